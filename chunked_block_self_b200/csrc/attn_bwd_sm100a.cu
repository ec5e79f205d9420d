// attn_bwd_sm100a.cu -- gradient of block attention and of full-utterance
// attention on B200 (sm_100a), the probabilities recomputed from the
// forward's log-sum-exp.
//
// For every segment (a block of an utterance, or the whole utterance) and
// head, with s = softmax_scale, all sums over the segment's frames:
//     P_ij  = exp(s q_i.k_j - lse_i)        delta_i = sum_d dO_id O_id
//     dS_ij = P_ij (dO_i.v_j - delta_i)
//     dV_j  = sum_i P_ij dO_i     dQ_i = s sum_j dS_ij k_j
//     dK_j  = s sum_i dS_ij q_i
//
// Two kinds of work item, each owning 128 rows of one head and walking the
// segment's other side in tiles of 64, so that every sum stays in the owner's
// TMEM accumulators: no atomics, no partial sums in memory, the same bits every
// time.  With X, Y the owner's and x, y the tile's matrices:
//   kind 0 (dK, dV): owner K, V (rows = keys), tiles Q, dO
//     S = X x^T, D = Y y^T (both transposed: row = key, column = query),
//     acc0 (dK) += dS x,  acc1 (dV) += P y
//   kind 1 (dQ): owner Q, dO (rows = queries), tiles K, V
//     S = X x^T, D = Y y^T,  acc0 (dQ) += dS x
// P is formed twice (once per kind): 7 products of 2*64 FLOP and 2 exps per
// (query, key) pair instead of 5 and 1.  A single pass would have to sum dQ
// across owners, in fp32 atomics or in partial sums added in order (32 KB per
// 128 x 128 pairs, half of that with owners of 256 keys); it was not built.
//
// One persistent CTA per SM, 20 warps:
//   warp 0   TMA producer: owner tiles (two stages), the segment's tiles into
//            a ring of eight; publishes every item's descriptor.
//   warp 1   issues S, warp 2 issues D (one elected lane each), each after
//            zeroing its operand's rows past the segment up to the MMA's
//            16-row granule (their P and dS are 0, but 0 * Inf would be NaN).
//   warp 3   owns TMEM and issues the accumulating MMAs (one elected lane).
//   warps 4-19  elementwise, two streams of two warpgroups on alternate tiles:
//            a lane owns one row of the tile (its TMEM lane), warpgroup g the
//            columns 32 (g & 1) .. + 31.  P = exp2(S s log2e - lse log2e) and
//            dS = P (D - delta) in fp32, each rounded once to bf16 and written
//            over S.  lse and delta belong to the lane's row (kind 1), or to the
//            columns (kind 0: fetched one tile ahead, +inf and 0 past the
//            segment, so that P and dS vanish there).  At the end of an item the
//            output rows: acc times s, rounded to bf16, the segment's rows only.
// TMEM (512 columns): stream p at 192 p: two S buffers of 64 (after use: P of
// the group's columns in its first 16, dS in its last 16), D at + 128; acc0 at
// 384, acc1 at 448.
//
// P and dS are rounded because the accumulating MMAs take 16-bit A operands at
// the full rate; the forward rounds its P alike.  Against 64 bits each gradient
// is then off by 0.0024 (relative, L2), 0.0017 of it the rounding of the result.
//
// What bounds it: the chain of a tile (S, read, exp, D, dS, write, accumulate)
// takes about 2.4 k cycles, and two chains are in flight: about 1.2 k cycles a
// tile, beside 512 for its 8192 exps and 512 (kind 1) or 640 (kind 0) for its
// MMAs.  16 clips of 1950-4700 frames, 16 heads: 2.95 ms, 0.81 PFLOP/s over the
// 7 products (0.49 of a measured bf16 GEMM), 0.58 over the formula's 5.  The
// registers decide: 94 of the 96 that 640 threads leave, none spilled.  Beside
// 200 KB of shared memory a spill lives in L2, and every form with more rows or
// chains in flight that spilled was slower (three streams, decoupled buffers of
// P and dS: 15 to 40 %).  Tiles of 128 rows in one chain of 32-column groups
// come out alike on long clips and 3 to 15 % behind on blocks.
//
// Every mbarrier wait is bounded; on expiry the CTA drains its copies and
// MMAs in flight, frees TMEM and returns.
#include <cmath>

#include "attn_bwd.cuh"
#include "nle.h"
#include "nle_device.cuh"
#include "nle_host.h"

namespace {

using namespace nle;

constexpr int kElem0 = 4;                            // first elementwise warp
constexpr int kElemWarps = 16;                       // four groups of four, one per TMEM lane quarter
constexpr int kThreads = 32 * (kElem0 + kElemWarps); // 640
constexpr int kCols = 32;                            // tile columns of a group
constexpr int kRows = 128;                           // owner rows
constexpr int kTile = 64;                            // rows of a tile
constexpr int kRowBytes = 128;                       // one frame of one head: 64 bf16
constexpr uint32_t kBoxBytes = kTile * kRowBytes;    // 8 KB: every TMA box is 64 frames
constexpr uint32_t kMatBytes = kRows * kRowBytes;    // X or Y: 16 KB
constexpr uint32_t kPairBytes = 2 * kMatBytes;       // X, Y
constexpr uint32_t kStageBytes = 2 * kBoxBytes;      // x, y
constexpr uint32_t kColBytes = 2 * kCols * 4;        // an elementwise warp's columns: -lse (log2 domain), -delta
constexpr uint32_t kRing = 8;                        // tiles in flight
constexpr int kDescRing = 4;
constexpr int kDescReaders = 3 + kElemWarps;         // S, D, accumulating and elementwise warps
// shared memory: two owner stages, the tile ring, the tiles' columns, the barriers
constexpr uint32_t kRingOff = 2 * kPairBytes;
constexpr uint32_t kColOff = kRingOff + kRing * kStageBytes;
constexpr uint32_t kBarsOff = kColOff + kElemWarps * kColBytes;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kStreamCols = 192, kDCol = 128, kAcc0 = 384, kAcc1 = 448;

// One work item as the producer publishes it (rows < 0: no further item).
struct ItemDesc {
    int f0, rows;   // owner rows
    int s0, T;      // the segment
    int h, kind;
};

struct Bars {
    uint64_t own_full[2];
    uint64_t own_empty[2];          // 2 arrivals: the item's last S and last D MMA have completed
    uint64_t t_full[kRing];
    uint64_t t_empty[kRing];        // the tile's accumulating MMAs have completed
    uint64_t s_full[4];             // by tile & 3
    uint64_t s_empty[4];            // the accumulating MMAs that read P, dS have completed
    uint64_t p_full[4];             // kElemWarps / 2 arrivals: P and dS written
    uint64_t d_full[2];             // by tile & 1
    uint64_t d_empty[2];            // kElemWarps / 2 arrivals: D has been read
    uint64_t acc_full;              // the item's accumulators are complete
    uint64_t acc_empty;             // kElemWarps arrivals: they have been read
    uint64_t mma_done[3];
    uint64_t desc_full[kDescRing];
    uint64_t desc_empty[kDescRing]; // kDescReaders arrivals
    ItemDesc desc[kDescRing];
    uint32_t tmem_base;
    int abort_flag;
};

struct Params {
    const int32_t *cu;
    int n_seq;
    int total;
    int heads;
    int block;          // frames per segment; 0: whole utterances
    int xtiles;         // owner tiles per block (block mode)
    float scale, scale_log2;
    const float *lse;   // [heads][total]
    const float *delta; // [heads][total]
    __nv_bfloat16 *dq, *dk, *dv;
    long long out_stride;   // elements between gradient frames
    int32_t *status;
    unsigned long long wait_ns;
    int flags;
};

// The CTA's items in order: item i = blockIdx.x + n * gridDim.x =
// ((u * X + x) * H + h) * 2 + c; u = 128-row unit of an utterance (X = 1), or
// block, whose owner tile x may not exist.  The kind is c, flipped on odd n:
// gridDim.x is even, so each CTA gets both kinds in turn and every (u, x, h)
// both kinds once.
struct ItemWalk {
    PlanWalker w;
    long long i;
    int n;

    __device__ __forceinline__ void init(const Params &p, int lane)
    {
        w.init(p.cu, p.n_seq, p.total, p.block ? p.block : kRows, lane);
        i = blockIdx.x;
        n = 0;
    }

    __device__ __forceinline__ bool next(const Params &p, int lane, ItemDesc &d)
    {
        for (;;) {
            const long long uxh = i >> 1, ux = uxh / p.heads;
            d.h = (int)(uxh - ux * p.heads);
            d.kind = ((int)i ^ n) & 1;
            i += gridDim.x;
            ++n;
            int f0, L, seq;
            if (p.block) {
                const long long u = ux / p.xtiles;
                const int x = (int)(ux - u * p.xtiles);
                if (!w.find(u, lane, f0, L, seq))
                    return false;
                if (x * kRows >= L)
                    continue;
                d.s0 = f0;
                d.T = L;
                d.f0 = f0 + x * kRows;
                d.rows = min(kRows, L - x * kRows);
            } else {
                if (!w.find(ux, lane, f0, L, seq))
                    return false;
                d.s0 = __ldg(p.cu + seq);
                d.T = __ldg(p.cu + seq + 1) - d.s0;
                d.f0 = f0;
                d.rows = L;
            }
            return true;
        }
    }
};

// A reader's walk over the published descriptors: waits for entry n.
struct DescReader {
    int n;
    __device__ __forceinline__ bool next(Bars *bars, const Params &p, volatile int *abort_flag, ItemDesc &d)
    {
        const int j = n % kDescRing;
        if (!wait_bar(smem_u32(&bars->desc_full[j]), (uint32_t)(n / kDescRing) & 1, abort_flag, p.wait_ns, p.status))
            return false;
        d = bars->desc[j];
        __syncwarp();
        if ((threadIdx.x & 31) == 0)
            mbar_arrive(smem_u32(&bars->desc_empty[j]));
        ++n;
        return d.rows >= 0;
    }
};

// One tile for one lane: P and dS of the warpgroup's 32 columns, written over
// its columns of S (P, kind 0 only, over the first 16, dS over the rest).
// neg_lse2, neg_delta: -lse log2e and -delta of the lane's row (kind 1); cl:
// those of the columns, in shared memory (kind 0).  valid: columns inside the
// segment; kind 1 masks the others by index (kind 0's have lse = +inf, so
// P = 0, and zeroed operands, so D = 0).  False if the wait for D ran out.
template <bool kDQ>
__device__ __forceinline__ bool elem_tile(uint32_t tS, uint32_t tD, int valid, float sl2, float neg_lse2,
                                          float neg_delta, uint32_t cl, Bars *bars,
                                          int stream, uint32_t d_parity, const Params &p, volatile int *abort_flag)
{
    uint32_t s[kCols], pk[kCols / 2];
    tmem_ld32_nowait(tS, s);
    tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < kCols; ++i)
        reg_fence(s[i]);
    const uint64_t k2 = pair(sl2, sl2);
    uint64_t pr[kCols / 2];
#pragma unroll
    for (int i = 0; i < kCols / 4; ++i) {
        uint64_t l0, l1;
        if (kDQ) {
            l0 = l1 = pair(neg_lse2, neg_lse2);
        } else {
            lds_pairs(cl + 16 * i, l0, l1);
        }
        const uint64_t y0 = fma2(pair(s[4 * i], s[4 * i + 1]), k2, l0);
        const uint64_t y1 = fma2(pair(s[4 * i + 2], s[4 * i + 3]), k2, l1);
        float a, b;
        unpair(y0, a, b);
        pr[2 * i] = pair(ex2_approx(a), ex2_approx(b));
        unpair(y1, a, b);
        pr[2 * i + 1] = pair(ex2_approx(a), ex2_approx(b));
        if (!kDQ && (i & 1)) {   // at most two loads of column values ahead of their use
            pair_fence(pr[2 * i]);
            pair_fence(pr[2 * i + 1]);
        }
    }
    if (!kDQ) {
#pragma unroll
        for (int i = 0; i < kCols / 2; ++i) {
            float a, b;
            unpair(pr[i], a, b);
            pk[i] = pack_bf16x2(a, b);
        }
        tmem_st16p(tS, pk);
    }
    if (!wait_bar(smem_u32(&bars->d_full[stream]), d_parity, abort_flag, p.wait_ns, p.status))
        return false;
    tc_fence_after();
    // D in two halves: 16 registers fewer at once, which is what keeps the 96
    // registers from spilling (beside 200 KB of shared memory spills live in L2)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        uint32_t d[16], dk[8];
        tmem_ld16_nowait(tD + 16 * h, d);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 16; ++i)
            reg_fence(d[i]);
        if (h) {
            tc_fence_before();
            __syncwarp();
            if ((threadIdx.x & 31) == 0)
                mbar_arrive(smem_u32(&bars->d_empty[stream]));
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint64_t l0, l1;
            if (kDQ) {
                l0 = l1 = pair(neg_delta, neg_delta);
            } else {
                lds_pairs(cl + 4 * kCols + 16 * (4 * h + i), l0, l1);
            }
            const uint64_t g0 = mul2(pr[8 * h + 2 * i], add2(pair(d[4 * i], d[4 * i + 1]), l0));
            const uint64_t g1 = mul2(pr[8 * h + 2 * i + 1], add2(pair(d[4 * i + 2], d[4 * i + 3]), l1));
            float a, b;
            unpair(g0, a, b);
            dk[2 * i] = pack_bf16x2(a, b);
            unpair(g1, a, b);
            dk[2 * i + 1] = pack_bf16x2(a, b);
        }
        if (kDQ && valid < kCols) {   // warp-uniform: the segment's last tile
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int c = 16 * h + 2 * i;
                dk[i] = c + 1 < valid ? dk[i] : c < valid ? dk[i] & 0xffffu : 0u;
            }
        }
        tmem_st8p(tS + kCols / 2 + 8 * h, dk);
    }
    tmem_wait_st();
    return true;
}

__global__ void __launch_bounds__(kThreads, 1)
    attn_bwd_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                    const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_do,
                    const Params p)
{
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t own_base = smem_u32(smem);
    const uint32_t ring_base = own_base + kRingOff;
    float *cols = reinterpret_cast<float *>(smem + kColOff);   // per elementwise warp: -lse2[32], -delta[32]
    Bars *bars = reinterpret_cast<Bars *>(smem + kBarsOff);
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;

    // ------------------------------------------------------------ set-up
    if (threadIdx.x == 0) {
        for (int s = 0; s < 2; ++s) {
            mbar_init(smem_u32(&bars->own_full[s]), 1);
            mbar_init(smem_u32(&bars->own_empty[s]), 2);
            mbar_init(smem_u32(&bars->d_full[s]), 1);
            mbar_init(smem_u32(&bars->d_empty[s]), kElemWarps / 2);
        }
        for (int s = 0; s < 4; ++s) {
            mbar_init(smem_u32(&bars->s_full[s]), 1);
            mbar_init(smem_u32(&bars->s_empty[s]), 1);
            mbar_init(smem_u32(&bars->p_full[s]), kElemWarps / 2);
        }
        for (int s = 0; s < (int)kRing; ++s) {
            mbar_init(smem_u32(&bars->t_full[s]), 1);
            mbar_init(smem_u32(&bars->t_empty[s]), 1);
        }
        mbar_init(smem_u32(&bars->acc_full), 1);
        mbar_init(smem_u32(&bars->acc_empty), kElemWarps);
        for (int s = 0; s < 3; ++s)
            mbar_init(smem_u32(&bars->mma_done[s]), 1);
        for (int j = 0; j < kDescRing; ++j) {
            mbar_init(smem_u32(&bars->desc_full[j]), 1);
            mbar_init(smem_u32(&bars->desc_empty[j]), kDescReaders);
        }
        bars->abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 3) {
        tmem_alloc(smem_u32(&bars->tmem_base), kTmemCols);
        tmem_relinquish();
    }
    if (threadIdx.x == 64) {
        tma_prefetch_desc(&tm_q);
        tma_prefetch_desc(&tm_k);
        tma_prefetch_desc(&tm_v);
        tma_prefetch_desc(&tm_do);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bars->tmem_base;
    volatile int *abort_flag = &bars->abort_flag;
    const unsigned long long wait_ns = p.wait_ns;

    if (warp == 0) {
        // ======================================================== producer
        ItemWalk it;
        it.init(p, lane);
        const bool skip0 = (p.flags & NLE_FLAG_TEST_SKIP_FIRST_LOAD) != 0;
        int n = 0;    // items published
        int nown = 0; // owner stages claimed
        int nt = 0;   // tiles claimed
        bool stop = false;
        auto publish = [&](const ItemDesc &d) -> bool {
            const int j = n % kDescRing;
            if (n >= kDescRing && !wait_bar(smem_u32(&bars->desc_empty[j]), (uint32_t)(n / kDescRing - 1) & 1,
                                            abort_flag, wait_ns, p.status))
                return false;
            if (lane == 0) {
                bars->desc[j] = d;
                mbar_arrive(smem_u32(&bars->desc_full[j]));
            }
            __syncwarp();
            ++n;
            return true;
        };
        ItemDesc d;
        while (!stop && it.next(p, lane, d)) {
            if (!publish(d)) {
                stop = true;
                break;
            }
            const int os = nown & 1;
            if (nown >= 2 && !wait_bar(smem_u32(&bars->own_empty[os]), (uint32_t)((nown >> 1) - 1) & 1, abort_flag,
                                       wait_ns, p.status)) {
                stop = true;
                break;
            }
            if (lane == 0 && !(skip0 && nown == 0)) {
                const uint32_t bar = smem_u32(&bars->own_full[os]);
                const uint32_t dst = own_base + os * kPairBytes;
                const int boxes = d.rows > kTile ? 2 : 1;
                mbar_arrive_expect_tx(bar, 2 * boxes * kBoxBytes);
                for (int x = 0; x < boxes; ++x) {
                    tma_load(dst + x * kBoxBytes, d.kind ? &tm_q : &tm_k, d.h * 64, d.f0 + x * kTile, bar);
                    tma_load(dst + kMatBytes + x * kBoxBytes, d.kind ? &tm_do : &tm_v, d.h * 64, d.f0 + x * kTile, bar);
                }
            }
            __syncwarp();
            ++nown;
            for (int j = 0; j * kTile < d.T; ++j) {
                const int s = nt % (int)kRing;
                const uint32_t u = (uint32_t)(nt / (int)kRing);
                if (u > 0 && !wait_bar(smem_u32(&bars->t_empty[s]), (u - 1) & 1, abort_flag, wait_ns, p.status)) {
                    stop = true;
                    break;
                }
                if (lane == 0) {
                    const uint32_t bar = smem_u32(&bars->t_full[s]);
                    const uint32_t dst = ring_base + s * kStageBytes;
                    mbar_arrive_expect_tx(bar, kStageBytes);
                    tma_load(dst, d.kind ? &tm_k : &tm_q, d.h * 64, d.s0 + j * kTile, bar);
                    tma_load(dst + kBoxBytes, d.kind ? &tm_v : &tm_do, d.h * 64, d.s0 + j * kTile, bar);
                }
                __syncwarp();
                ++nt;
            }
        }
        if (it.w.bad && lane == 0)
            report(p.status, NLE_ERR_INVALID_ARG);
        if (!stop)
            publish(ItemDesc{0, -1, 0, 0, 0, 0});
        // drain: the last copy into each stage must land before exit
        if (lane == 0) {
            for (int m = nown - 2; m < nown; ++m)
                if (m >= 0 && !(skip0 && m == 0))
                    wait_bar_drain(smem_u32(&bars->own_full[m & 1]), (uint32_t)(m >> 1) & 1, wait_ns);
            for (int m = nt - (int)kRing; m < nt; ++m)
                if (m >= 0)
                    wait_bar_drain(smem_u32(&bars->t_full[m % (int)kRing]), (uint32_t)(m / (int)kRing) & 1, wait_ns);
        }
        __syncwarp();
    } else if (warp == 1 || warp == 2) {
        // ======================================================== S (warp 1) and D (warp 2) MMAs
        const bool is_d = warp == 2;
        DescReader rd{0};
        ItemDesc d;
        uint32_t nt = 0, n = 0;
        const uint64_t own0 = smem_desc_sw128(own_base + (is_d ? kMatBytes : 0), 16, 1024);
        const uint64_t ring0 = smem_desc_sw128(ring_base + (is_d ? kBoxBytes : 0), 16, 1024);
        const uint32_t sh = is_d ? 1 : 2;   // D has one buffer a stream (two in all), S two (four)
        uint64_t *full = is_d ? bars->d_full : bars->s_full, *empty = is_d ? bars->d_empty : bars->s_empty;
        bool ok = true;
        while (ok && rd.next(bars, p, abort_flag, d)) {
            const uint32_t os = n & 1;
            if (!wait_bar(smem_u32(&bars->own_full[os]), (n >> 1) & 1, abort_flag, wait_ns, p.status))
                break;
            const uint64_t da = own0 + os * (kPairBytes >> 4);
            for (int left = __shfl_sync(kFull, d.T, 0); left > 0; left -= kTile, ++nt) {
                const uint32_t s = nt % kRing, b = nt & ((1u << sh) - 1), u = nt >> sh;
                if (!wait_bar(smem_u32(&bars->t_full[s]), (nt / kRing) & 1, abort_flag, wait_ns, p.status) ||
                    (u > 0 && !wait_bar(smem_u32(&empty[b]), (u - 1) & 1, abort_flag, wait_ns, p.status))) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                if (left < kTile && (left & 15)) {
                    // rows past the segment up to the MMA's granule: their P
                    // and dS are 0, but 0 * Inf would be NaN
                    uint4 *z = reinterpret_cast<uint4 *>(smem + kRingOff + s * kStageBytes + (is_d ? kBoxBytes : 0) +
                                                         left * kRowBytes);
                    for (int i = lane; i < (16 - (left & 15)) * (kRowBytes / 16); i += 32)
                        z[i] = make_uint4(0, 0, 0, 0);
                    fence_proxy_async_smem();
                    __syncwarp();
                }
                const uint64_t db = ring0 + s * (kStageBytes >> 4);
                const uint32_t id = idesc_bf16_f32(128, left < kTile ? (left + 15) & ~15 : kTile, false);
                const uint32_t t = tmem + (nt & 1) * kStreamCols + (is_d ? kDCol : ((nt >> 1) & 1) * kTile);
                // K steps of 16 elements = 32 bytes inside the 128-byte swizzle atom
                if (elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        mma_ss(t, da + 2 * kk, db + 2 * kk, id, kk > 0 ? 1u : 0u);
                    mma_commit(smem_u32(&full[b]));
                    if (left <= kTile)   // the item's last use of its owner matrix
                        mma_commit(smem_u32(&bars->own_empty[os]));
                }
                __syncwarp();
            }
            ++n;
        }
        // every MMA must finish before TMEM is released
        if (elect_one()) {
            mma_commit(smem_u32(&bars->mma_done[is_d]));
            wait_bar_drain(smem_u32(&bars->mma_done[is_d]), 0, wait_ns);
        }
        __syncwarp();
    } else if (warp == 3) {
        // ======================================================== accumulating MMAs
        DescReader rd{0};
        ItemDesc d;
        uint32_t nt = 0, n = 0;
        const uint64_t ring0 = smem_desc_sw128(ring_base, 0, 1024);
        constexpr uint32_t id = idesc_bf16_f32(128, 64, true);
        bool ok = true;
        while (ok && rd.next(bars, p, abort_flag, d)) {
            const bool both = __shfl_sync(kFull, d.kind, 0) == 0;
            uint32_t acc = 0;
            // p_full of a tile speaks for one stream's warps only: the other's
            // may still be reading the last item's accumulators
            if (n > 0 && !wait_bar(smem_u32(&bars->acc_empty), (n - 1) & 1, abort_flag, wait_ns, p.status))
                break;
            ++n;
            for (int left = __shfl_sync(kFull, d.T, 0); left > 0; left -= kTile, ++nt) {
                const uint32_t s = nt % kRing, b = nt & 3;
                if (!wait_bar(smem_u32(&bars->p_full[b]), (nt >> 2) & 1, abort_flag, wait_ns, p.status)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                // N = 64 is one 128-byte swizzle atom along N; K steps of 16
                // rows advance the start by 2048 bytes
                const uint64_t dx = ring0 + s * (kStageBytes >> 4), dy = dx + (kBoxBytes >> 4);
                const uint32_t a = tmem + (nt & 1) * kStreamCols + ((nt >> 1) & 1) * kTile;
                const int steps = left < kTile ? (left + 15) >> 4 : kTile / 16;
                if (elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < kTile / 16; ++kk) {
                        if (kk < steps) {
                            const uint32_t ak = a + (kk >> 1) * kCols + (kk & 1) * 8;
                            const uint64_t row = (uint64_t)(kk * (16 * kRowBytes >> 4));
                            if (both)
                                mma_ts(tmem + kAcc1, ak, dy + row, id, kk ? 1u : acc);
                            mma_ts(tmem + kAcc0, ak + kCols / 2, dx + row, id, kk ? 1u : acc);
                        }
                    }
                    mma_commit(smem_u32(&bars->s_empty[b]));
                    mma_commit(smem_u32(&bars->t_empty[s]));
                    if (left <= kTile)
                        mma_commit(smem_u32(&bars->acc_full));
                }
                __syncwarp();
                acc = 1;
            }
        }
        if (elect_one()) {
            mma_commit(smem_u32(&bars->mma_done[2]));
            wait_bar_drain(smem_u32(&bars->mma_done[2]), 0, wait_ns);
        }
        __syncwarp();
    } else if (warp >= kElem0) {
        // ======================================================== elementwise
        const int g = (warp - kElem0) >> 2;   // group: stream g >> 1, columns 32 (g & 1) .. + 31
        const int stream = g >> 1, c0 = kCols * (g & 1);
        const int qq = warp & 3;              // TMEM lane quarter of this warp
        const uint32_t lanes = (uint32_t)(qq * 32) << 16;
        const uint32_t tstream = tmem + stream * kStreamCols + c0 + lanes;
        const int row = qq * 32 + lane;
        float *cl = cols + (warp - kElem0) * (2 * kCols);
        const uint32_t cl32 = smem_u32(cl);
        DescReader rd{0};
        // lse and delta of an item: of this lane's row (kind 1), or of the
        // lane's column in tile j (kind 0; nothing past the segment: P = 0)
        auto fetch = [&](const ItemDesc &d, int j, float &l, float &dl) {
            const int c = j * kTile + c0 + lane;
            const bool in = d.kind ? row < d.rows : c < d.T;
            const size_t at = (size_t)d.h * p.total + (d.kind ? d.f0 + row : d.s0 + c);
            l = in ? __ldg(p.lse + at) : d.kind ? 0.f : INFINITY;
            dl = in ? __ldg(p.delta + at) : 0.f;
        };
        ItemDesc d, dn;
        int nt0 = 0, n = 0;   // the item's first tile; items
        float vl = 0.f, vd = 0.f;
        bool ok = rd.next(bars, p, abort_flag, d);
        if (ok)
            fetch(d, stream, vl, vd);
        for (; ok; ++n) {
            const bool active = qq * 32 < d.rows;   // warp-uniform
            const int tiles = (d.T + kTile - 1) / kTile;
            const float neg_lse2 = vl * -kLog2e, neg_delta = -vd;   // kind 1
            // the stream's tiles of the item
            for (int j = (nt0 ^ stream) & 1; j < tiles; j += 2) {
                const int nt = nt0 + j, b = nt & 3;
                const int valid = min(kTile, d.T - j * kTile) - c0;   // columns of this group in the segment
                const uint32_t dpar = (uint32_t)(nt >> 1) & 1;
                if (d.kind == 0) {
                    // the columns' values, for the whole warp
                    __syncwarp();
                    cl[lane] = vl * -kLog2e;
                    cl[kCols + lane] = -vd;
                    __syncwarp();
                    if (j + 2 < tiles)
                        fetch(d, j + 2, vl, vd);
                }
                if (!wait_bar(smem_u32(&bars->s_full[b]), ((uint32_t)nt >> 2) & 1, abort_flag, wait_ns, p.status)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                if (active && valid > 0) {
                    const uint32_t tS = tstream + ((nt >> 1) & 1) * kTile, tD = tstream + kDCol;
                    ok = d.kind ? elem_tile<true>(tS, tD, valid, p.scale_log2, neg_lse2, neg_delta, cl32,
                                                  bars, stream, dpar, p, abort_flag)
                                : elem_tile<false>(tS, tD, valid, p.scale_log2, neg_lse2, neg_delta, cl32,
                                                   bars, stream, dpar, p, abort_flag);
                } else {
                    ok = wait_bar(smem_u32(&bars->d_full[stream]), dpar, abort_flag, wait_ns, p.status);
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(smem_u32(&bars->d_empty[stream]));
                }
                if (!ok)
                    break;
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(smem_u32(&bars->p_full[b]));
            }
            if (!ok)
                break;
            nt0 += tiles;
            // the next item's values travel while this one's output is stored
            const bool have = rd.next(bars, p, abort_flag, dn);
            if (have)
                fetch(dn, (nt0 ^ stream) & 1, vl, vd);
            // ---------------------------------------------- output rows
            if (!wait_bar(smem_u32(&bars->acc_full), (uint32_t)n & 1, abort_flag, wait_ns, p.status))
                break;
            tc_fence_after();
            if (active && (d.kind == 0 || g < 2)) {
                const int c = 32 * (g & 1);
                const long long at = (d.f0 + qq * 32) * p.out_stride + d.h * 64 + c;
                uint32_t o[16];
                load_acc(tmem + (g < 2 ? kAcc0 : kAcc1) + c + lanes, g < 2 ? p.scale : 1.f, o);
                store_rows(o, (d.kind ? p.dq : g < 2 ? p.dk : p.dv) + at, p.out_stride, d.rows - qq * 32);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(smem_u32(&bars->acc_empty));
            d = dn;
            ok = have;
        }
    }

    // ------------------------------------------------------------ teardown
    tc_fence_before();
    __syncthreads();
    if (warp == 3) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

// delta[h][f] = sum_d dO O (fp32): eight lanes per head row, four heads of a
// frame per warp load.  Memory-bound: reads O and dO once.  Not unrolled: the
// unrolled loop takes 46 registers instead of 29 and runs 40 warps per SM, not 64
// (41 -> 51 us on the batch of 128 utterances).
__global__ void __launch_bounds__(256)
    attn_delta_kernel(const uint4 *out, const uint4 *dout, float *delta, int total, int heads)
{
    const int lane = threadIdx.x & 31;
    const long long rows = (long long)total * heads;
#pragma unroll 1
    for (long long r0 = ((long long)blockIdx.x * 8 + (threadIdx.x >> 5)) * 4; r0 < rows; r0 += (long long)gridDim.x * 32) {
        const long long r = r0 + (lane >> 3);
        float s = 0.f;
        int f = 0, h = 0;
        if (r < rows) {
            f = (int)(r / heads);
            h = (int)(r - (long long)f * heads);
            const uint4 a = __ldg(out + r * 8 + (lane & 7));
            const uint4 b = __ldg(dout + r * 8 + (lane & 7));
            const uint32_t av[4] = {a.x, a.y, a.z, a.w}, bv[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                s = fmaf(__uint_as_float(av[i] << 16), __uint_as_float(bv[i] << 16), s);
                s = fmaf(__uint_as_float(av[i] & 0xffff0000u), __uint_as_float(bv[i] & 0xffff0000u), s);
            }
        }
        s += __shfl_xor_sync(kFull, s, 1);
        s += __shfl_xor_sync(kFull, s, 2);
        s += __shfl_xor_sync(kFull, s, 4);
        if (r < rows && (lane & 7) == 0)
            delta[(size_t)h * total + f] = s;
    }
}

// block = 0: whole utterances.
int launch_attn_bwd(const nle_attn_bwd_args *a, int block, void *stream)
{
    if (!a || a->n_seq < 0 || a->total_frames < 0 || a->heads <= 0 || block < 0 || a->wait_limit_ns < 0)
        return NLE_ERR_INVALID_ARG;
    if (a->d_head != 64 || block > 256 || a->total_frames > 0x7fffffffLL)
        return NLE_ERR_UNSUPPORTED;
    const int xtiles = block ? (block + kRows - 1) / kRows : 1;
    // upper bound on work items: two kinds, each utterance at most T/unit + 1 units
    const long long units = a->n_seq + a->total_frames / (block ? block : kRows);
    if (units > 0x7fffffffLL || units * xtiles * 2 > 0x7fffffffLL / a->heads)
        return NLE_ERR_UNSUPPORTED;
    if (a->n_seq == 0 || a->total_frames == 0)
        return NLE_OK;
    const void *ptrs[] = {a->q, a->k, a->v, a->out, a->dout, a->dq, a->dk, a->dv, a->lse, a->cu_seqlens, a->workspace};
    for (const void *x : ptrs)
        if (!x)
            return NLE_ERR_INVALID_ARG;
    const int64_t dense = (int64_t)a->heads * 64;
    const int64_t stride = a->row_stride_qkv ? a->row_stride_qkv : dense;
    const int64_t dstride = a->row_stride_dqkv ? a->row_stride_dqkv : dense;
    if (stride < dense || dstride < dense || dense > 0x7fffffffLL || stride > (1ll << 38) || dstride > (1ll << 38))
        return NLE_ERR_INVALID_ARG;
    if (stride % 8 != 0 || dstride % 8 != 0)
        return NLE_ERR_MISALIGNED;
    for (int i = 0; i < 8; ++i)
        if (!nle::aligned16(ptrs[i]))
            return NLE_ERR_MISALIGNED;
    for (int i = 8; i < 11; ++i)
        if (!nle::aligned4(ptrs[i]))
            return NLE_ERR_MISALIGNED;
    if (!nle::aligned4(a->dev_status))
        return NLE_ERR_MISALIGNED;
    // what is written (dq, dk, dv, workspace) begins at no other buffer's start
    for (int i = 5; i < 11; ++i)
        for (int j = 0; j < i; ++j)
            if (ptrs[i] == ptrs[j] && (i < 8 || i == 10 || j >= 5))
                return NLE_ERR_INVALID_ARG;

    nle::DeviceInfo di;
    int dev = 0;
    if (!nle::current_device_info(&di, &dev))
        return NLE_ERR_CUDA;
    if (di.cc_major != 10)
        return NLE_ERR_UNSUPPORTED;
    const long long items = units * xtiles * 2 * a->heads;
    // an even grid: the two kinds of an owner tile are taken in the same round
    const int grid = (int)(items < (di.sm_count & ~1) ? items : (di.sm_count & ~1));
    // the kernel counts the tiles that a CTA walks in 32 bits
    if ((items / grid + 1) * ((block ? block : a->total_frames) / kTile + 1) > 0x7fffffffLL)
        return NLE_ERR_UNSUPPORTED;

    const double scale = a->softmax_scale > 0.f ? (double)a->softmax_scale : 1.0 / std::sqrt((double)a->d_head);
    const float scale_log2 = (float)(scale * 1.4426950408889634);
    float *delta = static_cast<float *>(a->workspace);
    const unsigned long long wait_ns = a->wait_limit_ns > 0 ? (unsigned long long)a->wait_limit_ns : 1000000000ull;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    // Blocks longer than one key tile, and a (block, head) for every SM by the
    // bound `units`: whole blocks on chip.  Whole blocks against tiles, us, with
    // delta's 41 in both: batch of 128 utterances, blocks of 97: 461, 410; 128:
    // 375, 352 (one key tile leaves the second half of that kernel idle); 129:
    // 543, 606; 160: 467, 518; 200: 404, 502; 256: 393, 459.  Few items of 200
    // frames, L2 flushed: 64: 24.6, 20.5; 96: 24.6, 24.6; 128: 26.6, 28.7; 160
    // (a second round for twelve SMs): 36.8, 32.8; 256: 38.9, 41.0.  The bound
    // counts an utterance of exactly one block twice, so 74 such items already
    // pass for 148; and it is block_frames that is looked at, not the utterances:
    // 512 of 100-128 frames take whole blocks too (377 against 363; of 40-80
    // frames 360 against 272).
    const bool whole = block && !(a->flags & NLE_FLAG_SPLIT_ITEMS) &&
                       ((a->flags & NLE_FLAG_WHOLE_ITEMS) || (block > kRows && units * a->heads >= di.sm_count));
    if (whole) {
        nle::BlockBwdArgs b{};
        b.q = a->q;
        b.k = a->k;
        b.v = a->v;
        b.out = a->out;
        b.dout = a->dout;
        b.lse = a->lse;
        b.delta = delta;
        b.dq = a->dq;
        b.dk = a->dk;
        b.dv = a->dv;
        b.cu = a->cu_seqlens;
        b.status = a->dev_status;
        b.total = a->total_frames;
        b.stride = stride;
        b.dstride = dstride;
        b.n_seq = a->n_seq;
        b.heads = a->heads;
        b.block = block;
        b.scale = (float)scale;
        b.scale_log2 = scale_log2;
        b.wait_ns = wait_ns;
        b.flags = a->flags;
        return nle::launch_block_bwd(b, di, dev, units * a->heads, st);
    }

    Params p{};
    p.cu = a->cu_seqlens;
    p.n_seq = a->n_seq;
    p.total = (int)a->total_frames;
    p.heads = a->heads;
    p.block = block;
    p.xtiles = xtiles;
    // above half the SM's: one CTA per SM (it owns all TMEM)
    const size_t smem = kBarsOff + ((sizeof(Bars) + 127) / 128) * 128 + 1024;
    if (smem > (size_t)di.smem_optin)
        return NLE_ERR_UNSUPPORTED;
    p.scale = (float)scale;
    p.scale_log2 = scale_log2;
    p.lse = a->lse;
    p.delta = delta;
    p.dq = static_cast<__nv_bfloat16 *>(a->dq);
    p.dk = static_cast<__nv_bfloat16 *>(a->dk);
    p.dv = static_cast<__nv_bfloat16 *>(a->dv);
    p.out_stride = dstride;
    p.status = a->dev_status;
    p.wait_ns = wait_ns;
    p.flags = a->flags;

    CUtensorMap tq, tk, tv, tdo;
    const uint64_t cols = (uint64_t)dense, rows = (uint64_t)a->total_frames;
    if (!nle::encode_tmap_bf16_2d(&tq, a->q, cols, rows, stride, 64, kTile) ||
        !nle::encode_tmap_bf16_2d(&tk, a->k, cols, rows, stride, 64, kTile) ||
        !nle::encode_tmap_bf16_2d(&tv, a->v, cols, rows, stride, 64, kTile) ||
        !nle::encode_tmap_bf16_2d(&tdo, a->dout, cols, rows, dense, 64, kTile))
        return NLE_ERR_CUDA;
    if (!nle::allow_max_dynamic_smem(reinterpret_cast<const void *>(attn_bwd_kernel), dev, di.smem_optin))
        return NLE_ERR_CUDA;
    const int rc = nle::launch_attn_delta(a->out, a->dout, delta, a->total_frames, a->heads, di, st);
    if (rc != NLE_OK)
        return rc;
    attn_bwd_kernel<<<grid, kThreads, smem, st>>>(tq, tk, tv, tdo, p);
    return cudaGetLastError() == cudaSuccess ? NLE_OK : NLE_ERR_CUDA;
}

} // namespace

namespace nle {

int launch_attn_delta(const void *out, const void *dout, float *delta, int64_t total, int heads, const DeviceInfo &di,
                      cudaStream_t st)
{
    const long long grid = (total * heads + 31) / 32, most = 16ll * di.sm_count;
    attn_delta_kernel<<<(unsigned)(grid < most ? grid : most), 256, 0, st>>>(
        static_cast<const uint4 *>(out), static_cast<const uint4 *>(dout), delta, (int)total, heads);
    return cudaGetLastError() == cudaSuccess ? NLE_OK : NLE_ERR_CUDA;
}

} // namespace nle

extern "C" int nle_block_attn_bwd(const nle_attn_bwd_args *args, int block_frames, void *stream)
{
    if (block_frames <= 0)
        return NLE_ERR_INVALID_ARG;
    return launch_attn_bwd(args, block_frames, stream);
}

extern "C" int nle_varlen_attn_bwd(const nle_attn_bwd_args *args, void *stream)
{
    return launch_attn_bwd(args, 0, stream);
}
