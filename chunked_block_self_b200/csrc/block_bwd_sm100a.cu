// block_bwd_sm100a.cu -- gradient of block attention, whole blocks at a time,
// on B200 (sm_100a).  The formulas are those of attn_bwd_sm100a.cu, whose
// kernel walks either side of a segment of any length and therefore forms
// every probability twice.  Here a block (at most 256 frames) of one head
// stays on chip: S and D are formed once, and dQ, dK and dV of the block are
// all summed in TMEM, 5 products and one exp per (query, key) pair.
//
// Work item = (block, head).  Key tile c = keys 128c..128c+127 (at most two),
// unit = (key tile, 64 queries): with rows = keys and columns = queries
//     S = K_c Q_u^T,  D = V_c dO_u^T          (M = 128, N <= 64, K = 64)
//     P = exp2(S s log2e - lse log2e), dS = P (D - delta)   (elementwise)
//     dV_c += P dO_u     A = P in TMEM (over S), B = dO rows
//     dK_c += dS Q_u     A = dS in shared memory, K-major, B = Q rows
//     dQ_x += dS^T K_c   A = the same shared memory read M-major: 128 queries
//                        (two units), K = the tile's keys, B = K rows
// dS is written once, as 64-query chunks of 128-byte rows (one key each),
// 128-byte swizzled: a row-major operand for dK and a column-major one for dQ.
//
// One persistent CTA per SM, 20 warps:
//   warp 0   TMA producer: K, Q, V, dO of an item, one box each, into a ring
//            of matrix slots; publishes the item's descriptor.
//   warp 1   issues S and D.
//   warp 2   issues dV, dK and dQ.
//   warp 3   owns TMEM; zeroes operand rows past the block (up to the MMAs'
//            16-row granule: their P and dS are 0, but 0 * Inf would be NaN)
//            and stages the block's lse and delta (+inf and 0 past it).
//   warps 4-19  elementwise, two groups of eight warps on alternate units
//            (group g: S, D buffer g): a lane owns one key of the tile, a
//            warp half of the unit's columns.  They also store the results:
//            a key tile's after the first unit of the next, so that its last
//            MMAs run under arithmetic.
// TMEM (512 columns): S, D of group g at 128 g and 128 g + 64 (P over S: warp
// half j's in columns 32j..32j+15), dQ_0, dQ_1 at 256 and 320, dK at 384, dV
// at 448.
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
constexpr int kElemWarps = 16;                       // two groups of eight
constexpr int kThreads = 32 * (kElem0 + kElemWarps); // 640
constexpr int kKeys = 128;                           // keys of a tile (MMA M)
constexpr int kUnit = 64;                            // queries of a unit
constexpr int kCols = 32;                            // columns of an elementwise warp
constexpr int kRowBytes = 128;                       // one frame of one head: 64 bf16
constexpr uint32_t kTileBytes = kKeys * kRowBytes;   // 16 KB
constexpr uint32_t kChunkBytes = kKeys * kRowBytes;  // dS of a unit: 128 keys x 64 queries
constexpr int kMaxSlots = 8;
constexpr int kMats = 4;                             // K, Q, V, dO
constexpr int kDescRing = 4;
constexpr int kDescReaders = 3 + kElemWarps;         // both MMA, fix-up and elementwise warps
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kGroupCols = 128, kDCol = 64, kQAcc = 256, kKAcc = 384, kVAcc = 448;

struct ItemDesc {
    int f0, L, h;   // the block (L < 0: no further item)
};

struct Bars {
    uint64_t m_full[kMaxSlots];
    uint64_t m_empty[kMaxSlots];    // the item's last MMAs have completed
    uint64_t ready[2];              // by item: matrices checked, columns staged
    uint64_t cols_empty[2];         // kElemWarps arrivals: the item's columns are no longer read
    uint64_t s_full[2], d_full[2];  // by group
    uint64_t d_empty[2];            // 8 arrivals: D has been read
    uint64_t p_full[2];             // 8 arrivals: P and dS written
    uint64_t p_empty[2];            // the unit's dV and dK MMAs have completed (P)
    uint64_t dq_done[2];            // the key tile's dQ_x MMAs have completed (dS chunks 2x, 2x + 1)
    uint64_t acc_full;              // the key tile's sums (the item's, on its last) are complete
    uint64_t acc_empty;             // kElemWarps arrivals: they have been read
    uint64_t mma_done[2];
    uint64_t desc_full[kDescRing];
    uint64_t desc_empty[kDescRing];
    ItemDesc desc[kDescRing];
    uint32_t tmem_base;
    int abort_flag;
};

struct Params {
    const int32_t *cu;
    int n_seq, total, heads, block;
    int slots;
    uint32_t slot_bytes, ds_off, col_off, bars_off;
    float scale, scale_log2;
    const float *lse, *delta;   // [heads][total]
    __nv_bfloat16 *dq, *dk, *dv;
    long long out_stride;
    int32_t *status;
    unsigned long long wait_ns;
    int flags;
};

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
        return d.L >= 0;
    }
};

// Results waiting to be stored: a key tile's dK, dV and, with its item's
// last tile, the item's dQ.
struct Pending {
    int f0, L, h, c;
    bool have, last;
};

__global__ void __launch_bounds__(kThreads, 1)
    block_bwd_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                     const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_do,
                     const Params p)
{
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t base = smem_u32(smem);
    const uint32_t ds_base = base + p.ds_off;
    float *cols = reinterpret_cast<float *>(smem + p.col_off);   // per item parity: -lse2[256], -delta[256]
    Bars *bars = reinterpret_cast<Bars *>(smem + p.bars_off);
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;

    // ------------------------------------------------------------ set-up
    if (threadIdx.x == 0) {
        for (int s = 0; s < p.slots; ++s) {
            mbar_init(smem_u32(&bars->m_full[s]), 1);
            mbar_init(smem_u32(&bars->m_empty[s]), 1);
        }
        for (int g = 0; g < 2; ++g) {
            mbar_init(smem_u32(&bars->ready[g]), 1);
            mbar_init(smem_u32(&bars->cols_empty[g]), kElemWarps);
            mbar_init(smem_u32(&bars->s_full[g]), 1);
            mbar_init(smem_u32(&bars->d_full[g]), 1);
            mbar_init(smem_u32(&bars->d_empty[g]), kElemWarps / 2);
            mbar_init(smem_u32(&bars->p_full[g]), kElemWarps / 2);
            mbar_init(smem_u32(&bars->p_empty[g]), 1);
            mbar_init(smem_u32(&bars->dq_done[g]), 1);
            mbar_init(smem_u32(&bars->mma_done[g]), 1);
        }
        mbar_init(smem_u32(&bars->acc_full), 1);
        mbar_init(smem_u32(&bars->acc_empty), kElemWarps);
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
    auto wait = [&](uint64_t *bar, uint32_t parity) {
        return wait_bar(smem_u32(bar), parity & 1, abort_flag, wait_ns, p.status);
    };

    if (warp == 0) {
        // ======================================================== producer
        PlanWalker w;
        w.init(p.cu, p.n_seq, p.total, p.block, lane);
        const bool skip0 = (p.flags & NLE_FLAG_TEST_SKIP_FIRST_LOAD) != 0;
        const uint64_t pol = policy_evict_first();   // every matrix is read once
        const uint32_t bytes = (uint32_t)p.block * kRowBytes;
        int n = 0;      // items published
        int nm = 0;     // matrices claimed
        bool stop = false;
        auto publish = [&](const ItemDesc &d) -> bool {
            const int j = n % kDescRing;
            if (n >= kDescRing && !wait(&bars->desc_empty[j], (uint32_t)(n / kDescRing - 1)))
                return false;
            if (lane == 0) {
                bars->desc[j] = d;
                mbar_arrive(smem_u32(&bars->desc_full[j]));
            }
            __syncwarp();
            ++n;
            return true;
        };
        for (long long i = blockIdx.x; !stop; i += gridDim.x) {
            ItemDesc d;
            int seq;
            const long long b = i / p.heads;
            d.h = (int)(i - b * p.heads);
            if (!w.find(b, lane, d.f0, d.L, seq))
                break;
            if (!publish(d)) {
                stop = true;
                break;
            }
            for (int m = 0; m < kMats; ++m) {
                const int s = nm % p.slots, u = nm / p.slots;
                if (u > 0 && !wait(&bars->m_empty[s], (uint32_t)(u - 1))) {
                    stop = true;
                    break;
                }
                if (lane == 0 && !(skip0 && nm == 0)) {
                    const uint32_t bar = smem_u32(&bars->m_full[s]);
                    mbar_arrive_expect_tx(bar, bytes);
                    tma_load_2d(base + s * p.slot_bytes, m == 0 ? &tm_k : m == 1 ? &tm_q : m == 2 ? &tm_v : &tm_do,
                                d.h * 64, d.f0, bar, pol);
                }
                __syncwarp();
                ++nm;
            }
        }
        if (w.bad && lane == 0)
            report(p.status, NLE_ERR_INVALID_ARG);
        if (!stop)
            publish(ItemDesc{0, -1, 0});
        // drain: the last copy into each slot must land before exit
        if (lane == 0)
            for (int m = nm - p.slots; m < nm; ++m)
                if (m >= 0 && !(skip0 && m == 0))
                    wait_bar_drain(smem_u32(&bars->m_full[m % p.slots]), (uint32_t)(m / p.slots) & 1, wait_ns);
        __syncwarp();
    } else if (warp == 1) {
        // ======================================================== S and D MMAs
        DescReader rd{0};
        ItemDesc d;
        uint32_t n = 0, t = 0;   // items, units
        int slot = 0;
        bool ok = true;
        while (ok && rd.next(bars, p, abort_flag, d)) {
            if (!wait(&bars->ready[n & 1], n >> 1))
                break;
            const int L = __shfl_sync(kFull, d.L, 0);
            uint32_t at[kMats];
            for (int m = 0; m < kMats; ++m) {
                at[m] = base + slot * p.slot_bytes;
                slot = slot + 1 == p.slots ? 0 : slot + 1;
            }
            const uint64_t dk0 = smem_desc_sw128(at[0], 16, 1024), dq0 = smem_desc_sw128(at[1], 16, 1024);
            const uint64_t dv0 = smem_desc_sw128(at[2], 16, 1024), do0 = smem_desc_sw128(at[3], 16, 1024);
            for (int c = 0; ok && c * kKeys < L; ++c) {
                for (int u = 0; u * kUnit < L; ++u, ++t) {
                    const uint32_t g = t & 1, use = t >> 1;
                    const uint32_t id = idesc_bf16_f32(128, min(kUnit, (L - u * kUnit + 15) & ~15), false);
                    const uint32_t ts = tmem + g * kGroupCols;
                    const uint64_t ca = (uint64_t)c * (kTileBytes >> 4), ub = (uint64_t)u * (kUnit * kRowBytes >> 4);
                    if (use > 0 && !wait(&bars->p_empty[g], use - 1)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    // K steps of 16 elements = 32 bytes inside the 128-byte swizzle atom
                    if (elect_one()) {
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            mma_ss(ts, dk0 + ca + 2 * kk, dq0 + ub + 2 * kk, id, kk > 0 ? 1u : 0u);
                        mma_commit(smem_u32(&bars->s_full[g]));
                    }
                    __syncwarp();
                    if (use > 0 && !wait(&bars->d_empty[g], use - 1)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    if (elect_one()) {
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            mma_ss(ts + kDCol, dv0 + ca + 2 * kk, do0 + ub + 2 * kk, id, kk > 0 ? 1u : 0u);
                        mma_commit(smem_u32(&bars->d_full[g]));
                    }
                    __syncwarp();
                }
            }
            ++n;
        }
        // every MMA must finish before TMEM is released
        if (elect_one()) {
            mma_commit(smem_u32(&bars->mma_done[0]));
            wait_bar_drain(smem_u32(&bars->mma_done[0]), 0, wait_ns);
        }
        __syncwarp();
    } else if (warp == 2) {
        // ======================================================== dV, dK and dQ MMAs
        DescReader rd{0};
        ItemDesc d;
        uint32_t t = 0, kt = 0;   // units, key tiles
        int slot = 0;
        constexpr uint32_t id = idesc_bf16_f32(128, 64, true), id_q = id | (1u << 15);   // id_q: A is M-major too
        bool ok = true;
        while (ok && rd.next(bars, p, abort_flag, d)) {
            const int L = __shfl_sync(kFull, d.L, 0);
            uint32_t at[kMats];
            const int slot0 = slot;
            for (int m = 0; m < kMats; ++m) {
                at[m] = base + slot * p.slot_bytes;
                slot = slot + 1 == p.slots ? 0 : slot + 1;
            }
            // N = 64 is one 128-byte swizzle atom along N; K steps of 16 rows
            // advance the start by 2048 bytes
            const uint64_t bk = smem_desc_sw128(at[0], 0, 1024), bq = smem_desc_sw128(at[1], 0, 1024);
            const uint64_t bo = smem_desc_sw128(at[3], 0, 1024);
            for (int c = 0; ok && c * kKeys < L; ++c, ++kt) {
                // p_full speaks for one group: the other's warps may still be
                // reading the last tile's sums
                if (kt > 0 && !wait(&bars->acc_empty, kt - 1)) {
                    ok = false;
                    break;
                }
                const int ksteps = (min(kKeys, L - c * kKeys) + 15) >> 4;
                const bool last_c = (c + 1) * kKeys >= L;
                for (int u = 0; u * kUnit < L; ++u, ++t) {
                    const uint32_t g = t & 1;
                    if (!wait(&bars->p_full[g], t >> 1)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const int steps = (min(kUnit, L - u * kUnit) + 15) >> 4;
                    const uint64_t ub = (uint64_t)u * (kUnit * kRowBytes >> 4);
                    const uint64_t ak = smem_desc_sw128(ds_base + u * kChunkBytes, 16, 1024);
                    const bool last_u = (u + 1) * kUnit >= L;
                    const uint32_t ap = tmem + g * kGroupCols;
                    if (elect_one()) {
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk) {
                            if (kk < steps) {
                                const uint64_t row = ub + kk * (16 * kRowBytes >> 4);
                                const uint32_t acc = u > 0 || kk > 0 ? 1u : 0u;
                                mma_ts(tmem + kVAcc, ap + (kk >> 1) * 32 + (kk & 1) * 8, bo + row, id, acc);
                                mma_ss(tmem + kKAcc, ak + 2 * kk, bq + row, id, acc);
                            }
                        }
                        mma_commit(smem_u32(&bars->p_empty[g]));
                        if ((u & 1) || last_u) {
                            const int x = u >> 1;
                            const uint64_t aq = smem_desc_sw128(ds_base + 2 * x * kChunkBytes, kChunkBytes, 1024);
                            for (int kk = 0; kk < ksteps; ++kk) {
                                const uint64_t row = kk * (16 * kRowBytes >> 4);
                                mma_ss(tmem + kQAcc + 64 * x, aq + row, bk + (uint64_t)c * (kTileBytes >> 4) + row, id_q,
                                       c > 0 || kk > 0 ? 1u : 0u);
                            }
                            mma_commit(smem_u32(&bars->dq_done[x]));
                        }
                        if (last_u) {
                            mma_commit(smem_u32(&bars->acc_full));
                            if (last_c)   // the item's matrices are free
                                for (int m = 0; m < kMats; ++m)
                                    mma_commit(smem_u32(&bars->m_empty[slot0 + m < p.slots ? slot0 + m
                                                                                           : slot0 + m - p.slots]));
                        }
                    }
                    __syncwarp();
                }
            }
        }
        if (elect_one()) {
            mma_commit(smem_u32(&bars->mma_done[1]));
            wait_bar_drain(smem_u32(&bars->mma_done[1]), 0, wait_ns);
        }
        __syncwarp();
    } else if (warp == 3) {
        // ======================================================== operand check and columns
        DescReader rd{0};
        ItemDesc d;
        uint32_t n = 0;
        int nm = 0;
        bool ok = true;
        while (ok && rd.next(bars, p, abort_flag, d)) {
            float l[8], dl[8];
            const size_t at = (size_t)d.h * p.total + d.f0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int c = lane + 32 * i;
                l[i] = c < d.L ? __ldg(p.lse + at + c) : INFINITY;
                dl[i] = c < d.L ? __ldg(p.delta + at + c) : 0.f;
            }
            if (n >= 2 && !wait(&bars->cols_empty[n & 1], (n >> 1) - 1))
                break;
            float *cl = cols + (n & 1) * 512;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                cl[lane + 32 * i] = l[i] * -kLog2e;
                cl[256 + lane + 32 * i] = -dl[i];
            }
            const int pad = -d.L & 15;
            for (int m = 0; m < kMats; ++m, ++nm) {
                const int s = nm % p.slots;
                if (!wait(&bars->m_full[s], (uint32_t)(nm / p.slots))) {
                    ok = false;
                    break;
                }
                uint4 *z = reinterpret_cast<uint4 *>(smem + s * p.slot_bytes + d.L * kRowBytes);
                for (int i = lane; i < pad * (kRowBytes / 16); i += 32)
                    z[i] = make_uint4(0, 0, 0, 0);
            }
            if (!ok)
                break;
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(smem_u32(&bars->ready[n & 1]));
            __syncwarp();
            ++n;
        }
    } else {
        // ======================================================== elementwise
        const int e = warp - kElem0;
        const int g = e >> 3, half = (e >> 2) & 1;   // group; half of the unit's columns
        const int qq = warp & 3;                     // TMEM lane quarter of this warp
        const int row = qq * 32 + lane;              // key of the tile
        const uint32_t lanes = (uint32_t)(qq * 32) << 16;
        const uint32_t tS = tmem + g * kGroupCols + kCols * half + lanes;
        const uint64_t k2 = pair(p.scale_log2, p.scale_log2);
        DescReader rd{0};
        ItemDesc d;
        uint32_t n = 0, t = 0, kt = 0;       // items, units, key tiles
        uint32_t nx[2] = {0, 0};             // key tiles that had queries in half x of the block
        Pending pend{};
        bool ok = true;

        // Stores the pending results once they are complete.
        auto store = [&]() -> bool {
            if (!pend.have)
                return true;
            pend.have = false;
            if (!wait(&bars->acc_full, kt - 1))
                return false;
            tc_fence_after();
            // dK by the first group, dV by the second; half of the columns per warp
            const int nk = pend.L - pend.c * kKeys;
            const int f = pend.f0 + pend.c * kKeys + row;
            if (qq * 32 < nk)
                store_acc(tmem + (g ? kVAcc : kKAcc) + kCols * half + lanes, g ? 1.f : p.scale,
                          (g ? p.dv : p.dk) + (long long)f * p.out_stride + pend.h * 64 + kCols * half, row < nk);
            if (pend.last) {   // dQ of queries 128 g .. by group g
                const int nq = pend.L - g * kKeys;
                if (qq * 32 < nq)
                    store_acc(tmem + kQAcc + 64 * g + kCols * half + lanes, p.scale,
                              p.dq + (long long)(pend.f0 + g * kKeys + row) * p.out_stride + pend.h * 64 + kCols * half,
                              row < nq);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(smem_u32(&bars->acc_empty));
            return true;
        };

        for (; ok && rd.next(bars, p, abort_flag, d); ++n) {
            if (!wait(&bars->ready[n & 1], n >> 1)) {
                ok = false;
                break;
            }
            const float *cl = cols + (n & 1) * 512;
            for (int c = 0; ok && c * kKeys < d.L; ++c) {
                const bool active = c * kKeys + qq * 32 < d.L;   // warp-uniform
                const bool row_ok = c * kKeys + row < d.L;
                for (int u = 0; u * kUnit < d.L; ++u, ++t) {
                    if ((t & 1) != (uint32_t)g)
                        continue;
                    const uint32_t use = t >> 1;
                    const int c0 = u * kUnit + kCols * half;   // first query of the warp's columns
                    const int x = u >> 1;
                    if (!wait(&bars->s_full[g], use)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const bool work = active && c0 < d.L;      // warp-uniform
                    uint64_t pr[kCols / 2];
                    uint32_t pk[kCols / 2];
                    if (work) {
                        uint32_t s[kCols];
                        tmem_ld32_nowait(tS, s);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < kCols; ++i)
                            reg_fence(s[i]);
#pragma unroll
                        for (int i = 0; i < kCols / 4; ++i) {
                            const float4 l = reinterpret_cast<const float4 *>(cl + c0)[i];
                            const uint64_t y0 = fma2(pair(s[4 * i], s[4 * i + 1]), k2, pair(l.x, l.y));
                            const uint64_t y1 = fma2(pair(s[4 * i + 2], s[4 * i + 3]), k2, pair(l.z, l.w));
                            float a, b;
                            unpair(y0, a, b);
                            pr[2 * i] = pair(ex2_approx(a), ex2_approx(b));
                            unpair(y1, a, b);
                            pr[2 * i + 1] = pair(ex2_approx(a), ex2_approx(b));
                        }
#pragma unroll
                        for (int i = 0; i < kCols / 2; ++i) {
                            float a, b;
                            unpair(pr[i], a, b);
                            pk[i] = pack_bf16x2(a, b);
                        }
                        tmem_st16p(tS, pk);
                    }
                    if (!wait(&bars->d_full[g], use)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    if (work) {
                        uint32_t dd[kCols];
                        tmem_ld32_nowait(tS + kDCol, dd);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < kCols; ++i)
                            reg_fence(dd[i]);
#pragma unroll
                        for (int i = 0; i < kCols / 4; ++i) {
                            const float4 l = reinterpret_cast<const float4 *>(cl + 256 + c0)[i];
                            pr[2 * i] = mul2(pr[2 * i], add2(pair(dd[4 * i], dd[4 * i + 1]), pair(l.x, l.y)));
                            pr[2 * i + 1] = mul2(pr[2 * i + 1], add2(pair(dd[4 * i + 2], dd[4 * i + 3]), pair(l.z, l.w)));
                        }
#pragma unroll
                        for (int i = 0; i < kCols / 2; ++i) {
                            float a, b;
                            unpair(pr[i], a, b);
                            // keys past the block: nothing to dQ
                            pk[i] = row_ok ? pack_bf16x2(a, b) : 0u;
                        }
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(smem_u32(&bars->d_empty[g]));
                    // the last key tile's dQ no longer reads these chunks
                    if (nx[x] > 0 && !wait(&bars->dq_done[x], nx[x] - 1)) {
                        ok = false;
                        break;
                    }
                    if (work) {
                        uint8_t *dst = smem + p.ds_off + u * kChunkBytes + row * kRowBytes;
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            *reinterpret_cast<uint4 *>(dst + ((4 * half + i) ^ (row & 7)) * 16) =
                                make_uint4(pk[4 * i], pk[4 * i + 1], pk[4 * i + 2], pk[4 * i + 3]);
                        fence_proxy_async_smem();
                        tmem_wait_st();
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(smem_u32(&bars->p_full[g]));
                    if (!store()) {
                        ok = false;
                        break;
                    }
                }
                if (!ok || !store()) {   // a tile without a unit for this group
                    ok = false;
                    break;
                }
                ++nx[0];
                if (d.L > kKeys)
                    ++nx[1];
                pend = Pending{d.f0, d.L, d.h, c, true, (c + 1) * kKeys >= d.L};
                ++kt;
            }
            if (!ok)
                break;
            __syncwarp();
            if (lane == 0)
                mbar_arrive(smem_u32(&bars->cols_empty[n & 1]));
        }
        if (ok)
            store();
    }

    // ------------------------------------------------------------ teardown
    tc_fence_before();
    __syncthreads();
    if (warp == 3) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

} // namespace

namespace nle {

int launch_block_bwd(const BlockBwdArgs &a, const DeviceInfo &di, int dev, long long items, cudaStream_t st)
{
    Params p{};
    p.cu = a.cu;
    p.n_seq = a.n_seq;
    p.total = (int)a.total;
    p.heads = a.heads;
    p.block = a.block;
    // every slot holds the block rounded up to the MMAs' 16-row granule; the
    // 128-row operands of K and V read past their slot, into the next ones
    // or dS (their surplus rows reach no result)
    p.slot_bytes = (uint32_t)((a.block + 15) / 16 * 16 * kRowBytes);
    const uint32_t chunks = (uint32_t)((a.block + kKeys - 1) / kKeys) * 2;
    const uint32_t ds_bytes = chunks * kChunkBytes;
    const uint32_t tail = 2 * 512 * 4 + ((sizeof(Bars) + 127) / 128) * 128 + 1024;
    int slots = (int)((di.smem_optin - ds_bytes - tail) / p.slot_bytes);
    if (slots > kMaxSlots)
        slots = kMaxSlots;
    if (slots < kMats)
        return NLE_ERR_UNSUPPORTED;
    p.slots = slots;
    p.ds_off = slots * p.slot_bytes;
    p.col_off = p.ds_off + ds_bytes;
    p.bars_off = p.col_off + 2 * 512 * 4;
    size_t smem = p.ds_off + ds_bytes + tail;
    // one CTA per SM: it owns all 512 TMEM columns
    if (smem <= (size_t)di.smem_optin / 2)
        smem = (size_t)di.smem_optin / 2 + 1024;
    p.scale = a.scale;
    p.scale_log2 = a.scale_log2;
    p.lse = a.lse;
    p.delta = a.delta;
    p.dq = static_cast<__nv_bfloat16 *>(a.dq);
    p.dk = static_cast<__nv_bfloat16 *>(a.dk);
    p.dv = static_cast<__nv_bfloat16 *>(a.dv);
    p.out_stride = a.dstride;
    p.status = a.status;
    p.wait_ns = a.wait_ns;
    p.flags = a.flags;
    CUtensorMap tq, tk, tv, tdo;
    const uint64_t cols = (uint64_t)a.heads * 64, rows = (uint64_t)a.total;
    if (!encode_tmap_bf16_2d(&tq, a.q, cols, rows, a.stride, 64, a.block) ||
        !encode_tmap_bf16_2d(&tk, a.k, cols, rows, a.stride, 64, a.block) ||
        !encode_tmap_bf16_2d(&tv, a.v, cols, rows, a.stride, 64, a.block) ||
        !encode_tmap_bf16_2d(&tdo, a.dout, cols, rows, cols, 64, a.block))
        return NLE_ERR_CUDA;
    if (!allow_max_dynamic_smem(reinterpret_cast<const void *>(block_bwd_kernel), dev, di.smem_optin))
        return NLE_ERR_CUDA;
    const int grid = (int)(items < di.sm_count ? items : di.sm_count);
    block_bwd_kernel<<<grid, kThreads, smem, st>>>(tq, tk, tv, tdo, p);
    return cudaGetLastError() == cudaSuccess ? NLE_OK : NLE_ERR_CUDA;
}

} // namespace nle
