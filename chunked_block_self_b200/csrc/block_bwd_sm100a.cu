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
//     dV_c += P dO_u     A = P in TMEM (over D), B = dO rows
//     dK_c += dS Q_u     A = dS in shared memory, K-major, B = Q rows
//     dQ_x += dS^T K_c   A = the same shared memory read M-major: 128 queries
//                        (two units), K = the tile's keys, B = K rows
// P and dS are rounded once to bf16, the type that the MMAs take at the full
// rate (errors as in attn_bwd_sm100a.cu).  dS is written once, as 64-query chunks of 128-byte rows (one key each),
// 128-byte swizzled: a row-major operand for dK and a column-major one for dQ.
//
// One persistent CTA per SM, 16 warps:
//   warp 0   TMA producer: K, Q, V, dO of an item, one box each; publishes the
//            item's descriptor.  Where dS leaves room for more than one item's
//            matrices, K, Q, dO, V have two slots each in that order; of the
//            others the next item's are fetched into L2 meanwhile.
//   warp 1   issues S and D: an item's first two S before its V and dO are
//            there, then S and D of a unit in turn.
//   warp 2   issues dV (as soon as P is written), dK and dQ.
//   warp 3   owns TMEM; zeroes operand rows past the block (up to the MMAs'
//            16-row granule: their P and dS are 0, but 0 * Inf would be NaN)
//            and stages the block's lse and delta (+inf and 0 past it).
//   warps 4-7   results: a key tile's dK and dV, an item's dQ.
//   warps 8-15  elementwise, two groups of four warps on alternate units
//            (group g: S, D buffer g): a lane owns one key of the tile.
// TMEM (512 columns): S, D of group g at 128 g and 128 g + 64 (P over D's
// first 32 columns, so that the group's next S need not wait for dV), dQ_0,
// dQ_1 at 256 and 320, dK at 384, dV at 448.
//
// What bounds it: a 200-frame block of one head takes 17 k cycles.  2.7 k of
// them wait for its V and dO, which have one slot each; its eight units follow
// at 1.8 k each, two in flight: the elementwise work of one is about 2 k (512
// for its exps), the hops between its warps and the issue of its MMAs as much
// again, the tensor pipe busy for 0.9 k.  HBM would allow 8 k.  The batch of
// 128 utterances (16 heads, 58,903 frames, 5,648 items): 0.36 ms, and 0.04 ms
// for delta: 2.4 TB/s of the operator's bytes.  Steps that paid, on a batch of
// 34,512 frames: no spilled registers (388 -> 293 us; beside 200 KB of shared
// memory a spill lives in L2), results on warps of their own and S ahead
// (-> 266), elementwise code short enough for the instruction cache and the
// first S ahead of V and dO (-> 248; alone 262 and 309), dV before dS and S, D
// in turn (-> 243).  Four elementwise groups of 32 columns: 253; delta formed
// here by four more warps: 260.
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

constexpr int kEpi0 = 4;                             // first of four result warps
constexpr int kElem0 = 8;                            // first elementwise warp
constexpr int kElemWarps = 8;                        // two groups of four
constexpr int kThreads = 32 * (kElem0 + kElemWarps); // 512
constexpr int kKeys = 128;                           // keys of a tile (MMA M)
constexpr int kUnit = 64;                            // queries of a unit
constexpr int kRowBytes = 128;                       // one frame of one head: 64 bf16
constexpr uint32_t kTileBytes = kKeys * kRowBytes;   // 16 KB
constexpr uint32_t kChunkBytes = kKeys * kRowBytes;  // dS of a unit: 128 keys x 64 queries
constexpr int kMaxSlots = 8;
constexpr int kMats = 4;
enum { kMatK, kMatQ, kMatO, kMatV };                 // O: dO
constexpr int kDescRing = 4;
constexpr int kDescReaders = 3 + 4 + kElemWarps;     // both MMA, check, result and elementwise warps
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kGroupCols = 128, kDCol = 64, kQAcc = 256, kKAcc = 384, kVAcc = 448;

struct ItemDesc {
    int f0, L, h;   // the block (L < 0: no further item)
};

struct Bars {
    uint64_t m_full[kMaxSlots];
    uint64_t m_empty[kMaxSlots];    // the item's last MMAs on the matrix have completed
    uint64_t ready_s[2];            // by item: K and Q checked, columns staged
    uint64_t ready_d[2];            // by item: V and dO checked
    uint64_t cols_empty[2];         // kElemWarps arrivals: the item's columns are no longer read
    uint64_t s_full[2], d_full[2];  // by group
    uint64_t s_empty[2];            // 4 arrivals: S has been read
    uint64_t p_full[2];             // 4 arrivals: P written, D read
    uint64_t ds_full[4];            // by unit & 3; 4 arrivals: dS written
    uint64_t p_empty[2];            // the unit's dV MMAs have completed (P, over D)
    uint64_t dq_done[2];            // the key tile's dQ_x MMAs have completed (dS chunks 2x, 2x + 1)
    uint64_t idle;                  // 4 arrivals: the group without a unit in an item of one unit
    uint64_t acc_full;              // the key tile's sums (the item's, on its last) are complete
    uint64_t acc_empty;             // 4 arrivals: dK and dV have been read
    uint64_t dq_empty;              // 4 arrivals: the item's dQ has been read
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

// A box into L2, ahead of its load.
__device__ __forceinline__ void tma_prefetch_2d(const CUtensorMap *tm, int x, int y)
{
    asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];"
                 ::"l"(reinterpret_cast<uint64_t>(tm)), "r"(x), "r"(y)
                 : "memory");
}

// Matrix m of item n: the first slots - 4 of K, Q, dO, V have two slots each.
struct Slot {
    int at, use;   // slot; how often it was used before
    __device__ __forceinline__ Slot(int m, int n, int slots)
    {
        const int two = slots - kMats;
        const bool twice = m < two;
        at = m + min(m, two) + (twice ? n & 1 : 0);
        use = twice ? n >> 1 : n;
    }
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

// A unit for a warp without keys in the tile: it only keeps the barriers' count.
__device__ __forceinline__ bool unit_idle(Bars *bars, int g, int x, uint32_t use, uint32_t nx, const Params &p,
                                          volatile int *abort_flag)
{
    if (!wait_bar(smem_u32(&bars->s_full[g]), use & 1, abort_flag, p.wait_ns, p.status))
        return false;
    __syncwarp();
    if ((threadIdx.x & 31) == 0)
        mbar_arrive(smem_u32(&bars->s_empty[g]));
    if (!wait_bar(smem_u32(&bars->d_full[g]), use & 1, abort_flag, p.wait_ns, p.status))
        return false;
    __syncwarp();
    if ((threadIdx.x & 31) == 0)
        mbar_arrive(smem_u32(&bars->p_full[g]));
    return nx == 0 || wait_bar(smem_u32(&bars->dq_done[x]), (nx - 1) & 1, abort_flag, p.wait_ns, p.status);
}

// A unit for one lane (one key), 32 queries at a time (rolled: the two groups
// walk this code at different places, and the longer straight line missed the
// instruction cache): P to TMEM over D, dS to the lane's row of the
// shared-memory chunk (128-byte swizzle).  halves: 32-query parts inside the
// block.  cl: the queries' -lse log2e, and 256 floats on their -delta.  Keys
// past the block (not row_ok) give dS = 0: dQ sums over all keys of the MMAs'
// 16-row granule.
__device__ __forceinline__ bool unit_work(uint32_t tS, uint32_t cl, uint8_t *dst, int row, bool row_ok, int halves,
                                          Bars *bars, int g, int x, uint32_t use, uint32_t nx, const Params &p,
                                          volatile int *abort_flag)
{
    if (!wait_bar(smem_u32(&bars->s_full[g]), use & 1, abort_flag, p.wait_ns, p.status))
        return false;
    tc_fence_after();
    const uint64_t k2 = pair(p.scale_log2, p.scale_log2);
    const uint32_t tP = tS + kDCol;
#pragma unroll 1
    for (int h = 0; h < halves; ++h) {
        uint32_t s[32];
        tmem_ld32_nowait(tS + 32 * h, s);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 32; ++i)
            reg_fence(s[i]);
        if (h + 1 == halves) {
            tc_fence_before();
            __syncwarp();
            if ((threadIdx.x & 31) == 0)
                mbar_arrive(smem_u32(&bars->s_empty[g]));
        }
        uint64_t pr[16];
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            uint64_t l0, l1;
            lds_pairs(cl + 128 * h + 16 * q, l0, l1);
            const uint64_t y0 = fma2(pair(s[4 * q], s[4 * q + 1]), k2, l0);
            const uint64_t y1 = fma2(pair(s[4 * q + 2], s[4 * q + 3]), k2, l1);
            float a, b;
            unpair(y0, a, b);
            pr[2 * q] = pair(ex2_approx(a), ex2_approx(b));
            unpair(y1, a, b);
            pr[2 * q + 1] = pair(ex2_approx(a), ex2_approx(b));
        }
        // D, and the last key tile's dQ no longer reads this half's chunks
        if (h == 0 && (!wait_bar(smem_u32(&bars->d_full[g]), use & 1, abort_flag, p.wait_ns, p.status) ||
                       (nx > 0 &&
                        !wait_bar(smem_u32(&bars->dq_done[x]), (nx - 1) & 1, abort_flag, p.wait_ns, p.status))))
            return false;
        tc_fence_after();
        uint32_t d[32], pk[16];
        tmem_ld32_nowait(tP + 32 * h, d);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float a, b;
            unpair(pr[i], a, b);
            pk[i] = pack_bf16x2(a, b);
        }
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 32; ++i)
            reg_fence(d[i]);
        tmem_st16p(tP + 16 * h, pk);   // over columns of D that are in registers or past
        if (h + 1 == halves) {   // dV, and after it the next unit's D, need not wait for dS
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if ((threadIdx.x & 31) == 0)
                mbar_arrive(smem_u32(&bars->p_full[g]));
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t o[4];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int q = 2 * i + j;
                uint64_t l0, l1;
                lds_pairs(cl + 1024 + 128 * h + 16 * q, l0, l1);
                const uint64_t g0 = mul2(pr[2 * q], add2(pair(d[4 * q], d[4 * q + 1]), l0));
                const uint64_t g1 = mul2(pr[2 * q + 1], add2(pair(d[4 * q + 2], d[4 * q + 3]), l1));
                float a, b;
                unpair(g0, a, b);
                o[2 * j] = row_ok ? pack_bf16x2(a, b) : 0u;
                unpair(g1, a, b);
                o[2 * j + 1] = row_ok ? pack_bf16x2(a, b) : 0u;
            }
            *reinterpret_cast<uint4 *>(dst + ((4 * h + i) ^ (row & 7)) * 16) = make_uint4(o[0], o[1], o[2], o[3]);
        }
    }
    fence_proxy_async_smem();
    return true;
}

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
            mbar_init(smem_u32(&bars->ready_s[g]), 1);
            mbar_init(smem_u32(&bars->ready_d[g]), 1);
            mbar_init(smem_u32(&bars->cols_empty[g]), kElemWarps);
            mbar_init(smem_u32(&bars->s_full[g]), 1);
            mbar_init(smem_u32(&bars->d_full[g]), 1);
            mbar_init(smem_u32(&bars->s_empty[g]), kElemWarps / 2);
            mbar_init(smem_u32(&bars->p_full[g]), kElemWarps / 2);
            mbar_init(smem_u32(&bars->ds_full[g]), kElemWarps / 2);
            mbar_init(smem_u32(&bars->ds_full[2 + g]), kElemWarps / 2);
            mbar_init(smem_u32(&bars->p_empty[g]), 1);
            mbar_init(smem_u32(&bars->dq_done[g]), 1);
            mbar_init(smem_u32(&bars->mma_done[g]), 1);
        }
        mbar_init(smem_u32(&bars->idle), kElemWarps / 2);
        mbar_init(smem_u32(&bars->acc_full), 1);
        mbar_init(smem_u32(&bars->acc_empty), 4);
        mbar_init(smem_u32(&bars->dq_empty), 4);
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

    if (warp < kEpi0) {
        if (warp == 0) {
            // ======================================================== producer
            PlanWalker w;
            w.init(p.cu, p.n_seq, p.total, p.block, lane);
            const bool skip0 = (p.flags & NLE_FLAG_TEST_SKIP_FIRST_LOAD) != 0;
            const uint64_t pol = policy_evict_first();   // every matrix is read once
            const uint32_t bytes = (uint32_t)p.block * kRowBytes;
            int n = 0;      // items published
            int last = kMats;   // matrices claimed of the last of them
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
                // V's slot is free after the last item's last D, dO's after its
                // last dV: both before the item's end
                for (last = 0; last < kMats; ++last) {
                    const int m = last < 2 ? last : last == 2 ? kMatV : kMatO;
                    if (last == 2 && n > 1 && lane == 0) {
                        tma_prefetch_2d(&tm_v, d.h * 64, d.f0);
                        tma_prefetch_2d(&tm_do, d.h * 64, d.f0);
                    }
                    const Slot s(m, n - 1, p.slots);
                    if (s.use > 0 && !wait(&bars->m_empty[s.at], (uint32_t)(s.use - 1))) {
                        stop = true;
                        break;
                    }
                    if (lane == 0 && !(skip0 && n == 1 && last == 0)) {
                        const uint32_t bar = smem_u32(&bars->m_full[s.at]);
                        mbar_arrive_expect_tx(bar, bytes);
                        tma_load_2d(base + s.at * p.slot_bytes,
                                    m == kMatK ? &tm_k : m == kMatQ ? &tm_q : m == kMatV ? &tm_v : &tm_do, d.h * 64,
                                    d.f0, bar, pol);
                    }
                    __syncwarp();
                }
            }
            if (w.bad && lane == 0)
                report(p.status, NLE_ERR_INVALID_ARG);
            const int items = n;
            if (!stop)
                publish(ItemDesc{0, -1, 0});
            // drain: the last copy into each slot must land before exit
            if (lane == 0)
                for (int j = 0; j < kMats; ++j) {
                    const int m = j < 2 ? j : j == 2 ? kMatV : kMatO;
                    const int claimed = items - (j >= last ? 1 : 0);
                    for (int i = max(claimed - (m < p.slots - kMats ? 2 : 1), 0); i < claimed; ++i) {
                        const Slot s(m, i, p.slots);
                        if (!(skip0 && i == 0 && j == 0))
                            wait_bar_drain(smem_u32(&bars->m_full[s.at]), (uint32_t)s.use & 1, wait_ns);
                    }
                }
            __syncwarp();
        } else if (warp == 1) {
            // ======================================================== S and D MMAs
            DescReader rd{0};
            ItemDesc d;
            uint32_t n = 0, t = 0;   // items, units
            bool ok = true;
            while (ok && rd.next(bars, p, abort_flag, d)) {
                if (!wait(&bars->ready_s[n & 1], n >> 1))
                    break;
                const int L = __shfl_sync(kFull, d.L, 0);
                auto mat = [&](int m) {
                    return smem_desc_sw128(base + Slot(m, (int)n, p.slots).at * p.slot_bytes, 16, 1024);
                };
                const uint64_t dk0 = mat(kMatK), dq0 = mat(kMatQ), dv0 = mat(kMatV), do0 = mat(kMatO);
                const int v_slot = Slot(kMatV, (int)n, p.slots).at;
                const int nu = (L + kUnit - 1) / kUnit, units = nu * ((L + kKeys - 1) / kKeys);
                // the item's first two S before its V and dO have arrived; then
                // S and D of a unit in turn, as the units before them end
                int sc = 0, su = 0, dc = 0, du = 0;   // key tile and 64-query part of the next S and D
                for (int i = 0, si = 0; ok && i < units; ++i) {
                    for (; ok && si < units && si < max(i + 1, 2); ++si) {
                        const uint32_t g = (t + si) & 1, use = (t + si) >> 1;
                        const uint32_t id = idesc_bf16_f32(128, min(kUnit, (L - su * kUnit + 15) & ~15), false);
                        const uint64_t a = dk0 + sc * (kTileBytes >> 4), b = dq0 + su * (kUnit * kRowBytes >> 4);
                        if (use > 0 && !wait(&bars->s_empty[g], use - 1)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        // K steps of 16 elements = 32 bytes inside the 128-byte swizzle atom
                        if (elect_one()) {
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk)
                                mma_ss(tmem + g * kGroupCols, a + 2 * kk, b + 2 * kk, id, kk > 0 ? 1u : 0u);
                            mma_commit(smem_u32(&bars->s_full[g]));
                        }
                        __syncwarp();
                        if (++su == nu) {
                            su = 0;
                            ++sc;
                        }
                    }
                    const uint32_t g = (t + i) & 1, use = (t + i) >> 1;
                    const uint32_t id = idesc_bf16_f32(128, min(kUnit, (L - du * kUnit + 15) & ~15), false);
                    const uint64_t a = dv0 + dc * (kTileBytes >> 4), b = do0 + du * (kUnit * kRowBytes >> 4);
                    if (!ok || (i == 0 && !wait(&bars->ready_d[n & 1], n >> 1)) ||
                        (use > 0 && !wait(&bars->p_empty[g], use - 1))) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    if (elect_one()) {
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            mma_ss(tmem + g * kGroupCols + kDCol, a + 2 * kk, b + 2 * kk, id, kk > 0 ? 1u : 0u);
                        mma_commit(smem_u32(&bars->d_full[g]));
                        if (i + 1 == units)
                            mma_commit(smem_u32(&bars->m_empty[v_slot]));
                    }
                    __syncwarp();
                    if (++du == nu) {
                        du = 0;
                        ++dc;
                    }
                }
                t += units;
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
            uint32_t t = 0, kt = 0, n = 0, idle = 0;   // units, key tiles, items, items of one unit
            constexpr uint32_t id = idesc_bf16_f32(128, 64, true), id_q = id | (1u << 15);   // id_q: A is M-major too
            bool ok = true;
            while (ok && rd.next(bars, p, abort_flag, d)) {
                const int L = __shfl_sync(kFull, d.L, 0);
                const int sk = Slot(kMatK, (int)n, p.slots).at, sq = Slot(kMatQ, (int)n, p.slots).at;
                const int so = Slot(kMatO, (int)n, p.slots).at;
                // N = 64 is one 128-byte swizzle atom along N; K steps of 16 rows
                // advance the start by 2048 bytes
                const uint64_t bk = smem_desc_sw128(base + sk * p.slot_bytes, 0, 1024);
                const uint64_t bq = smem_desc_sw128(base + sq * p.slot_bytes, 0, 1024);
                const uint64_t bo = smem_desc_sw128(base + so * p.slot_bytes, 0, 1024);
                for (int c = 0; ok && c * kKeys < L; ++c, ++kt) {
                    // the last tile's dK and dV have been read
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
                        const uint32_t ap = tmem + g * kGroupCols + kDCol;
                        if (elect_one()) {
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk)
                                if (kk < steps)
                                    mma_ts(tmem + kVAcc, ap + kk * 8, bo + ub + kk * (16 * kRowBytes >> 4), id,
                                           u > 0 || kk > 0 ? 1u : 0u);
                            mma_commit(smem_u32(&bars->p_empty[g]));
                            if (last_u && last_c)
                                mma_commit(smem_u32(&bars->m_empty[so]));
                        }
                        __syncwarp();
                        // dS; and for the item's first dQ: the last item's has been read
                        if (!wait(&bars->ds_full[t & 3], t >> 2) || (L <= kUnit && !wait(&bars->idle, idle++)) ||
                            (c == 0 && (u == 1 || (u == 0 && last_u)) && n > 0 && !wait(&bars->dq_empty, n - 1))) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        if (elect_one()) {
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk)
                                if (kk < steps)
                                    mma_ss(tmem + kKAcc, ak + 2 * kk, bq + ub + kk * (16 * kRowBytes >> 4), id,
                                           u > 0 || kk > 0 ? 1u : 0u);
                            if (last_u && last_c)
                                mma_commit(smem_u32(&bars->m_empty[sq]));
                            if ((u & 1) || last_u) {
                                const int x = u >> 1;
                                const uint64_t aq = smem_desc_sw128(ds_base + 2 * x * kChunkBytes, kChunkBytes, 1024);
                                for (int kk = 0; kk < ksteps; ++kk) {
                                    const uint64_t row = kk * (16 * kRowBytes >> 4);
                                    mma_ss(tmem + kQAcc + 64 * x, aq + row, bk + c * (kTileBytes >> 4) + row, id_q,
                                           c > 0 || kk > 0 ? 1u : 0u);
                                }
                                mma_commit(smem_u32(&bars->dq_done[x]));
                            }
                            if (last_u) {
                                mma_commit(smem_u32(&bars->acc_full));
                                if (last_c)
                                    mma_commit(smem_u32(&bars->m_empty[sk]));
                            }
                        }
                        __syncwarp();
                    }
                }
                ++n;
            }
            if (elect_one()) {
                mma_commit(smem_u32(&bars->mma_done[1]));
                wait_bar_drain(smem_u32(&bars->mma_done[1]), 0, wait_ns);
            }
            __syncwarp();
        } else {
            // ======================================================== operand check and columns
            DescReader rd{0};
            ItemDesc d;
            uint32_t n = 0;
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
                for (int half = 0; ok && half < 2; ++half) {   // K and Q, then V and dO
                    for (int m = 2 * half; m < 2 * half + 2; ++m) {
                        const Slot s(m, (int)n, p.slots);
                        if (!wait(&bars->m_full[s.at], (uint32_t)s.use)) {
                            ok = false;
                            break;
                        }
                        uint4 *z = reinterpret_cast<uint4 *>(smem + s.at * p.slot_bytes + d.L * kRowBytes);
                        for (int i = lane; i < pad * (kRowBytes / 16); i += 32)
                            z[i] = make_uint4(0, 0, 0, 0);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (ok && lane == 0)
                        mbar_arrive(smem_u32(&(half ? bars->ready_d : bars->ready_s)[n & 1]));
                    __syncwarp();
                }
                ++n;
            }
        }
    } else if (warp < kElem0) {
        // ======================================================== results
        const int qq = warp & 3;   // TMEM lane quarter of this warp
        const uint32_t lanes = (uint32_t)(qq * 32) << 16;
        DescReader rd{0};
        ItemDesc d;
        uint32_t kt = 0;   // key tiles
        bool ok = true;
        while (ok && rd.next(bars, p, abort_flag, d)) {
            for (int c = 0; c * kKeys < d.L; ++c, ++kt) {
                if (!wait(&bars->acc_full, kt)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                // rows that are not there are read too and stored by nothing
                const int nk = d.L - c * kKeys - qq * 32;
                const long long at = (long long)(d.f0 + c * kKeys + qq * 32) * p.out_stride + d.h * 64;
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    uint32_t o[2][16];
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        load_acc(tmem + (m ? kVAcc : kKAcc) + 32 * h + lanes, m ? 1.f : p.scale, o[h]);
                    if (m) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0)
                            mbar_arrive(smem_u32(&bars->acc_empty));
                    }
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        store_rows(o[h], (m ? p.dv : p.dk) + at + 32 * h, p.out_stride, nk);
                }
                if ((c + 1) * kKeys < d.L)
                    continue;
                // the item's last key tile: dQ
                for (int x = 0; x * kKeys < d.L; ++x) {
                    uint32_t o[2][16];
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        load_acc(tmem + kQAcc + 64 * x + 32 * h + lanes, p.scale, o[h]);
                    if ((x + 1) * kKeys >= d.L) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0)
                            mbar_arrive(smem_u32(&bars->dq_empty));
                    }
                    const long long aq = (long long)(d.f0 + x * kKeys + qq * 32) * p.out_stride + d.h * 64;
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        store_rows(o[h], p.dq + aq + 32 * h, p.out_stride, d.L - x * kKeys - qq * 32);
                }
            }
        }
    } else {
        // ======================================================== elementwise
        const int g = (warp - kElem0) >> 2;          // group
        const int qq = warp & 3;                     // TMEM lane quarter of this warp
        const int row = qq * 32 + lane;              // key of the tile
        const uint32_t lanes = (uint32_t)(qq * 32) << 16;
        const uint32_t tS = tmem + g * kGroupCols + lanes;
        DescReader rd{0};
        ItemDesc d;
        uint32_t n = 0, t = 0;               // items; units before the tile
        uint32_t nx0 = 0, nx1 = 0;           // key tiles that had queries in half 0, 1 of the block
        bool ok = true;
        for (; ok && rd.next(bars, p, abort_flag, d); ++n) {
            if (!wait(&bars->ready_s[n & 1], n >> 1))
                break;
            const uint32_t cl = smem_u32(cols) + (n & 1) * 2048;
            for (int c = 0; ok && c * kKeys < d.L; ++c) {
                const bool active = c * kKeys + qq * 32 < d.L;   // warp-uniform
                const bool row_ok = c * kKeys + row < d.L;
                // the group's units of the tile
                const int u0 = (t ^ g) & 1;
                for (int u = u0; u * kUnit < d.L; u += 2) {
                    const uint32_t use = (t + u) >> 1;
                    const int c0 = u * kUnit;           // first query of the unit
                    const bool two = c0 + 32 < d.L;    // warp-uniform: queries in the unit's second half
                    const uint32_t nx = u >> 1 ? nx1 : nx0;
                    uint8_t *dst = smem + p.ds_off + u * kChunkBytes + row * kRowBytes;
                    const int x = u >> 1;
                    ok = !active ? unit_idle(bars, g, x, use, nx, p, abort_flag)
                                 : unit_work(tS, cl + 4 * c0, dst, row, row_ok, two ? 2 : 1, bars, g, x, use, nx, p,
                                             abort_flag);
                    // no unit of this group in the other half: its phase is
                    // waited for all the same, before the half's next one can
                    // end (a parity wait only tells the phase before apart)
                    if (ok && d.L > kKeys && (2 + u0) * kUnit >= d.L && nx1 > 0 && !wait(&bars->dq_done[1], nx1 - 1))
                        ok = false;
                    if (!ok)
                        break;
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(smem_u32(&bars->ds_full[(t + u) & 3]));
                }
                if (ok && u0 * kUnit >= d.L) {   // no unit at all: the same, and warp 2 waits for it
                    if (nx0 > 0 && !wait(&bars->dq_done[0], nx0 - 1))
                        ok = false;
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(smem_u32(&bars->idle));
                }
                t += (d.L + kUnit - 1) / kUnit;
                ++nx0;
                nx1 += d.L > kKeys;
            }
            __syncwarp();
            if (lane == 0)
                mbar_arrive(smem_u32(&bars->cols_empty[n & 1]));
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
    const int rc = launch_attn_delta(a.out, a.dout, a.delta, a.total, a.heads, di, st);
    if (rc != NLE_OK)
        return rc;
    const int grid = (int)(items < di.sm_count ? items : di.sm_count);
    block_bwd_kernel<<<grid, kThreads, smem, st>>>(tq, tk, tv, tdo, p);
    return cudaGetLastError() == cudaSuccess ? NLE_OK : NLE_ERR_CUDA;
}

} // namespace nle
