// attn_bwd.cuh -- pieces shared by the attention gradient kernels (sm_100a).
#pragma once

#include "nle_device.cuh"
#include "nle_host.h"

namespace nle {

constexpr float kLog2e = 1.4426950408889634f;

// 2-D tiled TMA load (no multicast) with the default L2 policy.
__device__ __forceinline__ void tma_load(uint32_t dst, const void *tmap, int32_t x, int32_t y, uint32_t bar)
{
    asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes"
                 " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
                 "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(bar)
                 : "memory");
}

// ---------------------------------------------------------------- packed fp32 pairs
__device__ __forceinline__ uint64_t pair(uint32_t lo, uint32_t hi)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
    return r;
}

__device__ __forceinline__ uint64_t pair(float lo, float hi)
{
    return pair(__float_as_uint(lo), __float_as_uint(hi));
}

__device__ __forceinline__ void unpair(uint64_t p, float &lo, float &hi)
{
    uint32_t a, b;
    asm("mov.b64 {%0, %1}, %2;" : "=r"(a), "=r"(b) : "l"(p));
    lo = __uint_as_float(a);
    hi = __uint_as_float(b);
}

// Keeps the compiler from moving a pair's computation across this point.
__device__ __forceinline__ void pair_fence(uint64_t &x)
{
    asm volatile("" : "+l"(x));
}

// Four consecutive fp32 of shared memory as two pairs; not moved across fences.
__device__ __forceinline__ void lds_pairs(uint32_t addr, uint64_t &a, uint64_t &b)
{
    asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];" : "=l"(a), "=l"(b) : "r"(addr));
}

__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// 32 fp32 columns of an accumulator row (one row per lane), times f, as 16
// packed bf16 pairs.
__device__ __forceinline__ void load_acc(uint32_t tacc, float f, uint32_t (&o)[16])
{
    uint32_t r[32];
    tmem_ld32_nowait(tacc, r);
    tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < 32; ++i)
        reg_fence(r[i]);
#pragma unroll
    for (int i = 0; i < 16; ++i)
        o[i] = pack_bf16x2(__uint_as_float(r[2 * i]) * f, __uint_as_float(r[2 * i + 1]) * f);
}

// Stores such rows (64 bytes each, row i of the warp at dst + i * stride
// elements, rows < n).  A lane's row is four 16-byte pieces; stored as they
// are, every store would touch 32 lines.  The pieces are transposed within
// quads of lanes first (two butterfly steps), so that a store covers 64 bytes
// of eight rows.  Whole warp.
__device__ __forceinline__ void store_rows(const uint32_t (&o)[16], __nv_bfloat16 *dst, long long stride, int n)
{
    const int lane = threadIdx.x & 31;
    const bool odd = lane & 1, high = lane & 2;
    uint4 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        v[i] = make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
    auto swap = [](uint4 &a, uint4 &b, bool up, int m) {
        // the lane keeps one of a, b and gets the other's counterpart from its partner
        uint4 t = up ? a : b;
        t.x = __shfl_xor_sync(kFull, t.x, m);
        t.y = __shfl_xor_sync(kFull, t.y, m);
        t.z = __shfl_xor_sync(kFull, t.z, m);
        t.w = __shfl_xor_sync(kFull, t.w, m);
        if (up)
            a = t;
        else
            b = t;
    };
    swap(v[0], v[1], odd, 1);
    swap(v[2], v[3], odd, 1);
    swap(v[0], v[2], high, 2);
    swap(v[1], v[3], high, 2);
    // v[k]: piece lane & 3 of row (lane & ~3) + k
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int r = (lane & ~3) + k;
        if (r < n)
            *reinterpret_cast<uint4 *>(dst + r * stride + (lane & 3) * 8) = v[k];
    }
}

// delta[h][f] = sum_d dout_fhd out_fhd of every frame, into the workspace.
int launch_attn_delta(const void *out, const void *dout, float *delta, int64_t total, int heads, const DeviceInfo &di,
                      cudaStream_t st);

// The gradient of block attention, whole blocks at a time
// (block_bwd_sm100a.cu): delta and the gradient, launched once all of its own
// checks have passed; items: an upper bound of the (block, head) pairs.
struct BlockBwdArgs {
    const void *q, *k, *v, *out, *dout;
    const float *lse;
    float *delta;
    void *dq, *dk, *dv;
    const int32_t *cu;
    int32_t *status;
    int64_t total, stride, dstride;
    int n_seq, heads, block;
    float scale, scale_log2;
    unsigned long long wait_ns;
    int flags;
};
int launch_block_bwd(const BlockBwdArgs &a, const DeviceInfo &di, int dev, long long items, cudaStream_t st);

} // namespace nle
