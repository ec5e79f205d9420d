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

// 32 columns of an accumulator row, times f, to bf16 at dst.
__device__ __forceinline__ void store_acc(uint32_t tacc, float f, __nv_bfloat16 *dst, bool row_ok)
{
    uint32_t o[32];
    tmem_ld32_nowait(tacc, o);
    tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < 32; ++i)
        reg_fence(o[i]);
    if (row_ok) {
#pragma unroll
        for (int i = 0; i < 32; i += 8)
            *reinterpret_cast<uint4 *>(dst + i) =
                make_uint4(pack_bf16x2(__uint_as_float(o[i]) * f, __uint_as_float(o[i + 1]) * f),
                           pack_bf16x2(__uint_as_float(o[i + 2]) * f, __uint_as_float(o[i + 3]) * f),
                           pack_bf16x2(__uint_as_float(o[i + 4]) * f, __uint_as_float(o[i + 5]) * f),
                           pack_bf16x2(__uint_as_float(o[i + 6]) * f, __uint_as_float(o[i + 7]) * f));
    }
}

// The gradient of block attention, whole blocks at a time
// (block_bwd_sm100a.cu), after delta has been computed; items: an upper bound
// of the (block, head) pairs.
struct BlockBwdArgs {
    const void *q, *k, *v, *dout;
    const float *lse, *delta;
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
