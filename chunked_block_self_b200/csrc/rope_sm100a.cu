// rope_sm100a.cu -- per-head RMS norm of queries and keys with the rotary
// position rotation in one pass, and its gradient, on B200 (sm_100a).
//
// For every frame f and head, x = one row of 64 values:
//     z = w * x * r,  r = 1 / sqrt(mean(x^2) + eps)      (z = x without norm)
//     (y_a, y_b) = c * (z_a cos t - z_b sin t, z_b cos t + z_a sin t)
// for each rotated pair (a, b) = (j, j + R/2) or, interleaved, (2j, 2j + 1),
// t = pos(f) * inv_freq[j], c = rot_scale; elements past R = rot_dim pass
// through.  Gradient, with dz the same rotation of dy by -t (times c):
//     g = w * dz,   dx = r * (g - n * mean(g * n)),  n = x * r,
//     dw = sum over frames and heads of dz * n.
//
// Both directions move each byte once and are HBM-bound.  A warp takes one
// frame at a time: lane = (head group 0..3, 16-byte chunk 0..7), so a warp
// load covers four 128-byte head rows and every sum over a row is three
// shuffles.  The frame's angles are formed once per warp, one pair per lane,
// and shared by all its heads through shuffles; the frequency is kept in
// fp64 as turns per position, so a position of 10^8 still gives an angle
// exact to fp32.  All arithmetic on values is fp32 with one rounding to bf16
// at the store.  A row is read completely (its chunks meet in shuffles)
// before any of it is written, so the output may be the input.
//
// The weight gradient is summed in fp32 per lane over the frames of a
// persistent CTA, then over the CTA's warps, written as one partial row per
// CTA, and a second kernel adds the partial rows in their order in fp64:
// no atomics, the same bits every time on one device.
#include <cmath>

#include "nle.h"
#include "nle_device.cuh"
#include "nle_host.h"

namespace {

using namespace nle;

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kMaxPartials = NLE_ROPE_BWD_WORKSPACE_BYTES / (2 * 64 * (int)sizeof(float));

struct Rows {
    const uint8_t *src;   // dy in the backward pass
    const uint8_t *x;     // backward with norm: the rows that were normalised
    uint8_t *dst;
    long long src_stride, x_stride, dst_stride;   // bytes between frames
    const __nv_bfloat16 *w;
    int heads;
};

struct RParams {
    Rows q, k;
    const int32_t *cu;          // null: every frame, positions given
    const int32_t *positions;   // null: the frame's index inside its utterance
    int n_seq;
    int total;
    int unit;                   // frames per CTA unit
    const double *inv_freq;
    int rot_dim;
    float rot_scale;            // negative-angle (transposed) rotation: see back
    int back;
    float eps;
    float *partial;             // [gridDim.x][2][64] weight-gradient sums
    int32_t *status;
};

struct Chunk {
    float v[8];
};

__device__ __forceinline__ Chunk unpack(const uint4 &u)
{
    Chunk c;
    const uint32_t r[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        c.v[2 * i] = __uint_as_float(r[i] << 16);
        c.v[2 * i + 1] = __uint_as_float(r[i] & 0xffff0000u);
    }
    return c;
}

__device__ __forceinline__ uint4 pack(const Chunk &c)
{
    return make_uint4(pack_bf16x2(c.v[0], c.v[1]), pack_bf16x2(c.v[2], c.v[3]), pack_bf16x2(c.v[4], c.v[5]),
                      pack_bf16x2(c.v[6], c.v[7]));
}

__device__ __forceinline__ uint4 shfl4(const uint4 &u, int src)
{
    return make_uint4(__shfl_sync(kFull, u.x, src), __shfl_sync(kFull, u.y, src), __shfl_sync(kFull, u.z, src),
                      __shfl_sync(kFull, u.w, src));
}

// sum over the 8 lanes of a head row
__device__ __forceinline__ float row_sum(float s)
{
    s += __shfl_xor_sync(kFull, s, 1);
    s += __shfl_xor_sync(kFull, s, 2);
    s += __shfl_xor_sync(kFull, s, 4);
    return s;
}

// What a lane knows of the rotation of its chunk: for pair layout "half",
// element e is paired with element e of lane `partner`'s chunk; interleaved,
// with its neighbour.  cs/sn of the frame: half, one per element (sn signed
// for the element's side of the pair); interleaved, one per pair.
template <bool kInter>
struct Turn {
    float cs[kInter ? 4 : 8], sn[kInter ? 4 : 8];
};

struct LanePlan {
    int chunk, partner;
    bool rotated;     // the chunk lies within rot_dim
    int angle0;       // lane that holds the chunk's first angle
    float side;       // half layout: -1 for the first member of the pair, +1 for the second
    double turns;     // this lane's frequency in turns per position
};

template <bool kInter>
__device__ __forceinline__ LanePlan lane_plan(const RParams &p, int lane)
{
    LanePlan l;
    l.chunk = lane & 7;
    const int nrot = p.rot_dim >> 3;   // rotated chunks (even: rot_dim % 16 == 0)
    l.rotated = l.chunk < nrot;
    if (kInter) {
        l.partner = lane;
        l.angle0 = l.rotated ? 4 * l.chunk : 0;
        l.side = 1.f;
    } else {
        const int hc = nrot >> 1;
        const bool first = l.chunk < hc;
        l.partner = !l.rotated ? lane : first ? lane + hc : lane - hc;
        l.angle0 = !l.rotated ? 0 : 8 * (first ? l.chunk : l.chunk - hc);
        l.side = first ? -1.f : 1.f;
    }
    l.turns = lane < (p.rot_dim >> 1) ? p.inv_freq[lane] * 0.15915494309189533577 : 0.0;   // 1 / (2 pi)
    return l;
}

// The frame's angles: lane j forms pair j's, every lane collects its chunk's.
template <bool kInter>
__device__ __forceinline__ Turn<kInter> frame_turn(const RParams &p, const LanePlan &l, int pos)
{
    const double t = (double)pos * l.turns;
    const float half_turns = (float)(2.0 * (t - rint(t)));   // in [-1, 1]
    float s, c;
    sincospif(half_turns, &s, &c);
    c *= p.rot_scale;
    s *= p.back ? -p.rot_scale : p.rot_scale;
    Turn<kInter> u;
#pragma unroll
    for (int e = 0; e < (kInter ? 4 : 8); ++e) {
        u.cs[e] = __shfl_sync(kFull, c, l.angle0 + e);
        u.sn[e] = __shfl_sync(kFull, s, l.angle0 + e) * l.side;
    }
    return u;
}

// y = rotation of the chunk z; zp: the partner chunk (half layout)
template <bool kInter>
__device__ __forceinline__ Chunk rotate(const Chunk &z, const Chunk &zp, const Turn<kInter> &u, bool rotated)
{
    Chunk y;
    if (kInter) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float a = z.v[2 * i], b = z.v[2 * i + 1];
            y.v[2 * i] = rotated ? a * u.cs[i] - b * u.sn[i] : a;
            y.v[2 * i + 1] = rotated ? b * u.cs[i] + a * u.sn[i] : b;
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            y.v[e] = rotated ? z.v[e] * u.cs[e] + zp.v[e] * u.sn[e] : z.v[e];
    }
    return y;
}

constexpr int kBatch = 4;   // head rows per lane with their loads in flight together (16 heads of a frame)

// The forward pass of a frame as two factors per element: y_e = r (a_e x_e +
// b_e x_p), p the other member of the pair, r the row's 1 / rms (1 without
// norm).  The weights go into a and b once per frame and tensor, which halves
// the arithmetic per head: with it the batch-128 workload (16 + 16 heads,
// 59,062 frames) went from 128 to 113 us, and with both tensors' first loads
// issued together to 99 us, 4.9 TB/s, 0.76 of the measured copy rate.
struct Factors {
    float a[8], b[8];
};

template <bool kNorm, bool kInter>
__device__ __forceinline__ Factors factors(const Turn<kInter> &u, const uint4 &w, const uint4 &wp, bool rotated)
{
    Factors f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float c = u.cs[kInter ? e >> 1 : e], s = u.sn[kInter ? e >> 1 : e];
        f.a[e] = rotated ? c : 1.f;
        f.b[e] = !rotated ? 0.f : kInter && !(e & 1) ? -s : s;
    }
    if (kNorm) {
        const Chunk ww = unpack(w), pw = unpack(wp);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            f.a[e] *= ww.v[e];
            if (!kInter)   // an unrotated chunk is its own partner
                f.b[e] *= pw.v[e];
            else if (rotated)
                f.b[e] *= ww.v[e ^ 1];
        }
    }
    return f;
}

// The rows of a batch of a frame's heads (zeros past the last head).
__device__ __forceinline__ void load_batch(const Rows &r, long long f, const LanePlan &l, int h0, int lane,
                                           uint4 (&in)[kBatch])
{
    const uint8_t *src = r.src + f * r.src_stride + l.chunk * 16;
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
        const int h = h0 + 4 * b + (lane >> 3);
        in[b] = h < r.heads ? *reinterpret_cast<const uint4 *>(src + (long long)h * 128) : make_uint4(0, 0, 0, 0);
    }
}

// All heads of one tensor and frame: y = rotate(norm(x)).  in: the first batch.
template <bool kNorm, bool kInter>
__device__ __forceinline__ void forward_heads(const Rows &r, long long f, const LanePlan &l, const Factors &u, float eps,
                                              int lane, uint4 (&in)[kBatch])
{
    const int hg = lane >> 3;
    uint8_t *dst = r.dst + f * r.dst_stride + l.chunk * 16;
    for (int h0 = 0; h0 < r.heads; h0 += 4 * kBatch) {
        if (h0 > 0)
            load_batch(r, f, l, h0, lane, in);
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            if (h0 + 4 * b >= r.heads)
                break;   // warp-uniform
            const int h = h0 + 4 * b + hg;
            const Chunk x = unpack(in[b]);
            const Chunk xp = kInter ? x : unpack(shfl4(in[b], l.partner));
            float rr = 1.f;
            if (kNorm) {
                float ss = 0.f;
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    ss = fmaf(x.v[e], x.v[e], ss);
                rr = rsqrtf(row_sum(ss) * (1.f / 64.f) + eps);
            }
            Chunk y;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                // unrotated elements take nothing of their neighbour: 0 * Inf is NaN
                const float xo = !kInter ? xp.v[e] : !kNorm || l.rotated ? x.v[e ^ 1] : 0.f;
                y.v[e] = fmaf(u.b[e], xo, u.a[e] * x.v[e]);
                if (kNorm)
                    y.v[e] *= rr;
            }
            if (h < r.heads)   // untouched elements keep their bits (a NaN's too)
                *reinterpret_cast<uint4 *>(dst + (long long)h * 128) = kNorm || l.rotated ? pack(y) : in[b];
        }
    }
}

// The next unit of frames: [f0, f0 + n) of the utterance that starts at `start`.
__device__ __forceinline__ bool unit_at(const RParams &p, PlanWalker &w, long long u, int lane, int &f0, int &n,
                                        int &start)
{
    if (!p.cu) {
        if (u * p.unit >= p.total)
            return false;
        f0 = (int)(u * p.unit);
        n = min(p.unit, p.total - f0);
        start = 0;
        return true;
    }
    int seq;
    if (!w.find(u, lane, f0, n, seq))
        return false;
    start = __ldg(p.cu + seq);
    return true;
}

__device__ __forceinline__ uint4 load_w(const Rows &r, int chunk)
{
    return r.w ? __ldg(reinterpret_cast<const uint4 *>(r.w) + chunk) : make_uint4(0, 0, 0, 0);
}

// Keeps the compiler from unpacking the weights once for all frames (32
// registers instead of 16, and with them a CTA fewer per SM).
__device__ __forceinline__ void keep_packed(uint4 &a, uint4 &b, uint4 &c, uint4 &d)
{
    asm volatile("" : "+r"(a.x), "+r"(a.y), "+r"(a.z), "+r"(a.w), "+r"(b.x), "+r"(b.y), "+r"(b.z), "+r"(b.w));
    asm volatile("" : "+r"(c.x), "+r"(c.y), "+r"(c.z), "+r"(c.w), "+r"(d.x), "+r"(d.y), "+r"(d.z), "+r"(d.w));
}

// One CTA per unit of 8 or 32 frames, whose warps walk cu_seqlens from its start, 32
// utterances a step: four steps at most for 128 utterances, but the walks of all
// CTAs together grow with the square of the utterances (16 + 16 heads, 59,000
// frames in 128 utterances 102 us, in 1,000 158, 60,000 in 4,000 617; the
// gradient, whose CTAs are persistent and walk once, 150, 166 and 197).
template <bool kNorm, bool kInter>
__global__ void __launch_bounds__(kThreads) qk_rope_kernel(const RParams p)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    PlanWalker w;
    if (p.cu)
        w.init(p.cu, p.n_seq, p.total, p.unit, lane);
    int f0, n, start;
    const bool have = unit_at(p, w, blockIdx.x, lane, f0, n, start);
    if (p.cu && w.bad && threadIdx.x == 0)
        report(p.status, NLE_ERR_INVALID_ARG);
    if (!have)
        return;
    const LanePlan l = lane_plan<kInter>(p, lane);
    uint4 wq = load_w(p.q, l.chunk), wk = load_w(p.k, l.chunk);
    uint4 wqp = shfl4(wq, l.partner), wkp = shfl4(wk, l.partner);
    for (int i = warp; i < n; i += kWarps) {
        const long long f = f0 + i;
        const int pos = p.positions ? __ldg(p.positions + f) : (int)f - start;
        // both tensors' first heads are on their way while the angles are formed
        uint4 q0[kBatch], k0[kBatch];
        load_batch(p.q, f, l, 0, lane, q0);
        load_batch(p.k, f, l, 0, lane, k0);
        const Turn<kInter> u = frame_turn<kInter>(p, l, pos);
        keep_packed(wq, wqp, wk, wkp);
        forward_heads<kNorm, kInter>(p.q, f, l, factors<kNorm, kInter>(u, wq, wqp, l.rotated), p.eps, lane, q0);
        forward_heads<kNorm, kInter>(p.k, f, l, factors<kNorm, kInter>(u, wk, wkp, l.rotated), p.eps, lane, k0);
    }
}

constexpr int kBwdBatch = 4;
constexpr int kBwdCtas = 2;   // persistent CTAs per SM

// All heads of one tensor and frame: dx, and this lane's share of dw.
template <bool kInter>
__device__ __forceinline__ void backward_heads(const Rows &r, long long f, const LanePlan &l, const Turn<kInter> &u,
                                               const uint4 &w, float eps, int lane, float (&dw)[8])
{
    const int hg = lane >> 3;
    const uint8_t *src = r.src + f * r.src_stride + l.chunk * 16;
    const uint8_t *xs = r.x + f * r.x_stride + l.chunk * 16;
    uint8_t *dst = r.dst + f * r.dst_stride + l.chunk * 16;
    const Chunk ww = unpack(w);
    for (int h0 = 0; h0 < r.heads; h0 += 4 * kBwdBatch) {
        uint4 dy[kBwdBatch], xx[kBwdBatch];
#pragma unroll
        for (int b = 0; b < kBwdBatch; ++b) {
            const int h = h0 + 4 * b + hg;
            const bool in = h < r.heads;
            // past the last head dy = 0 and x = 1: r is finite whatever eps
            // (0 * r of a zero row with eps = 0 would be NaN), dw gets 0
            dy[b] = in ? *reinterpret_cast<const uint4 *>(src + (long long)h * 128) : make_uint4(0, 0, 0, 0);
            xx[b] = in ? *reinterpret_cast<const uint4 *>(xs + (long long)h * 128)
                       : make_uint4(0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u);
        }
#pragma unroll
        for (int b = 0; b < kBwdBatch; ++b) {
            if (h0 + 4 * b >= r.heads)
                break;   // warp-uniform
            const int h = h0 + 4 * b + hg;
            const Chunk d = unpack(dy[b]);
            Chunk dp = d;
            if (!kInter)
                dp = unpack(shfl4(dy[b], l.partner));
            const Chunk dz = rotate<kInter>(d, dp, u, l.rotated);
            const Chunk x = unpack(xx[b]);
            float ss = 0.f, gx = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                ss = fmaf(x.v[e], x.v[e], ss);
                gx = fmaf(dz.v[e] * ww.v[e], x.v[e], gx);
            }
            const float rr = rsqrtf(row_sum(ss) * (1.f / 64.f) + eps);
            // mean(g * n) * r, n = x * r
            const float m = row_sum(gx) * (1.f / 64.f) * rr * rr;
            Chunk dx;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                dx.v[e] = rr * (dz.v[e] * ww.v[e] - x.v[e] * m);
                dw[e] = fmaf(dz.v[e], x.v[e] * rr, dw[e]);
            }
            if (h < r.heads)
                *reinterpret_cast<uint4 *>(dst + (long long)h * 128) = pack(dx);
        }
    }
}

// The gradient with weights: two persistent CTAs per SM (128 registers: the
// sums of dw and four heads' dy and x in flight), 6 bytes per element.  Batch of
// 128 utterances (16 + 16 heads, 59,062 frames): 141 us and 6.5 us for the
// partial rows' sum, 4.9 TB/s together, 0.76 of the measured copy rate.
template <bool kInter>
__global__ void __launch_bounds__(kThreads, kBwdCtas) qk_norm_rope_bwd_kernel(const RParams p)
{
    __shared__ float sums[kWarps][2][64];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    PlanWalker w;
    if (p.cu)
        w.init(p.cu, p.n_seq, p.total, p.unit, lane);
    const LanePlan l = lane_plan<kInter>(p, lane);
    const uint4 wq = load_w(p.q, l.chunk), wk = load_w(p.k, l.chunk);
    float dwq[8] = {}, dwk[8] = {};
    for (long long un = blockIdx.x;; un += gridDim.x) {
        int f0, n, start;
        if (!unit_at(p, w, un, lane, f0, n, start))
            break;
        for (int i = warp; i < n; i += kWarps) {
            const long long f = f0 + i;
            const int pos = p.positions ? __ldg(p.positions + f) : (int)f - start;
            const Turn<kInter> u = frame_turn<kInter>(p, l, pos);
            backward_heads<kInter>(p.q, f, l, u, wq, p.eps, lane, dwq);
            backward_heads<kInter>(p.k, f, l, u, wk, p.eps, lane, dwk);
        }
    }
    if (p.cu && w.bad && threadIdx.x == 0)
        report(p.status, NLE_ERR_INVALID_ARG);
    // lanes of the same chunk, then the CTA's warps, in a fixed order
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        dwq[e] += __shfl_xor_sync(kFull, dwq[e], 8);
        dwq[e] += __shfl_xor_sync(kFull, dwq[e], 16);
        dwk[e] += __shfl_xor_sync(kFull, dwk[e], 8);
        dwk[e] += __shfl_xor_sync(kFull, dwk[e], 16);
        if (lane < 8) {
            sums[warp][0][lane * 8 + e] = dwq[e];
            sums[warp][1][lane * 8 + e] = dwk[e];
        }
    }
    __syncthreads();
    if (threadIdx.x < 128) {
        float s = 0.f;
        for (int i = 0; i < kWarps; ++i)
            s += sums[i][threadIdx.x >> 6][threadIdx.x & 63];
        p.partial[(size_t)blockIdx.x * 128 + threadIdx.x] = s;
    }
}

// dw = the CTAs' partial rows added in a fixed order (fp64)
__global__ void __launch_bounds__(1024) dw_reduce_kernel(const float *partial, int n, float *dw_q, float *dw_k)
{
    __shared__ double part[16][64];
    const int col = threadIdx.x & 63, row = threadIdx.x >> 6;
    double s = 0.0;
#pragma unroll 4
    for (int i = row; i < n; i += 16)
        s += (double)partial[(size_t)i * 128 + blockIdx.x * 64 + col];
    part[row][col] = s;
    __syncthreads();
    float *dw = blockIdx.x ? dw_k : dw_q;
    if (row == 0 && dw) {
        for (int i = 1; i < 16; ++i)
            s += part[i][col];
        dw[col] = (float)s;
    }
}

// One tensor's pointers and strides (elements); dense rows when stride is 0.
int check_rows(const void *ptr, int64_t *stride, int heads)
{
    const int64_t dense = (int64_t)heads * 64;
    if (*stride == 0)
        *stride = dense;
    if (!ptr || *stride < dense || *stride > (1ll << 40))
        return NLE_ERR_INVALID_ARG;
    if (*stride % 8 != 0 || !nle::aligned16(ptr))
        return NLE_ERR_MISALIGNED;
    return NLE_OK;
}

// A buffer of a call.  tensor: 0 (q), 1 (k): the sources and the output of
// one tensor, which may be one buffer (at one stride); -1: of its own.
struct Buffer {
    const void *p;
    int tensor;
    bool written;
};

// Does anything written begin where another buffer does?
template <int n>
bool written_twice(const Buffer (&b)[n])
{
    for (int i = 0; i < n; ++i)
        for (int j = 0; j < i; ++j) {
            const bool own = b[i].tensor >= 0 && b[i].tensor == b[j].tensor && b[i].written != b[j].written;
            if (b[i].p && b[i].p == b[j].p && (b[i].written || b[j].written) && !own)
                return true;
        }
    return false;
}

// Shared checks of the two entry points; *work: there is something to do.
int check_plan(const nle_rope_plan *r, bool *work)
{
    *work = false;
    if (!r || r->n_seq < 0 || r->total_frames < 0 || r->q_heads < 0 || r->k_heads < 0 ||
        r->q_heads + (long long)r->k_heads < 1 || r->rot_dim < 0 || !(r->eps >= 0.f) ||
        (r->interleaved != 0 && r->interleaved != 1))
        return NLE_ERR_INVALID_ARG;
    if (r->d_head != 64 || r->rot_dim > 64 || r->rot_dim % 16 != 0 || r->total_frames > 0x7fffffffLL ||
        r->q_heads > (1 << 20) || r->k_heads > (1 << 20))
        return NLE_ERR_UNSUPPORTED;
    // both tensors are normalised, or neither
    if ((r->q_weight == nullptr) != (r->k_weight == nullptr) && r->q_heads > 0 && r->k_heads > 0)
        return NLE_ERR_INVALID_ARG;
    if (r->total_frames == 0 || (r->cu_seqlens && r->n_seq == 0))
        return NLE_OK;
    if ((r->rot_dim > 0 && !r->inv_freq) || (!r->cu_seqlens && !r->positions))
        return NLE_ERR_INVALID_ARG;
    if ((r->q_weight && !nle::aligned16(r->q_weight)) || (r->k_weight && !nle::aligned16(r->k_weight)))
        return NLE_ERR_MISALIGNED;
    if (!nle::aligned4(r->cu_seqlens) || !nle::aligned4(r->positions) || !nle::aligned4(r->dev_status) ||
        (r->rot_dim > 0 && (reinterpret_cast<uintptr_t>(r->inv_freq) & 7)))
        return NLE_ERR_MISALIGNED;
    *work = true;
    return NLE_OK;
}

int fill_params(const nle_rope_plan *r, RParams *p, nle::DeviceInfo *di)
{
    int dev = 0;
    if (!nle::current_device_info(di, &dev))
        return NLE_ERR_CUDA;
    if (di->cc_major != 10)
        return NLE_ERR_UNSUPPORTED;
    p->cu = r->cu_seqlens;
    p->positions = r->positions;
    p->n_seq = r->n_seq;
    p->total = (int)r->total_frames;
    p->inv_freq = r->inv_freq;
    p->rot_dim = r->rot_dim;
    p->rot_scale = r->rot_scale == 0.f ? 1.f : r->rot_scale;
    p->eps = r->eps;
    p->status = r->dev_status;
    return NLE_OK;
}

long long units_bound(const RParams &p)
{
    return (p.cu ? (long long)p.n_seq : 1) + p.total / p.unit;
}

// The rotation (and norm) of both tensors, one CTA per unit.
int launch_rope(RParams &p, bool norm, bool inter, const nle::DeviceInfo &di, void *stream)
{
    // a frame per warp until the batch fills the GPU eight CTAs deep, then
    // four frames per warp (the plan walk and angle set-up amortised)
    p.unit = p.total <= 8 * kWarps * di.sm_count ? kWarps : 4 * kWarps;
    const long long grid = units_bound(p);
    if (grid > 0x7fffffffLL)
        return NLE_ERR_UNSUPPORTED;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (norm)
        inter ? qk_rope_kernel<true, true><<<(unsigned)grid, kThreads, 0, st>>>(p)
              : qk_rope_kernel<true, false><<<(unsigned)grid, kThreads, 0, st>>>(p);
    else
        inter ? qk_rope_kernel<false, true><<<(unsigned)grid, kThreads, 0, st>>>(p)
              : qk_rope_kernel<false, false><<<(unsigned)grid, kThreads, 0, st>>>(p);
    return cudaGetLastError() == cudaSuccess ? NLE_OK : NLE_ERR_CUDA;
}

} // namespace

extern "C" int nle_qk_norm_rope_fwd(const nle_rope_plan *plan, const void *q, int64_t q_stride, const void *k,
                                    int64_t k_stride, void *q_out, int64_t q_out_stride, void *k_out,
                                    int64_t k_out_stride, void *stream)
{
    bool work;
    int rc = check_plan(plan, &work);
    if (rc != NLE_OK || !work)
        return rc;
    const bool norm = plan->q_weight || plan->k_weight;
    struct {
        const void *src;
        int64_t ss;
        void *dst;
        int64_t ds;
        int heads;
        const void *w;
    } t[2] = {{q, q_stride, q_out, q_out_stride, plan->q_heads, plan->q_weight},
              {k, k_stride, k_out, k_out_stride, plan->k_heads, plan->k_weight}};
    RParams p{};
    for (int i = 0; i < 2; ++i) {
        if (t[i].heads == 0)
            continue;
        if (norm && !t[i].w)
            return NLE_ERR_INVALID_ARG;
        if ((rc = check_rows(t[i].src, &t[i].ss, t[i].heads)) != NLE_OK ||
            (rc = check_rows(t[i].dst, &t[i].ds, t[i].heads)) != NLE_OK)
            return rc;
        if (t[i].src == t[i].dst && t[i].ss != t[i].ds)   // in place: the same frames
            return NLE_ERR_INVALID_ARG;
        Rows &r = i ? p.k : p.q;
        r.src = static_cast<const uint8_t *>(t[i].src);
        r.dst = static_cast<uint8_t *>(t[i].dst);
        r.src_stride = t[i].ss * 2;
        r.dst_stride = t[i].ds * 2;
        r.heads = t[i].heads;
        r.w = static_cast<const __nv_bfloat16 *>(t[i].w);
    }
    if (written_twice<10>({{p.q.src, 0, false}, {p.k.src, 1, false}, {p.q.dst, 0, true}, {p.k.dst, 1, true},
                           {plan->q_weight, -1, false}, {plan->k_weight, -1, false}, {plan->inv_freq, -1, false},
                           {plan->cu_seqlens, -1, false}, {plan->positions, -1, false}, {plan->dev_status, -1, false}}))
        return NLE_ERR_INVALID_ARG;
    nle::DeviceInfo di;
    if ((rc = fill_params(plan, &p, &di)) != NLE_OK)
        return rc;
    return launch_rope(p, norm, plan->interleaved != 0, di, stream);
}

extern "C" int nle_qk_norm_rope_bwd(const nle_rope_plan *plan, const void *dq_out, int64_t dq_out_stride,
                                    const void *dk_out, int64_t dk_out_stride, const void *q, int64_t q_stride,
                                    const void *k, int64_t k_stride, void *dq, int64_t dq_stride, void *dk,
                                    int64_t dk_stride, float *dq_weight, float *dk_weight, void *workspace,
                                    void *stream)
{
    bool work;
    int rc = check_plan(plan, &work);
    if (rc != NLE_OK)
        return rc;
    const bool norm = plan->q_weight || plan->k_weight;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (!work) {
        // no frames: the weight gradients are empty sums
        for (float *dw : {dq_weight, dk_weight})
            if (norm && dw && cudaMemsetAsync(dw, 0, 64 * sizeof(float), st) != cudaSuccess)
                return NLE_ERR_CUDA;
        return NLE_OK;
    }
    struct {
        const void *src;
        int64_t ss;
        const void *x;
        int64_t xs;
        void *dst;
        int64_t ds;
        int heads;
        const void *w;
    } t[2] = {{dq_out, dq_out_stride, q, q_stride, dq, dq_stride, plan->q_heads, plan->q_weight},
              {dk_out, dk_out_stride, k, k_stride, dk, dk_stride, plan->k_heads, plan->k_weight}};
    RParams p{};
    for (int i = 0; i < 2; ++i) {
        if (t[i].heads == 0)
            continue;
        if (norm && !t[i].w)
            return NLE_ERR_INVALID_ARG;
        if ((rc = check_rows(t[i].src, &t[i].ss, t[i].heads)) != NLE_OK ||
            (norm && (rc = check_rows(t[i].x, &t[i].xs, t[i].heads)) != NLE_OK) ||
            (rc = check_rows(t[i].dst, &t[i].ds, t[i].heads)) != NLE_OK)
            return rc;
        if ((t[i].src == t[i].dst && t[i].ss != t[i].ds) ||   // in place: the same frames
            (norm && t[i].x == t[i].dst && t[i].xs != t[i].ds))
            return NLE_ERR_INVALID_ARG;
        Rows &r = i ? p.k : p.q;
        r.src = static_cast<const uint8_t *>(t[i].src);
        r.x = static_cast<const uint8_t *>(t[i].x);
        r.dst = static_cast<uint8_t *>(t[i].dst);
        r.src_stride = t[i].ss * 2;
        r.x_stride = t[i].xs * 2;
        r.dst_stride = t[i].ds * 2;
        r.heads = t[i].heads;
        r.w = static_cast<const __nv_bfloat16 *>(t[i].w);
    }
    if (norm && !workspace)
        return NLE_ERR_INVALID_ARG;
    if (norm && (!nle::aligned16(workspace) || !nle::aligned4(dq_weight) || !nle::aligned4(dk_weight)))
        return NLE_ERR_MISALIGNED;
    if (written_twice<15>({{p.q.src, 0, false}, {p.k.src, 1, false}, {norm ? p.q.x : nullptr, 0, false},
                           {norm ? p.k.x : nullptr, 1, false}, {p.q.dst, 0, true}, {p.k.dst, 1, true},
                           {norm ? dq_weight : nullptr, -1, true}, {norm ? dk_weight : nullptr, -1, true},
                           {norm ? workspace : nullptr, -1, true}, {plan->q_weight, -1, false},
                           {plan->k_weight, -1, false}, {plan->inv_freq, -1, false}, {plan->cu_seqlens, -1, false},
                           {plan->positions, -1, false}, {plan->dev_status, -1, false}}))
        return NLE_ERR_INVALID_ARG;
    nle::DeviceInfo di;
    if ((rc = fill_params(plan, &p, &di)) != NLE_OK)
        return rc;
    p.back = 1;
    if (!norm)   // the transposed rotation alone
        return launch_rope(p, false, plan->interleaved != 0, di, stream);
    p.partial = static_cast<float *>(workspace);
    p.unit = kWarps;
    long long grid = units_bound(p);
    if (grid > (long long)kBwdCtas * di.sm_count)
        grid = (long long)kBwdCtas * di.sm_count;
    if (grid > kMaxPartials)
        grid = kMaxPartials;
    if (plan->interleaved)
        qk_norm_rope_bwd_kernel<true><<<(unsigned)grid, kThreads, 0, st>>>(p);
    else
        qk_norm_rope_bwd_kernel<false><<<(unsigned)grid, kThreads, 0, st>>>(p);
    if (cudaGetLastError() != cudaSuccess)
        return NLE_ERR_CUDA;
    dw_reduce_kernel<<<2, 1024, 0, st>>>(p.partial, (int)grid, dq_weight, dk_weight);
    return cudaGetLastError() == cudaSuccess ? NLE_OK : NLE_ERR_CUDA;
}
