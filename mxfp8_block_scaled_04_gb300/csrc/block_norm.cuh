// The norms around a block fused with its gate and residual scale, and their gradients; formulas in include/block_norm.h.
//
// A CTA takes a row at a time and a thread V vectors of 8 columns of it, so that every input is read once and each
// output written once, with the row's sums (of y^2, then of h'^2; backward: y^2, h'^2 and dx w h' together, then b n1) formed
// between.  The next row is loaded before this one is worked on.  Bound by HBM for many rows, by the
// chain of loads, two reductions and stores (launch included) for few.
//
// The weights' gradients are sums over the rows: a CTA keeps its own in shared memory (each thread its columns), writes them
// to the workspace at its end, and a second kernel adds the CTAs' in order.
#pragma once

#include <cstdint>

#include "ptx.cuh"

namespace mxfp8 {

constexpr int kNormCtas = 2 * 152;  // CTAs whose partial sums the workspace holds

struct NormParams {
    const void *y, *h;                 // backward: h is the stream behind the block
    const void *dh_out, *dx;
    int64_t T, ldy, ldh, lddh, lddx;
    int H, vecs;
    int gate_kind;
    float scale, eps;
    const float *pre, *post, *gate;
    void *h_out, *x;
    void *dh, *dy;
    float *dpre, *dpost, *dgate, *partial;
};

// Eight elements of a row as they are stored.
template <bool F32>
struct Row8 {
    uint4 lo, hi;  // BF16: lo alone
};
template <>
struct Row8<false> {
    uint4 lo;
};

__device__ __forceinline__ uint4 load_stream(const void *p)
{
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}

template <bool F32>
__device__ __forceinline__ Row8<F32> load_row8(const void *base, int64_t at)
{
    Row8<F32> r;
    const unsigned char *p = static_cast<const unsigned char *>(base) + at * (F32 ? 4 : 2);
    r.lo = load_stream(p);
    if constexpr (F32)
        r.hi = load_stream(p + 16);
    return r;
}
template <bool F32>
__device__ __forceinline__ void widen8(const Row8<F32> &r, float (&v)[8])
{
    if constexpr (F32) {
        const uint32_t w[8] = {r.lo.x, r.lo.y, r.lo.z, r.lo.w, r.hi.x, r.hi.y, r.hi.z, r.hi.w};
#pragma unroll
        for (int k = 0; k < 8; ++k)
            v[k] = __uint_as_float(w[k]);
    } else {
        const uint32_t w[4] = {r.lo.x, r.lo.y, r.lo.z, r.lo.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            v[2 * k] = bf16_lo(w[k]);
            v[2 * k + 1] = bf16_hi(w[k]);
        }
    }
}
__device__ __forceinline__ uint32_t round_bf16x2(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// Store eight elements; v becomes what was stored.
template <bool F32>
__device__ __forceinline__ void store8(void *base, int64_t at, float (&v)[8], bool write = true)
{
    unsigned char *p = static_cast<unsigned char *>(base) + at * (F32 ? 4 : 2);
    if constexpr (F32) {
        if (write) {
            *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
            *reinterpret_cast<float4 *>(p + 16) = make_float4(v[4], v[5], v[6], v[7]);
        }
    } else {
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            w[k] = round_bf16x2(v[2 * k], v[2 * k + 1]);
            v[2 * k] = bf16_lo(w[k]);
            v[2 * k + 1] = bf16_hi(w[k]);
        }
        if (write)
            *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}
// Eight values of a weight (kept in L1: every row reads them).
__device__ __forceinline__ void weight8(const float *w, int at, float (&v)[8])
{
    const float4 a = __ldg(reinterpret_cast<const float4 *>(w + at)), b = __ldg(reinterpret_cast<const float4 *>(w + at + 4));
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}

// Sums of N values over the CTA, the same in every thread; one barrier.  `turn` alternates between two buffers, so that a
// buffer is written again only after a barrier that follows its last reads.
template <int N>
__device__ __forceinline__ void row_sums(float (&s)[N], float (*buffer)[4][32], int &turn, int lane, int warp, int warps)
{
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
#pragma unroll
        for (int n = 0; n < N; ++n)
            s[n] += __shfl_xor_sync(0xFFFFFFFFu, s[n], d);
    if (lane == 0) {
#pragma unroll
        for (int n = 0; n < N; ++n)
            buffer[turn][n][warp] = s[n];
    }
    __syncthreads();
#pragma unroll
    for (int n = 0; n < N; ++n)
        s[n] = lane < warps ? buffer[turn][n][lane] : 0.f;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
#pragma unroll
        for (int n = 0; n < N; ++n)
            s[n] += __shfl_xor_sync(0xFFFFFFFFu, s[n], d);
    turn ^= 1;
}

template <int V>
constexpr int kNormThreads = V == 1 ? 1024 : 512;

template <bool YF32, bool HF32, int V>
__global__ void __launch_bounds__(kNormThreads<V>) block_norm_kernel(const NormParams p)
{
    __shared__ float buffer[2][4][32];
    pdl_wait_and_release();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nt = blockDim.x, warps = nt >> 5;
    int turn = 0;
    Row8<YF32> yr[V];
    Row8<HF32> hr[V];
    auto load = [&](int64_t row) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int j = tid + i * nt;
            yr[i] = Row8<YF32>{};
            hr[i] = Row8<HF32>{};
            if (j < p.vecs && row < p.T) {
                if (p.y != nullptr)
                    yr[i] = load_row8<YF32>(p.y, row * p.ldy + 8 * j);
                hr[i] = load_row8<HF32>(p.h, row * p.ldh + 8 * j);
            }
        }
    };
    load(blockIdx.x);
    const float inv = 1.0f / static_cast<float>(p.H);
    for (int64_t row = blockIdx.x; row < p.T; row += gridDim.x) {
        float a[V][8];
        float s[1] = {0.f};
#pragma unroll
        for (int i = 0; i < V; ++i) {
            widen8<YF32>(yr[i], a[i]);
#pragma unroll
            for (int k = 0; k < 8; ++k)
                s[0] = fmaf(a[i][k], a[i][k], s[0]);
        }
        float factor = p.gate_kind == 2 ? __ldg(p.gate + row) : 1.0f;
        if (p.post != nullptr) {
            row_sums<1>(s, buffer, turn, lane, warp, warps);
            factor *= rsqrtf(s[0] * inv + p.eps);
        }
        s[0] = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int j = tid + i * nt;
            float h[8];
            widen8<HF32>(hr[i], h);
            if (j < p.vecs) {
                float w[8];
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    a[i][k] *= factor;
                if (p.post != nullptr) {
                    weight8(p.post, 8 * j, w);
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        a[i][k] *= w[k];
                }
                if (p.gate_kind == 1) {
                    weight8(p.gate, 8 * j, w);
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        a[i][k] *= w[k];
                }
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    a[i][k] = fmaf(p.scale, h[k], a[i][k]);
                store8<HF32>(p.h_out, row * p.H + 8 * j, a[i], p.h_out != nullptr);
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    s[0] = fmaf(a[i][k], a[i][k], s[0]);
            }
        }
        load(row + gridDim.x);
        if (p.pre != nullptr) {
            row_sums<1>(s, buffer, turn, lane, warp, warps);
            const float r = rsqrtf(s[0] * inv + p.eps);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int j = tid + i * nt;
                if (j < p.vecs) {
                    float w[8];
                    weight8(p.pre, 8 * j, w);
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        a[i][k] = a[i][k] * r * w[k];
                    store8<false>(p.x, row * p.H + 8 * j, a[i]);
                }
            }
        }
    }
}

// acc[0 .. 7] += v, in shared memory that this thread alone uses.
__device__ __forceinline__ void add8(float *acc, const float (&v)[8])
{
    float4 *q = reinterpret_cast<float4 *>(acc);
    float4 a = q[0], b = q[1];
    a.x += v[0], a.y += v[1], a.z += v[2], a.w += v[3], b.x += v[4], b.y += v[5], b.z += v[6], b.w += v[7];
    q[0] = a;
    q[1] = b;
}

template <bool YF32, bool HF32, int V>
__global__ void __launch_bounds__(kNormThreads<V>) block_norm_backward_kernel(const NormParams p)
{
    extern __shared__ float4 norm_smem[];
    __shared__ float buffer[2][4][32];
    pdl_wait_and_release();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nt = blockDim.x, warps = nt >> 5;
    int turn = 0;
    // this CTA's sums, an array of H for each that is wanted
    float *sums = reinterpret_cast<float *>(norm_smem);
    const bool channel = p.gate_kind == 1;
    float *const acc_pre = p.dpre != nullptr ? sums : nullptr;
    float *const acc_post = p.dpost != nullptr ? sums + (p.dpre != nullptr ? p.H : 0) : nullptr;
    float *const acc_gate = p.dgate != nullptr && channel ? sums + ((p.dpre != nullptr) + (p.dpost != nullptr)) * p.H : nullptr;
    const int arrays = (acc_pre != nullptr) + (acc_post != nullptr) + (acc_gate != nullptr);
    for (int n = 0; n < arrays; ++n)
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int j = tid + i * nt;
            if (j < p.vecs) {
                norm_smem[n * 2 * p.vecs + 2 * j] = make_float4(0.f, 0.f, 0.f, 0.f);
                norm_smem[n * 2 * p.vecs + 2 * j + 1] = make_float4(0.f, 0.f, 0.f, 0.f);
            }
        }
    Row8<YF32> yr[V];
    Row8<HF32> hr[V], gr[V];
    Row8<false> xr[V];
    auto load = [&](int64_t row) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int j = tid + i * nt;
            yr[i] = Row8<YF32>{};
            hr[i] = gr[i] = Row8<HF32>{};
            xr[i] = Row8<false>{};
            if (j < p.vecs && row < p.T) {
                if (p.y != nullptr)
                    yr[i] = load_row8<YF32>(p.y, row * p.ldy + 8 * j);
                if (p.dx != nullptr) {
                    hr[i] = load_row8<HF32>(p.h, row * p.ldh + 8 * j);
                    xr[i] = load_row8<false>(p.dx, row * p.lddx + 8 * j);
                }
                if (p.dh_out != nullptr)
                    gr[i] = load_row8<HF32>(p.dh_out, row * p.lddh + 8 * j);
            }
        }
    };
    const float inv = 1.0f / static_cast<float>(p.H);
    const bool second = p.post != nullptr || (p.gate_kind == 2 && p.dgate != nullptr);
    for (int64_t row = blockIdx.x; row < p.T; row += gridDim.x) {
        load(row);
        float s[3] = {0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int j = tid + i * nt;
            float y[8], h[8], d[8], w[8];
            widen8<YF32>(yr[i], y);
            widen8<HF32>(hr[i], h);
            widen8<false>(xr[i], d);
            if (p.pre != nullptr && j < p.vecs)
                weight8(p.pre, 8 * j, w);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                s[0] = fmaf(y[k], y[k], s[0]);
                s[1] = fmaf(h[k], h[k], s[1]);
                if (p.pre != nullptr && j < p.vecs)
                    s[2] = fmaf(d[k] * w[k], h[k], s[2]);
            }
        }
        row_sums<3>(s, buffer, turn, lane, warp, warps);
        const float r1 = p.post != nullptr ? rsqrtf(s[0] * inv + p.eps) : 1.0f;
        const float r2 = rsqrtf(s[1] * inv + p.eps);
        const float c2 = r2 * s[2] * inv;  // mean(t n2)
        const float token = p.gate_kind == 2 ? __ldg(p.gate + row) : 1.0f;
        float g[V][8];
        float m[1] = {0.f};
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int j = tid + i * nt;
            widen8<HF32>(gr[i], g[i]);
            if (j < p.vecs) {
                float w[8], y[8];
                if (p.dx != nullptr) {
                    float h[8], d[8];
                    widen8<HF32>(hr[i], h);
                    widen8<false>(xr[i], d);
                    weight8(p.pre, 8 * j, w);
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const float n = h[k] * r2;
                        g[i][k] = fmaf(r2, fmaf(-n, c2, d[k] * w[k]), g[i][k]);
                        d[k] *= n;
                    }
                    if (acc_pre != nullptr)
                        add8(acc_pre + 8 * j, d);
                }
                if (p.dh != nullptr) {
                    float v[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        v[k] = p.scale * g[i][k];
                    store8<HF32>(p.dh, row * p.H + 8 * j, v);
                }
                widen8<YF32>(yr[i], y);
                float q[8];  // n1, times the weight's share below
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    q[k] = y[k] * r1;
                if (acc_gate != nullptr) {
                    float v[8];
                    if (p.post != nullptr)
                        weight8(p.post, 8 * j, w);
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        v[k] = g[i][k] * q[k] * (p.post != nullptr ? w[k] : 1.0f);
                    add8(acc_gate + 8 * j, v);
                }
                if (channel) {
                    weight8(p.gate, 8 * j, w);
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        g[i][k] *= w[k];
                }
                if (acc_post != nullptr) {
                    float v[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        v[k] = token * g[i][k] * q[k];
                    add8(acc_post + 8 * j, v);
                }
                if (p.post != nullptr) {
                    weight8(p.post, 8 * j, w);
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        g[i][k] *= w[k];
                }
                if (second) {
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        m[0] = fmaf(g[i][k], q[k], m[0]);
                }
            }
        }
        if (second)
            row_sums<1>(m, buffer, turn, lane, warp, warps);
        if (p.gate_kind == 2 && p.dgate != nullptr && tid == 0)
            p.dgate[row] = m[0];
        if (p.dy != nullptr) {
            const float c1 = p.post != nullptr ? r1 * m[0] * inv : 0.f;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int j = tid + i * nt;
                if (j < p.vecs) {
                    float y[8];
                    widen8<YF32>(yr[i], y);
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        y[k] = token * r1 * fmaf(-y[k], c1, g[i][k]);
                    store8<YF32>(p.dy, row * p.H + 8 * j, y);
                }
            }
        }
    }
    for (int n = 0; n < arrays; ++n)
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int j = tid + i * nt;
            if (j < p.vecs) {
                float4 *to = reinterpret_cast<float4 *>(p.partial + (static_cast<int64_t>(blockIdx.x) * arrays + n) * p.H + 8 * j);
                to[0] = norm_smem[n * 2 * p.vecs + 2 * j];
                to[1] = norm_smem[n * 2 * p.vecs + 2 * j + 1];
            }
        }
}

// The CTAs' sums, in order: a warp takes 32 columns of an array's rows w, w + 8, ...; the eight warps' are added in order.
constexpr int kNormReduceThreads = 256;
__global__ void __launch_bounds__(kNormReduceThreads) block_norm_reduce_kernel(const float *partial, int ctas, int arrays, int H, float *a, float *b, float *c)
{
    __shared__ float part[8][32];
    pdl_wait_and_release();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t col = blockIdx.x * int64_t{32} + lane, width = static_cast<int64_t>(arrays) * H;  // H is a multiple of 8
    float s = 0.f;
    if (col < width)
        for (int r = warp; r < ctas; r += 8)
            s += partial[r * width + col];
    part[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && col < width) {
#pragma unroll
        for (int w = 1; w < 8; ++w)
            s += part[w][lane];
        const int n = static_cast<int>(col / H);
        (n == 0 ? a : n == 1 ? b : c)[col - static_cast<int64_t>(n) * H] = s;
    }
}

}  // namespace mxfp8
