// The norms around a block fused with its gate and residual scale, and their gradients; formulas in include/block_norm.h.
//
// A CTA takes a row at a time and a thread V vectors of 8 columns of it, so that every input is read once and each
// output written once, with the row's sums (of y^2, then of h'^2; backward: y^2, h'^2 and dx w h' together, then b n1) formed
// between.  Rows up to 8192 columns come through a ring of shared-memory stages, filled by bulk copies while the rows before
// them are worked on; longer ones are loaded by the threads.  Bound by HBM for many rows, by the chain of loads, two
// reductions and stores (launch included) for few.
//
// The weights' gradients are sums over the rows: each thread adds up its columns' (in registers; in shared memory for long
// rows), a CTA writes its sums to the workspace at its end, and a second kernel adds the CTAs' in order.  With a
// gate per channel sum(g n1) serves both: dpost = gate times it, dgate = w_post times it.
#pragma once

#include <cstdint>

#include "ptx.cuh"
#include "tcgen05.cuh"

namespace mxfp8 {

constexpr int kNormSms = 152;
constexpr int kNormThreads = 512;
constexpr int kNormMaxStages = 4;
constexpr int64_t kNormWait = 4000000000;  // cycles: about 2 s
// CTAs whose partial sums the workspace holds, for rows of H columns.
inline int norm_ctas(int64_t H) { return kNormSms * (H > 4096 ? 1 : H > 2048 ? 2 : H > 1024 ? 4 : 8); }

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
    int stages;                        // of the ring
    bool keep;                         // the weights are kept in shared memory, before the ring
    unsigned *fault;
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

// Sums over the CTA (at most 16 warps), the same in every thread; one barrier.  `turn` alternates between two buffers, so
// that a buffer is written again only after a barrier that follows its last reads; the warps that a CTA does not have count
// zeros, which clear() leaves there (before a barrier).
struct RowSums {
    float buffer[2][16][4];

    __device__ __forceinline__ void clear()
    {
        for (int i = threadIdx.x; i < 2 * 16 * 4; i += blockDim.x)
            (&buffer[0][0][0])[i] = 0.f;
    }
    __device__ __forceinline__ float one(float s, int &turn, int lane, int warp)
    {
#pragma unroll
        for (int d = 16; d > 0; d >>= 1)
            s += __shfl_xor_sync(0xFFFFFFFFu, s, d);
        if (lane == 0)
            buffer[turn][warp][0] = s;
        __syncthreads();
        s = buffer[turn][lane & 15][0];
#pragma unroll
        for (int d = 8; d > 0; d >>= 1)
            s += __shfl_xor_sync(0xFFFFFFFFu, s, d);
        turn ^= 1;
        return s;
    }
    // Three sums.  Each exchange with a lane half as far halves the values that a lane carries (12 shuffles for 30).
    __device__ __forceinline__ void three(float (&s)[3], int &turn, int lane, int warp)
    {
        const bool b4 = lane & 16, b3 = lane & 8;
        const float a0 = (b4 ? s[2] : s[0]) + __shfl_xor_sync(0xFFFFFFFFu, b4 ? s[0] : s[2], 16);
        const float a1 = (b4 ? 0.f : s[1]) + __shfl_xor_sync(0xFFFFFFFFu, b4 ? s[1] : 0.f, 16);
        float v = (b3 ? a1 : a0) + __shfl_xor_sync(0xFFFFFFFFu, b3 ? a0 : a1, 8);  // the sum numbered lane / 8
#pragma unroll
        for (int d = 4; d > 0; d >>= 1)
            v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
        if ((lane & 7) == 0)
            buffer[turn][warp][lane >> 3] = v;
        __syncthreads();
        v = buffer[turn][lane >> 2][lane & 3] + buffer[turn][8 + (lane >> 2)][lane & 3];
#pragma unroll
        for (int d = 16; d > 2; d >>= 1)
            v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
#pragma unroll
        for (int n = 0; n < 3; ++n)
            s[n] = __shfl_sync(0xFFFFFFFFu, v, n);
        turn ^= 1;
    }
};

// The ring: stage n % stages holds the CTA's n-th row of each input, one after the other.
struct RowSource {
    const void *base[4];
    int64_t pitch[4];  // bytes
    int bytes[4];      // of a row; 0: not read
    int at[4];         // offset in a stage
    int stage;         // bytes
};
__device__ __forceinline__ void add_source(RowSource &s, int n, const void *base, int64_t ld, int H, int size)
{
    s.base[n] = base;
    s.pitch[n] = ld * size;
    s.bytes[n] = base != nullptr ? H * size : 0;
    s.at[n] = s.stage;
    s.stage += s.bytes[n];
}
template <int N>
__device__ __forceinline__ void fetch_row(const RowSource &s, uint32_t smem, uint32_t bar, int64_t row)
{
    mbar_arrive_expect_tx(bar, static_cast<uint32_t>(s.stage));
#pragma unroll
    for (int n = 0; n < N; ++n)
        if (s.bytes[n] != 0)
            bulk_load(smem + s.at[n], static_cast<const unsigned char *>(s.base[n]) + row * s.pitch[n], static_cast<uint32_t>(s.bytes[n]), bar);
}
// Eight elements from a stage (zeros for an input that is not read).
template <bool F32>
__device__ __forceinline__ Row8<F32> stage_row8(const unsigned char *stage, const RowSource &s, int n, int j)
{
    Row8<F32> r{};
    if (s.bytes[n] != 0) {
        const uint4 *q = reinterpret_cast<const uint4 *>(stage + s.at[n]) + j * (F32 ? 2 : 1);
        r.lo = q[0];
        if constexpr (F32)
            r.hi = q[1];
    }
    return r;
}

// A row's vectors for the passes over it.  From a stage of the ring they are read each time that they are wanted, which keeps
// them out of the registers that the sums need; a long row's are loaded once.
template <bool YF32, bool HF32>
struct StageRow {
    const unsigned char *stage;
    const RowSource &src;
    int vecs;

    __device__ __forceinline__ Row8<YF32> y(int, int j) const { return at<YF32>(0, j); }
    __device__ __forceinline__ Row8<HF32> h(int, int j) const { return at<HF32>(1, j); }
    __device__ __forceinline__ Row8<HF32> g(int, int j) const { return at<HF32>(2, j); }
    __device__ __forceinline__ Row8<false> x(int, int j) const { return at<false>(3, j); }
    template <bool F32>
    __device__ __forceinline__ Row8<F32> at(int n, int j) const
    {
        return j < vecs ? stage_row8<F32>(stage, src, n, j) : Row8<F32>{};
    }
};
template <bool YF32, bool HF32, int V, bool BACKWARD>
struct LoadedRow {
    Row8<YF32> y_[V];
    Row8<HF32> h_[V], g_[BACKWARD ? V : 1];
    Row8<false> x_[BACKWARD ? V : 1];

    __device__ __forceinline__ LoadedRow(const NormParams &p, int64_t row)
    {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int j = threadIdx.x + i * blockDim.x;
            y_[i] = Row8<YF32>{};
            h_[i] = Row8<HF32>{};
            if (j < p.vecs && p.y != nullptr)
                y_[i] = load_row8<YF32>(p.y, row * p.ldy + 8 * j);
            if (j < p.vecs && (!BACKWARD || p.dx != nullptr))
                h_[i] = load_row8<HF32>(p.h, row * p.ldh + 8 * j);
            if constexpr (BACKWARD) {
                g_[i] = Row8<HF32>{};
                x_[i] = Row8<false>{};
                if (j < p.vecs && p.dx != nullptr)
                    x_[i] = load_row8<false>(p.dx, row * p.lddx + 8 * j);
                if (j < p.vecs && p.dh_out != nullptr)
                    g_[i] = load_row8<HF32>(p.dh_out, row * p.lddh + 8 * j);
            }
        }
    }
    __device__ __forceinline__ Row8<YF32> y(int i, int) const { return y_[i]; }
    __device__ __forceinline__ Row8<HF32> h(int i, int) const { return h_[i]; }
    __device__ __forceinline__ Row8<HF32> g(int i, int) const { return g_[i]; }
    __device__ __forceinline__ Row8<false> x(int i, int) const { return x_[i]; }
};

// w_post * gate of vector j, the factors of a channel behind the block: from `back`, where the CTA keeps the products, or
// from the two.  False without either.
__device__ __forceinline__ bool back_weight8(const NormParams &p, const float *back, int j, float (&w)[8])
{
    if (back != nullptr) {
        const float4 a = reinterpret_cast<const float4 *>(back)[2 * j], b = reinterpret_cast<const float4 *>(back)[2 * j + 1];
        w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
        return true;
    }
    const bool channel = p.gate_kind == 1;
    if (p.post != nullptr)
        weight8(p.post, 8 * j, w);
    if (channel) {
        float v[8];
        weight8(p.gate, 8 * j, v);
#pragma unroll
        for (int k = 0; k < 8; ++k)
            w[k] = p.post != nullptr ? w[k] * v[k] : v[k];
    }
    return p.post != nullptr || channel;
}

// y, h -> h', x of one row.
template <bool YF32, bool HF32, int V, typename Row, typename Between>
__device__ __forceinline__ void norm_row(const NormParams &p, int64_t row, float inv, const float *back, RowSums &sums, int &turn, int lane, int warp, const Row &in,
                                         Between &&between)
{
    const int tid = threadIdx.x, nt = blockDim.x;
    float a[V][8];
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        widen8<YF32>(in.y(i, tid + i * nt), a[i]);
#pragma unroll
        for (int k = 0; k < 8; ++k)
            s = fmaf(a[i][k], a[i][k], s);
    }
    float factor = p.gate_kind == 2 ? __ldg(p.gate + row) : 1.0f;
    s = sums.one(s, turn, lane, warp);
    between();
    if (p.post != nullptr)
        factor *= rsqrtf(s * inv + p.eps);
    s = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int j = tid + i * nt;
        if (j < p.vecs) {
            float w[8], h[8];
            widen8<HF32>(in.h(i, j), h);
#pragma unroll
            for (int k = 0; k < 8; ++k)
                a[i][k] *= factor;
            if (back_weight8(p, back, j, w)) {
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
                s = fmaf(a[i][k], a[i][k], s);
        }
    }
    if (p.pre != nullptr) {
        s = sums.one(s, turn, lane, warp);
        const float r = rsqrtf(s * inv + p.eps);
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

// Eight values of a weight that may be kept in shared memory.
__device__ __forceinline__ void kept8(const float *w, int j, float (&v)[8])
{
    const float4 a = reinterpret_cast<const float4 *>(w)[2 * j], b = reinterpret_cast<const float4 *>(w)[2 * j + 1];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
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

// One row's gradients; add_pre and add_post take vector i's terms of the sums over rows (dx n2; token gate g n1).
template <bool YF32, bool HF32, int V, typename Row, typename Between, typename AddPre, typename AddPost>
__device__ __forceinline__ void norm_row_backward(const NormParams &p, int64_t row, float inv, const float *pre_weight, const float *back, RowSums &sums, int &turn, int lane,
                                                  int warp, const Row &in, Between &&between, AddPre &&add_pre, AddPost &&add_post)
{
    const int tid = threadIdx.x, nt = blockDim.x;
    const bool second = p.post != nullptr || (p.gate_kind == 2 && p.dgate != nullptr);
    float s[3] = {0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int j = tid + i * nt;
        float y[8], h[8], d[8], w[8];
        widen8<YF32>(in.y(i, j), y);
        widen8<HF32>(in.h(i, j), h);
        widen8<false>(in.x(i, j), d);
        const bool pre = p.dx != nullptr && j < p.vecs;
        if (pre)
            kept8(pre_weight, j, w);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            s[0] = fmaf(y[k], y[k], s[0]);
            s[1] = fmaf(h[k], h[k], s[1]);
            if (pre)
                s[2] = fmaf(d[k] * w[k], h[k], s[2]);
        }
    }
    sums.three(s, turn, lane, warp);
    between();
    const float r1 = p.post != nullptr ? rsqrtf(s[0] * inv + p.eps) : 1.0f;
    const float r2 = rsqrtf(s[1] * inv + p.eps);
    const float c2 = r2 * s[2] * inv;  // mean(t n2)
    const float token = p.gate_kind == 2 ? __ldg(p.gate + row) : 1.0f;
    float g[V][8];
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int j = tid + i * nt;
        widen8<HF32>(in.g(i, j), g[i]);
        if (j < p.vecs) {
            float w[8], q[8];
            if (p.dx != nullptr) {
                float h[8], d[8];
                widen8<HF32>(in.h(i, j), h);
                widen8<false>(in.x(i, j), d);
                kept8(pre_weight, j, w);
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const float n = h[k] * r2;
                    g[i][k] = fmaf(r2, fmaf(-n, c2, d[k] * w[k]), g[i][k]);
                    d[k] *= n;
                }
                add_pre(i, d);
            }
            if (p.dh != nullptr) {
                float v[8];
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    v[k] = p.scale * g[i][k];
                store8<HF32>(p.dh, row * p.H + 8 * j, v);
            }
            widen8<YF32>(in.y(i, j), q);
            {
                float v[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    q[k] *= r1;  // n1
                    v[k] = token * g[i][k] * q[k];
                }
                add_post(i, v);
            }
            if (back_weight8(p, back, j, w)) {
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    g[i][k] *= w[k];
            }
            if (second) {
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    m = fmaf(g[i][k], q[k], m);
            }
        }
    }
    if (second)
        m = sums.one(m, turn, lane, warp);
    if (p.gate_kind == 2 && p.dgate != nullptr && tid == 0)
        p.dgate[row] = m;
    if (p.dy != nullptr) {
        const float c1 = p.post != nullptr ? r1 * m * inv : 0.f, factor = token * r1;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int j = tid + i * nt;
            if (j < p.vecs) {
                float y[8];
                widen8<YF32>(in.y(i, j), y);
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    y[k] = factor * fmaf(-y[k], c1, g[i][k]);
                store8<YF32>(p.dy, row * p.H + 8 * j, y);
            }
        }
    }
}

// The products of w_post and gate of this thread's columns into shared memory at `kept`, which then points behind them.
// (Only the thread that writes them reads them.)
template <int V>
__device__ __forceinline__ const float *keep_back(const NormParams &p, float *&kept)
{
    if (!p.keep || (p.post == nullptr && p.gate_kind != 1))
        return nullptr;
    float *const back = kept;
    for (int i = 0; i < V; ++i) {
        const int j = threadIdx.x + i * blockDim.x;
        if (j < p.vecs) {
            float w[8];
            back_weight8(p, nullptr, j, w);
            store8<true>(back, 8 * j, w);
        }
    }
    kept += p.H;
    return back;
}

// The ring's part of a kernel: run(row, stage, between) for each of the CTA's rows, where `between` is called by all threads
// after a barrier that follows their last reads of the stage before.
template <int N, typename Run>
__device__ __forceinline__ void ring_rows(const NormParams &p, const RowSource &src, unsigned char *smem, uint64_t *full, Run &&run)
{
    const int tid = threadIdx.x;
    const uint32_t base = smem_u32(smem), full0 = smem_u32(full);
    if (tid == 0) {
        for (int s = 0; s < p.stages; ++s)
            mbar_init(full0 + 8 * s, 1);
        fence_mbar_init();
        for (int s = 0; s < p.stages; ++s) {
            const int64_t row = blockIdx.x + int64_t{s} * gridDim.x;
            if (row < p.T)
                fetch_row<N>(src, base + s * src.stage, full0 + 8 * s, row);
        }
    }
    __syncthreads();
    int slot = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int64_t row = blockIdx.x; row < p.T; row += gridDim.x) {
        if (ok && !mbar_wait_cycles(full0 + 8 * slot, phase, kNormWait)) {  // a copy that never lands: its rows are garbage, and told
            ok = false;
            atomicOr(p.fault, 1u);
        }
        run(row, smem + slot * src.stage, [&]() {
            const int64_t next = row + (int64_t{p.stages} - 1) * gridDim.x;  // into the stage of the row before
            if (tid == 0 && row != blockIdx.x && next < p.T) {
                const int s = slot == 0 ? p.stages - 1 : slot - 1;
                fetch_row<N>(src, base + s * src.stage, full0 + 8 * s, next);
            }
        });
        if (++slot == p.stages) {
            slot = 0;
            phase ^= 1;
        }
    }
}

template <bool YF32, bool HF32, int V>
__global__ void __launch_bounds__(kNormThreads, V == 2 ? 2 : 1) block_norm_ring_kernel(const NormParams p)
{
    extern __shared__ float4 norm_smem[];
    __shared__ RowSums sums;
    __shared__ uint64_t full[kNormMaxStages];
    pdl_wait_and_release();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nt = blockDim.x;
    const float inv = 1.0f / static_cast<float>(p.H);
    int turn = 0;
    sums.clear();
    RowSource src{};
    add_source(src, 0, p.y, p.ldy, p.H, YF32 ? 4 : 2);
    add_source(src, 1, p.h, p.ldh, p.H, HF32 ? 4 : 2);
    float *kept = reinterpret_cast<float *>(norm_smem);
    const float *back = keep_back<V>(p, kept);
    ring_rows<2>(p, src, reinterpret_cast<unsigned char *>(kept), full, [&](int64_t row, const unsigned char *stage, auto &&between) {
        norm_row<YF32, HF32, V>(p, row, inv, back, sums, turn, lane, warp, StageRow<YF32, HF32>{stage, src, p.vecs}, between);
    });
}

template <bool YF32, bool HF32, int V>
__global__ void __launch_bounds__(kNormThreads) block_norm_long_kernel(const NormParams p)
{
    __shared__ RowSums sums;
    pdl_wait_and_release();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nt = blockDim.x;
    const float inv = 1.0f / static_cast<float>(p.H);
    int turn = 0;
    sums.clear();
    __syncthreads();
    for (int64_t row = blockIdx.x; row < p.T; row += gridDim.x) {
        norm_row<YF32, HF32, V>(p, row, inv, nullptr, sums, turn, lane, warp, LoadedRow<YF32, HF32, V, false>(p, row), [] {});
    }
}

// A CTA's sums over its rows: [2][H] of the workspace (dx n2, then g n1).
template <int V>
__device__ __forceinline__ float *partial_of(const NormParams &p, int n, int j)
{
    return p.partial + (static_cast<int64_t>(blockIdx.x) * 2 + n) * p.H + 8 * j;
}

template <bool YF32, bool HF32, int V>
__global__ void __launch_bounds__(kNormThreads) block_norm_backward_ring_kernel(const NormParams p)
{
    extern __shared__ float4 norm_smem[];
    __shared__ RowSums sums;
    __shared__ uint64_t full[kNormMaxStages];
    pdl_wait_and_release();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nt = blockDim.x;
    const float inv = 1.0f / static_cast<float>(p.H);
    int turn = 0;
    sums.clear();
    RowSource src{};
    add_source(src, 0, p.y, p.ldy, p.H, YF32 ? 4 : 2);
    add_source(src, 1, p.dx != nullptr ? p.h : nullptr, p.ldh, p.H, HF32 ? 4 : 2);
    add_source(src, 2, p.dh_out, p.lddh, p.H, HF32 ? 4 : 2);
    add_source(src, 3, p.dx, p.lddx, p.H, 2);
    float acc[2][V][8];
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
        for (int k = 0; k < 8; ++k)
            acc[0][i][k] = acc[1][i][k] = 0.f;
    float *kept = reinterpret_cast<float *>(norm_smem);
    const float *back = keep_back<V>(p, kept), *pre = p.pre;
    if (p.keep && p.pre != nullptr) {
        for (int i = 0; i < V; ++i) {
            const int j = tid + i * nt;
            if (j < p.vecs) {
                float w[8];
                weight8(p.pre, 8 * j, w);
                store8<true>(kept, 8 * j, w);
            }
        }
        pre = kept;
        kept += p.H;
    }
    ring_rows<4>(p, src, reinterpret_cast<unsigned char *>(kept), full, [&](int64_t row, const unsigned char *stage, auto &&between) {
        auto add = [&](int n, int i, const float (&v)[8]) {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                acc[n][i][k] += v[k];
        };
        norm_row_backward<YF32, HF32, V>(p, row, inv, pre, back, sums, turn, lane, warp, StageRow<YF32, HF32>{stage, src, p.vecs}, between, [&](int i, const float (&v)[8]) { add(0, i, v); },
                                         [&](int i, const float (&v)[8]) { add(1, i, v); });
    });
    if (p.partial != nullptr) {
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int j = tid + i * nt;
                if (j < p.vecs) {
                    float4 *to = reinterpret_cast<float4 *>(partial_of<V>(p, n, j));
                    to[0] = make_float4(acc[n][i][0], acc[n][i][1], acc[n][i][2], acc[n][i][3]);
                    to[1] = make_float4(acc[n][i][4], acc[n][i][5], acc[n][i][6], acc[n][i][7]);
                }
            }
    }
}

template <bool YF32, bool HF32, int V>
__global__ void __launch_bounds__(kNormThreads) block_norm_backward_long_kernel(const NormParams p)
{
    extern __shared__ float4 norm_smem[];  // the CTA's sums [2][H]
    __shared__ RowSums sums;
    pdl_wait_and_release();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nt = blockDim.x;
    const float inv = 1.0f / static_cast<float>(p.H);
    int turn = 0;
    sums.clear();
    __syncthreads();
    float *acc = reinterpret_cast<float *>(norm_smem);
    auto each = [&](auto &&f) {
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (tid + i * nt < p.vecs)
                    f(n, tid + i * nt, reinterpret_cast<float4 *>(acc + n * p.H + 8 * (tid + i * nt)));
    };
    each([](int, int, float4 *a) { a[0] = a[1] = make_float4(0.f, 0.f, 0.f, 0.f); });
    for (int64_t row = blockIdx.x; row < p.T; row += gridDim.x) {
        norm_row_backward<YF32, HF32, V>(p, row, inv, p.pre, nullptr, sums, turn, lane, warp, LoadedRow<YF32, HF32, V, true>(p, row), [] {},
                                         [&](int i, const float (&v)[8]) { add8(acc + 8 * (tid + i * nt), v); },
                                         [&](int i, const float (&v)[8]) { add8(acc + p.H + 8 * (tid + i * nt), v); });
    }
    if (p.partial != nullptr)
        each([&](int n, int j, float4 *a) {
            float4 *to = reinterpret_cast<float4 *>(partial_of<V>(p, n, j));
            to[0] = a[0];
            to[1] = a[1];
        });
}

// The CTAs' sums, in order: a warp takes 32 columns of rows w, w + 8, ...; the eight warps' are added in order.
constexpr int kNormReduceThreads = 256;
__global__ void __launch_bounds__(kNormReduceThreads) block_norm_reduce_kernel(const NormParams p, int ctas)
{
    __shared__ float part[8][32];
    pdl_wait_and_release();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t col = blockIdx.x * int64_t{32} + lane, width = 2 * static_cast<int64_t>(p.H);
    float s = 0.f;
    if (col < width) {
#pragma unroll 4
        for (int r = warp; r < ctas; r += 8)
            s += p.partial[r * width + col];
    }
    part[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && col < width) {
#pragma unroll
        for (int w = 1; w < 8; ++w)
            s += part[w][lane];
        const bool channel = p.gate_kind == 1;
        if (col < p.H) {
            if (p.dpre != nullptr)
                p.dpre[col] = s;
        } else {
            const int c = static_cast<int>(col) - p.H;
            if (p.dpost != nullptr)
                p.dpost[c] = channel ? p.gate[c] * s : s;
            if (p.dgate != nullptr && channel)
                p.dgate[c] = p.post != nullptr ? p.post[c] * s : s;
        }
    }
}

}  // namespace mxfp8
