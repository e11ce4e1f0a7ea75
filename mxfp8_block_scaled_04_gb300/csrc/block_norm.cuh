// The norms around a block fused with its gate and residual scale, and their gradients; formulas in include/block_norm.h.
//
// A CTA takes a row at a time and a thread V vectors of 8 columns of it, so that every input is read once and each
// output written once, with the row's sums (of y^2, then of h'^2; backward: y^2, h'^2 and dx w h' together, then b n1) formed
// between.  Rows come through a ring of shared-memory stages, filled by bulk copies while the rows before them are worked
// on, and a stage is read again in every pass over its row, which leaves the registers to the sums.  Rows of more than
// kNormShare columns are shared by the two CTAs of a cluster, half each, which exchange their sums.
//
// The weights' gradients are sums over the rows: each thread adds up its columns' in registers, a CTA writes its sums to the
// workspace at its end, and a second kernel adds the CTAs' in order.  With a gate per channel sum(g n1) serves both:
// dpost = gate times it, dgate = w_post times it.
//
// Measured (8192x7168, y bf16, both weights, a gate per channel): forward 76 us with a bf16 stream (6.1 TB/s), 115 with fp32;
// gradients 123 (5.7 TB/s) and 181.  4000x16384: 95 and 174.  Bound by HBM; by the chain of loads, reductions and stores for few
// rows (16x7168 4.7 and 9.5 us, launches included) and by issue for short ones (16000x1024 gradients 45 us, 4.4 TB/s).
#pragma once

#include <cstdint>

#include "ptx.cuh"
#include "tcgen05.cuh"

namespace mxfp8 {

constexpr int kNormSms = 152;
constexpr int kNormThreads = 512;
constexpr int kNormMaxStages = 4;
constexpr int kNormShare = 8192;           // most columns of a CTA
constexpr int64_t kNormWait = 4000000000;  // cycles: about 2 s
constexpr int64_t kNormDrain = 400000000;
// Most rows in work at once, whose CTAs' sums the workspace holds, for rows of H columns.
inline int norm_rows(int64_t H) { return H > kNormShare ? kNormSms / 2 : kNormSms * (H > 4096 ? 1 : H > 2048 ? 2 : H > 1024 ? 4 : 8); }

struct NormParams {
    const void *y, *h;                 // backward: h is the stream behind the block
    const void *dh_out, *dx;
    int64_t T, ldy, ldh, lddh, lddx;
    int H, vecs;                       // vecs: of the row
    int gate_kind;
    float scale, eps;
    const float *pre, *post, *gate;
    void *h_out, *x;
    void *dh, *dy;
    float *dpre, *dpost, *dgate, *partial;
    int stages;                        // of the ring
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

// Eight fp32 values as four pairs, for the packed operations (half the instructions; each lane rounds as a scalar).
struct Vec8 {
    uint64_t p[4];

    static __device__ __forceinline__ Vec8 splat(float a) { return {f2_splat(a), f2_splat(a), f2_splat(a), f2_splat(a)}; }
};
__device__ __forceinline__ Vec8 operator*(const Vec8 &a, const Vec8 &b) { return {f2_mul(a.p[0], b.p[0]), f2_mul(a.p[1], b.p[1]), f2_mul(a.p[2], b.p[2]), f2_mul(a.p[3], b.p[3])}; }
__device__ __forceinline__ Vec8 operator*(const Vec8 &a, float b)
{
    const uint64_t s = f2_splat(b);
    return {f2_mul(a.p[0], s), f2_mul(a.p[1], s), f2_mul(a.p[2], s), f2_mul(a.p[3], s)};
}
__device__ __forceinline__ Vec8 operator+(const Vec8 &a, const Vec8 &b) { return {f2_add(a.p[0], b.p[0]), f2_add(a.p[1], b.p[1]), f2_add(a.p[2], b.p[2]), f2_add(a.p[3], b.p[3])}; }
__device__ __forceinline__ Vec8 fma8(const Vec8 &a, const Vec8 &b, const Vec8 &c)
{
    return {f2_fma(a.p[0], b.p[0], c.p[0]), f2_fma(a.p[1], b.p[1], c.p[1]), f2_fma(a.p[2], b.p[2], c.p[2]), f2_fma(a.p[3], b.p[3], c.p[3])};
}
__device__ __forceinline__ Vec8 fma8(const Vec8 &a, float b, const Vec8 &c)
{
    const uint64_t s = f2_splat(b);
    return {f2_fma(a.p[0], s, c.p[0]), f2_fma(a.p[1], s, c.p[1]), f2_fma(a.p[2], s, c.p[2]), f2_fma(a.p[3], s, c.p[3])};
}
// sum += a . b, in two strands that total() adds.
__device__ __forceinline__ void dot8(uint64_t &sum, const Vec8 &a, const Vec8 &b)
{
#pragma unroll
    for (int k = 0; k < 4; ++k)
        sum = f2_fma(a.p[k], b.p[k], sum);
}
__device__ __forceinline__ float total(uint64_t sum)
{
    float lo, hi;
    f2_unpack(sum, lo, hi);
    return lo + hi;
}

template <bool F32>
__device__ __forceinline__ Vec8 widen8(const Row8<F32> &r)
{
    if constexpr (F32) {
        const uint32_t w[8] = {r.lo.x, r.lo.y, r.lo.z, r.lo.w, r.hi.x, r.hi.y, r.hi.z, r.hi.w};
        Vec8 v;
#pragma unroll
        for (int k = 0; k < 4; ++k)
            v.p[k] = f2_pack(__uint_as_float(w[2 * k]), __uint_as_float(w[2 * k + 1]));
        return v;
    } else {
        const uint32_t w[4] = {r.lo.x, r.lo.y, r.lo.z, r.lo.w};
        Vec8 v;
#pragma unroll
        for (int k = 0; k < 4; ++k)
            v.p[k] = f2_pack(bf16_lo(w[k]), bf16_hi(w[k]));
        return v;
    }
}
__device__ __forceinline__ uint32_t round_bf16x2(uint64_t pair)
{
    float lo, hi;
    f2_unpack(pair, lo, hi);
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// Store eight elements; v becomes what was stored.
template <bool F32>
__device__ __forceinline__ void store8(void *base, int64_t at, Vec8 &v, bool write = true)
{
    unsigned char *p = static_cast<unsigned char *>(base) + at * (F32 ? 4 : 2);
    if constexpr (F32) {
        if (write) {
            *reinterpret_cast<ulonglong2 *>(p) = make_ulonglong2(v.p[0], v.p[1]);
            *reinterpret_cast<ulonglong2 *>(p + 16) = make_ulonglong2(v.p[2], v.p[3]);
        }
    } else {
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            w[k] = round_bf16x2(v.p[k]);
            v.p[k] = f2_pack(bf16_lo(w[k]), bf16_hi(w[k]));
        }
        if (write)
            *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}
// Vector j of a weight: through L1 (every row reads them), or from shared memory where the CTA keeps it.
__device__ __forceinline__ Vec8 weight8(const float *w, int j)
{
    const ulonglong2 a = __ldg(reinterpret_cast<const ulonglong2 *>(w) + 2 * j), b = __ldg(reinterpret_cast<const ulonglong2 *>(w) + 2 * j + 1);
    return {a.x, a.y, b.x, b.y};
}
__device__ __forceinline__ Vec8 kept8(const float *w, int j)
{
    const ulonglong2 a = reinterpret_cast<const ulonglong2 *>(w)[2 * j], b = reinterpret_cast<const ulonglong2 *>(w)[2 * j + 1];
    return {a.x, a.y, b.x, b.y};
}

// Sums over a row's CTAs (of at most 16 warps each), the same in every thread; one barrier.  `count` of the sums so far: they
// alternate between two buffers, so that a buffer is written again only after a barrier that follows its last reads; the warps that a CTA does not have count
// zeros, which clear() leaves there (before a barrier).
struct RowSums {
    float buffer[2][16][4];
    float4 inbox[2];      // the peer's sums
    uint64_t arrived[2];

    template <int CTAS>
    __device__ __forceinline__ void clear()
    {
        for (int i = threadIdx.x; i < 2 * 16 * 4; i += blockDim.x)
            (&buffer[0][0][0])[i] = 0.f;
        if constexpr (CTAS == 2) {
            if (threadIdx.x == 0) {
                mbar_init(smem_u32(&arrived[0]), 1);
                mbar_init(smem_u32(&arrived[1]), 1);
                fence_mbar_init();
            }
            cluster_sync();
        }
    }
    // Four sums.  Each exchange with a lane half as far halves the values that a lane carries (13 shuffles for 40).  With two
    // CTAs to a row each sends its sums to the other's inbox, a store that the other's barrier counts; an inbox is written again
    // only after the message between has been received, and so after its reads.
    template <int CTAS>
    __device__ __forceinline__ void four(float (&s)[4], int &count, bool &lost, int lane, int warp, unsigned *fault)
    {
        const int turn = count & 1;
        const bool b4 = lane & 16, b3 = lane & 8;
        const float a0 = (b4 ? s[2] : s[0]) + __shfl_xor_sync(0xFFFFFFFFu, b4 ? s[0] : s[2], 16);
        const float a1 = (b4 ? s[3] : s[1]) + __shfl_xor_sync(0xFFFFFFFFu, b4 ? s[1] : s[3], 16);
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
        for (int n = 0; n < 4; ++n)
            s[n] = __shfl_sync(0xFFFFFFFFu, v, n);
        if constexpr (CTAS == 2) {
            const uint32_t bar = smem_u32(&arrived[turn]), peer = cluster_rank() ^ 1;
            if (threadIdx.x == 0) {
                mbar_arrive_expect_tx(bar, 16);
                asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(
                                 map_to_rank(smem_u32(&inbox[turn]), peer)),
                             "f"(s[0]), "f"(s[1]), "f"(s[2]), "f"(s[3]), "r"(map_to_rank(bar, peer))
                             : "memory");
            }
            if (!lost && !mbar_wait_cluster(bar, (count >> 1) & 1, kNormWait)) {  // sums that never come: waited for once, and told
                lost = true;
                atomicOr(fault, 1u);
            }
            const float4 other = inbox[turn];
            s[0] += other.x, s[1] += other.y, s[2] += other.z, s[3] += other.w;
        }
        ++count;
    }
    template <int CTAS>
    __device__ __forceinline__ float one(float s, int &count, bool &lost, int lane, int warp, unsigned *fault)
    {
        if constexpr (CTAS == 2) {
            float t[4] = {s, 0.f, 0.f, 0.f};
            four<2>(t, count, lost, lane, warp, fault);
            return t[0];
        }
        const int turn = count & 1;
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
        ++count;
        return s;
    }
};

// The ring: stage n % stages holds the CTA's n-th row of each input, one after the other.
struct RowSource {
    const void *base[4];  // at the CTA's first column
    int64_t pitch[4];  // bytes
    int bytes[4];      // of a row; 0: not read
    int at[4];         // offset in a stage
    int stage;         // bytes
};
// The CTA's columns, in vectors.
struct Share {
    int first, vecs;
};
template <int CTAS>
__device__ __forceinline__ Share my_share(const NormParams &p)
{
    if constexpr (CTAS == 1)
        return {0, p.vecs};
    const int half = (p.vecs + 1) / 2, rank = static_cast<int>(cluster_rank());
    return {rank * half, rank == 0 ? half : p.vecs - half};
}
__device__ __forceinline__ void add_source(RowSource &s, int n, const void *base, int64_t ld, const Share &c, int size)
{
    s.base[n] = static_cast<const unsigned char *>(base) + c.first * 8 * size;
    s.pitch[n] = ld * size;
    s.bytes[n] = base != nullptr ? c.vecs * 8 * size : 0;
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

// A row's vectors for the passes over it, read from its stage each time that they are wanted, which keeps them out of the
// registers that the sums need.
template <bool YF32, bool HF32>
struct StageRow {
    const unsigned char *stage;
    const RowSource &src;
    int vecs;

    __device__ __forceinline__ Row8<YF32> y(int j) const { return at<YF32>(0, j); }
    __device__ __forceinline__ Row8<HF32> h(int j) const { return at<HF32>(1, j); }
    __device__ __forceinline__ Row8<HF32> g(int j) const { return at<HF32>(2, j); }
    __device__ __forceinline__ Row8<false> x(int j) const { return at<false>(3, j); }
    template <bool F32>
    __device__ __forceinline__ Row8<F32> at(int n, int j) const
    {
        return j < vecs ? stage_row8<F32>(stage, src, n, j) : Row8<F32>{};
    }
};
template <bool KEPT>
__device__ __forceinline__ Vec8 weight8_of(const float *w, int first, int j) { return KEPT ? kept8(w, j) : weight8(w, first + j); }

// Whether channels have a factor behind the block: w_post, a gate or both.
__device__ __forceinline__ bool has_back(const NormParams &p) { return p.post != nullptr || p.gate_kind == 1; }
// Its vector j of the CTA's, which begin at `first`: from `back`, where the CTA keeps the products, or (KEPT false) from the two.
template <bool KEPT>
__device__ __forceinline__ Vec8 back_weight8(const NormParams &p, const float *back, int first, int j)
{
    if constexpr (KEPT)
        return kept8(back, j);
    j += first;
    if (p.gate_kind != 1)
        return weight8(p.post, j);
    return p.post != nullptr ? weight8(p.post, j) * weight8(p.gate, j) : weight8(p.gate, j);
}

// y, h -> h', x of one row.
template <bool YF32, bool HF32, int V, bool KEPT, int CTAS, typename Row, typename Between>
__device__ __forceinline__ void norm_row(const NormParams &p, const Share &c, int64_t row, float inv, const float *back, RowSums &sums, int &count, bool &lost, int lane, int warp, const Row &in,
                                         Between &&between)
{
    const int tid = threadIdx.x, nt = blockDim.x;
    Vec8 a[V];
    uint64_t s2 = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        a[i] = widen8<YF32>(in.y(tid + i * nt));
        dot8(s2, a[i], a[i]);
    }
    float factor = p.gate_kind == 2 ? __ldg(p.gate + row) : 1.0f;
    const float s = sums.one<CTAS>(total(s2), count, lost, lane, warp, p.fault);
    between();
    if (p.post != nullptr)
        factor *= rsqrtf(s * inv + p.eps);
    s2 = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int j = tid + i * nt;
        if (j < c.vecs) {
            a[i] = a[i] * factor;
            if (has_back(p))
                a[i] = a[i] * back_weight8<KEPT>(p, back, c.first, j);
            a[i] = fma8(widen8<HF32>(in.h(j)), p.scale, a[i]);
            store8<HF32>(p.h_out, row * p.H + 8 * (c.first + j), a[i], p.h_out != nullptr);
            dot8(s2, a[i], a[i]);
        }
    }
    if (p.pre != nullptr) {
        const float r = rsqrtf(sums.one<CTAS>(total(s2), count, lost, lane, warp, p.fault) * inv + p.eps);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int j = tid + i * nt;
            if (j < c.vecs) {
                Vec8 x = a[i] * r * weight8(p.pre, c.first + j);
                store8<false>(p.x, row * p.H + 8 * (c.first + j), x);
            }
        }
    }
}

// The gradients of a row in three passes, with the row's sums between them: y^2, h'^2 and dx w_pre h' before the second, which
// leaves the sum of b n1 (or of g u) for the third.
template <bool YF32, bool HF32, int V, bool KEPT, typename Row>
__device__ __forceinline__ void backward_sums(const NormParams &p, const Share &c, const float *pre_weight, const Row &in, float (&s)[4])
{
    uint64_t sy = 0, sh = 0, sd = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int j = threadIdx.x + i * blockDim.x;
        const Vec8 y = widen8<YF32>(in.y(j)), h = widen8<HF32>(in.h(j));
        dot8(sy, y, y);
        dot8(sh, h, h);
        if (p.dx != nullptr && j < c.vecs)
            dot8(sd, widen8<false>(in.x(j)) * weight8_of<KEPT>(pre_weight, c.first, j), h);
    }
    s[0] = total(sy);
    s[1] = total(sh);
    s[2] = total(sd);
}

struct RowFactors {
    float r1, r2, c2, token;  // c2: mean(t n2)
};
__device__ __forceinline__ RowFactors row_factors(const NormParams &p, int64_t row, float inv, const float (&s)[4])
{
    RowFactors f;
    f.r1 = p.post != nullptr ? rsqrtf(s[0] * inv + p.eps) : 1.0f;
    f.r2 = rsqrtf(s[1] * inv + p.eps);
    f.c2 = f.r2 * s[2] * inv;
    f.token = p.gate_kind == 2 ? __ldg(p.gate + row) : 1.0f;
    return f;
}

// g becomes b without the token's gate; y the row's elements of y; add_pre and add_post take vector i's terms of the sums over
// rows (dx n2; token gate g n1).
template <bool YF32, bool HF32, int V, bool KEPT, typename Row, typename AddPre, typename AddPost>
__device__ __forceinline__ float backward_apply(const NormParams &p, const Share &c, int64_t row, const RowFactors &f, const float *pre_weight, const float *back, const Row &in, Vec8 (&g)[V],
                                                Row8<YF32> (&y)[V], AddPre &&add_pre, AddPost &&add_post)
{
    uint64_t sm = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int j = threadIdx.x + i * blockDim.x;
        y[i] = in.y(j);
        if (j < c.vecs) {
            g[i] = widen8<HF32>(in.g(j));
            if (p.dx != nullptr) {
                const Vec8 n = widen8<HF32>(in.h(j)) * f.r2, d = widen8<false>(in.x(j));
                g[i] = fma8(fma8(n, -f.c2, d * weight8_of<KEPT>(pre_weight, c.first, j)), f.r2, g[i]);
                add_pre(i, d, n);
            }
            if (p.dh != nullptr) {
                Vec8 v = g[i] * p.scale;
                store8<HF32>(p.dh, row * p.H + 8 * (c.first + j), v);
            }
            const Vec8 n1 = widen8<YF32>(y[i]) * f.r1;
            add_post(i, g[i] * f.token, n1);
            if (has_back(p))
                g[i] = g[i] * back_weight8<KEPT>(p, back, c.first, j);
            dot8(sm, g[i], n1);
        }
    }
    return total(sm);
}

// m: the sum of b n1 without the token's gate.
template <bool YF32, int V>
__device__ __forceinline__ void backward_store(const NormParams &p, const Share &c, int64_t row, float inv, const RowFactors &f, float m, const Vec8 (&g)[V], const Row8<YF32> (&y)[V])
{
    if (p.gate_kind == 2 && p.dgate != nullptr && threadIdx.x == 0 && c.first == 0)
        p.dgate[row] = m;
    if (p.dy == nullptr)
        return;
    const float c1 = p.post != nullptr ? f.r1 * m * inv : 0.f, factor = f.token * f.r1;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int j = threadIdx.x + i * blockDim.x;
        if (j < c.vecs) {
            Vec8 v = fma8(widen8<YF32>(y[i]), -c1, g[i]) * factor;
            store8<YF32>(p.dy, row * p.H + 8 * (c.first + j), v);
        }
    }
}

// The products of w_post and gate of this thread's columns into shared memory at `kept`, which then points behind them.
// (Only the thread that writes them reads them.)
template <int V, bool KEEP>
__device__ __forceinline__ const float *keep_back(const NormParams &p, const Share &c, float *&kept)
{
    if (!KEEP || !has_back(p))
        return nullptr;
    float *const back = kept;
    for (int i = 0; i < V; ++i) {
        const int j = threadIdx.x + i * blockDim.x;
        if (j < c.vecs) {
            Vec8 w = back_weight8<false>(p, nullptr, c.first, j);
            store8<true>(back, 8 * j, w);
        }
    }
    kept += 8 * c.vecs;
    return back;
}

// The ring's state: each of the CTA's rows in turn.
struct Ring {
    unsigned char *smem;
    uint32_t base, full0;
    int slot, phase;
    bool ok;

    template <int N>
    __device__ __forceinline__ void start(const NormParams &p, const RowSource &src, unsigned char *memory, uint64_t *full, int64_t first, int64_t step)
    {
        smem = memory;
        base = smem_u32(memory);
        full0 = smem_u32(full);
        slot = phase = 0;
        ok = true;
        if (threadIdx.x == 0) {
            for (int s = 0; s < p.stages; ++s)
                mbar_init(full0 + 8 * s, 1);
            fence_mbar_init();
            for (int s = 0; s < p.stages; ++s) {
                const int64_t row = first + s * step;
                if (row < p.T)
                    fetch_row<N>(src, base + s * src.stage, full0 + 8 * s, row);
            }
        }
        __syncthreads();
    }
    // The next row's stage, once its copies have landed.
    __device__ __forceinline__ const unsigned char *next(const NormParams &p, const RowSource &src)
    {
        if (ok && !mbar_wait_cycles(full0 + 8 * slot, phase, kNormWait)) {  // a copy that never lands: the rows are garbage, and told
            ok = false;
            atomicOr(p.fault, 1u);
        }
        const unsigned char *at = smem + slot * src.stage;
        if (++slot == p.stages) {
            slot = 0;
            phase ^= 1;
        }
        return at;
    }
    // After a wait that ran out: the copies that are still in flight, for a while.
    __device__ __forceinline__ void drain(const NormParams &p)
    {
        if (!ok)
            for (int s = 0; s < p.stages; ++s)
                mbar_wait_cycles(full0 + 8 * s, s >= slot ? phase : phase ^ 1, kNormDrain);
    }
    // Row `row` into a stage whose readers have all passed a barrier since; behind: how many stages before the next one.
    template <int N>
    __device__ __forceinline__ void refill(const NormParams &p, const RowSource &src, int behind, int64_t row)
    {
        if (threadIdx.x == 0 && ok && row < p.T) {
            const int s = slot >= behind ? slot - behind : slot - behind + p.stages;
            fetch_row<N>(src, base + s * src.stage, full0 + 8 * s, row);
        }
    }
};

template <bool YF32, bool HF32, int V, bool KEEP, int CTAS>
__global__ void __launch_bounds__(kNormThreads, V == 2 ? 2 : 1) block_norm_kernel(const NormParams p)
{
    extern __shared__ float4 norm_smem[];
    __shared__ RowSums sums;
    __shared__ uint64_t full[kNormMaxStages];
    pdl_wait_and_release();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const float inv = 1.0f / static_cast<float>(p.H);
    const int64_t first = blockIdx.x / CTAS, step = gridDim.x / CTAS;
    const Share c = my_share<CTAS>(p);
    int count = 0;
    bool lost = false;
    sums.clear<CTAS>();
    RowSource src{};
    add_source(src, 0, p.y, p.ldy, c, YF32 ? 4 : 2);
    add_source(src, 1, p.h, p.ldh, c, HF32 ? 4 : 2);
    float *kept = reinterpret_cast<float *>(norm_smem);
    const float *back = keep_back<V, KEEP>(p, c, kept);
    Ring ring;
    ring.start<2>(p, src, reinterpret_cast<unsigned char *>(kept), full, first, step);
    for (int64_t row = first; row < p.T; row += step) {
        const StageRow<YF32, HF32> in{ring.next(p, src), src, c.vecs};
        // behind the row's first barrier nobody reads the row before it any more
        norm_row<YF32, HF32, V, KEEP, CTAS>(p, c, row, inv, back, sums, count, lost, lane, warp, in, [&]() {
            if (row != first)
                ring.refill<2>(p, src, 2, row + (p.stages - 1) * step);
        });
    }
    ring.drain(p);
}

template <bool YF32, bool HF32, int V, bool KEEP, int CTAS>
__global__ void __launch_bounds__(kNormThreads) block_norm_backward_kernel(const NormParams p)
{
    extern __shared__ float4 norm_smem[];
    __shared__ RowSums sums;
    __shared__ uint64_t full[kNormMaxStages];
    pdl_wait_and_release();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nt = blockDim.x;
    const float inv = 1.0f / static_cast<float>(p.H);
    const int64_t first = blockIdx.x / CTAS, step = gridDim.x / CTAS;
    const Share c = my_share<CTAS>(p);
    int count = 0;
    bool lost = false;
    sums.clear<CTAS>();
    RowSource src{};
    add_source(src, 0, p.y, p.ldy, c, YF32 ? 4 : 2);
    add_source(src, 1, p.dx != nullptr ? p.h : nullptr, p.ldh, c, HF32 ? 4 : 2);
    add_source(src, 2, p.dh_out, p.lddh, c, HF32 ? 4 : 2);
    add_source(src, 3, p.dx, p.lddx, c, 2);
    Vec8 acc[2][V];
#pragma unroll
    for (int i = 0; i < V; ++i)
        acc[0][i] = acc[1][i] = Vec8::splat(0.f);
    float *kept = reinterpret_cast<float *>(norm_smem);
    const float *back = keep_back<V, KEEP>(p, c, kept), *pre = KEEP ? kept : p.pre;
    if (KEEP && p.pre != nullptr) {
        for (int i = 0; i < V; ++i) {
            const int j = tid + i * nt;
            if (j < c.vecs) {
                Vec8 w = weight8(p.pre, c.first + j);
                store8<true>(kept, 8 * j, w);
            }
        }
        kept += 8 * c.vecs;
    }
    Ring ring;
    ring.start<4>(p, src, reinterpret_cast<unsigned char *>(kept), full, first, step);
    // A row's second pass and the next row's first share one exchange of sums.
    const unsigned char *stage = ring.next(p, src);
    float s[4];
    backward_sums<YF32, HF32, V, KEEP>(p, c, pre, StageRow<YF32, HF32>{stage, src, c.vecs}, s);
    s[3] = 0.f;
    sums.four<CTAS>(s, count, lost, lane, warp, p.fault);
    for (int64_t row = first; row < p.T; row += step) {
        const RowFactors f = row_factors(p, row, inv, s);
        Vec8 g[V];
        Row8<YF32> y[V];
        const float m = backward_apply<YF32, HF32, V, KEEP>(
            p, c, row, f, pre, back, StageRow<YF32, HF32>{stage, src, c.vecs}, g, y, [&](int i, const Vec8 &d, const Vec8 &n) { acc[0][i] = fma8(d, n, acc[0][i]); },
            [&](int i, const Vec8 &v, const Vec8 &n) { acc[1][i] = fma8(v, n, acc[1][i]); });
        const bool more = row + step < p.T;
        if (more) {
            stage = ring.next(p, src);
            backward_sums<YF32, HF32, V, KEEP>(p, c, pre, StageRow<YF32, HF32>{stage, src, c.vecs}, s);
        }
        s[3] = m;
        sums.four<CTAS>(s, count, lost, lane, warp, p.fault);
        if (more)
            ring.refill<4>(p, src, 2, row + p.stages * step);
        backward_store<YF32, V>(p, c, row, inv, f, s[3], g, y);
    }
    ring.drain(p);
    if (p.partial != nullptr) {  // a row of [2][H] per CTA (per cluster): dx n2, then g n1
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int j = tid + i * nt;
                if (j < c.vecs) {
                    store8<true>(p.partial + (first * 2 + n) * p.H, 8 * (c.first + j), acc[n][i]);
                }
            }
    }
}

// The CTAs' sums, in order: a warp takes 32 columns of every W-th CTA's; the W warps' are added in order.  W is 8, or 32 for the
// many CTAs of short rows (16000x1024, 1064 CTAs: gradients 50 -> 45 us; for 152 and fewer 8 are as fast or faster).
constexpr int kNormReduceFew = 256, kNormReduceMany = 1024, kNormReduceCtas = 256;
__global__ void __launch_bounds__(kNormReduceMany) block_norm_reduce_kernel(const NormParams p, int ctas)
{
    __shared__ float part[32][32];
    pdl_wait_and_release();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int64_t col = blockIdx.x * int64_t{32} + lane, width = 2 * static_cast<int64_t>(p.H);
    float s = 0.f;
    if (col < width) {
#pragma unroll 4
        for (int r = warp; r < ctas; r += warps)
            s += p.partial[r * width + col];
    }
    part[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && col < width) {
        for (int w = 1; w < warps; ++w)
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
