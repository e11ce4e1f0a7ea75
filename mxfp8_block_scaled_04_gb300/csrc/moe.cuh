// Expert routing, its gradient, the dispatch plan and the combination of the experts' rows (sm_103a);
// formulas and contracts in include/moe.h.  All sums and scores are fp32; every result is deterministic.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>

#include "ptx.cuh"

namespace mxfp8 {

constexpr int kRouteThreads = 256;
constexpr int kRouteMaxE = 512;
constexpr unsigned kAll = 0xFFFFFFFFu;

struct RouteParams {
    const void *logits;
    int64_t T, ld;
    int E, k, groups, topk_groups;
    bool sigmoid, renorm;
    bool vec;        // a lane's experts load (and store) as vectors
    bool vec16;      // backward: rows of dlogits are whole 16-byte vectors
    float scale;
    const float *bias;
    int32_t *indices;
    float *weights;
    // backward
    const int32_t *idx_in;
    const float *dweights;
    void *dlogits;
};

// One warp routes one token.  Lane l holds the VPL consecutive experts from l * VPL (32 * VPL is E rounded up to
// a power of two), so the lowest lane of a ballot holds the lowest index, equal groups are runs of lanes, and
// the softmax's sum by halves is first lane l with l ^ 16, l ^ 8, ..., then a lane's own values.
template <int VPL, bool F32>
__device__ __forceinline__ void load_row(const RouteParams &p, int64_t t, int lane, float (&l)[VPL], float fill)
{
    constexpr int kBytes = VPL * (F32 ? 4 : 2);
    const int e0 = lane * VPL;
    if (p.vec) {
        if (e0 < p.E) {
            const unsigned char *src = static_cast<const unsigned char *>(p.logits) + (t * p.ld + e0) * (F32 ? 4 : 2);
            uint32_t w[kBytes / 4 > 0 ? kBytes / 4 : 1];
            if constexpr (kBytes >= 16) {
#pragma unroll
                for (int i = 0; i < kBytes / 16; ++i) {
                    const uint4 q = reinterpret_cast<const uint4 *>(src)[i];
                    w[4 * i] = q.x, w[4 * i + 1] = q.y, w[4 * i + 2] = q.z, w[4 * i + 3] = q.w;
                }
            } else if constexpr (kBytes == 8) {
                const uint2 q = *reinterpret_cast<const uint2 *>(src);
                w[0] = q.x, w[1] = q.y;
            } else if constexpr (kBytes == 4) {
                w[0] = *reinterpret_cast<const uint32_t *>(src);
            } else {
                w[0] = *reinterpret_cast<const uint16_t *>(src);
            }
#pragma unroll
            for (int i = 0; i < VPL; ++i)
                l[i] = F32 ? __uint_as_float(w[F32 ? i : 0]) : (i & 1 ? bf16_hi(w[i / 2]) : bf16_lo(w[i / 2]));
            return;
        }
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            l[i] = fill;
        return;
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        l[i] = fill;
        if (e0 + i < p.E) {
            if constexpr (F32)
                l[i] = static_cast<const float *>(p.logits)[t * p.ld + e0 + i];
            else
                l[i] = __bfloat162float(static_cast<const __nv_bfloat16 *>(p.logits)[t * p.ld + e0 + i]);
        }
    }
}

__device__ __forceinline__ float max_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// exp(l - max) / sum for the row; experts past E (filled with -inf) get 0.  A row of -inf only: all 0; with a NaN: all NaN.
template <int VPL>
__device__ __forceinline__ void softmax_row(float (&l)[VPL], float (&s)[VPL])
{
    float m = l[0];
#pragma unroll
    for (int i = 1; i < VPL; ++i)
        m = max_nan(m, l[i]);
#pragma unroll
    for (int d = 16; d; d >>= 1)
        m = max_nan(m, __shfl_xor_sync(kAll, m, d));
    const bool none = m == -__int_as_float(0x7F800000);
    float r[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        s[i] = none ? 0.f : expf(l[i] - m);
        r[i] = s[i];
    }
#pragma unroll
    for (int d = 16; d; d >>= 1)
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            r[i] += __shfl_xor_sync(kAll, r[i], d);
#pragma unroll
    for (int h = VPL / 2; h; h >>= 1)
#pragma unroll
        for (int i = 0; i < h; ++i)
            r[i] += r[i + h];
#pragma unroll
    for (int i = 0; i < VPL; ++i)
        s[i] = none ? s[i] : s[i] / r[0];
}

// 1 / (1 + exp(-l)), the quotient rounded to nearest.  Up to 2^126 the reciprocal is the hardware's estimate
// and one correction with fused multiply-adds (P. Markstein, "Computation of elementary functions on the IBM RISC
// System/6000 processor", 1990): the correctly rounded one for every fp32 number in [1, 2^126], which
// tests/reciprocal_check.cu compares one by one.
constexpr float kReciprocalMax = 8.507059173023462e37f;  // 2^126
__device__ __forceinline__ float reciprocal_fast(float y)
{
    float q;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(q) : "f"(y));
    return fmaf(q, fmaf(-y, q, 1.0f), q);
}
__device__ __forceinline__ float sigmoid_exact(float l)
{
    const float y = 1.0f + expf(-l);
    return y > kReciprocalMax ? __frcp_rn(y) : reciprocal_fast(y);
}
template <int VPL>
__device__ __forceinline__ void sigmoid_row(const float (&l)[VPL], float (&s)[VPL])
{
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        const float y = 1.0f + expf(-l[i]);
        s[i] = reciprocal_fast(y);
        top = fmaxf(top, y);
    }
    if (top > kReciprocalMax) {
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            s[i] = sigmoid_exact(l[i]);
    }
}

// Order of keys as integers: NaN below every number, -0 equal to 0; 0 is left for "cannot be chosen".
__device__ __forceinline__ uint32_t order_key(float x)
{
    const uint32_t b = __float_as_uint(x + 0.0f);
    return x != x ? 1u : (b & 0x80000000u) ? ~b : b | 0x80000000u;
}

// order_key of a number (not NaN, not -0).
__device__ __forceinline__ uint32_t order_key_number(float x)
{
    const uint32_t b = __float_as_uint(x);
    return b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
}

// Falling order, by Batcher's odd-even merge network (VPL a power of two).
template <int A, int B, int VPL>
__device__ __forceinline__ void order_two(uint32_t (&v)[VPL])
{
    const uint32_t a = v[A], b = v[B];
    v[A] = max(a, b);
    v[B] = min(a, b);
}
template <int LO, int N, int R, int VPL>
__device__ __forceinline__ void merge_keys(uint32_t (&v)[VPL])
{
    if constexpr (2 * R < N) {
        merge_keys<LO, N, 2 * R>(v);
        merge_keys<LO + R, N, 2 * R>(v);
#pragma unroll
        for (int i = LO + R; i + R < LO + N; i += 2 * R) {
            const uint32_t a = v[i], b = v[i + R];
            v[i] = max(a, b);
            v[i + R] = min(a, b);
        }
    } else {
        order_two<LO, LO + R>(v);
    }
}
template <int VPL, int LO = 0, int N = VPL>
__device__ __forceinline__ void sort_keys(uint32_t (&v)[VPL])
{
    if constexpr (N > 1) {
        sort_keys<VPL, LO, N / 2>(v);
        sort_keys<VPL, LO + N / 2, N / 2>(v);
        merge_keys<LO, N, 1>(v);
    }
}

// The chosen are found by value: each lane sorts its keys, and k times the largest head of all lanes leaves (one
// warp-wide maximum, one ballot).  Which expert of the lane it was is looked up once, for all k at a time.  Bound by
// issue, about 690 warp instructions per token in 72% of the issue slots (65536x256 fp32, sigmoid, bias, 4 of 8 groups,
// 8 experts: 57 us; 128 us when each choice searched its lane again; the logits alone are 10 us of HBM).
template <int VPL, bool F32>
__global__ void __launch_bounds__(kRouteThreads) moe_route_kernel(const RouteParams p)
{
    constexpr float kNegInf = -__builtin_huge_valf();
    __shared__ __align__(16) float rows[kRouteThreads / 32][32 * VPL];
    __shared__ __align__(16) uint32_t keys[kRouteThreads / 32][32 * VPL];
    pdl_wait_and_release();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float *row = rows[warp];
    const int gs = p.E / p.groups;
    const int run = gs / VPL;  // lanes of a group, where a group is an aligned run of them
    const bool limited = p.topk_groups < p.groups, runs = run * VPL == gs && (run & (run - 1)) == 0;
    float b[VPL];
    if (p.bias != nullptr) {
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            b[i] = lane * VPL + i < p.E ? p.bias[lane * VPL + i] : 0.f;
    }
    for (int64_t t = blockIdx.x * int64_t{kRouteThreads / 32} + warp; t < p.T; t += gridDim.x * int64_t{kRouteThreads / 32}) {
        float l[VPL], s[VPL];
        uint32_t key[VPL];
        load_row<VPL, F32>(p, t, lane, l, kNegInf);
        if (p.sigmoid) {
            sigmoid_row<VPL>(l, s);
        } else {
            softmax_row<VPL>(l, s);
        }
        float kf[VPL], nan = 0.f;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            kf[i] = p.bias != nullptr ? s[i] + b[i] : l[i] + 0.0f;  // a sum of a score is never -0
            key[i] = order_key_number(kf[i]);
            nan = max_nan(nan, kf[i]);
        }
        if (nan != nan || p.E != 32 * VPL) {
#pragma unroll
            for (int i = 0; i < VPL; ++i)
                key[i] = lane * VPL + i >= p.E ? 0u : kf[i] != kf[i] ? 1u : key[i];
        }
        __syncwarp();  // the token before is done with the arrays
        if (limited && !runs) {
            // lanes rank whole groups from shared memory
#pragma unroll
            for (int i = 0; i < VPL; ++i)
                row[lane * VPL + i] = kf[i];
            __syncwarp();
            uint32_t rank[VPL];  // groups lane, lane + 32, ...: no more of them than experts
#pragma unroll
            for (int n = 0; n < VPL; ++n) {
                rank[n] = 0;
                const int g = lane + 32 * n;
                if (g < p.groups) {
                    uint32_t a = 0, c = 0;
                    float va = 0.f, vc = 0.f;
                    for (int i = 0; i < gs; ++i) {
                        const float v = row[g * gs + i];
                        const uint32_t u = order_key(v);
                        if (u > a) {
                            c = a, vc = va;
                            a = u, va = v;
                        } else if (u > c) {
                            c = u, vc = v;
                        }
                    }
                    rank[n] = p.bias == nullptr || gs == 1 ? a : order_key(va + vc);
                }
            }
            uint32_t taken = 0;  // bit n: group lane + 32 n is kept
            for (int j = 0; j < p.topk_groups; ++j) {
                uint32_t top = 0;
                int at = 0;
#pragma unroll
                for (int n = 0; n < VPL; ++n)
                    if (rank[n] > top) {
                        top = rank[n];
                        at = n;
                    }
                const uint32_t best = __reduce_max_sync(kAll, top);
                const int g = __reduce_min_sync(kAll, top == best ? lane + 32 * at : 1 << 20);
                if (lane == (g & 31)) {
                    taken |= 1u << (g >> 5);
#pragma unroll
                    for (int n = 0; n < VPL; ++n)
                        rank[n] = n == (g >> 5) ? 0u : rank[n];
                }
            }
#pragma unroll
            for (int i = 0; i < VPL; ++i) {
                const int g = (lane * VPL + i) / gs;
                const uint32_t kept = __shfl_sync(kAll, taken, g & 31);
                if (!(g < p.groups && (kept >> (g >> 5)) & 1))
                    key[i] = 0;
            }
            __syncwarp();
        }
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            row[lane * VPL + i] = s[i];
            keys[warp][lane * VPL + i] = key[i];
        }
        sort_keys<VPL>(key);
        if (limited && runs) {
            uint32_t rank = key[0];
            if (p.bias == nullptr) {
                for (int d = 1; d < run; d <<= 1)
                    rank = max(rank, __shfl_xor_sync(kAll, rank, d));
            } else {
                uint32_t a = key[0], c = VPL > 1 ? key[VPL > 1 ? 1 : 0] : 0u;  // the two largest
                for (int d = 1; d < run; d <<= 1) {
                    const uint32_t oa = __shfl_xor_sync(kAll, a, d), oc = __shfl_xor_sync(kAll, c, d);
                    c = max(max(c, oc), min(a, oa));
                    a = max(a, oa);
                }
                auto value = [](uint32_t u) { return u == 1u ? __uint_as_float(0x7FC00000u) : __uint_as_float(u & 0x80000000u ? u & 0x7FFFFFFFu : ~u); };
                rank = order_key(gs > 1 ? value(a) + value(c) : value(a));
            }
            if (lane * VPL >= p.E || (lane & (run - 1)) != 0)
                rank = 0;  // one lane stands for a group
            bool keep = false;
            for (int j = 0; j < p.topk_groups; ++j) {
                const uint32_t best = __reduce_max_sync(kAll, rank);
                const int src = __ffs(__ballot_sync(kAll, rank == best)) - 1;
                rank = lane == src ? 0u : rank;
                keep |= (lane & ~(run - 1)) == src;
            }
            key[0] = keep ? key[0] : 0u;  // a lane whose head cannot be chosen is never asked for the next
        }
        uint32_t my_key = 0;
        int my_src = 0;
        for (int j = 0; j < p.k; ++j) {
            const uint32_t best = __reduce_max_sync(kAll, key[0]);
            const int src = __ffs(__ballot_sync(kAll, key[0] == best)) - 1;
            if (lane == j)
                my_key = best, my_src = src;
            if (lane == src) {
#pragma unroll
                for (int i = 0; i + 1 < VPL; ++i)
                    key[i] = key[i + 1];
                key[VPL - 1] = 0;
            }
        }
        __syncwarp();
        // the expert: the first of lane my_src's with that key, past those that earlier choices of the same key took
        int my_idx = 0;
        {
            const bool mine = lane < p.k;
            const unsigned same = __match_any_sync(kAll, mine ? my_key : 0u) & __match_any_sync(kAll, mine ? my_src : 32 + lane);
            int skip = __popc(same & ((1u << lane) - 1));
            uint32_t their[VPL];
#pragma unroll
            for (int i = 0; i < VPL; ++i)
                their[i] = keys[warp][my_src * VPL + i];
            if (__any_sync(kAll, mine && skip > 0)) {
#pragma unroll
                for (int i = 0; i < VPL; ++i)
                    if (their[i] == my_key && skip-- == 0)
                        my_idx = i;
            } else {
#pragma unroll
                for (int i = VPL - 1; i >= 0; --i)
                    my_idx = their[i] == my_key ? i : my_idx;
            }
            my_idx += my_src * VPL;
        }
        const float my_p = lane < p.k ? row[my_idx] : 0.f;
        float w = my_p;
        if (p.renorm) {
            float total = my_p;
#pragma unroll
            for (int d = 16; d; d >>= 1)
                total += __shfl_xor_sync(kAll, total, d);
            w = total == 0.f ? 0.f : my_p / total;
        }
        if (lane < p.k) {
            p.indices[t * p.k + lane] = my_idx;
            p.weights[t * p.k + lane] = p.scale * w;
        }
    }
}

// Gradient of the sigmoid scores: only the chosen logits count.  A warp takes 32 / KP tokens at once (KP: k rounded up
// to a power of two), one lane per choice, so that the dependent loads of several tokens are in flight together;
// then it writes the tokens' rows as zeros and the chosen entries over them.  Bound by those writes (65536x256 fp32, k = 8:
// 18 us; one token per warp through shared memory 42).
template <bool F32>
__device__ __forceinline__ void store_logit(void *out, int64_t at, float v)
{
    if constexpr (F32)
        static_cast<float *>(out)[at] = v;
    else
        static_cast<__nv_bfloat16 *>(out)[at] = __float2bfloat16_rn(v);
}

template <int KP, bool F32>
__global__ void __launch_bounds__(kRouteThreads) moe_route_backward_sigmoid_kernel(const RouteParams p)
{
    constexpr int kTokens = 32 / KP;
    pdl_wait_and_release();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int j = lane % KP;
    for (int64_t t0 = (blockIdx.x * int64_t{kRouteThreads / 32} + warp) * kTokens; t0 < p.T; t0 += gridDim.x * int64_t{kRouteThreads / 32} * kTokens) {
        const int64_t t = t0 + lane / KP;
        const bool there = t < p.T && j < p.k;
        const int idx = there ? p.idx_in[t * p.k + j] : -1;
        float d = there ? p.scale * p.dweights[t * p.k + j] : 0.f;
        const bool live = idx >= 0 && idx < p.E;
        float pj = 0.f;
        if (live) {
            const int64_t at = t * p.ld + idx;
            pj = sigmoid_exact(F32 ? static_cast<const float *>(p.logits)[at] : __bfloat162float(static_cast<const __nv_bfloat16 *>(p.logits)[at]));
        }
        // the rows' zeros go out while the loads are under way
        for (int n = 0; n < kTokens && t0 + n < p.T; ++n) {
            const int64_t row = (t0 + n) * p.E;
            if (p.vec16) {
                constexpr int kElems = F32 ? 4 : 8;
                for (int e = lane * kElems; e < p.E; e += 32 * kElems)
                    *reinterpret_cast<uint4 *>(static_cast<unsigned char *>(p.dlogits) + (row + e) * (F32 ? 4 : 2)) = make_uint4(0, 0, 0, 0);
            } else {
                for (int e = lane; e < p.E; e += 32)
                    store_logit<F32>(p.dlogits, row + e, 0.f);
            }
        }
        d = live ? d : 0.f;
        if (p.renorm) {
            float total = pj, dot = d * pj;
#pragma unroll
            for (int o = KP / 2; o; o >>= 1) {
                total += __shfl_xor_sync(kAll, total, o);
                dot += __shfl_xor_sync(kAll, dot, o);
            }
            d = total == 0.f || !live ? 0.f : (d - dot / total) / total;
        }
        const int name = live ? idx + (lane / KP) * kRouteMaxE : -1 - lane;
        const unsigned same = __match_any_sync(kAll, name);
        float sum = d;
        if (__any_sync(kAll, (same & (same - 1)) != 0)) {  // an index named twice: its parts in order
            sum = 0.f;
            for (int i = 0; i < KP; ++i) {
                const int other = __shfl_sync(kAll, name, (lane & ~(KP - 1)) + i);
                const float od = __shfl_sync(kAll, d, (lane & ~(KP - 1)) + i);
                sum += other == name ? od : 0.f;
            }
        }
        __syncwarp();  // the zeros come first
        if (live)
            store_logit<F32>(p.dlogits, t * p.E + idx, sum * pj * (1.f - pj));
    }
}

// One warp per token for the softmax scores, which every logit of the row moves.  Bound by latency: a token is a chain of
// loads, reductions over lanes and passes through shared memory (65536x256 fp32, k = 8, renormalised: 49 us where the
// bytes take 20; 490 warp instructions per token, 59% of the issue slots).
template <int VPL, bool F32>
__global__ void __launch_bounds__(kRouteThreads) moe_route_backward_kernel(const RouteParams p)
{
    constexpr float kNegInf = -__builtin_huge_valf();
    __shared__ float rows[kRouteThreads / 32][32 * VPL];
    pdl_wait_and_release();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float *row = rows[warp];
    for (int64_t t = blockIdx.x * int64_t{kRouteThreads / 32} + warp; t < p.T; t += gridDim.x * int64_t{kRouteThreads / 32}) {
        const int idx = lane < p.k ? p.idx_in[t * p.k + lane] : -1;
        const bool live = idx >= 0 && idx < p.E;
        float d = live ? p.scale * p.dweights[t * p.k + lane] : 0.f;
        float l[VPL], s[VPL], pj = 0.f;
        load_row<VPL, F32>(p, t, lane, l, kNegInf);
        softmax_row<VPL>(l, s);
        __syncwarp();
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            row[lane * VPL + i] = s[i];
        __syncwarp();
        if (live)
            pj = row[idx];
        __syncwarp();
        float total = pj, dot = d * pj;
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            total += __shfl_xor_sync(kAll, total, o);
            dot += __shfl_xor_sync(kAll, dot, o);
        }
        if (p.renorm) {
            d = total == 0.f || !live ? 0.f : (d - dot / total) / total;
            dot = d * pj;
#pragma unroll
            for (int o = 16; o; o >>= 1)
                dot += __shfl_xor_sync(kAll, dot, o);
        }
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            row[lane * VPL + i] = 0.f;
        __syncwarp();
        const unsigned same = __match_any_sync(kAll, live ? idx : -1 - lane);
        if (__any_sync(kAll, (same & (same - 1)) != 0)) {
            for (int j = 0; j < p.k; ++j) {  // an index named twice: in order
                if (lane == j && live)
                    row[idx] += d;
                __syncwarp();
            }
        } else if (live) {
            row[idx] = d;
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            s[i] *= row[lane * VPL + i] - dot;
        }
        const int e0 = lane * VPL;
        const int64_t at = t * p.E + e0;
        if (p.vec && e0 < p.E) {
            constexpr int kBytes = VPL * (F32 ? 4 : 2);
            uint32_t w[VPL];
            if constexpr (F32) {
#pragma unroll
                for (int i = 0; i < VPL; ++i)
                    w[i] = __float_as_uint(s[i]);
            } else if constexpr (VPL >= 2) {
#pragma unroll
                for (int i = 0; i < VPL / 2; ++i)
                    w[i] = static_cast<uint32_t>(__bfloat16_as_ushort(__float2bfloat16_rn(s[2 * i]))) |
                           (static_cast<uint32_t>(__bfloat16_as_ushort(__float2bfloat16_rn(s[2 * i + 1]))) << 16);
            }
            unsigned char *dst = static_cast<unsigned char *>(p.dlogits) + at * (F32 ? 4 : 2);
            if constexpr (kBytes >= 16) {
#pragma unroll
                for (int i = 0; i < kBytes / 16; ++i)
                    reinterpret_cast<uint4 *>(dst)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
            } else if constexpr (kBytes == 8) {
                *reinterpret_cast<uint2 *>(dst) = make_uint2(w[0], w[1]);
            } else if constexpr (kBytes == 4) {
                *reinterpret_cast<uint32_t *>(dst) = w[0];
            } else {
                *reinterpret_cast<__nv_bfloat16 *>(dst) = __float2bfloat16_rn(s[0]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < VPL; ++i) {
                if (e0 + i < p.E) {
                    if constexpr (F32)
                        static_cast<float *>(p.dlogits)[at + i] = s[i];
                    else
                        static_cast<__nv_bfloat16 *>(p.dlogits)[at + i] = __float2bfloat16_rn(s[i]);
                }
            }
        }
    }
}

// ---- dispatch plan: a stable counting sort of the choices by expert ------------------------------------

constexpr int kPlanThreads = 256;
constexpr int kPlanWarps = kPlanThreads / 32;

struct PlanParams {
    const int32_t *indices;
    int64_t n;
    int k, E, chunks;
    int64_t chunk;       // choices per CTA, a multiple of kPlanThreads
    int32_t *counts;     // [chunks][E + 1]
    int64_t *offsets;
    int32_t *slots, *tokens;
};

// Choices outside [0, E) form a last bucket E, whose rows follow those of the experts.
__device__ __forceinline__ int plan_bucket(int e, int E) { return e >= 0 && e < E ? e : E; }

// How many choices of each chunk go to each bucket.
__global__ void __launch_bounds__(kPlanThreads) moe_count_kernel(const PlanParams p)
{
    __shared__ int hist[kRouteMaxE + 1];
    pdl_wait_and_release();
    for (int e = threadIdx.x; e <= p.E; e += kPlanThreads)
        hist[e] = 0;
    __syncthreads();
    const int64_t begin = blockIdx.x * p.chunk, end = min(begin + p.chunk, p.n);
    for (int64_t i = begin + threadIdx.x; i < end; i += kPlanThreads)
        atomicAdd(&hist[plan_bucket(p.indices[i], p.E)], 1);
    __syncthreads();
    for (int e = threadIdx.x; e <= p.E; e += kPlanThreads)
        p.counts[static_cast<int64_t>(blockIdx.x) * (p.E + 1) + e] = hist[e];
}

// Ranks the choices of one chunk: first row of each expert (scan over the experts) + the expert's choices in
// the chunks before + in the warps before (each warp owns a contiguous part) + in the lanes before.  Bound by latency:
// 65536 choices over 64 experts 4 + 10 us (count, rank), 128 choices 5 us in one launch.
__global__ void __launch_bounds__(kPlanThreads) moe_rank_kernel(const PlanParams p)
{
    __shared__ int part[kPlanWarps][kRouteMaxE + 1];  // choices per warp, then the warp's next row
    __shared__ int before[kRouteMaxE + 1], total[kRouteMaxE + 1];
    __shared__ int scan[kPlanWarps];
    pdl_wait_and_release();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    for (int e = tid; e < kPlanWarps * (kRouteMaxE + 1); e += kPlanThreads)
        (&part[0][0])[e] = 0;
    __syncthreads();
    const int64_t begin = blockIdx.x * p.chunk, end = min(begin + p.chunk, p.n);
    const int64_t share = p.chunk / kPlanWarps;
    const int64_t w0 = begin + warp * share, w1 = min(w0 + share, end);
    for (int64_t i = w0 + lane; i < w1; i += 32)
        atomicAdd(&part[warp][plan_bucket(p.indices[i], p.E)], 1);
    __syncthreads();
    for (int e = tid; e <= p.E; e += kPlanThreads) {
        int b = 0, a = 0;
        if (p.chunks > 1) {
#pragma unroll 8
            for (int c = 0; c < p.chunks; ++c) {
                const int v = p.counts[static_cast<int64_t>(c) * (p.E + 1) + e];
                b += c < static_cast<int>(blockIdx.x) ? v : 0;
                a += v;
            }
        } else {
            for (int w = 0; w < kPlanWarps; ++w)
                a += part[w][e];
        }
        before[e] = b;
        total[e] = a;
    }
    __syncthreads();
    // exclusive scan of the totals over the experts, two per thread
    const int e0 = 2 * tid;
    const int a0 = e0 < p.E ? total[e0] : 0, a1 = e0 + 1 < p.E ? total[e0 + 1] : 0;
    int incl = a0 + a1;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int v = __shfl_up_sync(kAll, incl, d);
        if (lane >= d)
            incl += v;
    }
    if (lane == 31)
        scan[warp] = incl;
    __syncthreads();
    int base = 0, all = 0;
    for (int w = 0; w < kPlanWarps; ++w) {
        base += w < warp ? scan[w] : 0;
        all += scan[w];
    }
    auto place = [&](int e, int first) {  // first row of bucket e -> each warp's first row in it
        if (blockIdx.x == 0)
            p.offsets[e] = first;
        int at = first + before[e];
        for (int w = 0; w < kPlanWarps; ++w) {
            const int c = part[w][e];
            part[w][e] = at;
            at += c;
        }
    };
    const int first = base + incl - a0 - a1;
    if (e0 < p.E)
        place(e0, first);
    if (e0 + 1 < p.E)
        place(e0 + 1, first + a0);
    if (tid == 0)
        place(p.E, all);
    __syncthreads();
    for (int64_t i0 = w0; i0 < w1; i0 += 32) {
        const int64_t i = i0 + lane;
        const int e = i < w1 ? plan_bucket(p.indices[i], p.E) : -1;
        const unsigned same = __match_any_sync(kAll, e);
        const int rank = __popc(same & ((1u << lane) - 1));
        const int at = e >= 0 ? part[warp][e] + rank : 0;
        __syncwarp();
        if (e >= 0 && rank == 0)
            part[warp][e] += __popc(same);
        __syncwarp();
        if (e >= 0) {
            p.slots[i] = e < p.E ? at : -2 - at;
            p.tokens[at] = e < p.E ? static_cast<int32_t>(i / p.k) : -1;
        }
    }
}

// ---- combination -----------------------------------------------------------------------------------------

constexpr int kCombineThreads = 128;

__device__ __forceinline__ void unpack8(const uint4 &q, float (&v)[8])
{
    v[0] = bf16_lo(q.x), v[1] = bf16_hi(q.x), v[2] = bf16_lo(q.y), v[3] = bf16_hi(q.y);
    v[4] = bf16_lo(q.z), v[5] = bf16_hi(q.z), v[6] = bf16_lo(q.w), v[7] = bf16_hi(q.w);
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    return static_cast<uint32_t>(__bfloat16_as_ushort(__float2bfloat16_rn(lo))) | (static_cast<uint32_t>(__bfloat16_as_ushort(__float2bfloat16_rn(hi))) << 16);
}
__device__ __forceinline__ uint4 pack8(const float (&v)[8])
{
    return make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
}

struct CombineParams {
    const uint4 *y, *dout;
    const int32_t *slots;
    const float *weights;
    int64_t R, T;
    int vecs, k, col_blocks;   // 16-byte vectors per row
    uint4 *out, *dy;
    float *dweights;
};

// A thread owns 8 columns of one token and reads its k rows eight at a time, so that eight loads are in flight.
// Bound by HBM: 8192 tokens of 8 x 7168 161 us, 6.6 TB/s.
__global__ void __launch_bounds__(kCombineThreads) moe_combine_kernel(const CombineParams p)
{
    pdl_wait_and_release();
    for (int64_t b = blockIdx.x; b < p.T * p.col_blocks; b += gridDim.x) {
        const int64_t t = b / p.col_blocks;
        const int c = static_cast<int>(b - t * p.col_blocks) * kCombineThreads + threadIdx.x;
        if (c >= p.vecs)
            continue;
        float acc[8] = {};
        for (int j0 = 0; j0 < p.k; j0 += 8) {
            uint4 q[8];
            float w[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                q[j] = make_uint4(0, 0, 0, 0);
                w[j] = 0.f;
                if (j0 + j < p.k) {
                    const int64_t s = p.slots[t * p.k + j0 + j];
                    if (s >= 0 && s < p.R) {
                        q[j] = p.y[s * p.vecs + c];
                        w[j] = p.weights != nullptr ? p.weights[t * p.k + j0 + j] : 1.f;
                    }
                }
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                float v[8];
                unpack8(q[j], v);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    acc[i] = fmaf(w[j], v[i], acc[i]);
            }
        }
        p.out[t * p.vecs + c] = pack8(acc);
    }
}

constexpr int kCombineBwdThreads = 128;

// One CTA per token: dout is read once per eight choices; the dot products are summed per thread over its
// columns, then over lanes, then over warps, in that order.  Bound by HBM: 8192 tokens of 8 x 7168 307 us, 6.5 TB/s
// (128 threads walk the 896 vectors of a row in seven whole steps; 256 in three and a half took 340).
__global__ void __launch_bounds__(kCombineBwdThreads) moe_combine_backward_kernel(const CombineParams p)
{
    __shared__ float sums[8][kCombineBwdThreads / 32];
    pdl_wait_and_release();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x) {
        for (int j0 = 0; j0 < p.k; j0 += 8) {
            int64_t s[8], o[8];  // the row read, and the row of dy written (-1: none)
            float w[8], dot[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                s[j] = o[j] = -1;
                w[j] = 0.f;
                dot[j] = 0.f;
                if (j0 + j < p.k) {
                    const int64_t v = p.slots[t * p.k + j0 + j];
                    s[j] = v >= 0 && v < p.R ? v : -1;
                    o[j] = v >= 0 ? s[j] : -2 - v < p.R ? -2 - v : -1;
                    if (s[j] >= 0)
                        w[j] = p.weights != nullptr ? p.weights[t * p.k + j0 + j] : 1.f;
                }
            }
            for (int c = tid; c < p.vecs; c += kCombineBwdThreads) {
                float d[8];
                unpack8(p.dout[t * p.vecs + c], d);
                uint4 q[8];
                if (p.dweights != nullptr) {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        q[j] = s[j] >= 0 ? p.y[s[j] * p.vecs + c] : make_uint4(0, 0, 0, 0);
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    if (p.dweights != nullptr && s[j] >= 0) {
                        float v[8];
                        unpack8(q[j], v);
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            dot[j] = fmaf(d[i], v[i], dot[j]);
                    }
                    if (p.dy != nullptr && o[j] >= 0) {
                        float g[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            g[i] = s[j] >= 0 ? w[j] * d[i] : 0.f;
                        p.dy[o[j] * p.vecs + c] = pack8(g);
                    }
                }
            }
            if (p.dweights != nullptr) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
#pragma unroll
                    for (int h = 16; h; h >>= 1)
                        dot[j] += __shfl_xor_sync(kAll, dot[j], h);
                    if (lane == 0)
                        sums[j][warp] = dot[j];
                }
                __syncthreads();
                if (tid < 8 && j0 + tid < p.k) {
                    float a = 0.f;
                    for (int i = 0; i < kCombineBwdThreads / 32; ++i)
                        a += sums[tid][i];
                    p.dweights[t * p.k + j0 + tid] = a;
                }
                __syncthreads();
            }
        }
    }
}

}  // namespace mxfp8
