// C ABI of expert routing, dispatch plan and combination (declarations and contract in include/moe.h):
// host-side checks and launches; the device code is in moe.cuh.
#include <cstdint>

#include "../../include/moe.h"
#include "host.h"
#include "moe.cuh"

namespace {

using namespace mxfp8;

constexpr int64_t kMaxDim = int64_t{1} << 31;
constexpr int64_t kMaxGrid = 1 << 20;

unsigned grid_of(int64_t blocks) { return static_cast<unsigned>(blocks < kMaxGrid ? blocks : kMaxGrid); }

// Choices per CTA of the plan: 1024 up to 152 CTAs' worth (one per SM; a constant, since the workspace's size is asked for
// without a device), then n spread over at most 152 CTAs (each CTA reads every chunk's counts, so their number is bounded).  Measured with 256 / 1024 / 4096 (us): 2048 choices over 64 experts
// 4.0 / 5.1 / 7.8, 65536 over 64 12.2 / 7.7 / 10.6, 65536 over 256 18.7 / 9.1 / 11.7.
int64_t plan_chunk(int64_t n)
{
    const int64_t even = (n + 151) / 152;
    const int64_t chunk = even > 1024 ? even : 1024;
    return (chunk + kPlanThreads - 1) / kPlanThreads * kPlanThreads;
}

int64_t plan_chunks(int64_t n) { return n > 0 ? (n + plan_chunk(n) - 1) / plan_chunk(n) : 1; }

mxfp8_status_t check_route(const void *logits, int type, int64_t T, int64_t E, int64_t ld, const moe_route_config_t *cfg, bool forward)
{
    if (cfg == nullptr)
        return MXFP8_ERR_NULL;
    for (int r : cfg->reserved)
        if (r != 0)
            return MXFP8_ERR_FORMAT;
    if ((type != MXFP4_BF16 && type != MXFP4_F32) || (cfg->score != MOE_SOFTMAX && cfg->score != MOE_SIGMOID) ||
        (cfg->renormalize != 0 && cfg->renormalize != 1))
        return MXFP8_ERR_FORMAT;
    if (T < 0 || T >= kMaxDim || E < 1 || ld < E || ld >= kMaxDim)
        return MXFP8_ERR_SHAPE;
    if (E > MXFP8_MAX_GROUPS)
        return MXFP8_ERR_GROUPS;
    if (cfg->top_k < 1 || cfg->top_k > MOE_MAX_TOPK || cfg->top_k > E)
        return MXFP8_ERR_SHAPE;
    if (forward) {
        if (cfg->num_groups < 1 || E % cfg->num_groups || cfg->topk_groups < 1 || cfg->topk_groups > cfg->num_groups)
            return MXFP8_ERR_GROUPS;
        if (cfg->top_k > E / cfg->num_groups * cfg->topk_groups)
            return MXFP8_ERR_SHAPE;
    }
    if (T > 0 && logits == nullptr)
        return MXFP8_ERR_NULL;
    if (!is_aligned(logits, type == MXFP4_F32 ? 4 : 2) || !is_aligned(cfg->bias, 4))
        return MXFP8_ERR_ALIGN;
    return MXFP8_OK;
}

// Experts per lane: E / 32 rounded up to a power of two.
int lane_experts(int64_t E)
{
    int v = 1;
    while (v * 32 < E)
        v *= 2;
    return v;
}

// Resident CTAs that take tokens in turn (the row set-up is paid once per warp).
template <typename K>
mxfp8_status_t launch_resident(K *kern, KernelSetup &setup, int64_t blocks, const RouteParams &p, cudaStream_t stream)
{
    int device = 0, ctas = 0;
    mxfp8_status_t st;
    if ((st = active_device(&device)) != MXFP8_OK || (st = setup(kern, device, kRouteThreads, 0, &ctas)) != MXFP8_OK)
        return st;
    return launch_serialized(kern, dim3(static_cast<unsigned>(blocks < ctas ? blocks : ctas)), kRouteThreads, 0, 1, stream, p);
}

template <bool BACKWARD, int VPL>
mxfp8_status_t launch_route_vpl(const RouteParams &p, int type, cudaStream_t stream)
{
    static KernelSetup f32, bf16;
    const int64_t blocks = (p.T + kRouteThreads / 32 - 1) / (kRouteThreads / 32);
    if constexpr (BACKWARD)
        return type == MXFP4_F32 ? launch_resident(moe_route_backward_kernel<VPL, true>, f32, blocks, p, stream)
                                 : launch_resident(moe_route_backward_kernel<VPL, false>, bf16, blocks, p, stream);
    else
        return type == MXFP4_F32 ? launch_resident(moe_route_kernel<VPL, true>, f32, blocks, p, stream)
                                 : launch_resident(moe_route_kernel<VPL, false>, bf16, blocks, p, stream);
}

template <bool BACKWARD>
mxfp8_status_t launch_route(const RouteParams &p, int type, int vpl, cudaStream_t stream)
{
    switch (vpl) {
    case 1: return launch_route_vpl<BACKWARD, 1>(p, type, stream);
    case 2: return launch_route_vpl<BACKWARD, 2>(p, type, stream);
    case 4: return launch_route_vpl<BACKWARD, 4>(p, type, stream);
    case 8: return launch_route_vpl<BACKWARD, 8>(p, type, stream);
    default: return launch_route_vpl<BACKWARD, 16>(p, type, stream);
    }
}

template <bool F32>
mxfp8_status_t launch_sigmoid_backward(const RouteParams &p, cudaStream_t stream)
{
    int kp = 1;
    while (kp < p.k)
        kp *= 2;
    const int64_t warps = (p.T * kp + 31) / 32;
    const dim3 grid(grid_of((warps + kRouteThreads / 32 - 1) / (kRouteThreads / 32)));
    auto launch = [&](auto *kern) { return launch_serialized(kern, grid, kRouteThreads, 0, 1, stream, p); };
    switch (kp) {
    case 1: return launch(moe_route_backward_sigmoid_kernel<1, F32>);
    case 2: return launch(moe_route_backward_sigmoid_kernel<2, F32>);
    case 4: return launch(moe_route_backward_sigmoid_kernel<4, F32>);
    case 8: return launch(moe_route_backward_sigmoid_kernel<8, F32>);
    case 16: return launch(moe_route_backward_sigmoid_kernel<16, F32>);
    default: return launch(moe_route_backward_sigmoid_kernel<32, F32>);
    }
}

// Whether every lane's share of a row can be read (and written) in vectors: the row pitch in bytes and the base are
// multiples of the vector, and E of a lane's experts.
bool vector_rows(const void *base, int64_t pitch, int64_t E, int vpl, int type)
{
    const int64_t size = type == MXFP4_F32 ? 4 : 2;
    const int64_t bytes = vpl * size < 16 ? vpl * size : 16;
    return E % vpl == 0 && pitch * size % bytes == 0 && is_aligned(base, static_cast<uintptr_t>(bytes));
}

mxfp8_status_t check_combine(int64_t R, int64_t H, int64_t T, int k)
{
    if (R < 0 || H < 0 || H % 8 || T < 0 || R >= kMaxDim || H >= kMaxDim || T >= kMaxDim || k < 1 || k > MOE_MAX_TOPK)
        return MXFP8_ERR_SHAPE;
    return MXFP8_OK;
}

}  // namespace

extern "C" {

mxfp8_status_t moe_route(const void *logits, int type, int64_t T, int64_t E, int64_t ld, const moe_route_config_t *cfg, int32_t *indices,
                         float *weights, void *stream)
{
    mxfp8_status_t st = check_route(logits, type, T, E, ld, cfg, true);
    if (st != MXFP8_OK)
        return st;
    if (T > 0 && (indices == nullptr || weights == nullptr))
        return MXFP8_ERR_NULL;
    if (!is_aligned(indices, 4) || !is_aligned(weights, 4))
        return MXFP8_ERR_ALIGN;
    int device = 0;
    if ((st = active_device(&device)) != MXFP8_OK)
        return st;
    for (const void *ptr : {logits, static_cast<const void *>(cfg->bias), static_cast<const void *>(indices), static_cast<const void *>(weights)})
        if (!pointer_on_device(ptr, device))
            return MXFP8_ERR_DEVICE;
    if (T == 0)
        return MXFP8_OK;
    const int vpl = lane_experts(E);
    RouteParams p{};
    p.logits = logits;
    p.T = T;
    p.ld = ld;
    p.E = static_cast<int>(E);
    p.k = cfg->top_k;
    p.groups = cfg->num_groups;
    p.topk_groups = cfg->topk_groups;
    p.sigmoid = cfg->score == MOE_SIGMOID;
    p.renorm = cfg->renormalize != 0;
    p.scale = cfg->scale;
    p.bias = cfg->bias;
    p.indices = indices;
    p.weights = weights;
    p.vec = vector_rows(logits, ld, E, vpl, type);
    return launch_route<false>(p, type, vpl, static_cast<cudaStream_t>(stream));
}

mxfp8_status_t moe_route_backward(const void *logits, int type, int64_t T, int64_t E, int64_t ld, const moe_route_config_t *cfg,
                                  const int32_t *indices, const float *dweights, void *dlogits, void *stream)
{
    mxfp8_status_t st = check_route(logits, type, T, E, ld, cfg, false);
    if (st != MXFP8_OK)
        return st;
    if (T > 0 && (indices == nullptr || dweights == nullptr || dlogits == nullptr))
        return MXFP8_ERR_NULL;
    if (!is_aligned(indices, 4) || !is_aligned(dweights, 4) || !is_aligned(dlogits, type == MXFP4_F32 ? 4 : 2))
        return MXFP8_ERR_ALIGN;
    int device = 0;
    if ((st = active_device(&device)) != MXFP8_OK)
        return st;
    for (const void *ptr : {logits, static_cast<const void *>(indices), static_cast<const void *>(dweights), static_cast<const void *>(dlogits)})
        if (!pointer_on_device(ptr, device))
            return MXFP8_ERR_DEVICE;
    if (T == 0)
        return MXFP8_OK;
    const int vpl = lane_experts(E);
    RouteParams p{};
    p.logits = logits;
    p.T = T;
    p.ld = ld;
    p.E = static_cast<int>(E);
    p.k = cfg->top_k;
    p.sigmoid = cfg->score == MOE_SIGMOID;
    p.renorm = cfg->renormalize != 0;
    p.scale = cfg->scale;
    p.idx_in = indices;
    p.dweights = dweights;
    p.dlogits = dlogits;
    p.vec = vector_rows(logits, ld, E, vpl, type) && vector_rows(dlogits, E, E, vpl, type);
    p.vec16 = E * (type == MXFP4_F32 ? 4 : 2) % 16 == 0 && is_aligned(dlogits, 16);
    if (p.sigmoid)
        return type == MXFP4_F32 ? launch_sigmoid_backward<true>(p, static_cast<cudaStream_t>(stream))
                                 : launch_sigmoid_backward<false>(p, static_cast<cudaStream_t>(stream));
    return launch_route<true>(p, type, vpl, static_cast<cudaStream_t>(stream));
}

size_t moe_plan_workspace_bytes(int64_t n, int64_t E)
{
    if (n < 0 || n >= kMaxDim || E < 1 || E > MXFP8_MAX_GROUPS)
        return 0;
    const int64_t chunks = plan_chunks(n);
    return chunks > 1 ? static_cast<size_t>(chunks * (E + 1)) * sizeof(int32_t) : 0;
}

mxfp8_status_t moe_plan(const int32_t *indices, int64_t n, int k, int64_t E, int64_t *offsets, int32_t *slots, int32_t *tokens, void *workspace,
                        void *stream_)
{
    if (n < 0 || n >= kMaxDim || k < 1 || k > MOE_MAX_TOPK || n % k)
        return MXFP8_ERR_SHAPE;
    if (E < 1 || E > MXFP8_MAX_GROUPS || offsets == nullptr)
        return MXFP8_ERR_GROUPS;
    if (n > 0 && (indices == nullptr || slots == nullptr || tokens == nullptr))
        return MXFP8_ERR_NULL;
    if (!is_aligned(indices, 4) || !is_aligned(offsets, 8) || !is_aligned(slots, 4) || !is_aligned(tokens, 4) || !is_aligned(workspace, 4))
        return MXFP8_ERR_ALIGN;
    if (moe_plan_workspace_bytes(n, E) > 0 && workspace == nullptr)
        return MXFP8_ERR_WORKSPACE;
    int device = 0;
    mxfp8_status_t st = active_device(&device);
    if (st != MXFP8_OK)
        return st;
    for (const void *ptr : {static_cast<const void *>(indices), static_cast<const void *>(offsets), static_cast<const void *>(slots),
                            static_cast<const void *>(tokens), static_cast<const void *>(workspace)})
        if (!pointer_on_device(ptr, device))
            return MXFP8_ERR_DEVICE;
    PlanParams p{};
    p.indices = indices;
    p.n = n;
    p.k = k;
    p.E = static_cast<int>(E);
    p.chunk = plan_chunk(n);
    p.chunks = static_cast<int>(plan_chunks(n));
    p.counts = static_cast<int32_t *>(workspace);
    p.offsets = offsets;
    p.slots = slots;
    p.tokens = tokens;
    cudaStream_t stream = static_cast<cudaStream_t>(stream_);
    const dim3 grid(static_cast<unsigned>(p.chunks));
    if (p.chunks > 1 && (st = launch_serialized(moe_count_kernel, grid, kPlanThreads, 0, 1, stream, p)) != MXFP8_OK)
        return st;
    return launch_serialized(moe_rank_kernel, grid, kPlanThreads, 0, 1, stream, p);
}

mxfp8_status_t moe_combine(const void *y, int64_t R, int64_t H, const int32_t *slots, const float *weights, int64_t T, int k, void *out, void *stream)
{
    mxfp8_status_t st = check_combine(R, H, T, k);
    if (st != MXFP8_OK)
        return st;
    const bool empty = T == 0 || H == 0;
    if (!empty && (slots == nullptr || out == nullptr || (y == nullptr && R > 0)))
        return MXFP8_ERR_NULL;
    if (!is_aligned(y, 16) || !is_aligned(out, 16) || !is_aligned(slots, 4) || !is_aligned(weights, 4))
        return MXFP8_ERR_ALIGN;
    int device = 0;
    if ((st = active_device(&device)) != MXFP8_OK)
        return st;
    for (const void *ptr : {y, static_cast<const void *>(slots), static_cast<const void *>(weights), static_cast<const void *>(out)})
        if (!pointer_on_device(ptr, device))
            return MXFP8_ERR_DEVICE;
    if (empty)
        return MXFP8_OK;
    CombineParams p{};
    p.y = static_cast<const uint4 *>(y);
    p.slots = slots;
    p.weights = weights;
    p.R = R;
    p.T = T;
    p.vecs = static_cast<int>(H / 8);
    p.k = k;
    p.col_blocks = (p.vecs + kCombineThreads - 1) / kCombineThreads;
    p.out = static_cast<uint4 *>(out);
    return launch_serialized(moe_combine_kernel, dim3(grid_of(T * p.col_blocks)), kCombineThreads, 0, 1, static_cast<cudaStream_t>(stream), p);
}

mxfp8_status_t moe_combine_backward(const void *dout, const void *y, int64_t R, int64_t H, const int32_t *slots, const float *weights, int64_t T, int k,
                                    void *dy, float *dweights, void *stream)
{
    mxfp8_status_t st = check_combine(R, H, T, k);
    if (st != MXFP8_OK)
        return st;
    if (T > 0 && (slots == nullptr || (dy == nullptr && dweights == nullptr)))
        return MXFP8_ERR_NULL;
    if (T > 0 && H > 0 && (dout == nullptr || (dweights != nullptr && y == nullptr && R > 0)))
        return MXFP8_ERR_NULL;
    if (!is_aligned(dout, 16) || !is_aligned(y, 16) || !is_aligned(dy, 16) || !is_aligned(slots, 4) || !is_aligned(weights, 4) ||
        !is_aligned(dweights, 4))
        return MXFP8_ERR_ALIGN;
    int device = 0;
    if ((st = active_device(&device)) != MXFP8_OK)
        return st;
    for (const void *ptr : {dout, y, static_cast<const void *>(slots), static_cast<const void *>(weights), static_cast<const void *>(dy),
                            static_cast<const void *>(dweights)})
        if (!pointer_on_device(ptr, device))
            return MXFP8_ERR_DEVICE;
    if (T == 0)
        return MXFP8_OK;
    CombineParams p{};
    p.y = static_cast<const uint4 *>(y);
    p.dout = static_cast<const uint4 *>(dout);
    p.slots = slots;
    p.weights = weights;
    p.R = R;
    p.T = T;
    p.vecs = static_cast<int>(H / 8);
    p.k = k;
    p.dy = static_cast<uint4 *>(dy);
    p.dweights = dweights;
    return launch_serialized(moe_combine_backward_kernel, dim3(grid_of(T)), kCombineBwdThreads, 0, 1, static_cast<cudaStream_t>(stream), p);
}

}  // extern "C"
