// C ABI of the norms around a block (declarations and contract in include/block_norm.h): host-side checks and launches;
// the device code is in block_norm.cuh.
#include <cstdint>
#include <mutex>
#include <type_traits>

#include "../../include/block_norm.h"
#include "block_norm.cuh"
#include "host.h"

namespace {

using namespace mxfp8;

constexpr int64_t kMaxDim = int64_t{1} << 31;
constexpr int kMostSmem = 224 * 1024;
constexpr int kRingBytes = 128 * 1024;

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

bool type_ok(int t) { return t == MXFP4_BF16 || t == MXFP4_F32; }

mxfp8_status_t check_config(const block_norm_config_t *cfg, int64_t T, int64_t H)
{
    if (cfg == nullptr)
        return MXFP8_ERR_NULL;
    for (int r : cfg->reserved)
        if (r != 0)
            return MXFP8_ERR_FORMAT;
    if (!type_ok(cfg->y_type) || !type_ok(cfg->h_type) || cfg->gate_kind < BLOCK_GATE_NONE || cfg->gate_kind > BLOCK_GATE_TOKEN)
        return MXFP8_ERR_FORMAT;
    if (T < 0 || T >= kMaxDim || H < 0 || H % 8 || H > BLOCK_NORM_MAX_H)
        return MXFP8_ERR_SHAPE;
    if ((cfg->gate_kind == BLOCK_GATE_NONE) != (cfg->gate == nullptr))
        return MXFP8_ERR_NULL;
    if (!is_aligned(cfg->pre_weight, 16) || !is_aligned(cfg->post_weight, 16) || !is_aligned(cfg->gate, cfg->gate_kind == BLOCK_GATE_TOKEN ? 4 : 16))
        return MXFP8_ERR_ALIGN;
    return MXFP8_OK;
}

bool pitch_ok(const void *p, int64_t ld, int64_t H) { return p == nullptr || (ld >= H && ld % 8 == 0 && ld < kMaxDim); }

// CTAs of a kernel that are resident at once: they depend on a call's threads and shared memory, few pairs of which occur (the
// table holds the last ones, without allocating).
template <auto *KERN>
mxfp8_status_t resident(int device, int threads, int smem, int64_t *ctas)
{
    struct Known {
        int device, threads, smem, per_sm;
    };
    static KernelSetup setup;  // opts the kernel in to the largest size
    static std::mutex mu;
    static Known known[16];
    static unsigned used = 0;
    int all = 0;
    const mxfp8_status_t st = setup(KERN, device, 32, kMostSmem, &all);
    if (st != MXFP8_OK)
        return st;
    std::lock_guard<std::mutex> lock(mu);
    int per_sm = 0;
    for (const Known &k : known)
        if (k.per_sm > 0 && k.device == device && k.threads == threads && k.smem == smem)
            per_sm = k.per_sm;
    if (per_sm == 0) {
        if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, KERN, threads, smem) != cudaSuccess || per_sm < 1) {
            cudaGetLastError();
            return MXFP8_ERR_LAUNCH;
        }
        known[used++ % 16] = {device, threads, smem, per_sm};
    }
    *ctas = static_cast<int64_t>(per_sm) * setup.sms[device];
    return MXFP8_OK;
}

template <auto *KERN, int CTAS>
mxfp8_status_t launch_rows(const NormParams &p, int threads, int smem, int64_t most, int device, cudaStream_t stream, int *rows)
{
    int64_t n = 0;
    const mxfp8_status_t st = resident<KERN>(device, threads, smem, &n);
    if (st != MXFP8_OK)
        return st;
    n = n / CTAS < most ? n / CTAS : most;
    n = n < 1 ? 1 : n < p.T ? n : p.T;
    *rows = static_cast<int>(n);
    return launch_serialized(KERN, dim3(static_cast<unsigned>(n * CTAS)), static_cast<unsigned>(threads), static_cast<size_t>(smem), CTAS, stream, p);
}

// element_bytes: of all inputs of a row, per column.
template <bool YF32, bool HF32, bool BACKWARD>
mxfp8_status_t launch_types(NormParams p, int element_bytes, int device, cudaStream_t stream, int *rows)
{
    const bool shared = p.H > kNormShare;  // two CTAs to a row
    const int vecs = shared ? (p.vecs + 1) / 2 : p.vecs;
    const int v = vecs <= kNormThreads ? 1 : 2;
    const int threads = static_cast<int>(ceil_div(ceil_div(vecs, v), 32) * 32);
    const int64_t most = BACKWARD ? norm_rows(p.H) : int64_t{1} << 20;
    // An SM's CTAs share kRingBytes for their rings (the rest is left to L1), with two stages at least.  With two vectors per
    // thread the weights are kept in shared memory where there is room (forward the factors behind the block alone), and a
    // backward ring, whose CTA has the SM to itself, takes all that is left.
    const int fits = 1024 / threads < 1 ? 1 : 1024 / threads < 8 ? 1024 / threads : 8;
    const int per_sm = BACKWARD && v == 2 ? 1 : fits;
    const int row_bytes = 8 * vecs * element_bytes;
    const int back = p.post != nullptr || p.gate_kind == BLOCK_GATE_CHANNEL ? vecs * 32 : 0, pre = BACKWARD && p.pre != nullptr ? vecs * 32 : 0;
    const bool keep = v == 2 && back + pre > 0 && 2 * row_bytes + back + pre <= kMostSmem / per_sm;
    const int room = BACKWARD && keep ? kMostSmem - back - pre : kRingBytes / per_sm;
    p.stages = room / row_bytes < 2 ? 2 : room / row_bytes < kNormMaxStages ? room / row_bytes : kNormMaxStages;
    const int smem = p.stages * row_bytes + (keep ? back + pre : 0);
    auto run = [&](auto vectors, auto kept, auto ctas) {
        if constexpr (BACKWARD)
            return launch_rows<block_norm_backward_kernel<YF32, HF32, vectors, kept, ctas>, ctas>(p, threads, smem, most, device, stream, rows);
        else
            return launch_rows<block_norm_kernel<YF32, HF32, vectors, kept, ctas>, ctas>(p, threads, smem, most, device, stream, rows);
    };
    using One = std::integral_constant<int, 1>;
    using Two = std::integral_constant<int, 2>;
    static_assert(kNormShare / 2 >= 8 * kNormThreads, "half of a shared row is two vectors per thread");
    if (shared)
        return keep ? run(Two{}, std::true_type{}, Two{}) : run(Two{}, std::false_type{}, Two{});
    if (v == 1)
        return run(One{}, std::false_type{}, One{});
    return keep ? run(Two{}, std::true_type{}, One{}) : run(Two{}, std::false_type{}, One{});
}

template <bool BACKWARD>
mxfp8_status_t launch(const NormParams &p, const block_norm_config_t *cfg, int element_bytes, int device, cudaStream_t stream, int *rows)
{
    const bool y32 = cfg->y_type == MXFP4_F32, h32 = cfg->h_type == MXFP4_F32;
    return y32 ? (h32 ? launch_types<true, true, BACKWARD>(p, element_bytes, device, stream, rows) : launch_types<true, false, BACKWARD>(p, element_bytes, device, stream, rows))
               : (h32 ? launch_types<false, true, BACKWARD>(p, element_bytes, device, stream, rows) : launch_types<false, false, BACKWARD>(p, element_bytes, device, stream, rows));
}

NormParams params(const block_norm_config_t *cfg, int64_t T, int64_t H)
{
    NormParams p{};
    p.T = T;
    p.H = static_cast<int>(H);
    p.vecs = static_cast<int>(H / 8);
    p.gate_kind = cfg->gate_kind;
    p.scale = cfg->scale;
    p.eps = cfg->eps;
    p.pre = cfg->pre_weight;
    p.post = cfg->post_weight;
    p.gate = cfg->gate;
    return p;
}

}  // namespace

extern "C" {

mxfp8_status_t block_norm(const block_norm_config_t *cfg, int64_t T, int64_t H, const void *y, int64_t ldy, const void *h, int64_t ldh, void *h_out, void *x,
                          void *stream)
{
    mxfp8_status_t st = check_config(cfg, T, H);
    if (st != MXFP8_OK)
        return st;
    if (!pitch_ok(y, ldy, H) || !pitch_ok(h, ldh, H))
        return MXFP8_ERR_SHAPE;
    if (T > 0 && H > 0) {
        if (h == nullptr || (h_out == nullptr && x == nullptr) || (x == nullptr) != (cfg->pre_weight == nullptr) ||
            (y == nullptr && (cfg->post_weight != nullptr || cfg->gate != nullptr)))
            return MXFP8_ERR_NULL;
    }
    if (!is_aligned(y, 16) || !is_aligned(h, 16) || !is_aligned(h_out, 16) || !is_aligned(x, 16))
        return MXFP8_ERR_ALIGN;
    int device = 0;
    if ((st = active_device(&device)) != MXFP8_OK)
        return st;
    for (const void *ptr : {y, h, static_cast<const void *>(h_out), static_cast<const void *>(x), static_cast<const void *>(cfg->pre_weight),
                            static_cast<const void *>(cfg->post_weight), static_cast<const void *>(cfg->gate)})
        if (!pointer_on_device(ptr, device))
            return MXFP8_ERR_DEVICE;
    if (T == 0 || H == 0)
        return MXFP8_OK;
    NormParams p = params(cfg, T, H);
    p.y = y;
    p.ldy = ldy;
    p.h = h;
    p.ldh = ldh;
    p.h_out = h_out;
    p.x = x;
    if ((p.fault = fault_word_address(device)) == nullptr)
        return MXFP8_ERR_DEVICE;
    const int hs = cfg->h_type == MXFP4_F32 ? 4 : 2, ys = cfg->y_type == MXFP4_F32 ? 4 : 2;
    int rows = 0;
    return launch<false>(p, cfg, hs + (y != nullptr ? ys : 0), device, static_cast<cudaStream_t>(stream), &rows);
}

size_t block_norm_backward_workspace_bytes(int64_t T, int64_t H)
{
    if (T <= 0 || T >= kMaxDim || H <= 0 || H > BLOCK_NORM_MAX_H)
        return 0;
    return static_cast<size_t>(T < norm_rows(H) ? T : norm_rows(H)) * 2 * static_cast<size_t>(H) * sizeof(float);
}

mxfp8_status_t block_norm_backward(const block_norm_config_t *cfg, int64_t T, int64_t H, const void *dh_out, int64_t lddh, const void *dx, int64_t lddx,
                                   const void *y, int64_t ldy, const void *h_out, int64_t ldh, void *dh, void *dy, float *dpre, float *dpost,
                                   float *dgate, void *workspace, void *stream_)
{
    mxfp8_status_t st = check_config(cfg, T, H);
    if (st != MXFP8_OK)
        return st;
    if (!pitch_ok(dh_out, lddh, H) || !pitch_ok(dx, lddx, H) || !pitch_ok(y, ldy, H) || !pitch_ok(h_out, ldh, H))
        return MXFP8_ERR_SHAPE;
    if ((dpost != nullptr && cfg->post_weight == nullptr) || (dgate != nullptr && cfg->gate == nullptr) || (dpre != nullptr && cfg->pre_weight == nullptr))
        return MXFP8_ERR_NULL;
    if (T > 0 && H > 0) {
        const bool needs_y = (cfg->post_weight != nullptr && (dy != nullptr || dpost != nullptr)) || dgate != nullptr;
        if ((dh_out == nullptr && dx == nullptr) || (dx != nullptr && (cfg->pre_weight == nullptr || h_out == nullptr)) || (needs_y && y == nullptr) ||
            (dh == nullptr && dy == nullptr && dpre == nullptr && dpost == nullptr && dgate == nullptr))
            return MXFP8_ERR_NULL;
        if ((dpre != nullptr || dpost != nullptr || dgate != nullptr) && workspace == nullptr)
            return MXFP8_ERR_WORKSPACE;
    }
    if (!is_aligned(dh_out, 16) || !is_aligned(dx, 16) || !is_aligned(y, 16) || !is_aligned(h_out, 16) || !is_aligned(dh, 16) || !is_aligned(dy, 16) ||
        !is_aligned(dpre, 4) || !is_aligned(dpost, 4) || !is_aligned(dgate, 4) || !is_aligned(workspace, 16))
        return MXFP8_ERR_ALIGN;
    int device = 0;
    if ((st = active_device(&device)) != MXFP8_OK)
        return st;
    for (const void *ptr : {dh_out, dx, y, h_out, static_cast<const void *>(dh), static_cast<const void *>(dy), static_cast<const void *>(dpre),
                            static_cast<const void *>(dpost), static_cast<const void *>(dgate), static_cast<const void *>(workspace),
                            static_cast<const void *>(cfg->pre_weight), static_cast<const void *>(cfg->post_weight),
                            static_cast<const void *>(cfg->gate)})
        if (!pointer_on_device(ptr, device))
            return MXFP8_ERR_DEVICE;
    cudaStream_t stream = static_cast<cudaStream_t>(stream_);
    auto zero = [&](float *out, int64_t n) {
        if (out == nullptr || n == 0 || cudaMemsetAsync(out, 0, static_cast<size_t>(n) * sizeof(float), stream) == cudaSuccess)
            return MXFP8_OK;
        cudaGetLastError();
        return MXFP8_ERR_LAUNCH;
    };
    const bool per_token = cfg->gate_kind == BLOCK_GATE_TOKEN;
    if (H == 0)  // sums over no columns
        return zero(per_token ? dgate : nullptr, T);
    if (T == 0) {  // sums over no rows
        for (float *out : {dpre, dpost, per_token ? nullptr : dgate})
            if ((st = zero(out, H)) != MXFP8_OK)
                return st;
        return MXFP8_OK;
    }
    NormParams p = params(cfg, T, H);
    p.y = y;
    p.ldy = ldy;
    p.h = h_out;
    p.ldh = ldh;
    p.dh_out = dh_out;
    p.lddh = lddh;
    p.dx = dx;
    p.lddx = lddx;
    p.dh = dh;
    p.dy = dy;
    p.dpre = dpre;
    p.dpost = dpost;
    p.dgate = dgate;
    const bool sums = dpre != nullptr || dpost != nullptr || (dgate != nullptr && cfg->gate_kind == BLOCK_GATE_CHANNEL);
    p.partial = sums ? static_cast<float *>(workspace) : nullptr;
    if ((p.fault = fault_word_address(device)) == nullptr)
        return MXFP8_ERR_DEVICE;
    const int hs = cfg->h_type == MXFP4_F32 ? 4 : 2, ys = cfg->y_type == MXFP4_F32 ? 4 : 2;
    const int element_bytes = (y != nullptr ? ys : 0) + (dx != nullptr ? hs + 2 : 0) + (dh_out != nullptr ? hs : 0);
    int rows = 0;
    if ((st = launch<true>(p, cfg, element_bytes, device, stream, &rows)) != MXFP8_OK || !sums)
        return st;
    return launch_serialized(block_norm_reduce_kernel, dim3(static_cast<unsigned>(ceil_div(2 * H, 32))),
                             rows > kNormReduceCtas ? kNormReduceMany : kNormReduceFew, 0, 1, stream, p, rows);
}

}  // extern "C"
