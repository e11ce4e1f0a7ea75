// C ABI of the MXFP4 cast and products (declarations and contract in include/mxfp4.h): host-side checks,
// tensor maps and launches; the device code is in mxfp4_cast.cuh and mxfp4_gemm.cuh.
#include <atomic>
#include <cstdint>
#include <mutex>

#include "../../include/mxfp4.h"
#include "host.h"
#include "mxfp4_cast.cuh"
#include "mxfp4_gemm.cuh"
#include "mxfp4_pair.cuh"
#include "mxfp4_split.cuh"

namespace {

using namespace mxfp8;

constexpr int64_t kMaxDim = int64_t{1} << 31;
constexpr int64_t kLongRow = int64_t{1} << 29;  // columns whose scales' offsets pass 31 bits

// Products by CTA pairs need more rows than one 128-row tile and tiles for most of the 76 pairs; experts' products that
// many rows per expert on average.  Measured (us, pairs / the other kernel), dense rows x N x K: 256x8192x8192 (32 tiles)
// 14.7 / 12.5, 1024x4096x4096 (64) 10.5 / 10.7, 512x8192x8192 (64) 15.5 / 17.3, 128x28672x8192 (one row tile) 28 / 25,
// 192x28672x8192 (112) 30 / 35; 64 experts of 2048 x 7168 with 64, 96, 128, 192, 256 rows: 95 / 87, 98 / 90, 101 / 107,
// 107 / 139, 131 / 177.
constexpr int64_t kPairMinTiles = 64;
constexpr int64_t kPairMinGroupRows = 128;

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

bool type_ok(int t) { return t == MXFP4_BF16 || t == MXFP4_F32; }

mxfp8_status_t sm_count(int device, int *sms)
{
    static std::atomic<int> cached[kMaxDevices];
    if (device < 0 || device >= kMaxDevices)
        return MXFP8_ERR_DEVICE;
    int n = cached[device].load(std::memory_order_relaxed);
    if (n == 0) {
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, device) != cudaSuccess) {
            cudaGetLastError();
            return MXFP8_ERR_DEVICE;
        }
        cached[device].store(n, std::memory_order_relaxed);
    }
    *sms = n;
    return MXFP8_OK;
}

template <bool F32, bool COL, bool GROUPED>
mxfp8_status_t launch_cast_as(const CastParams &p, int64_t tiles, int device, cudaStream_t stream)
{
    static KernelSetup setup;
    constexpr int smem = kCastSmem;
    int ctas = 0;
    const mxfp8_status_t st = setup(mxfp4_cast_kernel<F32, COL, GROUPED>, device, kCastThreads, smem, &ctas);
    if (st != MXFP8_OK)
        return st;
    const unsigned grid = static_cast<unsigned>(tiles < ctas ? tiles : ctas);
    return launch_serialized(mxfp4_cast_kernel<F32, COL, GROUPED>, dim3(grid), kCastThreads, smem, 1, stream, p);
}

mxfp8_status_t code_map(CUtensorMap *map, const void *codes, int64_t rows, int64_t row_bytes, int box_rows)
{
    PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
    if (enc == nullptr)
        return MXFP8_ERR_DEVICE;
    cuuint64_t dims[2] = {static_cast<cuuint64_t>(row_bytes), static_cast<cuuint64_t>(rows)};
    cuuint64_t strides[1] = {static_cast<cuuint64_t>(row_bytes)};
    cuuint32_t box[2] = {128, static_cast<cuuint32_t>(box_rows)};
    cuuint32_t estr[2] = {1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(codes), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? MXFP8_OK
               : MXFP8_ERR_LAUNCH;
}

template <bool F32>
mxfp8_status_t launch_group_as(const CUtensorMap &pm, const CUtensorMap &qm, const GemmParams &p, int64_t tiles, int device, cudaStream_t stream)
{
    static KernelSetup setup;
    constexpr int smem = kGroupSmem + kEpiBytes<F32>;
    int ctas = 0;
    const mxfp8_status_t st = setup(mxfp4_group_kernel<F32>, device, kGemmThreads, smem, &ctas);
    if (st != MXFP8_OK)
        return st;
    const unsigned grid = static_cast<unsigned>(tiles < ctas ? tiles : ctas);
    return launch_serialized(mxfp4_group_kernel<F32>, dim3(grid), kGemmThreads, smem, 1, stream, pm, qm, p);
}

// The scale plane as rows of 512-byte tiles, in boxes of 1024 bytes (one stage) x box_rows tile rows.
mxfp8_status_t scale_map(CUtensorMap *map, const void *scale, int64_t tile_rows, int64_t kc, int box_rows)
{
    PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
    if (enc == nullptr)
        return MXFP8_ERR_DEVICE;
    cuuint64_t dims[2] = {static_cast<cuuint64_t>(kc) * 128, static_cast<cuuint64_t>(tile_rows)};
    cuuint64_t strides[1] = {static_cast<cuuint64_t>(kc) * 512};
    cuuint32_t box[2] = {256, static_cast<cuuint32_t>(box_rows)};
    cuuint32_t estr[2] = {1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, const_cast<void *>(scale), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? MXFP8_OK
               : MXFP8_ERR_LAUNCH;
}

// The pair kernel.  p_rows: rows of P's map (all experts); plane rows likewise.
template <bool F32, bool GROUPED>
mxfp8_status_t launch_pair_as(const GemmParams &p, const void *p_codes, int64_t p_rows, int64_t p_plane_rows, const void *q_codes,
                              int64_t q_plane_rows, int64_t row_bytes, int64_t tiles, int device, cudaStream_t stream)
{
    static KernelSetup setup;
    constexpr int smem = kPairSmem + kEpiBytes<F32>;
    int ctas = 0;
    mxfp8_status_t st = setup(mxfp4_pair_kernel<F32, GROUPED>, device, kGemmThreads, smem, &ctas);
    if (st != MXFP8_OK)
        return st;
    CUtensorMap pm, qm, qpm, psm, qsm;
    if ((st = code_map(&pm, p_codes, p_rows, row_bytes, 128)) != MXFP8_OK || (st = code_map(&qm, q_codes, p.Q, row_bytes, 128)) != MXFP8_OK ||
        (st = code_map(&qpm, q_codes, p.Q, row_bytes, 32)) != MXFP8_OK || (st = scale_map(&psm, p.p_scale, p_plane_rows, p.kc, 1)) != MXFP8_OK || (st = scale_map(&qsm, p.q_scale, q_plane_rows, p.kc, 2)) != MXFP8_OK)
        return st;
    const int64_t pairs = tiles < ctas / 2 ? tiles : ctas / 2;
    return launch_serialized(mxfp4_pair_kernel<F32, GROUPED>, dim3(static_cast<unsigned>(2 * pairs)), kGemmThreads, smem, 2, stream, pm, qm, qpm,
                             psm, qsm, p);
}

// The kernel for few tiles.  S CTAs share a tile's K: the most (1, 2, 4, 8) for which all CTAs are resident at once, two
// per SM where the weights' bytes are the time (64 rows or fewer), one per SM above.  Measured (us, S = 1 / 2 / 4 / 8,
// rows x N x K): 1x4096x4096 13.0 / 12.9 / 12.9 / 10.9, 16x8192x28672 50 / 40 / 33 / 40, 100x512x16384 31 / 23 / 17 / 15;
// where they are not all resident S = 1 is fastest (1x28672x8192 33 / 38 / 42 / 52, 333x4096x4096 15 / 17 / 23 / 33).
template <int QROWS, int STAGES, bool F32>
mxfp8_status_t launch_split_as(const GemmParams &p, const CUtensorMap &pm, const CUtensorMap &qm, int64_t tiles, int splits, int device,
                               cudaStream_t stream)
{
    using Shape = SplitShape<QROWS, STAGES>;
    static KernelSetup setup;
    static_assert(Shape::kStage * STAGES >= QROWS * kGemmRows * 4 && Shape::kStage * STAGES >= kEpiBytes<F32>,
                  "partial sums and the epilogue's buffers fit the stages");
    int ctas = 0;
    const mxfp8_status_t st = setup(mxfp4_split_kernel<QROWS, STAGES, F32>, device, kGemmThreads, Shape::kSmem, &ctas);
    if (st != MXFP8_OK)
        return st;
    return launch_serialized(mxfp4_split_kernel<QROWS, STAGES, F32>, dim3(static_cast<unsigned>(tiles * splits)), kGemmThreads, Shape::kSmem, splits,
                             stream, pm, qm, p, splits);
}

template <bool F32>
mxfp8_status_t launch_split(const GemmParams &p_, const void *p_codes, const void *q_codes, int64_t row_bytes, int device, cudaStream_t stream)
{
    GemmParams p = p_;
    // small boxes for few tokens: rows past Q cost the copy engine as much as others (1x8192x28672: 23.9 us in boxes of 32
    // rows, 22.0 in boxes of 16)
    p.q_box = p.Q <= 16 ? 16 : p.Q <= 32 ? 32 : 128;
    CUtensorMap pm, qm;
    mxfp8_status_t st;
    if ((st = code_map(&pm, p_codes, p.P, row_bytes, kGemmRows)) != MXFP8_OK || (st = code_map(&qm, q_codes, p.Q, row_bytes, p.q_box)) != MXFP8_OK)
        return st;
    int sms = 0;
    if ((st = sm_count(device, &sms)) != MXFP8_OK)
        return st;
    const int64_t tiles = static_cast<int64_t>(p.p_tiles) * p.q_tiles, room = p.Q <= 64 ? 2 * sms : sms;
    int splits = 1;
    while (splits < 8 && tiles * splits * 2 <= room && splits * 2 <= p.k_iters)
        splits *= 2;
    if (p.Q <= 32)
        return launch_split_as<32, 4, F32>(p, pm, qm, tiles, splits, device, stream);
    // one CTA per SM is all there is: more stages in its shared memory
    if (tiles * splits <= sms)
        return launch_split_as<128, 5, F32>(p, pm, qm, tiles, splits, device, stream);
    return launch_split_as<128, 3, F32>(p, pm, qm, tiles, splits, device, stream);
}

// Checks and parameters that both products share.  Q: the tokens' rows; P: the weights' rows (per expert).
mxfp8_status_t gemm_params(GemmParams *p, const void *q_codes, const void *q_scale, int64_t Q, const void *p_codes, const void *p_scale, int64_t P,
                           int64_t K, void *out, int out_type, int64_t ldo)
{
    if (!type_ok(out_type))
        return MXFP8_ERR_FORMAT;
    if (Q < 0 || P < 0 || K < 0 || Q >= kMaxDim || P >= kMaxDim || K >= kMaxDim || ldo < P)
        return MXFP8_ERR_SHAPE;
    const int64_t tiles = ceil_div(P, kGemmRows) * ceil_div(Q, 128);
    if (tiles >= kMaxDim)
        return MXFP8_ERR_SHAPE;
    if (Q > 0 && P > 0) {
        if (out == nullptr || (K > 0 && (q_codes == nullptr || q_scale == nullptr || p_codes == nullptr || p_scale == nullptr)))
            return MXFP8_ERR_NULL;
    }
    if (!is_aligned(q_codes, 16) || !is_aligned(q_scale, 16) || !is_aligned(p_codes, 16) || !is_aligned(p_scale, 16) ||
        !is_aligned(out, out_type == MXFP4_F32 ? 4 : 2))
        return MXFP8_ERR_ALIGN;
    const int64_t pad = ceil_div(K, 32) * 32;
    *p = GemmParams{};
    p->p_scale = static_cast<const uint8_t *>(p_scale);
    p->q_scale = static_cast<const uint8_t *>(q_scale);
    p->P = P;
    p->Q = Q;
    p->kc = static_cast<int>(ceil_div(K, 128));
    p->k_iters = static_cast<int>(ceil_div(K, 256));
    p->k64 = static_cast<int>(ceil_div(pad, 64));
    p->p_tiles = static_cast<int>(ceil_div(P, kGemmRows));
    p->p_planes = p->p_tiles;
    p->q_tiles = static_cast<int>(ceil_div(Q, 128));
    p->out = out;
    p->ldo = ldo;
    const int size = out_type == MXFP4_F32 ? 4 : 2;
    p->vec_out = is_aligned(out, 16) && ldo * size % 16 == 0 && P * size % 16 == 0;
    return MXFP8_OK;
}

mxfp8_status_t zero_rows(void *out, int64_t rows, int64_t cols, int64_t ld, int type, cudaStream_t stream)
{
    const size_t e = type == MXFP4_F32 ? 4 : 2;
    if (cudaMemset2DAsync(out, static_cast<size_t>(ld) * e, 0, static_cast<size_t>(cols) * e, static_cast<size_t>(rows), stream) != cudaSuccess) {
        cudaGetLastError();
        return MXFP8_ERR_LAUNCH;
    }
    return MXFP8_OK;
}

}  // namespace

extern "C" {

size_t mxfp4_row_bytes(int64_t cols) { return cols <= 0 ? 0 : static_cast<size_t>(ceil_div(cols, 32)) * 16; }

size_t mxfp4_scale_bytes(int64_t rows, int64_t cols)
{
    return rows <= 0 || cols <= 0 ? 0 : static_cast<size_t>(ceil_div(rows, 128)) * static_cast<size_t>(ceil_div(cols, 128)) * 512;
}

size_t mxfp4_grouped_scale_bytes(int64_t total_rows, int64_t cols, int num_groups)
{
    if (total_rows <= 0 || cols <= 0 || num_groups < 1)
        return 0;
    const int64_t tiles = total_rows / 128 + (num_groups < total_rows ? num_groups : total_rows);
    return static_cast<size_t>(tiles) * static_cast<size_t>(ceil_div(cols, 128)) * 512;
}

mxfp8_status_t mxfp4_quantize(const void *x, int x_type, int64_t M, int64_t N, int64_t ldx, void *out_row, void *scale_row, void *out_col,
                              void *scale_col, const float *noop, void *stream_)
{
    if (!type_ok(x_type))
        return MXFP8_ERR_FORMAT;
    if (M < 0 || N < 0 || N % 8 || ldx % 8 || ldx < N || M >= kMaxDim || N >= kMaxDim || ldx >= kMaxDim)
        return MXFP8_ERR_SHAPE;
    const int64_t tiles = ceil_div(M, kCastTile) * ceil_div(N, kCastTile);
    if (tiles >= kMaxDim - (int64_t{1} << 20))
        return MXFP8_ERR_SHAPE;
    if (tiles > 0) {
        if (x == nullptr || (out_row == nullptr) != (scale_row == nullptr) || (out_col == nullptr) != (scale_col == nullptr) ||
            (out_row == nullptr && out_col == nullptr))
            return MXFP8_ERR_NULL;
    }
    if (!is_aligned(x, 16) || !is_aligned(out_row, 16) || !is_aligned(out_col, 16) || !is_aligned(scale_row, 4) || !is_aligned(scale_col, 4) ||
        !is_aligned(noop, 4))
        return MXFP8_ERR_ALIGN;
    int device = 0;
    mxfp8_status_t st = active_device(&device);
    if (st != MXFP8_OK)
        return st;
    for (const void *ptr : {x, static_cast<const void *>(out_row), static_cast<const void *>(scale_row), static_cast<const void *>(out_col),
                            static_cast<const void *>(scale_col), static_cast<const void *>(noop)})
        if (!pointer_on_device(ptr, device))
            return MXFP8_ERR_DEVICE;
    if (tiles == 0)
        return MXFP8_OK;
    CastParams p{};
    p.x = x;
    p.M = M;
    p.N = N;
    p.ldx = ldx;
    p.T = M;
    p.out_row = static_cast<uint8_t *>(out_row);
    p.scale_row = static_cast<uint8_t *>(scale_row);
    p.out_col = static_cast<uint8_t *>(out_col);
    p.scale_col = static_cast<uint8_t *>(scale_col);
    p.noop = noop;
    p.row_tiles = static_cast<int>(ceil_div(M, kCastTile));
    p.col_tiles = static_cast<int>(ceil_div(N, kCastTile));
    p.row_pitch = ceil_div(N, 32) * 16;
    p.col_pitch = ceil_div(M, 32) * 16;
    cudaStream_t stream = static_cast<cudaStream_t>(stream_);
    const bool col = out_col != nullptr;
    if (x_type == MXFP4_F32)
        return col ? launch_cast_as<true, true, false>(p, tiles, device, stream) : launch_cast_as<true, false, false>(p, tiles, device, stream);
    return col ? launch_cast_as<false, true, false>(p, tiles, device, stream) : launch_cast_as<false, false, false>(p, tiles, device, stream);
}

// The two-step form's cast of the T rows: codes, then (16-byte aligned) the plane.
size_t mxfp4_quantize_grouped_workspace_bytes(int64_t T, int64_t N, int64_t total_rows)
{
    if (T <= 0 || N <= 0 || total_rows <= T)
        return 0;
    return static_cast<size_t>(T) * mxfp4_row_bytes(N) + mxfp4_scale_bytes(T, N);
}

mxfp8_status_t mxfp4_quantize_grouped(const void *x, int x_type, int64_t T, int64_t N, int64_t ldx, const int32_t *rows, int64_t total_rows,
                                      int num_groups, const int64_t *offsets, void *out, void *scale, int *err_flag, void *workspace, void *stream_)
{
    if (!type_ok(x_type))
        return MXFP8_ERR_FORMAT;
    if (T < 0 || total_rows < 0 || N < 0 || N % 8 || ldx % 8 || ldx < N || T >= kMaxDim || total_rows >= kMaxDim || N >= kMaxDim ||
        ldx >= kMaxDim || (rows == nullptr && total_rows > T))
        return MXFP8_ERR_SHAPE;
    if (num_groups < 1 || num_groups > MXFP8_MAX_GROUPS || offsets == nullptr)
        return MXFP8_ERR_GROUPS;
    const int64_t col_tiles = ceil_div(N, kCastTile);
    const int64_t bound = (total_rows / kCastTile + num_groups) * col_tiles;
    if (bound >= kMaxDim - (int64_t{1} << 20))
        return MXFP8_ERR_SHAPE;
    const bool empty = total_rows == 0 || N == 0;
    if (!empty && (out == nullptr || scale == nullptr || (x == nullptr && T > 0)))
        return MXFP8_ERR_NULL;
    if (!is_aligned(x, 16) || !is_aligned(out, 16) || !is_aligned(scale, 4) || !is_aligned(rows, 4) || !is_aligned(offsets, 8) ||
        !is_aligned(err_flag, 4) || !is_aligned(workspace, 16))
        return MXFP8_ERR_ALIGN;
    int device = 0;
    mxfp8_status_t st = active_device(&device);
    if (st != MXFP8_OK)
        return st;
    for (const void *ptr : {x, static_cast<const void *>(rows), static_cast<const void *>(workspace), static_cast<const void *>(offsets), static_cast<const void *>(out),
                            static_cast<const void *>(scale), static_cast<const void *>(err_flag)})
        if (!pointer_on_device(ptr, device))
            return MXFP8_ERR_DEVICE;
    if (empty)
        return MXFP8_OK;
    CastParams p{};
    p.x = x;
    p.M = total_rows;
    p.N = N;
    p.ldx = ldx;
    p.T = T;
    p.out_row = static_cast<uint8_t *>(out);
    p.scale_row = static_cast<uint8_t *>(scale);
    p.col_tiles = static_cast<int>(col_tiles);
    p.row_pitch = ceil_div(N, 32) * 16;
    p.rows = rows;
    p.offsets = offsets;
    p.err_flag = err_flag;
    p.num_groups = num_groups;
    cudaStream_t stream = static_cast<cudaStream_t>(stream_);
    if (rows != nullptr && workspace != nullptr && total_rows > T && T > 0) {
        // more rows than tokens: cast every token once, then gather
        auto *codes = static_cast<uint8_t *>(workspace), *plane = codes + T * p.row_pitch;
        if ((st = mxfp4_quantize(x, x_type, T, N, ldx, codes, plane, nullptr, nullptr, nullptr, stream_)) != MXFP8_OK)
            return st;
        GatherParams g{};
        g.codes = codes;
        g.scale = plane;
        g.T = T;
        g.R = total_rows;
        g.N = N;
        g.pitch = p.row_pitch;
        g.col_tiles = p.col_tiles;
        g.rows = rows;
        g.offsets = offsets;
        g.num_groups = num_groups;
        g.out = p.out_row;
        g.out_scale = p.scale_row;
        g.err_flag = err_flag;
        static KernelSetup setup;
        int ctas = 0;
        if ((st = setup(mxfp4_gather_kernel, device, 256, 0, &ctas)) != MXFP8_OK)
            return st;
        const int64_t units = (total_rows / kCastTile + num_groups) * ceil_div(col_tiles, kGatherTiles);
        return launch_serialized(mxfp4_gather_kernel, dim3(static_cast<unsigned>(units < ctas ? units : ctas)), 256, 0, 1, stream, g);
    }
    return x_type == MXFP4_F32 ? launch_cast_as<true, false, true>(p, bound, device, stream)
                               : launch_cast_as<false, false, true>(p, bound, device, stream);
}

mxfp8_status_t mxfp4_dequantize(const void *codes, const void *scale, int64_t rows, int64_t cols, void *out, int out_type, void *stream_)
{
    if (!type_ok(out_type))
        return MXFP8_ERR_FORMAT;
    if (rows < 0 || cols < 0 || rows >= kMaxDim || cols >= kMaxDim)
        return MXFP8_ERR_SHAPE;
    const bool empty = rows == 0 || cols == 0;
    if (!empty && (codes == nullptr || scale == nullptr || out == nullptr))
        return MXFP8_ERR_NULL;
    if (!is_aligned(codes, 16) || !is_aligned(out, 16))
        return MXFP8_ERR_ALIGN;
    int device = 0;
    mxfp8_status_t st = active_device(&device);
    if (st != MXFP8_OK)
        return st;
    if (!pointer_on_device(codes, device) || !pointer_on_device(scale, device) || !pointer_on_device(out, device))
        return MXFP8_ERR_DEVICE;
    if (empty)
        return MXFP8_OK;
    const int per = out_type == MXFP4_F32 ? 4 : 8;  // elements of a 16-byte vector
    const bool vec = cols % per == 0;
    const int64_t vecs = ceil_div(cols, per) + (vec ? 0 : 1);  // a row that starts off a vector touches one more
    const int64_t groups = ceil_div(rows, vec ? kDecodeRows<true> : kDecodeRows<false>);
    // a row's vectors over blocks of up to 256 threads, as evenly as whole warps allow
    const unsigned threads = static_cast<unsigned>(ceil_div(ceil_div(vecs, ceil_div(vecs, 256)), 32) * 32);
    const dim3 grid(static_cast<unsigned>(ceil_div(vecs, threads)), static_cast<unsigned>(groups < 65535 ? groups : 65535));
    cudaStream_t stream = static_cast<cudaStream_t>(stream_);
    const auto *c = static_cast<const uint8_t *>(codes);
    const auto *s = static_cast<const uint8_t *>(scale);
    const int64_t pitch = ceil_div(cols, 32) * 16, col_tiles = ceil_div(cols, 128);
    auto launch = [&](auto *kern) { return launch_serialized(kern, grid, threads, 0, 1, stream, c, s, rows, cols, pitch, col_tiles, out); };
    if (cols >= kLongRow) {
        if (!vec)
            return out_type == MXFP4_F32 ? launch(mxfp4_decode_kernel<true, false, true>) : launch(mxfp4_decode_kernel<false, false, true>);
        return out_type == MXFP4_F32 ? launch(mxfp4_decode_kernel<true, true, true>) : launch(mxfp4_decode_kernel<false, true, true>);
    }
    if (!vec)
        return out_type == MXFP4_F32 ? launch(mxfp4_decode_kernel<true, false, false>) : launch(mxfp4_decode_kernel<false, false, false>);
    return out_type == MXFP4_F32 ? launch(mxfp4_decode_kernel<true, true, false>) : launch(mxfp4_decode_kernel<false, true, false>);
}

mxfp8_status_t mxfp4_matmul(const void *a_codes, const void *a_scale, int64_t M, const void *b_codes, const void *b_scale, int64_t N, int64_t K,
                            void *out, int out_type, int64_t ldo, void *stream_)
{
    GemmParams p;
    mxfp8_status_t st = gemm_params(&p, a_codes, a_scale, M, b_codes, b_scale, N, K, out, out_type, ldo);
    if (st != MXFP8_OK)
        return st;
    int device = 0;
    if ((st = active_device(&device)) != MXFP8_OK)
        return st;
    for (const void *ptr : {a_codes, a_scale, b_codes, b_scale, static_cast<const void *>(out)})
        if (!pointer_on_device(ptr, device))
            return MXFP8_ERR_DEVICE;
    if (M == 0 || N == 0)
        return MXFP8_OK;
    cudaStream_t stream = static_cast<cudaStream_t>(stream_);
    if (K == 0)
        return zero_rows(out, M, N, ldo, out_type, stream);
    if ((p.fault = fault_word_address(device)) == nullptr)
        return MXFP8_ERR_DEVICE;
    const int64_t row_bytes = ceil_div(K, 32) * 16;
    const int64_t pair_tiles = ceil_div(N, kPairRows) * ceil_div(M, kPairRows);
    if (M > 128 && pair_tiles >= kPairMinTiles) {
        p.p_tiles = static_cast<int>(ceil_div(N, kPairRows));
        p.q_tiles = static_cast<int>(ceil_div(M, kPairRows));
        return out_type == MXFP4_F32
                   ? launch_pair_as<true, false>(p, b_codes, N, p.p_planes, a_codes, ceil_div(M, 128), row_bytes, pair_tiles, device, stream)
                   : launch_pair_as<false, false>(p, b_codes, N, p.p_planes, a_codes, ceil_div(M, 128), row_bytes, pair_tiles, device, stream);
    }
    return out_type == MXFP4_F32 ? launch_split<true>(p, b_codes, a_codes, row_bytes, device, stream)
                                 : launch_split<false>(p, b_codes, a_codes, row_bytes, device, stream);
}

mxfp8_status_t mxfp4_matmul_grouped(const void *a_codes, const void *a_scale, int64_t total_rows, int num_groups, const int64_t *offsets,
                                    const void *b_codes, const void *b_scale, int64_t N, int64_t K, void *out, int out_type, int *err_flag,
                                    void *stream_)
{
    GemmParams p;
    mxfp8_status_t st = gemm_params(&p, a_codes, a_scale, total_rows, b_codes, b_scale, N, K, out, out_type, N);
    if (st != MXFP8_OK)
        return st;
    if (num_groups < 1 || num_groups > MXFP8_MAX_GROUPS || offsets == nullptr)
        return MXFP8_ERR_GROUPS;
    const int64_t bound = (total_rows / 128 + num_groups) * static_cast<int64_t>(p.p_tiles);
    if (bound >= kMaxDim - (int64_t{1} << 20) || num_groups * N >= kMaxDim)
        return MXFP8_ERR_SHAPE;
    if (!is_aligned(offsets, 8) || !is_aligned(err_flag, 4))
        return MXFP8_ERR_ALIGN;
    int device = 0;
    if ((st = active_device(&device)) != MXFP8_OK)
        return st;
    for (const void *ptr : {a_codes, a_scale, b_codes, b_scale, static_cast<const void *>(out), static_cast<const void *>(offsets),
                            static_cast<const void *>(err_flag)})
        if (!pointer_on_device(ptr, device))
            return MXFP8_ERR_DEVICE;
    if (total_rows == 0 || N == 0)
        return MXFP8_OK;
    cudaStream_t stream = static_cast<cudaStream_t>(stream_);
    if (K == 0)
        return zero_rows(out, total_rows, N, N, out_type, stream);
    if ((p.fault = fault_word_address(device)) == nullptr)
        return MXFP8_ERR_DEVICE;
    p.offsets = offsets;
    p.num_groups = num_groups;
    p.err_flag = err_flag;
    const int64_t row_bytes = ceil_div(K, 32) * 16;
    if (total_rows >= kPairMinGroupRows * num_groups && total_rows / kPairRows * ceil_div(N, kPairRows) >= kPairMinTiles) {
        const int64_t q_planes = static_cast<int64_t>(mxfp4_grouped_scale_bytes(total_rows, K, num_groups) / 512) / p.kc;
        p.p_tiles = static_cast<int>(ceil_div(N, kPairRows));
        const int64_t pair_bound = (total_rows / kPairRows + num_groups) * p.p_tiles;
        return out_type == MXFP4_F32 ? launch_pair_as<true, true>(p, b_codes, num_groups * N, int64_t{num_groups} * p.p_planes, a_codes, q_planes,
                                                                  row_bytes, pair_bound, device, stream)
                                     : launch_pair_as<false, true>(p, b_codes, num_groups * N, int64_t{num_groups} * p.p_planes, a_codes, q_planes,
                                                                   row_bytes, pair_bound, device, stream);
    }
    CUtensorMap pm, qm;
    p.q_box = 32;
    if ((st = code_map(&pm, b_codes, num_groups * N, row_bytes, kGemmRows)) != MXFP8_OK ||
        (st = code_map(&qm, a_codes, total_rows, row_bytes, p.q_box)) != MXFP8_OK)
        return st;
    return out_type == MXFP4_F32 ? launch_group_as<true>(pm, qm, p, bound, device, stream)
                                 : launch_group_as<false>(pm, qm, p, bound, device, stream);
}

}  // extern "C"
