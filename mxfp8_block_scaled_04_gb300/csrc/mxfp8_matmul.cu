// C ABI of the experts' products in MXFP8 (declarations and contract in include/mxfp8_matmul.h): host-side checks, tensor
// maps and launches; the device code is in mxfp8_pair.cuh.
#include <cstdint>

#include "../../include/mxfp8_matmul.h"
#include "empty_sum.cuh"
#include "host.h"
#include "mxfp8_pair.cuh"

namespace {

using namespace mxfp8;

constexpr int64_t kMaxDim = int64_t{1} << 31;

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

mxfp8_status_t encode(CUtensorMap *map, CUtensorMapDataType type, int rank, const void *at, const cuuint64_t *dims, const cuuint64_t *strides,
                      const cuuint32_t *box, CUtensorMapSwizzle swizzle)
{
    PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
    if (enc == nullptr)
        return MXFP8_ERR_DEVICE;
    const cuuint32_t estr[3] = {1, 1, 1};
    return enc(map, type, static_cast<cuuint32_t>(rank), const_cast<void *>(at), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? MXFP8_OK
               : MXFP8_ERR_LAUNCH;
}

// Codes [rows, cols] in boxes of 128 columns x box_rows.
mxfp8_status_t code_map(CUtensorMap *map, const void *codes, int64_t rows, int64_t cols, int box_rows)
{
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(cols)};
    const cuuint32_t box[2] = {128, static_cast<cuuint32_t>(box_rows)};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, codes, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

// The same codes without a swizzle, in boxes that are only read before the first row: zeros.
mxfp8_status_t zeros_map(CUtensorMap *map, const void *codes, int64_t rows, int64_t cols, int box_rows)
{
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(cols)};
    const cuuint32_t box[2] = {128, static_cast<cuuint32_t>(box_rows)};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, codes, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_NONE);
}

// Experts' codes [groups, rows, cols]: an expert's rows end in zeros, not in the next expert's.
mxfp8_status_t weight_map(CUtensorMap *map, const void *codes, int64_t groups, int64_t rows, int64_t cols)
{
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(groups)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(cols * rows)};
    const cuuint32_t box[3] = {128, 128, 1};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, codes, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

// A scale plane as tile_rows rows of kc tiles of 512 bytes, in boxes of one tile x box_rows tile rows.  (A map has a row at least;
// of a plane without one the kernel reads none.)
mxfp8_status_t scale_map(CUtensorMap *map, const void *scale, int64_t tile_rows, int64_t kc, int box_rows)
{
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(kc) * 128, static_cast<cuuint64_t>(tile_rows < 1 ? 1 : tile_rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(kc) * 512};
    const cuuint32_t box[2] = {128, static_cast<cuuint32_t>(box_rows)};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, scale, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_NONE);
}

// The weight gradients [groups, N, K] in boxes of 128 bytes x 32 rows: what lies past an expert's rows is not written.
mxfp8_status_t gradient_map(CUtensorMap *map, void *out, int64_t groups, int64_t N, int64_t K, bool f32)
{
    const int64_t size = f32 ? 4 : 2;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(K), static_cast<cuuint64_t>(N), static_cast<cuuint64_t>(groups)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(K * size), static_cast<cuuint64_t>(N * K * size)};
    const cuuint32_t box[3] = {static_cast<cuuint32_t>(128 / size), 32, 1};
    return encode(map, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, out, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

struct Maps {
    CUtensorMap p, q, q_part, p_scale, q_scale, out, zeros, zero_row;
};

template <int MODE, bool F32>
mxfp8_status_t launch_pair(const Product8Params &p, const Maps &m, int64_t tiles, int device, cudaStream_t stream)
{
    static KernelSetup setup;
    constexpr int smem = kP8Smem + kP8Epilogue<MODE, F32>;
    int ctas = 0;
    const mxfp8_status_t st = setup(mxfp8_pair_kernel<MODE, F32>, device, kP8Threads<MODE>, smem, &ctas);
    if (st != MXFP8_OK)
        return st;
    const int64_t pairs = tiles < ctas / 2 ? tiles : ctas / 2;
    return launch_serialized(mxfp8_pair_kernel<MODE, F32>, dim3(static_cast<unsigned>(2 * pairs)), kP8Threads<MODE>, smem, 2, stream, m.p, m.q, m.q_part,
                             m.p_scale, m.q_scale, m.out, m.zeros, m.zero_row, p);
}

}  // namespace

extern "C" {

mxfp8_status_t mxfp8_matmul_grouped(int product, const void *a, const void *a_scale, size_t a_scale_bytes, int a_fmt, const void *b,
                                    const void *b_scale, size_t b_scale_bytes, int b_fmt, int64_t total_rows, int64_t N, int64_t K, int num_groups,
                                    const int64_t *offsets, void *out, int out_type, int *err_flag, void *stream_)
{
    if (product < MXFP8_FORWARD || product > MXFP8_WEIGHT_GRADIENT || (out_type != MXFP4_BF16 && out_type != MXFP4_F32) ||
        (a_fmt != MXFP8_E4M3 && a_fmt != MXFP8_E5M2) || (b_fmt != MXFP8_E4M3 && b_fmt != MXFP8_E5M2))
        return MXFP8_ERR_FORMAT;
    if (total_rows < 0 || N < 0 || K < 0 || total_rows >= kMaxDim || N >= kMaxDim || K >= kMaxDim || N % 16 || K % 16)
        return MXFP8_ERR_SHAPE;
    if (num_groups < 1 || num_groups > MXFP8_MAX_GROUPS || offsets == nullptr)
        return MXFP8_ERR_GROUPS;
    if (num_groups * N >= kMaxDim)
        return MXFP8_ERR_SHAPE;
    const bool wgrad = product == MXFP8_WEIGHT_GRADIENT;
    const int64_t P = product == MXFP8_INPUT_GRADIENT ? K : N, sum = wgrad ? total_rows : product == MXFP8_FORWARD ? K : N;
    const int64_t p_tiles = ceil_div(P, kP8Tile), q_tiles = ceil_div(K, kP8Tile);
    const int64_t tiles = wgrad ? num_groups * p_tiles * q_tiles : (total_rows / kP8Tile + num_groups) * p_tiles;
    // the weight gradient's tile rows of scales, all planes' together
    const int64_t linear = (total_rows / 128 + num_groups) * ceil_div(N > K ? N : K, 128);
    if (tiles >= kMaxDim - (int64_t{1} << 20) || (wgrad && linear >= kMaxDim))
        return MXFP8_ERR_SHAPE;
    const int64_t out_rows = wgrad ? num_groups * N : total_rows;
    const int64_t cols = wgrad ? K : P;
    const bool empty = out_rows == 0 || cols == 0;
    const int64_t kc = ceil_div(sum, 128);  // tiles along the summed dimension (forward, input gradient)
    if (!empty) {
        if (out == nullptr || (sum > 0 && (a == nullptr || a_scale == nullptr || b == nullptr || b_scale == nullptr)))
            return MXFP8_ERR_NULL;
        if (!wgrad && static_cast<int64_t>(b_scale_bytes / 512) < num_groups * ceil_div(P, 128) * kc)
            return MXFP8_ERR_WORKSPACE;
    }
    if (!is_aligned(a, 16) || !is_aligned(a_scale, 16) || !is_aligned(b, 16) || !is_aligned(b_scale, 16) || !is_aligned(out, 16) ||
        !is_aligned(offsets, 8) || !is_aligned(err_flag, 4))
        return MXFP8_ERR_ALIGN;
    int device = 0;
    mxfp8_status_t st = active_device(&device);
    if (st != MXFP8_OK)
        return st;
    for (const void *ptr : {a, a_scale, b, b_scale, static_cast<const void *>(out), static_cast<const void *>(offsets),
                            static_cast<const void *>(err_flag)})
        if (!pointer_on_device(ptr, device))
            return MXFP8_ERR_DEVICE;
    cudaStream_t stream = static_cast<cudaStream_t>(stream_);
    if (empty || sum == 0) {
        EmptySumParams e{};
        e.offsets = offsets;
        e.num_groups = num_groups;
        e.total = total_rows;
        e.out = out;
        e.count = out_rows * cols;
        e.cols = cols;
        e.err_flag = err_flag;
        return launch_empty_sum(e, out_type == MXFP4_F32, stream);
    }
    Product8Params p{};
    if ((p.fault = fault_word_address(device)) == nullptr)
        return MXFP8_ERR_DEVICE;
    p.P = P;
    p.Q = wgrad ? K : total_rows;
    p.sum = sum;
    p.kc = static_cast<int>(kc);
    p.k_iters = static_cast<int>(kc);
    p.p_tiles = static_cast<int>(p_tiles);
    p.q_tiles = static_cast<int>(q_tiles);
    p.p_planes = static_cast<int>(ceil_div(P, 128));
    p.p_ct = static_cast<int>(ceil_div(N, 128));
    p.q_ct = static_cast<int>(ceil_div(K, 128));
    p.out = out;
    p.ldo = P;
    p.vec_out = true;  // N and K are multiples of 16
    p.offsets = offsets;
    p.num_groups = num_groups;
    p.err_flag = err_flag;
    // the weight gradient has the gradient on the accumulator's lanes, the other two the weights
    const int p_fmt = wgrad ? a_fmt : b_fmt, q_fmt = wgrad ? b_fmt : a_fmt;
    p.formats = (static_cast<uint32_t>(p_fmt) << 7) | (static_cast<uint32_t>(q_fmt) << 10);
    const int64_t unit = wgrad ? 512 : kc * 512;
    const int64_t a_tile_rows = static_cast<int64_t>(a_scale_bytes) / unit, b_tile_rows = static_cast<int64_t>(b_scale_bytes) / unit;
    p.p_tile_rows = wgrad ? a_tile_rows : b_tile_rows;
    p.q_tile_rows = wgrad ? b_tile_rows : a_tile_rows;
    const bool f32 = out_type == MXFP4_F32;
    Maps m;
    if (wgrad) {
        if ((st = code_map(&m.p, a, total_rows, N, 128)) != MXFP8_OK || (st = code_map(&m.q, b, total_rows, K, 128)) != MXFP8_OK ||
            (st = scale_map(&m.p_scale, a_scale, a_tile_rows, 1, 1)) != MXFP8_OK || (st = scale_map(&m.q_scale, b_scale, b_tile_rows, 1, 1)) != MXFP8_OK ||
            (st = zeros_map(&m.zeros, a, total_rows, N, kZeroRows)) != MXFP8_OK || (st = zeros_map(&m.zero_row, a, total_rows, N, 1)) != MXFP8_OK ||
            (st = gradient_map(&m.out, out, num_groups, N, K, f32)) != MXFP8_OK)
            return st;
        m.q_part = m.q;
    } else {
        if ((st = weight_map(&m.p, b, num_groups, N, K)) != MXFP8_OK || (st = code_map(&m.q, a, total_rows, sum, 128)) != MXFP8_OK ||
            (st = code_map(&m.q_part, a, total_rows, sum, 32)) != MXFP8_OK || (st = scale_map(&m.p_scale, b_scale, b_tile_rows, kc, 1)) != MXFP8_OK ||
            (st = scale_map(&m.q_scale, a_scale, a_tile_rows, kc, 2)) != MXFP8_OK)
            return st;
        m.out = m.zeros = m.zero_row = m.q;
    }
    switch (product) {
    case MXFP8_FORWARD:
        return f32 ? launch_pair<kForward, true>(p, m, tiles, device, stream) : launch_pair<kForward, false>(p, m, tiles, device, stream);
    case MXFP8_INPUT_GRADIENT:
        return f32 ? launch_pair<kInputGrad, true>(p, m, tiles, device, stream) : launch_pair<kInputGrad, false>(p, m, tiles, device, stream);
    default:
        return f32 ? launch_pair<kWeightGrad, true>(p, m, tiles, device, stream) : launch_pair<kWeightGrad, false>(p, m, tiles, device, stream);
    }
}

}  // extern "C"
