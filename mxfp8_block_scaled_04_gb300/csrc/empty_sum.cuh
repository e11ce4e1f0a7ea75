// Experts' products with nothing to sum, or with nothing to write: the offsets are checked as the products check them
// (groups.cuh), the output becomes zeros where they are good, and the error flag is set as there.  Bound by launch and latency.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>

#include "host.h"
#include "ptx.cuh"

namespace mxfp8 {

constexpr int kEmptySumThreads = 256, kEmptySumCtas = 1216;

struct EmptySumParams {
    const int64_t *offsets;
    int num_groups;
    int64_t total;        // rows that the offsets divide
    const int32_t *rows;  // which of T rows each is, or NULL: one that does not exist becomes NaN
    int64_t T;
    void *out;
    int64_t count, cols;  // elements in all, of a row
    int *err_flag;
};

// A product's output [total, cols].
inline EmptySumParams empty_sum(const int64_t *offsets, int num_groups, int64_t total, const int32_t *rows, int64_t T, void *out, int64_t cols, int *err_flag)
{
    return {offsets, num_groups, total, rows, T, out, total * cols, cols, err_flag};
}

template <bool F32>
__global__ void __launch_bounds__(kEmptySumThreads) empty_sum_kernel(const EmptySumParams p)
{
    pdl_wait_and_release();
    const int tid = threadIdx.x;
    int bad = tid == 0 && (p.offsets[0] != 0 || p.offsets[p.num_groups] > p.total);
    for (int g = tid; g < p.num_groups; g += kEmptySumThreads)
        bad |= p.offsets[g + 1] < p.offsets[g];
    if (__syncthreads_or(bad)) {
        if (blockIdx.x == 0 && tid == 0 && p.err_flag != nullptr)
            atomicOr(p.err_flag, 1);
        return;
    }
    const int64_t end = p.offsets[p.num_groups];  // rows from here on belong to no expert
    const int64_t first = blockIdx.x * int64_t{kEmptySumThreads} + tid, step = gridDim.x * int64_t{kEmptySumThreads};
    auto missing = [&](int64_t r) { return p.rows != nullptr && r < end && (p.rows[r] < 0 || p.rows[r] >= p.T); };
    bool told = p.rows == nullptr && end < p.total;
    for (int64_t r = first; p.rows != nullptr && r < p.total; r += step)
        told |= missing(r) || (r >= end && p.rows[r] >= 0);
    if (told && p.err_flag != nullptr)
        atomicOr(p.err_flag, 1);
    for (int64_t i = first; i < p.count; i += step) {
        const float v = missing(i / p.cols) ? __uint_as_float(0x7FFFFFFFu) : 0.f;
        if constexpr (F32)
            static_cast<float *>(p.out)[i] = v;
        else
            static_cast<__nv_bfloat16 *>(p.out)[i] = __float2bfloat16_rn(v);
    }
}

inline mxfp8_status_t launch_empty_sum(const EmptySumParams &p, bool f32, cudaStream_t stream)
{
    if (p.count == 0 && p.err_flag == nullptr)
        return MXFP8_OK;
    const int64_t rows = p.rows != nullptr ? p.total : 1, work = p.count > rows ? p.count : rows;
    const int64_t ctas = (work + kEmptySumThreads - 1) / kEmptySumThreads;
    const dim3 grid(static_cast<unsigned>(ctas < 1 ? 1 : ctas < kEmptySumCtas ? ctas : kEmptySumCtas));
    return f32 ? launch_serialized(empty_sum_kernel<true>, grid, kEmptySumThreads, 0, 1, stream, p)
               : launch_serialized(empty_sum_kernel<false>, grid, kEmptySumThreads, 0, 1, stream, p);
}

}  // namespace mxfp8
