// Compares the routing's reciprocal with the correctly rounded one, bit for bit, for every fp32 number in [1, 2^126].
// Built and run by test_reciprocal_gpu.py.
#include <cstdint>

#include "moe.cuh"

namespace {

// One thread per mantissa, all exponents in turn.  out[0]: numbers compared; out[1]: differences; out[2]: one of the numbers
// that differ (its bits).
__global__ void compare(unsigned long long *out)
{
    const uint32_t mantissa = blockIdx.x * blockDim.x + threadIdx.x;
    if (mantissa >= 1u << 23)
        return;
    unsigned n = 0, differ = 0;
    for (uint32_t e = 127; e <= 253; ++e) {
        const float y = __uint_as_float(e << 23 | mantissa);
        if (y > mxfp8::kReciprocalMax)
            break;
        ++n;
        if (__float_as_uint(mxfp8::reciprocal_fast(y)) != __float_as_uint(__frcp_rn(y))) {
            ++differ;
            out[2] = __float_as_uint(y);
        }
    }
    atomicAdd(&out[0], static_cast<unsigned long long>(n));
    if (differ)
        atomicAdd(&out[1], static_cast<unsigned long long>(differ));
}

}  // namespace

extern "C" int reciprocal_compare(unsigned long long *out)
{
    compare<<<(1 << 23) / 256, 256>>>(out);
    const cudaError_t launched = cudaGetLastError();
    return static_cast<int>(launched != cudaSuccess ? launched : cudaDeviceSynchronize());
}
