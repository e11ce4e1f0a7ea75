// Host helpers shared by the library's translation units (defined in api.cu).
#pragma once

#include <cstdint>
#include <mutex>

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include "../../include/mxfp8.h"

namespace mxfp8 {

// The driver's tensor-map encoder, or nullptr.
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();

// Is p device (or managed) memory of `device`?  NULL passes.
bool pointer_on_device(const void *p, int device);

// The calling thread's current device.
mxfp8_status_t active_device(int *device);

// Count one kernel launch (mxfp8_kernel_launch_count).
void count_launch();

// Device address of the library's fault word on the current device (mxfp8_device_fault_word reads it),
// looked up once per device; nullptr if that fails.
unsigned int *fault_word_address(int device);

inline bool is_aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

constexpr int kMaxDevices = 64;

// One per kernel: on its first call on a device opts the kernel in to `smem` bytes; gives the CTAs resident at once.
struct KernelSetup {
    std::mutex mu;
    int sms[kMaxDevices] = {};
    int per_sm[kMaxDevices] = {};

    template <typename K>
    mxfp8_status_t operator()(K *kern, int device, int threads, int smem, int *ctas)
    {
        std::lock_guard<std::mutex> lock(mu);
        if (device < 0 || device >= kMaxDevices)
            return MXFP8_ERR_DEVICE;
        if (per_sm[device] == 0) {
            int n = 0, s = 0;
            if (cudaDeviceGetAttribute(&s, cudaDevAttrMultiProcessorCount, device) != cudaSuccess ||
                cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess ||
                cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kern, threads, smem) != cudaSuccess || n < 1) {
                cudaGetLastError();
                return MXFP8_ERR_LAUNCH;
            }
            sms[device] = s;
            per_sm[device] = n;
        }
        *ctas = per_sm[device] * sms[device];
        return MXFP8_OK;
    }
};

// Launch with programmatic stream serialisation (and, with cluster > 1, in thread-block clusters of that
// many consecutive blocks).  Only kernels whose threads all wait (griddepcontrol.wait) before their first
// global access are launched this way.  The exception: a products' kernel behind mxfp4_parts_kernel reads weights, their scales
// and offsets before it waits.  That holds because the parts' kernel is the launch just before it, writes none of these, and
// waits before it lets the next one start, so that whatever wrote them has ended; nothing may be launched between the two.
template <typename... Params, typename... Args>
mxfp8_status_t launch_serialized(void (*kern)(Params...), dim3 grid, unsigned block, size_t smem, int cluster,
                                 cudaStream_t stream, Args &&...args)
{
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, std::forward<Args>(args)...);
    const cudaError_t last = cudaGetLastError();
    count_launch();
    return e == cudaSuccess && last == cudaSuccess ? MXFP8_OK : MXFP8_ERR_LAUNCH;
}

}  // namespace mxfp8
