// Host-side helpers shared by the library's CUDA translation units
// (definitions in sherry_cuda.cu unless inline).
#pragma once

#include <atomic>
#include <cstddef>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "sherry.h"

namespace sherry {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline int cuda_status(cudaError_t e) { return e == cudaSuccess ? SHERRY_OK : SHERRY_ERR_CUDA; }

struct DeviceInfo {
    bool checked = false;
    bool ok = false;
    int sms = 0;
    int max_smem_optin = 0;
};

// The current device (SHERRY_ERR_DEVICE unless it is sm_100).
int device_info(DeviceInfo* out);

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn encode_fn();

// int8 rows x [M][K], ld bytes apart: boxes of 128 bytes x bn rows, 128-byte swizzle.
int make_x_map(CUtensorMap* map, const int8_t* x, int64_t M, int64_t K, int64_t ld, int bn);

// The device status word of the current device.
unsigned* device_status_ptr();

// Buffers set aside by sherry_reserve on the current device
// (SHERRY_ERR_WORKSPACE when smaller than asked for): the split-K workspace,
// and the int8 activations with their scales.
int get_workspace(size_t bytes, void** out);
int get_act_buffer(size_t bytes, void** out);
size_t act_buffer_bytes(int64_t M, int64_t K);

// Launch with programmatic dependent launch: the kernel may start while the
// previous kernel on the stream finishes; it orders itself with
// griddepcontrol.wait before touching anything that kernel may write.
// With a cluster shape, in thread-block clusters.
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream, dim3 cluster,
                       Args... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster.x;
    attr[1].val.clusterDim.y = cluster.y;
    attr[1].val.clusterDim.z = cluster.z;
    cfg.attrs = attr;
    cfg.numAttrs = cluster.x * cluster.y * cluster.z > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream, Args... args)
{
    return launch_pdl(kernel, grid, block, smem, stream, dim3(1, 1, 1), args...);
}

// Runs `set` once per device (function attributes belong to a context); a
// device beyond the 64 tracked runs it every time.
template <class F>
int once_per_device(std::atomic<uint64_t>& done, F set)
{
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return SHERRY_ERR_CUDA;
    const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
    if (done.load(std::memory_order_acquire) & bit) return SHERRY_OK;
    if (set() != cudaSuccess) return SHERRY_ERR_CUDA;
    done.fetch_or(bit, std::memory_order_release);
    return SHERRY_OK;
}

}  // namespace sherry
