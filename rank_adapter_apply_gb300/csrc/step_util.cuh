// Shared by the drafted-token step's calls (base_linear.cu, rope.cu,
// tree_attention.cu, verify_drafts.cu): argument errors, launch errors and
// element access by type.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdarg>
#include <cstdint>
#include <cstdio>

#include "device_util.cuh"
#include "kernels.cuh"
#include "rank_adapter_apply.h"

namespace lora {
namespace step {

// Record a formatted message for lora_last_error() and return `code`.
inline int fail(int code, const char *fmt, ...) {
    char buf[256];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    return set_last_error(code, buf);
}

inline int launched(const char *what, cudaError_t e) {
    if (e == cudaSuccess) return LORA_OK;
    return fail(LORA_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

// SMs of the current device, 0 where there is none.
inline int sm_count() {
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return 0;
    return n;
}

// Launch in clusters of `cluster` CTAs (1: none) with programmatic stream
// serialization: the kernel calls grid_dependency_wait() before it touches
// memory, so its launch alone overlaps the end of the kernel before it.
template <typename... KArgs, typename... Args>
inline cudaError_t launch_step(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, int cluster, cudaStream_t st,
                               const Args &...args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

inline bool aligned16(const void *p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

// Whether rows of `len` elements at i * s0 + j * s1, i < n0 and j < n1, lie apart: the rows of an output that one call
// writes in no order.
inline bool rows_apart(long long n0, long long s0, long long n1, long long s1, long long len) {
    using wide = __int128;
    if (n0 < 1 || n1 < 1) return true;
    const wide a = s0 < 0 ? -(wide)s0 : s0, b = s1 < 0 ? -(wide)s1 : s1;
    if ((n0 > 1 && a < len) || (n1 > 1 && b < len)) return false;
    if (n0 == 1 || n1 == 1 || a >= (n1 - 1) * b + len || b >= (n0 - 1) * a + len) return true;
    for (wide j = 1; j < n1; ++j) {                        // neither inside the other: the rows next to i = 0's j-th
        const wide i = j * b / a;
        if ((i < n0 && j * b - i * a < len) || (i + 1 < n0 && (i + 1) * a - j * b < len)) return false;
    }
    return true;
}

inline bool known_dtype(int dtype) { return dtype == LORA_DTYPE_F32 || dtype == LORA_DTYPE_BF16; }

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// The elements of 16 bytes.
template <typename T>
__device__ __forceinline__ void unpack(const uint4 &v, float (&f)[16 / sizeof(T)]);
template <>
__device__ __forceinline__ void unpack<float>(const uint4 &v, float (&f)[4]) {
    f[0] = __uint_as_float(v.x), f[1] = __uint_as_float(v.y), f[2] = __uint_as_float(v.z), f[3] = __uint_as_float(v.w);
}
template <>
__device__ __forceinline__ void unpack<__nv_bfloat16>(const uint4 &v, float (&f)[8]) {
    f[0] = bf_lo(v.x), f[1] = bf_hi(v.x), f[2] = bf_lo(v.y), f[3] = bf_hi(v.y);
    f[4] = bf_lo(v.z), f[5] = bf_hi(v.z), f[6] = bf_lo(v.w), f[7] = bf_hi(v.w);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

}  // namespace step
}  // namespace lora
