// The driver's encoder of tensor maps, asked for once.
#pragma once

#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <atomic>

namespace lora {
namespace step {

inline PFN_cuTensorMapEncodeTiled_v12000 map_encoder() {
    static std::atomic<PFN_cuTensorMapEncodeTiled_v12000> known{nullptr};
    PFN_cuTensorMapEncodeTiled_v12000 fn = known.load(std::memory_order_acquire);
    if (fn) return fn;
    cudaDriverEntryPointQueryResult q;
    void *p = nullptr;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess || !p)
        return nullptr;
    fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    known.store(fn, std::memory_order_release);
    return fn;
}

}  // namespace step
}  // namespace lora
