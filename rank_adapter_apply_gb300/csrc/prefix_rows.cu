// lora_prefix_attention in bf16, up to 16 rows of an entry: the single tokens and small
// trees of a decoding step, whose keys are read for a few rows. Two warps to a scheduler, each
// with its own ring, keep up to 128 KB of keys and values in flight on an SM. 200 requests with
// contexts of up to 1000, 8 heads of 128: 87 us, 4.7 TB/s (6 / 10 / 12 warps 95 / 96 / 93).
#include "prefix_rows.cuh"

#include <atomic>

namespace lora {
namespace tree {
namespace {

constexpr int kWarps = 8, kThreads = 32 * kWarps;

template <int DP>
__global__ void __launch_bounds__(kThreads, 1) prefix_rows_kernel(TreeArgs a, Plan plan) {
    extern __shared__ __align__(128) unsigned char smem[];
    grid_dependency_wait();
    grid_launch_dependents();
    rows::work<DP, kWarps, kThreads>(a, plan, smem);
}

template <int DP>
cudaError_t launch(const TreeArgs &a, const Plan &plan, cudaStream_t st) {
    static std::atomic<uint64_t> ready{0};
    constexpr int kSmem = sizeof(rows::Memory<DP, kWarps, kThreads>);
    if (!device_bit(ready)) {
        const cudaError_t e = cudaFuncSetAttribute(prefix_rows_kernel<DP>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
        if (e != cudaSuccess) return e;
        set_device_bit(ready);
    }
    return launch_step(prefix_rows_kernel<DP>, dim3(plan.ctas / kWarps), dim3(kThreads), kSmem, 1, st, a, plan);
}

}  // namespace

// plan.ctas becomes the number of warps: each has two parts of 16 rows.
cudaError_t launch_rows(const TreeArgs &a, Plan &plan, cudaStream_t st) {
    plan.ctas = plan.ctas / 2 * kWarps;
    return a.head_dim <= 64 ? launch<64>(a, plan, st) : launch<128>(a, plan, st);
}

}  // namespace tree
}  // namespace lora
