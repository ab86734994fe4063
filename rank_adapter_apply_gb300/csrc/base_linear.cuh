// lora_base_linear: what its kernels share (base_linear.cu, base_linear_tc.cu).
#pragma once

#include "step_util.cuh"

#include <atomic>

namespace lora {
namespace linear {

struct LinearArgs {
    const void *x;
    const uint8_t *qweight;
    const void *scales;
    const uint8_t *zeros;
    void *y;
    long long x_stride, y_stride;
    int n_tokens, d_in, d_out, group;
};

constexpr int kMaxCluster = 8;

// Clusters of c CTAs of `threads` threads that the current device holds at once; asked of the runtime once. `known`
// is the caller's, one of a kernel and number of threads.
struct ActiveClusters {
    std::atomic<int> count[kMaxCluster + 1];       // 1 + the answer
    std::atomic<int> device;                        // 1 + the device they are of
};
template <typename Kernel>
int active_clusters(Kernel kernel, int threads, size_t smem, int c, ActiveClusters &known) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    const bool same = known.device.load(std::memory_order_acquire) == dev + 1;
    int n = same ? known.count[c].load(std::memory_order_relaxed) : 0;
    if (n > 0) return n - 1;
    if (!same) {
        for (auto &k : known.count) k.store(0, std::memory_order_relaxed);
        known.device.store(dev + 1, std::memory_order_release);
    }
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(c);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = c;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) {
        cudaGetLastError();
        n = 0;
    }
    known.count[c].store(n + 1, std::memory_order_relaxed);
    return n;
}

// On the 5th-generation tensor cores (base_linear_tc.cu): whether TMA can load an x of several rows in bf16 (fp32 it takes
// as it is), and the launch.
bool tc_takes(const LinearArgs &a);
cudaError_t launch_tc(const LinearArgs &a, int dtype, int sms, cudaStream_t st);
// CTAs whose bounded waits gave up.
cudaError_t read_timeouts(unsigned *count);

}  // namespace linear
}  // namespace lora
