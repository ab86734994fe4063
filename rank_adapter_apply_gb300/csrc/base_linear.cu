// lora_base_linear: y = W x for a few tokens, W in 4 bits with group scales.
#include "step_util.cuh"

namespace lora {
namespace {

using namespace step;

struct LinearArgs {
    const void *x;
    const uint8_t *qweight;
    const void *scales;
    const uint8_t *zeros;
    void *y;
    long long x_stride, y_stride;
    int n_tokens, d_in, d_out, group;
};

// One warp per output row and TT tokens: a lane takes eight columns (one
// 32-bit word of the row) at a time, in fp32.
template <typename T, int TT>
__global__ void __launch_bounds__(256) linear_rows_kernel(LinearArgs a) {
    const int lane = threadIdx.x & 31;
    const int row = blockIdx.x * 8 + (threadIdx.x >> 5);
    const int t0 = blockIdx.y * TT;
    if (row >= a.d_out) return;
    const int nt = min(TT, a.n_tokens - t0);
    const int words = a.d_in / 8, groups = a.d_in / a.group;
    const uint32_t *w = reinterpret_cast<const uint32_t *>(a.qweight + (size_t)row * (a.d_in / 2));
    const T *sc = static_cast<const T *>(a.scales) + (size_t)row * groups;
    const uint8_t *zr = a.zeros ? a.zeros + (size_t)row * groups : nullptr;
    const T *x = static_cast<const T *>(a.x) + (size_t)t0 * a.x_stride;
    float acc[TT];
#pragma unroll
    for (int t = 0; t < TT; ++t) acc[t] = 0.f;
    for (int i = lane; i < words; i += 32) {
        const uint32_t q = w[i];
        const int g = i * 8 / a.group;
        const float s = to_f32(sc[g]);
        const float z = zr ? (float)zr[g] : 8.f;
        float n[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) n[j] = (float)((q >> (4 * j)) & 15u) - z;
#pragma unroll
        for (int t = 0; t < TT; ++t) {
            if (t < nt) {
                const T *xt = x + (size_t)t * a.x_stride + i * 8;
                float p = 0.f;
#pragma unroll
                for (int j = 0; j < 8; ++j) p = fmaf(n[j], to_f32(xt[j]), p);
                acc[t] = fmaf(s, p, acc[t]);
            }
        }
    }
#pragma unroll
    for (int t = 0; t < TT; ++t) {
        const float v = warp_sum(acc[t]);
        if (lane == 0 && t < nt) static_cast<T *>(a.y)[(size_t)(t0 + t) * a.y_stride + row] = from_f32<T>(v);
    }
}

template <typename T>
cudaError_t launch_rows(const LinearArgs &a, cudaStream_t st) {
    constexpr int TT = 8;
    dim3 grid((a.d_out + 7) / 8, (a.n_tokens + TT - 1) / TT);
    linear_rows_kernel<T, TT><<<grid, 256, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace
}  // namespace lora

using namespace lora;
using namespace lora::step;

extern "C" int lora_base_linear(const lora_base_linear_desc *d, void *stream) {
    if (!d) return fail(LORA_ERR_ARG, "base_linear: NULL descriptor");
    if (!known_dtype(d->dtype)) return fail(LORA_ERR_ARG, "base_linear: unknown dtype %d", d->dtype);
    if (d->group != 32 && d->group != 64 && d->group != 128)
        return fail(LORA_ERR_ARG, "base_linear: group %d is not 32, 64 or 128", d->group);
    if (d->n_tokens < 0 || d->d_in < 1 || d->d_out < 1 || d->d_in % d->group != 0)
        return fail(LORA_ERR_ARG, "base_linear: n_tokens %d, d_in %d (a multiple of group %d), d_out %d", d->n_tokens,
                    d->d_in, d->group, d->d_out);
    if (d->n_tokens > (1 << 19)) return fail(LORA_ERR_ARG, "base_linear: n_tokens %d is above 524288", d->n_tokens);
    if (d->n_tokens == 0) return LORA_OK;
    if (!d->x || !d->qweight || !d->scales || !d->y) return fail(LORA_ERR_ARG, "base_linear: NULL pointer argument");
    if (!aligned16(d->qweight)) return fail(LORA_ERR_ARG, "base_linear: qweight must be 16-byte aligned");
    if (d->n_tokens > 1 && (d->x_stride < d->d_in || d->y_stride < d->d_out))
        return fail(LORA_ERR_ARG, "base_linear: row strides %lld, %lld are below d_in, d_out", (long long)d->x_stride,
                    (long long)d->y_stride);
    LinearArgs a{d->x,        d->qweight,  d->scales, d->zeros, d->y,    (long long)d->x_stride,
                 (long long)d->y_stride, d->n_tokens, d->d_in,   d->d_out, d->group};
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t e =
        d->dtype == LORA_DTYPE_BF16 ? launch_rows<__nv_bfloat16>(a, st) : launch_rows<float>(a, st);
    return launched("base_linear", e);
}
