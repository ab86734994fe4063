// lora_norm_rope: the norm of every query and key head, then the rotary positions
// and the append of k and v to the paged cache, in one pass over the rows.
//
//   y = x / sqrt(mean(x^2) + eps) * w,  (a, b) -> (a cos - b sin, a sin + b cos)
//
// The sum of squares, the norm and the turn are fp32 and the result is rounded once;
// between the norm and the rotation nothing is rounded or written. A row is read once
// and written once, as in lora_rope, whose layout of threads it keeps.
#include "rope_common.cuh"

#include <cmath>

namespace lora {
namespace {

using namespace step;
using namespace rope;

struct NormArgs {
    RopeArgs r;
    const void *q_weight, *k_weight;       // nullptr: ones
    long long q_weight_head, k_weight_head;
    float eps;
};

// The weight of head row r (q heads, then k); nullptr: ones.
template <typename T>
__device__ __forceinline__ const T *weight_of(const NormArgs &n, int r) {
    const bool q = r < n.r.n_heads;
    const T *w = static_cast<const T *>(q ? n.q_weight : n.k_weight);
    return w ? w + (q ? r * n.q_weight_head : (r - n.r.n_heads) * n.k_weight_head) : nullptr;
}

// Any layout: one warp per head row of one token; the row is read again for the turn.
// Bound by its issue slots; for rows that are not whole 16-byte vectors or longer
// than 64 of them.
template <typename T, bool kInterleaved>
__global__ void __launch_bounds__(256) norm_rows_kernel(NormArgs n) {
    const RopeArgs &a = n.r;
    grid_dependency_wait();
    grid_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int rows = a.n_heads + 2 * a.n_kv;
    const long long item = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (item >= (long long)a.n_tokens * rows) return;
    const long long t = item / rows;
    const int r = (int)(item % rows), pos = a.positions[t];
    if (pos < 0 || pos >= a.n_positions) return;
    const Row<T> w = row_of<T>(a, t, r, cache_place(a, t));
    if (!w.dst) return;
    if (!w.turned) {
        for (int i = lane; i < a.head_dim; i += 32) w.dst[i] = w.src[i];
        return;
    }
    const T *weight = weight_of<T>(n, r);
    float sum = 0.f;
    for (int i = lane; i < a.head_dim; i += 32) {
        const float x = to_f32(w.src[i]);
        sum = fmaf(x, x, sum);
    }
    const float inv = rsqrtf(warp_sum(sum) / (float)a.head_dim + n.eps);
    auto normed = [&](int i) { return to_f32(w.src[i]) * inv * (weight ? to_f32(weight[i]) : 1.f); };
    const int half = a.rot_dim / 2;
    const float *row = a.table + (size_t)pos * a.rot_dim;
    for (int j = lane; j < half; j += 32) {
        const float c = row[j], s = row[half + j];
        const int i0 = kInterleaved ? 2 * j : j, i1 = kInterleaved ? 2 * j + 1 : j + half;
        const float x0 = normed(i0), x1 = normed(i1);
        w.dst[i0] = from_f32<T>(x0 * c - x1 * s);
        w.dst[i1] = from_f32<T>(x0 * s + x1 * c);
    }
    for (int i = a.rot_dim + lane; i < a.head_dim; i += 32) w.dst[i] = from_f32<T>(normed(i));
}

// Rows in 16-byte vectors: a unit is two vectors of a row that are turned together (as
// in lora_rope), or two neighbours past rot_dim and in v. blockDim.x is the units of a
// row rounded up to a power of two, so that a row's sum of squares stays in a part of a
// warp. A thread takes its unit of kRows rows of one token, with all loads in flight
// before the first is used.
template <typename T, bool kInterleaved, int kRows>
__global__ void __launch_bounds__(256) norm_vectors_kernel(NormArgs n) {
    constexpr int N = 16 / sizeof(T);
    const RopeArgs &a = n.r;
    grid_dependency_wait();
    grid_launch_dependents();
    const long long t = blockIdx.x;
    const int u = threadIdx.x, rows = a.n_heads + 2 * a.n_kv, r0 = (blockIdx.y * blockDim.y + threadIdx.y) * kRows;
    const int vectors = a.head_dim / N, rot_vectors = a.rot_dim / N, half = a.rot_dim / 2;
    const int pos = a.positions[t];
    const long long at = cache_place(a, t);
    if (pos < 0 || pos >= a.n_positions) return;           // the whole block
    // this unit's vectors in a row that is normed and turned, and in one that is copied
    const bool turns = kInterleaved ? 2 * u < rot_vectors : u < rot_vectors / 2;
    const int v0 = kInterleaved || !turns ? 2 * u : u, v1 = kInterleaved || !turns ? 2 * u + 1 : u + rot_vectors / 2;
    Row<T> w[kRows];
    uint4 x0[kRows], x1[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        w[i].dst = nullptr;
        w[i].turned = false;
        x0[i] = x1[i] = make_uint4(0, 0, 0, 0);
        if (r0 + i < rows) w[i] = row_of<T>(a, t, r0 + i, at);
        if (!w[i].dst) continue;
        const int e0 = w[i].turned ? v0 : 2 * u, e1 = w[i].turned ? v1 : 2 * u + 1;
        if (e0 < vectors) x0[i] = *reinterpret_cast<const uint4 *>(w[i].src + e0 * N);
        if (e1 < vectors) x1[i] = *reinterpret_cast<const uint4 *>(w[i].src + e1 * N);
    }
    // N angles: of elements 2u N .. (interleaved: of N pairs) or u N ..
    float c[N], s[N];
    if (turns) {
        const float *row = a.table + (size_t)pos * a.rot_dim + u * N;
#pragma unroll
        for (int j = 0; j < N; ++j) {
            c[j] = row[j];
            s[j] = row[half + j];
        }
    }
    float w0[N], w1[N];                                      // the weights of the row before, mostly this one's, too
    const T *held = nullptr;
#pragma unroll
    for (int j = 0; j < N; ++j) w0[j] = w1[j] = 1.f;
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const bool turned = w[i].turned;
        float f0[N], f1[N];
        unpack<T>(x0[i], f0);
        unpack<T>(x1[i], f1);
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < N; ++j) sum = fmaf(f0[j], f0[j], fmaf(f1[j], f1[j], sum));
        // every lane takes part, whatever its row
        for (int o = blockDim.x >> 1; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (!w[i].dst) continue;
        const int e0 = turned ? v0 : 2 * u, e1 = turned ? v1 : 2 * u + 1;
        if (turned) {
            const float inv = rsqrtf(sum / (float)a.head_dim + n.eps);
            const T *weight = weight_of<T>(n, r0 + i);
            if (weight != held) {
                held = weight;
                if (weight) {
                    if (v0 < vectors) unpack<T>(*reinterpret_cast<const uint4 *>(weight + v0 * N), w0);
                    if (v1 < vectors) unpack<T>(*reinterpret_cast<const uint4 *>(weight + v1 * N), w1);
                } else {
#pragma unroll
                    for (int j = 0; j < N; ++j) w0[j] = w1[j] = 1.f;
                }
            }
#pragma unroll
            for (int j = 0; j < N; ++j) {
                f0[j] = f0[j] * inv * w0[j];
                f1[j] = f1[j] * inv * w1[j];
            }
            if (turns) {
                float g0[N], g1[N];
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    if (kInterleaved) {                    // pairs (2j, 2j + 1) of the two vectors in a row
                        const int p = j % (N / 2) * 2;
                        float(&f)[N] = j < N / 2 ? f0 : f1;
                        float(&g)[N] = j < N / 2 ? g0 : g1;
                        g[p] = f[p] * c[j] - f[p + 1] * s[j];
                        g[p + 1] = f[p] * s[j] + f[p + 1] * c[j];
                    } else {
                        g0[j] = f0[j] * c[j] - f1[j] * s[j];
                        g1[j] = f0[j] * s[j] + f1[j] * c[j];
                    }
                }
                x0[i] = pack(g0);
                x1[i] = pack(g1);
            } else {
                x0[i] = pack(f0);
                x1[i] = pack(f1);
            }
        }
        if (e0 < vectors) *reinterpret_cast<uint4 *>(w[i].dst + e0 * N) = x0[i];
        if (e1 < vectors) *reinterpret_cast<uint4 *>(w[i].dst + e1 * N) = x1[i];
    }
}

template <typename T>
bool weights_by_vectors(const NormArgs &n) {
    constexpr int N = 16 / sizeof(T);
    return aligned16(n.q_weight) && aligned16(n.k_weight) && n.q_weight_head % N == 0 && n.k_weight_head % N == 0;
}

template <typename T, bool kInterleaved, int kRows>
cudaError_t launch_vectors(const NormArgs &n, int units, cudaStream_t st) {
    const int rows = n.r.n_heads + 2 * n.r.n_kv;
    const int need = (rows + kRows - 1) / kRows;             // rows of threads
    const int fit = 256 / units, blocks = (need + fit - 1) / fit, whole = 32 / units;
    const int each = ((need + blocks - 1) / blocks + whole - 1) / whole * whole;   // whole warps: their lanes add up together
    return launch_step(norm_vectors_kernel<T, kInterleaved, kRows>, dim3(n.r.n_tokens, blocks), dim3(units, each), 0, 1, st, n);
}

template <typename T, bool kInterleaved>
cudaError_t launch_norm(const NormArgs &n, int sms, cudaStream_t st) {
    const RopeArgs &a = n.r;
    const long long rows = (long long)a.n_tokens * (a.n_heads + 2 * a.n_kv);
    int units = 1;
    while (units < (a.head_dim / (int)(16 / sizeof(T)) + 1) / 2) units *= 2;
    if (units <= 32 && by_vectors<T>(a, kInterleaved) && weights_by_vectors<T>(n))
        return rows <= 64ll * sms ? launch_vectors<T, kInterleaved, 1>(n, units, st)
                                  : launch_vectors<T, kInterleaved, 4>(n, units, st);
    return launch_step(norm_rows_kernel<T, kInterleaved>, dim3((unsigned)((rows + 7) / 8)), dim3(256), 0, 1, st, n);
}

}  // namespace
}  // namespace lora

using namespace lora;
using namespace lora::step;
using namespace lora::rope;

extern "C" int lora_norm_rope(const lora_norm_rope_desc *d, void *stream) {
    if (!d) return fail(LORA_ERR_ARG, "norm_rope: NULL descriptor");
    bool nothing;
    const int rc = check(&d->rope, "norm_rope", &nothing);
    if (rc != LORA_OK) return rc;
    if (d->rope.inverse) return fail(LORA_ERR_ARG, "norm_rope: inverse is not 0 (the norm has no inverse here)");
    if (!(d->eps >= 0.f) || !std::isfinite(d->eps)) return fail(LORA_ERR_ARG, "norm_rope: eps must be finite and not negative");
    if (d->q_weight_head < 0 || d->k_weight_head < 0)
        return fail(LORA_ERR_ARG, "norm_rope: the weights' strides %lld, %lld are negative", (long long)d->q_weight_head,
                    (long long)d->k_weight_head);
    if (nothing) return LORA_OK;
    const NormArgs n{arguments(&d->rope), d->q_weight, d->k_weight, d->q_weight_head, d->k_weight_head, d->eps};
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int sms = sm_count();
    if (sms < 1) return fail(LORA_ERR_CUDA, "norm_rope: no CUDA device");
    cudaError_t e;
    if (d->rope.dtype == LORA_DTYPE_BF16)
        e = d->rope.interleaved ? launch_norm<__nv_bfloat16, true>(n, sms, st) : launch_norm<__nv_bfloat16, false>(n, sms, st);
    else
        e = d->rope.interleaved ? launch_norm<float, true>(n, sms, st) : launch_norm<float, false>(n, sms, st);
    return launched("norm_rope", e);
}
