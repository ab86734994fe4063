// Rotary positions: lora_rope_table (angles) and lora_rope (the rotation of q
// and k, with the append of k and v to a paged cache).
#include "step_util.cuh"

#include <cmath>

namespace lora {
namespace {

using namespace step;

// ---- the table -----------------------------------------------------------------
// Angles are formed in double (position * f has to be exact to ~1e-8 at
// positions of 1e6 and more, where a product in fp32 is off by 0.06 rad) and
// cos and sin rounded once.
struct TableArgs {
    float *table;
    int n_positions, half, scaling;
    double base, factor, original, low_freq, high_freq;
    double ramp_lo, ramp_hi, magnitude;
};

__device__ double pair_frequency(const TableArgs &a, int j) {
    const double f = pow(a.base, -(double)j / a.half);
    switch (a.scaling) {
        case LORA_ROPE_LINEAR:
            return f / a.factor;
        case LORA_ROPE_PIECES: {
            const double wave = 2.0 * M_PI / f;
            if (wave < a.original / a.high_freq) return f;
            if (wave > a.original / a.low_freq) return f / a.factor;
            const double m = (a.original / wave - a.low_freq) / (a.high_freq - a.low_freq);
            return (1.0 - m) * f / a.factor + m * f;
        }
        case LORA_ROPE_YARN: {
            const double ramp = fmin(fmax((j - a.ramp_lo) / fmax(a.ramp_hi - a.ramp_lo, 0.001), 0.0), 1.0);
            return f * (1.0 - ramp) + f / a.factor * ramp;
        }
        default:
            return f;
    }
}

constexpr int kTableRows = 64;   // positions of one block: the frequency of a pair is formed once for them

__global__ void __launch_bounds__(256) rope_table_kernel(TableArgs a) {
    const int p0 = blockIdx.x * kTableRows, p1 = min(p0 + kTableRows, a.n_positions);
    for (int j = threadIdx.x; j < a.half; j += blockDim.x) {
        const double f = pair_frequency(a, j);
        for (int p = p0; p < p1; ++p) {
            double s, c;
            sincos((double)p * f, &s, &c);
            float *row = a.table + (size_t)p * (2 * a.half);
            row[j] = (float)(c * a.magnitude);
            row[a.half + j] = (float)(s * a.magnitude);
        }
    }
}

// ---- the rotation ----------------------------------------------------------------
struct RopeArgs {
    const void *q, *k, *v;
    void *q_out, *k_cache, *v_cache;
    const int64_t *slots;
    const int32_t *positions;
    const float *table;
    long long q_token, q_head, qo_token, qo_head, k_token, k_head, v_token, v_head, c_page, c_slot, c_head;
    long long n_slots;
    int n_positions, page_size, n_tokens, n_heads, n_kv, head_dim, rot_dim, inverse;
};

// One warp per head row of one token; a lane takes pairs one by one.
template <typename T, bool kInterleaved>
__global__ void __launch_bounds__(256) rope_rows_kernel(RopeArgs a) {
    const int lane = threadIdx.x & 31;
    const int rows = a.n_heads + 2 * a.n_kv;
    const long long item = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (item >= (long long)a.n_tokens * rows) return;
    const int t = (int)(item / rows), r = (int)(item % rows);
    const int pos = a.positions[t];
    if (pos < 0 || pos >= a.n_positions) return;
    const T *src;
    T *dst;
    if (r < a.n_heads) {
        src = static_cast<const T *>(a.q) + t * a.q_token + r * a.q_head;
        dst = static_cast<T *>(a.q_out) + t * a.qo_token + r * a.qo_head;
    } else {
        const long long slot = a.slots[t];
        if (slot < 0 || slot >= a.n_slots) return;
        const bool is_v = r >= a.n_heads + a.n_kv;
        const int h = r - a.n_heads - (is_v ? a.n_kv : 0);
        const long long at = slot / a.page_size * a.c_page + slot % a.page_size * a.c_slot + h * a.c_head;
        src = is_v ? static_cast<const T *>(a.v) + t * a.v_token + h * a.v_head
                   : static_cast<const T *>(a.k) + t * a.k_token + h * a.k_head;
        dst = static_cast<T *>(is_v ? a.v_cache : a.k_cache) + at;
        if (is_v) {
            for (int i = lane; i < a.head_dim; i += 32) dst[i] = src[i];
            return;
        }
    }
    const int half = a.rot_dim / 2;
    const float *row = a.table + (size_t)pos * a.rot_dim;
    for (int j = lane; j < half; j += 32) {
        const float c = row[j], s = a.inverse ? -row[half + j] : row[half + j];
        const int i0 = kInterleaved ? 2 * j : j, i1 = kInterleaved ? 2 * j + 1 : j + half;
        const float x0 = to_f32(src[i0]), x1 = to_f32(src[i1]);
        dst[i0] = from_f32<T>(x0 * c - x1 * s);
        dst[i1] = from_f32<T>(x0 * s + x1 * c);
    }
    for (int i = a.rot_dim + lane; i < a.head_dim; i += 32) dst[i] = src[i];
}

template <typename T>
cudaError_t launch_rope(const RopeArgs &a, int interleaved, cudaStream_t st) {
    const long long items = (long long)a.n_tokens * (a.n_heads + 2 * a.n_kv);
    const unsigned grid = (unsigned)((items + 7) / 8);
    if (interleaved)
        rope_rows_kernel<T, true><<<grid, 256, 0, st>>>(a);
    else
        rope_rows_kernel<T, false><<<grid, 256, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace
}  // namespace lora

using namespace lora;
using namespace lora::step;

extern "C" int lora_rope_table(float *table, int n_positions, int rot_dim, int scaling, double base, double factor,
                               double original, double low_freq, double high_freq, void *stream) {
    if (n_positions < 0 || rot_dim < 2 || rot_dim > 512 || rot_dim % 2 != 0)
        return fail(LORA_ERR_ARG, "rope_table: n_positions %d, rot_dim %d (even, 2..512)", n_positions, rot_dim);
    if (scaling < LORA_ROPE_PLAIN || scaling > LORA_ROPE_YARN)
        return fail(LORA_ERR_ARG, "rope_table: unknown scaling %d", scaling);
    if (!(base > 1.0) || !std::isfinite(base)) return fail(LORA_ERR_ARG, "rope_table: base must be above 1");
    if (scaling != LORA_ROPE_PLAIN && (!(factor >= 1.0) || !std::isfinite(factor)))
        return fail(LORA_ERR_ARG, "rope_table: factor must be at least 1");
    if (scaling == LORA_ROPE_BASE && rot_dim < 4) return fail(LORA_ERR_ARG, "rope_table: rot_dim below 4");
    if ((scaling == LORA_ROPE_PIECES || scaling == LORA_ROPE_YARN) &&
        (!(original >= 1.0) || !std::isfinite(original) || !(low_freq > 0.0) || !(high_freq > low_freq) ||
         !std::isfinite(high_freq)))
        return fail(LORA_ERR_ARG, "rope_table: original >= 1 and 0 < low_freq < high_freq are needed");
    if (n_positions == 0) return LORA_OK;
    if (!table) return fail(LORA_ERR_ARG, "rope_table: NULL table");
    TableArgs a{table, n_positions, rot_dim / 2, scaling, base, factor, original, low_freq, high_freq, 0.0, 0.0, 1.0};
    if (scaling == LORA_ROPE_BASE) a.base = base * std::pow(factor, rot_dim / (rot_dim - 2.0));
    if (scaling == LORA_ROPE_YARN) {
        const double lb = 2.0 * std::log(base);
        a.ramp_lo = std::fmax(std::floor(rot_dim * std::log(original / (2.0 * M_PI * high_freq)) / lb), 0.0);
        a.ramp_hi = std::fmin(std::ceil(rot_dim * std::log(original / (2.0 * M_PI * low_freq)) / lb), rot_dim - 1.0);
        a.magnitude = factor > 1.0 ? 0.1 * std::log(factor) + 1.0 : 1.0;
    }
    rope_table_kernel<<<(n_positions + kTableRows - 1) / kTableRows, 256, 0, static_cast<cudaStream_t>(stream)>>>(a);
    return launched("rope_table", cudaGetLastError());
}

extern "C" int lora_rope(const lora_rope_desc *d, void *stream) {
    if (!d) return fail(LORA_ERR_ARG, "rope: NULL descriptor");
    if (!known_dtype(d->dtype)) return fail(LORA_ERR_ARG, "rope: unknown dtype %d", d->dtype);
    if (d->n_tokens < 0 || d->n_heads < 0 || d->n_kv_heads < 0 || d->head_dim < 2 || d->head_dim > 1024 ||
        d->n_heads > 65536 || d->n_kv_heads > 65536)
        return fail(LORA_ERR_ARG, "rope: n_tokens %d, n_heads %d, n_kv_heads %d, head_dim %d (2..1024)", d->n_tokens,
                    d->n_heads, d->n_kv_heads, d->head_dim);
    if (d->rot_dim < 2 || d->rot_dim % 2 != 0 || d->rot_dim > d->head_dim)
        return fail(LORA_ERR_ARG, "rope: rot_dim %d must be even and at most head_dim %d", d->rot_dim, d->head_dim);
    if (d->n_positions < 0) return fail(LORA_ERR_ARG, "rope: n_positions %d", d->n_positions);
    const bool append = d->n_kv_heads > 0;
    if (append && (d->page_size < 1 || d->n_pages < 0 || d->n_pages > INT64_MAX / d->page_size))
        return fail(LORA_ERR_ARG, "rope: page_size %d, n_pages %lld", d->page_size, (long long)d->n_pages);
    const long long items = (long long)d->n_tokens * (d->n_heads + 2ll * d->n_kv_heads);
    if (items > (1ll << 33)) return fail(LORA_ERR_ARG, "rope: too many rows (%lld)", items);
    if (items == 0) return LORA_OK;
    if (!d->positions || (!d->table && d->n_positions > 0) || (d->n_heads > 0 && (!d->q || !d->q_out)) ||
        (append && (!d->k || !d->v || !d->k_cache || !d->v_cache || !d->slots)))
        return fail(LORA_ERR_ARG, "rope: NULL pointer argument");
    RopeArgs a{d->q,       d->k,         d->v,          d->q_out,       d->k_cache,     d->v_cache,   d->slots,
               d->positions, d->table,   d->q_token,    d->q_head,      d->q_out_token, d->q_out_head, d->k_token,
               d->k_head,  d->v_token,   d->v_head,     d->cache_page,  d->cache_slot,  d->cache_head,
               append ? (long long)d->n_pages * d->page_size : 0,
               d->n_positions, append ? d->page_size : 1, d->n_tokens, d->n_heads, d->n_kv_heads, d->head_dim,
               d->rot_dim, d->inverse};
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t e = d->dtype == LORA_DTYPE_BF16 ? launch_rope<__nv_bfloat16>(a, d->interleaved, st)
                                                      : launch_rope<float>(a, d->interleaved, st);
    return launched("rope", e);
}
