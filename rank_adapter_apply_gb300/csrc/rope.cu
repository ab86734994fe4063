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
// cos and sin rounded once. Bound by the double precision units; built once.
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

// Where head row r of token t (q heads, then k, then v) is read and written.
template <typename T>
struct Row {
    const T *src;
    T *dst;          // nullptr: the row is not written
    bool turned;
};

template <typename T>
__device__ __forceinline__ Row<T> row_of(const RopeArgs &a, long long t, int r, long long cache_at) {
    Row<T> w{};
    if (r < a.n_heads) {
        w.src = static_cast<const T *>(a.q) + t * a.q_token + r * a.q_head;
        w.dst = static_cast<T *>(a.q_out) + t * a.qo_token + r * a.qo_head;
        w.turned = true;
        return w;
    }
    r -= a.n_heads;
    w.turned = r < a.n_kv;
    const int h = w.turned ? r : r - a.n_kv;
    w.src = w.turned ? static_cast<const T *>(a.k) + t * a.k_token + h * a.k_head
                     : static_cast<const T *>(a.v) + t * a.v_token + h * a.v_head;
    if (cache_at >= 0) w.dst = static_cast<T *>(w.turned ? a.k_cache : a.v_cache) + cache_at + h * a.c_head;
    return w;
}

// Element offset of the token's place in the caches, -1: it has none.
__device__ __forceinline__ long long cache_place(const RopeArgs &a, long long t) {
    if (a.n_kv == 0) return -1;
    const long long slot = a.slots[t];
    if (slot < 0 || slot >= a.n_slots) return -1;
    if ((slot >> 31) == 0) {                               // 32-bit division where it will do
        const uint32_t page = (uint32_t)slot / (uint32_t)a.page_size;
        return page * a.c_page + ((uint32_t)slot - page * (uint32_t)a.page_size) * a.c_slot;
    }
    return slot / a.page_size * a.c_page + slot % a.page_size * a.c_slot;
}

// Any layout: one warp per head row of one token, a lane takes pairs one by one. Bound by
// its issue slots; for rows that are not whole 16-byte vectors.
template <typename T, bool kInterleaved>
__global__ void __launch_bounds__(256) rope_rows_kernel(RopeArgs a) {
    grid_dependency_wait();
    grid_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int rows = a.n_heads + 2 * a.n_kv;
    const long long item = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (item >= (long long)a.n_tokens * rows) return;
    const long long t = item / rows;
    const int pos = a.positions[t];
    if (pos < 0 || pos >= a.n_positions) return;
    const Row<T> w = row_of<T>(a, t, (int)(item % rows), cache_place(a, t));
    if (!w.dst) return;
    const int half = a.rot_dim / 2;
    const float *row = a.table + (size_t)pos * a.rot_dim;
    if (w.turned) {
        for (int j = lane; j < half; j += 32) {
            const float c = row[j], s = a.inverse ? -row[half + j] : row[half + j];
            const int i0 = kInterleaved ? 2 * j : j, i1 = kInterleaved ? 2 * j + 1 : j + half;
            const float x0 = to_f32(w.src[i0]), x1 = to_f32(w.src[i1]);
            w.dst[i0] = from_f32<T>(x0 * c - x1 * s);
            w.dst[i1] = from_f32<T>(x0 * s + x1 * c);
        }
    }
    for (int i = (w.turned ? a.rot_dim : 0) + lane; i < a.head_dim; i += 32) w.dst[i] = w.src[i];
}

// Rows in 16-byte vectors. A unit is two vectors of a row that are turned
// together: halves: vectors u and u + rot_dim / 2 elements; interleaved: vectors 2u
// and 2u + 1; past rot_dim (and in v): two neighbours to copy. A block has `units`
// lanes for a row (unit = threadIdx.x) times blockDim.y rows; a thread takes its
// unit of kRows rows of one token, whose cosines and sines it reads once, with all
// loads in flight before the first is used. Bound by memory: 16384 tokens of 64 + 8 heads
// of 128, with the append, 110 us, 6.2 TB/s; 1021 tokens of 28 + 4 heads of 80 in fp32 6.9
// us from memory, 3.5 TB/s (the launch is 1.5 of them); 8 tokens of 32 + 8 heads 1.6 us in a
// graph, a launch and one round of reads.
__device__ __forceinline__ uint4 pack(const float (&f)[4]) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
}
__device__ __forceinline__ uint4 pack(const float (&f)[8]) {
    return make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
}

template <typename T, bool kInterleaved, int kRows>
__global__ void __launch_bounds__(512) rope_vectors_kernel(RopeArgs a) {
    constexpr int N = 16 / sizeof(T);
    grid_dependency_wait();
    grid_launch_dependents();
    const long long t = blockIdx.x;
    const int u = threadIdx.x, rows = a.n_heads + 2 * a.n_kv, r0 = (blockIdx.y * blockDim.y + threadIdx.y) * kRows;
    const int vectors = a.head_dim / N, rot_vectors = a.rot_dim / N, half = a.rot_dim / 2;
    const int pos = a.positions[t];
    const long long at = cache_place(a, t);
    if (pos < 0 || pos >= a.n_positions) return;
    // this unit's vectors in a row that is turned, and in one that is copied
    const bool turns = kInterleaved ? 2 * u < rot_vectors : u < rot_vectors / 2;
    const int v0 = kInterleaved || !turns ? 2 * u : u, v1 = kInterleaved || !turns ? 2 * u + 1 : u + rot_vectors / 2;
    Row<T> w[kRows];
    uint4 x0[kRows], x1[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        w[i].dst = nullptr;
        if (r0 + i < rows) w[i] = row_of<T>(a, t, r0 + i, at);
        if (!w[i].dst) continue;
        const int e0 = w[i].turned ? v0 : 2 * u, e1 = w[i].turned ? v1 : 2 * u + 1;
        x0[i] = *reinterpret_cast<const uint4 *>(w[i].src + e0 * N);
        if (e1 < vectors) x1[i] = *reinterpret_cast<const uint4 *>(w[i].src + e1 * N);
    }
    // N angles: of elements 2u N .. (interleaved: of N pairs) or u N ..
    float c[N], s[N];
    if (turns) {
        const float *row = a.table + (size_t)pos * a.rot_dim + u * N;
#pragma unroll
        for (int j = 0; j < N; ++j) {
            c[j] = row[j];
            s[j] = a.inverse ? -row[half + j] : row[half + j];
        }
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        if (!w[i].dst) continue;
        int e0 = 2 * u, e1 = 2 * u + 1;
        if (w[i].turned) {
            e0 = v0, e1 = v1;
            if (turns) {
                float f0[N], f1[N], g0[N], g1[N];
                unpack<T>(x0[i], f0);
                unpack<T>(x1[i], f1);
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
            }
        }
        *reinterpret_cast<uint4 *>(w[i].dst + e0 * N) = x0[i];
        if (e1 < vectors) *reinterpret_cast<uint4 *>(w[i].dst + e1 * N) = x1[i];
    }
}

// Whether every row is whole 16-byte vectors at 16-byte addresses and the pairs
// fall into units.
template <typename T>
bool by_vectors(const RopeArgs &a, bool interleaved) {
    constexpr int N = 16 / sizeof(T);
    bool ok = a.head_dim % N == 0 && a.rot_dim % (interleaved ? N : 2 * N) == 0 && (a.head_dim / N + 1) / 2 <= 128;
    // an interleaved unit may not be half turned and half copied
    ok = ok && (a.rot_dim / N % 2 == 0);
    const long long q[] = {a.q_token, a.q_head, a.qo_token, a.qo_head};
    const long long kv[] = {a.k_token, a.k_head, a.v_token, a.v_head, a.c_page, a.c_slot, a.c_head};
    if (a.n_heads > 0) {
        ok = ok && aligned16(a.q) && aligned16(a.q_out);
        for (long long s : q) ok = ok && s % N == 0;
    }
    if (a.n_kv > 0) {
        ok = ok && aligned16(a.k) && aligned16(a.v) && aligned16(a.k_cache) && aligned16(a.v_cache);
        for (long long s : kv) ok = ok && s % N == 0;
    }
    return ok;
}

template <typename T, bool kInterleaved, int kRows>
cudaError_t launch_vectors(const RopeArgs &a, cudaStream_t st) {
    constexpr int N = 16 / sizeof(T);
    const int rows = a.n_heads + 2 * a.n_kv, units = (a.head_dim / N + 1) / 2;
    const int need = (rows + kRows - 1) / kRows;             // rows of threads
    const int fit = 256 / units > 0 ? 256 / units : 1;
    const int blocks = (need + fit - 1) / fit, each = (need + blocks - 1) / blocks;
    return launch_step(rope_vectors_kernel<T, kInterleaved, kRows>, dim3(a.n_tokens, blocks), dim3(units, each), 0, 1, st, a);
}

template <typename T, bool kInterleaved>
cudaError_t launch_rope(const RopeArgs &a, int sms, cudaStream_t st) {
    const long long rows = (long long)a.n_tokens * (a.n_heads + 2 * a.n_kv);
    if (by_vectors<T>(a, kInterleaved))
        // rows of a thread, one / four: 8 tokens of 48 rows 1.9 / 2.8 us, 128 2.4 / 2.9, 256 3.1 / 3.2, 512 4.8 / 4.1, 1024
        // 8.1 / 7.5
        return rows <= 64ll * sms ? launch_vectors<T, kInterleaved, 1>(a, st) : launch_vectors<T, kInterleaved, 4>(a, st);
    return launch_step(rope_rows_kernel<T, kInterleaved>, dim3((unsigned)((rows + 7) / 8)), dim3(256), 0, 1, st, a);
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
    if (!rows_apart(d->n_tokens, d->q_out_token, d->n_heads, d->q_out_head, d->head_dim))
        return fail(LORA_ERR_ARG, "rope: the rows of q_out overlap (strides %lld, %lld)", (long long)d->q_out_token,
                    (long long)d->q_out_head);
    if (append && (!rows_apart(d->n_pages, d->cache_page, d->page_size, d->cache_slot, d->head_dim) ||
                   !rows_apart(d->n_pages, d->cache_page, d->n_kv_heads, d->cache_head, d->head_dim) ||
                   !rows_apart(d->page_size, d->cache_slot, d->n_kv_heads, d->cache_head, d->head_dim)))
        return fail(LORA_ERR_ARG, "rope: rows of the caches overlap (strides %lld, %lld, %lld)", (long long)d->cache_page,
                    (long long)d->cache_slot, (long long)d->cache_head);
    RopeArgs a{d->q,       d->k,         d->v,          d->q_out,       d->k_cache,     d->v_cache,   d->slots,
               d->positions, d->table,   d->q_token,    d->q_head,      d->q_out_token, d->q_out_head, d->k_token,
               d->k_head,  d->v_token,   d->v_head,     d->cache_page,  d->cache_slot,  d->cache_head,
               append ? (long long)d->n_pages * d->page_size : 0,
               d->n_positions, append ? d->page_size : 1, d->n_tokens, d->n_heads, d->n_kv_heads, d->head_dim,
               d->rot_dim, d->inverse};
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int sms = sm_count();
    if (sms < 1) return fail(LORA_ERR_CUDA, "rope: no CUDA device");
    cudaError_t e;
    if (d->dtype == LORA_DTYPE_BF16)
        e = d->interleaved ? launch_rope<__nv_bfloat16, true>(a, sms, st) : launch_rope<__nv_bfloat16, false>(a, sms, st);
    else
        e = d->interleaved ? launch_rope<float, true>(a, sms, st) : launch_rope<float, false>(a, sms, st);
    return launched("rope", e);
}
