// Shared by lora_rope (rope.cu) and lora_norm_rope (norm_rope.cu): arguments and
// their checks, where rows are read and written, rows in 16-byte vectors.
#pragma once

#include "step_util.cuh"

namespace lora {
namespace rope {

using namespace step;

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

// Element offset of a slot in the caches, -1: it is none of theirs.
__device__ __forceinline__ long long place_of(const RopeArgs &a, long long slot) {
    if (slot < 0 || slot >= a.n_slots) return -1;
    if ((slot >> 31) == 0) {                               // 32-bit division where it will do
        const uint32_t page = (uint32_t)slot / (uint32_t)a.page_size;
        return page * a.c_page + ((uint32_t)slot - page * (uint32_t)a.page_size) * a.c_slot;
    }
    return slot / a.page_size * a.c_page + slot % a.page_size * a.c_slot;
}

// Element offset of the token's place in the caches, -1: it has none.
__device__ __forceinline__ long long cache_place(const RopeArgs &a, long long t) {
    return a.n_kv == 0 ? -1 : place_of(a, a.slots[t]);
}

__device__ __forceinline__ uint4 pack(const float (&f)[4]) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
}
__device__ __forceinline__ uint4 pack(const float (&f)[8]) {
    return make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
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

// The checks of a call, under its name; *nothing: there is nothing to do.
inline int check(const lora_rope_desc *d, const char *name, bool *nothing) {
    *nothing = false;
    if (!known_dtype(d->dtype)) return fail(LORA_ERR_ARG, "%s: unknown dtype %d", name, d->dtype);
    if (d->n_tokens < 0 || d->n_heads < 0 || d->n_kv_heads < 0 || d->head_dim < 2 || d->head_dim > 1024 ||
        d->n_heads > 65536 || d->n_kv_heads > 65536)
        return fail(LORA_ERR_ARG, "%s: n_tokens %d, n_heads %d, n_kv_heads %d, head_dim %d (2..1024)", name, d->n_tokens,
                    d->n_heads, d->n_kv_heads, d->head_dim);
    if (d->rot_dim < 2 || d->rot_dim % 2 != 0 || d->rot_dim > d->head_dim)
        return fail(LORA_ERR_ARG, "%s: rot_dim %d must be even and at most head_dim %d", name, d->rot_dim, d->head_dim);
    if (d->n_positions < 0) return fail(LORA_ERR_ARG, "%s: n_positions %d", name, d->n_positions);
    const bool append = d->n_kv_heads > 0;
    if (append && (d->page_size < 1 || d->n_pages < 0 || d->n_pages > INT64_MAX / d->page_size))
        return fail(LORA_ERR_ARG, "%s: page_size %d, n_pages %lld", name, d->page_size, (long long)d->n_pages);
    const long long items = (long long)d->n_tokens * (d->n_heads + 2ll * d->n_kv_heads);
    if (items > (1ll << 33)) return fail(LORA_ERR_ARG, "%s: too many rows (%lld)", name, items);
    *nothing = items == 0;
    if (items == 0) return LORA_OK;
    if (!d->positions || (!d->table && d->n_positions > 0) || (d->n_heads > 0 && (!d->q || !d->q_out)) ||
        (append && (!d->k || !d->v || !d->k_cache || !d->v_cache || !d->slots)))
        return fail(LORA_ERR_ARG, "%s: NULL pointer argument", name);
    if (!rows_apart(d->n_tokens, d->q_out_token, d->n_heads, d->q_out_head, d->head_dim))
        return fail(LORA_ERR_ARG, "%s: the rows of q_out overlap (strides %lld, %lld)", name, (long long)d->q_out_token,
                    (long long)d->q_out_head);
    if (append && (!rows_apart(d->n_pages, d->cache_page, d->page_size, d->cache_slot, d->head_dim) ||
                   !rows_apart(d->n_pages, d->cache_page, d->n_kv_heads, d->cache_head, d->head_dim) ||
                   !rows_apart(d->page_size, d->cache_slot, d->n_kv_heads, d->cache_head, d->head_dim)))
        return fail(LORA_ERR_ARG, "%s: rows of the caches overlap (strides %lld, %lld, %lld)", name, (long long)d->cache_page,
                    (long long)d->cache_slot, (long long)d->cache_head);
    return LORA_OK;
}

inline RopeArgs arguments(const lora_rope_desc *d) {
    const bool append = d->n_kv_heads > 0;
    return {d->q, d->k, d->v, d->q_out, d->k_cache, d->v_cache, d->slots,
            d->positions, d->table, d->q_token, d->q_head, d->q_out_token, d->q_out_head, d->k_token,
            d->k_head, d->v_token, d->v_head, d->cache_page, d->cache_slot, d->cache_head,
            append ? (long long)d->n_pages * d->page_size : 0,
            d->n_positions, append ? d->page_size : 1, d->n_tokens, d->n_heads, d->n_kv_heads, d->head_dim,
            d->rot_dim, d->inverse};
}

}  // namespace rope
}  // namespace lora
