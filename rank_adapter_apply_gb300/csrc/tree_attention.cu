// lora_tree_attention: attention of drafted trees over a paged cache.
#include "step_util.cuh"

#include <cmath>

namespace lora {
namespace {

using namespace step;

struct TreeArgs {
    const void *q, *k_cache, *v_cache;
    void *out;
    float *lse;
    const int32_t *page_table, *ctx_lens, *node_starts;
    const uint64_t *tree_mask;
    long long q_token, q_head, c_page, c_slot, c_head, o_token, o_head, table_stride, n_pages;
    float scale;
    int page_size, table_pages, mask_words, n_requests, n_tokens, n_heads, n_kv, head_dim;
};

__device__ __forceinline__ int node_start(const TreeArgs &a, int b) {
    return min(max(a.node_starts[b], 0), a.n_tokens);
}

// Request that owns node `t`: the last b with node_starts[b] <= t, or -1.
__device__ int request_of(const TreeArgs &a, int t) {
    int lo = 0, hi = a.n_requests;           // invariant: start(lo) <= t < start(hi), if any
    if (node_start(a, 0) > t || node_start(a, a.n_requests) <= t) return -1;
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (node_start(a, mid) <= t) lo = mid; else hi = mid;
    }
    return lo;
}

__device__ __forceinline__ float4 load4(const float *p) { return *reinterpret_cast<const float4 *>(p); }
__device__ __forceinline__ float4 load4(const __nv_bfloat16 *p) {
    const uint2 u = *reinterpret_cast<const uint2 *>(p);
    return make_float4(bf_lo(u.x), bf_hi(u.x), bf_lo(u.y), bf_hi(u.y));
}
__device__ __forceinline__ void store4(float *p, float4 v) { *reinterpret_cast<float4 *>(p) = v; }
__device__ __forceinline__ void store4(__nv_bfloat16 *p, float4 v) {
    *reinterpret_cast<uint2 *>(p) = make_uint2(pack_bf16(v.x, v.y), pack_bf16(v.z, v.w));
}

// One CTA of four warps for each query row; a warp takes every fourth key, a
// lane four elements of the head; the running maximum and sum in fp32, the
// four warps joined at the end.
template <typename T>
__global__ void __launch_bounds__(128) tree_rows_kernel(TreeArgs a) {
    const int t = blockIdx.x, h = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int b = request_of(a, t);
    if (b < 0) return;
    const int start = node_start(a, b), nodes = node_start(a, b + 1) - start, self = t - start;
    const long long ctx = max(a.ctx_lens[b], 0);
    long long keys = ctx + nodes;
    const long long room = (long long)a.table_pages * a.page_size;
    if (keys > room) keys = room;
    const bool mine = lane * 4 < a.head_dim;
    const float4 q = mine ? load4(static_cast<const T *>(a.q) + t * a.q_token + h * a.q_head + lane * 4)
                          : make_float4(0.f, 0.f, 0.f, 0.f);
    const long long head_at = (long long)(h / (a.n_heads / a.n_kv)) * a.c_head + lane * 4;
    const int32_t *pages = a.page_table + b * a.table_stride;
    float m = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (long long p = warp; p < keys; p += 4) {
        if (p >= ctx) {
            const long long j = p - ctx;
            bool sees = j <= self;
            if (a.tree_mask)
                sees = j < 64ll * a.mask_words && (a.tree_mask[(size_t)t * a.mask_words + j / 64] >> (j % 64) & 1);
            if (!sees) continue;
        }
        const int page = pages[p / a.page_size];
        if (page < 0 || page >= a.n_pages) continue;
        const long long at = page * a.c_page + p % a.page_size * a.c_slot + head_at;
        float4 k = make_float4(0.f, 0.f, 0.f, 0.f), v = k;
        if (mine) {
            k = load4(static_cast<const T *>(a.k_cache) + at);
            v = load4(static_cast<const T *>(a.v_cache) + at);
        }
        const float s = warp_sum(q.x * k.x + q.y * k.y + q.z * k.z + q.w * k.w) * a.scale;
        const float m2 = fmaxf(m, s);
        if (m2 == -INFINITY) continue;
        const float keep = expf(m - m2), w = expf(s - m2);
        m = m2;
        l = l * keep + w;
        o.x = o.x * keep + w * v.x;
        o.y = o.y * keep + w * v.y;
        o.z = o.z * keep + w * v.z;
        o.w = o.w * keep + w * v.w;
    }
    __shared__ float sm[4], sl[4];
    __shared__ float4 so[4][32];
    if (lane == 0) sm[warp] = m, sl[warp] = l;
    so[warp][lane] = o;
    __syncthreads();
    if (warp != 0) return;
    const float top = fmaxf(fmaxf(sm[0], sm[1]), fmaxf(sm[2], sm[3]));
    float sum = 0.f;
    o = make_float4(0.f, 0.f, 0.f, 0.f);
    if (top != -INFINITY) {
        for (int w = 0; w < 4; ++w) {
            const float f = expf(sm[w] - top);
            sum += f * sl[w];
            o.x += f * so[w][lane].x;
            o.y += f * so[w][lane].y;
            o.z += f * so[w][lane].z;
            o.w += f * so[w][lane].w;
        }
        const float r = 1.f / sum;
        o = make_float4(o.x * r, o.y * r, o.z * r, o.w * r);
    }
    if (mine) store4(static_cast<T *>(a.out) + t * a.o_token + h * a.o_head + lane * 4, o);
    if (a.lse && lane == 0) a.lse[(size_t)t * a.n_heads + h] = top == -INFINITY ? -INFINITY : top + logf(sum);
}

bool shape_ok(int n_requests, int n_tokens, int n_heads, int n_kv, int head_dim, int dtype) {
    return known_dtype(dtype) && n_requests >= 0 && n_tokens >= 0 && n_heads >= 1 && n_heads <= 65535 && n_kv >= 1 &&
           n_heads % n_kv == 0 && head_dim >= 8 && head_dim <= 128 && head_dim % 8 == 0;
}

}  // namespace
}  // namespace lora

using namespace lora;
using namespace lora::step;

extern "C" size_t lora_tree_attention_workspace_bytes(int n_requests, int n_tokens, int n_heads, int n_kv_heads,
                                                      int head_dim, int dtype) {
    if (!shape_ok(n_requests, n_tokens, n_heads, n_kv_heads, head_dim, dtype)) return 0;
    return 256;
}

extern "C" int lora_tree_attention(const lora_tree_attention_desc *d, void *stream) {
    if (!d) return fail(LORA_ERR_ARG, "tree_attention: NULL descriptor");
    if (!shape_ok(d->n_requests, d->n_tokens, d->n_heads, d->n_kv_heads, d->head_dim, d->dtype))
        return fail(LORA_ERR_ARG,
                    "tree_attention: dtype %d, n_requests %d, n_tokens %d, n_heads %d (a multiple of n_kv_heads %d), "
                    "head_dim %d (a multiple of 8, 8..128)",
                    d->dtype, d->n_requests, d->n_tokens, d->n_heads, d->n_kv_heads, d->head_dim);
    if (d->page_size < 1 || d->table_pages < 0 || d->n_pages < 0 || d->mask_words < 0)
        return fail(LORA_ERR_ARG, "tree_attention: page_size %d, table_pages %d, n_pages %lld, mask_words %d",
                    d->page_size, d->table_pages, (long long)d->n_pages, d->mask_words);
    if (!std::isfinite(d->scale)) return fail(LORA_ERR_ARG, "tree_attention: scale is not finite");
    if (d->n_tokens == 0 || d->n_requests == 0) return LORA_OK;
    if (!d->q || !d->out || !d->ctx_lens || !d->node_starts || (d->table_pages > 0 && !d->page_table) ||
        (d->n_pages > 0 && (!d->k_cache || !d->v_cache)))
        return fail(LORA_ERR_ARG, "tree_attention: NULL pointer argument");
    if (d->tree_mask && d->mask_words == 0) return fail(LORA_ERR_ARG, "tree_attention: mask_words is 0");
    const long long eb = d->dtype == LORA_DTYPE_F32 ? 4 : 2;
    const long long strides[] = {(long long)d->q_token,   (long long)d->q_head,     (long long)d->cache_page,
                                 (long long)d->cache_slot, (long long)d->cache_head, (long long)d->out_token,
                                 (long long)d->out_head};
    bool ok = aligned16(d->q) && aligned16(d->out) && aligned16(d->k_cache) && aligned16(d->v_cache);
    for (long long s : strides) ok = ok && s * eb % 16 == 0;
    if (!ok) return fail(LORA_ERR_ARG, "tree_attention: q, out and cache pointers and strides must be multiples of 16 bytes");
    const size_t need = lora_tree_attention_workspace_bytes(d->n_requests, d->n_tokens, d->n_heads, d->n_kv_heads,
                                                            d->head_dim, d->dtype);
    if (!d->workspace || d->workspace_bytes < need || reinterpret_cast<uintptr_t>(d->workspace) % 256)
        return fail(LORA_ERR_ARG, "tree_attention: workspace of %zu bytes, 256-byte aligned, is needed", need);
    TreeArgs a{d->q,       d->k_cache,   d->v_cache,   d->out,       d->lse,       d->page_table, d->ctx_lens,
               d->node_starts, d->tree_mask, d->q_token, d->q_head,  d->cache_page, d->cache_slot, d->cache_head,
               d->out_token, d->out_head, d->table_stride, d->n_pages, d->scale,   d->page_size,  d->table_pages,
               d->mask_words, d->n_requests, d->n_tokens, d->n_heads, d->n_kv_heads, d->head_dim};
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    dim3 grid(d->n_tokens, d->n_heads);
    if (d->dtype == LORA_DTYPE_BF16)
        tree_rows_kernel<__nv_bfloat16><<<grid, 128, 0, st>>>(a);
    else
        tree_rows_kernel<float><<<grid, 128, 0, st>>>(a);
    return launched("tree_attention", cudaGetLastError());
}
