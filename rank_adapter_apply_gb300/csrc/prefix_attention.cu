// lora_prefix_attention: attention of requests that share a prefix of their context.
//
// Entries are of two kinds: a group, whose rows are those of all its requests and whose
// keys are the prefix, read once for each tile of its rows, and a request with its own keys. In bf16
// few rows go to single warps (prefix_rows.cuh) and many to tiles of 128 on the
// 5th-generation tensor cores (tree_attention_tc.cu, which takes up the few rows as its
// CTAs are done); fp32 goes to the FMA units (tree_attention_f32.cu). A row's two
// results, and the parts of a unit that was cut, are joined in fp32 by the last kernel:
// O = sum 2^(m_i - m) O_i, l = sum 2^(m_i - m) l_i, m = max m_i, out = O / l.
//
// 64 requests behind two prefixes of 8192, own contexts of up to 1000, 32 heads over 8 of 128:
// 69 us; keys and values are read in 29. Of it the prefixes take 25, the requests' keys some
// 25 at 5 TB/s, the rest are the beginnings of the three parts and the join. 256 requests behind
// 32768 keys, 64 heads over 8: 370 us, the products alone 148; the prefix's part runs at 1.2
// PFLOP/s (the chain of scores, softmax, second product), the requests' 0.5 GB at 5 TB/s.
// 3 requests behind 777: 12.5 us in a graph, 13.2 a call: two launches and five dependent reads.
#include "tree_common.cuh"

#include <algorithm>
#include <cmath>

namespace lora {
namespace {

using namespace step;
using namespace tree;

// Rows up to which eight warps, and two, join one. Calls with eight / two / one warps, us, a group behind 1000 keys with
// contexts of up to 300: 96 rows 13.0 / 16.8 / 22.0, 768 17.8 / 19.5 / 23.1, 2048 30.0 / 27.4 / 29.3, 2400 33.8 / 29.7 / 31.0, 4096 56 /
// 49.6 / 47.7, 9600 80 / 61.7 / 58.5, 16384 122 / 91 / 85. (Eight are right below some 1200 rows, two up to some 3000: what
// lies between these and the limits below loses 2 to 4 us.)
constexpr long long kJoin8 = 2400, kJoin2 = 9600;

struct JoinArgs {
    TreeArgs a;
    Plan plan[2];                                        // of the groups' and of the requests' launch
    int m_rows[2];                                       // rows of their parts
};

// kEach warps of a block join a row: its parts of the group's unit and of the request's, in a
// row, are dealt to them. All that is read first is read at once; whether the group's entry is
// the row's own is known only later. Latency: two rounds of reads where a warp has at most
// kAhead parts.
template <typename T, int DP, int kEach>
__global__ void __launch_bounds__(256) prefix_join_kernel(const __grid_constant__ JoinArgs args) {
    constexpr int V = Joined<DP>::V, kAhead = 4;
    __shared__ float so[8][DP];
    __shared__ float2 sm[8];
    const TreeArgs &a = args.a;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = warp % kEach;
    grid_dependency_wait();
    grid_launch_dependents();
    const size_t rows = (size_t)a.n_tokens * a.n_heads, row = (size_t)blockIdx.x * (8 / kEach) + warp / kEach;
    const bool real = row < rows;
    const int token = real ? (int)(row / a.n_heads) : 0, head = real ? (int)(row % a.n_heads) : 0;
    int4 named[2];
    named[0] = named[1] = make_int4(0, 0, 0, -1);
    int g0 = 0, g1 = 0;
    if (real) named[1] = a.row_at[rows + row];
    if (real && a.n_groups > 0) {
        named[0] = a.row_at[row];
        g0 = group_start(a, 0);
        g1 = group_start(a, a.n_groups);
    }
    const int first = node_start(a, 0), last = node_start(a, a.n_requests);
    const bool mine = real && token >= first && token < last;            // of a request
    if (a.n_groups > 0 && (token < node_start(a, g0) || token >= node_start(a, g1))) named[0].w = -1;   // of no group
    int parts[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        // what starts that fall leave there leads nowhere
        const int4 n = named[k];
        const bool ok = mine && n.w == (int)row && n.y >= 0 && n.x >= 0 && n.x < args.plan[k].ctas &&
                        n.y <= args.plan[k].ctas - n.x && n.z >= 0 && n.z < args.m_rows[k];
        parts[k] = ok ? max(n.y, 1) : 0;
    }
    Joined<DP> all;
#pragma unroll
    for (int e = 0; e < V; ++e) all.o[e] = 0.f;
    const int n_parts = parts[0] + parts[1];
    for (int p0 = sub; p0 < n_parts; p0 += kEach * kAhead) {
        alignas(4 * V) float v[kAhead][V];
        float2 ml[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int i = p0 + u * kEach;
            if (i >= n_parts) break;
            const int k = i < parts[0] ? 0 : 1, p = k == 0 ? i : i - parts[0];
            const int4 n = k == 0 ? named[0] : named[1];
            const float *o = a.row_o + ((size_t)k * rows + row) * DP;
            const float2 *stat = a.row_ml + (size_t)k * rows + row;
            if (n.y > 0) {
                const size_t at = (size_t)(p == 0 ? 2 * n.x + 1 : 2 * (n.x + p)) * args.m_rows[k] + n.z;
                o = args.plan[k].part + at * DP;
                stat = args.plan[k].stat + at;
            }
            ml[u] = *stat;
            if constexpr (V == 4)
                *reinterpret_cast<float4 *>(v[u]) = *reinterpret_cast<const float4 *>(o + lane * V);
            else
                *reinterpret_cast<float2 *>(v[u]) = *reinterpret_cast<const float2 *>(o + lane * V);
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
            if (p0 + u * kEach < n_parts) all.add(ml[u], v[u]);
    }
    if constexpr (kEach > 1) {
#pragma unroll
        for (int e = 0; e < V; ++e) so[warp][lane * V + e] = all.o[e];
        if (lane == 0) sm[warp] = make_float2(all.m, all.l);
        __syncthreads();
        if (sub > 0) return;
#pragma unroll
        for (int w = 1; w < kEach; ++w) {
            float v[V];
#pragma unroll
            for (int e = 0; e < V; ++e) v[e] = so[warp + w][lane * V + e];
            all.add(sm[warp + w], v);
        }
    }
    if (mine) store_joined<T, DP>(a, token, head, all);
}

// Entries [first, first + count).
TreeArgs entries_of(TreeArgs a, int first, int count) {
    a.first = first;
    a.count = count;
    return a;
}

template <typename T, int DP>
cudaError_t launch_prefix(const TreeArgs &a, const Plan &groups, const Plan &requests, cudaStream_t st) {
    constexpr bool kBf16 = sizeof(T) == 2;
    const double group = a.n_heads / a.n_kv;
    JoinArgs join{a, {groups, requests}, {0, 0}};
    // Rows of a tile for n entries with up to so many pages of keys. In bf16 the warps' tiles of 16 read the keys again for
    // each tile, mostly from L2; the 5th-generation tensor cores read them once for 128 rows, but their kernel takes some
    // 20 us, and layouts that it does not take stay on 16 (256x1 of 8192, 64 heads over 8: 133 us with pages of 64, 584 with
    // pages of 12). Bytes read by the warps, and us with both kinds on 16 / with the wide one on 128: 55 MB (100x2 of 300) 40 / 62,
    // 65 MB (16x1 of 4000 in 2 groups) 23 / 29, 142 MB (requests of 16x16 of 1000) 49 / 31, 201 MB (12x1 of 16384) 45 / 36.
    // In fp32 tiles of 64 rows feed the FMA units better, and take a launch of their own beside 16: all wide entries take
    // them, or none. us with 16 / 64: 8 MB (8x4 of 500) 15 / 29, 20 MB (24x2 of 1024) 28 / 32, 50 MB (32x2 of 2000)
    // 46 / 45, 262 MB (32x4 of 4000) 153 / 91
    auto rows_of = [&](int n) { return a.n_tokens * group / std::max(n, 1); };
    auto bytes = [&](int n, double pages) {
        return std::ceil(rows_of(n) / 16.0) * n * a.n_kv * pages * a.page_size * a.head_dim * 2.0 * sizeof(T);
    };
    auto wide_bytes = [&](int n, int pages) { return rows_of(n) <= 16.0 ? 0.0 : bytes(n, pages); };
    const double wide = wide_bytes(a.n_groups, a.prefix_pages) + wide_bytes(a.n_requests, a.table_pages);
    auto tile = [&](int n, int pages) {
        if (!kBf16) return rows_of(n) <= 16.0 || wide <= 30e6 ? 16 : 64;
        return rows_of(n) <= 16.0 || bytes(n, pages) <= 80e6 || !tc_takes(a) ? 16 : 128;
    };
    int of_requests = tile(a.n_requests, a.table_pages);
    int of_groups = a.n_groups > 0 ? tile(a.n_groups, a.prefix_pages) : of_requests;
    const TreeArgs all = entries_of(a, 0, a.n_groups + a.n_requests), groups_alone = entries_of(a, 0, a.n_groups);
    const TreeArgs requests_alone = entries_of(a, a.n_groups, a.n_requests);
    Plan *const plan = join.plan;
    cudaError_t e = cudaErrorNotSupported;
    if (!kBf16) {
        if (of_groups == of_requests) {
            plan[0] = plan[1];
            e = launch_f32(all, plan[1], of_requests, st);
        } else {
            e = launch_f32(groups_alone, plan[0], of_groups, st);
            if (e == cudaSuccess) e = launch_f32(requests_alone, plan[1], of_requests, st);
        }
    } else {
        if (of_groups == 128 && of_requests == 128) {
            e = launch_mixed(all, plan[1], entries_of(a, 0, 0), plan[0], st);
            plan[0] = plan[1];
        } else if (of_groups == 128) {
            e = launch_mixed(groups_alone, plan[0], requests_alone, plan[1], st);
        } else if (of_requests == 128) {
            e = launch_mixed(requests_alone, plan[1], groups_alone, plan[0], st);
        }
        if (e == cudaErrorNotSupported) {
            of_groups = of_requests = 16;
            e = launch_rows(all, plan[1], st);
            plan[0] = plan[1];
        }
    }
    if (e != cudaSuccess) return e;
    join.m_rows[0] = of_groups;
    join.m_rows[1] = of_requests;
    const long long rows = (long long)a.n_tokens * a.n_heads;
    auto join_by = [&](auto kernel, int each) {
        return launch_step(kernel, dim3((unsigned)((rows * each + 7) / 8)), dim3(256), 0, 1, st, join);
    };
    if (rows <= kJoin8) return join_by(prefix_join_kernel<T, DP, 8>, 8);
    if (rows <= kJoin2) return join_by(prefix_join_kernel<T, DP, 2>, 2);
    return join_by(prefix_join_kernel<T, DP, 1>, 1);
}

size_t padded(size_t bytes) { return (bytes + 255) / 256 * 256; }

}  // namespace
}  // namespace lora

using namespace lora;
using namespace lora::step;

extern "C" size_t lora_prefix_attention_workspace_bytes(int n_requests, int n_groups, int n_tokens, int n_heads,
                                                        int n_kv_heads, int head_dim, int dtype) {
    if (n_groups < 0 || !tree::shape_ok(n_requests, n_tokens, n_heads, n_kv_heads, head_dim, dtype) ||
        (long long)n_tokens * n_heads > (1 << 30))
        return 0;
    // the parts of two launches, then two results of every row and where they are
    const size_t rows = 2 * (size_t)n_tokens * n_heads;
    return 2 * padded(tree::plan_bytes()) + padded(rows * (head_dim <= 64 ? 64 : 128) * sizeof(float)) +
           padded(rows * sizeof(float2)) + padded(rows * sizeof(int4));
}

extern "C" int lora_prefix_attention(const lora_prefix_attention_desc *d, void *stream) {
    if (!d) return fail(LORA_ERR_ARG, "prefix_attention: NULL descriptor");
    const lora_tree_attention_desc &t = d->tree;
    if (d->n_groups < 0 || d->n_groups > INT32_MAX - std::max(t.n_requests, 0) || d->prefix_pages < 0 || d->prefix_stride < 0)
        return fail(LORA_ERR_ARG, "prefix_attention: n_groups %d, prefix_pages %d, prefix_stride %lld", d->n_groups,
                    d->prefix_pages, (long long)d->prefix_stride);
    bool nothing;
    const int rc = tree::check(&t, "prefix_attention",
                               lora_prefix_attention_workspace_bytes(t.n_requests, d->n_groups, t.n_tokens, t.n_heads,
                                                                     t.n_kv_heads, t.head_dim, t.dtype),
                               &nothing);
    if (rc != LORA_OK || nothing) return rc;
    if (d->n_groups > 0 && (!d->prefix_lens || !d->group_starts || (d->prefix_pages > 0 && !d->prefix_table)))
        return fail(LORA_ERR_ARG, "prefix_attention: NULL pointer argument");
    TreeArgs a = tree::arguments(&t);
    const int ctas = tree::grid_of_device();
    if (ctas < 1) return fail(LORA_ERR_CUDA, "prefix_attention: no CUDA device");
    const size_t plan = padded(tree::plan_bytes()), rows = 2 * (size_t)a.n_tokens * a.n_heads;
    unsigned char *ws = static_cast<unsigned char *>(t.workspace);
    const Plan groups = tree::plan_at(ws, ctas), requests = tree::plan_at(ws + plan, ctas);
    a.row_o = reinterpret_cast<float *>(ws + 2 * plan);
    const size_t o_bytes = padded(rows * (a.head_dim <= 64 ? 64 : 128) * sizeof(float));
    a.row_ml = reinterpret_cast<float2 *>(ws + 2 * plan + o_bytes);
    a.row_at = reinterpret_cast<int4 *>(ws + 2 * plan + o_bytes + padded(rows * sizeof(float2)));
    a.prefix_table = d->prefix_table;
    a.prefix_stride = d->prefix_stride;
    a.prefix_lens = d->prefix_lens;
    a.group_starts = d->group_starts;
    a.n_groups = d->n_groups;
    a.prefix_pages = d->prefix_pages;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (t.dtype == LORA_DTYPE_BF16)
        e = a.head_dim <= 64 ? launch_prefix<__nv_bfloat16, 64>(a, groups, requests, st)
                             : launch_prefix<__nv_bfloat16, 128>(a, groups, requests, st);
    else
        e = a.head_dim <= 64 ? launch_prefix<float, 64>(a, groups, requests, st)
                             : launch_prefix<float, 128>(a, groups, requests, st);
    return launched("prefix_attention", e);
}
