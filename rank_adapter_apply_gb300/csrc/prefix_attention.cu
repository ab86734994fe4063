// lora_prefix_attention: attention of requests that share a prefix of their context.
//
// The kernels are lora_tree_attention's, over the entries of two kinds: a group, whose
// rows are those of all its requests and whose keys are the prefix, read once for them
// all, and a request with its own keys. Where both kinds take row tiles of one kernel
// they go in one launch; else the groups', which have more rows, go first, in tiles
// of 128 on the 5th-generation tensor cores. A row's two results, and the parts of a unit
// that was cut, are joined in fp32 by the last kernel: O = sum 2^(m_i - m) O_i,
// l = sum 2^(m_i - m) l_i, m = max m_i, out = O / l.
#include "tree_common.cuh"

#include <algorithm>

namespace lora {
namespace {

using namespace step;
using namespace tree;

struct JoinArgs {
    TreeArgs a;
    Plan plan[2];                                        // of the groups' and of the requests' launch
    int m_rows[2];                                       // rows of their parts
};

// A warp joins a row, or the eight of a block, which have the parts dealt to them: few
// rows are cut into many parts.
template <typename T, int DP, bool kBlock>
__global__ void __launch_bounds__(256) prefix_join_kernel(const __grid_constant__ JoinArgs args) {
    constexpr int V = Joined<DP>::V, kAhead = 4;
    __shared__ float so[kBlock ? 8 : 1][DP];
    __shared__ float2 sm[kBlock ? 8 : 1];
    const TreeArgs &a = args.a;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    grid_dependency_wait();
    grid_launch_dependents();
    const size_t rows = (size_t)a.n_tokens * a.n_heads, row = kBlock ? blockIdx.x : (size_t)blockIdx.x * 8 + warp;
    if (row >= rows) return;
    const int token = (int)(row / a.n_heads), head = (int)(row % a.n_heads);
    if (token < node_start(a, 0) || token >= node_start(a, a.n_requests)) return;   // of no request
    Joined<DP> all;
#pragma unroll
    for (int e = 0; e < V; ++e) all.o[e] = 0.f;
#pragma unroll
    for (int kind = 0; kind < 2; ++kind) {
        if (kind == 0 && (a.n_groups == 0 || token < node_start(a, group_start(a, 0)) ||
                          token >= node_start(a, group_start(a, a.n_groups))))
            continue;                                    // of no group
        const Plan &plan = args.plan[kind];
        const size_t at = kind * rows + row;
        const int4 named = a.row_at[at];
        // what starts that fall leave there leads nowhere
        if (named.w != (int)row || named.y < 0 || named.x < 0 || named.x >= plan.ctas || named.y > plan.ctas - named.x ||
            named.z < 0 || named.z >= args.m_rows[kind])
            continue;
        const int parts = max(named.y, 1);
        auto source = [&](int p) -> size_t {
            return (size_t)(p == 0 ? 2 * named.x + 1 : 2 * (named.x + p)) * args.m_rows[kind] + named.z;
        };
        const float *from = named.y == 0 ? a.row_o + at * DP : plan.part;
        const float2 *stat = named.y == 0 ? a.row_ml + at : plan.stat;
        constexpr int kStep = kBlock ? 8 : 1;
        for (int p0 = kBlock ? warp : 0; p0 < parts; p0 += kStep * kAhead) {
            alignas(4 * V) float v[kAhead][V];
            float2 ml[kAhead];
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const int p = p0 + u * kStep;
                if (p >= parts) break;
                const size_t s = named.y == 0 ? 0 : source(p);
                ml[u] = stat[s];
                const float *src = from + s * DP + lane * V;
                if constexpr (V == 4)
                    *reinterpret_cast<float4 *>(v[u]) = *reinterpret_cast<const float4 *>(src);
                else
                    *reinterpret_cast<float2 *>(v[u]) = *reinterpret_cast<const float2 *>(src);
            }
#pragma unroll
            for (int u = 0; u < kAhead; ++u)
                if (p0 + u * kStep < parts) all.add(ml[u], v[u]);
        }
    }
    if constexpr (kBlock) {
#pragma unroll
        for (int e = 0; e < V; ++e) so[warp][lane * V + e] = all.o[e];
        if (lane == 0) sm[warp] = make_float2(all.m, all.l);
        __syncthreads();
        if (warp > 0) return;
        for (int w = 1; w < 8; ++w) {
            float v[V];
#pragma unroll
            for (int e = 0; e < V; ++e) v[e] = so[w][lane * V + e];
            all.add(sm[w], v);
        }
    }
    store_joined<T, DP>(a, token, head, all);
}

// Entries [first, first + count) in tiles of `rows`, which become what the kernel took.
cudaError_t launch_entries(TreeArgs a, bool bf16, Plan &plan, int first, int count, int &rows, cudaStream_t st) {
    a.first = first;
    a.count = count;
    if (!bf16) return launch_f32(a, plan, rows, st);
    if (rows == 16) return launch_rows(a, plan, st);
    if (rows == 128) {
        const cudaError_t e = launch_tc(a, plan, st);
        if (e != cudaErrorNotSupported) return e;
        rows = 32;
    }
    return launch_mma(a, plan, rows, st);
}

template <typename T, int DP>
cudaError_t launch_prefix(const TreeArgs &a, const Plan &groups, const Plan &requests, cudaStream_t st) {
    constexpr bool kBf16 = sizeof(T) == 2;
    const double all = (double)a.n_tokens * (a.n_heads / a.n_kv);
    JoinArgs join{a, {groups, requests}, {0, 0}};
    auto tile = [&](double rows) { return kBf16 ? rows_of_tile(rows, tc_takes(a)) : rows <= 16.0 ? 16 : 64; };
    int of_requests = tile(all / a.n_requests), of_groups = a.n_groups > 0 ? tile(all / a.n_groups) : of_requests;
    cudaError_t e;
    if (kBf16 ? (of_groups == 128) == (of_requests == 128) : of_groups == of_requests) {
        of_requests = std::max(of_groups, of_requests);
        e = launch_entries(a, kBf16, join.plan[1], 0, a.n_groups + a.n_requests, of_requests, st);
        of_groups = of_requests;
        join.plan[0] = join.plan[1];
    } else {
        e = launch_entries(a, kBf16, join.plan[0], 0, a.n_groups, of_groups, st);
        if (e == cudaSuccess) e = launch_entries(a, kBf16, join.plan[1], a.n_groups, a.n_requests, of_requests, st);
    }
    if (e != cudaSuccess) return e;
    join.m_rows[0] = of_groups;
    join.m_rows[1] = of_requests;
    const long long rows = (long long)a.n_tokens * a.n_heads;
    if (rows <= 8 * groups.ctas)
        return launch_step(prefix_join_kernel<T, DP, true>, dim3((unsigned)rows), dim3(256), 0, 1, st, join);
    return launch_step(prefix_join_kernel<T, DP, false>, dim3((unsigned)((rows + 7) / 8)), dim3(256), 0, 1, st, join);
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
