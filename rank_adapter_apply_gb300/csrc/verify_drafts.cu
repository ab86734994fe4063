// lora_verify_drafts: acceptance of drafted trees against the target's
// probabilities, from given random numbers.
#include "step_util.cuh"

namespace lora {
namespace {

using namespace step;

constexpr int kMaxNodes = 1024;   // nodes of a request that are looked at
constexpr int kMaxCluster = 8;

struct VerifyArgs {
    const void *target, *draft;
    const int32_t *tokens, *parents, *node_starts;
    const float *uniforms, *noise;
    int32_t *path, *n_accepted, *next_token;
    long long target_row, draft_row, noise_row;
    int max_path, n_requests, n_nodes, vocab;
};

// What is left of the target's row after the rejections so far, at one token.
// The product is rounded before the difference, as the plain formula does.
__device__ __forceinline__ float rest(float p, float q, float a) { return fmaxf(__fsub_rn(p, __fmul_rn(a, q)), 0.f); }

template <int kThreads>
struct Shared {
    float sum[2][kThreads / 32 + 1];                 // warps' sums, and the CTA's, of passes in turn
    unsigned long long best[kThreads / 32 + 1];
    int parent[kMaxNodes];                           // of a node that may be tried: its parent; else -1
    int token[kMaxNodes];
    float p[kMaxNodes], q[kMaxNodes], u[kMaxNodes];  // target and draft at its token in its parent's rows
    int gone[kMaxNodes];                             // tokens rejected at the current node
};

// A request belongs to the CTAs of a cluster. Each of them walks the tree alike,
// from the nodes' values gathered at the start; a pass over a row of the
// vocabulary is cut among them, and its sum or maximum put together through
// distributed shared memory in a fixed order. A first child needs no pass: S_0 is 1.
// So a request reads one row of p, q and noise, and p and q once more for each
// rejection that is followed by another sibling.
//
// What bounds it: for large batches memory (256 requests of 8 nodes, vocabulary 131072, two
// fp32 rows and the noise: 78 us in a graph, 5.1 TB/s of what one pass reads, 86-90 us in a
// stream of calls, and a rejection reads more); for few the chain of passes, each a round of
// reads and two cluster barriers (32x13 of 100003 18 us, 1x5 of 32000 6 us).
// Visit a CTA's part of a row: f(v, p[v], q[v], noise[v]) for every index v, in
// rising order within a thread. Whole 16-byte vectors of p, at whatever element
// the row's first one starts, are dealt to the cluster; the elements before and
// after them go to its first and last CTA one by one. kBatch vectors of a thread
// are in flight together. Where q does not start at the same place within 16
// bytes as p, or noise not at 16 bytes, they are read element by element.
template <typename T, bool kQ, bool kNoise, int kThreads, class F>
__device__ __forceinline__ void visit(const T *p, const T *q, const float *noise, int vocab, int rank, int cluster,
                                      F &&f) {
    constexpr int N = 16 / sizeof(T), kBatch = sizeof(T) == 4 ? 2 : 1;
    const int tid = threadIdx.x;
    const int head = min((int)((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15) / (int)sizeof(T), vocab);
    const int vectors = (vocab - head) / N, tail = head + vectors * N;
    const bool q_vec = kQ && ((reinterpret_cast<uintptr_t>(p) ^ reinterpret_cast<uintptr_t>(q)) & 15) == 0;
    const bool n_vec = kNoise && (reinterpret_cast<uintptr_t>(noise + head) & 15) == 0;
    auto one = [&](int v) { f(v, to_f32(p[v]), kQ ? to_f32(q[v]) : 0.f, kNoise ? noise[v] : 0.f); };
    if (rank == 0 && tid < head) one(tid);
    const int lo = (int)((long long)vectors * rank / cluster), hi = (int)((long long)vectors * (rank + 1) / cluster);
    for (int i0 = lo + tid; i0 < hi; i0 += kThreads * kBatch) {
        uint4 pv[kBatch], qv[kBatch];
        alignas(16) float nv[kBatch][N];
#pragma unroll
        for (int e = 0; e < kBatch; ++e) {
            const int i = i0 + e * kThreads, v = head + i * N;
            if (i >= hi) break;
            pv[e] = *reinterpret_cast<const uint4 *>(p + v);
            if (kQ) {
                if (q_vec) {
                    qv[e] = *reinterpret_cast<const uint4 *>(q + v);
                } else {
                    alignas(16) T t[N];
#pragma unroll
                    for (int j = 0; j < N; ++j) t[j] = q[v + j];
                    qv[e] = *reinterpret_cast<const uint4 *>(t);
                }
            }
            if (kNoise) {
                if (n_vec) {
#pragma unroll
                    for (int j = 0; j < N; j += 4)
                        *reinterpret_cast<float4 *>(&nv[e][j]) = *reinterpret_cast<const float4 *>(noise + v + j);
                } else {
#pragma unroll
                    for (int j = 0; j < N; ++j) nv[e][j] = noise[v + j];
                }
            }
        }
#pragma unroll
        for (int e = 0; e < kBatch; ++e) {
            const int i = i0 + e * kThreads;
            if (i >= hi) break;
            float pf[N], qf[N];
            unpack<T>(pv[e], pf);
            if (kQ) unpack<T>(qv[e], qf);
#pragma unroll
            for (int j = 0; j < N; ++j) f(head + i * N + j, pf[j], kQ ? qf[j] : 0.f, kNoise ? nv[e][j] : 0.f);
        }
    }
    if (rank == cluster - 1 && tail + tid < vocab) one(tail + tid);
}

template <typename T, bool kDraft, int kThreads>
__global__ void __launch_bounds__(kThreads, 1024 / kThreads) verify_kernel(VerifyArgs a, int cluster) {
    __shared__ Shared<kThreads> sh;
    const int b = blockIdx.x / cluster, rank = blockIdx.x % cluster, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    grid_dependency_wait();
    grid_launch_dependents();
    const int start = min(max(a.node_starts[b], 0), a.n_nodes);
    const int nodes = min(max(min(a.node_starts[b + 1], a.n_nodes) - start, 0), kMaxNodes);
    const T *target = static_cast<const T *>(a.target), *draft = static_cast<const T *>(a.draft);
    for (int c = tid; c < nodes; c += kThreads) {
        const int x = a.tokens[start + c];
        int up = a.parents[start + c];
        if (up < 0 || up >= c || x < 0 || x >= a.vocab) up = -1;
        sh.parent[c] = up;
        sh.token[c] = x;
        sh.u[c] = a.uniforms[start + c];
        sh.p[c] = up < 0 ? 0.f : to_f32(target[(long long)(start + up) * a.target_row + x]);
        sh.q[c] = kDraft && up >= 0 ? to_f32(draft[(long long)(start + up) * a.draft_row + x]) : 1.f;
    }
    __syncthreads();
    const uint32_t sum_at = smem_u32(&sh.sum[0][kThreads / 32]);
    int node = 0, count = 0, rejected = 0, passes = 0;
    float alpha = 0.f;
    const T *p = nullptr, *q = nullptr;

    auto left_at = [&](float pv, float qv, int v) -> float {
        float r = kDraft ? rest(pv, qv, alpha) : pv;
        if constexpr (!kDraft)
            for (int i = 0; i < rejected; ++i) r = sh.gone[i] == v ? 0.f : r;
        return r;
    };

    auto row_sum = [&]() -> float {
        float s = 0.f;
        visit<T, kDraft, false, kThreads>(p, q, nullptr, a.vocab, rank, cluster,
                                          [&](int v, float pv, float qv, float) { s += left_at(pv, qv, v); });
        float *buf = sh.sum[passes & 1];
        s = warp_sum(s);
        if (lane == 0) buf[warp] = s;
        __syncthreads();
        s = buf[0];
        for (int w = 1; w < kThreads / 32; ++w) s += buf[w];
        if (cluster > 1) {
            if (tid == 0) buf[kThreads / 32] = s;
            cluster_sync_all();
            // buffers take turns: one is written again only after the barrier of the pass in between
            const uint32_t at = sum_at + (passes & 1) * sizeof(sh.sum[0]);
            float t = 0.f;
            for (int r = 0; r < cluster; ++r) t += __uint_as_float(ld_peer_u32(map_peer(at, r)));
            s = t;
        }
        ++passes;
        return s;
    };

    while (nodes > 0) {
        p = target + (long long)(start + node) * a.target_row;
        q = kDraft ? draft + (long long)(start + node) * a.draft_row : nullptr;
        alpha = 0.f;
        rejected = 0;
        float left = 1.f;
        int went = -1;
        if (count == a.max_path) break;
        for (int c = node + 1; c < nodes; ++c) {
            if (sh.parent[c] != node) continue;
            if (rejected > 0) left = row_sum();
            const int x = sh.token[c];
            const float px = left_at(sh.p[c], sh.q[c], x);
            if (__fmul_rn(sh.u[c], __fmul_rn(sh.q[c], left)) < px) {
                went = c;
                break;
            }
            alpha += left;
            if (!kDraft) {
                __syncthreads();                     // nobody reads the list any more
                if (tid == 0) sh.gone[rejected] = x;
                __syncthreads();
            }
            ++rejected;
        }
        if (went < 0) break;
        node = went;
        if (rank == 0 && tid == 0) a.path[(size_t)b * a.max_path + count] = node;
        ++count;
    }
    if (rank == 0)
        for (int i = count + tid; i < a.max_path; i += kThreads) a.path[(size_t)b * a.max_path + i] = -1;

    // ---- the next token: the largest rest / noise, ties to the lowest index
    int next = -1;
    const float *noise = a.noise + (long long)b * a.noise_row;
    for (int round = 0; round < 2 && next < 0 && nodes > 0; ++round) {     // the second: the row itself, R being zero
        if (round == 1) {
            if (rejected == 0) break;
            alpha = 0.f;
            rejected = 0;
        }
        float top = 0.f, low = 0.f;                  // this thread's best quotient, and a little less
        int at = -1;
        auto compare = [&](int v, float pv, float qv, float nv) {
            const float r = left_at(pv, qv, v);
            // the quotient only where the product says that it may be the largest yet
            if (r > low * nv) {
                const float key = __fdiv_rn(r, nv);
                if (key > top) top = key, at = v, low = key * (1.f - 0x1p-20f);
            }
        };
        if (kDraft && rejected > 0)
            visit<T, true, true, kThreads>(p, q, noise, a.vocab, rank, cluster, compare);
        else
            visit<T, false, true, kThreads>(p, nullptr, noise, a.vocab, rank, cluster,
                                            [&](int v, float pv, float, float nv) { compare(v, pv, 0.f, nv); });
        // positive floats order as their bits do; the lower index wins a tie
        unsigned long long mine =
            at < 0 ? 0ull : (unsigned long long)__float_as_uint(top) << 32 | (0xffffffffu - (unsigned)at);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const unsigned long long other = __shfl_xor_sync(0xffffffffu, mine, o);
            mine = other > mine ? other : mine;
        }
        if (lane == 0) sh.best[warp] = mine;
        __syncthreads();
        for (int w = 0; w < kThreads / 32; ++w) mine = sh.best[w] > mine ? sh.best[w] : mine;
        if (cluster > 1) {
            if (tid == 0) sh.best[kThreads / 32] = mine;
            cluster_sync_all();
            const uint32_t peer = smem_u32(&sh.best[kThreads / 32]);
            for (int r = 0; r < cluster; ++r) {
                const uint32_t w = map_peer(peer, r);
                const unsigned long long other = (unsigned long long)ld_peer_u32(w + 4) << 32 | ld_peer_u32(w);
                mine = other > mine ? other : mine;
            }
            cluster_sync_all();                      // the peers have read this CTA's, which may be written again
        } else {
            __syncthreads();
        }
        if (mine) next = (int)(0xffffffffu - (unsigned)(mine & 0xffffffffu));
    }
    if (rank == 0 && tid == 0) {
        a.n_accepted[b] = count;
        a.next_token[b] = next;
    }
    if (cluster > 1) cluster_sync_all();             // no CTA leaves while a peer may read its sums
}

template <typename T, bool kDraft, int kThreads>
cudaError_t launch_threads(const VerifyArgs &a, int cluster, cudaStream_t st) {
    return launch_step(verify_kernel<T, kDraft, kThreads>, dim3((unsigned)a.n_requests * cluster), dim3(kThreads), 0, cluster,
                       st, a, cluster);
}

// CTAs for a request: 1024 threads of them fit an SM, and few requests are cut
// further, over at most eight CTAs; where even those leave room, they are larger.
// Trees of 13 nodes over 100003 tokens in bf16, clusters until 2 / 6 / 12 CTAs to an SM:
// 256 requests 73 / 65 / 75 us, 512 151 / 121 / 114, 32 and fewer alike. CTAs of 256 / 512
// threads: 1 request 12.0 / 11.0 us, 32 17.6 / 17.3, 64 25.1 / 33.8, 256 65 / 77.
template <typename T, bool kDraft>
cudaError_t launch_verify(const VerifyArgs &a, int sms, cudaStream_t st) {
    int cluster = 1;
    while (cluster < kMaxCluster && (long long)a.n_requests * cluster < 6ll * sms) cluster *= 2;
    if ((long long)a.n_requests * cluster <= 2ll * sms) return launch_threads<T, kDraft, 512>(a, cluster, st);
    return launch_threads<T, kDraft, 256>(a, cluster, st);
}

}  // namespace
}  // namespace lora

using namespace lora;
using namespace lora::step;

extern "C" int lora_verify_drafts(const lora_verify_desc *d, void *stream) {
    if (!d) return fail(LORA_ERR_ARG, "verify_drafts: NULL descriptor");
    if (!known_dtype(d->dtype)) return fail(LORA_ERR_ARG, "verify_drafts: unknown dtype %d", d->dtype);
    if (d->n_requests < 0 || d->n_nodes < 0 || d->vocab < 1 || d->max_path < 0)
        return fail(LORA_ERR_ARG, "verify_drafts: n_requests %d, n_nodes %d, vocab %d, max_path %d", d->n_requests,
                    d->n_nodes, d->vocab, d->max_path);
    if (d->n_requests == 0) return LORA_OK;
    if (!d->node_starts || !d->n_accepted || !d->next_token || !d->noise || (d->max_path > 0 && !d->path) ||
        (d->n_nodes > 0 && (!d->target || !d->tokens || !d->parents || !d->uniforms)))
        return fail(LORA_ERR_ARG, "verify_drafts: NULL pointer argument");
    VerifyArgs a{d->target,   d->draft, d->tokens,     d->parents,    d->node_starts,
                 d->uniforms, d->noise, d->path,       d->n_accepted, d->next_token,
                 d->target_row, d->draft_row, d->noise_row, d->max_path, d->n_requests, d->n_nodes, d->vocab};
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int sms = sm_count();
    if (sms < 1) return fail(LORA_ERR_CUDA, "verify_drafts: no CUDA device");
    cudaError_t e;
    if (d->dtype == LORA_DTYPE_BF16)
        e = d->draft ? launch_verify<__nv_bfloat16, true>(a, sms, st) : launch_verify<__nv_bfloat16, false>(a, sms, st);
    else
        e = d->draft ? launch_verify<float, true>(a, sms, st) : launch_verify<float, false>(a, sms, st);
    return launched("verify_drafts", e);
}
