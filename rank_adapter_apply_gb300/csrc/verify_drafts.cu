// lora_verify_drafts: acceptance of drafted trees against the target's
// probabilities, from given random numbers.
#include "step_util.cuh"

namespace lora {
namespace {

using namespace step;

constexpr int kMaxNodes = 1024;   // nodes of a request that are looked at
constexpr int kThreads = 512;

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

// Sum over the block (every thread gets it); the order is fixed by the thread count.
__device__ float block_sum(float v, float *buf) {
    v = warp_sum(v);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
    __syncthreads();
    float s = 0.f;
    for (int w = 0; w < kThreads / 32; ++w) s += buf[w];
    return s;
}

// One CTA for each request. The walk is the same in every thread.
template <typename T>
__global__ void __launch_bounds__(kThreads) verify_kernel(VerifyArgs a) {
    __shared__ float buf[kThreads / 32];
    __shared__ unsigned long long best;
    __shared__ int gone[kMaxNodes];      // without draft: the tokens rejected at the current node
    const int b = blockIdx.x, tid = threadIdx.x;
    const int start = min(max(a.node_starts[b], 0), a.n_nodes);
    const int nodes = min(max(min(a.node_starts[b + 1], a.n_nodes) - start, 0), kMaxNodes);
    const int32_t *parents = a.parents + start, *tokens = a.tokens + start;
    int node = 0, count = 0, rejected = 0;
    float alpha = 0.f;
    const T *p = nullptr, *q = nullptr;
    while (nodes > 0) {
        p = static_cast<const T *>(a.target) + (size_t)(start + node) * a.target_row;
        q = a.draft ? static_cast<const T *>(a.draft) + (size_t)(start + node) * a.draft_row : nullptr;
        alpha = 0.f;
        rejected = 0;
        float left = 1.f;
        int went = -1;
        if (count == a.max_path) break;
        for (int c = node + 1; c < nodes; ++c) {
            if (parents[c] != node) continue;
            const int x = tokens[c];
            if (x < 0 || x >= a.vocab) continue;
            if (rejected > 0) {           // what is left after the last rejection
                float s = 0.f;
                for (int v = tid; v < a.vocab; v += kThreads) {
                    float r = q ? rest(to_f32(p[v]), to_f32(q[v]), alpha) : to_f32(p[v]);
                    if (!q)
                        for (int i = 0; i < rejected; ++i) r = gone[i] == v ? 0.f : r;
                    s += r;
                }
                left = block_sum(s, buf);
            }
            float px = to_f32(p[x]);
            const float qx = q ? to_f32(q[x]) : 1.f;
            if (q)
                px = rest(px, qx, alpha);
            else
                for (int i = 0; i < rejected; ++i) px = gone[i] == x ? 0.f : px;
            if (__fmul_rn(a.uniforms[start + c], __fmul_rn(qx, left)) < px) {
                went = c;
                break;
            }
            alpha += left;
            __syncthreads();
            if (tid == 0) gone[rejected] = x;
            ++rejected;
            __syncthreads();
        }
        if (went < 0) break;
        node = went;
        if (tid == 0) a.path[(size_t)b * a.max_path + count] = node;
        ++count;
    }
    for (int i = count + tid; i < a.max_path; i += kThreads) a.path[(size_t)b * a.max_path + i] = -1;
    // The next token: the largest rest / noise, ties to the lowest index.
    int next = -1;
    const float *noise = a.noise + (size_t)b * a.noise_row;
    for (int round = 0; round < 2 && next < 0 && nodes > 0; ++round) {   // the second: the row itself, R being zero
        if (tid == 0) best = 0;
        __syncthreads();
        unsigned long long mine = 0;
        for (int v = tid; v < a.vocab; v += kThreads) {
            float r = to_f32(p[v]);
            if (round == 0) {
                if (q && rejected > 0) r = rest(r, to_f32(q[v]), alpha);
                if (!q)
                    for (int i = 0; i < rejected; ++i) r = gone[i] == v ? 0.f : r;
            }
            if (r > 0.f) {
                const float key = __fdiv_rn(r, noise[v]);
                // positive floats order as their bits do; the lower index wins a tie
                const unsigned long long k = ((unsigned long long)__float_as_uint(key) << 32) | (0xffffffffu - v);
                if (key > 0.f && k > mine) mine = k;
            }
        }
        atomicMax(&best, mine);
        __syncthreads();
        if (best) next = (int)(0xffffffffu - (unsigned)(best & 0xffffffffu));
        __syncthreads();
    }
    if (tid == 0) {
        a.n_accepted[b] = count;
        a.next_token[b] = next;
    }
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
    if (d->dtype == LORA_DTYPE_BF16)
        verify_kernel<__nv_bfloat16><<<d->n_requests, kThreads, 0, st>>>(a);
    else
        verify_kernel<float><<<d->n_requests, kThreads, 0, st>>>(a);
    return launched("verify_drafts", cudaGetLastError());
}
