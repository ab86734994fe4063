// lora_sample_tokens: the next token of each row under temperature, top-k, top-p and
// min-p, from given random numbers.
#include "step_util.cuh"

#include <cfloat>
#include <climits>

namespace lora {
namespace {

using namespace step;

constexpr int kMaxCluster = 8;
constexpr int kHeldLogits = 64;   // of a thread, in registers
constexpr int kRejections = 6;    // races lost before the border is found by bisection

struct SampleArgs {
    const void *logits;
    const float *noise, *temperature, *top_p, *min_p;
    const int32_t *top_k;
    int32_t *tokens;
    float *logprobs;
    long long logits_row, noise_row;
    int n_rows, vocab;
};

// What the CTAs of a cluster put together in a pass.
struct alignas(16) Part {
    unsigned long long best;      // quotient's bits, then the complement of the index: the largest wins
    float sum;                    // (first pass: the maximum)
    uint32_t n;                   // (first pass: the bits of the lower bound)
};

// A place in the row's order: largest logit first, of equal ones the lowest index.
struct Place {
    float x;
    int i;
    // whether token v with logit y is in front of it
    __device__ __forceinline__ bool behind(float y, int v) const { return y > x || (y == x && v < i); }
    // places as numbers: the further to the front, the larger
    __device__ __forceinline__ unsigned long long number() const {
        const uint32_t b = __float_as_uint(x);
        return (unsigned long long)(b & 0x80000000u ? ~b : b | 0x80000000u) << 32 | (0xffffffffu - (unsigned)i);
    }
    __device__ __forceinline__ static Place of(unsigned long long n) {
        const uint32_t o = (uint32_t)(n >> 32);
        return {__uint_as_float(o & 0x80000000u ? o & 0x7fffffffu : ~o),
                (int)min(0xffffffffu - (uint32_t)n, (uint32_t)INT_MAX)};
    }
};

// A NaN counts as -inf, +inf as the largest number: differences from the maximum are then never NaN.
__device__ __forceinline__ float clean(float x) { return fminf(fmaxf(x, -INFINITY), FLT_MAX); }

// The largest p / noise yet. The quotient is formed only where a product says that it may be one.
struct Race {
    float top = 0.f, low = 0.f;
    int at = -1;
    __device__ __forceinline__ void enter(int v, float p, float n) {
        if (p > low * n) {
            const float key = __fdiv_rn(p, n);
            if (key > top || (key == top && v < at)) top = key, at = v, low = key * (1.f - 0x1p-20f);
        }
    }
    // positive floats order as their bits do; the lower index wins a tie
    __device__ __forceinline__ unsigned long long best() const {
        return at < 0 ? 0ull : (unsigned long long)__float_as_uint(top) << 32 | (0xffffffffu - (unsigned)at);
    }
};

// A row belongs to the CTAs of a cluster; a thread keeps up to 64 of its logits in
// registers (what is past them it reads again). Nothing is sorted:
//
//   1. the maximum; for top-k, a logit that at least k tokens reach: every warp takes the
//      ceil(k / warps)-th of its lanes' maxima, and the lowest of these is one;
//   2. the sum of p = exp((x - max) / t), and the race: the token with the largest
//      p / noise among those that may win;
//   3. the tokens in front of the winner are counted and their mass is summed. Each
//      filter keeps the first tokens of the order, so the winner is drawn if fewer than
//      k are in front and their mass is below top_p; if not, no token behind it is kept,
//      either, and the race is run again among those in front of it.
//
// The winner of a race over more than the kept tokens that is a kept one is the winner
// among these, so the draw is that of the filtered distribution. A race is lost with the
// probability of what the filters cut of the tokens in it; after six losses the border
// is found by bisection of the order's places instead.
template <typename T, int kThreads>
__global__ void __launch_bounds__(kThreads, 512 / kThreads) sample_kernel(SampleArgs a, int cluster) {
    constexpr int N = 16 / sizeof(T), kWarps = kThreads / 32, kHeld = kHeldLogits / N, kBatch = 16 / N;
    __shared__ Part parts[2][kWarps + 1];            // the warps', and the CTA's, of passes in turn
    const int row = blockIdx.x / cluster, rank = blockIdx.x % cluster, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    grid_dependency_wait();
    grid_launch_dependents();
    const T *logits = static_cast<const T *>(a.logits) + (long long)row * a.logits_row;
    const float *noise = a.noise + (long long)row * a.noise_row;

    // Whole 16-byte vectors, at whatever element the row's first one starts, are dealt to the cluster; an element
    // before or after them goes to a thread of the first or last CTA.
    const int head = min((int)((16 - (reinterpret_cast<uintptr_t>(logits) & 15)) & 15) / (int)sizeof(T), a.vocab);
    const int vectors = (a.vocab - head) / N, tail = head + vectors * N;
    const int lo = (int)((long long)vectors * rank / cluster), hi = (int)((long long)vectors * (rank + 1) / cluster);
    const int odd = rank == 0 && tid < head                                      ? tid
                    : rank == cluster - 1 && kThreads - 1 - tid < a.vocab - tail ? tail + kThreads - 1 - tid
                                                                                 : -1;
    uint4 held[kHeld];
#pragma unroll
    for (int j = 0; j < kHeld; ++j) {
        const int i = lo + tid + j * kThreads;
        if (i < hi) held[j] = *reinterpret_cast<const uint4 *>(logits + head + i * N);
    }
    const float odd_x = odd >= 0 ? clean(to_f32(logits[odd])) : -INFINITY;

    const float t = a.temperature ? a.temperature[row] : 1.f, top_p = a.top_p ? a.top_p[row] : 1.f;
    const float min_p = a.min_p && a.min_p[row] > 0.f ? a.min_p[row] : 0.f;
    const int top_k = a.top_k && a.top_k[row] > 0 ? a.top_k[row] : INT_MAX;
    // one token is kept: the first in the order
    bool first_only = !(t > 0.f) || top_k == 1 || top_p <= 0.f || min_p > 1.f;
    const float inv_t = t > 0.f ? fminf(fmaxf(__fdiv_rn(1.f, t), FLT_MIN), FLT_MAX) : 1.f;
    // every token is in the race: its noise is read in vectors, and brought to L2 while the logits come
    const int of_warp = (top_k - 1) / (kWarps * cluster) + 1;
    const bool dense = !first_only && min_p == 0.f && of_warp > 32 && (reinterpret_cast<uintptr_t>(noise + head) & 15) == 0;
    if (dense && tid == 0 && hi > lo)
        prefetch_l2_bulk(noise + head + lo * N, (uint32_t)min(hi - lo, kHeld * kThreads) * N * 4u);

    int passes = 0;
    // The cluster's value from the threads': join(a, b) over lanes, warps and CTAs, in one order.
    auto together = [&](Part mine, auto &&join) -> Part {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            mine = join(mine, Part{__shfl_xor_sync(0xffffffffu, mine.best, o), __shfl_xor_sync(0xffffffffu, mine.sum, o),
                                   __shfl_xor_sync(0xffffffffu, mine.n, o)});
        Part *buf = parts[passes & 1];
        if (lane == 0) buf[warp] = mine;
        __syncthreads();
        mine = buf[0];
        for (int w = 1; w < kWarps; ++w) mine = join(mine, buf[w]);
        if (cluster > 1) {
            if (tid == 0) buf[kWarps] = mine;
            cluster_sync_all();
            // buffers take turns: one is written again only after the barrier of the pass in between
            const uint32_t at = smem_u32(&buf[kWarps]);
            for (int r = 0; r < cluster; ++r) {
                const float4 v = ld_peer_f4(map_peer(at, r));
                const Part p{(unsigned long long)__float_as_uint(v.y) << 32 | __float_as_uint(v.x), v.z, __float_as_uint(v.w)};
                mine = r == 0 ? p : join(mine, p);
            }
        }
        ++passes;
        return mine;
    };
    auto add = [](const Part &p, const Part &q) { return Part{p.best > q.best ? p.best : q.best, p.sum + q.sum, p.n + q.n}; };
    auto vector = [&](int i, const uint4 &v, auto &&f) {
        float x[N];
        unpack<T>(v, x);
#pragma unroll
        for (int e = 0; e < N; ++e) f(head + i * N + e, clean(x[e]));
    };
    auto each = [&](auto &&f) {                      // f(index, logit) for this thread's tokens, in rising order but for odd's
        if (odd >= 0) f(odd, odd_x);
#pragma unroll
        for (int j = 0; j < kHeld; ++j) {
            const int i = lo + tid + j * kThreads;
            if (i < hi) vector(i, held[j], f);
        }
        for (int i = lo + tid + kHeld * kThreads; i < hi; i += kThreads)
            vector(i, *reinterpret_cast<const uint4 *>(logits + head + i * N), f);
    };

    // ---- 1: the maximum, and what at least top_k tokens reach
    float most = -INFINITY;
    each([&](int, float x) { most = fmaxf(most, x); });
    float reached = -INFINITY;
    if (!first_only && of_warp <= 32) {              // the lanes' maxima sorted, the largest in lane 0
        float v = most;
#pragma unroll
        for (int size = 2; size <= 32; size *= 2)
#pragma unroll
            for (int o = size / 2; o > 0; o /= 2) {
                const float w = __shfl_xor_sync(0xffffffffu, v, o);
                v = ((lane & o) == 0) == ((lane & size) == 0) ? fmaxf(v, w) : fminf(v, w);
            }
        reached = __shfl_sync(0xffffffffu, v, of_warp - 1);
    }
    const Part first = together(Part{0ull, most, (uint32_t)(Place{reached, 0}.number() >> 32)},
                                [](const Part &p, const Part &q) {
                                    return Part{0ull, fmaxf(p.sum, q.sum), min(p.n, q.n)};
                                });
    const float top = first.sum;
    int token = -1;
    float logprob = -INFINITY;
    if (top > -INFINITY) {
        auto prob = [&](float x) { return expf((x - top) * inv_t); };
        Place limit = Place::of((unsigned long long)first.n << 32);      // only tokens in front of it are in the race
        const bool by_mass = top_p < 1.f, tested = !first_only && (by_mass || top_k < a.vocab);
        float rest = 0.f, total = 0.f;               // p of all tokens but the maxima, which are 1 each, and of all
        uint32_t tops = 0;
        bool found = false;                          // the border: the tokens in the race are the kept ones
        for (int round = 0;; ++round) {
            // ---- 2: the sum and the race
            float sum = 0.f;
            uint32_t n = 0;
            Race race;
            auto enter = [&](int v, float x, float p, float nv) {
                if (x == top)
                    ++n;
                else
                    sum += p;
                race.enter(v, p, nv);
            };
            if (dense && round == 0) {
                if (odd >= 0) enter(odd, odd_x, prob(odd_x), noise[odd]);
#pragma unroll
                for (int j0 = 0; j0 < kHeld; j0 += kBatch) {
                    alignas(16) float nv[kBatch][N];
#pragma unroll
                    for (int b = 0; b < kBatch; ++b) {
                        const int i = lo + tid + (j0 + b) * kThreads;
                        if (i < hi)
#pragma unroll
                            for (int e = 0; e < N; e += 4)
                                *reinterpret_cast<float4 *>(&nv[b][e]) = *reinterpret_cast<const float4 *>(noise + head + i * N + e);
                    }
#pragma unroll
                    for (int b = 0; b < kBatch; ++b) {
                        const int i = lo + tid + (j0 + b) * kThreads;
                        float x[N];
                        unpack<T>(held[j0 + b], x);
                        if (i < hi)
#pragma unroll
                            for (int e = 0; e < N; ++e) enter(head + i * N + e, clean(x[e]), prob(clean(x[e])), nv[b][e]);
                    }
                }
                for (int i = lo + tid + kHeld * kThreads; i < hi; i += kThreads)
                    vector(i, *reinterpret_cast<const uint4 *>(logits + head + i * N),
                           [&](int v, float x) { enter(v, x, prob(x), noise[v]); });
            } else {
                each([&](int v, float x) {
                    const float p = prob(x);
                    if (x == top)
                        ++n;
                    else
                        sum += p;
                    if (first_only ? x == top : limit.behind(x, v) && p >= min_p) race.enter(v, first_only ? 1.f : p, first_only ? 1.f : noise[v]);
                });
            }
            const Part all = together(Part{race.best(), sum, n}, add);
            if (round == 0) {
                rest = all.sum;
                tops = all.n;
                total = rest + (float)tops;
            }
            if (all.best == 0) {                     // no noise was a positive number: the first in the order
                if (first_only) break;
                first_only = true;
                continue;
            }
            token = (int)(0xffffffffu - (unsigned)(all.best & 0xffffffffu));
            if (!tested || found || first_only) break;
            // ---- 3: whether the winner is kept
            Place at{clean(to_f32(logits[token])), token};
            unsigned long long no = 0, yes = 0;      // of the bisection: places not kept and kept
            bool kept;
            for (;;) {
                float mass = 0.f;
                uint32_t front = 0;
                each([&](int v, float x) {
                    if (at.behind(x, v)) {
                        ++front;
                        if (by_mass) mass += prob(x);
                    }
                });
                const Part p = together(Part{0ull, mass, front}, add);
                kept = p.n < (uint32_t)top_k && (!by_mass || p.sum < top_p * total);
                if (yes == 0) {                      // the winner's place
                    if (kept || round < kRejections) break;
                    no = at.number();
                    yes = Place{top, 0}.number();
                } else {
                    (kept ? yes : no) = no + (yes - no) / 2;
                }
                if (yes - no <= 1) {
                    found = true;
                    break;
                }
                at = Place::of(no + (yes - no) / 2);
            }
            if (kept && yes == 0) break;
            limit = found ? Place::of(no) : at;
        }
        logprob = -(logf((float)tops) + log1pf(rest / (float)tops));
        if (token >= 0) logprob += (clean(to_f32(logits[token])) - top) * inv_t;
    }
    if (rank == 0 && tid == 0) {
        a.tokens[row] = token;
        if (a.logprobs) a.logprobs[row] = logprob;
    }
    if (cluster > 1) cluster_sync_all();             // no CTA leaves while a peer may read its part
}

template <typename T>
cudaError_t launch_sample(const SampleArgs &a, int sms, cudaStream_t st) {
    constexpr int kThreads = 256;
    int cluster = 1;
    while (cluster < kMaxCluster &&
           ((long long)cluster * kThreads * kHeldLogits < a.vocab || (long long)a.n_rows * cluster < sms))
        cluster *= 2;
    return launch_step(sample_kernel<T, kThreads>, dim3((unsigned)a.n_rows * cluster), dim3(kThreads), 0, cluster, st, a,
                       cluster);
}

}  // namespace
}  // namespace lora

using namespace lora;
using namespace lora::step;

extern "C" int lora_sample_tokens(const lora_sample_desc *d, void *stream) {
    if (!d) return fail(LORA_ERR_ARG, "sample_tokens: NULL descriptor");
    if (!known_dtype(d->dtype)) return fail(LORA_ERR_ARG, "sample_tokens: unknown dtype %d", d->dtype);
    if (d->n_rows < 0 || d->n_rows > (1 << 27) || d->vocab < 1)
        return fail(LORA_ERR_ARG, "sample_tokens: n_rows %d (0..2^27), vocab %d", d->n_rows, d->vocab);
    if (d->logits_row < 0 || d->noise_row < 0)
        return fail(LORA_ERR_ARG, "sample_tokens: the strides %lld, %lld are negative", (long long)d->logits_row,
                    (long long)d->noise_row);
    if (d->n_rows == 0) return LORA_OK;
    if (!d->logits || !d->noise || !d->tokens) return fail(LORA_ERR_ARG, "sample_tokens: NULL pointer argument");
    const SampleArgs a{d->logits, d->noise,    d->temperature, d->top_p,     d->min_p,  d->top_k,
                       d->tokens, d->logprobs, d->logits_row,  d->noise_row, d->n_rows, d->vocab};
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int sms = sm_count();
    if (sms < 1) return fail(LORA_ERR_CUDA, "sample_tokens: no CUDA device");
    const cudaError_t e =
        d->dtype == LORA_DTYPE_BF16 ? launch_sample<__nv_bfloat16>(a, sms, st) : launch_sample<float>(a, sms, st);
    return launched("sample_tokens", e);
}
