// lora_sample_tokens: the next token of each row under temperature, top-k, top-p and
// min-p, from given random numbers.
#include "step_util.cuh"

#include <algorithm>
#include <atomic>
#include <cfloat>
#include <climits>

namespace lora {
namespace {

using namespace step;

constexpr int kMaxCluster = 8;
constexpr int kSliceBytes = 64 * 1024;   // of a CTA's logits in shared memory: three CTAs fit an SM
constexpr int kRejections = 6;           // races lost before the border is found by bisection

struct SampleArgs {
    const void *logits;
    const float *noise, *temperature, *top_p, *min_p;
    const int32_t *top_k;
    int32_t *tokens;
    float *logprobs;
    long long logits_row, noise_row;
    int n_rows, vocab, cluster, slots;       // slots: vectors of a CTA in shared memory
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

// A NaN counts as -inf, +inf as the type's largest number: differences from the maximum are then never NaN.
template <typename T>
__device__ __forceinline__ float clean(float x) {
    return fminf(fmaxf(x, -INFINITY), sizeof(T) == 4 ? FLT_MAX : __uint_as_float(0x7f7f0000u));
}
template <typename T>
__device__ __forceinline__ uint4 clean_vector(const uint4 &v) {
    float x[16 / sizeof(T)];
    unpack<T>(v, x);
#pragma unroll
    for (float &e : x) e = clean<T>(e);
    if constexpr (sizeof(T) == 4)
        return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
    else
        return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
}

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ void st_peer_part(uint32_t cluster_addr, const Part &p) {
    asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(cluster_addr), "r"((uint32_t)p.best),
                 "r"((uint32_t)(p.best >> 32)), "r"(__float_as_uint(p.sum)), "r"(p.n) : "memory");
}

// The largest p / noise yet, and a little less: what is below it need not be divided.
struct Race {
    float top = 0.f, low = 0.f;
    int at = -1;
    __device__ __forceinline__ void enter(int v, float p, float n) {
        const float key = __fdiv_rn(p, n);
        // 2^-15: more than the fast exponential is off by
        if (key > top || (key == top && v < at)) top = key, at = v, low = key * (1.f - 0x1p-15f);
    }
    // positive floats order as their bits do; the lower index wins a tie
    __device__ __forceinline__ unsigned long long best() const {
        return at < 0 ? 0ull : (unsigned long long)__float_as_uint(top) << 32 | (0xffffffffu - (unsigned)at);
    }
};

// A row belongs to the CTAs of a cluster, which keep its logits in shared memory (what
// is past 64 KB of a CTA is read again). Nothing is sorted:
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
__global__ void __launch_bounds__(kThreads, 768 / kThreads) sample_kernel(SampleArgs a) {
    constexpr int N = 16 / sizeof(T), kWarps = kThreads / 32, kBatch = 16 / N;
    extern __shared__ __align__(16) uint4 slice[];
    __shared__ Part warps[2][kWarps], ctas[2][kMaxCluster];          // of passes in turn
    static_assert(kSliceBytes / 16 % kThreads == 0, "the vectors past the slice begin at thread 0");
    const int cluster = a.cluster;
    const int row = blockIdx.x / cluster, rank = blockIdx.x % cluster, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (cluster > 1) cluster_arrive_relaxed();       // a peer that has come this far may be written to
    grid_dependency_wait();
    grid_launch_dependents();
    const T *logits = static_cast<const T *>(a.logits) + (long long)row * a.logits_row;
    const float *noise = a.noise + (long long)row * a.noise_row;

    // Whole 16-byte vectors, at whatever element the row's first one starts, are dealt to the cluster; an element
    // before or after them goes to a thread of the first or last CTA. A thread reads the vectors that it has copied.
    const int head = min((int)((16 - (reinterpret_cast<uintptr_t>(logits) & 15)) & 15) / (int)sizeof(T), a.vocab);
    const int vectors = (a.vocab - head) / N, tail = head + vectors * N;
    const int lo = (int)((long long)vectors * rank / cluster), n_vec = (int)((long long)vectors * (rank + 1) / cluster) - lo;
    const int held = min(n_vec, a.slots), base = head + lo * N;
    for (int j = tid; j < held; j += kThreads) cp_async16(&slice[j], logits + base + j * N);
    cp_async_commit();
    const int odd = rank == 0 && tid < head                                      ? tid
                    : rank == cluster - 1 && kThreads - 1 - tid < a.vocab - tail ? tail + kThreads - 1 - tid
                                                                                 : -1;
    const float odd_x = odd >= 0 ? clean<T>(to_f32(logits[odd])) : -INFINITY;

    const float t = a.temperature ? a.temperature[row] : 1.f, top_p = a.top_p ? a.top_p[row] : 1.f;
    const float min_p = a.min_p && a.min_p[row] > 0.f ? a.min_p[row] : 0.f;
    const int top_k = a.top_k && a.top_k[row] > 0 ? a.top_k[row] : INT_MAX;
    // one token is kept: the first in the order
    bool first_only = !(t > 0.f) || top_k == 1 || top_p <= 0.f || min_p > 1.f;
    const float inv_t = t > 0.f ? fminf(fmaxf(__fdiv_rn(1.f, t), FLT_MIN), FLT_MAX) : 1.f;
    // every token is in the race: its noise is read in vectors, and brought to L2 while the logits come
    const int of_warp = (top_k - 1) / (kWarps * cluster) + 1;
    const bool dense = !first_only && min_p == 0.f && of_warp > 32 && (reinterpret_cast<uintptr_t>(noise + base) & 15) == 0;
    if (dense && tid == 0 && held > 0) prefetch_l2_bulk(noise + base, (uint32_t)held * N * 4u);

    int passes = 0;
    // The cluster's value from the threads': join(a, b) over lanes, warps and CTAs, in one order.
    auto together = [&](Part mine, auto &&join) -> Part {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            mine = join(mine, Part{__shfl_xor_sync(0xffffffffu, mine.best, o), __shfl_xor_sync(0xffffffffu, mine.sum, o),
                                   __shfl_xor_sync(0xffffffffu, mine.n, o)});
        const int buf = passes++ & 1;                // written again only after the barriers of the pass in between
        if (lane == 0) warps[buf][warp] = mine;
        __syncthreads();
        mine = warps[buf][0];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) mine = join(mine, warps[buf][w]);
        if (cluster > 1) {
            if (tid < cluster) st_peer_part(map_peer(smem_u32(&ctas[buf][rank]), tid), mine);
            cluster_sync_all();
            mine = ctas[buf][0];
            for (int r = 1; r < cluster; ++r) mine = join(mine, ctas[buf][r]);
        }
        return mine;
    };
    auto add = [](const Part &p, const Part &q) { return Part{p.best > q.best ? p.best : q.best, p.sum + q.sum, p.n + q.n}; };
    auto vector = [&](int j) -> uint4 {
        return j < held ? slice[j] : clean_vector<T>(*reinterpret_cast<const uint4 *>(logits + base + j * N));
    };

    // ---- 1: the maximum, and what at least top_k tokens reach
    cp_async_wait_all();
    float most = odd_x;
    bool unclean = false;
    for (int j = tid; j < n_vec; j += kThreads) {
        float x[N];
        unpack<T>(vector(j), x);
#pragma unroll
        for (int e = 0; e < N; ++e) {
            most = fmaxf(most, x[e]);
            unclean = unclean || x[e] != x[e];
        }
    }
    if (unclean || most == INFINITY) {
        for (int j = tid; j < held; j += kThreads) slice[j] = clean_vector<T>(slice[j]);
        most = clean<T>(most);
    }
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
    if (cluster > 1) cluster_wait_acquire();
    const Part first = together(Part{0ull, most, (uint32_t)(Place{reached, 0}.number() >> 32)},
                                [](const Part &p, const Part &q) {
                                    return Part{0ull, fmaxf(p.sum, q.sum), min(p.n, q.n)};
                                });
    const float top = first.sum;
    int token = -1;
    float logprob = -INFINITY;
    if (top > -INFINITY) {
        const float c2 = inv_t * 1.4426950408889634f;
        auto prob = [&](float x) { return expf((x - top) * inv_t); };
        auto about = [&](float x) { return exp2_fast((x - top) * c2); };     // within 2^-17 where it is not below 2^-126
        Place limit = Place::of((unsigned long long)first.n << 32);          // only tokens in front of it are in the race
        // and no logit below this has p >= min_p
        const float floor_x = min_p > 0.f ? top + (logf(min_p) - 0.01f) / inv_t - fabsf(top) * 0x1p-22f : -INFINITY;
        const bool by_mass = top_p < 1.f, tested = !first_only && (by_mass || top_k < a.vocab);
        float rest = 0.f, total = 0.f;               // p of all tokens but the maxima, which are 1 each, and of all
        uint32_t tops = 0;
        bool found = false;                          // the border: the tokens in the race are the kept ones
        for (int round = 0;; ++round) {
            // ---- 2: the sum and the race
            Race race;
            float sum = 0.f;
            uint32_t n = 0;
            const float gate = first_only ? top : fmaxf(limit.x, floor_x);
            auto enter = [&](int v, float x) {       // exactly
                if (first_only) {
                    if (x == top) race.enter(v, 1.f, 1.f);
                } else if (limit.behind(x, v)) {
                    const float p = prob(x);
                    if (p >= min_p) race.enter(v, p, noise[v]);
                }
            };
            if (odd >= 0) {
                if (odd_x < top) sum = about(odd_x);
                if (odd_x >= gate) enter(odd, odd_x);
            }
            if (dense && round == 0) {
                for (int j0 = tid; j0 < held; j0 += kBatch * kThreads) {
                    alignas(16) float nv[kBatch][N];
#pragma unroll
                    for (int b = 0; b < kBatch; ++b) {
                        const int j = j0 + b * kThreads;
                        if (j < held)
#pragma unroll
                            for (int e = 0; e < N; e += 4)
                                *reinterpret_cast<float4 *>(&nv[b][e]) = *reinterpret_cast<const float4 *>(noise + base + j * N + e);
                    }
#pragma unroll
                    for (int b = 0; b < kBatch; ++b) {
                        const int j = j0 + b * kThreads;
                        if (j >= held) break;
                        float x[N];
                        unpack<T>(slice[j], x);
#pragma unroll
                        for (int e = 0; e < N; ++e) {
                            const float p = about(x[e]);
                            sum += p;
                            if (p > race.low * nv[b][e]) race.enter(base + j * N + e, prob(x[e]), nv[b][e]);
                        }
                    }
                }
            }
            for (int j = tid + (dense && round == 0 ? held + kThreads - 1 - (held + kThreads - 1) % kThreads : 0); j < n_vec;
                 j += kThreads) {
                float x[N], most_x = -INFINITY;
                unpack<T>(vector(j), x);
#pragma unroll
                for (int e = 0; e < N; ++e) {
                    if (round == 0) sum += about(x[e]);
                    most_x = fmaxf(most_x, x[e]);
                }
                if (most_x >= gate)
#pragma unroll
                    for (int e = 0; e < N; ++e)
                        if (x[e] >= gate) enter(base + j * N + e, x[e]);
            }
            if (round == 0 && most == top) {         // the maxima apart: 1 swallows what it is added to
                sum = odd >= 0 && odd_x < top ? about(odd_x) : 0.f;
                n = odd >= 0 && odd_x == top;
                for (int j = tid; j < n_vec; j += kThreads) {
                    float x[N];
                    unpack<T>(vector(j), x);
#pragma unroll
                    for (int e = 0; e < N; ++e) {
                        if (x[e] == top)
                            ++n;
                        else
                            sum += about(x[e]);
                    }
                }
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
            Place at{clean<T>(to_f32(logits[token])), token};
            unsigned long long no = 0, yes = 0;      // of the bisection: places not kept and kept
            bool kept;
            for (;;) {
                float mass = 0.f;
                uint32_t front = 0;
                auto count = [&](int v, float x) {
                    if (at.behind(x, v)) {
                        ++front;
                        mass += about(x);
                    }
                };
                if (odd >= 0) count(odd, odd_x);
                for (int j = tid; j < n_vec; j += kThreads) {
                    float x[N], most_x = -INFINITY;
                    unpack<T>(vector(j), x);
#pragma unroll
                    for (int e = 0; e < N; ++e) most_x = fmaxf(most_x, x[e]);
                    if (most_x >= at.x)
#pragma unroll
                        for (int e = 0; e < N; ++e) count(base + j * N + e, x[e]);
                }
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
        if (token >= 0) logprob += (clean<T>(to_f32(logits[token])) - top) * inv_t;
    }
    if (rank == 0 && tid == 0) {
        a.tokens[row] = token;
        if (a.logprobs) a.logprobs[row] = logprob;
    }
    if (cluster > 1) cluster_sync_all();             // no CTA leaves while a peer may write its parts there
}

template <typename T>
cudaError_t launch_sample(SampleArgs a, int sms, cudaStream_t st) {
    constexpr int kThreads = 256, N = 16 / sizeof(T);
    auto kernel = sample_kernel<T, kThreads>;
    static std::atomic<uint64_t> ready{0};
    if (!device_bit(ready)) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSliceBytes);
        if (e != cudaSuccess) return e;
        set_device_bit(ready);
    }
    a.cluster = 1;
    while (a.cluster < kMaxCluster && ((long long)a.cluster * kSliceBytes < (long long)a.vocab * (int)sizeof(T) ||
                                       (long long)a.n_rows * a.cluster < 2 * sms))
        a.cluster *= 2;
    const int vectors = a.vocab / N;
    a.slots = std::min((vectors + a.cluster - 1) / a.cluster, kSliceBytes / 16);
    return launch_step(kernel, dim3((unsigned)a.n_rows * a.cluster), dim3(kThreads), (size_t)a.slots * 16, a.cluster, st, a);
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
                       d->tokens, d->logprobs, d->logits_row,  d->noise_row, d->n_rows, d->vocab, 1,         0};
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int sms = sm_count();
    if (sms < 1) return fail(LORA_ERR_CUDA, "sample_tokens: no CUDA device");
    const cudaError_t e =
        d->dtype == LORA_DTYPE_BF16 ? launch_sample<__nv_bfloat16>(a, sms, st) : launch_sample<float>(a, sms, st);
    return launched("sample_tokens", e);
}
