// lora_sample_tokens: the next token of each row under temperature, top-k, top-p and
// min-p, from given random numbers.
#include "step_util.cuh"

#include <algorithm>
#include <atomic>
#include <cfloat>
#include <climits>
#include <type_traits>

namespace lora {
namespace {

using namespace step;

constexpr int kMaxCluster = 8;
constexpr int kSliceBytes = 64 * 1024;   // of a CTA's logits in shared memory: three CTAs fit an SM
constexpr int kBins = 256;               // of 1/8: down to 2^-32 of the largest p
// Tokens of a race that a CTA lists. us with 128 / 512 / 1024: 1 row of 32000 8.2 / 7.5 / 7.5, 77 of 65537 with top-k 23.3 / 20.0 /
// 20.1, 256 of 131072 102 / 102 / 122 (three CTAs no longer fit an SM), 64 of 100003 with k = 1000 49 / 39 / 39.
constexpr int kListed = 512;
// Races lost before the border is found by bisection, a pass for each halving. us with 2 / 6 / 12: 64 rows of 32000 nearly equal logits,
// top-p 0.5 72 / 32 / 32, top-p 0.1 129 / 84 / 54, k = 50 166 / 155 / 132; 64 of 100003 with k = 20 71 / 33 / 33; the others
// alike. A race that is lost in vain costs two passes.
constexpr int kRejections = 6;

struct SampleArgs {
    const void *logits;
    const float *noise, *temperature, *top_p, *min_p;
    const int32_t *top_k;
    int32_t *tokens;
    float *logprobs;
    long long logits_row, noise_row;
    int n_rows, vocab, cluster, slots;       // slots: vectors of a CTA in shared memory
};

// What the warps of a cluster put together in a pass: a race's winner (at < 0: none), its logit and noise; p of the
// tokens but the maxima, which are counted, by the maximum of the warp's CTA.
struct alignas(16) Part {
    int at;
    float x, noise, most;
    float sum;
    uint32_t n;
    uint32_t pad[2];
};

// Bits that order as the floats do, and back.
__device__ __forceinline__ uint32_t ordered(float x) {
    const uint32_t b = __float_as_uint(x);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float unordered(uint32_t o) {
    return __uint_as_float(o & 0x80000000u ? o & 0x7fffffffu : ~o);
}

// A place in the row's order: largest logit first, of equal ones the lowest index.
struct Place {
    float x;
    int i;
    // whether token v with logit y is in front of it
    __device__ __forceinline__ bool behind(float y, int v) const { return y > x || (y == x && v < i); }
    // places as numbers: the further to the front, the larger
    __device__ __forceinline__ unsigned long long number() const {
        return (unsigned long long)ordered(x) << 32 | (0xffffffffu - (unsigned)i);
    }
    __device__ __forceinline__ static Place of(unsigned long long n) {
        return {unordered((uint32_t)(n >> 32)), (int)min(0xffffffffu - (uint32_t)n, (uint32_t)INT_MAX)};
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

__device__ __forceinline__ void st_peer(uint32_t cluster_addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(cluster_addr), "r"(a), "r"(b), "r"(c), "r"(d)
                 : "memory");
}

__device__ __forceinline__ float warp_max(float v) { return unordered(__reduce_max_sync(0xffffffffu, ordered(v))); }

// p / noise exactly, of a token that may be drawn: with p >= min_p, and 2^-126 (the loops' exponential flushes what is
// smaller, so that a limit is needed that holds wherever a token is looked at). Not inlined: few tokens come to it, and it
// would be in the loops' way.
__device__ __noinline__ float quotient(float below_top, float inv_t, float min_p, float n) {
    const float p = expf(below_top * inv_t);
    return p >= fmaxf(min_p, FLT_MIN) ? __fdiv_rn(p, n) : -1.f;
}

// The largest p / noise yet, and twice a little less: what has a 2 p / noise below it need not be divided.
struct Race {
    float top = 0.f, low = 0.f, x = 0.f, noise = 0.f;
    int at = -1;
    __device__ __forceinline__ void enter(int v, float key, float xv, float nv) {
        // 2^-15: more than the fast exponential and quotient's are apart
        if (key > top || (key == top && v < at))
            top = key, at = v, x = xv, noise = nv, low = fmaxf(low, fminf(key, 0.5f * FLT_MAX) * (2.f - 0x1p-14f));
    }
    // the warp's best in all lanes: positive floats order as their bits do, the lower index wins a tie
    __device__ __forceinline__ void of_warp() {
        const uint32_t key = at < 0 ? 0u : __float_as_uint(top), best = __reduce_max_sync(0xffffffffu, key);
        const int first = __reduce_min_sync(0xffffffffu, key == best && at >= 0 ? at : INT_MAX);
        const int src = __ffs(__ballot_sync(0xffffffffu, at == first && key == best)) - 1;
        if (src < 0) {
            at = -1;
            return;
        }
        top = __shfl_sync(0xffffffffu, top, src);
        x = __shfl_sync(0xffffffffu, x, src);
        noise = __shfl_sync(0xffffffffu, noise, src);
        at = first;
    }
};

// What p / noise of a token above the limit, of parts whose winners are below it, stays under: p of their winners is below
// 2^-126, and no p / noise of theirs is above the winner's.
__device__ __noinline__ float most_behind(const Part *parts, int n_parts, float top, float inv_t) {
    float most = 0.f;
    for (int i = threadIdx.x & 31; i < n_parts; i += 32) {
        const Part p = parts[i];
        if (p.at >= 0 && quotient(p.x - top, inv_t, 0.f, p.noise) < 0.f) most = fmaxf(most, __fdiv_rn(2.f * FLT_MIN, p.noise));
    }
    return warp_max(most);
}

// A row belongs to the CTAs of a cluster, which keep its logits in shared memory (what
// is past 64 KB of a CTA is read again). Nothing is sorted:
//
//   1. the maximum; for top-k, a logit that at least k tokens reach: every CTA counts the
//      maxima of its vectors by their distance from its largest, an eighth of a power of two
//      of p to a bin, until ceil(k / CTAs) are there, and the lowest of these is one;
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
//
// A row is a cluster's: its logits are read from memory once and stay in shared memory. 256 rows
// of 131072 in fp32, top-p alone: 102 us, where logits and noise, which every row then reads whole,
// take 40 from memory: three passes over shared memory, exponentials and exchanges between
// CTAs follow one another, with three CTAs on an SM to fill the gaps (barriers, the
// arithmetic's own results and shared memory are the stalls, issue slots are busy for 40 %). 32 rows
// of 100003 with filters of all kinds 18 us, one of 32000 7.5: a launch and a chain of five exchanges. 64
// rows of 151936 in fp32, top-p alone: 60 us, 78 MB: the tokens past a CTA's 64 KB are listed in vain
// and gone over again. (A maximum of
// each vector in place of its tokens for top-k's bound 149 -> 107 us; 384 or 512 threads,
// 16 CTAs to a cluster and rows brought to L2 ahead were slower.)
template <typename T, int kThreads>
__global__ void __launch_bounds__(kThreads, 768 / kThreads) sample_kernel(SampleArgs a) {
    constexpr int N = 16 / sizeof(T), kWarps = kThreads / 32, kBatch = 8 / N;
    extern __shared__ __align__(16) uint4 slice[];
    __shared__ Part parts[2][kMaxCluster * kWarps];                  // of the cluster's warps, of passes in turn
    __shared__ uint32_t bins[kBins];
    __shared__ float of_cta[kWarps];
    __shared__ uint32_t bound;                       // bits of a race's bound
    __shared__ float2 listed[kListed];               // (logit, index's bits) of tokens in the race
    __shared__ int n_listed;
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
    const bool dense_row = !first_only && min_p == 0.f && top_k >= a.vocab && (reinterpret_cast<uintptr_t>(noise + base) & 15) == 0;
    if (dense_row && tid == 0 && held > 0) prefetch_l2_bulk(noise + base, (uint32_t)held * N * 4u);

    int passes = 0;
    const int n_parts = cluster * kWarps;
    // A warp's part to the CTAs of the cluster, and a barrier; a lane then has the parts `lane` and `lane + 32` of theirs.
    auto exchange = [&](const Part &p) -> const Part * {
        Part *buf = parts[passes++ & 1];             // written again only after the barrier of the pass in between
        if (lane < cluster) {
            const uint32_t at = smem_u32(&buf[rank * kWarps + warp]);
            const uint32_t to = cluster > 1 ? map_peer(at, lane) : at;
            st_peer(to, p.at, __float_as_uint(p.x), __float_as_uint(p.noise), __float_as_uint(p.most));
            st_peer(to + 16, __float_as_uint(p.sum), p.n, 0, 0);
        }
        if (cluster > 1)
            cluster_sync_all();
        else
            __syncthreads();
        return buf;
    };
    auto vector = [&](int j) -> uint4 {
        return j < held ? slice[j] : clean_vector<T>(*reinterpret_cast<const uint4 *>(logits + base + j * N));
    };

    auto each = [&](int from, auto &&f) {            // f(vector's number, its logits) from vector `from` of the thread on
        int j = from;
#pragma unroll 4
        for (; j < held; j += kThreads) {
            float x[N];
            unpack<T>(slice[j], x);
            f(j, x);
        }
        for (; j < n_vec; j += kThreads) {
            float x[N];
            unpack<T>(vector(j), x);
            f(j, x);
        }
    };

    // ---- 1: the maximum, and what at least top_k tokens reach
    cp_async_wait_all();
    float most = odd_x, nan = 0.f;
    each(tid, [&](int, const float (&x)[N]) {
#pragma unroll
        for (int e = 0; e < N; ++e) {
            most = fmaxf(most, x[e]);
            nan = x[e] != x[e] ? 1.f : nan;
        }
    });
    if (nan > 0.f || most == INFINITY) {
        for (int j = tid; j < held; j += kThreads) slice[j] = clean_vector<T>(slice[j]);
        most = clean<T>(most);
    }
    // the CTA's
    const float of_warp = warp_max(most);
    if (lane == 0) of_cta[warp] = of_warp;
    if (tid == 0) bound = 0;
    const bool bounded = !first_only && top_k < a.vocab;
    if (bounded)
        for (int i = tid; i < kBins; i += kThreads) bins[i] = 0;
    __syncthreads();
    float top = of_cta[0];                           // of the CTA, then of the row
#pragma unroll
    for (int w = 1; w < kWarps; ++w) top = fmaxf(top, of_cta[w]);
    const float c2 = fminf(inv_t * 1.4426950408889634f, FLT_MAX);    // logits to powers of two
    float reached = -INFINITY;
    if (bounded && top > -INFINITY) {
        const float largest = top;
        each(tid, [&](int, const float (&x)[N]) {
            float most_x = -INFINITY;
#pragma unroll
            for (int e = 0; e < N; ++e) most_x = fmaxf(most_x, x[e]);
            const float bin = (largest - most_x) * c2 * 8.f;
            if (bin < (float)kBins) atomicAdd(&bins[(int)bin], 1u);
        });
        __syncthreads();
        {
            // every warp finds the bin for itself: lane's eight bins, then up to the lane
            constexpr int kEach = kBins / 32;
            const uint32_t need = (uint32_t)((top_k - 1) / cluster + 1);
            uint32_t n[kEach], upto = 0;
#pragma unroll
            for (int i = 0; i < kEach; ++i) upto += n[i] = bins[lane * kEach + i];
            uint32_t before = upto;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t v = __shfl_up_sync(0xffffffffu, before, o);
                if (lane >= o) before += v;
            }
            before -= upto;
            int bin = kBins;
#pragma unroll
            for (int i = 0; i < kEach; ++i) {
                before += n[i];
                if (before >= need && bin == kBins) bin = lane * kEach + i;
            }
            bin = __reduce_min_sync(0xffffffffu, bin);
            // the bin's far edge, and what the difference and its product may be off by
            if (bin < kBins) reached = largest - (float)(bin + 1) * 1.0001f / (8.f * c2) - fabsf(largest) * 0x1p-22f;
        }
    }
    if (cluster > 1) cluster_wait_acquire();         // of the arrival at the start
    int token = -1;
    float logprob = -INFINITY;
    Place limit{-INFINITY, INT_MAX};                 // only tokens in front of it are in the race
    if (!dense_row) {
        // the row's maximum and bound; where all tokens are in the race they are not needed before it
        const Part *p = exchange(Part{0, 0.f, 0.f, top, reached, 0, {0, 0}});
        float m = -INFINITY, r = INFINITY;
        for (int i = lane; i < n_parts; i += 32) m = fmaxf(m, p[i].most), r = fminf(r, p[i].sum);
        top = warp_max(m);
        limit.x = -warp_max(-r);
    }
    if (dense_row || top > -INFINITY) {
        // By the maximum that is known: the CTA's in a dense row's first round. The roundings of the difference, of 1 / t, of
        // c2 and of the product move the argument by 2^-24 of itself each, and p by as much of |ln p|: with the constant's and
        // the exponential's own, p is within 2^-24 (5 |ln p| + 4) where it is not below 2^-126. quotient's argument shares the
        // first two: for |ln p| up to 87.4 the two are apart by less than 2^-15.5.
        auto about = [&](float x) { return exp2_fast((x - top) * c2); };
        // 2 p as near: not flushed for any p that quotient takes
        auto twice = [&](float x) { return exp2_fast(fmaf(x - top, c2, 1.f)); };
        // no logit below this has p >= min_p
        const float floor_x = min_p > 0.f ? top + (logf(min_p) - 0.01f) / inv_t - fabsf(top) * 0x1p-22f : -INFINITY;
        const bool by_mass = top_p < 1.f, tested = !first_only && (by_mass || top_k < a.vocab);
        float rest = 0.f, total = 0.f, token_x = 0.f;    // p of all tokens but the maxima, which are 1 each, and of all
        uint32_t tops = 0, in_race = 0;              // in_race: of later rounds
        bool found = false;                          // the border: the tokens in the race are the kept ones
        for (int round = 0;; ++round) {
            // ---- 2: the sum and the race
            Race race;
            float sum = 0.f;
            uint32_t n = 0;
            const float gate = first_only ? top : fmaxf(limit.x, floor_x);
            auto enter = [&](int v, float x, float nv) {                     // exactly, of tokens that may win
                if (first_only ? x == top : limit.behind(x, v))
                    race.enter(v, first_only ? 1.f : quotient(x - top, inv_t, min_p, nv), x, nv);
            };
            // All tokens, with their noise in vectors where it can be. A quotient is formed where a product says that it may
            // be the largest yet of the CTA's threads, which have the bound from one another; the first comes from quick
            // quotients. (With a bound of its own, some lane of a warp divides in most steps.)
            auto race_all = [&](auto gated) {
                constexpr bool kGated = decltype(gated)::value;
                const bool in_vectors = !kGated || (reinterpret_cast<uintptr_t>(noise + base) & 15) == 0;
                const int end = kGated ? n_vec : held;
                alignas(16) float nv[kBatch][N], next[kBatch][N];
                if (!kGated) sum *= 2.f;                     // so are the p that are added
                auto load = [&](int j0) {
#pragma unroll
                    for (int b = 0; b < kBatch; ++b) {
                        const int j = j0 + lane + b * kThreads;
                        if (j >= end || first_only) continue;
                        const float *src = noise + base + j * N;
                        if (in_vectors) {
#pragma unroll
                            for (int e = 0; e < N; e += 4) *reinterpret_cast<float4 *>(&next[b][e]) = *reinterpret_cast<const float4 *>(src + e);
                        } else {
#pragma unroll
                            for (int e = 0; e < N; ++e) next[b][e] = src[e];
                        }
                    }
                };
#pragma unroll
                for (int i = 0; i < kBatch * N; ++i) next[i / N][i % N] = 1.f;
                load(tid - lane);
                for (int j0 = tid - lane; j0 < end; j0 += kBatch * kThreads) {      // a warp's lanes together
#pragma unroll
                    for (int i = 0; i < kBatch * N; ++i) nv[i / N][i % N] = next[i / N][i % N];
                    load(j0 + kBatch * kThreads);
                    float x[kBatch][N], p[kBatch][N];        // p: twice p
#pragma unroll
                    for (int b = 0; b < kBatch; ++b) {
                        const int j = j0 + lane + b * kThreads;
                        if (j < end) {
                            unpack<T>(kGated ? vector(j) : slice[j], x[b]);
                        } else {
#pragma unroll
                            for (int e = 0; e < N; ++e) x[b][e] = -INFINITY;
                        }
#pragma unroll
                        for (int e = 0; e < N; ++e) {
                            p[b][e] = twice(x[b][e]);
                            if (!kGated) sum += p[b][e];
                            if (kGated && !(x[b][e] >= gate)) p[b][e] = 0.f;
                        }
                    }
                    if (!kGated && j0 < kThreads) {
                        float quick = 0.f;
#pragma unroll
                        for (int b = 0; b < kBatch; ++b)
#pragma unroll
                            for (int e = 0; e < N; ++e)
                                quick = fmaxf(quick, nv[b][e] >= FLT_MIN ? __fdividef(p[b][e], nv[b][e]) : 0.f);
                        race.low = fmaxf(race.low, fminf(warp_max(quick), FLT_MAX) * (1.f - 0x1p-14f));
                        if (lane == 0) atomicMax(&bound, __float_as_uint(race.low));
                    }
                    if (!kGated) race.low = fmaxf(race.low, __uint_as_float(*reinterpret_cast<volatile uint32_t *>(&bound)));
                    bool some = false;
#pragma unroll
                    for (int b = 0; b < kBatch; ++b)
#pragma unroll
                        for (int e = 0; e < N; ++e) some |= p[b][e] > race.low * nv[b][e];
                    if (__any_sync(0xffffffffu, some)) {
#pragma unroll
                        for (int b = 0; b < kBatch; ++b)
#pragma unroll
                            for (int e = 0; e < N; ++e)
                                if (p[b][e] > race.low * nv[b][e])
                                    enter(base + (j0 + lane + b * kThreads) * N + e, x[b][e], nv[b][e]);
                        race.low = warp_max(race.low);
                        if (!kGated && lane == 0) atomicMax(&bound, __float_as_uint(race.low));
                    }
                }
                if (!kGated) sum *= 0.5f;
            };
            const bool all_in = dense_row && round == 0;
            if (top > -INFINITY) {                   // a CTA of a dense row may have nothing
                if (odd >= 0) {
                    if (odd_x < top) sum = about(odd_x);
                    if (odd_x >= gate) enter(odd, odd_x, noise[odd]);
                }
                if (all_in) race_all(std::false_type{});
                if (!all_in || n_vec > held) {
                    int count = kListed + 1;
                    if (in_race <= (uint32_t)(kListed / 2 * cluster)) {
                        // few tokens are in the race: they are listed, and their noise is read by all threads at once
                        if (tid == 0) n_listed = 0;
                        __syncthreads();
                        each(tid + (all_in ? held : 0), [&](int j, const float (&x)[N]) {
                            float most_x = -INFINITY;
#pragma unroll
                            for (int e = 0; e < N; ++e) {
                                if (round == 0) sum += about(x[e]);
                                most_x = fmaxf(most_x, x[e]);
                            }
                            if (most_x >= gate) {
#pragma unroll
                                for (int e = 0; e < N; ++e) {
                                    const int v = base + j * N + e;
                                    if (x[e] < gate || (first_only ? x[e] < top : !limit.behind(x[e], v))) continue;
                                    const int at = atomicAdd(&n_listed, 1);
                                    if (at < kListed) listed[at] = make_float2(x[e], __int_as_float(v));
                                }
                            }
                        });
                        __syncthreads();
                        count = n_listed;
                    }
                    if (count <= kListed) {
                        for (int i = tid; i < count; i += kThreads) {
                            const int v = __float_as_int(listed[i].y);
                            enter(v, listed[i].x, first_only ? 1.f : noise[v]);
                        }
                    } else {
                        race_all(std::true_type{});
                    }
                    __syncthreads();                 // nobody reads the list any more
                }
                if (round == 0) {
                    // The maxima apart, for 1 swallows what it is added to: the lanes of a warp that has one sum its tokens
                    // again together.
                    if (most == top) {
                        sum = odd >= 0 && odd_x < top ? about(odd_x) : 0.f;
                        n = odd >= 0 && odd_x == top;
                    }
                    for (uint32_t left = __ballot_sync(0xffffffffu, most == top); left; left &= left - 1) {
                        const int other = __ffs(left) - 1;
                        for (int j = tid - lane + other + lane * kThreads; j < n_vec; j += 32 * kThreads) {
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
                }
            }
            race.of_warp();
            const Part *parts_of_all = exchange(Part{race.at, race.x, race.noise, top, warp_sum(sum), __reduce_add_sync(0xffffffffu, n), {0, 0}});
            Race best;
            float m = top;
            if (all_in) {
                for (int i = lane; i < n_parts; i += 32) m = fmaxf(m, parts_of_all[i].most);
                m = warp_max(m);
                if (m == -INFINITY) break;           // a row of -inf alone
            }
            top = m;
            float of_rest = 0.f;
            uint32_t of_tops = 0;
            bool far = false;                        // a part's winner is below the limit
            for (int i = lane; i < n_parts; i += 32) {
                const Part p = parts_of_all[i];
                if (p.most == top)
                    of_rest += p.sum, of_tops += p.n;
                else
                    of_rest += (p.sum + (float)p.n) * exp2_fast((p.most - top) * c2);
                if (p.at < 0) continue;
                const float key = first_only ? 1.f : quotient(p.x - top, inv_t, min_p, p.noise);
                best.enter(p.at, key, p.x, p.noise);
                far = far || key < 0.f;
            }
            best.of_warp();
            if (round == 0) {
                rest = warp_sum(of_rest);
                tops = __reduce_add_sync(0xffffffffu, of_tops);
                total = rest + (float)tops;
            }
            // In a dense row a CTA's winner may be below the limit of the row's maximum, which the CTA did not know, in front of
            // a token above it that could win: the race is run again by the row's maximum. Noise of the exponential
            // distribution is never as small as that needs.
            const bool again =
                round == 0 && __any_sync(0xffffffffu, far) && most_behind(parts_of_all, n_parts, top, inv_t) >= best.top;
            if (best.at < 0 || again) {              // not again: no noise was a positive number, the first in the order
                if (first_only) break;
                first_only = !again;
                in_race = again ? UINT32_MAX : 0;
                continue;
            }
            token = best.at;
            token_x = best.x;
            if (!tested || found || first_only) break;
            // ---- 3: whether the winner is kept
            Place at{best.x, token};
            unsigned long long no = 0, yes = 0;      // of the bisection: places not kept and kept,
            uint32_t front_no = 0, front_yes = 0;    // and the tokens in front of them
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
                each(tid, [&](int j, const float (&x)[N]) {
                    float most_x = -INFINITY;
#pragma unroll
                    for (int e = 0; e < N; ++e) most_x = fmaxf(most_x, x[e]);
                    if (most_x >= at.x) {
#pragma unroll
                        for (int e = 0; e < N; ++e) count(base + j * N + e, x[e]);
                    }
                });
                const Part *p = exchange(Part{0, 0.f, 0.f, 0.f, warp_sum(mass), __reduce_add_sync(0xffffffffu, front), {0, 0}});
                mass = 0.f;
                front = 0;
                for (int i = lane; i < n_parts; i += 32) mass += p[i].sum, front += p[i].n;
                mass = warp_sum(mass);
                front = __reduce_add_sync(0xffffffffu, front);
                kept = front < (uint32_t)top_k && (!by_mass || mass < top_p * total);
                if (yes == 0) {                      // the winner's place
                    in_race = front;
                    if (kept || round < kRejections) break;
                    no = at.number(), front_no = front;
                    yes = Place{top, 0}.number(), front_yes = 0;
                } else if (kept) {
                    yes = no + (yes - no) / 2, front_yes = front;
                } else {
                    no = no + (yes - no) / 2, front_no = front;
                }
                // at most one token between them: what is in front of it is in front of `yes`, so it is kept
                if (front_no - front_yes <= 1) {
                    found = true;
                    in_race = front_no;
                    break;
                }
                at = Place::of(no + (yes - no) / 2);
            }
            if (kept && yes == 0) break;
            limit = found ? Place::of(no) : at;
        }
        if (top > -INFINITY) {
            logprob = -(logf((float)tops) + log1pf(rest / (float)tops));
            if (token >= 0) logprob += (token_x - top) * inv_t;
        }
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
