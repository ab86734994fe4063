// lora_norm_rope: the norm of every query and key head, then the rotary positions
// and the append of k and v to the paged cache, in one pass over the rows.
//
//   y = x / sqrt(mean(x^2) + eps) * w,  (a, b) -> (a cos - b sin, a sin + b cos)
//
// The sum of squares, the norm and the turn are fp32 and the result is rounded once;
// between the norm and the rotation nothing is rounded or written. A row is read once
// and written once, as in lora_rope, whose layout of threads it keeps.
//
// 16384 tokens, 64 + 8 + 8 heads of 128 in bf16: 123 us, 5.5 TB/s of 6.8 (100 us); issue slots
// are busy for two thirds and waits for the arithmetic's own results are the first stall. 8 tokens
// 2.2 us in a graph, the launch and one chain of reads.
#include "rope_common.cuh"

#include <algorithm>
#include <atomic>
#include <climits>
#include <cmath>

namespace lora {
namespace {

using namespace step;
using namespace rope;

struct NormArgs {
    RopeArgs r;
    const void *q_weight, *k_weight;       // nullptr: ones
    long long q_weight_head, k_weight_head;
    float eps, one_over_dim;
};

// The weight of head row r (q heads, then k); nullptr: ones.
template <typename T>
__device__ __forceinline__ const T *weight_of(const NormArgs &n, int r) {
    const bool q = r < n.r.n_heads;
    const T *w = static_cast<const T *>(q ? n.q_weight : n.k_weight);
    return w ? w + (q ? r * n.q_weight_head : (r - n.r.n_heads) * n.k_weight_head) : nullptr;
}

// Any layout: one warp per head row of one token; the row is read again for the turn.
// Bound by its issue slots; for rows that are not whole 16-byte vectors or longer
// than 64 of them.
template <typename T, bool kInterleaved>
__global__ void __launch_bounds__(256) norm_rows_kernel(NormArgs n) {
    const RopeArgs &a = n.r;
    grid_dependency_wait();
    grid_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int rows = a.n_heads + 2 * a.n_kv;
    const long long item = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (item >= (long long)a.n_tokens * rows) return;
    const long long t = item / rows;
    const int r = (int)(item % rows), pos = a.positions[t];
    if (pos < 0 || pos >= a.n_positions) return;
    const Row<T> w = row_of<T>(a, t, r, cache_place(a, t));
    if (!w.dst) return;
    if (!w.turned) {
        for (int i = lane; i < a.head_dim; i += 32) w.dst[i] = w.src[i];
        return;
    }
    const T *weight = weight_of<T>(n, r);
    float sum = 0.f;
    for (int i = lane; i < a.head_dim; i += 32) {
        const float x = to_f32(w.src[i]);
        sum = fmaf(x, x, sum);
    }
    const float inv = rsqrtf(fmaf(warp_sum(sum), n.one_over_dim, n.eps));
    auto normed = [&](int i) { return to_f32(w.src[i]) * inv * (weight ? to_f32(weight[i]) : 1.f); };
    const int half = a.rot_dim / 2;
    const float *row = a.table + (size_t)pos * a.rot_dim;
    for (int j = lane; j < half; j += 32) {
        const float c = row[j], s = row[half + j];
        const int i0 = kInterleaved ? 2 * j : j, i1 = kInterleaved ? 2 * j + 1 : j + half;
        const float x0 = normed(i0), x1 = normed(i1);
        w.dst[i0] = from_f32<T>(x0 * c - x1 * s);
        w.dst[i1] = from_f32<T>(x0 * s + x1 * c);
    }
    for (int i = a.rot_dim + lane; i < a.head_dim; i += 32) w.dst[i] = from_f32<T>(normed(i));
}

// The elements of 16 bytes in pairs.
template <typename T>
__device__ __forceinline__ void unpack2(const uint4 &v, uint64_t (&f)[8 / sizeof(T)]) {
    float x[16 / sizeof(T)];
    unpack<T>(v, x);
#pragma unroll
    for (int i = 0; i < (int)(8 / sizeof(T)); ++i) f[i] = pair(x[2 * i], x[2 * i + 1]);
}
template <typename T>
__device__ __forceinline__ uint4 pack2(const uint64_t (&f)[8 / sizeof(T)]) {
    float x[16 / sizeof(T)];
#pragma unroll
    for (int i = 0; i < (int)(8 / sizeof(T)); ++i) unpair(f[i], x[2 * i], x[2 * i + 1]);
    return pack(x);
}
__device__ __forceinline__ uint64_t swapped(uint64_t v) {
    float lo, hi;
    unpair(v, lo, hi);
    return pair(hi, lo);
}

// Rows in 16-byte vectors: a unit is two vectors of a row that are turned together (as
// in lora_rope), or two neighbours past rot_dim and in v. A row's units, rounded up to a
// power of two, are lanes in a row, so that its sum of squares stays in a part of a
// warp. Weights, cosines and sines make the four coefficients of a unit, mostly the same for
// many rows of a token:
//   y0 = (x0 A0 + x1 B0) / rms, y1 = (x1 A1 + x0 B1) / rms
// (interleaved: each vector with its pairs swapped instead of the other vector).
template <typename T, bool kInterleaved>
struct Units {
    static constexpr int N = 16 / sizeof(T), P = N / 2;
    const NormArgs &n;
    int u, vectors, v0, v1, normed, rows;
    bool turns;                                            // in a row that is normed and turned
    uint64_t a0[P], a1[P], b0[P], b1[P];

    __device__ __forceinline__ explicit Units(const NormArgs &args) : n(args) {
        const RopeArgs &a = n.r;
        const int rot_vectors = a.rot_dim / N;
        u = threadIdx.x;
        vectors = a.head_dim / N;
        turns = kInterleaved ? 2 * u < rot_vectors : u < rot_vectors / 2;
        v0 = kInterleaved || !turns ? 2 * u : u;
        v1 = kInterleaved || !turns ? 2 * u + 1 : u + rot_vectors / 2;
        normed = a.n_heads + a.n_kv;
        rows = normed + a.n_kv;
    }
    // Element offset of row r in its token's q, k or v, and in what is written; which of them. They fit 32 bits.
    __device__ __forceinline__ int source(int r) const {
        const RopeArgs &a = n.r;
        return r < a.n_heads ? r * (int)a.q_head : r < normed ? (r - a.n_heads) * (int)a.k_head : (r - normed) * (int)a.v_head;
    }
    __device__ __forceinline__ int target(int r) const {
        const RopeArgs &a = n.r;
        return r < a.n_heads ? r * (int)a.qo_head : (r < normed ? r - a.n_heads : r - normed) * (int)a.c_head;
    }
    template <typename U>
    __device__ __forceinline__ U *of_row(int r, U *q, U *k, U *v) const {
        return r < n.r.n_heads ? q : r < normed ? k : v;
    }
    __device__ __forceinline__ int first_vector(int r) const { return r < normed ? v0 : 2 * u; }
    __device__ __forceinline__ int second_vector(int r) const { return r < normed ? v1 : 2 * u + 1; }
    __device__ __forceinline__ void weights(const T *weight, uint4 &w0, uint4 &w1) const {
        if (weight && v0 < vectors) w0 = *reinterpret_cast<const uint4 *>(weight + v0 * N);
        if (weight && v1 < vectors) w1 = *reinterpret_cast<const uint4 *>(weight + v1 * N);
    }
    // From the unit's weights (none: ones) and the token's angles, rot_dim / 2 cosines, then as many sines.
    __device__ __forceinline__ void coefficients(bool some, const uint4 &wv0, const uint4 &wv1, const float *angles) {
        uint64_t w0[P], w1[P];
        unpack2<T>(wv0, w0);
        unpack2<T>(wv1, w1);
#pragma unroll
        for (int i = 0; i < P; ++i) {
            if (!some) w0[i] = w1[i] = pair(1.f, 1.f);
            a0[i] = w0[i], a1[i] = w1[i], b0[i] = b1[i] = 0;
        }
        if (!turns) return;
        // N angles: of elements 2u N .. (interleaved: of N pairs) or u N ..
        alignas(16) float c[N], s[N];
#pragma unroll
        for (int j = 0; j < N; j += 4) {
            *reinterpret_cast<float4 *>(c + j) = *reinterpret_cast<const float4 *>(angles + u * N + j);
            *reinterpret_cast<float4 *>(s + j) = *reinterpret_cast<const float4 *>(angles + n.r.rot_dim / 2 + u * N + j);
        }
#pragma unroll
        for (int i = 0; i < P; ++i) {
            if (kInterleaved) {                            // pair i of the vectors has angles i and P + i
                b0[i] = mul2(swapped(w0[i]), pair(-s[i], s[i]));
                b1[i] = mul2(swapped(w1[i]), pair(-s[P + i], s[P + i]));
                a0[i] = mul2(w0[i], pair(c[i], c[i]));
                a1[i] = mul2(w1[i], pair(c[P + i], c[P + i]));
            } else {
                b0[i] = mul2(w1[i], pair(-s[2 * i], -s[2 * i + 1]));
                b1[i] = mul2(w0[i], pair(s[2 * i], s[2 * i + 1]));
                a0[i] = mul2(w0[i], pair(c[2 * i], c[2 * i + 1]));
                a1[i] = mul2(w1[i], pair(c[2 * i], c[2 * i + 1]));
            }
        }
    }
    // A row's unit, normed and turned where it is to be; every lane of the warp calls it.
    __device__ __forceinline__ void turn(uint4 &v0, uint4 &v1, bool is_normed) const {
        uint64_t x0[P], x1[P], sums[2] = {0, 0};
        unpack2<T>(v0, x0);
        unpack2<T>(v1, x1);
#pragma unroll
        for (int j = 0; j < P; ++j) {
            sums[0] = fma2(x0[j], x0[j], sums[0]);
            sums[1] = fma2(x1[j], x1[j], sums[1]);
        }
        float sum, other;
        unpair(add2(sums[0], sums[1]), sum, other);
        sum += other;
#pragma unroll
        for (int o = 1; o < 32; o *= 2)
            if (o < (int)blockDim.x) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (!is_normed) return;
        const float rms = rsqrtf(fmaf(sum, n.one_over_dim, n.eps));
        const uint64_t inv = pair(rms, rms);
        uint64_t y0[P], y1[P];
#pragma unroll
        for (int j = 0; j < P; ++j) {
            x0[j] = mul2(x0[j], inv);
            x1[j] = mul2(x1[j], inv);
            y0[j] = mul2(x0[j], a0[j]);
            y1[j] = mul2(x1[j], a1[j]);
        }
        if (turns) {                                       // not by zero: an infinity past rot_dim stays where it is
#pragma unroll
            for (int j = 0; j < P; ++j) {
                y0[j] = fma2(kInterleaved ? swapped(x0[j]) : x1[j], b0[j], y0[j]);
                y1[j] = fma2(kInterleaved ? swapped(x1[j]) : x0[j], b1[j], y1[j]);
            }
        }
        v0 = pack2<T>(y0);
        v1 = pack2<T>(y1);
    }
};

// Few rows: a thread takes its unit of one row. It is latency: a launch, the position, the angles.
template <typename T, bool kInterleaved>
__global__ void __launch_bounds__(256) norm_vectors_kernel(NormArgs n) {
    constexpr int N = 16 / sizeof(T);
    const RopeArgs &a = n.r;
    grid_dependency_wait();
    grid_launch_dependents();
    const long long t = blockIdx.x;
    Units<T, kInterleaved> unit(n);
    const int r = blockIdx.y * blockDim.y + threadIdx.y, pos = a.positions[t];
    const long long at = cache_place(a, t);
    const bool there = pos >= 0 && pos < a.n_positions && r < (at >= 0 ? unit.rows : a.n_heads);
    const int e0 = unit.first_vector(r), e1 = unit.second_vector(r);
    uint4 x0 = make_uint4(0, 0, 0, 0), x1 = x0, w0 = x0, w1 = x0;
    const T *weight = nullptr;
    if (there) {
        const T *src = unit.of_row(r, static_cast<const T *>(a.q) + t * a.q_token, static_cast<const T *>(a.k) + t * a.k_token,
                                   static_cast<const T *>(a.v) + t * a.v_token) + unit.source(r);
        if (e0 < unit.vectors) x0 = *reinterpret_cast<const uint4 *>(src + e0 * N);
        if (e1 < unit.vectors) x1 = *reinterpret_cast<const uint4 *>(src + e1 * N);
        if (r < unit.normed) {
            weight = weight_of<T>(n, r);
            unit.weights(weight, w0, w1);
            unit.coefficients(weight, w0, w1, a.table + (size_t)pos * a.rot_dim);
        }
    }
    unit.turn(x0, x1, there && r < unit.normed);
    if (!there) return;
    T *dst = unit.of_row(r, static_cast<T *>(a.q_out) + t * a.qo_token, static_cast<T *>(a.k_cache) + at,
                         static_cast<T *>(a.v_cache) + at) + unit.target(r);
    if (e0 < unit.vectors) *reinterpret_cast<uint4 *>(dst + e0 * N) = x0;
    if (e1 < unit.vectors) *reinterpret_cast<uint4 *>(dst + e1 * N) = x1;
}

// Many rows: a block goes over tokens, `rounds` rows of a token to a thread, with the rows and
// angles of the next kStages - 1 tokens on their way to shared memory. Rows do not wait for
// the token's position, which is read a token earlier than its angles. (Blocks of one token each
// wait for position, rows and angles in turn: 145 us for 16384 tokens of 64 + 8 heads.) Threads x
// blocks of an SM for the same: 96 x 5 124 us, 128 x 4 126, 128 x 5 123, 160 x 4 128, 192 x 4 156,
// 320 x 2 157. kTail: a row has fewer than two vectors for each of its lanes.
constexpr int kStages = 2, kStreamThreads = 128, kStreamBlocks = 5;   // blocks of an SM

struct Stream {
    int rounds, chunk;                                     // chunk: rows of a token that a block takes
    int stage_bytes;
};

template <typename T, bool kInterleaved, bool kTail>
__global__ void __launch_bounds__(kStreamThreads, kStreamBlocks) norm_stream_kernel(NormArgs n, Stream how) {
    constexpr int N = 16 / sizeof(T);
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ long long places[kStages];                  // of the stages' tokens: in the caches, or -1
    __shared__ int found[kStages];                         // whether the position is in the table
    const RopeArgs &a = n.r;
    grid_dependency_wait();
    grid_launch_dependents();
    Units<T, kInterleaved> unit(n);
    const int threads = blockDim.x * blockDim.y, tid = threadIdx.y * blockDim.x + threadIdx.x;
    const int r0 = blockIdx.y * how.chunk, r1 = min(r0 + how.chunk, unit.rows);
    const int x_bytes = how.stage_bytes - a.rot_dim * 4;
    const int tokens = (a.n_tokens - (int)blockIdx.x + (int)gridDim.x - 1) / (int)gridDim.x;   // of this block
    auto token = [&](int i) { return (long long)blockIdx.x + (long long)i * gridDim.x; };
    int pos = 0;                                           // of the next token to be loaded
    long long slot = -1;
    auto look = [&](int i) {
        if (i >= tokens) return;
        pos = a.positions[token(i)];
        if (tid == 0 && a.n_kv > 0) slot = a.slots[token(i)];
    };
    auto load = [&](int i) {
        if (i < tokens) {
            const int stage = i % kStages;
            unsigned char *to = smem + stage * how.stage_bytes;
            const long long t = token(i);
            const T *q = static_cast<const T *>(a.q) + t * a.q_token, *k = static_cast<const T *>(a.k) + t * a.k_token;
            const T *v = static_cast<const T *>(a.v) + t * a.v_token;
            unsigned char *mine = to + tid * 16;
            for (int r = r0 + (int)threadIdx.y; r < r1; r += blockDim.y, mine += 32 * threads) {
                const T *src = unit.of_row(r, q, k, v) + unit.source(r);
                const int e0 = unit.first_vector(r), e1 = unit.second_vector(r);
                if (e0 < unit.vectors) cp_async16(mine, src + e0 * N);
                if (e1 < unit.vectors) cp_async16(mine + 16 * threads, src + e1 * N);
            }
            const bool ok = pos >= 0 && pos < a.n_positions;
            if (ok)
                for (int j = tid; j < a.rot_dim / 4; j += threads)
                    cp_async16(to + x_bytes + j * 16, a.table + (size_t)pos * a.rot_dim + j * 4);
            if (tid == 0) {
                places[stage] = place_of(a, slot);
                found[stage] = ok;
            }
        }
        cp_async_commit();
    };
    for (int i = 0; i < kStages - 1; ++i) {
        look(i);
        load(i);
    }
    look(kStages - 1);
    // weights that are the same for all heads stay in registers
    uint4 qw0 = make_uint4(0, 0, 0, 0), qw1 = qw0, kw0 = qw0, kw1 = qw0;
    unit.weights(static_cast<const T *>(n.q_weight), qw0, qw1);
    unit.weights(static_cast<const T *>(n.k_weight), kw0, kw1);
    for (int i = 0; i < tokens; ++i) {
        asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
        __syncthreads();                                   // token i is here, and everyone is done with the one before
        load(i + kStages - 1);
        look(i + kStages);
        const int stage = i % kStages;
        if (!found[stage]) continue;
        const unsigned char *from = smem + stage * how.stage_bytes;
        const float *angles = reinterpret_cast<const float *>(from + x_bytes);
        const long long at = places[stage], t = token(i);
        T *q = static_cast<T *>(a.q_out) + t * a.qo_token, *k = static_cast<T *>(a.k_cache) + at, *v = static_cast<T *>(a.v_cache) + at;
        const int written = at >= 0 ? r1 : min(r1, a.n_heads);
        int held = -1;                                     // the coefficients are those of the queries (0) or keys (1)
        const unsigned char *mine = from + tid * 16;
        int r = r0 + (int)threadIdx.y;
        for (int j = 0; j < how.rounds; ++j, r += blockDim.y, mine += 32 * threads) {
            uint4 x0 = *reinterpret_cast<const uint4 *>(mine), x1 = *reinterpret_cast<const uint4 *>(mine + 16 * threads);
            const int e0 = unit.first_vector(r), e1 = unit.second_vector(r);
            if (kTail) {                                   // lanes without a vector, which was not copied
                if (e0 >= unit.vectors) x0 = make_uint4(0, 0, 0, 0);
                if (e1 >= unit.vectors) x1 = make_uint4(0, 0, 0, 0);
            }
            const bool norm = r < unit.normed;
            if (norm) {
                const int kind = r < a.n_heads ? 0 : 1;
                const long long head = kind ? n.k_weight_head : n.q_weight_head;
                const bool some = kind ? n.k_weight : n.q_weight;
                if (some && head != 0) {
                    uint4 w0 = make_uint4(0, 0, 0, 0), w1 = w0;
                    unit.weights(weight_of<T>(n, r), w0, w1);
                    unit.coefficients(true, w0, w1, angles);
                } else if (held != kind) {
                    unit.coefficients(some, kind ? kw0 : qw0, kind ? kw1 : qw1, angles);
                    held = kind;
                }
            }
            unit.turn(x0, x1, norm);
            if (r >= written) continue;
            T *dst = unit.of_row(r, q, k, v) + unit.target(r);
            if (!kTail || e0 < unit.vectors) *reinterpret_cast<uint4 *>(dst + e0 * N) = x0;
            if (!kTail || e1 < unit.vectors) *reinterpret_cast<uint4 *>(dst + e1 * N) = x1;
        }
    }
}

// What by_vectors asks of the rows, of the weights and the table, too.
template <typename T>
bool weights_by_vectors(const NormArgs &n) {
    constexpr int N = 16 / sizeof(T);
    for (long long s : {n.r.q_head, n.r.qo_head})
        if (s > INT_MAX / (n.r.n_heads + 1) || s < INT_MIN / (n.r.n_heads + 1)) return false;
    for (long long s : {n.r.k_head, n.r.v_head, n.r.c_head})
        if (s > INT_MAX / (n.r.n_kv + 1) || s < INT_MIN / (n.r.n_kv + 1)) return false;
    return aligned16(n.r.table) && n.r.rot_dim % 8 == 0 && aligned16(n.q_weight) && aligned16(n.k_weight) && n.q_weight_head % N == 0 && n.k_weight_head % N == 0;
}

template <typename T, bool kInterleaved>
cudaError_t launch_vectors(const NormArgs &n, int units, cudaStream_t st) {
    const int rows = n.r.n_heads + 2 * n.r.n_kv, whole = 32 / units;
    const int fit = 256 / units, blocks = (rows + fit - 1) / fit, each = (rows + blocks - 1) / blocks;
    // whole warps: their lanes add up together
    return launch_step(norm_vectors_kernel<T, kInterleaved>, dim3(n.r.n_tokens, blocks),
                       dim3(units, (each + whole - 1) / whole * whole), 0, 1, st, n);
}

template <typename T, bool kInterleaved, bool kTail>
cudaError_t launch_stream(const NormArgs &n, int units, int sms, cudaStream_t st) {
    constexpr int kBytes = 24 * 1024;
    auto kernel = norm_stream_kernel<T, kInterleaved, kTail>;
    static std::atomic<uint64_t> ready{0};
    if (!device_bit(ready)) {
        const cudaError_t e =
            cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kStages * (kBytes + 4096));
        if (e != cudaSuccess) return e;
        set_device_bit(ready);
    }
    const int rows = n.r.n_heads + 2 * n.r.n_kv, whole = 32 / units, row_bytes = units * 32;
    // chunks of a token's rows that fit a stage, each in rounds of whole warps
    const int chunks = (rows * row_bytes + kBytes - 1) / kBytes, per = (rows + chunks - 1) / chunks;
    const int rounds = std::max((per * units + kStreamThreads - 1) / kStreamThreads, 1);
    const int y = ((per + rounds - 1) / rounds + whole - 1) / whole * whole;
    Stream how;
    how.rounds = rounds;
    how.chunk = per;
    how.stage_bytes = rounds * y * units * 32 + n.r.rot_dim * 4;
    // as many blocks as run at once: of the largest stages four fit an SM's 228 KB, each with 1 KB of the system's
    const int fit = std::min(kStreamBlocks, 228 * 1024 / (kStages * how.stage_bytes + 1024 + 128));
    const int blocks = std::max(std::min(n.r.n_tokens, fit * sms / chunks), 1);
    return launch_step(kernel, dim3(blocks, chunks), dim3(units, y), (size_t)kStages * how.stage_bytes, 1, st, n, how);
}

template <typename T, bool kInterleaved>
cudaError_t launch_norm(const NormArgs &n, int sms, cudaStream_t st) {
    const RopeArgs &a = n.r;
    const long long rows = (long long)a.n_tokens * (a.n_heads + 2 * a.n_kv);
    int units = 1;
    while (units < (a.head_dim / (int)(16 / sizeof(T)) + 1) / 2) units *= 2;
    if (units <= 32 && by_vectors<T>(a, kInterleaved) && weights_by_vectors<T>(n)) {
        // The stream's blocks need a few tokens each, and a token two rounds. In bf16, 32 + 8 heads of 128, rows one by one /
        // streamed: 512 tokens 4.9 / 5.1 us, 1024 8.1 / 8.1, 2048 17.0 / 13.9, 4096 33.0 / 24.9, 8192 68 / 45; 16 + 4 heads of
        // 256, 2000 tokens 16.9 / 14.1; 8 + 2 heads of 64, 4096 tokens 5.9 / 9.7
        if (rows <= 300ll * sms || (a.n_heads + 2 * a.n_kv) * units < 256) return launch_vectors<T, kInterleaved>(n, units, st);
        return units * 2 * (int)(16 / sizeof(T)) == a.head_dim ? launch_stream<T, kInterleaved, false>(n, units, sms, st)
                                                               : launch_stream<T, kInterleaved, true>(n, units, sms, st);
    }
    return launch_step(norm_rows_kernel<T, kInterleaved>, dim3((unsigned)((rows + 7) / 8)), dim3(256), 0, 1, st, n);
}

}  // namespace
}  // namespace lora

using namespace lora;
using namespace lora::step;
using namespace lora::rope;

extern "C" int lora_norm_rope(const lora_norm_rope_desc *d, void *stream) {
    if (!d) return fail(LORA_ERR_ARG, "norm_rope: NULL descriptor");
    bool nothing;
    const int rc = check(&d->rope, "norm_rope", &nothing);
    if (rc != LORA_OK) return rc;
    if (d->rope.inverse) return fail(LORA_ERR_ARG, "norm_rope: inverse is not 0 (the norm has no inverse here)");
    if (!(d->eps >= 0.f) || !std::isfinite(d->eps)) return fail(LORA_ERR_ARG, "norm_rope: eps must be finite and not negative");
    if (d->q_weight_head < 0 || d->k_weight_head < 0)
        return fail(LORA_ERR_ARG, "norm_rope: the weights' strides %lld, %lld are negative", (long long)d->q_weight_head,
                    (long long)d->k_weight_head);
    if (nothing) return LORA_OK;
    NormArgs n{arguments(&d->rope), nullptr, nullptr, 0, 0, d->eps, 1.f / (float)d->rope.head_dim};
    // a weight of no heads is not looked at, not even for its alignment
    if (d->rope.n_heads > 0) n.q_weight = d->q_weight, n.q_weight_head = d->q_weight_head;
    if (d->rope.n_kv_heads > 0) n.k_weight = d->k_weight, n.k_weight_head = d->k_weight_head;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int sms = sm_count();
    if (sms < 1) return fail(LORA_ERR_CUDA, "norm_rope: no CUDA device");
    cudaError_t e;
    if (d->rope.dtype == LORA_DTYPE_BF16)
        e = d->rope.interleaved ? launch_norm<__nv_bfloat16, true>(n, sms, st) : launch_norm<__nv_bfloat16, false>(n, sms, st);
    else
        e = d->rope.interleaved ? launch_norm<float, true>(n, sms, st) : launch_norm<float, false>(n, sms, st);
    return launched("norm_rope", e);
}
