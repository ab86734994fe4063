// lora_tree_attention and lora_prefix_attention in fp32: tiles of M rows and 64 keys on the FMA units.
//
// 128 threads; a half-warp (16 lanes) owns M / 8 rows. Scores: a lane has those rows
// against keys lane, lane + 16, + 32, + 48, so a row's maximum and sum are a
// half-warp's. The weights go to shared memory over the keys they were formed
// from, and a lane sums DP / 16 columns of O for the same rows. FMA-bound for 64
// rows (a shared-memory wavefront feeds 8 or more FMA instructions); for few rows
// 16 are taken, so that little is computed for rows that do not exist. The split of the
// work and the join are those of the tensor-core kernels. Two CTAs of an SM load
// and compute in turn. 64 nodes, 64 heads over 8, ctx 32768: 1.55 ms, 44 TFLOP/s.
#include "tree_common.cuh"

#include <atomic>

namespace lora {
namespace tree {
namespace {

constexpr int kThreads = 128;

template <int DP, int M>
struct F32 {
    static constexpr int R = M / 8;                            // rows of a half-warp
    static constexpr int C = DP / 16;                          // columns of a lane in O
    static constexpr int kRow = DP + 4;                        // floats of a staged row of Q and K: 16 lanes' keys differ
                                                               // in their banks
    static constexpr int kW = kTileKeys + 4;                   // floats of a row of weights
    static constexpr int kKeys = kTileKeys * kRow > M * kW ? kTileKeys * kRow : M * kW;
    static constexpr int kSmem = (M * kRow + kKeys + kTileKeys * DP) * 4;
};

template <int DP, int M, bool kPrefix>
__global__ void __launch_bounds__(kThreads, 2) tree_f32_kernel(TreeArgs a, Plan plan) {
    using T = F32<DP, M>;
    constexpr int R = T::R, C = T::C, kPieces = DP / 4;
    extern __shared__ __align__(128) unsigned char smem[];
    float *qs = reinterpret_cast<float *>(smem), *ks = qs + M * T::kRow, *vs = ks + T::kKeys;
    __shared__ long long scratch[kScratch + kThreads / 32], offs[kTileKeys];
    __shared__ uint32_t valid[2];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, half = tid >> 4, l16 = tid & 15;
    const int group = a.n_heads / a.n_kv, row0 = half * R;     // this half-warp's rows of the tile
    grid_dependency_wait();
    grid_launch_dependents();                                  // the join kernel waits for this grid's end itself
    if (!kPrefix && tid == 0) plan.seg[blockIdx.x] = make_int4(0, 0, 0, 0);
    Share share;
    if (!find_share<kThreads, kPrefix>(a, M, scratch, share)) return;
    Cursor c = share.start;
    const int n_tiles = share.n_tiles;
    const float c2 = a.scale * 1.4426950408889634f;            // scores in powers of two

    float o[R][C], m[R], l[R];
    int seg_first = c.tile;
    for (int i = 0; i < n_tiles; ++i) {
        const bool first = i == 0 || c.tile == 0;
        __syncthreads();                                       // everyone is done with the tile before
        if (tid < kTileKeys) {
            const long long off = key_offset<kPrefix>(a, c, tid);
            offs[tid] = off;
            const uint32_t ok = __ballot_sync(0xffffffffu, off >= 0);
            if (lane == 0) valid[warp] = ok;
        }
        if (first) {
            for (int n = tid; n < M * kPieces; n += kThreads) {
                const int r = n / kPieces, p = n % kPieces, row = c.row_tile * M + r, node = row / group;
                const bool ok = node < c.r.nodes && p * 4 < a.head_dim;
                const long long at = (c.r.start + node) * a.q_token + (c.head * group + row % group) * a.q_head + p * 4;
                copy16(smem_u32(qs + r * T::kRow + p * 4), static_cast<const float *>(a.q) + (ok ? at : 0), ok);
            }
#pragma unroll
            for (int r = 0; r < R; ++r) {
                m[r] = -INFINITY;
                l[r] = 0.f;
#pragma unroll
                for (int e = 0; e < C; ++e) o[r][e] = 0.f;
            }
            seg_first = c.tile;
        }
        __syncthreads();
        const long long head_at = (long long)c.head * a.c_head;
#pragma unroll 4
        for (int n = tid; n < kTileKeys * kPieces; n += kThreads) {
            const int k = n / kPieces, p = n % kPieces;
            const long long off = offs[k];
            const bool ok = off >= 0 && p * 4 < a.head_dim;
            const long long at = ok ? off + head_at + p * 4 : 0;
            copy16(smem_u32(ks + k * T::kRow + p * 4), static_cast<const float *>(a.k_cache) + at, ok);
            copy16(smem_u32(vs + k * DP + p * 4), static_cast<const float *>(a.v_cache) + at, ok);
        }
        cp_async_commit();
        cp_async_wait_all();
        __syncthreads();

        // ---- scores
        float s[R][4];
#pragma unroll
        for (int r = 0; r < R; ++r) s[r][0] = s[r][1] = s[r][2] = s[r][3] = 0.f;
#pragma unroll 2
        for (int d = 0; d < DP; d += 4) {
            float4 k4[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) k4[j] = *reinterpret_cast<const float4 *>(ks + (l16 + 16 * j) * T::kRow + d);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const float4 q4 = *reinterpret_cast<const float4 *>(qs + (row0 + r) * T::kRow + d);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    s[r][j] = fmaf(q4.x, k4[j].x, fmaf(q4.y, k4[j].y, fmaf(q4.z, k4[j].z, fmaf(q4.w, k4[j].w, s[r][j]))));
            }
        }
        // ---- keys a row does not see
        const int p0 = c.tile * kTileKeys;
        const uint64_t there = valid[0] | (uint64_t)valid[1] << 32;
        const bool masked = there != ~0ull || p0 + kTileKeys > c.r.ctx;
        bool hidden = false;                                   // a key that is there but that a row skips
#pragma unroll
        for (int r = 0; r < R; ++r) {
            uint64_t seen = ~0ull;
            if (masked) {
                const int node = (c.row_tile * M + row0 + r) / group;
                seen = node < c.r.nodes ? seen_keys(a, c.r, node, p0) & there : 0;
                hidden = hidden || (node < c.r.nodes && seen != there);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) s[r][j] = seen >> (l16 + 16 * j) & 1 ? s[r][j] * c2 : -INFINITY;
        }
        __syncthreads();                                       // K has been read: the weights take its place
        // ---- running maximum and sum, weights
#pragma unroll
        for (int r = 0; r < R; ++r) {
            float top = fmaxf(fmaxf(s[r][0], s[r][1]), fmaxf(s[r][2], s[r][3]));
#pragma unroll
            for (int x = 8; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
            top = fmaxf(top, m[r]);
            const float base = top == -INFINITY ? 0.f : top;
            const float keep = exp2f(m[r] - base);
            m[r] = top;
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float w = exp2f(s[r][j] - base);
                sum += w;
                ks[(row0 + r) * T::kW + l16 + 16 * j] = w;
            }
            l[r] = l[r] * keep + sum;                          // this lane's keys; joined at the end
#pragma unroll
            for (int e = 0; e < C; ++e) o[r][e] *= keep;
        }
        // A weight of zero times an infinity or NaN is NaN: where a row skips a key, values that are not finite are
        // looked for, and such a tile is summed without the zero weights.
        bool skip_zero = false;
        if (masked && __syncthreads_or(hidden)) {
            bool odd = false;
            for (int n = tid; n < kTileKeys * DP; n += kThreads) odd = odd || !isfinite(vs[n]);
            skip_zero = __syncthreads_or(odd);
        }
        __syncwarp();                                          // a half-warp reads its own rows' weights
        if (skip_zero) {
            for (int k = 0; k < kTileKeys; ++k)
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const float w = ks[(row0 + r) * T::kW + k];
                    if (w == 0.f) continue;
#pragma unroll
                    for (int e = 0; e < C; ++e) o[r][e] = fmaf(w, vs[k * DP + (e / 4) * 64 + l16 * 4 + e % 4], o[r][e]);
                }
        } else {
#pragma unroll 2
            for (int k = 0; k < kTileKeys; k += 4) {
                float4 w4[R];
#pragma unroll
                for (int r = 0; r < R; ++r) w4[r] = *reinterpret_cast<const float4 *>(ks + (row0 + r) * T::kW + k);
#pragma unroll
                for (int e = 0; e < C; e += 4) {               // columns 64 (e / 4) + 4 l16 .. + 3
                    float4 v4[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        v4[j] = *reinterpret_cast<const float4 *>(vs + (k + j) * DP + (e / 4) * 64 + l16 * 4);
#pragma unroll
                    for (int r = 0; r < R; ++r) {
                        o[r][e] = fmaf(w4[r].x, v4[0].x, fmaf(w4[r].y, v4[1].x, fmaf(w4[r].z, v4[2].x, fmaf(w4[r].w, v4[3].x, o[r][e]))));
                        o[r][e + 1] = fmaf(w4[r].x, v4[0].y, fmaf(w4[r].y, v4[1].y, fmaf(w4[r].z, v4[2].y, fmaf(w4[r].w, v4[3].y, o[r][e + 1]))));
                        o[r][e + 2] = fmaf(w4[r].x, v4[0].z, fmaf(w4[r].y, v4[1].z, fmaf(w4[r].z, v4[2].z, fmaf(w4[r].w, v4[3].z, o[r][e + 2]))));
                        o[r][e + 3] = fmaf(w4[r].x, v4[0].w, fmaf(w4[r].y, v4[1].w, fmaf(w4[r].z, v4[2].w, fmaf(w4[r].w, v4[3].w, o[r][e + 3]))));
                    }
                }
            }
        }
        if (c.tile + 1 == c.r.key_tiles || i + 1 == n_tiles) {
            const bool starts = seg_first == 0, ends = c.tile + 1 == c.r.key_tiles;
            const long long slot = 2ll * blockIdx.x + (starts ? 1 : 0);
#pragma unroll
            for (int r = 0; r < R; ++r) {
#pragma unroll
                for (int x = 8; x > 0; x >>= 1) l[r] += __shfl_xor_sync(0xffffffffu, l[r], x);
                const int row = c.row_tile * M + row0 + r, node = row / group;
                if (node >= c.r.nodes) continue;
                const long long token = c.r.start + node;
                const int head = c.head * group + row % group;
                // a row without keys is 0; one whose scores are all NaN also has m = -inf, but its l is NaN
                const bool none = l[r] == 0.f, done = !kPrefix && starts && ends;
                const float inv = !done ? 1.f : l[r] > 0.f ? 1.f / l[r] : l[r];
                float *dst = done ? static_cast<float *>(a.out) + token * a.o_token + (long long)head * a.o_head
                                  : plan.part + (slot * M + row0 + r) * DP;
                float2 *stat = plan.stat + slot * M + row0 + r;
                if constexpr (kPrefix) {
                    const size_t at = row_index(a, c, token, head);
                    if (starts && ends) dst = a.row_o + at * DP, stat = a.row_ml + at;
                    if (starts && l16 == 0) name_parts(a, at, ends ? 0 : parts_of(share, c), row0 + r);
                }
#pragma unroll
                for (int e = 0; e < C; e += 4) {
                    const int col = (e / 4) * 64 + l16 * 4;
                    if (!done || col < a.head_dim)
                        *reinterpret_cast<float4 *>(dst + col) =
                            done && none ? make_float4(0.f, 0.f, 0.f, 0.f)
                                         : make_float4(o[r][e] * inv, o[r][e + 1] * inv, o[r][e + 2] * inv, o[r][e + 3] * inv);
                }
                if (l16 == 0) {
                    if (!done)
                        *stat = make_float2(m[r], l[r]);
                    else if (a.lse)
                        a.lse[token * a.n_heads + head] = none ? -INFINITY : m[r] * 0.6931471805599453f + logf(l[r]);
                }
            }
            if (!kPrefix && tid == 0 && starts && !ends)
                plan.seg[blockIdx.x] = make_int4(c.b, c.row_tile, c.head, parts_of(share, c));
        }
        if (i + 1 < n_tiles) next_tile<kPrefix>(a, c, M);
    }
}

template <int DP, int M, bool kPrefix>
cudaError_t launch(const TreeArgs &a, const Plan &plan, cudaStream_t st) {
    static std::atomic<uint64_t> ready{0};
    auto kernel = tree_f32_kernel<DP, M, kPrefix>;
    if (!device_bit(ready)) {
        const cudaError_t e =
            cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, F32<DP, M>::kSmem);
        if (e != cudaSuccess) return e;
        set_device_bit(ready);
    }
    return launch_step(kernel, dim3(plan.ctas), dim3(kThreads), F32<DP, M>::kSmem, 1, st, a, plan);
}

template <int DP, int M>
cudaError_t launch_call(const TreeArgs &a, const Plan &plan, cudaStream_t st) {
    return a.row_o ? launch<DP, M, true>(a, plan, st) : launch<DP, M, false>(a, plan, st);
}

}  // namespace

cudaError_t launch_f32(const TreeArgs &a, const Plan &plan, int m_rows, cudaStream_t st) {
    if (a.head_dim <= 64) return m_rows == 16 ? launch_call<64, 16>(a, plan, st) : launch_call<64, 64>(a, plan, st);
    return m_rows == 16 ? launch_call<128, 16>(a, plan, st) : launch_call<128, 64>(a, plan, st);
}

}  // namespace tree
}  // namespace lora
