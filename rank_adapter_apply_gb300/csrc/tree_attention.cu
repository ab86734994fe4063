// lora_tree_attention: attention of drafted trees over a paged cache.
#include "base_linear.cuh"
#include "tree_common.cuh"

#include <algorithm>
#include <atomic>
#include <cmath>

namespace lora {
namespace {

using namespace step;
using namespace tree;

// ---- bf16, up to 32 rows a tile: mma.sync over the paged cache -------------------
// Four warps share a tile of 16 or 32 rows and 64 keys, by rows and by keys; K and V
// come by cp.async through the page table into a ring, a softmax with a running maximum
// and sum goes over the tiles, and O stays in registers. For long contexts it is bound by
// memory (16 requests of 7 nodes, ctx 8192, 32 heads over 8: 90 us, 4.7 TB/s); for few
// keys by the latency of two launches and a tile or two (1x8 ctx 777: 12.7 us).

constexpr int kStages = 3;

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
template <int DP, int WM, int WN>
struct Tile {
    static constexpr int M = 16 * WM, NK = kTileKeys / WN, kWarps = WM * WN, kThreads = 32 * kWarps;
    static constexpr int kRowBytes = DP * 2, kHalf = kTileKeys * kRowBytes, kStage = 2 * kHalf;
    // stages, then a ring of the tiles' key offsets and valid-key masks (one place more than stages: a tile's are
    // written while the tile one stage-count before it may still be read), then the search's scratch
    static constexpr int kRing = kStages + 1;
    static constexpr int kOff = kStages * kStage, kValid = kOff + kRing * kTileKeys * 8;
    static constexpr int kStart = kValid + kRing * 8, kSmem = kStart + (kScratch + kThreads / 32) * 8;
};

template <int DP, int WM, int WN>
__global__ void __launch_bounds__(128, 2) tree_tiles_kernel(TreeArgs a, Plan plan) {
    using T = Tile<DP, WM, WN>;
    constexpr int kPieces = DP / 8;                     // 16-byte pieces of a row
    extern __shared__ __align__(128) unsigned char smem[];
    long long *offs = reinterpret_cast<long long *>(smem + T::kOff);        // element offset of a key's row, -1: none
    uint32_t *valid = reinterpret_cast<uint32_t *>(smem + T::kValid);       // two words a tile
    long long *scratch = reinterpret_cast<long long *>(smem + T::kStart);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int wm = warp % WM, wn = warp / WM, g4 = lane >> 2, t4 = lane & 3;
    const int group = a.n_heads / a.n_kv;

    grid_dependency_wait();
    grid_launch_dependents();                            // the join kernel waits for this grid's end itself
    if (tid == 0) plan.seg[blockIdx.x] = make_int4(0, 0, 0, 0);
    Share share;
    if (!find_share<T::kThreads>(a, T::M, scratch, share)) return;
    Cursor load = share.start;
    Cursor c = load;                                     // the tile being computed; `load` runs ahead of it
    Cursor look = load;                                  // the tile whose page ids are being read: one further ahead
    const int n_tiles = (int)(share.hi - share.lo);

    // Offsets of tile i's keys: read into a register by threads 0..63, stored to the ring at the end of the step.
    auto read_off = [&](const Cursor &u) -> long long { return tid < kTileKeys ? key_offset(a, u, tid) : -1; };
    auto store_off = [&](int i, long long off) {
        if (tid >= kTileKeys) return;
        offs[i % T::kRing * kTileKeys + tid] = off;
        const uint32_t ok = __ballot_sync(0xffffffffu, off >= 0);
        if (lane == 0) valid[i % T::kRing * 2 + warp] = ok;
    };
    auto issue = [&](int i, const Cursor &u) {
        const uint32_t base = smem_u32(smem) + i % kStages * T::kStage;
        const int piece = tid % kPieces;
        const bool in_head = piece * 8 < a.head_dim;
        const long long at0 = u.head * a.c_head + piece * 8;
#pragma unroll
        for (int n = 0; n < kTileKeys * kPieces / T::kThreads; ++n) {
            const int k = tid / kPieces + n * (T::kThreads / kPieces);
            const long long off = offs[i % T::kRing * kTileKeys + k];
            const bool ok = off >= 0 && in_head;
            const long long at = ok ? off + at0 : 0;
            const uint32_t dst = base + k * T::kRowBytes + ((piece ^ (k & 7)) << 4);
            copy16(dst, static_cast<const __nv_bfloat16 *>(a.k_cache) + at, ok);
            copy16(dst + T::kHalf, static_cast<const __nv_bfloat16 *>(a.v_cache) + at, ok);
        }
    };

    // fill: offsets of the first tiles, then their copies; one commit group a tile
    long long pending = -1;
    for (int i = 0; i < kStages - 1; ++i) {
        if (i < n_tiles) {
            store_off(i, read_off(look));
            next_tile(a, look, T::M);
        }
    }
    __syncthreads();
    for (int i = 0; i < kStages - 1; ++i) {
        if (i < n_tiles) {
            issue(i, load);
            next_tile(a, load, T::M);
        }
        cp_async_commit();
    }
    if (kStages - 1 < n_tiles) store_off(kStages - 1, read_off(look));

    uint32_t q[DP / 16][4];
    float o[DP / 8][4], m[2], l[2];
    const float scale = a.scale == 0.f ? 1.f : fabsf(a.scale);
    const float c2 = scale * 1.4426950408889634f;        // scores in powers of two
    bool fresh = true;
    int seg_first = c.tile;
    const uint32_t lm_row = lane & 7, lm_hi = (lane >> 3) & 1, lm_top = lane >> 4;

    for (int i = 0; i < n_tiles; ++i) {
        if (fresh) {                                     // a new unit: its query rows, straight into fragments
            const __nv_bfloat16 *qp = static_cast<const __nv_bfloat16 *>(a.q);
#pragma unroll
            for (int hrow = 0; hrow < 2; ++hrow) {
                const int row = c.row_tile * T::M + wm * 16 + g4 + hrow * 8;
                const int node = row / group;
                const bool ok = node < c.r.nodes;
                const long long at = ok ? (c.r.start + node) * a.q_token + (c.head * group + row % group) * a.q_head : 0;
#pragma unroll
                for (int ks = 0; ks < DP / 16; ++ks)
#pragma unroll
                    for (int up = 0; up < 2; ++up) {
                        const int col = ks * 16 + up * 8 + t4 * 2;
                        uint32_t v = 0;
                        if (ok && col < a.head_dim) v = *reinterpret_cast<const uint32_t *>(qp + at + col);
                        if (a.scale < 0.f) v ^= 0x80008000u;
                        if (a.scale == 0.f) v = 0;
                        q[ks][up * 2 + hrow] = v;
                    }
            }
#pragma unroll
            for (int d = 0; d < DP / 8; ++d) o[d][0] = o[d][1] = o[d][2] = o[d][3] = 0.f;
            m[0] = m[1] = -INFINITY;
            l[0] = l[1] = 0.f;
            seg_first = c.tile;
            fresh = false;
        }
        asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
        __syncthreads();                                 // tile i is here, and everyone is done with tile i - 1
        if (i + kStages - 1 < n_tiles) {
            issue(i + kStages - 1, load);
            next_tile(a, load, T::M);
            next_tile(a, look, T::M);
        }
        cp_async_commit();
        if (i + kStages < n_tiles) pending = read_off(look);

        // ---- scores of this warp's rows and keys
        const uint32_t kb = smem_u32(smem) + i % kStages * T::kStage, vb = kb + T::kHalf;
        float s[T::NK / 8][4];
#pragma unroll
        for (int n = 0; n < T::NK / 8; ++n) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
#pragma unroll
        for (int ks = 0; ks < DP / 16; ++ks) {
#pragma unroll
            for (int n = 0; n < T::NK / 16; ++n) {
                uint32_t kf[4];
                const uint32_t key = wn * T::NK + n * 16 + lm_top * 8 + lm_row;
                ldsm4(kf, kb + key * T::kRowBytes + (((ks * 2 + lm_hi) ^ (key & 7)) << 4));
                mma_bf16(s[2 * n], q[ks][0], q[ks][1], q[ks][2], q[ks][3], kf[0], kf[1]);
                mma_bf16(s[2 * n + 1], q[ks][0], q[ks][1], q[ks][2], q[ks][3], kf[2], kf[3]);
            }
        }
        // ---- keys a row does not see
        const int p0 = c.tile * kTileKeys;
        const uint64_t there = valid[i % T::kRing * 2] | (uint64_t)valid[i % T::kRing * 2 + 1] << 32;
        bool hidden = false;                             // a key that is there but that one of this thread's rows skips
        const bool masked = there != ~0ull || p0 + kTileKeys > c.r.ctx;
        if (masked) {
#pragma unroll
            for (int hrow = 0; hrow < 2; ++hrow) {
                const int node = (c.row_tile * T::M + wm * 16 + g4 + hrow * 8) / group;
                uint64_t seen = 0;
                if (node < c.r.nodes) {
                    seen = seen_keys(a, c.r, node, p0) & there;
                    hidden = hidden || seen != there;
                }
                seen >>= wn * T::NK;
#pragma unroll
                for (int n = 0; n < T::NK / 8; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        if (!(seen >> (n * 8 + t4 * 2 + e) & 1)) s[n][hrow * 2 + e] = -INFINITY;
            }
        }
        // ---- running maximum and sum
        float top[2] = {m[0], m[1]};
#pragma unroll
        for (int n = 0; n < T::NK / 8; ++n) {
            top[0] = fmaxf(top[0], fmaxf(s[n][0], s[n][1]));
            top[1] = fmaxf(top[1], fmaxf(s[n][2], s[n][3]));
        }
#pragma unroll
        for (int hrow = 0; hrow < 2; ++hrow) {
            top[hrow] = fmaxf(top[hrow], __shfl_xor_sync(0xffffffffu, top[hrow], 1));
            top[hrow] = fmaxf(top[hrow], __shfl_xor_sync(0xffffffffu, top[hrow], 2));
        }
        const bool moved = top[0] != m[0] || top[1] != m[1];
        const float base0 = top[0] == -INFINITY ? 0.f : top[0] * c2, base1 = top[1] == -INFINITY ? 0.f : top[1] * c2;
        if (__any_sync(0xffffffffu, moved)) {
            const float k0 = exp2_fast(fmaf(m[0], c2, -base0)), k1 = exp2_fast(fmaf(m[1], c2, -base1));
            l[0] *= k0;
            l[1] *= k1;
#pragma unroll
            for (int d = 0; d < DP / 8; ++d) {
                o[d][0] *= k0;
                o[d][1] *= k0;
                o[d][2] *= k1;
                o[d][3] *= k1;
            }
            m[0] = top[0];
            m[1] = top[1];
        }
        uint32_t pf[T::NK / 8][2];
#pragma unroll
        for (int n = 0; n < T::NK / 8; ++n) {
            const float e0 = exp2_fast(fmaf(s[n][0], c2, -base0)), e1 = exp2_fast(fmaf(s[n][1], c2, -base0));
            const float e2 = exp2_fast(fmaf(s[n][2], c2, -base1)), e3 = exp2_fast(fmaf(s[n][3], c2, -base1));
            l[0] += e0 + e1;
            l[1] += e2 + e3;
            // weights to bf16 for the second product: 2^-9 relative, below the output's own rounding; their sum
            // l stays in fp32 and unrounded
            pf[n][0] = pack_bf16(e0, e1);
            pf[n][1] = pack_bf16(e2, e3);
        }
        // A weight of zero times an infinity or NaN is NaN: where a row skips a key that is there (the whole block
        // decides alike, in tiles of tree keys only), values that are not finite are looked for, and such a tile
        // is summed key by key without the zero weights.
        bool by_key = false;
        if (masked && __syncthreads_or(hidden)) {
            uint32_t odd = 0;
            for (int n = tid; n < T::kHalf / 16; n += T::kThreads) {
                const uint4 v = *reinterpret_cast<const uint4 *>(smem + i % kStages * T::kStage + T::kHalf + n * 16);
                odd |= ((v.x & 0x7f807f80u) + 0x00800080u) | ((v.y & 0x7f807f80u) + 0x00800080u) |
                       ((v.z & 0x7f807f80u) + 0x00800080u) | ((v.w & 0x7f807f80u) + 0x00800080u);
            }
            by_key = __syncthreads_or((odd & 0x80008000u) != 0);
        }
        if (by_key) {
            // the weights go where the keys lay (every warp has its scores by now): [M][64] bf16
            uint32_t *w = reinterpret_cast<uint32_t *>(smem + i % kStages * T::kStage);
#pragma unroll
            for (int n = 0; n < T::NK / 8; ++n)
#pragma unroll
                for (int hrow = 0; hrow < 2; ++hrow)
                    w[(wm * 16 + g4 + hrow * 8) * 32 + (wn * T::NK + n * 8) / 2 + t4] = pf[n][hrow];
            __syncwarp();
            for (int k = wn * T::NK; k < (wn + 1) * T::NK; ++k) {
                const __nv_bfloat16 *wb = reinterpret_cast<const __nv_bfloat16 *>(w);
                const float w0 = to_f32(wb[(wm * 16 + g4) * 64 + k]), w1 = to_f32(wb[(wm * 16 + g4 + 8) * 64 + k]);
                const unsigned char *vr = smem + i % kStages * T::kStage + T::kHalf + k * T::kRowBytes + t4 * 4;
#pragma unroll
                for (int d = 0; d < DP / 8; ++d) {
                    const uint32_t v = *reinterpret_cast<const uint32_t *>(vr + ((d ^ (k & 7)) << 4));
                    if (w0 != 0.f) o[d][0] = fmaf(w0, bf_lo(v), o[d][0]), o[d][1] = fmaf(w0, bf_hi(v), o[d][1]);
                    if (w1 != 0.f) o[d][2] = fmaf(w1, bf_lo(v), o[d][2]), o[d][3] = fmaf(w1, bf_hi(v), o[d][3]);
                }
            }
        } else {
#pragma unroll
            for (int n = 0; n < T::NK / 16; ++n) {
#pragma unroll
                for (int d = 0; d < DP / 16; ++d) {
                    uint32_t vf[4];
                    const uint32_t key = wn * T::NK + n * 16 + lm_hi * 8 + lm_row;
                    ldsm4_t(vf, vb + key * T::kRowBytes + (((d * 2 + lm_top) ^ (key & 7)) << 4));
                    mma_bf16(o[2 * d], pf[2 * n][0], pf[2 * n][1], pf[2 * n + 1][0], pf[2 * n + 1][1], vf[0], vf[1]);
                    mma_bf16(o[2 * d + 1], pf[2 * n][0], pf[2 * n][1], pf[2 * n + 1][0], pf[2 * n + 1][1], vf[2], vf[3]);
                }
            }
        }
        // ---- the unit or the share ends: join the warps and write
        if (c.tile + 1 == c.r.key_tiles || i + 1 == n_tiles) {
#pragma unroll
            for (int hrow = 0; hrow < 2; ++hrow) {
                l[hrow] += __shfl_xor_sync(0xffffffffu, l[hrow], 1);
                l[hrow] += __shfl_xor_sync(0xffffffffu, l[hrow], 2);
                m[hrow] = m[hrow] == -INFINITY ? -INFINITY : m[hrow] * c2;
            }
            if constexpr (WN > 1) {
                // the warps that share rows, through the stage just consumed (the next copies into it are issued
                // after the next step's barrier)
                float *buf = reinterpret_cast<float *>(smem + i % kStages * T::kStage);   // [WN - 1][M][DP + 2]
                __syncthreads();
                if (wn > 0) {
#pragma unroll
                    for (int hrow = 0; hrow < 2; ++hrow) {
                        float *r = buf + ((size_t)(wn - 1) * T::M + wm * 16 + g4 + hrow * 8) * (DP + 2);
#pragma unroll
                        for (int d = 0; d < DP / 8; ++d)
                            *reinterpret_cast<float2 *>(r + d * 8 + t4 * 2) =
                                make_float2(o[d][hrow * 2], o[d][hrow * 2 + 1]);
                        if (t4 == 0) *reinterpret_cast<float2 *>(r + DP) = make_float2(m[hrow], l[hrow]);
                    }
                }
                __syncthreads();
                if (wn == 0) {
#pragma unroll
                    for (int w = 1; w < WN; ++w)
#pragma unroll
                        for (int hrow = 0; hrow < 2; ++hrow) {
                            const float *r = buf + ((size_t)(w - 1) * T::M + wm * 16 + g4 + hrow * 8) * (DP + 2);
                            const float2 ml = *reinterpret_cast<const float2 *>(r + DP);
                            const float t = fmaxf(m[hrow], ml.x), b = t == -INFINITY ? 0.f : t;
                            const float f = exp2_fast(m[hrow] - b), h = exp2_fast(ml.x - b);
                            m[hrow] = t;
                            l[hrow] = l[hrow] * f + ml.y * h;
#pragma unroll
                            for (int d = 0; d < DP / 8; ++d) {
                                const float2 v = *reinterpret_cast<const float2 *>(r + d * 8 + t4 * 2);
                                o[d][hrow * 2] = o[d][hrow * 2] * f + v.x * h;
                                o[d][hrow * 2 + 1] = o[d][hrow * 2 + 1] * f + v.y * h;
                            }
                        }
                }
            }
            const bool starts = seg_first == 0, ends = c.tile + 1 == c.r.key_tiles;
            if (wn == 0) {
#pragma unroll
                for (int hrow = 0; hrow < 2; ++hrow) {
                    const int r = wm * 16 + g4 + hrow * 8;
                    const int row = c.row_tile * T::M + r, node = row / group;
                    if (node >= c.r.nodes) continue;
                    if (starts && ends) {
                        const long long token = c.r.start + node;
                        const int head = c.head * group + row % group;
                        const float inv = l[hrow] > 0.f ? 1.f / l[hrow] : l[hrow];
                        __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(a.out) + token * a.o_token + head * a.o_head;
                        // a row without keys is 0; one whose scores are all NaN also has m = -inf (fmaxf drops them),
                        // but its l is NaN
                        const bool none = l[hrow] == 0.f;
#pragma unroll
                        for (int d = 0; d < DP / 8; ++d)
                            if (d * 8 < a.head_dim)
                                *reinterpret_cast<uint32_t *>(out + d * 8 + t4 * 2) =
                                    none ? 0u : pack_bf16(o[d][hrow * 2] * inv, o[d][hrow * 2 + 1] * inv);
                        if (a.lse && t4 == 0)
                            a.lse[token * a.n_heads + head] =
                                none ? -INFINITY : m[hrow] * 0.6931471805599453f + logf(l[hrow]);
                    } else {
                        const long long slot = 2ll * blockIdx.x + (starts ? 1 : 0);
                        float *part = plan.part + (slot * T::M + r) * DP;
#pragma unroll
                        for (int d = 0; d < DP / 8; ++d)
                            *reinterpret_cast<float2 *>(part + d * 8 + t4 * 2) =
                                make_float2(o[d][hrow * 2], o[d][hrow * 2 + 1]);
                        if (t4 == 0) plan.stat[slot * T::M + r] = make_float2(m[hrow], l[hrow]);
                    }
                }
            }
            if (tid == 0 && starts && !ends) {
                plan.seg[blockIdx.x] = make_int4(c.b, c.row_tile, c.head, parts_of(share, c, i));
            }
            fresh = true;
        }
        if (i + kStages < n_tiles) store_off(i + kStages, pending);
        next_tile(a, c, T::M);
    }
}

// Join the parts of the unit that goes on past CTA blockIdx.x's share. A warp takes
// kR rows, with kAhead parts of each in flight; with kR = 1, for few units cut into
// many parts, above 24 parts the warps of a block share the parts of its eight rows
// instead. It is latency: a launch, one read of the segment and one or more rounds
// of reads, 4 of the 12.6 us of 1x8 ctx 777 (2 / 4 / 8 / 16 parts ahead: 13.8 /
// 13.0 / 12.6 / 13.8). (One row to a warp and four: 1x8 ctx 777 12.7 and 16.0 us,
// 32x16 ctx 4096 89.4 and 89.0. 38 parts, 1x6 ctx 3000: 24.5 us row after row, 17.6
// so.)
template <int DP>
struct Joined {
    static constexpr int V = DP / 32;                    // columns of a lane
    float o[V], m = -INFINITY, l = 0.f;
    __device__ __forceinline__ void add(float2 ml, const float (&v)[V]) {
        const float t = fmaxf(m, ml.x), b = t == -INFINITY ? 0.f : t;
        const float f = exp2_fast(m - b), h = exp2_fast(ml.x - b);
        m = t;
        l = l * f + ml.y * h;
#pragma unroll
        for (int e = 0; e < V; ++e) o[e] = o[e] * f + v[e] * h;
    }
};

template <typename T, int DP>
__device__ __forceinline__ void store_joined(const TreeArgs &a, const int4 &seg, int start, int row, const Joined<DP> &j) {
    constexpr int V = Joined<DP>::V;
    const int lane = threadIdx.x & 31, group = a.n_heads / a.n_kv, head = seg.z * group + row % group;
    const long long token = start + row / group;
    const bool none = j.l == 0.f;                        // m is -inf for a row of NaN scores, too
    const float inv = j.l > 0.f ? 1.f / j.l : j.l;       // a NaN stays one
    T *out = static_cast<T *>(a.out) + token * a.o_token + (long long)head * a.o_head + lane * V;
    if (lane * V < a.head_dim) {
#pragma unroll
        for (int e = 0; e < V; e += 2) {
            const float x = none ? 0.f : j.o[e] * inv, y = none ? 0.f : j.o[e + 1] * inv;
            if constexpr (sizeof(T) == 2)
                *reinterpret_cast<uint32_t *>(out + e) = pack_bf16(x, y);
            else
                *reinterpret_cast<float2 *>(out + e) = make_float2(x, y);
        }
    }
    if (a.lse && lane == 0) a.lse[token * a.n_heads + head] = none ? -INFINITY : j.m * 0.6931471805599453f + logf(j.l);
}

template <typename T, int DP, int M, int kR>
__global__ void __launch_bounds__(256) tree_join_kernel(TreeArgs a, Plan plan, int m_rows) {
    constexpr int V = Joined<DP>::V, kAhead = kR == 1 ? 8 : 2, kMany = 24, kShared = kR == 1 ? 8 : 1;
    __shared__ float so[kShared][kShared][DP];               // of a warp's parts, of a row
    __shared__ float2 sm[kShared][kShared];
    grid_dependency_wait();
    grid_launch_dependents();
    const int4 seg = plan.seg[blockIdx.x];
    if (seg.w == 0) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, group = a.n_heads / a.n_kv;
    const int start = node_start(a, seg.x);
    const int rows = min((node_start(a, seg.x + 1) - start) * group - seg.y * m_rows, m_rows);
    auto read = [&](int part, int r, float2 &ml, float (&v)[V]) {
        const long long slot = part == 0 ? 2ll * blockIdx.x + 1 : 2ll * (blockIdx.x + part);
        ml = plan.stat[slot * M + r];
        const float *src = plan.part + (slot * M + r) * DP + lane * V;
        if constexpr (V == 4) {
            *reinterpret_cast<float4 *>(v) = *reinterpret_cast<const float4 *>(src);
        } else {
            *reinterpret_cast<float2 *>(v) = *reinterpret_cast<const float2 *>(src);
        }
    };
    if constexpr (kR == 1) {
        if (seg.w > kMany) {                                 // a warp adds every eighth part of the block's eight rows
            const int r0 = blockIdx.y * 8;
            if (r0 >= rows) return;
            Joined<DP> j[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
#pragma unroll
                for (int e = 0; e < V; ++e) j[i].o[e] = 0.f;
            for (int p = warp; p < seg.w; p += 8) {
                alignas(4 * V) float v[8][V];
                float2 ml[8];
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (r0 + i < rows) read(p, r0 + i, ml[i], v[i]);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (r0 + i < rows) j[i].add(ml[i], v[i]);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
#pragma unroll
                for (int e = 0; e < V; ++e) so[warp][i][lane * V + e] = j[i].o[e];
                if (lane == 0) sm[warp][i] = make_float2(j[i].m, j[i].l);
            }
            __syncthreads();
            if (r0 + warp >= rows) return;
            Joined<DP> all;
#pragma unroll
            for (int e = 0; e < V; ++e) all.o[e] = 0.f;
            for (int w = 0; w < 8; ++w) {
                float v[V];
#pragma unroll
                for (int e = 0; e < V; ++e) v[e] = so[w][warp][lane * V + e];
                all.add(sm[w][warp], v);
            }
            store_joined<T, DP>(a, seg, start, seg.y * m_rows + r0 + warp, all);
            return;
        }
    }
    const int r0 = (blockIdx.y * 8 + warp) * kR;
    if (r0 >= rows) return;
    Joined<DP> j[kR];
#pragma unroll
    for (int k = 0; k < kR; ++k)
#pragma unroll
        for (int e = 0; e < V; ++e) j[k].o[e] = 0.f;
    for (int p = 0; p < seg.w; p += kAhead) {
        alignas(4 * V) float v[kAhead][kR][V];
        float2 ml[kAhead][kR];
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
#pragma unroll
            for (int k = 0; k < kR; ++k)
                if (p + u < seg.w && r0 + k < rows) read(p + u, r0 + k, ml[u][k], v[u][k]);
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
#pragma unroll
            for (int k = 0; k < kR; ++k)
                if (p + u < seg.w && r0 + k < rows) j[k].add(ml[u][k], v[u][k]);
    }
#pragma unroll
    for (int k = 0; k < kR; ++k)
        if (r0 + k < rows) store_joined<T, DP>(a, seg, start, seg.y * m_rows + r0 + k, j[k]);
}

constexpr int kMaxRows = 128;
constexpr int kMaxCtas = 2 * 160;

// The row tile by the average rows (nodes times query heads of a key/value head) of a request: how they are spread over
// the requests only the device knows, so one wide tree among many single nodes goes in many small tiles (64 requests, ctx
// 4096, 32 heads over 8: all of one node 176 us, one of them of 64 nodes 234). Measured with equal requests: 8, ctx 4096,
// 32 heads over 8, tiles of 16 / 32 / 128 rows: 8 rows 34.6 / 35.4 / 35.6 us, 16 rows 36.0 / 36.3 / 35.5, 24 rows 45.1 /
// 38.0 / 36.8, 32 rows 45.5 / 38.2 / 37.4, 48 rows 58.9 / 50.9 / 38.9, 128 rows 119 / 80 / 47. For few keys 32 beats 128
// up to 32 rows: 1x8 ctx 777 12.7 and 14.8, 4x8 ctx 500 13.6 and 17.7.
int rows_of_tile(const TreeArgs &a) {
    const double rows = (double)a.n_tokens * (a.n_heads / a.n_kv) / a.n_requests;
    return rows <= 16.0 ? 16 : rows <= 32.0 || !tc_takes(a) ? 32 : 128;
}

size_t plan_bytes(int ctas) {
    return (size_t)ctas * sizeof(int4) + 2 * (size_t)ctas * kMaxRows * (128 * sizeof(float) + sizeof(float2));
}

template <int DP, int WM>
cudaError_t launch_tiles(const TreeArgs &a, const Plan &plan, cudaStream_t st) {
    using T = Tile<DP, WM, 4 / WM>;
    auto kernel = tree_tiles_kernel<DP, WM, 4 / WM>;
    static std::atomic<uint64_t> ready{0};
    if (!device_bit(ready)) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, T::kSmem);
        if (e != cudaSuccess) return e;
        set_device_bit(ready);
    }
    return launch_step(kernel, dim3(plan.ctas), dim3(T::kThreads), T::kSmem, 1, st, a, plan);
}

template <typename T, int DP, int M>
cudaError_t launch_join(const TreeArgs &a, const Plan &plan, int m_rows, cudaStream_t st) {
    // few units: each is cut into many parts, and the rows need the blocks
    const double units = (double)a.n_requests * a.n_kv *
                         std::max(1.0, (double)a.n_tokens * (a.n_heads / a.n_kv) / a.n_requests / m_rows);
    if (units * 8 < plan.ctas)
        return launch_step(tree_join_kernel<T, DP, M, 1>, dim3(plan.ctas, M / 8), dim3(256), 0, 1, st, a, plan, m_rows);
    constexpr int kR = M >= 32 ? 4 : 2;
    return launch_step(tree_join_kernel<T, DP, M, kR>, dim3(plan.ctas, M / 8 / kR), dim3(256), 0, 1, st, a, plan, m_rows);
}

template <int DP>
cudaError_t launch_bf16(const TreeArgs &a, const Plan &plan, cudaStream_t st) {
    const int rows = rows_of_tile(a);
    cudaError_t e = cudaErrorNotSupported;
    if (rows == 128) {
        e = launch_tc(a, plan, st);
        if (e == cudaSuccess) return launch_join<__nv_bfloat16, DP, 128>(a, plan, tc_rows(a), st);
    }
    if (rows == 16) {
        e = launch_tiles<DP, 1>(a, plan, st);
        return e != cudaSuccess ? e : launch_join<__nv_bfloat16, DP, 16>(a, plan, 16, st);
    }
    if (e != cudaErrorNotSupported) return e;
    e = launch_tiles<DP, 2>(a, plan, st);
    return e != cudaSuccess ? e : launch_join<__nv_bfloat16, DP, 32>(a, plan, 32, st);
}

template <int DP>
cudaError_t launch_fp32(const TreeArgs &a, const Plan &plan, cudaStream_t st) {
    // rows beyond a request's cost their FMAs all the same: 8 requests, ctx 4096, tiles of 16 / 64 rows: 16 rows 117 / 182
    // us, 24 rows 211 / 183
    const int rows = (double)a.n_tokens * (a.n_heads / a.n_kv) / a.n_requests <= 16.0 ? 16 : 64;
    const cudaError_t e = launch_f32(a, plan, rows, st);
    if (e != cudaSuccess) return e;
    return rows == 16 ? launch_join<float, DP, 16>(a, plan, 16, st) : launch_join<float, DP, 64>(a, plan, 64, st);
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
    // the largest grid of any GPU this library is built for: the size does not depend on the device
    return plan_bytes(kMaxCtas);
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
    if ((long long)d->n_tokens * d->n_heads > (1 << 30))
        return fail(LORA_ERR_ARG, "tree_attention: n_tokens %d times n_heads %d is above 2^30", d->n_tokens,
                    d->n_heads);
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
    for (long long s : strides) ok = ok && s >= 0 && s * eb % 16 == 0;
    if (!ok)
        return fail(LORA_ERR_ARG, "tree_attention: q, out and cache pointers and strides must be multiples of 16 bytes, "
                                  "no stride negative");
    if (!rows_apart(d->n_tokens, d->out_token, d->n_heads, d->out_head, d->head_dim))
        return fail(LORA_ERR_ARG, "tree_attention: the rows of out overlap (strides %lld, %lld)", (long long)d->out_token,
                    (long long)d->out_head);
    const size_t need = lora_tree_attention_workspace_bytes(d->n_requests, d->n_tokens, d->n_heads, d->n_kv_heads,
                                                            d->head_dim, d->dtype);
    if (!d->workspace || d->workspace_bytes < need || reinterpret_cast<uintptr_t>(d->workspace) % 256)
        return fail(LORA_ERR_ARG, "tree_attention: workspace of %zu bytes, 256-byte aligned, is needed", need);
    TreeArgs a{d->q,       d->k_cache,   d->v_cache,   d->out,       d->lse,       d->page_table, d->ctx_lens,
               d->node_starts, d->tree_mask, d->q_token, d->q_head,  d->cache_page, d->cache_slot, d->cache_head,
               d->out_token, d->out_head, d->table_stride, d->n_pages, d->scale,   d->page_size,  d->table_pages,
               d->mask_words, d->n_requests, d->n_tokens, d->n_heads, d->n_kv_heads, d->head_dim};
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int sms = sm_count();
    if (sms < 1) return fail(LORA_ERR_CUDA, "tree_attention: no CUDA device");
    Plan plan;
    plan.ctas = std::min(std::max(2 * sms, 64), kMaxCtas);          // 64: a group of every class fits
    plan.part = static_cast<float *>(d->workspace);
    plan.stat = reinterpret_cast<float2 *>(plan.part + 2 * (size_t)plan.ctas * kMaxRows * 128);
    plan.seg = reinterpret_cast<int4 *>(plan.stat + 2 * (size_t)plan.ctas * kMaxRows);
    cudaError_t e;
    if (d->dtype == LORA_DTYPE_BF16)
        e = d->head_dim <= 64 ? launch_bf16<64>(a, plan, st) : launch_bf16<128>(a, plan, st);
    else
        e = d->head_dim <= 64 ? launch_fp32<64>(a, plan, st) : launch_fp32<128>(a, plan, st);
    return launched("tree_attention", e);
}

extern "C" int lora_step_wait_timeouts(uint64_t *count) {
    if (!count) return fail(LORA_ERR_ARG, "step_wait_timeouts: NULL pointer argument");
    unsigned n = 0, of_linear = 0;
    // the copies below wait for the default stream and those that it waits for, not for non-blocking streams
    cudaError_t e = cudaDeviceSynchronize();
    if (e == cudaSuccess) e = read_timeouts(&n);
    if (e == cudaSuccess) e = linear::read_timeouts(&of_linear);
    if (e != cudaSuccess) return launched("step_wait_timeouts", e);
    *count = (uint64_t)n + of_linear;
    return LORA_OK;
}
