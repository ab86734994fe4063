// Device code of lora_prefix_attention in bf16 for up to 16 rows of an entry
// (prefix_rows.cu) and beside the 5th-generation tensor cores (tree_attention_tc.cu):
// A warp works alone: row tiles of 16 on mma.sync, 16 keys a step, K and V by cp.async
// through the page table into a ring of its own, O in registers, no barrier but the warp's.
// The steps of all units (entry, head, row tile), in a row, with a few more for each unit's
// beginning and end, are dealt to the warps in equal shares, so that ragged lengths and
// many short units cost each warp alike. (Tiles of 64 keys shared by a block's four warps and dealt
// without the units' own cost: 64 requests with contexts of up to 1000 take 64 us, the same
// number of keys in contexts of 500 41.)
#pragma once

#include "tree_common.cuh"

#include <climits>

namespace lora {
namespace tree {
namespace rows {

constexpr int kRows = 16, kKeys = 16;
// A step is computed while the next is on its way. Shared memory that the rings leave is the cache that the copies pass
// through: with three stages, and 28 KB of it, 200 requests with contexts of up to 1000 take 102 us, with two 87.
constexpr int kStages = 2;
constexpr int kUnitCost = 2;                   // steps that a unit's beginning and end are worth
// Steps of a warp's share, at least: the join reads a part for each. us with 2 / 3 / 4: 3x1 of 777 12.2 / 12.6 / 13.1, 8x1 of
// 2000 17.1 / 15.9 / 15.6, 12x1 of 16384 33.8 / 34.9 / 36.3
constexpr int kLeast = 3;

// What a step's computation has to know of it.
struct Step {
    int start, nodes, ctx, keys;
    int row_tile, head, step, there;           // there: the keys that are there
    int last, starts, ends, parts;             // last: of the warp's part of its unit, which has the unit's first or last step
    int group;                                 // whether the entry is a group
};

// Shared memory: the warps' rings, then what the shares are found with and the steps in the rings.
template <int DP, int kWarps, int kThreads>
struct Memory {
    static constexpr int kRowBytes = DP * 2, kHalf = kKeys * kRowBytes, kStage = 2 * kHalf;
    unsigned char rings[kWarps][kStages * kStage];
    Step steps[kWarps][kStages + 1];
    long long sums[kThreads / 32], first_of[kWarps];
    int entry_of[kWarps];
    Request entries[kThreads];                         // where there are no more
};

// Where a warp is in the units' steps.
struct Place {
    Request r;
    long long col, hi;
    int b, head, row_tile, step, steps;
};

__device__ __forceinline__ int steps_of(const Request &r) { return max((r.keys + kKeys - 1) / kKeys, 1); }
__device__ __forceinline__ long long cost_of(const TreeArgs &a, const Request &r) {
    return (long long)r.row_tiles * a.n_kv * (steps_of(r) + kUnitCost);
}

// The first unit after the one at p, at its first step. known: the entries, or nullptr.
__device__ __noinline__ inline void next_place(const TreeArgs &a, const Request *known, Place &p) {
    p.step = 0;
    if (++p.row_tile < p.r.row_tiles) return;
    p.row_tile = 0;
    if (++p.head < a.n_kv) return;
    p.head = 0;
    do {
        if (++p.b >= a.count) {
            p.col = p.hi;
            return;
        }
        p.r = known ? known[p.b] : request<true>(a, p.b, kRows);
    } while (p.r.row_tiles == 0);
    p.steps = steps_of(p.r);
}

// Whether there is a step after this one.
__device__ __forceinline__ bool advance(const TreeArgs &a, const Request *known, Place &p) {
    ++p.col;
    if (++p.step == p.steps) {
        p.col += kUnitCost;
        if (p.col < p.hi) next_place(a, known, p);
    }
    return p.col < p.hi;
}

// A CTA's work. kWarps of its kThreads / 32 warps have shares; all threads call it.
template <int DP, int kWarps, int kThreads>
__device__ __forceinline__ void work(const TreeArgs &a, const Plan &plan, unsigned char *smem) {
    using R = Memory<DP, kWarps, kThreads>;
    constexpr int kPieces = DP / 8;                    // 16-byte pieces of a row
    R &sm = *reinterpret_cast<R *>(smem);
    auto &steps = sm.steps;
    auto &sums = sm.sums;
    auto &first_of = sm.first_of;
    auto &entry_of = sm.entry_of;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g4 = lane >> 2, t4 = lane & 3;
    const int group = a.n_heads / a.n_kv;

    // ---- the warps' shares: neighbours in different blocks
    auto scanned = [&](long long n) {                  // up to this thread, of the block
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long v = __shfl_up_sync(0xffffffffu, n, o);
            if (lane >= o) n += v;
        }
        __syncthreads();
        if (lane == 31) sums[warp] = n;
        __syncthreads();
        for (int w = 0; w < warp; ++w) n += sums[w];
        return n;
    };
    long long total = 0, mine = 0, upto = 0;
    const Request *const known = a.count <= kThreads ? sm.entries : nullptr;
    for (int b0 = 0; b0 < a.count; b0 += kThreads) {
        const int b = b0 + tid;
        mine = 0;
        if (b < a.count) {
            const Request r = request<true>(a, b, kRows);
            sm.entries[tid] = r;
            mine = cost_of(a, r);
        }
        upto = scanned(mine);
        __syncthreads();
        if (tid == kThreads - 1) sums[0] = upto;
        __syncthreads();
        total += sums[0];
    }
    const int worker = warp < kWarps ? warp * (int)gridDim.x + (int)blockIdx.x : INT_MAX;
    const long long workers = min((long long)plan.ctas, (total + kLeast - 1) / kLeast);
    const long long lo = worker < workers ? scaled(total, worker, workers) : total;
    const long long hi = worker < workers ? scaled(total, worker + 1, workers) : total;
    if (lane == 0 && warp < kWarps) first_of[warp] = lo, entry_of[warp] = -1;
    __syncthreads();
    // the entry of each warp's first step
    long long before = 0;
    for (int b0 = 0; b0 < a.count; b0 += kThreads) {
        const int b = b0 + tid;
        if (a.count > kThreads) {
            mine = b < a.count ? cost_of(a, request<true>(a, b, kRows)) : 0;
            upto = scanned(mine);
        }
        for (int w = 0; w < kWarps; ++w) {
            const long long x = first_of[w] - before;
            if (entry_of[w] < 0 && upto - mine <= x && x < upto) entry_of[w] = b;
        }
        __syncthreads();
        for (int w = 0; w < kWarps; ++w)
            if (entry_of[w] == b && first_of[w] >= 0) first_of[w] -= before + upto - mine, first_of[w] = ~first_of[w];
        __syncthreads();
        if (tid == kThreads - 1) sums[0] = upto;
        __syncthreads();
        before += sums[0];
    }
    if (lo >= hi) return;
    Place load;
    load.b = entry_of[warp];
    load.r = known ? known[load.b] : request<true>(a, load.b, kRows);
    load.steps = steps_of(load.r);
    load.hi = hi;
    load.col = lo;
    {
        const long long at = ~first_of[warp], unit = scaled(at, 1, load.steps + kUnitCost);
        load.head = (int)scaled(unit, 1, load.r.row_tiles);
        load.row_tile = (int)(unit - (long long)load.head * load.r.row_tiles);
        load.step = (int)(at - unit * (load.steps + kUnitCost));
        if (load.step >= load.steps) {                 // in a unit's end
            load.col += load.steps + kUnitCost - load.step;
            if (load.col >= hi) return;
            next_place(a, known, load);
            if (load.col >= hi) return;
        }
    }
    int from = load.step;                              // the first step of the warp's part of the unit at `load`
    auto worker_of = [&](long long x) { return (int)scaled((x + 1) * workers - 1, 1, total); };

    unsigned char *ring = sm.rings[warp];
    const uint32_t ring_at = smem_u32(ring);
    // lane k < 16: element offset of the step's key k, -1: nobody sees it
    auto look = [&](const Place &p) -> long long {
        const int key = p.step * kKeys + lane;
        if (lane >= kKeys || key >= p.r.keys) return -1;
        const int at = key / a.page_size, id = table_row<true>(a, p.b)[at];
        return id >= 0 && id < a.n_pages ? id * a.c_page + (key - at * a.page_size) * a.c_slot : -1;
    };
    bool more = true;
    auto issue = [&](int i, long long off) {           // step i, which `load` is at, and to the next
        const uint32_t to = ring_at + i % kStages * R::kStage;
        const int piece = lane % kPieces;
        const bool in_head = piece * 8 < a.head_dim;
        const long long at0 = load.head * a.c_head + piece * 8;
#pragma unroll
        for (int n = 0; n < kKeys * kPieces / 32; ++n) {
            const int k = lane / kPieces + n * (32 / kPieces);
            const long long o = __shfl_sync(0xffffffffu, off, k);
            const bool ok = o >= 0 && in_head;
            const long long at = ok ? o + at0 : 0;
            const uint32_t dst = to + k * R::kRowBytes + ((piece ^ (k & 7)) << 4);
            copy16(dst, static_cast<const __nv_bfloat16 *>(a.k_cache) + at, ok);
            copy16(dst + R::kHalf, static_cast<const __nv_bfloat16 *>(a.v_cache) + at, ok);
        }
        const int there = (int)__ballot_sync(0xffffffffu, off >= 0);
        Step s{load.r.start, load.r.nodes, load.r.ctx, load.r.keys, load.row_tile, load.head, load.step, there,
               0, from == 0, 0, 0, is_group<true>(a, load.b)};
        s.ends = load.step + 1 == load.steps;
        s.last = s.ends || load.col + 1 >= load.hi;
        if (s.last && s.starts && !s.ends) s.parts = worker_of(load.col - load.step + load.steps - 1) - worker + 1;
        if (lane == 0) steps[warp][i % (kStages + 1)] = s;
        more = advance(a, known, load);
        if (s.last) from = load.step;
    };
    long long off = look(load);
    int loaded = 0;                                    // steps that are there or on their way
    for (int i = 0; i < kStages - 1; ++i) {
        if (more) {
            issue(loaded++, off);
            if (more) off = look(load);
        }
        cp_async_commit();
    }
    uint32_t q[DP / 16][4];
    float o[DP / 8][4], m[2], l[2];
    const float scale = a.scale == 0.f ? 1.f : fabsf(a.scale);
    const float c2 = scale * 1.4426950408889634f;      // scores in powers of two
    bool fresh = true, over = false;
    const uint32_t lm_row = lane & 7, lm_hi = (lane >> 3) & 1, lm_top = lane >> 4;
    for (int i = 0; !over; ++i) {
        __syncwarp();                                  // the warp is done with the step before
        over = !more && i + 1 == loaded;               // with more to come, loaded is i + kStages - 1
        if (more) {
            issue(loaded++, off);
            if (more) off = look(load);
        }
        cp_async_commit();
        const Step c = steps[warp][i % (kStages + 1)];
        if (fresh) {                                   // a unit's first step here: its query rows, straight into fragments
            const __nv_bfloat16 *qp = static_cast<const __nv_bfloat16 *>(a.q);
#pragma unroll
            for (int hrow = 0; hrow < 2; ++hrow) {
                const int row = c.row_tile * kRows + g4 + hrow * 8, node = row / group;
                const bool ok = node < c.nodes;
                const long long at = ok ? (c.start + node) * a.q_token + (c.head * group + row % group) * a.q_head : 0;
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
            fresh = false;
        }
        asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
        __syncwarp();                                  // step i is here
        // ---- scores
        const uint32_t kb = ring_at + i % kStages * R::kStage, vb = kb + R::kHalf;
        float s[2][4] = {};
#pragma unroll
        for (int ks = 0; ks < DP / 16; ++ks) {
            uint32_t kf[4];
            const uint32_t key = lm_top * 8 + lm_row;
            ldsm4(kf, kb + key * R::kRowBytes + (((ks * 2 + lm_hi) ^ (key & 7)) << 4));
            mma_bf16(s[0], q[ks][0], q[ks][1], q[ks][2], q[ks][3], kf[0], kf[1]);
            mma_bf16(s[1], q[ks][0], q[ks][1], q[ks][2], q[ks][3], kf[2], kf[3]);
        }
        // ---- keys a row does not see
        const int p0 = c.step * kKeys;
        bool hidden = false;                           // a key that is there but that one of this thread's rows skips
        if (c.there != 0xffff || (p0 + kKeys > c.ctx && !c.group)) {
#pragma unroll
            for (int hrow = 0; hrow < 2; ++hrow) {
                const int node = (c.row_tile * kRows + g4 + hrow * 8) / group;
                uint32_t seen = 0;
                if (node < c.nodes) {
                    const Request r{c.start, c.nodes, 0, 0, c.ctx, c.keys};
                    seen = c.group ? 0xffffu : (uint32_t)seen_keys(a, r, node, p0);
                    seen &= c.there;
                    hidden = hidden || (int)seen != c.there;
                }
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        if (!(seen >> (n * 8 + t4 * 2 + e) & 1)) s[n][hrow * 2 + e] = -INFINITY;
            }
        }
        // ---- running maximum and sum
        float top[2] = {fmaxf(m[0], fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[1][0], s[1][1]))),
                        fmaxf(m[1], fmaxf(fmaxf(s[0][2], s[0][3]), fmaxf(s[1][2], s[1][3])))};
#pragma unroll
        for (int x = 1; x <= 2; ++x) {
            top[0] = fmaxf(top[0], __shfl_xor_sync(0xffffffffu, top[0], x));
            top[1] = fmaxf(top[1], __shfl_xor_sync(0xffffffffu, top[1], x));
        }
        // The products are rounded by themselves: a row whose maximum stands is kept by a factor of exactly 1, whatever the
        // others do.
        const float base0 = top[0] == -INFINITY ? 0.f : __fmul_rn(top[0], c2);
        const float base1 = top[1] == -INFINITY ? 0.f : __fmul_rn(top[1], c2);
        if (__any_sync(0xffffffffu, top[0] != m[0] || top[1] != m[1])) {
            const float k0 = exp2_fast(__fmul_rn(m[0], c2) - base0), k1 = exp2_fast(__fmul_rn(m[1], c2) - base1);
            l[0] *= k0;
            l[1] *= k1;
#pragma unroll
            for (int d = 0; d < DP / 8; ++d) o[d][0] *= k0, o[d][1] *= k0, o[d][2] *= k1, o[d][3] *= k1;
            m[0] = top[0];
            m[1] = top[1];
        }
        uint32_t pf[2][2];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            const float e0 = exp2_fast(fmaf(s[n][0], c2, -base0)), e1 = exp2_fast(fmaf(s[n][1], c2, -base0));
            const float e2 = exp2_fast(fmaf(s[n][2], c2, -base1)), e3 = exp2_fast(fmaf(s[n][3], c2, -base1));
            l[0] += e0 + e1;
            l[1] += e2 + e3;
            // weights to bf16 for the second product: half a step, 2^-8 relative at most, of either sign from key to key, so that
            // a row of many keys is off by less than its output's own rounding; their sum l stays in fp32 and unrounded
            pf[n][0] = pack_bf16(e0, e1);
            pf[n][1] = pack_bf16(e2, e3);
        }
        // A weight of zero times an infinity or NaN is NaN: where a row skips a key that is there, values that are not
        // finite are looked for, and such a step is summed key by key without the zero weights.
        bool by_key = false;
        if (__any_sync(0xffffffffu, hidden)) {
            uint32_t odd = 0;
            for (int n = lane; n < R::kHalf / 16; n += 32) {
                const uint4 v = *reinterpret_cast<const uint4 *>(ring + i % kStages * R::kStage + R::kHalf + n * 16);
                odd |= ((v.x & 0x7f807f80u) + 0x00800080u) | ((v.y & 0x7f807f80u) + 0x00800080u) |
                       ((v.z & 0x7f807f80u) + 0x00800080u) | ((v.w & 0x7f807f80u) + 0x00800080u);
            }
            by_key = __any_sync(0xffffffffu, (odd & 0x80008000u) != 0);
        }
        if (by_key) {
            // the weights go where the keys lay: [16][16] bf16
            uint32_t *w = reinterpret_cast<uint32_t *>(ring + i % kStages * R::kStage);
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int hrow = 0; hrow < 2; ++hrow) w[(g4 + hrow * 8) * 8 + n * 4 + t4] = pf[n][hrow];
            __syncwarp();
            const __nv_bfloat16 *wb = reinterpret_cast<const __nv_bfloat16 *>(w);
            for (int k = 0; k < kKeys; ++k) {
                const float w0 = to_f32(wb[g4 * 16 + k]), w1 = to_f32(wb[(g4 + 8) * 16 + k]);
                const unsigned char *vr = ring + i % kStages * R::kStage + R::kHalf + k * R::kRowBytes + t4 * 4;
#pragma unroll
                for (int d = 0; d < DP / 8; ++d) {
                    const uint32_t v = *reinterpret_cast<const uint32_t *>(vr + ((d ^ (k & 7)) << 4));
                    if (w0 != 0.f) o[d][0] = fmaf(w0, bf_lo(v), o[d][0]), o[d][1] = fmaf(w0, bf_hi(v), o[d][1]);
                    if (w1 != 0.f) o[d][2] = fmaf(w1, bf_lo(v), o[d][2]), o[d][3] = fmaf(w1, bf_hi(v), o[d][3]);
                }
            }
        } else {
#pragma unroll
            for (int d = 0; d < DP / 16; ++d) {
                uint32_t vf[4];
                const uint32_t key = lm_hi * 8 + lm_row;
                ldsm4_t(vf, vb + key * R::kRowBytes + (((d * 2 + lm_top) ^ (key & 7)) << 4));
                mma_bf16(o[2 * d], pf[0][0], pf[0][1], pf[1][0], pf[1][1], vf[0], vf[1]);
                mma_bf16(o[2 * d + 1], pf[0][0], pf[0][1], pf[1][0], pf[1][1], vf[2], vf[3]);
            }
        }
        // ---- the warp's part of the unit ends
        if (c.last) {
#pragma unroll
            for (int hrow = 0; hrow < 2; ++hrow) {
                l[hrow] += __shfl_xor_sync(0xffffffffu, l[hrow], 1);
                l[hrow] += __shfl_xor_sync(0xffffffffu, l[hrow], 2);
                const int r = g4 + hrow * 8, row = c.row_tile * kRows + r, node = row / group;
                if (node >= c.nodes) continue;
                const size_t rows = (size_t)a.n_tokens * a.n_heads;
                const size_t at = (c.group ? 0 : rows) + (size_t)(c.start + node) * a.n_heads + c.head * group + row % group;
                const long long slot = 2ll * worker + (c.starts ? 1 : 0);
                const bool whole = c.starts && c.ends;
                float *part = whole ? a.row_o + at * DP : plan.part + (slot * kRows + r) * DP;
                float2 *stat = whole ? a.row_ml + at : plan.stat + slot * kRows + r;
#pragma unroll
                for (int d = 0; d < DP / 8; ++d)
                    *reinterpret_cast<float2 *>(part + d * 8 + t4 * 2) = make_float2(o[d][hrow * 2], o[d][hrow * 2 + 1]);
                if (t4 == 0) {
                    *stat = make_float2(m[hrow] == -INFINITY ? -INFINITY : m[hrow] * c2, l[hrow]);
                    if (c.starts)
                        a.row_at[at] = make_int4(worker, whole ? 0 : c.parts, r, (int)(at < rows ? at : at - rows));
                }
            }
            fresh = true;
        }
    }
}

}  // namespace rows
}  // namespace tree
}  // namespace lora
