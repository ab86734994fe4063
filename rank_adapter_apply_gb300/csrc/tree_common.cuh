// Shared by the kernels of lora_tree_attention and lora_prefix_attention
// (tree_attention.cu, tree_attention_tc.cu, tree_attention_f32.cu,
// prefix_attention.cu): arguments, the units of work and their split.
#pragma once

#include "step_util.cuh"

namespace lora {
namespace tree {

using namespace step;

struct TreeArgs {
    const void *q, *k_cache, *v_cache;
    void *out;
    float *lse;
    const int32_t *page_table, *ctx_lens, *node_starts;
    const uint64_t *tree_mask;
    long long q_token, q_head, c_page, c_slot, c_head, o_token, o_head, table_stride, n_pages;
    float scale;
    int page_size, table_pages, mask_words, n_requests, n_tokens, n_heads, n_kv, head_dim;
    // lora_prefix_attention alone. Its work is that of n_groups + n_requests entries: a group's rows are those of its
    // requests and its keys the prefix; then the requests with their own keys. A launch does `count` of them from `first`
    // on. Results of a row go to row_o, row_ml (of a group's entry, then of a request's: [2][n_tokens * n_heads]) or
    // to the parts that row_at names.
    const int32_t *prefix_table, *prefix_lens, *group_starts;
    long long prefix_stride;
    int n_groups, prefix_pages, first, count;
    float *row_o;             // [..][DP] unnormalised O; nullptr: a call of lora_tree_attention
    float2 *row_ml;           // (m, l)
    int4 *row_at;             // (CTA of the first part, parts: 0 is row_o, row of the tile, token * n_heads + head)
};

__device__ __forceinline__ int node_start(const TreeArgs &a, int b) {
    return min(max(a.node_starts[b], 0), a.n_tokens);
}

// The work of the kernels. A unit is (request, row tile, key/value head): the query
// rows of one tile (a node's query heads that share the key/value head lie side by
// side) against all keys of the request in tiles of 64. Row tiles of one request
// read the same keys, so they are put side by side in blocks of up to eight, and the
// blocks of k row tiles are class k. The key tiles of a class's blocks, in a row,
// are its columns; they are dealt in equal shares to groups of k CTAs, of which each
// takes one row tile of the block. So the CTAs of a group read the same keys at the
// same time, and memory gives them once (4 requests of up to 64 nodes, 64 heads over
// 8, 32768 keys: 1.5 GB a call when the row tiles went one after another). A share
// may start and end inside a unit, so ragged lengths cost nothing, and a unit is
// split over many CTAs where there are few. A CTA that covers a whole unit writes its
// result; the others write (O, m, l) to the workspace, and the join kernel joins them.
constexpr int kTileKeys = 64;

struct Plan {                 // workspace regions
    float *part;              // [2 * ctas][M][DP] unnormalised O
    float2 *stat;             // [2 * ctas][M] (m, l), m in powers of two
    int4 *seg;                // [ctas] (request, row tile, head, parts) of the unit that starts in a CTA's share and
                              // goes on past it; parts = 0: there is none
    int ctas;
};
// Part slots: 2c + 1 holds the first part of the unit that goes on past CTA c's
// share, 2c the part of the unit that began before it.

// 16 bytes to shared memory, zeros when !ok (the source is then not read).
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool ok) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0) : "memory");
}
__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Four 8 x 8 matrices of 16-bit elements, plain and transposed.
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}

struct Request {
    int start, nodes, row_tiles, key_tiles, ctx, keys;
};

// The entries of a launch, and entry b's row of page ids. kPrefix: a call of lora_prefix_attention.
template <bool kPrefix>
__device__ __forceinline__ int entries(const TreeArgs &a) {
    return kPrefix ? a.count : a.n_requests;
}
template <bool kPrefix>
__device__ __forceinline__ bool is_group(const TreeArgs &a, int b) {
    return kPrefix && a.first + b < a.n_groups;
}
template <bool kPrefix>
__device__ __forceinline__ const int32_t *table_row(const TreeArgs &a, int b) {
    if (is_group<kPrefix>(a, b)) return a.prefix_table + (a.first + b) * a.prefix_stride;
    return a.page_table + (kPrefix ? a.first + b - a.n_groups : b) * a.table_stride;
}
// First request of group g.
__device__ __forceinline__ int group_start(const TreeArgs &a, int g) {
    return min(max(a.group_starts[g], 0), a.n_requests);
}

// Not inlined, like everything that a tile in the middle of a unit does not need: a warp of a role runs alone on its
// scheduler, and straight code that does not fit the instruction cache would be its pace.
template <bool kPrefix>
__device__ __noinline__ inline Request request(const TreeArgs &a, int b, int m_rows) {
    Request r;
    const bool shared = is_group<kPrefix>(a, b);
    int n = b;
    if constexpr (kPrefix) n = shared ? a.first + b : a.first + b - a.n_groups;
    if (shared) {
        r.start = node_start(a, group_start(a, n));
        r.nodes = max(node_start(a, group_start(a, n + 1)) - r.start, 0);
        r.ctx = max(a.prefix_lens[n], 0);
    } else {
        r.start = node_start(a, n);
        r.nodes = max(node_start(a, n + 1) - r.start, 0);
        r.ctx = max(a.ctx_lens[n], 0);
    }
    // keys that fit the page table; the largest count is a multiple of the tile below 2^31
    const long long room = min((long long)(shared ? a.prefix_pages : a.table_pages) * a.page_size, 0x7fffffc0ll);
    r.keys = (int)min((long long)r.ctx + (shared ? 0 : r.nodes), room);
    r.row_tiles = (r.nodes * (a.n_heads / a.n_kv) + m_rows - 1) / m_rows;
    r.key_tiles = max((r.keys + kTileKeys - 1) / kTileKeys, 1);   // one for rows without keys, too
    return r;
}

constexpr int kMaxClass = 8;

// Blocks of class k among a request's row tiles; the last, of less than eight, comes after the others.
__device__ __forceinline__ int blocks_of(int row_tiles, int k) {
    return k == kMaxClass ? row_tiles / kMaxClass : row_tiles % kMaxClass == k;
}

// Where a CTA is in the columns of its class `k`, of whose blocks it takes row tile `row`.
struct Cursor {
    Request r;
    int b, row_tile, head, tile, k, row;
};

// The next request of the class is looked for by the whole warp, 32 at a time: one after the other they took 18 us of a
// CTA whose class has few requests among 41. All lanes call it with the same cursor.
template <bool kPrefix>
__device__ __noinline__ inline void next_unit(const TreeArgs &a, Cursor &c, int m_rows) {
    c.tile = 0;
    if (++c.head < a.n_kv) return;
    c.head = 0;
    if (c.k == kMaxClass && (c.row_tile += kMaxClass) / kMaxClass < c.r.row_tiles / kMaxClass) return;
    const int n = entries<kPrefix>(a), lane = threadIdx.x & 31;
    uint32_t found = 0;
    for (int b0 = c.b + 1; found == 0; b0 += 32) {
        if (b0 >= n) {
            c.b = n;
            return;
        }
        Request r{};
        if (b0 + lane < n) r = request<kPrefix>(a, b0 + lane, m_rows);
        found = __ballot_sync(0xffffffffu, blocks_of(r.row_tiles, c.k) > 0);
        const int at = __ffs(found) - 1;                     // -1, of nobody: any lane
        c.b = b0 + at;
        c.r = {__shfl_sync(0xffffffffu, r.start, at),     __shfl_sync(0xffffffffu, r.nodes, at),
               __shfl_sync(0xffffffffu, r.row_tiles, at), __shfl_sync(0xffffffffu, r.key_tiles, at),
               __shfl_sync(0xffffffffu, r.ctx, at),       __shfl_sync(0xffffffffu, r.keys, at)};
    }
    c.row_tile = (c.k == kMaxClass ? 0 : c.r.row_tiles - c.k) + c.row;
}

template <bool kPrefix>
__device__ __forceinline__ void next_tile(const TreeArgs &a, Cursor &c, int m_rows) {
    if (++c.tile < c.r.key_tiles) return;
    Cursor next = c;                                     // c itself stays in registers
    next_unit<kPrefix>(a, next, m_rows);
    c = next;
}

// Bits 0..63: which of the tile's keys p0 .. p0 + 63 node i (row `token`) sees.
__device__ __noinline__ inline uint64_t seen_keys(const TreeArgs &a, const Request &r, int i, int p0) {
    const int in_ctx = r.ctx - p0;
    uint64_t seen = in_ctx >= 64 ? ~0ull : in_ctx <= 0 ? 0ull : (1ull << in_ctx) - 1;
    if (in_ctx >= 64) return seen;
    const int j0 = -in_ctx;                             // the node that is the tile's first key
    if (!a.tree_mask) {
        const int n = in_ctx + i + 1;                   // keys up to the node itself
        return n >= 64 ? ~0ull : n <= 0 ? 0ull : (1ull << n) - 1;
    }
    const uint64_t *m = a.tree_mask + (size_t)(r.start + i) * a.mask_words;
    if (j0 < 0) return seen | m[0] << (-j0);
    const int w = j0 >> 6, sh = j0 & 63;
    if (w < a.mask_words) seen = m[w] >> sh;
    if (sh && w + 1 < a.mask_words) seen |= m[w + 1] << (64 - sh);
    return seen;
}

// A CTA's share of its class's columns: [lo, hi) of total, dealt to `used` groups of which its is number `group`, the
// tiles in it and where it starts. false: it has none. scratch: kScratch words and one for each warp. Every thread calls
// it. kUnit: columns without a tile that follow a unit's, for what its beginning and end cost.
constexpr int kScratch = 2 + kMaxClass;
struct Share {
    long long lo, hi, total, used;
    int group, n_tiles;
    Cursor start;
};

// x * y / z, in 32 bits where they will do.
__device__ __forceinline__ long long scaled(long long x, long long y, long long z) {
    const long long p = x * y;
    return (p | z) >> 32 == 0 ? (long long)((uint32_t)p / (uint32_t)z) : p / z;
}

template <int kThreads, bool kPrefix, int kUnit = 0>
__device__ inline bool find_share(const TreeArgs &a, int m_rows, long long *scratch, Share &s) {
    constexpr int kWarps = kThreads / 32;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, n_entries = entries<kPrefix>(a);
    long long *columns = scratch + 2, *sums = scratch + kScratch;    // of class k at k - 1; of the warps' requests
    // Up to 32 requests: every warp finds it all for itself, a lane to a request. What the warps write to shared memory
    // is the same, and none waits for another.
    const bool few = n_entries <= 32;
    const int each = few ? 32 : kThreads, me = few ? lane : tid;
    if (!few) {
        if (tid < kScratch) scratch[tid] = tid == 0 ? -1 : 0;
        __syncthreads();
    }
    Request mine{};                                          // request `me`: the only ones in most calls
    long long my_columns = 0;                                // few: of class lane + 1
    for (int b0 = 0; b0 < n_entries; b0 += each) {
        const int b = b0 + me;
        Request r{};
        if (b < n_entries) r = request<kPrefix>(a, b, m_rows);
        if (b0 == 0) mine = r;
        const uint32_t some = __reduce_or_sync(0xffffffffu, (r.row_tiles % kMaxClass ? 1u << r.row_tiles % kMaxClass : 0u) |
                                                                (r.row_tiles >= kMaxClass ? 1u << kMaxClass : 0u));
        for (uint32_t left = some; left; left &= left - 1) {
            const int k = __ffs(left) - 1;
            const long long n = (long long)blocks_of(r.row_tiles, k) * (r.key_tiles + kUnit) * a.n_kv;
            const uint32_t lo = __reduce_add_sync(0xffffffffu, (uint32_t)n & 0xffffffu);
            const uint32_t hi = __reduce_add_sync(0xffffffffu, (uint32_t)(n >> 24));
            const unsigned long long sum = lo + ((unsigned long long)hi << 24);
            if (few)
                my_columns = lane == k - 1 ? (long long)sum : my_columns;
            else if (lane == 0)
                atomicAdd(reinterpret_cast<unsigned long long *>(columns) + k - 1, sum);
        }
    }
    if (few) {
        if (lane < kMaxClass) columns[lane] = my_columns;
        __syncwarp();
    } else {
        __syncthreads();
    }
    const int grid = gridDim.x;
    long long all = 0;
    uint32_t present = 0;                                    // classes with columns
#pragma unroll
    for (int k = 1; k <= kMaxClass; ++k) {
        const long long n = columns[k - 1];
        all += k * n;
        present |= n > 0 ? 1u << k : 0u;
    }
    if (all == 0) return false;
    // The longest share t: the least of 32 from what equal shares would be, 0.65 % apart, with which the groups, of
    // whole numbers, fit the grid. They do by 1.14 times that: rounding up costs 1 + 2 + .. + 8 CTAs at most. CTAs that
    // are left go to the widest class that takes them; to one class alone all go.
    long long t = 0;
    int spare = grid;
    if (present & (present - 1)) {
        for (long long even = scaled(all + grid - 1, 1, grid);; even *= 2) {     // a grid of 216 CTAs or more never doubles
            t = even + scaled(even * lane + 154, 1, 155);
            long long ctas = 0;
            for (uint32_t left = present; left; left &= left - 1) {
                const int k = __ffs(left) - 1;
                ctas += k * scaled(columns[k - 1] + t - 1, 1, t);
            }
            const uint32_t fits = __ballot_sync(0xffffffffu, ctas <= grid);
            if (fits == 0) continue;
            t = __shfl_sync(0xffffffffu, t, __ffs(fits) - 1);
            spare = grid - (int)__shfl_sync(0xffffffffu, ctas, __ffs(fits) - 1);
            break;
        }
    } else {
        spare = grid - (__ffs(present) - 1);                 // a group of the one class
    }
    int k = 0, at_cta = blockIdx.x;
    for (uint32_t left = present; left;) {
        k = 31 - __clz(left);
        left ^= 1u << k;
        const long long need = present & (present - 1) ? scaled(columns[k - 1] + t - 1, 1, t) : 1;
        s.used = min(need + spare / k, columns[k - 1]);
        spare -= (int)(s.used - need) * k;
        if (at_cta < k * s.used) break;
        at_cta -= k * (int)s.used;
        k = 0;
    }
    if (k == 0) return false;
    s.total = columns[k - 1];
    s.start.k = k;
    s.start.row = (int)scaled(at_cta, 1, s.used);
    s.group = at_cta - s.start.row * (int)s.used;
    s.lo = scaled(s.total, s.group, s.used);
    s.hi = scaled(s.total, s.group + 1, s.used);
    auto scan = [&](long long n) {
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long v = __shfl_up_sync(0xffffffffu, n, o);
            if (lane >= o) n += v;
        }
        return n;
    };
    // of an entry with `units` units before it and its columns from `first` on: columns without a tile before column x
    auto idle = [&](long long x, long long first, long long units, int key_tiles) -> long long {
        const long long at = x - first, unit = scaled(at, 1, key_tiles + kUnit), rest = at - unit * (key_tiles + kUnit);
        return (units + unit) * kUnit + max(rest - key_tiles, 0ll);
    };
    long long before = 0;                                    // columns of the requests before the share's first
    long long idle_lo = 0, idle_hi = 0;
    if (few) {
        const long long units = (long long)blocks_of(mine.row_tiles, k) * a.n_kv, n = units * (mine.key_tiles + kUnit);
        const long long upto = scan(n);
        const int b = __ffs(__ballot_sync(0xffffffffu, upto - n <= s.lo && s.lo < upto)) - 1;
        before = __shfl_sync(0xffffffffu, upto - n, b);
        s.start.b = b;
        s.start.r = {__shfl_sync(0xffffffffu, mine.start, b),     __shfl_sync(0xffffffffu, mine.nodes, b),
                     __shfl_sync(0xffffffffu, mine.row_tiles, b), __shfl_sync(0xffffffffu, mine.key_tiles, b),
                     __shfl_sync(0xffffffffu, mine.ctx, b),       __shfl_sync(0xffffffffu, mine.keys, b)};
        if constexpr (kUnit > 0) {
            const long long units_before = scan(units) - units;
            const int e = __ffs(__ballot_sync(0xffffffffu, upto - n < s.hi && s.hi <= upto)) - 1;
            idle_lo = idle(s.lo, before, __shfl_sync(0xffffffffu, units_before, b), s.start.r.key_tiles);
            idle_hi = idle(s.hi, __shfl_sync(0xffffffffu, upto - n, e), __shfl_sync(0xffffffffu, units_before, e),
                           __shfl_sync(0xffffffffu, mine.key_tiles, e));
        }
    } else {
        long long units_before = 0;
        if constexpr (kUnit > 0) {                           // the columns have been read: their place is free
            __syncthreads();
            if (tid == 0) scratch[3] = -1;
            __syncthreads();
        }
        for (int b0 = 0; b0 < n_entries; b0 += kThreads) {    // ends in the chunk that holds the share's last column
            const int b = b0 + tid;
            if (b0 > 0 && b < n_entries) mine = request<kPrefix>(a, b, m_rows);
            const long long units = b < n_entries ? (long long)blocks_of(mine.row_tiles, k) * a.n_kv : 0;
            const long long n = units * (mine.key_tiles + kUnit);
            long long upto = scan(n);
            if (lane == 31) sums[warp] = upto;
            __syncthreads();
            for (int w = 0; w < warp; ++w) upto += sums[w];
            upto += before;
            const bool first = upto - n <= s.lo && s.lo < upto, last = upto - n < s.hi && s.hi <= upto;
            if (first) {
                scratch[0] = b, scratch[1] = upto - n;
                const int words[] = {mine.start, mine.nodes, mine.row_tiles, mine.key_tiles, mine.ctx, mine.keys};
#pragma unroll
                for (int i = 0; i < 6; ++i) reinterpret_cast<int *>(scratch + 4)[i] = words[i];
            }
            for (int w = 0; w < kWarps; ++w) before += sums[w];
            __syncthreads();
            if constexpr (kUnit > 0) {
                long long u = scan(units);
                if (lane == 31) sums[warp] = u;
                __syncthreads();
                for (int w = 0; w < warp; ++w) u += sums[w];
                u += units_before - units;
                if (first) scratch[2] = idle(s.lo, upto - n, u, mine.key_tiles);
                if (last) scratch[3] = idle(s.hi, upto - n, u, mine.key_tiles);
                for (int w = 0; w < kWarps; ++w) units_before += sums[w];
                __syncthreads();
                if (scratch[3] >= 0) break;
            } else if (scratch[0] >= 0) {
                break;
            }
        }
        if (scratch[0] < 0) return false;                    // not reached
        if constexpr (kUnit > 0) idle_lo = scratch[2], idle_hi = scratch[3];
        before = scratch[1];
        s.start.b = (int)scratch[0];
        const int *r = reinterpret_cast<const int *>(scratch + 4);
        s.start.r = {r[0], r[1], r[2], r[3], r[4], r[5]};
    }
    s.n_tiles = (int)(s.hi - s.lo - (idle_hi - idle_lo));
    if (s.n_tiles == 0) return false;
    const int wide = s.start.r.key_tiles + kUnit;
    const long long at = s.lo - before, unit = scaled(at, 1, wide), block = scaled(unit, 1, a.n_kv);
    s.start.tile = (int)(at - unit * wide);
    s.start.head = (int)(unit - block * a.n_kv);
    s.start.row_tile = (k == kMaxClass ? (int)block * kMaxClass : s.start.r.row_tiles - k) + s.start.row;
    if (kUnit > 0 && s.start.tile >= s.start.r.key_tiles) next_unit<kPrefix>(a, s.start, m_rows);
    return true;
}

// Parts of the unit at cursor c whose tile is the share's last, and not the unit's:
// group floor(((x + 1) used - 1) / total) has column x. The CTAs of neighbouring
// groups with the same row are neighbours.
__device__ __forceinline__ int parts_of(const Share &s, const Cursor &c) {
    const long long x = s.hi - 1 + (c.r.key_tiles - 1 - c.tile);
    const long long p = (x + 1) * s.used - 1;
    return (int)scaled(p, 1, s.total) - s.group + 1;
}

// Element offset of key `key` of the cursor's tile in the caches, -1: nobody sees it.
template <bool kPrefix>
__device__ __forceinline__ long long key_offset(const TreeArgs &a, const Cursor &u, int key) {
    const int p = u.tile * kTileKeys + key;
    if (p >= u.r.keys) return -1;
    const int at = p / a.page_size, id = table_row<kPrefix>(a, u.b)[at];
    return id >= 0 && id < a.n_pages ? id * a.c_page + (p - at * a.page_size) * a.c_slot : -1;
}

// Where a row's result goes in a call of lora_prefix_attention: the index of row_o and row_ml for one that is whole, and
// row_at's entry of the unit that starts in this CTA's share.
__device__ __forceinline__ size_t row_index(const TreeArgs &a, const Cursor &c, long long token, int head) {
    const size_t rows = (size_t)a.n_tokens * a.n_heads, row = (size_t)token * a.n_heads + head;
    return is_group<true>(a, c.b) ? row : rows + row;
}
__device__ __forceinline__ void name_parts(const TreeArgs &a, size_t index, int parts, int r) {
    const size_t rows = (size_t)a.n_tokens * a.n_heads;
    a.row_at[index] = make_int4(blockIdx.x, parts, r, (int)(index < rows ? index : index - rows));
}

// O, maximum (in powers of two) and sum of a row, a lane's columns, joined part by part.
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

// A row's output and log-sum-exp, by a warp.
template <typename T, int DP>
__device__ __forceinline__ void store_joined(const TreeArgs &a, long long token, int head, const Joined<DP> &j) {
    constexpr int V = Joined<DP>::V;
    const int lane = threadIdx.x & 31;
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

constexpr int kMaxRows = 128;
constexpr int kMaxCtas = 2 * 160;

// tree_attention.cu: the checks of a call under its name (*nothing: there is nothing to do; need: the least workspace),
// its arguments, CTAs of a kernel on the current device (0: there is none), a workspace's bytes for them.
int check(const lora_tree_attention_desc *d, const char *name, size_t need, bool *nothing);
bool shape_ok(int n_requests, int n_tokens, int n_heads, int n_kv, int head_dim, int dtype);
TreeArgs arguments(const lora_tree_attention_desc *d);
int grid_of_device();
size_t plan_bytes();
Plan plan_at(void *workspace, int ctas);

// prefix_rows.cu: row tiles of 16 by single warps, which become the plan's CTAs (lora_prefix_attention alone).
cudaError_t launch_rows(const TreeArgs &a, Plan &plan, cudaStream_t st);

// tree_attention_tc.cu: row tiles of up to 128 on the 5th-generation tensor cores,
// for the calls that it takes; the rows of a tile. launch_tc returns
// cudaErrorNotSupported where the driver refuses a tensor map (nothing is queued).
bool tc_takes(const TreeArgs &a);
int tc_rows(const TreeArgs &a);
cudaError_t launch_tc(const TreeArgs &a, const Plan &plan, cudaStream_t st);
// lora_prefix_attention: the entries of `wide` on that kernel, then, where there are any, those of `narrow` by single warps
// of the same CTAs, which become its plan's CTAs.
cudaError_t launch_mixed(const TreeArgs &wide, const Plan &wide_plan, const TreeArgs &narrow, Plan &narrow_plan,
                         cudaStream_t st);
// CTAs of its kernel on the current device whose bounded waits gave up so far.
cudaError_t read_timeouts(unsigned *count);

// tree_attention_f32.cu: row tiles of 16 or 64 in fp32.
cudaError_t launch_f32(const TreeArgs &a, const Plan &plan, int m_rows, cudaStream_t st);

}  // namespace tree
}  // namespace lora
