// Shared by the tensor-core kernels of lora_tree_attention (tree_attention.cu,
// tree_attention_tc.cu): arguments, the units of work and their split.
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

struct Request {
    int start, nodes, row_tiles, key_tiles, ctx, keys;
};

// Not inlined, like everything that a tile in the middle of a unit does not need: a warp of a role runs alone on its
// scheduler, and straight code that does not fit the instruction cache would be its pace.
__device__ __noinline__ inline Request request(const TreeArgs &a, int b, int m_rows) {
    Request r;
    r.start = node_start(a, b);
    r.nodes = max(node_start(a, b + 1) - r.start, 0);
    // keys that fit the page table; the largest count is a multiple of the tile below 2^31
    const long long room = min((long long)a.table_pages * a.page_size, 0x7fffffc0ll);
    r.ctx = max(a.ctx_lens[b], 0);
    r.keys = (int)min((long long)r.ctx + r.nodes, room);
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

__device__ __noinline__ inline void next_unit(const TreeArgs &a, Cursor &c, int m_rows) {
    c.tile = 0;
    if (++c.head < a.n_kv) return;
    c.head = 0;
    if (c.k == kMaxClass && (c.row_tile += kMaxClass) / kMaxClass < c.r.row_tiles / kMaxClass) return;
    do {
        if (++c.b >= a.n_requests) return;
        c.r = request(a, c.b, m_rows);
    } while (blocks_of(c.r.row_tiles, c.k) == 0);
    c.row_tile = (c.k == kMaxClass ? 0 : c.r.row_tiles - c.k) + c.row;
}

__device__ __forceinline__ void next_tile(const TreeArgs &a, Cursor &c, int m_rows) {
    if (++c.tile < c.r.key_tiles) return;
    Cursor next = c;                                     // c itself stays in registers
    next_unit(a, next, m_rows);
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

// A CTA's share of its class's columns: [lo, hi) of total, dealt to `used` groups of which its is number `group`, and
// where it starts. false: it has none. scratch: kScratch words and one for each warp. Every thread calls it.
constexpr int kScratch = 2 + kMaxClass;
struct Share {
    long long lo, hi, total, used;
    int group;
    Cursor start;
};

// x * y / z, in 32 bits where they will do.
__device__ __forceinline__ long long scaled(long long x, long long y, long long z) {
    const long long p = x * y;
    return (p | z) >> 32 == 0 ? (long long)((uint32_t)p / (uint32_t)z) : p / z;
}

template <int kThreads>
__device__ inline bool find_share(const TreeArgs &a, int m_rows, long long *scratch, Share &s) {
    constexpr int kWarps = kThreads / 32;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    long long *columns = scratch + 2, *sums = scratch + kScratch;    // of class k at k - 1; of the warps' requests
    // Up to 32 requests: every warp finds it all for itself, a lane to a request. What the warps write to shared memory
    // is the same, and none waits for another.
    const bool few = a.n_requests <= 32;
    const int each = few ? 32 : kThreads, me = few ? lane : tid;
    if (!few) {
        if (tid < kScratch) scratch[tid] = tid == 0 ? -1 : 0;
        __syncthreads();
    }
    Request mine{};                                          // request `me`: the only ones in most calls
    long long my_columns = 0;                                // few: of class lane + 1
    for (int b0 = 0; b0 < a.n_requests; b0 += each) {
        const int b = b0 + me;
        Request r{};
        if (b < a.n_requests) r = request(a, b, m_rows);
        if (b0 == 0) mine = r;
        const uint32_t some = __reduce_or_sync(0xffffffffu, (r.row_tiles % kMaxClass ? 1u << r.row_tiles % kMaxClass : 0u) |
                                                                (r.row_tiles >= kMaxClass ? 1u << kMaxClass : 0u));
        for (uint32_t left = some; left; left &= left - 1) {
            const int k = __ffs(left) - 1;
            const long long n = (long long)blocks_of(r.row_tiles, k) * r.key_tiles * a.n_kv;
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
    long long before = 0;                                    // columns of the requests before the share's first
    if (few) {
        const long long n = (long long)blocks_of(mine.row_tiles, k) * mine.key_tiles * a.n_kv, upto = scan(n);
        const int b = __ffs(__ballot_sync(0xffffffffu, upto - n <= s.lo && s.lo < upto)) - 1;
        before = __shfl_sync(0xffffffffu, upto - n, b);
        s.start.b = b;
        s.start.r = {__shfl_sync(0xffffffffu, mine.start, b),     __shfl_sync(0xffffffffu, mine.nodes, b),
                     __shfl_sync(0xffffffffu, mine.row_tiles, b), __shfl_sync(0xffffffffu, mine.key_tiles, b),
                     __shfl_sync(0xffffffffu, mine.ctx, b),       __shfl_sync(0xffffffffu, mine.keys, b)};
    } else {
        for (int b0 = 0; b0 < a.n_requests; b0 += kThreads) {    // ends in the chunk that holds column lo < total
            const int b = b0 + tid;
            if (b0 > 0 && b < a.n_requests) mine = request(a, b, m_rows);
            const long long n = b < a.n_requests ? (long long)blocks_of(mine.row_tiles, k) * mine.key_tiles * a.n_kv : 0;
            long long upto = scan(n);
            if (lane == 31) sums[warp] = upto;
            __syncthreads();
            for (int w = 0; w < warp; ++w) upto += sums[w];
            upto += before;
            if (upto - n <= s.lo && s.lo < upto) scratch[0] = b, scratch[1] = upto - n;
            for (int w = 0; w < kWarps; ++w) before += sums[w];
            __syncthreads();
            if (scratch[0] >= 0) break;
        }
        if (scratch[0] < 0) return false;                    // not reached
        before = scratch[1];
        s.start.b = (int)scratch[0];
        s.start.r = request(a, s.start.b, m_rows);
    }
    const long long at = s.lo - before, unit = scaled(at, 1, s.start.r.key_tiles), block = scaled(unit, 1, a.n_kv);
    s.start.tile = (int)(at - unit * s.start.r.key_tiles);
    s.start.head = (int)(unit - block * a.n_kv);
    s.start.row_tile = (k == kMaxClass ? (int)block * kMaxClass : s.start.r.row_tiles - k) + s.start.row;
    return true;
}

// Parts of the unit at cursor c whose tile is the share's tile i and the last of
// the share: group floor(((x + 1) used - 1) / total) has column x. The CTAs of
// neighbouring groups with the same row are neighbours.
__device__ __forceinline__ int parts_of(const Share &s, const Cursor &c, int i) {
    const long long x = s.lo + i + (c.r.key_tiles - 1 - c.tile);
    const long long p = (x + 1) * s.used - 1;
    return (int)scaled(p, 1, s.total) - s.group + 1;
}

// Element offset of key `key` of the cursor's tile in the caches, -1: nobody sees it.
__device__ __forceinline__ long long key_offset(const TreeArgs &a, const Cursor &u, int key) {
    const int p = u.tile * kTileKeys + key;
    if (p >= u.r.keys) return -1;
    const int at = p / a.page_size, id = a.page_table[u.b * a.table_stride + at];
    return id >= 0 && id < a.n_pages ? id * a.c_page + (p - at * a.page_size) * a.c_slot : -1;
}

// tree_attention_tc.cu: row tiles of up to 128 on the 5th-generation tensor cores,
// for the calls that it takes; the rows of a tile. launch_tc returns
// cudaErrorNotSupported where the driver refuses a tensor map (nothing is queued).
bool tc_takes(const TreeArgs &a);
int tc_rows(const TreeArgs &a);
cudaError_t launch_tc(const TreeArgs &a, const Plan &plan, cudaStream_t st);
// CTAs of its kernel on the current device whose bounded waits gave up so far.
cudaError_t read_timeouts(unsigned *count);

// tree_attention_f32.cu: row tiles of 16 or 64 in fp32.
cudaError_t launch_f32(const TreeArgs &a, const Plan &plan, int m_rows, cudaStream_t st);

}  // namespace tree
}  // namespace lora
