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

// The work of the tensor-core kernels. A unit is (request, row tile, key/value
// head): the query rows of one tile (a node's query heads that share the key/value
// head lie side by side) against all keys of the request in tiles of 64. The key
// tiles of all units, in a row, are dealt to the CTAs in equal shares: a share is a
// run of tiles that may start and end inside a unit, so ragged lengths cost
// nothing, and a unit is split over many CTAs where there are few. A CTA that
// covers a whole unit writes its result; the others write (O, m, l) to the
// workspace, and the join kernel joins them.
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

// Where a CTA is in the run of tiles.
struct Cursor {
    Request r;
    int b, row_tile, head, tile;
};

__device__ __noinline__ inline void next_unit(const TreeArgs &a, Cursor &c, int m_rows) {
    c.tile = 0;
    if (++c.head < a.n_kv) return;
    c.head = 0;
    if (++c.row_tile < c.r.row_tiles) return;
    c.row_tile = 0;
    do {
        if (++c.b >= a.n_requests) return;
        c.r = request(a, c.b, m_rows);
    } while (c.r.row_tiles == 0);
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

// A CTA's share of the tiles: [lo, hi) of total, dealt to `used` CTAs, and where it
// starts. false: it has none. scratch: 2 kWarps + 2 words. Every thread calls it.
struct Share {
    long long lo, hi, total, used;
    Cursor start;
};

// x * y / z, in 32 bits where they will do.
__device__ __forceinline__ long long scaled(long long x, long long y, long long z) {
    const long long p = x * y;
    return p >> 32 == 0 ? (long long)((uint32_t)p / (uint32_t)z) : p / z;
}

template <int kThreads>
__device__ inline bool find_share(const TreeArgs &a, int m_rows, long long *scratch, Share &s) {
    constexpr int kWarps = kThreads / 32;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    // tiles of the requests tid, tid + kThreads, ..; of the first of them and its prefix sum, which is all in most calls
    Request mine{};
    long long n0 = 0, sum = 0;
    for (int b = tid; b < a.n_requests; b += kThreads) {
        const Request r = request(a, b, m_rows);
        const long long n = (long long)r.row_tiles * r.key_tiles * a.n_kv;
        if (b == tid) mine = r, n0 = n;
        sum += n;
    }
    long long upto = n0, all = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long v = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += v;
    }
    if (a.n_requests > kThreads) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
    }
    if (lane == 31) scratch[2 + warp] = upto, scratch[2 + kWarps + warp] = a.n_requests > kThreads ? all : upto;
    if (tid == 0) scratch[0] = -1;
    __syncthreads();
    s.total = 0;
    long long before = 0;
    for (int w = 0; w < kWarps; ++w) s.total += scratch[2 + kWarps + w];
    s.used = min((long long)gridDim.x, s.total);
    if (blockIdx.x >= s.used) return false;
    s.lo = scaled(s.total, blockIdx.x, s.used);
    s.hi = scaled(s.total, blockIdx.x + 1, s.used);
    for (int b0 = 0; b0 < a.n_requests; b0 += kThreads) {    // ends in the chunk that holds tile lo < total
        const int b = b0 + tid;
        if (b0 > 0) {
            n0 = 0;
            if (b < a.n_requests) {
                mine = request(a, b, m_rows);
                n0 = (long long)mine.row_tiles * mine.key_tiles * a.n_kv;
            }
            upto = n0;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long v = __shfl_up_sync(0xffffffffu, upto, o);
                if (lane >= o) upto += v;
            }
            __syncthreads();
            if (lane == 31) scratch[2 + warp] = upto;
            __syncthreads();
        }
        for (int w = 0; w < warp; ++w) upto += scratch[2 + w];
        upto += before;
        if (upto - n0 <= s.lo && s.lo < upto) scratch[0] = b, scratch[1] = upto - n0;
        for (int w = 0; w < kWarps; ++w) before += scratch[2 + w];
        __syncthreads();
        if (scratch[0] >= 0) break;
    }
    if (scratch[0] < 0) return false;                        // not reached
    s.start.b = (int)scratch[0];
    s.start.r = request(a, s.start.b, m_rows);
    const long long at = s.lo - scratch[1], unit = scaled(at, 1, s.start.r.key_tiles);
    s.start.tile = (int)(at - unit * s.start.r.key_tiles);
    s.start.row_tile = (int)scaled(unit, 1, a.n_kv);
    s.start.head = (int)(unit - (long long)s.start.row_tile * a.n_kv);
    return true;
}

// Parts of the unit at cursor c whose tile is the share's tile i and the last of
// the share: CTA floor(((x + 1) used - 1) / total) has tile x.
__device__ __forceinline__ int parts_of(const Share &s, const Cursor &c, int i) {
    const long long x = s.lo + i + (c.r.key_tiles - 1 - c.tile);
    const long long p = (x + 1) * s.used - 1;
    return (int)scaled(p, 1, s.total) - (int)blockIdx.x + 1;
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
