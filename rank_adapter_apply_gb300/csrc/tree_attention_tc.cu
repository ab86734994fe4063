// lora_tree_attention, row tiles of 128 on the 5th-generation tensor cores.
//
// Scores S = Q K^T (128 rows x 64 keys) and O += P V are tcgen05 products with
// their accumulators in tensor memory; P goes back into S's columns in bf16 and is
// the A operand of the second product from there. 192 threads:
//   warps 0-3  softmax: thread = row = tensor-memory lane, so the running maximum
//              and sum need no exchange; at a unit's end they write its result;
//   warp 4     loads: TMA boxes of up to 64 cache rows of a page into a ring of
//              16 KB items (K and V alternate), Q at a unit's start;
//   warp 5     one thread issues the products.
// S is double-buffered: the scores of tile i + 1 are formed while the softmax of
// tile i runs. Two CTAs fit an SM (256 tensor-memory columns and 113 KB each).
//
// The maximum is a reference that moves only when a row's scores pass it by 2^8:
// P and l share it, so the quotient does not depend on it, P stays below 2^8 (bf16
// has the range) and O in tensor memory is rescaled a few times in a unit at most.
//
// A weight of zero times an infinity or NaN is NaN, so a V row that is not finite
// may not meet a row that skips it. Only tree keys, and what lies past the last
// key, can be skipped: in tiles with such keys the softmax warps look through V,
// clear the rows that are not finite, and the rows that see one of them add it in
// fp32 at the end of the unit.
//
// What bounds it: 4 requests of up to 64 nodes, ctx 32768, 64 heads over 8 take 202 us
// with the join in a graph, 971 TFLOP/s. The product pipe is busy for 63 % of it (64 keys at a time,
// Q is read from shared memory again for each), and a CTA's chain scores, softmax, weights
// to tensor memory, second product, next scores is as long as the two CTAs of an SM can
// hide. 32 requests of up to 16 nodes, ctx 4096, 32 heads over 8: 89 us, 4.7 TB/s of keys
// and values, with half of the 128 lanes empty.
#include "tree_common.cuh"
#include "tc_util.cuh"
#include "tensor_map.cuh"

#include <atomic>

namespace lora {
namespace tree {
namespace {

constexpr int kRows = 128;                     // lanes of an accumulator; rows of a tile: whole nodes, at most this
constexpr int kThreads = 192;
constexpr int kItems = 5;                      // ring of K and V items
constexpr int kMeta = 4;                       // ring of the tiles' masks
constexpr uint32_t kWaitLimit = 1u << 18;       // polls, of some microseconds each: about a second

template <int DP>
struct Tc {
    static constexpr int kHalves = DP / 64;    // columns in blocks of 64: rows of 128 bytes, 128-byte swizzle
    static constexpr int kItem = kTileKeys * DP * 2, kQ = kRows * DP * 2;
    static constexpr int kSmem = kQ + kItems * kItem;
};

struct Meta {
    uint32_t valid[2];                         // keys that are there
    uint32_t first;                            // first tile of a unit in this share
};

struct TcArgs {
    CUtensorMap q, k, v;                       // boxes of 64 columns: q {group heads, whole nodes}, k, v {box rows}
    TreeArgs a;
    Plan plan;
    int box;                                   // cache rows of a box: a power of two, 8..64
    int slot_first;                            // order of the cache maps' dimensions: columns, place, head, page (else
                                               // columns, head, place, page)
};

__device__ __forceinline__ void tma_3d(uint32_t dst, const CUtensorMap *map, int c0, int c1, int c2, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
        ::"r"(dst), "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void tma_4d(uint32_t dst, const CUtensorMap *map, int c0, int c1, int c2, int c3,
                                       uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
        "[%6];" ::"r"(dst), "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(smem_u32(bar)) : "memory");
}

__device__ __noinline__ bool wait_long(uint64_t *bar, uint32_t parity, volatile int *err) {
    if (*err) return false;
    if (mbar_wait_bounded(bar, parity, kWaitLimit)) return true;
    *err = 1;
    return false;
}

// o[0..31] += the weight times V of every key of tiles first .. c.tile that row
// `node` sees and whose V row is not finite (columns d .. d + 31).
__device__ __noinline__ void add_poison(const TreeArgs &a, const Cursor &c, int first, int node, int head, int d, float c2,
                                        float m, float *o) {
    const __nv_bfloat16 *q =
        static_cast<const __nv_bfloat16 *>(a.q) + (c.r.start + node) * a.q_token + (long long)head * a.q_head;
    Cursor at = c;
    for (at.tile = first; at.tile <= c.tile; ++at.tile) {
        const uint64_t seen = seen_keys(a, c.r, node, at.tile * kTileKeys);
        for (int k = 0; k < kTileKeys; ++k) {
            const long long off = seen >> k & 1 ? key_offset(a, at, k) : -1;
            if (off < 0) continue;
            const __nv_bfloat16 *kp = static_cast<const __nv_bfloat16 *>(a.k_cache) + off + (long long)c.head * a.c_head;
            const __nv_bfloat16 *vp = static_cast<const __nv_bfloat16 *>(a.v_cache) + off + (long long)c.head * a.c_head;
            bool bad = false;
            float dot = 0.f;
            for (int e = 0; e < a.head_dim; ++e) {
                bad = bad || !isfinite(to_f32(vp[e]));
                dot = fmaf(to_f32(q[e]), to_f32(kp[e]), dot);
            }
            const float x = a.scale < 0.f ? -dot : a.scale == 0.f ? 0.f : dot;
            const float weight = exp2_fast(fmaf(x, c2, m == -INFINITY ? 0.f : -m));
            if (!bad || weight == 0.f) continue;
            for (int e = 0; e < 32 && d + e < a.head_dim; ++e) o[e] = fmaf(weight, to_f32(vp[d + e]), o[e]);
        }
    }
}

// CTAs whose bounded waits gave up (lora_step_wait_timeouts).
__device__ unsigned g_gave_up = 0;

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
        "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};"
        ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
          "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]),
          "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]),
          "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}

// B operand with its rows (N) contiguous: 64 of them in the 128 bytes of a k, eight
// ks 1024 bytes further, the next 64 rows one block of the tile further.
__device__ __forceinline__ uint64_t desc_n_major(uint32_t addr, uint32_t block_bytes) {
    uint64_t d = 0;
    d |= (uint64_t)((addr & 0x3FFFFu) >> 4);
    d |= (uint64_t)((block_bytes >> 4) & 0x3FFFu) << 16;
    d |= (uint64_t)((1024u >> 4) & 0x3FFFu) << 32;
    d |= (uint64_t)1 << 46;
    d |= (uint64_t)tc::kSwz128 << 61;
    return d;
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
    uint64_t v;
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(lo), "f"(hi));
    return v;
}
__device__ __forceinline__ void unpair(uint64_t v, float &lo, float &hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

// Whether a 16-byte piece of bf16 holds an infinity or NaN.
__device__ __forceinline__ bool odd_piece(const uint4 &v) {
    return ((((v.x & 0x7f807f80u) + 0x00800080u) | ((v.y & 0x7f807f80u) + 0x00800080u) |
             ((v.z & 0x7f807f80u) + 0x00800080u) | ((v.w & 0x7f807f80u) + 0x00800080u)) & 0x80008000u) != 0;
}

template <int DP>
__global__ void __launch_bounds__(kThreads, 2) tree_tc_kernel(const __grid_constant__ TcArgs args) {
    using C = Tc<DP>;
    extern __shared__ __align__(1024) unsigned char smem[];
    __shared__ uint64_t full[kItems], empty[kItems], meta_full[kMeta], s_full[2], p_ready[2], pv_done[2], q_full, drained, looked;
    __shared__ int poison_at[2];                       // 1 + the last tile (even, odd) whose V had a row that is not finite
    __shared__ Meta meta[kMeta];
    __shared__ long long scratch[kScratch + kThreads / 32];
    __shared__ uint32_t tmem_base;
    __shared__ int error;
    volatile int *err = &error;

    const TreeArgs &a = args.a;
    const Plan &plan = args.plan;
    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), group = a.n_heads / a.n_kv;
    const int rows = kRows / group * group;            // of a tile
    grid_dependency_wait();
    grid_launch_dependents();                          // the join kernel waits for this grid's end itself
    if (tid == 0) plan.seg[blockIdx.x] = make_int4(0, 0, 0, 0);
    Share share;
    if (!find_share<kThreads>(a, rows, scratch, share)) return;
    const int n_tiles = (int)(share.hi - share.lo);
    if (tid == 0) {
        for (int i = 0; i < kItems; ++i) mbar_init(&full[i], 1), mbar_init(&empty[i], 1);
        for (int i = 0; i < kMeta; ++i) mbar_init(&meta_full[i], 1);
        for (int i = 0; i < 2; ++i) mbar_init(&s_full[i], 1), mbar_init(&p_ready[i], 4), mbar_init(&pv_done[i], 1);
        mbar_init(&q_full, 1);
        mbar_init(&drained, 1);
        mbar_init(&looked, 4);
        error = 0;
        poison_at[0] = poison_at[1] = 0;
        fence_mbar_init();
        tc::prefetch_tensormap(&args.q);
        tc::prefetch_tensormap(&args.k);
        tc::prefetch_tensormap(&args.v);
    }
    if (warp == 5) {
        tc::tmem_alloc(&tmem_base, 256);
        tc::tmem_relinquish();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = tmem_base, tmem_o = tmem + 128;   // S of the two buffers at columns 0 and 64, O at 128
    const uint32_t q_at = smem_u32(smem), ring = q_at + C::kQ;
    auto wait = [&](uint64_t *bar, uint32_t phase) -> bool {
        return mbar_try_wait(bar, phase & 1u) || wait_long(bar, phase & 1u, err);
    };
    // A wait of a warp: where it gave up for one lane, all leave.
    auto together = [](bool ok) -> bool { return __all_sync(0xffffffffu, ok); };
    // Items are loaded in the order in which the products take them, K0 K1 V0 K2 V1 .., round and round the ring; a
    // role steps through them with a place and the parity of its round.
    auto step = [](int &place, uint32_t &round) {
        if (++place == kItems) place = 0, round ^= 1u;
    };
    auto place_v = [&](int i) { return (i + 1 < n_tiles ? 2 * i + 2 : 2 * i + 1) % kItems; };
    auto round_v = [&](int i) { return (uint32_t)((i + 1 < n_tiles ? 2 * i + 2 : 2 * i + 1) / kItems); };

    if (warp == 4) {
        // ---------------- loads: lane b < 64 / box loads box b of a tile ----------------
        // The lanes hold the pages of 32 boxes of the request in a row (a tile's boxes lie in one such run): the run
        // in use, the one after it, whose reads are in flight meanwhile, and the first, where the next head begins.
        const int boxes = kTileKeys / args.box;
        Cursor u = share.start;
        struct Run {
            int page, place;                           // page -1: no such box
        };
        auto read_run = [&](int run) -> Run {
            // unsigned: the run after the last may begin past 2^31
            const uint32_t p = ((uint32_t)run * 32 + lane) * (uint32_t)args.box, at = p / (uint32_t)a.page_size;
            return {p < (uint32_t)u.r.keys ? a.page_table[u.b * a.table_stride + at] : -1, (int)(p - at * (uint32_t)a.page_size)};
        };
        int run_b = -1, run_at = 0;                    // request, and number of the run in use
        Run now{}, ahead{}, head_run{};
        int at = 0, units = 0, issued = 0, k_at = 0;   // the ring's next place, and that of the last K
        uint32_t round = 0, k_round = 0;
        struct Box {
            int page, c1, c2;                          // the cache maps' outer coordinates
        } last{};                                      // of the tile whose V is still to be loaded
        auto load = [&](const CUtensorMap *map, const Box &b) -> bool {
            if (!together(wait(&empty[at], round ^ 1u))) return false;   // at once in the first round
            if (lane == 0) mbar_arrive_expect_tx(&full[at], C::kItem);
            __syncwarp();
            if (lane < boxes) {
                const uint32_t dst = ring + at * C::kItem + lane * args.box * 128;
#pragma unroll
                for (int h = 0; h < C::kHalves; ++h)
                    tma_4d(dst + h * (C::kItem / C::kHalves), map, h * 64, b.c1, b.c2, b.page, &full[at]);
            }
            step(at, round);
            ++issued;
            return true;
        };
        int i = 0;
        for (; i < n_tiles; ++i) {
            const int box0 = u.tile * boxes, run = box0 >> 5;
            if (run_b != u.b || run != run_at) {
                if (run_b != u.b) head_run = read_run(0);
                now = run == 0 ? head_run : run_b == u.b && run == run_at + 1 ? ahead : read_run(run);
                run_b = u.b;
                run_at = run;
                ahead = read_run(run + 1);
            }
            const int from = (box0 & 31) + lane;       // lanes past the tile's boxes read a lane that nobody uses
            int page = __shfl_sync(0xffffffffu, now.page, from & 31);
            const int place = __shfl_sync(0xffffffffu, now.place, from & 31);
            uint32_t lo = ~0u, hi = ~0u;               // the tile's keys that are there
            const bool whole = lane >= boxes ||
                               (page >= 0 && page < (int)a.n_pages && (box0 + lane + 1) * args.box <= u.r.keys);
            if (!__all_sync(0xffffffffu, whole)) {
                // rows of the box that hold keys; a page outside the cache reads zeros
                int n = lane < boxes ? min(max(u.r.keys - (box0 + lane) * args.box, 0), args.box) : 0;
                if (n == 0 || page < 0 || page >= a.n_pages) page = (int)a.n_pages, n = 0;
                const uint64_t bits = n == 64 ? ~0ull : ((1ull << n) - 1) << (lane * args.box & 63);
                lo = __reduce_or_sync(0xffffffffu, (uint32_t)bits);
                hi = __reduce_or_sync(0xffffffffu, (uint32_t)(bits >> 32));
            }
            const Box here{page, args.slot_first ? place : u.head, args.slot_first ? u.head : place};
            const bool first = i == 0 || u.tile == 0;
            if (first) {
                // the last scores of the unit before have been formed: Q may be overwritten
                if (i > 0 && !together(wait(&empty[k_at], k_round))) break;
                if (lane == 0) {
                    mbar_arrive_expect_tx(&q_full, rows * DP * 2);
                    for (int h = 0; h < C::kHalves; ++h)
                        tma_3d(q_at + h * (kRows * 128), &args.q, h * 64, u.head * group,
                               u.r.start + u.row_tile * (rows / group), &q_full);
                }
                ++units;
            }
            k_at = at, k_round = round;
            if (!load(&args.k, here)) break;
            if (lane == 0) {
                Meta &m = meta[i % kMeta];
                m.valid[0] = lo;
                m.valid[1] = hi;
                m.first = first;
                tc::mbar_arrive(&meta_full[i % kMeta]);
            }
            if (i > 0 && !load(&args.v, last)) break;
            last = here;
            next_tile(a, u, rows);
        }
        if (i == n_tiles) load(&args.v, last);
        // no copy is in flight when the CTA ends
        for (int j = max(issued - kItems, 0); j < issued; ++j)
            mbar_wait_bounded(&full[j % kItems], (uint32_t)(j / kItems) & 1u, kWaitLimit);
        if (units > 0) mbar_wait_bounded(&q_full, (uint32_t)(units - 1) & 1u, kWaitLimit);
    } else if (warp == 5) {
        // ---------------- products ----------------
        // The whole warp runs the loop, so that addresses and descriptors stay in uniform registers; one lane's
        // instructions count.
        const uint32_t lead = tc::elect_one(), tm = __shfl_sync(0xffffffffu, tmem, 0), tm_o = tm + 128;
        constexpr uint32_t idesc_s = tc::idesc_bf16(kRows, kTileKeys);
        constexpr uint32_t idesc_o = tc::idesc_bf16(kRows, DP) | (1u << 16);    // B (V) with N contiguous
        // descriptors of the operands' first slices; slices and places differ in the address field alone
        const uint64_t q_desc = tc::smem_desc(q_at, 128, tc::kSwz128), k_desc = tc::smem_desc(ring, 128, tc::kSwz128);
        const uint64_t v_desc = desc_n_major(ring, C::kItem / C::kHalves);
        const int n = __shfl_sync(0xffffffffu, n_tiles, 0);
        int at = 0, units = 0;
        uint32_t round = 0;
        for (int i = 0; i <= n; ++i) {
            if (i < n) {
                const bool ok = wait(&full[at], round) && wait(&meta_full[i % kMeta], (uint32_t)(i / kMeta)) &&
                                (!meta[i % kMeta].first || wait(&q_full, (uint32_t)units++)) &&
                                (i < 2 || wait(&pv_done[i & 1], (uint32_t)((i - 2) >> 1)));      // P of tile i - 2 was read
                if (!together(ok)) break;
                tc::fence_after_sync();
                const uint64_t kd = k_desc + (uint64_t)(at * (C::kItem >> 4));
#pragma unroll
                for (int k = 0; k < DP / 16; ++k)
                    tc::mma_bf16_lead(tm + (i & 1) * 64, q_desc + (k >> 2) * (kRows * 128 >> 4) + (k & 3) * 2,
                                 kd + (k >> 2) * (C::kItem / 2 >> 4) + (k & 3) * 2, idesc_s, k > 0, lead);
                tc::mma_commit_lead(&empty[at], lead);
                tc::mma_commit_lead(&s_full[i & 1], lead);
                step(at, round);
            }
            if (i > 0) {
                const int t = i - 1;
                if (!together(wait(&p_ready[t & 1], (uint32_t)(t >> 1)) && wait(&full[at], round))) break;
                tc::fence_after_sync();
                const uint32_t more = meta[t % kMeta].first == 0;
                const uint64_t vd = v_desc + (uint64_t)(at * (C::kItem >> 4));
#pragma unroll
                for (int k = 0; k < kTileKeys / 16; ++k)
                    tc::mma_bf16_tmem_a_lead(tm_o, tm + (t & 1) * 64 + k * 8, vd + k * (2048 >> 4), idesc_o, more | (k > 0),
                                                 lead);
                tc::mma_commit_lead(&empty[at], lead);
                tc::mma_commit_lead(&pv_done[t & 1], lead);
                step(at, round);
            }
        }
        // every product is done before tensor memory is freed
        tc::mma_commit_lead(&drained, lead);
        mbar_wait_bounded(&drained, 0, kWaitLimit);
    } else {
        // ---------------- softmax: thread = row ----------------
        const uint32_t lanes = (uint32_t)(warp * 32) << 16;
        const float c2 = (a.scale == 0.f ? 1.f : fabsf(a.scale)) * 1.4426950408889634f;   // scores in powers of two
        Cursor c = share.start;
        float m = -INFINITY, l = 0.f;                  // m: the reference, in powers of two
        int seg_first = c.tile, node = 0, head = 0;
        uint32_t looks = 0;                            // tiles whose V was looked through
        bool poison = false, idle = false;             // idle: no row of this warp exists
        for (int i = 0; i < n_tiles; ++i) {
            const bool first = i == 0 || c.tile == 0;
            if (first) {
                m = -INFINITY, l = 0.f, seg_first = c.tile, poison = false;
                const int row = c.row_tile * rows + tid;
                node = tid < rows ? row / group : c.r.nodes;
                head = c.head * group + row % group;
                idle = __all_sync(0xffffffffu, node >= c.r.nodes);
            }
            if (!together(wait(&meta_full[i % kMeta], (uint32_t)(i / kMeta)) && wait(&s_full[i & 1], (uint32_t)(i >> 1)))) break;
            tc::fence_after_sync();
            const uint64_t there = meta[i % kMeta].valid[0] | (uint64_t)meta[i % kMeta].valid[1] << 32;
            const int p0 = c.tile * kTileKeys;
            if (!idle) {
                uint32_t raw[64];
                tc::tmem_ld64_sync(tmem + lanes + (i & 1) * 64, raw);
                float(&s)[64] = reinterpret_cast<float(&)[64]>(raw);
                if (a.scale <= 0.f) {
#pragma unroll
                    for (int k = 0; k < 64; ++k) s[k] = a.scale < 0.f ? -s[k] : 0.f;
                }
                if (there != ~0ull || p0 + kTileKeys > c.r.ctx) {
                    const uint64_t seen = node < c.r.nodes ? seen_keys(a, c.r, node, p0) & there : 0;
                    const uint32_t lo = (uint32_t)seen, hi = (uint32_t)(seen >> 32);
#pragma unroll
                    for (int k = 0; k < 32; ++k) {
                        if (!(lo >> k & 1)) s[k] = -INFINITY;
                        if (!(hi >> k & 1)) s[k + 32] = -INFINITY;
                    }
                }
                float top = s[0], top2 = s[1];
#pragma unroll
                for (int k = 2; k < 64; k += 2) top = fmaxf(top, s[k]), top2 = fmaxf(top2, s[k + 1]);
                top = fmaxf(top, top2) * c2;
                const bool move = top > m + 8.f;
                if (__any_sync(0xffffffffu, move)) {
                    const float f = move ? exp2_fast(m - top) : 1.f;
                    if (move) m = top;
                    l *= f;
                    if (!first) {                          // O of the tiles before, once it is complete
                        if (!together(wait(&pv_done[(i - 1) & 1], (uint32_t)((i - 1) >> 1)))) break;
                        tc::fence_after_sync();
#pragma unroll 1
                        for (int d = 0; d < DP; d += 32) {
                            uint32_t o[32];
                            tc::tmem_ld32_sync(tmem_o + lanes + d, o);
#pragma unroll
                            for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
                            tmem_st32(tmem_o + lanes + d, o);
                        }
                    }
                }
                const float minus = m == -INFINITY ? 0.f : -m;
                const uint64_t cc = pair(c2, c2), mm = pair(minus, minus);
                uint32_t p[32];
                uint64_t sums[2] = {pair(l, 0.f), pair(0.f, 0.f)};
#pragma unroll
                for (int k = 0; k < 32; ++k) {
                    float e0, e1;
                    unpair(fma2(pair(s[2 * k], s[2 * k + 1]), cc, mm), e0, e1);
                    e0 = exp2_fast(e0);
                    e1 = exp2_fast(e1);
                    sums[k & 1] = add2(sums[k & 1], pair(e0, e1));
                    // weights to bf16 for the second product: 2^-9 relative, below the output's own rounding; their sum
                    // l stays in fp32 and unrounded
                    p[k] = pack_bf16(e0, e1);
                }
                float l0, l1;
                unpair(add2(sums[0], sums[1]), l0, l1);
                l = l0 + l1;
                tmem_st32(tmem + lanes + (i & 1) * 64, p);
                tc::tmem_st_wait();
            }
            if (p0 + kTileKeys > min(c.r.ctx, c.r.keys)) {
                // some row may skip a key of this tile: no V row with an infinity or NaN in it may stay
                const int vp = place_v(i);
                if (!together(wait(&full[vp], round_v(i)))) break;
                // two threads for a row
                constexpr int kPieces = DP / 16;
                unsigned char *v = smem + C::kQ + vp * C::kItem + (tid >> 1) * 128 +
                                   (tid & 1) * (C::kHalves == 2 ? C::kItem / 2 : 64);
                bool bad = false;
#pragma unroll
                for (int k = 0; k < kPieces; ++k) bad = bad || odd_piece(*reinterpret_cast<const uint4 *>(v + k * 16));
                bad = __shfl_xor_sync(0xffffffffu, (int)bad, 1) || bad;
                if (bad) {
#pragma unroll
                    for (int k = 0; k < kPieces; ++k) *reinterpret_cast<uint4 *>(v + k * 16) = make_uint4(0, 0, 0, 0);
                    if (there >> (tid >> 1) & 1) poison_at[i & 1] = i + 1;
                }
                tc::fence_proxy_async_smem();
                // the four warps meet at a barrier whose wait is bounded, too: one of them may have given up
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&looked);
                if (!together(wait(&looked, looks++))) break;
                poison = poison || *reinterpret_cast<volatile int *>(&poison_at[i & 1]) == i + 1;
            }
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&p_ready[i & 1]);       // one of a warp: arrivals at one address queue up

            if (c.tile + 1 == c.r.key_tiles || i + 1 == n_tiles) {
                // ---- the unit or the share ends: write
                const bool starts = seg_first == 0, ends = c.tile + 1 == c.r.key_tiles;
                if (!together(wait(&pv_done[i & 1], (uint32_t)(i >> 1)))) break;
                tc::fence_after_sync();
                // a row without keys is 0; one whose scores are all NaN also has m = -inf, but its l is NaN
                const bool mine = node < c.r.nodes, none = l == 0.f, done = starts && ends;
                const long long token = c.r.start + node, slot = 2ll * blockIdx.x + (starts ? 1 : 0);
                const float inv = !done ? 1.f : l > 0.f ? 1.f / l : l;
                __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(a.out) + token * a.o_token + head * a.o_head;
                float *part = plan.part + (slot * kRows + tid) * DP;
#pragma unroll 1
                for (int d = 0; d < DP; d += 32) {
                    uint32_t o[32];
                    tc::tmem_ld32_sync(tmem_o + lanes + d, o);
                    if (poison && mine) {
                        float t[32];
#pragma unroll
                        for (int k = 0; k < 32; ++k) t[k] = __uint_as_float(o[k]);
                        add_poison(a, c, max(seg_first, min(c.r.ctx, c.r.keys) / kTileKeys), node, head, d, c2, m, t);
#pragma unroll
                        for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(t[k]);
                    }
                    if (mine && done) {
#pragma unroll
                        for (int k = 0; k < 32; k += 8) {
                            if (d + k >= a.head_dim) break;
                            float v[8];
#pragma unroll
                            for (int e = 0; e < 8; ++e) v[e] = none ? 0.f : __uint_as_float(o[k + e]) * inv;
                            *reinterpret_cast<uint4 *>(out + d + k) =
                                make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]),
                                           pack_bf16(v[6], v[7]));
                        }
                    } else if (mine) {
#pragma unroll
                        for (int k = 0; k < 32; k += 4)
                            *reinterpret_cast<uint4 *>(part + d + k) = make_uint4(o[k], o[k + 1], o[k + 2], o[k + 3]);
                    }
                    __syncwarp();
                }
                if (mine && done && a.lse)
                    a.lse[token * a.n_heads + head] = none ? -INFINITY : m * 0.6931471805599453f + logf(l);
                if (mine && !done) plan.stat[slot * kRows + tid] = make_float2(m, l);
                if (tid == 0 && starts && !ends)
                    plan.seg[blockIdx.x] = make_int4(c.b, c.row_tile, c.head, parts_of(share, c, i));
                tc::fence_before_sync();
            }
            __syncwarp();
            next_tile(a, c, rows);
        }
    }
    tc::fence_before_sync();
    __syncthreads();
    if (tid == 0 && error) atomicAdd(&g_gave_up, 1u);
    if (warp == 5) {
        tc::fence_after_sync();
        tc::tmem_dealloc(tmem, 256);
    }
}

// A bf16 map of `rank` dimensions, boxes of 64 columns, 128-byte swizzle. The
// stride of a dimension of one element is never used: any legal one stands in.
bool encode(CUtensorMap *map, const void *base, int rank, const cuuint64_t *dims, const long long *strides,
            const cuuint32_t *box) {
    cuuint64_t bytes[3];
    const cuuint32_t ones[4] = {1, 1, 1, 1};
    for (int i = 0; i + 1 < rank; ++i) bytes[i] = dims[i + 1] == 1 ? 16 : (cuuint64_t)strides[i] * 2;
    const auto fn = map_encoder();
    return fn && fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void *>(base), dims, bytes, box, ones,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Cache rows of a box: what divides a page and the tile.
int box_of(int page_size) {
    int box = kTileKeys;
    while (page_size % box) box /= 2;
    return box;
}

template <int DP>
cudaError_t launch(const TreeArgs &a, const Plan &plan, cudaStream_t st) {
    static std::atomic<uint64_t> ready{0};
    if (!device_bit(ready)) {
        const cudaError_t e =
            cudaFuncSetAttribute(tree_tc_kernel<DP>, cudaFuncAttributeMaxDynamicSharedMemorySize, Tc<DP>::kSmem);
        if (e != cudaSuccess) return e;
        set_device_bit(ready);
    }
    const int group = a.n_heads / a.n_kv;
    TcArgs args;
    args.a = a;
    args.plan = plan;
    args.box = box_of(a.page_size);
    const cuuint64_t q_dims[] = {(cuuint64_t)a.head_dim, (cuuint64_t)a.n_heads, (cuuint64_t)a.n_tokens};
    const long long q_strides[] = {a.q_head, a.q_token};
    const cuuint32_t q_box[] = {64, (cuuint32_t)group, (cuuint32_t)(kRows / group)};
    args.slot_first = a.c_slot < a.c_head;
    const cuuint64_t heads = a.n_kv, places = a.page_size;
    const cuuint32_t box = args.box;
    const bool sf = args.slot_first;
    const cuuint64_t c_dims[] = {(cuuint64_t)a.head_dim, sf ? places : heads, sf ? heads : places, (cuuint64_t)a.n_pages};
    const long long c_strides[] = {sf ? a.c_slot : a.c_head, sf ? a.c_head : a.c_slot, a.c_page};
    const cuuint32_t c_box[] = {64, sf ? box : 1, sf ? 1 : box, 1};
    if (!encode(&args.q, a.q, 3, q_dims, q_strides, q_box) || !encode(&args.k, a.k_cache, 4, c_dims, c_strides, c_box) ||
        !encode(&args.v, a.v_cache, 4, c_dims, c_strides, c_box))
        return cudaErrorNotSupported;
    return launch_step(tree_tc_kernel<DP>, dim3(plan.ctas), dim3(kThreads), Tc<DP>::kSmem, 1, st, args);
}

}  // namespace

cudaError_t read_timeouts(unsigned *count) { return cudaMemcpyFromSymbol(count, g_gave_up, sizeof *count); }

// Whether strides s of dimensions of n elements, innermost first, rise and are
// those of a tensor map: 0 < s < 2^40 bytes.
static bool rising(const long long *s, const long long *n, int count) {
    long long last = 0;
    for (int i = 0; i < count; ++i) {
        if (n[i] == 1) continue;
        if (s[i] <= last || s[i] >= 1ll << 39) return false;
        last = s[i];
    }
    return true;
}

// Pages in boxes of eight rows or more (the swizzle's period), whole nodes in a
// tile, a query's heads within its token, pages outermost in the cache.
bool tc_takes(const TreeArgs &a) {
    const int group = a.n_heads / a.n_kv;
    if (box_of(a.page_size) < 8 || group > kRows || a.n_pages < 1 || a.n_pages >= INT32_MAX) return false;
    const long long q[] = {a.q_head, a.q_token}, qn[] = {a.n_heads, a.n_tokens};
    const bool sf = a.c_slot < a.c_head;
    const long long c[] = {sf ? a.c_slot : a.c_head, sf ? a.c_head : a.c_slot, a.c_page};
    const long long cn[] = {sf ? a.page_size : a.n_kv, sf ? a.n_kv : a.page_size, a.n_pages};
    return rising(q, qn, 2) && rising(c, cn, 3);
}

int tc_rows(const TreeArgs &a) { return kRows / (a.n_heads / a.n_kv) * (a.n_heads / a.n_kv); }

cudaError_t launch_tc(const TreeArgs &a, const Plan &plan, cudaStream_t st) {
    return a.head_dim <= 64 ? launch<64>(a, plan, st) : launch<128>(a, plan, st);
}

}  // namespace tree
}  // namespace lora
