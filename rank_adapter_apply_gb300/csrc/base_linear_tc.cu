// lora_base_linear on the 5th-generation tensor cores.
//
// A CTA takes 128 rows of W, up to N tokens and, as one of the CTAs of a cluster, a
// range of the columns. Blocks of 256 columns of the 4-bit words and of x come by
// TMA into a ring; x is the B operand as it lies. Thread = row = tensor-memory
// lane: the words of its row become (n - z) / 64 in registers, exact in bf16, and go to
// tensor memory as the A operand. The products within one group are exact, their sum is
// fp32; it comes back to the row's thread, which scales it into its fp32 accumulators. So
// no weight is ever rounded.
//
// An x in fp32 is cut by eight more warps into three bf16 parts of eight bits each that
// sum to it exactly from 2^-103 on, where all three are normal numbers; of a smaller x
// less than 2^-125 is lost. They lie side by side as three times the tokens in one
// product, and their sums meet in the row's accumulators.
//
// S sets of four warps take units of up to 128 columns in turn, each with its own A and
// D in tensor memory, so the reads, the conversion, the products and the sums of S units
// overlap. One warp issues the copies, one the products. At the end the sets' and the
// cluster's parts are added in a fixed order.
//
// What bounds it: 64x5120x8192 with groups of 64 takes 12.6 us (1.9 TB/s of words, 426
// TFLOP/s; the same on mma.sync 29.9 us), 17x14336x4096 with groups of 32 and zeros 15.8
// us (23.4). No pipe of a busy SM is above a half: issue slots 45 %, integer pipe 35 %,
// products 23 % of 64x5120x8192. It is the chain of a unit, reading, ten instructions for
// eight values, tensor memory, products, sums, that two or three sets do not hide, and a
// third set has no room for its D. 128 rows to a CTA leave SMs idle (4096 rows: 128 CTAs
// of 152), and the launch, the first loads and the cluster's end take 4 us of a call. In
// fp32 64x5120x8192 takes 35 us: cutting x, for each 128 rows again, is its pace. Above 64
// tokens W is converted again for every 64 (32 in fp32).
#include "base_linear.cuh"
#include "tc_util.cuh"
#include "tensor_map.cuh"

#include <algorithm>

namespace lora {
namespace linear {
namespace {

using namespace step;

constexpr int kRows = 128;
constexpr uint32_t kWaitLimit = 1u << 18;       // polls, of some microseconds each: about a second

template <typename X_, int N_, int S_>
struct TcTile {
    using X = X_;                                                   // type of x, scales and y
    static constexpr int N = N_, S = S_;                            // tokens, sets of warps
    static constexpr int kParts = sizeof(X) == 4 ? 3 : 1;           // bf16 parts of x
    static constexpr int ND = kParts * N;                           // columns of D, rows of B: the parts side by side
    static constexpr int kWBytes = kRows * 128, kStage = kWBytes + ND * 512;    // 256 columns of W, and of x
    static constexpr int kStages = 192 * 1024 / kStage, kSmem = kStages * kStage;
    static constexpr int kCutters = kParts == 3 ? 8 : 0;             // warps that cut x
    static constexpr int kThreads = (4 * S + 2 + kCutters) * 32;
    static_assert(S * N * kRows * 4 <= kSmem, "the sets' sums take the ring's place");
};

struct TcArgs {
    CUtensorMap w, x;                                               // boxes: 128 bytes x 128 rows; bf16: 64 columns x N tokens
    LinearArgs a;
    int cluster, x_vec, y_vec, group_vec;                                  // group_vec: a unit's scales, zeros in one load
};

__device__ unsigned g_gave_up = 0;

__device__ __noinline__ bool wait_long(uint64_t *bar, uint32_t parity, volatile int *err) {
    if (*err) return false;
    if (mbar_wait_bounded(bar, parity, kWaitLimit)) return true;
    *err = 1;
    return false;
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
        ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
          "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

// The eight 4-bit values n of a word less the zero z, over 64, in bf16 and in order. Bits v < 256 of a bf16 are the
// number v 2^-133, subnormal or not, so a byte and a byte of zero are a value with no more ado: n 2^-133 2^127, or, of
// the byte's upper half, 16 n 2^-133 2^123, and minus_z = -z / 64, twice, added in the same exact operation. (With masks
// and an exponent put on by hand it took 13 instructions for a word, not 10: 64x5120x8192 14.8 -> 12.7 us.)
__device__ __forceinline__ void integers(uint32_t w, uint32_t minus_z, uint32_t *out) {
    const uint32_t even = w & 0x0f0f0f0fu, odd = w & 0xf0f0f0f0u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t v;                                                 // selector 8 | i: the sign of byte i of even, zero
        asm("prmt.b32 %0, %1, %2, %3;" : "=r"(v) : "r"(even), "r"(odd), "r"(i | (8 | i) << 4 | (4 + i) << 8 | (8 | i) << 12));
        asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(out[i]) : "r"(v), "r"(0x7d007f00u), "r"(minus_z));
    }
}

__device__ __forceinline__ uint64_t pair(uint32_t lo, uint32_t hi) {
    uint64_t v;
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "r"(lo), "r"(hi));
    return v;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}

// A unit is what a set converts at a time: as many columns, up to 128, as tensor memory holds of A and of a D for each
// of their groups. Returned in pieces of 32 columns, like GU.
template <int N, int S, int GU>
struct Unit {
    static constexpr bool k4 = S * (4 * 16 + 4 / GU * N) <= 512, k2 = GU <= 2 && S * (2 * 16 + 2 / GU * N) <= 512;
    static constexpr int kPieces = k4 ? 4 : k2 ? 2 : GU;
};

// Eight fp32 values (zeros where !there) as three bf16 each that sum to them (exactly from 2^-103 on): the upper eight
// significand bits, cut, the eight after them, and the rest. An infinity or NaN is the first part alone.
__device__ __forceinline__ void cut(const float (&v)[8], bool there, uint4 (&part)[3]) {
    uint32_t h[3][8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float x = there ? v[e] : 0.f;
        h[0][e] = __float_as_uint(x) & 0xffff0000u;
        const float rest = fabsf(x) < INFINITY ? x - __uint_as_float(h[0][e]) : 0.f;
        if (x != x) h[0][e] |= 0x00400000u;                         // a NaN whose upper half reads as an infinity
        h[1][e] = __float_as_uint(rest) & 0xffff0000u;
        h[2][e] = __float_as_uint(rest - __uint_as_float(h[1][e]));
    }
#pragma unroll
    for (int p = 0; p < 3; ++p)
        part[p] = make_uint4(__byte_perm(h[p][0], h[p][1], 0x7632), __byte_perm(h[p][2], h[p][3], 0x7632),
                             __byte_perm(h[p][4], h[p][5], 0x7632), __byte_perm(h[p][6], h[p][7], 0x7632));
}

template <class C, int GU, bool kZeros>   // GU: groups are GU * 32 columns
__global__ void __launch_bounds__(C::kThreads, 1) linear_tc_kernel(const __grid_constant__ TcArgs args) {
    extern __shared__ __align__(1024) unsigned char smem[];
    __shared__ uint64_t full[C::kStages], empty[C::kStages], a_ready[C::S], done[C::S], drained;
    __shared__ uint32_t tmem_base;
    __shared__ int error;
    volatile int *err = &error;
    constexpr int N = C::N, ND = C::ND, S = C::S, U = Unit<ND, S, GU>::kPieces, kUnits = 8 / U, kGroups = U / GU;   // units of a block, groups of a unit
    constexpr int kSetColumns = U * 16 + kGroups * ND;               // of tensor memory: A, the groups' D
    constexpr uint32_t kColumns = S * kSetColumns <= 128 ? 128 : S * kSetColumns <= 256 ? 256 : 512;
    static_assert(S * kSetColumns <= 512, "tensor memory");
    using X = typename C::X;
    const LinearArgs &a = args.a;
    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), cluster = args.cluster;
    const int rank = blockIdx.x % cluster, row0 = blockIdx.x / cluster * kRows, tok0 = blockIdx.y * N;
    const int blocks = (a.d_in + 255) / 256, groups = a.d_in / (GU * 32);
    const int b_lo = (int)((long long)blocks * rank / cluster), b_hi = (int)((long long)blocks * (rank + 1) / cluster);
    const int u_lo = b_lo * kUnits, n_units = min(b_hi * kUnits, (groups + kGroups - 1) / kGroups) - u_lo;

    if (tid == 0) {
        for (int i = 0; i < C::kStages; ++i) mbar_init(&full[i], 1 + C::kCutters), mbar_init(&empty[i], 5 * kUnits);
        for (int i = 0; i < S; ++i) mbar_init(&a_ready[i], 4), mbar_init(&done[i], 1);
        mbar_init(&drained, 1);
        error = 0;
        fence_mbar_init();
        tc::prefetch_tensormap(&args.w);
        if (C::kParts == 1) tc::prefetch_tensormap(&args.x);
    }
    if (warp == 4 * S + 1) {
        tc::tmem_alloc(&tmem_base, kColumns);
        tc::tmem_relinquish();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    grid_dependency_wait();
    grid_launch_dependents();
    const uint32_t tmem = tmem_base, ring = smem_u32(smem);
    auto wait = [&](uint64_t *bar, uint32_t phase) -> bool {
        return mbar_try_wait(bar, phase & 1u) || wait_long(bar, phase & 1u, err);
    };
    // A wait of a warp: where it gave up for one lane, all leave.
    auto together = [](bool ok) -> bool { return __all_sync(0xffffffffu, ok); };

    float *red = reinterpret_cast<float *>(smem);                   // [S][N][kRows]
    uint64_t acc[N / 2];
    if (warp == 4 * S) {
        // ---------------- copies ----------------
        if (lane == 0) {
            int i = 0;
            for (; i < b_hi - b_lo; ++i) {
                const int st = i % C::kStages, b = b_lo + i;
                if (i >= C::kStages && !wait(&empty[st], (uint32_t)(i / C::kStages - 1))) break;
                unsigned char *to = smem + st * C::kStage;
                mbar_arrive_expect_tx(&full[st], C::kParts == 1 ? C::kStage : C::kWBytes);
                tc::tma_load_2d(to, &args.w, b * 128, row0, &full[st]);
#pragma unroll
                for (int h = 0; h < 4 && C::kParts == 1; ++h)
                    tc::tma_load_2d(to + C::kWBytes + h * N * 128, &args.x, b * 256 + h * 64, tok0, &full[st]);
            }
            // no copy is in flight when the ring is taken over
            for (int j = max(i - C::kStages, 0); j < i; ++j)
                mbar_wait_bounded(&full[j % C::kStages], (uint32_t)(j / C::kStages) & 1u, kWaitLimit);
        }
    } else if (warp == 4 * S + 1) {
        // ---------------- products ----------------
        // The whole warp runs the loop, so that addresses and descriptors are uniform; one lane's instructions count.
        constexpr uint32_t idesc = tc::idesc_bf16(kRows, ND);
        const uint32_t lead = tc::elect_one();
        const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
        const uint64_t x_desc = tc::smem_desc(ring + C::kWBytes, 128, tc::kSwz128);
        for (int u = 0; u < n_units; ++u) {
            const int i = u / kUnits, st = i % C::kStages, set = u % S;
            if (!together(wait(&full[st], (uint32_t)(i / C::kStages)) && wait(&a_ready[set], (uint32_t)(u / S)))) break;
            tc::fence_after_sync();
            const uint32_t at = tm + set * kSetColumns;
            const uint64_t xd = x_desc + (uint64_t)(st * (C::kStage >> 4));
#pragma unroll
            for (int k = 0; k < U * 2; ++k) {
                const int kk = (u % kUnits) * U * 2 + k;            // of the block's sixteen products
                tc::mma_bf16_tmem_a_lead(at + U * 16 + k / (GU * 2) * ND, at + k * 8,
                                         xd + (kk >> 2) * (ND * 128 >> 4) + (kk & 3) * 2, idesc, k % (GU * 2) > 0, lead);
            }
            tc::mma_commit_lead(&done[set], lead);
            tc::mma_commit_lead(&empty[st], lead);
        }
        tc::mma_commit_lead(&drained, lead);
        mbar_wait_bounded(&drained, 0, kWaitLimit);
    } else if (warp > 4 * S + 1) {
        // ---------------- x in fp32: three bf16 parts in the layout that TMA gives bf16 ----------------
        if constexpr (C::kParts == 3) {
            const int first = warp - (4 * S + 2);
            constexpr int kMine = N / 8;
            const float *x = static_cast<const float *>(a.x);
            alignas(16) float next[kMine][8];
            // No branch around a load, so that all are in flight: what is not there reads the first columns, for nothing.
            // Ordinary loads, since x may have been written while this kernel was already running.
            auto fetch = [&](int i) {
                const int k = (b_lo + i) * 256 + lane * 8;
#pragma unroll
                for (int r = 0; r < kMine; ++r) {
                    const int t = tok0 + first + r * 8;
                    const float *p = t < a.n_tokens && k < a.d_in ? x + (long long)t * a.x_stride + k : x;
                    if (args.x_vec) {
                        *reinterpret_cast<float4 *>(next[r]) = *reinterpret_cast<const float4 *>(p);
                        *reinterpret_cast<float4 *>(next[r] + 4) = *(reinterpret_cast<const float4 *>(p) + 1);
                    } else {
#pragma unroll
                        for (int e = 0; e < 8; ++e) next[r][e] = p[e];
                    }
                }
            };
            fetch(0);
            for (int i = 0; i < b_hi - b_lo; ++i) {
                const int st = i % C::kStages, k = (b_lo + i) * 256 + lane * 8;
                uint4 part[kMine][3];
#pragma unroll
                for (int r = 0; r < kMine; ++r) cut(next[r], tok0 + first + r * 8 < a.n_tokens && k < a.d_in, part[r]);
                if (i + 1 < b_hi - b_lo) fetch(i + 1);
                if (!together(i < C::kStages || wait(&empty[st], (uint32_t)(i / C::kStages - 1)))) break;
                unsigned char *to = smem + st * C::kStage + C::kWBytes + (lane >> 3) * (ND * 128);
#pragma unroll
                for (int r = 0; r < kMine; ++r) {
                    const int n = first + r * 8;
#pragma unroll
                    for (int e = 0; e < 3; ++e)
                        *reinterpret_cast<uint4 *>(to + (e * N + n) * 128 + (((lane & 7) ^ (n & 7)) << 4)) = part[r][e];
                }
                tc::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&full[st]);
            }
        }
    } else {
        // ---------------- conversion and sums: thread = row ----------------
        const int set = warp >> 2, row = tid & 127;
        const size_t wrow = min(row0 + row, a.d_out - 1);           // a row past d_out is not stored
        const X *scales = static_cast<const X *>(a.scales) + wrow * groups;
        const uint8_t *zeros = kZeros ? a.zeros + wrow * groups : nullptr;
        const uint32_t at = tmem + set * kSetColumns + ((uint32_t)(warp & 3) << 21);
        const unsigned char *wsrc = smem + row * 128;
        const int swz = row & 7;
#pragma unroll
        for (int n = 0; n < N / 2; ++n) acc[n] = 0;
        constexpr int kScaleWords = C::kParts == 3 ? kGroups : (kGroups + 1) / 2;
        uint32_t sc[kScaleWords] = {};                              // of the unit whose products run; bf16: two to a word
        uint32_t z = 0;                                             // of the unit to be converted, a byte to a group
        auto load_zeros = [&](int u) {
            const int of = (u_lo + u) * kGroups;
            if (kGroups > 1 && args.group_vec) {
                if (u < n_units)
                    z = kGroups == 4 ? *reinterpret_cast<const uint32_t *>(zeros + of) : *reinterpret_cast<const uint16_t *>(zeros + of);
                return;
            }
            z = 0;
#pragma unroll
            for (int g = 0; g < kGroups; ++g)
                if (u < n_units && of + g < groups) z |= (uint32_t)zeros[of + g] << (8 * g);
        };
        auto load_scales = [&](int u, uint32_t (&v)[kScaleWords]) {
            const int of = (u_lo + u) * kGroups;
            if (kGroups > 1 && args.group_vec) {
                if constexpr (kScaleWords == 4) {
                    const uint4 w = *reinterpret_cast<const uint4 *>(scales + of);
                    v[0] = w.x, v[1] = w.y, v[2] = w.z, v[3] = w.w;
                } else if constexpr (kScaleWords == 2) {
                    const uint2 w = *reinterpret_cast<const uint2 *>(scales + of);
                    v[0] = w.x, v[1] = w.y;
                } else {
                    v[0] = *reinterpret_cast<const uint32_t *>(scales + of);
                }
                return;
            }
            if constexpr (C::kParts == 3) {
#pragma unroll
                for (int g = 0; g < kGroups; ++g) v[g] = of + g < groups ? reinterpret_cast<const uint32_t *>(scales)[of + g] : 0u;
            } else {
                const uint16_t *s16 = reinterpret_cast<const uint16_t *>(scales);
#pragma unroll
                for (int g = 0; g < kGroups; g += 2)
                    v[g / 2] =
                        (of + g < groups ? s16[of + g] : 0u) | (g + 1 < kGroups && of + g + 1 < groups ? s16[of + g + 1] : 0u) << 16;
            }
        };
        auto scale_of = [&](int g) {
            return C::kParts == 3 ? __uint_as_float(sc[g]) : g & 1 ? bf_hi(sc[g / 2]) : bf_lo(sc[g / 2]);
        };
        if (kZeros) load_zeros(set);
        auto drain = [&]() {
#pragma unroll
            for (int g = 0; g < kGroups; ++g) {
                const uint32_t f = __float_as_uint(scale_of(g));
                const uint64_t ss = pair(f, f);
#pragma unroll
                for (int n = 0; n < ND; n += 16) {
                    uint32_t d[16];
                    tc::tmem_ld16_sync(at + U * 16 + g * ND + n, d);
                    const int to = n % N / 2;
#pragma unroll
                    for (int k = 0; k < 8; ++k) acc[to + k] = fma2(pair(d[2 * k], d[2 * k + 1]), ss, acc[to + k]);
                }
            }
        };
        bool ok = true;
        int it = 0;
        for (int u = set; u < n_units; u += S, ++it) {
            const int i = u / kUnits, st = i % C::kStages;
            uint32_t sc_next[kScaleWords];
            load_scales(u, sc_next);
            uint32_t zz[kGroups];                                   // -z / 64, twice
#pragma unroll
            for (int g = 0; g < kGroups; ++g) {
                zz[g] = 0xbe00be00u;                                // z = 8
                if (kZeros) {
                    const uint32_t zb = __float_as_uint((float)min(z >> (8 * g) & 255u, 128u) * -0.015625f) >> 16;
                    zz[g] = zb | zb << 16;
                }
            }
            if (kZeros) load_zeros(u + S);
            ok = together(wait(&full[st], (uint32_t)(i / C::kStages)));
            if (!ok) break;
            uint4 w[U];
#pragma unroll
            for (int j = 0; j < U; ++j)
                w[j] = *reinterpret_cast<const uint4 *>(wsrc + st * C::kStage + ((((u % kUnits) * U + j) ^ swz) << 4));
            uint32_t f[16];
            auto convert = [&](int j) {
                const uint32_t of[4] = {w[j].x, w[j].y, w[j].z, w[j].w};
#pragma unroll
                for (int k = 0; k < 4; ++k) integers(of[k], zz[j / GU], f + 4 * k);
            };
            convert(0);
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&empty[st]);
            if (it > 0) {
                ok = together(wait(&done[set], (uint32_t)(it - 1)));
                if (!ok) break;
                tc::fence_after_sync();
                drain();
            }
            tmem_st16(at, f);
#pragma unroll
            for (int j = 1; j < U; ++j) {
                convert(j);
                tmem_st16(at + j * 16, f);
            }
            tc::tmem_st_wait();
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&a_ready[set]);
#pragma unroll
            for (int g = 0; g < kScaleWords; ++g) sc[g] = sc_next[g];
        }
        if (ok && it > 0 && together(wait(&done[set], (uint32_t)(it - 1)))) {
            tc::fence_after_sync();
            drain();
        }
    }
    // ---- the sets' and the cluster's parts, added in a fixed order; the ring is done with
    tc::fence_before_sync();
    __syncthreads();
    if (warp < 4 * S) {
        float *mine = red + (warp >> 2) * N * kRows + (tid & 127);
#pragma unroll
        for (int n = 0; n < N / 2; ++n) {
            mine[2 * n * kRows] = __uint_as_float((uint32_t)acc[n]);
            mine[(2 * n + 1) * kRows] = __uint_as_float((uint32_t)(acc[n] >> 32));
        }
    }
    if (warp == 4 * S + 1) {
        tc::fence_after_sync();
        tc::tmem_dealloc(tmem, kColumns);
    }
    __syncthreads();
    const int nt = min(N, a.n_tokens - tok0), items = nt * (kRows / 4);
    float4 *sum = reinterpret_cast<float4 *>(red);
    auto add = [](float4 &s, const float4 &v) { s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w; };
    auto of_sets = [&](int i) {
        float4 s = sum[i];
#pragma unroll
        for (int p = 1; p < S; ++p) add(s, sum[p * N * (kRows / 4) + i]);
        return make_float4(s.x * 64.f, s.y * 64.f, s.z * 64.f, s.w * 64.f);      // integers() gives 64ths
    };
    auto store = [&](int i, const float4 &s) {
        const int r = row0 + (i & 31) * 4;
        X *y = static_cast<X *>(a.y) + (size_t)(tok0 + (i >> 5)) * a.y_stride + r;
        if (args.y_vec && r + 4 <= a.d_out) {
            if constexpr (C::kParts == 3)
                *reinterpret_cast<float4 *>(y) = s;
            else
                *reinterpret_cast<uint2 *>(y) = make_uint2(pack_bf16(s.x, s.y), pack_bf16(s.z, s.w));
        } else {
            const float v[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (r + e < a.d_out) y[e] = from_f32<X>(v[e]);
        }
    };
    if (cluster == 1) {
        for (int i = tid; i < items; i += C::kThreads) store(i, of_sets(i));
    } else {
        for (int i = tid; i < items; i += C::kThreads) sum[i] = of_sets(i);
        cluster_sync_all();
        const int lo = items * rank / cluster, hi = items * (rank + 1) / cluster;
        for (int i = lo + tid; i < hi; i += C::kThreads) {
            float4 v[kMaxCluster];
#pragma unroll
            for (int p = 0; p < kMaxCluster; ++p)
                if (p < cluster) v[p] = ld_peer_f4(map_peer(ring + i * 16, p));
#pragma unroll
            for (int p = 1; p < kMaxCluster; ++p)
                if (p < cluster) add(v[0], v[p]);
            store(i, v[0]);
        }
        cluster_sync_all();                                         // the peers have read this CTA's sums
    }
    if (tid == 0 && error) atomicAdd(&g_gave_up, 1u);
}

bool encode(CUtensorMap *map, CUtensorMapDataType type, CUtensorMapSwizzle swizzle, const void *base, long long columns,
            long long rows, long long row_bytes, int box_columns, int box_rows) {
    const cuuint64_t dims[] = {(cuuint64_t)columns, (cuuint64_t)rows}, bytes[] = {rows == 1 ? 16 : (cuuint64_t)row_bytes};
    const cuuint32_t box[] = {(cuuint32_t)box_columns, (cuuint32_t)box_rows}, ones[] = {1, 1};
    const auto fn = map_encoder();
    return fn && fn(map, type, 2, const_cast<void *>(base), dims, bytes, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
                    CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <class C, int GU, bool kZeros>
cudaError_t launch(const LinearArgs &a, int sms, cudaStream_t st) {
    auto kernel = linear_tc_kernel<C, GU, kZeros>;
    static std::atomic<uint64_t> ready{0};
    if (!device_bit(ready)) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
        if (e != cudaSuccess) return e;
        set_device_bit(ready);
    }
    static ActiveClusters known;
    const int blocks = (a.d_in + 255) / 256, tok_tiles = (a.n_tokens + C::N - 1) / C::N;
    const long long tiles = (long long)((a.d_out + kRows - 1) / kRows) * tok_tiles;
    // CTAs of a cluster: the least of an estimate in clocks, 5000 for a round of CTAs (launch, first loads, sums), 3000 for a
    // cluster's sums, 900 for a block of columns. It came within 1 % of the fastest of 1..8 for each of 45 shapes of
    // 512 to 14336 columns and rows and 16 to 64 tokens. 32 tokens with 1 / 2 / 3 / 4 / 8: 4096x4096 11.8 / 9.3 / 8.2 / 7.4 / 18.2 us (two
    // rounds), 4096x14336 12.4 / 19.0 / 24.4 / 28.1 / 49.6, 4096x1024 11.4 / 9.0 / 7.7 / 6.7 / 6.1.
    int cluster = 1;
    long long least = INT64_MAX;
    for (int c = 1; c <= kMaxCluster && (c == 1 || c <= blocks); ++c) {
        const int at_once = active_clusters(kernel, C::kThreads, C::kSmem, c, known);
        if (at_once < 1) continue;
        const long long rounds = (tiles + at_once - 1) / at_once;
        const long long cost = rounds * (5000 + (c > 1 ? 3000 : 0) + (long long)((blocks + c - 1) / c) * 900);
        if (cost < least) least = cost, cluster = c;
    }
    TcArgs args;
    args.a = a;
    args.cluster = cluster;
    args.x_vec = aligned16(a.x) && a.x_stride % 4 == 0;
    args.y_vec = reinterpret_cast<uintptr_t>(a.y) % (4 * sizeof(typename C::X)) == 0 && a.y_stride % 4 == 0;
    constexpr int kGroups = Unit<C::ND, C::S, GU>::kPieces / GU;
    args.group_vec = a.d_in / (GU * 32) % kGroups == 0 && reinterpret_cast<uintptr_t>(a.scales) % (sizeof(typename C::X) * kGroups) == 0 &&
                     reinterpret_cast<uintptr_t>(a.zeros) % kGroups == 0;
    if (!encode(&args.w, CU_TENSOR_MAP_DATA_TYPE_UINT8, CU_TENSOR_MAP_SWIZZLE_128B, a.qweight, a.d_in / 2, a.d_out, a.d_in / 2,
                128, kRows) ||
        (C::kParts == 1 &&
         !encode(&args.x, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, CU_TENSOR_MAP_SWIZZLE_128B, a.x, a.d_in, a.n_tokens,
                 a.x_stride * 2, 64, C::N)))
        return cudaErrorNotSupported;
    const dim3 grid((a.d_out + kRows - 1) / kRows * cluster, tok_tiles);
    return launch_step(kernel, grid, dim3(C::kThreads), C::kSmem, cluster, st, args);
}

// Sets of warps, measured with two / three: 17x14336x4096 with groups of 32 and zeros 15.7 / 17.1 us (two sets have room
// for the four D of 128 columns, three for those of 64), 64 tokens of it 20.5 / 19.7, 64x5120x8192 with groups of 64 12.5 /
// 14.4, 16x5120x8192 9.4 / 9.4, 17x4096x14336 with groups of 128 12.1 / 11.7.
template <typename X, int N>
cudaError_t launch_group(const LinearArgs &a, int sms, cudaStream_t st) {
    using Narrow = TcTile<X, N, sizeof(X) == 4 || N == 32 ? 2 : 3>;
    using Wide = TcTile<X, N, sizeof(X) == 4 || N == 64 ? 2 : 3>;
    switch (a.group) {
        case 32: return a.zeros ? launch<Narrow, 1, true>(a, sms, st) : launch<Narrow, 1, false>(a, sms, st);
        case 64: return a.zeros ? launch<Wide, 2, true>(a, sms, st) : launch<Wide, 2, false>(a, sms, st);
        default: return a.zeros ? launch<Wide, 4, true>(a, sms, st) : launch<Wide, 4, false>(a, sms, st);
    }
}

}  // namespace

cudaError_t read_timeouts(unsigned *count) { return cudaMemcpyFromSymbol(count, g_gave_up, sizeof *count); }

bool tc_takes(const LinearArgs &a) {
    return aligned16(a.x) && a.x_stride % 8 == 0 && a.x_stride < 1ll << 38;
}

cudaError_t launch_tc(const LinearArgs &a, int dtype, int sms, cudaStream_t st) {
    // three parts of 64 tokens would leave a ring of one stage
    if (dtype == LORA_DTYPE_F32) return a.n_tokens <= 16 ? launch_group<float, 16>(a, sms, st) : launch_group<float, 32>(a, sms, st);
    using X = __nv_bfloat16;
    if (a.n_tokens <= 16) return launch_group<X, 16>(a, sms, st);
    if (a.n_tokens <= 32) return launch_group<X, 32>(a, sms, st);
    return launch_group<X, 64>(a, sms, st);
}

}  // namespace linear
}  // namespace lora
