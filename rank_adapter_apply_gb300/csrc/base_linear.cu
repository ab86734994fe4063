// lora_base_linear: y = W x for a few tokens, W in 4 bits with group scales.
#include "base_linear.cuh"

#include <algorithm>

namespace lora {
namespace linear {
namespace {

using namespace step;

// bf16 on mma.sync. A CTA of up to 12 warps takes 16 rows of W to a warp and, as
// one of the CTAs of a cluster, a range of the columns; warps and cluster are
// chosen so that the CTAs fill the SMs evenly (launch_tiles). Each warp streams its
// rows' 4-bit words from global memory into registers, kAhead blocks of 128 columns
// ahead, and meets nobody on the way; x of a slice of KS columns lies in shared
// memory for all of them. A product mma(W 16 x 16, x^T 16 x 8) has the rows of W as
// its rows and eight tokens as its columns. The 4-bit values become (n - z) / 64 in
// registers, exact in bf16 (nibbles()). So the products within a group are exact,
// and the group's fp32 sum is scaled once. At the end the cluster's parts are added
// in a fixed order through distributed shared memory: no workspace, no atomics.
//
// What bounds it: for one token the words of W ought to, and a third to a half of
// their rate is reached (W from memory: 1x4096x4096 6.1 us, 1.4 TB/s; 1x4096x14336
// 11.2 us, 2.7 TB/s): the launch, the first loads and the cluster's end take 3 us
// of a call. Where x is not aligned it also serves many tokens, and the products
// take over (64x5120x8192 29.9 us).
//
// Order of the columns. A block of 128 columns is four units of two products. Lane
// t of a quad loads 16 bytes of a row, columns 32 t .. 32 t + 31. With groups of 128
// its word u is its part of unit u. With groups of 64 or 32 a unit has to stay
// within a group, so the quad first exchanges words (exchange()). Within a word the
// halves of a register are nibbles 16 bits apart: 0 4 | 1 5 | 2 6 | 3 7. x is put
// into the same order when it is staged (x_place() and the byte permutes).
template <int NT_, int KS_, int kAhead_, int kCtas_, int kMaxWarps_>
struct LinearTile {
    static constexpr int NT = NT_, KS = KS_, kAhead = kAhead_, kCtas = kCtas_;
    static constexpr int kMaxWarps = kMaxWarps_, T = 8 * NT;        // tokens
    static constexpr int kXRow = KS * 2, kPlane = T * kXRow;        // bytes of a staged row, of x
    static constexpr int kParted = T * (16 * kMaxWarps + 1) * 4;    // bytes of the parts of the sums, at most
    static constexpr int kSmem = kPlane > kParted ? kPlane : kParted;
    static_assert(KS % (128 * kAhead) == 0, "a slice is whole rounds of the register ring");
};

// Nibbles 0 and 4 (kHigh: 1 and 5) of w, less the zero, over 64. Bits v < 256 of a bf16 are the number v 2^-133,
// subnormal or not: n 2^-133 2^127 or 16 n 2^-133 2^123, and minus_z = -z / 64, twice, added in the same exact operation.
template <bool kHigh>
__device__ __forceinline__ uint32_t nibbles(uint32_t w, uint32_t minus_z) {
    uint32_t v;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;"
        : "=r"(v) : "r"(w & (kHigh ? 0x00f000f0u : 0x000f000fu)), "r"(kHigh ? 0x7d007d00u : 0x7f007f00u), "r"(minus_z));
    return v;
}

// The first product of a group: D = A * B.
__device__ __forceinline__ void mma_bf16_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
        "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};\n"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

// W is read once: 16 bytes past the L1.
__device__ __forceinline__ uint4 load_w(const uint8_t *p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}

// Eight consecutive bf16 of x, zeros when !ok. Ordinary loads: the kernel before may still have been writing x when this
// one started, and the read-only path asks for memory that nobody writes as long as the kernel runs. (The weights are.)
__device__ __forceinline__ uint4 load_x(const __nv_bfloat16 *p, bool ok, bool vec) {
    if (!ok) return make_uint4(0, 0, 0, 0);
    if (vec) return *reinterpret_cast<const uint4 *>(p);
    const uint16_t *e = reinterpret_cast<const uint16_t *>(p);
    return make_uint4(e[0] | (uint32_t)e[1] << 16, e[2] | (uint32_t)e[3] << 16, e[4] | (uint32_t)e[5] << 16,
                      e[6] | (uint32_t)e[7] << 16);
}

// Words of a quad's 16 bytes each into units: w[u] becomes this lane's word of unit u.
template <int GU>
__device__ __forceinline__ void exchange(uint32_t (&w)[4], int t4) {
    if constexpr (GU <= 2) {
        // lanes t and t ^ 2: the lower keeps its words 0, 1 and gives 2, 3
        const bool up = t4 & 2;
        const uint32_t a = __shfl_xor_sync(0xffffffffu, up ? w[0] : w[2], 2);
        const uint32_t b = __shfl_xor_sync(0xffffffffu, up ? w[1] : w[3], 2);
        if (up)
            w[0] = a, w[1] = b;
        else
            w[2] = a, w[3] = b;
    }
    if constexpr (GU == 1) {
        // now w[0..1] are of pieces 0, 1 and w[2..3] of pieces 2, 3: lanes t and t ^ 1
        const bool up = t4 & 1;
        const uint32_t a = __shfl_xor_sync(0xffffffffu, up ? w[0] : w[1], 1);
        const uint32_t b = __shfl_xor_sync(0xffffffffu, up ? w[2] : w[3], 1);
        if (up)
            w[0] = a, w[2] = b;
        else
            w[1] = a, w[3] = b;
    }
}

// Where eight columns of x (piece q of a block's 16) go: 4 * unit + lane of the quad.
template <int GU>
__device__ __forceinline__ int x_place(int q) {
    if constexpr (GU == 4) return (q & 3) * 4 + (q >> 2);
    // lane t has, of each half block, words 2 (t >> 1) and the next of piece t & 1
    if constexpr (GU == 2) return ((q >> 3) * 2 + (q & 1)) * 4 + (q >> 2 & 1) + (q >> 1 & 1) * 2;
    return q;                                                       // a full transpose: unit u is piece u
}

template <class C, int GU, bool kZeros>   // GU: groups are GU * 32 columns
__global__ void __launch_bounds__(32 * C::kMaxWarps, C::kCtas) linear_tiles_kernel(LinearArgs a, int cluster, int x_vec) {
    extern __shared__ __align__(128) unsigned char smem[];
    constexpr int kGroups = 4 / GU, kSliceBlocks = C::KS / 128, kAhead = C::kAhead;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g4 = lane >> 2, t4 = lane & 3;
    const int warps = blockDim.x >> 5, rows = 16 * warps;
    const int rank = blockIdx.x % cluster, row0 = blockIdx.x / cluster * rows, tok0 = blockIdx.y * C::T;
    const int nt = min(C::T, a.n_tokens - tok0);
    const int groups = a.d_in / (GU * 32), blocks = (a.d_in + 127) / 128;
    const int b_lo = (int)((long long)blocks * rank / cluster), b_hi = (int)((long long)blocks * (rank + 1) / cluster);
    using X = __nv_bfloat16;
    const X *x = static_cast<const X *>(a.x) + (size_t)tok0 * a.x_stride;

    grid_dependency_wait();
    grid_launch_dependents();
    // ---- this lane's rows: words, scales and zeros of a block. A row past d_out reads the last row (nobody stores
    // what comes of it), and columns past d_in meet an x of zero.
    const int r_in = warp * 16 + g4;                                // and r_in + 8
    const uint8_t *wsrc[2];
    const X *ssrc[2];
    const uint8_t *zsrc[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const size_t row = min(row0 + r_in + h * 8, a.d_out - 1);
        wsrc[h] = a.qweight + row * (a.d_in / 2) + (size_t)b_lo * 64 + t4 * 16;
        ssrc[h] = static_cast<const X *>(a.scales) + row * groups + b_lo * kGroups + t4 % kGroups;
        zsrc[h] = kZeros ? a.zeros + row * groups + b_lo * kGroups + t4 % kGroups : nullptr;
    }
    uint4 w[kAhead][2];
    X sc[kAhead][2];
    uint32_t zr[kAhead][2];
    // block i of the round whose first block is b (the pointers are at b)
    auto fetch = [&](int i, int b, int slot) {
        if (b + i >= b_hi) return;
        const bool in = GU == 4 || (b + i) * 128 + t4 * 32 < a.d_in;
        const bool gin = GU == 4 || (b + i) * kGroups + t4 % kGroups < groups;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            w[slot][h] = in ? load_w(wsrc[h] + i * 64) : make_uint4(0, 0, 0, 0);
            sc[slot][h] = gin ? __ldg(ssrc[h] + i * kGroups) : from_f32<X>(0.f);
            if (kZeros) zr[slot][h] = gin ? __ldg(zsrc[h] + i * kGroups) : 0;
        }
    };
#pragma unroll
    for (int i = 0; i < kAhead; ++i) fetch(i, b_lo, i);

    float acc[C::NT][4];
#pragma unroll
    for (int n = 0; n < C::NT; ++n) acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.f;

    for (int s_lo = b_lo; s_lo < b_hi; s_lo += kSliceBlocks) {
        // ---- x of the slice: rows past the tokens and columns past d_in are zero
        const int n_blocks = min(kSliceBlocks, b_hi - s_lo);
        if (s_lo != b_lo) __syncthreads();
        // A warp takes a block's 16 pieces of two tokens at a time: piece and place of a lane are always the same.
        constexpr int kBatch = C::NT == 1 ? 4 : 8;    // pieces of a thread whose loads are in flight
        const int q = lane & 15, odd = lane >> 4;                   // odd token of the pair
        unsigned char *dst = smem + odd * C::kXRow + ((x_place<GU>(q) ^ (odd << 2)) << 4);
        const int pairs = s_lo == b_lo ? C::T / 2 : (nt + 1) / 2;   // rows past the tokens are cleared once
        for (int i0 = warp; i0 < pairs * kSliceBlocks; i0 += warps * kBatch) {
            uint4 v[kBatch];
#pragma unroll
            for (int e = 0; e < kBatch; ++e) {
                const int i = i0 + e * warps, t = i / kSliceBlocks * 2 + odd, blk = i % kSliceBlocks;
                const int k = (s_lo + blk) * 128 + q * 8;
                v[e] = load_x(x + (size_t)t * a.x_stride + k, t < nt && blk < n_blocks && k < a.d_in, x_vec);
            }
#pragma unroll
            for (int e = 0; e < kBatch; ++e) {
                const int i = i0 + e * warps, t2 = i / kSliceBlocks * 2, blk = i % kSliceBlocks;
                if (t2 >= C::T) break;
                const uint4 &o = v[e];
                *reinterpret_cast<uint4 *>(dst + t2 * C::kXRow + blk * 256) =
                    make_uint4(__byte_perm(o.x, o.z, 0x5410), __byte_perm(o.x, o.z, 0x7632), __byte_perm(o.y, o.w, 0x5410),
                               __byte_perm(o.y, o.w, 0x7632));
            }
        }
        __syncthreads();
        // lane t4's piece of unit u: place 4 u + t4, odd tokens with the halves of eight places swapped
        const unsigned char *xbase = smem + g4 * C::kXRow + ((t4 ^ ((g4 & 1) << 2)) << 4);
        const int x_odd = (g4 & 1) ? -64 : 64;
        for (int r0 = 0; r0 < n_blocks; r0 += kAhead, xbase += kAhead * 256) {
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                if (r0 + i >= n_blocks) break;
                uint32_t wd[2][4], z[2];
                float sf[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    wd[h][0] = w[i][h].x, wd[h][1] = w[i][h].y, wd[h][2] = w[i][h].z, wd[h][3] = w[i][h].w;
                    exchange<GU>(wd[h], t4);
                    sf[h] = to_f32(sc[i][h]);
                    z[h] = 0xbe00be00u;                             // -8 / 64, twice
                    if (kZeros) {
                        const uint32_t zb = __float_as_uint((float)min(zr[i][h], 128u) * -0.015625f) >> 16;
                        z[h] = zb | zb << 16;
                    }
                }
                fetch(i + kAhead, s_lo + r0, i);
                float part[C::NT][4];
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    uint32_t f[2][4];
                    const uint32_t z0 = kZeros && kGroups > 1 ? __shfl_sync(0xffffffffu, z[0], u / GU, 4) : z[0];
                    const uint32_t z1 = kZeros && kGroups > 1 ? __shfl_sync(0xffffffffu, z[1], u / GU, 4) : z[1];
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        f[half][0] = nibbles<false>(wd[0][u] >> (8 * half), z0);
                        f[half][1] = nibbles<false>(wd[1][u] >> (8 * half), z1);
                        f[half][2] = nibbles<true>(wd[0][u] >> (8 * half), z0);
                        f[half][3] = nibbles<true>(wd[1][u] >> (8 * half), z1);
                    }
#pragma unroll
                    for (int n = 0; n < C::NT; ++n) {
                        const uint4 b =
                            *reinterpret_cast<const uint4 *>(xbase + n * 8 * C::kXRow + i * 256 + (u >> 1) * 128 + (u & 1) * x_odd);
                        if (u % GU == 0)
                            mma_bf16_first(part[n], f[0], b.x, b.y);
                        else
                            mma_bf16(part[n], f[0][0], f[0][1], f[0][2], f[0][3], b.x, b.y);
                        mma_bf16(part[n], f[1][0], f[1][1], f[1][2], f[1][3], b.z, b.w);
                    }
                    if (u % GU == GU - 1) {
                        const float s0 = kGroups > 1 ? __shfl_sync(0xffffffffu, sf[0], u / GU, 4) : sf[0];
                        const float s1 = kGroups > 1 ? __shfl_sync(0xffffffffu, sf[1], u / GU, 4) : sf[1];
#pragma unroll
                        for (int n = 0; n < C::NT; ++n) {
                            acc[n][0] = fmaf(s0, part[n][0], acc[n][0]);
                            acc[n][1] = fmaf(s0, part[n][1], acc[n][1]);
                            acc[n][2] = fmaf(s1, part[n][2], acc[n][2]);
                            acc[n][3] = fmaf(s1, part[n][3], acc[n][3]);
                        }
                    }
                }
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                wsrc[h] += kAhead * 64;
                ssrc[h] += kAhead * kGroups;
                if (kZeros) zsrc[h] += kAhead * kGroups;
            }
        }
    }
    // ---- the cluster's parts, added in a fixed order
    __syncthreads();
    float *red = reinterpret_cast<float *>(smem);                   // [T][red_row]
    const int red_row = rows + 1;
#pragma unroll
    for (int n = 0; n < C::NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e)
            red[(n * 8 + t4 * 2 + (e & 1)) * red_row + r_in + (e >> 1) * 8] = acc[n][e];
    if (cluster > 1)
        cluster_sync_all();
    else
        __syncthreads();
    const int r_lo = rows * rank / cluster, slice = rows * (rank + 1) / cluster - r_lo;
    const uint32_t red_at = smem_u32(red);
    for (int i = tid; i < nt * slice; i += 32 * warps) {
        const int t = i / slice, r = r_lo + i % slice, at = t * red_row + r;
        if (row0 + r >= a.d_out) continue;
        float sum = red[at];
        if (cluster > 1) {
            float v[kMaxCluster];
#pragma unroll
            for (int p = 0; p < kMaxCluster; ++p)
                v[p] = p < cluster ? __uint_as_float(ld_peer_u32(map_peer(red_at, p) + at * 4)) : 0.f;
            sum = v[0];
#pragma unroll
            for (int p = 1; p < kMaxCluster; ++p) sum += v[p];
        }
        static_cast<X *>(a.y)[(size_t)(tok0 + t) * a.y_stride + row0 + r] = from_f32<X>(sum * 64.f);       // nibbles() gives 64ths
    }
    if (cluster > 1) cluster_sync_all();                            // the peers have read this CTA's parts
}

template <class C, int GU, bool kZeros>
cudaError_t launch_tiles(const LinearArgs &a, int sms, cudaStream_t st) {
    auto kernel = linear_tiles_kernel<C, GU, kZeros>;
    static std::atomic<uint64_t> ready{0};
    if (!device_bit(ready)) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
        if (e != cudaSuccess) return e;
        set_device_bit(ready);
    }
    // Warps of a CTA and CTAs of a cluster: the least of an estimate in clocks. A round of CTAs costs about 5000 (launch,
    // first loads, the cluster's sums) and for each block of columns the latency of a warp's chain, 900, and the issue
    // slots or tensor time of every warp of the SM's four schedulers, with the staging of x. A round is what the device
    // holds at once: clusters fill whole places of a GPC. It comes within 10 % of what was measured: 1x4096x4096 8 warps,
    // clusters of 8: 5.7 us; 7 and 4: 7.1; 7 and 8, in two rounds: 8.9. 1x14336x4096: 8, 8: 13.0; 7, 4: 20.7.
    // 1x4096x14336: 6, 2: 10.5; 8, 2: 12.0; 4, 5, in two rounds: 15.4.
    const int tok_tiles = (a.n_tokens + C::T - 1) / C::T, blocks = (a.d_in + 127) / 128;
    constexpr int kIssue = (150 + 28 * C::NT) / 4, kTensor = 16 * C::NT;
    static ActiveClusters known[C::kMaxWarps + 1];
    int warps = C::kMaxWarps, cluster = 1;
    long long least = INT64_MAX;
    for (int w = C::kMaxWarps; w >= 4; --w)
        for (int c = 1; c <= kMaxCluster && (c == 1 || c <= blocks); ++c) {
            const long long clusters = (long long)((a.d_out + 16 * w - 1) / (16 * w)) * tok_tiles;
            const int at_once = active_clusters(kernel, 32 * w, C::kSmem, c, known[w]);
            if (at_once < 1) continue;
            const long long rounds = (clusters + at_once - 1) / at_once;
            const long long on_sm = (std::min<long long>(clusters, at_once) * c + sms - 1) / sms;
            const long long cost = rounds * (5000 + (long long)((blocks + c - 1) / c) *
                                                        (900 + on_sm * (w * std::max(kIssue, kTensor) + 2 * C::T)));
            if (cost < least) least = cost, warps = w, cluster = c;
        }
    const int x_vec = aligned16(a.x) && a.x_stride % 8 == 0;
    const dim3 grid((a.d_out + 16 * warps - 1) / (16 * warps) * cluster, tok_tiles);
    return launch_step(kernel, grid, dim3(32 * warps), C::kSmem, cluster, st, a, cluster, x_vec);
}

template <class C, int GU>
cudaError_t launch_zeros(const LinearArgs &a, int sms, cudaStream_t st) {
    return a.zeros ? launch_tiles<C, GU, true>(a, sms, st) : launch_tiles<C, GU, false>(a, sms, st);
}

template <class C>
cudaError_t launch_group(const LinearArgs &a, int sms, cudaStream_t st) {
    switch (a.group) {
        case 32: return launch_zeros<C, 1>(a, sms, st);
        case 64: return launch_zeros<C, 2>(a, sms, st);
        default: return launch_zeros<C, 4>(a, sms, st);
    }
}

// The kernel and its tokens' tile. bf16 from 4 tokens goes to the 5th-generation tensor cores where TMA can load x (16-byte
// aligned rows), measured for 4096x4096, 5120x8192 and 4096x14336 (d_in x d_out), W from memory: 2 tokens 6.3 / 10.6 / 11.4
// us here and 6.5 / 10.0 / 11.6 there, 4 tokens 6.5 / 10.4 / 12.0 and 6.5 / 10.0 / 11.6, 8 tokens 6.9 / 10.8 / 12.7 and 6.6 /
// 10.0 / 11.6; from L2, 16 tokens 8.3 / 12.7 / 14.9 and 6.3 / 9.5 / 11.5, 64 tokens 15.1 / 29.9 / 32.3 and 8.0 / 12.5 /
// 13.4. fp32 always goes there (with three products for each here, 1 token 8.8 / 16.5 / 19.0 us against 7.6 / 13.0 / 16.5, 64
// tokens 41 / 71 / 88 against 16.6 / 34.9 / 55.5). Here, up to 16 tokens: two CTAs of eight warps to an SM. Above, the
// accumulators want the registers of twelve warps to an SM, in one CTA, whose copy of x then serves more rows (48 tokens:
// 12.5 / 23.4 / 26.2 us, against 14.1 / 25.5 / 32.1 with two CTAs of eight).
cudaError_t launch_linear(const LinearArgs &a, int dtype, int sms, cudaStream_t st) {
    if (dtype == LORA_DTYPE_F32 || (a.n_tokens >= 4 && tc_takes(a))) return launch_tc(a, dtype, sms, st);
    if (a.n_tokens <= 8) return launch_group<LinearTile<1, 2048, 4, 2, 8>>(a, sms, st);
    if (a.n_tokens <= 16) return launch_group<LinearTile<2, 2048, 4, 2, 8>>(a, sms, st);
    if (a.n_tokens <= 32) return launch_group<LinearTile<4, 1024, 4, 1, 12>>(a, sms, st);
    return launch_group<LinearTile<8, 1024, 1, 1, 12>>(a, sms, st);
}

}  // namespace
}  // namespace linear
}  // namespace lora

using namespace lora;
using namespace lora::linear;
using namespace lora::step;

extern "C" int lora_base_linear(const lora_base_linear_desc *d, void *stream) {
    if (!d) return fail(LORA_ERR_ARG, "base_linear: NULL descriptor");
    if (!known_dtype(d->dtype)) return fail(LORA_ERR_ARG, "base_linear: unknown dtype %d", d->dtype);
    if (d->group != 32 && d->group != 64 && d->group != 128)
        return fail(LORA_ERR_ARG, "base_linear: group %d is not 32, 64 or 128", d->group);
    if (d->n_tokens < 0 || d->d_in < 1 || d->d_out < 1 || d->d_in % d->group != 0)
        return fail(LORA_ERR_ARG, "base_linear: n_tokens %d, d_in %d (a multiple of group %d), d_out %d", d->n_tokens,
                    d->d_in, d->group, d->d_out);
    if (d->n_tokens > (1 << 18)) return fail(LORA_ERR_ARG, "base_linear: n_tokens %d is above 262144", d->n_tokens);
    if (d->n_tokens == 0) return LORA_OK;
    if (!d->x || !d->qweight || !d->scales || !d->y) return fail(LORA_ERR_ARG, "base_linear: NULL pointer argument");
    if (!aligned16(d->qweight)) return fail(LORA_ERR_ARG, "base_linear: qweight must be 16-byte aligned");
    if (d->n_tokens > 1 && (d->x_stride < d->d_in || d->y_stride < d->d_out))
        return fail(LORA_ERR_ARG, "base_linear: row strides %lld, %lld are below d_in, d_out", (long long)d->x_stride,
                    (long long)d->y_stride);
    LinearArgs a{d->x,        d->qweight,  d->scales, d->zeros, d->y,    (long long)d->x_stride,
                 (long long)d->y_stride, d->n_tokens, d->d_in,   d->d_out, d->group};
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int sms = sm_count();
    if (sms < 1) return fail(LORA_ERR_CUDA, "base_linear: no CUDA device");
    return launched("base_linear", launch_linear(a, d->dtype, sms, st));
}
