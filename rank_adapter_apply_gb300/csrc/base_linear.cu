// lora_base_linear: y = W x for a few tokens, W in 4 bits with group scales.
#include "step_util.cuh"

#include <atomic>

namespace lora {
namespace {

using namespace step;

struct LinearArgs {
    const void *x;
    const uint8_t *qweight;
    const void *scales;
    const uint8_t *zeros;
    void *y;
    long long x_stride, y_stride;
    int n_tokens, d_in, d_out, group;
};

// One warp per output row and TT tokens: a lane takes eight columns (one
// 32-bit word of the row) at a time, in fp32.
template <typename T, int TT>
__global__ void __launch_bounds__(256) linear_rows_kernel(LinearArgs a) {
    const int lane = threadIdx.x & 31;
    const int row = blockIdx.x * 8 + (threadIdx.x >> 5);
    const int t0 = blockIdx.y * TT;
    if (row >= a.d_out) return;
    const int nt = min(TT, a.n_tokens - t0);
    const int words = a.d_in / 8, groups = a.d_in / a.group;
    const uint32_t *w = reinterpret_cast<const uint32_t *>(a.qweight + (size_t)row * (a.d_in / 2));
    const T *sc = static_cast<const T *>(a.scales) + (size_t)row * groups;
    const uint8_t *zr = a.zeros ? a.zeros + (size_t)row * groups : nullptr;
    const T *x = static_cast<const T *>(a.x) + (size_t)t0 * a.x_stride;
    float acc[TT];
#pragma unroll
    for (int t = 0; t < TT; ++t) acc[t] = 0.f;
    for (int i = lane; i < words; i += 32) {
        const uint32_t q = w[i];
        const int g = i * 8 / a.group;
        const float s = to_f32(sc[g]);
        const float z = zr ? fminf((float)zr[g], 128.f) : 8.f;
        float n[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) n[j] = (float)((q >> (4 * j)) & 15u) - z;
#pragma unroll
        for (int t = 0; t < TT; ++t) {
            if (t < nt) {
                const T *xt = x + (size_t)t * a.x_stride + i * 8;
                float p = 0.f;
#pragma unroll
                for (int j = 0; j < 8; ++j) p = fmaf(n[j], to_f32(xt[j]), p);
                acc[t] = fmaf(s, p, acc[t]);
            }
        }
    }
#pragma unroll
    for (int t = 0; t < TT; ++t) {
        const float v = warp_sum(acc[t]);
        if (lane == 0 && t < nt) static_cast<T *>(a.y)[(size_t)(t0 + t) * a.y_stride + row] = from_f32<T>(v);
    }
}

// ---- bf16: tensor-core tiles --------------------------------------------------------
//
// A CTA takes R rows of W and, as one of the CK CTAs of a cluster, a slice of
// the columns, in chunks of KC columns staged by asynchronous copies. Its eight
// warps are WR groups of 16 * MT rows times WK groups of the chunk's columns. A
// product mma(W 16 x 16, x^T 16 x 8) has the rows of W as its rows and eight
// tokens as its columns. The 4-bit values become bf16 integers in registers:
// 0x4300 | n is 128 + n, and subtracting 128 + z leaves n - z exactly. So the
// products within a group are exact in fp32, and the group's fp32 sum is scaled
// once. A column order within eight columns that suits the unpacking (0 4, 1 5, 2
// 6, 3 7: nibbles 16 bits apart) is used for W and x alike. At the end the warps'
// and the cluster's parts are added in a fixed order through (distributed) shared
// memory: no workspace, no atomics.
template <int NT_, int MT_, int WR_, int KC_, int kStages_, int kCtas_>
struct LinearTile {
    static constexpr int NT = NT_, MT = MT_, WR = WR_, KC = KC_, kStages = kStages_, kCtas = kCtas_;
    static constexpr int WK = 8 / WR, R = WR * 16 * MT, T = 8 * NT, KW = KC / WK;
    static constexpr int kWRow = KC / 2, kXRow = KC * 2;            // bytes of a staged row
    static constexpr int kWStage = R * kWRow, kStage = kWStage + T * kXRow;
    static constexpr int kRedRow = R + 1;                           // floats of a token's row of the parts
    static constexpr int kRed = WK * T * kRedRow * 4;
    static constexpr int kSmem = kStages * kStage > kRed ? kStages * kStage : kRed;
    static_assert(KW % 128 == 0 && kWRow % 128 == 0, "a warp's columns come in blocks of 128");
};

__device__ __forceinline__ uint32_t nibbles(uint32_t w, uint32_t zz) {
    uint32_t v;
    asm("lop3.b32 %0, %1, 0x000f000f, 0x43004300, 0xea;" : "=r"(v) : "r"(w));     // (w & mask) | magic
    __nv_bfloat162 h = __hsub2(*reinterpret_cast<__nv_bfloat162 *>(&v), *reinterpret_cast<__nv_bfloat162 *>(&zz));
    return *reinterpret_cast<uint32_t *>(&h);
}

template <class C, int GU>   // GU: groups are GU * 32 columns
__global__ void __launch_bounds__(256, C::kCtas) linear_tiles_kernel(LinearArgs a, int cluster, int x_vec) {
    extern __shared__ __align__(128) unsigned char smem[];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g4 = lane >> 2, t4 = lane & 3;
    const int wr = warp % C::WR, wk = warp / C::WR;
    const int rank = blockIdx.x % cluster, row0 = blockIdx.x / cluster * C::R, tok0 = blockIdx.y * C::T;
    const int nt = min(C::T, a.n_tokens - tok0);
    const int groups = a.d_in / a.group, chunks = (a.d_in + C::KC - 1) / C::KC;
    const int c_lo = (int)((long long)chunks * rank / cluster), c_hi = (int)((long long)chunks * (rank + 1) / cluster);
    const __nv_bfloat16 *x = static_cast<const __nv_bfloat16 *>(a.x) + (size_t)tok0 * a.x_stride;
    const __nv_bfloat16 *scales = static_cast<const __nv_bfloat16 *>(a.scales);

    // rows of x past the tokens are zero in every stage and never copied to
    for (int i = tid; i < C::kStages * (C::T - nt) * (C::kXRow / 16); i += 256) {
        const int st = i / ((C::T - nt) * (C::kXRow / 16)), at = i % ((C::T - nt) * (C::kXRow / 16));
        *reinterpret_cast<uint4 *>(smem + st * C::kStage + C::kWStage + nt * C::kXRow + at * 16) = make_uint4(0, 0, 0, 0);
    }
    auto issue = [&](int chunk, int st) {
        unsigned char *base = smem + st * C::kStage;
        const int k0 = chunk * C::KC;
        constexpr int kWPieces = C::kWRow / 16, kXPieces = C::kXRow / 16;
#pragma unroll
        for (int i = 0; i < C::R * kWPieces / 256; ++i) {
            const int n = tid + i * 256, r = n / kWPieces, p = n % kWPieces;
            const bool ok = row0 + r < a.d_out && k0 + p * 32 < a.d_in;
            const uint8_t *src = a.qweight + (ok ? (size_t)(row0 + r) * (a.d_in / 2) + k0 / 2 + p * 16 : 0);
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                             smem_u32(base + r * C::kWRow + ((p ^ (r & 7)) << 4))),
                         "l"(src), "r"(ok ? 16 : 0)
                         : "memory");
        }
        for (int n = tid; n < nt * kXPieces; n += 256) {
            const int t = n / kXPieces, p = n % kXPieces;
            unsigned char *dst = base + C::kWStage + t * C::kXRow + ((p ^ ((t & 1) << 2)) << 4);
            const bool ok = k0 + p * 8 < a.d_in;                    // d_in is a multiple of 32
            const __nv_bfloat16 *src = x + (ok ? (size_t)t * a.x_stride + k0 + p * 8 : 0);
            if (x_vec) {
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src),
                             "r"(ok ? 16 : 0)
                             : "memory");
            } else {
                *reinterpret_cast<uint4 *>(dst) = ok ? load8_bf16(reinterpret_cast<const uint16_t *>(src), 0, 8, true, 0)
                                                     : make_uint4(0, 0, 0, 0);
            }
        }
    };
    // Scales and zeros of one block of 128 columns: lane t4 of a quad has the block's group t4 / GU..., of both rows
    struct Groups {
        float s[C::MT][2];
        uint32_t z[C::MT][2];
    };
    auto read_groups = [&](int chunk, int block) {
        Groups g;
        const int k = chunk * C::KC + wk * C::KW + block * 128 + t4 / GU * GU * 32, gi = k / (GU * 32);
#pragma unroll
        for (int mt = 0; mt < C::MT; ++mt)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int row = row0 + (wr * C::MT + mt) * 16 + g4 + h * 8;
                const bool ok = row < a.d_out && chunk < c_hi && gi < groups;
                const size_t at = ok ? (size_t)row * groups + gi : 0;
                g.s[mt][h] = ok ? __bfloat162float(scales[at]) : 0.f;
                // 128 + z as a bf16 pair: exact up to 256
                const uint32_t z = a.zeros && ok ? min((int)a.zeros[at], 128) : 8;
                const uint32_t b = __float_as_uint(128.f + (float)z) >> 16;
                g.z[mt][h] = b | b << 16;
            }
        return g;
    };

    float acc[C::MT][C::NT][4];
#pragma unroll
    for (int mt = 0; mt < C::MT; ++mt)
#pragma unroll
        for (int n = 0; n < C::NT; ++n) acc[mt][n][0] = acc[mt][n][1] = acc[mt][n][2] = acc[mt][n][3] = 0.f;

    for (int s = 0; s < C::kStages - 1; ++s) {
        if (c_lo + s < c_hi) issue(c_lo + s, s);
        cp_async_commit();
    }
    constexpr int kBlocks = C::KW / 128;
    Groups now = read_groups(c_lo, 0);
    for (int c = c_lo, st = 0; c < c_hi; ++c, st = st + 1 == C::kStages ? 0 : st + 1) {
        asm volatile("cp.async.wait_group %0;" ::"n"(C::kStages - 2) : "memory");
        // this thread's pieces of x into the order of the unpacked weights: 0 4 | 1 5 | 2 6 | 3 7
        for (int n = tid; n < nt * (C::kXRow / 16); n += 256) {
            uint4 *v = reinterpret_cast<uint4 *>(smem + st * C::kStage + C::kWStage + n * 16);
            const uint4 o = *v;
            *v = make_uint4(__byte_perm(o.x, o.z, 0x5410), __byte_perm(o.x, o.z, 0x7632), __byte_perm(o.y, o.w, 0x5410),
                            __byte_perm(o.y, o.w, 0x7632));
        }
        __syncthreads();
        if (c + C::kStages - 1 < c_hi) issue(c + C::kStages - 1, st == 0 ? C::kStages - 1 : st - 1);
        cp_async_commit();
        const unsigned char *wbase = smem + st * C::kStage, *xbase = wbase + C::kWStage;
#pragma unroll
        for (int blk = 0; blk < kBlocks; ++blk) {
            const Groups next = blk + 1 < kBlocks ? read_groups(c, blk + 1) : read_groups(c + 1, 0);
            float part[C::MT][C::NT][4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {                           // units of 32 columns
                if (u % GU == 0) {
#pragma unroll
                    for (int mt = 0; mt < C::MT; ++mt)
#pragma unroll
                        for (int n = 0; n < C::NT; ++n)
                            part[mt][n][0] = part[mt][n][1] = part[mt][n][2] = part[mt][n][3] = 0.f;
                }
                const int piece = (wk * C::KW + blk * 128) / 32 + u;
                uint32_t w[C::MT][2], zz[C::MT][2];
#pragma unroll
                for (int mt = 0; mt < C::MT; ++mt)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int r = (wr * C::MT + mt) * 16 + g4 + h * 8;
                        w[mt][h] = *reinterpret_cast<const uint32_t *>(wbase + r * C::kWRow + ((piece ^ (r & 7)) << 4) + t4 * 4);
                        zz[mt][h] = __shfl_sync(0xffffffffu, now.z[mt][h], u, 4);
                    }
                uint32_t f[C::MT][2][4];
#pragma unroll
                for (int mt = 0; mt < C::MT; ++mt)
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        f[mt][half][0] = nibbles(w[mt][0] >> (8 * half), zz[mt][0]);
                        f[mt][half][1] = nibbles(w[mt][1] >> (8 * half), zz[mt][1]);
                        f[mt][half][2] = nibbles(w[mt][0] >> (8 * half + 4), zz[mt][0]);
                        f[mt][half][3] = nibbles(w[mt][1] >> (8 * half + 4), zz[mt][1]);
                    }
#pragma unroll
                for (int n = 0; n < C::NT; ++n) {
                    const int t = n * 8 + g4;
                    const uint4 b = *reinterpret_cast<const uint4 *>(xbase + t * C::kXRow +
                                                                     (((piece * 4 + t4) ^ ((t & 1) << 2)) << 4));
#pragma unroll
                    for (int mt = 0; mt < C::MT; ++mt) {
                        mma_bf16(part[mt][n], f[mt][0][0], f[mt][0][1], f[mt][0][2], f[mt][0][3], b.x, b.y);
                        mma_bf16(part[mt][n], f[mt][1][0], f[mt][1][1], f[mt][1][2], f[mt][1][3], b.z, b.w);
                    }
                }
                if (u % GU == GU - 1) {
#pragma unroll
                    for (int mt = 0; mt < C::MT; ++mt) {
                        const float s0 = __shfl_sync(0xffffffffu, now.s[mt][0], u, 4);
                        const float s1 = __shfl_sync(0xffffffffu, now.s[mt][1], u, 4);
#pragma unroll
                        for (int n = 0; n < C::NT; ++n) {
                            acc[mt][n][0] = fmaf(s0, part[mt][n][0], acc[mt][n][0]);
                            acc[mt][n][1] = fmaf(s0, part[mt][n][1], acc[mt][n][1]);
                            acc[mt][n][2] = fmaf(s1, part[mt][n][2], acc[mt][n][2]);
                            acc[mt][n][3] = fmaf(s1, part[mt][n][3], acc[mt][n][3]);
                        }
                    }
                }
            }
            now = next;
        }
    }
    // ---- parts of the warps and the cluster, added in a fixed order
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();
    float *red = reinterpret_cast<float *>(smem);                   // [WK][T][kRedRow]
#pragma unroll
    for (int mt = 0; mt < C::MT; ++mt)
#pragma unroll
        for (int n = 0; n < C::NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int r = (wr * C::MT + mt) * 16 + g4 + (e >> 1) * 8, t = n * 8 + t4 * 2 + (e & 1);
                red[(wk * C::T + t) * C::kRedRow + r] = acc[mt][n][e];
            }
    if (cluster > 1)
        cluster_sync_all();
    else
        __syncthreads();
    const int slice = C::R / cluster, r_lo = rank * slice;
    const uint32_t red_at = smem_u32(red);
    for (int i = tid; i < nt * slice; i += 256) {
        const int t = i / slice, r = r_lo + i % slice;
        if (row0 + r >= a.d_out) continue;
        float sum = 0.f;
        for (int p = 0; p < cluster; ++p) {
            const uint32_t peer = cluster > 1 ? map_peer(red_at, p) : red_at;
#pragma unroll
            for (int k = 0; k < C::WK; ++k) {
                const uint32_t at = peer + ((k * C::T + t) * C::kRedRow + r) * 4;
                float v;
                if (cluster > 1)
                    v = __uint_as_float(ld_peer_u32(at));
                else
                    v = red[(k * C::T + t) * C::kRedRow + r];
                sum += v;
            }
        }
        static_cast<__nv_bfloat16 *>(a.y)[(size_t)(tok0 + t) * a.y_stride + row0 + r] = __float2bfloat16_rn(sum);
    }
    if (cluster > 1) cluster_sync_all();                            // the peers have read this CTA's parts
}

template <class C, int GU>
cudaError_t launch_tiles(const LinearArgs &a, int sms, cudaStream_t st) {
    auto kernel = linear_tiles_kernel<C, GU>;
    static std::atomic<uint64_t> ready{0};
    if (!device_bit(ready)) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
        if (e != cudaSuccess) return e;
        set_device_bit(ready);
    }
    const int row_blocks = (a.d_out + C::R - 1) / C::R, tok_blocks = (a.n_tokens + C::T - 1) / C::T;
    const int chunks = (a.d_in + C::KC - 1) / C::KC;
    int cluster = 1;
    while (cluster < 8 && 2 * cluster <= chunks && (long long)row_blocks * tok_blocks * cluster < sms) cluster *= 2;
    const int x_vec = aligned16(a.x) && a.x_stride % 8 == 0;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(row_blocks * cluster, tok_blocks);
    cfg.blockDim = dim3(256);
    cfg.dynamicSmemBytes = C::kSmem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, a, cluster, x_vec);
}

template <class C>
cudaError_t launch_group(const LinearArgs &a, int sms, cudaStream_t st) {
    switch (a.group) {
        case 32: return launch_tiles<C, 1>(a, sms, st);
        case 64: return launch_tiles<C, 2>(a, sms, st);
        default: return launch_tiles<C, 4>(a, sms, st);
    }
}

// Tokens of a CTA's tile and, with them, its rows: the more tokens, the more
// rows share their copy of x.
cudaError_t launch_bf16(const LinearArgs &a, int sms, cudaStream_t st) {
    if (a.n_tokens <= 8) return launch_group<LinearTile<1, 1, 2, 512, 4, 3>>(a, sms, st);
    if (a.n_tokens <= 16) return launch_group<LinearTile<2, 1, 4, 512, 3, 2>>(a, sms, st);
    if (a.n_tokens <= 32) return launch_group<LinearTile<4, 1, 8, 256, 3, 2>>(a, sms, st);
    return launch_group<LinearTile<8, 1, 8, 256, 2, 2>>(a, sms, st);
}

template <typename T>
cudaError_t launch_rows(const LinearArgs &a, cudaStream_t st) {
    constexpr int TT = 8;
    dim3 grid((a.d_out + 7) / 8, (a.n_tokens + TT - 1) / TT);
    linear_rows_kernel<T, TT><<<grid, 256, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace
}  // namespace lora

using namespace lora;
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
    if (d->dtype == LORA_DTYPE_F32) return launched("base_linear", launch_rows<float>(a, st));
    const int sms = sm_count();
    if (sms < 1) return fail(LORA_ERR_CUDA, "base_linear: no CUDA device");
    return launched("base_linear", launch_bf16(a, sms, st));
}
