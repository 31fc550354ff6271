// matvec.cu -- products of a few bf16 token vectors with a weight matrix held
// in 4 bits with group scales, in the quantisers' own row-major layouts:
//   y[t, n] = sum_k x[t, k] * s[n, k / G] * c[n, k]
// c E2M1, s UE8M0 with G = 32 (MX) or UE4M3 with G = 16 (NVFP4).  Every weight
// byte is used once per 8 tokens, so the kernel is bound by the HBM stream of
// N K (1/2 + 1/G) bytes.
//
// A block's eight warps cut K into eight slices and walk over tiles of 16
// rows; a warp streams its slice of a tile through a ring of cp.async stages
// (16-byte pieces, no waits on other warps), and multiplies on the tensor
// cores: mma.m16n8k16 with the weights as the 16-row operand and 8 tokens as
// the other, so 1 to 8 tokens cost the same.  c is exact in fp16.  The tokens
// are brought to fp16 too, each token's slice scaled by a power of two that
// puts its largest finite magnitude in [2^14, 2^15): bf16's 8 bits fit, and an
// element loses bits only below 2^-31 of that largest one (it is then off by
// at most 2^-40 of it, less than a rounding of the fp32 sum).  The group
// scale multiplies the fp32 sum of its group.  The eight slices' sums meet in
// shared memory and are added in slice order.
#include <cuda_fp16.h>

#include "moe_common.cuh"
#include "moe_internal.h"

namespace moe {
namespace {

constexpr int kMvWarps = 8;
constexpr int kMvRows = 16;                        // rows of a tile (MMA M)
constexpr int kMvTokens = 8;                       // tokens of a pass (MMA N)
constexpr int kMvChunk = 512;                      // K elements of a stage
constexpr int kMvRowBytes = kMvChunk / 2 + 16;     // padded: a quad's words of 8 rows fall into 32 banks
constexpr int kMvStageBytes = kMvRows * kMvRowBytes;
constexpr int kMvStages = 3;
constexpr int kMvRingBytes = kMvWarps * kMvStages * kMvStageBytes;
constexpr int kMvMaxXBytes = 116 * 1024;           // tokens held in shared memory
constexpr int kMvMaxK = 57344;                     // one token fits there
static_assert(kMvRingBytes + kMvMaxXBytes + 2 * kMvWarps * kMvRows * kMvTokens * 4 <= 232448, "shared memory budget");
static_assert((2 * kMvMaxK + 127) / 128 * 128 + 64 <= kMvMaxXBytes, "one token");

struct MatvecArgs {
    const __nv_bfloat16 *x;   // [T, K]
    const uint8_t *w;         // [N, K / 2]
    const uint8_t *sf;        // [N, K / G]
    __nv_bfloat16 *y;         // [T, N]
    int T, N, K;
    int tokens;               // tokens of a pass (blockIdx.y), <= kMvTokens
    int slice;                // K elements of a warp's slice, a multiple of 32
    int x_stride;             // bytes of a token in shared memory
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool real) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(real ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}

// The two E2M1 codes of byte b of w as fp16 (the low nibble in the low half).
__device__ __forceinline__ uint32_t e2m1x2_to_half2(uint32_t w, int b) {
    const __half2_raw h = __nv_cvt_fp4x2_to_halfraw2(__nv_fp4x2_storage_t((w >> (8 * b)) & 0xFFu), __NV_E2M1);
    return uint32_t(h.x) | (uint32_t(h.y) << 16);
}

__device__ __forceinline__ void mma_16x8x16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                            uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 2^(b - 127), b = 255 is NaN (the fp32 value of an UE8M0 byte).
__device__ __forceinline__ float ue8m0_value(uint32_t b) {
    return __uint_as_float(b == 0u ? 0x00400000u : b == 255u ? 0x7FC00000u : b << 23);
}
// The value of an UE4M3 byte (bit 7 is unused), 0x7F is NaN.
__device__ __forceinline__ float ue4m3_value(uint32_t b) {
    const uint32_t c = b & 0x7Fu;
    return c == 0x7Fu ? __uint_as_float(0x7FC00000u) : e4m3_mag_value(c);
}

// acc += d * scale: rows g (first two sums) and g + 8 (last two).
__device__ __forceinline__ void add_group(float (&acc)[4], const float (&d)[4], float s0, float s1) {
    acc[0] = fmaf(d[0], s0, acc[0]);
    acc[1] = fmaf(d[1], s0, acc[1]);
    acc[2] = fmaf(d[2], s1, acc[2]);
    acc[3] = fmaf(d[3], s1, acc[3]);
}

template <bool kNv>
__global__ void __launch_bounds__(kMvWarps * 32) fp4_matvec_kernel(const MatvecArgs args) {
    constexpr int kGroup = kNv ? 16 : 32;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float sums[2][kMvWarps][kMvRows * kMvTokens];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, t = lane & 3;
    const int tok0 = int(blockIdx.y) * args.tokens;
    const int ntok = min(args.tokens, args.T - tok0);
    const int k_lo = min(warp * args.slice, args.K), k_hi = min(k_lo + args.slice, args.K);
    const int chunks = (k_hi - k_lo + kMvChunk - 1) / kMvChunk;
    const int tiles = (args.N + kMvRows - 1) / kMvRows;
    uint8_t *xs = smem;
    uint8_t *ring = smem + args.tokens * args.x_stride + warp * kMvStages * kMvStageBytes;
    const int64_t w_ld = args.K / 2, sf_ld = args.K / kGroup;

    pdl_wait();
    pdl_trigger();
    // stage `i` of this warp's stream: chunk i % chunks of tile blockIdx.x + (i / chunks) gridDim.x
    int load_tile = blockIdx.x, load_chunk = 0, load_slot = 0;
    auto load_next = [&]() {
        if (load_tile < tiles && chunks > 0) {
            const int k0 = k_lo + load_chunk * kMvChunk;
            const int pieces = (min(kMvChunk, k_hi - k0)) / 32;  // 16-byte pieces of a row, 1 .. 16
            const uint32_t dst = smem_u32(ring + load_slot * kMvStageBytes);
#pragma unroll
            for (int i = 0; i < kMvRows * 16 / 32; ++i) {
                const int r = i * 2 + (lane >> 4), p = lane & 15;
                const int n = load_tile * kMvRows + r;
                const bool real = n < args.N;
                if (p < pieces)
                    cp_async16(dst + r * kMvRowBytes + p * 16, args.w + (real ? n : 0) * w_ld + k0 / 2 + p * 16, real);
            }
            if (++load_chunk == chunks) {
                load_chunk = 0;
                load_tile += gridDim.x;
            }
        }
        cp_async_commit();
        if (++load_slot == kMvStages) load_slot = 0;
    };
#pragma unroll
    for (int i = 0; i < kMvStages - 1; ++i) load_next();

    // this warp's slice of the tokens in fp16
    float unscale[2] = {0.0f, 0.0f};  // of tokens 2t and 2t + 1, the columns of this lane's sums
    for (int j = 0; j < ntok; ++j) {
        const __nv_bfloat16 *xr = args.x + int64_t(tok0 + j) * args.K;
        float amax = 0.0f;
        for (int k = k_lo + lane * 2; k < k_hi; k += 64) {
            const float2 v = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(xr + k));
            const float a = fabsf(v.x), b = fabsf(v.y);
            if (a <= 3.4e38f) amax = fmaxf(amax, a);
            if (b <= 3.4e38f) amax = fmaxf(amax, b);
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, d));
        // 2^shift brings amax into [2^14, 2^15); both factors are normal numbers
        const int shift = min(max(14 - (int(__float_as_uint(amax) >> 23) - 127), -113), 126);
        const float mul = amax > 0.0f ? __uint_as_float(uint32_t(127 + shift) << 23) : 1.0f;
        const float inv = amax > 0.0f ? __uint_as_float(uint32_t(127 - shift) << 23) : 1.0f;
        if (j == 2 * t) unscale[0] = inv;
        if (j == 2 * t + 1) unscale[1] = inv;
        for (int k = k_lo + lane * 2; k < k_hi; k += 64) {
            const float2 v = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(xr + k));
            *reinterpret_cast<__half2 *>(xs + j * args.x_stride + k * 2) = __floats2half2_rn(v.x * mul, v.y * mul);
        }
    }
    __syncwarp();

    const uint8_t *xrow = xs + min(g, ntok - 1) * args.x_stride;  // token g
    int slot = 0, buf = 0;
    for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x, buf ^= 1) {
        float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        const int n0 = tile * kMvRows + g;
        const uint8_t *s0 = args.sf + int64_t(min(n0, args.N - 1)) * sf_ld;
        const uint8_t *s1 = args.sf + int64_t(min(n0 + 8, args.N - 1)) * sf_ld;
        for (int c = 0; c < chunks; ++c) {
            cp_async_wait<kMvStages - 2>();
            __syncwarp();  // this stage has landed for every lane, and the one before it is read
            load_next();
            const uint8_t *st = ring + slot * kMvStageBytes + g * kMvRowBytes;
            const int k0 = k_lo + c * kMvChunk;
            const int groups = min(kMvChunk, k_hi - k0) / 32;
#pragma unroll 4
            for (int i = 0; i < groups; ++i) {
                const int k = k0 + i * 32;
                if constexpr (kNv) {
                    // a group of 16 is one step: lane t holds its elements 4t .. 4t + 3
#pragma unroll
                    for (int s = 0; s < 2; ++s) {
                        const uint32_t wa = *reinterpret_cast<const uint16_t *>(st + i * 16 + s * 8 + t * 2);
                        const uint32_t wb =
                            *reinterpret_cast<const uint16_t *>(st + i * 16 + s * 8 + t * 2 + 8 * kMvRowBytes);
                        const uint2 xv = *reinterpret_cast<const uint2 *>(xrow + (k + s * 16 + t * 4) * 2);
                        float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                        mma_16x8x16(d, e2m1x2_to_half2(wa, 0), e2m1x2_to_half2(wb, 0), e2m1x2_to_half2(wa, 1),
                                    e2m1x2_to_half2(wb, 1), xv.x, xv.y);
                        const int sg = k / 16 + s;
                        add_group(acc, d, ue4m3_value(__ldg(s0 + sg)), ue4m3_value(__ldg(s1 + sg)));
                    }
                } else {
                    // a group of 32 is two steps: lane t holds its elements 8t .. 8t + 7
                    const uint32_t wa = *reinterpret_cast<const uint32_t *>(st + i * 16 + t * 4);
                    const uint32_t wb = *reinterpret_cast<const uint32_t *>(st + i * 16 + t * 4 + 8 * kMvRowBytes);
                    const uint4 xv = *reinterpret_cast<const uint4 *>(xrow + (k + t * 8) * 2);
                    float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                    mma_16x8x16(d, e2m1x2_to_half2(wa, 0), e2m1x2_to_half2(wb, 0), e2m1x2_to_half2(wa, 1),
                                e2m1x2_to_half2(wb, 1), xv.x, xv.y);
                    mma_16x8x16(d, e2m1x2_to_half2(wa, 2), e2m1x2_to_half2(wb, 2), e2m1x2_to_half2(wa, 3),
                                e2m1x2_to_half2(wb, 3), xv.z, xv.w);
                    add_group(acc, d, ue8m0_value(__ldg(s0 + k / 32)), ue8m0_value(__ldg(s1 + k / 32)));
                }
            }
            if (++slot == kMvStages) slot = 0;
        }
        // rows g and g + 8, tokens 2t and 2t + 1 of this slice
        float *mine = sums[buf][warp];
        mine[g * kMvTokens + 2 * t] = acc[0] * unscale[0];
        mine[g * kMvTokens + 2 * t + 1] = acc[1] * unscale[1];
        mine[(g + 8) * kMvTokens + 2 * t] = acc[2] * unscale[0];
        mine[(g + 8) * kMvTokens + 2 * t + 1] = acc[3] * unscale[1];
        __syncthreads();
        if (threadIdx.x < kMvRows * kMvTokens) {
            const int j = threadIdx.x >> 4, r = threadIdx.x & 15;
            const int n = tile * kMvRows + r;
            if (j < ntok && n < args.N) {
                float v = 0.0f;
#pragma unroll
                for (int i = 0; i < kMvWarps; ++i) v += sums[buf][i][r * kMvTokens + j];
                args.y[int64_t(tok0 + j) * args.N + n] = __float2bfloat16_rn(v);
            }
        }
    }
}

template <bool kNv>
cudaError_t launch_matvec(const MatvecArgs &a, dim3 grid, size_t smem, cudaStream_t stream) {
    const cudaError_t e = set_max_dynamic_smem(reinterpret_cast<const void *>(fp4_matvec_kernel<kNv>),
                                               kMvRingBytes + kMvMaxXBytes);
    if (e != cudaSuccess) return e;
    return launch_pdl(fp4_matvec_kernel<kNv>, grid, dim3(kMvWarps * 32), smem, stream, a);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" moe_status_t moe_fp4_matvec(const void *x_bf16, const void *w_fp4, const void *w_sf, void *y_bf16, int T,
                                       int N, int K, int format, moe_stream_t stream) {
    if (T < 0 || N <= 0 || K <= 0 || (format != MOE_FP4_MX && format != MOE_FP4_NVFP4)) return MOE_ERR_INVALID_ARG;
    if (K % 32 || K > kMvMaxK || T > 65535) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (T == 0) return MOE_OK;
    if (!x_bf16 || !w_fp4 || !w_sf || !y_bf16 || !aligned(x_bf16, 16) || !aligned(w_fp4, 16) || !aligned(y_bf16, 2))
        return MOE_ERR_INVALID_ARG;
    DeviceScope dev(y_bf16);
    if (dev.status != MOE_OK) return dev.status;
    MatvecArgs a{};
    a.x = static_cast<const __nv_bfloat16 *>(x_bf16);
    a.w = static_cast<const uint8_t *>(w_fp4);
    a.sf = static_cast<const uint8_t *>(w_sf);
    a.y = static_cast<__nv_bfloat16 *>(y_bf16);
    a.T = T;
    a.N = N;
    a.K = K;
    // the tokens of a quarter-warp's 16-byte reads are 64 bytes apart modulo 128
    a.x_stride = (2 * K + 127) / 128 * 128 + 64;
    if (a.x_stride > kMvMaxXBytes) return MOE_ERR_UNSUPPORTED_SHAPE;
    const int fit = kMvMaxXBytes / a.x_stride;
    a.tokens = T < kMvTokens ? T : kMvTokens;
    if (a.tokens > fit) a.tokens = fit;
    a.slice = (K / 32 + kMvWarps - 1) / kMvWarps * 32;
    const int tiles = (N + kMvRows - 1) / kMvRows, sms = num_sms();
    const dim3 grid(unsigned(tiles < sms ? tiles : sms), unsigned((T + a.tokens - 1) / a.tokens));
    const size_t smem = size_t(a.tokens) * a.x_stride + kMvRingBytes;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e =
        format == MOE_FP4_NVFP4 ? launch_matvec<true>(a, grid, smem, st) : launch_matvec<false>(a, grid, smem, st);
    return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
