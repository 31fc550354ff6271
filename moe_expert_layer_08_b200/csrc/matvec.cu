// matvec.cu -- products of a few bf16 token vectors with a weight matrix held
// in 4 bits with group scales, in the quantisers' own row-major layouts:
//   y[t, n] = sum_k x[t, k] * s[n, k / G] * c[n, k]
// c E2M1, s UE8M0 with G = 32 (MX) or UE4M3 with G = 16 (NVFP4).  Every weight
// byte is used once per 8 tokens, so the kernel is bound by the HBM stream of
// N K (1/2 + 1/G) bytes.
//
// A block has two teams of eight warps; a team cuts K into eight slices and
// walks over tiles of 16 rows.  A warp streams its slice of a tile, weights and
// scales, through its own ring of cp.async stages (no waits on other warps), and
// multiplies on the tensor cores: mma.m16n8k16 with the weights as the 16-row
// operand and 8 tokens as the other, so 1 to 8 tokens cost the same.  c is exact
// in fp16.  The tokens are brought to fp16 too, each token's slice scaled by a
// power of two that puts its largest finite magnitude in [2^14, 2^15): bf16's 8
// bits fit, and an element loses bits only below 2^-31 of that largest one (it
// is then off by at most 2^-40 of it, less than a rounding of the fp32 sum).
// The group scale multiplies the fp32 sum of its group.  The eight slices' sums
// meet in shared memory and are added in slice order.
#include <cuda_fp16.h>

#include "moe_common.cuh"
#include "moe_internal.h"

namespace moe {
namespace {

constexpr int kMvWarps = 8;                        // of a team: slices of K
constexpr int kMvTeams = 2;
constexpr int kMvRows = 16;                        // rows of a tile (MMA M)
constexpr int kMvTokens = 8;                       // tokens of a pass (MMA N)
constexpr int kMvChunk = 256;                      // K elements of a stage
constexpr int kMvRowBytes = kMvChunk / 2 + 16;     // padded: a quad's words of 8 rows fall into 32 banks
// a row's scales of a stage (at most 16 bytes) inside two aligned 16-byte
// pieces, padded likewise
constexpr int kMvScaleBytes = 48;
constexpr int kMvStageBytes = kMvRows * (kMvRowBytes + kMvScaleBytes);
constexpr int kMvSumBytes = 2 * kMvTeams * kMvWarps * kMvRows * kMvTokens * 4;
constexpr int kMvMaxSmem = 232448;
constexpr int kMvMaxK = 57344;
constexpr int mv_fixed_bytes(int stages) { return kMvTeams * kMvWarps * stages * kMvStageBytes + kMvSumBytes; }
static_assert(mv_fixed_bytes(2) + (2 * kMvMaxK + 127) / 128 * 128 + 64 <= kMvMaxSmem, "one token of the largest K");

// The E2M1 codes in bits 4j.. and 4j + 16.. of w as fp16 times 2^-14: sign,
// exponent and mantissa bits in place (E2M1's bits are those of an fp16 number
// with another exponent bias, subnormals included).  The shifts are products
// with factors the compiler does not know, which go to the multiply-add pipe:
// the integer pipe, at half its rate, bounds this kernel.  (The conversion
// instruction ran at a fraction of that: 39 us at N = 14336, K = 7168; byte
// permutes 29 us.)
struct PairFactors {
    uint32_t mag[3], sign[3];  // 2^(9 - 4j), 2^(12 - 4j)
};
struct MatvecArgs {
    const __nv_bfloat16 *x;   // [T, K]
    const uint8_t *w;         // [N, K / 2]
    const uint8_t *sf;        // [N, K / G]
    __nv_bfloat16 *y;         // [T, N]
    int T, N, K;
    int tokens;               // tokens of a pass (blockIdx.y), <= kMvTokens
    int slice;                // K elements of a warp's slice, a multiple of 32
    int x_stride;             // bytes of a token in shared memory
    PairFactors factors;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}

template <int j>
__device__ __forceinline__ uint32_t e2m1_pair(uint32_t w, const PairFactors &f) {
    if constexpr (j == 3) return (w & 0x80008000u) | ((w >> 3) & 0x0E000E00u);
    else return (w & (0x00070007u << (4 * j))) * f.mag[j] + (w & (0x00080008u << (4 * j))) * f.sign[j];
}

// d = a b + c: c is zero for the first step of a group
__device__ __forceinline__ void mma_16x8x16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                            uint32_t b0, uint32_t b1, const float (&c)[4]) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%10, %11, %12, %13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
}

// 2^(b - 127) for a UE8M0 byte b <= 254 (a subnormal for b = 0), infinity for 255.
__device__ __forceinline__ float ue8m0_value(uint32_t b) { return __uint_as_float(max(b << 23, 0x00400000u)); }
// 2^-8 times the value of a UE4M3 byte below 0x7F (bit 7 is not read): its bits
// are those of an fp16 number with an exponent bias of 15 instead of 7.
__device__ __forceinline__ float ue4m3_value_256th(uint32_t b) {
    __half_raw h;
    h.x = static_cast<unsigned short>((b & 0x7Fu) << 7);
    return __half2float(__half(h));
}

// acc += d * scale: rows g (first two sums) and g + 8 (last two).
__device__ __forceinline__ void add_group(float (&acc)[4], const float (&d)[4], float s0, float s1) {
    acc[0] = fmaf(d[0], s0, acc[0]);
    acc[1] = fmaf(d[1], s0, acc[1]);
    acc[2] = fmaf(d[2], s1, acc[2]);
    acc[3] = fmaf(d[3], s1, acc[3]);
}

template <bool kNv, int kStages>
__global__ void __launch_bounds__(kMvTeams * kMvWarps * 32, 1) fp4_matvec_kernel(const MatvecArgs args) {
    constexpr int kGroup = kNv ? 16 : 32;
    extern __shared__ __align__(128) uint8_t smem[];
    const int wid = threadIdx.x >> 5, team = wid / kMvWarps, warp = wid % kMvWarps, lane = threadIdx.x & 31;
    const int g = lane >> 2, t = lane & 3;
    const int tok0 = int(blockIdx.y) * args.tokens;
    const int ntok = min(args.tokens, args.T - tok0);
    const int k_lo = min(warp * args.slice, args.K), k_hi = min(k_lo + args.slice, args.K);
    const int chunks = (k_hi - k_lo + kMvChunk - 1) / kMvChunk;
    const int tiles = (args.N + kMvRows - 1) / kMvRows;
    const int first = int(blockIdx.x) + team * int(gridDim.x), step = kMvTeams * int(gridDim.x);
    uint8_t *ring = smem + wid * kStages * kMvStageBytes;
    float *sums = reinterpret_cast<float *>(smem + kMvTeams * kMvWarps * kStages * kMvStageBytes) +
                  team * 2 * kMvWarps * kMvRows * kMvTokens;
    uint8_t *xs = smem + mv_fixed_bytes(kStages);
    const int64_t w_ld = args.K / 2, sf_ld = args.K / kGroup, sf_end = args.N * sf_ld;

    pdl_wait();
    pdl_trigger();
    // the stages of this warp's stream in order: the chunks of its tiles
    int load_tile = first, load_chunk = 0, load_slot = 0;
    auto load_next = [&]() {
        if (load_tile < tiles && chunks > 0) {
            const int k0 = k_lo + load_chunk * kMvChunk;
            const int elems = min(kMvChunk, k_hi - k0);
            const uint32_t dst = smem_u32(ring + load_slot * kMvStageBytes);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = i * 4 + (lane >> 3), p = lane & 7;
                const int n = load_tile * kMvRows + r;
                const bool real = n < args.N;
                if (p * 32 < elems)
                    cp_async16(dst + r * kMvRowBytes + p * 16, args.w + (real ? n : 0) * w_ld + k0 / 2 + p * 16,
                               real ? 16 : 0);
            }
            // the aligned 16-byte pieces that hold the scales, cut at the array's end
            const int n = load_tile * kMvRows + (lane >> 1);
            const int64_t s = int64_t(n) * sf_ld + k0 / kGroup, p = (s & ~int64_t(15)) + (lane & 1) * 16;
            if (n < args.N && p < s + elems / kGroup)
                cp_async16(dst + kMvRows * kMvRowBytes + (lane >> 1) * kMvScaleBytes + (lane & 1) * 16, args.sf + p,
                           int(min(int64_t(16), sf_end - p)));
            if (++load_chunk == chunks) {
                load_chunk = 0;
                load_tile += step;
            }
        }
        cp_async_commit();
        if (++load_slot == kStages) load_slot = 0;
    };
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) load_next();

    // the tokens' slices in fp16: each of the two warps of a slice takes every second token
    float *unscales = sums + kMvWarps * kMvRows * kMvTokens;  // in the second buffer of sums until the first tile ends
    float unscale[2];                                         // of tokens 2t and 2t + 1, the columns of this lane's sums
    for (int j = 0; j < ntok; ++j) {
        const __nv_bfloat16 *xr = args.x + int64_t(tok0 + j) * args.K;
        float amax = 0.0f;
        for (int k = k_lo + lane * 8; k < k_hi; k += 256) {
            const uint4 u = *reinterpret_cast<const uint4 *>(xr + k);
            const uint32_t v[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float a = __uint_as_float((v[i] << 16) & 0x7FFFFFFFu), b = __uint_as_float(v[i] & 0x7FFF0000u);
                if (a <= 3.4e38f) amax = fmaxf(amax, a);
                if (b <= 3.4e38f) amax = fmaxf(amax, b);
            }
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, d));
        // 2^shift brings amax into [2^14, 2^15); both factors are normal numbers
        const int shift = min(max(14 - (int(__float_as_uint(amax) >> 23) - 127), -113), 126);
        const float mul = amax > 0.0f ? __uint_as_float(uint32_t(127 + shift) << 23) : 1.0f;
        if (lane == 0) unscales[warp * kMvTokens + j] = amax > 0.0f ? __uint_as_float(uint32_t(127 - shift) << 23) : 1.0f;
        if ((j & 1) == team)
            for (int k = k_lo + lane * 8; k < k_hi; k += 256) {
                const uint4 u = *reinterpret_cast<const uint4 *>(xr + k);
                const uint32_t v[4] = {u.x, u.y, u.z, u.w};
                // in the order of the decoded weights: NVFP4 elements 0 and 2, 1 and 3, 4
                // and 6, 5 and 7, MX elements 0 and 4, 1 and 5, 2 and 6, 3 and 7
                uint32_t h[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int lo = kNv ? (i & 1) + 4 * (i >> 1) : i, hi = lo + (kNv ? 2 : 4);
                    const auto value = [&](int e) { return __uint_as_float(e & 1 ? v[e >> 1] & 0xFFFF0000u : v[e >> 1] << 16); };
                    const __half2 p = __floats2half2_rn(value(lo) * mul, value(hi) * mul);
                    h[i] = *reinterpret_cast<const uint32_t *>(&p);
                }
                *reinterpret_cast<uint4 *>(xs + j * args.x_stride + k * 2) = make_uint4(h[0], h[1], h[2], h[3]);
            }
    }
    __syncthreads();
    unscale[0] = 2 * t < ntok ? unscales[warp * kMvTokens + 2 * t] : 0.0f;
    unscale[1] = 2 * t + 1 < ntok ? unscales[warp * kMvTokens + 2 * t + 1] : 0.0f;

    const uint8_t *xrow = xs + min(g, ntok - 1) * args.x_stride;  // token g
    int slot = 0, buf = 0;
    for (int tile = first; tile < tiles; tile += step, buf ^= 1) {
        float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        // rows g and g + 8 have a NaN scale: the largest byte of UE4M3; for UE8M0, whose
        // byte 255 becomes an infinity, the sum of zero times the scales
        uint32_t top0 = 0, top1 = 0;
        float nan0 = 0.0f, nan1 = 0.0f;
        // where rows g and g + 8 have their first scale inside its 16-byte piece
        const int64_t s0 = (int64_t(tile) * kMvRows + g) * sf_ld + k_lo / kGroup, s1 = s0 + 8 * sf_ld;
        for (int c = 0; c < chunks; ++c) {
            cp_async_wait<kStages - 2>();
            __syncwarp();  // this stage has landed for every lane, and the one before it is read
            load_next();
            const uint8_t *st = ring + slot * kMvStageBytes + g * kMvRowBytes;
            const uint8_t *sc = ring + slot * kMvStageBytes + kMvRows * kMvRowBytes + g * kMvScaleBytes;
            const uint8_t *sc0 = sc + ((s0 + c * (kMvChunk / kGroup)) & 15);
            const uint8_t *sc1 = sc + 8 * kMvScaleBytes + ((s1 + c * (kMvChunk / kGroup)) & 15);
            const uint8_t *xk = xrow + (k_lo + c * kMvChunk) * 2;
            const float zero[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            // 32 elements: two groups of 16 or one of 32
            auto block = [&](int i) {
                float d[4];
                uint32_t a[4];
                if constexpr (kNv) {
                    // a group of 16 is one step: lane t holds its elements 4t .. 4t + 3
#pragma unroll
                    for (int s = 0; s < 2; ++s) {
                        const uint32_t wa = *reinterpret_cast<const uint16_t *>(st + i * 16 + s * 8 + t * 2);
                        const uint32_t wb =
                            *reinterpret_cast<const uint16_t *>(st + i * 16 + s * 8 + t * 2 + 8 * kMvRowBytes);
                        const uint2 xv = *reinterpret_cast<const uint2 *>(xk + (i * 32 + s * 16 + t * 4) * 2);
                        const uint32_t pa = __byte_perm(wa, 0u, 0x4140u), pb = __byte_perm(wb, 0u, 0x4140u);
                        a[0] = e2m1_pair<0>(pa, args.factors);
                        a[1] = e2m1_pair<0>(pb, args.factors);
                        a[2] = e2m1_pair<1>(pa, args.factors);
                        a[3] = e2m1_pair<1>(pb, args.factors);
                        mma_16x8x16(d, a[0], a[1], a[2], a[3], xv.x, xv.y, zero);
                        const uint32_t b0 = sc0[2 * i + s] & 0x7Fu, b1 = sc1[2 * i + s] & 0x7Fu;
                        top0 = max(top0, b0);
                        top1 = max(top1, b1);
                        add_group(acc, d, ue4m3_value_256th(b0), ue4m3_value_256th(b1));
                    }
                } else {
                    // a group of 32 is two steps: lane t holds its elements 8t .. 8t + 7
                    const uint32_t wa = *reinterpret_cast<const uint32_t *>(st + i * 16 + t * 4);
                    const uint32_t wb = *reinterpret_cast<const uint32_t *>(st + i * 16 + t * 4 + 8 * kMvRowBytes);
                    const uint4 xv = *reinterpret_cast<const uint4 *>(xk + (i * 32 + t * 8) * 2);
                    a[0] = e2m1_pair<0>(wa, args.factors);
                    a[1] = e2m1_pair<0>(wb, args.factors);
                    a[2] = e2m1_pair<1>(wa, args.factors);
                    a[3] = e2m1_pair<1>(wb, args.factors);
                    mma_16x8x16(d, a[0], a[1], a[2], a[3], xv.x, xv.y, zero);
                    a[0] = e2m1_pair<2>(wa, args.factors);
                    a[1] = e2m1_pair<2>(wb, args.factors);
                    a[2] = e2m1_pair<3>(wa, args.factors);
                    a[3] = e2m1_pair<3>(wb, args.factors);
                    mma_16x8x16(d, a[0], a[1], a[2], a[3], xv.z, xv.w, d);
                    const float f0 = ue8m0_value(sc0[i]), f1 = ue8m0_value(sc1[i]);
                    nan0 = fmaf(f0, 0.0f, nan0);
                    nan1 = fmaf(f1, 0.0f, nan1);
                    add_group(acc, d, f0, f1);
                }
            };
            const int blocks = min(kMvChunk, k_hi - k_lo - c * kMvChunk) / 32;
            if (blocks == kMvChunk / 32) {
#pragma unroll
                for (int i = 0; i < kMvChunk / 32; ++i) block(i);
            } else {
#pragma unroll 1
                for (int i = 0; i < blocks; ++i) block(i);
            }
            if (++slot == kStages) slot = 0;
        }
        if (kNv) {
            nan0 = top0 == 0x7Fu ? __uint_as_float(0x7FC00000u) : 0.0f;
            nan1 = top1 == 0x7Fu ? __uint_as_float(0x7FC00000u) : 0.0f;
        }
        // 2^14 for the codes, 2^8 for the UE4M3 scales' exponent bias
        constexpr float kBack = kNv ? 0x1p22f : 0x1p14f;
        // rows g and g + 8, tokens 2t and 2t + 1 of this slice
        float *mine = sums + (buf * kMvWarps + warp) * kMvRows * kMvTokens;
        mine[g * kMvTokens + 2 * t] = (acc[0] * kBack + nan0) * unscale[0];
        mine[g * kMvTokens + 2 * t + 1] = (acc[1] * kBack + nan0) * unscale[1];
        mine[(g + 8) * kMvTokens + 2 * t] = (acc[2] * kBack + nan1) * unscale[0];
        mine[(g + 8) * kMvTokens + 2 * t + 1] = (acc[3] * kBack + nan1) * unscale[1];
        asm volatile("bar.sync %0, %1;" ::"r"(1 + team), "r"(kMvWarps * 32) : "memory");
        const int id = warp * 32 + lane;
        if (id < kMvRows * ntok) {
            const int j = id >> 4, r = id & 15;
            const int n = tile * kMvRows + r;
            if (n < args.N) {
                float v = 0.0f;
#pragma unroll
                for (int i = 0; i < kMvWarps; ++i)
                    v += sums[(buf * kMvWarps + i) * kMvRows * kMvTokens + r * kMvTokens + j];
                args.y[int64_t(tok0 + j) * args.N + n] = __float2bfloat16_rn(v);
            }
        }
    }
}

template <bool kNv, int kStages>
cudaError_t launch_matvec(const MatvecArgs &a, dim3 grid, cudaStream_t stream) {
    const cudaError_t e =
        set_max_dynamic_smem(reinterpret_cast<const void *>(fp4_matvec_kernel<kNv, kStages>), kMvMaxSmem);
    if (e != cudaSuccess) return e;
    return launch_pdl(fp4_matvec_kernel<kNv, kStages>, grid, dim3(kMvTeams * kMvWarps * 32),
                      size_t(mv_fixed_bytes(kStages) + a.tokens * a.x_stride), stream, a);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" moe_status_t moe_fp4_matvec(const void *x_bf16, const void *w_fp4, const void *w_sf, void *y_bf16, int T,
                                       int N, int K, int format, moe_stream_t stream) {
    if (T < 0 || N <= 0 || K <= 0 || (format != MOE_FP4_MX && format != MOE_FP4_NVFP4)) return MOE_ERR_INVALID_ARG;
    if (K % 32 || K > kMvMaxK || T > 65535) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (T == 0) return MOE_OK;
    if (!x_bf16 || !w_fp4 || !w_sf || !y_bf16 || !aligned(x_bf16, 16) || !aligned(w_fp4, 16) ||
        !aligned(w_sf, 16) || !aligned(y_bf16, 2))
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
    a.factors = {{512, 32, 2}, {4096, 256, 16}};
    // the tokens of a quarter-warp's 16-byte reads are 64 bytes apart modulo 128
    a.x_stride = (2 * K + 127) / 128 * 128 + 64;
    const auto fits = [&](int stages) { return (kMvMaxSmem - mv_fixed_bytes(stages)) / a.x_stride; };
    a.tokens = T < kMvTokens ? T : kMvTokens;
    if (a.tokens > fits(2)) a.tokens = fits(2);
    a.slice = (K / 32 + kMvWarps - 1) / kMvWarps * 32;
    const int tiles = (N + kMvRows - 1) / kMvRows, sms = num_sms();
    const dim3 grid(unsigned(tiles < sms ? tiles : sms), unsigned((T + a.tokens - 1) / a.tokens));
    const bool nv = format == MOE_FP4_NVFP4;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    // as many stages in flight as the tokens leave room for
    const cudaError_t e = a.tokens <= fits(4)   ? (nv ? launch_matvec<true, 4>(a, grid, st) : launch_matvec<false, 4>(a, grid, st))
                          : a.tokens <= fits(3) ? (nv ? launch_matvec<true, 3>(a, grid, st) : launch_matvec<false, 3>(a, grid, st))
                                                : (nv ? launch_matvec<true, 2>(a, grid, st) : launch_matvec<false, 2>(a, grid, st));
    return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
