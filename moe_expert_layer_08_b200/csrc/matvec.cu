// matvec.cu -- products of a few bf16 token vectors with a weight matrix held
// in 4 bits with group scales, in the quantisers' own row-major layouts:
//   y[t, n] = sum_k x[t, k] * s[n, k / G] * c[n, k]
// c E2M1, s UE8M0 with G = 32 (MX) or UE4M3 with G = 16 (NVFP4).  Every weight
// byte is used once per 8 tokens, so the floor is the HBM stream of N K (1/2 + 1/G)
// bytes.
//
// A block's 16 warps are two teams, each with a tile of 16 rows at a time and K cut
// into eight slices (a tile costs a team about 100 instructions besides its
// weights: as one team of 16 slices 30.1 us instead of 27.2 at N = 14336, K =
// 7168).  A warp streams its slice of a tile through its
// own ring (TMA boxes of 16 rows x 128 bytes, the scales by cp.async; no waits on
// other warps), and multiplies on the tensor cores: mma.m16n8k16 with the weights
// as the 16-row operand and 8 tokens as the other, so 1 to 8 tokens cost the
// same.  c is exact in fp16.  The tokens are brought to fp16 too, each token
// scaled by a power of two that puts its largest finite magnitude in [2^15, 2^16):
// bf16's 8 bits fit (65280 at most), and an element loses bits only below 2^-32 of
// that largest one (it is then off by half of fp16's smallest step, 2^-25, so by at
// most 2^-40 of that one, less than a rounding of the fp32 sum).  The group scale
// multiplies the fp32 sum of its group.  The slices' sums meet in shared memory and are added in slice order.
// With K a multiple of 128 the block-scaled tensor cores take longer rows and larger
// MX matrices, and NVFP4 ones for up to four tokens, in a kernel without decoding; this
// one takes the rest, and tokens too long for that one's shared memory.
// What keeps it from its floor is the decoding, about 50 instructions per warp and 512
// weights against 11 cycles of an SM's share of HBM, and the chain of decoding, MMA and
// scaling that each group waits for: at N = 14336, K = 7168, eight NVFP4 tokens, 36 us,
// issue 56 %, tensor 7 %, DRAM 17 %.
#include <cuda_fp16.h>

#include "moe_common.cuh"
#include "moe_internal.h"

namespace moe {
namespace {

constexpr int kMvWarps = 16;
constexpr int kMvTeams = 2;
constexpr int kMvSlices = kMvWarps / kMvTeams;     // of K, one per warp of a team
constexpr int kMvRows = 16;                        // rows of a tile (MMA M)
constexpr int kMvTokens = 8;                       // tokens of a pass (MMA N)
constexpr int kMvChunk = 256;                      // K elements of a stage: 128 bytes of codes a row
constexpr int kMvCodeBytes = kMvRows * 128;        // of a stage
constexpr int kMvScaleBytes = kMvRows * 32;        // of a stage: two aligned pieces around a row's scales
constexpr int kMvSumBytes = 2 * kMvWarps * kMvRows * kMvTokens * 4;
constexpr int kMvMaxBytes = kMvTokens * 4 + 96;  // the tokens' largest magnitudes
constexpr int kMvMaxSmem = 232448;
constexpr int kMvMaxK = 57344;
// a stage's scales as fp32, per warp
constexpr int mv_float_bytes(bool nv) { return kMvRows * (nv ? 64 : 32); }
constexpr int mv_fixed_bytes(bool nv, int stages) {
    return 1024 + kMvWarps * (stages * (kMvCodeBytes + kMvScaleBytes + 8) + mv_float_bytes(nv)) + kMvSumBytes + kMvMaxBytes;
}
static_assert(mv_fixed_bytes(true, 2) + (2 * kMvMaxK + 127) / 128 * 128 + 64 <= kMvMaxSmem, "one token of the largest K");

// The E2M1 codes in bits 4j.. and 4j + 16.. of w as fp16 times 2^-14: sign,
// exponent and mantissa bits in place (E2M1's bits are those of an fp16 number
// with another exponent bias, subnormals included).  The shifts are products
// with factors the compiler does not know, which go to the multiply-add pipe:
// the integer pipe runs at half its rate.  (The conversion
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
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%10, %11, %12, %13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
}

// 2^(b - 127) for a UE8M0 byte b (a subnormal for 0, NaN for 255).
__device__ __forceinline__ float ue8m0_value(uint32_t b) {
    return __uint_as_float(b == 255u ? 0x7FC00000u : max(b << 23, 0x00400000u));
}
// 2^-8 times the value of a UE4M3 byte (bit 7 is not read, 0x7F is NaN): its bits
// are those of an fp16 number with an exponent bias of 15 instead of 7.
__device__ __forceinline__ float ue4m3_value_256th(uint32_t b) {
    __half_raw h;
    h.x = static_cast<unsigned short>((b & 0x7Fu) << 7);
    return (b & 0x7Fu) == 0x7Fu ? __uint_as_float(0x7FC00000u) : __half2float(__half(h));
}

// acc += d * scale: rows g (first two sums) and g + 8 (last two).
__device__ __forceinline__ void add_group(float (&acc)[4], const float (&d)[4], float s0, float s1) {
    acc[0] = fmaf(d[0], s0, acc[0]);
    acc[1] = fmaf(d[1], s0, acc[1]);
    acc[2] = fmaf(d[2], s1, acc[2]);
    acc[3] = fmaf(d[3], s1, acc[3]);
}

// Results of an MX matrix by definition, those of a thread (rows row, row + step, ... of a
// token) that are not finite although the token is small: with 2^m the power of two of the
// token's largest element, its sums are kept 2^(1 - m) times as large as its results, and
// pass fp32's range before these do where m < 1.  Only scales of more than 2^110 lead there
// (a slice's groups are at most 224, a group's sum at most 768 times its scale); a result
// stays without one in its row, and with a NaN in the token (halves: the token in fp16,
// read by the lanes of its half of the warp that are here together).
__device__ __noinline__ void mx_again(__nv_bfloat16 *y, const __nv_bfloat16 *x, const uint8_t *halves, const uint8_t *w,
                                      const uint8_t *sf, int row, int step, int N, int K) {
    const uint32_t lane = threadIdx.x & 31, here = __activemask(), half = here & (lane < 16 ? 0xFFFFu : 0xFFFF0000u);
    bool nan = false;
#pragma unroll 4
    for (int k = __popc(half & ((1u << lane) - 1)) * 8; k < K; k += __popc(half) * 8) {
        const uint4 h = *reinterpret_cast<const uint4 *>(halves + k * 2);
        const uint32_t m = __vmaxu2(__vmaxu2(h.x & 0x7FFF7FFFu, h.y & 0x7FFF7FFFu), __vmaxu2(h.z & 0x7FFF7FFFu, h.w & 0x7FFF7FFFu));
        nan |= max(m & 0xFFFFu, m >> 16) > 0x7C00u;
    }
    if (__ballot_sync(here, nan) & half) return;
#pragma unroll 1
    for (; row < N; row += step) {
        if (fabsf(__bfloat162float(y[row])) <= 3.4e38f) continue;
        const uint8_t *codes = w + int64_t(row) * (K / 2), *scales = sf + int64_t(row) * (K / 32);
        bool large = false;
#pragma unroll 16
        for (int i = 0; i < K / 32; ++i) large |= scales[i] > 237 && scales[i] < 255;
        if (!large) continue;
        float v = 0.0f;
#pragma unroll 1
        for (int i = 0; i < K / 32; ++i) {
            float sum = 0.0f;
#pragma unroll 4
            for (int k = 32 * i; k < 32 * i + 32; ++k) {
                const uint32_t c = codes[k / 2] >> (4 * (k & 1)) & 15u, m = c & 7u;
                const float mag = m < 4 ? 0.5f * float(m) : m == 4 ? 2.0f : m == 5 ? 3.0f : m == 6 ? 4.0f : 6.0f;
                sum = fmaf(__bfloat162float(x[k]), c & 8u ? -mag : mag, sum);
            }
            v = fmaf(sum, ue8m0_value(scales[i]), v);
        }
        y[row] = __float2bfloat16_rn(v);
    }
}

// Where a wait that gave up leaves its mark (the outputs become NaN).
__device__ int g_matvec_err[8];

template <bool kNv, int kStages>
__global__ void __launch_bounds__(kMvWarps * 32, 1)
    fp4_matvec_kernel(const __grid_constant__ CUtensorMap tmap_w, const MatvecArgs args) {
    constexpr int kGroup = kNv ? 16 : 32;
    constexpr int kChunkScales = kMvChunk / kGroup;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ volatile int abort_flag;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, t = lane & 3;
    const int tok0 = int(blockIdx.y) * args.tokens;
    const int ntok = min(args.tokens, args.T - tok0);
    const int units = args.K / 32, team = warp / kMvSlices, mine = warp % kMvSlices;
    const int k_lo = mine * units / kMvSlices * 32, k_hi = (mine + 1) * units / kMvSlices * 32;
    const int chunks = (k_hi - k_lo + kMvChunk - 1) / kMvChunk;
    const int tiles = (args.N + kMvRows - 1) / kMvRows;
    const int first = int(blockIdx.x) + team * int(gridDim.x), step = kMvTeams * int(gridDim.x);
    uint8_t *codes = smem + warp * kStages * kMvCodeBytes;
    uint8_t *scales = smem + kMvWarps * kStages * kMvCodeBytes + warp * kStages * kMvScaleBytes;
    uint8_t *floats = smem + kMvWarps * kStages * (kMvCodeBytes + kMvScaleBytes) + warp * mv_float_bytes(kNv);
    uint8_t *after = smem + kMvWarps * (kStages * (kMvCodeBytes + kMvScaleBytes) + mv_float_bytes(kNv));
    float *sums = reinterpret_cast<float *>(after);
    uint64_t *bars = reinterpret_cast<uint64_t *>(after + kMvSumBytes) + warp * kStages;
    uint8_t *xs = after + kMvSumBytes + kMvWarps * kStages * 8 + kMvMaxBytes;
    const int64_t sf_ld = args.K / kGroup, sf_end = args.N * sf_ld;

    uint32_t *tops = reinterpret_cast<uint32_t *>(after + kMvSumBytes + kMvWarps * kStages * 8);  // [token]
    if (threadIdx.x == 0) abort_flag = 0;
    if (threadIdx.x < kMvTokens) tops[threadIdx.x] = 0;
    if (lane == 0) {
        for (int s = 0; s < kStages; ++s) mbar_init(&bars[s], 1);  // this warp's own
        fence_mbar_init();
    }
    __syncthreads();
    pdl_wait();
    pdl_trigger();
    const uint64_t pol = policy_evict_first();
    // The stages of this warp's stream in order: the chunks of its tiles. Lane 0
    // brings the codes; every lane a 16-byte piece of a row's scales (the two
    // aligned pieces around them, cut at the array's end).
    int load_tile = first, load_chunk = 0, load_slot = 0;
    const int piece_row = lane >> 1;
    int64_t at = 0;  // of this lane's row of the tile, the first scale of the chunk
    auto load_next = [&]() {
        if (load_tile < tiles && chunks > 0) {
            const int k0 = k_lo + load_chunk * kMvChunk;
            if (lane == 0) {
                mbar_arrive_expect_tx(&bars[load_slot], kMvCodeBytes);
                tma_load_2d(codes + load_slot * kMvCodeBytes, &tmap_w, &bars[load_slot], k0 / 2, load_tile * kMvRows, pol);
            }
            if (load_chunk == 0) at = min(load_tile * kMvRows + piece_row, args.N - 1) * sf_ld + k_lo / kGroup;
            const int64_t p = (at & ~int64_t(15)) + (lane & 1) * 16;
            if ((lane & 1) == 0 || (int(at) & 15) + kChunkScales > 16) {
                const int64_t left = sf_end - p;
                if (left > 0)
                    cp_async16(smem_u32(scales + load_slot * kMvScaleBytes + lane * 16), args.sf + p, left < 16 ? int(left) : 16);
            }
            at += kChunkScales;
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

    // The tokens in fp16, in the order of the decoded weights: NVFP4 elements 0 and 2, 1
    // and 3, 4 and 6, 5 and 7, MX elements 0 and 4, 1 and 5, 2 and 6, 3 and 7.  First
    // every token's largest finite magnitude, then the values; a warp has every so many
    // 256 elements of one token.  (Little code: a block runs through it once, and
    // fetching eight tokens' copies of it took 0.6 us each.)
    const int x_tok = warp % ntok, x_step = (kMvWarps - x_tok + ntok - 1) / ntok * 256;
    const __nv_bfloat16 *x = args.x + int64_t(tok0 + x_tok) * args.K;
    uint32_t top = 0;
#pragma unroll 4
    for (int k = warp / ntok * 256 + lane * 8; k < args.K; k += x_step) {
        const uint4 raw = __ldg(reinterpret_cast<const uint4 *>(x + k));
        const uint32_t v[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t a = v[i] & 0x7FFFu, b = v[i] >> 16 & 0x7FFFu;
            if (a < 0x7F80u) top = max(top, a);
            if (b < 0x7F80u) top = max(top, b);
        }
    }
    top = __reduce_max_sync(0xFFFFFFFFu, top);
    if (lane == 0) atomicMax(&tops[x_tok], top);
    __syncthreads();
    // 2^shift brings the largest magnitude into [2^15, 2^16); it and 2^-shift are normal numbers
    const auto shift_of = [&](int j) { return min(15 - (int(tops[j] >> 7) - 127), 126); };
    {
        const float mul = tops[x_tok] ? __uint_as_float(uint32_t(127 + shift_of(x_tok)) << 23) : 1.0f;
        uint8_t *to = xs + x_tok * args.x_stride;
#pragma unroll 2
        for (int k = warp / ntok * 256 + lane * 8; k < args.K; k += x_step) {
            const uint4 raw = __ldg(reinterpret_cast<const uint4 *>(x + k));
            const uint32_t v[4] = {raw.x, raw.y, raw.z, raw.w};
            uint32_t h[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int lo = kNv ? (i & 1) + 4 * (i >> 1) : i, hi = lo + (kNv ? 2 : 4);
                const auto value = [&](int e) { return __uint_as_float(e & 1 ? v[e >> 1] & 0xFFFF0000u : v[e >> 1] << 16); };
                const __half2 p = __floats2half2_rn(value(lo) * mul, value(hi) * mul);
                h[i] = *reinterpret_cast<const uint32_t *>(&p);
            }
            *reinterpret_cast<uint4 *>(to + k * 2) = make_uint4(h[0], h[1], h[2], h[3]);
        }
    }
    __syncthreads();
    // What brings the sums of tokens 2t and 2t + 1, this lane's columns, back.  MX: with the
    // 2^14 of the codes, 2^-112 to 2^126, in one factor (2^14 first would take results of 2^114
    // out of fp32's range).  NVFP4: 2^22 for codes and scales comes first, for sums that are
    // below 2^21 whatever the token.
    float unscale[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int j = 2 * t + i;
        unscale[i] = __uint_as_float(uint32_t(127 + (kNv ? 0 : 14) - (j < ntok && tops[j] ? shift_of(j) : 0)) << 23);
    }

    const uint8_t *xrow = xs + min(g, ntok - 1) * args.x_stride + (kNv ? t * 8 : t * 16);  // token g
    int slot = 0, buf = 0;
    uint32_t phase = 0;
    bool ok = true, again = false;  // again: a result of this thread's is not finite
    const int swz = g * 16;  // 16-byte pieces of a row of codes: piece ^ row % 8
    for (int tile = first; tile < tiles; tile += step, buf ^= 1) {
        float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        // where this lane's row of the tile (two lanes a row) has its first scale
        int64_t first_scale = min(tile * kMvRows + piece_row, args.N - 1) * sf_ld + k_lo / kGroup;
        for (int c = 0; c < chunks; ++c) {
            cp_async_wait<kStages - 2>();
            ok = mbar_wait_cycles(&bars[slot], phase, &abort_flag, g_matvec_err, 61) && ok;
            __syncwarp();  // this stage has landed for every lane, and the one before it is read
            load_next();
            // the stage's scales as fp32: half a row per lane
            {
                const uint8_t *sc = scales + slot * kMvScaleBytes + piece_row * 32 + (int(first_scale) & 15) +
                                    (lane & 1) * (kChunkScales / 2);
                const int r = piece_row;
                float f[kChunkScales / 2];
#pragma unroll
                for (int i = 0; i < kChunkScales / 2; ++i) f[i] = kNv ? ue4m3_value_256th(sc[i]) : ue8m0_value(sc[i]);
#pragma unroll
                for (int i = 0; i < kChunkScales / 8; ++i) {
                    const int piece = (lane & 1) * (kChunkScales / 8) + i;
                    uint8_t *to = floats + (kNv ? r * 64 + ((piece ^ (r >> 1 & 3)) << 4) : r * 32 + ((piece ^ (r >> 2 & 1)) << 4));
                    *reinterpret_cast<float4 *>(to) = make_float4(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]);
                }
                first_scale += kChunkScales;
            }
            __syncwarp();
            const uint8_t *st = codes + slot * kMvCodeBytes + g * 128;
            const uint8_t *xk = xrow + (k_lo + c * kMvChunk) * 2;
            const float zero[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            // four scales of rows g and g + 8 (the swizzle is the same for both)
            auto four = [&](int row, int piece) {
                return *reinterpret_cast<const float4 *>(
                    floats + (kNv ? row * 64 + ((piece ^ (g >> 1 & 3)) << 4) : row * 32 + ((piece ^ (g >> 2 & 1)) << 4)));
            };
            // 32 elements: two groups of 16 or one of 32
            auto block = [&](int i, float s0, float s1, float s2, float s3) {
                float d[4];
                uint32_t a[4];
                const uint8_t *row = st + ((i << 4) ^ swz);
                if constexpr (kNv) {
                    // a group of 16 is one step: lane t holds its elements 4t .. 4t + 3
#pragma unroll
                    for (int s = 0; s < 2; ++s) {
                        const uint32_t wa = *reinterpret_cast<const uint16_t *>(row + s * 8 + t * 2);
                        const uint32_t wb = *reinterpret_cast<const uint16_t *>(row + s * 8 + t * 2 + 8 * 128);
                        const uint2 xv = *reinterpret_cast<const uint2 *>(xk + (i * 32 + s * 16) * 2);
                        const uint32_t pa = __byte_perm(wa, 0u, 0x4140u), pb = __byte_perm(wb, 0u, 0x4140u);
                        a[0] = e2m1_pair<0>(pa, args.factors);
                        a[1] = e2m1_pair<0>(pb, args.factors);
                        a[2] = e2m1_pair<1>(pa, args.factors);
                        a[3] = e2m1_pair<1>(pb, args.factors);
                        mma_16x8x16(d, a[0], a[1], a[2], a[3], xv.x, xv.y, zero);
                        add_group(acc, d, s ? s2 : s0, s ? s3 : s1);
                    }
                } else {
                    // a group of 32 is two steps: lane t holds its elements 8t .. 8t + 7
                    const uint32_t wa = *reinterpret_cast<const uint32_t *>(row + t * 4);
                    const uint32_t wb = *reinterpret_cast<const uint32_t *>(row + t * 4 + 8 * 128);
                    const uint4 xv = *reinterpret_cast<const uint4 *>(xk + i * 32 * 2);
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
                    add_group(acc, d, s0, s1);
                }
            };
            const int blocks = min(kMvChunk, k_hi - k_lo - c * kMvChunk) / 32;
            constexpr int kPer = kNv ? 2 : 4;  // blocks of four scales a row
            auto quad = [&](int i0) {          // four blocks
#pragma unroll
                for (int i = i0; i < i0 + 4; i += kPer) {
                    const float4 u = four(g, i / kPer), v = four(g + 8, i / kPer);
                    if constexpr (kNv) {
                        block(i, u.x, v.x, u.y, v.y);
                        block(i + 1, u.z, v.z, u.w, v.w);
                    } else {
                        block(i, u.x, v.x, 0.0f, 0.0f);
                        block(i + 1, u.y, v.y, 0.0f, 0.0f);
                        block(i + 2, u.z, v.z, 0.0f, 0.0f);
                        block(i + 3, u.w, v.w, 0.0f, 0.0f);
                    }
                }
            };
            if (blocks == kMvChunk / 32) {
                quad(0);
                quad(4);
            } else {
                if (blocks >= 4) quad(0);
#pragma unroll 1
                for (int i = blocks & 4; i < blocks; ++i) {
                    const float4 u = four(g, i / kPer), v = four(g + 8, i / kPer);
                    if constexpr (kNv) {
                        const bool odd = i & 1;
                        block(i, odd ? u.z : u.x, odd ? v.z : v.x, odd ? u.w : u.y, odd ? v.w : v.y);
                    } else {
                        const int k = i & 3;
                        block(i, k == 0 ? u.x : k == 1 ? u.y : k == 2 ? u.z : u.w,
                              k == 0 ? v.x : k == 1 ? v.y : k == 2 ? v.z : v.w, 0.0f, 0.0f);
                    }
                }
            }
            if (++slot == kStages) {
                slot = 0;
                phase ^= 1u;
            }
        }
        const float back = !ok ? __uint_as_float(0x7FC00000u) : kNv ? 0x1p22f : 1.0f;
        // rows g and g + 8, tokens 2t and 2t + 1 of this slice
        float *part = sums + (buf * kMvWarps + warp) * kMvRows * kMvTokens;
        part[g * kMvTokens + 2 * t] = acc[0] * back * unscale[0];
        part[g * kMvTokens + 2 * t + 1] = acc[1] * back * unscale[1];
        part[(g + 8) * kMvTokens + 2 * t] = acc[2] * back * unscale[0];
        part[(g + 8) * kMvTokens + 2 * t + 1] = acc[3] * back * unscale[1];
        asm volatile("bar.sync %0, %1;" ::"r"(1 + team), "n"(kMvSlices * 32) : "memory");
        const int id = mine * 32 + lane;
        if (id < kMvRows * ntok) {
            const int j = id >> 4, r = id & 15;
            const int n = tile * kMvRows + r;
            if (n < args.N) {
                float v = 0.0f;
#pragma unroll
                for (int i = 0; i < kMvSlices; ++i)
                    v += sums[(buf * kMvWarps + team * kMvSlices + i) * kMvRows * kMvTokens + r * kMvTokens + j];
                again |= !(fabsf(v) <= 3.4028235e38f);
                args.y[int64_t(tok0 + j) * args.N + n] = __float2bfloat16_rn(v);
            }
        }
    }
    if (!kNv && again) {
        // (its own stores, which a thread sees; inside the loop the call cost launches of 3 us
        // 0.1 us each)
        const int id = mine * 32 + lane, j = id >> 4;
        if (tops[j] < 128u << 7)  // the token is below two
            mx_again(args.y + int64_t(tok0 + j) * args.N, args.x + int64_t(tok0 + j) * args.K, xs + j * args.x_stride, args.w,
                     args.sf, first * kMvRows + (id & 15), step * kMvRows, args.N, args.K);
    }
    if (abort_flag) {
        // a wait gave up: a quarter of a second, in which the copies under way land
        const long long t0 = clock64();
        while (clock64() - t0 < kWaitTimeoutCycles / 8) {
        }
    }
}

// Bytes of a token in shared memory: those of a quarter-warp's 16-byte reads are 64 bytes
// apart modulo 128.
int mv_token_bytes(int K) { return (2 * K + 127) / 128 * 128 + 64; }
// Tokens that fit beside a number of stages.
int mv_tokens_beside(bool nv, int K, int stages) { return (kMvMaxSmem - 16 - mv_fixed_bytes(nv, stages)) / mv_token_bytes(K); }
// Tokens of a pass over the weights.
int mv_pass_tokens(bool nv, int T, int K) {
    const int most = mv_tokens_beside(nv, K, 2), tokens = T < kMvTokens ? T : kMvTokens;
    return tokens < most ? tokens : most;
}

template <bool kNv, int kStages>
cudaError_t launch_matvec(const CUtensorMap &tmap_w, const MatvecArgs &a, dim3 grid, cudaStream_t stream) {
    const cudaError_t e =
        set_max_dynamic_smem(reinterpret_cast<const void *>(fp4_matvec_kernel<kNv, kStages>), kMvMaxSmem - 16);
    if (e != cudaSuccess) return e;
    return launch_pdl(fp4_matvec_kernel<kNv, kStages>, grid, dim3(kMvWarps * 32),
                      size_t(mv_fixed_bytes(kNv, kStages) + a.tokens * a.x_stride), stream, tmap_w, a);
}

}  // namespace

// Fitted to the measurements at the choice between the kernels (off by 9 % in the root mean
// square): the tokens' preparation and a block's tiles of 16 rows, by their elements and by
// the stages of a slice (a last one that is no half or whole costs more), as often as the
// passes fill the device.
double fp4_matvec_mma_us(bool nv, int T, int N, int K) {
    const int tokens = mv_pass_tokens(nv, T, K), passes = (T + tokens - 1) / tokens, sms = num_sms();
    const int64_t row_tiles = (int64_t(N) + kMvRows - 1) / kMvRows, blocks = row_tiles < sms ? row_tiles : sms;
    const int slice = (K / 32 + kMvSlices - 1) / kMvSlices * 32, chunks = (slice + kMvChunk - 1) / kMvChunk;
    const double times = double((blocks * passes + sms - 1) / sms), tiles = double((row_tiles + blocks - 1) / blocks);
    const double k = K / 1000.0, prepare = (nv ? 0.11 : 0.08) * k * T / passes;
    const double tile = nv ? 0.4 + 0.37 * k + 0.22 * chunks + (slice % 128 ? 0.1 : 0.0)
                           : 0.28 + 0.21 * k + 0.17 * chunks + (slice % 128 ? 0.18 : 0.0);
    return 0.5 + times * (0.8 + prepare + tiles * tile + (nv ? 0.12 : 0.24) * k);
}
}  // namespace moe

using namespace moe;

extern "C" moe_status_t moe_fp4_matvec(const void *x_bf16, const void *w_fp4, const void *w_sf, void *y_bf16, int T,
                                       int N, int K, int format, moe_stream_t stream) {
    if (T < 0 || N <= 0 || K <= 0 || (format != MOE_FP4_MX && format != MOE_FP4_NVFP4)) return MOE_ERR_INVALID_ARG;
    if (K % 32 || K > kMvMaxK || T > 65535 || N > kMaxRows) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (T == 0) return MOE_OK;
    if (!x_bf16 || !w_fp4 || !w_sf || !y_bf16 || !aligned(x_bf16, 16) || !aligned(w_fp4, 16) ||
        !aligned(w_sf, 16) || !aligned(y_bf16, 2))
        return MOE_ERR_INVALID_ARG;
    DeviceScope dev(y_bf16);
    if (dev.status != MOE_OK) return dev.status;
    cudaError_t e = cudaSuccess;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (fp4_matvec_tc(format == MOE_FP4_NVFP4, x_bf16, w_fp4, w_sf, y_bf16, T, N, K, st, &e))
        return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
    MatvecArgs a{};
    a.x = static_cast<const __nv_bfloat16 *>(x_bf16);
    a.w = static_cast<const uint8_t *>(w_fp4);
    a.sf = static_cast<const uint8_t *>(w_sf);
    a.y = static_cast<__nv_bfloat16 *>(y_bf16);
    a.T = T;
    a.N = N;
    a.K = K;
    a.factors = {{512, 32, 2}, {4096, 256, 16}};
    a.x_stride = mv_token_bytes(K);
    const bool nv = format == MOE_FP4_NVFP4;
    const auto fits = [&](int stages) { return mv_tokens_beside(nv, K, stages); };
    a.tokens = mv_pass_tokens(nv, T, K);
    const int tiles = (N + kMvRows - 1) / kMvRows, sms = num_sms();
    const dim3 grid(unsigned(tiles < sms ? tiles : sms), unsigned((T + a.tokens - 1) / a.tokens));
    CUtensorMap tm;
    if (!encode_bytes_rows(&tm, w_fp4, uint64_t(K / 2), uint64_t(N), kMvRows)) return MOE_ERR_CUDA;
    // as many stages in flight as the tokens leave room for
    e = a.tokens <= fits(4)   ? (nv ? launch_matvec<true, 4>(tm, a, grid, st) : launch_matvec<false, 4>(tm, a, grid, st))
        : a.tokens <= fits(3) ? (nv ? launch_matvec<true, 3>(tm, a, grid, st) : launch_matvec<false, 3>(tm, a, grid, st))
                              : (nv ? launch_matvec<true, 2>(tm, a, grid, st) : launch_matvec<false, 2>(tm, a, grid, st));
    return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
