// matvec_tc.cu -- the product of a few bf16 token vectors with a weight matrix held in
// 4 bits, on the block-scaled tensor cores, for K a multiple of 128:
//   y[t, n] = sum_k x[t, k] * s[n, k / G] * c[n, k]
// c E2M1, s UE8M0 with G = 32 (MX) or UE4M3 with G = 16 (NVFP4, one to four tokens);
// bound by the HBM stream of N K (1/2 + 1/G) bytes once nothing is done per weight.
// (Decoding the codes in registers for mma.sync is bound by the integer pipe, at a
// third of that stream.)  So tcgen05.mma.kind::mxf8f6f4 takes the codes as they are, as
// its 128-row E2M1 operand, and everything else is per token or per group.
//
// The tokens are the E4M3 operand, each element as four columns whose scales carry
// the piece's weight: with 2^e the smallest power with max|x| <= 448 * 2^e over the
// element's 32,
//   x 2^-e = p0 + 2^-4 p1 + 2^-22 p2 + 2^-26 p3,
// each piece the rounding of what the ones before it left.  p0 and p1 hold an
// element of at least 2^-6 exactly (four bits each of bf16's eight), p2 and p3 what
// is below E4M3's subnormals: an element is off by at most 2^-36 * 2^e, 2^-43 of the
// largest of its 32.  E4M3 has no infinities: an element that is not finite enters as
// zero and its token's results are computed again by definition.
//
// MX: the weights' scales go to the tensor cores too, and a tile's sums stay in TMEM
// over all of K.  NVFP4: its scales are no power of two, so the weights' scales are
// ones there, each MMA (32 elements) has columns of its own, twice the pieces (the
// halves of the 32 apart, zeros elsewhere), and the draining warps multiply a group's
// sum by its row's scale: with more than four tokens that is more work than decoding.
//
// A block streams tiles of up to 128 rows and a part of K, 256 elements a stage (with
// 128 the loading thread, at 340 cycles a stage, held everything up), to its shared
// memory by TMA (which spreads the 4-bit codes to bytes) with the stage's scales by
// cp.async beside them; blocks of a cluster have the parts of K of the same rows, write
// their fp32 sums to the block that adds a row's (in part order) through distributed
// shared memory, and prepare their part of the tokens once, for all their tiles.  A
// tcgen05 instruction costs its thread about 75 cycles, so two to four threads issue,
// each every second to fourth stage, with sums of its own.  The rows of a tile are as
// few as fill every cluster equally often.
// N = 14336, K = 7168: MX 14.4 us for one token and 20.5 for eight, NVFP4 18.5, 20.4 and
// 25.8 for one, two and four (by mma.sync 27, 30, 32, 33 and 34).  While it streams, one
// MX token's blocks take the HBM's rate; 2.4 us pass before (the tokens) and 2.5 after
// (sums, the cluster).  The operand of eight MX or four NVFP4 tokens leaves room for four
// stages, which are too few to cover a load's latency; NVFP4 is bound by its two issuers,
// 1000 cycles a stage.
#include "moe_common.cuh"
#include "moe_internal.h"

namespace moe {
namespace {

constexpr int kMxBlockK = 128;       // K elements of a block of codes and its scale image
constexpr int kMxStageBlocks = 2;    // blocks of a stage
constexpr int kMxPieces = 4;         // of a token's element: MMA columns
constexpr int kMxTokens = 8;         // of a pass
constexpr int kMxIssuers = 4;        // at most
constexpr int kMxMaxStages = 6;
constexpr int kMxNvTokens = 4;       // of a pass with NVFP4 weights, at most
constexpr int kMxSets = 2;           // NVFP4: issuers, each with four draining warps of its own
constexpr int kMxMaxParts = 8;
constexpr int kMxSmem = 232448;
// warps: 0 loads codes, 1-4 scales (a thread a row), 5-19 prepare the tokens, then
// 5-8 issue and 16-19 (NVFP4: 12-19) drain
constexpr int kMxThreads = 20 * 32;
constexpr int kMxPrepWarp = 5, kMxPrepWarps = 15;
// TMEM columns: two accumulators per issuer, the stages' scale images of both operands
constexpr int kMxAccCols = kMxPieces * kMxTokens;
static_assert(kMxAccCols == 32, "one load of an accumulator");
constexpr int kMxSfaCol = 2 * kMxIssuers * kMxAccCols;
constexpr int kMxSfCols = 4 * kMxStageBlocks;  // of a stage and operand
constexpr int kMxSfbCol = kMxSfaCol + kMxSfCols * kMxMaxStages;
static_assert(kMxSfbCol + kMxSfCols * kMxMaxStages <= 512, "TMEM");
constexpr int kMxMisc = 512;
// TMEM columns with NVFP4: the sums of four MMAs, 16 columns each (eight a token), or of
// two for three and four tokens, two buffers an issuer; scales as above
constexpr int kNvBufCols = 64;
constexpr int kNvSfaCol = 2 * kMxSets * kNvBufCols, kNvSfbCol = kNvSfaCol + 4 * kMxSets;
static_assert(kNvSfbCol + kMxSfCols * kMxMaxStages <= 512, "TMEM");

struct MxArgs {
    const __nv_bfloat16 *x;   // [T, K]
    const uint8_t *w;         // [N, K / 2]
    const uint8_t *sf;        // [N, K / 32] or [N, K / 16]
    __nv_bfloat16 *y;         // [T, N]
    int T, N, K;
    int tokens;               // of a pass (blockIdx.y)
    int cols;                 // of the tokens' operand in shared memory, a multiple of 8
    int rows;                 // of a tile, a multiple of 8
    int parts;                // of K: blocks of a cluster
    int blocks;               // of 128 elements of a part, at most
    int rounds;               // tiles of a cluster, at most
    int stages, issuers;      // the first a multiple of the second: a ring slot is always the same issuer's
};
// The MMA reads 128 rows of a stage, N in steps of 16 of the tokens and 32 rows of a
// scale image, whatever of them is in use: the rest are other bytes of the block's
// memory, in rows and columns that nobody reads.  So a stage holds a tile's rows, a
// block of tokens its columns, and the regions lie in an order in which no such read
// leaves them.
__host__ __device__ inline int mx_stage_bytes(const MxArgs &a) { return kMxStageBlocks * a.rows * 128; }
// scales of a stage: an image a block, or 16 bytes a row
__host__ __device__ constexpr int mx_scale_bytes(bool nv) { return nv ? kTileRows * 16 : kMxStageBlocks * kSfBlockBytes; }
int mx_smem_bytes(bool nv, const MxArgs &a, int stages) {
    const int ring = stages * mx_stage_bytes(a);
    const int rest = a.blocks * a.cols * (128 + 16) + stages * mx_scale_bytes(nv) + (nv ? kSfBlockBytes : 0) +
                     a.rounds * a.tokens * kTileRows * 4 * (nv ? kMxSets : 1) + kMxMisc;
    // the last stage's 128 rows end inside
    return 1024 + ring + (rest > kTileRows * 128 ? rest : kTileRows * 128);
}

__device__ int g_matvec_tc_err[8];  // where a wait that gave up leaves its mark (the outputs become NaN)

__device__ __forceinline__ uint32_t cluster_rank_of() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
// To this block's shared address `at` in block `cta` of the cluster.
__device__ __forceinline__ void cluster_put(uint32_t at, int cta, uint32_t v) {
    uint32_t remote;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(at), "r"(cta));
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(remote), "r"(v) : "memory");
}
// (without an order of this thread's accesses: for the others' having begun alone)
__device__ __forceinline__ void cluster_arrive_relaxed() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ bool mx_warp_wait(uint64_t *bar, uint32_t parity, volatile int *abort, int where) {
    return __all_sync(0xFFFFFFFFu, mbar_wait_cycles(bar, parity, abort, g_matvec_tc_err, where));
}
// Eight bf16; elements that are not finite as zeros.
__device__ __forceinline__ bool finite8(uint4 u, float (&v)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    bool fine = true;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        v[i] = __uint_as_float(i & 1 ? w[i >> 1] & 0xFFFF0000u : w[i >> 1] << 16);
        if (!(fabsf(v[i]) <= 3.4e38f)) {
            v[i] = 0.0f;
            fine = false;
        }
    }
    return fine;
}
// E4M3 codes of v.
__device__ __forceinline__ uint2 piece_of(const float (&v)[8]) {
    uint32_t h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __nv_cvt_float2_to_fp8x2(make_float2(v[2 * i], v[2 * i + 1]), __NV_SATFINITE, __NV_E4M3);
    return make_uint2(h[0] | h[1] << 16, h[2] | h[3] << 16);
}
// What the codes left of v, times `next`.
__device__ __forceinline__ void leave(float (&v)[8], uint2 piece, float next) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t two = (i & 2 ? piece.y : piece.x) >> (16 * (i & 1)) & 0xFFFFu;
        const __half2 h = __half2(__nv_cvt_fp8x2_to_halfraw2(__nv_fp8x2_storage_t(two), __NV_E4M3));
        v[2 * i] = (v[2 * i] - __low2float(h)) * next;
        v[2 * i + 1] = (v[2 * i + 1] - __high2float(h)) * next;
    }
}

// kNvTokens: 0 with MX weights, else up to how many tokens of NVFP4 ones, 2 or 4.
template <int kNvTokens>
__global__ void __launch_bounds__(kMxThreads, 1)
    fp4_matvec_tc_kernel(const __grid_constant__ CUtensorMap tmap_w, const MxArgs args) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *ring = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int kStages = args.stages;
    constexpr bool kNv = kNvTokens > 0;
    constexpr int kUnitMmas = kNvTokens == 4 ? 2 : 4, kMmaCols = kNvBufCols / kUnitMmas;  // of a buffer of sums
    constexpr int kEpiWarp = kNv ? 12 : 16, kSets = kNv ? kMxSets : 1, kTokenCols = kNv ? 2 * kMxPieces : kMxPieces;
    constexpr int kScaleBytes = mx_scale_bytes(kNv), kGroup = kNv ? 16 : 32;
    const int stage_bytes = mx_stage_bytes(args);
    uint8_t *toks = ring + kStages * stage_bytes;                      // [block][column] 128 bytes, swizzled
    uint8_t *sfa = toks + args.blocks * args.cols * 128;               // [stage] images, or rows of 16 bytes
    uint8_t *sfb = sfa + kStages * kScaleBytes;                        // [block][column] 16 bytes, 4 of them scales
    uint8_t *ones = sfb + args.blocks * args.cols * 16;                // NVFP4: an image of ones
    // [part][set][round][token][this block's rows]
    float *sums = reinterpret_cast<float *>(ones + (kNv ? kSfBlockBytes : 0));
    uint64_t *full = reinterpret_cast<uint64_t *>(sums + kSets * args.rounds * args.tokens * kTileRows);
    uint64_t *empty = full + kMxMaxStages;
    uint64_t *tmem_full = empty + kMxMaxStages;   // [2]; NVFP4: [issuer][2]
    uint64_t *tmem_empty = tmem_full + 4;
    uint64_t *mma_done = tmem_empty + 4;          // [issuer]
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(mma_done + kMxIssuers);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_holder + 1);
    uint32_t *bad = tmem_holder + 2;              // tokens with an element that is not finite
    uint32_t *flags = bad + 1;                    // [part] its bad tokens; bit 31: a wait of its gave up
    static_assert((2 * kMxMaxStages + 8 + kMxIssuers) * 8 + (3 + kMxMaxParts) * 4 <= kMxMisc, "barriers and flags");

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int parts = args.parts, part = parts > 1 ? int(cluster_rank_of()) : 0;
    const int all_blocks = args.K / kMxBlockK, all_pairs = (all_blocks + 1) / 2;
    const int pair0 = part * all_pairs / parts, kb0 = pair0 * kMxStageBlocks;
    const int pairs = (part + 1) * all_pairs / parts - pair0;  // stages of a tile
    const int blocks = min(pairs * kMxStageBlocks, all_blocks - kb0);
    const int issuers = args.issuers;
    const int tiles = (args.N + args.rows - 1) / args.rows;
    const int first = int(blockIdx.x) / parts, step = int(gridDim.x) / parts;
    const int own_rows = kTileRows / parts;  // of a tile, added and written by this block
    const int tok0 = int(blockIdx.y) * args.tokens, ntok = min(args.tokens, args.T - tok0);

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&full[s], 1 + 128);  // the codes' copy, the threads that bring scales
            mbar_init(&empty[s], kNv ? 1 + 4 : 1);  // the MMAs, the warps that read scales
        }
        for (int b = 0; b < 4; ++b) {
            mbar_init(&tmem_full[b], kNv ? 1 : issuers);
            mbar_init(&tmem_empty[b], 4);
        }
        for (int i = 0; i < kMxIssuers; ++i) mbar_init(&mma_done[i], 1);
        *abort_flag = 0;
        *bad = 0;
        fence_mbar_init();
        prefetch_tmap(&tmap_w);
    }
    if (warp == kMxPrepWarp) {
        tmem_alloc(tmem_holder, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    cluster_arrive_relaxed();  // waited for before this block's first write to another: they have all begun
    const uint32_t tmem = *tmem_holder;
    pdl_wait();
    if (threadIdx.x == 0) pdl_trigger();

    if (warp == 0) {
        if (lane == 0) {
            // ------------------------------------------------------------ codes
            const uint64_t pol = policy_evict_first();
            int stage = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (int tile = first; ok && tile < tiles; tile += step)
                for (int s = 0; s < pairs; ++s) {
                    ok = mbar_wait_cycles(&empty[stage], phase ^ 1u, abort_flag, g_matvec_tc_err, 71);
                    if (!ok) break;
                    // (a block past K is filled with zeros, and its bytes count)
                    mbar_arrive_expect_tx(&full[stage], uint32_t(kMxStageBlocks * args.rows * 64));
                    tma_load_4d(ring + stage * stage_bytes, &tmap_w, &full[stage], 0, tile * args.rows, 0, kb0 + s * kMxStageBlocks, pol);
                    if (++stage == kStages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
        }
        __syncwarp();
    } else if (warp < kMxPrepWarp) {
        // ---------------------------------------------------------------- scales: thread = row
        // MX: four bytes a block, to row r's place in the image, (r % 32) * 16 + (r / 32) * 4;
        // NVFP4: eight a block, both at once where they are aligned
        const int r = int(threadIdx.x) - 32;
        const int64_t ld = args.K / kGroup;
        const uint32_t dst = smem_u32(sfa) + uint32_t(kNv ? r * 16 : (r & 31) * 16 + (r >> 5) * 4);
        const bool whole = args.K % (kMxStageBlocks * kMxBlockK) == 0;
        int stage = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (int tile = first; ok && tile < tiles; tile += step) {
            const int n = tile * args.rows + r;
            const bool real = r < args.rows && n < args.N;
            const uint8_t *src = args.sf + (real ? n * ld : 0) + kb0 * (kMxBlockK / kGroup);
            for (int s = 0; s < pairs; ++s) {
                ok = mx_warp_wait(&empty[stage], phase ^ 1u, abort_flag, 73);
                if (!ok) break;
                if constexpr (kNv) {
                    const uint32_t to = dst + stage * kScaleBytes;
                    const uint8_t *from = src + s * 16;
                    if (real && whole)
                        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
                    else if (real) {
#pragma unroll
                        for (int b = 0; b < kMxStageBlocks; ++b)
                            if (kMxStageBlocks * s + b < blocks)
                                asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(to + b * 8), "l"(from + b * 8) : "memory");
                    }
                } else {
#pragma unroll
                    for (int b = 0; b < kMxStageBlocks; ++b)
                        if (real && kMxStageBlocks * s + b < blocks)
                            asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(
                                             dst + (stage * kMxStageBlocks + b) * kSfBlockBytes),
                                         "l"(src + (kMxStageBlocks * s + b) * 4)
                                         : "memory");
                }
                asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(&full[stage])) : "memory");
                if (++stage == kStages) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
    } else {
        // ---------------------------------------------------------------- tokens
        // a unit is a stage's 256 elements of a token, eight per lane
        const int w0 = warp - kMxPrepWarp, block = lane >> 4;
        const int s_step = kMxPrepWarps / ntok, t_step = kMxPrepWarps - s_step * ntok;
        struct Unit {
            int s, t;
        };
        auto next = [&](Unit &u) {  // kMxPrepWarps further, stage by stage over the tokens
            u.s += s_step;
            u.t += t_step;
            if (u.t >= ntok) {
                u.t -= ntok;
                ++u.s;
            }
        };
        auto inside = [&](Unit u) { return kMxStageBlocks * u.s + block < blocks; };
        auto fetch = [&](Unit u) {
            const int64_t at = int64_t(tok0 + u.t) * args.K + (kb0 + kMxStageBlocks * u.s) * kMxBlockK + lane * 8;
            return inside(u) ? __ldg(reinterpret_cast<const uint4 *>(args.x + at)) : make_uint4(0, 0, 0, 0);
        };
        auto put = [&](Unit u, uint4 raw) {
            float v[8], amax = 0.0f;
            if (!finite8(raw, v)) atomicOr(bad, 1u << u.t);
#pragma unroll
            for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(v[i]));
            amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
            amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
            // at least -101: the last piece's scale is 2^-127 there, and bf16's smallest
            // subnormal a multiple of its step
            const int e = max(scale_exponent<true>(amax), -101);
            const float m = exp2_neg(e);
            bool low = false;  // an element below 2^-6 may need the last two pieces
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                v[i] *= m;
                low |= v[i] != 0.0f && fabsf(v[i]) < 0.015625f;
            }
            low = __any_sync(0xFFFFFFFFu, low);
            const int kb = kMxStageBlocks * u.s + block, col = kTokenCols * u.t;
            uint8_t *to = toks + (kb * args.cols + col) * 128 + (lane & 1) * 8;
            const int slot = (lane & 15) >> 1;
            uint8_t *image = sfb + (kb * args.cols + col) * 16 + (lane >> 2 & 3);
            uint2 piece[kMxPieces];
            piece[0] = piece_of(v);
            leave(v, piece[0], 16.0f);
            piece[1] = piece_of(v);
            piece[2] = piece[3] = make_uint2(0, 0);
            if (low) {
                leave(v, piece[1], 262144.0f);
                piece[2] = piece_of(v);
                leave(v, piece[2], 16.0f);
                piece[3] = piece_of(v);
            }
            if (inside(u)) {
                const int half = kNv ? lane >> 1 & 1 : 0;  // of a group of 32 the 16 this lane's are in
#pragma unroll
                for (int p = 0; p < kMxPieces; ++p) {
                    auto place = [&](int c) { return reinterpret_cast<uint2 *>(to + c * 128 + ((slot ^ ((col + c) & 7)) << 4)); };
                    *place(half * kMxPieces + p) = piece[p];
                    if (kNv) *place((1 - half) * kMxPieces + p) = make_uint2(0, 0);
                    if ((lane & 3) == 0) {
                        const uint8_t scale = uint8_t(e + 127 - (p == 0 ? 0 : p == 1 ? 4 : p == 2 ? 22 : 26));
                        image[p * 16] = scale;
                        if (kNv) image[(kMxPieces + p) * 16] = scale;
                    }
                }
            }
        };
        // (one copy of the code, which every block fetches anew: units come three ahead)
        Unit u = {w0 / ntok, w0 % ntok}, ahead = u;
        uint4 raw[3];
#pragma unroll
        for (int i = 0; i < 3; ++i, next(ahead)) raw[i] = fetch(ahead);
#pragma unroll 1
        for (; u.s < pairs; next(u), next(ahead)) {
            put(u, raw[0]);
            raw[0] = raw[1];
            raw[1] = raw[2];
            raw[2] = fetch(ahead);
        }
        if (kNv && w0 == 0) reinterpret_cast<uint4 *>(ones)[lane] = make_uint4(0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu);
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        asm volatile("bar.sync 1, %0;" ::"n"(kMxPrepWarps * 32) : "memory");

        if (w0 < issuers) {
            if (lane == 0) {
                // -------------------------------------------------------- MMA issuer
                bool ok = true;
                // NVFP4: a block's MMAs each have columns of their own; the weights' scales are
                // for the draining warps
                const uint32_t unit = tmem + uint32_t(kNvSfaCol + 4 * w0);
                if constexpr (kNv) tc_cp_sf(unit, smem_desc_sf(smem_u32(ones)));
                const uint32_t mma_n = uint32_t((args.cols + 15) / 16 * 16);
                int stage = w0, li = 0, s = w0, used = 0;  // s: this issuer's next stage, counted in the tile
                uint32_t phase = 0;
                for (int tile = first; ok && tile < tiles; tile += step, ++li, s -= pairs) {
                    const int buf = li & 1, s_first = s;
                    if (!kNv && !mbar_wait_cycles(&tmem_empty[buf], (uint32_t(li >> 1) & 1u) ^ 1u, abort_flag, g_matvec_tc_err, 75))
                        break;
                    tc_fence_after();
                    const uint32_t acc = tmem + uint32_t((buf * kMxIssuers + w0) * kMxAccCols);
                    for (; s < pairs; s += issuers) {
                        ok = mbar_wait_cycles(&full[stage], phase, abort_flag, g_matvec_tc_err, 76);
                        if (!ok) break;
                        if constexpr (kNv) {
                            const uint32_t colb = tmem + uint32_t(kNvSfbCol + kMxSfCols * stage);
#pragma unroll
                            for (int m0 = 0; m0 < 4 * kMxStageBlocks; m0 += kUnitMmas) {  // a buffer of the stage's MMAs
                                const int h = m0 / 4, kb = kMxStageBlocks * s + h, b = used & 1;
                                if (kb >= blocks) break;
                                ok = mbar_wait_cycles(&tmem_empty[2 * w0 + b], (uint32_t(used >> 1) & 1u) ^ 1u, abort_flag,
                                                      g_matvec_tc_err, 78);
                                if (!ok) break;
                                tc_fence_after();
                                const uint32_t d = tmem + uint32_t((2 * w0 + b) * kNvBufCols);
                                if (m0 % 4 == 0) tc_cp_sf(colb + 4 * h, smem_desc_sf(smem_u32(sfb + kb * args.cols * 16)));
                                const uint64_t ad = smem_desc_sw128(smem_u32(ring + stage * stage_bytes + h * args.rows * 128));
                                const uint64_t bd = smem_desc_sw128(smem_u32(toks + kb * args.cols * 128));
#pragma unroll
                                for (int m = 0; m < kUnitMmas; ++m) {
                                    const int ks = m0 % 4 + m;
                                    tc_mma_mxf8f6f4(d + uint32_t(m * kMmaCols), ad + uint64_t(2 * ks), bd + uint64_t(2 * ks),
                                                    idesc_mxf8f6f4(uint32_t(kMmaCols), uint32_t(ks)), unit, colb + 4 * h, 0u);
                                }
                                tc_commit(&tmem_full[2 * w0 + b]);
                                ++used;
                            }
                            if (!ok) break;
                            tc_commit(&empty[stage]);
                            stage += issuers;
                            if (stage >= kStages) {
                                stage -= kStages;
                                phase ^= 1u;
                            }
                            continue;
                        }
                        // the scales were written by ordinary accesses of other threads
                        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                        tc_fence_after();
                        const uint32_t col = tmem + uint32_t(kMxSfaCol + kMxSfCols * stage);
                        const uint32_t colb = tmem + uint32_t(kMxSfbCol + kMxSfCols * stage);
#pragma unroll
                        for (int b = 0; b < kMxStageBlocks; ++b) {
                            const int kb = kMxStageBlocks * s + b;
                            if (kb >= blocks) break;
                            tc_cp_sf(col + 4 * b, smem_desc_sf(smem_u32(sfa + (stage * kMxStageBlocks + b) * kSfBlockBytes)));
                            tc_cp_sf(colb + 4 * b, smem_desc_sf(smem_u32(sfb + kb * args.cols * 16)));
                            const uint64_t ad = smem_desc_sw128(smem_u32(ring + stage * stage_bytes + b * args.rows * 128));
                            const uint64_t bd = smem_desc_sw128(smem_u32(toks + kb * args.cols * 128));
#pragma unroll
                            for (int ks = 0; ks < 4; ++ks)
                                tc_mma_mxf8f6f4(acc, ad + uint64_t(2 * ks), bd + uint64_t(2 * ks), idesc_mxf8f6f4(mma_n, uint32_t(ks)),
                                                col + 4 * b, colb + 4 * b, s > s_first || b || ks ? 1u : 0u);
                        }
                        tc_commit(&empty[stage]);
                        stage += issuers;
                        if (stage >= kStages) {
                            stage -= kStages;
                            phase ^= 1u;
                        }
                    }
                    if (!ok) break;
                    if (!kNv) tc_commit(&tmem_full[buf]);
                }
                // all issued MMAs must be finished before TMEM is released
                tc_commit(&mma_done[w0]);
                const long long t0 = clock64();
                while (!mbar_try_wait(&mma_done[w0], 0) && clock64() - t0 < kWaitTimeoutCycles) {
                }
            }
            __syncwarp();
        } else if (warp >= kEpiWarp) {
            // ------------------------------------------------------------ sums: thread = row
            const int q = warp & 3, row = q * 32 + lane, adds = row / own_rows;  // the block that adds this row's
            int li = 0;
            cluster_wait();
            if constexpr (kNv) {
                // every second stage: the sums of its 16 groups of 16 times the row's scales
                const int set = (warp - kEpiWarp) >> 2;
                int s = set, stage = set, used = 0;
                uint32_t phase = 0;
                bool ok = true;
                for (int tile = first; ok && tile < tiles; tile += step, ++li, s -= pairs) {
                    float acc[kNvTokens] = {};
                    bool nan = false;
                    for (; ok && s < pairs; s += kMxSets) {
                        ok = mx_warp_wait(&full[stage], phase, abort_flag, 79);
                        if (!ok) break;
                        const uint4 sc = *reinterpret_cast<const uint4 *>(sfa + stage * kScaleBytes + row * 16);
                        const uint32_t scales[4] = {sc.x, sc.y, sc.z, sc.w};
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&empty[stage]);
                        auto scale = [&](int g) {
                            // 2^-8 times a UE4M3 byte's value: its bits are those of an fp16 number of another bias
                            const uint32_t byte = scales[g >> 2] >> (8 * (g & 3)) & 0x7Fu;
                            nan |= byte == 0x7Fu;
                            __half_raw h;
                            h.x = static_cast<unsigned short>(byte << 7);
                            return __half2float(__half(h));
                        };
                        auto four = [](const uint32_t *r) {
                            return __uint_as_float(r[0]) + (__uint_as_float(r[1]) + (__uint_as_float(r[2]) + __uint_as_float(r[3])));
                        };
#pragma unroll
                        for (int m0 = 0; m0 < 4 * kMxStageBlocks; m0 += kUnitMmas) {
                            const int b = used & 1;
                            if (kMxStageBlocks * s + m0 / 4 >= blocks) break;
                            ok = mx_warp_wait(&tmem_full[2 * set + b], uint32_t(used >> 1) & 1u, abort_flag, 77);
                            if (!ok) break;
                            tc_fence_after();
                            const uint32_t d = tmem + (uint32_t(q * 32) << 16) + uint32_t((2 * set + b) * kNvBufCols);
#pragma unroll
                            for (int c = 0; c < kNvBufCols; c += 32) {
                                uint32_t r[32];
                                tmem_ld_32x32(d + uint32_t(c), r);
                                tmem_ld_wait();
                                // columns of an MMA: a token's first 16 elements' four pieces, its last 16's, the next token's
#pragma unroll
                                for (int m = 0; m < 32 / kMmaCols; ++m)
#pragma unroll
                                    for (int half = 0; half < 2; ++half) {
                                        const float f = scale(2 * (m0 + c / kMmaCols + m) + half);
#pragma unroll
                                        for (int t = 0; t < kNvTokens; ++t)
                                            if (t < ntok) acc[t] = fmaf(four(r + m * kMmaCols + 8 * t + 4 * half), f, acc[t]);
                                    }
                            }
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(&tmem_empty[2 * set + b]);
                            ++used;
                        }
                        stage += kMxSets;
                        if (stage >= kStages) {
                            stage -= kStages;
                            phase ^= 1u;
                        }
                    }
                    const uint32_t to =
                        smem_u32(sums + ((part * kMxSets + set) * args.rounds + li) * args.tokens * own_rows + row % own_rows);
#pragma unroll
                    for (int t = 0; t < kNvTokens; ++t)
                        if (t < ntok)
                            cluster_put(to + uint32_t(t * own_rows * 4), adds, nan ? 0x7FC00000u : __float_as_uint(acc[t] * 256.0f));
                }
            }
            for (int tile = first; !kNv && tile < tiles; tile += step, ++li) {
                const int buf = li & 1;
                if (!mx_warp_wait(&tmem_full[buf], uint32_t(li >> 1) & 1u, abort_flag, 77)) break;
                tc_fence_after();
                // issuer i has stages of this tile if its first one is before the tile's end
                const int lead = li * pairs % issuers;
                auto has = [&](int i) { return i < issuers && (i >= lead ? i - lead : i + issuers - lead) < pairs; };
                const uint32_t to = smem_u32(sums + (part * args.rounds + li) * args.tokens * own_rows + row % own_rows);
                const uint32_t acc = tmem + (uint32_t(q * 32) << 16) + uint32_t(buf * kMxIssuers * kMxAccCols);
                float v[kMxTokens];
#pragma unroll
                for (int t = 0; t < kMxTokens; ++t) v[t] = 0.0f;
                for (int i = 0; i < issuers; ++i) {
                    if (!has(i)) continue;
                    uint32_t r[32];
                    tmem_ld_32x32(acc + uint32_t(i * kMxAccCols), r);
                    tmem_ld_wait();
#pragma unroll
                    for (int t = 0; t < kMxTokens; ++t)
                        v[t] += __uint_as_float(r[4 * t]) +
                                (__uint_as_float(r[4 * t + 1]) + (__uint_as_float(r[4 * t + 2]) + __uint_as_float(r[4 * t + 3])));
                }
#pragma unroll
                for (int t = 0; t < kMxTokens; ++t)
                    if (t < ntok) cluster_put(to + uint32_t(t * own_rows * 4), adds, __float_as_uint(v[t]));
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&tmem_empty[buf]);
            }
        }
    }
    __syncwarp();
    if (warp < kEpiWarp) cluster_wait();
    __syncthreads();
    if (threadIdx.x < parts) cluster_put(smem_u32(flags + part), int(threadIdx.x), *bad | (*abort_flag ? 1u << 31 : 0u));
    __syncwarp();
    tc_fence_before();
    cluster_arrive();
    cluster_wait();
    tc_fence_after();
    if (*abort_flag && threadIdx.x == 0) {
        // a wait gave up (else every copy has been consumed): a quarter of a second, in which copies land
        const long long t0 = clock64();
        while (clock64() - t0 < kWaitTimeoutCycles / 8) {
        }
    }
    if (warp == kMxPrepWarp) tmem_dealloc(tmem, 512);

    // The parts' sums of this block's rows, in part order.
    uint32_t wrong = 0;
    for (int p = 0; p < parts; ++p) wrong |= flags[p];
    const int rounds = first < tiles ? (tiles - first + step - 1) / step : 0;
    const int per_tile = own_rows * ntok;
    for (int i = threadIdx.x; i < rounds * per_tile; i += kMxThreads) {
        const int li = i / per_tile, t = (i - li * per_tile) / own_rows, own = i - li * per_tile - t * own_rows;
        const int r = part * own_rows + own, n = (first + li * step) * args.rows + r;
        if (r >= args.rows || n >= args.N || (wrong >> t & 1u)) continue;
        const float *at = sums + (li * args.tokens + t) * own_rows + own;
        float v = 0.0f;
        for (int p = 0; p < parts * kSets; ++p) v += at[p * args.rounds * args.tokens * own_rows];
        if (wrong >> 31) v = __uint_as_float(0x7FC00000u);
        args.y[int64_t(tok0 + t) * args.N + n] = __float2bfloat16_rn(v);
    }
    if (wrong & 0x7FFFFFFFu) {
        // tokens with infinities or NaN: the sum of these elements' products, a warp per result
        constexpr float kMag[8] = {0.0f, 0.5f, 1.0f, 1.5f, 2.0f, 3.0f, 4.0f, 6.0f};
        for (int i = warp; i < rounds * per_tile; i += kMxThreads / 32) {
            const int li = i / per_tile, t = (i - li * per_tile) / own_rows, own = i - li * per_tile - t * own_rows;
            const int r = part * own_rows + own, n = (first + li * step) * args.rows + r;
            if (r >= args.rows || n >= args.N || !(wrong >> t & 1u)) continue;
            float v = 0.0f;
            for (int k = lane; k < args.K; k += 32) {
                const uint32_t c = args.w[int64_t(n) * (args.K / 2) + k / 2] >> (4 * (k & 1)) & 15u;
                const uint32_t s = args.sf[int64_t(n) * (args.K / kGroup) + k / kGroup];
                float scale = __uint_as_float(s == 255u ? 0x7FC00000u : max(s << 23, 0x00400000u));
                if constexpr (kNv) {
                    __half_raw h;
                    h.x = static_cast<unsigned short>((s & 0x7Fu) << 7);
                    scale = (s & 0x7Fu) == 0x7Fu ? __uint_as_float(0x7FC00000u) : __half2float(__half(h)) * 256.0f;
                }
                // (a finite element changes nothing beside them, but 6 times it may pass fp32's range;
                // its scale may be NaN)
                const float x = __bfloat162float(args.x[int64_t(tok0 + t) * args.K + k]);
                v += (fabsf(x) <= 3.4e38f ? 0.0f : x * (c & 8u ? -kMag[c & 7u] : kMag[c & 7u])) * scale;
            }
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
            if (lane == 0) args.y[int64_t(tok0 + t) * args.N + n] = __float2bfloat16_rn(v);
        }
    }
}

}  // namespace

bool fp4_matvec_tc(bool nv, const void *x, const void *w, const void *sf, void *y, int T, int N, int K, cudaStream_t stream,
                   cudaError_t *status) {
    if (K % kMxBlockK || !aligned(w, 32) || (nv && T > kMxNvTokens)) return false;
    // This kernel or the other, by the two estimates in us.  Of a launch of this one: its
    // start and end, the rows that its blocks stream (in 128 K elements), the tokens that
    // they prepare, and the ends of a block's tiles; as often as its passes fill the device.
    // On 2530 sizes, 1 to 32 tokens, K from 512 to 57344, N from 1 to 65536, the choice took
    // 0.5 % more time than the faster kernel in the mean and 29 % at most.  us, this / the
    // other, MX: one row of K = 4096, T = 1 4.5 / 4.3, of 7168 5.2 / 6.4, T = 8 6.5 / 10.2;
    // 2048 x 2048, T = 1 6.3 / 3.3, T = 8 6.4 / 4.3; 1024 x 7168, T = 1 6.6 / 6.7, T = 8 8.0 /
    // 10.4; 4096 x 4096, T = 1 6.9 / 6.7, T = 8 8.3 / 8.9; 16384 x 512, T = 1 6.4 / 7.8; T = 16:
    // 12288 x 2048 21.4 / 18.0, 4096 x 8192 21.3 / 37.4; NVFP4: 2048 x 4096, T = 2 6.8 / 5.6,
    // 4096 x 7168, T = 2 9.1 / 12.3, T = 4 12.1 / 13.5.
    const double other = fp4_matvec_mma_us(nv, T, N, K), ends = nv ? (T <= 2 ? 4.5 : 5.5) : 5.0;
    if (other <= ends - 0.3) return false;
    const auto run = !nv ? fp4_matvec_tc_kernel<0> : T <= 2 ? fp4_matvec_tc_kernel<2> : fp4_matvec_tc_kernel<4>;
    const void *kernel = reinterpret_cast<const void *>(run);
    *status = set_max_dynamic_smem(kernel, kMxSmem);
    if (*status != cudaSuccess) return true;
    const int all_blocks = K / kMxBlockK;
    MxArgs a{}, best{};
    a.x = static_cast<const __nv_bfloat16 *>(x);
    a.w = static_cast<const uint8_t *>(w);
    a.sf = static_cast<const uint8_t *>(sf);
    a.y = static_cast<__nv_bfloat16 *>(y);
    a.T = T;
    a.N = N;
    a.K = K;
    a.tokens = T < kMxTokens ? T : kMxTokens;
    a.cols = nv ? 2 * kMxPieces * a.tokens : (kMxPieces * a.tokens + 7) / 8 * 8;
    // The parts of K that leave a block the least to stream (the rows of a stage count as
    // 72 at least, what its instructions take, and a block of a token as 14), while its
    // tokens and sums leave room.
    int64_t best_rows = 0, clusters = 0, fit = 0;
    for (a.parts = 1; a.parts <= kMxMaxParts && 2 * a.parts <= all_blocks + 1; a.parts *= 2) {
        const int64_t units = resident_clusters(kernel, a.parts, kMxThreads, kMxSmem);
        a.rounds = int((N + kTileRows * units - 1) / (kTileRows * units));
        a.rows = int((N + a.rounds * units - 1) / (a.rounds * units) + 7) / 8 * 8;
        a.blocks = ((all_blocks + 1) / 2 + a.parts - 1) / a.parts * 2;
        if (a.blocks > 1024 || a.rounds > 1024) continue;
        a.stages = mx_smem_bytes(nv, a, kMxMaxStages) <= kMxSmem ? kMxMaxStages : 4;
        if (mx_smem_bytes(nv, a, a.stages) > kMxSmem) continue;
        a.issuers = nv ? kMxSets : a.stages == 4 ? 4 : 3;
        const int64_t stream_rows = (int64_t(a.rounds) * (a.rows > 72 ? a.rows : 72) + 14 * a.tokens) * a.blocks;
        if (best.parts == 0 || stream_rows < best_rows) {
            best = a;
            best_rows = stream_rows;
            const int64_t tiles = (N + a.rows - 1) / a.rows;
            clusters = tiles < units ? tiles : units;
            fit = units;
        }
    }
    if (best.parts == 0) return false;
    const int64_t passes = (T + best.tokens - 1) / best.tokens, times = (clusters * passes + fit - 1) / fit;
    const double rows = double(best.rounds) * (best.rows > 72 ? best.rows : 72) * best.blocks, prepared = double(best.tokens) * best.blocks;
    const double row_us = !nv ? 0.0012 : T <= 2 ? 0.0021 : 0.0022, token_us = !nv ? 0.018 : T <= 2 ? 0.05 : 0.053;
    const double end_us = !nv ? 0.47 : T <= 2 ? 0.26 : 0.62;
    if (double(times) * (ends + row_us * rows + token_us * prepared + end_us * (best.rounds - 1)) - (nv ? 0.0 : 0.3) >= other)
        return false;
    CUtensorMap tm;
    *status = cudaErrorUnknown;
    if (!encode_weights4(&tm, w, uint64_t(N), uint64_t(K / 2), 1, uint64_t(K / 2), uint64_t(all_blocks), kMxBlockK / 2,
                         best.rows, 1, kMxStageBlocks))
        return true;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(clusters * best.parts), unsigned(passes));
    cfg.blockDim = dim3(kMxThreads);
    // All of an SM's, whatever is used: a block holds all of its TMEM until its cluster has
    // met, so blocks of two clusters on two SMs, each with one waiting for the other's
    // TMEM, would wait for good.
    cfg.dynamicSmemBytes = size_t(kMxSmem);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = unsigned(best.parts);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    *status = cudaLaunchKernelEx(&cfg, run, tm, best);
    return true;
}

}  // namespace moe
