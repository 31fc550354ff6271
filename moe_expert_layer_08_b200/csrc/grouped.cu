// grouped.cu -- products of the experts' bf16 weights with ragged groups of
// rows, and their two gradients.  Rows offsets[e] .. offsets[e+1]-1 of the row
// operands belong to expert e:
//   product          y[r, n]     = sum_k x[r, k] W[e, n, k]
//   input gradient   dx[r, k]    = sum_n dy[r, n] W[e, n, k]
//   weight gradient  dW[e, n, k] = sum_{r of e} dy[r, n] x[r, k]
// bf16 operands, fp32 sums in TMEM (tcgen05.mma.kind::f16), one rounding to
// bf16 at the end.  In all three a work item is a strip of the output features
// (one or two MMA tiles, the M side) times up to kN columns of the N side: rows of one
// expert (product, input gradient; N is the row count rounded up to 16, so a
// ragged group costs what it has and not a full tile) or 256 columns of k
// (weight gradient).  Large loads run on pairs of CTAs (tcgen05 cta_group::2):
// a strip of 512 features, each CTA with 256 of them and half of the N side in
// its shared memory, 48 KB from L2 per 1024 MMA cycles and SM instead of 64.  Few
// items of a long contraction are shared by clusters instead: a block has a part of
// it, and some columns of the parts' fp32 sums to add, in part order.  Operands come by TMA
// straight from the caller's row-major tensors in whichever major order the
// contraction finds them:
//                    M side                     N side
//   product          W rows n, K-major          x rows, K-major
//   input gradient   W columns k, MN-major      dy rows, K-major
//   weight gradient  dy columns n, MN-major     x columns k, MN-major
// Columns past a feature width and rows of W past its expert read as zeros
// through the tensor maps.  The weight gradient's contraction runs over rows,
// so the rows of the next group inside its last 16-row step are zeroed in
// shared memory on both sides (a product with zero alone would let a NaN of
// the neighbour through).
#include "moe_common.cuh"
#include "moe_internal.h"
#include "row_chunks.h"

namespace moe {
namespace {

// The workspace of calls whose status nobody reads, on every stream and in every graph
// of a device: memory of the library's own, since an allocator's block may have an
// earlier owner whose work on one stream is still to come.
__device__ __align__(256) uint8_t g_grouped_unread[kHdrBytes];

enum GroupedMode { kProduct = 0, kGradInput = 1, kGradWeight = 2 };

constexpr int kBlockK = 64;    // contraction elements of a pipeline stage (one 128-byte swizzled row)
constexpr int kRowBox = 32;    // rows of one TMA box of a K-major N side
constexpr int kChunkBlock = 16;  // row chunks that share a strip's weights before the next strip
constexpr int kMaxSmem = 232448;
// warps: 0 loads, 1 and 2 issue, 3 zeroes the weight gradient's tails; 4-19
// drain the tiles in turn, four warps a block of 32 columns
constexpr int kEpiWarps = 16;
constexpr int kThreads = 32 * (4 + kEpiWarps);

// kN: columns of the N side an item may have.  Fewer columns leave room for more
// stages of weights in flight; more columns cost fewer operand bytes per MMA.
// kTiles: 128-row MMA tiles of a CTA's strip.  With one there is TMEM for two
// accumulators, so that the next item's MMAs run while the last one's are
// drained, at 64 operand bytes per MMA cycle and SM instead of 48.
template <int kMode, int kN, int kTiles>
struct GroupedCfg {
    // per epilogue warp, results on their way out: 16 rows x 32 features, or of the
    // weight gradient 32 rows x 32 columns
    static constexpr int kStageOutBytes = kEpiWarps * (kMode == kGradWeight ? 32 : 16) * 64;
    static constexpr int kStrip = kTiles * kTileRows;     // output features of an item per CTA
    static constexpr bool kPair = kN >= 160;
    static constexpr int kCtas = kPair ? 2 : 1;
    static constexpr int kABytes = kStrip * kBlockK * 2;  // 16 KB a tile
    static constexpr int kBRows = (kN / kCtas + kRowBox - 1) / kRowBox * kRowBox;
    static constexpr int kBBytes = kBRows * kBlockK * 2;
    static constexpr int kStageBytes = kABytes + kBBytes;
    static constexpr int kBufs = kTiles * kN <= 256 ? 2 : 1;        // accumulator buffers of a tile
    static constexpr int kTmemCols = kN == 64 ? 128 * kTiles : 512;
    static constexpr bool kSplits = kN == 64 && kTiles == 1;        // may share an item's contraction among a cluster
    static constexpr int kMisc = 512;
    static constexpr int kMaxStages = 10;
    // barriers, the results' way out and the group table beside the stages
    static constexpr int fixed_bytes(int E) { return 1024 + kStageOutBytes + kMisc + 8 * (E + 1); }
    static constexpr int stages(int E) {
        return (kMaxSmem - fixed_bytes(E)) / kStageBytes < kMaxStages ? (kMaxSmem - fixed_bytes(E)) / kStageBytes : kMaxStages;
    }
    static_assert(stages(kMaxExperts) >= 3, "shared memory budget");
    static_assert(!kSplits || kN * kTileRows * 4 <= 3 * kStageBytes, "a part's sums fit the ring");
    static_assert(kTiles * kBufs * kN <= kTmemCols, "TMEM allocation");
};

struct GroupedArgs {
    const int *offsets;   // [E + 1]
    __nv_bfloat16 *out;
    int *hdr;             // workspace header (error word)
    int R, E;
    int D;                // output features: N (product, weight gradient's rows) or K (input gradient)
    int C;                // contraction length of the product and input gradient
    int K;                // weight gradient: columns of dW
    int chunks_m, chunks_n;  // MN-major operands: their maps have 64-column chunks as a dimension, two of them a box
    int zero_unused;      // product, input gradient: write zeros to the rows of no expert
    int stages;           // of the operand ring
    int split;            // parts of the contraction, the CTAs of a cluster (then one item per cluster)
};

// Shared-memory matrix descriptor, MN-major, 128-byte swizzle: boxes of 64 MN
// x 64 contraction elements (a contraction row is 128 bytes), 8-row groups
// 1024 B apart (SBO), the next 64 MN elements one box further (LBO).
__device__ __forceinline__ uint64_t smem_desc_mn_sw128(uint32_t saddr) {
    uint64_t d = 0;
    d |= uint64_t((saddr >> 4) & 0x3FFFu);
    d |= uint64_t((64 * 128) >> 4) << 16;   // LBO
    d |= uint64_t(1024 >> 4) << 32;         // SBO
    d |= uint64_t(1) << 46;                 // descriptor version (sm_100)
    d |= uint64_t(2) << 61;                 // SWIZZLE_128B
    return d;
}

// TMA store of a box from shared memory (this thread's own bulk group).
__device__ __forceinline__ void tma_store_3d(const CUtensorMap *map, const void *src, int c0, int c1, int c2) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(smem_u32(src)), "r"(c0), "r"(c1), "r"(c2)
                 : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
// This thread's stores have read their shared memory / are complete.
__device__ __forceinline__ void tma_store_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void tma_store_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// 32 lanes x 16 columns of 32-bit words.
__device__ __forceinline__ void tmem_ld_32x16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}

// One step of a warp's inclusive maximum / sum scans.
__device__ __forceinline__ int warp_scan_max(int v, int lane) {
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xFFFFFFFFu, v, d);
        if (lane >= d) v = max(v, o);
    }
    return v;
}
__device__ __forceinline__ int warp_scan_sum(int v, int lane) {
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xFFFFFFFFu, v, d);
        if (lane >= d) v += o;
    }
    return v;
}

// Work item u: expert, first output feature of its strip, and the N side: rows
// [row0, row0 + cols) or columns [col0, col0 + cols) of dW.
struct Item {
    int e, d0, n0, cols;
    int kblocks;   // stages
    int tail;      // weight gradient: rows of the last stage (1 .. 64)
};

// Walks the items of one CTA in ascending order; every role keeps its own.
template <int kMode, int kN, int kTiles>
struct Walker {
    static constexpr int kItemStrip = GroupedCfg<kMode, kN, kTiles>::kStrip * GroupedCfg<kMode, kN, kTiles>::kCtas;
    const int *row_of;   // [E + 1] group starts, ascending
    const int *item_of;  // [E + 1] first item of each expert
    int E, strips, kb_const, K, D;
    int e = 0;

    __device__ __forceinline__ Item at(int u) {
        Item it;
        if constexpr (kMode == kGradWeight) {
            const int kt = (K + kN - 1) / kN;
            const int per = strips * kt;
            it.e = u / per;
            const int l = u - it.e * per;
            it.d0 = (l / kt) * kItemStrip;
            it.n0 = (l % kt) * kN;
            it.cols = min(kN, K - it.n0);
            const int rows = row_of[it.e + 1] - row_of[it.e];
            it.kblocks = (rows + kBlockK - 1) / kBlockK;
            it.tail = rows - (it.kblocks - 1) * kBlockK;
        } else {
            while (item_of[e + 1] <= u) ++e;
            it.e = e;
            const int l = u - item_of[e];
            const int r0 = row_of[e], rows = row_of[e + 1] - r0;
            const RowChunks chunks = row_chunks(rows, kN);
            const int nch = chunks.count, size = chunks.size;
            // blocks of kChunkBlock row chunks; inside one, strip by strip over its chunks
            const int b = l / (kChunkBlock * strips);
            const int rem = l - b * kChunkBlock * strips;
            const int width = min(kChunkBlock, nch - b * kChunkBlock);
            const int c = b * kChunkBlock + rem % width;
            it.d0 = (rem / width) * kItemStrip;
            it.n0 = r0 + c * size;
            it.cols = min(size, rows - c * size);
            it.kblocks = kb_const;
            it.tail = kBlockK;
        }
        return it;
    }
};

// ---- CTA pairs
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
// Every thread of both CTAs.
__device__ __forceinline__ void cluster_barrier() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Two floats at this CTA's shared address `at`, of CTA `cta` of the cluster.
__device__ __forceinline__ float2 cluster_load(uint32_t at, int cta) {
    uint32_t remote;
    float2 v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(at), "r"(cta));
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(remote) : "memory");
    return v;
}
// The first CTA's barrier at this CTA's address `bar`.
__device__ __forceinline__ uint32_t leader_bar(uint64_t *bar) {
    uint32_t remote;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(remote) : "r"(smem_u32(bar)));
    return remote;
}
// TMA loads (no multicast) into this CTA that complete on a barrier of the pair.
__device__ __forceinline__ void tma_load_2d_pair(void *dst, const CUtensorMap *map, uint32_t bar, int c0, int c1,
                                                 uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%3, %4}], [%2], %5;" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "l"(policy)
        : "memory");
}
__device__ __forceinline__ void tma_load_3d_pair(void *dst, const CUtensorMap *map, uint32_t bar, int c0, int c1, int c2,
                                                 uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%3, %4, %5}], [%2], %6;" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "l"(policy)
        : "memory");
}
__device__ __forceinline__ void tma_load_4d_pair(void *dst, const CUtensorMap *map, uint32_t bar, int c0, int c1, int c2,
                                                 int c3, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%3, %4, %5, %6}], [%2], %7;" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "l"(policy)
        : "memory");
}
// Arrive on the first CTA's barrier at this CTA's address `bar`.
__device__ __forceinline__ void mbar_arrive_leader(uint64_t *bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(leader_bar(bar)) : "memory");
}
// mbar_wait_cycles with the acquire of what the other CTA did before it arrived.
__device__ __forceinline__ bool mbar_try_wait_cluster(uint64_t *bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}\n"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0u;
}
__device__ __forceinline__ bool mbar_wait_cluster(uint64_t *bar, uint32_t parity, volatile int *abort, int *err, int where) {
    return mbar_try_wait_cluster(bar, parity) ||
           (mbar_wait_cycles_slow(bar, parity, abort, err, where) && mbar_try_wait_cluster(bar, parity));
}
// The pair's D[M = 256, N] (+)= A . B^T: rows 0-127 of A and D are the first
// CTA's, and so is the first half of B's N; descriptors hold for both CTAs.
__device__ __forceinline__ void tc_mma_bf16_pair(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                                 uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// Arrive on the barrier at `bar` in both CTAs when this thread's MMAs complete.
__device__ __forceinline__ void tc_commit_pair(uint64_t *bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_u32(bar)),
        "h"(static_cast<uint16_t>(3))
        : "memory");
}
// Arrive on this CTA's barrier alone.
template <bool kPair>
__device__ __forceinline__ void tc_commit_own(uint64_t *bar) {
    if constexpr (kPair)
        asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
                     : "memory");
    else
        tc_commit(bar);
}
template <bool kPair>
__device__ __forceinline__ void tmem_alloc_for(uint32_t *dst_smem, uint32_t ncols) {
    if constexpr (kPair) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst_smem)), "r"(ncols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    } else {
        tmem_alloc(dst_smem, ncols);
        tmem_relinquish();
    }
}
template <bool kPair>
__device__ __forceinline__ void tmem_dealloc_for(uint32_t taddr, uint32_t ncols) {
    if constexpr (kPair)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
    else
        tmem_dealloc(taddr, ncols);
}

// A bounded wait of a whole warp: true for all of its lanes or for none.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, volatile int *abort, int *err, int where) {
    return __all_sync(0xFFFFFFFFu, mbar_wait_cycles(bar, parity, abort, err, where));
}

template <int kMode, int kN, int kTiles>
__global__ void __launch_bounds__(kThreads, 1)
    grouped_kernel(const __grid_constant__ CUtensorMap tmap_m, const __grid_constant__ CUtensorMap tmap_n,
                   const __grid_constant__ CUtensorMap tmap_out, const GroupedArgs args) {
    using C = GroupedCfg<kMode, kN, kTiles>;
    const int kStages = args.stages;
    constexpr bool kPair = C::kPair;
    constexpr int kCtas = C::kCtas;
    static_assert(kPair || kMode != kGradWeight, "the weight gradient runs on pairs");
    constexpr bool kMMn = kMode != kProduct;         // M side MN-major
    constexpr bool kNMn = kMode == kGradWeight;      // N side MN-major
    extern __shared__ uint8_t smem_raw[];
    uint8_t *tiles = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *stage_out = tiles + kStages * C::kStageBytes;
    uint64_t *full = reinterpret_cast<uint64_t *>(stage_out + C::kStageOutBytes);
    uint64_t *empty = full + kStages;
    // weight gradient, a stage whose tail rows are to be zeroed: landed in this CTA;
    // zeroed in both (the first CTA's). Every other stage completes on `full` (a
    // pair's on the first CTA's).
    uint64_t *landed = empty + kStages;
    uint64_t *zeroed = landed + kStages;
    uint64_t *tmem_full = zeroed + kStages;       // [tile][buf]
    uint64_t *tmem_empty = tmem_full + 4;        // [tile][buf]
    uint64_t *mma_done = tmem_empty + 4;         // [tile]
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(mma_done + 2);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_holder + 1);
    int *row_of = reinterpret_cast<int *>(reinterpret_cast<uint8_t *>(full) + C::kMisc);
    int *item_of = row_of + args.E + 1;
    static_assert((4 * C::kMaxStages + 10) * 8 + 8 <= C::kMisc, "barriers and flags");

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], kTiles);  // the issuers
            mbar_init(&landed[s], 1);
            mbar_init(&zeroed[s], 2);
        }
        for (int b = 0; b < 4; ++b) {
            mbar_init(&tmem_full[b], 1);
            mbar_init(&tmem_empty[b], kCtas * kEpiWarps / kTiles);
        }
        mbar_init(&mma_done[0], 1);
        mbar_init(&mma_done[1], 1);
        *abort_flag = 0;
        fence_mbar_init();
        prefetch_tmap(&tmap_m);
        prefetch_tmap(&tmap_n);
    }
    if (warp == 1) tmem_alloc_for<kPair>(tmem_holder, C::kTmemCols);
    const int rank = kPair ? int(cluster_rank()) : 0;  // blocks 2i and 2i + 1 are a pair
    const int split = C::kSplits ? args.split : 1, cut = split > 1 ? int(cluster_rank()) : 0;
    const int first = int(blockIdx.x) / (kCtas * split), step = int(gridDim.x) / (kCtas * split);
    constexpr int kItemStrip = C::kStrip * kCtas;
    const int strips = (args.D + kItemStrip - 1) / kItemStrip;
    pdl_wait();
    if (warp == 0) {
        // Group starts: the running maximum of the offsets clamped to [0, R],
        // so a bad array never leads out of the row operands; and each
        // expert's first item.
        int carry_row = 0, carry_item = 0, bad = 0;
        for (int b = 0; b <= args.E; b += 32) {
            const int i = b + lane;
            const int raw = i <= args.E ? __ldg(args.offsets + i) : args.R;
            const int clamped = min(max(raw, 0), args.R);
            const int row = max(warp_scan_max(clamped, lane), carry_row);
            if (i <= args.E) {
                bad |= row != raw;
                row_of[i] = row;
            }
            carry_row = __shfl_sync(0xFFFFFFFFu, row, 31);
        }
        __syncwarp();
        if constexpr (kMode != kGradWeight) {
            for (int b = 0; b < args.E; b += 32) {
                const int i = b + lane;
                const int n = i < args.E ? (row_of[i + 1] - row_of[i] + kN - 1) / kN * strips : 0;
                const int incl = warp_scan_sum(n, lane) + carry_item;
                if (i < args.E) item_of[i + 1] = incl;
                carry_item = __shfl_sync(0xFFFFFFFFu, incl, 31);
            }
            if (lane == 0) item_of[0] = 0;
        }
        bad = __any_sync(0xFFFFFFFFu, bad);
        // the call's error word (timeouts are added two seconds later at the earliest)
        if (blockIdx.x == 0 && lane == 0) {
            args.hdr[kHdrTimeoutWhere] = 0;
            args.hdr[kHdrError] = bad ? kDevErrBadRouting : 0;
        }
    }
    tc_fence_before();
    if constexpr (kPair)
        cluster_barrier();  // and the other CTA's barriers and TMEM are set up
    else
        __syncthreads();
    tc_fence_after();
    if (threadIdx.x == 0) pdl_trigger();
    const uint32_t tmem = *tmem_holder;

    Walker<kMode, kN, kTiles> walk;
    walk.row_of = row_of;
    walk.item_of = item_of;
    walk.E = args.E;
    walk.strips = strips;
    walk.kb_const = (args.C + kBlockK - 1) / kBlockK;
    walk.K = args.K;
    walk.D = args.D;
    const int num_items = kMode == kGradWeight ? args.E * strips * ((args.K + kN - 1) / kN) : item_of[args.E];
    int *err = args.hdr;
    // features of tile a of this CTA: the pair's tile a is its CTAs' 128 rows side by side
    auto tile_row = [&](const Item &it, int a) { return it.d0 + (kCtas * a + rank) * kTileRows; };
    auto two_tiles = [&](const Item &it) { return kTiles == 2 && it.d0 + kCtas * kTileRows < args.D; };
    // this CTA's stages of an item
    auto kb_lo = [&](const Item &it) { return C::kSplits ? it.kblocks * cut / split : 0; };
    auto kb_hi = [&](const Item &it) { return C::kSplits ? it.kblocks * (cut + 1) / split : it.kblocks; };
    // stage kb of a weight gradient's item ends inside a 16-row step
    auto tail_stage = [](const Item &it, int kb) {
        return kMode == kGradWeight && kb == it.kblocks - 1 && it.tail % 16 != 0;
    };
    // this CTA's part of the N side
    auto part = [&](const Item &it) { return (it.cols + 15) / 16 * 16 / kCtas; };

    if (warp == 0) {
        if (lane == 0) {
            // ------------------------------------------------------------ loads
            const uint64_t pol_once = policy_evict_first(), pol_n = policy_evict_last();
            int stage = 0;
            uint32_t phase = 0, filled = 0, fill_parity = 0;
            bool ok = true;
            for (int u = first; ok && u < num_items; u += step) {
                const Item it = walk.at(u);
                const int tiles_m = two_tiles(it) ? 2 : 1;
                // the weights are read once, or by an expert's row chunks at about the same
                // time (64 experts of 32 rows, 1024 x 1024: 29.8 us, 33.4 with all to be kept)
                const uint64_t pol_m = kMode != kGradWeight && row_of[it.e + 1] - row_of[it.e] <= kN ? pol_once : pol_n;
                const int n_part = part(it), n0 = it.n0 + rank * n_part;
                // (a load costs this thread about 190 cycles: the rows of large parts come in one)
                const bool big = !kNMn && n_part > C::kBRows / 2;
                const int boxes_n = kNMn ? (n_part + 63) / 64 : big ? C::kBRows / kRowBox : (n_part + kRowBox - 1) / kRowBox;
                const uint32_t bytes = uint32_t(tiles_m * kTileRows * 128 + boxes_n * (kNMn ? 64 : kRowBox) * 128);
                for (int kb = kb_lo(it); kb < kb_hi(it); ++kb) {
                    if (!mbar_wait_cycles(&empty[stage], phase ^ 1u, abort_flag, err, 31)) {
                        ok = false;
                        break;
                    }
                    uint8_t *a = tiles + stage * C::kStageBytes, *b = a + C::kABytes;
                    // both CTAs of a pair load the same number of bytes
                    const bool own = tail_stage(it, kb);
                    uint64_t *bar = own ? &landed[stage] : &full[stage];
                    if (own || rank == 0) mbar_arrive_expect_tx(bar, own ? bytes : kCtas * bytes);
                    const uint32_t signal = kPair && !own ? leader_bar(bar) : smem_u32(bar);
                    auto load_2d = [&](uint8_t *dst, const CUtensorMap *map, int c0, int c1, uint64_t pol) {
                        if constexpr (kPair)
                            tma_load_2d_pair(dst, map, signal, c0, c1, pol);
                        else
                            tma_load_2d(dst, map, bar, c0, c1, pol);
                    };
                    auto load_3d = [&](uint8_t *dst, const CUtensorMap *map, int c0, int c1, int c2, uint64_t pol) {
                        if constexpr (kPair)
                            tma_load_3d_pair(dst, map, signal, c0, c1, c2, pol);
                        else
                            tma_load_3d(dst, map, bar, c0, c1, c2, pol);
                    };
                    const int k = kb * kBlockK;
                    if constexpr (kMode == kProduct) {
                        for (int t = 0; t < tiles_m; ++t)
                            load_3d(a + t * kTileRows * 128, &tmap_m, k, tile_row(it, t), it.e, pol_m);
                    } else if (args.chunks_m) {
                        for (int t = 0; t < tiles_m; ++t) {
                            uint8_t *to = a + t * kTileRows * 128;
                            if constexpr (kMode == kGradWeight) {
                                load_3d(to, &tmap_m, 0, row_of[it.e] + k, tile_row(it, t) / 64, pol_m);
                            } else if constexpr (kPair) {
                                tma_load_4d_pair(to, &tmap_m, signal, 0, k, tile_row(it, t) / 64, it.e, pol_m);
                            } else {
                                tma_load_4d(to, &tmap_m, bar, 0, k, tile_row(it, t) / 64, it.e, pol_m);
                            }
                        }
                    } else {
                        for (int t = 0; t < 2 * tiles_m; ++t) {
                            const int d = tile_row(it, t >> 1) + (t & 1) * 64;
                            if constexpr (kMode == kGradInput)
                                load_3d(a + t * 64 * 128, &tmap_m, d, k, it.e, pol_m);
                            else
                                load_2d(a + t * 64 * 128, &tmap_m, d, row_of[it.e] + k, pol_m);
                        }
                    }
                    if (big) {
                        load_2d(b, &tmap_out, k, n0, pol_n);  // (those maps' boxes: kBRows rows)
                    } else if (kNMn && args.chunks_n) {
                        load_3d(b, &tmap_n, 0, row_of[it.e] + k, n0 / 64, pol_n);
                    } else {
                        for (int t = 0; t < boxes_n; ++t) {
                            if constexpr (kNMn)
                                load_2d(b + t * 64 * 128, &tmap_n, n0 + t * 64, row_of[it.e] + k, pol_n);
                            else
                                load_2d(b + t * kRowBox * 128, &tmap_n, k, n0 + t * kRowBox, pol_n);
                        }
                    }
                    filled |= 1u << stage;
                    fill_parity = (fill_parity & ~(1u << stage)) | (phase << stage);
                    if (++stage == kStages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            // Every issued copy must have landed before the CTA may exit, and a pair's
            // last commits must have reached it: both are so once its stages are
            // consumed.  After a wait that gave up nothing consumes them: a quarter of
            // a second, in which copies land.
            for (int s = 0; s < kStages; ++s)
                if (filled >> s & 1u) mbar_wait_cycles(&empty[s], fill_parity >> s & 1u, abort_flag, err, 37);
            if (*abort_flag) {
                const long long t0 = clock64();
                while (clock64() - t0 < kWaitTimeoutCycles / 8) {
                }
            }
        }
        __syncwarp();
    } else if (warp == 1 || warp == 2) {
        if (lane == 0 && rank == 0 && warp <= kTiles) {
            // ------------------------------------------------------------ MMA issuer of tile a
            const int a = warp - 1;
            auto wait = [&](uint64_t *bar, uint32_t parity, int where) {
                return kPair ? mbar_wait_cluster(bar, parity, abort_flag, err, where)
                             : mbar_wait_cycles(bar, parity, abort_flag, err, where);
            };
            auto commit = [&](uint64_t *bar) {
                if constexpr (kPair)
                    tc_commit_pair(bar);
                else
                    tc_commit(bar);
            };
            int stage = 0, li = 0;
            uint32_t full_uses = 0, zeroed_uses = 0;  // per stage, of each barrier: its phase
            bool ok = true;
            for (int u = first; ok && u < num_items; u += step) {
                const Item it = walk.at(u);
                if (it.kblocks == 0) continue;
                const bool valid = a == 0 || two_tiles(it);
                const uint32_t n = uint32_t((it.cols + 15) / 16 * 16);
                const uint32_t idesc = idesc_bf16(n) + (kPair ? (128u >> 4) << 24 : 0u)  // M = 256
                                       + (kMMn ? 1u << 15 : 0u) + (kNMn ? 1u << 16 : 0u);
                const int buf = li % C::kBufs;
                const uint32_t use = uint32_t(li / C::kBufs) & 1u;
                if (valid) {
                    if (!wait(&tmem_empty[2 * a + buf], use ^ 1u, 32)) break;
                    tc_fence_after();
                    ++li;
                }
                const uint32_t acc = tmem + uint32_t((buf * kTiles + a) * kN);
                const int kb0 = kb_lo(it);
                for (int kb = kb0; kb < kb_hi(it); ++kb) {
                    if (tail_stage(it, kb)) {
                        ok = wait(&zeroed[stage], zeroed_uses >> stage & 1u, 34);
                        zeroed_uses ^= 1u << stage;
                    } else {
                        ok = mbar_wait_cycles(&full[stage], full_uses >> stage & 1u, abort_flag, err, 33);
                        full_uses ^= 1u << stage;
                    }
                    if (!ok) break;
                    tc_fence_after();
                    if (valid) {
                        const int steps = kMode == kGradWeight && kb == it.kblocks - 1 ? (it.tail + 15) / 16 : kBlockK / 16;
                        const uint32_t st = smem_u32(tiles + stage * C::kStageBytes);
                        const uint32_t sa = st + uint32_t(a * kTileRows * 128), sb = st + C::kABytes;
                        const uint64_t adesc = kMMn ? smem_desc_mn_sw128(sa) : smem_desc_sw128(sa);
                        const uint64_t bdesc = kNMn ? smem_desc_mn_sw128(sb) : smem_desc_sw128(sb);
                        // a step is 16 contraction elements: 32 bytes inside the swizzled
                        // row (K-major) or 16 rows of 128 bytes (MN-major), in 16-byte units
                        for (int ks = 0; ks < steps; ++ks) {
                            const uint64_t ad = adesc + uint64_t(ks * (kMMn ? 128 : 2)), bd = bdesc + uint64_t(ks * (kNMn ? 128 : 2));
                            if constexpr (kPair)
                                tc_mma_bf16_pair(acc, ad, bd, idesc, kb > kb0 || ks ? 1u : 0u);
                            else
                                tc_mma_bf16(acc, ad, bd, idesc, kb > kb0 || ks ? 1u : 0u);
                        }
                    }
                    commit(&empty[stage]);
                    if (++stage == kStages) stage = 0;
                }
                if (!ok) break;
                if (valid) commit(&tmem_full[2 * a + buf]);
            }
            // all issued MMAs must be finished before TMEM is released
            tc_commit_own<kPair>(&mma_done[a]);
            const long long t0 = clock64();
            while (!mbar_try_wait(&mma_done[a], 0) && clock64() - t0 < kWaitTimeoutCycles) {
            }
        }
        __syncwarp();
    } else if (warp == 3) {
        if constexpr (kMode == kGradWeight) {
            // ------------------------------------------------------------ tail rows
            // The rows of the next group (or past the tensor) inside the last 16-row
            // step of an item, zeroed on both sides; a row is 128 bytes in every box,
            // so the swizzle inside it does not matter.
            int stage = 0;
            uint32_t landed_uses = 0;
            for (int u = first; u < num_items; u += step) {
                const Item it = walk.at(u);
                if (it.kblocks == 0) continue;
                const int last = (stage + it.kblocks - 1) % kStages;
                if (tail_stage(it, it.kblocks - 1)) {
                    if (!warp_wait(&landed[last], landed_uses >> last & 1u, abort_flag, err, 35)) break;
                    landed_uses ^= 1u << last;
                    uint8_t *a = tiles + last * C::kStageBytes + it.tail * 128;
                    constexpr int kBoxes = C::kStageBytes / (64 * 128);
                    for (int r = lane >> 3; r < 16 - it.tail % 16; r += 4)
#pragma unroll
                        for (int box = 0; box < kBoxes; ++box)
                            *reinterpret_cast<uint4 *>(a + box * 64 * 128 + r * 128 + (lane & 7) * 16) = make_uint4(0, 0, 0, 0);
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                    if (lane == 0) mbar_arrive_leader(&zeroed[last]);
                }
                stage = (last + 1) % kStages;
            }
        }
        __syncwarp();
    } else {
        // ---------------------------------------------------------------- epilogue of tile a
        constexpr int kGroups = kEpiWarps / 4 / kTiles;  // warps of a tile's lane quarter: every kGroups-th block of columns
        const int a = ((warp - 4) >> 2) % kTiles, q = warp & 3, group = ((warp - 4) >> 2) / kTiles;
        uint16_t *out_block = reinterpret_cast<uint16_t *>(stage_out + (warp - 4) * (C::kStageOutBytes / kEpiWarps));  // [row][32 features]
        if constexpr (kMode != kGradWeight) {
            if (args.zero_unused) {
                // rows before the first group and behind the last, 8 columns per store
                const int64_t v_row = args.D / 8;
                const int64_t head = row_of[0], behind = args.R - row_of[args.E];
                const int64_t total = (head + behind) * v_row;
                uint4 *o = reinterpret_cast<uint4 *>(args.out);
                constexpr int kWide = 32 * kEpiWarps;
                for (int64_t i = int64_t(blockIdx.x) * kWide + (threadIdx.x - 128); i < total;
                     i += int64_t(gridDim.x) * kWide) {
                    const int64_t r = i / v_row;
                    const int64_t row = r < head ? r : r - head + row_of[args.E];
                    o[row * v_row + (i - r * v_row)] = make_uint4(0, 0, 0, 0);
                }
            }
        }
        int li = 0;
        for (int u = first; u < num_items; u += step) {
            const Item it = walk.at(u);
            if (a == 1 && !two_tiles(it)) continue;
            const int d = tile_row(it, a) + q * 32 + lane;
            if constexpr (kMode == kGradWeight) {
                if (it.kblocks == 0) {
                    // an expert without rows: zeros, a warp row by row
                    const int pieces = it.cols / 8, rows = min(kTileRows, args.D - tile_row(it, a));
                    for (int r = q + 4 * group; r < rows; r += 4 * kGroups) {
                        uint4 *o = reinterpret_cast<uint4 *>(
                            args.out + (int64_t(it.e) * args.D + tile_row(it, a) + r) * args.K + it.n0);
                        if (lane < pieces) o[lane] = make_uint4(0, 0, 0, 0);
                    }
                    continue;
                }
            }
            const int buf = li % C::kBufs;
            const uint32_t use = uint32_t(li / C::kBufs) & 1u;
            if (!warp_wait(&tmem_full[2 * a + buf], use, abort_flag, err, 36)) break;
            tc_fence_after();
            ++li;
            const uint32_t acc = tmem + (uint32_t(q * 32) << 16) + uint32_t((buf * kTiles + a) * kN);
            const int blocks = (it.cols + 31) / 32;
            if (split > 1) {
                // a part of the contraction: its fp32 sums, [column][128 features], to the
                // ring (every stage of it has been consumed), for the whole cluster
                float *sums = reinterpret_cast<float *>(tiles) + q * 32 + lane;
#pragma unroll 1
                for (int cb = group; cb < blocks; cb += kGroups)
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        uint32_t v[16];
                        tmem_ld_32x16(acc + uint32_t(cb * 32 + half * 16), v);
                        tmem_ld_wait();
#pragma unroll
                        for (int j = 0; j < 16; ++j) sums[(cb * 32 + half * 16 + j) * kTileRows] = __uint_as_float(v[j]);
                    }
                break;
            }
            // Everything that reads TMEM first, rounded and packed in pairs of columns,
            // so that the next item's MMAs wait for as little as they can.
            constexpr int kMine = (kN / 32 + kGroups - 1) / kGroups;
            uint32_t h[kMine][16];
#pragma unroll
            for (int m = 0; m < kMine; ++m) {
                const int cb = kGroups * m + group;
                if (cb < blocks) {
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        uint32_t v[16];
                        tmem_ld_32x16(acc + uint32_t(cb * 32 + half * 16), v);
                        tmem_ld_wait();
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const __nv_bfloat162 p =
                                __floats2bfloat162_rn(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1]));
                            h[m][8 * half + j] = *reinterpret_cast<const uint32_t *>(&p);
                        }
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if constexpr (kPair)
                    mbar_arrive_leader(&tmem_empty[2 * a + buf]);
                else
                    mbar_arrive(&tmem_empty[2 * a + buf]);
            }
#pragma unroll
            for (int m = 0; m < kMine; ++m) {
                const int cb = kGroups * m + group;
                if (cb >= blocks) break;
                const int left = it.cols - cb * 32;
                if constexpr (kMode == kGradWeight) {
                    // thread = row n of dW, 32 consecutive columns k: a 32 x 32 box through
                    // shared memory (64-byte rows, 64-byte swizzle); the map cuts it at the
                    // last row and column.  (Stores from the registers cost the L1 a cycle
                    // per row: 933 us instead of 701 for 48 experts of 128 rows, 4096 x 7168.)
                    if (lane == 0) tma_store_wait_read();
                    __syncwarp();
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        *reinterpret_cast<uint4 *>(out_block + lane * 32 + ((j ^ ((lane >> 1) & 3)) * 8)) =
                            make_uint4(h[m][4 * j], h[m][4 * j + 1], h[m][4 * j + 2], h[m][4 * j + 3]);
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                    if (lane == 0 && d < args.D) tma_store_3d(&tmap_out, out_block, it.n0 + cb * 32, d, it.e);
                } else {
                    // thread = output feature d, 32 consecutive rows: turned around in
                    // shared memory, then 16 bytes of 8 rows at a time per warp
                    const int d8 = tile_row(it, a) + q * 32 + (lane & 3) * 8;  // D % 8 == 0
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const uint32_t pair = h[m][8 * half + j];
                            out_block[(2 * j) * 32 + lane] = static_cast<uint16_t>(pair);
                            out_block[(2 * j + 1) * 32 + lane] = static_cast<uint16_t>(pair >> 16);
                        }
                        __syncwarp();
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const int r = i * 8 + (lane >> 2);
                            const uint4 piece = *reinterpret_cast<const uint4 *>(out_block + r * 32 + (lane & 3) * 8);
                            if (16 * half + r < left && d8 < args.D)
                                *reinterpret_cast<uint4 *>(args.out + int64_t(it.n0 + cb * 32 + 16 * half + r) * args.D +
                                                           d8) = piece;
                        }
                        __syncwarp();
                    }
                }
            }
        }
        if (kMode == kGradWeight && lane == 0) tma_store_wait_all();
        __syncwarp();
    }
    if constexpr (C::kSplits)
        if (split > 1) {
            // the parts' sums, added in the order of the parts: every split-th column here
            cluster_barrier();
            if (warp >= 4 && first < num_items) {
                const Item it = walk.at(first);
                const int id = int(threadIdx.x) - 128, d = (id & 63) * 2;
                for (int c = cut + split * (id >> 6); c < it.cols && it.d0 + d < args.D; c += split * (kEpiWarps / 2)) {
                    const uint32_t at = smem_u32(reinterpret_cast<float *>(tiles) + c * kTileRows + d);
                    float2 v = make_float2(0.0f, 0.0f);
                    for (int p = 0; p < split; ++p) {
                        const float2 u = cluster_load(at, p);
                        v.x += u.x;
                        v.y += u.y;
                    }
                    *reinterpret_cast<__nv_bfloat162 *>(args.out + int64_t(it.n0 + c) * args.D + it.d0 + d) =
                        __floats2bfloat162_rn(v.x, v.y);
                }
            }
            cluster_barrier();  // the other parts have read this CTA's sums
        }
    tc_fence_before();
    if constexpr (kPair)
        cluster_barrier();  // the other CTA's MMAs, arrivals and commits for this one are over
    else
        __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc_for<kPair>(tmem, C::kTmemCols);
}

template <int kMode, int kN, int kTiles>
cudaError_t launch_grouped(const CUtensorMap &tmap_m, const CUtensorMap &tmap_n, const CUtensorMap &tmap_out,
                           GroupedArgs a, int64_t items, cudaStream_t stream) {
    using C = GroupedCfg<kMode, kN, kTiles>;
    a.stages = C::stages(a.E);
    const cudaError_t e = set_max_dynamic_smem(reinterpret_cast<const void *>(grouped_kernel<kMode, kN, kTiles>), kMaxSmem);
    if (e != cudaSuccess) return e;
    const int64_t groups = num_sms() / (C::kCtas * a.split);
    const int grid = int(items < groups ? items : groups) * C::kCtas * a.split;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(grid));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = size_t(C::fixed_bytes(a.E) + a.stages * C::kStageBytes);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = unsigned(C::kCtas * a.split);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = C::kCtas * a.split > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, grouped_kernel<kMode, kN, kTiles>, tmap_m, tmap_n, tmap_out, a);
}

// A configuration of the product and the input gradient.
struct Choice {
    int kn, tiles, split;
    int64_t items;  // at most, whatever the groups
};

// The one of the shortest time by an estimate in SM cycles from the sizes alone (the
// groups are on the device: half of the experts are taken to have 3/4 of the mean
// load, half 5/4).  A stage costs the longest of its MMAs (2 cycles a column and
// tile), of the ring's round trip (4000 cycles over its stages), and of what L2
// delivers to all CTAs at work (4840 bytes a cycle); an item its stages and the fill,
// longer with one accumulator.  On 40 loads, even and Zipf-like, from 1 x 1024 x 1024
// to 16384 x 4096 x 2048, both directions, its choice took 1.5 % more time than the
// best one in the mean and 25 % at most.  Examples, product: 8 experts, 2048 rows,
// 1024 x 1024: 12.8 us with 160 columns and one tile, 19.8 with 256 and two; 16
// experts, 16384 rows, 4096 x 2048: 313 and 203; 48 experts, 8 rows, 4096 x 7168: 86
// and 78, and 70 with 64 columns and two tiles.  A contraction in parts: 16 rows,
// 4096 x 4096: 26.6 us whole, 16.9 in two, 12.7 in four.
template <int kMode>
Choice choose(int R, int E, int D, int contraction) {
    const int sms = num_sms(), kblocks = (contraction + kBlockK - 1) / kBlockK, experts = R < E ? R : E;
    const double mean = double(R) / experts;
    auto larger = [](double a, double b) { return a > b ? a : b; };
    Choice best = {};
    double best_time = 0;
    for (int kn : {64, 160, 256}) {
        if (kn > 64 && mean <= 16) break;  // 48 experts, 8 rows, Zipf-like: 46.0 us, 54.9 with 160 columns
        for (int tiles = 1; tiles <= (kn == 160 ? 1 : 2); ++tiles) {
            const int ctas = kn >= 160 ? 2 : 1, units = sms / ctas;
            const int64_t strips = (D + kTileRows * tiles * ctas - 1) / (kTileRows * tiles * ctas);
            const int64_t most = (R + int64_t(experts) * (kn - 1)) / kn * strips;
            const double chunks =
                experts == 1 ? (R + int64_t(kn) - 1) / kn : (larger(1.0, 0.75 * mean / kn) + larger(1.0, 1.25 * mean / kn)) / 2;
            const double cols = larger(16.0, mean / chunks), items = experts * chunks * double(strips);
            const double bytes = tiles * 16384 + int((cols + 31) / 32) * 4096.0 / ctas;
            const int ring = 214000 / (tiles * 16384 + kn * 128 / ctas);
            const double mma = larger(280.0, 2.0 * tiles * cols);
            for (int split = 1; split <= 8; split *= 2) {
                // one item per cluster, and stages enough in each part
                if (split > 1 && (kn > 64 || tiles > 1 || kblocks < 4 * split ||
                                  most > resident_clusters(reinterpret_cast<const void *>(grouped_kernel<kMode, 64, 1>), split,
                                                           kThreads, kMaxSmem)))
                    break;
                const double rounds = larger(1.0, items * split / units), at_work = items * split < units ? items * split : units;
                const double stage = larger(larger(mma, 4000.0 / ring), bytes * at_work * ctas / 4840);
                const double time = 3000 + rounds * (stage * kblocks / split + (tiles * kn > 256 ? 2000 : 1000)) + (split > 1 ? 2500 : 0);
                if (best.kn == 0 || time < best_time) {
                    best_time = time;
                    best = {kn, tiles, split, most};
                }
            }
        }
    }
    return best;
}

template <int kMode>
cudaError_t launch_rows(const CUtensorMap &tm, const CUtensorMap &tn, const void *rows, GroupedArgs a, cudaStream_t stream) {
    const cudaError_t e = set_max_dynamic_smem(reinterpret_cast<const void *>(grouped_kernel<kMode, 64, 1>), kMaxSmem);
    if (e != cudaSuccess) return e;
    const Choice c = choose<kMode>(a.R, a.E, a.D, a.C);
    a.split = c.split;
    CUtensorMap tb;  // the rows in boxes as large as a stage's part
    const int box = c.kn == 64 ? GroupedCfg<kMode, 64, 1>::kBRows
                    : c.kn == 160 ? GroupedCfg<kMode, 160, 1>::kBRows : GroupedCfg<kMode, 256, 1>::kBRows;
    if (!encode_bf16_rows(&tb, rows, uint64_t(a.C), uint64_t(a.R), box)) return cudaErrorInvalidValue;
    switch (c.kn + c.tiles) {
        case 64 + 1: return launch_grouped<kMode, 64, 1>(tm, tn, tb, a, c.items, stream);
        case 64 + 2: return launch_grouped<kMode, 64, 2>(tm, tn, tb, a, c.items, stream);
        case 160 + 1: return launch_grouped<kMode, 160, 1>(tm, tn, tb, a, c.items, stream);
        case 256 + 1: return launch_grouped<kMode, 256, 1>(tm, tn, tb, a, c.items, stream);
        default: return launch_grouped<kMode, 256, 2>(tm, tn, tb, a, c.items, stream);
    }
}

moe_status_t check_grouped(int R, int E, int N, int K) {
    if (R < 0 || E <= 0 || N <= 0 || K <= 0) return MOE_ERR_INVALID_ARG;
    if (R > kMaxRows || E > kMaxExperts || N % 8 || K % 8 || N > kGroupedMaxWidth || K > kGroupedMaxWidth) return MOE_ERR_UNSUPPORTED_SHAPE;
    // every expert's items fit an int: strips <= 1024, chunks <= R / 64 + E
    if ((int64_t(R) / 64 + E) * ((int64_t(N > K ? N : K) + kTileRows - 1) / kTileRows) > 2000000000ll ||
        int64_t(E) * ((N + 255) / 256) * ((K + 255) / 256) > 2000000000ll)
        return MOE_ERR_UNSUPPORTED_SHAPE;
    return MOE_OK;
}

// The product (grad = false: rows x [R, K] -> out [R, N]) or the input
// gradient (rows dy [R, N] -> out [R, K]).
moe_status_t run_rows(bool grad, const void *rows, const void *w, const int32_t *offsets, void *out, int R, int E,
                      int N, int K, int zero_unused, void *workspace, size_t ws_bytes, moe_stream_t stream) {
    moe_status_t s = check_grouped(R, E, N, K);
    if (s != MOE_OK) return s;
    if (R == 0) return MOE_OK;
    if (!rows || !w || !offsets || !out || !workspace || !aligned(rows, 16) || !aligned(w, 16) ||
        !aligned(offsets, 4) || !aligned(out, 16) || !aligned(workspace, 256))
        return MOE_ERR_INVALID_ARG;
    if (ws_bytes < size_t(kHdrBytes)) return MOE_ERR_WORKSPACE_TOO_SMALL;
    DeviceScope dev(out);
    if (dev.status != MOE_OK) return dev.status;
    GroupedArgs a{};
    a.offsets = offsets;
    a.out = static_cast<__nv_bfloat16 *>(out);
    a.hdr = static_cast<int *>(workspace);
    a.R = R;
    a.E = E;
    a.D = grad ? K : N;
    a.C = grad ? N : K;
    a.K = K;
    a.zero_unused = zero_unused;
    CUtensorMap tm, tn;
    a.chunks_m = grad && K % 64 == 0;
    if (!(a.chunks_m ? encode_bf16_chunks(&tm, 4, w, uint64_t(K), uint64_t(N), uint64_t(E), kBlockK)
                     : encode_bf16_3d(&tm, w, uint64_t(K), uint64_t(N), uint64_t(E), grad ? kBlockK : kTileRows)) ||
        !encode_bf16_rows(&tn, rows, uint64_t(a.C), uint64_t(R), kRowBox))
        return MOE_ERR_CUDA;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = grad ? launch_rows<kGradInput>(tm, tn, rows, a, st) : launch_rows<kProduct>(tm, tn, rows, a, st);
    return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

moe_status_t moe_grouped_workspace_bytes(size_t *bytes) {
    if (!bytes) return MOE_ERR_INVALID_ARG;
    *bytes = kHdrBytes;
    return MOE_OK;
}

moe_status_t moe_grouped_unread_workspace(int device, void **workspace) {
    if (device < 0 || !workspace) return MOE_ERR_INVALID_ARG;
    int current = -1;
    if (cudaGetDevice(&current) != cudaSuccess) return MOE_ERR_CUDA;
    if (current != device && cudaSetDevice(device) != cudaSuccess) {
        cudaGetLastError();
        return MOE_ERR_CUDA;
    }
    void *p = nullptr;
    const cudaError_t e = cudaGetSymbolAddress(&p, g_grouped_unread);
    if (e != cudaSuccess) cudaGetLastError();
    if (current != device) cudaSetDevice(current);
    if (e != cudaSuccess || !p) return MOE_ERR_CUDA;
    *workspace = p;
    return MOE_OK;
}

moe_status_t moe_grouped_matmul(const void *x_bf16, const void *w_bf16, const int32_t *offsets, void *y_bf16, int R,
                                int E, int N, int K, int zero_unused, void *workspace, size_t ws_bytes,
                                moe_stream_t stream) {
    return run_rows(false, x_bf16, w_bf16, offsets, y_bf16, R, E, N, K, zero_unused, workspace, ws_bytes, stream);
}

moe_status_t moe_grouped_matmul_grad_input(const void *dy_bf16, const void *w_bf16, const int32_t *offsets,
                                           void *dx_bf16, int R, int E, int N, int K, int zero_unused, void *workspace,
                                           size_t ws_bytes, moe_stream_t stream) {
    return run_rows(true, dy_bf16, w_bf16, offsets, dx_bf16, R, E, N, K, zero_unused, workspace, ws_bytes, stream);
}

moe_status_t moe_grouped_matmul_grad_weight(const void *dy_bf16, const void *x_bf16, const int32_t *offsets,
                                            void *dw_bf16, int R, int E, int N, int K, void *workspace, size_t ws_bytes,
                                            moe_stream_t stream) {
    moe_status_t s = check_grouped(R, E, N, K);
    if (s != MOE_OK) return s;
    if (!dw_bf16 || !offsets || !workspace || !aligned(dw_bf16, 16) || !aligned(offsets, 4) ||
        !aligned(workspace, 256) || (R > 0 && (!dy_bf16 || !x_bf16 || !aligned(dy_bf16, 16) || !aligned(x_bf16, 16))))
        return MOE_ERR_INVALID_ARG;
    if (ws_bytes < size_t(kHdrBytes)) return MOE_ERR_WORKSPACE_TOO_SMALL;
    DeviceScope dev(dw_bf16);
    if (dev.status != MOE_OK) return dev.status;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (R == 0) {
        // no rows to map: every gradient is zero, and the error word says so
        cudaError_t e = cudaMemsetAsync(dw_bf16, 0, size_t(E) * size_t(N) * size_t(K) * 2, st);
        if (e == cudaSuccess) e = cudaMemsetAsync(workspace, 0, kHdrBytes, st);
        return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
    }
    GroupedArgs a{};
    a.offsets = offsets;
    a.out = static_cast<__nv_bfloat16 *>(dw_bf16);
    a.hdr = static_cast<int *>(workspace);
    a.R = R;
    a.E = E;
    a.D = N;
    a.K = K;
    CUtensorMap tm, tn, to;
    a.chunks_m = N % 64 == 0;
    a.chunks_n = K % 256 == 0;  // every item has its 256 columns: a CTA's begin at a chunk
    if (!(a.chunks_m ? encode_bf16_chunks(&tm, 3, dy_bf16, uint64_t(N), uint64_t(R), 1, kBlockK)
                     : encode_bf16_rows(&tm, dy_bf16, uint64_t(N), uint64_t(R), kBlockK)) ||
        !(a.chunks_n ? encode_bf16_chunks(&tn, 3, x_bf16, uint64_t(K), uint64_t(R), 1, kBlockK)
                     : encode_bf16_rows(&tn, x_bf16, uint64_t(K), uint64_t(R), kBlockK)) ||
        !encode_bf16_3d(&to, dw_bf16, uint64_t(K), uint64_t(N), uint64_t(E), 32, 32))
        return MOE_ERR_CUDA;
    a.split = 1;
    // strips of 512 rows of dW per pair, or of 256 while they would leave most pairs
    // idle (2 experts of 512 x 512, 4096 rows: 26.3 -> 20.9 us; at 64 items 11.6 against 12.5)
    const int64_t items = int64_t(E) * ((N + 511) / 512) * ((K + 255) / 256);
    const cudaError_t e = items <= 32 ? launch_grouped<kGradWeight, 256, 1>(tm, tn, to, a, 2 * items, st)
                                      : launch_grouped<kGradWeight, 256, 2>(tm, tn, to, a, items, st);
    return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
