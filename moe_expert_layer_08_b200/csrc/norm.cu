// norm.cu -- the root-mean-square norms around the expert layer, fused with
// what stands next to them, and their gradients:
//   before   y = x rstd w,  rstd = (mean(x^2) + eps)^-1/2, as bf16 and/or as
//            the layer's quantised input (E4M3 codes of bf16(y) with a UE8M0
//            scale per 32: what moe_quantize_fp8 makes of y)
//   after    out = a residual + g * (x rstd w), g a gate per channel, per
//            token, per element or none
// and, with xhat = x rstd and dz the gradient that reaches x rstd w,
//   dx = rstd (dz w - xhat mean(dz w xhat)) [+ the residual branch's gradient]
//   dw = sum_t dz xhat,  dg = dout (x rstd w) summed to g's shape.
// All four are bound by HBM.  A block takes every gridDim.x-th row with its
// columns fixed to its threads (8 at a time, 16-byte accesses), so the column
// sums of the gradients stay in registers over the rows.  A thread brings its
// own pieces of the rows ahead into its own part of a shared-memory ring
// (cp.async), so several rows a block are in flight and no barrier is needed
// to read them.  Sums are fp32; the column sums of the blocks are written out
// and added in block order by a second kernel, so results do not depend on
// timing.
#include "moe_common.cuh"
#include "moe_internal.h"

namespace moe {
namespace {

constexpr int kNormMaxH = 16384;
constexpr int kNormMaxBlocks = 512;  // column sums a workspace holds: the gradients' blocks, at most

struct Bf16x8 {
    uint4 u;
    __device__ __forceinline__ float2 pair(int i) const {
        const uint32_t w = i == 0 ? u.x : i == 1 ? u.y : i == 2 ? u.z : u.w;
        return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
    }
};

__device__ __forceinline__ Bf16x8 load8(const __nv_bfloat16 *p) {
    Bf16x8 v;
    v.u = __ldg(reinterpret_cast<const uint4 *>(p));
    return v;
}
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&p);
}
__device__ __forceinline__ Bf16x8 pack8(const float (&v)[8]) {
    Bf16x8 r;
    r.u = make_uint4(pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7]));
    return r;
}
__device__ __forceinline__ void store8(__nv_bfloat16 *p, const Bf16x8 &v) { *reinterpret_cast<uint4 *>(p) = v.u; }

// The block's sum of v (and of w), in every thread.  `red` holds two sets of
// 2 x 32 floats; the caller alternates them, so one barrier a call is enough.
__device__ __forceinline__ float2 block_sum(float v, float w, float (*red)[32]) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
        w += __shfl_xor_sync(0xFFFFFFFFu, w, d);
    }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
    if (lane == 0) {
        red[0][warp] = v;
        red[1][warp] = w;
    }
    __syncthreads();
    v = lane < nw ? red[0][lane] : 0.0f;
    w = lane < nw ? red[1][lane] : 0.0f;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
        w += __shfl_xor_sync(0xFFFFFFFFu, w, d);
    }
    return make_float2(v, w);
}

struct NormArgs {
    const __nv_bfloat16 *x, *weight, *residual, *gate;
    __nv_bfloat16 *y;      // before: y (or null); after: out
    uint8_t *q, *sf;       // before: codes and scales (or null)
    float *rstd_out;       // [T] or null
    int T, H;
    float eps, alpha;
    int gate_kind;
    // gradients
    const __nv_bfloat16 *dy;        // before: dy; after: dout
    const __nv_bfloat16 *dres_in;   // before: the residual branch's gradient (or null)
    const float *rstd;
    __nv_bfloat16 *dx, *dres;
    float *part;                    // [blocks][1 or 2][H] column sums
    void *dgate;                    // per token: f32 [T]; per element: bf16 [T, H]
};

// Rows ahead in shared memory: more where a row has fewer streams.
constexpr int norm_depth(int streams) { return 5 - streams; }

// The ring of one thread's pieces: kStreams inputs of a row, norm_depth rows.
template <int kVecs, int kStreams>
struct RowRing {
    static constexpr int kDepth = norm_depth(kStreams);
    uint4 *mine;               // this thread's first piece
    const __nv_bfloat16 *src[kStreams];
    int T, H, row, slot;       // the next row to bring, and where

    __device__ __forceinline__ uint4 *at(int slot_, int stream, int i) const {
        return mine + ((slot_ * kStreams + stream) * kVecs + i) * blockDim.x;
    }
    __device__ __forceinline__ void next() {
        if (row < T) {
#pragma unroll
            for (int s = 0; s < kStreams; ++s)
#pragma unroll
                for (int i = 0; i < kVecs; ++i) {
                    const int c = threadIdx.x + i * blockDim.x;
                    if (c < H / 8)
                        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(at(slot, s, i))),
                                     "l"(src[s] + int64_t(row) * H + c * 8)
                                     : "memory");
                }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        row += gridDim.x;
        if (++slot == kDepth) slot = 0;
    }
    // All but the newest kDepth - 1 rows have landed (for this thread).
    __device__ __forceinline__ void wait() const {
        asm volatile("cp.async.wait_group %0;" ::"n"(kDepth - 1) : "memory");
    }
    __device__ __forceinline__ Bf16x8 get(int slot_, int stream, int i) const {
        Bf16x8 v;
        v.u = *at(slot_, stream, i);
        return v;
    }
};

// Forward of both norms. kVecs: 8-column pieces of a row per thread. Streams:
// x; after: x, residual and, for a gate per element, that.
template <int kVecs, bool kAfter, int kStreams>
__global__ void __launch_bounds__(kVecs == 1 ? 1024 : 512, kVecs == 1 ? 1 : 2) norm_kernel(const NormArgs a) {
    extern __shared__ uint4 ring_smem[];
    __shared__ float red[2][2][32];
    const int nvec = a.H / 8;
    pdl_wait();
    pdl_trigger();
    RowRing<kVecs, kStreams> ring;
    ring.mine = ring_smem + threadIdx.x;
    ring.src[0] = a.x;
    if constexpr (kStreams > 1) ring.src[1] = a.residual;
    if constexpr (kStreams > 2) ring.src[2] = a.gate;
    ring.T = a.T;
    ring.H = a.H;
    ring.row = blockIdx.x;
    ring.slot = 0;
#pragma unroll
    for (int d = 0; d < ring.kDepth - 1; ++d) ring.next();
    int flip = 0, slot = 0;
    for (int row = blockIdx.x; row < a.T; row += gridDim.x, flip ^= 1) {
        const int64_t base = int64_t(row) * a.H;
        ring.next();
        ring.wait();
        float ss = 0.0f;
#pragma unroll
        for (int i = 0; i < kVecs; ++i)
            if (int(threadIdx.x + i * blockDim.x) < nvec) {
                const Bf16x8 x = ring.get(slot, 0, i);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 v = x.pair(j);
                    ss = fmaf(v.x, v.x, ss);
                    ss = fmaf(v.y, v.y, ss);
                }
            }
        const float rstd = __frsqrt_rn(block_sum(ss, 0.0f, red[flip]).x / float(a.H) + a.eps);
        if (a.rstd_out && threadIdx.x == 0) a.rstd_out[row] = rstd;
        float tgate = 1.0f;
        if (kAfter && a.gate_kind == MOE_GATE_TOKEN) tgate = __bfloat162float(a.gate[row]);
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            const int c = threadIdx.x + i * blockDim.x;
            const bool in = c < nvec;
            float v[8];
            if (in) {
                const Bf16x8 x = ring.get(slot, 0, i), w = load8(a.weight + c * 8);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 xv = x.pair(j), wv = w.pair(j);
                    v[2 * j] = xv.x * rstd * wv.x;
                    v[2 * j + 1] = xv.y * rstd * wv.y;
                }
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = 0.0f;
            }
            if constexpr (kAfter) {
                if (in) {
                    const Bf16x8 r = ring.get(slot, 1, i);
                    Bf16x8 g;
                    if constexpr (kStreams > 2) {
                        g = ring.get(slot, 2, i);
                    } else {
                        if (a.gate_kind == MOE_GATE_CHANNEL) g = load8(a.gate + c * 8);
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float2 rv = r.pair(j);
                        float2 gv = make_float2(tgate, tgate);
                        if (kStreams > 2 || a.gate_kind == MOE_GATE_CHANNEL) gv = g.pair(j);
                        v[2 * j] = fmaf(gv.x, v[2 * j], a.alpha * rv.x);
                        v[2 * j + 1] = fmaf(gv.y, v[2 * j + 1], a.alpha * rv.y);
                    }
                    store8(a.y + base + c * 8, pack8(v));
                }
            } else {
                const Bf16x8 y = pack8(v);
                if (a.y && in) store8(a.y + base + c * 8, y);
                if (a.q) {
                    // a group of 32 columns is four neighbouring lanes
                    float amax = 0.0f;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float2 b = y.pair(j);
                        v[2 * j] = b.x;
                        v[2 * j + 1] = b.y;
                        amax = fmaxf(amax, fmaxf(fabsf(b.x), fabsf(b.y)));
                    }
                    amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
                    amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
                    const int e = scale_exponent<true>(amax);
                    const float m = exp2_neg(e);
                    uint32_t code[2];
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const float s[4] = {v[4 * j] * m, v[4 * j + 1] * m, v[4 * j + 2] * m, v[4 * j + 3] * m};
                        code[j] = to_e4m3x4(s);
                    }
                    if (in) {
                        *reinterpret_cast<uint2 *>(a.q + base + c * 8) = make_uint2(code[0], code[1]);
                        if ((threadIdx.x & 3) == 0) a.sf[(base + c * 8) / 32] = uint8_t(e + 127);
                    }
                }
            }
        }
        if (++slot == ring.kDepth) slot = 0;
    }
}

// Gradients of both norms: dx, the residual branch, per-token and per-element
// gates; the column sums of the weight (and of a per-channel gate) per block.
// Streams: dy, x; then before: the residual branch's gradient if there is one,
// after: a gate per element.
template <int kVecs, bool kAfter, int kStreams>
__global__ void __launch_bounds__(kVecs == 1 ? 1024 : 512, kVecs == 2 ? 2 : 1) norm_backward_kernel(const NormArgs a) {
    extern __shared__ uint4 ring_smem[];
    __shared__ float red[2][2][32];
    const int nvec = a.H / 8;
    const bool channel = kAfter && kStreams == 2 && a.gate_kind == MOE_GATE_CHANNEL;
    pdl_wait();
    pdl_trigger();
    RowRing<kVecs, kStreams> ring;
    ring.mine = ring_smem + threadIdx.x;
    ring.src[0] = a.dy;
    ring.src[1] = a.x;
    if constexpr (kStreams > 2) ring.src[2] = kAfter ? a.gate : a.dres_in;
    ring.T = a.T;
    ring.H = a.H;
    ring.row = blockIdx.x;
    ring.slot = 0;
#pragma unroll
    for (int d = 0; d < ring.kDepth - 1; ++d) ring.next();
    float dw[kVecs][8], dg[kAfter && kStreams == 2 ? kVecs : 1][8];
#pragma unroll
    for (int i = 0; i < kVecs; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            dw[i][j] = 0.0f;
            if (kAfter && kStreams == 2) dg[i][j] = 0.0f;
        }
    int flip = 0, slot = 0;
    for (int row = blockIdx.x; row < a.T; row += gridDim.x, flip ^= 1) {
        const int64_t base = int64_t(row) * a.H;
        const float rstd = a.rstd[row];
        float tgate = 1.0f;
        if (kAfter && a.gate_kind == MOE_GATE_TOKEN) tgate = __bfloat162float(a.gate[row]);
        ring.next();
        ring.wait();
        // the gate of piece i (its elements, or one value for all of them)
        auto gate_of = [&](int i, int c, Bf16x8 &g) {
            if constexpr (kAfter) {
                if constexpr (kStreams > 2)
                    g = ring.get(slot, 2, i);
                else if (channel)
                    g = load8(a.gate + c * 8);
            }
        };
        float dot = 0.0f, tsum = 0.0f;
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            const int c = threadIdx.x + i * blockDim.x;
            if (c >= nvec) continue;
            const Bf16x8 dy = ring.get(slot, 0, i), x = ring.get(slot, 1, i), w = load8(a.weight + c * 8);
            Bf16x8 g;
            gate_of(i, c, g);
            float de[8];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 x2 = x.pair(j), d2 = dy.pair(j), w2 = w.pair(j);
                const float2 xh = make_float2(x2.x * rstd, x2.y * rstd);
                float2 dz = d2;
                if constexpr (kAfter) {
                    float2 g2 = make_float2(tgate, tgate);
                    if (kStreams > 2 || channel) g2 = g.pair(j);
                    dz = make_float2(d2.x * g2.x, d2.y * g2.y);
                    de[2 * j] = d2.x * (xh.x * w2.x);
                    de[2 * j + 1] = d2.y * (xh.y * w2.y);
                    if constexpr (kStreams == 2) {
                        dg[i][2 * j] += de[2 * j];
                        dg[i][2 * j + 1] += de[2 * j + 1];
                        tsum += de[2 * j];
                        tsum += de[2 * j + 1];
                    }
                }
                dw[i][2 * j] = fmaf(dz.x, xh.x, dw[i][2 * j]);
                dw[i][2 * j + 1] = fmaf(dz.y, xh.y, dw[i][2 * j + 1]);
                dot = fmaf(dz.x * w2.x, xh.x, dot);
                dot = fmaf(dz.y * w2.y, xh.y, dot);
            }
            if constexpr (kAfter && kStreams > 2)
                store8(static_cast<__nv_bfloat16 *>(a.dgate) + base + c * 8, pack8(de));
        }
        const float2 s = block_sum(dot, tsum, red[flip]);
        const float mean = s.x / float(a.H);
        if (kAfter && a.gate_kind == MOE_GATE_TOKEN && threadIdx.x == 0) static_cast<float *>(a.dgate)[row] = s.y;
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            const int c = threadIdx.x + i * blockDim.x;
            if (c >= nvec) continue;
            const Bf16x8 dy = ring.get(slot, 0, i), x = ring.get(slot, 1, i), w = load8(a.weight + c * 8);
            Bf16x8 g, add;
            gate_of(i, c, g);
            if constexpr (!kAfter && kStreams > 2) add = ring.get(slot, 2, i);
            float v[8], r[8];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 x2 = x.pair(j), d2 = dy.pair(j), w2 = w.pair(j);
                const float2 xh = make_float2(x2.x * rstd, x2.y * rstd);
                float2 dz = d2;
                if constexpr (kAfter) {
                    float2 g2 = make_float2(tgate, tgate);
                    if (kStreams > 2 || channel) g2 = g.pair(j);
                    dz = make_float2(d2.x * g2.x, d2.y * g2.y);
                    r[2 * j] = a.alpha * d2.x;
                    r[2 * j + 1] = a.alpha * d2.y;
                }
                v[2 * j] = rstd * (dz.x * w2.x - xh.x * mean);
                v[2 * j + 1] = rstd * (dz.y * w2.y - xh.y * mean);
                if constexpr (!kAfter && kStreams > 2) {
                    const float2 a2 = add.pair(j);
                    v[2 * j] += a2.x;
                    v[2 * j + 1] += a2.y;
                }
            }
            store8(a.dx + base + c * 8, pack8(v));
            if (kAfter) store8(a.dres + base + c * 8, pack8(r));
        }
        if (++slot == ring.kDepth) slot = 0;
    }
    float *p = a.part + int64_t(blockIdx.x) * (channel ? 2 : 1) * a.H;
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
        const int c = threadIdx.x + i * blockDim.x;
        if (c >= nvec) continue;
        reinterpret_cast<float4 *>(p + c * 8)[0] = make_float4(dw[i][0], dw[i][1], dw[i][2], dw[i][3]);
        reinterpret_cast<float4 *>(p + c * 8)[1] = make_float4(dw[i][4], dw[i][5], dw[i][6], dw[i][7]);
        if constexpr (kAfter && kStreams == 2)
            if (channel) {
                reinterpret_cast<float4 *>(p + a.H + c * 8)[0] = make_float4(dg[i][0], dg[i][1], dg[i][2], dg[i][3]);
                reinterpret_cast<float4 *>(p + a.H + c * 8)[1] = make_float4(dg[i][4], dg[i][5], dg[i][6], dg[i][7]);
            }
    }
}

// The blocks' column sums [blocks][cols] added up in a fixed order: 32 columns
// a block, 16 warps each taking every 16th partial, their sums added in warp
// order.  Columns 0 .. H-1 are dw, H .. 2H-1 a per-channel dgate.
constexpr int kColumnWarps = 16;
__global__ void __launch_bounds__(kColumnWarps * 32) column_sums_kernel(const float *part, int blocks, int cols, int H,
                                                                        float *dw, float *dg) {
    __shared__ float s[kColumnWarps][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int c = blockIdx.x * 32 + lane;
    pdl_wait();
    float v = 0.0f;
    if (c < cols) {
#pragma unroll 8
        for (int b = warp; b < blocks; b += kColumnWarps) v += part[int64_t(b) * cols + c];
    }
    s[warp][lane] = v;
    __syncthreads();
    if (warp == 0 && c < cols) {
        v = 0.0f;
#pragma unroll
        for (int i = 0; i < kColumnWarps; ++i) v += s[i][lane];
        (c < H ? dw : dg)[c < H ? c : c - H] = v;
    }
}

// Threads, 8-column pieces per thread and ring bytes of a row of H columns.
struct RowShape {
    int threads, vecs, bytes;
};
RowShape row_shape(int H, int vecs, int streams) {
    const int nvec = H / 8;
    while ((nvec + vecs - 1) / vecs > (vecs == 1 ? 1024 : 512)) vecs *= 2;  // H <= 16384: at most 4
    const int threads = ((nvec + vecs - 1) / vecs + 31) / 32 * 32;
    return {threads, vecs, threads * vecs * 16 * streams * norm_depth(streams)};
}
// Blocks of a launch: what one SM holds (64 registers a thread) on every SM.
int row_blocks(int T, const RowShape &s, int most_per_sm) {
    int per_sm = 1024 / s.threads;
    const int by_smem = 232448 / (s.bytes + 2048);
    if (per_sm > by_smem) per_sm = by_smem;
    if (per_sm > most_per_sm) per_sm = most_per_sm;
    if (per_sm < 1) per_sm = 1;
    const int cap = num_sms() * per_sm;
    return T < cap ? T : cap;
}

moe_status_t check_norm(int T, int H, float eps) {
    if (T < 0 || H <= 0 || !(eps > 0.0f) || !(eps <= 3.4e38f)) return MOE_ERR_INVALID_ARG;
    if (H % 8 || H > kNormMaxH) return MOE_ERR_UNSUPPORTED_SHAPE;
    return MOE_OK;
}

template <int kVecs, bool kAfter, int kStreams>
cudaError_t launch_norm(const NormArgs &a, const RowShape &s, cudaStream_t stream) {
    const cudaError_t e =
        set_max_dynamic_smem(reinterpret_cast<const void *>(norm_kernel<kVecs, kAfter, kStreams>), s.bytes);
    if (e != cudaSuccess) return e;
    return launch_pdl(norm_kernel<kVecs, kAfter, kStreams>, dim3(unsigned(row_blocks(a.T, s, 8))),
                      dim3(unsigned(s.threads)), size_t(s.bytes), stream, a);
}

template <bool kAfter, int kStreams>
moe_status_t run_norm(const NormArgs &a, cudaStream_t stream) {
    // a decode batch: one piece per thread, for latency; else four, for fewer barriers a byte
    const RowShape s = row_shape(a.H, a.T <= num_sms() ? 1 : 4, kStreams);
    const cudaError_t e = s.vecs == 1   ? launch_norm<1, kAfter, kStreams>(a, s, stream)
                          : s.vecs == 2 ? launch_norm<2, kAfter, kStreams>(a, s, stream)
                                        : launch_norm<4, kAfter, kStreams>(a, s, stream);
    return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

template <int kVecs, bool kAfter, int kStreams>
cudaError_t launch_norm_backward(const NormArgs &a, const RowShape &s, int grid, cudaStream_t stream) {
    const cudaError_t e =
        set_max_dynamic_smem(reinterpret_cast<const void *>(norm_backward_kernel<kVecs, kAfter, kStreams>), s.bytes);
    if (e != cudaSuccess) return e;
    return launch_pdl(norm_backward_kernel<kVecs, kAfter, kStreams>, dim3(unsigned(grid)), dim3(unsigned(s.threads)),
                      size_t(s.bytes), stream, a);
}

template <bool kAfter, int kStreams>
moe_status_t run_norm_backward(const NormArgs &a, float *dw, float *dg, cudaStream_t stream) {
    const RowShape s = row_shape(a.H, a.T <= num_sms() ? 1 : 2, kStreams);
    // few blocks: each leaves column sums to write and add
    int grid = row_blocks(a.T, s, 3);
    if (grid > kNormMaxBlocks) grid = kNormMaxBlocks;
    cudaError_t e = s.vecs == 1   ? launch_norm_backward<1, kAfter, kStreams>(a, s, grid, stream)
                    : s.vecs == 2 ? launch_norm_backward<2, kAfter, kStreams>(a, s, grid, stream)
                                  : launch_norm_backward<4, kAfter, kStreams>(a, s, grid, stream);
    if (e == cudaSuccess) {
        const int cols = a.H * (kAfter && a.gate_kind == MOE_GATE_CHANNEL ? 2 : 1);
        e = launch_pdl(column_sums_kernel, dim3(unsigned((cols + 31) / 32)), dim3(kColumnWarps * 32), 0, stream,
                       static_cast<const float *>(a.part), grid, cols, a.H, dw, dg);
    }
    return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

bool bad_gate(int kind) { return kind < MOE_GATE_NONE || kind > MOE_GATE_FULL; }

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

moe_status_t moe_norm_before(const void *x_bf16, const void *weight_bf16, int T, int H, float eps, void *y_bf16,
                             void *y_fp8, void *y_sf, float *rstd, moe_stream_t stream) {
    const moe_status_t s = check_norm(T, H, eps);
    if (s != MOE_OK) return s;
    if ((!y_fp8) != (!y_sf)) return MOE_ERR_INVALID_ARG;
    if (y_fp8 && H % 32) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (T == 0) return MOE_OK;
    if (!x_bf16 || !weight_bf16 || (!y_bf16 && !y_fp8) || !aligned(x_bf16, 16) || !aligned(weight_bf16, 16) ||
        !aligned(y_bf16, 16) || !aligned(y_fp8, 16) || !aligned(rstd, 4))
        return MOE_ERR_INVALID_ARG;
    DeviceScope dev(x_bf16);
    if (dev.status != MOE_OK) return dev.status;
    NormArgs a{};
    a.x = static_cast<const __nv_bfloat16 *>(x_bf16);
    a.weight = static_cast<const __nv_bfloat16 *>(weight_bf16);
    a.y = static_cast<__nv_bfloat16 *>(y_bf16);
    a.q = static_cast<uint8_t *>(y_fp8);
    a.sf = static_cast<uint8_t *>(y_sf);
    a.rstd_out = rstd;
    a.T = T;
    a.H = H;
    a.eps = eps;
    return run_norm<false, 1>(a, reinterpret_cast<cudaStream_t>(stream));
}

moe_status_t moe_norm_after(const void *x_bf16, const void *residual_bf16, const void *weight_bf16,
                            const void *gate_bf16, int gate_kind, int T, int H, float eps, float residual_scale,
                            void *out_bf16, float *rstd, moe_stream_t stream) {
    const moe_status_t s = check_norm(T, H, eps);
    if (s != MOE_OK) return s;
    if (bad_gate(gate_kind) || !(residual_scale >= -3.4e38f && residual_scale <= 3.4e38f)) return MOE_ERR_INVALID_ARG;
    if (T == 0) return MOE_OK;
    if (!x_bf16 || !residual_bf16 || !weight_bf16 || !out_bf16 || (gate_kind != MOE_GATE_NONE && !gate_bf16) ||
        !aligned(x_bf16, 16) || !aligned(residual_bf16, 16) || !aligned(weight_bf16, 16) || !aligned(out_bf16, 16) ||
        !aligned(gate_bf16, gate_kind == MOE_GATE_TOKEN ? 2 : 16) || !aligned(rstd, 4))
        return MOE_ERR_INVALID_ARG;
    DeviceScope dev(x_bf16);
    if (dev.status != MOE_OK) return dev.status;
    NormArgs a{};
    a.x = static_cast<const __nv_bfloat16 *>(x_bf16);
    a.residual = static_cast<const __nv_bfloat16 *>(residual_bf16);
    a.weight = static_cast<const __nv_bfloat16 *>(weight_bf16);
    a.gate = static_cast<const __nv_bfloat16 *>(gate_bf16);
    a.gate_kind = gate_kind;
    a.y = static_cast<__nv_bfloat16 *>(out_bf16);
    a.rstd_out = rstd;
    a.T = T;
    a.H = H;
    a.eps = eps;
    a.alpha = residual_scale;
    return gate_kind == MOE_GATE_FULL ? run_norm<true, 3>(a, reinterpret_cast<cudaStream_t>(stream))
                                      : run_norm<true, 2>(a, reinterpret_cast<cudaStream_t>(stream));
}

moe_status_t moe_norm_workspace_bytes(int T_max, int H, size_t *bytes) {
    if (!bytes || T_max < 0 || H <= 0) return MOE_ERR_INVALID_ARG;
    if (H % 8 || H > kNormMaxH) return MOE_ERR_UNSUPPORTED_SHAPE;
    *bytes = size_t(kNormMaxBlocks) * 2 * size_t(H) * sizeof(float);
    return MOE_OK;
}

moe_status_t moe_norm_before_backward(const void *dy_bf16, const void *x_bf16, const void *weight_bf16,
                                      const float *rstd, const void *dresidual_bf16, int T, int H, void *dx_bf16,
                                      float *dweight, void *workspace, size_t ws_bytes, moe_stream_t stream) {
    moe_status_t s = check_norm(T, H, 1.0f);
    if (s != MOE_OK) return s;
    if (!dweight || !aligned(dweight, 4)) return MOE_ERR_INVALID_ARG;
    if (T > 0 && (!dy_bf16 || !x_bf16 || !weight_bf16 || !rstd || !dx_bf16 || !workspace || !aligned(dy_bf16, 16) ||
                  !aligned(x_bf16, 16) || !aligned(weight_bf16, 16) || !aligned(rstd, 4) ||
                  !aligned(dresidual_bf16, 16) || !aligned(dx_bf16, 16) || !aligned(workspace, 256)))
        return MOE_ERR_INVALID_ARG;
    size_t need = 0;
    moe_norm_workspace_bytes(T, H, &need);
    if (T > 0 && ws_bytes < need) return MOE_ERR_WORKSPACE_TOO_SMALL;
    DeviceScope dev(dweight);
    if (dev.status != MOE_OK) return dev.status;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (T == 0)
        return cudaMemsetAsync(dweight, 0, sizeof(float) * size_t(H), st) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
    NormArgs a{};
    a.dy = static_cast<const __nv_bfloat16 *>(dy_bf16);
    a.x = static_cast<const __nv_bfloat16 *>(x_bf16);
    a.weight = static_cast<const __nv_bfloat16 *>(weight_bf16);
    a.rstd = rstd;
    a.dres_in = static_cast<const __nv_bfloat16 *>(dresidual_bf16);
    a.T = T;
    a.H = H;
    a.dx = static_cast<__nv_bfloat16 *>(dx_bf16);
    a.part = static_cast<float *>(workspace);
    return a.dres_in ? run_norm_backward<false, 3>(a, dweight, nullptr, st)
                     : run_norm_backward<false, 2>(a, dweight, nullptr, st);
}

moe_status_t moe_norm_after_backward(const void *dout_bf16, const void *x_bf16, const void *weight_bf16,
                                     const float *rstd, const void *gate_bf16, int gate_kind, int T, int H,
                                     float residual_scale, void *dx_bf16, void *dresidual_bf16, float *dweight,
                                     void *dgate, void *workspace, size_t ws_bytes, moe_stream_t stream) {
    moe_status_t s = check_norm(T, H, 1.0f);
    if (s != MOE_OK) return s;
    if (bad_gate(gate_kind) || !(residual_scale >= -3.4e38f && residual_scale <= 3.4e38f) || !dweight ||
        !aligned(dweight, 4) || (gate_kind == MOE_GATE_CHANNEL && (!dgate || !aligned(dgate, 4))))
        return MOE_ERR_INVALID_ARG;
    if (T > 0 &&
        (!dout_bf16 || !x_bf16 || !weight_bf16 || !rstd || !dx_bf16 || !dresidual_bf16 || !workspace ||
         !aligned(dout_bf16, 16) || !aligned(x_bf16, 16) || !aligned(weight_bf16, 16) || !aligned(rstd, 4) ||
         !aligned(dx_bf16, 16) || !aligned(dresidual_bf16, 16) || !aligned(workspace, 256) ||
         (gate_kind != MOE_GATE_NONE && (!gate_bf16 || !dgate)) ||
         !aligned(gate_bf16, gate_kind == MOE_GATE_TOKEN ? 2 : 16) ||
         !aligned(dgate, gate_kind == MOE_GATE_FULL ? 16 : 4)))
        return MOE_ERR_INVALID_ARG;
    size_t need = 0;
    moe_norm_workspace_bytes(T, H, &need);
    if (T > 0 && ws_bytes < need) return MOE_ERR_WORKSPACE_TOO_SMALL;
    DeviceScope dev(dweight);
    if (dev.status != MOE_OK) return dev.status;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (T == 0) {
        cudaError_t e = cudaMemsetAsync(dweight, 0, sizeof(float) * size_t(H), st);
        if (e == cudaSuccess && gate_kind == MOE_GATE_CHANNEL) e = cudaMemsetAsync(dgate, 0, sizeof(float) * size_t(H), st);
        return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
    }
    NormArgs a{};
    a.dy = static_cast<const __nv_bfloat16 *>(dout_bf16);
    a.x = static_cast<const __nv_bfloat16 *>(x_bf16);
    a.weight = static_cast<const __nv_bfloat16 *>(weight_bf16);
    a.rstd = rstd;
    a.gate = static_cast<const __nv_bfloat16 *>(gate_bf16);
    a.gate_kind = gate_kind;
    a.T = T;
    a.H = H;
    a.alpha = residual_scale;
    a.dx = static_cast<__nv_bfloat16 *>(dx_bf16);
    a.dres = static_cast<__nv_bfloat16 *>(dresidual_bf16);
    a.dgate = gate_kind == MOE_GATE_CHANNEL ? nullptr : dgate;
    a.part = static_cast<float *>(workspace);
    if (gate_kind == MOE_GATE_FULL) return run_norm_backward<true, 3>(a, dweight, nullptr, st);
    return run_norm_backward<true, 2>(a, dweight, gate_kind == MOE_GATE_CHANNEL ? static_cast<float *>(dgate) : nullptr,
                                      st);
}

}  // extern "C"
