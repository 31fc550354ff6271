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
// All four are bound by HBM.  A row's columns are fixed to the threads that take
// it (8 at a time, 16-byte accesses), so the weights' gradients stay in
// registers over the rows.  A thread brings its own pieces of the rows ahead
// into its own part of a shared-memory ring (cp.async), so rows are in flight
// and no barrier is needed to read them.  The arithmetic is on pairs of columns
// (fp32x2 instructions; with rows of a block in groups and scale bytes straight from
// the bits they took the quantised norm of 8192 x 7168 from 71.7 to 53.3 us, later
// steps to 44).  Sums are fp32; the column sums of the blocks are written out and added
// in block order by a second kernel, so results do not depend on timing.
#include "moe_common.cuh"
#include "moe_internal.h"

namespace moe {
namespace {

constexpr int kNormMaxH = 16384;
constexpr int kNormMaxBlocks = 512;  // column sums a workspace holds: the gradients' blocks, at most

// Pairs of fp32 values.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 r;
    asm("{\n\t.reg .b64 a, b, r;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "mul.rn.f32x2 r, a, b;\n\tmov.b64 {%0, %1}, r;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 r;
    asm("{\n\t.reg .b64 a, b, c, r;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
        "fma.rn.f32x2 r, a, b, c;\n\tmov.b64 {%0, %1}, r;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return r;
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// Eight bf16 values as four pairs.
struct Bf16x8 {
    uint32_t u[4];
    __device__ __forceinline__ float2 pair(int i) const {
        return make_float2(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xFFFF0000u));
    }
    __device__ __forceinline__ void set(int i, float2 v) {
        const __nv_bfloat162 p = __floats2bfloat162_rn(v.x, v.y);
        u[i] = *reinterpret_cast<const uint32_t *>(&p);
    }
};
__device__ __forceinline__ Bf16x8 as_bf16x8(uint4 v) { return {{v.x, v.y, v.z, v.w}}; }
__device__ __forceinline__ Bf16x8 load8(const __nv_bfloat16 *p) {
    return as_bf16x8(__ldg(reinterpret_cast<const uint4 *>(p)));
}
__device__ __forceinline__ void store8(__nv_bfloat16 *p, const Bf16x8 &v) {
    *reinterpret_cast<uint4 *>(p) = make_uint4(v.u[0], v.u[1], v.u[2], v.u[3]);
}

// Eight rounded columns to E4M3 with their group's UE8M0 scale; a group of 32
// columns is four neighbouring lanes.  The rule and the codes of
// moe_quantize_fp8 (the scale byte straight from the bits: the exponent field of
// amax plus one where its fraction is above 0.75, less 8, at least 0; zero has
// 127).
struct Quantised {
    uint32_t code[2], sf;
};
__device__ __forceinline__ Quantised quantise8(const Bf16x8 &y) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t a = y.u[i] & 0x7FFF7FFFu;
        const __nv_bfloat162 r =
            __hmax2(*reinterpret_cast<const __nv_bfloat162 *>(&m), *reinterpret_cast<const __nv_bfloat162 *>(&a));
        m = *reinterpret_cast<const uint32_t *>(&r);
    }
    float amax = fmaxf(__uint_as_float(m << 16), __uint_as_float(m & 0xFFFF0000u));
    amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
    const uint32_t bits = __float_as_uint(amax);
    const int field = max(int((bits + 0x1FFFFFu) >> 23) - 8, 0);
    Quantised q;
    q.sf = bits == 0u ? 127u : uint32_t(field);
    const float2 inv = both(__uint_as_float((254u - q.sf) << 23));
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float2 a = mul2(y.pair(2 * i), inv), b = mul2(y.pair(2 * i + 1), inv);
        const uint32_t lo = __nv_cvt_float2_to_fp8x2(a, __NV_SATFINITE, __NV_E4M3);
        const uint32_t hi = __nv_cvt_float2_to_fp8x2(b, __NV_SATFINITE, __NV_E4M3);
        // (the sign bits, for NaN: every other code has its value's already)
        q.code[i] = (lo | hi << 16) | (__byte_perm(y.u[2 * i], y.u[2 * i + 1], 0x7531u) & 0x80808080u);
    }
    return q;
}

// The sums of kCount values over the `warps` warps that take a row, in all of
// their threads; `warp` is this one's number among them.  The warps' sums meet in
// `red` (zero beyond `warps`) and every thread adds them in the same order.  The
// caller alternates two sets of `red`, so one barrier a call is enough: number
// `bar`, for one row group of several in a block.
template <int kCount>
__device__ __forceinline__ void row_sum(float (&v)[kCount], float (*red)[32], int warp, int warps, int bar) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
#pragma unroll
        for (int c = 0; c < kCount; ++c) v[c] += __shfl_xor_sync(0xFFFFFFFFu, v[c], d);
    if (warps == 1) return;
    if ((threadIdx.x & 31) == 0)
#pragma unroll
        for (int c = 0; c < kCount; ++c) red[c][warp] = v[c];
    asm volatile("bar.sync %0, %1;" ::"r"(bar), "r"(warps * 32) : "memory");
    // (each thread adding all of them up from memory: 49.0 us instead of 46.3 for 8192
    // x 7168 to FP8, where instructions count)
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int c = 0; c < kCount; ++c) {
        float t = red[c][warps > 16 ? lane : lane & 15];
        if (warps > 16) t += __shfl_xor_sync(0xFFFFFFFFu, t, 16);
#pragma unroll
        for (int d = 8; d > 0; d >>= 1) t += __shfl_xor_sync(0xFFFFFFFFu, t, d);
        v[c] = t;
    }
}
__device__ __forceinline__ void clear(float *red, int count) {
    for (int i = threadIdx.x; i < count; i += blockDim.x) red[i] = 0.0f;
    __syncthreads();
}

struct NormArgs {
    const __nv_bfloat16 *x, *weight, *residual, *gate;
    __nv_bfloat16 *y;      // before: y (or null); after: out
    uint8_t *q, *sf;       // before: codes and scales (or null)
    float *rstd_out;       // [T] or null
    int T, H;
    int groups, row_threads;  // gradients: rows a block takes at a time, threads of each
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

// Rows of the forward kernels' rings: one being worked on, the others on their
// way (a block is one of several on its SM).
constexpr int norm_depth(int streams) { return streams == 1 ? 3 : 2; }
// The gradients work on two rows at a time up to this width, with as many on
// their way, and on one with one on its way above.
constexpr int kNormTwoRowsH = 8192;

// The ring of one thread's pieces: kStreams inputs of a row, kDepth rows.
template <int kVecs, int kStreams, int kDepth>
struct RowRing {
    uint32_t mine;             // this thread's first piece (shared memory), and the bytes to its next
    uint32_t piece;
    const __nv_bfloat16 *src[kStreams];  // this thread's first columns of the next row to bring
    int64_t step;              // elements to the row after that
    int T, row, row_step, slot, first, apart, nvec;

    // `threads` take a row, this one from column 8 * first on
    template <int kAhead>
    __device__ __forceinline__ void start(uint4 *smem, int first_, int threads, int H, int T_, int row_, int row_step_) {
        mine = smem_u32(smem + threadIdx.x);
        piece = blockDim.x * 16u;
        first = first_;
        apart = threads;
        nvec = H / 8;
        T = T_;
        row = row_;
        row_step = row_step_;
        step = int64_t(row_step_) * H;
        slot = 0;
#pragma unroll
        for (int s = 0; s < kStreams; ++s) src[s] += int64_t(row_) * H + first_ * 8;
#pragma unroll
        for (int d = 0; d < kAhead; ++d) next();
    }
    __device__ __forceinline__ bool has(int i) const { return first + i * apart < nvec; }
    __device__ __forceinline__ void next() {
        if (row < T) {
#pragma unroll
            for (int s = 0; s < kStreams; ++s)
#pragma unroll
                for (int i = 0; i < kVecs; ++i)
                    if (has(i))
                        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                                         mine + ((slot * kStreams + s) * kVecs + i) * piece),
                                     "l"(src[s] + i * apart * 8)
                                     : "memory");
#pragma unroll
            for (int s = 0; s < kStreams; ++s) src[s] += step;
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        row += row_step;
        if (++slot == kDepth) slot = 0;
    }
    // All but the newest kLeft rows have landed (for this thread).
    template <int kLeft>
    __device__ __forceinline__ void wait() const {
        asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
    }
    __device__ __forceinline__ Bf16x8 get(int slot_, int stream, int i) const {
        Bf16x8 v;
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(v.u[0]), "=r"(v.u[1]), "=r"(v.u[2]), "=r"(v.u[3])
                     : "r"(mine + ((slot_ * kStreams + stream) * kVecs + i) * piece)
                     : "memory");
        return v;
    }
};

// Forward of both norms. kVecs: 8-column pieces of a row per thread, whose
// weights (and gate per channel) stay in registers. Streams: x; after: x,
// residual and, for a gate per element, that.
template <int kVecs, bool kAfter, int kStreams>
__global__ void __launch_bounds__(1024, 1) norm_kernel(const NormArgs a) {
    extern __shared__ uint4 ring_smem[];
    __shared__ __align__(16) float red[2][1][32];
    constexpr int kDepth = norm_depth(kStreams);
    const int tid = threadIdx.x;
    pdl_wait();
    pdl_trigger();
    RowRing<kVecs, kStreams, kDepth> ring;
    ring.src[0] = a.x;
    if constexpr (kStreams > 1) ring.src[1] = a.residual;
    if constexpr (kStreams > 2) ring.src[2] = a.gate;
    ring.template start<kDepth - 1>(ring_smem, tid, blockDim.x, a.H, a.T, blockIdx.x, gridDim.x);
    const int warp = tid >> 5, warps = blockDim.x >> 5;
    const float inv_h = 1.0f / float(a.H);
    Bf16x8 w[kVecs], gc[kAfter && kStreams == 2 ? kVecs : 1];
#pragma unroll
    for (int i = 0; i < kVecs; ++i)
        if (ring.has(i)) {
            w[i] = load8(a.weight + (tid + i * blockDim.x) * 8);
            if (kAfter && kStreams == 2 && a.gate_kind == MOE_GATE_CHANNEL) gc[i] = load8(a.gate + (tid + i * blockDim.x) * 8);
        }
    clear(&red[0][0][0], 2 * 32);
    // the token's gate, brought a row ahead
    const bool token = kAfter && a.gate_kind == MOE_GATE_TOKEN;
    __nv_bfloat16 next_gate = __float2bfloat16_rn(1.0f);
    if (token && blockIdx.x < a.T) next_gate = a.gate[blockIdx.x];
    int flip = 0, slot = 0;
    for (int row = blockIdx.x; row < a.T; row += gridDim.x, flip ^= 1) {
        const int64_t base = int64_t(row) * a.H + tid * 8;
        const float tgate = __bfloat162float(next_gate);
        if (token && row + int(gridDim.x) < a.T) next_gate = a.gate[row + gridDim.x];
        ring.next();
        ring.template wait<kDepth - 1>();
        float2 ss = both(0.0f);
        Bf16x8 x[kVecs];
#pragma unroll
        for (int i = 0; i < kVecs; ++i)
            if (ring.has(i)) {
                x[i] = ring.get(slot, 0, i);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 v = x[i].pair(j);
                    ss = fma2(v, v, ss);
                }
            }
        float sum[1] = {ss.x + ss.y};
        row_sum(sum, red[flip], warp, warps, 0);
        // within 2 ulp, far below the sums' own rounding (correctly rounded: 46.3 us instead of 43.9)
        const float rstd = rsqrtf(sum[0] * inv_h + a.eps);
        if (a.rstd_out && tid == 0) a.rstd_out[row] = rstd;
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            const bool in = ring.has(i);
            const int col = i * blockDim.x * 8;  // from this thread's first
            Bf16x8 y;
            if (in) {
                float2 v[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) v[j] = mul2(mul2(x[i].pair(j), both(rstd)), w[i].pair(j));
                if constexpr (kAfter) {
                    const Bf16x8 r = ring.get(slot, 1, i);
                    Bf16x8 g;
                    if constexpr (kStreams > 2)
                        g = ring.get(slot, 2, i);
                    else
                        g = gc[i];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        float2 gv = both(tgate);
                        if (kStreams > 2 || a.gate_kind == MOE_GATE_CHANNEL) gv = g.pair(j);
                        v[j] = fma2(gv, v[j], mul2(both(a.alpha), r.pair(j)));
                    }
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) y.set(j, v[j]);
                if (kAfter || a.y) store8(a.y + base + col, y);
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) y.u[j] = 0u;
            }
            if constexpr (!kAfter) {
                if (a.q) {
                    const Quantised q = quantise8(y);
                    if (in) {
                        *reinterpret_cast<uint2 *>(a.q + base + col) = make_uint2(q.code[0], q.code[1]);
                        if ((tid & 3) == 0) a.sf[(base + col) >> 5] = uint8_t(q.sf);
                    }
                }
            }
        }
        if (++slot == kDepth) slot = 0;
    }
}

// Gradients of both norms: dx, the residual branch, per-token and per-element
// gates; the column sums of the weight (and of a per-channel gate) per block.
// A block's threads are `groups` groups of `row_threads`, each with rows of its
// own, so that short rows leave few column sums too; a group works on kRows rows
// between two meetings of its threads.  kHold: the weights and a gate per channel
// stay in registers.  Streams: dy, x; then before: the residual branch's gradient
// if there is one, after: a gate per element.
template <int kVecs, bool kAfter, int kStreams, int kRows, bool kHold>
__global__ void __launch_bounds__(512, 1) norm_backward_kernel(const NormArgs a) {
    extern __shared__ uint4 ring_smem[];
    __shared__ __align__(16) float red[2][2][16][kRows][32];
    constexpr bool kChannelToo = kAfter && kStreams == 2;  // the gate may be per channel
    constexpr int kDepth = 2 * kRows;
    const bool channel = kChannelToo && a.gate_kind == MOE_GATE_CHANNEL;
    const bool token = kChannelToo && a.gate_kind == MOE_GATE_TOKEN;
    const int group = int(threadIdx.x) / a.row_threads, tid = int(threadIdx.x) - group * a.row_threads;
    const int first = int(blockIdx.x) * a.groups + group, step = int(gridDim.x) * a.groups;
    const int warp = tid >> 5, warps = a.row_threads >> 5;
    pdl_wait();
    pdl_trigger();
    RowRing<kVecs, kStreams, kDepth> ring;
    ring.src[0] = a.dy;
    ring.src[1] = a.x;
    if constexpr (kStreams > 2) ring.src[2] = kAfter ? a.gate : a.dres_in;
    ring.template start<kRows>(ring_smem, tid, a.row_threads, a.H, a.T, first, step);
    float2 dw[kVecs][4], dg[kChannelToo ? kVecs : 1][4];
    float2 wf[kHold ? kVecs : 1][4], gf[kHold && kChannelToo ? kVecs : 1][4];
    auto column = [&](int i) { return (tid + i * a.row_threads) * 8; };
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            dw[i][j] = both(0.0f);
            if (kChannelToo) dg[i][j] = both(0.0f);
        }
        if (kHold && ring.has(i)) {
            const Bf16x8 w = load8(a.weight + column(i));
            Bf16x8 g;
            if (channel) g = load8(a.gate + column(i));
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                wf[i][j] = w.pair(j);
                if (kChannelToo && channel) gf[i][j] = g.pair(j);
            }
        }
    }
    clear(&red[0][0][0][0][0], 2 * 2 * 16 * kRows * 32);
    const float inv_h = 1.0f / float(a.H);
    // the rows' scalars, brought as far ahead as their elements
    float next_rstd[kRows] = {};
    __nv_bfloat16 next_gate[kRows] = {};
    auto fetch = [&](int row0) {
#pragma unroll
        for (int r = 0; r < kRows; ++r)
            if (row0 + r * step < a.T) {
                next_rstd[r] = a.rstd[row0 + r * step];
                if (token) next_gate[r] = a.gate[row0 + r * step];
            }
    };
    fetch(first);
    int flip = 0, slot0 = 0;
    for (int row0 = first; row0 < a.T; row0 += kRows * step, flip ^= 1) {
        float rstd[kRows], tgate[kRows], dots[kRows] = {}, tsums[kRows] = {};
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            rstd[r] = next_rstd[r];
            tgate[r] = token ? __bfloat162float(next_gate[r]) : 1.0f;
            ring.next();
        }
        fetch(row0 + kRows * step);
        ring.template wait<kRows>();
        // weight and gate of piece i: from registers or memory
        auto weight_of = [&](int i, Bf16x8 &w) {
            if (!kHold) w = load8(a.weight + column(i));
        };
        auto gate_of = [&](int slot, int i, Bf16x8 &g) {
            if constexpr (kAfter && kStreams > 2)
                g = ring.get(slot, 2, i);
            else if (!kHold && channel)
                g = load8(a.gate + column(i));
        };
        // dz of pair j, the gradient that reaches xhat w
        auto dz_of = [&](float2 d, int r, int i, int j, const Bf16x8 &g) {
            if constexpr (!kAfter) return d;
            if constexpr (kStreams > 2) return mul2(d, g.pair(j));
            return mul2(d, channel ? (kHold ? gf[kChannelToo ? i : 0][j] : g.pair(j)) : both(tgate[r]));
        };
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            const int row = row0 + r * step;
            if (row >= a.T) continue;
            const int slot = slot0 + r;
            float2 dot = both(0.0f), tsum = both(0.0f);
#pragma unroll
            for (int i = 0; i < kVecs; ++i) {
                if (!ring.has(i)) continue;
                const Bf16x8 dy = ring.get(slot, 0, i), x = ring.get(slot, 1, i);
                Bf16x8 w, g, de;
                weight_of(i, w);
                gate_of(slot, i, g);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 d = dy.pair(j), w2 = kHold ? wf[i][j] : w.pair(j), xh = mul2(x.pair(j), both(rstd[r]));
                    const float2 dz = dz_of(d, r, i, j, g);
                    if constexpr (kAfter) {
                        const float2 z = mul2(xh, w2);
                        if constexpr (kStreams > 2) {
                            de.set(j, mul2(d, z));
                        } else {
                            if (channel) dg[i][j] = fma2(d, z, dg[i][j]);
                            if (token) tsum = fma2(d, z, tsum);
                        }
                    }
                    dw[i][j] = fma2(dz, xh, dw[i][j]);
                    dot = fma2(mul2(dz, w2), xh, dot);
                }
                if constexpr (kAfter && kStreams > 2)
                    store8(static_cast<__nv_bfloat16 *>(a.dgate) + int64_t(row) * a.H + column(i), de);
            }
            dots[r] = dot.x + dot.y;
            tsums[r] = tsum.x + tsum.y;
        }
        row_sum(dots, red[flip][0][group], warp, warps, 1 + group);
        if (token) {
            row_sum(tsums, red[flip][1][group], warp, warps, 1 + group);
#pragma unroll
            for (int r = 0; r < kRows; ++r)
                if (tid == 0 && row0 + r * step < a.T) static_cast<float *>(a.dgate)[row0 + r * step] = tsums[r];
        }
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            const int row = row0 + r * step;
            if (row >= a.T) continue;
            const int slot = slot0 + r;
            const float2 mean = both(-dots[r] * inv_h);
#pragma unroll
            for (int i = 0; i < kVecs; ++i) {
                if (!ring.has(i)) continue;
                const int64_t at = int64_t(row) * a.H + column(i);
                const Bf16x8 dy = ring.get(slot, 0, i), x = ring.get(slot, 1, i);
                Bf16x8 w, g, add, out, res;
                weight_of(i, w);
                gate_of(slot, i, g);
                if constexpr (!kAfter && kStreams > 2) add = ring.get(slot, 2, i);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 d = dy.pair(j), xh = mul2(x.pair(j), both(rstd[r]));
                    const float2 dzw = mul2(dz_of(d, r, i, j, g), kHold ? wf[i][j] : w.pair(j));
                    float2 v = mul2(both(rstd[r]), fma2(xh, mean, dzw));
                    if constexpr (!kAfter && kStreams > 2) v = fma2(both(1.0f), add.pair(j), v);
                    out.set(j, v);
                    if (kAfter) res.set(j, mul2(both(a.alpha), d));
                }
                store8(a.dx + at, out);
                if (kAfter) store8(a.dres + at, res);
            }
        }
        slot0 = slot0 ? 0 : kRows;
    }
    // the groups' column sums, added in group order through the ring's memory
    asm volatile("cp.async.wait_all;" ::: "memory");
    float *sums = reinterpret_cast<float *>(ring_smem);  // [group][1 or 2][H]
    const int cols = (channel ? 2 : 1) * a.H;
    float *p = a.part + int64_t(blockIdx.x) * cols;
    __syncthreads();
    float *to = a.groups > 1 ? sums + group * cols : p;
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
        if (!ring.has(i)) continue;
        const int c = column(i);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            *reinterpret_cast<float2 *>(to + c + 2 * j) = dw[i][j];
            if (kChannelToo && channel) *reinterpret_cast<float2 *>(to + a.H + c + 2 * j) = dg[i][j];
        }
    }
    if (a.groups > 1) {
        __syncthreads();
        for (int c = threadIdx.x; c < cols; c += blockDim.x) {
            float v = 0.0f;
            for (int g = 0; g < a.groups; ++g) v += sums[g * cols + c];
            p[c] = v;
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

// Threads of a row of H columns, `vecs` 8-column pieces each.
int row_threads(int H, int vecs) { return ((H / 8 + vecs - 1) / vecs + 31) / 32 * 32; }
constexpr int kSmSmem = 228 * 1024;  // shared memory of an SM, 1 KB of it per resident block

moe_status_t check_norm(int T, int H, float eps) {
    if (T < 0 || H <= 0 || !(eps > 0.0f) || !(eps <= 3.4e38f)) return MOE_ERR_INVALID_ARG;
    if (H % 8 || H > kNormMaxH || T > kMaxRows) return MOE_ERR_UNSUPPORTED_SHAPE;
    return MOE_OK;
}

template <int kVecs, bool kAfter, int kStreams>
cudaError_t launch_norm(const NormArgs &a, cudaStream_t stream) {
    const int threads = row_threads(a.H, kVecs), bytes = threads * kVecs * 16 * kStreams * norm_depth(kStreams);
    const cudaError_t e = set_max_dynamic_smem(reinterpret_cast<const void *>(norm_kernel<kVecs, kAfter, kStreams>), bytes);
    if (e != cudaSuccess) return e;
    // as many blocks as fit at once (64 registers a thread), each with every gridDim-th row
    const int by_threads = 1024 / threads, by_smem = kSmSmem / (bytes + 2048);
    int per_sm = by_threads < by_smem ? by_threads : by_smem;
    if (per_sm < 1) per_sm = 1;
    const int cap = num_sms() * per_sm;
    return launch_pdl(norm_kernel<kVecs, kAfter, kStreams>, dim3(unsigned(a.T < cap ? a.T : cap)), dim3(unsigned(threads)),
                      size_t(bytes), stream, a);
}

template <bool kAfter, int kStreams>
moe_status_t run_norm(const NormArgs &a, cudaStream_t stream) {
    // a decode batch: one piece per thread, for latency; else two, which is also
    // what 1024 threads need for the widest rows
    const bool one = a.T <= num_sms() && a.H <= 8192;
    const cudaError_t e =
        one ? launch_norm<1, kAfter, kStreams>(a, stream) : launch_norm<2, kAfter, kStreams>(a, stream);
    return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

template <int kVecs, bool kAfter, int kStreams, int kRows, bool kHold>
cudaError_t launch_norm_backward(NormArgs a, float *dw, float *dg, cudaStream_t stream) {
    const auto kernel = norm_backward_kernel<kVecs, kAfter, kStreams, kRows, kHold>;
    const int cols = a.H * (kAfter && a.gate_kind == MOE_GATE_CHANNEL ? 2 : 1);
    a.row_threads = row_threads(a.H, kVecs);
    a.groups = 512 / a.row_threads;
    if (a.groups > 15) a.groups = 15;  // named barriers
    const int rows_per_block = (a.T + num_sms() - 1) / num_sms();
    if (a.groups > rows_per_block) a.groups = rows_per_block;
    int bytes = a.row_threads * a.groups * kVecs * 16 * kStreams * 2 * kRows;
    if (a.groups > 1 && bytes < a.groups * cols * 4) bytes = a.groups * cols * 4;
    cudaError_t e = set_max_dynamic_smem(reinterpret_cast<const void *>(kernel), bytes);
    if (e != cudaSuccess) return e;
    const int needed = (a.T + a.groups - 1) / a.groups;
    int grid = num_sms() < kNormMaxBlocks ? num_sms() : kNormMaxBlocks;
    if (grid > needed) grid = needed;
    e = launch_pdl(kernel, dim3(unsigned(grid)), dim3(unsigned(a.row_threads * a.groups)), size_t(bytes), stream, a);
    if (e != cudaSuccess) return e;
    return launch_pdl(column_sums_kernel, dim3(unsigned((cols + 31) / 32)), dim3(kColumnWarps * 32), 0, stream,
                      static_cast<const float *>(a.part), grid, cols, a.H, dw, dg);
}

template <bool kAfter, int kStreams>
moe_status_t run_norm_backward(const NormArgs &a, float *dw, float *dg, cudaStream_t stream) {
    const cudaError_t e = a.H <= kNormTwoRowsH ? launch_norm_backward<2, kAfter, kStreams, 2, true>(a, dw, dg, stream)
                                               : launch_norm_backward<4, kAfter, kStreams, 1, false>(a, dw, dg, stream);
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
