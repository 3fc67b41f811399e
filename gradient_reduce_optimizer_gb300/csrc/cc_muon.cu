// Muon: the orthogonalisation of matrices by Newton-Schulz products
// (cc_muon_orthogonalise) and the fused data-parallel Muon step
// (cc_fused_dp_muon), include/cc_dp.h.
//
//   X <- G / (|G|_F + eps), then `steps` times X <- a X + (b A + c A A) X with
//   A = X X^T (matrices taller than wide: from the right with A = X^T X)
// applies x -> a x + b x^3 + c x^5 to the singular values of X and keeps its
// singular vectors; Muon's coefficients drive every one of them towards 1.
//
// Arithmetic.  The products run on the tensor cores on fp16 operands with
// fp32 accumulation (cc_muon_gemm.cu).  What their roundings cost follows from the
// singular values' spread (tests/test_gpu_muon_spectra.py has the formula, and
// holds the kernels to 1.2 times it): 7e-4 of the result on a Gaussian matrix,
// 6e-3 where one direction is all of it.  Three things keep 11-bit operands
// accurate, each checked against 64 bits:
//  * the first step reads G itself, not normalised: 16-bit matrices in place,
//    fp32 ones (and the step's update) as bf16, which has their range, plus
//    their rounding's own bf16 as a low part.  1/(|G|_F + eps) multiplies the
//    accumulators.  bf16 operands cost little there: what the first products
//    add to a X is small next to it wherever singular values still have to
//    grow (a Gaussian matrix's error changes by less than 2%; where one direction
//    is all of the matrix, fp32's products of its bf16 part cost 5.7e-3, bf16's
//    and fp16's own 3.6e-3 and 5.3e-3);
//  * in all but the last two steps X carries a low part (the rounding of its
//    fp16 value, itself in 8 bits, e5m2: three more bits of each element, and
//    half the bytes of a second fp16) that joins the term a X.  There X's small
//    singular values are still growing by up to a a step next to large ones,
//    and a rounding of X relative to the large ones would grow with them.
//    On a matrix of rank 8 plus 5% noise the result's error falls from 1.5e-2
//    to 1.2e-3;
//  * in the last three steps, where the singular values of X approach 1, the
//    polynomial is expanded around A = t I (t = 1/4, 1/2, 3/4): a + b l + c l^2
//    = a' + b' (l - t) + c (l - t)^2.  The terms no longer cancel, so
//    rounding A and P costs less (1.5e-3 to 0.8e-3 on a Gaussian matrix).
// Matrices with a side of at most 64 take fp32 products (cc_muon_small.cu).
// Momentum, master weights, norms and sums are fp32.

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "cc_dp_device.cuh"
#include "cc_dp_internal.h"
#include "cc_muon_internal.h"
#include "cc_trace.h"

namespace ccdp {
namespace muon {
namespace {

constexpr int kThreads = 256;
constexpr unsigned kAll = 0xFFFFFFFFu;

__device__ __forceinline__ void pdl_launch() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

__device__ __forceinline__ float block_sum(float v) {
    __shared__ float buf[kThreads / 32];
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(kAll, v, d);
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x / 32] = v;
    __syncthreads();
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) s += buf[w];
    __syncthreads();
    return s;
}

__device__ __forceinline__ float load_as_float(const void *p, int dtype, size_t i) {
    if (dtype == CC_DTYPE_F32) return static_cast<const float *>(p)[i];
    if (dtype == CC_DTYPE_BF16) return __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i]);
    return __half2float(static_cast<const __half *>(p)[i]);
}

// Eight consecutive elements at a 16-byte boundary.
__device__ __forceinline__ void load8(const void *p, int dtype, size_t i, float (&f)[8]) {
    if (dtype == CC_DTYPE_F32) {
        const float4 a = *reinterpret_cast<const float4 *>(static_cast<const float *>(p) + i);
        const float4 b = *reinterpret_cast<const float4 *>(static_cast<const float *>(p) + i + 4);
        f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
        f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    } else {
        const uint4 q = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p) + i);
        if (dtype == CC_DTYPE_BF16) {
            dev::widen8(q, f);
        } else {
            const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 v = __half22float2(*reinterpret_cast<const __half2 *>(&w[e]));
                f[2 * e] = v.x;
                f[2 * e + 1] = v.y;
            }
        }
    }
}

struct Source {
    const void *p;
    int dtype;
    int rows, cols;
    size_t ld, stride;       // elements between rows, between matrices
    bool vec;                // rows of 16-byte vectors of 8 elements
};

// v as bf16 and the bf16 of what that leaves; a and b share a word.
__device__ __forceinline__ void split2(float a, float b, uint32_t &hi, uint32_t &lo) {
    hi = dev::pack_bf16x2(a, b);
    lo = dev::pack_bf16x2(a - dev::bf16_lo(hi), b - dev::bf16_hi(hi));
}

// Sums of squares (CTA q of a matrix: vectors q, q + parts, ...), and with x
// the matrices laid out for TMA (rows ld elements apart): 16-bit ones copied,
// fp32 ones as bf16 and low part.  HBM bytes bound it: 24 x 4096 x 1024 bf16 in 40
// us, 5.0 TB/s.  (A pass of its own, because the first product needs no norm:
// it only has to be known when that product's tiles leave.)
__global__ void __launch_bounds__(kThreads)
squares_kernel(const __grid_constant__ Source s, float *partial, unsigned *done, uint16_t *x,
               uint16_t *lo, size_t ld, size_t stride) {
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        done[blockIdx.y] = done[gridDim.y + blockIdx.y] = 0;
    }
    const size_t src = static_cast<size_t>(blockIdx.y) * s.stride;
    const size_t dst = static_cast<size_t>(blockIdx.y) * stride;
    const size_t per_row = (static_cast<size_t>(s.cols) + 7) / 8;
    const size_t total = per_row * s.rows;
    float sum = 0.0f;
#pragma unroll 2
    for (size_t i = static_cast<size_t>(blockIdx.x) * kThreads + threadIdx.x; i < total;
         i += static_cast<size_t>(gridDim.x) * kThreads) {
        const size_t r = i / per_row;
        const int c = static_cast<int>(i - r * per_row) * 8;
        const size_t at = src + r * s.ld + c;
        float f[8];
        if (s.vec) {
            load8(s.p, s.dtype, at, f);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                f[e] = c + e < s.cols ? load_as_float(s.p, s.dtype, at + e) : 0.0f;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) sum = __fmaf_rn(f[e], f[e], sum);
        if (x) {
            uint32_t h[4], l[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (s.dtype == CC_DTYPE_F16) {
                    const __half2 q = __floats2half2_rn(f[2 * e], f[2 * e + 1]);   // exact
                    h[e] = *reinterpret_cast<const uint32_t *>(&q);
                } else {
                    split2(f[2 * e], f[2 * e + 1], h[e], l[e]);
                }
            }
            const size_t to = dst + r * ld + c;
            *reinterpret_cast<uint4 *>(x + to) = make_uint4(h[0], h[1], h[2], h[3]);
            if (lo) *reinterpret_cast<uint4 *>(lo + to) = make_uint4(l[0], l[1], l[2], l[3]);
        }
    }
    sum = block_sum(sum);
    if (threadIdx.x == 0) partial[static_cast<size_t>(blockIdx.y) * kMaxParts + blockIdx.x] = sum;
}

struct MomentumArgs {
    const void *grads[CC_MAX_R];
    const float *acc[CC_MAX_R];          // all null without accumulation
    size_t offset[CC_MUON_MAX_MATRICES];
    float *momentum;
    float *u;                            // fp32 [matrix][span], or null and
    uint16_t *hi, *lo;                   // bf16 and its low part, rows ld apart
    float *partial;
    unsigned *done;                      // cleared for the iteration
    size_t elems, span;                  // of one matrix: its size, its place
    size_t ld;
    int cols;
    bool small_index;                    // elems below 2^32
    int R;
    float inv_scale, beta, one_minus_beta;
    int nesterov;
};

// Zeros from a row's end at `last` to the next 16-byte boundary.
__device__ __forceinline__ void pad_row(const MomentumArgs &p, size_t last) {
    for (int k = 1; k <= (8 - p.cols % 8) % 8; ++k) p.hi[last + k] = p.lo[last + k] = 0;
}

// g = sum of the replicas / grad_scale, momentum' = beta momentum + (1-beta) g,
// u = (1-beta) g + beta momentum' (Nesterov) or momentum'; and the sums of u^2.
// The replicas are summed in replica order, each operation one rounding.  u
// goes out as the iteration reads it.  2 R + 12 bytes an element and HBM's rate:
// 96 x 1024 x 1024 of R = 8 in 421 us, 6.7 TB/s.
// MOST: the replicas whose loads are on their way at once; fewer of them leave
// registers for more warps (us, sixteen and as many as there are: R = 8, 33 x 2332 x
// 1101 449 and 370, R = 2, 59 x 263 x 3223 229 and 137).
template <int MOST>
__global__ void __launch_bounds__(kThreads, MOST <= 4 ? 4 : MOST <= 8 ? 3 : 2)
momentum_kernel(const __grid_constant__ MomentumArgs p) {
    pdl_launch();
    __shared__ __align__(16) uint16_t staged[2][kThreads * 8];
    const int lane = threadIdx.x & 31;
    const int b = blockIdx.y;
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        p.done[b] = p.done[gridDim.y + b] = 0;
    }
    const size_t off = p.offset[b];
    const size_t place = static_cast<size_t>(b) * p.span;
    const size_t vecs = p.elems / 8;
    const bool accumulate = p.acc[0] != nullptr;
    float sum = 0.0f;
    auto finish = [&](float s, float m, float &m_new, float &v) {
        const float g = __fmul_rn(s, p.inv_scale);
        m_new = __fadd_rn(__fmul_rn(p.beta, m), __fmul_rn(p.one_minus_beta, g));
        v = p.nesterov ? __fadd_rn(__fmul_rn(p.one_minus_beta, g), __fmul_rn(p.beta, m_new)) : m_new;
        sum = __fmaf_rn(v, v, sum);
    };
    const bool ragged = !p.u && p.cols % 8 != 0;
    for (size_t i0 = static_cast<size_t>(blockIdx.x) * kThreads; i0 < vecs;
         i0 += static_cast<size_t>(gridDim.x) * kThreads) {
        const size_t i = i0 + threadIdx.x;
        if (i < vecs) {
            const size_t e = off + i * 8;
            uint4 q[MOST];
#pragma unroll
            for (int r = 0; r < MOST; ++r)
                if (r < p.R) q[r] = __ldcs(reinterpret_cast<const uint4 *>(
                                 static_cast<const uint16_t *>(p.grads[r]) + e));
            const float4 ma = *reinterpret_cast<const float4 *>(p.momentum + e);
            const float4 mb = *reinterpret_cast<const float4 *>(p.momentum + e + 4);
            float s[8];
#pragma unroll
            for (int r = 0; r < MOST; ++r)
                if (r < p.R) {
                    if (accumulate) {
                        const float4 aa = __ldcs(reinterpret_cast<const float4 *>(p.acc[r] + e));
                        const float4 ab = __ldcs(reinterpret_cast<const float4 *>(p.acc[r] + e + 4));
                        float t[8] = {aa.x, aa.y, aa.z, aa.w, ab.x, ab.y, ab.z, ab.w};
                        dev::add8_bf16(t, q[r]);
#pragma unroll
                        for (int k = 0; k < 8; ++k) s[k] = r == 0 ? t[k] : __fadd_rn(s[k], t[k]);
                    } else if (r == 0) {
                        dev::widen8(q[0], s);
                    } else {
                        dev::add8_bf16(s, q[r]);
                    }
                }
            const float m[8] = {ma.x, ma.y, ma.z, ma.w, mb.x, mb.y, mb.z, mb.w};
            float mn[8], v[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) finish(s[k], m[k], mn[k], v[k]);
            *reinterpret_cast<float4 *>(p.momentum + e) = make_float4(mn[0], mn[1], mn[2], mn[3]);
            *reinterpret_cast<float4 *>(p.momentum + e + 4) = make_float4(mn[4], mn[5], mn[6], mn[7]);
            if (p.u) {
                float *u = p.u + place + i * 8;
                *reinterpret_cast<float4 *>(u) = make_float4(v[0], v[1], v[2], v[3]);
                *reinterpret_cast<float4 *>(u + 4) = make_float4(v[4], v[5], v[6], v[7]);
            } else {
                uint32_t h[4], l[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) split2(v[2 * k], v[2 * k + 1], h[k], l[k]);
                size_t to = place + i * 8;
                if (p.ld != static_cast<size_t>(p.cols) && !ragged) {
                    const size_t row = p.small_index ? static_cast<uint32_t>(i * 8) /
                                                           static_cast<uint32_t>(p.cols)
                                                     : i * 8 / p.cols;
                    to += row * (p.ld - p.cols);
                }
                uint16_t *hi = ragged ? staged[0] + threadIdx.x * 8 : p.hi + to;
                uint16_t *lo = ragged ? staged[1] + threadIdx.x * 8 : p.lo + to;
                *reinterpret_cast<uint4 *>(hi) = make_uint4(h[0], h[1], h[2], h[3]);
                *reinterpret_cast<uint4 *>(lo) = make_uint4(l[0], l[1], l[2], l[3]);
            }
        }
        if (ragged) {
            // Rows of the iteration's matrices start on 128 bytes, the slab's do not: by
            // way of shared memory, so that a warp writes its 256 elements side by side.
            __syncwarp();
            const size_t i_warp = i - lane;
            const size_t first = i_warp * 8 + lane;
            const int n = i_warp < vecs ? static_cast<int>(min(vecs - i_warp, size_t{32})) * 8 : 0;
            size_t row = p.small_index ? static_cast<uint32_t>(first) / static_cast<uint32_t>(p.cols)
                                       : first / p.cols;
            int col = static_cast<int>(first - row * p.cols);
            for (int k = lane; k < n; k += 32) {
                const size_t to = place + row * p.ld + col;
                p.hi[to] = staged[0][(threadIdx.x - lane) * 8 + k];
                p.lo[to] = staged[1][(threadIdx.x - lane) * 8 + k];
                if (col + 1 == p.cols) pad_row(p, to);
                col += 32;                               // rows are longer than 64
                if (col >= p.cols) {
                    col -= p.cols;
                    ++row;
                }
            }
            __syncwarp();
        }
    }
    const size_t i = vecs * 8 + threadIdx.x;             // the last elems % 8
    if (blockIdx.x == 0 && i < p.elems) {
        float s = 0.0f;
        for (int r = 0; r < p.R; ++r) {
            float t = dev::bf16_at(p.grads[r], off + i);
            if (accumulate) t = __fadd_rn(p.acc[r][off + i], t);
            s = r == 0 ? t : __fadd_rn(s, t);
        }
        float mn, v;
        finish(s, p.momentum[off + i], mn, v);
        p.momentum[off + i] = mn;
        if (p.u) {
            p.u[place + i] = v;
        } else {
            uint32_t h, l;
            split2(v, 0.0f, h, l);
            const size_t row = i / p.cols, to = place + row * p.ld + (i - row * p.cols);
            p.hi[to] = static_cast<uint16_t>(h);
            p.lo[to] = static_cast<uint16_t>(l);
            if (i + 1 == p.elems) pad_row(p, to);
        }
    }
    sum = block_sum(sum);
    if (threadIdx.x == 0) p.partial[static_cast<size_t>(b) * kMaxParts + blockIdx.x] = sum;
}

// ---- host side -------------------------------------------------------------------

size_t up(size_t v, size_t to) { return (v + to - 1) / to * to; }

// Elements from one 16-bit row to the next: rows that start between 32-byte
// sectors cost a fifth of the products' time (a step of 12 x 3254 x 355: 53 us, of
// 352 columns 45), so they start on 128 bytes where they would.
size_t row_of(size_t cols) { return cols % 16 == 0 ? cols : up(cols, 64); }

// Where everything lies in a workspace for `count` matrices of rows x cols.
struct Plan {
    int count, rows, cols, small;
    bool tall;
    size_t ld, stride;           // of X
    size_t ld8;                  // of its 8-bit low part
    size_t lda, stride_a;        // of A and P
    size_t at_done, at_partial, at_x0, at_x1, at_lo, at_lo8, at_a, at_p, at_split, bytes;
    bool has_split;
    bool is_small;               // cc_muon_small.cu: u, the partial Gram matrices, Q
    size_t span;                 // of u
    size_t at_u, at_gram, at_q;
};

int make_plan(int count, int rows, int cols, Plan *p) {
    if (count < 0 || rows < 0 || cols < 0)
        return fail(CC_ERR_INVALID, "count=%d rows=%d cols=%d must be >= 0", count, rows, cols);
    constexpr int kMostSide = 1 << 20;
    if (rows > kMostSide || cols > kMostSide)
        return fail(CC_ERR_INVALID, "rows=%d cols=%d above %d", rows, cols, kMostSide);
    p->count = count;
    p->rows = rows;
    p->cols = cols;
    p->small = std::min(rows, cols);
    p->tall = rows > cols;
    p->ld = row_of(static_cast<size_t>(cols));
    p->stride = p->ld * rows;
    p->ld8 = up(static_cast<size_t>(cols), 64);
    p->lda = row_of(static_cast<size_t>(p->small));
    p->stride_a = p->lda * p->small;
    p->span = up(static_cast<size_t>(rows) * cols, 8);
    size_t at = 0;
    bool fits = true;                    // (one matrix's parts are below 2^43 bytes)
    auto take = [&](size_t bytes_each) {
        const size_t here = at;
        size_t all;
        fits = fits && !__builtin_mul_overflow(bytes_each, static_cast<size_t>(count), &all) &&
               all <= SIZE_MAX / 16;
        at += fits ? up(all, 256) : 0;
        return here;
    };
    auto too_large = [&] {
        return fail(CC_ERR_INVALID, "%d matrices of %d x %d are too large", count, rows, cols);
    };
    p->at_done = take(2 * sizeof(unsigned));
    p->at_partial = take(kMaxParts * sizeof(float));
    p->is_small = p->small <= kSmallSide;
    if (p->is_small) {
        const size_t square = static_cast<size_t>(kSmallSide) * kSmallSide * sizeof(float);
        p->at_u = take(4 * p->span);
        p->at_gram = take(square * small_parts(count, std::max(rows, cols)));
        p->at_q = take(square);
        p->bytes = at;
        return fits ? CC_OK : too_large();
    }
    p->at_x0 = take(2 * p->stride);
    p->at_x1 = take(2 * p->stride);
    p->at_lo = take(2 * p->stride);
    p->at_lo8 = take(p->ld8 * rows);
    p->at_a = take(2 * p->stride_a);
    p->at_p = take(2 * p->stride_a);
    p->has_split = (count == 1 && p->small > kSplitSide) ||
                   (count <= kMostPieces && p->small <= kSplitSide &&
                    std::max(rows, cols) >= kSplitLong);
    p->at_split = at;
    if (p->has_split) at += kMostPieces * kPieceBytes;
    p->bytes = at;
    return fits ? CC_OK : too_large();
}

// CTAs a matrix for the elementwise passes: two vectors of 8 elements a
// thread at least, four waves of the GPU over all matrices at most.
int parts_of(size_t elems, int count) {
    const size_t most = std::max<size_t>(1, 8 * 608 / static_cast<size_t>(count));
    const size_t per = static_cast<size_t>(kThreads) * 8 * 2;
    return static_cast<int>(std::min<size_t>({std::max<size_t>((elems + per - 1) / per, 1), most,
                                              static_cast<size_t>(kMaxParts)}));
}

// Columns up to the next 16-byte boundary.
int padded(int cols) { return static_cast<int>(up(static_cast<size_t>(cols), 8)); }

// The iteration over matrices `g` with their sums of squares in place.
Iteration iteration(const Plan &pl, const Batch &g, void *g_lo, bool bf16, int parts,
                    unsigned char *ws, const float *coeffs, int steps, float eps) {
    // Rows up to the next 16-byte boundary: zeros there stay zeros, and boxes are
    // cut off at whole 16 bytes.
    const Batch x{ws + pl.at_x0, pl.count, pl.rows, padded(pl.cols), pl.ld, pl.stride};
    const Batch a{ws + pl.at_a, pl.count, pl.small, padded(pl.small), pl.lda, pl.stride_a};
    Iteration it{};
    it.rows = pl.rows;
    it.cols = pl.cols;
    it.g = g;
    it.g_lo = x;
    it.g_lo.p = g_lo;
    it.bf16 = bf16;
    it.x[0] = it.x[1] = x;
    it.x[1].p = ws + pl.at_x1;
    it.lo = Batch{ws + pl.at_lo8, pl.count, pl.rows, static_cast<int>(pl.ld8), pl.ld8,
                  pl.ld8 * pl.rows};
    it.a = it.p = a;
    it.p.p = ws + pl.at_p;
    it.partial = reinterpret_cast<const float *>(ws + pl.at_partial);
    it.parts = parts;
    it.eps = eps;
    it.coeffs = coeffs;
    it.steps = steps;
    it.done = reinterpret_cast<unsigned *>(ws + pl.at_done);
    it.split = pl.has_split ? reinterpret_cast<float *>(ws + pl.at_split) : nullptr;
    return it;
}

int check_iteration(const float *coeffs, int steps, float eps) {
    if (steps < 1 || steps > CC_MUON_MAX_STEPS)
        return fail(CC_ERR_INVALID, "steps=%d must be in 1..%d", steps, CC_MUON_MAX_STEPS);
    if (!coeffs) return fail(CC_ERR_INVALID, "coeffs is NULL");
    for (int i = 0; i < 3 * steps; ++i)
        if (!(std::fabs(coeffs[i]) <= 100.0f))
            return fail(CC_ERR_INVALID, "coeffs[%d]=%g must be within [-100, 100]", i, coeffs[i]);
    if (!std::isfinite(eps) || eps < 0.0f)
        return fail(CC_ERR_INVALID, "eps=%g must be finite and >= 0", eps);
    return CC_OK;
}

struct Range {
    uintptr_t lo, hi;
    bool written;
    const char *name;
    int index;
    bool host_ok;
};

// Checked ranges of one call, at most kMost.
struct Ranges {
    static constexpr int kMost = 3 * CC_MAX_R + 4;
    Range r[kMost];
    int count = 0;
    int add(const void *p, size_t bytes, size_t align, bool written, const char *name, int index,
            bool host_ok = false) {
        if (!p) return fail(CC_ERR_INVALID, "%s[%d] is NULL", name, index);
        const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
        if (lo % align != 0)
            return fail(CC_ERR_MISALIGNED, "%s[%d]=%p is not %zu-byte aligned", name, index, p,
                        align);
        r[count++] = {lo, lo + bytes, written, name, index, host_ok};
        return CC_OK;
    }
    int check() const {
        for (int i = 0; i < count; ++i)
            for (int j = i + 1; j < count; ++j)
                if ((r[i].written || r[j].written) && r[i].lo < r[j].hi && r[j].lo < r[i].hi)
                    return fail(CC_ERR_ALIAS, "%s[%d] overlaps %s[%d]", r[i].name, r[i].index,
                                r[j].name, r[j].index);
        int st = ensure_device();
        for (int i = 0; st == CC_OK && i < count; ++i)
            st = check_slab_range(reinterpret_cast<const void *>(r[i].lo), r[i].hi - r[i].lo,
                                  r[i].name, r[i].host_ok);
        return st;
    }
};

int check_workspace(Ranges *rg, const Plan &pl, void *workspace, size_t workspace_bytes) {
    if (workspace_bytes < pl.bytes)
        return fail(CC_ERR_INVALID, "workspace of %zu bytes, %d matrices of %d x %d need %zu",
                    workspace_bytes, pl.count, pl.rows, pl.cols, pl.bytes);
    return rg->add(workspace, pl.bytes, 256, true, "workspace", 0);
}

}  // namespace
}  // namespace muon
}  // namespace ccdp

using namespace ccdp;
using namespace ccdp::muon;

extern "C" {

int cc_muon_workspace(int count, int rows, int cols, size_t *bytes) {
    if (!bytes) return fail(CC_ERR_INVALID, "bytes is NULL");
    *bytes = 0;
    Plan pl{};
    const int st = make_plan(count, rows, cols, &pl);
    if (st != CC_OK) return st;
    if (count > 0 && rows > 0 && cols > 0) *bytes = pl.bytes;
    return CC_OK;
}

int cc_muon_orthogonalise(const void *g, size_t ldg, size_t strideg, void *out, size_t ldo,
                          size_t strideo, int count, int rows, int cols, int g_dtype,
                          const float *coeffs, int steps, float eps, void *workspace,
                          size_t workspace_bytes, void *stream) {
    TraceRange call("cc_muon_orthogonalise", static_cast<uint64_t>(count));
    Plan pl{};
    int st = make_plan(count, rows, cols, &pl);
    if (st != CC_OK) return st;
    if (count > 65535) return fail(CC_ERR_INVALID, "count=%d above 65535", count);
    if (g_dtype != CC_DTYPE_BF16 && g_dtype != CC_DTYPE_F16 && g_dtype != CC_DTYPE_F32)
        return fail(CC_ERR_INVALID, "g_dtype=%d unknown", g_dtype);
    if ((st = check_iteration(coeffs, steps, eps)) != CC_OK) return st;
    if (count == 0 || rows == 0 || cols == 0) return CC_OK;
    const size_t elem = g_dtype == CC_DTYPE_F32 ? 4 : 2;
    const size_t limit = SIZE_MAX / 16 / (static_cast<size_t>(rows) * count);
    for (const size_t ld : {ldg, ldo})
        if (ld < static_cast<size_t>(cols) || ld > limit)
            return fail(CC_ERR_INVALID, "row stride %zu for cols=%d", ld, cols);
    const size_t one_g = (static_cast<size_t>(rows) - 1) * ldg + cols;
    const size_t one_o = (static_cast<size_t>(rows) - 1) * ldo + cols;
    if (count > 1 && (strideg < one_g || strideo < one_o || strideg > SIZE_MAX / 16 / count ||
                      strideo > SIZE_MAX / 16 / count))
        return fail(CC_ERR_INVALID, "matrix strides %zu, %zu below a matrix's extent", strideg,
                    strideo);
    Ranges rg;
    if ((st = rg.add(g, ((count - 1) * strideg + one_g) * elem, elem, false, "g", 0)) != CC_OK)
        return st;
    if ((st = rg.add(out, ((count - 1) * strideo + one_o) * 2, 2, true, "out", 0)) != CC_OK)
        return st;
    if ((st = check_workspace(&rg, pl, workspace, workspace_bytes)) != CC_OK) return st;
    if ((st = rg.check()) != CC_OK) return st;

    const cudaStream_t cs = static_cast<cudaStream_t>(stream);
    unsigned char *ws = static_cast<unsigned char *>(workspace);
    const PlainOut po{static_cast<__nv_bfloat16 *>(out), ldo, strideo};
    if (pl.is_small)
        return small_out({g, g_dtype, pl.small, std::max(rows, cols), pl.tall, ldg, strideg}, count,
                         coeffs, steps, eps, reinterpret_cast<float *>(ws + pl.at_gram),
                         reinterpret_cast<float *>(ws + pl.at_q), po, false, cs);
    const size_t step = count > 1 ? strideg : 0;
    const bool aligned = reinterpret_cast<uintptr_t>(g) % 16 == 0 && ldg * elem % 16 == 0 &&
                         step * elem % 16 == 0;
    const Source s{g, g_dtype, rows, cols, ldg, strideg, aligned && cols % 8 == 0};
    // 16-bit matrices that TMA can walk are read in place
    const bool in_place = elem == 2 && aligned;
    const bool split = g_dtype == CC_DTYPE_F32;
    uint16_t *x0 = in_place ? nullptr : reinterpret_cast<uint16_t *>(ws + pl.at_x0);
    uint16_t *lo = split ? reinterpret_cast<uint16_t *>(ws + pl.at_lo) : nullptr;
    const int parts = parts_of(static_cast<size_t>(rows) * cols, count);
    squares_kernel<<<dim3(parts, count), kThreads, 0, cs>>>(
        s, reinterpret_cast<float *>(ws + pl.at_partial),
        reinterpret_cast<unsigned *>(ws + pl.at_done), x0, lo, pl.ld, pl.stride);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return fail_cuda(e, "sum of squares launch");
    const Batch gb = in_place ? Batch{g, count, rows, cols, ldg, count > 1 ? strideg : rows * ldg}
                              : Batch{x0, count, rows, padded(cols), pl.ld, pl.stride};
    return iterate_out(iteration(pl, gb, lo, g_dtype != CC_DTYPE_F16, parts, ws, coeffs, steps, eps),
                       po, cs);
}

int cc_fused_dp_muon(const void *const *grads, const float *const *acc, float *master,
                     float *momentum, void *const *params_out, size_t n, int R,
                     const size_t *offsets, int count, int rows, int cols, float lr, float beta,
                     int nesterov, float weight_decay, float update_scale, const float *coeffs,
                     int steps, float eps, float grad_scale, void *workspace,
                     size_t workspace_bytes, void *stream) {
    TraceRange call("cc_fused_dp_muon", static_cast<uint64_t>(count));
    if (R < 1 || R > CC_MAX_R) return fail(CC_ERR_INVALID, "R=%d must be in 1..%d", R, CC_MAX_R);
    Plan pl{};
    int st = make_plan(count, rows, cols, &pl);
    if (st != CC_OK) return st;
    if (count > CC_MUON_MAX_MATRICES)
        return fail(CC_ERR_INVALID, "count=%d above %d", count, CC_MUON_MAX_MATRICES);
    if (!std::isfinite(lr) || lr < 0.0f) return fail(CC_ERR_INVALID, "lr=%g must be finite and >= 0", lr);
    if (!std::isfinite(beta) || beta < 0.0f || beta >= 1.0f)
        return fail(CC_ERR_INVALID, "beta=%g must be in [0, 1)", beta);
    if (!std::isfinite(weight_decay) || weight_decay < 0.0f)
        return fail(CC_ERR_INVALID, "weight_decay=%g must be finite and >= 0", weight_decay);
    if (!std::isfinite(update_scale) || update_scale < 0.0f)
        return fail(CC_ERR_INVALID, "update_scale=%g must be finite and >= 0", update_scale);
    if (!std::isfinite(grad_scale) || grad_scale <= 0.0f || !std::isfinite(1.0f / grad_scale))
        return fail(CC_ERR_INVALID, "grad_scale=%g must be finite and > 0", grad_scale);
    if ((st = check_iteration(coeffs, steps, eps)) != CC_OK) return st;
    if (count == 0 || rows == 0 || cols == 0) return CC_OK;
    if (!grads || !params_out || !offsets)
        return fail(CC_ERR_INVALID, "grads/params_out/offsets arrays are NULL");
    if (n > SIZE_MAX / 8) return fail(CC_ERR_INVALID, "n=%zu too large", n);

    const size_t elems = static_cast<size_t>(rows) * cols;
    MomentumArgs m{};
    StepOut so{};
    bool sorted = true;
    for (int i = 0; i < count; ++i) {
        if (offsets[i] % CC_PAD_ELEMS != 0)
            return fail(CC_ERR_MISALIGNED, "offsets[%d]=%zu is not a multiple of %d", i,
                        offsets[i], CC_PAD_ELEMS);
        if (offsets[i] > n || elems > n - offsets[i])
            return fail(CC_ERR_INVALID, "matrix %d: [%zu, %zu + %zu) not inside [0, %zu)", i,
                        offsets[i], offsets[i], elems, n);
        if (i > 0 && offsets[i] < offsets[i - 1] + elems) sorted = false;
        m.offset[i] = so.offset[i] = offsets[i];
    }
    if (!sorted)
        for (int i = 0; i < count; ++i)
            for (int j = i + 1; j < count; ++j)
                if (offsets[i] < offsets[j] + elems && offsets[j] < offsets[i] + elems)
                    return fail(CC_ERR_ALIAS, "matrices %d and %d overlap", i, j);
    Ranges rg;
    for (int r = 0; r < R; ++r) {
        m.grads[r] = grads[r];
        m.acc[r] = acc ? acc[r] : nullptr;
        so.out[r] = params_out[r];
        if ((st = rg.add(grads[r], 2 * n, 16, false, "grads", r, true)) != CC_OK) return st;
        if ((st = rg.add(params_out[r], 2 * n, 16, true, "params_out", r, true)) != CC_OK) return st;
        if (acc && (st = rg.add(acc[r], 4 * n, 16, false, "acc", r)) != CC_OK) return st;
    }
    if ((st = rg.add(master, 4 * n, 16, true, "master", 0)) != CC_OK) return st;
    if ((st = rg.add(momentum, 4 * n, 16, true, "momentum", 0)) != CC_OK) return st;
    if ((st = check_workspace(&rg, pl, workspace, workspace_bytes)) != CC_OK) return st;
    if ((st = rg.check()) != CC_OK) return st;

    const cudaStream_t cs = static_cast<cudaStream_t>(stream);
    unsigned char *ws = static_cast<unsigned char *>(workspace);
    const int parts = parts_of(elems, count);
    m.momentum = momentum;
    if (pl.is_small) {
        m.u = reinterpret_cast<float *>(ws + pl.at_u);
        m.span = pl.span;
    } else {
        m.hi = reinterpret_cast<uint16_t *>(ws + pl.at_x0);
        m.lo = reinterpret_cast<uint16_t *>(ws + pl.at_lo);
        m.span = pl.stride;
    }
    m.partial = reinterpret_cast<float *>(ws + pl.at_partial);
    m.done = reinterpret_cast<unsigned *>(ws + pl.at_done);
    m.elems = elems;
    m.ld = pl.ld;
    m.cols = cols;
    m.small_index = elems <= UINT32_MAX;
    m.R = R;
    m.inv_scale = 1.0f / grad_scale;
    m.beta = beta;
    m.one_minus_beta = 1.0f - beta;
    m.nesterov = nesterov != 0;
    if (R <= 4) momentum_kernel<4><<<dim3(parts, count), kThreads, 0, cs>>>(m);
    else if (R <= 8) momentum_kernel<8><<<dim3(parts, count), kThreads, 0, cs>>>(m);
    else momentum_kernel<CC_MAX_R><<<dim3(parts, count), kThreads, 0, cs>>>(m);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return fail_cuda(e, "momentum launch");
    so.master = master;
    so.R = R;
    so.decay = 1.0f - lr * weight_decay;
    so.lr_scale = lr * update_scale;
    if (pl.is_small)
        return small_step({m.u, CC_DTYPE_F32, pl.small, std::max(rows, cols), pl.tall,
                           static_cast<size_t>(cols), pl.span},
                          count, coeffs, steps, eps, reinterpret_cast<float *>(ws + pl.at_gram),
                          reinterpret_cast<float *>(ws + pl.at_q), so, true, cs);
    return iterate_step(iteration(pl, {m.hi, count, rows, padded(cols), pl.ld, pl.stride}, m.lo, true,
                                  parts, ws, coeffs, steps, eps),
                        so, cs);
}

}  // extern "C"
