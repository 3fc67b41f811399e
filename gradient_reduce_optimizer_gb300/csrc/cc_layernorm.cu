// Layer norm, forward and backward, with the reduction of the weight's and
// bias's gradients over the rows (include/cc_dp.h, cc_layernorm_forward and
// cc_layernorm_backward).
//
// Forward, per row of `cols` elements:
//   s    = x + residual, rounded once to the activations' type (or s = x)
//   mean = sum(s) / cols,  rstd = 1 / sqrt(sum((s - mean)^2) / cols + eps)
//   y    = (s - mean) * rstd * weight + bias
// The row stays in registers between the two sums, so the variance is the
// exact two-pass form (no cancellation of E[s^2] - mean^2) at one read.  The
// second pass also sums s - mean, which is what the first one's roundings left: in
// a row that is all but constant it corrects the mean, the variance and y.  (rstd
// is up to 1/sqrt(eps) there, and would make much of an ulp of the mean.)
//
// Backward, with h = (x - mean) * rstd and t = dy * weight:
//   dx = rstd * (t - mean(t) - h * mean(t * h)) (+ dsum)
//   dweight = sum over rows of dy * h,   dbias = sum over rows of dy
// Persistent CTAs walk the rows; every thread owns fixed columns and keeps
// their two running column sums in registers, so the activations are read
// once for dx and for the column sums alike.  Each CTA then writes one row of
// partial column sums, and a second kernel adds the CTAs' rows in CTA order:
// no atomics, the same bits on every run.
//
// Everything is computed in fp32 whatever the types in memory, and each
// result is rounded once.  HBM bytes bound the large sizes (each activation
// tensor moves once); launches bound the small ones, so every kernel's launch
// overlaps the end of the one before it (griddepcontrol).  That one may still be
// writing what this one reads, so no load takes the read-only path.
//
// Rows in whole 16-byte vectors take ln_fwd_kernel and ln_bwd_kernel, others
// ln_fwd_scalar_kernel and ln_bwd_kernel's RAGGED form, and rows that are wide or
// oddly placed the any-shape kernels.

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>

#include "cc_dp_internal.h"
#include "cc_tc_device.cuh"
#include "cc_trace.h"

namespace ccdp {

// Set by a wait for a row's copies that ran out.
__device__ unsigned int g_ln_status = 0;

namespace {

using namespace tc;

constexpr unsigned kStatusRows = 4096u;

constexpr int kSms = 152;
constexpr int kFwdWarps = 4;            // warps of a CTA of the warp-per-row kernels
constexpr int kScalarThreads = 256;     // CTA of the any-shape kernels
constexpr unsigned kAll = 0xFFFFFFFFu;

// ---- types in memory --------------------------------------------------------

// The kV<T> elements of one 16-byte access, as they lie in memory.
template <typename T> struct Pack;
template <typename T> constexpr int kV = 16 / static_cast<int>(sizeof(T));
template <> struct Pack<float> {
    float4 q;
    __device__ void get(float (&f)[4]) const {
        f[0] = q.x; f[1] = q.y; f[2] = q.z; f[3] = q.w;
    }
    __device__ void put(const float (&f)[4]) { q = make_float4(f[0], f[1], f[2], f[3]); }
    __device__ void load(const float *p) { q = *reinterpret_cast<const float4 *>(p); }
    // vector v of a row in shared memory
    __device__ void take(const unsigned char *row, int v) {
        q = reinterpret_cast<const float4 *>(row)[v];
    }
    __device__ void store(float *p) const { *reinterpret_cast<float4 *>(p) = q; }
};

__device__ __forceinline__ float2 unpack2(uint32_t w, __nv_bfloat16) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
__device__ __forceinline__ float2 unpack2(uint32_t w, __half) {
    return __half22float2(*reinterpret_cast<const __half2 *>(&w));
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi, __nv_bfloat16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi, __half) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

template <typename T> struct Pack16 {
    uint4 q;
    __device__ void get(float (&f)[8]) const {
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 v = unpack2(w[i], T{});
            f[2 * i] = v.x;
            f[2 * i + 1] = v.y;
        }
    }
    __device__ void put(const float (&f)[8]) {
        q = make_uint4(pack2(f[0], f[1], T{}), pack2(f[2], f[3], T{}), pack2(f[4], f[5], T{}),
                       pack2(f[6], f[7], T{}));
    }
    __device__ void load(const T *p) { q = *reinterpret_cast<const uint4 *>(p); }
    __device__ void take(const unsigned char *row, int v) {
        q = reinterpret_cast<const uint4 *>(row)[v];
    }
    __device__ void store(T *p) const { *reinterpret_cast<uint4 *>(p) = q; }
};
template <> struct Pack<__nv_bfloat16> : Pack16<__nv_bfloat16> {};
template <> struct Pack<__half> : Pack16<__half> {};

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f(__half v) { return __half2float(v); }
template <typename T> __device__ __forceinline__ T from_f(float v);
template <> __device__ __forceinline__ float from_f<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) {
    return __float2bfloat16_rn(v);
}
template <> __device__ __forceinline__ __half from_f<__half>(float v) { return __float2half_rn(v); }

// A parameter vector (weight or bias) of a type known at run time: all the
// parameters of a call share it, so its branches are uniform.
struct Param {
    const void *p;      // null: every element is `fill`
    int dtype;
    bool vec;           // 16-byte aligned
    float fill;
    __device__ __forceinline__ float at(size_t i) const {
        if (!p) return fill;
        if (dtype == CC_DTYPE_F32) return static_cast<const float *>(p)[i];
        if (dtype == CC_DTYPE_BF16) return to_f(static_cast<const __nv_bfloat16 *>(p)[i]);
        return to_f(static_cast<const __half *>(p)[i]);
    }
    // Elements i to i + V - 1, i a multiple of V.
    template <int V> __device__ __forceinline__ void vector(size_t i, float (&f)[V]) const {
        if (!p || !vec) {
#pragma unroll
            for (int e = 0; e < V; ++e) f[e] = at(i + e);
        } else if (dtype == CC_DTYPE_F32) {
#pragma unroll
            for (int e = 0; e < V; e += 4) {
                const float4 q =
                    *reinterpret_cast<const float4 *>(static_cast<const float *>(p) + i + e);
                f[e] = q.x; f[e + 1] = q.y; f[e + 2] = q.z; f[e + 3] = q.w;
            }
        } else {
#pragma unroll
            for (int e = 0; e < V; e += 4) {
                const uint2 q =
                    *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(p) + i + e);
                const float2 lo = dtype == CC_DTYPE_BF16 ? unpack2(q.x, __nv_bfloat16{})
                                                         : unpack2(q.x, __half{});
                const float2 hi = dtype == CC_DTYPE_BF16 ? unpack2(q.y, __nv_bfloat16{})
                                                         : unpack2(q.y, __half{});
                f[e] = lo.x; f[e + 1] = lo.y; f[e + 2] = hi.x; f[e + 3] = hi.y;
            }
        }
    }
};

__device__ __forceinline__ void store_param(void *p, int dtype, size_t i, float v) {
    if (dtype == CC_DTYPE_F32) static_cast<float *>(p)[i] = v;
    else if (dtype == CC_DTYPE_BF16) static_cast<__nv_bfloat16 *>(p)[i] = from_f<__nv_bfloat16>(v);
    else static_cast<__half *>(p)[i] = from_f<__half>(v);
}

__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_launch() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// Two fp32 values to an instruction.
using f2 = unsigned long long;
__device__ __forceinline__ f2 pair(float lo, float hi) {
    f2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ float2 both(f2 a) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a));
    return r;
}
__device__ __forceinline__ float add(f2 a) { return both(a).x + both(a).y; }
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
    f2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
    f2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
    f2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

// ---- sums over a row --------------------------------------------------------

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(kAll, v, d);
    return v;
}

__device__ __forceinline__ float2 warp_sum2(float a, float b) {
    return make_float2(warp_sum(a), warp_sum(b));
}

// The CTA's sums of a and b, the same on every thread; `buf` holds 64 floats
// and alternates between two buffers so that one barrier a call is enough.
__device__ __forceinline__ float2 block_sum2(float a, float b, float *buf) {
    a = warp_sum(a);
    b = warp_sum(b);
    const int warps = (blockDim.x + 31) / 32;
    if ((threadIdx.x & 31) == 0) {
        buf[threadIdx.x / 32] = a;
        buf[32 + threadIdx.x / 32] = b;
    }
    __syncthreads();
    const int lane = threadIdx.x & 31;
    a = warp_sum(lane < warps ? buf[lane] : 0.0f);
    b = warp_sum(lane < warps ? buf[32 + lane] : 0.0f);
    return make_float2(a, b);
}

// The two sums over a group of warps that share a row: half the lanes carry on
// with each, so five exchanges do for both; buf is the group's, for this row.
// `go`, the same on a warp's lanes, becomes false on all of the group's warps if
// it is on one; quit: the group's flag for this row, 0 until a warp sets it.
__device__ __forceinline__ float2 group_sum2(float a, float b, float2 *buf, int group, int warps,
                                             volatile int *quit, bool &go) {
    const int lane = threadIdx.x & 31;
    float keep = lane & 16 ? b : a;
    keep += __shfl_xor_sync(kAll, lane & 16 ? a : b, 16);
#pragma unroll
    for (int d = 8; d > 0; d >>= 1) keep += __shfl_xor_sync(kAll, keep, d);
    a = __shfl_sync(kAll, keep, 0);
    b = __shfl_sync(kAll, keep, 16);
    if (warps == 1) return make_float2(a, b);
    if (lane == 0) buf[threadIdx.x / 32 % warps] = make_float2(a, b);
    if (!go) *quit = 1;
    asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(32 * warps) : "memory");
    go = *quit == 0;
    const float2 v = lane < warps ? buf[lane] : make_float2(0.0f, 0.0f);
    a = warp_sum(v.x);
    b = warp_sum(v.y);
    return make_float2(a, b);
}

// ---- forward ----------------------------------------------------------------

// A row's statistics from its first mean m and the sums of the deviations d from
// it and of their squares: the mean, 1 / sqrt(variance + eps), and the shift that
// makes d * rstd + shift the normalised element.  m is off by some ulps of the
// row's largest elements, the mean c of the deviations by some of theirs: c
// corrects m where they are small next to it (a deviation below |m| / 16), and
// would only add its own roundings to it elsewhere.
struct RowStats {
    float mean, rstd, shift;
};
__device__ __forceinline__ RowStats row_stats(float m, float sum_d, float sum_d2, float inv_cols,
                                              float eps) {
    float c = sum_d * inv_cols;
    float var = sum_d2 * inv_cols;
    if (!(256.0f * var < m * m)) c = 0.0f;
    var = __fmaf_rn(-c, c, var);
    if (var < 0.0f) var = 0.0f;                       // a rounding; NaN stays
    const float rstd = __frsqrt_rn(var + eps);
    return {m + c, rstd, -c * rstd};
}

template <typename T>
struct FwdArgs {
    const T *x, *residual;        // residual null: none
    T *y, *sum_out;               // sum_out null: not kept
    Param weight, bias;
    float *mean, *rstd;           // null: not kept
    size_t rows, cols, ldx, ldr, ldy, lds;
    float eps, inv_cols;
};

// One row on blockDim.x threads (BLOCK) or one warp, NV vectors a thread: four,
// which keeps 64 bytes (128 with a residual) a thread on their way and leaves room
// for 24 and more warps an SM.  Rows are not walked by persistent CTAs here: with
// little state to a row, new CTAs hide more latency than a ring of stages did
// (16384 x 1024: 32 us).  16384 x 1024 bf16 with residual and sum in 24.5 us, 5.5
// TB/s; 8192 x 3072 fp32 in 34.2 us, 5.9 TB/s (a device copy of as many bytes takes
// 2 us less); 512 x 1024 in 3.9 us, which is the call's time on the CPU.
template <typename T, int NV, bool BLOCK>
__global__ void __launch_bounds__(BLOCK ? 1024 : 32 * kFwdWarps)
ln_fwd_kernel(const __grid_constant__ FwdArgs<T> p) {
    __shared__ float buf[BLOCK ? 128 : 1];
    const int L = BLOCK ? static_cast<int>(blockDim.x) : 32;
    const int lane = BLOCK ? static_cast<int>(threadIdx.x) : static_cast<int>(threadIdx.x & 31);
    const size_t row = BLOCK ? blockIdx.x
                             : static_cast<size_t>(blockIdx.x) * (blockDim.x / 32) + threadIdx.x / 32;
    pdl_wait();
    pdl_launch();
    if (!BLOCK && row >= p.rows) return;
    constexpr int V = kV<T>;
    const int nvec = static_cast<int>(p.cols / V);
    float f[NV][V];
    const T *x = p.x + row * p.ldx;
    if (p.residual) {
        const T *r = p.residual + row * p.ldr;
        Pack<T> a[NV], b[NV];
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int v = lane + k * L;
            if (v < nvec) {
                a[k].load(x + static_cast<size_t>(v) * V);
                b[k].load(r + static_cast<size_t>(v) * V);
            }
        }
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int v = lane + k * L;
            if (v < nvec) {
                float g[V];
                a[k].get(f[k]);
                b[k].get(g);
#pragma unroll
                for (int e = 0; e < V; ++e) f[k][e] += g[e];
                a[k].put(f[k]);                 // the sum as the activations' type holds it
                a[k].get(f[k]);
                if (p.sum_out) a[k].store(p.sum_out + row * p.lds + static_cast<size_t>(v) * V);
            }
        }
    } else {
        Pack<T> a[NV];
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int v = lane + k * L;
            if (v < nvec) a[k].load(x + static_cast<size_t>(v) * V);
        }
#pragma unroll
        for (int k = 0; k < NV; ++k)
            if (lane + k * L < nvec) a[k].get(f[k]);
    }
    float s = 0.0f;
#pragma unroll
    for (int k = 0; k < NV; ++k)
        if (lane + k * L < nvec) {
#pragma unroll
            for (int e = 0; e < V; ++e) s += f[k][e];
        }
    s = BLOCK ? block_sum2(s, 0.0f, buf).x : warp_sum(s);
    const float mean = s * p.inv_cols;
    const f2 less = pair(-mean, -mean);
    f2 c = 0, q = 0;
#pragma unroll
    for (int k = 0; k < NV; ++k)
        if (lane + k * L < nvec) {
#pragma unroll
            for (int e = 0; e < V; e += 2) {
                const f2 d = add2(pair(f[k][e], f[k][e + 1]), less);
                c = add2(c, d);
                q = fma2(d, d, q);
                f[k][e] = both(d).x;
                f[k][e + 1] = both(d).y;
            }
        }
    const float2 sums = BLOCK ? block_sum2(add(c), add(q), buf + 64) : warp_sum2(add(c), add(q));
    const RowStats st = row_stats(mean, sums.x, sums.y, p.inv_cols, p.eps);
    if (lane == 0) {
        if (p.mean) p.mean[row] = st.mean;
        if (p.rstd) p.rstd[row] = st.rstd;
    }
    T *y = p.y + row * p.ldy;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int v = lane + k * L;
        if (v < nvec) {
            float w[V], b[V];
            p.weight.vector(static_cast<size_t>(v) * V, w);
            p.bias.vector(static_cast<size_t>(v) * V, b);
#pragma unroll
            for (int e = 0; e < V; ++e)
                f[k][e] = __fmaf_rn(__fmaf_rn(f[k][e], st.rstd, st.shift), w[e], b[e]);
            Pack<T> o;
            o.put(f[k]);
            o.store(y + static_cast<size_t>(v) * V);
        }
    }
}

// Rows that cannot be read in 16-byte vectors: NE elements a thread, one by one
// and all in flight at once, a warp or (BLOCK) a CTA a row.  A warp's accesses
// are 32 elements side by side wherever the row starts; they cost more
// instructions than vectors, but no masks, no shifts and no edges.  (The
// aligned vectors that a row touches, masked at its ends, were slower: 16384 x
// 1023 bf16 with its residual took 66 us, this takes 40; of 1024, 24.)
template <typename T, int NE, bool BLOCK>
__global__ void __launch_bounds__(BLOCK ? 1024 : 32 * kFwdWarps)
ln_fwd_scalar_kernel(const __grid_constant__ FwdArgs<T> p) {
    __shared__ float buf[BLOCK ? 128 : 1];
    const int L = BLOCK ? static_cast<int>(blockDim.x) : 32;
    const int lane = BLOCK ? static_cast<int>(threadIdx.x) : static_cast<int>(threadIdx.x & 31);
    const size_t row = BLOCK ? blockIdx.x
                             : static_cast<size_t>(blockIdx.x) * (blockDim.x / 32) + threadIdx.x / 32;
    pdl_wait();
    pdl_launch();
    if (!BLOCK && row >= p.rows) return;
    const int cols = static_cast<int>(p.cols);
    const T *x = p.x + row * p.ldx + lane;
    float f[NE];
    if (p.residual) {
        const T *r = p.residual + row * p.ldr + lane;
        T a[NE], b[NE];
#pragma unroll
        for (int k = 0; k < NE; ++k)
            if (lane + k * L < cols) {
                a[k] = x[k * L];
                b[k] = r[k * L];
            }
        T *sum = p.sum_out ? p.sum_out + row * p.lds + lane : nullptr;
#pragma unroll
        for (int k = 0; k < NE; ++k)
            if (lane + k * L < cols) {
                const T v = from_f<T>(to_f(a[k]) + to_f(b[k]));
                if (sum) sum[k * L] = v;
                f[k] = to_f(v);
            }
    } else {
        T a[NE];
#pragma unroll
        for (int k = 0; k < NE; ++k)
            if (lane + k * L < cols) a[k] = x[k * L];
#pragma unroll
        for (int k = 0; k < NE; ++k)
            if (lane + k * L < cols) f[k] = to_f(a[k]);
    }
    float s = 0.0f;
#pragma unroll
    for (int k = 0; k < NE; ++k)
        if (lane + k * L < cols) s += f[k];
    const float mean = (BLOCK ? block_sum2(s, 0.0f, buf).x : warp_sum(s)) * p.inv_cols;
    const f2 less = pair(-mean, -mean);
    f2 c = 0, q = 0;
#pragma unroll
    for (int k = 0; k < NE; k += 2) {
        // what lies past the row deviates by nothing
        if (lane + k * L >= cols) f[k] = mean;
        if (lane + (k + 1) * L >= cols) f[k + 1] = mean;
        const f2 d = add2(pair(f[k], f[k + 1]), less);
        c = add2(c, d);
        q = fma2(d, d, q);
        f[k] = both(d).x;
        f[k + 1] = both(d).y;
    }
    const float2 sums = BLOCK ? block_sum2(add(c), add(q), buf + 64) : warp_sum2(add(c), add(q));
    const RowStats st = row_stats(mean, sums.x, sums.y, p.inv_cols, p.eps);
    if (lane == 0) {
        if (p.mean) p.mean[row] = st.mean;
        if (p.rstd) p.rstd[row] = st.rstd;
    }
    T *y = p.y + row * p.ldy + lane;
    // Loads of parameters do not overtake stores of y; where a thread has many, all
    // of them come first (bf16, us, first and in turn: 16384 x 333 11.1 and 13.2,
    // 3001 x 8191 65 and 74; with eight a warp's lane 20000 x 61 6.8 and 6.3).
    constexpr bool kAllFirst = NE > 8;
    // the parameters' types, told apart once
    auto finish = [&](auto weight, auto bias) {
#pragma unroll
        for (int k = 0; k < NE; ++k)
            if (lane + k * L < cols) {
                f[k] = __fmaf_rn(__fmaf_rn(f[k], st.rstd, st.shift), weight(k * L), bias(k * L));
                if (!kAllFirst) y[k * L] = from_f<T>(f[k]);
            }
        if constexpr (kAllFirst) {
#pragma unroll
            for (int k = 0; k < NE; ++k)
                if (lane + k * L < cols) y[k * L] = from_f<T>(f[k]);
        }
    };
    if (p.weight.p && p.bias.p && p.weight.dtype == CC_DTYPE_F32) {
        const float *w = static_cast<const float *>(p.weight.p) + lane;
        const float *b = static_cast<const float *>(p.bias.p) + lane;
        finish([&](int i) { return w[i]; }, [&](int i) { return b[i]; });
    } else {
        finish([&](int i) { return p.weight.at(lane + i); }, [&](int i) { return p.bias.at(lane + i); });
    }
}

// Any shape, alignment and row stride: one CTA a row, element by element; the
// row is read again for each of the three passes (from L1/L2).
template <typename T>
__global__ void __launch_bounds__(kScalarThreads)
ln_fwd_any_kernel(const __grid_constant__ FwdArgs<T> p) {
    __shared__ float buf[128];
    pdl_wait();
    pdl_launch();
    const size_t row = blockIdx.x;
    const T *x = p.x + row * p.ldx;
    const T *r = p.residual ? p.residual + row * p.ldr : nullptr;
    auto at = [&](size_t i) {
        const float v = to_f(x[i]);
        return r ? to_f(from_f<T>(v + to_f(r[i]))) : v;
    };
    float s = 0.0f;
    for (size_t i = threadIdx.x; i < p.cols; i += kScalarThreads) s += at(i);
    const float mean = block_sum2(s, 0.0f, buf).x * p.inv_cols;
    float q = 0.0f, c = 0.0f;
    for (size_t i = threadIdx.x; i < p.cols; i += kScalarThreads) {
        const float d = at(i) - mean;
        c += d;
        q = __fmaf_rn(d, d, q);
    }
    const float2 sums = block_sum2(c, q, buf + 64);
    const RowStats st = row_stats(mean, sums.x, sums.y, p.inv_cols, p.eps);
    if (threadIdx.x == 0) {
        if (p.mean) p.mean[row] = st.mean;
        if (p.rstd) p.rstd[row] = st.rstd;
    }
    for (size_t i = threadIdx.x; i < p.cols; i += kScalarThreads) {
        const float v = at(i);
        if (p.sum_out) p.sum_out[row * p.lds + i] = from_f<T>(v);
        p.y[row * p.ldy + i] =
            from_f<T>(__fmaf_rn(__fmaf_rn(v - mean, st.rstd, st.shift), p.weight.at(i),
                                p.bias.at(i)));
    }
}

// ---- ragged rows --------------------------------------------------------------
//
// Contiguous rows whose length is no multiple of a vector's V elements start
// anywhere between two 16-byte boundaries.  They are read and written in the
// aligned vectors they touch all the same: vector v of a row holds its columns
// v V - phase .. (phase: the row's first element within its vector), and only
// the first and the last vector, shared with the neighbouring rows, are masked
// and stored element by element.  The parameters lie in shared memory in fp32,
// one word further on every 32, so that the lanes' reads V words apart meet no
// bank twice; V zeros stand before and after them.

// Words of a parameter row in shared memory, and of element i (-V .. cols + V).
__host__ __device__ constexpr size_t ragged_words(size_t cols, int v) {
    return (cols + 2 * v) + (cols + 2 * v) / 32 + 1;
}
template <int V> __device__ __forceinline__ uint32_t ragged_word(int i) {
    const uint32_t at = static_cast<uint32_t>(i + V);
    return at + (at >> 5);
}
template <int V> __device__ __forceinline__ void ragged_row(float *row, const Param &from, int cols) {
    if (threadIdx.x < V) {
        row[ragged_word<V>(static_cast<int>(threadIdx.x) - V)] = 0.0f;
        row[ragged_word<V>(cols + static_cast<int>(threadIdx.x))] = 0.0f;
    }
    const int step = 4 * static_cast<int>(blockDim.x);
#pragma unroll 4
    for (int i = 4 * static_cast<int>(threadIdx.x); i < cols; i += step) {
        float f[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        if (i + 4 <= cols) {
            from.vector(i, f);
        } else {
#pragma unroll
            for (int e = 0; e < 3; ++e)
                if (i + e < cols) f[e] = from.at(i + e);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (i + e < cols) row[ragged_word<V>(i + e)] = f[e];
    }
}
template <int V>
__device__ __forceinline__ void ragged_take(const float *row, int c0, float (&f)[V]) {
#pragma unroll
    for (int e = 0; e < V; ++e) f[e] = row[ragged_word<V>(c0 + e)];
}
// Columns c0 .. of a row to memory: a whole vector, or what of it is the row's.
template <typename T, int V>
__device__ __forceinline__ void ragged_store(T *row, int c0, int cols, const float (&f)[V]) {
    if (c0 >= 0 && c0 + V <= cols) {
        Pack<T> a;
        a.put(f);
        a.store(row + c0);
    } else {
#pragma unroll
        for (int e = 0; e < V; ++e)
            if (c0 + e >= 0 && c0 + e < cols) row[c0 + e] = from_f<T>(f[e]);
    }
}

// ---- backward ---------------------------------------------------------------

template <typename T>
struct BwdArgs {
    const T *dy, *x, *dsum;       // dsum null: none
    T *dx;
    Param weight;
    const float *mean, *rstd;
    float *partial;               // the column sums, [gridDim.x][2][cols], or null and
    void *dweight, *dbias;        // the results (of one CTA), each null: not wanted
    int param_dtype;
    size_t rows, cols, lddy, ldx, ldds, lddx;
    float cols_f, inv_cols;
    uint32_t skip;                // the row whose fill never comes (failure injection),
    unsigned long long limit_ns;  // or kNoRow; how long a wait lasts
};
constexpr uint32_t kNoRow = 0xFFFFFFFFu;

// What a CTA that gave up leaves in place of its partial column sums, so that
// none are made from them: a signalling NaN, which no sum is.
constexpr uint32_t kUnfinished = 0x7FA05EADu;

// ---- rows on their way ------------------------------------------------------
//
// The vector kernels are persistent, and rows come by bulk copies into a ring
// of shared-memory stages, a row of every group of warps to a stage.  The bytes in
// flight that HBM's latency asks for (about 70 KB an SM) then cost no
// registers: held in registers, the next row left room for too few warps (the
// backward pass streamed at half of HBM's rate).

__device__ __forceinline__ bool elect_one() {
    uint32_t one;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
    return one != 0;
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes,
                                          uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes"
                 " [%0], [%1], %2, [%3];"
                 ::"r"(dst), "l"(src), "r"(bytes), "r"(bar) : "memory");
}

// Without copies in flight the next rows' latency would be exposed: while a
// block of rows is worked on, the next `stages` - 1 are on their way.
constexpr int kMostStages = 8;

// Bytes of a tensor's rows in a stage (ragged ones with what they share of a
// vector at either end).
__host__ __device__ constexpr uint32_t bwd_pitch(uint32_t groups, uint32_t bytes, bool ragged) {
    return ragged ? (groups * bytes + 45) / 16 * 16 : groups * bytes;
}

// Threads of a CTA, for the registers a thread's E elements take.
constexpr int bwd_threads(int elements, bool hold) {
    return !hold || elements <= 8 ? 1024 : elements <= 16 ? 640 : 384;
}
constexpr int kMostGroups = 15;         // named barriers 1 to 15

// 16384 x 1024 bf16 with dsum in 30.1 us with the columns' kernel, 4.5 TB/s; 8192 x
// 3072 fp32 in 55.4 us, 5.5 TB/s; 512 x 1024 in 8.1 us.  What is left of the large
// ones is the tail: the columns' sums across warps, then the second launch (4 to 5
// us of the GPU's time, half of it hidden).
//
// Rows walk: `warps` warps a row, NV vectors a thread.  Every thread keeps the
// column sums of its own columns in registers, and between the row's two sums
// and dx also h and t (HOLD; without it the widest rows' threads read the row
// twice from shared memory).  RAGGED rows (above) come into shared memory as
// they lie, with the same phase; a thread's columns stay its own because the
// rows of a group of warps are a multiple of eight apart.
template <typename T, int NV, bool HOLD, bool RAGGED>
__global__ void __launch_bounds__(bwd_threads(NV *kV<T>, HOLD))
ln_bwd_kernel(const __grid_constant__ BwdArgs<T> p, int warps, int stages) {
    extern __shared__ __align__(128) unsigned char smem[];
    constexpr int V = kV<T>, H = V / 2;
    __shared__ __align__(8) uint64_t full[kMostStages], empty[kMostStages];
    __shared__ float2 sums[2][32];
    __shared__ int quit[2][32];           // by turns, as the sums
    const int threads = static_cast<int>(blockDim.x);
    const int groups = threads / (32 * warps);
    const int group = static_cast<int>(threadIdx.x) / (32 * warps);
    const int lane = static_cast<int>(threadIdx.x) % (32 * warps);
    const int cols = static_cast<int>(p.cols);
    const uint32_t rows = static_cast<uint32_t>(p.rows);
    // a group's rows all start at the same phase: of a vector, and in the stage
    const uint32_t start = RAGGED ? static_cast<uint32_t>(static_cast<size_t>(blockIdx.x) * groups *
                                                          p.cols * sizeof(T) % 16) +
                                        group * static_cast<uint32_t>(p.cols * sizeof(T))
                                  : group * static_cast<uint32_t>(p.cols * sizeof(T));
    const int phase = RAGGED ? static_cast<int>(start % 16 / sizeof(T)) : 0;
    const int nvec = RAGGED ? (phase + cols + V - 1) / V : cols / V;
    const uint32_t bytes = static_cast<uint32_t>(p.cols * sizeof(T));
    const uint32_t pitch = bwd_pitch(groups, bytes, RAGGED);   // a tensor's part of a stage
    const uint32_t stage_bytes = (p.dsum ? 3 : 2) * pitch;
    // the weight, as float4s: the first four of every vector, then the last
    // four, so that a warp's reads meet no bank twice
    float4 *w_row = reinterpret_cast<float4 *>(smem + stages * stage_bytes);
    if (threadIdx.x == 0) {
        for (int q = 0; q < stages; ++q) {
            mbar_init(smem_u32(&full[q]), 1);
            mbar_init(smem_u32(&empty[q]), threads / 32);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (threadIdx.x < 64) quit[threadIdx.x / 32][threadIdx.x % 32] = 0;
    __syncthreads();
    pdl_wait();

    // A stage holds one row of each group of each tensor; warp 0 fills it, with
    // one copy a tensor where the rows lie one after another.
    const uint32_t step = gridDim.x * groups;
    auto fill_one = [&](const T *src, size_t ld, uint32_t at, uint32_t first, uint32_t n,
                        uint32_t bar) {
        if (ld == p.cols) {
            if (elect_one()) bulk_load(at, src + first * ld, n * bytes, bar);
        } else {
            for (uint32_t r = threadIdx.x; r < n; r += 32)
                bulk_load(at + r * bytes, src + (first + r) * ld, bytes, bar);
        }
    };
    uint32_t fills = 0;                               // bit q: stage q's copies, modulo 2
    auto fill = [&](int q, uint32_t first) {
        if (p.skip - first < static_cast<uint32_t>(groups)) return;
        fills ^= 1u << q;
        const uint32_t n = min(static_cast<uint32_t>(groups), rows - first);
        const uint32_t bar = smem_u32(&full[q]), at = smem_u32(smem) + q * stage_bytes;
        if constexpr (RAGGED) {
            // the aligned vectors that the rows touch, but nothing past the tensor's
            // end: of its last vector the elements one by one
            const size_t from = static_cast<size_t>(first) * bytes, all = p.rows * bytes;
            const size_t lo = from / 16 * 16, end = (from + n * bytes + 15) / 16 * 16;
            size_t hi = end;
            if (end > all) {
                hi = all / 16 * 16;
                const size_t i = hi / sizeof(T) + threadIdx.x;
                if (i * sizeof(T) < all) {
                    T *to = reinterpret_cast<T *>(smem + q * stage_bytes + (i * sizeof(T) - lo));
                    to[0] = p.dy[i];
                    to[pitch / sizeof(T)] = p.x[i];
                    if (p.dsum) to[2 * pitch / sizeof(T)] = p.dsum[i];
                }
                __syncwarp();
            }
            if (elect_one()) {
                const uint32_t size = static_cast<uint32_t>(hi - lo);
                mbar_arrive_expect_tx(bar, (p.dsum ? 3 : 2) * size);
                if (size > 0) {
                    const size_t e = lo / sizeof(T);
                    bulk_load(at, p.dy + e, size, bar);
                    bulk_load(at + pitch, p.x + e, size, bar);
                    if (p.dsum) bulk_load(at + 2 * pitch, p.dsum + e, size, bar);
                }
            }
        } else {
            if (elect_one()) mbar_arrive_expect_tx(bar, (p.dsum ? 3 : 2) * n * bytes);
            __syncwarp();
            fill_one(p.dy, p.lddy, at, first, n, bar);
            fill_one(p.x, p.ldx, at + pitch, first, n, bar);
            if (p.dsum) fill_one(p.dsum, p.ldds, at + 2 * pitch, first, n, bar);
        }
        __syncwarp();
    };
    const bool filler = threadIdx.x < 32;
    uint32_t first = blockIdx.x * groups;
    if (filler)
        for (int q = 0; q < stages && first + q * step < rows; ++q) fill(q, first + q * step);
    if constexpr (RAGGED) {
        ragged_row<V>(reinterpret_cast<float *>(w_row), p.weight, cols);
    } else {
        for (int i = threadIdx.x; i < nvec * (V / 4); i += threads) {
            float f[4];
            p.weight.vector(static_cast<size_t>(i % nvec) * V + i / nvec * 4, f);
            w_row[i] = make_float4(f[0], f[1], f[2], f[3]);
        }
    }
    float nmean = 0.0f, nrstd = 0.0f;
    if (first + group < rows) {
        nmean = p.mean[first + group];
        nrstd = p.rstd[first + group];
    }
    __syncthreads();
    pdl_launch();

    f2 dw[NV][H], db[NV][H];
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int e = 0; e < H; ++e) dw[k][e] = db[k][e] = 0;
    // dy, h and t = dy * weight of one vector of a row in shared memory
    auto vector = [&](const unsigned char *in, int v, f2 mean2, f2 rstd2, f2 (&y)[H], f2 (&h)[H], f2 (&t)[H]) {
        Pack<T> a;
        float f[V];
        a.take(in, v);
        a.get(f);
#pragma unroll
        for (int e = 0; e < H; ++e) y[e] = pair(f[2 * e], f[2 * e + 1]);
        const int c0 = v * V - phase;
        const bool edge = RAGGED && (c0 < 0 || c0 + V > cols);
        if (edge) {                                   // the neighbours' elements: dy = 0
#pragma unroll
            for (int e = 0; e < V; ++e)
                if (c0 + e < 0 || c0 + e >= cols) f[e] = 0.0f;
#pragma unroll
            for (int e = 0; e < H; ++e) y[e] = pair(f[2 * e], f[2 * e + 1]);
        }
        a.take(in + pitch, v);
        a.get(f);
        if (edge) {                                   // and h = 0
            const float mean = -both(mean2).x;
#pragma unroll
            for (int e = 0; e < V; ++e)
                if (c0 + e < 0 || c0 + e >= cols) f[e] = mean;
        }
#pragma unroll
        for (int e = 0; e < H; ++e)
            h[e] = mul2(add2(pair(f[2 * e], f[2 * e + 1]), mean2), rstd2);
        if constexpr (RAGGED) {
            ragged_take(reinterpret_cast<const float *>(w_row), c0, f);
#pragma unroll
            for (int e = 0; e < H; ++e) t[e] = mul2(y[e], pair(f[2 * e], f[2 * e + 1]));
        } else {
#pragma unroll
            for (int e = 0; e < H; e += 2) {
                const float4 w = w_row[e / 2 * nvec + v];
                t[e] = mul2(y[e], pair(w.x, w.y));
                t[e + 1] = mul2(y[e + 1], pair(w.z, w.w));
            }
        }
    };
    // A bounded wait of a warp.  After one that ran out the warp, and with it the
    // others that share its rows, waits for nothing more and leaves: no dx from a
    // stage that was not filled, and no column sums of this CTA.
    auto wait = [&](uint64_t *bar, uint32_t parity) {
        const bool there = mbar_wait(smem_u32(bar), parity, p.limit_ns);
        if (!there) atomicOr(&g_ln_status, kStatusRows);
        return __all_sync(kAll, there) != 0;
    };
    bool go = true;
    int turn = 0, stage = 0, before = 0;              // before: the stage before this one
    uint32_t parity = 0, parity_before = 0;
    for (bool later = false; first < rows; first += step, later = true, turn ^= 1) {
        const uint32_t row = first + group;
        const float rstd = nrstd;
        const f2 mean2 = pair(-nmean, -nmean), rstd2 = pair(rstd, rstd);
        if (row + step < rows) {
            nmean = p.mean[row + step];
            nrstd = p.rstd[row + step];
        }
        // The stage before this one is filled anew as soon as every warp has
        // read it, most likely by now.
        if (filler && later && stages > 1 && first + (stages - 1) * step < rows) {
            go = wait(&empty[before], parity_before);
            if (go) fill(before, first + (stages - 1) * step);
        }
        go = go && wait(&full[stage], parity);
        const unsigned char *in = smem + stage * stage_bytes + start / 16 * 16;
        if (row < rows) {
        f2 h[HOLD ? NV : 1][H], t[HOLD ? NV : 1][H];
        f2 s1 = 0, s2 = 0;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int v = lane + k * 32 * warps, at = HOLD ? k : 0;
            if (v < nvec) {
                f2 y[H];
                vector(in, v, mean2, rstd2, y, h[at], t[at]);
#pragma unroll
                for (int e = 0; e < H; ++e) {
                    s1 = add2(s1, t[at][e]);
                    s2 = fma2(t[at][e], h[at][e], s2);
                    dw[k][e] = fma2(y[e], h[at][e], dw[k][e]);
                    db[k][e] = add2(db[k][e], y[e]);
                }
            }
        }
        const float2 a = both(s1), b = both(s2);
        const float2 s = group_sum2(a.x + a.y, b.x + b.y, sums[turn] + group * warps, group, warps,
                                    &quit[turn][group], go);
        if (!go) break;
        // The mean of t a quotient, not a product with 1 / cols, and taken off before rstd is
        // multiplied: equal gradients leave nothing.
        const float m1 = -__fdiv_rn(s.x, p.cols_f), m2 = -(s.y * p.inv_cols);
        const f2 m1s = pair(m1, m1), m2s = pair(m2, m2);
        T *dx = p.dx + row * p.lddx;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int v = lane + k * 32 * warps, at = HOLD ? k : 0;
            if (v < nvec) {
                if (!HOLD) {
                    f2 y[H];
                    vector(in, v, mean2, rstd2, y, h[0], t[0]);
                }
                float o[V];
#pragma unroll
                for (int e = 0; e < H; ++e) {
                    const float2 d = both(mul2(fma2(h[at][e], m2s, add2(t[at][e], m1s)), rstd2));
                    o[2 * e] = d.x;
                    o[2 * e + 1] = d.y;
                }
                Pack<T> out;
                if (p.dsum) {
                    float g[V];
                    out.take(in + 2 * pitch, v);
                    out.get(g);
#pragma unroll
                    for (int e = 0; e < V; ++e) o[e] += g[e];
                }
                if constexpr (RAGGED) {
                    ragged_store(dx, v * V - phase, cols, o);
                } else {
                    out.put(o);
                    out.store(dx + v * V);
                }
            }
        }
        }
        if (!go) break;
        __syncwarp();
        if ((threadIdx.x & 31) == 0) mbar_arrive(smem_u32(&empty[stage]));
        if (filler && stages == 1 && first + step < rows) {
            go = wait(&empty[0], parity);
            if (go) fill(0, first + step);
        }
        before = stage;
        parity_before = parity;
        if (++stage == stages) {
            stage = 0;
            parity ^= 1u;
        }
    }
    if (filler && !go)                                // let the copies in flight land
        for (int q = 0; q < stages; ++q) mbar_wait(smem_u32(&full[q]), (fills >> q & 1u) ^ 1u);
    if (!p.partial && !p.dweight && !p.dbias) return;
    // the groups' sums in group order, dweight then dbias, in the stages' place
    float *out = p.partial + static_cast<size_t>(blockIdx.x) * 2 * p.cols;
    float *cross = reinterpret_cast<float *>(smem);
    const bool only = !p.partial;                     // these are the results already
    if (__syncthreads_or(!go)) {
        if (!only)
            for (int c = threadIdx.x; c < 2 * cols; c += threads) out[c] = __uint_as_float(kUnfinished);
        return;
    }
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        const bool direct = groups == 1 && !only;
        float *to = direct ? out + which * p.cols : cross + static_cast<size_t>(group) * cols;
        if (!direct) __syncthreads();
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int v = lane + k * 32 * warps;
            if (v < nvec && RAGGED) {
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float2 two = both(which ? db[k][e / 2] : dw[k][e / 2]);
                    const int c = v * V - phase + e;
                    if (c >= 0 && c < cols) to[c] = e % 2 ? two.y : two.x;
                }
            } else if (v < nvec) {
#pragma unroll
                for (int e = 0; e < H; e += 2) {
                    const float2 lo = both(which ? db[k][e] : dw[k][e]);
                    const float2 hi = both(which ? db[k][e + 1] : dw[k][e + 1]);
                    reinterpret_cast<float4 *>(to + static_cast<size_t>(v) * V)[e / 2] =
                        make_float4(lo.x, lo.y, hi.x, hi.y);
                }
            }
        }
        if (direct) continue;
        __syncthreads();
        for (int c = threadIdx.x; c < cols; c += threads) {
            float s = cross[c];
            for (int g = 1; g < groups; ++g) s += cross[g * cols + c];
            void *result = which ? p.dbias : p.dweight;
            if (!only) out[static_cast<size_t>(which) * p.cols + c] = s;
            else if (result) store_param(result, p.param_dtype, c, s);
        }
    }
}

// Any shape, alignment and row stride: one CTA a row at a time, element by
// element; the column sums live in the CTA's own row of the workspace, where
// each column is always the same thread's.  Their traffic, and one element an
// access, make it slow: 16384 x 1024 bf16 with dsum, rows 1027 elements apart, 275
// us; 2000 x 16392 725 (of 16384 in vectors 86).
template <typename T>
__global__ void __launch_bounds__(kScalarThreads)
ln_bwd_any_kernel(const __grid_constant__ BwdArgs<T> p) {
    __shared__ float buf[128];
    pdl_wait();
    pdl_launch();
    float *dw = p.partial ? p.partial + static_cast<size_t>(blockIdx.x) * 2 * p.cols : nullptr;
    float *db = dw ? dw + p.cols : nullptr;
    if (dw)
        for (size_t i = threadIdx.x; i < p.cols; i += kScalarThreads) dw[i] = db[i] = 0.0f;
    int which = 0;
    for (size_t row = blockIdx.x; row < p.rows; row += gridDim.x, which ^= 1) {
        const T *dy = p.dy + row * p.lddy;
        const T *x = p.x + row * p.ldx;
        const float mean = p.mean[row], rstd = p.rstd[row];
        float s1 = 0.0f, s2 = 0.0f;
        for (size_t i = threadIdx.x; i < p.cols; i += kScalarThreads) {
            const float y = to_f(dy[i]);
            const float h = (to_f(x[i]) - mean) * rstd;
            const float t = y * p.weight.at(i);
            s1 += t;
            s2 = __fmaf_rn(t, h, s2);
            if (dw) {
                dw[i] = __fmaf_rn(y, h, dw[i]);
                db[i] += y;
            }
        }
        const float2 s = block_sum2(s1, s2, buf + 64 * which);
        s1 = __fdiv_rn(s.x, p.cols_f);
        s2 = s.y * p.inv_cols;
        for (size_t i = threadIdx.x; i < p.cols; i += kScalarThreads) {
            const float h = (to_f(x[i]) - mean) * rstd;
            float o = rstd * ((to_f(dy[i]) * p.weight.at(i) - s1) - h * s2);
            if (p.dsum) o += to_f(p.dsum[row * p.ldds + i]);
            p.dx[row * p.lddx + i] = from_f<T>(o);
        }
    }
}

// The column sums of the CTAs' partial rows, in CTA order within each of
// kSlices interleaved slices, the slices then in order.  Where a CTA gave up
// nothing is written.
constexpr int kColsPerBlock = 32;
constexpr int kSlices = 16;

__global__ void __launch_bounds__(kColsPerBlock * kSlices)
ln_bwd_columns_kernel(const float *partial, int count, size_t cols, void *dweight, void *dbias,
                      int dtype) {
    __shared__ float sum[kSlices][kColsPerBlock];
    pdl_wait();
    pdl_launch();
    const int c = threadIdx.x % kColsPerBlock, slice = threadIdx.x / kColsPerBlock;
    const size_t col = static_cast<size_t>(blockIdx.x) * kColsPerBlock + c;
    const int which = blockIdx.y;
    void *out = which ? dbias : dweight;
    if (!out) return;
    float s = 0.0f;
    bool whole = true;
    if (col < cols)
#pragma unroll 8
        for (int q = slice; q < count; q += kSlices) {
            const float v = partial[(static_cast<size_t>(q) * 2 + which) * cols + col];
            whole = whole && __float_as_uint(v) != kUnfinished;
            s += v;
        }
    sum[slice][c] = s;
    if (__syncthreads_or(!whole)) return;
    if (slice == 0 && col < cols) {
#pragma unroll
        for (int k = 1; k < kSlices; ++k) s += sum[k][c];
        store_param(out, dtype, col, s);
    }
}

// ---- dispatch ---------------------------------------------------------------

// How rows are walked: nv 16-byte vectors (or elements) a thread, `warps` warps a
// row.  Rows of more than 16384 elements take the any-shape kernels; so do, in the
// backward pass, rows off 16-byte boundaries that are not contiguous either, and
// the few whose stage would not fit in shared memory.
struct Shape {
    enum Kind { kVector, kRagged, kScalar, kAny } kind;
    int nv, warps, threads;
    unsigned grid;
    int stages;                   // backward: of a ring
    size_t smem;
    bool hold;
    bool direct;                  // backward: one CTA, which makes the column sums' results
};
constexpr size_t kMostCols = 16384;
constexpr size_t kSharedMost = 220 * 1024;       // shared memory of a CTA

int threads_of(size_t nvec, int nv) {
    return static_cast<int>((nvec + nv * 32 - 1) / (nv * 32) * 32);
}

// Rows as they can be read.
enum class Rows { kVector, kRagged, kAny };

Shape forward_shape(size_t rows, size_t cols, size_t elem, Rows how) {
    if (cols > kMostCols)
        return {Shape::kAny, 0, 0, kScalarThreads, static_cast<unsigned>(rows), 0, 0, true, false};
    Shape s{};
    const bool vector = how == Rows::kVector;
    s.kind = vector ? Shape::kVector : Shape::kScalar;
    const size_t n = vector ? cols * elem / 16 : cols;
    if (vector) s.nv = n <= 32 ? 1 : n <= 64 ? 2 : 4;
    // Element by element: sixteen a thread, and eight where a warp does (bf16, us,
    // sixteen and eight: 16384 x 333 10.4 and, in two warps, 17.4; 16384 x 1023 39.7
    // and 39.0; 2000 x 5001 27.5 and 29.2).
    else s.nv = n <= 256 ? 8 : 16;
    s.threads = threads_of(n, s.nv);
    s.warps = s.threads / 32;
    // few rows: over all SMs, rather than all a CTA's warps
    const size_t each = s.warps > 1 ? 1 : std::min<size_t>((rows + kSms - 1) / kSms, kFwdWarps);
    if (each > 1) s.threads = static_cast<int>(32 * each);
    s.grid = static_cast<unsigned>((rows + each - 1) / each);
    return s;
}

// tensors: rows of this many inputs are read for one row of dx.  One CTA an SM.
Shape backward_shape(size_t rows, size_t cols, size_t elem, Rows how, int tensors) {
    const int v = 16 / static_cast<int>(elem);
    const bool ragged = how == Rows::kRagged;
    const size_t weight = (ragged ? ragged_words(cols, v) * 4 + 15 : cols * 4) / 16 * 16;
    auto stage_of = [&](size_t groups) {
        return static_cast<size_t>(tensors) * bwd_pitch(static_cast<uint32_t>(groups),
                                                        static_cast<uint32_t>(cols * elem), ragged);
    };
    if (how == Rows::kAny || cols > kMostCols || stage_of(1) + weight > kSharedMost)
        return {Shape::kAny, 0, 0, kScalarThreads,
                static_cast<unsigned>(std::min<size_t>(rows, 2 * kSms)), 0, 0, true, false};
    const size_t nvec = ragged ? (cols + 2 * v - 2) / v : cols / v;
    Shape s{};
    s.kind = ragged ? Shape::kRagged : Shape::kVector;
    const int full = 32 / v;                          // vectors of 32 elements
    s.nv = nvec <= 32 ? 1 : nvec <= 64 ? 2 : nvec <= 128 ? 4 : full;
    s.hold = true;
    s.warps = threads_of(nvec, s.nv) / 32;
    if (s.warps > 12) {
        s.nv = full / 2;
        s.hold = false;
        s.warps = threads_of(nvec, s.nv) / 32;
        if (s.warps > 32)
            return {Shape::kAny, 0, 0, kScalarThreads,
                    static_cast<unsigned>(std::min<size_t>(rows, 2 * kSms)), 0, 0, true, false};
    }
    const int most = bwd_threads(s.nv * v, s.hold) / 32 / s.warps;
    // few rows: over all SMs, rather than all a CTA's groups
    const size_t held = std::min(most, s.warps == 1 ? 32 : kMostGroups);
    size_t groups = std::clamp<size_t>((rows + kSms - 1) / kSms, 1, held);
    // two stages each, where they fit
    while (groups > 1 && 2 * stage_of(groups) + weight > kSharedMost) --groups;
    // Rows that one CTA takes at once: it makes the column sums' results too, and
    // the second launch is saved, where it has the threads for it (7 x 105 fp32 5.9
    // -> 4.4 us, 12 x 1024 bf16 6.1 -> 5.9; 5 x 1024 6.2 -> 6.4, 1 x 1024 6.1 -> 10.8).
    if (rows <= held && stage_of(rows) + weight <= kSharedMost &&
        rows * s.warps * 32 * 4 >= cols) {
        groups = rows;
        s.direct = true;
    }
    s.threads = static_cast<int>(groups) * s.warps * 32;
    s.stages = static_cast<int>(
        std::clamp<size_t>((kSharedMost - weight) / stage_of(groups), 1, kMostStages));
    s.grid = static_cast<unsigned>(std::min<size_t>((rows + groups - 1) / groups, kSms));
    // the groups' column sums take the stages' place
    s.smem = s.stages * stage_of(groups) + weight;
    if (groups > 1 || s.direct) s.smem = std::max(s.smem, groups * cols * 4);
    return s;
}
static_assert(kSms % 8 == 0, "the rows of a group: a multiple of eight apart");

// Let a kernel have kSharedMost of shared memory on this device, once: the call
// takes the CPU a good part of a small launch's time.
cudaError_t allow_shared_memory(const void *kernel) {
    static std::atomic<uintptr_t> done[64];
    int device = 0;
    cudaError_t e = cudaGetDevice(&device);
    if (e != cudaSuccess) return e;
    const uintptr_t key = reinterpret_cast<uintptr_t>(kernel) + static_cast<uintptr_t>(device);
    for (auto &slot : done) {
        uintptr_t is = slot.load(std::memory_order_acquire);
        if (is == key) return cudaSuccess;
        if (is != 0) continue;
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 static_cast<int>(kSharedMost));
        if (e == cudaSuccess) slot.compare_exchange_strong(is, key, std::memory_order_release);
        return e;
    }
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                static_cast<int>(kSharedMost));
}

// Kernels wait for the work before them on the device (griddepcontrol.wait), so
// their launch overlaps its end.
template <typename... P, typename... A>
cudaError_t launch(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t stream,
                   A... args) {
    if (smem > 40 * 1024) {               // 48 KB with the static part need no leave
        const cudaError_t e = allow_shared_memory(reinterpret_cast<const void *>(kernel));
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <typename T>
cudaError_t launch_fwd(const FwdArgs<T> &a, Rows how, cudaStream_t stream) {
    const Shape s = forward_shape(a.rows, a.cols, sizeof(T), how);
    if (s.kind == Shape::kAny)
        return launch(ln_fwd_any_kernel<T>, dim3(s.grid), s.threads, 0, stream, a);
    if (s.kind == Shape::kScalar) {
        auto kernel = s.warps > 1  ? ln_fwd_scalar_kernel<T, 16, true>
                      : s.nv == 8 ? ln_fwd_scalar_kernel<T, 8, false>
                                  : ln_fwd_scalar_kernel<T, 16, false>;
        return launch(kernel, dim3(s.grid), s.threads, 0, stream, a);
    }
    auto kernel = s.warps > 1  ? ln_fwd_kernel<T, 4, true>
                  : s.nv == 1 ? ln_fwd_kernel<T, 1, false>
                  : s.nv == 2 ? ln_fwd_kernel<T, 2, false>
                              : ln_fwd_kernel<T, 4, false>;
    return launch(kernel, dim3(s.grid), s.threads, 0, stream, a);
}

template <typename T, bool RAGGED> auto bwd_kernel(const Shape &s) {
    constexpr int kFull = 32 / kV<T>;                 // vectors of 32 elements
    return !s.hold     ? ln_bwd_kernel<T, kFull / 2, false, RAGGED>
           : s.nv == 1 ? ln_bwd_kernel<T, 1, true, RAGGED>
           : s.nv == 2 ? ln_bwd_kernel<T, 2, true, RAGGED>
           : s.nv == 4 ? ln_bwd_kernel<T, 4, true, RAGGED>
                       : ln_bwd_kernel<T, kFull, true, RAGGED>;
}

// One-shot injected stall of this thread's next backward launch
// (cc_inject_layernorm_stall): the row whose fill is skipped, or -1, and the
// limit of that launch's waits.
thread_local long long g_stall_row = -1;
thread_local unsigned long long g_stall_ns = 0;

template <typename T>
cudaError_t launch_bwd(BwdArgs<T> a, Rows how, void *dweight, void *dbias, int dtype,
                       cudaStream_t stream) {
    const Shape s = backward_shape(a.rows, a.cols, sizeof(T), how, a.dsum ? 3 : 2);
    if (g_stall_row >= 0 && s.kind != Shape::kAny) {
        a.skip = static_cast<uint32_t>(g_stall_row);
        a.limit_ns = g_stall_ns;
        g_stall_row = -1;
    }
    if (s.direct) {
        a.partial = nullptr;
        a.dweight = dweight;
        a.dbias = dbias;
        a.param_dtype = dtype;
    }
    cudaError_t e = cudaSuccess;
    if (a.rows > 0) {
        e = s.kind == Shape::kAny
                ? launch(ln_bwd_any_kernel<T>, dim3(s.grid), s.threads, 0, stream, a)
                : launch(s.kind == Shape::kRagged ? bwd_kernel<T, true>(s) : bwd_kernel<T, false>(s),
                         dim3(s.grid), s.threads, s.smem, stream, a, s.warps, s.stages);
        if (e != cudaSuccess) return e;
    }
    if ((dweight || dbias) && !s.direct) {
        const dim3 grid(static_cast<unsigned>((a.cols + kColsPerBlock - 1) / kColsPerBlock), 2);
        e = launch(ln_bwd_columns_kernel, grid, kColsPerBlock * kSlices, 0, stream,
                   static_cast<const float *>(a.partial), a.rows > 0 ? static_cast<int>(s.grid) : 0,
                   a.cols, dweight, dbias, dtype);
    }
    return e;
}

// ---- argument checks ---------------------------------------------------------

size_t dtype_size(int dtype) { return dtype == CC_DTYPE_F32 ? 4 : 2; }

bool known_dtype(int d) {
    return d == CC_DTYPE_BF16 || d == CC_DTYPE_F16 || d == CC_DTYPE_F32;
}

// The ranges of one call: collected, compared with one another, then looked
// up in the device's allocations.  At most kMost of them.
struct Ranges {
    static constexpr int kMost = 12;
    struct One {
        uintptr_t lo, hi;
        bool written;
        const char *name;
    } r[kMost];
    int count = 0;

    int add(const void *p, size_t bytes, size_t align, bool written, const char *name) {
        if (!p) return fail(CC_ERR_INVALID, "%s is NULL", name);
        const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
        if (lo % align != 0)
            return fail(CC_ERR_MISALIGNED, "%s=%p is not %zu-byte aligned", name, p, align);
        r[count++] = {lo, lo + bytes, written, name};
        return CC_OK;
    }
    // rows of cols elements, ld elements apart
    int add_rows(const void *p, size_t rows, size_t cols, size_t ld, size_t elem, bool written,
                 const char *name) {
        if (ld < cols)
            return fail(CC_ERR_INVALID, "%s: row stride %zu is below cols=%zu", name, ld, cols);
        if (rows > 0 && ld > (SIZE_MAX / 8 - cols) / rows)
            return fail(CC_ERR_INVALID, "%s: %zu rows of stride %zu are too large", name, rows, ld);
        return add(p, rows == 0 ? 0 : ((rows - 1) * ld + cols) * elem, elem, written, name);
    }
    int check() const {
        for (int i = 0; i < count; ++i)
            for (int j = i + 1; j < count; ++j)
                if ((r[i].written || r[j].written) && r[i].lo < r[j].hi && r[j].lo < r[i].hi)
                    return fail(CC_ERR_ALIAS, "%s overlaps %s", r[i].name, r[j].name);
        int st = ensure_device();
        Allocation last{0, 0};
        for (int i = 0; st == CC_OK && i < count; ++i)
            if (r[i].hi > r[i].lo)
                st = check_device_range(reinterpret_cast<const void *>(r[i].lo),
                                        r[i].hi - r[i].lo, r[i].name, &last);
        return st;
    }
};

// How the rows of all of a call's tensors can be read: in whole 16-byte vectors;
// or, all of them contiguous from a 16-byte boundary on, as ragged ones.
struct Reading {
    size_t cols, elem;
    bool vector, ragged = true;
    Reading(size_t cols_, size_t elem_)
        : cols(cols_), elem(elem_), vector(cols_ * elem_ % 16 == 0) {}
    void add(const void *p, size_t ld) {
        if (p == nullptr) return;
        const bool aligned = reinterpret_cast<uintptr_t>(p) % 16 == 0;
        vector = vector && aligned && ld * elem % 16 == 0;
        ragged = ragged && aligned && ld == cols;
    }
    Rows rows() const { return vector ? Rows::kVector : ragged ? Rows::kRagged : Rows::kAny; }
};

Param param_of(const void *p, int dtype, float fill) {
    return {p, dtype, reinterpret_cast<uintptr_t>(p) % 16 == 0, fill};
}

int check_common(size_t rows, size_t cols, int act_dtype, int param_dtype) {
    if (!known_dtype(act_dtype)) return fail(CC_ERR_INVALID, "act_dtype=%d unknown", act_dtype);
    if (!known_dtype(param_dtype))
        return fail(CC_ERR_INVALID, "param_dtype=%d unknown", param_dtype);
    if (rows > 0x7FFFFFFFu) return fail(CC_ERR_INVALID, "rows=%zu above 2^31 - 1", rows);
    if (cols > 0x7FFFFFFFu) return fail(CC_ERR_INVALID, "cols=%zu above 2^31 - 1", cols);
    return CC_OK;
}

template <typename T>
int forward_typed(const void *x, size_t ldx, const void *residual, size_t ldr,
                  const void *weight, const void *bias, void *y, size_t ldy, void *sum_out,
                  size_t lds, float *mean, float *rstd, size_t rows, size_t cols, float eps,
                  int param_dtype, cudaStream_t stream) {
    FwdArgs<T> a{static_cast<const T *>(x), static_cast<const T *>(residual),
                 static_cast<T *>(y), static_cast<T *>(sum_out),
                 param_of(weight, param_dtype, 1.0f), param_of(bias, param_dtype, 0.0f),
                 mean, rstd, rows, cols, ldx, ldr, ldy, lds, eps,
                 1.0f / static_cast<float>(cols)};
    Reading how(cols, sizeof(T));
    how.add(x, ldx);
    how.add(residual, ldr);
    how.add(y, ldy);
    how.add(sum_out, lds);
    const cudaError_t e = launch_fwd<T>(a, how.rows(), stream);
    return e == cudaSuccess ? CC_OK : fail_cuda(e, "layer norm forward launch");
}

template <typename T>
int backward_typed(const void *dy, size_t lddy, const void *x, size_t ldx, const void *weight,
                   const float *mean, const float *rstd, const void *dsum, size_t ldds,
                   void *dx, size_t lddx, void *dweight, void *dbias, size_t rows, size_t cols,
                   int param_dtype, float *workspace, cudaStream_t stream) {
    BwdArgs<T> a{static_cast<const T *>(dy), static_cast<const T *>(x),
                 static_cast<const T *>(dsum), static_cast<T *>(dx),
                 param_of(weight, param_dtype, 1.0f), mean, rstd,
                 dweight || dbias ? workspace : nullptr, nullptr, nullptr, param_dtype,
                 rows, cols, lddy, ldx, ldds, lddx, static_cast<float>(cols),
                 1.0f / static_cast<float>(cols), kNoRow, kTimeoutNs};
    Reading how(cols, sizeof(T));
    how.add(dy, lddy);
    how.add(x, ldx);
    how.add(dsum, ldds);
    how.add(dx, lddx);
    const cudaError_t e = launch_bwd<T>(a, how.rows(), dweight, dbias, param_dtype, stream);
    return e == cudaSuccess ? CC_OK : fail_cuda(e, "layer norm backward launch");
}

// The largest workspace any alignment of these rows takes: a row of partial
// sums a CTA, and no kernel runs more CTAs than this.
size_t bwd_workspace_bytes(size_t rows, size_t cols) {
    return std::min<size_t>(rows, 2 * kSms) * 2 * cols * sizeof(float);
}

}  // namespace

void arm_layernorm_stall(long long row, unsigned long long limit_ns) {
    g_stall_row = row;
    g_stall_ns = limit_ns;
}

cudaError_t read_ln_status(unsigned *status, bool clear) {
    cudaError_t e = cudaMemcpyFromSymbol(status, g_ln_status, sizeof(unsigned));
    if (e == cudaSuccess && clear) {
        const unsigned zero = 0;
        e = cudaMemcpyToSymbol(g_ln_status, &zero, sizeof(unsigned));
    }
    return e;
}

}  // namespace ccdp

using namespace ccdp;

extern "C" {

int cc_layernorm_forward(const void *x, size_t ldx, const void *residual, size_t ldr,
                         const void *weight, const void *bias, void *y, size_t ldy,
                         void *sum_out, size_t lds, float *mean, float *rstd, size_t rows,
                         size_t cols, float eps, int act_dtype, int param_dtype, void *stream) {
    TraceRange call("cc_layernorm_forward", rows);
    int st = check_common(rows, cols, act_dtype, param_dtype);
    if (st != CC_OK) return st;
    if (!(eps >= 0.0f) || eps > 3.4e38f)
        return fail(CC_ERR_INVALID, "eps=%g must be finite and >= 0", eps);
    if (sum_out && !residual) return fail(CC_ERR_INVALID, "sum_out without a residual");
    if (rows == 0 || cols == 0) return CC_OK;
    const size_t a = dtype_size(act_dtype), pb = dtype_size(param_dtype);
    Ranges rg;
    if ((st = rg.add_rows(x, rows, cols, ldx, a, false, "x")) != CC_OK) return st;
    if (residual && (st = rg.add_rows(residual, rows, cols, ldr, a, false, "residual")) != CC_OK)
        return st;
    if (weight && (st = rg.add(weight, cols * pb, pb, false, "weight")) != CC_OK) return st;
    if (bias && (st = rg.add(bias, cols * pb, pb, false, "bias")) != CC_OK) return st;
    if ((st = rg.add_rows(y, rows, cols, ldy, a, true, "y")) != CC_OK) return st;
    if (sum_out && (st = rg.add_rows(sum_out, rows, cols, lds, a, true, "sum_out")) != CC_OK)
        return st;
    if (mean && (st = rg.add(mean, rows * 4, 4, true, "mean")) != CC_OK) return st;
    if (rstd && (st = rg.add(rstd, rows * 4, 4, true, "rstd")) != CC_OK) return st;
    if ((st = rg.check()) != CC_OK) return st;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    switch (act_dtype) {
        case CC_DTYPE_BF16:
            return forward_typed<__nv_bfloat16>(x, ldx, residual, ldr, weight, bias, y, ldy,
                                                sum_out, lds, mean, rstd, rows, cols, eps,
                                                param_dtype, s);
        case CC_DTYPE_F16:
            return forward_typed<__half>(x, ldx, residual, ldr, weight, bias, y, ldy, sum_out,
                                         lds, mean, rstd, rows, cols, eps, param_dtype, s);
        default:
            return forward_typed<float>(x, ldx, residual, ldr, weight, bias, y, ldy, sum_out,
                                        lds, mean, rstd, rows, cols, eps, param_dtype, s);
    }
}

int cc_layernorm_backward_workspace(size_t rows, size_t cols, size_t *bytes) {
    if (!bytes) return fail(CC_ERR_INVALID, "bytes is NULL");
    *bytes = 0;
    const int st = check_common(rows, cols, CC_DTYPE_F32, CC_DTYPE_F32);
    if (st != CC_OK) return st;
    *bytes = bwd_workspace_bytes(rows, cols);
    return CC_OK;
}

int cc_layernorm_backward(const void *dy, size_t lddy, const void *x, size_t ldx,
                          const void *weight, const float *mean, const float *rstd,
                          const void *dsum, size_t ldds, void *dx, size_t lddx, void *dweight,
                          void *dbias, size_t rows, size_t cols, int act_dtype, int param_dtype,
                          void *workspace, size_t workspace_bytes, void *stream) {
    TraceRange call("cc_layernorm_backward", rows);
    int st = check_common(rows, cols, act_dtype, param_dtype);
    if (st != CC_OK) return st;
    if (cols == 0 || (rows == 0 && !dweight && !dbias)) return CC_OK;
    const size_t a = dtype_size(act_dtype), pb = dtype_size(param_dtype);
    Ranges rg;
    if (rows > 0) {
        if ((st = rg.add_rows(dy, rows, cols, lddy, a, false, "dy")) != CC_OK) return st;
        if ((st = rg.add_rows(x, rows, cols, ldx, a, false, "x")) != CC_OK) return st;
        if ((st = rg.add(mean, rows * 4, 4, false, "mean")) != CC_OK) return st;
        if ((st = rg.add(rstd, rows * 4, 4, false, "rstd")) != CC_OK) return st;
        if (dsum && (st = rg.add_rows(dsum, rows, cols, ldds, a, false, "dsum")) != CC_OK)
            return st;
        if ((st = rg.add_rows(dx, rows, cols, lddx, a, true, "dx")) != CC_OK) return st;
    }
    if (weight && (st = rg.add(weight, cols * pb, pb, false, "weight")) != CC_OK) return st;
    if (dweight && (st = rg.add(dweight, cols * pb, pb, true, "dweight")) != CC_OK) return st;
    if (dbias && (st = rg.add(dbias, cols * pb, pb, true, "dbias")) != CC_OK) return st;
    if ((dweight || dbias) && rows > 0) {
        const size_t need = bwd_workspace_bytes(rows, cols);
        if (workspace_bytes < need)
            return fail(CC_ERR_INVALID, "workspace of %zu bytes, %zu rows of %zu need %zu",
                        workspace_bytes, rows, cols, need);
        if ((st = rg.add(workspace, need, 16, true, "workspace")) != CC_OK) return st;
    }
    if ((st = rg.check()) != CC_OK) return st;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    float *ws = static_cast<float *>(workspace);
    switch (act_dtype) {
        case CC_DTYPE_BF16:
            return backward_typed<__nv_bfloat16>(dy, lddy, x, ldx, weight, mean, rstd, dsum,
                                                 ldds, dx, lddx, dweight, dbias, rows, cols,
                                                 param_dtype, ws, s);
        case CC_DTYPE_F16:
            return backward_typed<__half>(dy, lddy, x, ldx, weight, mean, rstd, dsum, ldds, dx,
                                          lddx, dweight, dbias, rows, cols, param_dtype, ws, s);
        default:
            return backward_typed<float>(dy, lddy, x, ldx, weight, mean, rstd, dsum, ldds, dx,
                                         lddx, dweight, dbias, rows, cols, param_dtype, ws, s);
    }
}

}  // extern "C"
