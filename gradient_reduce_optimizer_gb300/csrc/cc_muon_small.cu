// The Newton-Schulz iteration for matrices whose shorter side m is at most 64
// (adapters, heads), in fp32 throughout.
//
// Two things differ from the tensor-core path.  A tile of the tensor cores is
// 128 wide, so such matrices would leave most of it empty over fifteen
// dependent products; and the roundings of 11-bit operands average out over m
// rows, which few rows do not do (up to 1e-2 of the result at m = 3).  Here
// every iterate is a polynomial of the first Gram matrix, X_k = Q_k X_0 with
// Q_k and A_k = X_k X_k^T both m x m and commuting:
//   P = a I + b A + c A A,   Q <- P Q,   A <- P (A P),
// so the long side is read twice only, in three launches:
//   gram     partial sums of G G^T over slices of the long side;
//   iterate  one CTA a matrix: adds the slices in order, takes |G|_F from the
//            trace, runs all steps in shared memory, leaves Q / (|G|_F + eps);
//   apply    Q G, to bf16 or into the parameters.
// In fp32 the Gram matrix resolves singular values down to 2^-12 of the
// largest, the same relative to which their growth by a^steps stays small; the
// 11-bit path could not do this (it would need its A to 2^-22).  1e-6 of the result
// off on Gaussian matrices, up to 7e-4 where singular values lie there.
//
// What bounds it is the iterate kernel's chain of products: 7 x 64 x 2744 fp32 takes
// 75 us, 60 x 64 x 300 68, a step of 7 x 64 x 2744 with eight replicas 99.
// m = 64 takes 17 products of 64^3 in one CTA, 64 x (two 16-byte reads, 16
// FMAs) a thread each.

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "cc_dp_internal.h"
#include "cc_muon_internal.h"

namespace ccdp {
namespace muon {
namespace {

constexpr int kM = kSmallSide;            // 64
constexpr int kThreads = 256;             // 16 x 16 threads of 4 x 4 elements
constexpr int kPad = kM + 4;              // row stride in shared memory, in floats

__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_launch() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

__device__ __forceinline__ float as_float(const void *p, int dtype, size_t i) {
    if (dtype == CC_DTYPE_F32) return static_cast<const float *>(p)[i];
    if (dtype == CC_DTYPE_BF16) return __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i]);
    return __half2float(static_cast<const __half *>(p)[i]);
}

// c[4][4] += sum over k < len of x[k][4 i ..] y[k][4 j ..]
__device__ __forceinline__ void outer(const float (*x)[kPad], const float (*y)[kPad], int len, int i,
                                      int j, float (&c)[4][4]) {
#pragma unroll 4
    for (int k = 0; k < len; ++k) {
        const float4 a = *reinterpret_cast<const float4 *>(&x[k][4 * i]);
        const float4 b = *reinterpret_cast<const float4 *>(&y[k][4 * j]);
        const float av[4] = {a.x, a.y, a.z, a.w}, bv[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int s = 0; s < 4; ++s) c[r][s] = __fmaf_rn(av[r], bv[s], c[r][s]);
    }
}

// 64 entries of the long side from k0 on, as tile[k][i] with i on the shorter
// side; zero outside the matrix.
__device__ __forceinline__ void load_tile(const SmallSource &s, int b, int k0, float (*tile)[kPad]) {
    const size_t base = static_cast<size_t>(b) * s.stride;
    for (int e = threadIdx.x; e < kM * kM; e += kThreads) {
        const int fast = e % kM, slow = e / kM;      // fast: along a row of the matrix
        const int i = s.tall ? fast : slow, k = s.tall ? slow : fast;
        float v = 0.0f;
        if (i < s.m && k0 + k < s.n) {
            const size_t at = s.tall ? static_cast<size_t>(k0 + k) * s.ld + i
                                     : static_cast<size_t>(i) * s.ld + k0 + k;
            v = as_float(s.p, s.dtype, base + at);
        }
        tile[k][i] = v;
    }
}

__global__ void __launch_bounds__(kThreads)
small_gram_kernel(const __grid_constant__ SmallSource s, float *partial) {
    __shared__ __align__(16) float tile[kM][kPad];
    pdl_wait();
    pdl_launch();
    const int i = threadIdx.x / 16, j = threadIdx.x % 16;
    float c[4][4] = {};
    for (int k0 = blockIdx.x * kM; k0 < s.n; k0 += gridDim.x * kM) {
        load_tile(s, blockIdx.y, k0, tile);
        __syncthreads();
        outer(tile, tile, kM, i, j, c);
        __syncthreads();
    }
    float *out = partial + (static_cast<size_t>(blockIdx.y) * gridDim.x + blockIdx.x) * kM * kM;
#pragma unroll
    for (int r = 0; r < 4; ++r)
        *reinterpret_cast<float4 *>(out + (4 * i + r) * kM + 4 * j) =
            make_float4(c[r][0], c[r][1], c[r][2], c[r][3]);
}

struct SmallCoeffs {
    float v[CC_MUON_MAX_STEPS][3];
    int steps;
};

constexpr int kIterateBytes = 4 * kM * kPad * static_cast<int>(sizeof(float));
// More than half of an SM's: with an SM for every matrix, no two share one.  (They are
// placed while the Gram kernel's CTAs still run, and would gather on the SMs that are
// free first: a step of 7 x 64 x 2744 in 20 us instead of 9.)
constexpr int kIterateAlone = 116 * 1024;

__global__ void __launch_bounds__(kThreads)
small_iterate_kernel(const float *partial, int parts, int m, float eps,
                     const __grid_constant__ SmallCoeffs co, float *q_out) {
    extern __shared__ __align__(16) float smem[];
    using Mat = float (*)[kPad];
    Mat A = reinterpret_cast<Mat>(smem);
    Mat P = A + kM, Q = P + kM, T = Q + kM;
    __shared__ float inv_slot;
    const int i = threadIdx.x / 16, j = threadIdx.x % 16;
    auto put = [&](Mat to, const float (&c)[4][4]) {
#pragma unroll
        for (int r = 0; r < 4; ++r)
            *reinterpret_cast<float4 *>(&to[4 * i + r][4 * j]) =
                make_float4(c[r][0], c[r][1], c[r][2], c[r][3]);
    };
    pdl_wait();
    pdl_launch();
    float g[4][4] = {};
    const float *src = partial + static_cast<size_t>(blockIdx.x) * parts * kM * kM;
    for (int q = 0; q < parts; ++q)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const float4 v =
                *reinterpret_cast<const float4 *>(src + (q * kM + 4 * i + r) * kM + 4 * j);
            g[r][0] += v.x;
            g[r][1] += v.y;
            g[r][2] += v.z;
            g[r][3] += v.w;
        }
    put(A, g);
    __syncthreads();
    if (threadIdx.x < 32) {
        float v = A[threadIdx.x][threadIdx.x] + A[threadIdx.x + 32][threadIdx.x + 32];
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
        if (threadIdx.x == 0) inv_slot = __fdiv_rn(1.0f, __fadd_rn(__fsqrt_rn(v), eps));
    }
    __syncthreads();
    const float inv = inv_slot;
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int s = 0; s < 4; ++s) g[r][s] = g[r][s] * inv * inv;
    put(A, g);
    __syncthreads();
    const bool mine = 4 * i < m && 4 * j < m;         // this thread's block holds entries
    for (int k = 0; k < co.steps; ++k) {
        const float a = co.v[k][0], b = co.v[k][1], c2 = co.v[k][2];
        const bool last = k == co.steps - 1;
        float c[4][4] = {};
        if (mine) {
            outer(A, A, m, i, j, c);
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    c[r][s] = __fmaf_rn(c2, c[r][s], b * A[4 * i + r][4 * j + s]);
                    if (4 * i + r == 4 * j + s) c[r][s] += a;
                }
            put(P, c);
            if (k == 0) put(Q, c);
        }
        __syncthreads();
        float t[4][4] = {};
        if (k > 0) {
            if (mine) outer(P, Q, m, i, j, t);        // P Q
            __syncthreads();
            if (mine) put(Q, t);
        }
        if (!last) {
            float u[4][4] = {};
            if (mine) {
                outer(A, P, m, i, j, u);              // A P
                put(T, u);
            }
            __syncthreads();
            // P (A P), of which one triangle counts for both: outer() reads its first
            // operand across, and an A that its roundings have made unsymmetric goes
            // astray from step to step (a matrix of rank one came out 8e-3 off, and so
            // 2e-4).
            float w[4][4] = {};
            if (mine && j >= i) {
                outer(P, T, m, i, j, w);
                if (i == j) {
#pragma unroll
                    for (int r = 1; r < 4; ++r)
#pragma unroll
                        for (int s = 0; s < r; ++s) w[r][s] = w[s][r];
                } else {
#pragma unroll
                    for (int s = 0; s < 4; ++s)
                        *reinterpret_cast<float4 *>(&A[4 * j + s][4 * i]) =
                            make_float4(w[0][s], w[1][s], w[2][s], w[3][s]);
                }
                put(A, w);
            }
        }
        __syncthreads();
    }
    float *out = q_out + static_cast<size_t>(blockIdx.x) * kM * kM;
    for (int e = threadIdx.x; e < kM * kM; e += kThreads) {
        const int r = e / kM, s = e % kM;
        out[e] = r < m && s < m ? Q[s][r] * inv : 0.0f;   // as outer() reads it
    }
}

// STEP: the parameter update, else bf16 matrices.
template <bool STEP, typename Extra>
__global__ void __launch_bounds__(kThreads)
small_apply_kernel(const __grid_constant__ SmallSource s, const float *q_in,
                   const __grid_constant__ Extra extra) {
    __shared__ __align__(16) float tile[kM][kPad];     // [k on the long side][i]
    __shared__ __align__(16) float xt[kM][kPad];       // [i][k]
    __shared__ __align__(16) float q[kM][kPad];
    const int b = blockIdx.y;
    pdl_wait();
    pdl_launch();
    for (int e = threadIdx.x; e < kM * kM; e += kThreads)
        q[e / kM][e % kM] = q_in[static_cast<size_t>(b) * kM * kM + e];
    const int i = threadIdx.x / 16, j = threadIdx.x % 16;
    for (int k0 = blockIdx.x * kM; k0 < s.n; k0 += gridDim.x * kM) {
        load_tile(s, b, k0, tile);
        __syncthreads();
        for (int e = threadIdx.x; e < kM * kM; e += kThreads) xt[e % kM][e / kM] = tile[e / kM][e % kM];
        __syncthreads();
        float c[4][4] = {};
        outer(q, xt, s.m, i, j, c);                    // q: Q across
        __syncthreads();
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int t = 0; t < 4; ++t) tile[4 * j + t][4 * i + r] = c[r][t];
        __syncthreads();
        for (int e = threadIdx.x; e < kM * kM; e += kThreads) {
            const int fast = e % kM, slow = e / kM;
            const int ii = s.tall ? fast : slow, k = s.tall ? slow : fast;
            if (ii >= s.m || k0 + k >= s.n) continue;
            const size_t row = s.tall ? k0 + k : ii, col = s.tall ? ii : k0 + k;
            const float y = tile[k][ii];
            if constexpr (STEP) {
                const size_t at = extra.offset[b] + row * (s.tall ? s.m : s.n) + col;
                const float w = __fsub_rn(__fmul_rn(extra.master[at], extra.decay),
                                          __fmul_rn(extra.lr_scale, y));
                extra.master[at] = w;
                const __nv_bfloat16 o = __float2bfloat16_rn(w);
                for (int r = 0; r < extra.R; ++r) static_cast<__nv_bfloat16 *>(extra.out[r])[at] = o;
            } else {
                extra.p[static_cast<size_t>(b) * extra.stride + row * extra.ld + col] =
                    __float2bfloat16_rn(y);
            }
        }
        __syncthreads();
    }
}

template <typename... P, typename... A>
cudaError_t launch_chained(void (*kernel)(P...), dim3 grid, size_t smem, cudaStream_t stream,
                           bool chain, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = chain ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <bool STEP, typename Extra>
int run(const SmallSource &s, int count, const float *coeffs, int steps, float eps, float *partial,
        float *q, const Extra &extra, bool chain, cudaStream_t stream) {
    const int parts = small_parts(count, s.n);
    cudaError_t e = launch_chained(small_gram_kernel, dim3(parts, count), 0, stream, chain, s, partial);
    if (e != cudaSuccess) return fail_cuda(e, "Gram launch");
    SmallCoeffs co{};
    for (int k = 0; k < steps; ++k)
        for (int v = 0; v < 3; ++v) co.v[k][v] = coeffs[3 * k + v];
    co.steps = steps;
    e = cudaFuncSetAttribute(reinterpret_cast<const void *>(small_iterate_kernel),
                             cudaFuncAttributeMaxDynamicSharedMemorySize, kIterateAlone);
    if (e != cudaSuccess) return fail_cuda(e, "shared memory attribute");
    e = launch_chained(small_iterate_kernel, dim3(count),
                       count <= 152 ? kIterateAlone : kIterateBytes, stream, true,
                       static_cast<const float *>(partial), parts, s.m, eps, co, q);
    if (e != cudaSuccess) return fail_cuda(e, "iteration launch");
    // enough CTAs for the GPU, a tile of 64 at least each
    const int tiles = (s.n + kM - 1) / kM;
    const int wide = std::min(tiles, std::max(1, 4 * 152 / count));
    e = launch_chained(small_apply_kernel<STEP, Extra>, dim3(wide, count), 0, stream, true, s,
                       static_cast<const float *>(q), extra);
    return e == cudaSuccess ? CC_OK : fail_cuda(e, "apply launch");
}

}  // namespace

int small_parts(int count, int n) {
    const int tiles = (n + kM - 1) / kM;
    return std::max(1, std::min({tiles, 64, 4 * 152 / std::max(count, 1)}));
}

int small_out(const SmallSource &s, int count, const float *coeffs, int steps, float eps,
              float *partial, float *q, const PlainOut &out, bool chain, cudaStream_t stream) {
    return run<false>(s, count, coeffs, steps, eps, partial, q, out, chain, stream);
}

int small_step(const SmallSource &s, int count, const float *coeffs, int steps, float eps,
               float *partial, float *q, const StepOut &out, bool chain, cudaStream_t stream) {
    return run<true>(s, count, coeffs, steps, eps, partial, q, out, chain, stream);
}

}  // namespace muon
}  // namespace ccdp
