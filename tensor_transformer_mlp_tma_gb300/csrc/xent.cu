// Row kernels of the vocabulary cross entropy (the products run in tc_gemm.cu and
// simt_gemm.cu).  With logits S = X W^T [T, V], per token
//   lse = log sum_v exp S_v,   loss = lse - S_y,   dS = (exp(S - lse) - 1[y]) g.
// No [T, V] array exists: the product's epilogue leaves one (max, sum of
// exponentials) pair per token and 128 vocabulary rows, which combine_kernel joins.
// All statistics are fp32.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "kernels.h"
#include "launch.cuh"
#include "ptx.cuh"

namespace tpmlp {
namespace xent {

constexpr uint32_t STATUS_INVALID_ARG = 1;  // TPMLP_ERR_INVALID_ARG

// (m, s) stands for the sum s * exp(m).  An empty pair is (-inf, 0); a NaN or
// +inf logit leaves NaN in s, which every join keeps.
__device__ __forceinline__ void join(float &m, float &s, float m2, float s2) {
    const float mx = fmaxf(m, m2);
    const float base = mx == -INFINITY ? 0.0f : mx;
    s = s * expf(m - base) + s2 * expf(m2 - base);
    m = mx;
}

// Whether row's target takes part: not the ignored index and a row of W.  A target
// outside the vocabulary is reported once in the status word and not read.
__device__ __forceinline__ bool target_ok(const RowArgs &a, int64_t row) {
    const int64_t t = a.target[row];
    if (t == a.ignore_index) return false;
    if (t >= 0 && t < a.vocab) return true;
    if (atomicCAS(a.status, 0u, STATUS_INVALID_ARG) == 0u) atomicExch(a.status + 1, static_cast<uint32_t>(row));
    return false;
}

// loss and lse of 32 tokens per block: lane = token (the partials of one group are
// contiguous over tokens), the warps take every 32nd group and join theirs through
// shared memory, in a fixed order.  Reads 8 bytes per token and 128 vocabulary rows,
// 1/(32 h) of the product's FLOPs in bytes; bound by latency.
constexpr int COMBINE_WARPS = 32;
__global__ void __launch_bounds__(32 * COMBINE_WARPS) combine_kernel(const RowArgs a, float *loss, float *lse) {
    __shared__ float2 sh[COMBINE_WARPS][32];
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * 32 + lane;
    float m = -INFINITY, s = 0.0f;
    if (row < a.tokens) {
#pragma unroll 4
        for (int64_t g = w; g < a.groups; g += COMBINE_WARPS) {
            const float2 p = a.part[g * a.tokens + row];
            join(m, s, p.x, p.y);
        }
    }
    sh[w][lane] = make_float2(m, s);
    __syncthreads();
    for (int half = COMBINE_WARPS / 2; half > 0; half >>= 1) {
        if (w < half) {
            const float2 o = sh[w + half][lane];
            join(m, s, o.x, o.y);
            sh[w][lane] = make_float2(m, s);
        }
        __syncthreads();
    }
    if (w == 0 && row < a.tokens) {
        const float l = logf(s);
        lse[row] = m + l;
        // the difference of the two large terms first, then the small one
        loss[row] = target_ok(a, row) ? (m - a.target_logit[row]) + l : 0.0f;
    }
}

// g of every token for the backward pass: 0 where the target does not take part.
__global__ void row_g_kernel(const RowArgs a, const float *dloss, float *row_g) {
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const int64_t row = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
    if (row < a.tokens) row_g[row] = target_ok(a, row) ? dloss[row] : 0.0f;
}

// Fixed-order sum of the fp32 matrices that split products left, rounded once to the
// output's type.  V columns per thread.  Memory bound: 4 bytes per split and element.
template <typename T, int V>
__global__ void __launch_bounds__(256) sum_splits_kernel(const float *in, int splits, int64_t rows, int64_t cols,
                                                         int64_t ld, T *out) {
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const int64_t per_row = cols / V, n = rows * per_row, step = rows * ld;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < n;
         i += static_cast<int64_t>(gridDim.x) * 256) {
        const int64_t r = i / per_row, c = (i - r * per_row) * V;
        const float *src = in + r * ld + c;
        float v[V];
#pragma unroll
        for (int j = 0; j < V; ++j) v[j] = 0.0f;
        for (int k = 0; k < splits; ++k, src += step) {
            if constexpr (V == 4) {
                const float4 w = *reinterpret_cast<const float4 *>(src);
                v[0] += w.x, v[1] += w.y, v[2] += w.z, v[3] += w.w;
            } else {
                v[0] += *src;
            }
        }
        T *dst = out + r * cols + c;
        if constexpr (sizeof(T) == 4 && V == 4) {
            *reinterpret_cast<float4 *>(dst) = make_float4(v[0], v[1], v[2], v[3]);
        } else if constexpr (sizeof(T) == 4) {
            dst[0] = v[0];
        } else if constexpr (V == 4) {
            const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
            *reinterpret_cast<uint2 *>(dst) =
                make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
        } else {
            dst[0] = __float2bfloat16_rn(v[0]);
        }
    }
}

// x = p0 + p1 + p2 in bf16: the first two cut off after eight bits of the significand, so
// that the three together hold its 24 bits (a value too large to round to bf16 does not
// become infinite; an infinite one has parts inf, 0, 0).  Four columns per thread.
// Memory bound: 4 bytes read, 6 written per element.
__global__ void __launch_bounds__(256) split3_kernel(const float *in, int64_t rows, int64_t cols, int64_t ld,
                                                     __nv_bfloat16 *out) {
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const int64_t n = rows * ld;
    for (int64_t i = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * 4; i < n;
         i += static_cast<int64_t>(gridDim.x) * 1024) {
        const int64_t r = i / ld, c = i - r * ld;
        float v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = c + j < cols ? in[r * cols + c + j] : 0.0f;
#pragma unroll
        for (int part = 0; part < 3; ++part) {
            __nv_bfloat16 h[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float hi = part < 2 ? __uint_as_float(__float_as_uint(v[j]) & 0xFFFF0000u) : v[j];
                h[j] = __float2bfloat16_rn(hi);
                v[j] = isinf(v[j]) ? 0.0f : v[j] - hi;
            }
            *reinterpret_cast<uint2 *>(out + part * n + i) = *reinterpret_cast<const uint2 *>(h);
        }
    }
}

// ---- FFMA path: the logits of one piece of the vocabulary are in memory (fp32) ----
constexpr int ROW_THREADS = 256;

// One (max, sum) pair of one token's logits of this piece, and its target's logit.
__global__ void __launch_bounds__(ROW_THREADS) piece_stats_kernel(const RowArgs a, const float *logits, int64_t n,
                                                                 int64_t col0, float2 *part) {
    __shared__ float2 sh[ROW_THREADS];
    const int64_t row = blockIdx.x;
    const float *x = logits + row * n;
    float m = -INFINITY, s = 0.0f;
    for (int64_t i = threadIdx.x; i < n; i += ROW_THREADS) join(m, s, x[i], 1.0f);
    sh[threadIdx.x] = make_float2(m, s);
    __syncthreads();
    for (int half = ROW_THREADS / 2; half > 0; half >>= 1) {
        if (threadIdx.x < static_cast<unsigned>(half)) {
            const float2 o = sh[threadIdx.x + half];
            join(m, s, o.x, o.y);
            sh[threadIdx.x] = make_float2(m, s);
        }
        __syncthreads();
    }
    if (threadIdx.x == 0) {
        part[row] = make_float2(m, s);
        const int64_t t = a.target[row];
        if (t != a.ignore_index && t >= col0 && t < col0 + n) a.target_logit[row] = x[t - col0];
    }
}

// dS of one token over this piece (fp32 in place, or bf16 beside the logits).
template <typename T>
__global__ void __launch_bounds__(ROW_THREADS) piece_grad_kernel(const RowArgs a, const float *logits, int64_t n,
                                                                int64_t col0, const float *lse, const float *row_g,
                                                                T *out) {
    const int64_t row = blockIdx.x;
    const float g = row_g[row], l = lse[row];
    const int64_t t = a.target[row] - col0;
    for (int64_t i = threadIdx.x; i < n; i += ROW_THREADS) {
        float v = 0.0f;
        if (g != 0.0f) {
            const float p = expf(logits[row * n + i] - l);
            v = (i == t ? p - 1.0f : p) * g;
        }
        if constexpr (sizeof(T) == 4)
            out[row * n + i] = v;
        else
            out[row * n + i] = __float2bfloat16_rn(v);
    }
}

// Blocks of 256 threads for n units of work, as many as stay resident.
static int64_t blocks_for(int64_t n) {
    const int64_t b = (n + 255) / 256;
    return b < 152 * 8 ? b : 152 * 8;
}

}  // namespace xent

cudaError_t launch_xent_combine(const RowArgs &a, float *loss, float *lse, cudaStream_t st) {
    return launch_pdl(xent::combine_kernel, dim3(static_cast<unsigned>((a.tokens + 31) / 32)), 32 * xent::COMBINE_WARPS, 0, st, a, loss, lse);
}

cudaError_t launch_xent_row_g(const RowArgs &a, const float *dloss, float *row_g, cudaStream_t st) {
    return launch_pdl(xent::row_g_kernel, dim3(static_cast<unsigned>((a.tokens + 255) / 256)), 256, 0, st, a, dloss, row_g);
}

cudaError_t launch_sum_splits(bool is_bf16, const float *in, int splits, int64_t rows, int64_t cols, int64_t ld,
                              void *out, cudaStream_t st) {
    const bool vec = cols % 4 == 0 && ld % 4 == 0 && (reinterpret_cast<uintptr_t>(out) & 15) == 0;
    const int64_t blocks = xent::blocks_for(rows * cols / (vec ? 4 : 1));
    if (is_bf16) {
        auto o = static_cast<__nv_bfloat16 *>(out);
        return vec ? launch_pdl(xent::sum_splits_kernel<__nv_bfloat16, 4>, dim3(static_cast<unsigned>(blocks)), 256, 0, st, in, splits, rows, cols, ld, o)
                   : launch_pdl(xent::sum_splits_kernel<__nv_bfloat16, 1>, dim3(static_cast<unsigned>(blocks)), 256, 0, st, in, splits, rows, cols, ld, o);
    }
    auto o = static_cast<float *>(out);
    return vec ? launch_pdl(xent::sum_splits_kernel<float, 4>, dim3(static_cast<unsigned>(blocks)), 256, 0, st, in, splits, rows, cols, ld, o)
               : launch_pdl(xent::sum_splits_kernel<float, 1>, dim3(static_cast<unsigned>(blocks)), 256, 0, st, in, splits, rows, cols, ld, o);
}

cudaError_t launch_split3(const float *in, int64_t rows, int64_t cols, int64_t ld, void *out, cudaStream_t st) {
    return launch_pdl(xent::split3_kernel, dim3(static_cast<unsigned>(xent::blocks_for(rows * ld / 4))), 256, 0, st, in, rows, cols, ld,
                        static_cast<__nv_bfloat16 *>(out));
}

cudaError_t launch_xent_piece_stats(const RowArgs &a, const float *logits, int64_t n, int64_t col0, float2 *part,
                                    cudaStream_t st) {
    xent::piece_stats_kernel<<<static_cast<unsigned>(a.tokens), xent::ROW_THREADS, 0, st>>>(a, logits, n, col0, part);
    return cudaGetLastError();
}

cudaError_t launch_xent_piece_grad(bool is_bf16, const RowArgs &a, const float *logits, int64_t n, int64_t col0,
                                   const float *lse, const float *row_g, void *out, cudaStream_t st) {
    const unsigned grid = static_cast<unsigned>(a.tokens);
    if (is_bf16)
        xent::piece_grad_kernel<<<grid, xent::ROW_THREADS, 0, st>>>(a, logits, n, col0, lse, row_g,
                                                                    static_cast<__nv_bfloat16 *>(out));
    else
        xent::piece_grad_kernel<<<grid, xent::ROW_THREADS, 0, st>>>(a, logits, n, col0, lse, row_g,
                                                                    static_cast<float *>(out));
    return cudaGetLastError();
}

}  // namespace tpmlp
