// Norm, scaling and padding of the Newton-Schulz orthogonalisation (the products run
// in tc_gemm.cu).  Each matrix G [rows, cols] becomes X = G / (|G|_F + eps), held as
// the sum of two fp16 matrices, hi + lo / lo_scale, of size [P, Q] (rows and cols rounded
// up to 64, the rest zero: zero rows and columns stay zero through every product).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "kernels.h"
#include "launch.cuh"
#include "ptx.cuh"

namespace tpmlp {
namespace ortho {

constexpr int THREADS = 256;

// Sum of squares over the whole fp32 range without overflow or underflow, after
// J. L. Blue, "A portable Fortran program to find the Euclidean norm of a vector"
// (ACM TOMS 4, 1978): large and small values are scaled by powers of two and summed
// apart from the ordinary ones.
struct Blue {
    float big, mid, small;
};
constexpr float kBig = 0x1p48f, kSmall = 0x1p-48f;      // limits of the ordinary values
constexpr float kBigScale = 0x1p-72f, kSmallScale = 0x1p72f;
__device__ __forceinline__ void add(Blue &b, float x) {
    const float ax = fabsf(x);
    if (ax > kBig) {  // also +-inf
        const float y = x * kBigScale;
        b.big = fmaf(y, y, b.big);
    } else if (ax < kSmall) {
        const float y = x * kSmallScale;
        b.small = fmaf(y, y, b.small);
    } else {  // also NaN
        b.mid = fmaf(x, x, b.mid);
    }
}

template <typename T>
__device__ __forceinline__ float value(T x);
template <>
__device__ __forceinline__ float value<float>(float x) {
    return x;
}
template <>
__device__ __forceinline__ float value<__nv_bfloat16>(__nv_bfloat16 x) {
    return __bfloat162float(x);
}

// Block sums of squares: blocks blockIdx.x = 0.. of matrix blockIdx.y, each over a
// contiguous range.  VEC: 16-byte loads (the matrix starts and ends on 16 bytes).
// Memory bound: one read of G.
template <typename T, bool VEC>
__global__ void __launch_bounds__(THREADS) norm_kernel(const T *G, int64_t n, int64_t per_block, Blue *part) {
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const T *g = G + static_cast<int64_t>(blockIdx.y) * n;
    const int64_t beg = static_cast<int64_t>(blockIdx.x) * per_block, end = min(beg + per_block, n);
    Blue b{0.0f, 0.0f, 0.0f};
    if constexpr (VEC) {
        constexpr int E = 16 / sizeof(T);
#pragma unroll 4
        for (int64_t i = beg + threadIdx.x * E; i < end; i += THREADS * E) {
            const uint4 w = __ldg(reinterpret_cast<const uint4 *>(g + i));
            const T *v = reinterpret_cast<const T *>(&w);
#pragma unroll
            for (int j = 0; j < E; ++j) add(b, value<T>(v[j]));
        }
    } else {
#pragma unroll 4
        for (int64_t i = beg + threadIdx.x; i < end; i += THREADS) add(b, value<T>(g[i]));
    }
    __shared__ Blue sh[THREADS / 32];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        b.big += __shfl_xor_sync(0xffffffffu, b.big, o);
        b.mid += __shfl_xor_sync(0xffffffffu, b.mid, o);
        b.small += __shfl_xor_sync(0xffffffffu, b.small, o);
    }
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = b;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < THREADS / 32; ++w) b.big += sh[w].big, b.mid += sh[w].mid, b.small += sh[w].small;
        part[static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x] = b;
    }
}

// scale / (|G| + eps) of one matrix from its block sums, in the same order in every
// block that asks.  The three sums meet in 64 bits, where none of them can overflow.
__device__ __forceinline__ float inverse_norm(const Blue *part, int n, float eps, float scale) {
    __shared__ double sh[THREADS / 32];
    __shared__ float result;
    double s = 0.0;
    for (int i = threadIdx.x; i < n; i += THREADS) {
        const Blue b = part[i];
        s += static_cast<double>(b.mid) + static_cast<double>(b.big) * 0x1p144 + static_cast<double>(b.small) * 0x1p-144;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < THREADS / 32; ++w) s += sh[w];
        // beyond the fp32 range (|G| < 2^-113 with eps = 0) the factor saturates
        result = static_cast<float>(fmin(static_cast<double>(scale) / (sqrt(s) + static_cast<double>(eps)), 0x1p127));
        if (s != s) result = nanf("");
    }
    __syncthreads();
    return result;
}

// hi and lo of 8 consecutive columns per thread; grid.x covers P * Q / 8, grid.y the
// matrices.  Memory bound: G read once more, 4 bytes written per element.
template <typename T, bool VEC>
__global__ void __launch_bounds__(THREADS) scale_kernel(const T *G, int64_t rows, int64_t cols, int64_t P, int64_t Q,
                                                        const Blue *part, int nparts, float eps, float scale,
                                                        __half *hi, __half *lo, float lo_scale) {
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const int64_t z = blockIdx.y;
    const float f = inverse_norm(part + z * nparts, nparts, eps, scale);
    const T *g = G + z * rows * cols;
    // UN loads in flight per thread before the first is used
    constexpr int UN = 4;
    const uint32_t per_row = static_cast<uint32_t>(Q / 8), total = static_cast<uint32_t>(P * Q / 8);
    const uint32_t stride = gridDim.x * THREADS;
    for (uint32_t i0 = blockIdx.x * THREADS + threadIdx.x; i0 < total; i0 += UN * stride) {
        float v[UN][8];
#pragma unroll
        for (int u = 0; u < UN; ++u) {
            const uint32_t i = i0 + u * stride;
            if (i >= total) break;
            const int64_t r = i / per_row, c = (i - static_cast<uint32_t>(r) * per_row) * 8;
            if (VEC && r < rows && c + 8 <= cols) {
                const uint4 *src = reinterpret_cast<const uint4 *>(g + r * cols + c);
                alignas(16) T t[8];
                *reinterpret_cast<uint4 *>(t) = __ldg(src);
                if constexpr (sizeof(T) == 4) *reinterpret_cast<uint4 *>(t + 4) = __ldg(src + 1);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[u][j] = value<T>(t[j]);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) v[u][j] = r < rows && c + j < cols ? value<T>(g[r * cols + c + j]) : 0.0f;
            }
        }
#pragma unroll
        for (int u = 0; u < UN; ++u) {
            const uint32_t i = i0 + u * stride;
            if (i >= total) break;
            alignas(16) __half h[8];
            alignas(16) __half l[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float x = v[u][j] * f;
                h[j] = __float2half_rn(x);
                l[j] = __float2half_rn((x - __half2float(h[j])) * lo_scale);
            }
            const int64_t o = z * P * Q + static_cast<int64_t>(i) * 8;
            *reinterpret_cast<uint4 *>(hi + o) = *reinterpret_cast<const uint4 *>(h);
            *reinterpret_cast<uint4 *>(lo + o) = *reinterpret_cast<const uint4 *>(l);
        }
    }
}

// The last step's result out of its padded array, where the output's rows are not
// multiples of 16 bytes (a TMA store cannot write them).
__global__ void __launch_bounds__(THREADS) unpad_kernel(const __nv_bfloat16 *in, int64_t rows, int64_t cols, int64_t P,
                                                        int64_t Q, __nv_bfloat16 *out) {
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    // a warp per row: its loads and stores of consecutive columns coalesce
    const int64_t z = blockIdx.y, warps = static_cast<int64_t>(gridDim.x) * (THREADS / 32);
    for (int64_t r = static_cast<int64_t>(blockIdx.x) * (THREADS / 32) + (threadIdx.x >> 5); r < rows; r += warps) {
        const __nv_bfloat16 *src = in + (z * P + r) * Q;
        __nv_bfloat16 *dst = out + (z * rows + r) * cols;
#pragma unroll 4
        for (int64_t c = threadIdx.x & 31; c < cols; c += 32) dst[c] = src[c];
    }
}

static unsigned grid_x(int64_t work, int64_t batch) {
    const int64_t blocks = (work + THREADS - 1) / THREADS;
    const int64_t most = (152 * 8 + batch - 1) / batch;
    return static_cast<unsigned>(blocks < most ? blocks : most);
}

template <typename T>
static cudaError_t launch_start(const OrthoStart &a, cudaStream_t st) {
    const int64_t n = a.rows * a.cols;
    const T *G = static_cast<const T *>(a.G);
    const bool aligned = (reinterpret_cast<uintptr_t>(G) & 15) == 0;
    const bool vec_all = aligned && n * sizeof(T) % 16 == 0;
    const bool vec_rows = aligned && a.cols % 8 == 0;
    const int64_t nb = ortho_norm_blocks(a.batch, n);
    const int64_t per = ((n + nb - 1) / nb + 15) / 16 * 16;
    const dim3 gn(static_cast<unsigned>(nb), static_cast<unsigned>(a.batch));
    Blue *part = static_cast<Blue *>(a.part);
    cudaError_t e = launch_pdl(vec_all ? norm_kernel<T, true> : norm_kernel<T, false>, gn, THREADS, 0, st, G, n, per, part);
    if (e != cudaSuccess) return e;
    const dim3 gs(grid_x(a.P * a.Q / 32, a.batch), static_cast<unsigned>(a.batch));
    __half *hi = static_cast<__half *>(a.hi), *lo = static_cast<__half *>(a.lo);
    return launch_pdl(vec_rows ? scale_kernel<T, true> : scale_kernel<T, false>, gs, THREADS, 0, st, G, a.rows, a.cols,
                      a.P, a.Q, part, static_cast<int>(nb), a.eps, a.scale, hi, lo, a.lo_scale);
}

}  // namespace ortho

int64_t ortho_norm_blocks(int64_t batch, int64_t n) {
    const int64_t most = (152 * 4 + batch - 1) / batch, want = (n + 8191) / 8192;
    return want < most ? want : most;
}

cudaError_t launch_ortho_start(bool is_bf16, const OrthoStart &a, cudaStream_t st) {
    return is_bf16 ? ortho::launch_start<__nv_bfloat16>(a, st) : ortho::launch_start<float>(a, st);
}

cudaError_t launch_ortho_unpad(const void *in, int64_t batch, int64_t rows, int64_t cols, int64_t P, int64_t Q,
                               void *out, cudaStream_t st) {
    const dim3 g(ortho::grid_x(rows * 32, batch), static_cast<unsigned>(batch));
    return launch_pdl(ortho::unpad_kernel, g, ortho::THREADS, 0, st, static_cast<const __nv_bfloat16 *>(in), rows, cols,
                      P, Q, static_cast<__nv_bfloat16 *>(out));
}

}  // namespace tpmlp
