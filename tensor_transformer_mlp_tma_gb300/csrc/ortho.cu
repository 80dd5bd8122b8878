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
// The limits and scales leave room for 2^34 squares of the largest value of each kind (2^126, 2^122,
// 2^106 in all), and the square of the smallest subnormal number is a normal one (2^-114).
constexpr float kBig = 0x1p46f, kSmall = 0x1p-56f;      // limits of the ordinary values
constexpr float kBigScale = 0x1p-84f, kSmallScale = 0x1p92f;
// N values at once, all into the sum that the largest of them belongs to: beside a value of
// 2^-56 or more, what underflows (below 2^-74) is too small to count.
template <int N>
__device__ __forceinline__ void add(Blue &b, const float (&x)[N]) {
    float m = 0.0f;
#pragma unroll
    for (int j = 0; j < N; ++j) m = fmaxf(m, fabsf(x[j]));
    if (m <= kBig && m >= kSmall) {
#pragma unroll
        for (int j = 0; j < N; ++j) b.mid = fmaf(x[j], x[j], b.mid);
    } else {
        const bool big = m > kBig;  // also +-inf; a NaN beside small values goes with them
        const float f = big ? kBigScale : kSmallScale;
        float s = big ? b.big : b.small;
#pragma unroll
        for (int j = 0; j < N; ++j) s = fmaf(x[j] * f, x[j] * f, s);
        (big ? b.big : b.small) = s;
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

// Sums over the block, in the same order in every block that asks.
__device__ __forceinline__ Blue block_sum(Blue b) {
    __shared__ Blue sh[THREADS / 32];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        b.big += __shfl_xor_sync(0xffffffffu, b.big, o);
        b.mid += __shfl_xor_sync(0xffffffffu, b.mid, o);
        b.small += __shfl_xor_sync(0xffffffffu, b.small, o);
    }
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = b;
    __syncthreads();
    b = sh[0];
#pragma unroll
    for (int w = 1; w < THREADS / 32; ++w) b.big += sh[w].big, b.mid += sh[w].mid, b.small += sh[w].small;
    return b;
}

// Block sums of squares: blocks blockIdx.x = 0.. of matrix blockIdx.y, each over a
// contiguous range.  VEC: 16-byte loads (the matrix starts and ends on 16 bytes).
// Memory bound: one read of G (4096 x 16384 in bf16: 31 us, 4.3 TB/s).
template <typename T, bool VEC>
__device__ __forceinline__ Blue sum_of_squares(const T *g, int64_t beg, int64_t end) {
    Blue b{0.0f, 0.0f, 0.0f};
    if constexpr (VEC) {
        constexpr int E = 16 / sizeof(T);
        constexpr int UN = 4;  // loads in flight before the first is used
        for (int64_t i = beg + threadIdx.x * E; i < end; i += UN * THREADS * E) {
            uint4 w[UN];
#pragma unroll
            for (int u = 0; u < UN; ++u)
                w[u] = i + u * THREADS * E < end ? __ldg(reinterpret_cast<const uint4 *>(g + i + u * THREADS * E))
                                                 : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
            for (int u = 0; u < UN; ++u) {
                const T *v = reinterpret_cast<const T *>(&w[u]);
                float x[E];
#pragma unroll
                for (int j = 0; j < E; ++j) x[j] = value<T>(v[j]);
                add(b, x);
            }
        }
    } else {
#pragma unroll 4
        for (int64_t i = beg + threadIdx.x; i < end; i += THREADS) {
            const float x[1] = {value<T>(g[i])};
            add(b, x);
        }
    }
    return b;
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(THREADS) norm_kernel(const T *G, int64_t n, int64_t per_block, Blue *part) {
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const T *g = G + static_cast<int64_t>(blockIdx.y) * n;
    const int64_t beg = static_cast<int64_t>(blockIdx.x) * per_block, end = min(beg + per_block, n);
    Blue b = sum_of_squares<T, VEC>(g, beg, end);
    b = block_sum(b);
    if (threadIdx.x == 0) part[static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x] = b;
}

// scale / (|G| + eps) from the three sums, as the product of f and the power of two `unit`.  The norm is
// sqrt(s) / unit, s the sum in the largest unit that has any (a sum two units down could not
// count); x unit f then neither overflows nor loses bits that count, whatever the norm: unit
// moves all values towards the ordinary ones.  fp32 throughout: 64-bit arithmetic here took
// longer than a block's share of the matrix.
// With POW2 f is the power of two below it, and `rest` (1 to 2) is what is left.
template <bool POW2>
__device__ __forceinline__ float inverse_norm(const Blue &b, float eps, float scale, float &unit, float &rest) {
    float s;
    if (b.big > 0.0f)
        s = b.big + b.mid * kBigScale * kBigScale, unit = kBigScale;
    else if (b.mid == 0.0f && b.small > 0.0f)
        s = b.small, unit = kSmallScale;
    else
        s = b.mid + b.small * (1.0f / kSmallScale) * (1.0f / kSmallScale), unit = 1.0f;
    if (b.big != b.big || b.mid != b.mid || b.small != b.small) s = nanf("");
    float f = __fdiv_rn(scale, __fsqrt_rn(s) + eps * unit);
    if (f > 0x1p127f) f = 0x1p127f;  // a zero matrix with eps = 0; not NaN
    rest = 1.0f;
    if (POW2 && f >= 0x1p-126f) {
        const float p = __uint_as_float(__float_as_uint(f) & 0x7F800000u);
        rest = f / p;
        f = p;
    }
    return f;
}

// hi and lo of 8 consecutive columns per thread; grid.y is the matrix.  Memory bound: G read
// once more, 4 bytes written per element (4096 x 16384: 86 us, 4.7 TB/s), or 2: with POW2
// (lo may then be null) X is scaled by the power of two below the factor, which leaves
// bf16 values exact in fp16 and their low part zero, and the rest of the factor goes to
// rest[matrix].
template <typename T, bool VEC, bool POW2>
__global__ void __launch_bounds__(THREADS) scale_kernel(const T *G, int64_t rows, int64_t cols, int64_t P, int64_t Q,
                                                        const Blue *part, int nparts, float eps, float scale,
                                                        __half *hi, __half *lo, float lo_scale, float *rest) {
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const int64_t z = blockIdx.y;
    Blue b{0.0f, 0.0f, 0.0f};
    for (int i = threadIdx.x; i < nparts; i += THREADS) {
        const Blue p = part[z * nparts + i];
        b.big += p.big, b.mid += p.mid, b.small += p.small;
    }
    float left, unit;
    const float f = inverse_norm<POW2>(block_sum(b), eps, scale, unit, left);
    if (POW2 && blockIdx.x == 0 && threadIdx.x == 0) rest[z] = left;
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
                const float x = v[u][j] * unit * f;
                h[j] = __float2half_rn(x);
                l[j] = __float2half_rn((x - __half2float(h[j])) * lo_scale);
            }
            const int64_t o = z * P * Q + static_cast<int64_t>(i) * 8;
            *reinterpret_cast<uint4 *>(hi + o) = *reinterpret_cast<const uint4 *>(h);
            if (!POW2 || lo) *reinterpret_cast<uint4 *>(lo + o) = *reinterpret_cast<const uint4 *>(l);
        }
    }
}

// The splits' sum of one 32 x 32 piece of A's lower triangle per block, stored where it is
// and transposed.  Memory bound: 4 bytes per split and element of the triangle, 4 written.
__global__ void __launch_bounds__(THREADS) gram_sum_kernel(const float *in, int splits, int64_t p, float scale,
                                                           __half *A) {
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    if (blockIdx.x > blockIdx.y) return;  // above the diagonal
    __shared__ float t[32][33];
    const int64_t step = static_cast<int64_t>(gridDim.z) * p * p, at = blockIdx.z * p * p;
    const int64_t r0 = blockIdx.y * 32, c0 = blockIdx.x * 32;
    const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float *src = in + at + (r0 + y + 8 * k) * p + c0 + x;
        float s = 0.0f;
        for (int i = 0; i < splits; ++i) s += src[i * step];
        s *= scale;
        A[at + (r0 + y + 8 * k) * p + c0 + x] = __float2half_rn(s);
        t[y + 8 * k][x] = s;
    }
    if (blockIdx.x == blockIdx.y) return;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 4; ++k) A[at + (c0 + y + 8 * k) * p + r0 + x] = __float2half_rn(t[x][y + 8 * k]);
}

// The last step's result out of its padded array, where the output's rows are not
// multiples of 16 bytes (a TMA store cannot write them).
__global__ void __launch_bounds__(THREADS) unpad_kernel(const __nv_bfloat16 *in, int64_t rows, int64_t cols, int64_t P,
                                                        int64_t Q, __nv_bfloat16 *out) {
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    // a warp per 128 columns of a row: consecutive columns coalesce, four loads at once
    const int64_t z = blockIdx.y;
    const uint32_t segs = static_cast<uint32_t>((cols + 127) / 128), total = static_cast<uint32_t>(rows) * segs;
    const int lane = threadIdx.x & 31;
    for (uint32_t i = blockIdx.x * (THREADS / 32) + (threadIdx.x >> 5); i < total; i += gridDim.x * (THREADS / 32)) {
        const int64_t r = i / segs, c0 = static_cast<int64_t>(i - static_cast<uint32_t>(r) * segs) * 128 + lane;
        const __nv_bfloat16 *src = in + (z * P + r) * Q;
        __nv_bfloat16 *dst = out + (z * rows + r) * cols;
        __nv_bfloat16 v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (c0 + 32 * j < cols) v[j] = src[c0 + 32 * j];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (c0 + 32 * j < cols) dst[c0 + 32 * j] = v[j];
    }
}

static unsigned grid_x(int64_t work, int64_t batch) {
    const int64_t blocks = (work + THREADS - 1) / THREADS;
    const int64_t most = (152 * 8 + batch - 1) / batch;
    return static_cast<unsigned>(blocks < most ? blocks : most);
}

template <typename T>
static cudaError_t launch_start(const OrthoStart &a, bool norm, cudaStream_t st) {
    const int64_t n = a.rows * a.cols;
    const T *G = static_cast<const T *>(a.G);
    const bool aligned = (reinterpret_cast<uintptr_t>(G) & 15) == 0;
    const bool vec_all = aligned && n * sizeof(T) % 16 == 0;
    const bool vec_rows = aligned && a.cols % 8 == 0;
    const int64_t nb = ortho_norm_blocks(a.batch, n);
    const int64_t per = ((n + nb - 1) / nb + 15) / 16 * 16;
    const dim3 gn(static_cast<unsigned>(nb), static_cast<unsigned>(a.batch));
    Blue *part = static_cast<Blue *>(a.part);
    if (norm)
        return launch_pdl(vec_all ? norm_kernel<T, true> : norm_kernel<T, false>, gn, THREADS, 0, st, G, n, per, part);
    const dim3 gs(grid_x(a.P * a.Q / 32, a.batch), static_cast<unsigned>(a.batch));
    __half *hi = static_cast<__half *>(a.hi), *lo = static_cast<__half *>(a.lo);
    auto kernel = a.rest ? (vec_rows ? scale_kernel<T, true, true> : scale_kernel<T, false, true>)
                         : (vec_rows ? scale_kernel<T, true, false> : scale_kernel<T, false, false>);
    return launch_pdl(kernel, gs, THREADS, 0, st, G, a.rows, a.cols, a.P, a.Q, part, static_cast<int>(nb), a.eps,
                      a.scale, hi, lo, a.lo_scale, a.rest);
}

}  // namespace ortho

int64_t ortho_norm_blocks(int64_t batch, int64_t n) {
    if (batch < 1) batch = 1;
    const int64_t most = (152 * 4 + batch - 1) / batch, want = (n + 8191) / 8192;
    return want < most ? want : most;
}

cudaError_t launch_ortho_norm(bool is_bf16, const OrthoStart &a, cudaStream_t st) {
    return is_bf16 ? ortho::launch_start<__nv_bfloat16>(a, true, st) : ortho::launch_start<float>(a, true, st);
}
cudaError_t launch_ortho_scale(bool is_bf16, const OrthoStart &a, cudaStream_t st) {
    return is_bf16 ? ortho::launch_start<__nv_bfloat16>(a, false, st) : ortho::launch_start<float>(a, false, st);
}

cudaError_t launch_ortho_gram_sum(const float *in, int splits, int64_t matrices, int64_t p, float scale, void *A,
                                  cudaStream_t st) {
    const dim3 g(static_cast<unsigned>(p / 32), static_cast<unsigned>(p / 32), static_cast<unsigned>(matrices));
    return launch_pdl(ortho::gram_sum_kernel, g, ortho::THREADS, 0, st, in, splits, p, scale, static_cast<__half *>(A));
}

cudaError_t launch_ortho_unpad(const void *in, int64_t batch, int64_t rows, int64_t cols, int64_t P, int64_t Q,
                               void *out, cudaStream_t st) {
    const dim3 g(ortho::grid_x(rows * ((cols + 127) / 128) * 32, batch), static_cast<unsigned>(batch));
    return launch_pdl(ortho::unpad_kernel, g, ortho::THREADS, 0, st, static_cast<const __nv_bfloat16 *>(in), rows, cols,
                      P, Q, static_cast<__nv_bfloat16 *>(out));
}

}  // namespace tpmlp
