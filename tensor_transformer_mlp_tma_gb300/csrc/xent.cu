// Row kernels of the vocabulary cross entropy (the products run in tc_gemm.cu and
// simt_gemm.cu).  With logits S = X W^T [T, V], per token
//   lse = log sum_v exp S_v,   loss = lse - S_y,   dS = (exp(S - lse) - 1[y]) g.
// No [T, V] array exists: the product's epilogue leaves one (max, sum of
// exponentials) pair per token and 16 to 128 vocabulary rows, which combine_kernel joins.
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
    s = s * __expf(m - base) + s2 * __expf(m2 - base);
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

__device__ __forceinline__ void finish_row(const RowArgs &a, int64_t row, float m, float s, float *loss, float *lse) {
    const float l = logf(s);
    lse[row] = m + l;
    // the difference of the two large terms first, then the small one
    loss[row] = target_ok(a, row) ? (m - __ldcg(a.target_logit + row)) + l : 0.0f;
}

// The last block of a grid to get here joins the blocks' pairs of up to 8 tokens, in order, a
// warp per token.  status[2] counts the blocks; the last one sets it back to zero.
__device__ __forceinline__ void last_block_joins(const RowArgs &a, float *loss, float *lse) {
    __shared__ bool last;
    __threadfence();  // this thread's partials and target logits, before its block is counted
    __syncthreads();
    if (threadIdx.x == 0) last = atomicAdd(a.status + 2, 1u) == gridDim.x - 1;
    __syncthreads();
    if (!last) return;
    __threadfence();
    if (threadIdx.x == 0) a.status[2] = 0u;
    const int lane = threadIdx.x & 31, row = threadIdx.x >> 5;
    if (row >= a.tokens) return;
    float m = -INFINITY, s = 0.0f;
    for (int64_t g = lane; g < gridDim.x; g += 32) {
        const float2 p = __ldcg(a.part + g * a.tokens + row);
        join(m, s, p.x, p.y);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        const float m2 = __shfl_xor_sync(0xffffffffu, m, off), s2 = __shfl_xor_sync(0xffffffffu, s, off);
        join(m, s, m2, s2);
    }
    if (lane == 0) finish_row(a, row, m, s, loss, lse);
}

// loss and lse of 32 tokens per block: lane = token (the partials of one group are
// contiguous over tokens), the warps take every 32nd group and join theirs through
// shared memory, in a fixed order.  Reads 8 bytes per token and 128 vocabulary rows,
// 1/(32 h) of the product's FLOPs in bytes; bound by latency (7 to 10 us).
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
    if (w == 0 && row < a.tokens) finish_row(a, row, m, s, loss, lse);
}

// ---- few tokens ------------------------------------------------------------------
// Statistics of up to T tokens (one in bf16, up to eight in fp32) in one pass over W: X sits in shared memory, every warp
// streams its share of W's rows, FEW_ROWS at a time, 512 bytes of each per load, and keeps its
// own online softmax.  A product of so few rows would waste the tensor core's tile, and
// its copies of 128-byte pieces of many rows read W at 3.2 to 3.6 TB/s (T = 1 to 8).
// Bound by W's bytes: h = 4096, V = 32768 in 47 us (5.7 TB/s) at T = 1, h = 8192, V = 50000
// at 6.4 TB/s.
// The backward pass runs the same kernels (GRAD) for dS, so that its logits are those of lse to
// the bit: 1 - p of a confident token is then as exact as the logits' differences.
constexpr int FEW_THREADS = 512, FEW_ROWS = 4;

// One token's row of dS, element by element.
struct GradRow {
    float lse, g;
    int64_t tcol;  // the target's column of this piece
};
__device__ __forceinline__ GradRow grad_row(const RowArgs &a, const FewGrad &d, int64_t t, float unit) {
    GradRow r = {0.0f, 0.0f, -1};
    if (t >= a.tokens) return r;
    const int64_t y = a.target[t];
    r.lse = d.lse[t];
    if (y != a.ignore_index && y >= 0 && y < d.all_vocab) r.g = __fdiv_rn(d.dloss[t], unit), r.tcol = y - d.col0;
    return r;
}
__device__ __forceinline__ float grad_unit(const RowArgs &a, const FewGrad &d) {
    const float unit = xent_find_unit(a.target, d.dloss, a.tokens, a.ignore_index, d.all_vocab);
    if (blockIdx.x == 0 && threadIdx.x == 0) *d.unit = unit;
    return unit;
}
template <typename E>
__device__ __forceinline__ void grad_put(const FewGrad &d, const GradRow &r, int64_t t, int64_t col, float z) {
    const float p = __expf(z - r.lse);
    float v = r.g == 0.0f ? 0.0f : (col == r.tcol ? p - 1.0f : p) * r.g;
    __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(d.out) + t * d.ld + col;
    if constexpr (sizeof(E) == 2) {
        *out = __float2bfloat16_rn(v);
    } else {
#pragma unroll
        for (int k = 0; k < 3; ++k, out += d.part) {
            const __nv_bfloat16 h = __float2bfloat16_rn(v);
            *out = h;
            v -= __bfloat162float(h);
        }
    }
}

// EC consecutive elements as fp32 pairs.
template <typename E, int EC>
struct Chunk;
template <>
struct Chunk<__nv_bfloat16, 8> {
    uint4 w;
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) { w = *reinterpret_cast<const uint4 *>(p); }
    __device__ __forceinline__ void stream(const __nv_bfloat16 *p) { w = __ldcs(reinterpret_cast<const uint4 *>(p)); }
    __device__ __forceinline__ void zero() { w = make_uint4(0u, 0u, 0u, 0u); }
    __device__ __forceinline__ float2 pair(int i) const {
        const uint32_t u = i == 0 ? w.x : (i == 1 ? w.y : (i == 2 ? w.z : w.w));
        return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xFFFF0000u));
    }
};
template <>
struct Chunk<float, 4> {
    float4 w;
    __device__ __forceinline__ void load(const float *p) { w = *reinterpret_cast<const float4 *>(p); }
    __device__ __forceinline__ void stream(const float *p) { w = __ldcs(reinterpret_cast<const float4 *>(p)); }
    __device__ __forceinline__ void zero() { w = make_float4(0.0f, 0.0f, 0.0f, 0.0f); }
    __device__ __forceinline__ float2 pair(int i) const {
        return i == 0 ? make_float2(w.x, w.y) : make_float2(w.z, w.w);
    }
};
template <>
struct Chunk<float, 1> {  // rows that do not start on 16 bytes
    float w;
    __device__ __forceinline__ void load(const float *p) { w = *p; }
    __device__ __forceinline__ void stream(const float *p) { w = __ldcs(p); }
    __device__ __forceinline__ void zero() { w = 0.0f; }
    __device__ __forceinline__ float2 pair(int) const { return make_float2(w, 0.0f); }
};

template <typename E, int EC, int T, bool GRAD>
__global__ void __launch_bounds__(FEW_THREADS, 1) few_kernel(const RowArgs a, const E *X, const E *W, int64_t h,
                                                            float2 *part, float *loss, float *lse, const FewGrad d) {
    extern __shared__ __align__(16) uint8_t few_smem[];
    E *xs = reinterpret_cast<E *>(few_smem);  // [T][h]
    __shared__ float2 sh[FEW_THREADS / 32][T];
    constexpr int N = FEW_ROWS * T, LOG = N == 4 ? 2 : (N == 8 ? 3 : (N == 16 ? 4 : 5)), PAIRS = EC == 1 ? 1 : EC / 2;
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    for (int64_t i = static_cast<int64_t>(threadIdx.x) * EC; i < T * h; i += FEW_THREADS * EC) {
        Chunk<E, EC> c;
        if (i < a.tokens * h)
            c.load(X + i);
        else
            c.zero();
        *reinterpret_cast<Chunk<E, EC> *>(xs + i) = c;
    }
    __syncthreads();
    // This warp's rows of W, a contiguous share.
    const int64_t warps = static_cast<int64_t>(gridDim.x) * (FEW_THREADS / 32);
    const int64_t id = static_cast<int64_t>(blockIdx.x) * (FEW_THREADS / 32) + w;
    const int64_t beg = a.vocab * id / warps, end = a.vocab * (id + 1) / warps;
    // After the reduction below lane l holds sum number l >> (5 - LOG): row / T, token % T.
    const int mine = lane >> (5 - LOG), my_row = mine / T, my_t = mine % T;
    int64_t target = -1;
    GradRow gr;
    if constexpr (GRAD) {
        // in fp32 dS keeps all its bits, and needs no unit
        gr = grad_row(a, d, my_t, sizeof(E) == 2 ? grad_unit(a, d) : 1.0f);
    } else if (my_t < a.tokens) {
        target = a.target[my_t];
        if (target == a.ignore_index) target = -1;
    }
    float m = -INFINITY, s = 0.0f;
    for (int64_t r0 = beg; r0 < end; r0 += FEW_ROWS) {
        float2 acc[N];
#pragma unroll
        for (int i = 0; i < N; ++i) acc[i] = make_float2(0.0f, 0.0f);
        const E *rows = W + r0 * h;
        const int n = static_cast<int>(min(static_cast<int64_t>(FEW_ROWS), end - r0));
#pragma unroll 2
        for (int64_t c = lane * EC; c < h; c += 32 * EC) {
            Chunk<E, EC> b[FEW_ROWS];
#pragma unroll
            for (int i = 0; i < FEW_ROWS; ++i) {
                if (i < n)
                    b[i].stream(rows + i * h + c);
                else
                    b[i].zero();
            }
#pragma unroll
            for (int t = 0; t < T; ++t) {
                Chunk<E, EC> x;
                x.load(xs + t * h + c);
#pragma unroll
                for (int j = 0; j < PAIRS; ++j) {
                    const float2 xv = x.pair(j);
#pragma unroll
                    for (int i = 0; i < FEW_ROWS; ++i)
                        acc[i * T + t] = ptx::fma2(b[i].pair(j), xv, acc[i * T + t]);
                }
            }
        }
        // Every lane has a share of all N sums; each exchange halves how many sums a lane
        // is concerned with.
        float v[N];
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = acc[i].x + acc[i].y;
#pragma unroll
        for (int q = 0; q < 5; ++q) {
            const int off = 16 >> q;
            if (q < LOG) {
                const int half = N >> (q + 1);
#pragma unroll
                for (int i = 0; i < half; ++i) {
                    const float send = (lane & off) ? v[i] : v[i + half];
                    const float keep = (lane & off) ? v[i + half] : v[i];
                    v[i] = keep + __shfl_xor_sync(0xffffffffu, send, off);
                }
            } else {
                v[0] += __shfl_xor_sync(0xffffffffu, v[0], off);
            }
        }
        if constexpr (GRAD) {
            // 2^(5 - LOG) lanes hold each sum
            if (my_row < n && my_t < a.tokens && (lane & (31 >> LOG)) == 0) grad_put<E>(d, gr, my_t, r0 + my_row, v[0]);
        } else if (my_row < n) {
            join(m, s, v[0], 1.0f);
            if (target == r0 + my_row) a.target_logit[my_t] = v[0];
        }
    }
    if constexpr (GRAD) return;
    // the rows of one token sit in lanes that differ in bits 4 and 3
#pragma unroll
    for (int off = 16; off >= 8; off >>= 1) {
        const float m2 = __shfl_xor_sync(0xffffffffu, m, off), s2 = __shfl_xor_sync(0xffffffffu, s, off);
        join(m, s, m2, s2);
    }
    if (mine < T) sh[w][mine] = make_float2(m, s);
    __syncthreads();
    if (threadIdx.x < a.tokens) {
        float2 p = sh[0][threadIdx.x];
        for (int i = 1; i < FEW_THREADS / 32; ++i) join(p.x, p.y, sh[i][threadIdx.x].x, sh[i][threadIdx.x].y);
        part[static_cast<int64_t>(blockIdx.x) * a.tokens + threadIdx.x] = p;
    }
    last_block_joins(a, loss, lse);
}

// The same for 2 to 8 bf16 tokens, where one FMA per weight and token would cost more than
// W's bytes: warp products of 16 rows of W with 8 tokens.  A dot product does not
// care in which order k comes, so each lane loads 16 contiguous bytes of two rows and
// takes them as its share of two 16-deep products, with the tokens' values at the same
// places; no shuffling, no staging of W.  The warps of a block share a group of 16
// rows by slices of k and add their sums in order through shared memory, so that the
// blocks' shares of the vocabulary stay even; two buffers let one barrier per group do.
// 51 us (5.3 TB/s) for T = 8, h = 4096, V = 32768, where one FMA per weight and token took 78.
// With 16 or 32 tokens the same kernel was no faster than the tcgen05 tiles.
constexpr int SLIM_ROWS = 16;

template <int SLIM_WARPS, bool GRAD>
__global__ void __launch_bounds__(32 * SLIM_WARPS, 16 / SLIM_WARPS) slim_kernel(const RowArgs a, const __nv_bfloat16 *X,
                                                              const __nv_bfloat16 *W, int64_t h, int hp,
                                                              float2 *part, float *loss, float *lse, const FewGrad fg) {
    extern __shared__ __align__(16) uint8_t slim_smem[];
    // [8][hp], hp = h rounded up to 32, and 8 more: a row's 16-byte pieces then start 4
    // banks after the row before, and the eight tokens that a load touches do not collide
    __nv_bfloat16 *xs = reinterpret_cast<__nv_bfloat16 *>(slim_smem);
    __shared__ float4 sums[2][SLIM_WARPS][32];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, q = lane & 3, r = lane >> 2;
    const int ld = hp + 8;
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    for (int i = threadIdx.x * 8; i < 8 * hp; i += 256 * SLIM_WARPS) {
        const int t = i / hp, c = i - t * hp;
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (t < a.tokens && c < h) v = *reinterpret_cast<const uint4 *>(X + t * h + c);
        *reinterpret_cast<uint4 *>(xs + t * ld + c) = v;
    }
    __syncthreads();
    int64_t target[2];
    float m[2], s[2];
    GradRow gr[2];
    float unit = 1.0f;
    if constexpr (GRAD) unit = grad_unit(a, fg);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int t = 2 * q + j;
        target[j] = -1;
        if constexpr (GRAD)
            gr[j] = grad_row(a, fg, t, unit);
        else if (t < a.tokens && a.target[t] != a.ignore_index) target[j] = a.target[t];
        m[j] = -INFINITY, s[j] = 0.0f;
    }
    int it = 0;
    for (int64_t r0 = static_cast<int64_t>(blockIdx.x) * SLIM_ROWS; r0 < a.vocab;
         r0 += static_cast<int64_t>(gridDim.x) * SLIM_ROWS, ++it) {
        const int rows = static_cast<int>(min(static_cast<int64_t>(SLIM_ROWS), a.vocab - r0));
        const __nv_bfloat16 *row0 = W + (r0 + r) * h + 8 * q, *row1 = row0 + 8 * h;
        const bool in0 = r < rows, in1 = r + 8 < rows;
        float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 8
        for (int c = 32 * w; c < hp; c += 32 * SLIM_WARPS) {
            const bool in = c + 8 * q < h;
            uint4 u = make_uint4(0u, 0u, 0u, 0u), v = u;
            if (in && in0) u = __ldcs(reinterpret_cast<const uint4 *>(row0 + c));
            if (in && in1) v = __ldcs(reinterpret_cast<const uint4 *>(row1 + c));
            const uint4 x = *reinterpret_cast<const uint4 *>(xs + r * ld + c + 8 * q);
            ptx::mma_bf16_16x8x16(d, u.x, v.x, u.y, v.y, x.x, x.y);
            ptx::mma_bf16_16x8x16(d, u.z, v.z, u.w, v.w, x.z, x.w);
        }
        const int buf = it & 1;
        sums[buf][w][lane] = make_float4(d[0], d[1], d[2], d[3]);
        __syncthreads();
        if (it % SLIM_WARPS == w) {  // the warps take turns
            float4 v = sums[buf][0][lane];
            for (int k = 1; k < SLIM_WARPS; ++k) {
                const float4 o = sums[buf][k][lane];
                v.x += o.x, v.y += o.y, v.z += o.z, v.w += o.w;
            }
            const float z[4] = {v.x, v.y, v.z, v.w};  // (row r, tokens 2q, 2q + 1), (row r + 8, the same)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int row = r + 8 * (j >> 1);
                if constexpr (GRAD) {
                    const int t = 2 * q + (j & 1);
                    if (row < rows && t < a.tokens) grad_put<__nv_bfloat16>(fg, gr[j & 1], t, r0 + row, z[j]);
                } else if (row < rows) {
                    join(m[j & 1], s[j & 1], z[j], 1.0f);
                    if (target[j & 1] == r0 + row) a.target_logit[2 * q + (j & 1)] = z[j];
                }
            }
        }
    }
    if constexpr (GRAD) return;
    // One token's rows: 8 lanes of every warp.
    float2 *all = reinterpret_cast<float2 *>(&sums[0][0][0]);  // [SLIM_WARPS][8]
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 2; ++j) {
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) {
            const float m2 = __shfl_xor_sync(0xffffffffu, m[j], off), s2 = __shfl_xor_sync(0xffffffffu, s[j], off);
            join(m[j], s[j], m2, s2);
        }
        if (r == 0) all[w * 8 + 2 * q + j] = make_float2(m[j], s[j]);
    }
    __syncthreads();
    if (threadIdx.x < a.tokens) {
        float2 p = all[threadIdx.x];
        for (int k = 1; k < SLIM_WARPS; ++k) join(p.x, p.y, all[k * 8 + threadIdx.x].x, all[k * 8 + threadIdx.x].y);
        part[static_cast<int64_t>(blockIdx.x) * a.tokens + threadIdx.x] = p;
    }
    last_block_joins(a, loss, lse);
}

// Fixed-order sum of the fp32 matrices that split products left, rounded once to the
// output's type.  V columns per thread.  Memory bound: 4 bytes per split and element.
template <typename T, int V>
__global__ void __launch_bounds__(256) sum_splits_kernel(const float *in, int splits, int64_t rows, int64_t cols,
                                                         int64_t ld, const float *unit_at, T *out) {
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const float unit = unit_at ? *unit_at : 1.0f;
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
#pragma unroll
        for (int j = 0; j < V; ++j) v[j] *= unit;
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

// x = p0 + p1 + p2 in bf16, each the rest before it rounded to eight bits, so that the
// three together hold all 24 (the largest fp32 numbers, which would round up to
// infinity, are cut off instead; an infinite one has parts inf, 0, 0).  Two matrices in one
// launch, a warp per row, four columns per lane.  Memory bound: 4 bytes read, 6 written
// per element.
__device__ __forceinline__ void split3(const Split3 &m, int64_t r, int lane) {
    const float *in = m.in + r * m.cols;
    const bool vec = m.cols % 4 == 0 && (reinterpret_cast<uintptr_t>(m.in) & 15) == 0;
    __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(m.out) + r * m.ld;
    const int64_t all = m.rows * m.ld;
#pragma unroll 4
    for (int64_t c = 4 * lane; c < m.ld; c += 128) {
        float v[4];
        if (vec && c < m.cols) {
            const float4 w = __ldg(reinterpret_cast<const float4 *>(in + c));
            v[0] = w.x, v[1] = w.y, v[2] = w.z, v[3] = w.w;
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = c + j < m.cols ? in[c + j] : 0.0f;
        }
        // numbers that no rounding makes infinite (all but the very largest, inf and NaN)
        const bool ordinary = fmaxf(fmaxf(fabsf(v[0]), fabsf(v[1])), fmaxf(fabsf(v[2]), fabsf(v[3]))) < 0x1p127f &&
                              v[0] == v[0] && v[1] == v[1] && v[2] == v[2] && v[3] == v[3];
#pragma unroll
        for (int part = 0; part < 3; ++part) {
            __nv_bfloat162 h[2] = {__floats2bfloat162_rn(v[0], v[1]), __floats2bfloat162_rn(v[2], v[3])};
            if (!ordinary) {
                __nv_bfloat16 *p = reinterpret_cast<__nv_bfloat16 *>(h);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (__hisinf(p[j]) && !isinf(v[j])) p[j] = __float2bfloat16_rz(v[j]);
            }
            const float2 lo = __bfloat1622float2(h[0]), up = __bfloat1622float2(h[1]);
            const float w[4] = {lo.x, lo.y, up.x, up.y};
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = !ordinary && isinf(v[j]) ? 0.0f : v[j] - w[j];
            *reinterpret_cast<uint2 *>(out + part * all + c) = *reinterpret_cast<const uint2 *>(h);
        }
    }
}
__global__ void __launch_bounds__(256) split3_kernel(const Split3 a, const Split3 b) {
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const int lane = threadIdx.x & 31;
    for (int64_t r = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5); r < a.rows + b.rows;
         r += static_cast<int64_t>(gridDim.x) * 8) {
        if (r < a.rows)
            split3(a, r, lane);
        else
            split3(b, r - a.rows, lane);
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
                                                                int64_t col0, const float *lse, const float *dloss,
                                                                T *out) {
    const int64_t row = blockIdx.x;
    const bool takes_part = a.target[row] != a.ignore_index && a.target[row] >= 0 && a.target[row] < a.vocab;
    const float g = takes_part ? dloss[row] : 0.0f, l = lse[row];
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

// Shared memory of the kernel that takes these tokens: X, for as many tokens as it is built for.
static int64_t few_smem(bool is_bf16, int64_t tokens, int64_t hidden) {
    if (is_bf16) return tokens <= 1 ? hidden * 2 : 8 * ((hidden + 31) / 32 * 32 + 8) * 2;
    return (tokens <= 2 ? tokens : (tokens <= 4 ? 4 : 8)) * hidden * 4;
}

bool xent_few(bool is_bf16, int64_t tokens, int64_t hidden) {
    if (tokens > 8) return false;
    return few_smem(is_bf16, tokens, hidden) <= XENT_FEW_SMEM;
}

int64_t xent_few_groups(int64_t vocab) {
    const int64_t b = (vocab + 15) / 16;
    return b < 304 ? b : 304;
}

namespace {
// What the two passes' launches of a few-token kernel have in common, and what each adds.
struct FewCall {
    RowArgs a;
    const void *X, *W;
    int64_t h;
    float2 *part;
    float *loss, *lse;
    FewGrad grad;
    cudaStream_t st;
};

template <bool GRAD, int WARPS>
cudaError_t launch_slim(const FewCall &c, int64_t smem) {
    auto kernel = xent::slim_kernel<WARPS, GRAD>;
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(XENT_FEW_SMEM));
    if (e != cudaSuccess) return e;
    return launch_pdl(kernel, dim3(static_cast<unsigned>(xent_few_groups(c.a.vocab))), 32 * WARPS,
                      static_cast<size_t>(smem), c.st, c.a, static_cast<const __nv_bfloat16 *>(c.X),
                      static_cast<const __nv_bfloat16 *>(c.W), c.h, static_cast<int>((c.h + 31) / 32 * 32), c.part,
                      c.loss, c.lse, c.grad);
}

template <bool GRAD, typename E, int EC, int T>
cudaError_t launch_few(const FewCall &c) {
    auto kernel = xent::few_kernel<E, EC, T, GRAD>;
    const size_t smem = static_cast<size_t>(T) * c.h * sizeof(E);
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(XENT_FEW_SMEM));
    if (e != cudaSuccess) return e;
    return launch_pdl(kernel, dim3(static_cast<unsigned>(xent_few_groups(c.a.vocab))), xent::FEW_THREADS, smem, c.st,
                      c.a, static_cast<const E *>(c.X), static_cast<const E *>(c.W), c.h, c.part, c.loss, c.lse, c.grad);
}

template <bool GRAD, typename E, int EC>
cudaError_t launch_few_t(const FewCall &c) {
    if (c.a.tokens <= 1) return launch_few<GRAD, E, EC, 1>(c);
    if (c.a.tokens <= 2) return launch_few<GRAD, E, EC, 2>(c);
    if (c.a.tokens <= 4) return launch_few<GRAD, E, EC, 4>(c);
    return launch_few<GRAD, E, EC, 8>(c);
}

// The choice depends on the tokens, h and the alignment alone, so that both passes and every
// piece of W (whose rows of 16 bytes start on 16 bytes) take the same kernel.
template <bool GRAD>
cudaError_t launch_few_any(bool is_bf16, const FewCall &c) {
    if (is_bf16) {
        if (c.a.tokens <= 1) return launch_few<GRAD, __nv_bfloat16, 8, 1>(c);
        // 16 warps per SM: two blocks, of which one computes while the other is at its barrier,
        // where two copies of X leave room for the loads in L1; one block of all 16 warps where
        // they do not (T = 4, V = 50000: h = 6144 4.4 TB/s with two blocks, h = 8192 5.8 with one).
        const int64_t smem = few_smem(true, c.a.tokens, c.h);
        return smem <= 72 * 1024 ? launch_slim<GRAD, 8>(c, smem) : launch_slim<GRAD, 16>(c, smem);
    }
    const uintptr_t both = reinterpret_cast<uintptr_t>(c.X) | reinterpret_cast<uintptr_t>(c.W);
    if (c.h % 4 == 0 && (both & 15) == 0) return launch_few_t<GRAD, float, 4>(c);
    return launch_few_t<GRAD, float, 1>(c);
}
}  // namespace

cudaError_t launch_xent_few(bool is_bf16, const RowArgs &a, const void *X, const void *W, int64_t h, float2 *part,
                            float *loss, float *lse, cudaStream_t st) {
    return launch_few_any<false>(is_bf16, {a, X, W, h, part, loss, lse, {}, st});
}

cudaError_t launch_xent_few_grad(bool is_bf16, const RowArgs &a, const void *X, const void *W, int64_t h,
                                 const FewGrad &d, cudaStream_t st) {
    return launch_few_any<true>(is_bf16, {a, X, W, h, nullptr, nullptr, nullptr, d, st});
}

cudaError_t launch_sum_splits(bool is_bf16, const float *in, int splits, int64_t rows, int64_t cols, int64_t ld,
                              const float *unit, void *out, cudaStream_t st) {
    const bool vec = cols % 4 == 0 && ld % 4 == 0 && (reinterpret_cast<uintptr_t>(out) & 15) == 0;
    const int64_t blocks = xent::blocks_for(rows * cols / (vec ? 4 : 1));
    if (is_bf16) {
        auto o = static_cast<__nv_bfloat16 *>(out);
        return vec ? launch_pdl(xent::sum_splits_kernel<__nv_bfloat16, 4>, dim3(static_cast<unsigned>(blocks)), 256, 0, st, in, splits, rows, cols, ld, unit, o)
                   : launch_pdl(xent::sum_splits_kernel<__nv_bfloat16, 1>, dim3(static_cast<unsigned>(blocks)), 256, 0, st, in, splits, rows, cols, ld, unit, o);
    }
    auto o = static_cast<float *>(out);
    return vec ? launch_pdl(xent::sum_splits_kernel<float, 4>, dim3(static_cast<unsigned>(blocks)), 256, 0, st, in, splits, rows, cols, ld, unit, o)
               : launch_pdl(xent::sum_splits_kernel<float, 1>, dim3(static_cast<unsigned>(blocks)), 256, 0, st, in, splits, rows, cols, ld, unit, o);
}

cudaError_t launch_split3(const Split3 &a, const Split3 &b, cudaStream_t st) {
    const int64_t blocks = xent::blocks_for((a.rows + b.rows) * 32);
    return launch_pdl(xent::split3_kernel, dim3(static_cast<unsigned>(blocks)), 256, 0, st, a, b);
}

cudaError_t launch_xent_piece_stats(const RowArgs &a, const float *logits, int64_t n, int64_t col0, float2 *part,
                                    cudaStream_t st) {
    xent::piece_stats_kernel<<<static_cast<unsigned>(a.tokens), xent::ROW_THREADS, 0, st>>>(a, logits, n, col0, part);
    return cudaGetLastError();
}

cudaError_t launch_xent_piece_grad(bool is_bf16, const RowArgs &a, const float *logits, int64_t n, int64_t col0,
                                   const float *lse, const float *dloss, void *out, cudaStream_t st) {
    const unsigned grid = static_cast<unsigned>(a.tokens);
    if (is_bf16)
        xent::piece_grad_kernel<<<grid, xent::ROW_THREADS, 0, st>>>(a, logits, n, col0, lse, dloss,
                                                                    static_cast<__nv_bfloat16 *>(out));
    else
        xent::piece_grad_kernel<<<grid, xent::ROW_THREADS, 0, st>>>(a, logits, n, col0, lse, dloss,
                                                                    static_cast<float *>(out));
    return cudaGetLastError();
}

}  // namespace tpmlp
