// Newton-Schulz steps on the Gram matrix alone.  With A_k = X_k X_k^T and
// B_k = a I + b A_k + c A_k^2, the step X_{k+1} = B_k X_k gives
//   A_{k+1} = B_k A_k B_k,   X_n = Q X_0,  Q = B_{n-1} ... B_1 B_0,
// so that n steps on a p x q matrix need X_0 twice, once for A_0 and once for Q X_0, and
// everything between is p x p.  For p <= 128 one CTA per matrix holds A, B and Q in
// shared memory and runs all steps without leaving the SM.
//
// Precision: A holds the squares of X's singular values and Q grows to a^n on the
// small ones, so 11-bit operands would not do.  Every matrix is the sum of two fp16
// matrices (22 bits) and a product is three: hi hi + hi lo + lo hi, in one fp32
// accumulator.  Against 64 bits that leaves errors of 1e-6 (Gaussian matrices) to
// 6e-4 (one singular value 1000 times the others), below the bf16 output's own, for five steps of
// a = 3.4; they grow with the square of the largest factor in Q, which bounds the use of this kernel
// (see ortho_layout).
// All factors are polynomials of A_0 and commute, but their roundings do not: an error
// that couples a large singular value i and a small one j is multiplied by
// B_i B_j (at most about 2.4) in B A B and by B_j^2 (up to 11.8 a step) in A B B, and by
// B_i (below 1) or B_j (3.4) in B Q or Q B.  The other forms lose three digits in
// five steps.
//
// Bound by the tensor core and by latency in turn: a step is three dependent products
// with a trip through tensor memory, registers and shared memory between them (the
// fourth, B Q, runs beside them).  Five steps take 37 us at p = 128, where the four
// products of a step are 3.2 of its 7 us, and 21 us at p = 16; up to 152 matrices at once.
// The fifteen launches that the steps on X itself need took 455 us for 32 matrices of
// 128 x 4096, which are now done in 83 us.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "kernels.h"
#include "launch.cuh"
#include "ptx.cuh"

namespace tpmlp {
namespace chain {

constexpr int PT = NS_CHAIN_P;           // rows and columns of the tile, 128
constexpr int THREADS = 512;             // warp w: TMEM lanes 32 (w % 4).., columns 32 (w / 4)..
// A matrix: two blocks of 64 columns, each 128 rows of the high part and then 128 rows of
// the low part, 128-byte swizzled.  As the second operand of a product the 256 rows of a
// block give hi and lo in one MMA.
constexpr uint32_t PART = PT * 128;      // from the high to the low part
constexpr uint32_t BLOCK = 2 * PART;     // from one block to the next
constexpr uint32_t MAT = 2 * BLOCK;
constexpr size_t SMEM = 3 * MAT + 1024;  // A, B, Q, and alignment
constexpr uint32_t TMEM_COLS = 512;      // two accumulators of 2 x 128 columns
constexpr uint32_t STATUS_TIMEOUT = 4;   // TPMLP_ERR_TIMEOUT

// A is stored times 2^13: its entries are at most 3.6, and 2^-25 / 2^13 is what the two parts
// can miss of the small ones.  B is stored as it is (at most 7.5, and 2^-25 of it is below
// the 22 bits of its large entries), so that a product with B keeps its scale.
constexpr float SA = 8192.0f;

// 32 values of one row, columns col .. col + 31, split into the two parts of the matrix at
// `mat`: 16-byte chunk j of a 128-byte row r sits at chunk j ^ (r & 7).
__device__ __forceinline__ void put(uint32_t mat, int row, int col, const float (&v)[32]) {
    const uint32_t base = mat + static_cast<uint32_t>(col >> 6) * BLOCK + static_cast<uint32_t>(row) * 128u;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        uint32_t h[4], l[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float a = v[8 * j + 2 * i], b = v[8 * j + 2 * i + 1];
            h[i] = ptx::f16x2_satfinite(a, b);
            const __half2 hh = *reinterpret_cast<__half2 *>(&h[i]);
            l[i] = ptx::f16x2_satfinite(a - __low2float(hh), b - __high2float(hh));
        }
        const uint32_t at = base + (static_cast<uint32_t>((((col & 63) >> 3) + j) ^ (row & 7)) << 4);
        ptx::st_shared_v4(at, h[0], h[1], h[2], h[3]);
        ptx::st_shared_v4(at + PART, l[0], l[1], l[2], l[3]);
    }
}

// Descriptor of a 128-byte-swizzled K-major operand; 16 columns on are 32 bytes on.
__device__ __forceinline__ uint64_t operand(uint32_t at) { return ptx::sdesc_sw128(at, 16, 1024); }

// X Y^T for two matrices in shared memory of n columns each (n a multiple of 16), issued by one
// thread: D[0, 128) = X_hi Y_hi^T and D[128, 256) = X_hi Y_lo^T by MMAs of 256 columns, then
// D[128, 256) += X_lo Y_hi^T.  Their sum is the product.  (Three MMAs of 128 columns in the
// place of one of 256 and one of 128 read the operands from shared memory more often
// than the tensor core can take them: 12% of the kernel's time.)
__device__ __forceinline__ void multiply(uint32_t d, uint32_t x, uint32_t y, int n) {
    constexpr uint32_t WIDE = ptx::idesc_f16_f32(PT, 2 * PT, false, false);
    const uint32_t narrow = ptx::idesc_f16_f32(PT, n, false, false);
    const uint64_t xh = operand(x), xl = operand(x + PART), yh = operand(y);
    // the address field counts 16 bytes
    const auto step = [](int k) { return static_cast<uint64_t>((k >> 2) * (BLOCK >> 4) + (k & 3) * 2); };
    for (int k = 0; k < n / 16; ++k) ptx::umma_f16_ss(d, xh + step(k), yh + step(k), WIDE, k > 0);
    for (int k = 0; k < n / 16; ++k) ptx::umma_f16_ss(d + PT, xl + step(k), yh + step(k), narrow, 1u);
}

__global__ void __launch_bounds__(THREADS, 1) chain_kernel(const NsChain c) {
    extern __shared__ uint8_t raw[];
    __shared__ __align__(8) uint64_t bars[3];
    __shared__ uint32_t tmem_sh;
    __shared__ volatile int abort_sh;
    const uint32_t base = (ptx::smem_u32(raw) + 1023u) & ~1023u;
    const uint32_t mA = base, mB = base + MAT, mQ = base + 2 * MAT;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int row = 32 * (warp & 3) + lane, col0 = 32 * (warp >> 2);
    const int n = c.size;
    const bool mine_in = col0 < n;  // warps whose columns are all padding only keep step
    const uint32_t bar[2] = {ptx::smem_u32(&bars[0]), ptx::smem_u32(&bars[1])};
    if (threadIdx.x == 0) {
        ptx::mbar_init(bar[0], 1);
        ptx::mbar_init(bar[1], 1);
        ptx::mbar_init(ptx::smem_u32(&bars[2]), 1);
        abort_sh = 0;
        ptx::fence_mbar_init();
    }
    if (warp == 0) {
        ptx::tmem_alloc(ptx::smem_u32(&tmem_sh), TMEM_COLS);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = tmem_sh;
    const uint32_t mine = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16) + static_cast<uint32_t>(col0);
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();

    // A_0: the sum of the splits' Gram matrices.  They are symmetric, so a thread reads its
    // row as a column and a warp's loads are contiguous.
    const int64_t z = blockIdx.x, P = c.P;
    float A[32];  // times SA
#pragma unroll
    for (int i = 0; i < 32; ++i) A[i] = 0.0f;
    const float rest = c.rest ? c.rest[z] : 1.0f;
    if (row < n && col0 < n) {
        const float *src = c.gram + z * P * P + col0 * P + row;
        for (int s = 0; s < c.splits; ++s, src += c.matrices * P * P)
#pragma unroll
            for (int i = 0; i < 32; ++i) A[i] += src[i * P];
#pragma unroll
        for (int i = 0; i < 32; ++i) A[i] = col0 + i < n ? A[i] * (c.unit * rest * rest * SA) : 0.0f;
    }

    // Each product belongs to one of two barriers; `start` runs once every thread's
    // shared-memory writes and tensor-memory reads before it are done.
    uint32_t phase[2] = {0u, 0u};
    bool ok = true;
    auto start = [&](auto issue) {
        ptx::fence_proxy_async_smem();
        ptx::tc_fence_before();
        __syncthreads();
        if (threadIdx.x == 0) {
            ptx::tc_fence_after();
            issue();
        }
    };
    auto wait = [&](int b) {
        if (!ptx::mbar_wait(bar[b], phase[b], c.wait_ns, &abort_sh)) {
            ok = false;
            abort_sh = 1;
        }
        phase[b] ^= 1u;
        ptx::tc_fence_after();
    };
    auto load = [&](int acc, float (&v)[32]) {
        uint32_t r[32], l[32];
        ptx::tmem_ld_32x32b_x32(mine + static_cast<uint32_t>(acc * 2 * PT), r);
        ptx::tmem_ld_32x32b_x32(mine + static_cast<uint32_t>(acc * 2 * PT + PT), l);
        ptx::tmem_ld_wait(r);
        ptx::tmem_ld_wait(l);
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]) + __uint_as_float(l[i]);
    };
    float v[32];
    put(mA, row, col0, A);
    const bool on_diagonal = (warp & 3) == (warp >> 2);  // this warp's block holds the diagonal
    const float ca = c.b * (1.0f / SA), cs = c.c * (1.0f / (SA * SA));
    // A wait that runs out leaves `ok` false in at least one thread and raises the
    // flag that ends every other wait at once; the steps are then gone through without
    // waiting, so that all threads meet at the same barriers.
    for (int k = 0; k < c.steps; ++k) {
        const bool last = k == c.steps - 1;
        start([&] {
            multiply(tmem, mA, mA, n);
            ptx::umma_commit(bar[0]);
        });
        wait(0);
        if (mine_in) {
            load(0, v);
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = fmaf(cs, v[i], ca * A[i]);
            if (on_diagonal) {
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    if (lane == i) v[i] += c.a;
            }
            put(mB, row, col0, v);
            if (k == 0) {  // Q^T = B_0
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] *= c.q_scale * rest;
                put(mQ, row, col0, v);
            }
        }
        if (k == 0 && last) break;
        // B A first: the chain goes on with it, while Q^T B = (B Q)^T has time until the step's end.
        start([&] {
            if (!last) {
                multiply(tmem, mB, mA, n);
                ptx::umma_commit(bar[0]);
            }
            if (k > 0) {
                multiply(tmem + 2 * PT, mQ, mB, n);
                ptx::umma_commit(bar[1]);
            }
        });
        if (!last) {
            wait(0);
            if (mine_in) {  // B A takes A's place
                load(0, v);
                put(mA, row, col0, v);
            }
            start([&] {
                multiply(tmem, mB, mA, n);  // B (B A)^T = B A B
                ptx::umma_commit(bar[0]);
            });
        }
        if (k > 0) {
            wait(1);
            if (mine_in) {
                load(1, v);
                put(mQ, row, col0, v);
            }
        }
        if (last) break;
        wait(0);
        if (mine_in) {
            load(0, A);
            put(mA, row, col0, A);
        }
    }
    // Given up: once more for the products in flight, so that they do not outlive the
    // shared and tensor memory that they use.
    ok = !__syncthreads_or(!ok);
    if (!ok) {
        if (threadIdx.x == 0) {
            ptx::umma_commit(ptx::smem_u32(&bars[2]));
            ptx::mbar_wait(ptx::smem_u32(&bars[2]), 0, c.wait_ns, nullptr);
            if (c.status && atomicCAS(c.status, 0u, STATUS_TIMEOUT) == 0u) atomicExch(c.status + 1, 8u);
        }
        __syncthreads();
    }

    // Q from Q^T in shared memory, every thread what it wrote itself: element (row, col) of
    // Q^T to row col of Q, where a warp's 32 rows are neighbours.  Past the rows and columns
    // in use the tile holds anything; there Q is zero, since the product Q X runs over them.
    if (row < P && col0 < P) {
#pragma unroll
        for (int part = 0; part < 2; ++part) {
            __half *out = static_cast<__half *>(c.Q) + ((part * c.matrices + z) * P + col0) * P + row;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint32_t w[4] = {0u, 0u, 0u, 0u};
                if (mine_in && row < n)
                    ptx::ld_shared_v4(mQ + part * PART + static_cast<uint32_t>(col0 >> 6) * BLOCK +
                                          static_cast<uint32_t>(row) * 128u +
                                          (static_cast<uint32_t>((((col0 & 63) >> 3) + j) ^ (row & 7)) << 4),
                                      w[0], w[1], w[2], w[3]);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const __half2 h = *reinterpret_cast<const __half2 *>(&w[i]);
                    const int col = 8 * j + 2 * i;
                    const bool in = col0 + col < n;  // n is even
                    out[col * P] = in ? __low2half(h) : __half(0.0f);
                    out[(col + 1) * P] = in ? __high2half(h) : __half(0.0f);
                }
            }
        }
    }
    ptx::tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, TMEM_COLS);
    }
}

}  // namespace chain

cudaError_t launch_ns_chain(const NsChain &c, cudaStream_t st) {
    // per call: the attribute belongs to the current device
    const cudaError_t e = cudaFuncSetAttribute(chain::chain_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>(chain::SMEM));
    if (e != cudaSuccess) return e;
    return launch_pdl(chain::chain_kernel, dim3(static_cast<unsigned>(c.matrices)), chain::THREADS, chain::SMEM, st, c);
}

}  // namespace tpmlp
