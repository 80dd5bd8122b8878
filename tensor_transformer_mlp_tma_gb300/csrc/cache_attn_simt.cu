// Attention over a paged cache on FFMA kernels: fp32 caches, and bf16 ones whose layout the
// tensor-core kernel does not take; any page size.
//
//   O = softmax(scale Q K^T over the visible keys) V,  one pass over the keys with the running
//   maximum m and sum l of each row:  m' = max(m, max s),  l' = l 2^(m - m') + sum 2^(s - m'),
//   O' = O 2^(m - m') + P V,  s in units of log2.
//
// K of the next tile is on its way while the weights and outputs of one are formed, V while the scores are
// (fp32 rows on 16 bytes: by asynchronous copies; two blocks per SM hide the rest).
//
// A block takes 32 rows (tokens and the heads that share their keys) and 64 keys at a time, all
// of them in shared memory in fp32.  Many rows are bound by instructions and shared memory's rate (56 and 50 %
// of the cycles before two products went to an instruction): a thread forms up to 8 scores of one key, then 4 x 4
// outputs (4 prompt chunks of 300 to 512 tokens in fp32: 16.2 ms, 27 TFLOP/s); few by the turns of a tile's
// copies, barriers and sums (64 sequences of one token, 2.4 GB: 515 us, 4.6 TB/s).  bf16 goes through registers on its
// way, 8 bytes (or, where rows are not on 16, one element) at a time, and waits for each: 1.3 ms (0.9 TB/s) and 22 ms
// (20 TFLOP/s) for the same two in bf16 with pages of 1, 4 or 20 tokens.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <mutex>
#include <type_traits>

#include "cache_attn.cuh"
#include "launch.cuh"
#include "ptx.cuh"

namespace tpmlp {
namespace cattn {

constexpr int SR = CACHE_ATTN_SIMT_ROWS;
constexpr int SK = 64;
constexpr int STHREADS = 256, WARPS = STHREADS / 32;
constexpr int P_LD = SK + 4;
// Minus infinity in the place of a score says that the row does not see the key.  A visible score of minus infinity becomes
// LOWEST; a row's maximum begins at the next number above it, 2^104 away: the weight is zero, whatever else the row sees.
constexpr float LOWEST = -0x1.fffffep+127f, LEAST_MAXIMUM = -0x1.fffffcp+127f;

__device__ __forceinline__ float4 get4(const float *p, bool vec) {
    return vec ? *reinterpret_cast<const float4 *>(p) : make_float4(p[0], p[1], p[2], p[3]);
}
__device__ __forceinline__ float4 get4(const __nv_bfloat16 *p, bool vec) {
    if (!vec) return make_float4(__bfloat162float(p[0]), __bfloat162float(p[1]), __bfloat162float(p[2]), __bfloat162float(p[3]));
    const uint2 w = *reinterpret_cast<const uint2 *>(p);
    const __nv_bfloat162 lo = *reinterpret_cast<const __nv_bfloat162 *>(&w.x), hi = *reinterpret_cast<const __nv_bfloat162 *>(&w.y);
    return make_float4(__low2float(lo), __high2float(lo), __low2float(hi), __high2float(hi));
}

inline size_t simt_smem(int d) {
    return sizeof(float) * (static_cast<size_t>(SR) * d + SK * (d + 4) + SK * d + SR * P_LD + 3 * SR);
}

// Scores of a key and NR rows, four apart from q on.  (A constant number of them: with a test per row the rows' loads
// waited for one another, and everything took twice as long.)
template <int NR>
__device__ __forceinline__ void scores(float (&s)[SR / 4], const float *q, const float *k, int d) {
    float2 t[NR] = {};  // sums of even and odd components: two products to an instruction
#pragma unroll 2
    for (int e = 0; e < d; e += 4) {
        const float4 x = *reinterpret_cast<const float4 *>(k + e);
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            const float4 y = *reinterpret_cast<const float4 *>(q + 4 * i * d + e);
            t[i] = ptx::fma2(make_float2(y.x, y.y), make_float2(x.x, x.y), t[i]);
            t[i] = ptx::fma2(make_float2(y.z, y.w), make_float2(x.z, x.w), t[i]);
        }
    }
#pragma unroll
    for (int i = 0; i < NR; ++i) s[i] = t[i].x + t[i].y;
}

// Weights of a tile in place of its scores, and the rows' new maxima, sums and factors; a warp takes NR rows, eight apart,
// side by side.
template <int NR>
__device__ __forceinline__ void weights(float *P, float *m_sh, float *l_sh, float *f_sh, int warp, int lane, int rows) {
    float s[NR][2], top[NR], sum[NR], m[NR];
#pragma unroll
    for (int i = 0; i < NR; ++i) {
        const int row = warp + WARPS * i;
        const bool have = row < rows;
        s[i][0] = have ? P[row * P_LD + lane] : -INFINITY;
        s[i][1] = have ? P[row * P_LD + lane + 32] : -INFINITY;
        m[i] = have ? m_sh[row] : -INFINITY;
        top[i] = fmaxf(s[i][0], s[i][1]);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int i = 0; i < NR; ++i) top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], o));
#pragma unroll
    for (int i = 0; i < NR; ++i) {
        const int row = warp + WARPS * i;
        top[i] = fmaxf(m[i], top[i]);
        // masked weights are marked by a negative number, not by zero: 0 x NaN would be NaN
        const float p0 = s[i][0] == -INFINITY ? -1.0f : exp2f(s[i][0] - top[i]), p1 = s[i][1] == -INFINITY ? -1.0f : exp2f(s[i][1] - top[i]);
        sum[i] = (s[i][0] == -INFINITY ? 0.0f : p0) + (s[i][1] == -INFINITY ? 0.0f : p1);
        if (row < rows) {
            P[row * P_LD + lane] = p0;
            P[row * P_LD + lane + 32] = p1;
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int i = 0; i < NR; ++i) sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], o);
    __syncwarp();
    if (lane == 0)
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            const int row = warp + WARPS * i;
            if (row < rows) {
                const float f = scale_of(m[i], top[i]);
                f_sh[row] = f, m_sh[row] = top[i], l_sh[row] = l_sh[row] * f + sum[i];
            }
        }
}

// Outputs of row quads quad0 and (TWO) quad1 from the keys of a group, four at a time.
template <bool TWO, bool MASKED>
__device__ __forceinline__ void outputs(float2 (&acc)[2][4][2], const float *P, const float *V, int d, int quad0, int quad1, int kg, int key_groups) {
    for (int key = 4 * kg; key < SK; key += 4 * key_groups) {
        float4 v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = *reinterpret_cast<const float4 *>(V + (key + k) * d);
#pragma unroll
        for (int h = 0; h < (TWO ? 2 : 1); ++h)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const float4 p = *reinterpret_cast<const float4 *>(P + (4 * (h == 0 ? quad0 : quad1) + r) * P_LD + key);
                const float pk[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (!MASKED || !(pk[k] < 0.0f)) {
                        const float2 p2 = make_float2(pk[k], pk[k]);
                        acc[h][r][0] = ptx::fma2(p2, make_float2(v[k].x, v[k].y), acc[h][r][0]);
                        acc[h][r][1] = ptx::fma2(p2, make_float2(v[k].z, v[k].w), acc[h][r][1]);
                    }
            }
    }
}

template <typename E>
__global__ void __launch_bounds__(STHREADS) simt_kernel(const CacheAttnArgs a) {
    extern __shared__ float4 smem4[];
    __shared__ typename Walk<SR, SK>::Shared wsh;
    __shared__ int64_t where_sh[2][SK];
    const int d = a.d, quads = d / 4, kld = d + 4;
    float *Q = reinterpret_cast<float *>(smem4), *K = Q + SR * d, *V = K + SK * kld, *P = V + SK * d;
    float *m_sh = P + SR * P_LD, *l_sh = m_sh + SR, *f_sh = l_sh + SR;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    Walk<SR, SK> walk;
    walk.begin(a, wsh);

    // the output's threads: `cols` of four components each, `groups` of them; with fewer row quads
    // than groups the keys are shared out too
    int cols = 1;
    while (cols < quads) cols *= 2;
    // (at most 32 groups: their sums are added up in the space of K, V and P, 128 d floats and more)
    const int groups = min(STHREADS / cols, 32), col = tid & (cols - 1), group = tid / cols;

    // K or V of a tile into shared memory, rows `ld` apart
    auto copy = [&](float *to, int ld, const void *base, const int64_t *where) {
        if (col < quads)
#pragma unroll 4
            for (int key = tid / cols; key < SK; key += STHREADS / cols) {
                const int64_t off = where[key];
                const E *from = static_cast<const E *>(base) + (off >= 0 ? off + 4 * col : 0);
                float *at = to + key * ld + 4 * col;
                if constexpr (std::is_same<E, float>::value) {
                    if (a.vec) {
                        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(ptx::smem_u32(at)), "l"(from), "r"(off >= 0 ? 16u : 0u)
                                     : "memory");
                        continue;
                    }
                }
                *reinterpret_cast<float4 *>(at) = off >= 0 ? get4(from, a.vec) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };

    bool posted = false;
    Unit u;
    while (walk.next(a, u)) {
        const int rq = (u.rows + 3) / 4;
        int rq2 = 1;
        while (rq2 < rq) rq2 *= 2;
        const int key_groups = rq2 < groups ? groups / rq2 : 1;
        const int quad0 = rq2 < groups ? group % rq2 : group, kg = rq2 < groups ? group / rq2 : 0;
        const bool mine = col < quads && group < groups;
        float2 acc[2][4][2] = {};
        __syncthreads();  // the unit before is done with shared memory
        for (int i = tid; i < SR * quads; i += STHREADS) {
            const int row = i / quads, e = (i - row * quads) * 4;
            float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (row < u.rows) {
                const int r = u.row0 + row, token = r / a.group;
                const int64_t at = (static_cast<int64_t>(u.s.q0 + token) * a.heads + u.head * a.group + (r - token * a.group)) * d + e;
                x = get4(static_cast<const E *>(a.q) + at, true);
            }
            *reinterpret_cast<float4 *>(Q + row * d + e) = x;
        }
        if (tid < SR) m_sh[tid] = LEAST_MAXIMUM, l_sh[tid] = 0.0f;
        // where a tile's keys lie: the page is looked up early, and used after the scores of the tile before
        auto look = [&](int t) {
            const int key = t * SK + tid;
            return tid < SK && key < u.s.len ? a.table[u.b * a.max_pages + static_cast<uint32_t>(key) / static_cast<uint32_t>(a.page_size)] : -1;
        };
        auto place = [&](int t, int page) {
            const int key = t * SK + tid;
            if (tid >= SK) return;
            int64_t off = -1;  // no key: zeros
            if (key < u.s.len) {
                if (page >= 0 && page < a.pages)
                    off = page * a.page_stride + u.head * a.head_stride +
                          static_cast<uint32_t>(key) % static_cast<uint32_t>(a.page_size) * a.token_stride;
                else
                    report(a, STATUS_INVALID, static_cast<uint32_t>(u.b));
            }
            where_sh[t & 1][tid] = off;
        };
        place(u.tile0, look(u.tile0));
        __syncthreads();
        copy(K, kld, a.k, where_sh[u.tile0 & 1]);
        copy(V, d, a.v, where_sh[u.tile0 & 1]);
        for (int t = u.tile0; t < u.tile0 + u.tiles; ++t) {
            const int key0 = t * SK;
            const bool masked = key0 + SK > u.s.prefix, more = t + 1 < u.tile0 + u.tiles;
            const int page = more ? look(t + 1) : -1;
            asm volatile("cp.async.wait_group 1;" ::: "memory");  // K
            __syncthreads();
            {
                // scores of one key and rows rg, rg + 4, ...
                const int key = tid & (SK - 1), rg = tid / SK;
                float s[SR / 4] = {};
                const int nr = (u.rows + 3) / 4;
                if (nr == 1)
                    scores<1>(s, Q + rg * d, K + key * kld, d);
                else if (nr == 2)
                    scores<2>(s, Q + rg * d, K + key * kld, d);
                else if (nr <= 4)
                    scores<4>(s, Q + rg * d, K + key * kld, d);
                else
                    scores<8>(s, Q + rg * d, K + key * kld, d);
#pragma unroll
                for (int i = 0; i < SR / 4; ++i)
                    if (i < nr) {
                        const int row = rg + 4 * i;
                        const bool seen = row < u.rows && (!masked || visible(a, u.s, (u.row0 + row) / a.group, key0 + key));
                        const float x = s[i] * a.scale_log2;
                        P[row * P_LD + key] = !seen ? -INFINITY : (x == -INFINITY ? LOWEST : x);
                    }
            }
            if (more) place(t + 1, page);
            __syncthreads();
            if (more) copy(K, kld, a.k, where_sh[(t + 1) & 1]);
            else asm volatile("cp.async.commit_group;" ::: "memory");
            if (u.rows <= WARPS)
                weights<1>(P, m_sh, l_sh, f_sh, warp, lane, u.rows);
            else
                weights<SR / WARPS>(P, m_sh, l_sh, f_sh, warp, lane, u.rows);
            asm volatile("cp.async.wait_group 1;" ::: "memory");  // V
            __syncthreads();
            if (mine && quad0 < rq) {
                const int quad1 = quad0 + groups < rq ? quad0 + groups : quad0;
                const bool two = quad1 != quad0;
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int row = 4 * (h == 0 ? quad0 : quad1) + r;
                        const float f = row < u.rows ? f_sh[row] : 1.0f;
#pragma unroll
                        for (int c = 0; c < 2; ++c) acc[h][r][c] = ptx::mul2(acc[h][r][c], make_float2(f, f));
                    }
                const float *v = V + 4 * col;
                if (two)
                    masked ? outputs<true, true>(acc, P, v, d, quad0, quad1, kg, key_groups)
                           : outputs<true, false>(acc, P, v, d, quad0, quad1, kg, key_groups);
                else
                    masked ? outputs<false, true>(acc, P, v, d, quad0, quad1, kg, key_groups)
                           : outputs<false, false>(acc, P, v, d, quad0, quad1, kg, key_groups);
            }
            __syncthreads();  // V is free
            if (more) copy(V, d, a.v, where_sh[(t + 1) & 1]);
        }
        __syncthreads();
        // the key groups' sums, through the space of K
        if (key_groups > 1) {
            float *sums = K;
            if (mine && kg > 0) {
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    put4(sums + (((kg - 1) * rq2 + quad0) * 4 + r) * d + 4 * col,
                         make_float4(acc[0][r][0].x, acc[0][r][0].y, acc[0][r][1].x, acc[0][r][1].y));
            }
            __syncthreads();
            if (mine && kg == 0) {
                for (int g = 1; g < key_groups; ++g)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const float4 x = *reinterpret_cast<const float4 *>(sums + (((g - 1) * rq2 + quad0) * 4 + r) * d + 4 * col);
                        acc[0][r][0] = ptx::add2(acc[0][r][0], make_float2(x.x, x.y)), acc[0][r][1] = ptx::add2(acc[0][r][1], make_float2(x.z, x.w));
                    }
            }
        }
        const int64_t piece = (2 * static_cast<int64_t>(blockIdx.x) + u.place) * SR;
        if (mine && kg == 0) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int quad = quad0 + h * groups;
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int row = 4 * quad + r;
                    if (quad >= rq || row >= u.rows) continue;
                    float4 x = make_float4(acc[h][r][0].x, acc[h][r][0].y, acc[h][r][1].x, acc[h][r][1].y);
                    if (u.cut) {
                        __stcg(reinterpret_cast<float4 *>(a.part + (piece + row) * d + 4 * col), x);
                    } else {
                        const float l = l_sh[row], inv = l == 0.0f ? 0.0f : 1.0f / l;
                        put4(out_row<E>(a, u, row) + 4 * col, make_float4(x.x * inv, x.y * inv, x.z * inv, x.w * inv));
                    }
                }
            }
        }
        if (u.cut && tid < u.rows) __stcg(a.part_ml + piece + tid, make_float2(m_sh[tid], l_sh[tid]));
        if (u.cut && u.place == 1) {
            if (tid == 0) post_cut(a, u.s.q0, u.head, u.row0, u.rows, walk.last_block(u));
            posted = true;
        }
    }
    if (!posted && tid == 0) post_cut(a, 0, 0, 0, 0, 0);
}

template <typename E>
cudaError_t launch_simt(const CacheAttnArgs &a, int blocks, cudaStream_t st) {
    static std::mutex mu;
    static bool set[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    {
        std::lock_guard<std::mutex> lk(mu);
        if (!set[dev]) {
            e = cudaFuncSetAttribute(simt_kernel<E>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     static_cast<int>(simt_smem(256)));
            if (e != cudaSuccess) return e;
            set[dev] = true;
        }
    }
    e = launch_pdl(simt_kernel<E>, dim3(static_cast<unsigned>(blocks)), STHREADS, simt_smem(a.d), st, a);
    return e == cudaSuccess ? launch_join<E, SR>(a, blocks, st) : e;
}

}  // namespace cattn

// Two blocks per SM where their shared memory fits (225 KB beside 1 KB each).
int cache_attn_simt_blocks(bool, int d, int num_sms) {
    const int per = 2 * (cattn::simt_smem(d) + 1024) <= 225 * 1024 ? 2 : 1;
    const int n = per * num_sms;
    return n < CACHE_ATTN_BLOCKS ? n : CACHE_ATTN_BLOCKS;
}

cudaError_t launch_cache_attn_simt(bool is_bf16, const CacheAttnArgs &a, int num_sms, cudaStream_t st) {
    const int blocks = cache_attn_simt_blocks(is_bf16, a.d, num_sms);
    return is_bf16 ? cattn::launch_simt<__nv_bfloat16>(a, blocks, st) : cattn::launch_simt<float>(a, blocks, st);
}

}  // namespace tpmlp
