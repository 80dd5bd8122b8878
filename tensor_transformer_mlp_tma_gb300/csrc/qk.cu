// Per-head norms of queries and keys with the position rotation in the same pass, its
// gradient, and the same pass writing keys and values into a paged cache.
//
//   norm:      y = g x r,  r = 1 / sqrt(mean(x^2) + eps)         (per head, gains g [d])
//   rotation:  (u, v) -> a (u cos f - v sin f, u sin f + v cos f),  f = position * theta_i
//   backward:  dy = the rotation's transpose of the incoming gradient,
//              dg = sum dy x r,  dx = r (dy g - x r mean(dy g x r))
//
// Angles.  position * theta_i in fp32 is off by 2^-24 of itself: 0.06 radians at position 10^6.
// theta_i is kept as turns in units of 2^-64, so that the product modulo 2^64 is the fraction of
// a turn, exact to position * 2^-65; its upper 32 bits go to sincospif.
//
// Bound by memory: each element is read once and written once.  A head is held by d / 16 (bf16)
// or d / 8 (fp32) lanes, sixteen bytes of first members and sixteen of second members of the
// pairs each, so the rotation needs no exchange and the norm a few shuffles; the sines of a
// token are computed once per block and read from shared memory by its heads.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "kernels.h"
#include "launch.cuh"
#include "ptx.cuh"

namespace tpmlp {
namespace qk {

constexpr int THREADS = 256;
constexpr int MAX_TOKENS = 4;      // tokens per block
constexpr int MAX_D = 256;
constexpr uint32_t STATUS_INVALID = 1;  // TPMLP_ERR_INVALID_ARG

// P pairs per lane.  VEC: rows are read in pieces of P elements, where every piece starts on
// its own size; else element by element.
template <typename T, int P_, bool VEC_>
struct Lanes {
    using E = T;
    static constexpr int P = P_;
    static constexpr bool VEC = VEC_;
    static constexpr int WORDS = 2 * P * sizeof(T) / 4;  // 32-bit words of a lane's 2P elements
};

// Where a lane's elements are: first members at a, a + step, ..., second members at b, b + step, ...
struct Place {
    int a, b, step;
    int pairs;    // pairs inside the head
    int rotated;  // of those, the first `rotated` rotate
};

template <int P>
__device__ __forceinline__ Place place(int unit, int d, int rot, bool interleaved) {
    const int p0 = unit * P, nf = rot / 2;
    Place at;
    at.pairs = min(max(d / 2 - p0, 0), P);
    at.rotated = min(max(nf - p0, 0), P);
    if (interleaved) {
        at.a = 2 * p0, at.b = 2 * p0 + 1, at.step = 2;
    } else if (at.rotated > 0) {
        at.a = p0, at.b = nf + p0, at.step = 1;
    } else {
        at.a = rot + 2 * (p0 - nf), at.b = at.a + 1, at.step = 2;
    }
    return at;
}

// The pairs of a half-layout lane that straddles the end of the rotated part (element-wise lanes
// only): pair i >= rotated is (rot + 2 j, rot + 2 j + 1).
__device__ __forceinline__ void straddle(const Place &at, int i, int unit_p0, int rot, bool interleaved, int &ia, int &ib) {
    if (!interleaved && at.rotated > 0 && i >= at.rotated) {
        ia = rot + 2 * (unit_p0 + i - rot / 2);
        ib = ia + 1;
    } else {
        ia = at.a + i * at.step;
        ib = at.b + i * at.step;
    }
}

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_f(float v, float &o) { o = v; }
__device__ __forceinline__ void from_f(float v, __nv_bfloat16 &o) { o = __float2bfloat16_rn(v); }

// A lane's elements as they are in memory.
template <typename L>
struct Raw {
    uint32_t w[L::WORDS];
};

template <int WORDS>
__device__ __forceinline__ void copy_in(uint32_t *w, const void *p) {
    if constexpr (WORDS == 4) {
        const uint4 v = *static_cast<const uint4 *>(p);
        w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    } else {
        const uint2 v = *static_cast<const uint2 *>(p);
        w[0] = v.x, w[1] = v.y;
    }
}
template <int WORDS>
__device__ __forceinline__ void copy_out(void *p, const uint32_t *w) {
    if constexpr (WORDS == 4)
        *static_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    else
        *static_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
}

// The two pieces of a vector lane: first and second members in the half layout, consecutive
// elements elsewhere.
template <typename L>
__device__ __forceinline__ int second_piece(const Place &at) {
    return at.step == 1 ? at.b : at.a + L::P;
}

template <typename L>
__device__ __forceinline__ Raw<L> load(const typename L::E *row, const Place &at, int p0, int rot, bool inter) {
    Raw<L> r;
    if constexpr (L::VEC) {
        if (at.pairs > 0) {
            copy_in<L::WORDS / 2>(r.w, row + at.a);
            copy_in<L::WORDS / 2>(r.w + L::WORDS / 2, row + second_piece<L>(at));
        } else {
#pragma unroll
            for (int i = 0; i < L::WORDS; ++i) r.w[i] = 0u;
        }
    } else {
        typename L::E e[2 * L::P];
#pragma unroll
        for (int i = 0; i < L::P; ++i) {
            int ia, ib;
            straddle(at, i, p0, rot, inter, ia, ib);
            from_f(0.0f, e[2 * i]), from_f(0.0f, e[2 * i + 1]);
            if (i < at.pairs) e[2 * i] = row[ia], e[2 * i + 1] = row[ib];
        }
        memcpy(r.w, e, sizeof(e));
    }
    return r;
}

// First members to u, second members to v.
template <typename L>
__device__ __forceinline__ void unpack(const Raw<L> &r, const Place &at, float (&u)[L::P], float (&v)[L::P]) {
    typename L::E e[2 * L::P];
    memcpy(e, r.w, sizeof(e));
    if (L::VEC && at.step == 1) {
#pragma unroll
        for (int i = 0; i < L::P; ++i) u[i] = to_f(e[i]), v[i] = to_f(e[L::P + i]);
    } else {
#pragma unroll
        for (int i = 0; i < L::P; ++i) u[i] = to_f(e[2 * i]), v[i] = to_f(e[2 * i + 1]);
    }
}

template <typename L>
__device__ __forceinline__ void store(typename L::E *row, const Place &at, int p0, int rot, bool inter,
                                      const float (&u)[L::P], const float (&v)[L::P]) {
    if constexpr (L::VEC) {
        if (at.pairs == 0) return;
        typename L::E e[2 * L::P];
        if (at.step == 1) {
#pragma unroll
            for (int i = 0; i < L::P; ++i) from_f(u[i], e[i]), from_f(v[i], e[L::P + i]);
        } else {
#pragma unroll
            for (int i = 0; i < L::P; ++i) from_f(u[i], e[2 * i]), from_f(v[i], e[2 * i + 1]);
        }
        Raw<L> r;
        memcpy(r.w, e, sizeof(e));
        copy_out<L::WORDS / 2>(row + at.a, r.w);
        copy_out<L::WORDS / 2>(row + second_piece<L>(at), r.w + L::WORDS / 2);
    } else {
#pragma unroll
        for (int i = 0; i < L::P; ++i) {
            int ia, ib;
            straddle(at, i, p0, rot, inter, ia, ib);
            if (i < at.pairs) from_f(u[i], row[ia]), from_f(v[i], row[ib]);
        }
    }
}

// A value copied unrounded.
template <typename L>
__device__ __forceinline__ void store_raw(typename L::E *row, const Place &at, int p0, int rot, bool inter, const Raw<L> &r) {
    if constexpr (L::VEC) {
        if (at.pairs == 0) return;
        copy_out<L::WORDS / 2>(row + at.a, r.w);
        copy_out<L::WORDS / 2>(row + second_piece<L>(at), r.w + L::WORDS / 2);
    } else {
        typename L::E e[2 * L::P];
        memcpy(e, r.w, sizeof(e));
#pragma unroll
        for (int i = 0; i < L::P; ++i) {
            int ia, ib;
            straddle(at, i, p0, rot, inter, ia, ib);
            if (i < at.pairs) row[ia] = e[2 * i], row[ib] = e[2 * i + 1];
        }
    }
}

// Amplitude times cosine and sine of every pair's angle, for `n` tokens from t0 on.
__device__ __forceinline__ void angles(const QkArgs &a, int64_t t0, int n, float *cosines, float *sines) {
    const int nf = a.rot / 2;
    for (int i = threadIdx.x; i < n * nf; i += THREADS) {
        const int tok = i / nf, f = i - tok * nf;
        const uint64_t turn = static_cast<uint64_t>(a.position[t0 + tok]) * a.turns[f];
        // half turns in [-1, 1)
        const float half = static_cast<float>(static_cast<int32_t>(turn >> 32)) * 0x1p-31f;
        float s, c;
        sincospif(half, &s, &c);
        cosines[i] = a.amplitude * c;
        sines[i] = a.amplitude * s;
    }
}

template <int P>
__device__ __forceinline__ void turn(float (&u)[P], float (&v)[P], const float *c, const float *s, int rotated, float sign) {
#pragma unroll
    for (int i = 0; i < P; ++i) {
        if (i < rotated) {
            const float ci = c[i], si = sign * s[i];
            const float x = u[i] * ci - v[i] * si;
            v[i] = u[i] * si + v[i] * ci;
            u[i] = x;
        }
    }
}

__device__ __forceinline__ float group_sum(float x, int lanes) {
    for (int o = lanes / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

template <typename E>
__device__ __forceinline__ const E *head_row(const HeadRows &h, int64_t token, int head, int per_shard, int d) {
    const int shard = head / per_shard;
    return static_cast<const E *>(h.p) + token * h.row + shard * h.shard + static_cast<int64_t>(head - shard * per_shard) * d;
}

// blockIdx.x: a group of `toks` tokens; blockIdx.y: a range of `rows` head rows of each.
template <typename L, bool APPEND>
__global__ void __launch_bounds__(THREADS)
    forward_kernel(const QkArgs a, int toks, int rows_per_block, int lanes) {
    using E = typename L::E;
    extern __shared__ float table[];
    __shared__ int64_t dst[MAX_TOKENS];
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const int64_t t0 = static_cast<int64_t>(blockIdx.x) * toks;
    const int n = static_cast<int>(min(static_cast<int64_t>(toks), a.tokens - t0));
    const int total = a.heads + (APPEND ? 2 : 1) * a.kv_heads;
    const int r0 = static_cast<int>(blockIdx.y) * rows_per_block, rows = min(rows_per_block, total - r0);
    const int nf = a.rot / 2, hq = a.heads / a.t, hk = a.kv_heads / a.t;
    const int lane = static_cast<int>(threadIdx.x) & (lanes - 1), p0 = lane * L::P;
    const int sub = static_cast<int>(threadIdx.x) / lanes, subs = THREADS / lanes;
    const Place at = place<L::P>(lane, a.d, a.rot, a.interleaved);
    const int items = n * rows;
    float *sines = table + toks * nf;

    struct Item {
        int tok, row;
        Raw<L> x;
    };
    auto fetch = [&](int i, Item &it) {
        it.tok = i / rows, it.row = r0 + i - it.tok * rows;
        const int64_t t = t0 + it.tok;
        const E *p = it.row < a.heads ? head_row<E>(a.q, t, it.row, hq, a.d)
                     : !APPEND || it.row < a.heads + a.kv_heads
                         ? head_row<E>(a.k, t, it.row - a.heads, hk, a.d)
                         : head_row<E>(a.v, t, it.row - a.heads - a.kv_heads, hk, a.d);
        it.x = load<L>(p, at, p0, a.rot, a.interleaved);
    };
    Item cur;
    if (sub < items) fetch(sub, cur);
    angles(a, t0, n, table, sines);
    if (APPEND && static_cast<int>(threadIdx.x) < n) {
        const int64_t slot = a.slot[t0 + threadIdx.x];
        int64_t where = -1;
        if (slot >= a.slots) {
            if (atomicCAS(a.status, 0u, STATUS_INVALID) == 0u) a.status[1] = static_cast<uint32_t>(t0 + threadIdx.x);
        } else if (slot >= 0) {
            where = slot / a.page_size * a.page_stride + slot % a.page_size * a.token_stride;
        }
        dst[threadIdx.x] = where;
    }
    __syncthreads();
    // every lane of a warp takes part in the shuffles; `live` says whether it has a row
    for (int i0 = 0; i0 < items; i0 += subs) {
        const int i = i0 + sub;
        const bool live = i < items;
        Item next;
        if (i + subs < items) fetch(i + subs, next);
        const bool value = APPEND && live && cur.row >= a.heads + a.kv_heads;
        const bool key = live && !value && cur.row >= a.heads;
        float u[L::P], v[L::P];
        if (live) unpack<L>(cur.x, at, u, v);
        if (a.norm) {
            float sum = 0.0f;
            if (live) {
#pragma unroll
                for (int j = 0; j < L::P; ++j) sum += u[j] * u[j] + v[j] * v[j];
            }
            const float r = rsqrtf(group_sum(sum, lanes) / static_cast<float>(a.d) + a.eps);
            if (live && !value) {
                float gu[L::P], gv[L::P];
                const E *gain = static_cast<const E *>(key ? a.gain_k : a.gain_q);
                unpack<L>(load<L>(gain, at, p0, a.rot, a.interleaved), at, gu, gv);
#pragma unroll
                for (int j = 0; j < L::P; ++j) u[j] *= r * gu[j], v[j] *= r * gv[j];
            }
        }
        if (live) {
            if (!value) turn<L::P>(u, v, table + cur.tok * nf + p0, sines + cur.tok * nf + p0, at.rotated, 1.0f);
            const int64_t t = t0 + cur.tok;
            if (!key && !value) {
                E *o = const_cast<E *>(head_row<E>(a.oq, t, cur.row, hq, a.d));
                store<L>(o, at, p0, a.rot, a.interleaved, u, v);
            } else if (!APPEND) {
                E *o = const_cast<E *>(head_row<E>(a.ok, t, cur.row - a.heads, hk, a.d));
                store<L>(o, at, p0, a.rot, a.interleaved, u, v);
            } else if (dst[cur.tok] >= 0) {
                if (key)
                    store<L>(static_cast<E *>(a.cache_k) + dst[cur.tok] + (cur.row - a.heads) * a.head_stride, at, p0,
                             a.rot, a.interleaved, u, v);
                else
                    store_raw<L>(static_cast<E *>(a.cache_v) + dst[cur.tok] +
                                     (cur.row - a.heads - a.kv_heads) * a.head_stride,
                                 at, p0, a.rot, a.interleaved, cur.x);
            }
        }
        cur = next;
    }
}

// Blocks [0, q_blocks) take the queries' rows, the others the keys'; each takes groups of `toks`
// tokens in turn, and leaves its sums of the gains' gradient in part[blockIdx.x][d].
template <typename L>
__global__ void __launch_bounds__(THREADS)
    backward_kernel(const QkArgs a, int toks, int q_blocks, int lanes) {
    using E = typename L::E;
    extern __shared__ float table[];
    __shared__ float sums[THREADS / 32][MAX_D];
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const bool key = static_cast<int>(blockIdx.x) >= q_blocks;
    const int block = static_cast<int>(blockIdx.x) - (key ? q_blocks : 0);
    const int blocks = key ? static_cast<int>(gridDim.x) - q_blocks : q_blocks;
    const int heads = key ? a.kv_heads : a.heads, per_shard = heads / a.t;
    const HeadRows &hx = key ? a.k : a.q, &hg = key ? a.dk : a.dq, &ho = key ? a.ok : a.oq;
    const int nf = a.rot / 2;
    const int lane = static_cast<int>(threadIdx.x) & (lanes - 1), p0 = lane * L::P;
    const int sub = static_cast<int>(threadIdx.x) / lanes, subs = THREADS / lanes;
    const Place at = place<L::P>(lane, a.d, a.rot, a.interleaved);
    float *sines = table + toks * nf;
    float gu[L::P], gv[L::P], su[L::P], sv[L::P];
#pragma unroll
    for (int j = 0; j < L::P; ++j) gu[j] = gv[j] = 1.0f, su[j] = sv[j] = 0.0f;
    if (a.norm)
        unpack<L>(load<L>(static_cast<const E *>(key ? a.gain_k : a.gain_q), at, p0, a.rot, a.interleaved), at, gu, gv);
    const int64_t groups = (a.tokens + toks - 1) / toks;
    for (int64_t group = block; group < groups; group += blocks) {
        const int64_t t0 = group * toks;
        const int n = static_cast<int>(min(static_cast<int64_t>(toks), a.tokens - t0));
        const int items = n * heads;
        struct Item {
            int tok, head;
            Raw<L> x, g;
        };
        auto fetch = [&](int i, Item &it) {
            it.tok = i / heads, it.head = i - it.tok * heads;
            it.g = load<L>(head_row<E>(hg, t0 + it.tok, it.head, per_shard, a.d), at, p0, a.rot, a.interleaved);
            if (a.norm)
                it.x = load<L>(head_row<E>(hx, t0 + it.tok, it.head, per_shard, a.d), at, p0, a.rot, a.interleaved);
        };
        Item cur;
        if (sub < items) fetch(sub, cur);
        __syncthreads();  // the table of the group before has been read
        angles(a, t0, n, table, sines);
        __syncthreads();
        for (int i0 = 0; i0 < items; i0 += subs) {
            const bool live = i0 + sub < items;
            Item next;
            if (i0 + sub + subs < items) fetch(i0 + sub + subs, next);
            float u[L::P], v[L::P];
            if (live) {
                unpack<L>(cur.g, at, u, v);
                turn<L::P>(u, v, table + cur.tok * nf + p0, sines + cur.tok * nf + p0, at.rotated, -1.0f);
            }
            if (a.norm) {
                float xu[L::P], xv[L::P], square = 0.0f, dot = 0.0f;
                if (live) {
                    unpack<L>(cur.x, at, xu, xv);
#pragma unroll
                    for (int j = 0; j < L::P; ++j) {
                        square += xu[j] * xu[j] + xv[j] * xv[j];
                        dot += gu[j] * u[j] * xu[j] + gv[j] * v[j] * xv[j];
                    }
                }
                for (int o = lanes / 2; o > 0; o >>= 1) {
                    square += __shfl_xor_sync(0xffffffffu, square, o);
                    dot += __shfl_xor_sync(0xffffffffu, dot, o);
                }
                const float inv_d = 1.0f / static_cast<float>(a.d);
                const float r = rsqrtf(square / static_cast<float>(a.d) + a.eps);
                const float m = r * dot * inv_d;  // mean of dy g x r
                if (live) {
#pragma unroll
                    for (int j = 0; j < L::P; ++j) {
                        const float hu = xu[j] * r, hv = xv[j] * r;
                        su[j] += u[j] * hu, sv[j] += v[j] * hv;
                        u[j] = r * (u[j] * gu[j] - hu * m);
                        v[j] = r * (v[j] * gv[j] - hv * m);
                    }
                }
            }
            if (live) {
                E *o = const_cast<E *>(head_row<E>(ho, t0 + cur.tok, cur.head, per_shard, a.d));
                store<L>(o, at, p0, a.rot, a.interleaved, u, v);
            }
            cur = next;
        }
    }
    if (!a.norm) return;
    // lanes of a warp that hold the same components, then the block's warps in order
#pragma unroll
    for (int j = 0; j < L::P; ++j) {
        for (int o = lanes; o < 32; o <<= 1) {
            su[j] += __shfl_xor_sync(0xffffffffu, su[j], o);
            sv[j] += __shfl_xor_sync(0xffffffffu, sv[j], o);
        }
    }
    const int warp = static_cast<int>(threadIdx.x) >> 5;
    if ((static_cast<int>(threadIdx.x) & 31) < lanes) {
#pragma unroll
        for (int j = 0; j < L::P; ++j) {
            if (j < at.pairs) {
                int ia, ib;
                if (L::VEC && at.step == 2)
                    ia = at.a + 2 * j, ib = ia + 1;
                else
                    straddle(at, j, p0, a.rot, a.interleaved, ia, ib);
                sums[warp][ia] = su[j];
                sums[warp][ib] = sv[j];
            }
        }
    }
    __syncthreads();
    for (int c = threadIdx.x; c < a.d; c += THREADS) {
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < THREADS / 32; ++w) s += sums[w][c];
        a.part[static_cast<int64_t>(blockIdx.x) * a.d + c] = s;
    }
}

// dgain[c] = sum of the blocks' part[.][c], in a fixed order.  blockIdx.y: queries or keys.
constexpr int GAIN_ROWS = 16;
template <typename E>
__global__ void __launch_bounds__(32 * GAIN_ROWS) gain_kernel(const QkArgs a, int q_blocks, int blocks) {
    __shared__ float sums[GAIN_ROWS][33];
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const bool key = blockIdx.y == 1;
    const int x = threadIdx.x & 31, y = threadIdx.x >> 5, c = blockIdx.x * 32 + x;
    const int first = key ? q_blocks : 0, last = key ? blocks : q_blocks;
    float s = 0.0f;
    if (c < a.d) {
#pragma unroll 4
        for (int b = first + y; b < last; b += GAIN_ROWS) s += a.part[static_cast<int64_t>(b) * a.d + c];
    }
    sums[y][x] = s;
    __syncthreads();
    if (y == 0 && c < a.d) {
#pragma unroll
        for (int i = 1; i < GAIN_ROWS; ++i) s += sums[i][x];
        from_f(s, static_cast<E *>(key ? a.dgain_k : a.dgain_q)[c]);
    }
}

// Blocks of the backward pass: four per SM of the 152, and no more than groups of tokens.
constexpr int BACKWARD_BLOCKS = 608;

template <typename F>
cudaError_t dispatch(bool is_bf16, const QkArgs &a, F f) {
    // sixteen-byte pieces of first and second members (bf16: 8 elements), eight-byte ones, or elements
    auto fits = [&](int p) { return a.vec && a.d % (2 * p) == 0 && (a.interleaved || a.rot % (2 * p) == 0) && a.rot % 2 == 0; };
    if (is_bf16) {
        if (fits(8)) return f(Lanes<__nv_bfloat16, 8, true>());
        if (fits(4)) return f(Lanes<__nv_bfloat16, 4, true>());
        return f(Lanes<__nv_bfloat16, 4, false>());
    }
    if (fits(4)) return f(Lanes<float, 4, true>());
    return f(Lanes<float, 4, false>());
}

int lanes_of(int d, int p) {
    int n = 1;
    while (n * 2 * p < d) n *= 2;
    return n;
}

}  // namespace qk

int64_t qk_partial_floats(int64_t tokens, int d) {
    return (tokens > 0 ? qk::BACKWARD_BLOCKS : 1) * static_cast<int64_t>(d);
}

cudaError_t launch_qk_forward(bool is_bf16, const QkArgs &a, bool append, cudaStream_t st) {
    return qk::dispatch(is_bf16, a, [&](auto L) {
        using Ln = decltype(L);
        const int lanes = qk::lanes_of(a.d, Ln::P), subs = qk::THREADS / lanes;
        const int rows = a.heads + (append ? 2 : 1) * a.kv_heads;
        // Many tokens: four per block, so that a thread computes about one sine; few: a row per
        // group of lanes, over as many blocks as that takes.
        const int toks = a.tokens * rows >= 152LL * 8 * subs ? qk::MAX_TOKENS : 1;
        const int per = toks > 1 ? rows : (rows < subs ? rows : subs);
        const dim3 grid(static_cast<unsigned>((a.tokens + toks - 1) / toks), static_cast<unsigned>((rows + per - 1) / per));
        const size_t smem = static_cast<size_t>(toks) * a.rot * sizeof(float);
        return append ? launch_pdl(qk::forward_kernel<Ln, true>, grid, qk::THREADS, smem, st, a, toks, per, lanes)
                      : launch_pdl(qk::forward_kernel<Ln, false>, grid, qk::THREADS, smem, st, a, toks, per, lanes);
    });
}

cudaError_t launch_qk_backward(bool is_bf16, const QkArgs &a, cudaStream_t st, int *launches) {
    *launches = 0;
    return qk::dispatch(is_bf16, a, [&](auto L) {
        using Ln = decltype(L);
        const int lanes = qk::lanes_of(a.d, Ln::P), subs = qk::THREADS / lanes;
        const int rows = a.heads + a.kv_heads;
        const int toks = a.tokens * rows >= 152LL * 8 * subs ? qk::MAX_TOKENS : 1;
        const int64_t groups = (a.tokens + toks - 1) / toks;
        // blocks in proportion to the rows
        int64_t nq = qk::BACKWARD_BLOCKS * static_cast<int64_t>(a.heads) / rows, nk = qk::BACKWARD_BLOCKS - nq;
        nq = nq < groups ? nq : groups;
        nk = nk < groups ? nk : groups;
        const size_t smem = static_cast<size_t>(toks) * a.rot * sizeof(float);
        cudaError_t e = launch_pdl(qk::backward_kernel<Ln>, dim3(static_cast<unsigned>(nq + nk)), qk::THREADS, smem, st, a,
                                   toks, static_cast<int>(nq), lanes);
        if (e != cudaSuccess) return e;
        ++*launches;
        if (!a.norm) return e;
        e = launch_pdl(qk::gain_kernel<typename Ln::E>, dim3(static_cast<unsigned>((a.d + 31) / 32), 2),
                       32 * qk::GAIN_ROWS, 0, st, a, static_cast<int>(nq), static_cast<int>(nq + nk));
        if (e == cudaSuccess) ++*launches;
        return e;
    });
}

}  // namespace tpmlp
