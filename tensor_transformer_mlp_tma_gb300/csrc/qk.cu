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
constexpr int WARPS = THREADS / 32;
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

// Amplitude times cosine and sine of every pair's angle at one token, by one warp.
__device__ __forceinline__ void angles(const QkArgs &a, int64_t token, float *cosines, float *sines) {
    const uint64_t position = static_cast<uint64_t>(a.position[token]);
    for (int f = threadIdx.x & 31; f < a.rot / 2; f += 32) {
        const uint64_t turn = position * a.turns[f];
        // half turns in [-1, 1)
        const float half = static_cast<float>(static_cast<int32_t>(turn >> 32)) * 0x1p-31f;
        float s, c;
        sincospif(half, &s, &c);
        cosines[f] = a.amplitude * c;
        sines[f] = a.amplitude * s;
    }
}

// What a lane's pairs are multiplied by: (u, v) -> (uu u + uv v, vu u + vv v), two pairs to a float2.
template <int P>
struct Factors {
    float2 uu[P / 2], uv[P / 2], vu[P / 2], vv[P / 2];
};

template <typename L>
__device__ __forceinline__ bool turns_pair(const Place &at, int i) {
    return L::VEC ? at.rotated > 0 : i < at.rotated;  // vector lanes rotate as a whole
}

template <int P>
__device__ __forceinline__ void table_row(const float *t, float (&x)[P]) {
#pragma unroll
    for (int i = 0; i < P; i += 4) {
        const float4 q = *reinterpret_cast<const float4 *>(t + i);
        x[i] = q.x, x[i + 1] = q.y, x[i + 2] = q.z, x[i + 3] = q.w;
    }
}

template <typename L>
__device__ __forceinline__ Factors<L::P> factors(const QkArgs &a, const void *gain, const Place &at, int p0, const float *cosines,
                                                 const float *sines) {
    constexpr int P = L::P;
    float gu[P], gv[P], c[P], s[P];
#pragma unroll
    for (int i = 0; i < P; ++i) gu[i] = gv[i] = 1.0f, c[i] = 1.0f, s[i] = 0.0f;
    if (a.norm) unpack<L>(load<L>(static_cast<const typename L::E *>(gain), at, p0, a.rot, a.interleaved), at, gu, gv);
    if (at.rotated > 0) table_row<P>(cosines + p0, c), table_row<P>(sines + p0, s);
    Factors<P> f;
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const bool r = turns_pair<L>(at, i);
        const float ci = r ? c[i] : 1.0f, si = r ? s[i] : 0.0f;
        (i & 1 ? f.uu[i / 2].y : f.uu[i / 2].x) = gu[i] * ci;
        (i & 1 ? f.uv[i / 2].y : f.uv[i / 2].x) = -gv[i] * si;
        (i & 1 ? f.vu[i / 2].y : f.vu[i / 2].x) = gu[i] * si;
        (i & 1 ? f.vv[i / 2].y : f.vv[i / 2].x) = gv[i] * ci;
    }
    return f;
}

__device__ __forceinline__ float group_sum(float x, int lanes) {
    for (int o = lanes / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// Heads of one array: the shard of a head by a multiplication.  inverse = ceil(2^32 / per) gives the
// quotient of heads below 2^32 / per; there are 2^16 at most, 2^15 per shard where there are several.
struct Shards {
    uint32_t per, inverse;
};
inline Shards shards_of(int heads, int t) {
    const uint32_t per = static_cast<uint32_t>(heads / t);
    return {per, t == 1 || per == 1 ? 0u : static_cast<uint32_t>(((1ull << 32) + per - 1) / per)};
}

template <typename E>
__device__ __forceinline__ const E *head_row(const HeadRows &h, int64_t token, int head, const Shards &s, int d) {
    const int shard = s.inverse == 0u ? (s.per == 1u ? head : 0) : static_cast<int>(__umulhi(static_cast<uint32_t>(head), s.inverse));
    return static_cast<const E *>(h.p) + token * h.row + shard * h.shard + static_cast<int64_t>(head - shard * static_cast<int>(s.per)) * d;
}

// A warp takes one token's heads, 32 / lanes at a time, or with few tokens a `split`-th of them; its
// factors stay in registers.
struct Split {
    int lanes;   // per head
    int split;   // warps per token
    Shards q, k;
};

template <typename L, bool APPEND>
__global__ void __launch_bounds__(THREADS) forward_kernel(const QkArgs a, const Split w) {
    using E = typename L::E;
    constexpr int P = L::P;
    __shared__ alignas(16) float cosines[WARPS][MAX_D / 2], sines[WARPS][MAX_D / 2];
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const int warp = static_cast<int>(threadIdx.x) >> 5;
    // (tokens times split is below 2^31, see split_of)
    const uint32_t work = blockIdx.x * WARPS + warp;
    const int64_t token = work / static_cast<uint32_t>(w.split);
    if (token >= a.tokens) return;
    const int part = static_cast<int>(work) - static_cast<int>(token) * w.split;
    const int rows = a.heads + (APPEND ? 2 : 1) * a.kv_heads;
    const int lane = static_cast<int>(threadIdx.x) & (w.lanes - 1), p0 = lane * P;
    const int each = 32 / w.lanes, sub = (static_cast<int>(threadIdx.x) & 31) / w.lanes, step = each * w.split;
    const Place at = place<P>(lane, a.d, a.rot, a.interleaved);

    auto fetch = [&](int row) {
        if (row < a.heads) return load<L>(head_row<E>(a.q, token, row, w.q, a.d), at, p0, a.rot, a.interleaved);
        row -= a.heads;
        if (!APPEND || row < a.kv_heads) return load<L>(head_row<E>(a.k, token, row, w.k, a.d), at, p0, a.rot, a.interleaved);
        return load<L>(head_row<E>(a.v, token, row - a.kv_heads, w.k, a.d), at, p0, a.rot, a.interleaved);
    };
    int row = part * each + sub;
    Raw<L> x = {}, next = {};
    if (row < rows) x = fetch(row);
    if (row + step < rows) next = fetch(row + step);
    if (a.rot > 0) angles(a, token, cosines[warp], sines[warp]);
    int64_t where = -1;
    if (APPEND) {
        const int64_t slot = a.slot[token];
        if (slot >= a.slots) {
            if (atomicCAS(a.status, 0u, STATUS_INVALID) == 0u) a.status[1] = static_cast<uint32_t>(token);
        } else if (slot >= 0) {
            where = slot / a.page_size * a.page_stride + slot % a.page_size * a.token_stride;
        }
    }
    __syncwarp();
    int kind = -1;  // of the factors at hand: 0 queries, 1 keys
    Factors<P> f;
    const float inv_d = 1.0f / static_cast<float>(a.d);
    for (int r0 = part * each; r0 < rows; r0 += step, row += step) {
        // two rows ahead in flight; every lane of the warp takes part in the shuffles
        Raw<L> after = {};
        if (row + 2 * step < rows) after = fetch(row + 2 * step);
        const int of = row < a.heads ? 0 : (!APPEND || row < a.heads + a.kv_heads ? 1 : 2);
        if (of < 2 && of != kind) {
            f = factors<L>(a, of ? a.gain_k : a.gain_q, at, p0, cosines[warp], sines[warp]);
            kind = of;
        }
        float u[P], v[P];
        unpack<L>(x, at, u, v);
        float r = 1.0f;
        if (a.norm) {
            float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
            for (int i = 0; i < P; ++i) sum = ptx::fma2(make_float2(u[i], v[i]), make_float2(u[i], v[i]), sum);
            r = rsqrtf(group_sum(sum.x + sum.y, w.lanes) * inv_d + a.eps);
        }
        if (row < rows) {
            if (of == 2) {
                if (where >= 0)
                    store_raw<L>(static_cast<E *>(a.cache_v) + where + (row - a.heads - a.kv_heads) * a.head_stride, at, p0,
                                 a.rot, a.interleaved, x);
            } else {
                const float2 rr = make_float2(r, r);
#pragma unroll
                for (int i = 0; i < P; i += 2) {
                    const float2 ui = make_float2(u[i], u[i + 1]), vi = make_float2(v[i], v[i + 1]);
                    float2 x0, x1;
                    if (L::VEC && at.rotated == 0) {  // not mixed: infinities stay where they are
                        x0 = ptx::mul2(ptx::mul2(ui, f.uu[i / 2]), rr);
                        x1 = ptx::mul2(ptx::mul2(vi, f.vv[i / 2]), rr);
                    } else {
                        x0 = ptx::mul2(ptx::fma2(ui, f.uu[i / 2], ptx::mul2(vi, f.uv[i / 2])), rr);
                        x1 = ptx::mul2(ptx::fma2(vi, f.vv[i / 2], ptx::mul2(ui, f.vu[i / 2])), rr);
                        if (!L::VEC) {
                            if (i >= at.rotated) x0.x = ui.x * f.uu[i / 2].x * r, x1.x = vi.x * f.vv[i / 2].x * r;
                            if (i + 1 >= at.rotated) x0.y = ui.y * f.uu[i / 2].y * r, x1.y = vi.y * f.vv[i / 2].y * r;
                        }
                    }
                    u[i] = x0.x, u[i + 1] = x0.y, v[i] = x1.x, v[i + 1] = x1.y;
                }
                if (of == 0)
                    store<L>(const_cast<E *>(head_row<E>(a.oq, token, row, w.q, a.d)), at, p0, a.rot, a.interleaved, u, v);
                else if (!APPEND)
                    store<L>(const_cast<E *>(head_row<E>(a.ok, token, row - a.heads, w.k, a.d)), at, p0, a.rot, a.interleaved, u, v);
                else if (where >= 0)
                    store<L>(static_cast<E *>(a.cache_k) + where + (row - a.heads) * a.head_stride, at, p0, a.rot, a.interleaved, u, v);
            }
        }
        x = next, next = after;
    }
}

// Blocks [0, q_blocks) take the queries, the others the keys; each warp takes tokens in turn (or
// parts of them) and leaves the block's sums of the gains' gradient in part[blockIdx.x][d].
template <typename L>
__global__ void __launch_bounds__(THREADS, 2) backward_kernel(const QkArgs a, const Split w, int q_blocks) {
    using E = typename L::E;
    constexpr int P = L::P;
    __shared__ alignas(16) float cosines[WARPS][MAX_D / 2], sines[WARPS][MAX_D / 2];
    __shared__ float sums[WARPS][MAX_D];
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const int warp = static_cast<int>(threadIdx.x) >> 5;
    const bool key = static_cast<int>(blockIdx.x) >= q_blocks;
    const int block = static_cast<int>(blockIdx.x) - (key ? q_blocks : 0);
    const int blocks = key ? static_cast<int>(gridDim.x) - q_blocks : q_blocks;
    const int heads = key ? a.kv_heads : a.heads;
    const Shards sh = key ? w.k : w.q;
    const HeadRows &hx = key ? a.k : a.q, &hg = key ? a.dk : a.dq, &ho = key ? a.ok : a.oq;
    const int lane = static_cast<int>(threadIdx.x) & (w.lanes - 1), p0 = lane * P;
    const int each = 32 / w.lanes, sub = (static_cast<int>(threadIdx.x) & 31) / w.lanes, step = each * w.split;
    const Place at = place<P>(lane, a.d, a.rot, a.interleaved);
    float gu[P], gv[P];
    float2 su[P / 2], sv[P / 2];
#pragma unroll
    for (int i = 0; i < P; ++i) gu[i] = gv[i] = 1.0f;
#pragma unroll
    for (int i = 0; i < P / 2; ++i) su[i] = sv[i] = make_float2(0.0f, 0.0f);
    if (a.norm)
        unpack<L>(load<L>(static_cast<const E *>(key ? a.gain_k : a.gain_q), at, p0, a.rot, a.interleaved), at, gu, gv);
    const float inv_d = 1.0f / static_cast<float>(a.d);
    struct Item {
        Raw<L> x, g;
    };
    const uint32_t all = static_cast<uint32_t>(a.tokens) * w.split;
    for (uint32_t work = block * WARPS + warp; work < all; work += blocks * WARPS) {
        const int64_t token = work / static_cast<uint32_t>(w.split);
        const int part = static_cast<int>(work) - static_cast<int>(token) * w.split;
        auto fetch = [&](int row) {
            Item it = {};
            if (row < heads) {
                it.g = load<L>(head_row<E>(hg, token, row, sh, a.d), at, p0, a.rot, a.interleaved);
                if (a.norm) it.x = load<L>(head_row<E>(hx, token, row, sh, a.d), at, p0, a.rot, a.interleaved);
            }
            return it;
        };
        int row = part * each + sub;
        Item cur = fetch(row);
        __syncwarp();  // the table of the token before has been read
        if (a.rot > 0) angles(a, token, cosines[warp], sines[warp]);
        __syncwarp();
        float c[P], s[P];
#pragma unroll
        for (int i = 0; i < P; ++i) c[i] = 1.0f, s[i] = 0.0f;
        if (at.rotated > 0) table_row<P>(cosines[warp] + p0, c), table_row<P>(sines[warp] + p0, s);
        for (int r0 = part * each; r0 < heads; r0 += step, row += step) {
            const Item next = fetch(row + step);
            float u[P], v[P];
            unpack<L>(cur.g, at, u, v);
#pragma unroll
            for (int i = 0; i < P; i += 2) {
                if (L::VEC && at.rotated == 0) continue;
                const float2 ui = make_float2(u[i], u[i + 1]), vi = make_float2(v[i], v[i + 1]);
                const float2 ci = make_float2(c[i], c[i + 1]), si = make_float2(s[i], s[i + 1]);
                const float2 x0 = ptx::fma2(ui, ci, ptx::mul2(vi, si));
                const float2 x1 = ptx::fma2(vi, ci, ptx::mul2(ui, make_float2(-si.x, -si.y)));
                if (L::VEC || i < at.rotated) u[i] = x0.x, v[i] = x1.x;
                if (L::VEC || i + 1 < at.rotated) u[i + 1] = x0.y, v[i + 1] = x1.y;
            }
            if (a.norm) {
                float xu[P], xv[P];
                unpack<L>(cur.x, at, xu, xv);
                float2 square = make_float2(0.0f, 0.0f), dot = square;
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    const float2 xi = make_float2(xu[i], xv[i]);
                    square = ptx::fma2(xi, xi, square);
                    dot = ptx::fma2(ptx::mul2(make_float2(u[i], v[i]), xi), make_float2(gu[i], gv[i]), dot);
                }
                float sq = square.x + square.y, dt = dot.x + dot.y;
                for (int o = w.lanes / 2; o > 0; o >>= 1) {
                    sq += __shfl_xor_sync(0xffffffffu, sq, o);
                    dt += __shfl_xor_sync(0xffffffffu, dt, o);
                }
                const float r = rsqrtf(sq * inv_d + a.eps);
                // r (dy g - x r mean(dy g x r)) = r dy g - (r^3 mean(dy g x)) x
                const float m = -(r * r) * (r * (dt * inv_d));
                const float2 rr = make_float2(r, r), mm = make_float2(m, m);
                const bool live = row < heads;
#pragma unroll
                for (int i = 0; i < P; i += 2) {
                    const float2 ui = make_float2(u[i], u[i + 1]), vi = make_float2(v[i], v[i + 1]);
                    const float2 xi = make_float2(xu[i], xu[i + 1]), yi = make_float2(xv[i], xv[i + 1]);
                    if (live) {
                        su[i / 2] = ptx::fma2(ui, ptx::mul2(xi, rr), su[i / 2]);
                        sv[i / 2] = ptx::fma2(vi, ptx::mul2(yi, rr), sv[i / 2]);
                    }
                    const float2 x0 = ptx::fma2(ptx::mul2(ui, make_float2(gu[i], gu[i + 1])), rr, ptx::mul2(xi, mm));
                    const float2 x1 = ptx::fma2(ptx::mul2(vi, make_float2(gv[i], gv[i + 1])), rr, ptx::mul2(yi, mm));
                    u[i] = x0.x, u[i + 1] = x0.y, v[i] = x1.x, v[i + 1] = x1.y;
                }
            }
            if (row < heads) store<L>(const_cast<E *>(head_row<E>(ho, token, row, sh, a.d)), at, p0, a.rot, a.interleaved, u, v);
            cur = next;
        }
    }
    if (!a.norm) return;
    // lanes of a warp that hold the same components, then the block's warps in order
#pragma unroll
    for (int i = 0; i < P / 2; ++i) {
        for (int o = w.lanes; o < 32; o <<= 1) {
            su[i].x += __shfl_xor_sync(0xffffffffu, su[i].x, o);
            su[i].y += __shfl_xor_sync(0xffffffffu, su[i].y, o);
            sv[i].x += __shfl_xor_sync(0xffffffffu, sv[i].x, o);
            sv[i].y += __shfl_xor_sync(0xffffffffu, sv[i].y, o);
        }
    }
    if ((static_cast<int>(threadIdx.x) & 31) < w.lanes) {
#pragma unroll
        for (int i = 0; i < P; ++i) {
            if (i < at.pairs) {
                int ia, ib;
                straddle(at, i, p0, a.rot, a.interleaved, ia, ib);
                sums[warp][ia] = i & 1 ? su[i / 2].y : su[i / 2].x;
                sums[warp][ib] = i & 1 ? sv[i / 2].y : sv[i / 2].x;
            }
        }
    }
    __syncthreads();
    for (int c = threadIdx.x; c < a.d; c += THREADS) {
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < WARPS; ++i) s += sums[i][c];
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

// Blocks of the backward pass: two per SM of the 152, and no more than there is work for.
constexpr int BACKWARD_BLOCKS = 304;

template <typename F>
cudaError_t dispatch(bool is_bf16, const QkArgs &a, F f) {
    // Sixteen-byte pieces of first and second members (bf16: 8 elements), eight-byte ones, or elements.
    // 8192 tokens of 64 heads of 128: 63 us with the first, 106 with the second.
    auto fits = [&](int p) { return a.vec && a.d % (2 * p) == 0 && a.rot % (2 * p) == 0; };
    if (is_bf16) {
        if (fits(8)) return f(Lanes<__nv_bfloat16, 8, true>());
        if (fits(4)) return f(Lanes<__nv_bfloat16, 4, true>());
        return f(Lanes<__nv_bfloat16, 4, false>());
    }
    if (fits(4)) return f(Lanes<float, 4, true>());
    return f(Lanes<float, 4, false>());
}

// `rows` heads of each token, of which a warp takes 32 / lanes at once.  A warp per token where
// there are 16 warps for every SM, else as many as that takes, up to a step each.
Split split_of(const QkArgs &a, int pairs, int rows) {
    Split w;
    w.lanes = 1;
    while (w.lanes * 2 * pairs < a.d) w.lanes *= 2;
    const int each = 32 / w.lanes;
    const int64_t steps = (rows + each - 1) / each, want = (152 * 16 + a.tokens - 1) / a.tokens;
    w.split = static_cast<int>(want < steps ? want : steps);
    w.q = shards_of(a.heads, a.t), w.k = shards_of(a.kv_heads, a.t);
    return w;
}

}  // namespace qk

int64_t qk_partial_floats(int64_t tokens, int d) {
    return (tokens > 0 ? qk::BACKWARD_BLOCKS : 1) * static_cast<int64_t>(d);
}

cudaError_t launch_qk_forward(bool is_bf16, const QkArgs &a, bool append, cudaStream_t st) {
    return qk::dispatch(is_bf16, a, [&](auto L) {
        using Ln = decltype(L);
        const qk::Split w = qk::split_of(a, Ln::P, a.heads + (append ? 2 : 1) * a.kv_heads);
        const dim3 grid(static_cast<unsigned>((a.tokens * w.split + qk::WARPS - 1) / qk::WARPS));
        return append ? launch_pdl(qk::forward_kernel<Ln, true>, grid, qk::THREADS, 0, st, a, w)
                      : launch_pdl(qk::forward_kernel<Ln, false>, grid, qk::THREADS, 0, st, a, w);
    });
}

cudaError_t launch_qk_backward(bool is_bf16, const QkArgs &a, cudaStream_t st, int *launches) {
    *launches = 0;
    return qk::dispatch(is_bf16, a, [&](auto L) {
        using Ln = decltype(L);
        // queries and keys have warps of their own
        const qk::Split w = qk::split_of(a, Ln::P, a.heads > a.kv_heads ? a.heads : a.kv_heads);
        const int64_t most = (a.tokens * w.split + qk::WARPS - 1) / qk::WARPS;
        // blocks in proportion to the rows
        int64_t nq = qk::BACKWARD_BLOCKS * static_cast<int64_t>(a.heads) / (a.heads + a.kv_heads);
        nq = nq < 1 ? 1 : (nq > qk::BACKWARD_BLOCKS - 1 ? qk::BACKWARD_BLOCKS - 1 : nq);
        int64_t nk = qk::BACKWARD_BLOCKS - nq;
        nq = nq < most ? nq : most;
        nk = nk < most ? nk : most;
        cudaError_t e = launch_pdl(qk::backward_kernel<Ln>, dim3(static_cast<unsigned>(nq + nk)), qk::THREADS, 0, st, a, w,
                                   static_cast<int>(nq));
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
