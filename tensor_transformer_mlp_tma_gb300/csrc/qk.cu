// Per-head norms of queries and keys with the position rotation in the same pass, its
// gradient, and the same pass writing keys and values into a paged cache.
//
//   norm:      y = g x r,  r = 1 / sqrt(mean(x^2) + eps)         (per head, gains g [d])
//   rotation:  (u, v) -> a (u cos f - v sin f, u sin f + v cos f),  f = position * theta_i
//   backward:  dy = the rotation's transpose of the incoming gradient,
//              dg = sum dy x r,  dx = r (dy g - x r mean(dy g x r))
//
// Angles.  position * theta_i in fp32 is off by 2^-24 of itself: 0.06 radians at position 10^6.
// theta_i is kept as turns in units of 2^-64, rounded, so that the product modulo 2^64 is the fraction of
// a turn, off by position * 2^-65 at most; what it has beyond the nearest quarter goes to sincospif.
//
// Bound by memory: 8192 tokens of 32 heads of 128 with as many key heads (bf16, norm and rotation) take 45 us forward
// (0.27 GB, 5.9 TB/s) and 80 us backward (0.40 GB, 5.1 TB/s, with the gains' sums); fp32 86 us (6.3 TB/s) and 142 (5.7).  Each element is read once and
// written once.  A warp takes a token: its angles' factors stay in registers over the token's heads, and a head
// is held by d / 16 (bf16) or d / 8 (fp32) lanes, sixteen bytes of first members and sixteen of second members of the
// pairs each, so that the rotation needs no exchange and the norm a few shuffles.  Rows come by a queue of
// asynchronous copies into shared memory, four deep: held in registers, as many rows under way would halve the warps.
// With fewer tokens than warps a token's heads are shared out.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <mutex>

#include "kernels.h"
#include "launch.cuh"
#include "ptx.cuh"

namespace tpmlp {
namespace qk {

constexpr int THREADS = 256;
constexpr int WARPS = THREADS / 32;
// Rows on their way per lane: 32 (backward 64) bytes each.
constexpr int FORWARD_DEPTH = 4, BACKWARD_DEPTH = 4;
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

// Which P pairs of a head a lane holds.  Vector lanes have two pieces of P elements, A at a and B at b, which
// lie side by side over the lanes: a request for one of them is without gaps.
//   half:         pair i = (A[i], B[i]), of frequency fa + i; behind the rotated part A and B are halves of the rest
//   interleaved:  pair i = (A[2i], A[2i + 1]) of frequency fa + i, and then B's, from fb on
// `turn_a`, `turn_b`: whether the pairs of A and B rotate (half: the same).
// Element-wise lanes have the P pairs from `first` on, wherever those are, and the first `rotated` of them rotate.
struct Place {
    int a, b, fa, fb;
    bool turn_a, turn_b;
    int pairs;           // vector lanes: P or 0
    int first, rotated;
};

template <typename L>
__device__ __forceinline__ Place place(int lane, int d, int rot, bool interleaved) {
    constexpr int P = L::P;
    const int nf = rot / 2;
    Place at;
    at.first = lane * P;
    at.pairs = min(max(d / 2 - at.first, 0), P);
    at.rotated = min(max(nf - at.first, 0), P);
    if (interleaved) {
        at.a = P * lane, at.b = d / 2 + P * lane;
        at.fa = at.a / 2, at.fb = at.b / 2;
        at.turn_a = at.a < rot, at.turn_b = at.b < rot;
    } else {
        at.turn_a = at.turn_b = at.first < nf;
        at.fa = at.fb = at.first;
        at.a = at.turn_a ? at.first : rot + at.first - nf;
        at.b = at.a + (at.turn_a ? nf : (d - rot) / 2);
    }
    return at;
}

// The two elements of pair i.
template <typename L>
__device__ __forceinline__ void pair_at(const Place &at, int i, int rot, bool interleaved, int &ia, int &ib) {
    if (L::VEC) {
        ia = interleaved ? (i < L::P / 2 ? at.a + 2 * i : at.b + 2 * i - L::P) : at.a + i;
        ib = interleaved ? ia + 1 : at.b + i;
    } else {
        const int pair = at.first + i, nf = rot / 2;
        const bool apart = !interleaved && i < at.rotated;
        ia = apart ? pair : (interleaved ? 2 * pair : rot + 2 * (pair - nf));
        ib = apart ? nf + pair : ia + 1;
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

template <typename L>
__device__ __forceinline__ Raw<L> load(const typename L::E *row, const Place &at, int rot, bool inter) {
    Raw<L> r = {};
    if constexpr (L::VEC) {
        if (at.pairs > 0) {
            copy_in<L::WORDS / 2>(r.w, row + at.a);
            copy_in<L::WORDS / 2>(r.w + L::WORDS / 2, row + at.b);
        }
    } else {
        typename L::E e[2 * L::P];
#pragma unroll
        for (int i = 0; i < L::P; ++i) {
            int ia, ib;
            pair_at<L>(at, i, rot, inter, ia, ib);
            from_f(0.0f, e[2 * i]), from_f(0.0f, e[2 * i + 1]);
            if (i < at.pairs) e[2 * i] = row[ia], e[2 * i + 1] = row[ib];
        }
        memcpy(r.w, e, sizeof(e));
    }
    return r;
}

// A lane's queue of rows on their way: DEPTH of them are copied to places of its own in shared memory, which takes
// no registers while they come (element-wise lanes copy when they are asked for them).
template <typename L, int DEPTH>
struct Queue {
    static constexpr int PIECE = L::WORDS * 2;  // bytes
    static constexpr int BYTES = DEPTH * THREADS * 2 * PIECE;
    uint32_t base;
    __device__ explicit Queue(uint32_t smem) : base(smem + threadIdx.x * PIECE) {}
    __device__ __forceinline__ uint32_t place_of(int stage, int piece) const {
        return base + static_cast<uint32_t>(stage * 2 + piece) * (THREADS * PIECE);
    }
    __device__ __forceinline__ void push(int stage, const typename L::E *row, const Place &at, bool have) const {
        if constexpr (L::VEC) {
            if (have && at.pairs > 0) {
                copy(place_of(stage, 0), row + at.a);
                copy(place_of(stage, 1), row + at.b);
            }
        }
    }
    static __device__ __forceinline__ void copy(uint32_t to, const void *from) {
        if constexpr (PIECE == 16)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
        else
            asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(to), "l"(from) : "memory");
    }
    static __device__ __forceinline__ void commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
    // The oldest of DEPTH groups has landed.
    static __device__ __forceinline__ void wait() { asm volatile("cp.async.wait_group %0;" ::"n"(DEPTH - 1) : "memory"); }
    __device__ __forceinline__ Raw<L> take(int stage, const typename L::E *row, const Place &at, int rot, bool inter, bool have) const {
        Raw<L> r = {};
        if constexpr (L::VEC) {
            if (have && at.pairs > 0) {
                if constexpr (PIECE == 16) {
                    ptx::ld_shared_v4(place_of(stage, 0), r.w[0], r.w[1], r.w[2], r.w[3]);
                    ptx::ld_shared_v4(place_of(stage, 1), r.w[4], r.w[5], r.w[6], r.w[7]);
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) r.w[i] = ptx::ld_shared_u32(place_of(stage, i >> 1) + 4 * (i & 1));
                }
            }
        } else if (have) {
            r = load<L>(row, at, rot, inter);
        }
        return r;
    }
};

// First members to u, second members to v.
template <typename L>
__device__ __forceinline__ void unpack(const Raw<L> &r, bool inter, float (&u)[L::P], float (&v)[L::P]) {
    if constexpr (L::VEC && sizeof(typename L::E) == 2) {
        float lo[L::P], hi[L::P];  // of the words
#pragma unroll
        for (int i = 0; i < L::P; ++i) lo[i] = __uint_as_float(r.w[i] << 16), hi[i] = __uint_as_float(r.w[i] & 0xFFFF0000u);
#pragma unroll
        for (int i = 0; i < L::P; ++i) {
            u[i] = inter ? lo[i] : (i & 1 ? hi[i / 2] : lo[i / 2]);
            v[i] = inter ? hi[i] : (i & 1 ? hi[(L::P + i) / 2] : lo[(L::P + i) / 2]);
        }
        return;
    }
    typename L::E e[2 * L::P];
    memcpy(e, r.w, sizeof(e));
    if (L::VEC && !inter) {
#pragma unroll
        for (int i = 0; i < L::P; ++i) u[i] = to_f(e[i]), v[i] = to_f(e[L::P + i]);
    } else {
#pragma unroll
        for (int i = 0; i < L::P; ++i) u[i] = to_f(e[2 * i]), v[i] = to_f(e[2 * i + 1]);
    }
}

template <typename L>
__device__ __forceinline__ void store_raw(typename L::E *row, const Place &at, int rot, bool inter, const Raw<L> &r) {
    if constexpr (L::VEC) {
        if (at.pairs == 0) return;
        copy_out<L::WORDS / 2>(row + at.a, r.w);
        copy_out<L::WORDS / 2>(row + at.b, r.w + L::WORDS / 2);
    } else {
        typename L::E e[2 * L::P];
        memcpy(e, r.w, sizeof(e));
#pragma unroll
        for (int i = 0; i < L::P; ++i) {
            int ia, ib;
            pair_at<L>(at, i, rot, inter, ia, ib);
            if (i < at.pairs) row[ia] = e[2 * i], row[ib] = e[2 * i + 1];
        }
    }
}

template <typename L>
__device__ __forceinline__ void store(typename L::E *row, const Place &at, int rot, bool inter, const float (&u)[L::P],
                                      const float (&v)[L::P]) {
    if constexpr (L::VEC && sizeof(typename L::E) == 2) {
        Raw<L> r;
#pragma unroll
        for (int i = 0; i < L::P; ++i) {
            constexpr int H = L::P / 2;
            const int j = i < H ? 2 * i : 2 * (i - H);
            const float lo = inter ? u[i] : (i < H ? u[j] : v[j]), hi = inter ? v[i] : (i < H ? u[j + 1] : v[j + 1]);
            const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
            r.w[i] = *reinterpret_cast<const uint32_t *>(&b);
        }
        store_raw<L>(row, at, rot, inter, r);
        return;
    }
    typename L::E e[2 * L::P];
    if (L::VEC && !inter) {
#pragma unroll
        for (int i = 0; i < L::P; ++i) from_f(u[i], e[i]), from_f(v[i], e[L::P + i]);
    } else {
#pragma unroll
        for (int i = 0; i < L::P; ++i) from_f(u[i], e[2 * i]), from_f(v[i], e[2 * i + 1]);
    }
    Raw<L> r;
    memcpy(r.w, e, sizeof(e));
    store_raw<L>(row, at, rot, inter, r);
}

// Amplitude times cosine and sine of every pair's angle at one token, by one warp.
__device__ __forceinline__ void angles(const QkArgs &a, int64_t token, float *cosines, float *sines) {
    const uint64_t position = static_cast<uint64_t>(a.position[token]);
    for (int f = threadIdx.x & 31; f < a.rot / 2; f += 32) {
        const uint64_t turn = position * a.turns[f];
        // The nearest quarter, and the rest of at most an eighth of a turn: rounded to 24 bits, the rest is off by 2^-28
        // of a turn, where half turns from -1 to 1 would be by 2^-26 (an error of the sine of 1.6 steps of 2^-24).
        const uint32_t quarter = static_cast<uint32_t>((turn + (1ull << 61)) >> 62);
        const int32_t rest = static_cast<int32_t>((turn - (static_cast<uint64_t>(quarter) << 62)) >> 30);
        const float ac = (quarter + 1u) & 2u ? -a.amplitude : a.amplitude, as = quarter & 2u ? -a.amplitude : a.amplitude;
        float s, c;
        sincospif(static_cast<float>(rest) * 0x1p-33f, &s, &c);
        cosines[f] = ac * (quarter & 1u ? s : c);
        sines[f] = as * (quarter & 1u ? c : s);
    }
}

// What a lane's pairs are multiplied by: (u, v) -> (uu u + uv v, vu u + vv v), two pairs to a float2.
template <int P>
struct Factors {
    float2 uu[P / 2], uv[P / 2], vu[P / 2], vv[P / 2];
};

template <typename L>
__device__ __forceinline__ bool turns_pair(const Place &at, int i, bool inter) {
    return L::VEC ? (inter && i >= L::P / 2 ? at.turn_b : at.turn_a) : i < at.rotated;
}

// The pairs' entries of a table; where a pair does not rotate, `other`.
template <typename L>
__device__ __forceinline__ void entries(const float *table, const Place &at, bool inter, float other, float (&x)[L::P]) {
    constexpr int P = L::P;
#pragma unroll
    for (int i = 0; i < P; ++i) x[i] = other;
    if (at.pairs == 0) return;
    if constexpr (L::VEC) {
        const int second = inter ? at.fb : at.fa + P / 2;
        constexpr int H = P / 2;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (h == 0 ? !at.turn_a : !at.turn_b) continue;
            const float *t = table + (h == 0 ? at.fa : second);
#pragma unroll
            for (int i = 0; i < H; i += 2) {  // (frequencies of vector lanes begin at even places)
                const float2 q = *reinterpret_cast<const float2 *>(t + i);
                x[H * h + i] = q.x, x[H * h + i + 1] = q.y;
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < P; ++i)
            if (i < at.rotated) x[i] = table[at.first + i];
    }
}

template <typename L>
__device__ __forceinline__ Factors<L::P> factors(const QkArgs &a, const void *gain, const Place &at, const float *cosines, const float *sines) {
    constexpr int P = L::P;
    float gu[P], gv[P], c[P], s[P];
#pragma unroll
    for (int i = 0; i < P; ++i) gu[i] = gv[i] = 1.0f;
    if (a.norm) unpack<L>(load<L>(static_cast<const typename L::E *>(gain), at, a.rot, a.interleaved), a.interleaved, gu, gv);
    entries<L>(cosines, at, a.interleaved, 1.0f, c);
    entries<L>(sines, at, a.interleaved, 0.0f, s);
    Factors<P> f;
#pragma unroll
    for (int i = 0; i < P; i += 2) {
        f.uu[i / 2] = make_float2(gu[i] * c[i], gu[i + 1] * c[i + 1]);
        f.uv[i / 2] = make_float2(-gv[i] * s[i], -gv[i + 1] * s[i + 1]);
        f.vu[i / 2] = make_float2(gu[i] * s[i], gu[i + 1] * s[i + 1]);
        f.vv[i / 2] = make_float2(gv[i] * c[i], gv[i + 1] * c[i + 1]);
    }
    return f;
}

__device__ __forceinline__ float group_sum(float x, int lanes) {
    for (int o = lanes / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// Heads of one array, of one token: head h begins at h * step + (h / per shard) * gap.  The shard comes by a
// multiplication: inverse = ceil(2^32 / per) gives the quotient of heads below 2^32 / per; there are 2^16 at
// most, 2^15 per shard where there are several.
struct HeadMap {
    const void *p;
    int64_t row;
    uint32_t step, gap, inverse;
};
inline HeadMap map_of(const HeadRows &h, int heads, int t, int d) {
    const uint32_t per = static_cast<uint32_t>(heads / t);
    HeadMap m = {h.p, h.row, static_cast<uint32_t>(d), 0u, 0u};
    if (t > 1 && per == 1) m.step = static_cast<uint32_t>(h.shard);
    if (t > 1 && per > 1) {
        m.gap = static_cast<uint32_t>(h.shard - static_cast<int64_t>(per) * d);
        m.inverse = static_cast<uint32_t>(((1ull << 32) + per - 1) / per);
    }
    return m;
}

template <typename E>
__device__ __forceinline__ E *token_base(const HeadMap &m, int64_t token) {
    return const_cast<E *>(static_cast<const E *>(m.p)) + token * m.row;
}
__device__ __forceinline__ uint32_t head_at(const HeadMap &m, int head) {
    return static_cast<uint32_t>(head) * m.step + __umulhi(static_cast<uint32_t>(head), m.inverse) * m.gap;
}

// A warp takes one token's heads, 32 / lanes at a time, or with few tokens a `split`-th of them; its
// factors stay in registers.
struct Split {
    int lanes;   // per head
    int split;   // warps per token
    HeadMap q, k, v, oq, ok, dq, dk;
};

template <typename L, bool APPEND>
__global__ void __launch_bounds__(THREADS, 3) forward_kernel(const QkArgs a, const Split w) {
    using E = typename L::E;
    constexpr int P = L::P;
    extern __shared__ uint4 queue_mem[];
    const Queue<L, FORWARD_DEPTH> queue(ptx::smem_u32(queue_mem));
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
    const int lane = static_cast<int>(threadIdx.x) & (w.lanes - 1);
    const int each = 32 / w.lanes, sub = (static_cast<int>(threadIdx.x) & 31) / w.lanes, step = each * w.split;
    const bool inter = a.interleaved;
    const Place at = place<L>(lane, a.d, a.rot, inter);

    const E *const q = token_base<E>(w.q, token), *const k = token_base<E>(w.k, token), *const v_ = APPEND ? token_base<E>(w.v, token) : nullptr;
    E *const oq = token_base<E>(w.oq, token), *const ok = APPEND ? nullptr : token_base<E>(w.ok, token);
    auto from = [&](int row) {
        if (row < a.heads) return q + head_at(w.q, row);
        row -= a.heads;
        if (!APPEND || row < a.kv_heads) return k + head_at(w.k, row);
        return v_ + head_at(w.v, row - a.kv_heads);
    };
    int row = part * each + sub, ahead = row, stage = 0;
    auto push = [&](int at_stage) {
        if (L::VEC && ahead < rows) queue.push(at_stage, from(ahead), at, true);
        queue.commit();
        ahead += step;
    };
#pragma unroll
    for (int i = 0; i < FORWARD_DEPTH - 1; ++i) push(i);
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
        // every lane of the warp takes part in the shuffles, whether it has a row or not
        push(stage == 0 ? FORWARD_DEPTH - 1 : stage - 1);
        queue.wait();
        const bool have = row < rows;
        const Raw<L> x = queue.take(stage, L::VEC || !have ? nullptr : from(row), at, a.rot, inter, have);
        stage = stage == FORWARD_DEPTH - 1 ? 0 : stage + 1;
        const int of = row < a.heads ? 0 : (!APPEND || row < a.heads + a.kv_heads ? 1 : 2);
        if (of < 2 && of != kind) {
            f = factors<L>(a, of ? a.gain_k : a.gain_q, at, cosines[warp], sines[warp]);
            kind = of;
        }
        float u[P], v[P];
        unpack<L>(x, inter, u, v);
        float r = 1.0f;
        if (a.norm) {
            float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
            for (int i = 0; i < P; i += 2) {
                const float2 ui = make_float2(u[i], u[i + 1]), vi = make_float2(v[i], v[i + 1]);
                sum = ptx::fma2(ui, ui, sum);
                sum = ptx::fma2(vi, vi, sum);
            }
            r = rsqrtf(group_sum(sum.x + sum.y, w.lanes) * inv_d + a.eps);
        }
        if (have) {
            if (of == 2) {
                if (where >= 0)
                    store_raw<L>(static_cast<E *>(a.cache_v) + where + (row - a.heads - a.kv_heads) * a.head_stride, at, a.rot, inter, x);
            } else {
                const float2 rr = make_float2(r, r);
#pragma unroll
                for (int i = 0; i < P; i += 2) {
                    const float2 ui = make_float2(u[i], u[i + 1]), vi = make_float2(v[i], v[i + 1]);
                    float2 x0 = ptx::mul2(ui, f.uu[i / 2]), x1 = ptx::mul2(vi, f.vv[i / 2]);
                    // pairs that do not rotate are not mixed: infinities stay where they are
                    const float2 y0 = ptx::fma2(vi, f.uv[i / 2], x0), y1 = ptx::fma2(ui, f.vu[i / 2], x1);
                    const bool t0 = turns_pair<L>(at, i, inter), t1 = turns_pair<L>(at, i + 1, inter);
                    x0 = ptx::mul2(make_float2(t0 ? y0.x : x0.x, t1 ? y0.y : x0.y), rr);
                    x1 = ptx::mul2(make_float2(t0 ? y1.x : x1.x, t1 ? y1.y : x1.y), rr);
                    u[i] = x0.x, u[i + 1] = x0.y, v[i] = x1.x, v[i + 1] = x1.y;
                }
                if (of == 0)
                    store<L>(oq + head_at(w.oq, row), at, a.rot, inter, u, v);
                else if (!APPEND)
                    store<L>(ok + head_at(w.ok, row - a.heads), at, a.rot, inter, u, v);
                else if (where >= 0)
                    store<L>(static_cast<E *>(a.cache_k) + where + (row - a.heads) * a.head_stride, at, a.rot, inter, u, v);
            }
        }
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
    extern __shared__ uint4 queue_mem[];
    using Q = Queue<L, BACKWARD_DEPTH>;
    const Q grads(ptx::smem_u32(queue_mem)), inputs(ptx::smem_u32(queue_mem) + Q::BYTES);
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const int warp = static_cast<int>(threadIdx.x) >> 5;
    const bool key = static_cast<int>(blockIdx.x) >= q_blocks;
    const int block = static_cast<int>(blockIdx.x) - (key ? q_blocks : 0);
    const int blocks = key ? static_cast<int>(gridDim.x) - q_blocks : q_blocks;
    const int heads = key ? a.kv_heads : a.heads;
    const HeadMap hx = key ? w.k : w.q, hg = key ? w.dk : w.dq, ho = key ? w.ok : w.oq;
    const int lane = static_cast<int>(threadIdx.x) & (w.lanes - 1);
    const bool inter = a.interleaved;
    const int each = 32 / w.lanes, sub = (static_cast<int>(threadIdx.x) & 31) / w.lanes, step = each * w.split;
    const Place at = place<L>(lane, a.d, a.rot, inter);
    float gu[P], gv[P];
    float2 su[P / 2], sv[P / 2];
#pragma unroll
    for (int i = 0; i < P; ++i) gu[i] = gv[i] = 1.0f;
#pragma unroll
    for (int i = 0; i < P / 2; ++i) su[i] = sv[i] = make_float2(0.0f, 0.0f);
    if (a.norm)
        unpack<L>(load<L>(static_cast<const E *>(key ? a.gain_k : a.gain_q), at, a.rot, inter), inter, gu, gv);
    const float inv_d = 1.0f / static_cast<float>(a.d);
    // The rows that this lane takes, one after the other, and those that are on their way.
    const uint32_t all = static_cast<uint32_t>(a.tokens) * w.split;
    uint32_t work_ahead = block * WARPS + warp;
    int row_ahead = static_cast<int>(work_ahead % static_cast<uint32_t>(w.split)) * each + sub, stage = 0;
    auto settle = [&] {  // (a part of a token may have no rows at all)
        while (work_ahead < all && row_ahead - sub >= heads) {
            work_ahead += blocks * WARPS;
            row_ahead = static_cast<int>(work_ahead % static_cast<uint32_t>(w.split)) * each + sub;
        }
    };
    settle();
    auto push = [&](int at_stage) {
        if (L::VEC && work_ahead < all) {
            const int64_t token = work_ahead / static_cast<uint32_t>(w.split);
            if (row_ahead < heads) {
                grads.push(at_stage, token_base<E>(hg, token) + head_at(hg, row_ahead), at, true);
                if (a.norm) inputs.push(at_stage, token_base<E>(hx, token) + head_at(hx, row_ahead), at, true);
            }
            row_ahead += step;
            settle();
        }
        grads.commit();
    };
#pragma unroll
    for (int i = 0; i < BACKWARD_DEPTH - 1; ++i) push(i);
    for (uint32_t work = block * WARPS + warp; work < all; work += blocks * WARPS) {
        const int64_t token = work / static_cast<uint32_t>(w.split);
        const int part = static_cast<int>(work) - static_cast<int>(token) * w.split;
        if (part * each >= heads) continue;
        int row = part * each + sub;
        __syncwarp();  // the table of the token before has been read
        if (a.rot > 0) angles(a, token, cosines[warp], sines[warp]);
        __syncwarp();
        float c[P], s[P];
        entries<L>(cosines[warp], at, inter, 1.0f, c);
        entries<L>(sines[warp], at, inter, 0.0f, s);
        const E *const g_base = token_base<E>(hg, token), *const x_base = token_base<E>(hx, token);
        E *const o_base = token_base<E>(ho, token);
        for (int r0 = part * each; r0 < heads; r0 += step, row += step) {
            push(stage == 0 ? BACKWARD_DEPTH - 1 : stage - 1);
            grads.wait();
            const bool live = row < heads;
            const Raw<L> g = grads.take(stage, L::VEC || !live ? nullptr : g_base + head_at(hg, row), at, a.rot, inter, live);
            float u[P], v[P];
            unpack<L>(g, inter, u, v);
#pragma unroll
            for (int i = 0; i < P; i += 2) {
                const float2 ui = make_float2(u[i], u[i + 1]), vi = make_float2(v[i], v[i + 1]);
                const float2 ci = make_float2(c[i], c[i + 1]), si = make_float2(s[i], s[i + 1]);
                const float2 x0 = ptx::fma2(ui, ci, ptx::mul2(vi, si));
                const float2 x1 = ptx::fma2(vi, ci, ptx::mul2(ui, make_float2(-si.x, -si.y)));
                if (turns_pair<L>(at, i, inter)) u[i] = x0.x, v[i] = x1.x;
                if (turns_pair<L>(at, i + 1, inter)) u[i + 1] = x0.y, v[i + 1] = x1.y;
            }
            if (a.norm) {
                float xu[P], xv[P];
                unpack<L>(inputs.take(stage, L::VEC || !live ? nullptr : x_base + head_at(hx, row), at, a.rot, inter, live), inter, xu, xv);
                float2 square = make_float2(0.0f, 0.0f), dot = square;
#pragma unroll
                for (int i = 0; i < P; i += 2) {
                    const float2 xi = make_float2(xu[i], xu[i + 1]), yi = make_float2(xv[i], xv[i + 1]);
                    square = ptx::fma2(xi, xi, square);
                    square = ptx::fma2(yi, yi, square);
                    dot = ptx::fma2(ptx::mul2(make_float2(u[i], u[i + 1]), xi), make_float2(gu[i], gu[i + 1]), dot);
                    dot = ptx::fma2(ptx::mul2(make_float2(v[i], v[i + 1]), yi), make_float2(gv[i], gv[i + 1]), dot);
                }
                float sq = square.x + square.y, dt = dot.x + dot.y;
                for (int o = w.lanes / 2; o > 0; o >>= 1) {
                    sq += __shfl_xor_sync(0xffffffffu, sq, o);
                    dt += __shfl_xor_sync(0xffffffffu, dt, o);
                }
                const float r = rsqrtf(sq * inv_d + a.eps);
                // r (dy g - x r mean(dy g x r)), with no power of r above the first: r may be 1e20, or 1e-19
                const float m = -r * (r * (dt * inv_d));
                const float2 rr = make_float2(r, r), mm = make_float2(m, m);
#pragma unroll
                for (int i = 0; i < P; i += 2) {
                    const float2 ui = make_float2(u[i], u[i + 1]), vi = make_float2(v[i], v[i + 1]);
                    const float2 xi = make_float2(xu[i], xu[i + 1]), yi = make_float2(xv[i], xv[i + 1]);
                    if (live) {
                        su[i / 2] = ptx::fma2(ui, ptx::mul2(xi, rr), su[i / 2]);
                        sv[i / 2] = ptx::fma2(vi, ptx::mul2(yi, rr), sv[i / 2]);
                    }
                    const float2 x0 = ptx::mul2(ptx::fma2(ui, make_float2(gu[i], gu[i + 1]), ptx::mul2(xi, mm)), rr);
                    const float2 x1 = ptx::mul2(ptx::fma2(vi, make_float2(gv[i], gv[i + 1]), ptx::mul2(yi, mm)), rr);
                    u[i] = x0.x, u[i + 1] = x0.y, v[i] = x1.x, v[i + 1] = x1.y;
                }
            }
            if (live) store<L>(o_base + head_at(ho, row), at, a.rot, inter, u, v);
            stage = stage == BACKWARD_DEPTH - 1 ? 0 : stage + 1;
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
                pair_at<L>(at, i, a.rot, inter, ia, ib);
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

// Blocks of the backward pass: two per SM, and no more than there is work for; at most as many as the workspace has room for.
constexpr int MOST_BACKWARD_BLOCKS = 304;

template <typename F>
cudaError_t dispatch(bool is_bf16, const QkArgs &a, F f) {
    // Sixteen-byte pieces of first and second members (bf16: 8 elements), eight-byte ones, or elements.
    // 8192 tokens of 32 + 32 heads of 128 in bf16, forward and backward: 45 and 80 us with the first, 56 and 104 with the second
    // (120 of 128 rotate), 123 and 212 element by element (116 rotate; rows on 2 bytes 123 and 256).  fp32: 86 and 142 us
    // with sixteen-byte pieces, 139 and 227 element by element.
    auto fits = [&](int p) { return a.vec && a.d % (2 * p) == 0 && a.rot % (a.interleaved ? p : 2 * p) == 0; };
    if (is_bf16) {
        if (fits(8)) return f(Lanes<__nv_bfloat16, 8, true>());
        if (fits(4)) return f(Lanes<__nv_bfloat16, 4, true>());
        return f(Lanes<__nv_bfloat16, 4, false>());
    }
    if (fits(4)) return f(Lanes<float, 4, true>());
    return f(Lanes<float, 4, false>());
}

// More than 48 KB of shared memory (the kernels' own arrays among them) has to be asked for, once per device and kernel.
cudaError_t opt_in(const void *kernel, int bytes) {
    constexpr int MOST = 16;  // kernels here
    static std::mutex mu;
    static const void *done[64][MOST] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lk(mu);
    for (int i = 0; i < MOST; ++i) {
        if (done[dev][i] == kernel) return cudaSuccess;
        if (done[dev][i]) continue;
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e == cudaSuccess) done[dev][i] = kernel;
        return e;
    }
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

template <typename... P, typename... A>
cudaError_t launch(void (*kernel)(P...), dim3 grid, int smem, cudaStream_t st, A... args) {
    const cudaError_t e = smem > 0 ? opt_in(reinterpret_cast<const void *>(kernel), smem) : cudaSuccess;
    if (e != cudaSuccess) return e;
    return launch_pdl(kernel, grid, THREADS, static_cast<size_t>(smem), st, args...);
}

// `rows` heads of each token, of which a warp takes 32 / lanes at once.  A warp per token where that
// makes `warps` of them per SM, else as many as it takes, up to a step each.
Split split_of(const QkArgs &a, int pairs, int rows, int warps) {
    Split w;
    w.lanes = 1;
    while (w.lanes * 2 * pairs < a.d) w.lanes *= 2;
    const int each = 32 / w.lanes;
    const int64_t steps = (rows + each - 1) / each, want = (static_cast<int64_t>(a.sms) * warps + a.tokens - 1) / a.tokens;
    w.split = static_cast<int>(want < steps ? want : steps);
    w.q = map_of(a.q, a.heads, a.t, a.d), w.oq = map_of(a.oq, a.heads, a.t, a.d), w.dq = map_of(a.dq, a.heads, a.t, a.d);
    w.k = map_of(a.k, a.kv_heads, a.t, a.d), w.ok = map_of(a.ok, a.kv_heads, a.t, a.d), w.dk = map_of(a.dk, a.kv_heads, a.t, a.d);
    w.v = map_of(a.v, a.kv_heads, a.t, a.d);
    return w;
}

}  // namespace qk

int64_t qk_partial_floats(int64_t tokens, int d) {
    return (tokens > 0 ? qk::MOST_BACKWARD_BLOCKS : 1) * static_cast<int64_t>(d);
}

cudaError_t launch_qk_forward(bool is_bf16, const QkArgs &a, bool append, cudaStream_t st) {
    return qk::dispatch(is_bf16, a, [&](auto L) {
        using Ln = decltype(L);
        const qk::Split w = qk::split_of(a, Ln::P, a.heads + (append ? 2 : 1) * a.kv_heads, 32);
        const dim3 grid(static_cast<unsigned>((a.tokens * w.split + qk::WARPS - 1) / qk::WARPS));
        constexpr int smem = Ln::VEC ? qk::Queue<Ln, qk::FORWARD_DEPTH>::BYTES : 0;
        return append ? qk::launch(qk::forward_kernel<Ln, true>, grid, smem, st, a, w)
                      : qk::launch(qk::forward_kernel<Ln, false>, grid, smem, st, a, w);
    });
}

cudaError_t launch_qk_backward(bool is_bf16, const QkArgs &a, cudaStream_t st, int *launches) {
    *launches = 0;
    return qk::dispatch(is_bf16, a, [&](auto L) {
        using Ln = decltype(L);
        // queries and keys have warps of their own
        const qk::Split w = qk::split_of(a, Ln::P, a.heads > a.kv_heads ? a.heads : a.kv_heads, 16);
        const int64_t most = (a.tokens * w.split + qk::WARPS - 1) / qk::WARPS;
        // blocks in proportion to the rows
        const int64_t blocks = 2 * a.sms < qk::MOST_BACKWARD_BLOCKS ? 2 * a.sms : qk::MOST_BACKWARD_BLOCKS;
        int64_t nq = blocks * a.heads / (a.heads + a.kv_heads);
        nq = nq < 1 ? 1 : (nq > blocks - 1 ? blocks - 1 : nq);
        int64_t nk = blocks - nq;
        nq = nq < most ? nq : most;
        nk = nk < most ? nk : most;
        constexpr int smem = Ln::VEC ? 2 * qk::Queue<Ln, qk::BACKWARD_DEPTH>::BYTES : 0;
        cudaError_t e = qk::launch(qk::backward_kernel<Ln>, dim3(static_cast<unsigned>(nq + nk)), smem, st, a, w, static_cast<int>(nq));
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
