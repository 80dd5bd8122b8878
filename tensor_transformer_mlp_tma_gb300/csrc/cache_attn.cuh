// How attention over a paged cache is divided among the blocks, and how its pieces are joined.
//
// The new tokens of a sequence and the `group` query heads that share a key head are the rows of
// one product: row r is token r / group, head r % group of the group.  A unit is (sequence, key
// head, ROWS consecutive rows); its work is its tiles of KEYS keys.  The lengths are known on the
// device only (a captured graph is replayed with other lengths), so every block adds up the tiles
// of all units itself and takes an equal share [c total / blocks, (c + 1) total / blocks) of them
// in order: long sequences are cut wherever a share ends, short ones fill a block together, and
// the shares differ by one tile at most.
//
// A unit that lies in one block is written by it.  The pieces of a cut one go to the workspace as
// (maximum, sum, unnormalised output) in fp32, two places per block: [0] for a unit that began in
// an earlier block, [1] for one that begins in this block and goes on.  A second kernel joins them in
// the order of the keys, eight rows to a block, so that results do not depend on which block ends last.
// Left to one block per unit, the join of 8 units of 64 rows in 20 pieces each (one sequence of
// 131072 keys) took 30 us of 124; the second kernel takes 5 to 8, most of it its launch.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "kernels.h"
#include "launch.cuh"
#include "ptx.cuh"

namespace tpmlp {
namespace cattn {

constexpr uint32_t STATUS_INVALID = 1;  // TPMLP_ERR_INVALID_ARG

__device__ __forceinline__ void report(const CacheAttnArgs &a, uint32_t status, uint32_t detail) {
    if (atomicCAS(a.status, 0u, status) == 0u) a.status[1] = detail;
}

// One sequence's new tokens and keys.  What does not fit is reported (by one block): a sequence whose
// q_start decreases or leaves the tokens has none (its rows may be another's), and with a length
// that is too short for its tokens or too long for the table its rows see nothing.
struct Seq {
    int q0, n;         // first new token, their number
    int len, prefix;   // keys in all, keys before the new tokens'
};

__device__ __forceinline__ Seq sequence(const CacheAttnArgs &a, int64_t b, bool tell) {
    const int s0 = a.q_start[b], s1 = a.q_start[b + 1], len = a.kv_len[b];
    const bool starts = s0 >= 0 && s1 >= s0 && s1 <= a.tokens;
    Seq s;
    s.q0 = starts ? s0 : 0, s.n = starts ? s1 - s0 : 0;
    const bool fits = len >= s.n && len <= a.max_pages * a.page_size;
    s.len = fits ? len : 0;
    s.prefix = fits ? len - s.n : 0;
    if (!(starts && fits) && tell) report(a, STATUS_INVALID, static_cast<uint32_t>(b));
    return s;
}

// Whether row `token` (counted in its sequence) sees the key.
__device__ __forceinline__ bool visible(const CacheAttnArgs &a, const Seq &s, int token, int key) {
    const int j = key - s.prefix;
    if (j < 0) return true;
    if (key >= s.len) return false;
    if (!a.tree) return j <= token;
    if (j >= 64 * a.tree_words) return false;
    return (a.tree[static_cast<int64_t>(s.q0 + token) * a.tree_words + (j >> 6)] >> (j & 63)) & 1;
}

// Tokens that rows 0 .. rows - 1 reach into: rows / group, rounded up.
__device__ __forceinline__ int tokens_of(const CacheAttnArgs &a, int rows) { return (rows + a.group - 1) / a.group; }

template <int ROWS, int KEYS>
struct Tiles {
    static __device__ __forceinline__ int row_tiles(const CacheAttnArgs &a, const Seq &s) {
        return (s.n * a.group + ROWS - 1) / ROWS;
    }
    // Tiles of the keys that the first `tokens` new tokens see, one at least: rows that see nothing are
    // written too.
    static __device__ __forceinline__ int to(const CacheAttnArgs &a, const Seq &s, int tokens) {
        const int keys = a.tree || s.len == 0 ? s.len : s.prefix + tokens;
        return max(1, (keys + KEYS - 1) / KEYS);
    }
    static __device__ __forceinline__ int of(const CacheAttnArgs &a, const Seq &s, int rt) {
        return to(a, s, min(s.n, tokens_of(a, (rt + 1) * ROWS)));
    }
    static __device__ __forceinline__ int64_t per_head(const CacheAttnArgs &a, const Seq &s) {
        const int n = row_tiles(a, s);
        if (n == 0) return 0;
        const int last = to(a, s, s.n);
        if (a.tree || s.len == 0) return static_cast<int64_t>(n) * last;
        int64_t sum = last;
        const bool even = ROWS % a.group == 0;  // a tile's rows are whole tokens
        const int step = ROWS / a.group;
        for (int rt = 0; rt < n - 1; ++rt) sum += even ? to(a, s, (rt + 1) * step) : of(a, s, rt);
        return sum;
    }
};

struct Unit {
    Seq s;
    int b, head;          // sequence, key head
    int row0, rows;       // rows of the sequence
    int tile0, tiles;     // this block's tiles of the unit
    bool cut;             // the unit has tiles in other blocks
    int place;            // of this block's piece
    int64_t begin, end;   // the unit's tiles, counted among all
};


// x y / z for z > 0: most work has fewer than 2^32 / blocks tiles, for which 32 bits do.
__device__ __forceinline__ int64_t share(int64_t x, int64_t y, int64_t z) {
    const uint64_t product = static_cast<uint64_t>(x) * static_cast<uint64_t>(y);
    if ((product >> 32) == 0 && (z >> 32) == 0) return static_cast<uint32_t>(product) / static_cast<uint32_t>(z);
    return static_cast<int64_t>(product / static_cast<uint64_t>(z));
}

struct WalkShared {
    int64_t warp_sum[8];
    int b, head, rt, tile, count;
};

// A block's share of the work.
template <int ROWS, int KEYS>
struct Walk {
    using T = Tiles<ROWS, KEYS>;
    int64_t total, pos, end;   // tiles of all, of this block
    int blocks;
    int b, head, rt, tile;     // where pos is
    int count;                 // tiles of the unit

    using Shared = WalkShared;

    // All threads (at least 256) of the block.
    __device__ void begin(const CacheAttnArgs &a, Shared &sh) {
        const int tid = threadIdx.x, lane = tid & 31;
        const int per = static_cast<int>((a.batch + 255) / 256);
        const int s0 = tid * per, s1 = static_cast<int>(min(static_cast<int64_t>(s0) + per, a.batch));
        int64_t mine = 0;
        if (tid < 256)
            for (int i = s0; i < s1; ++i) mine += a.kv_heads * T::per_head(a, sequence(a, i, blockIdx.x == 0));
        int64_t scan = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t up = __shfl_up_sync(0xffffffffu, scan, o);
            if (lane >= o) scan += up;
        }
        if (tid < 256 && lane == 31) sh.warp_sum[tid >> 5] = scan;
        __syncthreads();
        int64_t before = 0;
        total = 0;
#pragma unroll
        for (int w = 0; w < 8; ++w) {
            if (w < (tid >> 5)) before += sh.warp_sum[w];
            total += sh.warp_sum[w];
        }
        blocks = static_cast<int>(total < gridDim.x ? total : gridDim.x);
        const int64_t c = blockIdx.x;
        pos = end = 0;
        if (c < blocks) pos = share(c, total, blocks), end = share(c + 1, total, blocks);
        int64_t at = before + scan - mine;
        if (tid < 256 && at <= pos && pos < at + mine && pos < end) {
            // the sequence, key head, rows and tile at pos
            for (int i = s0; i < s1; ++i) {
                const Seq s = sequence(a, i, false);
                const int64_t ph = T::per_head(a, s), cost = a.kv_heads * ph;
                if (pos < at + cost) {
                    int64_t off = pos - at;
                    sh.b = i;
                    sh.head = static_cast<int>(share(off, 1, ph));
                    off -= sh.head * ph;
                    int r = 0, n;
                    while (off >= (n = T::of(a, s, r))) off -= n, ++r;
                    sh.rt = r, sh.count = n, sh.tile = static_cast<int>(off);
                    break;
                }
                at += cost;
            }
        }
        __syncthreads();
        b = sh.b, head = sh.head, rt = sh.rt, tile = sh.tile, count = sh.count;
    }

    __device__ __forceinline__ bool next(const CacheAttnArgs &a, Unit &u) {
        if (pos >= end) return false;
        u.s = sequence(a, b, false);
        u.b = b, u.head = head, u.row0 = rt * ROWS;
        u.rows = min(ROWS, u.s.n * a.group - u.row0);
        u.tile0 = tile;
        u.tiles = static_cast<int>(min(static_cast<int64_t>(count - tile), end - pos));
        u.begin = pos - tile, u.end = u.begin + count;
        u.cut = u.tiles != count;
        u.place = tile == 0 ? 1 : 0;
        pos += u.tiles;
        if (pos < end) {  // the next unit
            tile = 0;
            Seq s = u.s;
            if (++rt >= T::row_tiles(a, s)) {
                rt = 0;
                if (++head >= a.kv_heads) {
                    head = 0;
                    do s = sequence(a, ++b, false);
                    while (s.n == 0);
                }
            }
            count = T::of(a, s, rt);
        }
        return true;
    }

    // The block of a cut unit's last tile: c with c total / blocks <= g < (c + 1) total / blocks (whole numbers).
    __device__ int last_block(const Unit &u) const { return static_cast<int>(share(u.end * blocks - 1, 1, total)); }
};

__device__ __forceinline__ float scale_of(float from, float to) { return from == to ? 1.0f : exp2f(from - to); }

__device__ __forceinline__ void put4(float *p, float4 v) { *reinterpret_cast<float4 *>(p) = v; }
__device__ __forceinline__ void put4(__nv_bfloat16 *p, float4 v) {
    __nv_bfloat162 lo = __floats2bfloat162_rn(v.x, v.y), hi = __floats2bfloat162_rn(v.z, v.w);
    uint2 w;
    w.x = *reinterpret_cast<uint32_t *>(&lo);
    w.y = *reinterpret_cast<uint32_t *>(&hi);
    *reinterpret_cast<uint2 *>(p) = w;
}

// The output row of a unit's row.
template <typename E, typename U>
__device__ __forceinline__ E *out_row(const CacheAttnArgs &a, const U &u, int row) {
    const int r = u.row0 + row, token = r / a.group;
    return static_cast<E *>(a.o) +
           (static_cast<int64_t>(u.s.q0 + token) * a.heads + u.head * a.group + (r - token * a.group)) * a.d;
}

// A unit that begins in a block and goes on, for the kernel that joins its pieces; rows = 0: none.
__device__ __forceinline__ void post_cut(const CacheAttnArgs &a, int q0, int head, int row0, int rows, int last) {
    int4 *to = reinterpret_cast<int4 *>(a.cuts) + 2 * blockIdx.x;
    to[0] = make_int4(rows, last, q0, head);
    to[1] = make_int4(row0, 0, 0, 0);
}

constexpr int JOIN_THREADS = 256, JOIN_ROWS = 8;

// blockIdx.x: the block that a unit begins in; blockIdx.y: eight of its rows.
template <typename E, int ROWS>
__global__ void __launch_bounds__(JOIN_THREADS, 4) join_kernel(const CacheAttnArgs a) {
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const int4 *cut = reinterpret_cast<const int4 *>(a.cuts) + 2 * blockIdx.x;
    const int4 c0 = __ldcg(cut);
    const int rows = c0.x, first = blockIdx.x, last = c0.y, from = JOIN_ROWS * blockIdx.y;
    if (from >= rows) return;
    const int row0 = __ldcg(cut + 1).x;
    const int quads = a.d / 4;
    for (int i = threadIdx.x; i < min(JOIN_ROWS, rows - from) * quads; i += JOIN_THREADS) {
        const int row = from + i / quads, e = (i % quads) * 4;
        float m = -INFINITY, l = 0.0f;
        float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        // four pieces under way at a time
        for (int c = first; c <= last; c += 4) {
            float2 ml[4];
            float4 y[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int from_block = min(c + k, last);
                const int64_t at = (2 * static_cast<int64_t>(from_block) + (from_block == first ? 1 : 0)) * ROWS + row;
                ml[k] = __ldcg(a.part_ml + at);
                y[k] = __ldcg(reinterpret_cast<const float4 *>(a.part + at * a.d + e));
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (c + k > last) break;
                const float top = fmaxf(m, ml[k].x), f = scale_of(m, top), g = scale_of(ml[k].x, top);
                l = l * f + ml[k].y * g;
                x.x = x.x * f + y[k].x * g;
                x.y = x.y * f + y[k].y * g;
                x.z = x.z * f + y[k].z * g;
                x.w = x.w * f + y[k].w * g;
                m = top;
            }
        }
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;  // a row that sees nothing: zeros
        const int r = row0 + row, token = r / a.group;
        E *o = static_cast<E *>(a.o) + (static_cast<int64_t>(c0.z + token) * a.heads + c0.w * a.group + (r - token * a.group)) * a.d + e;
        put4(o, make_float4(x.x * inv, x.y * inv, x.z * inv, x.w * inv));
    }
}

template <typename E, int ROWS>
cudaError_t launch_join(const CacheAttnArgs &a, int blocks, cudaStream_t st) {
    const int64_t all = a.tokens * a.group, rows = all < ROWS ? all : ROWS;
    const dim3 grid(static_cast<unsigned>(blocks), static_cast<unsigned>((rows + JOIN_ROWS - 1) / JOIN_ROWS));
    return launch_pdl(join_kernel<E, ROWS>, grid, JOIN_THREADS, 0, st, a);
}

}  // namespace cattn
}  // namespace tpmlp
