// Attention over a paged cache in bf16 on the tensor cores.
//
//   O = softmax(scale Q K^T over the visible keys) V,  one pass over the keys (cache_attn.cuh: who
//   takes which).
//
// Both products have the keys or the head's components as their 128 rows and the few queries as
// their columns, so that one token of one sequence costs a product of 16 columns and not of 128:
//   S^T [keys, rows] = K Q^T,   O^T [d, rows] += V^T P^T.
// K and V come by TMA as they lie in the cache, page by page: the same 128-byte-swizzled tile is a
// K-major operand for the first product and, transposed by the descriptor alone, an MN-major one
// for the second.  A thread holds one key's scores of up to 64 rows (TMEM lane = key): the weights go
// to shared memory as the line of that key, which again is an MN-major operand.
//
// A row's maximum runs over lanes, where it costs an exchange per row.  So the weights are
// 2^(s - m) with a reference m that is only renewed when some score of the tile is above it by more than
// 2^8: one comparison per score and one vote per tile; bf16 weights and fp32 sums hold 2^8 as well
// as 1.
//
// Two streams of four warps, each with scores, weights and outputs of its own, keep the tensor core
// and the arithmetic busy in turn: units of up to 64 rows give them alternate tiles (joined at
// the unit's end), units of more rows 64 rows each of the same tiles.
//
// Bound by reading the cache for up to about 128 rows, beyond that by the operands' way from shared
// memory to the tensor core.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <mutex>

#include "cache_attn.cuh"
#include "launch.cuh"
#include "ptx.cuh"
#include "tensormap.h"

namespace tpmlp {
namespace cattn {

constexpr int TR = CACHE_ATTN_TC_ROWS;  // rows per tile of a unit
constexpr int KEYS = 128;
constexpr int COLS = 64;                // rows per stream
// Two streams of a warpgroup each, and one whose first warp copies and second issues the products.
constexpr int TTHREADS = 384;
// Registers per thread: a stream's hold 64 scores and 64 sums.  Launched with 168 (three warpgroups in
// 65536), 224 + 224 + 56 = 3 x 168.
constexpr int STREAM_REGISTERS = 224, OTHER_REGISTERS = 56;
constexpr uint32_t BLOCK_BYTES = KEYS * 128;    // 128 keys of 64 components
constexpr uint32_t Q_BLOCK_BYTES = COLS * 128;  // 64 rows of 64 components
constexpr uint32_t P_BYTES = KEYS * 128;
constexpr float RENEW = 8.0f;           // log2 above the reference
constexpr uint32_t STATUS_TIMEOUT = 4;  // TPMLP_ERR_TIMEOUT
constexpr uint32_t SMALL_BYTES = 1536;

// NB blocks of 128 components of a head, each a slot of BLK blocks of 64.
template <int NB, int BLK>
struct Shape {
    static constexpr uint32_t SLOT = BLK * BLOCK_BYTES;
    static constexpr int Q_BLOCKS = NB * BLK;
    static constexpr uint32_t Q_BYTES = Q_BLOCKS * Q_BLOCK_BYTES;
    // 227 KB less the queries, the weights, the small arrays and 1 KB for alignment
    static constexpr int FIT = (232448 - 2 * static_cast<int>(Q_BYTES + P_BYTES) - static_cast<int>(SMALL_BYTES) - 1024) / static_cast<int>(SLOT);
    static constexpr int SLOTS = FIT < 10 ? FIT : 10;
    static constexpr uint32_t RING = SLOTS * SLOT;
    static constexpr uint32_t SMEM = RING + 2 * (Q_BYTES + P_BYTES) + SMALL_BYTES + 1024;
    static constexpr uint32_t TMEM = NB == 1 ? 256 : 512;  // columns: 2 x 64 of S, 2 x NB x 64 of O
};

struct Small {
    uint64_t full[10], empty[10];
    uint64_t s_full[2], p_full[2], o_done[2], q_full[2], drain;
    alignas(16) float m[2][COLS];  // references (log2), read four at a time
    uint32_t top[2][COLS]; // the tile's maxima, ordered as integers; then the factors
    uint8_t token[2][COLS]; // of a row, counted from the first row's token
    Walk<TR, KEYS>::Shared walk;
    uint32_t tmem;
    int skip[2];           // the weights' product has been done by the stream itself
    int last;
    volatile int abort;
};
static_assert(sizeof(Small) <= SMALL_BYTES && offsetof(Small, m) % 16 == 0, "small arrays");
static_assert(Shape<1, 1>::SLOTS == 10 && Shape<1, 2>::SLOTS == 5 && Shape<2, 2>::SLOTS == 4, "ring");

// Order of floats as unsigned integers (all above 0).
__device__ __forceinline__ uint32_t ordered(float x) {
    const uint32_t b = __float_as_uint(x);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float unordered(uint32_t o) { return __uint_as_float(o & 0x80000000u ? o & 0x7FFFFFFFu : ~o); }

// Ring position of a unit's i-th K or V tile: K0 K1 V0 K2 V1 ... V(n-1), NB slots each.
template <int NB>
__device__ __forceinline__ int k_pos(int i) {
    return NB * (i == 0 ? 0 : 2 * i - 1);
}
template <int NB>
__device__ __forceinline__ int v_pos(int i, int n) {
    return NB * (i < n - 1 ? 2 * i + 2 : 2 * n - 1);
}

template <int NB, int BLK>
struct Block {
    using S = Shape<NB, BLK>;
    const CacheAttnArgs &a;
    Small *sh;
    uint32_t ring, q, p;   // shared-memory addresses

    __device__ uint32_t slot(int pos) const { return ring + static_cast<uint32_t>(pos % S::SLOTS) * S::SLOT; }
    __device__ uint32_t full(int pos) const { return ptx::smem_u32(&sh->full[pos % S::SLOTS]); }
    __device__ uint32_t empty(int pos) const { return ptx::smem_u32(&sh->empty[pos % S::SLOTS]); }
    __device__ bool wait(uint32_t bar, uint32_t parity) const {
        if (ptx::mbar_wait(bar, parity, a.wait_ns, &sh->abort)) return true;
        sh->abort = 1;
        return false;
    }
    __device__ bool wait_full(int pos) const { return wait(full(pos), static_cast<uint32_t>(pos / S::SLOTS) & 1u); }
    __device__ bool wait_empty(int pos) const { return wait(empty(pos), (static_cast<uint32_t>(pos / S::SLOTS) & 1u) ^ 1u); }
    // Blocks of 64 components that block nb of a head has.
    __device__ int blocks(int nb) const { return min(BLK, (a.d - nb * 128 + 63) / 64); }
};

// Ring positions are counted modulo a multiple of the slots that keeps the phase.
template <int SLOTS>
__device__ __forceinline__ int wrap(int pos) {
    return pos % (2 * SLOTS * 4096);
}

// ---- copies: one warp --------------------------------------------------------------------------
template <int NB, int BLK>
__device__ void copy_role(const Block<NB, BLK> &B, Walk<TR, KEYS> walk, const CUtensorMap *mk, const CUtensorMap *mv,
                          int box) {
    using S = Shape<NB, BLK>;
    const CacheAttnArgs &a = B.a;
    const int lane = threadIdx.x & 31;
    const int pieces = KEYS / box;
    const unsigned page_size = static_cast<unsigned>(a.page_size);
    int pos = 0;
    int64_t issued = 0;
    bool ok = true;
    Unit u = {};
    // the page and row of this lane's piece of a tile; page -1: no keys there
    struct Piece {
        int page, row;
    };
    auto look = [&](int tile) {
        Piece x = {-1, 0};
        const int key = tile * KEYS + lane * box;
        if (lane < pieces && key < u.s.len) {
            const unsigned at = static_cast<unsigned>(key) / page_size;
            const int page = page_of(a, u.b, at);
            x.page = page < 0 ? static_cast<int>(a.pages) : page;  // past the last page: zeros
            x.row = key - static_cast<int>(at * page_size);
        }
        return x;
    };
    auto issue = [&](const CUtensorMap *map, const Piece &x) {
        const int valid = __popc(__ballot_sync(0xffffffffu, x.page >= 0));
        for (int nb = 0; nb < NB; ++nb) {
            ok = __shfl_sync(0xffffffffu, lane == 0 ? B.wait_empty(pos) : true, 0) && ok;
            if (!ok) return;
            const int blocks = B.blocks(nb);
            const uint32_t bar = B.full(pos), dst = B.slot(pos) + static_cast<uint32_t>(lane * box) * 128u;
            if (lane == 0) ptx::mbar_arrive_expect_tx(bar, static_cast<uint32_t>(valid * box * blocks) * 128u);
            __syncwarp();
            if (x.page >= 0)
                for (int k = 0; k < blocks; ++k)
                    ptx::tma_load_4d(dst + static_cast<uint32_t>(k) * BLOCK_BYTES, map, bar, nb * 128 + k * 64, x.row, u.head, x.page);
            pos = wrap<S::SLOTS>(pos + 1);
            ++issued;
        }
    };
    while (ok && walk.next(a, u)) {
        Piece here = look(u.tile0), next = {-1, 0};
        if (u.tiles > 1) next = look(u.tile0 + 1);
        issue(mk, here);
        for (int i = 0; ok && i < u.tiles; ++i) {
            Piece after = {-1, 0};
            if (i + 2 < u.tiles) after = look(u.tile0 + i + 2);
            if (i + 1 < u.tiles) issue(mk, next);
            if (ok) issue(mv, here);
            here = next, next = after;
        }
    }
    if (!ok) {
        if (lane == 0) report(a, STATUS_TIMEOUT, 1);
        // copies in flight land before anything goes on
        const int back = static_cast<int>(issued < S::SLOTS ? issued : S::SLOTS);
        for (int i = 1; i <= back; ++i) {
            const int at = pos - i < 0 ? pos - i + 2 * S::SLOTS * 4096 : pos - i;
            ptx::mbar_wait(B.full(at), static_cast<uint32_t>(at / S::SLOTS) & 1u, a.wait_ns, nullptr);
        }
    }
}

// ---- products: one thread ----------------------------------------------------------------------
template <int NB, int BLK>
__device__ void product_role(const Block<NB, BLK> &B, Walk<TR, KEYS> walk, uint32_t tmem) {
    using S = Shape<NB, BLK>;
    const CacheAttnArgs &a = B.a;
    Small *sh = B.sh;
    const int steps = (a.d + 15) / 16;
    int base = 0;
    uint32_t q_phase[2] = {0, 0}, p_phase[2] = {0, 0};
    bool ok = true;
    Unit u;
    auto bar = [&](uint64_t &x) { return ptx::smem_u32(&x); };
    while (ok && walk.next(a, u)) {
        const int n = u.tiles;
        const bool both = u.rows > COLS;  // both streams take every tile
        int width[2];
        width[0] = both ? COLS : (u.rows + 15) & ~15;
        width[1] = both ? (u.rows - COLS + 15) & ~15 : width[0];
        auto scores = [&](int s, int i, bool first) {
            if (first) {
                ok = ok && B.wait(bar(sh->q_full[s]), q_phase[s]);
                q_phase[s] ^= 1u;
            }
            if (!ok) return;
            ptx::tc_fence_after();
            const uint32_t idesc = ptx::idesc_bf16_f32(KEYS, width[s], false, false);
            const uint32_t d = tmem + static_cast<uint32_t>(s * COLS), q = B.q + static_cast<uint32_t>(s) * S::Q_BYTES;
            for (int nb = 0; nb < NB; ++nb) {
                const uint32_t tile = B.slot(wrap<S::SLOTS>(base + k_pos<NB>(i) + nb));
                for (int k = 0; k < 8 && nb * 8 + k < steps; ++k) {
                    const uint32_t ka = tile + static_cast<uint32_t>(k >> 2) * BLOCK_BYTES + (k & 3) * 32;
                    const uint32_t qa = q + static_cast<uint32_t>(nb * 2 + (k >> 2)) * Q_BLOCK_BYTES + (k & 3) * 32;
                    ptx::umma_f16_ss(d, ptx::sdesc_sw128(ka, 16, 1024), ptx::sdesc_sw128(qa, 16, 1024), idesc, nb + k > 0);
                }
            }
        };
        // the stream's weights of a tile are formed, and its scores have been read
        auto weights = [&](int s) {
            ok = ok && B.wait(bar(sh->p_full[s]), p_phase[s]);
            p_phase[s] ^= 1u;
        };
        auto outputs = [&](int s, int i, bool first) {
            if (!ok || sh->skip[s]) return;
            ptx::tc_fence_after();
            const uint32_t idesc = ptx::idesc_bf16_f32(128, width[s], true, true);
            for (int nb = 0; nb < NB; ++nb) {
                const uint32_t d = tmem + static_cast<uint32_t>(2 * COLS + (s * NB + nb) * COLS);
                const uint32_t va = B.slot(wrap<S::SLOTS>(base + v_pos<NB>(i, n) + nb)), pa = B.p + static_cast<uint32_t>(s) * P_BYTES;
                // (64 components: the second half of the 128 rows is whatever lies behind, and is not read)
                for (int k = 0; k < KEYS / 16; ++k)
                    ptx::umma_f16_ss(d, ptx::sdesc_sw128(va + k * 2048, BLOCK_BYTES, 1024),
                                     ptx::sdesc_sw128(pa + k * 2048, P_BYTES, 1024), idesc, !first || k > 0);
            }
        };
        auto release = [&](int pos) {
            for (int nb = 0; nb < NB; ++nb) ptx::umma_commit(B.empty(wrap<S::SLOTS>(base + pos + nb)));
        };
        auto arrived = [&](int pos) {
            for (int nb = 0; nb < NB; ++nb) ok = ok && B.wait_full(wrap<S::SLOTS>(base + pos + nb));
        };
        for (int i = 0; ok && i <= n; ++i) {
            if (i < n) arrived(k_pos<NB>(i));
            if (!both) {
                if (ok && i < n) {
                    scores(i & 1, i, i < 2);
                    if (!ok) break;
                    ptx::umma_commit(bar(sh->s_full[i & 1]));
                    release(k_pos<NB>(i));
                }
                if (ok && i > 0) {
                    arrived(v_pos<NB>(i - 1, n));
                    weights((i - 1) & 1);
                    outputs((i - 1) & 1, i - 1, i - 1 < 2);
                    if (!ok) break;
                    ptx::umma_commit(bar(sh->o_done[(i - 1) & 1]));
                    release(v_pos<NB>(i - 1, n));
                }
            } else {
                if (ok && i > 0) arrived(v_pos<NB>(i - 1, n));
                for (int s = 0; ok && s < 2; ++s) {
                    // the next scores first: the stream waits for them
                    if (i > 0) weights(s);
                    if (i < n) {
                        scores(s, i, i == 0);
                        if (!ok) break;
                        ptx::umma_commit(bar(sh->s_full[s]));
                    }
                    if (i > 0) {
                        outputs(s, i - 1, i == 1);
                        if (!ok) break;
                        ptx::umma_commit(bar(sh->o_done[s]));
                    }
                }
                if (!ok) break;
                if (i > 0) release(v_pos<NB>(i - 1, n));
                if (i < n) release(k_pos<NB>(i));
            }
        }
        base = wrap<S::SLOTS>(base + 2 * n * NB);
    }
    if (!ok) {
        report(a, STATUS_TIMEOUT, 2);
        // products in flight end before shared and tensor memory are given back
        ptx::umma_commit(bar(sh->drain));
        ptx::mbar_wait(bar(sh->drain), 0, a.wait_ns, nullptr);
    }
}

// ---- softmax: four warps per stream ------------------------------------------------------------
template <int NB, int BLK>
struct Stream {
    using S = Shape<NB, BLK>;
    const Block<NB, BLK> &B;
    const CacheAttnArgs &a;
    Small *sh;
    const int s, warp, lane, key;   // stream; warp of it; key of a tile (TMEM lane)
    const uint32_t scores, out, q, p;
    uint32_t s_phase = 0, o_phase = 0;
    bool failed = false;
    float l[4][16];                 // sums of this key's weights, per row

    __device__ Stream(const Block<NB, BLK> &b, uint32_t tmem, int stream)
        : B(b), a(b.a), sh(b.sh), s(stream), warp((threadIdx.x >> 5) & 3), lane(threadIdx.x & 31), key(threadIdx.x & 127),
          scores(tmem + (static_cast<uint32_t>(32 * ((threadIdx.x >> 5) & 3)) << 16) + static_cast<uint32_t>(stream * COLS)),
          out(tmem + (static_cast<uint32_t>(32 * ((threadIdx.x >> 5) & 3)) << 16) + static_cast<uint32_t>(2 * COLS + stream * NB * COLS)),
          q(b.q + static_cast<uint32_t>(stream) * S::Q_BYTES), p(b.p + static_cast<uint32_t>(stream) * P_BYTES) {}

    __device__ bool vote(bool x) const { return ptx::barrier_or(1 + s, 128, x); }
    __device__ void wait_out() {
        failed = !B.wait(ptx::smem_u32(&sh->o_done[s]), o_phase) || failed;
        o_phase ^= 1u;
        __syncwarp();
        ptx::tc_fence_after();
    }

    // Queries of rows row0 .. row0 + rows - 1 of the unit, zeros up to `width`, as the K-major operand.
    __device__ void load_q(const Unit &u, int row0, int rows, int width) {
        const int chunks = (a.d + 15) / 16 * 2;
        for (int i = key; i < width * chunks; i += 128) {
            const int row = i / chunks, c = i - row * chunks;
            uint4 x = make_uint4(0u, 0u, 0u, 0u);
            if (row < rows && c * 8 < a.d) {
                const int r = u.row0 + row0 + row, token = r / a.group;
                x = *reinterpret_cast<const uint4 *>(
                    static_cast<const __nv_bfloat16 *>(a.q) +
                    (static_cast<int64_t>(u.s.q0 + token) * a.heads + u.head * a.group + (r - token * a.group)) * a.d + c * 8);
            }
            ptx::st_shared_v4(q + static_cast<uint32_t>(c >> 3) * Q_BLOCK_BYTES + static_cast<uint32_t>(row) * 128u +
                                  (static_cast<uint32_t>((c & 7) ^ (row & 7)) << 4),
                              x.x, x.y, x.z, x.w);
        }
        const int first = (u.row0 + row0) / a.group;
        if (key < COLS) {
            sh->m[s][key] = -INFINITY;
            sh->token[s][key] = static_cast<uint8_t>((u.row0 + row0 + min(key, max(rows, 1) - 1)) / a.group - first);
        }
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&sh->q_full[s]));
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int j = 0; j < 16; ++j) l[c][j] = 0.0f;
    }

    __device__ void load_scores(uint32_t (&x)[4][16], int width) const {
#pragma unroll
        for (int c = 0; c < 4; ++c)
            if (16 * c < width) ptx::tmem_ld_32x32b_x16(scores + 16 * c, x[c]);
#pragma unroll
        for (int c = 0; c < 4; ++c)
            if (16 * c < width) ptx::tmem_ld_wait(x[c]);
    }

    // Bit r: row r sees this thread's key.  Rows behind the last see everything (their scores are zero).
    __device__ uint64_t seen(const Unit &u, int row0, int rows, int at) const {
        const uint64_t past = rows >= 64 ? 0ull : ~0ull << rows;
        const int j = at - u.s.prefix;
        if (j < 0) return ~0ull;
        if (at >= u.s.len) return past;
        if (!a.tree) {
            const int64_t from = static_cast<int64_t>(j) * a.group - (u.row0 + row0);  // rows of token j and later
            return (from <= 0 ? ~0ull : (from >= 64 ? 0ull : ~0ull << from)) | past;
        }
        if (j >= 64 * a.tree_words) return past;
        const int64_t *words = a.tree + static_cast<int64_t>(u.s.q0 + (u.row0 + row0) / a.group) * a.tree_words + (j >> 6);
        uint64_t bits = past;
        for (int r = 0; r < rows; ++r) {
            const uint64_t w = static_cast<uint64_t>(words[static_cast<int64_t>(sh->token[s][r]) * a.tree_words]);
            bits |= (w >> (j & 63) & 1ull) << r;
        }
        return bits;
    }

    // Renews the references from the tile's maxima; the sums and outputs so far take the factors.
    __device__ void renew(uint32_t (&x)[4][16], int width, bool masked, uint64_t sees, bool outputs) {
        if (key < COLS) sh->top[s][key] = 0u;
        vote(false);
        load_scores(x, width);
#pragma unroll
        for (int c = 0; c < 4; ++c)
            if (16 * c < width) {
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    float v = __uint_as_float(x[c][j]) * a.scale_log2;
                    if (masked && !(sees >> (16 * c + j) & 1ull)) v = -INFINITY;
                    v = ptx::warp_max_f32(v);
                    if (lane == ((16 * c + j) & 31)) atomicMax(&sh->top[s][16 * c + j], ordered(v));
                }
            }
        vote(false);
        if (key < width) {
            const float was = sh->m[s][key];
            float now = unordered(sh->top[s][key]);
            now = now > was ? now : was;  // NaN: as it was
            sh->m[s][key] = now;
            sh->top[s][key] = __float_as_uint(was == now ? 1.0f : exp2f(was - now));
        }
        vote(false);
        const uint32_t *factor = sh->top[s];
#pragma unroll
        for (int c = 0; c < 4; ++c)
            if (16 * c < width) {
#pragma unroll
                for (int j = 0; j < 16; ++j) l[c][j] *= __uint_as_float(factor[16 * c + j]);
            }
        if (outputs) {
#pragma unroll 1
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll 1
                for (int c = 0; c * 16 < width; ++c) {
                    uint32_t o[16];
                    ptx::tmem_ld_32x32b_x16(out + nb * COLS + 16 * c, o);
                    ptx::tmem_ld_wait(o);
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        o[j] = __float_as_uint(__uint_as_float(o[j]) * __uint_as_float(factor[16 * c + j]));
                    ptx::tmem_st_32x32b_x16(out + nb * COLS + 16 * c, o);
                }
            ptx::tmem_st_wait();
        }
    }

    // Values that are not finite would reach rows that do not see them (0 x NaN).  Those behind the
    // sequence's end are cleared; of a tile with others the stream forms the product itself, key by key.
    __device__ bool own_product(int pos, int at, int len, uint64_t sees, int width, bool first) {
        for (int nb = 0; nb < NB; ++nb) failed = !B.wait_full(wrap<S::SLOTS>(pos + nb)) || failed;
        bool odd = false;
        if (!failed) {
            for (int nb = 0; nb < NB; ++nb)
                for (int b = 0; b < B.blocks(nb); ++b) {
                    const uint32_t line = B.slot(wrap<S::SLOTS>(pos + nb)) + static_cast<uint32_t>(b) * BLOCK_BYTES + static_cast<uint32_t>(key) * 128u;
                    bool bad = false;
#pragma unroll
                    for (int c = 0; c < 8; ++c) {
                        uint32_t w[4];
                        ptx::ld_shared_v4(line + static_cast<uint32_t>((c ^ (key & 7)) << 4), w[0], w[1], w[2], w[3]);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            bad = bad || (w[i] & 0x7F80u) == 0x7F80u || (w[i] & 0x7F800000u) == 0x7F800000u;
                    }
                    if (bad && at >= len) {
#pragma unroll
                        for (int c = 0; c < 8; ++c) ptx::st_shared_v4(line + static_cast<uint32_t>(c << 4), 0u, 0u, 0u, 0u);
                    } else {
                        odd = odd || bad;
                    }
                }
        }
        if (!vote(odd && sees != ~0ull)) return false;
        // -0 marks a weight that is none
        const uint32_t line = p + static_cast<uint32_t>(key) * 128u;
        for (int r = 0; r < width; ++r)
            if (!(sees >> r & 1ull))
                asm volatile("st.shared.b16 [%0], %1;" ::"r"(line + (static_cast<uint32_t>((r >> 3) ^ (key & 7)) << 4) + (r & 7) * 2),
                             "h"(static_cast<uint16_t>(0x8000))
                             : "memory");
        vote(false);
#pragma unroll 1
        for (int nb = 0; nb < NB; ++nb) {
            const int e = key;  // component nb * 128 + key: this thread's TMEM lane
            const bool have = nb * 128 + e < a.d;
            const uint32_t v0 = B.slot(wrap<S::SLOTS>(pos + nb)) + static_cast<uint32_t>(have ? e >> 6 : 0) * BLOCK_BYTES + (e & 7) * 2;
#pragma unroll 1
            for (int c = 0; c * 16 < width; ++c) {
                uint32_t o[16];
                if (first) {
#pragma unroll
                    for (int j = 0; j < 16; ++j) o[j] = 0u;
                } else {
                    ptx::tmem_ld_32x32b_x16(out + nb * COLS + 16 * c, o);
                    ptx::tmem_ld_wait(o);
                }
#pragma unroll 1
                for (int k = 0; k < KEYS; ++k) {
                    uint16_t vb;
                    asm volatile("ld.shared.b16 %0, [%1];" : "=h"(vb) : "r"(v0 + k * 128 + (static_cast<uint32_t>(((e >> 3) & 7) ^ (k & 7)) << 4)));
                    const float v = __uint_as_float(static_cast<uint32_t>(vb) << 16);
                    uint32_t w[8];
                    ptx::ld_shared_v4(p + k * 128 + (static_cast<uint32_t>((2 * c) ^ (k & 7)) << 4), w[0], w[1], w[2], w[3]);
                    ptx::ld_shared_v4(p + k * 128 + (static_cast<uint32_t>((2 * c + 1) ^ (k & 7)) << 4), w[4], w[5], w[6], w[7]);
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        const uint32_t half = (j & 1 ? w[j >> 1] >> 16 : w[j >> 1] & 0xFFFFu);
                        if (half != 0x8000u)
                            o[j] = __float_as_uint(__uint_as_float(o[j]) + __uint_as_float(half << 16) * v);
                    }
                }
                ptx::tmem_st_32x32b_x16(out + nb * COLS + 16 * c, o);
            }
        }
        ptx::tmem_st_wait();
        return true;
    }

    // One tile: scores to weights.  k: how many this stream has done of the unit; pos: ring position of its V.
    __device__ bool tile(const Unit &u, int row0, int rows, int width, int t, int k, int pos, bool &fresh) {
        failed = !B.wait(ptx::smem_u32(&sh->s_full[s]), s_phase) || failed;
        s_phase ^= 1u;
        __syncwarp();
        ptx::tc_fence_after();
        const int at = t * KEYS + key;
        const bool masked = (t + 1) * KEYS > u.s.prefix;
        uint64_t sees = ~0ull;
        uint32_t x[4][16];
        load_scores(x, width);
        if (masked) sees = seen(u, row0, rows, at);
        bool high = fresh;
        if (!fresh) {
#pragma unroll
            for (int c = 0; c < 4; ++c)
                if (16 * c < width) {
#pragma unroll
                    for (int j = 0; j < 16; j += 4) {
                        const float4 m = *reinterpret_cast<const float4 *>(&sh->m[s][16 * c + j]);
                        const float mm[4] = {m.x, m.y, m.z, m.w};
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float y = fmaf(__uint_as_float(x[c][j + i]), a.scale_log2, -mm[i]);
                            x[c][j + i] = __float_as_uint(y);
                        }
                    }
                }
            if (masked) {
#pragma unroll
                for (int c = 0; c < 4; ++c)
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        if (!(sees >> (16 * c + j) & 1ull)) x[c][j] = 0xFF800000u;
            }
#pragma unroll
            for (int c = 0; c < 4; ++c)
                if (16 * c < width) {
#pragma unroll
                    for (int j = 0; j < 16; ++j) high = high || __uint_as_float(x[c][j]) > RENEW;
                }
        }
        bool waited = false;
        if (vote(high || failed)) {
            if (vote(failed)) return false;
            if (k > 0) {
                wait_out();
                waited = true;
            }
            renew(x, width, masked, sees, k > 0);
            fresh = false;
#pragma unroll
            for (int c = 0; c < 4; ++c)
                if (16 * c < width) {
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        const float m = sh->m[s][16 * c + j];
                        fresh = fresh || m == -INFINITY;
                        float y = m == -INFINITY ? __uint_as_float(x[c][j]) : fmaf(__uint_as_float(x[c][j]), a.scale_log2, -m);
                        if (masked && !(sees >> (16 * c + j) & 1ull)) y = -INFINITY;
                        x[c][j] = __float_as_uint(y);
                    }
                }
        }
        // the weights' space is read by the product of the tile before
        if (k > 0 && !waited) wait_out();
        const uint32_t line = p + static_cast<uint32_t>(key) * 128u;
#pragma unroll
        for (int c = 0; c < 4; ++c)
            if (16 * c < width) {
                uint32_t w[8];
#pragma unroll
                for (int j = 0; j < 16; j += 2) {
                    const float p0 = ptx::ex2_approx(__uint_as_float(x[c][j])), p1 = ptx::ex2_approx(__uint_as_float(x[c][j + 1]));
                    l[c][j] += p0;
                    l[c][j + 1] += p1;
                    const __nv_bfloat162 h = __floats2bfloat162_rn(p0, p1);
                    w[j >> 1] = *reinterpret_cast<const uint32_t *>(&h);
                }
                ptx::st_shared_v4(line + (static_cast<uint32_t>((2 * c) ^ (key & 7)) << 4), w[0], w[1], w[2], w[3]);
                ptx::st_shared_v4(line + (static_cast<uint32_t>((2 * c + 1) ^ (key & 7)) << 4), w[4], w[5], w[6], w[7]);
            }
        const bool own = masked && own_product(pos, at, u.s.len, sees, width, k == 0);
        if (key == 0) sh->skip[s] = own;
        ptx::fence_proxy_async_smem();
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&sh->p_full[s]));
        return true;
    }

    // The warp's sums of l, into the weights' space (no product reads it any more): [warp][row].
    __device__ void sum_l() {
        float v[64];
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int j = 0; j < 16; ++j) v[16 * c + j] = l[c][j];
        // halves the values at every exchange: lane ends with rows 2 lane and 2 lane + 1, bits reversed below
#pragma unroll
        for (int o = 16, n = 32; o > 0; o >>= 1, n >>= 1) {
            const bool up = lane & o;
#pragma unroll
            for (int i = 0; i < n; ++i) {
                const float send = up ? v[i] : v[i + n], keep = up ? v[i + n] : v[i];
                v[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
            }
        }
        const int row = (lane & 16 ? 32 : 0) + (lane & 8 ? 16 : 0) + (lane & 4 ? 8 : 0) + (lane & 2 ? 4 : 0) + (lane & 1 ? 2 : 0);
        const uint32_t to = p + static_cast<uint32_t>(warp * COLS + row) * 4u;
        asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(to), "f"(v[0]), "f"(v[1]) : "memory");
    }
};

__device__ __forceinline__ float ld_shared_f32(uint32_t at) { return __uint_as_float(ptx::ld_shared_u32(at)); }

template <int NB, int BLK>
__device__ void softmax_role(const Block<NB, BLK> &B, Walk<TR, KEYS> walk, uint32_t tmem, int s) {
    const CacheAttnArgs &a = B.a;
    Small *sh = B.sh;
    Stream<NB, BLK> st(B, tmem, s);
    int base = 0;
    Unit u;
    auto both_vote = [&](bool x) { return ptx::barrier_or(3, 256, x); };
    while (walk.next(a, u)) {
        const int n = u.tiles;
        const bool both = u.rows > COLS;
        const int row0 = both ? s * COLS : 0, rows = both ? min(COLS, u.rows - row0) : u.rows;
        const int width = (rows + 15) & ~15;
        const int mine = both ? n : (n + 1 - s) / 2;
        if (mine > 0) st.load_q(u, row0, rows, width);
        bool fresh = true, ok = true;
        if (mine > 0) st.vote(false);  // m and token are written
        for (int k = 0; ok && k < mine; ++k) {
            const int i = both ? k : 2 * k + s;
            ok = st.tile(u, row0, rows, width, u.tile0 + i, k, wrap<Shape<NB, BLK>::SLOTS>(base + v_pos<NB>(i, n)), fresh);
        }
        if (ok && mine > 0) {
            st.wait_out();
            st.sum_l();
        }
        base = wrap<Shape<NB, BLK>::SLOTS>(base + 2 * n * NB);
        if (both_vote(!ok || st.failed)) {
            // what this block would have added to cut units is counted, so that the next call finds
            // the counters at zero
            if (threadIdx.x == 0) {
                report(a, STATUS_TIMEOUT, 3);
                do {
                    if (u.cut && atomicAdd(a.counters + u.first, 1u) == static_cast<uint32_t>(u.last - u.first)) a.counters[u.first] = 0u;
                } while (walk.next(a, u));
            }
            return;
        }
        ptx::tc_fence_after();
        // Eight rows at a time: with the streams' tiles of the same rows, every other eight.
        const bool two = !both && n > 1;
        const int warp = st.warp, lane = st.lane;
        const uint32_t lanes = static_cast<uint32_t>(32 * warp) << 16;
        auto l_of = [&](int stream, int r) {
            const uint32_t at = B.p + static_cast<uint32_t>(stream) * P_BYTES + static_cast<uint32_t>(r) * 4u;
            return (ld_shared_f32(at) + ld_shared_f32(at + COLS * 4)) + (ld_shared_f32(at + 2 * COLS * 4) + ld_shared_f32(at + 3 * COLS * 4));
        };
        const int64_t piece = (2 * static_cast<int64_t>(blockIdx.x) + u.place) * TR;
        for (int c = both ? 0 : s; 8 * c < rows; c += both ? 1 : 2) {
            const int own = both ? s : 0;
            float f0[8], f1[8], top[8], sum[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int r = 8 * c + j;
                top[j] = sh->m[own][r];
                sum[j] = l_of(own, r);
                f0[j] = 1.0f, f1[j] = 0.0f;
                if (two) {
                    const float m0 = top[j], m1 = sh->m[1][r], l1 = l_of(1, r);
                    top[j] = fmaxf(m0, m1);
                    f0[j] = scale_of(m0, top[j]), f1[j] = scale_of(m1, top[j]);
                    sum[j] = sum[j] * f0[j] + l1 * f1[j];
                }
            }
            if (u.cut && warp == 0 && lane == 0) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (8 * c + j < rows) __stcg(a.part_ml + piece + row0 + 8 * c + j, make_float2(top[j], sum[j]));
            }
            for (int nb = 0; nb < NB; ++nb) {
                uint32_t o[8], o1[8];
                ptx::tmem_ld_32x32b_x8(tmem + lanes + static_cast<uint32_t>(2 * COLS + (own * NB + nb) * COLS + 8 * c), o);
                if (two) ptx::tmem_ld_32x32b_x8(tmem + lanes + static_cast<uint32_t>(2 * COLS + (NB + nb) * COLS + 8 * c), o1);
                ptx::tmem_ld_wait(o);
                if (two) ptx::tmem_ld_wait(o1);
                const int e = nb * 128 + 32 * warp + lane;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int r = 8 * c + j;
                    if (r >= rows || e >= a.d) continue;
                    float v = __uint_as_float(o[j]);
                    if (two) v = v * f0[j] + __uint_as_float(o1[j]) * f1[j];
                    if (u.cut) {
                        __stcg(a.part + (piece + row0 + r) * a.d + e, v);
                    } else {
                        v = sum[j] == 0.0f ? 0.0f : v / sum[j];
                        out_row<__nv_bfloat16>(a, u, row0 + r)[e] = __float2bfloat16_rn(v);
                    }
                }
            }
        }
        ptx::tc_fence_before();
        if (u.cut) __threadfence();
        both_vote(false);  // outputs, references and sums have been read
        if (u.cut) {
            if (threadIdx.x == 0) {
                const uint32_t pieces = static_cast<uint32_t>(u.last - u.first + 1);
                sh->last = atomicAdd(a.counters + u.first, 1u) == pieces - 1;
                if (sh->last) a.counters[u.first] = 0u;
                __threadfence();
            }
            both_vote(false);
            if (sh->last) join<__nv_bfloat16, TR>(a, u, threadIdx.x, 256);
        }
    }
}

template <int NB, int BLK>
__global__ void __launch_bounds__(TTHREADS, 1)
    tc_kernel(const CacheAttnArgs a, const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv, int box) {
    using S = Shape<NB, BLK>;
    extern __shared__ uint8_t raw[];
    const uint32_t start = (ptx::smem_u32(raw) + 1023u) & ~1023u;
    const uint32_t small_at = S::RING + 2 * (S::Q_BYTES + P_BYTES);
    Small *sh = reinterpret_cast<Small *>(raw + (start - ptx::smem_u32(raw)) + small_at);
    const Block<NB, BLK> B = {a, sh, start, start + S::RING, start + S::RING + 2 * S::Q_BYTES};
    const int warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) {
        for (int i = 0; i < S::SLOTS; ++i) {
            ptx::mbar_init(ptx::smem_u32(&sh->full[i]), 1);
            ptx::mbar_init(ptx::smem_u32(&sh->empty[i]), 1);
        }
        for (int s = 0; s < 2; ++s) {
            ptx::mbar_init(ptx::smem_u32(&sh->s_full[s]), 1);
            ptx::mbar_init(ptx::smem_u32(&sh->p_full[s]), 4);
            ptx::mbar_init(ptx::smem_u32(&sh->o_done[s]), 1);
            ptx::mbar_init(ptx::smem_u32(&sh->q_full[s]), 4);
            sh->skip[s] = 0;
        }
        ptx::mbar_init(ptx::smem_u32(&sh->drain), 1);
        sh->abort = 0;
        ptx::fence_mbar_init();
        ptx::prefetch_tensormap(&mk);
        ptx::prefetch_tensormap(&mv);
    }
    if (warp == 9) {
        ptx::tmem_alloc(ptx::smem_u32(&sh->tmem), S::TMEM);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    Walk<TR, KEYS> walk;
    walk.begin(a, sh->walk);  // with a __syncthreads
    ptx::tc_fence_after();
    const uint32_t tmem = sh->tmem;
    if (warp < 8) {
        ptx::more_registers<STREAM_REGISTERS>();
        softmax_role<NB, BLK>(B, walk, tmem, warp >> 2);
    } else {
        ptx::fewer_registers<OTHER_REGISTERS>();
        if (warp == 8)
            copy_role<NB, BLK>(B, walk, &mk, &mv, box);
        else if (warp == 9 && (threadIdx.x & 31) == 0)
            product_role<NB, BLK>(B, walk, tmem);
    }
    __syncwarp();
    ptx::tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, S::TMEM);
    }
}

// The cache as (component, row, head, page), a box of 64 components and `box` rows.
bool cache_map(CUtensorMap *m, const CacheAttnArgs &a, const void *base, int box) {
    const auto encode = tensor_map_encoder();
    if (!encode) {
        set_last_error("cuTensorMapEncodeTiled is not available from the driver");
        return false;
    }
    const cuuint64_t dims[4] = {static_cast<cuuint64_t>(a.d), static_cast<cuuint64_t>(a.page_size),
                                static_cast<cuuint64_t>(a.kv_heads), static_cast<cuuint64_t>(a.pages)};
    // a stride of a dimension of one is never used, but has to be a valid one
    const auto stride = [&](int64_t s, int64_t n) { return static_cast<cuuint64_t>(n > 1 ? s * 2 : 16 * ((a.d * 2 + 15) / 16)); };
    const cuuint64_t strides[3] = {stride(a.token_stride, a.page_size), stride(a.head_stride, a.kv_heads), stride(a.page_stride, a.pages)};
    const cuuint32_t boxes[4] = {64, static_cast<cuuint32_t>(box), 1, 1}, steps[4] = {1, 1, 1, 1};
    const CUresult r = encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(base), dims, strides, boxes, steps,
                              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS)
        set_last_error("cuTensorMapEncodeTiled failed (CUresult %d) for a cache of %lld pages of %lld rows", static_cast<int>(r),
                       static_cast<long long>(a.pages), static_cast<long long>(a.page_size));
    return r == CUDA_SUCCESS;
}

template <int NB, int BLK>
cudaError_t launch_tc(const CacheAttnArgs &a, int blocks, cudaStream_t st) {
    using S = Shape<NB, BLK>;
    static std::mutex mu;
    static bool set[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    {
        std::lock_guard<std::mutex> lk(mu);
        if (!set[dev]) {
            e = cudaFuncSetAttribute(tc_kernel<NB, BLK>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(S::SMEM));
            if (e != cudaSuccess) return e;
            set[dev] = true;
        }
    }
    // a box's rows lie in one page and in one tile
    int box = KEYS;
    while (a.page_size % box != 0) box /= 2;
    CUtensorMap mk, mv;
    if (!cache_map(&mk, a, a.k, box) || !cache_map(&mv, a, a.v, box)) return cudaErrorInvalidValue;
    return launch_pdl(tc_kernel<NB, BLK>, dim3(static_cast<unsigned>(blocks)), TTHREADS, S::SMEM, st, a, mk, mv, box);
}

}  // namespace cattn

bool cache_attn_tc(const CacheAttnArgs &a) { return a.vec && a.page_size % 8 == 0 && a.d % 8 == 0 && a.d <= 256; }

cudaError_t launch_cache_attn_tc(const CacheAttnArgs &a, int num_sms, cudaStream_t st) {
    if (a.d <= 64) return cattn::launch_tc<1, 1>(a, num_sms, st);
    if (a.d <= 128) return cattn::launch_tc<1, 2>(a, num_sms, st);
    return cattn::launch_tc<2, 2>(a, num_sms, st);
}

}  // namespace tpmlp
