// Attention over a paged cache in bf16 on the tensor cores.
//
//   O = softmax(scale Q K^T over the visible keys) V,  one pass over the keys (cache_attn.cuh: who
//   takes which).
//
// K and V come by TMA as they lie in the cache, page by page, in tiles of 128 keys: the same
// 128-byte-swizzled tile is a K-major operand for the first product and an MN-major one for the second.
// One warp copies K, one V, one issues the products, one hands out the units (sequence, key head, rows), and two
// streams of four warps, each with scores, weights and outputs of its own, take the tiles in turn, so that
// the tensor core and the arithmetic are both kept busy; they are added up at the unit's end.
//
// Few rows (Narrow): both products have the keys or the head's components as their 128 rows and the
// rows of queries as their columns, so that one token of one sequence costs a product of 16 columns and
// not of 128:
//   S^T [keys, rows] = K Q^T,   O^T [d, rows] += V^T P^T,   l^T += 1 P^T.
// A thread holds one key's scores of up to 64 rows (TMEM lane = key): the weights go to shared memory
// as the line of that key, an MN-major operand.  A row's maximum would run over lanes, an exchange per
// row: the reference is renewed by a vote (below), and the sums of the weights are a product with ones.
//
// More rows (Wide): S [rows, keys] = Q K^T, O [rows, d] += P V, a thread holding a row: maximum and sum are
// its own, masks are a row's 32 bits at a time, and the weights go back to tensor memory in place of the
// scores, as the second product's first operand: shared memory, which the products' operands keep busy,
// carries half as much as with the weights in it.  4 prompt chunks of 300 to 512 tokens over 3000 to 8192 keys,
// 64 heads on 8 of 128 components: 352 to 359 us, 1.25 PFLOP/s, in bursts of a few ms, and 380 to 400 (1.15) one after another
// for longer, when the power limit lowers the clock; with the weights in shared memory 622.
//
// In both the weights are 2^(s - m) with a reference m that is only renewed when some score of the tile is
// above it by more than 2^8: bf16 weights and fp32 sums hold 2^8 as well as 1, and outputs are
// scaled a few times per row instead of once per tile.
//
// The weights are rounded to bf16, because they are operands of a bf16 product whose other one is the cache as it is: at most
// 2^-8 of each, next to the 2^-8 of the rounded output (against 64 bits an output of the decoding batch is off by 2.3e-3, with
// weights in fp32 by 1.7e-3).  Two parts per weight would be two products of V instead of one.  Scores, references, sums and
// outputs are fp32; Narrow's sums are of the rounded weights (one more product), Wide's of the unrounded ones, which it has
// in registers when it adds them up.
//
// Narrow is bound by reading the cache: 64 sequences of one token, 1.19 GB: 185 us, 6.4 TB/s.  Wide is bound by the
// turns of a stream between its products and its exponentials, of about 1700 cycles each for a tile (the products of
// both streams' tiles alone are 1060), and at the units' ends by the outputs' way to memory.
// One sequence of one token over 2048 keys takes 16.4 us with the join, over a single key 9.9.
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

constexpr int KEYS = 128;
constexpr int COLS = 64;                // rows per stream
// Two streams of a warpgroup each, and one whose warps issue the products, copy K, copy V and plan.
constexpr int TTHREADS = 384;
constexpr uint32_t BLOCK_BYTES = KEYS * 128;    // 128 keys of 64 components
constexpr uint32_t Q_BLOCK_BYTES = 2 * COLS * 128;  // 128 rows (64 of each stream) of 64 components
constexpr uint32_t P_BYTES = KEYS * 128;
// What else a stream's weights' space holds while no product reads it: per warp and row a maximum or a
// sum; per row the factor of the outputs, that of the other stream's, and the output's row.
constexpr uint32_t P_WARPS = 0, P_FACTOR = 1024, P_OTHER = 1280, P_ROW = 1536;
constexpr float RENEW = 8.0f;           // log2 above the reference
constexpr uint32_t STATUS_TIMEOUT = 4;  // TPMLP_ERR_TIMEOUT
constexpr uint32_t SMALL_BYTES = 2048;

// NB blocks of 128 components of a head, each a slot of BLK blocks of 64.  WIDE: rows in lanes.
template <int NB, int BLK, bool WIDE>
struct Shape {
    static_assert(2 * COLS == CACHE_ATTN_TC_ROWS, "the workspace's pieces");
    static constexpr uint32_t SLOT = BLK * BLOCK_BYTES;
    static constexpr int Q_BLOCKS = NB * BLK;
    static constexpr uint32_t Q_BYTES = Q_BLOCKS * Q_BLOCK_BYTES;  // of both streams
    // 227 KB less the queries, the weights, the small arrays and 1 KB for alignment
    static constexpr uint32_t P_ALL = WIDE ? 0 : 2 * P_BYTES;
    static constexpr int FIT = (232448 - static_cast<int>(Q_BYTES + P_ALL) - static_cast<int>(SMALL_BYTES) - 1024) / static_cast<int>(SLOT);
    static constexpr int SLOTS = FIT < 10 ? FIT : 10;
    // V waits for the weights of its tile, K for nothing
    static constexpr int K_SLOTS = SLOTS / 2, V_SLOTS = SLOTS - K_SLOTS;
    static constexpr uint32_t RING = SLOTS * SLOT;
    static constexpr uint32_t SMEM = RING + Q_BYTES + P_ALL + SMALL_BYTES + 1024;
    static constexpr int ROWS = WIDE ? 2 * COLS : COLS;  // of a unit
};
constexpr uint32_t TMEM = 512;          // columns: 2 x 2 x 64 of S, 2 x NB x 64 of O, for NB = 1 2 x 64 of sums
constexpr uint32_t O_COLUMN = 4 * COLS, L_COLUMN = 6 * COLS;

// A unit as the planning warp hands it to the others.  tiles = 0: there are no more.
struct alignas(16) Job {
    Seq s;
    int b, head, row0, rows;
    int tile0, tiles, cut, place;
    int last, unused[3];   // last block of a unit that begins here and is cut
};
constexpr int JOBS = 3;
constexpr int JOB_READERS = 11;  // warps: the streams' eight, products, copies of K and of V

// Slots of a ring that have been copied to (a bit each), and the phase of the last copy into each.
struct Copied {
    uint32_t slots, phases;
};

struct Small {
    Job job[JOBS];
    uint64_t job_full[JOBS], job_empty[JOBS];
    uint64_t full[10], empty[10];  // of K's slots, then V's
    uint64_t s_full[2][2], p_full[2], o_done[2], q_full[2], drain;
    float m[2][COLS];      // references (log2)
    alignas(16) float ref[2][COLS];  // their negatives, 0 for a row that has seen nothing yet
    WalkShared walk;
    uint32_t tmem;
    int skip[2];           // the weights' product has been done by the stream itself
    alignas(16) uint32_t ones[96];  // in bf16: 128 x 16 of them, whose groups of 8 x 8 (128 bytes) begin 16 bytes apart
    Copied copied[2];      // K's and V's, when their roles have ended
    volatile int abort;
};
static_assert(sizeof(Small) <= SMALL_BYTES && offsetof(Small, ref) % 16 == 0, "small arrays");
static_assert(Shape<1, 1, false>::SLOTS == 10 && Shape<1, 2, false>::SLOTS == 5 && Shape<2, 2, false>::SLOTS == 4, "ring");
static_assert(Shape<1, 1, true>::SLOTS == 10 && Shape<1, 2, true>::SLOTS == 6 && Shape<2, 2, true>::SLOTS == 5, "ring");

template <int NB, int BLK, bool WIDE>
struct Block {
    using S = Shape<NB, BLK, WIDE>;
    const CacheAttnArgs &a;
    Small *sh;
    uint32_t ring, q, p;   // shared-memory addresses

    __device__ uint32_t bar(const uint64_t &x) const { return ptx::smem_u32(&x); }
    __device__ bool wait(uint32_t bar, uint32_t parity) const {
        if (ptx::mbar_try_wait(bar, parity)) return true;
        if (sh->abort) return false;
        // the clock is looked at only after many tries
#pragma unroll 1
        for (int i = 0; i < 64; ++i)
            if (ptx::mbar_try_wait(bar, parity)) return true;
        if (ptx::mbar_wait(bar, parity, a.wait_ns, &sh->abort)) return true;
        sh->abort = 1;
        return false;
    }
    // For copies and products under way after a wait has run out: 0.1 s at least, whatever the limit of waits.
    __device__ uint64_t drain_ns() const { return a.wait_ns > 100000000ull ? a.wait_ns : 100000000ull; }
    // `wait` for a whole warp.
    __device__ bool warp_wait(uint32_t bar, uint32_t parity) const {
        if (__all_sync(0xffffffffu, ptx::mbar_try_wait(bar, parity))) return true;
        return __all_sync(0xffffffffu, wait(bar, parity));
    }
    // Blocks of 64 components that block nb of a head has.
    __device__ int blocks(int nb) const { return min(BLK, (a.d - nb * 128 + 63) / 64); }
};

// A place in a ring.
struct Place {
    int slot = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next(int slots) {
        if (++slot == slots) slot = 0, phase ^= 1u;
    }
};

// Takes the jobs in order; all lanes of the warp.
template <int NB, int BLK, bool WIDE>
struct Jobs {
    const Block<NB, BLK, WIDE> &B;
    Place at;
    __device__ void read(Job &j, int slot) const {
        const uint32_t from = ptx::smem_u32(&B.sh->job[slot]);
        uint32_t w[16];
#pragma unroll
        for (int i = 0; i < 16; i += 4) ptx::ld_shared_v4(from + 4 * i, w[i], w[i + 1], w[i + 2], w[i + 3]);
        memcpy(&j, w, sizeof(j));
    }
    // The job at hand (waiting for it the first time), and the one behind it.
    __device__ bool peek(Job &j) const {
        if (!B.warp_wait(B.bar(B.sh->job_full[at.slot]), at.phase)) return false;
        read(j, at.slot);
        return true;
    }
    __device__ bool peek_next(Job &j) const {
        Place next = at;
        next.next(JOBS);
        if (!B.warp_wait(B.bar(B.sh->job_full[next.slot]), next.phase)) return false;
        read(j, next.slot);
        return true;
    }
    __device__ void release() {
        __syncwarp();
        if ((threadIdx.x & 31) == 0) ptx::mbar_arrive(B.bar(B.sh->job_empty[at.slot]));
        at.next(JOBS);
    }
    __device__ bool get(Job &j) {
        if (!peek(j)) return false;
        release();
        return true;
    }
};

// ---- planning: one warp ------------------------------------------------------------------------
// Reads the lengths and hands out the units ahead of time, so that no other warp waits for them, and
// brings the units' queries near.
template <int NB, int BLK, bool WIDE>
__device__ void plan_role(const Block<NB, BLK, WIDE> &B, Walk<Shape<NB, BLK, WIDE>::ROWS, KEYS> walk) {
    const CacheAttnArgs &a = B.a;
    const int lane = threadIdx.x & 31;
    Place at;
    Unit u = {};
    bool more = true;
    while (more) {
        more = walk.next(a, u);
        Job j = {};
        if (more) {
            j.s = u.s, j.b = u.b, j.head = u.head, j.row0 = u.row0, j.rows = u.rows;
            j.tile0 = u.tile0, j.tiles = u.tiles, j.cut = u.cut, j.place = u.place;
            if (u.cut && u.place == 1) j.last = walk.last_block(u);
        }
        if (!B.warp_wait(B.bar(B.sh->job_empty[at.slot]), at.phase ^ 1u)) return;
        if (lane == 0) {
            B.sh->job[at.slot] = j;
            ptx::mbar_arrive(B.bar(B.sh->job_full[at.slot]));
        }
        __syncwarp();
        at.next(JOBS);
        if (more) {
            // a line for every 64 components of every row
            const int per = (a.d + 63) / 64;
#pragma unroll 1
            for (int i = lane; i < u.rows * per; i += 32) {
                const int row = i / per, r = u.row0 + row, token = r / a.group;
                const __nv_bfloat16 *q = static_cast<const __nv_bfloat16 *>(a.q) +
                                         (static_cast<int64_t>(u.s.q0 + token) * a.heads + u.head * a.group + (r - token * a.group)) * a.d +
                                         (i - row * per) * 64;
                asm volatile("prefetch.global.L2 [%0];" ::"l"(q));
            }
        }
    }
}

// ---- copies: one warp for K, one for V -----------------------------------------------------------
template <int NB, int BLK, bool WIDE>
__device__ void copy_role(const Block<NB, BLK, WIDE> &B, bool values, const CUtensorMap *map, int box) {
    using S = Shape<NB, BLK, WIDE>;
    const CacheAttnArgs &a = B.a;
    const int lane = threadIdx.x & 31;
    const int pieces = KEYS / box;
    const unsigned page_size = static_cast<unsigned>(a.page_size);
    const bool leader = ptx::elect_one();
    const int first = values ? S::K_SLOTS : 0, slots = values ? S::V_SLOTS : S::K_SLOTS;
    const uint32_t ring = B.ring + static_cast<uint32_t>(first) * S::SLOT;
    const uint32_t full0 = B.bar(B.sh->full[first]), empty0 = B.bar(B.sh->empty[first]);
    Place at;
    Copied copied = {0, 0};
    bool ok = true;
    Jobs<NB, BLK, WIDE> jobs = {B, {}};
    Job job = {};
    int tile = 0;
    // A tile: key head and sequence (none: -1), and the page (as the table has it) and row of this lane's
    // piece; row -1: no keys there.  Looked up two tiles ahead: under load a word of the table takes as
    // long as a tile.
    struct Piece {
        int head, b, page, row;
    };
    auto look = [&] {
        Piece x = {-1, 0, 0, -1};
        if (tile == job.tiles) {
            tile = 0;
            if (job.head >= 0 && !jobs.get(job)) {
                ok = false;
                job.tiles = 0;
            }
            if (job.tiles == 0) {
                job.head = -1;
                return x;
            }
        }
        x.head = job.head, x.b = job.b;
        const int key = (job.tile0 + tile) * KEYS + lane * box;
        if (lane < pieces && key < job.s.len) {
            const unsigned n = static_cast<unsigned>(key) / page_size;
            x.page = a.table[job.b * a.max_pages + n];
            x.row = key - static_cast<int>(n * page_size);
        }
        ++tile;
        return x;
    };
    Piece next = {-1, 0, 0, -1}, after = next;
#pragma unroll 1
    for (int t = -2;; ++t) {
        Piece x = next;
        next = after;
        after = look();
        if (t < 0) continue;
        if (!ok || x.head < 0) break;
        if (x.row >= 0 && (x.page < 0 || x.page >= a.pages)) {
            report(a, STATUS_INVALID, static_cast<uint32_t>(x.b));
            x.page = static_cast<int>(a.pages);  // past the last page: zeros
        }
        const int valid = __popc(__ballot_sync(0xffffffffu, x.row >= 0));
#pragma unroll 1
        for (int nb = 0; nb < NB; ++nb) {
            ok = B.warp_wait(empty0 + 8 * at.slot, at.phase ^ 1u);
            if (!ok) break;
            const int blocks = B.blocks(nb);
            const uint32_t bar = full0 + 8 * at.slot, dst = ring + static_cast<uint32_t>(at.slot) * S::SLOT;
            if (leader) ptx::mbar_arrive_expect_tx(bar, static_cast<uint32_t>(valid * box * blocks) * 128u);
#pragma unroll 1
            for (int p = 0; p < valid; p += 4) {
                int page[4], row[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    page[j] = __shfl_sync(0xffffffffu, x.page, p + j);
                    row[j] = __shfl_sync(0xffffffffu, x.row, p + j);
                }
                if (leader) {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (p + j < valid) {
                            const uint32_t to = dst + static_cast<uint32_t>((p + j) * box) * 128u;
                            ptx::tma_load_4d(to, map, bar, nb * 128, row[j], x.head, page[j]);
                            if (BLK > 1 && blocks > 1) ptx::tma_load_4d(to + BLOCK_BYTES, map, bar, nb * 128 + 64, row[j], x.head, page[j]);
                        }
                }
            }
            copied.slots |= 1u << at.slot;
            copied.phases = (copied.phases & ~(1u << at.slot)) | at.phase << at.slot;
            at.next(slots);
        }
        if (!ok) break;
    }
    if (lane == 0) {
        B.sh->copied[values] = copied;
        if (!ok) report(a, STATUS_TIMEOUT, 1);
    }
}
// After a timeout: copies in flight land.  (Functions of their own: inlined they cost the drafts 1 us of 60.)
__device__ __noinline__ void drain_copies(uint32_t full0, Copied copied, uint64_t limit_ns) {
#pragma unroll 1
    for (int i = 0; copied.slots >> i != 0; ++i)
        if (copied.slots >> i & 1u) ptx::mbar_wait(full0 + 8 * i, copied.phases >> i & 1u, limit_ns, nullptr);
}

// ---- products: one warp --------------------------------------------------------------------------
// Narrow: scores run ahead of outputs by a tile per stream, which has two places for them.  Wide: a tile's
// weights lie in place of its scores, so that a place is free for new ones behind the product that reads
// them.  All products of Wide have one shape (128 x 128 x 16): the tensor core takes them in order.
template <int NB, int BLK, bool WIDE>
__device__ void product_role(const Block<NB, BLK, WIDE> &B, uint32_t tmem) {
    using S = Shape<NB, BLK, WIDE>;
    const CacheAttnArgs &a = B.a;
    Small *sh = B.sh;
    const int steps = (a.d + 15) / 16;
    const bool leader = ptx::elect_one();
    const uint32_t v_ring = B.ring + S::K_SLOTS * S::SLOT;
    const uint32_t k_full = B.bar(sh->full[0]), v_full = B.bar(sh->full[S::K_SLOTS]);
    const uint32_t to_empty = B.bar(sh->empty[0]) - k_full;
    Place kp, vp;
    const uint64_t ones = ptx::sdesc_plain(ptx::smem_u32(sh->ones), 16, 16);
    uint32_t q_phase = 0, p_phase = 0;  // a bit per stream
    bool ok = true;
    Jobs<NB, BLK, WIDE> jobs = {B, {}};
    Job u;
    auto queries = [&](int s) {
        ok = ok && B.warp_wait(B.bar(sh->q_full[s]), q_phase >> s & 1u);
        q_phase ^= 1u << s;
    };
    // the stream's weights of a tile are formed, and its scores have been read
    auto weights = [&](int s) {
        ok = ok && B.warp_wait(B.bar(sh->p_full[s]), p_phase >> s & 1u);
        p_phase ^= 1u << s;
    };
    // The next tile of a ring: its descriptors, and the barriers that give its slots back.
    auto take = [&](Place &at, int slots, uint32_t full, uint32_t ring, uint32_t lbo, uint64_t (&desc)[NB], uint32_t (&free)[NB]) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            ok = ok && B.warp_wait(full + 8 * at.slot, at.phase);
            desc[nb] = ptx::sdesc_sw128(ring + static_cast<uint32_t>(at.slot) * S::SLOT, lbo, 1024);
            free[nb] = full + to_empty + 8 * at.slot;
            at.next(slots);
        }
    };
    uint64_t kd[NB], vd[NB];
    uint32_t free[NB];
    auto take_k = [&] { take(kp, S::K_SLOTS, k_full, B.ring, 16, kd, free); };
    // (64 components: the second half of the 128 is whatever lies behind, and is not read)
    auto take_v = [&] { take(vp, S::V_SLOTS, v_full, v_ring, BLOCK_BYTES, vd, free); };
    // Scores of a tile, or a half of their products (steps of 16 components `from` to `to` of every block of 128).
    auto scores = [&](uint32_t d, uint32_t q0, uint32_t idesc, int from = 0, int to = 4 * BLK) {
        const uint64_t q = ptx::sdesc_sw128(q0, 16, 1024);
        // descriptors count 16 bytes: 16 components on are 2, 64 a block
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int c = from; c < to; ++c)
                if (nb * 8 + c < steps) {
                    const uint64_t kc = kd[nb] + static_cast<uint64_t>((c >> 2) * (BLOCK_BYTES >> 4) + (c & 3) * 2);
                    const uint64_t qc = q + static_cast<uint64_t>((nb * 2 + (c >> 2)) * (Q_BLOCK_BYTES >> 4) + (c & 3) * 2);
                    ptx::umma_f16_ss(d, WIDE ? qc : kc, WIDE ? kc : qc, idesc, nb + c > 0);
                }
    };
    auto give_back = [&] {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) ptx::umma_commit(free[nb]);
    };
    while (ok && (ok = jobs.get(u)) && u.tiles > 0) {
        const int n = u.tiles;
        if constexpr (WIDE) {
            // a scale below zero: the products with -Q
            const uint32_t s_desc = ptx::idesc_bf16_f32(128, KEYS, false, false) | (a.scale_log2 < 0.0f ? ptx::IDESC_NEGATE_A : 0u);
            const uint32_t o_desc = ptx::idesc_bf16_f32(128, 128, false, true);
            // Waits stand between products: the queue holds a few of them, and an open barrier too
            // takes 150 cycles and more to be seen, with shared memory as busy as it is.
            auto place = [&](int i) { return tmem + static_cast<uint32_t>(i & 1) * 128u; };
            auto have_scores = [&](int i, const uint32_t (&slots)[NB]) {
                ptx::umma_commit(B.bar(sh->s_full[NB == 1 ? i & 1 : 0][NB == 1 ? 0 : i & 1]));
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) ptx::umma_commit(slots[nb]);
            };
            queries(0), queries(1);
            for (int i = 0; ok && i < 2 && i < n; ++i) {
                take_k();
                if (!ok) break;
                ptx::tc_fence_after();
                if (leader) {
                    scores(place(i), B.q, s_desc);
                    have_scores(i, free);
                }
            }
            uint64_t v[NB];
            uint32_t v_free[NB];
            auto next_v = [&] {
                take_v();
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) v[nb] = vd[nb], v_free[nb] = free[nb];
            };
            if (ok) next_v();
#pragma unroll 1
            for (int o = 0; ok && o < n; ++o) {
                const int s = NB == 1 ? o & 1 : 0;
                weights(s);
                if (!ok) break;
                ptx::tc_fence_after();
                const bool skip = sh->skip[s] != 0, more = o + 2 < n;
                const uint32_t d = tmem + O_COLUMN + static_cast<uint32_t>(s) * 128u;
                auto outputs = [&](int from, int to) {
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                        for (int c = from; c < to; ++c)  // 16 keys on are 8 columns of weights
                            ptx::umma_f16_ts(d + nb * 128, place(o) + 8 * c, v[nb] + static_cast<uint64_t>(c * 128), o_desc,
                                             o >= (NB == 1 ? 2 : 1) || c > 0);
                };
                if (leader && !skip) outputs(0, KEYS / 32);
                if (more) take_k();
                if (!ok) break;
                ptx::tc_fence_after();
                if (leader) {
                    if (!skip) outputs(KEYS / 32, KEYS / 16);
                    if (NB > 1 || o + 2 >= n) ptx::umma_commit(B.bar(sh->o_done[s]));
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb) ptx::umma_commit(v_free[nb]);
                    if (more) scores(place(o), B.q, s_desc, 0, 2 * BLK);
                }
                uint32_t k_free[NB];
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) k_free[nb] = free[nb];
                // (NB = 2: the slots hold V of a tile and a half, and the next one comes late)
                if (NB == 1 && o + 1 < n) next_v();
                if (!ok) break;
                if (leader && more) {
                    scores(place(o), B.q, s_desc, 2 * BLK, 4 * BLK);
                    have_scores(o, k_free);
                }
                if (NB > 1 && o + 1 < n) next_v();
            }
        } else {
            const int width = (u.rows + 15) & ~15;
            const uint32_t s_desc = ptx::idesc_bf16_f32(KEYS, width, false, false), o_desc = ptx::idesc_bf16_f32(128, width, true, true);
#pragma unroll 1
            for (int i = 0; ok && i < n + 2; ++i) {
                if (i < n) {
                    const int s = i & 1, k = i >> 1;
                    take_k();
                    if (k == 0) queries(s);
                    if (!ok) break;
                    ptx::tc_fence_after();
                    if (leader) {
                        scores(tmem + static_cast<uint32_t>((2 * (k & 1) + s) * COLS), B.q + static_cast<uint32_t>(s) * COLS * 128u, s_desc);
                        ptx::umma_commit(B.bar(sh->s_full[s][k & 1]));
                        give_back();
                    }
                }
                const int o = i - 2;
                if (o >= 0) {
                    const int s = o & 1, k = o >> 1;
                    take_v();
                    weights(s);
                    if (!ok) break;
                    ptx::tc_fence_after();
                    if (leader) {
                        const uint64_t p = ptx::sdesc_sw128(B.p + static_cast<uint32_t>(s) * P_BYTES, P_BYTES, 1024);
                        if (sh->skip[s] == 0) {
                            const uint32_t d = tmem + O_COLUMN + static_cast<uint32_t>(s * COLS);
                            // 16 keys on are 128
#pragma unroll
                            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                                for (int c = 0; c < KEYS / 16; ++c)
                                    ptx::umma_f16_ss(d + nb * 2 * COLS, vd[nb] + static_cast<uint64_t>(c * 128), p + static_cast<uint64_t>(c * 128),
                                                     o_desc, k > 0 || c > 0);
                        }
                        if (NB == 1) {
                            // sums of the weights: one more product, with ones for V (each lane has all of them)
                            const uint32_t l_desc = ptx::idesc_bf16_f32(128, width, false, true);
                            const uint32_t d = tmem + L_COLUMN + static_cast<uint32_t>(s * COLS);
#pragma unroll
                            for (int c = 0; c < KEYS / 16; ++c)
                                ptx::umma_f16_ss(d, ones, p + static_cast<uint64_t>(c * 128), l_desc, k > 0 || c > 0);
                        }
                        ptx::umma_commit(B.bar(sh->o_done[s]));
                        give_back();
                    }
                }
            }
        }
    }
    if (!ok && leader) report(a, STATUS_TIMEOUT, 2);
}
// After a timeout: products in flight end.  (By the lane that issued them: elect_one's is always the same.)
__device__ __noinline__ void drain_products(uint32_t drain, uint64_t limit_ns) {
    if (ptx::elect_one()) {
        ptx::umma_commit(drain);
        ptx::mbar_wait(drain, 0, limit_ns, nullptr);
    }
}

// ---- softmax: four warps per stream ------------------------------------------------------------
// Loads and stores of tensor memory are instructions of whole warps: where lanes may have taken different ways before one (a wait,
// lanes without a row or a component, a vote, which brings the warps together but not their lanes), a __syncwarp stands before it.
// Code that runs once per unit or less is kept short, in loops: a line of instructions that is not in
// the cache costs about as much as eight of them that are.
template <int NB, int BLK, bool WIDE>
struct Stream {
    using S = Shape<NB, BLK, WIDE>;
    const Block<NB, BLK, WIDE> &B;
    const CacheAttnArgs &a;
    Small *sh;
    const int s, warp, lane, key;   // stream; warp of it; TMEM lane: Narrow's key of a tile, Wide's row of the unit
    const uint32_t tmem, q;         // tensor memory from this warp's lanes on; this stream's queries
    uint32_t scores;                // of the tile at hand
    uint32_t s_phase = 0, o_phase = 0;  // s_phase: a bit per place
    bool failed = false;

    __device__ Stream(const Block<NB, BLK, WIDE> &b, uint32_t tmem0, int stream)
        : B(b), a(b.a), sh(b.sh), s(stream), warp((threadIdx.x >> 5) & 3), lane(threadIdx.x & 31), key(threadIdx.x & 127),
          tmem(tmem0 + (static_cast<uint32_t>(32 * ((threadIdx.x >> 5) & 3)) << 16)), q(b.q + static_cast<uint32_t>(stream) * COLS * 128u) {}

    __device__ bool vote(bool x) const { return ptx::barrier_or(1 + s, 128, x); }
    __device__ void wait_out() {
        failed = !B.wait(ptx::smem_u32(&sh->o_done[s]), o_phase) || failed;
        o_phase ^= 1u;
        __syncwarp();
        ptx::tc_fence_after();
    }

    // Queries of rows row0 .. row0 + rows - 1 of the unit, zeros up to `width`, as the K-major operand.
    __device__ void load_q(const Job &u, int row0, int rows, int width) {
        // two threads per row, half of its chunks of 8 components each
        const int row = key >> 1, chunks = (a.d + 15) / 16;
        const int r = u.row0 + row0 + row, token = r / a.group;
        const __nv_bfloat16 *const from0 = static_cast<const __nv_bfloat16 *>(a.q);
        const __nv_bfloat16 *from = from0 +
                                    (static_cast<int64_t>(u.s.q0 + token) * a.heads + u.head * a.group + (r - token * a.group)) * a.d;
        if (row < width) {
            const uint32_t line = q + static_cast<uint32_t>(row) * 128u;
            const int odd = key & 1;
#pragma unroll 4
            for (int i = 0; i < chunks; ++i) {
                const int c = 2 * i + odd;
                const uint32_t have = row < rows && c * 8 < a.d ? 16u : 0u;  // 0: zeros are written
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                                 line + static_cast<uint32_t>(c >> 3) * Q_BLOCK_BYTES + (static_cast<uint32_t>((c & 7) ^ (row & 7)) << 4)),
                             "l"(have ? from + c * 8 : from0), "r"(have)
                             : "memory");
            }
        }
    }

    // They have landed.
    __device__ void have_q() {
        asm volatile("cp.async.wait_all;" ::: "memory");
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&sh->q_full[s]));
    }

    __device__ uint32_t v_slot(uint32_t pos) const { return B.ring + (S::K_SLOTS + pos % S::V_SLOTS) * S::SLOT; }

    // Values that are not finite would reach rows that do not see them (0 x NaN).  Those behind the
    // sequence's end are cleared; of a tile with others the stream forms the product itself, key by key.
    // Whether this thread's key (at) has such values.
    __device__ bool odd_values(uint32_t pos, int at, int len) {
        for (int nb = 0; nb < NB; ++nb)
            failed = !B.wait(B.bar(sh->full[S::K_SLOTS + (pos + nb) % S::V_SLOTS]), (pos + nb) / S::V_SLOTS & 1u) || failed;
        __syncwarp();
        bool odd = false;
        if (!failed) {
#pragma unroll 1
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll 1
                for (int b = 0; b < B.blocks(nb); ++b) {
                    const uint32_t line = v_slot(pos + nb) + static_cast<uint32_t>(b) * BLOCK_BYTES + static_cast<uint32_t>(key) * 128u;
                    // the largest size, NaN above all
                    __nv_bfloat162 top = __floats2bfloat162_rn(0.0f, 0.0f);
#pragma unroll
                    for (int c = 0; c < 8; ++c) {
                        uint32_t w[4];
                        ptx::ld_shared_v4(line + static_cast<uint32_t>((c ^ (key & 7)) << 4), w[0], w[1], w[2], w[3]);
#pragma unroll
                        for (int i = 0; i < 4; ++i) top = __hmax2_nan(top, __habs2(*reinterpret_cast<const __nv_bfloat162 *>(&w[i])));
                    }
                    const uint32_t t = *reinterpret_cast<const uint32_t *>(&top);
                    const bool bad = (t & 0x7F80u) == 0x7F80u || (t & 0x7F800000u) == 0x7F800000u;
                    if (bad && at >= len) {
#pragma unroll 1
                        for (int c = 0; c < 8; ++c) ptx::st_shared_v4(line + static_cast<uint32_t>(c << 4), 0u, 0u, 0u, 0u);
                    } else {
                        odd = odd || bad;
                    }
                }
        }
        return odd;
    }

    // A unit's queries and tiles of this stream.
    struct Part {
        int row0, rows, width, tiles;
    };
    __device__ Part part(const Job &x) const {
        Part y;
        y.row0 = WIDE ? s * COLS : 0, y.rows = x.rows - y.row0;  // (WIDE: of which 64 at most)
        y.width = WIDE ? COLS : (y.rows + 15) & ~15;
        y.tiles = WIDE && NB > 1 ? (s == 0 ? x.tiles : 0) : (x.tiles + 1 - s) / 2;
        return y;
    }
    // The queries of the next unit, as soon as the scores of the one before are complete.
    __device__ bool queries(const Job &x) {
        const Part y = part(x);
        const bool some = x.tiles > 0 && (WIDE || y.tiles > 0);
        if (some) load_q(x, y.row0, y.rows, y.width);
        return some;
    }

};

// Up to 64 rows: a thread per key.
template <int NB, int BLK>
struct Narrow : Stream<NB, BLK, false> {
    static constexpr bool WIDE = false;
    using Base = Stream<NB, BLK, WIDE>;
    using S = Shape<NB, BLK, WIDE>;
    using Base::B, Base::a, Base::sh, Base::s, Base::warp, Base::lane, Base::key, Base::tmem, Base::scores, Base::s_phase, Base::o_phase,
        Base::failed, Base::vote, Base::wait_out, Base::v_slot, Base::odd_values;
    const uint32_t scores0, out, p;
    float2 l[4];                    // NB = 2: sums of the weights of 8 rows over some of the warp's keys (see add_up)

    __device__ Narrow(const Block<NB, BLK, WIDE> &b, uint32_t tmem0, int stream)
        : Base(b, tmem0, stream), scores0(tmem + static_cast<uint32_t>(stream * COLS)),
          out(tmem + O_COLUMN + static_cast<uint32_t>(stream * COLS)), p(b.p + static_cast<uint32_t>(stream) * P_BYTES) {}

    __device__ void start() {
        if (key < COLS) sh->m[s][key] = -INFINITY;
        if (NB > 1) {
#pragma unroll
            for (int i = 0; i < 4; ++i) l[i] = make_float2(0.0f, 0.0f);
        }
        vote(false);
    }

    // Lanes that share a key's line in add_up, eight rows each: 2, 4 or 8, as a power of two.
    static __device__ __forceinline__ int line_bits(int width) { return width <= 16 ? 1 : (width <= 32 ? 2 : 3); }

    // Where tensor memory is full of outputs (NB = 2), a stream adds up the rounded weights itself, from their
    // place: a lane takes eight rows of every (32 / lanes)-th key of its warp.  (Sums of all rows for its own
    // key would be 64 registers.)
    __device__ void add_up(int width) {
        const int bits = line_bits(width), lanes = 1 << bits, chunk = lane & (lanes - 1);
        if (8 * chunk < width) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < lanes) {
                    const int k = (lane >> bits) + (i << (5 - bits));
                    uint32_t w[4];
                    ptx::ld_shared_v4(p + static_cast<uint32_t>(32 * warp + k) * 128u + (static_cast<uint32_t>(chunk ^ (k & 7)) << 4), w[0], w[1], w[2], w[3]);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        l[j] = ptx::add2(l[j], make_float2(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xFFFF0000u)));
                }
        }
    }

    // Bit r: row r sees this thread's key.  Rows behind the last see everything (their scores are zero).
    __device__ uint64_t seen(const Job &u, int rows, int at) const {
        const uint64_t past = rows >= 64 ? 0ull : ~0ull << rows;
        const int j = at - u.s.prefix;
        if (j < 0) return ~0ull;
        if (at >= u.s.len) return past;
        if (!a.tree) {
            const int64_t from = static_cast<int64_t>(j) * a.group - u.row0;  // rows of token j and later
            return (from <= 0 ? ~0ull : (from >= 64 ? 0ull : ~0ull << from)) | past;
        }
        if (j >= 64 * a.tree_words) return past;
        // token by token: `group` rows each, the first one's perhaps fewer
        const int r0 = u.row0, first = r0 / a.group, tokens = (r0 + rows - 1) / a.group - first + 1;
        const int64_t *words = a.tree + static_cast<int64_t>(u.s.q0 + first) * a.tree_words + (j >> 6);
        uint64_t bits = past;
        int begin = first * a.group - r0;
#pragma unroll 8
        for (int t = 0; t < tokens; ++t, begin += a.group) {
            const uint64_t w = static_cast<uint64_t>(words[static_cast<int64_t>(t) * a.tree_words]);
            const int b = max(begin, 0), e = min(begin + a.group, rows);
            const uint64_t span = (e >= 64 ? ~0ull : (1ull << e) - 1ull) & ~((1ull << b) - 1ull);
            if (w >> (j & 63) & 1ull) bits |= span;
        }
        return bits;
    }

    // Scores that a row does not see: what the scale turns into -infinity.
    __device__ void hide(uint64_t sees, int width) const {
        const uint32_t none = a.scale_log2 > 0.0f ? 0xFF800000u : 0x7F800000u;
#pragma unroll 1
        for (int c = 0; c < width; c += 16) {
            uint32_t x[16];
            ptx::tmem_ld_32x32b_x16(scores + c, x);
            ptx::tmem_ld_wait(x);
            const uint32_t bits = static_cast<uint32_t>(sees >> c);
#pragma unroll
            for (int j = 0; j < 16; ++j) x[j] = bits >> j & 1u ? x[j] : none;
            ptx::tmem_st_32x32b_x16(scores + c, x);
        }
        ptx::tmem_st_wait();
    }

    // Weights of the rows, rounded to bf16, two to a word; returns the largest exponent.
    __device__ float form(uint32_t (&w)[COLS / 2], int width) const {
        const float2 scale = make_float2(a.scale_log2, a.scale_log2);
        float top = -INFINITY;
        // 32 rows at a time: with all 64 loaded at once the registers do not suffice
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint32_t r[2][16];
#pragma unroll
            for (int c = 0; c < 2; ++c)
                if (32 * h + 16 * c < width) ptx::tmem_ld_32x32b_x16(scores + 32 * h + 16 * c, r[c]);
#pragma unroll
            for (int c = 0; c < 2; ++c)
                if (32 * h + 16 * c < width) {
                    ptx::tmem_ld_wait(r[c]);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float4 m = *reinterpret_cast<const float4 *>(&sh->ref[s][32 * h + 16 * c + 4 * j]);
                        const float2 lo = ptx::fma2(make_float2(__uint_as_float(r[c][4 * j]), __uint_as_float(r[c][4 * j + 1])), scale,
                                                    make_float2(m.x, m.y));
                        const float2 hi = ptx::fma2(make_float2(__uint_as_float(r[c][4 * j + 2]), __uint_as_float(r[c][4 * j + 3])), scale,
                                                    make_float2(m.z, m.w));
                        top = fmaxf(top, fmaxf(fmaxf(lo.x, lo.y), fmaxf(hi.x, hi.y)));
                        const __nv_bfloat162 e0 = __floats2bfloat162_rn(ptx::ex2_approx(lo.x), ptx::ex2_approx(lo.y)),
                                             e1 = __floats2bfloat162_rn(ptx::ex2_approx(hi.x), ptx::ex2_approx(hi.y));
                        w[16 * h + 8 * c + 2 * j] = *reinterpret_cast<const uint32_t *>(&e0);
                        w[16 * h + 8 * c + 2 * j + 1] = *reinterpret_cast<const uint32_t *>(&e1);
                    }
                }
        }
        return top;
    }

    // Renews the references from the tile's maxima; the sums and outputs so far take the factors.
    // Returns whether some row has seen nothing yet.
    __device__ bool renew(int width, bool more) {
#pragma unroll 1
        for (int c = 0; c < width; c += 16) {
            uint32_t x[16];
            __syncwarp();
            ptx::tmem_ld_32x32b_x16(scores + c, x);
            ptx::tmem_ld_wait(x);
            float top = 0.0f;  // lane j's: of row c + j
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                const float v = ptx::warp_max_f32(__uint_as_float(x[j]) * a.scale_log2);
                if (lane == j) top = v;
            }
            if (lane < 16) ptx::st_shared_u32(p + P_WARPS + static_cast<uint32_t>(warp * COLS + c + lane) * 4u, __float_as_uint(top));
        }
        vote(false);
        bool none = false;
        if (key < width) {
            const float was = sh->m[s][key];
            float now = was;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const float t = __uint_as_float(ptx::ld_shared_u32(p + P_WARPS + static_cast<uint32_t>(w * COLS + key) * 4u));
                now = t > now ? t : now;  // NaN: passed over
            }
            none = now == -INFINITY;
            sh->m[s][key] = now;
            sh->ref[s][key] = none ? 0.0f : -now;
            ptx::st_shared_u32(p + P_FACTOR + static_cast<uint32_t>(key) * 4u, __float_as_uint(was == now ? 1.0f : ptx::ex2_approx(was - now)));
        }
        const bool fresh = vote(none);
        __syncwarp();
        if (more) {
            if (NB > 1) {
                const uint32_t rows8 = p + P_FACTOR + static_cast<uint32_t>(lane & ((1 << line_bits(width)) - 1)) * 32u;
                uint32_t f[8];
                ptx::ld_shared_v4(rows8, f[0], f[1], f[2], f[3]);
                ptx::ld_shared_v4(rows8 + 16, f[4], f[5], f[6], f[7]);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    l[i] = ptx::mul2(l[i], make_float2(__uint_as_float(f[2 * i]), __uint_as_float(f[2 * i + 1])));
            }
            // (NB = 1: behind the outputs are the sums)
#pragma unroll 1
            for (int nb = 0; nb < 2; ++nb)
#pragma unroll 1
                for (int c = 0; c < width; c += 16) {
                    uint32_t o[16];
                    ptx::tmem_ld_32x32b_x16(out + nb * 2 * COLS + c, o);
                    ptx::tmem_ld_wait(o);
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        o[j] = __float_as_uint(__uint_as_float(o[j]) *
                                               __uint_as_float(ptx::ld_shared_u32(p + P_FACTOR + static_cast<uint32_t>(c + j) * 4u)));
                    ptx::tmem_st_32x32b_x16(out + nb * 2 * COLS + c, o);
                }
            ptx::tmem_st_wait();
            vote(false);  // the factors have been read: the weights come to their place
        }
        return fresh;
    }

    __device__ bool own_product(uint32_t pos, int at, int len, uint64_t sees, int width, bool first) {
        const bool odd = odd_values(pos, at, len);
        const bool own = vote(odd && sees != ~0ull);
        __syncwarp();
        if (!own) return false;
        // -0 marks a weight that is none
        const uint32_t line = p + static_cast<uint32_t>(key) * 128u;
        for (int r = 0; r < width; ++r)
            if (!(sees >> r & 1ull))
                asm volatile("st.shared.b16 [%0], %1;" ::"r"(line + (static_cast<uint32_t>((r >> 3) ^ (key & 7)) << 4) + (r & 7) * 2),
                             "h"(static_cast<uint16_t>(0x8000))
                             : "memory");
        vote(false);
        __syncwarp();
#pragma unroll 1
        for (int nb = 0; nb < NB; ++nb) {
            const int e = key;  // component nb * 128 + key: this thread's TMEM lane
            const bool have = nb * 128 + e < a.d;
            const uint32_t v0 = v_slot(pos + nb) + static_cast<uint32_t>(have ? e >> 6 : 0) * BLOCK_BYTES + (e & 7) * 2;
#pragma unroll 1
            for (int c = 0; c * 16 < width; ++c) {
                uint32_t o[16];
                if (first) {
#pragma unroll
                    for (int j = 0; j < 16; ++j) o[j] = 0u;
                } else {
                    ptx::tmem_ld_32x32b_x16(out + nb * 2 * COLS + 16 * c, o);
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
                __syncwarp();
                ptx::tmem_st_32x32b_x16(out + nb * 2 * COLS + 16 * c, o);
            }
        }
        ptx::tmem_st_wait();
        return true;
    }

    // One tile: scores to weights.  k: how many this stream has done of the unit; pos: of its V, counted in slots.
    __device__ bool tile(const Job &u, int rows, int width, int t, int k, uint32_t pos, bool &fresh) {
        failed = !B.wait(ptx::smem_u32(&sh->s_full[s][k & 1]), s_phase >> (k & 1) & 1u) || failed;
        s_phase ^= 1u << (k & 1);
        scores = scores0 + static_cast<uint32_t>((k & 1) * 2 * COLS);
        __syncwarp();
        ptx::tc_fence_after();
        const int at = t * KEYS + key;
        const bool masked = (t + 1) * KEYS > u.s.prefix;
        uint64_t sees = ~0ull;
        if (masked) {
            sees = seen(u, rows, at);
            __syncwarp();
            hide(sees, width);
        }
        uint32_t w[COLS / 2];
        int pass = fresh ? 1 : 0;
#pragma unroll 1
        for (;; ++pass) {
            if (pass == 1) {
                if (vote(failed)) return false;
                if (k > 0) wait_out();
                fresh = renew(width, k > 0);
            }
            const float top = form(w, width);
            if (pass == 1 || !vote(top > RENEW || failed)) break;
        }
        if (k > 0 && pass == 0) wait_out();  // their place is read by the product of the tile before
        const uint32_t line = p + static_cast<uint32_t>(key) * 128u;
#pragma unroll
        for (int c = 0; c < 8; ++c)
            if (8 * c < width)
                ptx::st_shared_v4(line + (static_cast<uint32_t>(c ^ (key & 7)) << 4), w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
        const bool own = masked && own_product(pos, at, u.s.len, sees, width, k == 0);
        if (key == 0) sh->skip[s] = own;
        ptx::fence_proxy_async_smem();
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&sh->p_full[s]));
        if (NB > 1) add_up(width);
        return true;
    }

    // The sums (NB = 2: each warp's), into the weights' space, which no product reads any more.
    __device__ void sum_l(int width) {
        if (NB == 1) {
            if (warp == 0)
#pragma unroll 1
                for (int c = 0; c < width; c += 16) {
                    uint32_t x[16];
                    __syncwarp();
                    ptx::tmem_ld_32x32b_x16(out + (L_COLUMN - O_COLUMN) + c, x);
                    ptx::tmem_ld_wait(x);
                    if (lane == 0)
#pragma unroll
                        for (int j = 0; j < 16; j += 4)
                            ptx::st_shared_v4(p + P_WARPS + static_cast<uint32_t>(c + j) * 4u, x[j], x[j + 1], x[j + 2], x[j + 3]);
                }
            return;
        }
        const int lanes = (1 << line_bits(width));
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 4; ++i)
            for (int o = lanes; o < 32; o <<= 1) {
                l[i].x += __shfl_xor_sync(0xffffffffu, l[i].x, o);
                l[i].y += __shfl_xor_sync(0xffffffffu, l[i].y, o);
            }
        vote(false);  // every warp has read its weights
        if (lane < lanes) {
            const uint32_t to = p + P_WARPS + static_cast<uint32_t>(warp * COLS + 8 * lane) * 4u;
            ptx::st_shared_v4(to, __float_as_uint(l[0].x), __float_as_uint(l[0].y), __float_as_uint(l[1].x), __float_as_uint(l[1].y));
            ptx::st_shared_v4(to + 16, __float_as_uint(l[2].x), __float_as_uint(l[2].y), __float_as_uint(l[3].x), __float_as_uint(l[3].y));
        }
    }
};

// Up to 128 rows: a thread per row.
template <int NB, int BLK>
struct Wide : Stream<NB, BLK, true> {
    static constexpr bool WIDE = true;
    using Base = Stream<NB, BLK, WIDE>;
    using S = Shape<NB, BLK, WIDE>;
    using Base::B, Base::a, Base::sh, Base::s, Base::warp, Base::lane, Base::key, Base::tmem, Base::scores, Base::s_phase, Base::o_phase,
        Base::failed, Base::vote, Base::wait_out, Base::v_slot, Base::odd_values;
    const uint32_t out;
    float m;                        // the row's reference (log2)
    float2 l[2];                    // its sum, in four parts
    int token;                      // its token
    int all;                        // keys that every row of the unit sees

    __device__ Wide(const Block<NB, BLK, WIDE> &b, uint32_t tmem0, int stream)
        : Base(b, tmem0, stream), out(tmem + O_COLUMN + static_cast<uint32_t>(stream) * 128u) {}

    // Bit i: the row sees key at + i.
    __device__ uint32_t sees_of(const Job &u, int at) const {
        const int left = u.s.len - at, j = at - u.s.prefix;
        const uint32_t bits = left >= 32 ? ~0u : (left <= 0 ? 0u : (1u << left) - 1u);
        if (j + 32 <= 0) return bits;
        if (!a.tree) {
            const int n = token + 1 - j;
            return n >= 32 ? bits : (n <= 0 ? 0u : bits & ((1u << n) - 1u));
        }
        const int64_t *words = a.tree + static_cast<int64_t>(u.s.q0 + token) * a.tree_words;
        auto word = [&](int i) { return i < a.tree_words ? static_cast<uint64_t>(words[i]) : 0ull; };
        uint64_t w;
        if (j < 0) {
            w = word(0) << -j | ((1ull << -j) - 1ull);
        } else {
            w = word(j >> 6) >> (j & 63);
            if ((j & 63) > 32) w |= word((j >> 6) + 1) << (64 - (j & 63));
        }
        return bits & static_cast<uint32_t>(w);
    }

    __device__ void hide(const Job &u, int at) const {
#pragma unroll 1
        for (int h = 0; h < KEYS; h += 32) {
            const uint32_t bits = sees_of(u, at + h);
            if (__all_sync(0xffffffffu, bits == ~0u)) continue;
#pragma unroll
            for (int c = 0; c < 32; c += 16) {
                uint32_t x[16];
                ptx::tmem_ld_32x32b_x16(scores + h + c, x);
                ptx::tmem_ld_wait(x);
#pragma unroll
                for (int j = 0; j < 16; ++j) x[j] = bits >> (c + j) & 1u ? x[j] : 0xFF800000u;
                ptx::tmem_st_32x32b_x16(scores + h + c, x);
            }
        }
        ptx::tmem_st_wait();
    }

    // The reference becomes the row's maximum so far (top: of this tile); its sum and outputs take the factor.
    __device__ void renew(float top, bool more) {
        const float now = top > m ? top : m;  // NaN: passed over
        const float f = m == now ? 1.0f : ptx::ex2_approx(m - now);
        m = now;
        l[0] = ptx::mul2(l[0], make_float2(f, f));
        l[1] = ptx::mul2(l[1], make_float2(f, f));
        if (more) {
#pragma unroll 1
            for (int c = 0; c < a.d; c += 16) {
                uint32_t o[16];
                ptx::tmem_ld_32x32b_x16(out + c, o);
                ptx::tmem_ld_wait(o);
#pragma unroll
                for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
                ptx::tmem_st_32x32b_x16(out + c, o);
            }
            ptx::tmem_st_wait();
        }
    }

    // Weights (in place of the scores: two to a word) and their sums.
    __device__ void form() {
        const float scale = fabsf(a.scale_log2), ref = m == -INFINITY ? 0.0f : -m;
        const float2 scale2 = make_float2(scale, scale), ref2 = make_float2(ref, ref);
        uint32_t x[2][32];
        ptx::tmem_ld_32x32b_x32(scores, x[0]);
#pragma unroll
        for (int h = 0; h < 4; ++h) {
            uint32_t (&r)[32] = x[h & 1];
            ptx::tmem_ld_wait(r);
            if (h < 3) ptx::tmem_ld_32x32b_x32(scores + 32 * (h + 1), x[(h + 1) & 1]);
            uint32_t w[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                const float2 e = ptx::fma2(make_float2(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1])), scale2, ref2);
                const float2 p2 = make_float2(ptx::ex2_approx(e.x), ptx::ex2_approx(e.y));
                l[j & 1] = ptx::add2(l[j & 1], p2);
                const __nv_bfloat162 b = __floats2bfloat162_rn(p2.x, p2.y);
                w[j] = *reinterpret_cast<const uint32_t *>(&b);
            }
            ptx::tmem_st_32x32b_x16(scores + 16 * h, w);
        }
        ptx::tmem_st_wait();
    }

    // The product of a tile with values that are not finite, from the weights as they were rounded.
    __device__ bool product(const Job &u, uint32_t pos, int at, bool first) {
        const bool own = vote(odd_values(pos, at + key, u.s.len));
        __syncwarp();
        if (!own) return false;
#pragma unroll 1
        for (int c = 0; c < a.d; c += 16) {
            const uint32_t v0 = v_slot(pos + (c >> 7)) + static_cast<uint32_t>((c >> 6) & 1) * BLOCK_BYTES;
            const uint32_t chunk = static_cast<uint32_t>(c >> 3) & 7u;
            uint32_t o[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) o[j] = 0u;
            if (!first) {
                ptx::tmem_ld_32x32b_x16(out + c, o);
                ptx::tmem_ld_wait(o);
            }
#pragma unroll 1
            for (int h = 0; h < KEYS; h += 16) {
                const uint32_t bits = sees_of(u, at + (h & ~31)) >> (h & 16);
                uint32_t w[8];
                __syncwarp();
                ptx::tmem_ld_32x32b_x8(scores + h / 2, w);
                ptx::tmem_ld_wait(w);
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                    const uint32_t line = v0 + static_cast<uint32_t>(h + k) * 128u;
                    uint32_t v[8];
                    ptx::ld_shared_v4(line + ((chunk ^ (k & 7)) << 4), v[0], v[1], v[2], v[3]);
                    ptx::ld_shared_v4(line + (((chunk + 1) ^ (k & 7)) << 4), v[4], v[5], v[6], v[7]);
                    if (bits >> k & 1u) {
                        const float p1 = __uint_as_float(k & 1 ? w[k >> 1] & 0xFFFF0000u : w[k >> 1] << 16);
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            o[j] = __float_as_uint(__uint_as_float(o[j]) +
                                                   p1 * __uint_as_float(j & 1 ? v[j >> 1] & 0xFFFF0000u : v[j >> 1] << 16));
                    }
                }
            }
            __syncwarp();
            ptx::tmem_st_32x32b_x16(out + c, o);
        }
        ptx::tmem_st_wait();
        return true;
    }

    __device__ void start(const Job &u) {
        token = (u.row0 + min(key, u.rows - 1)) / a.group;
        all = min(u.s.len, a.tree ? u.s.prefix : u.s.prefix + u.row0 / a.group + 1);
        m = -INFINITY;
        l[0] = l[1] = make_float2(0.0f, 0.0f);
    }

    // One tile, the unit's i-th and this stream's k-th.  A wait that failed makes the rest of them end at once.
    __device__ void tile(const Job &u, int i, int k, uint32_t pos) {
        const int place = NB == 1 ? 0 : k & 1;
        failed = !B.wait(ptx::smem_u32(&sh->s_full[s][place]), s_phase >> place & 1u) || failed;
        s_phase ^= 1u << place;
        scores = tmem + static_cast<uint32_t>(i & 1) * 128u;
        __syncwarp();
        ptx::tc_fence_after();
        const int at = (u.tile0 + i) * KEYS;
        const bool masked = at + KEYS > all;
        if (masked) hide(u, at);
        float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        {
            uint32_t x[2][32];
            ptx::tmem_ld_32x32b_x32(scores, x[0]);
#pragma unroll
            for (int h = 0; h < 4; ++h) {
                ptx::tmem_ld_wait(x[h & 1]);
                if (h < 3) ptx::tmem_ld_32x32b_x32(scores + 32 * (h + 1), x[(h + 1) & 1]);
#pragma unroll
                for (int j = 0; j < 32; j += 2)
                    top[(j >> 1) & 3] = fmaxf(top[(j >> 1) & 3], fmaxf(__uint_as_float(x[h & 1][j]), __uint_as_float(x[h & 1][j + 1])));
            }
        }
        const float most = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * fabsf(a.scale_log2);
        // (NB = 1: the scores come with the end of the stream's product before them, which was issued before)
        if (NB > 1 && k > 0) wait_out();
        if (__any_sync(0xffffffffu, most > m + RENEW)) renew(most, k > 0);
        form();
        const bool own = masked && product(u, pos, at, k == 0);
        if (key == 0) sh->skip[s] = own;
        if (masked) ptx::fence_proxy_async_smem();  // values that were cleared
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&sh->p_full[s]));
    }
};

template <int NB, int BLK>
__device__ void narrow_role(const Block<NB, BLK, false> &B, uint32_t tmem, int s) {
    const CacheAttnArgs &a = B.a;
    Small *sh = B.sh;
    Narrow<NB, BLK> st(B, tmem, s);
    const int key = st.key;
    uint32_t v_pos = 0;  // slots of V so far
    Jobs<NB, BLK, false> jobs = {B, {}};
    Job u;
    auto both_vote = [&](bool x) { return ptx::barrier_or(3, 256, x); };
    auto shared = [&](uint32_t at) { return __uint_as_float(ptx::ld_shared_u32(at)); };
    bool loaded = false, posted = false;
    // (both streams leave together: a barrier that only one of them comes to would wait forever)
    if (both_vote(!jobs.peek(u))) return;
    while (u.tiles > 0) {
        if (!loaded && st.queries(u)) st.have_q();
        loaded = false;
        const auto y = st.part(u);
        const int n = u.tiles, rows = u.rows, width = y.width;
        st.start();
        bool fresh = true, ok = true;
#pragma unroll 1
        for (int k = 0; ok && k < y.tiles; ++k) {
            const int i = 2 * k + s;
            ok = st.tile(u, rows, width, u.tile0 + i, k, v_pos + i * NB, fresh);
        }
        v_pos += n * NB;
        bool coming = false;
        if (ok && !st.failed && y.tiles > 0) {
            Job ahead;
            st.failed = !jobs.peek_next(ahead);
            if (!st.failed && ahead.tiles > 0) {
                coming = st.queries(ahead);
                loaded = true;
            }
        }
        if (ok && y.tiles > 0) {
            st.wait_out();
            st.sum_l(width);
        }
        if (coming) st.have_q();
        if (both_vote(!ok || st.failed)) return;
        ptx::tc_fence_after();
        jobs.read(u, jobs.at.slot);  // (not kept in registers over the tiles)
        // Streams that shared the rows out by tiles are added up here.  A thread per row: factors of the
        // outputs, and where the row goes.
        const bool two = n > 1;
        const int64_t piece = (2 * static_cast<int64_t>(blockIdx.x) + u.place) * COLS;
        if (key < rows) {
            auto sum = [&](int stream) {
                const uint32_t at = B.p + static_cast<uint32_t>(stream) * P_BYTES + P_WARPS + static_cast<uint32_t>(key) * 4u;
                return NB == 1 ? shared(at)
                               : (shared(at) + shared(at + COLS * 4)) + (shared(at + 2 * COLS * 4) + shared(at + 3 * COLS * 4));
            };
            float top = sh->m[0][key], total = sum(0), f0 = 1.0f, f1 = 0.0f;
            if (two) {
                const float m0 = top, m1 = sh->m[1][key];
                top = fmaxf(m0, m1);
                f0 = scale_of(m0, top), f1 = scale_of(m1, top);
                total = total * f0 + sum(1) * f1;
            }
            const int r = u.row0 + key, token = r / a.group;
            int to = token * a.heads + (r - token * a.group);
            if (u.cut) {
                if (s == 0) __stcg(a.part_ml + piece + key, make_float2(top, total));
                to = key;
            } else {
                const float inv = total == 0.0f ? 0.0f : 1.0f / total;  // a row that sees nothing: zeros
                f0 *= inv, f1 *= inv;
            }
            ptx::st_shared_u32(st.p + P_FACTOR + static_cast<uint32_t>(key) * 4u, __float_as_uint(f0));
            ptx::st_shared_u32(st.p + P_OTHER + static_cast<uint32_t>(key) * 4u, __float_as_uint(f1));
            ptx::st_shared_u32(st.p + P_ROW + static_cast<uint32_t>(key) * 4u, static_cast<uint32_t>(to));
        }
        st.vote(false);
        __syncwarp();
        float *part = a.part + piece * a.d;
        __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(a.o) + (static_cast<int64_t>(u.s.q0) * a.heads + u.head * a.group) * a.d;
        const uint32_t lanes = static_cast<uint32_t>(32 * st.warp) << 16;
#pragma unroll 1
        for (int nb = 0; nb < NB; ++nb) {
            const int e = nb * 128 + key;
#pragma unroll 1
            for (int c = 8 * s; c < rows; c += 16) {
                uint32_t x[8], y[8], f[8], g[8], to[8];
                ptx::tmem_ld_32x32b_x8(tmem + lanes + O_COLUMN + static_cast<uint32_t>(2 * nb * COLS + c), x);
                if (two) ptx::tmem_ld_32x32b_x8(tmem + lanes + O_COLUMN + static_cast<uint32_t>((2 * nb + 1) * COLS + c), y);
                const uint32_t at = st.p + P_FACTOR + static_cast<uint32_t>(c) * 4u;
                ptx::ld_shared_v4(at, f[0], f[1], f[2], f[3]);
                ptx::ld_shared_v4(at + 16, f[4], f[5], f[6], f[7]);
                ptx::ld_shared_v4(at + (P_ROW - P_FACTOR), to[0], to[1], to[2], to[3]);
                ptx::ld_shared_v4(at + (P_ROW - P_FACTOR) + 16, to[4], to[5], to[6], to[7]);
                if (two) {
                    ptx::ld_shared_v4(at + (P_OTHER - P_FACTOR), g[0], g[1], g[2], g[3]);
                    ptx::ld_shared_v4(at + (P_OTHER - P_FACTOR) + 16, g[4], g[5], g[6], g[7]);
                }
                ptx::tmem_ld_wait(x);
                if (two) ptx::tmem_ld_wait(y);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    float v = __uint_as_float(x[j]) * __uint_as_float(f[j]);
                    if (two) v += __uint_as_float(y[j]) * __uint_as_float(g[j]);
                    x[j] = __float_as_uint(v);
                }
                if (e < a.d) {
                    if (u.cut) {
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            if (c + j < rows) __stcg(part + static_cast<int64_t>(static_cast<int>(to[j])) * a.d + e, __uint_as_float(x[j]));
                    } else {
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            if (c + j < rows) o[static_cast<int64_t>(static_cast<int>(to[j])) * a.d + e] = __float2bfloat16_rn(__uint_as_float(x[j]));
                    }
                }
                __syncwarp();  // (lanes without a component; tensor memory is read by whole warps)
            }
        }
        ptx::tc_fence_before();
        if (u.cut && u.place == 1) {
            if (threadIdx.x == 0) post_cut(a, u.s.q0, u.head, u.row0, u.rows, u.last);
            posted = true;
        }
        jobs.release();
        if (both_vote(!jobs.peek(u))) return;  // (and outputs, references and sums have been read)
    }
    if (!posted && threadIdx.x == 0) post_cut(a, 0, 0, 0, 0, 0);
}

template <int NB, int BLK>
__device__ void wide_role(const Block<NB, BLK, true> &B, uint32_t tmem, int s) {
    const CacheAttnArgs &a = B.a;
    Wide<NB, BLK> st(B, tmem, s);
    const int key = st.key;
    uint32_t v_pos = 0;  // slots of V so far
    uint32_t other = 0;  // NB = 1: phase of the other stream's scores
    Jobs<NB, BLK, true> jobs = {B, {}};
    Job u;
    auto both_vote = [&](bool x) { return ptx::barrier_or(3, 256, x); };
    bool loaded = false, posted = false;
    // (both streams leave together: a barrier that only one of them comes to would wait forever)
    if (both_vote(!jobs.peek(u))) return;
    while (u.tiles > 0) {
        if (!loaded && st.queries(u)) st.have_q();
        const int n = u.tiles, rows = u.rows, tiles = st.part(u).tiles;
        st.start(u);
#pragma unroll 1
        for (int k = 0; k < tiles; ++k) {
            const int i = NB == 1 ? 2 * k + s : k;
            st.tile(u, i, k, v_pos + i * NB);
        }
        v_pos += n * NB;
        // The next unit's queries are on their way as soon as the last scores, this stream's or the other's, are complete.
        Job ahead;
        bool coming = false;
        if (NB == 1) {
            const int count = s == 0 ? n / 2 : (n + 1) / 2;  // tiles of the other stream
            if (((n - 1) & 1) != s) st.failed = !B.wait(B.bar(B.sh->s_full[1 - s][0]), (other + count - 1) & 1u) || st.failed;
            other = (other + count) & 1u;
            if (__all_sync(0xffffffffu, !st.failed)) {
                if (jobs.peek_next(ahead))
                    coming = st.queries(ahead);
                else
                    st.failed = true;
            }
        }
        if (tiles > 0) st.wait_out();
        __syncwarp();
        // the row's reference and sum, to both streams (in place of scores)
        {
            uint32_t ml[8] = {__float_as_uint(st.m), __float_as_uint((st.l[0].x + st.l[0].y) + (st.l[1].x + st.l[1].y))};
            if (tiles > 0) ptx::tmem_st_32x32b_x8(st.tmem + static_cast<uint32_t>(s) * 128u, ml);
            ptx::tmem_st_wait();
            ptx::tc_fence_before();
        }
        if (both_vote(st.failed)) return;
        ptx::tc_fence_after();
        if (NB > 1) {
            if (both_vote(!jobs.peek_next(ahead))) return;
            coming = st.queries(ahead);
        }
        loaded = true;
        jobs.read(u, jobs.at.slot);
        // streams that shared the tiles out are added up; each writes half of the components
        const bool two = NB == 1 && n > 1;
        uint32_t ml0[8], ml1[8];
        __syncwarp();
        ptx::tmem_ld_32x32b_x8(st.tmem, ml0);
        if (two) ptx::tmem_ld_32x32b_x8(st.tmem + 128, ml1);
        ptx::tmem_ld_wait(ml0);
        if (two) ptx::tmem_ld_wait(ml1);
        ptx::tc_fence_before();
        if (NB == 1 && coming) st.have_q();  // (the next scores come while the outputs are written)
        const float m0 = __uint_as_float(ml0[0]), m1 = two ? __uint_as_float(ml1[0]) : m0, top = two ? fmaxf(m0, m1) : m0;
        float f0 = two ? scale_of(m0, top) : 1.0f, f1 = two ? scale_of(m1, top) : 0.0f;
        float total = __uint_as_float(ml0[1]);
        if (two) total = total * f0 + __uint_as_float(ml1[1]) * f1;
        const bool have = key < rows;
        const int64_t piece = (2 * static_cast<int64_t>(blockIdx.x) + u.place) * (2 * COLS) + key;
        const int r = u.row0 + key, token = st.token;  // (of rows that there are)
        float *part_row = a.part + piece * a.d;
        __nv_bfloat16 *o_row = static_cast<__nv_bfloat16 *>(a.o) +
                               (static_cast<int64_t>(u.s.q0 + token) * a.heads + u.head * a.group + (r - token * a.group)) * a.d;
        if (u.cut) {
            if (have && s == 0) __stcg(a.part_ml + piece, make_float2(top, total));
        } else {
            const float inv = total == 0.0f ? 0.0f : 1.0f / total;  // a row that sees nothing: zeros
            f0 *= inv, f1 *= inv;
        }
        __syncwarp();  // (lanes without a row)
        constexpr int HALF = 32 * BLK * NB;
        const uint32_t outs = st.tmem + O_COLUMN;
#pragma unroll 1
        for (int c = s * HALF; c < min(a.d, (s + 1) * HALF); c += 8) {
            uint32_t x[8], x1[8];
            ptx::tmem_ld_32x32b_x8(outs + c, x);
            if (two) ptx::tmem_ld_32x32b_x8(outs + 128 + c, x1);
            ptx::tmem_ld_wait(x);
            if (two) ptx::tmem_ld_wait(x1);
            float v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                v[j] = __uint_as_float(x[j]) * f0;
                if (two) v[j] += __uint_as_float(x1[j]) * f1;
            }
            if (have && u.cut) {
                __stcg(reinterpret_cast<float4 *>(part_row + c), make_float4(v[0], v[1], v[2], v[3]));
                __stcg(reinterpret_cast<float4 *>(part_row + c + 4), make_float4(v[4], v[5], v[6], v[7]));
            } else if (have) {
                uint4 w;
                uint32_t *to = &w.x;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
                    to[j] = *reinterpret_cast<const uint32_t *>(&b);
                }
                *reinterpret_cast<uint4 *>(o_row + c) = w;
            }
            __syncwarp();  // (lanes without a row)
        }
        ptx::tc_fence_before();
        if (NB > 1 && coming) st.have_q();
        if (u.cut && u.place == 1) {
            if (threadIdx.x == 0) post_cut(a, u.s.q0, u.head, u.row0, u.rows, u.last);
            posted = true;
        }
        jobs.release();
        if (both_vote(!jobs.peek(u))) return;
    }
    if (!posted && threadIdx.x == 0) post_cut(a, 0, 0, 0, 0, 0);
}

template <int NB, int BLK, bool WIDE>
__global__ void __launch_bounds__(TTHREADS, 1)
    tc_kernel(const CacheAttnArgs a, const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv, int box) {
    using S = Shape<NB, BLK, WIDE>;
    extern __shared__ uint8_t raw[];
    const uint32_t start = (ptx::smem_u32(raw) + 1023u) & ~1023u;
    const uint32_t small_at = S::RING + S::Q_BYTES + S::P_ALL;
    Small *sh = reinterpret_cast<Small *>(raw + (start - ptx::smem_u32(raw)) + small_at);
    const Block<NB, BLK, WIDE> B = {a, sh, start, start + S::RING, start + S::RING + S::Q_BYTES};
    const int warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) {
        for (int i = 0; i < S::SLOTS; ++i) {
            ptx::mbar_init(ptx::smem_u32(&sh->full[i]), 1);
            ptx::mbar_init(ptx::smem_u32(&sh->empty[i]), 1);
        }
        for (int s = 0; s < 2; ++s) {
            ptx::mbar_init(ptx::smem_u32(&sh->s_full[s][0]), 1);
            ptx::mbar_init(ptx::smem_u32(&sh->s_full[s][1]), 1);
            ptx::mbar_init(ptx::smem_u32(&sh->p_full[s]), 4);
            ptx::mbar_init(ptx::smem_u32(&sh->o_done[s]), 1);
            ptx::mbar_init(ptx::smem_u32(&sh->q_full[s]), 4);
            sh->skip[s] = 0;
        }
        for (int i = 0; i < JOBS; ++i) {
            ptx::mbar_init(ptx::smem_u32(&sh->job_full[i]), 1);
            ptx::mbar_init(ptx::smem_u32(&sh->job_empty[i]), JOB_READERS);
        }
        ptx::mbar_init(ptx::smem_u32(&sh->drain), 1);
        sh->abort = 0;
        ptx::fence_mbar_init();
        ptx::prefetch_tensormap(&mk);
        ptx::prefetch_tensormap(&mv);
    }
    if (threadIdx.x < 96) {
        sh->ones[threadIdx.x] = 0x3F803F80u;
        ptx::fence_proxy_async_smem();
    }
    if (warp == 8) {
        ptx::tmem_alloc(ptx::smem_u32(&sh->tmem), TMEM);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    Walk<Shape<NB, BLK, WIDE>::ROWS, KEYS> walk;
    walk.begin(a, sh->walk);  // with a __syncthreads
    ptx::tc_fence_after();
    const uint32_t tmem = sh->tmem;
    if (warp < 8) {
        if constexpr (WIDE)
            wide_role<NB, BLK>(B, tmem, warp >> 2);
        else
            narrow_role<NB, BLK>(B, tmem, warp >> 2);
    } else if (warp == 8)
        product_role<NB, BLK, WIDE>(B, tmem);
    else if (warp < 11)
        copy_role<NB, BLK, WIDE>(B, warp == 10, warp == 10 ? &mv : &mk, box);
    else
        plan_role<NB, BLK, WIDE>(B, walk);
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncwarp();
    ptx::tc_fence_before();
    __syncthreads();
    if (sh->abort) {
        // A wait has run out.  A role that was done before that, its copies or products still under way, does not know of it:
        // only here have all roles ended.  What is in flight ends before shared and tensor memory are given back.
        if (warp == 8) drain_products(B.bar(sh->drain), B.drain_ns());
        if (warp == 9 || warp == 10) drain_copies(B.bar(sh->full[warp == 10 ? S::K_SLOTS : 0]), sh->copied[warp == 10], B.drain_ns());
        if (threadIdx.x == 0) {
            report(a, STATUS_TIMEOUT, 3);
            post_cut(a, 0, 0, 0, 0, 0);
        }
        __syncthreads();
    }
    if (warp == 8) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, TMEM);
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

template <int NB, int BLK, bool WIDE>
cudaError_t launch_tc(const CacheAttnArgs &a, int blocks, cudaStream_t st) {
    using S = Shape<NB, BLK, WIDE>;
    static std::mutex mu;
    static bool set[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    {
        std::lock_guard<std::mutex> lk(mu);
        if (!set[dev]) {
            e = cudaFuncSetAttribute(tc_kernel<NB, BLK, WIDE>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(S::SMEM));
            if (e != cudaSuccess) return e;
            set[dev] = true;
        }
    }
    // a box's rows lie in one page and in one tile
    int box = KEYS;
    while (a.page_size % box != 0) box /= 2;
    CUtensorMap mk, mv;
    if (!cache_map(&mk, a, a.k, box) || !cache_map(&mv, a, a.v, box)) return cudaErrorInvalidValue;
    e = launch_pdl(tc_kernel<NB, BLK, WIDE>, dim3(static_cast<unsigned>(blocks)), TTHREADS, S::SMEM, st, a, mk, mv, box);
    return e == cudaSuccess ? launch_join<__nv_bfloat16, S::ROWS>(a, blocks, st) : e;
}

}  // namespace cattn

bool cache_attn_tc(const CacheAttnArgs &a) { return a.vec && a.page_size % 8 == 0 && a.d % 8 == 0 && a.d <= 256; }

cudaError_t launch_cache_attn_tc(const CacheAttnArgs &a, int num_sms, cudaStream_t st) {
    // Rows in lanes above 32 rows per sequence (the lengths themselves are known on the device only).  Measured with
    // rows in lanes and in columns, us: 64 sequences of 128 components over 100 to 8192 keys with 4 rows 196 and 189, 16 rows
    // 220 and 199, 32 196 and 192, 40 193 and 193, 48 195 and 194, 64 189 and 199; 8 of them with 32 rows 39.3 and 38.5, 40 rows
    // 42.8 and 43.5, 64 43 and 47; 16 of 68 to 256 rows 65 and 85; one of 131072 keys the same within 1% from 8 to 64 rows.
    // The border moves with the components: with 64 of them 32 rows 141 and 150, with 256 of them 48 rows 451 and 401.
    const bool wide = a.tokens * a.group > 32 * a.batch;
    if (a.d <= 64) return wide ? cattn::launch_tc<1, 1, true>(a, num_sms, st) : cattn::launch_tc<1, 1, false>(a, num_sms, st);
    if (a.d <= 128) return wide ? cattn::launch_tc<1, 2, true>(a, num_sms, st) : cattn::launch_tc<1, 2, false>(a, num_sms, st);
    return wide ? cattn::launch_tc<2, 2, true>(a, num_sms, st) : cattn::launch_tc<2, 2, false>(a, num_sms, st);
}

}  // namespace tpmlp
