// Host-side launchers of the kernels behind the C ABI (internal to libtpmlp.so).
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace tpmlp {

// The unit that dS of bf16 is taken in: dS / unit is rounded and multiplied, and the products
// are multiplied by it in fp32.  The usual gradients of the losses are all the same (1 over
// the tokens of a mean); in units of their significand dS at a target is p - 1 times a power of
// two, where in the plain unit it is the same rounding of 1/n in every token, up to 2^-9 of dX and
// dW that does not average out.  The exponent stays with dS: only the significand rounds, and
// a unit of 1 to 2 takes no gradient out of range.  It is the significand of the first
// gradient that takes part: of a valid target, neither 0 nor subnormal, infinite or NaN.
// Prompts come first, and have no part; a whole warp looks at 256 tokens at a time.
#ifdef __CUDACC__
__device__ __forceinline__ float xent_find_unit(const int64_t *target, const float *dloss, int64_t tokens,
                                                int64_t ignore_index, int64_t vocab) {
    constexpr int UN = 8;  // loads in flight
    const int lane = threadIdx.x & 31;
    for (int64_t t0 = 0; t0 < tokens; t0 += 32 * UN) {
        float g[UN];
#pragma unroll
        for (int u = 0; u < UN; ++u) {
            const int64_t t = t0 + 32 * u + lane;
            const int64_t y = t < tokens ? target[t] : -1;
            const float d = t < tokens ? fabsf(dloss[t]) : 0.0f;
            g[u] = y != ignore_index && y >= 0 && y < vocab ? d : 0.0f;
        }
#pragma unroll
        for (int u = 0; u < UN; ++u) {
            const unsigned hit = __ballot_sync(0xffffffffu, g[u] >= 0x1p-126f && g[u] < INFINITY);
            if (hit) {
                const float first = __shfl_sync(0xffffffffu, g[u], __ffs(static_cast<int>(hit)) - 1);
                return __uint_as_float((__float_as_uint(first) & 0x007FFFFFu) | 0x3F800000u);
            }
        }
    }
    return 1.0f;
}
#endif

// Epilogues of the GEMM kernels.  Each names the step of the MLP it finishes.
enum Epi : int {
    EPI_BIAS_GELU = 0,  // H = acc + a (optional store), Y = GeLU(H) (optional) -- column-parallel GEMM
    EPI_FOLD_BIAS = 1,  // Z = b + ((Z_1 + Z_2) + ...)                      -- row-parallel GEMM
    EPI_DGELU = 2,      // dY = acc * GeLU'(H)                              -- dZ B^T
    EPI_STORE = 3,      // out = acc                                       -- dB, dA
    EPI_FOLD = 4,       // dX = ((P_1 + P_2) + ...)                        -- dY A^T
    EPI_ATTN_SCORE = 5, // S = scale * acc, -inf above the diagonal (causal), fp16 out -- Q K^T
    EPI_ATTN_DS = 6,    // dS = P * (acc - D[row]) * scale                  -- dO V^T -> dS
    EPI_XENT_STATS = 7, // per row: max and sum of exponentials per 128 columns, the target's logit -- X W^T
    EPI_XENT_GRAD = 8,  // dS = (exp(acc - lse[row]) - [col = target]) * g[row]  -- X W^T -> dS
    EPI_ACC32 = 9,      // out (fp32) = acc, or out += acc                  -- dX and dW, piece by piece
    EPI_FOLD32 = 20,    // ACC32 over K in nshards ranges, added up in fp32 -- dX and dW of fp32, from three parts
    EPI_NS_GRAM = 10,   // A = scale * acc, symmetric, fp16                 -- X X^T
    EPI_NS_POLY = 11,   // C = diag I + alpha A + scale * acc, symmetric, fp16 -- A A
    EPI_NS_UPDATE = 12, // X' = alpha hi + beta lo + scale * acc as hi' + lo', fp16 -- C X
    EPI_NS_LAST = 13,   // the same X', bf16                                -- C X, last step
    EPI_STORE_UNIT = 19, // out = acc * unit (see xent_find_unit)                 -- dX and dW of bf16
    EPI_NS_GRAMS = 18,  // A in fp32, lower triangle, over K in ksplit ranges -- X X^T
    EPI_NS_GRAM32 = 15, // A_0 in fp32 from X as two fp16 parts, K in nshards ranges added up in fp32 -- X X^T
    EPI_NS_FINAL = 16,  // bf16 out = scale * acc, both operands in two parts -- Q X
    EPI_XENT_FOLD = 17, // XENT_STATS over K in nshards ranges, added up in fp32
    EPI_XENT_GRAD3 = 14, // XENT_GRAD for fp32: dS as three bf16 parts      -- X W^T -> dS
};

// A per-head operand or output read or written in place inside a token-major
// array (rank 4 or 5), instead of a contiguous [batch][rows][cols] block (rank 3).
// Element (e, s) of problem z = b * heads + g, head g = i * hpt + j:
//   rank 4 (O, dO [T, h]):           base[(b*S + s) * ld + g * d + e]
//   rank 5 (Q, K, V inside QKV or dQKV [T, 3h], base at the Q/K/V column offset):
//                                     base[(b*S + s) * ld + i * coli + j * d + e]
struct HeadView {
    int rank;  // 3 (plain block), 4 or 5
    int64_t S, nb, heads, hpt, d, ld, coli;
};

// One GEMM  out[M,N] = sum_k opA(m,k) opB(k,n)  over row-major operands.
//   A operand: K-major ([M,K] row-major, a_mn = false) or MN-major ([K,M], a_mn = true)
//   B operand: K-major ([N,K] row-major, b_mn = false) or MN-major ([K,N], b_mn = true)
// The K range is split into `nshards` consecutive ranges of `kshard` elements;
// each range is accumulated on its own and, for the FOLD epilogues, the range
// partials are summed in ascending order.  For the other epilogues nshards = 1.
struct GemmArgs {
    const void *a;
    bool a_mn;
    const void *b;
    bool b_mn;
    int64_t M, N, K;
    int nshards;
    int64_t kshard;
    void *out0;        // H / Z / dY / dB / dA / dX
    void *out1;        // Y for EPI_BIAS_GELU (null: no activation); Y rebuilt from H for EPI_DGELU (optional)
    const void *aux;   // H for EPI_DGELU
    const void *bias;  // a for EPI_BIAS_GELU, b for EPI_FOLD_BIAS
    uint32_t *status;  // device status word
    uint64_t wait_ns;
    int group;         // raster: tiles walk `group` M-tiles (N-tiles if raster_n) fastest
    bool raster_n;
    bool cta_pair;     // tensor-core path: 256 x 256 tiles on CTA pairs (tcgen05 cta_group::2)
    float *colsum_part;  // EPI_DGELU on tensor cores: fp32 column sums per 32-row block [ceil(M/32), N]
    // Batched GEMMs: `batch` independent problems whose operands and outputs are
    // contiguous [batch][rows][cols] arrays (attention heads).  1 = plain GEMM.
    int64_t batch;
    float scale;          // EPI_ATTN_SCORE, EPI_ATTN_DS
    bool causal;          // EPI_ATTN_SCORE: mask columns past the row
    const float *rowvec;  // EPI_ATTN_DS: D, one fp32 per output row, [batch][M]
    // Causal per-head products (tensor-core path, square M = K, one shard): only
    // the k range the zero pattern leaves, in whole tiles.  1: k below the end of
    // the M-tile (P V, dS K); 2: k from the start of the M-tile on (P^T dO, dS^T Q).
    int causal_k;
    bool skip_upper;  // skip tiles wholly above the diagonal (scores, dS)
    // EPI_STORE with an MN-major A on tensor cores: also write bias_grad[n] =
    // sum_k B(k, n) (bf16), computed by the MMA from an extra M-tile whose A is
    // `ones`, a 64 x 64 bf16 block of ones (8 KiB, 16-byte aligned).
    const void *ones;
    void *bias_grad;
    // Per-head GEMMs addressing their operands and output in place (tensor-core
    // path; EPI_ATTN_SCORE, EPI_ATTN_DS, EPI_STORE): a rank of 0 or 3 is the
    // plain [batch][rows][cols] block.
    bool heads_layout;
    HeadView a_view, b_view, o_view;
    // Row pitches in elements of operand A and B and of the output (0: contiguous),
    // multiples of 8; batch must be 1 where one is set.
    int64_t lda, ldb, ldo;
    // EPI_XENT_*, EPI_FOLD32.  parts = 3: the operands are fp32 numbers given as the sum of
    // three bf16 matrices, a_part / b_part elements apart, and each k-block is
    // multiplied six times (every pair of parts but those below 2^-22).  ksplit > 1 (ACC32, FOLD32):
    // the K range in ksplit parts of nshards * kshard elements, each an output [M, N] of its
    // own, one after the other in out0.  XENT_FOLD, FOLD32 and the XENT_GRADs take K (of a split) in
    // nshards ranges of kshard elements (all pairs of parts in one accumulation where there is one range).
    int parts;
    int64_t a_part, b_part;
    int ksplit;
    bool small_tile;  // 128 x 128 tiles on single CTAs (XENT_GRAD, XENT_GRAD3, ACC32, FOLD32, STORE_UNIT)
    // EPI_XENT_STATS, EPI_XENT_GRAD: rows are tokens, columns vocabulary rows
    // col0 .. col0 + N - 1 of W.
    const int64_t *target;   // [M]
    int64_t ignore_index, col0, vocab;
    float2 *part;            // STATS: (max, sum) of column group k, row m, at part[k * M + m]
    float *target_logit;     // STATS: [M], written where the target is one of the columns
    const float *row_lse;    // GRAD: [M]
    const float *dloss;      // GRAD: [M]; a target that is ignored or outside [0, vocab) has none
    float *unit;             // GRAD: where its unit goes; EPI_STORE_UNIT: where it is read
    bool accumulate;         // EPI_ACC32, EPI_FOLD32: add to what out0 holds
    int tile_n;              // EPI_XENT_FOLD: columns per tile, a multiple of 32 up to 256 (0: 256)
    // EPI_NS_*: fp16 operands.  POLY reads A through aux; UPDATE and LAST read the
    // two parts of X through aux (high) and aux2 (low).  out0 / out1: X' high, low.
    // LAST writes an [batch][out_rows][out_cols] array, the rest of the tile is dropped.
    // GRAM32 and FINAL: X as two parts, or with x_single the high one alone.
    bool x_single;
    const void *aux2;
    float alpha, beta, diag;
    int64_t out_rows, out_cols;
};

// Column groups of the EPI_XENT_STATS partials: four per 512-wide tile (128 columns each), or
// two per tile of EPI_XENT_FOLD.
inline int64_t xent_groups(int64_t N, int tile_n) {
    return tile_n == 512 ? (N + 511) / 512 * 4 : (N + tile_n - 1) / tile_n * 2;
}

// Tensor-core path: bf16 operands, fp32 accumulation in TMEM (tcgen05).
cudaError_t launch_tc_gemm(Epi epi, const GemmArgs &g, int num_sms, cudaStream_t st);

// Whether launch_tc_gemm runs this product on 256 x 512 tiles (CTA pairs; the
// store (both operands MN-major or both K-major), bias + GeLU and GeLU'
// epilogues of one shard on plain operands) rather than 256 x 256.  TPMLP_WIDE=0 keeps 256 x 256 (a tuning knob, read per call).
bool tc_wide_tile(Epi epi, const GemmArgs &g);

// FFMA path: element type fp32 (is_bf16 = false) or bf16, fp32 accumulation.
cudaError_t launch_simt_gemm(Epi epi, bool is_bf16, const GemmArgs &g, cudaStream_t st);

// Deterministic column sums out[c] = sum_r x[r,c] in two launches (per-chunk fp32
// partials into `partials`, then an in-order sum of the chunks).
int64_t colsum_chunks(int64_t rows, int64_t cols);
cudaError_t launch_colsum(bool is_bf16, const void *x, int64_t rows, int64_t cols, float *partials,
                          void *out, cudaStream_t st, int *launches);

// Second pass alone: out[c] = sum over `chunks` rows of partials[k, c], in order.
// `ones` (optional): an 8 KiB block the kernel also fills with bf16 ones.
cudaError_t launch_colsum_final(bool is_bf16, const float *partials, int64_t chunks, int64_t cols, void *out,
                                cudaStream_t st, void *ones = nullptr);

// A kernel that waits on a barrier nothing arrives on and reports the timeout.
cudaError_t launch_timeout_probe(uint32_t *status, uint64_t wait_ns, cudaStream_t st);

// LayerNorm over the rows of a row-major [rows, h] matrix (fp32 statistics).
struct LnArgs {
    int64_t rows, h;
    float eps;
    const void *x;      // input rows
    const void *gamma;  // [h]
    const void *beta;   // [h] (forward)
    void *y;            // forward output
    float *mean;        // [rows]
    float *rstd;        // [rows]
    const void *dy;     // backward: gradient w.r.t. the output
    void *dx;           // backward: gradient w.r.t. the input
    void *dgamma;       // [h]
    void *dbeta;        // [h]
    float *partials;    // backward: ln_partial_floats(rows, h) floats of scratch
};
int64_t ln_partial_floats(int64_t rows, int64_t h);
cudaError_t launch_ln_forward(bool is_bf16, const LnArgs &a, cudaStream_t st);
cudaError_t launch_ln_backward(bool is_bf16, const LnArgs &a, cudaStream_t st, int *launches);

// Attention support.  Problem z = b*heads + g over `nb` sequences of S tokens;
// token-major O and dO are [T, h] with head g at columns [g*d, (g+1)*d).
struct HeadLayout {
    int64_t nb, S, h, heads, d;
};
// wtile > 0: each row writes P only up to the end of its wtile-wide column tile.
cudaError_t launch_softmax(const void *S, void *P, int64_t rows, int64_t cols, bool causal, int64_t wtile,
                           cudaStream_t st);
// D[z*S + s] = row dot of dO and O over head g's columns of token b*S + s (token-major inputs).
// `ones` (optional): an 8 KiB block the kernel also fills with bf16 ones.
cudaError_t launch_rowdot(const HeadLayout &L, const void *dO, const void *O, float *D, cudaStream_t st,
                          void *ones = nullptr);

// Vocabulary cross entropy: the kernels over token rows (xent.cu).
struct RowArgs {
    int64_t tokens, vocab, ignore_index;
    const int64_t *target;  // [tokens]
    const float2 *part;     // [groups][tokens]: (max, sum of exponentials)
    int64_t groups;
    float *target_logit;    // [tokens]
    uint32_t *status;
};
cudaError_t launch_xent_combine(const RowArgs &a, float *loss, float *lse, cudaStream_t st);
// Statistics of few tokens in one pass over W (xent_few says whether these are); partials in `groups` = xent_few_groups(vocab) groups.
constexpr int64_t XENT_FEW_SMEM = 192 * 1024;
bool xent_few(bool is_bf16, int64_t tokens, int64_t hidden);
int64_t xent_few_groups(int64_t vocab);
cudaError_t launch_xent_few(bool is_bf16, const RowArgs &a, const void *X, const void *W, int64_t hidden, float2 *part,
                            float *loss, float *lse, cudaStream_t st);
// dS of few tokens over vocabulary rows col0 .. col0 + RowArgs::vocab - 1, W at the first of them, from
// logits of the same bits as launch_xent_few's.  out: [tokens][ld] in bf16, in units of *unit, or
// for fp32 three such matrices, `part` elements apart.
struct FewGrad {
    const float *lse, *dloss;
    float *unit;
    void *out;
    int64_t ld, part, col0, all_vocab;
};
cudaError_t launch_xent_few_grad(bool is_bf16, const RowArgs &a, const void *X, const void *W, int64_t hidden,
                                 const FewGrad &d, cudaStream_t st);
// out[r][c] = sum over the `splits` matrices [rows][ld] of in, in order, in the output's type.
// With unit the sums are multiplied by *unit.
cudaError_t launch_sum_splits(bool is_bf16, const float *in, int splits, int64_t rows, int64_t cols, int64_t ld,
                              const float *unit, void *out, cudaStream_t st);
// fp32 [rows][cols] as three bf16 matrices [rows][ld], ld >= cols a multiple of 4, the rest zero.
struct Split3 {
    const float *in;
    int64_t rows, cols, ld;
    void *out;
};
cudaError_t launch_split3(const Split3 &a, const Split3 &b, cudaStream_t st);
// FFMA path: logits [tokens, n] of vocabulary rows col0 .. col0 + n - 1.
cudaError_t launch_xent_piece_stats(const RowArgs &a, const float *logits, int64_t n, int64_t col0, float2 *part,
                                    cudaStream_t st);
cudaError_t launch_xent_piece_grad(bool is_bf16, const RowArgs &a, const float *logits, int64_t n, int64_t col0,
                                   const float *lse, const float *dloss, void *out, cudaStream_t st);

// A [matrices][p][p] (fp16, whole) = scale * the sum of the splits' lower triangles
// [splits][matrices][p][p], in order.
cudaError_t launch_ortho_gram_sum(const float *in, int splits, int64_t matrices, int64_t p, float scale, void *A,
                                  cudaStream_t st);

// Newton-Schulz orthogonalisation (ortho.cu): X = G scale / (|G| + eps) as hi + lo / 2^11.
struct OrthoStart {
    const void *G;  // [batch][rows][cols]
    int64_t batch, rows, cols, P, Q;
    float eps, scale;
    void *part;     // ortho_norm_blocks(batch, rows * cols) * batch * 12 bytes
    void *hi, *lo;  // fp16 [batch][P][Q]
    float lo_scale; // lo holds the remainder times this
    float *rest;    // null: X scaled by the whole factor; else by the power of two below it, and the rest here
};
int64_t ortho_norm_blocks(int64_t batch, int64_t n);
// The block sums of the norms, then the scaled parts.
cudaError_t launch_ortho_norm(bool is_bf16, const OrthoStart &a, cudaStream_t st);
cudaError_t launch_ortho_scale(bool is_bf16, const OrthoStart &a, cudaStream_t st);
// The steps on p x p Gram matrices, p <= 128 (ns_chain.cu).
constexpr int NS_CHAIN_P = 128;
struct NsChain {
    int64_t matrices, P;  // P: 64 or 128, the row pitch and size in memory
    int size;             // rows and columns in use, a multiple of 16
    const float *gram;    // [splits][matrices][P][P]
    int splits;
    float unit;           // A_0 = unit * rest^2 * the sum of the splits
    const float *rest;    // [matrices]; Q is multiplied by it
    int steps;
    float a, b, c, q_scale;
    void *Q;              // fp16 [2][matrices][P][P]: high and low part of q_scale * Q
    uint32_t *status;
    uint64_t wait_ns;
};
cudaError_t launch_ns_chain(const NsChain &c, cudaStream_t st);
cudaError_t launch_ortho_unpad(const void *in, int64_t batch, int64_t rows, int64_t cols, int64_t P, int64_t Q,
                               void *out, cudaStream_t st);

// Norms of queries and keys per head and the position rotation (qk.cu).  Head j of shard i of
// token r is at p + r * row + i * shard + j * d, in elements.
struct HeadRows {
    const void *p;
    int64_t row, shard;
};
struct QkArgs {
    int sms;           // of the device
    int64_t tokens;
    int heads, kv_heads, t, d;
    int rot;           // components that rotate
    bool interleaved;  // pairs (2i, 2i + 1) instead of (i, i + rot / 2)
    bool norm;
    float eps, amplitude;
    HeadRows q, k, v;       // inputs (v: append only)
    HeadRows oq, ok;        // outputs: rotated (ok: not for append), or the gradients of q and k
    const void *gain_q, *gain_k;  // [d]
    const int64_t *position;      // [tokens]
    const uint64_t *turns;        // [rot / 2]: turns per position, times 2^64
    bool vec;               // every row start and stride on 16 bytes
    // append: token r's K and V go to slot[r] of the cache
    const int64_t *slot;
    void *cache_k, *cache_v;
    int64_t page_size, slots, page_stride, head_stride, token_stride;
    uint32_t *status;
    // backward: gradients of the rotated q and k
    HeadRows dq, dk;
    float *part;            // qk_partial_floats() floats
    void *dgain_q, *dgain_k;
};
int64_t qk_partial_floats(int64_t tokens, int d);
cudaError_t launch_qk_forward(bool is_bf16, const QkArgs &a, bool append, cudaStream_t st);
cudaError_t launch_qk_backward(bool is_bf16, const QkArgs &a, cudaStream_t st, int *launches);

// Attention of new tokens over a paged cache (cache_attn.cuh says how the work is divided).
struct CacheAttnArgs {
    int64_t tokens, batch, max_pages;
    int heads, kv_heads, group, d;  // group = heads / kv_heads
    const void *q;                  // [tokens][heads][d]
    void *o;
    const int32_t *q_start;         // [batch + 1]
    const int32_t *kv_len;          // [batch]
    const int32_t *table;           // [batch][max_pages]
    const int64_t *tree;            // [tokens][tree_words], null: causal
    int tree_words;
    float scale_log2;               // the scores' factor times log2(e)
    const void *k, *v;              // page p, head h, row r at p * page_stride + h * head_stride + r * token_stride
    int64_t pages, page_size, page_stride, head_stride, token_stride;
    bool vec;                       // rows start on 16 bytes
    uint32_t *status;
    void *cuts;                     // [blocks] of 32 bytes: the unit that begins in a block and goes on
    float *part;                    // [2 blocks][rows per tile][d]
    float2 *part_ml;                // [2 blocks][rows per tile]: maximum (log2), sum
    uint64_t wait_ns;
};
constexpr int CACHE_ATTN_BLOCKS = 320;    // at most
constexpr int CACHE_ATTN_TC_ROWS = 128;   // rows (token, head) of a tile: tensor-core and FFMA kernel
constexpr int CACHE_ATTN_SIMT_ROWS = 32;
int cache_attn_simt_blocks(bool is_bf16, int d, int num_sms);
cudaError_t launch_cache_attn_simt(bool is_bf16, const CacheAttnArgs &a, int num_sms, cudaStream_t st);
// bf16 on the tensor cores; cache_attn_tc says whether the cache's layout allows it.
bool cache_attn_tc(const CacheAttnArgs &a);
cudaError_t launch_cache_attn_tc(const CacheAttnArgs &a, int num_sms, cudaStream_t st);

// Records a description of the last failure of this host thread (read back by
// tpmlp_last_error()).
void set_last_error(const char *fmt, ...);

// Adds to the count reported by tpmlp_launch_count().
void add_launches(uint64_t n);

}  // namespace tpmlp
