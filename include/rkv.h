/*
 * rkv.h -- C ABI of librkv, the GB300 (sm_103a) implementation of R-KV's
 * decode-time KV-cache compression step.
 *
 * The operation (R-KV review, yoonschallenge.tistory.com/1236):
 *   - opening notes and summary-table row "Decoding-time compression
 *     scheme": the fixed cache B_budget and the buffer B_buffer of newly
 *     generated tokens are merged (here: rows 0..budget-1 followed by the
 *     buffer rows, n_cached rows in all); the newest n_obs (8) observation
 *     tokens are always kept; every other token is scored and only the top
 *     ones are kept, so that exactly `budget` rows remain.
 *   - row "importance": I_i is the softmax attention the n_obs observation
 *     queries give key i (mean over the queries, scale 1/sqrt(d), causal among
 *     the observation tokens), max-pooled over the G query heads that share
 *     the KV head.
 *   - row "redundancy": R_i is the mean cosine similarity of key i to the
 *     other n_cached-1 keys of the same KV head; a similar pair is one with
 *     cosine > tau; token i is protected (its above-tau similarities are
 *     dropped from its sum) when fewer than beta newer tokens are similar to
 *     it, i.e. the beta most recent tokens of a similar group are protected.
 *   - row "final selection criterion": Z_i = lambda*I_i - (1-lambda)*R_i
 *     (lambda = 0.1 on the page); ties go to the newer token.
 *   - question 2, cause 3: the kept K/V rows are copied into the new cache.
 *
 * One "problem" is one (layer, sequence, KV head).  All P problems of a call
 * share n_cached, budget and the parameters and are processed by one launch
 * per kernel.
 *
 * Layouts (every array contiguous, row-major; element type `dtype`):
 *   K, V                 [P, n_capacity, head_dim]; problem p starts at
 *                        element p*n_capacity*head_dim.  head_dim*elem_size
 *                        must be a multiple of 16 bytes and every base pointer
 *                        16-byte aligned.
 *   out_K, out_V         [P, out_capacity, head_dim] (out_capacity = 0 in the
 *                        descriptor means n_capacity): an out-of-place call
 *                        may write the kept rows into buffers of just
 *                        `budget` rows per problem.
 *   Q_obs                [P, G, n_obs, head_dim]: query q of query head g of
 *                        problem p.  Query head g of the G that share the KV
 *                        head of problem p.
 *   out_idx              [P, budget] int32.
 *   out_I, out_R, out_Z  [P, n_cached] float.
 *
 * Ownership and execution: every pointer is device memory owned by the
 * caller.  The calls never allocate or free device memory and never
 * synchronise: they check their arguments on the host, enqueue kernels on
 * `stream` (a cudaStream_t, or NULL for the legacy default stream) and return.
 * Results are valid in stream order.  Scratch memory is the caller's
 * `workspace` of at least rkv_workspace_size() bytes, 256-byte aligned; one
 * workspace must not be used by two calls that may overlap on the GPU.
 *
 * Errors: each call returns RKV_OK or an RKV_ERR_* code and enqueues nothing
 * on error.  Errors raised on the device (a bounded wait that timed out, an
 * index found out of range) are recorded in the workspace and read by
 * rkv_get_device_status().  Not thread-safe only where stated.
 */
#ifndef RKV_H
#define RKV_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

enum {
    RKV_OK = 0,
    RKV_ERR_INVALID_ARG = 1, /* a size, count or pointer is invalid */
    RKV_ERR_UNSUPPORTED = 2, /* dtype / head_dim / group size not supported */
    RKV_ERR_WORKSPACE = 3,   /* workspace missing, misaligned or too small */
    RKV_ERR_ALIAS = 4,       /* outputs partially overlap inputs */
    RKV_ERR_CUDA = 5,        /* a CUDA runtime call or launch failed */
    RKV_ERR_DEVICE = 6,      /* a kernel recorded an error (see status) */
    RKV_ERR_TOO_LARGE = 7    /* request exceeds rkv_compress_noalloc's scratch */
};

enum { RKV_DTYPE_BF16 = 0, RKV_DTYPE_FP32 = 1 };

/* Shape of one call's problems. */
typedef struct {
    int64_t num_problems; /* P = layers * sequences * kv_heads (>= 0)        */
    int32_t gqa_group;    /* G, query heads per KV head, 1..16               */
    int32_t head_dim;     /* d, 64 or 128                                    */
    int32_t n_capacity;   /* rows allocated per problem in K and V           */
    int32_t dtype;        /* RKV_DTYPE_BF16 or RKV_DTYPE_FP32 (K, V, Q, out) */
    int32_t out_capacity; /* rows per problem in out_K/out_V (and rkv_gather's
                             dst); 0 = n_capacity.  Must be >= budget, and 0 or
                             n_capacity for in-place compaction.             */
} rkv_desc;

/* Largest n_cached accepted by rkv_compress / rkv_score. */
#define RKV_MAX_TOKENS 32768

/* Bytes of workspace rkv_compress / rkv_score need for `desc` and n_cached
 * tokens with n_obs observation tokens.  0 if the arguments are invalid. */
size_t rkv_workspace_size(const rkv_desc* desc, int n_cached, int n_obs);

/* One compression round (the whole step above) for all P problems.
 *   n_cached   rows in use per problem (merged cache + buffer), <= n_capacity
 *   budget     rows kept per problem, n_obs <= budget <= n_capacity and
 *              budget <= out_capacity
 *   n_obs      observation tokens (the newest n_obs rows), >= 1
 *   lambda, beta, tau   the parameters of Z, protection and similarity
 *   out_K/out_V  receive the kept rows in ascending original position in
 *              their rows 0..budget-1; rows >= budget are not touched.  They
 *              may be K/V themselves (in-place compaction) but must not
 *              overlap them otherwise (RKV_ERR_ALIAS).
 *   out_idx    [P, budget]: kept original row indices, strictly ascending;
 *              the last n_obs are n_cached-n_obs .. n_cached-1.
 * n_cached <= budget evicts nothing: out_idx = 0..n_cached-1 then -1, and the
 * rows are copied only when the outputs are not the inputs. */
int rkv_compress(const rkv_desc* desc, const void* K, const void* V, const void* Q_obs,
                 int n_cached, int budget, int n_obs, float lambda, int beta, float tau,
                 void* out_K, void* out_V, int32_t* out_idx,
                 void* workspace, size_t workspace_bytes, void* stream);

/* The scores alone (for tests and analysis): out_I, out_R, out_Z
 * [P, n_cached].  Observation tokens get R = 0 and Z = +inf. */
int rkv_score(const rkv_desc* desc, const void* K, const void* Q_obs, int n_cached,
              int n_obs, float lambda, int beta, float tau,
              float* out_I, float* out_R, float* out_Z,
              void* workspace, size_t workspace_bytes, void* stream);

/* Variants of the scoring (all off: the step above).
 *   redundancy_softmax  the R-KV review, question 2, cause 3, lists a softmax
 *                       of the redundancy among the operations of a
 *                       compression round.  1: the candidates' redundancy
 *                       becomes R'_i = exp(R_i) / sum_{j<C} exp(R_j) (R_i as
 *                       above, C = n_cached - n_obs candidates), so it sums
 *                       to 1 over the candidates; 0: R as above.
 *   pool_window         w, odd, 1..RKV_MAX_POOL_WINDOW.  A SnapKV-style
 *                       pooling of the importance over positions (SnapKV is
 *                       the attention-only method the review compares
 *                       against): I'_i = max of I_j over the candidates j
 *                       with |j - i| <= (w-1)/2 (the window is cut at the
 *                       candidates' ends).  1: no pooling.
 *   sentences           a sentence-level penalty (below), or NULL.
 *   schedule            a recent window and sampled selection (below), or
 *                       NULL.  With a schedule the L newest rows take the
 *                       place of the observation tokens in everything that
 *                       follows (they are not candidates; Z = +inf, R = 0).
 * Z_i = lambda*I'_i - (1-lambda)*R'_i - pen_i; observation tokens keep their
 * I, get R = 0 and Z = +inf as before.  A NULL variant is all off. */
/* Sentence-level redundancy (the SkipKV review, yoonschallenge.tistory.com/
 * 1230, summary-table rows "Method 1: Sentence-level KV Storage Skipping",
 * "Final eviction score" and "Cache Range Monitoring").  A sentence is
 * represented by the mean of its tokens' last-layer hidden states
 * (rkv_sentence_reps computes it); when the cosine similarity of sentence a
 * and a later sentence b of the same sequence exceeds tau, a is the
 * redundant one.  Its penalty is pen_a = max of cos(a, b) over the later b
 * with cos(a, b) > tau (0 if none), and every cached row of sentence a has
 * pen_a subtracted from its Z, so redundant earlier sentences go first while
 * the budget still decides how many rows stay.  The sentence of each cached
 * row is tracked in seg_id, which the compression compacts along with the
 * rows (the cache-range mapping the review describes).
 *   reps      [num_seqs, max_sentences, hidden_dim] fp32 (rows >= count[s]
 *             ignored)
 *   count     [num_seqs] sentences in use per sequence (device memory)
 *   seg_id    [P, ld_seg] int32: sentence of cached row i of problem p, or
 *             -1 (ids outside 0..count-1 count as none).  Problem p belongs
 *             to sequence (p / heads) % num_seqs (problems ordered layer,
 *             sequence, head).  After rkv_compress_ex / rkv_paged_compress
 *             entries 0..budget-1 hold the kept rows' sentences.
 *   penalty   [num_seqs, max_sentences] fp32, written: pen_a per sentence.
 * All pointers are device memory owned by the caller. */
typedef struct {
    const float* reps;
    const int32_t* count;
    int32_t* seg_id;
    float* penalty;
    int64_t num_seqs;      /* >= 1 */
    int32_t heads;         /* >= 1 */
    int32_t max_sentences; /* 1 .. RKV_MAX_SENTENCES */
    int32_t hidden_dim;    /* 4 .. RKV_MAX_HIDDEN, a multiple of 4 */
    int32_t ld_seg;        /* row stride of seg_id, >= n_cached */
    float tau;             /* sentence-similarity threshold */
} rkv_sentences;
#define RKV_MAX_SENTENCES 65536
#define RKV_MAX_HIDDEN 16384

/* ForesightKV-style schedule and selection (the ForesightKV summary page,
 * gist.science/ko/paper/2602.03203, section "Dynamic eviction process"):
 * when the cache holds B + L rows the newest L are kept and the rest are
 * compressed to B - L by the scores; the decision takes the top K and then
 * samples (multinomial sampling) to add randomness.  The R-KV score Z stands
 * in for the page's learned scorer.  Here:
 *   - the newest L = recent_window rows (n_obs <= L <= budget) are kept like
 *     the observation tokens (which still supply the importance queries);
 *     the other C = n_cached - L rows are the candidates, k = budget - L of
 *     them are kept;
 *   - the pool is the top pool_size candidates by Z (ties to the newer);
 *   - k of the pool are drawn without replacement with probabilities
 *     proportional to exp(Z_i / temperature): exactly the k largest
 *     Z_i / temperature + g_i over the pool, g_i = -log(-log(u_i)) (Gumbel
 *     noise) from the caller's uniforms u [P, ld_uniforms] in [0, 1), so a
 *     seeded generator on the caller's side makes the draw reproducible.
 * pool_size == k is the deterministic top-k (uniforms may be NULL). */
typedef struct {
    int32_t recent_window;  /* L */
    int32_t pool_size;      /* K, k <= K <= C */
    float temperature;      /* > 0 */
    int32_t ld_uniforms;    /* >= C when uniforms are given */
    const float* uniforms;  /* [P, ld_uniforms]; needed when K > k */
} rkv_schedule;

typedef struct {
    int32_t redundancy_softmax;       /* 0 or 1 */
    int32_t pool_window;              /* odd, 1 .. RKV_MAX_POOL_WINDOW */
    const rkv_sentences* sentences;   /* NULL: no sentence-level penalty */
    const rkv_schedule* schedule;     /* NULL: keep the n_obs newest, top-k */
} rkv_variant;
#define RKV_MAX_POOL_WINDOW 255

/* Sentence representations: out_reps[s, a, :] = mean of hidden[s, t, :] over
 * the tokens t with token_seg[s, t] == a (zeros for a sentence without
 * tokens).  hidden [num_seqs, T, hidden_dim] (dtype bf16 or fp32), token_seg
 * [num_seqs, T] int32 (-1: no sentence; ids >= max_sentences ignored),
 * out_reps [num_seqs, max_sentences, hidden_dim] fp32. */
int rkv_sentence_reps(const void* hidden, const int32_t* token_seg, int64_t num_seqs, int T,
                      int hidden_dim, int dtype, int max_sentences, float* out_reps,
                      void* stream);

/* The penalties alone: writes sent->penalty from reps, count and tau. */
int rkv_sentence_penalty(const rkv_sentences* sent, void* stream);

/* rkv_compress / rkv_score with a variant (invalid variant fields:
 * RKV_ERR_INVALID_ARG).  rkv_score_ex's out_I and out_R are the I' and R'
 * that enter Z. */
int rkv_compress_ex(const rkv_desc* desc, const void* K, const void* V, const void* Q_obs,
                    int n_cached, int budget, int n_obs, float lambda, int beta, float tau,
                    const rkv_variant* variant, void* out_K, void* out_V, int32_t* out_idx,
                    void* workspace, size_t workspace_bytes, void* stream);
int rkv_score_ex(const rkv_desc* desc, const void* K, const void* Q_obs, int n_cached,
                 int n_obs, float lambda, int beta, float tau, const rkv_variant* variant,
                 float* out_I, float* out_R, float* out_Z,
                 void* workspace, size_t workspace_bytes, void* stream);

/* ---------------------------------------------------------------- paged --
 * The step on a paged KV cache.  The review (question 2, cause 4) names the
 * clash between pruning and a block-structured (PagedAttention) cache as a
 * main limitation: pruning re-lays the KV tensor out, and freeing the old
 * cache to allocate a compressed one costs memory management.  Here a
 * sequence's rows live in fixed-size blocks of a shared pool, compaction runs
 * in place inside the sequence's own blocks, and the blocks it empties are
 * handed back whole.
 *
 * Layout: K_pool, V_pool [num_blocks, num_kv_heads, block_size, head_dim]:
 * one (block, head) is a contiguous block_size x head_dim tile.  Sequence s
 * (one row of block_table [num_seqs, max_blocks_per_seq], int32) holds its
 * logical row r of head h at block block_table[s][r / block_size], row
 * r % block_size.  Problem p = s * num_kv_heads + h; Q_obs is
 * [P, G, n_obs, head_dim] and out_idx [P, budget] as for rkv_compress.
 * The entries 0 .. ceil(n_cached / block_size) - 1 of every table row must be
 * distinct valid block ids, not shared between sequences; entries outside
 * 0..num_blocks-1 are recorded as a device error and their rows skipped.
 *
 * Effect: for every problem the kept rows (out_idx) move to logical rows
 * 0..budget-1 of the same sequence and head, in place; rows past budget in
 * the last kept block are left as they were.  The blocks past the kept ones,
 * entries ceil(budget/bs) .. ceil(n_cached/bs) - 1 of each row, are no longer
 * used: their ids are written to out_freed [num_seqs, n_free] (n_free =
 * rkv_paged_freed_per_seq()) and the table entries are set to -1.  Rows after
 * n_cached in each sequence's last block (space it has not filled yet) are
 * neither read nor written, and blocks not named by the first
 * ceil(n_cached/bs) entries of any row are not touched. */
typedef struct {
    int64_t num_seqs;           /* S, rows of the block table (>= 0)         */
    int32_t num_kv_heads;       /* H, heads per block; P = S * H problems     */
    int32_t gqa_group;          /* G, query heads per KV head, 1..16          */
    int32_t head_dim;           /* d, 64 or 128                               */
    int32_t block_size;         /* rows per block, a power of two, 1..1024    */
    int32_t num_blocks;         /* blocks in each pool (>= 1)                 */
    int32_t max_blocks_per_seq; /* row stride of block_table (>= 1)           */
    int32_t dtype;              /* RKV_DTYPE_BF16 or RKV_DTYPE_FP32           */
} rkv_paged_desc;

/* Workspace bytes rkv_paged_compress needs for these arguments (0 if they
 * are invalid).  bf16 pools with blocks of at least 128 rows are read in
 * place by the tensor-core stages when the call's shapes fit them (n_cached
 * <= 4352, gqa_group * n_obs a multiple of 8 up to 128, beta <= 63): then the
 * size equals rkv_workspace_size() of the same problems.  Otherwise (blocks
 * under 128 rows, fp32 pools, the CUDA-core paths) it adds one contiguous
 * copy of the P problems' keys [P, n_cached, head_dim], which the key
 * statistics write for the later stages. */
size_t rkv_paged_workspace_size(const rkv_paged_desc* desc, int n_cached, int n_obs,
                                int beta);

/* Blocks freed per sequence: ceil(n_cached/bs) - ceil(budget/bs), or 0 when
 * n_cached <= budget; -1 if the arguments are invalid. */
int rkv_paged_freed_per_seq(const rkv_paged_desc* desc, int n_cached, int budget);

/* One compression round on the paged cache (see above).  n_cached <= budget:
 * out_idx is the identity and nothing moves or is freed.  Problems whose
 * scores, keys and kept indices exceed the fused selection kernel's shared
 * memory (8*(n_cached-n_obs) + 4*budget > 160 KB) return RKV_ERR_UNSUPPORTED. */
int rkv_paged_compress(const rkv_paged_desc* desc, void* K_pool, void* V_pool,
                       const void* Q_obs, int32_t* block_table, int n_cached, int budget,
                       int n_obs, float lambda, int beta, float tau,
                       const rkv_variant* variant, int32_t* out_idx, int32_t* out_freed,
                       void* workspace, size_t workspace_bytes, void* stream);

/* ------------------------------------------------------ the cache in use --
 * What a decode loop does with a paged cache between two compressions:
 * rotate the new tokens' queries and keys by their positions, write the new
 * rows through the block table (as they are, or at 4 or 8 bits), and attend over
 * the rows.  After a compression a row of the cache is no longer its token's
 * position, so the calls take the positions (int32 [tokens]) apart from the
 * rows (lens).
 *
 * lens [num_seqs] int32: the rows in use of each sequence, counted with the
 * tokens the call brings: the append writes rows lens[s] - n_s .. lens[s] - 1
 * and the attention that follows reads rows 0 .. lens[s] - 1.
 *
 * New tokens come as rows of heads (rkv_rows): value d of head h of token j
 * at data[j * token_stride + h * head_stride + d], or, in calls with the same
 * number of tokens for every sequence, of token i of sequence s at
 * data[s * seq_stride + i * token_stride + h * head_stride + d].  Strides
 * count elements; data and every stride used are multiples of 16 bytes, so a
 * slice of a fused projection is taken as it is.
 *
 * The launches of these calls may begin while the stream's last kernel ends
 * (programmatic dependent launch), and a call reads and writes nothing before
 * everything in front of it is over: results are in stream order as ever, also in
 * captured graphs. */
typedef struct {
    void* data;
    int64_t seq_stride;   /* unused where tokens are numbered through */
    int64_t token_stride;
    int64_t head_stride;
} rkv_rows;

/* Rotary positions.  Pair i (0 <= i < rot_dim / 2) of a head is turned by
 * pos * f_i:  (x, x') -> m (x cos - x' sin, x' cos + x sin), the pair being
 * elements (i, i + rot_dim / 2) or, interleaved, (2i, 2i + 1); elements past
 * rot_dim pass through.  f_i = base^(-2i / rot_dim), and for long contexts
 *   LINEAR    f_i / factor
 *   NTK       the base becomes base * factor^(rot_dim / (rot_dim - 2))
 *   BY_PARTS  with t_i = original_len * f_i / (2 pi) turns over the trained
 *             length and g = (t_i - low) / (high - low) cut to [0, 1]:
 *             f_i (g + (1 - g) / factor)
 * m = attn_factor (1 leaves lengths alone).  The plan is host memory, made
 * once: it holds each f_i as a 64-bit fixed-point part of a turn, so pos * f_i
 * is reduced exactly whatever the position (with angles of at most 1 radian a
 * position the result is off by less than 2^-22 turns at position 2^31, by less
 * than 2^-24 below 2^27; larger angles of a caller's own in proportion). */
enum {
    RKV_ROPE_NONE = 0,
    RKV_ROPE_LINEAR = 1,
    RKV_ROPE_NTK = 2,
    RKV_ROPE_BY_PARTS = 3
};
#define RKV_MAX_ROT_DIM 128
typedef struct {
    int32_t rot_dim;      /* even, 2 .. RKV_MAX_ROT_DIM                       */
    int32_t interleaved;  /* 0 or 1                                           */
    int32_t scaling;      /* RKV_ROPE_*                                       */
    double base;          /* > 0                                              */
    double factor;        /* > 0                                              */
    double original_len;  /* > 0 for BY_PARTS                                 */
    double low, high;     /* low < high for BY_PARTS                          */
    double attn_factor;   /* m, finite                                        */
} rkv_rope_config;
typedef struct {
    int32_t rot_dim;
    int32_t interleaved;
    float attn_factor;
    int32_t reserved;
    uint64_t turns[RKV_MAX_ROT_DIM / 2]; /* f_i / (2 pi) in units of 2^-64 turn */
} rkv_rope_plan;

/* Fill a plan from a configuration, or from rot_dim / 2 angles per position
 * (radians, finite) of the caller's own.  Host only. */
int rkv_rope_init(const rkv_rope_config* config, rkv_rope_plan* plan);
int rkv_rope_init_freqs(int rot_dim, int interleaved, const double* freqs, double attn_factor,
                        rkv_rope_plan* plan);

/* out = the rows of q (q_heads per token) and, unless k is NULL, of k
 * (k_heads per token) turned by their tokens' positions; inverse != 0 turns
 * by the opposite angles, which is the gradient's map (the transpose).
 * num_tokens tokens, tokens_per_seq of them (a divisor of num_tokens) per
 * sequence for seq_stride.  An output may be its input (same pointer and
 * strides), where q and k may be slices of one projection's rows; other
 * overlaps are RKV_ERR_ALIAS.  fp32 arithmetic, one rounding. */
int rkv_rope_apply(const rkv_rope_plan* plan, int dtype, int head_dim, int64_t num_tokens,
                   int64_t tokens_per_seq, const int32_t* positions, int inverse, int q_heads,
                   const rkv_rows* q, const rkv_rows* out_q, int k_heads, const rkv_rows* k,
                   const rkv_rows* out_k, void* stream);

/* Append to a paged cache (rkv_paged_desc; dtype is that of the pools and of
 * k, v, q).  With cu_tokens NULL every sequence brings new_per_seq tokens
 * (num_tokens = num_seqs * new_per_seq); otherwise sequence s brings tokens
 * cu_tokens[s] .. cu_tokens[s + 1] - 1 ([num_seqs + 1] int32 on the device,
 * ascending from 0), num_tokens bounds cu_tokens[num_seqs], and for tokens past
 * it (padding) nothing is written.  k and v have num_kv_heads heads.
 * With a rope, k is turned by positions (NULL: by the rows it is written to);
 * q (num_kv_heads * gqa_group heads; may be NULL) is turned the same way, or
 * copied without a rope, into out_q (which may be q, beside k and v of one
 * projection).  Rows outside the table
 * and ids that name no block are recorded as a device error in `workspace`
 * (NULL: not recorded; else 256-byte aligned, only its error word is used)
 * and not written.  Two tokens of a call must not share a row of the pool.
 * Nothing else of the pools changes. */
int rkv_paged_append(const rkv_paged_desc* desc, const rkv_rope_plan* rope, void* K_pool,
                     void* V_pool, const int32_t* block_table, const int32_t* lens,
                     int64_t num_tokens, int new_per_seq, const int32_t* cu_tokens,
                     const int32_t* positions, const rkv_rows* k, const rkv_rows* v,
                     const rkv_rows* q, const rkv_rows* out_q, void* workspace, void* stream);

/* A paged cache held in 4 bits.  Each row of head_dim values is stored in
 * groups of 32 neighbours as x ~ scale * code + low, with t(x) the fp32 nearest
 * to x - low:
 *   low   the largest bf16 that is not above the group's smallest value,
 *   scale the smallest bf16 that is not below the fp32 nearest to
 *         t(largest) / 15,
 *   code  the whole number nearest to t(x) * r, r the fp32 nearest to 1 / scale
 *         (0 where the scale is below 2^-126); halves go to even.
 * A group that holds a NaN or an infinity, or whose range passes the largest
 * float, reads as NaN.  codes [num_blocks, num_kv_heads, block_size,
 * head_dim / 2] bytes: with W = head_dim / 32, 16-bit word g * W + w of a row
 * holds values 32 w + 4 g .. 32 w + 4 g + 3 (lowest bits first), so that a
 * lane's share of every group lies together.  scales [num_blocks,
 * num_kv_heads, block_size, W, 2] bf16: (scale, low).  Codes are 16-byte
 * aligned, scales too. */
typedef struct {
    void* k_codes;
    void* k_scales;
    void* v_codes;
    void* v_scales;
} rkv_q4_cache;

/* rkv_paged_append into a 4-bit cache (desc->dtype: that of k, v and q). */
int rkv_q4_append(const rkv_paged_desc* desc, const rkv_rope_plan* rope,
                  const rkv_q4_cache* cache, const int32_t* block_table, const int32_t* lens,
                  int64_t num_tokens, int new_per_seq, const int32_t* cu_tokens,
                  const int32_t* positions, const rkv_rows* k, const rkv_rows* v,
                  const rkv_rows* q, const rkv_rows* out_q, void* workspace, void* stream);

/* Rows of a 4-bit cache as values: row first[s] + i (first NULL: i) of
 * sequence s and head h, i < n_rows, to out_K and out_V
 * [num_seqs * num_kv_heads, n_rows, head_dim] (desc->dtype; either may be
 * NULL), the layout rkv_score and rkv_compress take.  Rows at or past lens[s]
 * are not written. */
int rkv_q4_read(const rkv_paged_desc* desc, const rkv_q4_cache* cache,
                const int32_t* block_table, const int32_t* lens, const int32_t* first,
                int n_rows, void* out_K, void* out_V, void* workspace, void* stream);

/* A paged cache held in 8 bits: each row of head_dim values as x ~ scale * code,
 *   scale the fp32 nearest to the row's largest magnitude / 127,
 *   code  the whole number nearest to x * r, r the fp32 nearest to 1 / scale (0
 *         where the scale is below 2^-126); halves go to even; -127 .. 127.
 * A row that holds a NaN or an infinity reads as NaN.  codes [num_blocks,
 * num_kv_heads, block_size, head_dim] int8, in the values' order; scales
 * [num_blocks, num_kv_heads, block_size] fp32.  All four arrays are 16-byte
 * aligned. */
typedef struct {
    void* k_codes;
    void* k_scales;
    void* v_codes;
    void* v_scales;
} rkv_q8_cache;

/* rkv_paged_append into an 8-bit cache (desc->dtype: that of k, v and q). */
int rkv_q8_append(const rkv_paged_desc* desc, const rkv_rope_plan* rope,
                  const rkv_q8_cache* cache, const int32_t* block_table, const int32_t* lens,
                  int64_t num_tokens, int new_per_seq, const int32_t* cu_tokens,
                  const int32_t* positions, const rkv_rows* k, const rkv_rows* v,
                  const rkv_rows* q, const rkv_rows* out_q, void* workspace, void* stream);

/* rkv_q4_read of an 8-bit cache: scale * code, rounded to desc->dtype. */
int rkv_q8_read(const rkv_paged_desc* desc, const rkv_q8_cache* cache,
                const int32_t* block_table, const int32_t* lens, const int32_t* first,
                int n_rows, void* out_K, void* out_V, void* workspace, void* stream);

/* Attention of the newest n_new (1 .. RKV_MAX_NEW_TOKENS) tokens of every
 * sequence over its cache: token t sees rows j <= lens[s] - n_new + t,
 *   out[s, t, head] = sum_j p_j V_j,  p = softmax_j(scale * q . K_j)
 * with query heads h * gqa_group .. of KV head h.  A token that sees no row
 * (lens[s] < n_new, or 0), or only rows whose logits are -inf, gets zeros.  lse, unless NULL, receives
 * log(sum_j exp(scale * q . K_j)) [num_seqs, n_new, heads] fp32 (-inf where
 * nothing is seen).  Rows at or past lens[s] may hold anything, and what a row
 * holds that only the later of the new tokens see stays out of the earlier
 * ones.  max_rows (1 .. the table's rows, at most 2^30) bounds lens; a larger lens[s] is recorded as a device
 * error and cut to it, a negative one likewise to 0, and rows whose id names
 * no block are recorded and skipped.  Sums, the softmax's statistics and the
 * output before its one rounding are fp32; for the second product a bf16 cache
 * takes the probabilities as two bf16 parts, to 2^-16 of them (as one, to 2^-8,
 * where n_new * gqa_group is above 16), a 4-bit one those of the
 * lows too and probability times scale in
 * fp16 (in steps that follow the query's own largest such products; to two bf16
 * parts where a row's groups lie more than 2^8 apart), so that a row which a
 * query gives no weight, or does not see, may hold numbers of any size.  V's
 * scales and lows count in full from 2^-100 to 2^100.  A 4-bit cache takes a
 * query's elements relative to its row's largest (exact down to 2^-27 of it, the
 * others to 2^-35 of it; magnitudes below 2^115).  Logits (to base 2) may have any
 * size that fp32 holds: past 2^24 they are as coarse as fp32 is there.  The sums of
 * probabilities times V, before they are divided, are up to 2^8 sum |V| (fp32).
 * q, out: rkv_rows by sequence and token (bf16 for 4-bit caches). */
#define RKV_MAX_NEW_TOKENS 64
/* Bytes for the current device (the work is cut for its SMs) and any of the caches, of
 * these sizes or smaller ones (num_seqs, n_new, max_rows); 0: invalid sizes. */
size_t rkv_attention_workspace_size(const rkv_paged_desc* desc, int n_new, int max_rows);
int rkv_paged_attention(const rkv_paged_desc* desc, int n_new, const rkv_rows* q,
                        const void* K_pool, const void* V_pool, const int32_t* block_table,
                        const int32_t* lens, int max_rows, float scale, const rkv_rows* out,
                        float* lse, void* workspace, size_t workspace_bytes, void* stream);
int rkv_q4_attention(const rkv_paged_desc* desc, int n_new, const rkv_rows* q,
                     const rkv_q4_cache* cache, const int32_t* block_table,
                     const int32_t* lens, int max_rows, float scale, const rkv_rows* out,
                     float* lse, void* workspace, size_t workspace_bytes, void* stream);
/* The same over an 8-bit cache (q and out bf16).  Codes enter the products as
 * bf16 numbers, exactly; K's scale meets the logit and V's the probability in
 * fp32, and the probability times the scale goes on as a bf16 cache's
 * probabilities do (two bf16 parts, one where n_new * gqa_group is above 16).
 * What a hidden row holds, codes or scale, reaches no query.  Rows of V count in full where
 * their largest magnitude is 2^-100 or more, queries below 2^112 (q . code stays finite). */
int rkv_q8_attention(const rkv_paged_desc* desc, int n_new, const rkv_rows* q,
                     const rkv_q8_cache* cache, const int32_t* block_table,
                     const int32_t* lens, int max_rows, float scale, const rkv_rows* out,
                     float* lse, void* workspace, size_t workspace_bytes, void* stream);

/* Attention of a batch whose sequences share long prefixes (samples of one prompt,
 * requests over one document): rows of the pools that are held once, named by a
 * table of their own, and read once for all of their sequences.  rkv_paged_compress
 * wants a sequence's blocks for itself; a prefix is not compacted, so its blocks
 * stay as they are while the sequences' own rows, in block_table and lens, are
 * appended to and compressed as ever.
 *   table     [num_prefixes, max_blocks] int32 block ids
 *   lens      [num_prefixes] int32 rows of each prefix, 0 .. max_rows
 *   cu_seqs   [num_prefixes + 1] int32, ascending from 0: sequences cu_seqs[p] ..
 *             cu_seqs[p + 1] - 1 share prefix p, those from cu_seqs[num_prefixes]
 *             on have none.  NULL: every prefix has num_seqs / num_prefixes
 *             (a whole number) sequences, in order.
 * All on the device; num_prefixes 0 leaves the own rows. */
typedef struct {
    const int32_t* table;
    const int32_t* lens;
    const int32_t* cu_seqs;
    int32_t num_prefixes;
    int32_t max_blocks; /* row stride of table (>= 1) */
    int32_t max_rows;   /* bounds lens (>= 1), at most 2^30 and the table's rows */
} rkv_prefixes;

/* Bytes for the current device, of these sizes or smaller ones (num_seqs, n_new, the
 * max_rows of both, num_prefixes), over blocks of any size; 0: invalid sizes. */
size_t rkv_prefix_attention_workspace_size(const rkv_paged_desc* desc, int n_new, int max_rows,
                                           const rkv_prefixes* prefixes);

/* rkv_paged_attention where token t of sequence s sees all rows of its prefix and
 * then its own rows j <= lens[s] - n_new + t (max_rows bounds lens; a sequence may
 * have no rows of its own): one softmax over both; lse likewise.  What is said there
 * of sums, sizes of logits, hidden rows, bad ids and lengths holds here for both
 * tables; a cu_seqs that descends or passes the last sequence is recorded and cut.
 * The probabilities of a prefix's rows meet a bf16 V as one bf16 part (2^-8 of
 * them).  Prefixes are read by tensor-core kernels where the pools are bf16 with
 * blocks of 8 rows or more, else on the CUDA cores.  The work is cut for num_seqs /
 * num_prefixes sequences a prefix: sequences without one are better off in a call of their
 * own where they are many (results are the same). */
int rkv_prefix_attention(const rkv_paged_desc* desc, int n_new, const rkv_rows* q,
                         const void* K_pool, const void* V_pool, const rkv_prefixes* prefixes,
                         const int32_t* block_table, const int32_t* lens, int max_rows, float scale,
                         const rkv_rows* out, float* lse, void* workspace, size_t workspace_bytes,
                         void* stream);

/* The selection alone: for scores Z [P, n] (fp32), out_idx [P, budget] as
 * rkv_compress would produce it (top budget-n_obs of the candidates
 * 0..n-n_obs-1 by Z, ties to the larger index, then the n_obs observation
 * tokens, ascending).  Requires n_obs <= budget < n <= RKV_MAX_TOKENS. */
int rkv_select(int64_t num_problems, int n, const float* Z, int n_obs, int budget,
               int32_t* out_idx, void* stream);

/* The copy alone: dst[p, r, :] = src[p, idx[p, r], :] for r < budget where
 * idx >= 0; src laid out as K in `desc`, dst as out_K (out_capacity rows per
 * problem); idx rows strictly ascending.  dst may equal src (in place, with
 * out_capacity 0 or n_capacity) but must not overlap it otherwise. */
int rkv_gather(const rkv_desc* desc, const void* src, const int32_t* idx, int budget,
               void* dst, void* stream);

/* Clears the device error word at the start of `workspace` (enqueued on
 * `stream`).  Call once on a fresh workspace before its first use, unless the
 * workspace was allocated zero-filled. */
int rkv_workspace_init(void* workspace, void* stream);

/* Synchronises `stream`, returns the first error a kernel recorded in
 * `workspace` since the last call (RKV_OK if none) and clears it. */
int rkv_get_device_status(void* workspace, void* stream);

/* rkv_compress without a caller workspace.  The pages have no counterpart:
 * this is a deployment convenience for callers that may not allocate device
 * memory while they run (an engine plugin or custom op whose host framework
 * owns all device memory, a process whose memory is reserved up front for the
 * KV cache).  Same arguments, results and stream semantics as rkv_compress;
 * the scratch is a static array of RKV_NOALLOC_SCRATCH_BYTES inside the
 * library, held by every GPU that loads it until exit.  Requests whose
 * rkv_workspace_size() exceeds it return RKV_ERR_TOO_LARGE before anything is
 * enqueued (16 MiB holds the scratch of about 700 thousand token slots, e.g.
 * one Llama-8B layer at batch 64 with N = 1152, or 195 problems of 4096).
 * Never allocates or frees device memory.
 * Every call looks up the array's device address on the current device
 * (cudaGetSymbolAddress, a host-side lookup).  The first lookup on a device
 * may load the library's device code there; make the first call on each
 * device before any stream capture: if the lookup fails (for instance because
 * a capture forbids loading code), the call returns RKV_ERR_CUDA and enqueues
 * nothing.  All calls share the array.  Once a call's arguments pass their
 * checks it clears the array's device error word (enqueued on `stream` before
 * its kernels); a rejected call enqueues nothing.  Calls that may overlap on
 * the GPU race on the array and must be serialised by the caller. */
#define RKV_NOALLOC_SCRATCH_BYTES (16u << 20)
int rkv_compress_noalloc(const rkv_desc* desc, const void* K, const void* V, const void* Q_obs,
                         int n_cached, int budget, int n_obs, float lambda, int beta, float tau,
                         void* out_K, void* out_V, int32_t* out_idx, void* stream);

/* rkv_get_device_status for rkv_compress_noalloc's static scratch on the
 * current device: synchronises `stream`, returns RKV_ERR_DEVICE if a kernel
 * recorded an error there since the last read (and clears it), RKV_OK
 * otherwise. */
int rkv_noalloc_device_status(void* stream);

/* rkv_selftest_wait_timeout on the static scratch of the current device (the
 * error word that rkv_noalloc_device_status reads). */
int rkv_noalloc_selftest_wait_timeout(void* stream);

/* Self-test of the failure path: enqueues one bounded wait that nothing
 * completes (the primitive every wait of the kernels uses).  After its limit
 * (about a second) it records a timeout in `workspace`, which
 * rkv_get_device_status() then reports as RKV_ERR_DEVICE; the context stays
 * usable.  Nothing hangs and nothing traps. */
int rkv_selftest_wait_timeout(void* workspace, void* stream);

/* Human-readable name of an RKV_* code. */
const char* rkv_strerror(int code);

/* Step schedule of rkv_compress / rkv_compress_ex / rkv_paged_compress
 * (process-wide).  A call whose keys are bf16 rows with N <= 2048 (contiguous,
 * or a paged pool of blocks of 128 rows or more, grouped by whole sequences),
 * that passes no variant, whose selection fits the fused compaction and whose
 * stream is not being captured into a graph can run on two SM partitions of
 * the device (driver green contexts, created at the first such call and
 * kept): the problems are cut into `groups` equal groups; importance and Gram
 * of each group run on the tensor partition (about tensor_sms SMs), and each
 * group's selection and row copy run on the other SMs while the tensor
 * partition scores the next group (the last group's on the whole device).
 * It needs at least
 * 2 * groups * tensor_sms problems.  Results are bit for bit those of one
 * launch per stage over the whole device.
 *   mode RKV_SCHEDULE_ONE_LAUNCH: always one launch per stage;
 *   mode RKV_SCHEDULE_AUTO (default): grouped where a cost model of the
 *     kernels' measured per-problem times predicts a gain (the Llama-8B-shaped
 *     step: yes; a few thousand problems or long rows compacted in place: no;
 *     paged pools: never);
 *   mode RKV_SCHEDULE_GROUPED: grouped wherever the call is eligible.
 * Defaults: groups = 8, tensor_sms = 0 (112 of every 152 SMs).  Calls that
 * take the grouped schedule share the partitions' streams and run one after
 * another whatever stream they were given; where the driver offers no
 * partitions the one-launch schedule runs, and so it does under a profiler or
 * other tool injected into the process (CUDA_INJECTION64_PATH, or the
 * variables Nsight Compute sets: ncu cannot profile launches in a green
 * context).
 * rkv_compress_noalloc always takes the one-launch schedule.  Returns
 * RKV_ERR_INVALID_ARG for an unknown mode, groups outside 2..32 or
 * 0 < tensor_sms < 8. */
enum {
    RKV_SCHEDULE_ONE_LAUNCH = 0,
    RKV_SCHEDULE_AUTO = 1,
    RKV_SCHEDULE_GROUPED = 2
};
int rkv_set_overlap(int mode, int groups, int tensor_sms);

/* Launch trace (not thread-safe).  While enabled, each launch of the library
 * is preceded and followed, on its own stream, by a one-thread kernel that
 * stores the device's global nanosecond timer, so launches on the two SM
 * partitions of the grouped step (rkv_set_overlap) are placed on one clock.
 * Enabling clears the trace; up to 8192 launches are kept.  rkv_trace_read
 * synchronises the device, writes per launch (in enqueue order, up to
 * max_records) the kernel (index of rkv_kernel_name), the lane (0: the
 * caller's stream, 1: the tensor partition, 2: the other partition) and the
 * start and end stamps in ns, clears the trace and returns the number of
 * records written (a negative RKV_* code on a CUDA error).  Any output
 * pointer may be null. */
int rkv_trace_enable(int on);
int rkv_trace_read(int* kernel, int* lane, uint64_t* start_ns, uint64_t* end_ns,
                   int max_records);

/* Per-kernel timing (not thread-safe).  While enabled, each launch of the
 * library is bracketed by CUDA events on its stream.  rkv_timing_read waits for
 * the events, writes per-kernel totals (milliseconds) and launch counts for up
 * to `max_kernels` kernels in the order of rkv_kernel_name(), returns the
 * number of kernel kinds, and with reset != 0 clears the totals. */
int rkv_timing_enable(int on);
int rkv_timing_read(double* total_ms, int64_t* launches, int max_kernels, int reset);
const char* rkv_kernel_name(int kernel);

#ifdef __cplusplus
}
#endif
#endif /* RKV_H */
