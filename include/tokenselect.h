/*
 * tokenselect.h - C ABI of the token-level KV selection decode path (sm_103a).
 *
 * The method: TokenSelect ("TokenSelect: Efficient Long-Context Inference and
 * Length Extrapolation for LLMs via Dynamic Token-Level KV Cache Selection").
 * One decode step of one layer is, per sequence of the batch:
 *
 *   1. Selection Cache check: cos(Q, C_Q) >= theta reuses the cached indices
 *      (deep notes, Appendix Algorithm 1; review, section 3.2).
 *   2. Paged dot product: l[h][i] = alpha <q_h, K_{h/G}[i]> over all N cached
 *      tokens of the paged cache (deep notes, Appendix Algorithm 2).
 *   3. Head soft vote: v[i] = sum_h softmax_h(l[h])[i] (deep notes, "Head soft
 *      vote", equation T_head-soft-vote).
 *   4. Selection: TopK(v) over the candidates [s, N-w), or the shortest
 *      (vote desc, index asc) prefix with mass >= p*H, united with the sinks
 *      [0, s) and the local window [N-w, N) (review, section 4.2, "2K+512").
 *   5. Sparse attention over the selected tokens (deep notes, "Formalising
 *      selective sparse attention", equation for O-hat).
 *
 * Conventions for every call below:
 *  - Tensor arguments are DEVICE pointers owned by the caller. The library
 *    never frees them. A context owns its own device scratch; a cache handle
 *    owns C_Q and C_T. Both are freed by their destroy call.
 *  - Layouts are dense row-major. KV pools are [num_pages][H_kv][P][d] (fp32
 *    or bf16, 16-byte aligned base); token i of sequence b lives in page
 *    page_table[b * max_pages_per_seq + i / P] at slot i % P (page tables are
 *    int32 [B][max_pages_per_seq], entries past a sequence unused). Queries are
 *    fp32 [B][H][d]. Query head h reads KV head h / (H / H_kv).
 *  - 4-bit pools (TS_KV_Q4) are bytes [num_pages][H_kv][16 (d/2 + d/32)]. The
 *    block of a (page, KV head) holds codes [d/64][16 tokens][32 bytes] (byte j:
 *    element 2j of the 64 in the low half, 2j + 1 in the high half), then scales
 *    bf16 [d/64][16 tokens]. A code u stands for (u - 8) * scale. A group of 64
 *    elements is written with scale = bf16(max|x| / 7) and u = 8 + round(x /
 *    scale), ties to even: at most half a scale from x (and from 7 scales where
 *    the scale was rounded down). A group with a NaN or an infinity reads as NaN.
 *  - Work is enqueued on `stream` (a cudaStream_t; NULL is the legacy default
 *    stream) and returns before it runs. Argument and shape errors are
 *    reported synchronously by the return value, before anything is enqueued.
 *    Errors found on the device (a page id outside the pool, an output that
 *    does not fit, a wait that ran out) are recorded in the context's status
 *    word and read back with ts_get_status. Nothing aborts or traps.
 *  - A context is bound to the device current at ts_create (the packed calls,
 *    those for drafted tokens, ts_attend and every call over a 4-bit pool return TS_ERR_INVALID_ARG where
 *    another one is current) and is not thread safe: calls on one context must
 *    be serialised by the caller, and calls that share a context's scratch must
 *    go to one stream (or be ordered).
 */
#ifndef TOKENSELECT_H
#define TOKENSELECT_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct ts_ctx ts_ctx;     /* opaque; library-owned */
typedef struct ts_cache ts_cache; /* opaque; library-owned */
typedef struct ts_rope ts_rope;   /* opaque; library-owned, host memory only */

typedef enum {
  TS_OK = 0,
  TS_ERR_INVALID_ARG = 1,      /* null pointer, bad enum, negative size        */
  TS_ERR_SHAPE = 2,            /* sizes beyond what the context was created for */
  TS_ERR_UNSUPPORTED = 3,      /* head geometry without a compiled kernel       */
  TS_ERR_CUDA = 4,             /* a CUDA runtime call failed                    */
  TS_ERR_PAGE_OOB = 5,         /* device: page-table entry outside the pool     */
  TS_ERR_CAPACITY = 6,         /* device: selection larger than its buffer      */
  TS_ERR_TIMEOUT = 7,          /* device: a bounded wait ran out                */
  TS_ERR_COOP_UNAVAILABLE = 8, /* a cooperative launch was refused              */
  TS_ERR_SEQ_LEN = 9,          /* device: seq_lens[b] < 0 or above the maximum  */
  TS_ERR_SCRATCH_LIMIT = 10    /* beyond the fixed scratch of the no-alloc call */
} ts_status;

enum { TS_KV_F32 = 0, TS_KV_BF16 = 1, TS_KV_Q4 = 2 };
enum { TS_SELECT_TOPK = 0, TS_SELECT_TOPP = 1 };
/* Selection function whose per-token score the top-k ranks (TokenSelect deep
 * notes, "Evolution of the selection function"; TokenSelect review, section
 * 3.1 and the ablation of section 4.4 / table 4):
 *  HEAD_SOFT_VOTE  v_i = sum_h softmax(scale q_h.K^T)_i  (the method);
 *  LOGIT_SUM       s_i = sum_h scale q_h.k_{g(h),i}: plain TopK(Q.K^T) of the
 *                  concatenated heads, dominated by high-norm heads (signed);
 *  HEAD_HARD_VOTE  c_i = number of query heads whose own top-k over the
 *                  candidates [s, N-w) (ties to the lower index) holds i.
 * The two ablations serve top-k only and run on the multi-kernel path. */
enum { TS_SCORE_HEAD_SOFT_VOTE = 0, TS_SCORE_LOGIT_SUM = 1, TS_SCORE_HEAD_HARD_VOTE = 2 };

/* Shape of the model's attention and of the caller's pools, fixed per context. */
typedef struct {
  int n_q_heads;          /* H                                                  */
  int n_kv_heads;         /* H_kv, divides H                                    */
  int head_dim;           /* d (64 or 128)                                      */
  int page_size;          /* P tokens per page: 16, or 1 for a token-granular   */
                          /* pool (one token per page; separate kernels only)   */
  int kv_dtype;           /* TS_KV_F32, TS_KV_BF16 or TS_KV_Q4 (16-token pages, */
                          /* d 64 or 128, at most 16 query heads per KV head)   */
  int max_batch;          /* largest B of any call                              */
  int max_pages_per_seq;  /* page-table row stride; max tokens = this * P       */
  int64_t num_pages;      /* pool size in pages; larger page ids are errors     */
} ts_config;

/* Selection parameters (review, section 4.2: k = 2048, 4 sinks, 512 local;
 * deep notes, Algorithm 1: theta = 0.9). */
typedef struct {
  int mode;               /* TS_SELECT_TOPK or TS_SELECT_TOPP                   */
  int k;                  /* top-k budget over the candidates                   */
  int n_sink;             /* s: tokens [0, s) always kept                       */
  int n_local;            /* w: tokens [N-w, N) always kept                     */
  float top_p;            /* mass fraction for TOPP; >= 1 keeps every token     */
  float theta;            /* cache threshold; > 1 never hits                    */
  float softmax_scale;    /* alpha; 0 means 1/sqrt(d)                           */
  int score_fn;           /* TS_SCORE_*; 0 (the head soft vote) by default      */
} ts_select_params;

/* Context: validates and records cfg, allocates the device scratch for
 * max_batch sequences of max_pages_per_seq * page_size tokens on the current
 * device (that of ts_tree_attend is allocated by its first call). Returns TS_ERR_UNSUPPORTED for a head geometry with no kernel. */
ts_status ts_create(ts_ctx** out, const ts_config* cfg);
ts_status ts_destroy(ts_ctx* ctx);

/* Bytes of one page of a K pool (or a V pool) of this shape, all KV heads; 0
 * for a NULL cfg or an unknown kv_dtype. A pool has num_pages times as many. */
int64_t ts_page_bytes(const ts_config* cfg);

/* Selection Cache for n_layers layers of max_batch sequences: per (sequence,
 * layer) a first-query flag, C_Q (fp32 H*d) and C_T (int32, `capacity`
 * entries). Starts empty (every first query misses). */
ts_status ts_cache_create(ts_ctx* ctx, ts_cache** out, int n_layers, int capacity);
ts_status ts_cache_destroy(ts_cache* cache);
/* Marks every (sequence, layer) as empty again; enqueued on `stream`. */
ts_status ts_cache_reset(ts_cache* cache, void* stream);

/* Algorithm 1's test for one layer: hit[b] = 1 iff the entry of (b, layer)
 * is filled, and cos(q_b, C_Q) >= theta over the H*d query (fp32).
 * q [B][H][d]; hit uint8 [B]; cos_out fp32 [B] or NULL (NaN when empty). */
ts_status ts_cache_check(ts_ctx* ctx, ts_cache* cache, int layer, const float* q, int B,
                         float theta, uint8_t* hit, float* cos_out, void* stream);

/* Paged dot product + fused per-head softmax normaliser + head soft vote.
 * For each b with skip == NULL or skip[b] == 0:
 *   vote[b * vote_stride + i] = sum_h exp(l[h][i] - L_h),  i < seq_lens[b],
 * with l = scale * <q_h, K_{h/G}[i]> and L_h = log sum_i exp(l[h][i]).
 * The H x N logits are context scratch and are not returned. scale 0 means
 * 1/sqrt(d). seq_lens int32 [B] on the device, each in [0, max_pages_per_seq
 * * page_size]; vote_stride >= max_pages_per_seq * page_size. Entries past
 * seq_lens[b] and skipped rows are left untouched. */
ts_status ts_score(ts_ctx* ctx, const float* q, const void* k_pool, const int32_t* page_table,
                   const int32_t* seq_lens, int B, const uint8_t* skip, float scale,
                   float* vote, int64_t vote_stride, void* stream);

/* The per-token score of one selection function (params->score_fn, TS_SCORE_*)
 * for the top-k of ts_select: HEAD_SOFT_VOTE computes exactly what ts_score
 * does; LOGIT_SUM writes the signed sums of the per-head logits (rank them by
 * passing the same params to ts_select); HEAD_HARD_VOTE runs one top-k per
 * query head over the candidates [s, N-w) of params (k, n_sink, n_local; ties
 * to the lower index) and writes the vote counts as floats (exact small
 * integers, 0 outside the candidates). Every entry i < seq_lens[b] of a row
 * that is not skipped is written; layout and scale as in ts_score. */
ts_status ts_score_fn(ts_ctx* ctx, const ts_select_params* params, const float* q, const void* k_pool,
                      const int32_t* page_table, const int32_t* seq_lens, int B, const uint8_t* skip,
                      float* vote, int64_t vote_stride, void* stream);

/* Selection (top-k or top-p) united with sinks and window, ascending.
 * For each b: if hit != NULL and hit[b] != 0, the index set is rebuilt from
 * the cache entry (cached part within [s, N-w), plus the current sinks and
 * window); otherwise it is selected from vote and, if cache != NULL, the
 * entry of (b, layer) takes the selected part and q_b (Algorithm 1). Ties in
 * the vote go to the lower index. idx int32 [B][idx_stride] receives the
 * count[b] indices; a count above idx_stride (or a selected part above the
 * cache capacity) records TS_ERR_CAPACITY and writes nothing past the end.
 * q may be NULL when cache is NULL. With params->score_fn == LOGIT_SUM the
 * scores are ranked as signed values; top-p needs the head soft vote (its
 * mass is the vote's), else TS_ERR_INVALID_ARG. */
ts_status ts_select(ts_ctx* ctx, ts_cache* cache, int layer, const float* q, const float* vote,
                    int64_t vote_stride, const int32_t* seq_lens, int B, const uint8_t* hit,
                    const ts_select_params* params, int32_t* idx, int64_t idx_stride,
                    int32_t* count, void* stream);

/* Sparse attention: out[b][h] = softmax_i(scale q_h.K_i) V_i over the count[b]
 * indices idx[b * idx_stride + j] (split over the index list, merged by
 * log-sum-exp). out fp32 [B][H][d]; lse fp32 [B][H] or NULL. An empty index
 * list gives out = 0 and lse = -inf. */
ts_status ts_sparse_attend(ts_ctx* ctx, const float* q, const void* k_pool, const void* v_pool,
                           const int32_t* page_table, const int32_t* idx, int64_t idx_stride,
                           const int32_t* count, int B, float scale, float* out, float* lse,
                           void* stream);

/* Attention over the whole cache: ts_sparse_attend with every token i <
 * seq_lens[b] attended, without an index list. 4-bit pools (TS_KV_Q4) only,
 * else TS_ERR_UNSUPPORTED. A sequence of length 0 gives out = 0 and lse = -inf;
 * a length outside [0, max tokens] records TS_ERR_SEQ_LEN and is taken as 0;
 * the tokens of a page outside the pool are left out and TS_ERR_PAGE_OOB is
 * recorded. 64 elements of a value row that read as NaN make the same elements of
 * the outputs NaN, and no others. Repeated calls give the same bits. */
ts_status ts_attend(ts_ctx* ctx, const float* q, const void* k_pool, const void* v_pool, const int32_t* page_table,
                    const int32_t* seq_lens, int B, float scale, float* out, float* lse, void* stream);

/* Causal attention of whole prompts, packed one behind another: sequence b is
 * rows cu_rows[b] .. cu_rows[b + 1] - 1 of every tensor (cu_rows int32 [B + 1]
 * on the device, from 0, ascending, at most `total`; a length may be 0), and its
 * row i attends to rows 0 .. i of the same sequence:
 *   out[r][h] = softmax_j(scale <q[r][h], k[j][h/G]>) v[j][h/G],
 *   lse[r][h] = log sum_j exp(scale <q[r][h], k[j][h/G]>)   (lse NULL: not wanted).
 * q bf16 [total][H][d], k and v bf16 [total][H_kv][d], with q_stride, k_stride,
 * v_stride elements from row to row (dense inside a row), so that the three may
 * be column ranges of one projection: base pointers 16-byte aligned, strides
 * multiples of 8 and at least the row. out bf16 [total][H][d] with out_stride
 * likewise; lse fp32 [total][H]. Rows of out and lse from cu_rows[B] on are left
 * as they are. Scores, sums and outputs accumulate in fp32; the softmax weights
 * are rounded to bf16 for their product with v, the outputs once at the end (a
 * row's weights sum to 2^37 at most before they are divided, so values below 2^90
 * never pass fp32). No cache is read or written: the context gives the head
 * geometry (d 64 or 128, G <= 16, bf16 or 4-bit pools, else TS_ERR_UNSUPPORTED),
 * B <= max_batch, and a prompt may be longer than its max tokens. Boundaries that
 * are not as above record TS_ERR_SEQ_LEN: nothing is written for a sequence that
 * descends or ends beyond `total`. A row's result depends on no later row, on no other
 * sequence and on no row past the last one, whatever those hold (NaN and
 * infinities too). An infinite value that a row does see gives it an infinity, or
 * NaN where its weight is below fp32's range. Repeated calls give the same bits. */
ts_status ts_prompt_attend(ts_ctx* ctx, const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                           const void* v, int64_t v_stride, const int32_t* cu_rows, int B, int total, float scale,
                           void* out, int64_t out_stride, float* lse, void* stream);

/* Sparse attention for callers that cannot allocate device memory: the same
 * computation and the same kernel as ts_sparse_attend, but with no context.
 * The paper has no counterpart; this exists for callers that run where
 * cudaMalloc is unavailable or forbidden - inside a memory pool or arena they
 * do not own, under a framework allocator that must see every allocation, or
 * in a process that has to keep device memory fixed after start-up - and
 * so cannot create a context (ts_create allocates its scratch).
 * Its scratch (split partials, merge counters, a fallback status slot) is one
 * fixed static device array of 4 MiB + 16 KiB in the library, held by every
 * GPU that loads the library until the process exits. Limits: B <= 48,
 * n_kv_heads <= 64 (one merge counter per (sequence, KV head) in the head of
 * the array) and B * H_kv * G * (d + 2) <= 2^20 floats (one split per
 * (sequence, KV head) at that size); beyond them the call returns
 * TS_ERR_SCRATCH_LIMIT and enqueues nothing. A NaN scale returns
 * TS_ERR_INVALID_ARG, as in ts_sparse_attend, and 4-bit pools TS_ERR_UNSUPPORTED. It calls no cudaMalloc/cudaFree. The first call on a
 * device looks up the array's device address (cudaGetSymbolAddress) and the
 * SM count: make that first call before any stream capture on that device.
 * Every call clears the merge counters, then uses the shared array: calls
 * that overlap on the GPU (other streams, other threads) race on it and must
 * be serialised by the caller. Geometry: n_q_heads, n_kv_heads, head_dim,
 * kv_dtype as in ts_config; pools of num_pages pages; page_table int32
 * [B][max_pages_per_seq]. status: int32 on the device or NULL; receives the
 * first device error (0 otherwise is left unchanged). Other arguments as in
 * ts_sparse_attend. */
ts_status ts_sparse_attend_noalloc(int n_q_heads, int n_kv_heads, int head_dim, int kv_dtype,
                                   const float* q, const void* k_pool, const void* v_pool,
                                   int64_t num_pages, const int32_t* page_table,
                                   int max_pages_per_seq, const int32_t* idx, int64_t idx_stride,
                                   const int32_t* count, int B, float scale, float* out, float* lse,
                                   int32_t* status, void* stream);

/* One whole decode step of one layer, stream-ordered, no host synchronisation:
 * cache check (when cache != NULL and theta <= 1), score and vote for the
 * sequences that miss, selection (and cache update), sparse attention.
 * hit uint8 [B] (may be NULL) receives the cache decisions. vote receives the
 * votes of the missing sequences (may be NULL: context scratch is used).
 * Supported geometries run as one cooperative launch; repeated calls on the
 * same inputs give bit-identical results. params->score_fn other than the
 * head soft vote (the ablations) runs the multi-kernel path with that
 * selection function (the vote buffer then holds its scores); so does a
 * context with one-token pages or 4-bit pools. Environment switches, read once by
 * ts_create (comparisons and tests): TOKENSELECT_MULTI_KERNEL=1 keeps the
 * multi-kernel path; TOKENSELECT_NO_TC=1 scans on CUDA cores instead of tensor
 * cores; TOKENSELECT_SCAN_CLAIM=1 lets the CTAs claim scan pages from a shared
 * counter when at most two sequences are scanned (faster where SM bandwidth
 * differs, but no longer bit-identical from run to run);
 * TOKENSELECT_L2_BUDGET_MB sets the logit bytes one CUDA-core scan wave may
 * keep in L2; TOKENSELECT_TOPP_ATTEND=gather / range / range_tc fixes the top-p
 * attention (selected tokens shared out over the CTAs; each CTA's own scanned
 * range from the scan's logits, P.V on CUDA cores or on the tensor cores),
 * otherwise chosen per sequence by how dense the selection is; TS_DEBUG prints
 * launch diagnostics. */
ts_status ts_decode_step(ts_ctx* ctx, ts_cache* cache, int layer, const float* q,
                         const void* k_pool, const void* v_pool, const int32_t* page_table,
                         const int32_t* seq_lens, int B, const ts_select_params* params,
                         float* vote, int64_t vote_stride, int32_t* idx, int64_t idx_stride,
                         int32_t* count, float* out, float* lse, uint8_t* hit, void* stream);

/* Appends the current token's K and V rows to the paged pools before a
 * decode step (the harness step of reading R9: the current token is the last
 * cached position). For each b, k_new / v_new [B][H_kv][d] (device, kv_dtype
 * elements, 16-byte aligned) are written to pool[page][g][slot] of position
 * seq_lens[b] - 1, page = page_table[b][(seq_lens[b] - 1) / page_size]. A
 * length outside [1, max tokens] records TS_ERR_SEQ_LEN, a page outside the
 * pool TS_ERR_PAGE_OOB (nothing is written for that sequence). For a 4-bit pool
 * k_new / v_new are bf16 and the rows are quantised. */
ts_status ts_append_kv(ts_ctx* ctx, const void* k_new, const void* v_new, const int32_t* page_table,
                       const int32_t* seq_lens, int B, void* k_pool, void* v_pool, void* stream);

/* Appends the K and V rows of whole prompts (or of several tokens at once) to the
 * paged pools. Packed row r of sequence b (cu_rows[b] <= r < cu_rows[b + 1], as in
 * ts_prompt_attend) goes to position starts[b] + r - cu_rows[b] of that sequence
 * (starts int32 [B] on the device; NULL: 0). k / v [total][H_kv][d] in the pool's
 * element type (bf16 for a 4-bit pool, whose rows are quantised), k_stride and
 * v_stride elements from row to row, dense inside a row, rows 16-byte aligned. A
 * position outside [0, max tokens), or boundaries that are not ascending from 0 to at
 * most total, records TS_ERR_SEQ_LEN, a page outside the pool TS_ERR_PAGE_OOB; the
 * rows concerned (of a sequence that ends beyond total: all of its rows) are not
 * written. Rows from cu_rows[B] on are not written. Two rows
 * for one position leave one of them or, in a 4-bit pool, a mix of them. */
ts_status ts_append_prompt(ts_ctx* ctx, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                           const int32_t* cu_rows, const int32_t* starts, int B, int total,
                           const int32_t* page_table, void* k_pool, void* v_pool, void* stream);

/* Reads cached rows back as values: the inverse of ts_append_prompt, with the same
 * cu_rows, starts and errors. k_out / v_out fp32 [total][H_kv][d], dense, 16-byte
 * aligned, hold every pool type's values exactly; rows that are not read are left as
 * they are. */
ts_status ts_read_kv(ts_ctx* ctx, const int32_t* cu_rows, const int32_t* starts, int B, int total,
                     const int32_t* page_table, const void* k_pool, const void* v_pool, float* k_out,
                     float* v_out, void* stream);

/* Rotary positions. A head's first rot_dim elements are turned in pairs, (i, i + rot_dim/2) or, interleaved, (2i,
 * 2i + 1):  y1 = a (x1 cos t - x2 sin t), y2 = a (x2 cos t + x1 sin t), t = position * f_i; the others pass as they
 * are. f_i = base^(-2i/rot_dim) radians per position, then by `scaling` (with n = original, lengths in positions):
 *  PLAIN   f_i;
 *  LINEAR  f_i / factor;
 *  BASE    base * factor^(rot_dim/(rot_dim - 2)) in place of base;
 *  BANDS   t f_i + (1 - t) f_i / factor, t = (n f_i / 2pi - low) / (high - low) held to [0, 1]: pairs that turn more
 *          than `high` times within n positions keep their frequency, those below `low` turns are scaled;
 *  YARN    t f_i / factor + (1 - t) f_i, t = (i - i_high) / (i_low - i_high) held to [0, 1], where i_x is the pair
 *          that turns x times within n positions, i_high rounded down and at least 0, i_low rounded up and at most
 *          rot_dim - 1 (their difference at least 0.001); a = 0.1 ln(factor) + 1 for a factor above 1;
 *  GIVEN   freqs[rot_dim/2] (host memory, read by ts_rope_create).
 * a = attention where that is not 0, else 1 unless the rule names one. Angles, modulo a turn, are exact to 2^-32 of
 * it plus what `position` makes of the last bit of f_i / 2pi in fp64, for every int32 position, negative ones too; then they
 * are rounded to fp32, by up to 2^-26 of a turn (9.4e-8 radians, for those near half a turn). */
enum { TS_ROPE_PLAIN = 0, TS_ROPE_LINEAR = 1, TS_ROPE_BASE = 2, TS_ROPE_BANDS = 3, TS_ROPE_YARN = 4, TS_ROPE_GIVEN = 5 };
typedef struct {
  int rot_dim;            /* even, 2 to 128, at most the context's head_dim      */
  int interleaved;        /* 0: pairs (i, i + rot_dim/2); 1: pairs (2i, 2i + 1)  */
  int scaling;            /* TS_ROPE_*                                          */
  double base;            /* > 0                                                */
  double factor;          /* > 0; not read for PLAIN and GIVEN                  */
  int original;           /* context that the model was made for: BANDS, YARN   */
  double low, high;       /* turns within it, 0 < low < high: BANDS, YARN       */
  double attention;       /* factor of what is turned; 0: by the rule           */
  const double* freqs;    /* GIVEN, else NULL                                   */
} ts_rope_config;
/* Works out the frequencies on the host (no device memory: a handle serves every context and device). */
ts_status ts_rope_create(ts_rope** out, const ts_rope_config* cfg);
ts_status ts_rope_destroy(ts_rope* rope);
/* The handle's frequencies (rot_dim/2 of them, radians per position) and its factor a. */
ts_status ts_rope_read(const ts_rope* rope, double* freqs, double* attention);

/* Turns rows of heads by their positions: x and out [total][heads][d] (d the context's head_dim), dense inside a row,
 * x_stride and out_stride elements from row to row, each of type TS_KV_F32 or TS_KV_BF16; positions int32 [total] on
 * the device. Rows 16-byte aligned. Computed in fp32 and rounded once. out may be x where type and stride are the
 * same (another combination at one address is refused); otherwise they must not share memory. With the positions negated the call is its own transpose: the gradient
 * of x from that of out (and, where a is 1, the inverse). The context gives d and the device. */
ts_status ts_rotate(ts_ctx* ctx, const ts_rope* rope, const void* x, int64_t x_stride, int dtype, int heads,
                    const int32_t* positions, int total, void* out, int64_t out_stride, int out_dtype, void* stream);

/* ts_append_prompt with K rows turned on their way, exactly as ts_rotate (rounded to the rows' type, then quantised
 * for a 4-bit pool) and then ts_append_prompt would write them. Row r is turned by positions[r], which need not be
 * its place in the cache (drafts of one depth share a position). q and q_out NULL, or: the queries of the same rows,
 * q [total][H][d] of the rows' type with q_stride, are turned too, into q_out [total][H][d] of type q_out_dtype
 * (TS_KV_F32 for ts_decode_step and its kin, TS_KV_BF16 for ts_tree_attend) with q_out_stride; q_out may be q as in
 * ts_rotate. All `total` rows of q are turned, whether their K and V rows have a place or not. */
ts_status ts_append_rotated(ts_ctx* ctx, const ts_rope* rope, const void* k, int64_t k_stride, const void* v,
                            int64_t v_stride, const int32_t* positions, const int32_t* cu_rows, const int32_t* starts,
                            int B, int total, const int32_t* page_table, void* k_pool, void* v_pool, const void* q,
                            int64_t q_stride, void* q_out, int64_t q_out_stride, int q_out_dtype, void* stream);

/* Attention of drafted tokens over the whole cache. Packed rows cu_rows[b] .. cu_rows[b + 1] - 1 (cu_rows as in
 * ts_prompt_attend) are the queries of the last T_b = cu_rows[b + 1] - cu_rows[b] cached tokens of sequence b, which
 * are appended already: seq_lens[b] counts them. Row i of a sequence sees all tokens before seq_lens[b] - T_b, and of
 * the T_b drafts those j whose bit is set in its mask: mask int32 [total][mask_words] on the device, bit j % 32 of
 * word j / 32 (a tree: a row's own bit and its ancestors'; any set of bits is served, the row's own not implied).
 * mask NULL: the drafts j <= i, a chain. q bf16 [total][H][d] with q_stride, out bf16 [total][H][d] with out_stride,
 * lse fp32 [total][H] or NULL, alignment as in ts_prompt_attend. A row that sees nothing gives out = 0 and
 * lse = -inf. T_b may be 0; T_b above 1024, above 32 mask_words or above seq_lens[b], a length above the maximum, or
 * boundaries that are not ascending record TS_ERR_SEQ_LEN, and nothing is written for that sequence; total is at most
 * 2^24. The tokens of a
 * page outside the pool are left out and TS_ERR_PAGE_OOB is recorded. bf16 pools with d 64 or 128 and at most 16
 * query heads per KV head, else TS_ERR_UNSUPPORTED. Scores, sums and outputs accumulate in fp32; softmax weights are
 * rounded to bf16 for their product with v, outputs once at the end. A row's result depends on no draft that it does
 * not see and on nothing behind its sequence, whatever those hold (NaN and infinities too). A NaN score that a row sees makes
 * its outputs and lse NaN, a value that it sees and that is not finite makes that element not finite, however little it
 * weighs; rows of out and lse from
 * cu_rows[B] on are left as they are. Repeated calls give the same bits. A context's first call allocates its scratch
 * (512 (d + 2) fp32 for each SM: 40 MB at d 128; TS_ERR_CUDA, with nothing enqueued, where there is no room), also
 * one with total 0 and one whose stream is being captured; later calls allocate nothing. */
ts_status ts_tree_attend(ts_ctx* ctx, const void* q, int64_t q_stride, const void* k_pool, const void* v_pool,
                         const int32_t* page_table, const int32_t* seq_lens, const int32_t* cu_rows, const int32_t* mask,
                         int mask_words, int B, int total, float scale, void* out, int64_t out_stride, float* lse,
                         void* stream);

/* Which drafted tokens the target keeps, and the token behind them. Node 0 of a sequence's rows is the root, the last
 * token that is certain (its entries of tokens, parents and u are not read); node i > 0 holds the drafted token
 * tokens[r] behind node parents[r] < i (numbers within the sequence). target fp32 [total][vocab], target_stride
 * elements from row to row: the target's probabilities behind each node; draft likewise: those that the node's
 * children were drawn from, or NULL for drafts without probabilities. u fp32 [total] and u_next fp32 [B]: numbers
 * from [0, 1). From the root on, the children of the current node are tried in ascending order:
 *   with p and q the node's rows, c = 0, Z = 1, W = 1:  child x is taken iff u q(x) Z < max(p(x) - c q(x), 0) W;
 *   otherwise c += Z / W (where W > 0), Z = sum_i max(p(i) - c q(i), 0), and W -= q(x) if `distinct`
 * (distinct != 0: siblings were drawn without replacement, each from what its elder siblings left of q; 0: each
 * from q). draft NULL: x is taken iff u Z < p(x), otherwise Z -= p(x) and p(x) = 0. A child that is taken becomes the
 * current node; with none left next_token[b] is drawn from the residual r = max(p - c q, 0): the smallest i with
 * sum_{j <= i} r(j) > u_next[b] sum r (the last i with r(i) > 0 where rounding leaves none), from p where r is zero
 * throughout, -1 where p is too. Entries that are NaN or negative
 * count as 0. Sums are off by less than 2^-32 of them and 2^-45 of the sums of p and c q.
 * Tokens so drawn are distributed as the target's, where the rows of target and draft add up to 1: Z and W start at 1, not
 * at the rows' sums, and what a row misses of 1 (an fp32 softmax: about 1e-6) is carried along undivided. With
 * `distinct` it is off W, the mass that the elder siblings leave of q, so it shows where they leave little (a tenth of
 * W = 1e-5): a row whose first tokens hold nearly all of its mass wants few children, or rows that add up better.
 * path int32 [B][path_stride] receives the taken nodes in order, node 0 first, then -1; count int32 [B] how many.
 * More than path_stride record TS_ERR_CAPACITY (the first ones are written, count is the whole number). At most 1024
 * nodes per sequence; more, or boundaries that are not ascending, record TS_ERR_SEQ_LEN, count 0 and -1 (so does a
 * sequence without rows, without an error). A token outside [0, vocab) or a parent outside [0, i) records
 * TS_ERR_INVALID_ARG, and that node is passed over. vocab <= 2^20. The outputs must not share memory with the
 * inputs. The context gives max_batch, the device and the status word. */
ts_status ts_verify_tree(ts_ctx* ctx, const int32_t* tokens, const int32_t* parents, const int32_t* cu_rows, int B,
                         int total, int vocab, const float* target, int64_t target_stride, const float* draft,
                         int64_t draft_stride, const float* u, const float* u_next, int distinct, int32_t* path,
                         int64_t path_stride, int32_t* count, int32_t* next_token, void* stream);

/* Keeps the K and V rows of a path of drafts: of the last T_b = cu_rows[b + 1] - cu_rows[b] cached tokens (seq_lens[b]
 * counts them), row path[b][j] moves to row j for j < count[b], so that the path follows the certain tokens without a
 * gap. path and count as ts_verify_tree writes them: ascending within [0, T_b), count[b] in [0, min(T_b, path_stride)].
 * new_lens int32 [B] or NULL receives seq_lens[b] - T_b + count[b]; it must not share memory with the other
 * arrays. Every
 * pool type, values move as they are. n_layers pools each, layer_bytes from one to the next (a multiple of 16, at
 * least a pool; not read for one). A path that is not as above records TS_ERR_INVALID_ARG, a count above path_stride
 * TS_ERR_CAPACITY, boundaries or lengths that are not as in ts_tree_attend TS_ERR_SEQ_LEN: nothing moves for that
 * sequence and its length stays. A row with a page outside the pool records TS_ERR_PAGE_OOB and does not move. */
ts_status ts_keep_rows(ts_ctx* ctx, const int32_t* path, int64_t path_stride, const int32_t* count, const int32_t* cu_rows,
                       const int32_t* seq_lens, int B, int total, const int32_t* page_table, void* k_pool, void* v_pool,
                       int n_layers, int64_t layer_bytes, int32_t* new_lens, void* stream);

/* Block-level selection, the granularity the method argues against
 * (TokenSelect review, figure 2(b): InfLLM-style methods keep or drop whole
 * blocks; granularity 1 is token-level selection). From the votes of each
 * sequence (non-negative, e.g. from ts_score): blocks of `block` consecutive
 * tokens (the last one ragged) are scored by their largest vote, the
 * budget / block best blocks are taken (ties to the lower block) and every
 * token of them is written to idx [B][idx_stride] ascending, count [B]; a
 * list longer than idx_stride records TS_ERR_CAPACITY. No sinks, window or
 * cache: it serves the recall comparison of the two granularities. */
ts_status ts_select_blocks(ts_ctx* ctx, const float* vote, int64_t vote_stride, const int32_t* seq_lens, int B,
                           int block, int budget, int32_t* idx, int64_t idx_stride, int32_t* count,
                           void* stream);

/* Chunk-wise prefill selection (TokenSelect deep notes, "Optimising the
 * selection frequency of the prefill stage"; review, section 3.2): the c
 * queries of a prefill chunk, q fp32 [B][c][H][d] (16-byte aligned), are
 * averaged into one query per sequence, (1/c) sum_i q[b][i]; that mean query
 * is scored and selects once (head soft vote, top-k over [s, N-w) united
 * with sinks and window, ties to the lower index; no Selection Cache in
 * prefill), writing vote (or context scratch when NULL), idx [B][idx_stride]
 * ascending and count [B] as ts_decode_step does. The chunk's own tokens must
 * already be cached as the last c of seq_lens[b] tokens: query i attends to
 * the selected tokens at positions <= seq_lens[b] - c + i (causal), giving
 * out fp32 [B][c][H][d] and lse fp32 [B][c][H] (or NULL). The attention runs
 * on the tensor cores for bf16 pools with d = 64 or 128 (else
 * TS_ERR_UNSUPPORTED). params must be top-k with the head soft vote. */
ts_status ts_prefill_chunk(ts_ctx* ctx, const float* q, int c, const void* k_pool, const void* v_pool,
                           const int32_t* page_table, const int32_t* seq_lens, int B,
                           const ts_select_params* params, float* vote, int64_t vote_stride,
                           int32_t* idx, int64_t idx_stride, int32_t* count, float* out, float* lse,
                           void* stream);

/* Failure detection (no counterpart in the pages; the library's own safety
 * net). Every wait of the persistent decode-step kernel - its grid barriers
 * and its copy, tensor-core and accumulator waits - gives up after `ns`
 * nanoseconds (default 1 s): the kernel then records TS_ERR_TIMEOUT, raises an
 * abort word that the other CTAs see at their next barrier, waits (bounded)
 * for its own copies in flight, frees its tensor memory and returns, so the
 * context stays usable. The waits of ts_prefill_chunk, ts_prompt_attend and ts_tree_attend have
 * the same bound (each by itself; one of the longest lasts as long as 128 rows of
 * a prompt take), but what the last two have in flight when one runs out is
 * waited for as long as 1 s even where ns is less. The waits of the separate calls
 * (ts_score, ts_attend, ts_sparse_attend) keep the 1 s bound. ns == 0 is
 * TS_ERR_INVALID_ARG. */
ts_status ts_set_wait_limit(ts_ctx* ctx, uint64_t ns);

/* Fault injection for tests of the time-out path: the NEXT persistent
 * decode-step launch of this context makes CTA `cta` leave at its grid
 * barrier number `barrier` (0 = the first) without arriving, so that every
 * other CTA's bounded wait runs out (TS_ERR_TIMEOUT through ts_get_status).
 * Nothing faults, traps or hangs: the run-out is the ordinary bounded-wait
 * path, and the launch after it starts from clean barrier words. The request
 * is consumed by that one launch; a cta beyond the grid injects nothing. */
ts_status ts_inject_barrier_skip(ts_ctx* ctx, int cta, int barrier);

/* Synchronises `stream`, then reads and clears the device status word.
 * *device_status receives TS_OK or the first device error since the last read. */
ts_status ts_get_status(ts_ctx* ctx, ts_status* device_status, void* stream);

/* Static text for a status code. */
const char* ts_status_str(ts_status s);

/* Kernel timing (tracing). While enabled, every kernel launch of the library is
 * bracketed by a pair of CUDA events on its stream, tagged with its family;
 * inside a CUDA graph capture the events become event-record nodes that each
 * replay re-records. At most 256 brackets are held; later ones are dropped. */
enum {
  TS_PROF_CHECK = 0,   /* Selection Cache test                     */
  TS_PROF_SCORE = 1,   /* paged dot product + per-CTA normaliser    */
  TS_PROF_VOTE = 2,    /* head soft vote                            */
  TS_PROF_SELECT = 3,  /* radix selection, refresh and compaction   */
  TS_PROF_ATTEND = 4,  /* sparse attention + merge                  */
  TS_PROF_STEP = 5,    /* the persistent whole-step kernel          */
  TS_PROF_N = 6
};
typedef struct {
  double ms[TS_PROF_N];        /* summed device time per family */
  int64_t launches[TS_PROF_N]; /* brackets summed per family    */
} ts_profile;
ts_status ts_profile_enable(ts_ctx* ctx, int on);
/* Waits for the recorded brackets and ADDS their durations into *out. With
 * keep == 0 the brackets are released; keep != 0 leaves them registered so a
 * replayed CUDA graph can be read again after each replay. */
ts_status ts_profile_read(ts_ctx* ctx, ts_profile* out, int keep);

/* Number of kernel launches this context has issued (or captured into a CUDA
 * graph) since ts_create, counted on the host at each launch. */
ts_status ts_kernel_count(ts_ctx* ctx, int64_t* out);

/* Tracing: %globaltimer values (ns) at which CTA 0 of the last persistent
 * decode-step kernel reached its phase boundaries (0: start, 1: set-up done,
 * 2+3w / 3+3w / 4+3w: wave w scanned / partials written / barrier passed,
 * 20: scoring done, 21: radix levels done, 22: candidates gathered,
 * 23: selection done, 24: attention done, 25: last barrier passed,
 * 26: outputs merged, 27: end; 32..63 finer points inside the phases, see
 * the kernel source; 0 where not reached). Synchronises `stream`, copies 64
 * values to out64 (host) and clears them. */
ts_status ts_debug_phase_ns(ts_ctx* ctx, uint64_t* out64, void* stream);

/* Library version, e.g. 100 for 0.1.0. */
int ts_version(void);

#ifdef __cplusplus
}
#endif

#endif /* TOKENSELECT_H */
