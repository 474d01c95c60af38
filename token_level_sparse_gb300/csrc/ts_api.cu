// C ABI of libtokenselect: argument validation, context and cache lifetime,
// and the stream-ordered composition of one decode step.
#include <cmath>
#include <algorithm>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <initializer_list>
#include <new>

#include "ts_internal.h"

using namespace ts;

namespace {

template <typename T>
cudaError_t alloc(T** p, size_t n) {
  *p = nullptr;
  if (n == 0) n = 1;
  return cudaMalloc(reinterpret_cast<void**>(p), n * sizeof(T));
}

void free_ctx_buffers(ts_ctx* c) {
  for (auto& b : c->prof) {
    if (b.begin) cudaEventDestroy(b.begin);
    if (b.end) cudaEventDestroy(b.end);
    b.begin = b.end = nullptr;
  }
  cudaFree(c->status);
  cudaFree(c->logits);
  cudaFree(c->partials);
  cudaFree(c->stats);
  cudaFree(c->counters);
  cudaFree(c->sel_state);
  cudaFree(c->hist);
  cudaFree(c->mass_hist);
  cudaFree(c->chunk_counts);
  cudaFree(c->attn_part);
  cudaFree(c->vote);
  cudaFree(c->hit);
  cudaFree(c->qmean);
  cudaFree(c->blk_len);
  cudaFree(c->blk_idx);
  cudaFree(c->sel_rows);
  cudaFree(c->q4_part_o);
  cudaFree(c->q4_part_ml);
  cudaFree(c->tree_part_o);
  cudaFree(c->tree_part_ml);
  cudaFree(c->step_partials);
  cudaFree(c->step_hist);
  cudaFree(c->step_mass);
  cudaFree(c->cand_n);
  cudaFree(c->cands);
  cudaFree(c->cta_cnt);
  cudaFree(c->apart);
  cudaFree(c->step_wpart);
  cudaFree(c->gsync);
  cudaFree(c->phase_ns);
}

// Room for the parts of the tree attention (40 MB at d 128), made by a context's first call: most contexts see no drafts.
// The allocation is no part of a graph that the call is captured into.
ts_status tree_room(ts_ctx* c) {
  if (c->tree_part_ml) return TS_OK;
  const size_t slots = (size_t)tree_part_slots(c->num_sms);
  cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
  cudaError_t e = cudaThreadExchangeStreamCaptureMode(&mode);
  if (e != cudaSuccess) return cuda_status(e);
  e = alloc(&c->tree_part_o, slots * 256 * (size_t)c->cfg.head_dim);
  if (e == cudaSuccess) e = alloc(&c->tree_part_ml, slots * 256);
  if (e != cudaSuccess) {
    cudaFree(c->tree_part_o);
    c->tree_part_o = nullptr;
    cudaGetLastError();   // (the next launch asks for it)
  }
  cudaThreadExchangeStreamCaptureMode(&mode);
  return cuda_status(e);
}

float resolve_scale(const ts_ctx* ctx, float scale) {
  return scale == 0.f ? 1.f / std::sqrt((float)ctx->cfg.head_dim) : scale;
}

bool valid_params(const ts_select_params* p) {
  if (!p) return false;
  if (p->mode != TS_SELECT_TOPK && p->mode != TS_SELECT_TOPP) return false;
  if (p->k < 0 || p->n_sink < 0 || p->n_local < 0) return false;
  if (p->mode == TS_SELECT_TOPP && !(p->top_p > 0.f)) return false;
  if (std::isnan(p->theta) || std::isnan(p->softmax_scale)) return false;
  if (p->score_fn != TS_SCORE_HEAD_SOFT_VOTE && p->score_fn != TS_SCORE_LOGIT_SUM &&
      p->score_fn != TS_SCORE_HEAD_HARD_VOTE)
    return false;
  // the ablation selection functions are ranked by top-k only (top-p's mass is the soft vote's)
  if (p->score_fn != TS_SCORE_HEAD_SOFT_VOTE && p->mode != TS_SELECT_TOPK) return false;
  return true;
}

constexpr int kMaxRows = 1 << 30;                     // rows of one packed call
constexpr int64_t kMaxRowStride = (int64_t)1 << 31;   // elements from one packed row to the next
constexpr double kInv2Pi = 0x1.45f306dc9c883p-3, kInv2PiLow = -0x1.6b01ec5417056p-57;   // 1 / 2pi
constexpr int kMaxTreeRows = 1 << 24;                  // rows of one call for drafted tokens
constexpr int kMaxVocab = 1 << 20;                    // tokens of a vocabulary

cudaStream_t as_stream(void* s) { return static_cast<cudaStream_t>(s); }

// The current device is not the context's: its kernels would be launched where its memory is not.
bool elsewhere(const ts_ctx* ctx) {
  int device = -1;
  return cudaGetDevice(&device) != cudaSuccess || device != ctx->device;
}
bool aligned16(std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if (reinterpret_cast<uintptr_t>(p) % 16 != 0) return false;
  return true;
}
// n elements of 4 bytes from p on, and m from q on, share memory
bool overlap4(const void* p, int64_t n, const void* q, int64_t m) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
  return a < b + 4 * (uintptr_t)m && b < a + 4 * (uintptr_t)n;
}
bool q4_elsewhere(const ts_ctx* ctx) { return ctx->cfg.kv_dtype == TS_KV_Q4 && elsewhere(ctx); }

}  // namespace

extern "C" {

int ts_version(void) { return 100; }

const char* ts_status_str(ts_status s) {
  switch (s) {
    case TS_OK: return "ok";
    case TS_ERR_INVALID_ARG: return "invalid argument";
    case TS_ERR_SHAPE: return "shape outside the context's limits";
    case TS_ERR_UNSUPPORTED: return "head geometry not compiled";
    case TS_ERR_CUDA: return "CUDA runtime error";
    case TS_ERR_PAGE_OOB: return "page-table entry outside the pool";
    case TS_ERR_CAPACITY: return "selection larger than its output buffer";
    case TS_ERR_TIMEOUT: return "a bounded device wait ran out";
    case TS_ERR_COOP_UNAVAILABLE: return "cooperative launch refused";
    case TS_ERR_SEQ_LEN: return "sequence length outside [0, max tokens]";
    case TS_ERR_SCRATCH_LIMIT: return "size beyond the fixed scratch of the no-alloc call";
  }
  return "unknown status";
}

ts_status ts_create(ts_ctx** out, const ts_config* cfg) {
  if (!out || !cfg) return TS_ERR_INVALID_ARG;
  *out = nullptr;
  const ts_config& c = *cfg;
  if (c.n_q_heads < 1 || c.n_kv_heads < 1 || c.n_q_heads % c.n_kv_heads != 0) return TS_ERR_INVALID_ARG;
  if (c.max_batch < 1 || c.max_pages_per_seq < 1 || c.num_pages < 1 || c.head_dim < 1) return TS_ERR_INVALID_ARG;
  if (c.kv_dtype != TS_KV_F32 && c.kv_dtype != TS_KV_BF16 && c.kv_dtype != TS_KV_Q4) return TS_ERR_INVALID_ARG;
  if (c.page_size != kPage && c.page_size != 1) return TS_ERR_UNSUPPORTED;
  if (c.n_kv_heads > kCounterSlots - 2 || c.n_q_heads > 256) return TS_ERR_UNSUPPORTED;
  if ((int64_t)c.max_pages_per_seq * c.page_size > (int64_t)1 << 30) return TS_ERR_SHAPE;
  if (!score_supported(c)) return TS_ERR_UNSUPPORTED;

  ts_ctx* ctx = new (std::nothrow) ts_ctx();
  if (!ctx) return TS_ERR_CUDA;
  ctx->cfg = c;
  // environment switches, read here once (never per call):
  // TOKENSELECT_MULTI_KERNEL=1 keeps ts_decode_step on the multi-kernel path (tests, comparisons)
  if (const char* env = std::getenv("TOKENSELECT_MULTI_KERNEL")) ctx->use_step = !(env[0] == '1');
  // the persistent kernel's TMA page tiles are 16 tokens: a token-granular pool (one token per
  // page) takes the multi-kernel path
  if (c.page_size != kPage) ctx->use_step = false;
  ctx->page_shift = c.page_size == kPage ? 4 : 0;
  ctx->debug = std::getenv("TS_DEBUG") != nullptr;
  if (const char* env = std::getenv("TOKENSELECT_NO_TC")) ctx->no_tc = env[0] == '1';
  if (const char* env = std::getenv("TOKENSELECT_SCAN_CLAIM")) ctx->scan_claim = env[0] == '1';
  // TOKENSELECT_TOPP_ATTEND=gather / range / range_tc: the persistent kernel's top-p attention
  // always shares the selected tokens out over the CTAs, or always attends each CTA's own range
  // (when it may), with P.V on CUDA cores or on the tensor cores (bf16, d = 128)
  if (const char* env = std::getenv("TOKENSELECT_TOPP_ATTEND")) {
    if (std::strcmp(env, "gather") == 0) ctx->range_attend = 0;
    if (std::strcmp(env, "range") == 0) ctx->range_attend = 2;
    if (std::strcmp(env, "range_tc") == 0) {
      ctx->range_attend = 2;
      ctx->range_tc = true;
    }
  }
  if (const char* env = std::getenv("TOKENSELECT_L2_BUDGET_MB")) {
    const long mb = std::strtol(env, nullptr, 10);
    if (mb > 0) ctx->l2_budget = (int64_t)mb << 20;
  }
  if (cudaGetDevice(&ctx->device) != cudaSuccess ||
      cudaDeviceGetAttribute(&ctx->num_sms, cudaDevAttrMultiProcessorCount, ctx->device) != cudaSuccess) {
    delete ctx;
    return TS_ERR_CUDA;
  }
  const size_t B = c.max_batch, H = c.n_q_heads, HKV = c.n_kv_heads, G = H / HKV, D = c.head_dim;
  ctx->max_tokens = c.max_pages_per_seq * c.page_size;
  ctx->score_max_chunks = (ctx->max_tokens + kScorePagesPerCta * kPage - 1) / (kScorePagesPerCta * kPage);
  ctx->sel_max_chunks = (ctx->max_tokens + kSelChunk - 1) / kSelChunk;
  ctx->attn_splits = kAttnMaxSplits;
  const size_t T = ctx->max_tokens;
  cudaError_t e = cudaSuccess;
  auto chk = [&](cudaError_t r) {
    if (e == cudaSuccess) e = r;
  };
  const size_t NS = (size_t)ctx->num_sms;
  // [B][H][T] logits of the multi-kernel path; the persistent kernel keeps, per CTA, the
  // logits of its page range: at most (B*T/16 + NS) pages, which this also covers
  ctx->logits_floats = (int64_t)(B * H * T + H * NS * 2 * kPage);
  chk(alloc(&ctx->status, 1));
  chk(alloc(&ctx->logits, (size_t)ctx->logits_floats));
  const bool q4 = c.kv_dtype == TS_KV_Q4;
  if (!q4) {   // the persistent kernel, and the kernels of the other pools
    chk(alloc(&ctx->step_partials, B * NS * 2 * H));   // two partial rows per CTA where a tile holds two pages
    chk(alloc(&ctx->step_hist, B * kStepHistPerSeq));
    chk(alloc(&ctx->step_mass, B * kStepHistPerSeq));
    chk(alloc(&ctx->cand_n, B));
    chk(alloc(&ctx->cands, B * 2048));
    chk(alloc(&ctx->cta_cnt, B * NS * 4));
    chk(alloc(&ctx->apart, B * NS * H * (D + 2) + 2 * B * H));   // (max, sum) rows padded to an even count
    // per CTA: [sequence][scan warp][head] (max, sum exp) pairs of the CUDA-core scan
    chk(alloc(&ctx->step_wpart, NS * B * kMaxScanWarps * kMaxScanG * 2));
    chk(alloc(&ctx->sel_rows, NS * kStepFlagCap));
    chk(alloc(&ctx->partials, B * ctx->score_max_chunks * H));
    chk(alloc(&ctx->attn_part, B * HKV * kAttnMaxSplits * G * (D + 2)));
    chk(alloc(&ctx->qmean, B * H * D));
  } else {
    const size_t slots = (size_t)q4_part_slots(c, ctx->num_sms);
    chk(alloc(&ctx->q4_part_o, slots * H * D));
    chk(alloc(&ctx->q4_part_ml, slots * H));
  }
  chk(alloc(&ctx->gsync, 4));
  if (e == cudaSuccess) chk(cudaMemset(ctx->gsync, 0, 4 * sizeof(unsigned)));   // then kept zero by each launch
  chk(alloc(&ctx->phase_ns, 64));
  chk(alloc(&ctx->stats, B * H));
  chk(alloc(&ctx->counters, B * kCounterSlots));
  chk(alloc(&ctx->sel_state, B));
  chk(alloc(&ctx->hist, B * 2048));
  chk(alloc(&ctx->mass_hist, B * 2048));
  chk(alloc(&ctx->chunk_counts, B * ctx->sel_max_chunks));
  chk(alloc(&ctx->vote, B * T));
  chk(alloc(&ctx->hit, B));
  chk(alloc(&ctx->blk_len, B));
  chk(alloc(&ctx->blk_idx, B * T + B));
  if (e == cudaSuccess) chk(cudaMemset(ctx->status, 0, sizeof(int)));
  if (e == cudaSuccess) chk(cudaMemset(ctx->counters, 0, B * kCounterSlots * sizeof(unsigned)));
  if (e == cudaSuccess) chk(cudaMemset(ctx->hist, 0, B * 2048 * sizeof(unsigned)));
  if (e == cudaSuccess) chk(cudaMemset(ctx->mass_hist, 0, B * 2048 * sizeof(unsigned long long)));
  if (e == cudaSuccess) chk(cudaMemset(ctx->hit, 0, B));
  if (e == cudaSuccess) chk(cudaMemset(ctx->phase_ns, 0, 64 * sizeof(unsigned long long)));
  if (e == cudaSuccess) chk(cudaDeviceSynchronize());
  if (e != cudaSuccess) {
    free_ctx_buffers(ctx);
    delete ctx;
    return TS_ERR_CUDA;
  }
  *out = ctx;
  return TS_OK;
}

ts_status ts_destroy(ts_ctx* ctx) {
  if (!ctx) return TS_ERR_INVALID_ARG;
  cudaDeviceSynchronize();
  free_ctx_buffers(ctx);
  delete ctx;
  return TS_OK;
}

int64_t ts_page_bytes(const ts_config* c) {
  if (!c) return 0;
  const int64_t rows = (int64_t)c->n_kv_heads * c->page_size, d = c->head_dim;
  switch (c->kv_dtype) {
    case TS_KV_F32: return rows * d * 4;
    case TS_KV_BF16: return rows * d * 2;
    case TS_KV_Q4: return rows * (d / 2 + d / 32);
  }
  return 0;
}

ts_status ts_cache_create(ts_ctx* ctx, ts_cache** out, int n_layers, int capacity) {
  if (!ctx || !out || n_layers < 1 || capacity < 1) return TS_ERR_INVALID_ARG;
  *out = nullptr;
  ts_cache* c = new (std::nothrow) ts_cache();
  if (!c) return TS_ERR_CUDA;
  c->ctx = ctx;
  c->n_layers = n_layers;
  c->capacity = capacity;
  const size_t LB = (size_t)n_layers * ctx->cfg.max_batch;
  const size_t HD = (size_t)ctx->cfg.n_q_heads * ctx->cfg.head_dim;
  cudaError_t e = alloc(&c->cq, LB * HD);
  if (e == cudaSuccess) e = alloc(&c->ct, LB * capacity);
  if (e == cudaSuccess) e = alloc(&c->ct_count, LB);
  if (e == cudaSuccess) e = alloc(&c->filled, LB);
  if (e == cudaSuccess) e = cudaMemset(c->filled, 0, LB);
  if (e == cudaSuccess) e = cudaMemset(c->ct_count, 0, LB * sizeof(int32_t));
  if (e == cudaSuccess) e = cudaDeviceSynchronize();
  if (e != cudaSuccess) {
    cudaFree(c->cq);
    cudaFree(c->ct);
    cudaFree(c->ct_count);
    cudaFree(c->filled);
    delete c;
    return TS_ERR_CUDA;
  }
  *out = c;
  return TS_OK;
}

ts_status ts_cache_destroy(ts_cache* c) {
  if (!c) return TS_ERR_INVALID_ARG;
  cudaDeviceSynchronize();
  cudaFree(c->cq);
  cudaFree(c->ct);
  cudaFree(c->ct_count);
  cudaFree(c->filled);
  delete c;
  return TS_OK;
}

ts_status ts_cache_reset(ts_cache* c, void* stream) {
  if (!c) return TS_ERR_INVALID_ARG;
  return launch_cache_reset(c, as_stream(stream));
}

ts_status ts_cache_check(ts_ctx* ctx, ts_cache* cache, int layer, const float* q, int B, float theta,
                         uint8_t* hit, float* cos_out, void* stream) {
  if (!ctx || !cache || !q || !hit || cache->ctx != ctx) return TS_ERR_INVALID_ARG;
  if (layer < 0 || layer >= cache->n_layers || B < 1 || B > ctx->cfg.max_batch) return TS_ERR_SHAPE;
  if (std::isnan(theta)) return TS_ERR_INVALID_ARG;
  return launch_cache_check(ctx, cache, layer, q, B, theta, hit, cos_out, as_stream(stream));
}

ts_status ts_score(ts_ctx* ctx, const float* q, const void* k_pool, const int32_t* page_table,
                   const int32_t* seq_lens, int B, const uint8_t* skip, float scale, float* vote,
                   int64_t vote_stride, void* stream) {
  if (!ctx || !q || !k_pool || !page_table || !seq_lens || !vote) return TS_ERR_INVALID_ARG;
  if (q4_elsewhere(ctx)) return TS_ERR_INVALID_ARG;
  if (B < 1 || B > ctx->cfg.max_batch || vote_stride < ctx->max_tokens) return TS_ERR_SHAPE;
  if (std::isnan(scale)) return TS_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(k_pool) % 16 != 0) return TS_ERR_INVALID_ARG;
  ScoreCall c{q, k_pool, page_table, seq_lens, skip, B, resolve_scale(ctx, scale), vote, vote_stride};
  return launch_score(ctx, c, as_stream(stream));
}

ts_status ts_score_fn(ts_ctx* ctx, const ts_select_params* params, const float* q, const void* k_pool,
                      const int32_t* page_table, const int32_t* seq_lens, int B, const uint8_t* skip,
                      float* vote, int64_t vote_stride, void* stream) {
  if (!ctx || !q || !k_pool || !page_table || !seq_lens || !vote || !valid_params(params))
    return TS_ERR_INVALID_ARG;
  if (q4_elsewhere(ctx)) return TS_ERR_INVALID_ARG;
  if (B < 1 || B > ctx->cfg.max_batch || vote_stride < ctx->max_tokens) return TS_ERR_SHAPE;
  if (reinterpret_cast<uintptr_t>(k_pool) % 16 != 0) return TS_ERR_INVALID_ARG;
  ScoreCall c{q, k_pool, page_table, seq_lens, skip, B, resolve_scale(ctx, params->softmax_scale), vote,
              vote_stride};
  c.fn = params->score_fn;
  c.k = params->k;
  c.n_sink = params->n_sink;
  c.n_local = params->n_local;
  return launch_score(ctx, c, as_stream(stream));
}

ts_status ts_select(ts_ctx* ctx, ts_cache* cache, int layer, const float* q, const float* vote,
                    int64_t vote_stride, const int32_t* seq_lens, int B, const uint8_t* hit,
                    const ts_select_params* params, int32_t* idx, int64_t idx_stride, int32_t* count,
                    void* stream) {
  if (!ctx || !vote || !seq_lens || !idx || !count || !valid_params(params)) return TS_ERR_INVALID_ARG;
  if (B < 1 || B > ctx->cfg.max_batch || vote_stride < ctx->max_tokens || idx_stride < 1) return TS_ERR_SHAPE;
  if (hit && !cache) return TS_ERR_INVALID_ARG;
  if (cache) {
    if (cache->ctx != ctx || !q) return TS_ERR_INVALID_ARG;
    if (layer < 0 || layer >= cache->n_layers) return TS_ERR_SHAPE;
  }
  SelectCall c{cache, layer, q, vote, vote_stride, seq_lens, B, hit, *params, idx, idx_stride, count};
  return launch_select(ctx, c, as_stream(stream));
}

ts_status ts_sparse_attend(ts_ctx* ctx, const float* q, const void* k_pool, const void* v_pool,
                           const int32_t* page_table, const int32_t* idx, int64_t idx_stride,
                           const int32_t* count, int B, float scale, float* out, float* lse, void* stream) {
  if (!ctx || !q || !k_pool || !v_pool || !page_table || !idx || !count || !out) return TS_ERR_INVALID_ARG;
  if (q4_elsewhere(ctx)) return TS_ERR_INVALID_ARG;
  if (B < 1 || B > ctx->cfg.max_batch || idx_stride < 1) return TS_ERR_SHAPE;
  if (std::isnan(scale)) return TS_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(k_pool) % 16 != 0 || reinterpret_cast<uintptr_t>(v_pool) % 16 != 0)
    return TS_ERR_INVALID_ARG;
  AttendCall c{q, k_pool, v_pool, page_table, idx, idx_stride, count, B, resolve_scale(ctx, scale), out, lse};
  return launch_attend(ctx, c, as_stream(stream));
}

ts_status ts_decode_step(ts_ctx* ctx, ts_cache* cache, int layer, const float* q, const void* k_pool,
                         const void* v_pool, const int32_t* page_table, const int32_t* seq_lens, int B,
                         const ts_select_params* params, float* vote, int64_t vote_stride, int32_t* idx,
                         int64_t idx_stride, int32_t* count, float* out, float* lse, uint8_t* hit,
                         void* stream) {
  if (!ctx || !q || !k_pool || !v_pool || !page_table || !seq_lens || !idx || !count || !out ||
      !valid_params(params))
    return TS_ERR_INVALID_ARG;
  if (q4_elsewhere(ctx)) return TS_ERR_INVALID_ARG;
  if (B < 1 || B > ctx->cfg.max_batch || idx_stride < 1) return TS_ERR_SHAPE;
  if (cache && (cache->ctx != ctx || layer < 0 || layer >= cache->n_layers)) return TS_ERR_INVALID_ARG;
  if (!vote) {
    vote = ctx->vote;
    vote_stride = ctx->max_tokens;
  }
  if (vote_stride < ctx->max_tokens) return TS_ERR_SHAPE;
  if (reinterpret_cast<uintptr_t>(k_pool) % 16 != 0 || reinterpret_cast<uintptr_t>(v_pool) % 16 != 0)
    return TS_ERR_INVALID_ARG;
  cudaStream_t s = as_stream(stream);
  const float scale = resolve_scale(ctx, params->softmax_scale);
  const bool use_cache = cache != nullptr && params->theta <= 1.f;
  uint8_t* hbuf = hit ? hit : ctx->hit;
  ts_status st = TS_OK;
  if (ctx->use_step && step_supported(ctx->cfg) && B <= 64 && params->score_fn == TS_SCORE_HEAD_SOFT_VOTE) {
    // one persistent cooperative kernel for the whole step
    if (!use_cache && hit && cudaMemsetAsync(hit, 0, B, s) != cudaSuccess) return TS_ERR_CUDA;
    StepCall sc{};
    sc.phases = kPhaseScore | kPhaseSelect | kPhaseAttend | (use_cache ? kPhaseCheck : 0);
    sc.B = B;
    sc.q = q;
    sc.k_pool = k_pool;
    sc.v_pool = v_pool;
    sc.page_table = page_table;
    sc.seq_lens = seq_lens;
    sc.scale = scale;
    sc.theta = params->theta;
    sc.hit_in = nullptr;
    sc.hit_out = use_cache ? hbuf : nullptr;
    sc.cache = cache;
    sc.layer = layer;
    sc.params = *params;
    sc.vote = vote;
    sc.vote_stride = vote_stride;
    sc.idx = idx;
    sc.idx_stride = idx_stride;
    sc.count = count;
    sc.out = out;
    sc.lse = lse;
    st = launch_step(ctx, sc, s);
    if (ctx->debug) std::fprintf(stderr, "ts decode step: persistent kernel -> %s\n", ts_status_str(st));
    if (st != TS_ERR_COOP_UNAVAILABLE) return st;
    ctx->use_step = false;  // the multi-kernel path below from now on
  }
  if (use_cache) {
    st = launch_cache_check(ctx, cache, layer, q, B, params->theta, hbuf, nullptr, s);
    if (st != TS_OK) return st;
  } else if (hit) {
    if (cudaMemsetAsync(hit, 0, B, s) != cudaSuccess) return TS_ERR_CUDA;
  }
  const uint8_t* skip = use_cache ? hbuf : nullptr;
  ScoreCall sc{q, k_pool, page_table, seq_lens, skip, B, scale, vote, vote_stride};
  sc.fn = params->score_fn;
  sc.k = params->k;
  sc.n_sink = params->n_sink;
  sc.n_local = params->n_local;
  st = launch_score(ctx, sc, s);
  if (st != TS_OK) return st;
  SelectCall sel{cache, layer, q, vote, vote_stride, seq_lens, B, skip, *params, idx, idx_stride, count};
  st = launch_select(ctx, sel, s);
  if (st != TS_OK) return st;
  AttendCall ac{q, k_pool, v_pool, page_table, idx, idx_stride, count, B, scale, out, lse};
  return launch_attend(ctx, ac, s);
}

ts_status ts_prefill_chunk(ts_ctx* ctx, const float* q, int c, const void* k_pool, const void* v_pool,
                           const int32_t* page_table, const int32_t* seq_lens, int B, const ts_select_params* params,
                           float* vote, int64_t vote_stride, int32_t* idx, int64_t idx_stride, int32_t* count,
                           float* out, float* lse, void* stream) {
  if (!ctx || !q || !k_pool || !v_pool || !page_table || !seq_lens || !idx || !count || !out ||
      !valid_params(params))
    return TS_ERR_INVALID_ARG;
  if (params->mode != TS_SELECT_TOPK || params->score_fn != TS_SCORE_HEAD_SOFT_VOTE) return TS_ERR_INVALID_ARG;
  if (c < 1 || B < 1 || B > ctx->cfg.max_batch || idx_stride < 1) return TS_ERR_SHAPE;
  if (reinterpret_cast<uintptr_t>(k_pool) % 16 != 0 || reinterpret_cast<uintptr_t>(v_pool) % 16 != 0 ||
      reinterpret_cast<uintptr_t>(q) % 16 != 0)
    return TS_ERR_INVALID_ARG;
  if (!chunk_attend_supported(ctx->cfg)) return TS_ERR_UNSUPPORTED;
  if (!vote) {
    vote = ctx->vote;
    vote_stride = ctx->max_tokens;
  }
  if (vote_stride < ctx->max_tokens) return TS_ERR_SHAPE;
  cudaStream_t s = as_stream(stream);
  const float scale = resolve_scale(ctx, params->softmax_scale);
  // (1) the mean query of every chunk
  ts_status st = launch_chunk_mean(ctx, q, c, B, ctx->qmean, s);
  if (st != TS_OK) return st;
  // (2) one selection from it: score, vote and top-k (the persistent kernel without its attention)
  st = TS_ERR_COOP_UNAVAILABLE;
  if (ctx->use_step && step_supported(ctx->cfg) && B <= 64) {
    StepCall sc{};
    sc.phases = kPhaseScore | kPhaseSelect;
    sc.B = B;
    sc.q = ctx->qmean;
    sc.k_pool = k_pool;
    sc.v_pool = v_pool;
    sc.page_table = page_table;
    sc.seq_lens = seq_lens;
    sc.scale = scale;
    sc.theta = 2.f;
    sc.params = *params;
    sc.vote = vote;
    sc.vote_stride = vote_stride;
    sc.idx = idx;
    sc.idx_stride = idx_stride;
    sc.count = count;
    st = launch_step(ctx, sc, s);
    if (st != TS_OK && st != TS_ERR_COOP_UNAVAILABLE) return st;
  }
  if (st != TS_OK) {
    ScoreCall scc{ctx->qmean, k_pool, page_table, seq_lens, nullptr, B, scale, vote, vote_stride};
    st = launch_score(ctx, scc, s);
    if (st != TS_OK) return st;
    SelectCall sel{nullptr, 0, ctx->qmean, vote, vote_stride, seq_lens, B, nullptr, *params, idx, idx_stride, count};
    st = launch_select(ctx, sel, s);
    if (st != TS_OK) return st;
  }
  // (3) the chunk's queries attend causally to the shared selection, on the tensor cores
  ChunkAttendCall ac{q, c, k_pool, v_pool, page_table, seq_lens, idx, idx_stride, count, B, scale, out, lse};
  return launch_chunk_attend(ctx, ac, s);
}

ts_status ts_append_kv(ts_ctx* ctx, const void* k_new, const void* v_new, const int32_t* page_table,
                       const int32_t* seq_lens, int B, void* k_pool, void* v_pool, void* stream) {
  if (!ctx || !k_new || !v_new || !page_table || !seq_lens || !k_pool || !v_pool) return TS_ERR_INVALID_ARG;
  if (q4_elsewhere(ctx)) return TS_ERR_INVALID_ARG;
  if (B < 1 || B > ctx->cfg.max_batch) return TS_ERR_SHAPE;
  for (const void* p : {k_new, v_new, static_cast<const void*>(k_pool), static_cast<const void*>(v_pool)})
    if (reinterpret_cast<uintptr_t>(p) % 16 != 0) return TS_ERR_INVALID_ARG;
  return launch_append_kv(ctx, k_new, v_new, page_table, seq_lens, B, k_pool, v_pool, as_stream(stream));
}

ts_status ts_append_prompt(ts_ctx* ctx, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                           const int32_t* cu_rows, const int32_t* starts, int B, int total,
                           const int32_t* page_table, void* k_pool, void* v_pool, void* stream) {
  if (!ctx || !k || !v || !cu_rows || !page_table || !k_pool || !v_pool) return TS_ERR_INVALID_ARG;
  if (elsewhere(ctx)) return TS_ERR_INVALID_ARG;
  const ts_config& c = ctx->cfg;
  const int64_t row = (int64_t)c.n_kv_heads * c.head_dim, per16 = c.kv_dtype == TS_KV_F32 ? 4 : 8;
  if (B < 1 || B > c.max_batch || total < 0 || total > kMaxRows) return TS_ERR_SHAPE;
  if (k_stride < row || v_stride < row || k_stride > kMaxRowStride || v_stride > kMaxRowStride) return TS_ERR_SHAPE;
  if (k_stride % per16 != 0 || v_stride % per16 != 0) return TS_ERR_INVALID_ARG;
  for (const void* p : {k, v, static_cast<const void*>(k_pool), static_cast<const void*>(v_pool)})
    if (reinterpret_cast<uintptr_t>(p) % 16 != 0) return TS_ERR_INVALID_ARG;
  AppendPromptCall a{k, k_stride, v, v_stride, cu_rows, starts, B, total, page_table, k_pool, v_pool};
  return launch_append_prompt(ctx, a, as_stream(stream));
}

ts_status ts_read_kv(ts_ctx* ctx, const int32_t* cu_rows, const int32_t* starts, int B, int total,
                     const int32_t* page_table, const void* k_pool, const void* v_pool, float* k_out, float* v_out,
                     void* stream) {
  if (!ctx || !cu_rows || !page_table || !k_pool || !v_pool || !k_out || !v_out) return TS_ERR_INVALID_ARG;
  if (elsewhere(ctx)) return TS_ERR_INVALID_ARG;
  if (B < 1 || B > ctx->cfg.max_batch || total < 0 || total > kMaxRows) return TS_ERR_SHAPE;
  for (const void* p : {k_pool, v_pool, static_cast<const void*>(k_out), static_cast<const void*>(v_out)})
    if (reinterpret_cast<uintptr_t>(p) % 16 != 0) return TS_ERR_INVALID_ARG;
  return launch_read_kv(ctx, cu_rows, starts, B, total, page_table, k_pool, v_pool, k_out, v_out, as_stream(stream));
}

ts_status ts_attend(ts_ctx* ctx, const float* q, const void* k_pool, const void* v_pool, const int32_t* page_table,
                    const int32_t* seq_lens, int B, float scale, float* out, float* lse, void* stream) {
  if (!ctx || !q || !k_pool || !v_pool || !page_table || !seq_lens || !out) return TS_ERR_INVALID_ARG;
  if (elsewhere(ctx)) return TS_ERR_INVALID_ARG;
  if (B < 1 || B > ctx->cfg.max_batch) return TS_ERR_SHAPE;
  if (std::isnan(scale)) return TS_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(k_pool) % 16 != 0 || reinterpret_cast<uintptr_t>(v_pool) % 16 != 0)
    return TS_ERR_INVALID_ARG;
  if (ctx->cfg.kv_dtype != TS_KV_Q4) return TS_ERR_UNSUPPORTED;
  AttendCall c{q, k_pool, v_pool, page_table, nullptr, 0, nullptr, B, resolve_scale(ctx, scale), out, lse};
  return launch_attend_q4(ctx, c, seq_lens, as_stream(stream));
}

ts_status ts_prompt_attend(ts_ctx* ctx, const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                           const void* v, int64_t v_stride, const int32_t* cu_rows, int B, int total, float scale,
                           void* out, int64_t out_stride, float* lse, void* stream) {
  if (!ctx || !q || !k || !v || !cu_rows || !out) return TS_ERR_INVALID_ARG;
  if (elsewhere(ctx)) return TS_ERR_INVALID_ARG;
  const ts_config& c = ctx->cfg;
  const int64_t qrow = (int64_t)c.n_q_heads * c.head_dim, krow = (int64_t)c.n_kv_heads * c.head_dim;
  if (B < 1 || B > c.max_batch || total < 0 || total > kMaxRows) return TS_ERR_SHAPE;
  if (q_stride < qrow || out_stride < qrow || k_stride < krow || v_stride < krow) return TS_ERR_SHAPE;
  for (int64_t st : {q_stride, k_stride, v_stride, out_stride}) {
    if (st > kMaxRowStride) return TS_ERR_SHAPE;
    if (st % 8 != 0) return TS_ERR_INVALID_ARG;
  }
  for (const void* p : {q, k, v, static_cast<const void*>(out)})
    if (reinterpret_cast<uintptr_t>(p) % 16 != 0) return TS_ERR_INVALID_ARG;
  if (std::isnan(scale)) return TS_ERR_INVALID_ARG;
  if (!prompt_supported(c)) return TS_ERR_UNSUPPORTED;
  PromptCall a{q, q_stride, k, k_stride, v, v_stride, cu_rows, B, total, resolve_scale(ctx, scale), out, out_stride, lse};
  return launch_prompt_attend(ctx, a, as_stream(stream));
}

// Frequencies of every pair in radians per position, by the configuration's rule.
ts_status ts_rope_create(ts_rope** out, const ts_rope_config* cfg) {
  if (!out || !cfg) return TS_ERR_INVALID_ARG;
  *out = nullptr;
  const ts_rope_config& c = *cfg;
  if (c.rot_dim < 2 || c.rot_dim > 128 || c.rot_dim % 2 != 0) return TS_ERR_SHAPE;
  if (c.interleaved != 0 && c.interleaved != 1) return TS_ERR_INVALID_ARG;
  if (c.scaling < TS_ROPE_PLAIN || c.scaling > TS_ROPE_GIVEN) return TS_ERR_INVALID_ARG;
  if ((c.scaling == TS_ROPE_GIVEN) != (c.freqs != nullptr)) return TS_ERR_INVALID_ARG;
  const double pi = 3.14159265358979323846;
  if (c.scaling != TS_ROPE_GIVEN && !(std::isfinite(c.base) && c.base > 0.)) return TS_ERR_INVALID_ARG;
  if (c.scaling != TS_ROPE_GIVEN && c.scaling != TS_ROPE_PLAIN && !(std::isfinite(c.factor) && c.factor > 0.))
    return TS_ERR_INVALID_ARG;
  const bool ranged = c.scaling == TS_ROPE_BANDS || c.scaling == TS_ROPE_YARN;
  if (ranged && !(c.original > 0 && std::isfinite(c.low) && std::isfinite(c.high) && c.low > 0. && c.high > c.low))
    return TS_ERR_INVALID_ARG;
  if (c.scaling == TS_ROPE_YARN && c.base == 1.) return TS_ERR_INVALID_ARG;
  if (!std::isfinite(c.attention) || c.attention < 0.) return TS_ERR_INVALID_ARG;
  ts_rope* r = new (std::nothrow) ts_rope();
  if (!r) return TS_ERR_CUDA;
  r->rot_dim = c.rot_dim;
  r->interleaved = c.interleaved;
  const int n = c.rot_dim / 2;
  double base = c.base, first = 0., last = 0.;
  if (c.scaling == TS_ROPE_BASE && c.rot_dim > 2) base *= std::pow(c.factor, (double)c.rot_dim / (c.rot_dim - 2));
  if (c.scaling == TS_ROPE_YARN) {
    // the pairs that turn `high` and `low` times within the original context
    auto pair = [&](double turns) { return c.rot_dim * std::log(c.original / (2. * pi * turns)) / (2. * std::log(c.base)); };
    first = std::max(0., std::floor(pair(c.high)));
    last = std::min((double)c.rot_dim - 1., std::ceil(pair(c.low)));
  }
  for (int i = 0; i < n; ++i) {
    double f = c.scaling == TS_ROPE_GIVEN ? c.freqs[i] : std::pow(base, -2. * i / c.rot_dim);
    if (c.scaling == TS_ROPE_LINEAR) f /= c.factor;
    if (c.scaling == TS_ROPE_BANDS) {
      const double t = std::min(1., std::max(0., (c.original * f / (2. * pi) - c.low) / (c.high - c.low)));
      f = (1. - t) * f / c.factor + t * f;
    }
    if (c.scaling == TS_ROPE_YARN) {
      const double t = std::min(1., std::max(0., (i - first) / std::max(last - first, 0.001)));
      f = t * f / c.factor + (1. - t) * f;
    }
    if (!std::isfinite(f)) {
      delete r;
      return TS_ERR_INVALID_ARG;
    }
    r->freqs[i] = f;
    // f / 2pi modulo 1 in units of 2^-64: the product with 1 / 2pi (to 107 bits) in two parts, both exact modulo 1
    const double whole = std::fabs(f) * kInv2Pi, rest = std::fma(std::fabs(f), kInv2Pi, -whole) + std::fabs(f) * kInv2PiLow;
    const double turn = std::fmod(whole, 1.), more = std::fmod(rest, 1.);
    const uint64_t low = (uint64_t)std::ldexp(std::fabs(more), 64);
    const uint64_t u = (uint64_t)std::ldexp(turn, 64) + (more < 0. ? 0 - low : low);
    r->turns[i] = f < 0. ? 0 - u : u;
  }
  const double by_rule = c.scaling == TS_ROPE_YARN && c.factor > 1. ? 0.1 * std::log(c.factor) + 1. : 1.;
  r->factor = (float)(c.attention > 0. ? c.attention : by_rule);
  *out = r;
  return TS_OK;
}

ts_status ts_rope_destroy(ts_rope* rope) {
  if (!rope) return TS_ERR_INVALID_ARG;
  delete rope;
  return TS_OK;
}

ts_status ts_rope_read(const ts_rope* rope, double* freqs, double* attention) {
  if (!rope || !freqs || !attention) return TS_ERR_INVALID_ARG;
  for (int i = 0; i < rope->rot_dim / 2; ++i) freqs[i] = rope->freqs[i];
  *attention = rope->factor;
  return TS_OK;
}

ts_status ts_rotate(ts_ctx* ctx, const ts_rope* rope, const void* x, int64_t x_stride, int dtype, int heads,
                    const int32_t* positions, int total, void* out, int64_t out_stride, int out_dtype, void* stream) {
  if (!ctx || !rope || (total > 0 && (!x || !positions || !out))) return TS_ERR_INVALID_ARG;
  if (elsewhere(ctx)) return TS_ERR_INVALID_ARG;
  if ((dtype != TS_KV_F32 && dtype != TS_KV_BF16) || (out_dtype != TS_KV_F32 && out_dtype != TS_KV_BF16))
    return TS_ERR_INVALID_ARG;
  const ts_config& c = ctx->cfg;
  if (heads < 1 || heads > 4096 || total < 0 || total > kMaxRows || rope->rot_dim > c.head_dim) return TS_ERR_SHAPE;
  const int64_t row = (int64_t)heads * c.head_dim;
  if (x_stride < row || out_stride < row || x_stride > kMaxRowStride || out_stride > kMaxRowStride) return TS_ERR_SHAPE;
  if (x_stride % (dtype == TS_KV_F32 ? 4 : 8) != 0 || out_stride % (out_dtype == TS_KV_F32 ? 4 : 8) != 0)
    return TS_ERR_INVALID_ARG;
  if (!aligned16({x, out})) return TS_ERR_INVALID_ARG;
  if (x == out && (x_stride != out_stride || dtype != out_dtype) && total > 0) return TS_ERR_INVALID_ARG;
  RotateCall a{x, x_stride, dtype, heads, positions, total, out, out_stride, out_dtype};
  return launch_rotate(ctx, rope, a, as_stream(stream));
}

ts_status ts_append_rotated(ts_ctx* ctx, const ts_rope* rope, const void* k, int64_t k_stride, const void* v,
                            int64_t v_stride, const int32_t* positions, const int32_t* cu_rows, const int32_t* starts,
                            int B, int total, const int32_t* page_table, void* k_pool, void* v_pool, const void* q,
                            int64_t q_stride, void* q_out, int64_t q_out_stride, int q_out_dtype, void* stream) {
  if (!ctx || !rope || !cu_rows || !page_table || !k_pool || !v_pool) return TS_ERR_INVALID_ARG;
  if (total > 0 && (!k || !v || !positions)) return TS_ERR_INVALID_ARG;
  if ((q == nullptr) != (q_out == nullptr)) return TS_ERR_INVALID_ARG;
  if (elsewhere(ctx)) return TS_ERR_INVALID_ARG;
  const ts_config& c = ctx->cfg;
  const int64_t row = (int64_t)c.n_kv_heads * c.head_dim, qrow = (int64_t)c.n_q_heads * c.head_dim;
  const int64_t per16 = c.kv_dtype == TS_KV_F32 ? 4 : 8;
  if (B < 1 || B > c.max_batch || total < 0 || total > kMaxRows || rope->rot_dim > c.head_dim) return TS_ERR_SHAPE;
  if (k_stride < row || v_stride < row || k_stride > kMaxRowStride || v_stride > kMaxRowStride) return TS_ERR_SHAPE;
  if (k_stride % per16 != 0 || v_stride % per16 != 0) return TS_ERR_INVALID_ARG;
  if (q) {
    if (q_out_dtype != TS_KV_F32 && q_out_dtype != TS_KV_BF16) return TS_ERR_INVALID_ARG;
    if (q_stride < qrow || q_out_stride < qrow || q_stride > kMaxRowStride || q_out_stride > kMaxRowStride) return TS_ERR_SHAPE;
    if (q_stride % per16 != 0 || q_out_stride % (q_out_dtype == TS_KV_F32 ? 4 : 8) != 0) return TS_ERR_INVALID_ARG;
    if (q == q_out && (q_stride != q_out_stride || (q_out_dtype == TS_KV_F32) != (c.kv_dtype == TS_KV_F32)))
      return TS_ERR_INVALID_ARG;
  }
  if (!aligned16({k, v, k_pool, v_pool, q, q_out})) return TS_ERR_INVALID_ARG;
  AppendPromptCall a{k, k_stride, v, v_stride, cu_rows, starts, B, total, page_table, k_pool, v_pool};
  RotateCall r{q, q_stride, c.kv_dtype == TS_KV_F32 ? TS_KV_F32 : TS_KV_BF16, c.n_q_heads, positions, total, q_out, q_out_stride,
               q_out_dtype};
  return launch_append_rotated(ctx, rope, a, r, as_stream(stream));
}

ts_status ts_tree_attend(ts_ctx* ctx, const void* q, int64_t q_stride, const void* k_pool, const void* v_pool,
                         const int32_t* page_table, const int32_t* seq_lens, const int32_t* cu_rows, const int32_t* mask,
                         int mask_words, int B, int total, float scale, void* out, int64_t out_stride, float* lse,
                         void* stream) {
  if (!ctx || !k_pool || !v_pool || !page_table || !seq_lens || !cu_rows) return TS_ERR_INVALID_ARG;
  if (total > 0 && (!q || !out)) return TS_ERR_INVALID_ARG;
  if (elsewhere(ctx)) return TS_ERR_INVALID_ARG;
  const ts_config& c = ctx->cfg;
  const int64_t row = (int64_t)c.n_q_heads * c.head_dim;
  if (B < 1 || B > c.max_batch || total < 0 || total > kMaxRows) return TS_ERR_SHAPE;
  if (total > kMaxTreeRows) return TS_ERR_SHAPE;
  if (mask && (mask_words < 1 || mask_words > kMaxTree / 32)) return TS_ERR_SHAPE;
  if (q_stride < row || out_stride < row || q_stride > kMaxRowStride || out_stride > kMaxRowStride) return TS_ERR_SHAPE;
  if (q_stride % 8 != 0 || out_stride % 8 != 0 || !aligned16({q, k_pool, v_pool, out})) return TS_ERR_INVALID_ARG;
  if (std::isnan(scale)) return TS_ERR_INVALID_ARG;
  if (!tree_supported(c)) return TS_ERR_UNSUPPORTED;
  if (const ts_status st = tree_room(ctx); st != TS_OK) return st;
  TreeCall a{q, q_stride, k_pool, v_pool, page_table, seq_lens, cu_rows, mask, mask_words, B, total,
             resolve_scale(ctx, scale), out, out_stride, lse};
  return launch_tree_attend(ctx, a, as_stream(stream));
}

ts_status ts_verify_tree(ts_ctx* ctx, const int32_t* tokens, const int32_t* parents, const int32_t* cu_rows, int B,
                         int total, int vocab, const float* target, int64_t target_stride, const float* draft,
                         int64_t draft_stride, const float* u, const float* u_next, int distinct, int32_t* path,
                         int64_t path_stride, int32_t* count, int32_t* next_token, void* stream) {
  if (!ctx || !cu_rows || !u_next || !path || !count || !next_token) return TS_ERR_INVALID_ARG;
  if (total > 0 && (!tokens || !parents || !target || !u)) return TS_ERR_INVALID_ARG;
  if (elsewhere(ctx)) return TS_ERR_INVALID_ARG;
  if (B < 1 || B > ctx->cfg.max_batch || total < 0 || total > kMaxRows) return TS_ERR_SHAPE;
  if (vocab < 1 || vocab > kMaxVocab || path_stride < 1 || path_stride > kMaxRowStride) return TS_ERR_SHAPE;
  if (target_stride < vocab || (draft && draft_stride < vocab)) return TS_ERR_SHAPE;
  VerifyCall a{tokens, parents, cu_rows, B, total, vocab, target, target_stride, draft, draft_stride, u, u_next,
               distinct != 0, path, path_stride, count, next_token};
  return launch_verify(ctx, a, as_stream(stream));
}

ts_status ts_keep_rows(ts_ctx* ctx, const int32_t* path, int64_t path_stride, const int32_t* count, const int32_t* cu_rows,
                       const int32_t* seq_lens, int B, int total, const int32_t* page_table, void* k_pool, void* v_pool,
                       int n_layers, int64_t layer_bytes, int32_t* new_lens, void* stream) {
  if (!ctx || !path || !count || !cu_rows || !seq_lens || !page_table || !k_pool || !v_pool) return TS_ERR_INVALID_ARG;
  if (elsewhere(ctx)) return TS_ERR_INVALID_ARG;
  if (B < 1 || B > ctx->cfg.max_batch || total < 0 || total > kMaxRows) return TS_ERR_SHAPE;
  if (path_stride < 1 || path_stride > kMaxRowStride || n_layers < 1 || n_layers > 65535) return TS_ERR_SHAPE;
  if (n_layers > 1 && layer_bytes < ctx->cfg.num_pages * ts_page_bytes(&ctx->cfg)) return TS_ERR_SHAPE;
  if ((n_layers > 1 && layer_bytes % 16 != 0) || !aligned16({k_pool, v_pool})) return TS_ERR_INVALID_ARG;
  // (each of many CTAs reads these, one writes the new lengths)
  if (new_lens && (overlap4(new_lens, B, seq_lens, B) || overlap4(new_lens, B, count, B) || overlap4(new_lens, B, cu_rows, B + 1) ||
                   overlap4(new_lens, B, path, B * path_stride)))
    return TS_ERR_INVALID_ARG;
  KeepCall a{path, path_stride, count, cu_rows, seq_lens, B, total, page_table, k_pool, v_pool, n_layers, layer_bytes, new_lens};
  return launch_keep_rows(ctx, a, as_stream(stream));
}

ts_status ts_select_blocks(ts_ctx* ctx, const float* vote, int64_t vote_stride, const int32_t* seq_lens, int B,
                           int block, int budget, int32_t* idx, int64_t idx_stride, int32_t* count, void* stream) {
  if (!ctx || !vote || !seq_lens || !idx || !count) return TS_ERR_INVALID_ARG;
  if (block < 1 || budget < 0) return TS_ERR_INVALID_ARG;
  if (B < 1 || B > ctx->cfg.max_batch || vote_stride < ctx->max_tokens || idx_stride < 1) return TS_ERR_SHAPE;
  return launch_select_blocks(ctx, vote, vote_stride, seq_lens, B, block, budget, idx, idx_stride, count,
                              as_stream(stream));
}

ts_status ts_debug_phase_ns(ts_ctx* ctx, uint64_t* out64, void* stream) {
  if (!ctx || !out64) return TS_ERR_INVALID_ARG;
  if (cudaStreamSynchronize(as_stream(stream)) != cudaSuccess) return TS_ERR_CUDA;
  if (cudaMemcpy(out64, ctx->phase_ns, 64 * sizeof(uint64_t), cudaMemcpyDeviceToHost) != cudaSuccess)
    return TS_ERR_CUDA;
  return cudaMemset(ctx->phase_ns, 0, 64 * sizeof(uint64_t)) == cudaSuccess ? TS_OK : TS_ERR_CUDA;
}

ts_status ts_kernel_count(ts_ctx* ctx, int64_t* out) {
  if (!ctx || !out) return TS_ERR_INVALID_ARG;
  *out = ctx->kernels;
  return TS_OK;
}

ts_status ts_profile_enable(ts_ctx* ctx, int on) {
  if (!ctx) return TS_ERR_INVALID_ARG;
  if (on) {
    for (auto& b : ctx->prof) {
      if (!b.begin && cudaEventCreate(&b.begin) != cudaSuccess) return TS_ERR_CUDA;
      if (!b.end && cudaEventCreate(&b.end) != cudaSuccess) return TS_ERR_CUDA;
    }
  }
  ctx->prof_on = on != 0;
  return TS_OK;
}

ts_status ts_profile_read(ts_ctx* ctx, ts_profile* out, int keep) {
  if (!ctx || !out) return TS_ERR_INVALID_ARG;
  for (int i = 0; i < ctx->prof_used; ++i) {
    ProfBracket& b = ctx->prof[i];
    if (!b.recorded) continue;
    if (cudaEventSynchronize(b.end) != cudaSuccess) return TS_ERR_CUDA;
    float ms = 0.f;
    if (cudaEventElapsedTime(&ms, b.begin, b.end) != cudaSuccess) return TS_ERR_CUDA;
    out->ms[b.family] += ms;
    out->launches[b.family] += 1;
  }
  if (!keep) ctx->prof_used = 0;
  return TS_OK;
}

ts_status ts_set_wait_limit(ts_ctx* ctx, uint64_t ns) {
  if (!ctx || ns == 0) return TS_ERR_INVALID_ARG;
  ctx->wait_ns = ns;
  return TS_OK;
}

ts_status ts_inject_barrier_skip(ts_ctx* ctx, int cta, int barrier) {
  if (!ctx || cta < 0 || barrier < 0) return TS_ERR_INVALID_ARG;
  ctx->inject_skip_cta = cta;
  ctx->inject_skip_barrier = barrier;
  return TS_OK;
}

ts_status ts_get_status(ts_ctx* ctx, ts_status* device_status, void* stream) {
  if (!ctx || !device_status) return TS_ERR_INVALID_ARG;
  if (cudaStreamSynchronize(as_stream(stream)) != cudaSuccess) return TS_ERR_CUDA;
  int v = 0;
  if (cudaMemcpy(&v, ctx->status, sizeof(int), cudaMemcpyDeviceToHost) != cudaSuccess) return TS_ERR_CUDA;
  if (cudaMemset(ctx->status, 0, sizeof(int)) != cudaSuccess) return TS_ERR_CUDA;
  *device_status = static_cast<ts_status>(v);
  return TS_OK;
}

}  // extern "C"
