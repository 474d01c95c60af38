// Rows into and out of the paged pools: packed K and V rows of whole prompts (ts_append_prompt),
// one token per sequence into a 4-bit pool (ts_append_kv), and rows read back as fp32 values
// (ts_read_kv).
//
// Packed row r belongs to sequence b with cu[b] <= r < cu[b + 1] and goes to position
// starts[b] + r - cu[b]. A CTA takes a few neighbouring rows: it looks up their page and slot once,
// then its threads move 16 bytes (or, into and out of 4-bit blocks, 8 elements) each. Every byte is
// read and written once, so the copies are bound by memory; eight lanes share one 4-bit group
// of 64 elements, whose 32 code bytes of neighbouring tokens are contiguous in the block.
#include "ts_rows.cuh"

namespace ts {
namespace {

// bf16 and fp32 pools: rows copied as they are, 16 bytes per thread, four under way. Bound by memory: 33,122 rows
// of 8 KV heads of 128, K and V: 50 us, 5.5 TB/s read and written in bf16 (16- and one-token pages alike), 91 us and
// 6.0 TB/s in fp32.
__global__ void __launch_bounds__(rows_threads(1)) append_rows_kernel(const __grid_constant__ RowsArgs a, int row_bytes) {
  __shared__ int64_t place[kRowsPerCta];
  place_rows(a, place);
  const int cpr = row_bytes / 16, per_row = 2 * a.HKV * cpr;
  const int64_t r0 = (int64_t)blockIdx.x * a.rows_per_cta;
  const int ps = 1 << a.page_shift;
#pragma unroll 4
  for (int i = threadIdx.x; i < per_row * a.rows_per_cta; i += blockDim.x) {
    const int row = i / per_row, rem = i % per_row, isv = rem >= a.HKV * cpr;
    const int c = rem - isv * a.HKV * cpr, g = c / cpr, ch = c % cpr;
    const int64_t at = place[row];
    if (at < 0) continue;
    const uint4 v = *reinterpret_cast<const uint4*>(a.src[isv] + (r0 + row) * a.src_stride[isv] + (size_t)c * 16);
    const int64_t page = at >> a.page_shift, slot = at & (ps - 1);
    *reinterpret_cast<uint4*>(a.pool[isv] + ((page * a.HKV + g) * ps + slot) * row_bytes + ch * 16) = v;
  }
}

// 4-bit pools (q4_quantise8).
//
// Measured: 33,122 rows of 8 KV heads of 128, K and V: 43 us, 4.0 TB/s, bound by issue (with the divisions
// throughout 104 us; eight loads under way in place of four 2 us more).
template <int NB, int ROWS>
__global__ void __launch_bounds__(rows_threads(ROWS)) append_q4_kernel(const __grid_constant__ RowsArgs a) {
  __shared__ int64_t place[kRowsPerCta];
  constexpr int D = NB * 64, BLK = q4_block_bytes(D), CODES = q4_code_bytes(D), COLS = rows_threads(ROWS) / 8 / ROWS;
  constexpr int BATCH = 4;               // loads under way per thread
  const int groups = a.HKV * NB, lane8 = threadIdx.x & 7;
  // neighbouring groups of eight lanes take neighbouring rows of the same 64 elements: their codes
  // are neighbours in the block
  const int row = (threadIdx.x >> 3) % ROWS;
  const int64_t r = (int64_t)blockIdx.x * ROWS + row;
  const unsigned peers = 0xffu << (threadIdx.x & 24);
  uint4 raw[BATCH];
  auto load = [&](int i0) {
#pragma unroll
    for (int k = 0; k < BATCH; ++k) {
      const int i = i0 + k * COLS, isv = i >= groups, c = isv ? i - groups : i;
      raw[k] = r < a.total && i < 2 * groups ? ldg_nc128(a.src[isv] + r * a.src_stride[isv] + c * 128 + lane8 * 16)
                                             : make_uint4(0u, 0u, 0u, 0u);
    }
  };
  const int first = (threadIdx.x >> 3) / ROWS;
  load(first);                           // on their way while the rows' places are looked up
  place_rows(a, place);
  const int64_t at = place[row];
  const int slot = (int)(at & 15);
  for (int i0 = first; i0 < 2 * groups; i0 += BATCH * COLS) {
    if (i0 != first) load(i0);
#pragma unroll
    for (int k = 0; k < BATCH; ++k) {
      const int i = i0 + k * COLS, isv = i >= groups, c = isv ? i - groups : i, g = c / NB, nb = c % NB;
      if (i >= 2 * groups) break;        // (the same in all eight lanes)
      __nv_bfloat16 sb;
      const uint32_t w = q4_quantise8(raw[k], peers, sb);
      if (at >= 0) {
        unsigned char* base = a.pool[isv] + ((at >> 4) * a.HKV + g) * BLK;
        *reinterpret_cast<uint32_t*>(base + nb * 512 + slot * 32 + lane8 * 4) = w;
        if (lane8 == 0) *reinterpret_cast<__nv_bfloat16*>(base + CODES + nb * 32 + slot * 2) = sb;
      }
    }
  }
}

// Rows of a pool as fp32 values: exact for every pool type (a code times a bf16 scale has 12
// significant bits). Eight threads to 64 elements of one row, thread l elements 4l .. 4l + 3 and 32 + 4l .. ,
// so that each of its two stores fills whole sectors with its neighbours'. Bound by the values written:
// 33,122 rows of 8 KV heads of 128: from a 4-bit pool 48 us, 6.4 TB/s, from a bf16 pool 66 us, 6.2 TB/s, from an
// fp32 pool 84 us, 6.4 TB/s.
template <int kType>
struct RawQuads;                         // the raw elements of one thread
template <>
struct RawQuads<TS_KV_Q4> {
  uint32_t lo, hi, scale;
};
template <>
struct RawQuads<TS_KV_BF16> {
  uint2 lo, hi;
};
template <>
struct RawQuads<TS_KV_F32> {
  float4 lo, hi;
};

template <int kType, int ROWS>
__global__ void __launch_bounds__(rows_threads(ROWS)) read_rows_kernel(const __grid_constant__ RowsArgs a) {
  __shared__ int64_t place[kRowsPerCta];
  place_rows(a, place);
  constexpr int COLS = rows_threads(ROWS) / 8 / ROWS, BATCH = 4;
  const int NB = a.D / 64, groups = a.HKV * NB, lane8 = threadIdx.x & 7, ps = 1 << a.page_shift;
  const int row = (threadIdx.x >> 3) % ROWS;
  const int64_t r = (int64_t)blockIdx.x * ROWS + row;
  const int64_t at = place[row];
  if (at < 0) return;
  const int64_t page = at >> a.page_shift;
  const int slot = (int)(at & (ps - 1));
  const int codes = q4_code_bytes(a.D), blk = q4_block_bytes(a.D), half = NB >> 1;   // NB is 1 or 2
  for (int i0 = (threadIdx.x >> 3) / ROWS; i0 < 2 * groups; i0 += BATCH * COLS) {
    RawQuads<kType> raw[BATCH];
#pragma unroll
    for (int k = 0; k < BATCH; ++k) {
      const int i = i0 + k * COLS, isv = i >= groups, c = isv ? i - groups : i, g = c >> half, nb = c & half;
      if (i >= 2 * groups) break;
      if constexpr (kType == TS_KV_Q4) {
        const unsigned char* base = a.pool[isv] + (page * a.HKV + g) * blk;
        const unsigned char* piece = base + nb * 512 + slot * 32 + lane8 * 2;
        raw[k].lo = *reinterpret_cast<const uint16_t*>(piece);
        raw[k].hi = *reinterpret_cast<const uint16_t*>(piece + 16);
        raw[k].scale = *reinterpret_cast<const uint16_t*>(base + codes + nb * 32 + slot * 2);
      } else {
        using Quad = decltype(raw[k].lo);
        constexpr int ES = kType == TS_KV_BF16 ? 2 : 4;
        const unsigned char* src = a.pool[isv] + (((page * a.HKV + g) * ps + slot) * a.D + nb * 64 + lane8 * 4) * ES;
        raw[k].lo = *reinterpret_cast<const Quad*>(src);
        raw[k].hi = *reinterpret_cast<const Quad*>(src + 32 * ES);
      }
    }
#pragma unroll
    for (int k = 0; k < BATCH; ++k) {
      const int i = i0 + k * COLS, isv = i >= groups, c = isv ? i - groups : i;
      if (i >= 2 * groups) break;
      float4 lo, hi;
      if constexpr (kType == TS_KV_Q4) {
        const float s = bf16_bits_f(raw[k].scale);
        auto value = [&](uint32_t w, int e) { return (float)((int)((w >> (4 * e)) & 15u) - 8) * s; };
        lo = make_float4(value(raw[k].lo, 0), value(raw[k].lo, 1), value(raw[k].lo, 2), value(raw[k].lo, 3));
        hi = make_float4(value(raw[k].hi, 0), value(raw[k].hi, 1), value(raw[k].hi, 2), value(raw[k].hi, 3));
      } else if constexpr (kType == TS_KV_BF16) {
        auto quad = [](uint2 w) {
          return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u), __uint_as_float(w.y << 16),
                             __uint_as_float(w.y & 0xffff0000u));
        };
        lo = quad(raw[k].lo);
        hi = quad(raw[k].hi);
      } else {
        lo = raw[k].lo;
        hi = raw[k].hi;
      }
      float* dst = a.dst[isv] + r * a.HKV * a.D + c * 64 + lane8 * 4;
      *reinterpret_cast<float4*>(dst) = lo;
      *reinterpret_cast<float4*>(dst + 32) = hi;
    }
  }
}

// Rows of kept drafts to the front of their draft (ts_keep_rows): row path[j] of the last T rows goes to row j, for
// every layer. Places ascend and path[j] >= j, so row j is never the source of a later row: a thread moves its 16 bytes
// (of one head, K or V) of the rows one after another, eight loads under way before their stores, and needs nobody
// else. Bytes move as they are, whatever the pool's type (4-bit scales are two bytes of a token: a thread each). Bound by
// latency: page, row in, row out: one layer of one sequence 5 us, 32 layers of 16 sequences 7 us.
constexpr int kKeepThreads = 128, kKeepRows = 128, kKeepBatch = 8;

struct KeepArgs {
  const int32_t* path;
  int64_t path_stride;
  const int32_t* count;
  const int32_t* cu;
  int B, total;
  const int32_t* seq_lens;
  const int32_t* page_table;
  int pt_stride, page_shift;
  int64_t num_pages;
  int max_tokens, HKV, D;
  unsigned char* pool[2];
  int64_t layer_bytes;
  int32_t* new_lens;           // or null
  int* status;
};

template <int kType>
__global__ void __launch_bounds__(kKeepThreads) keep_rows_kernel(const __grid_constant__ KeepArgs a) {
  __shared__ int64_t s_src[kKeepRows], s_dst[kKeepRows];
  const int b = blockIdx.x, tid = threadIdx.x;
  const bool lead = blockIdx.y == 0 && blockIdx.z == 0;          // the CTA that reports for its sequence
  const int32_t* path = a.path + b * a.path_stride;
  const int c0 = a.cu[b], T = a.cu[b + 1] - c0, n = a.seq_lens[b], count = a.count[b];
  int err = 0;
  if (c0 < 0 || T < 0 || c0 + (int64_t)T > a.total || (b == 0 && c0 != 0) || n < T || n > a.max_tokens)
    err = TS_ERR_SEQ_LEN;
  else if (count > a.path_stride)
    err = TS_ERR_CAPACITY;
  else if (count < 0 || count > T)
    err = TS_ERR_INVALID_ARG;
  if (!err) {
    bool bad = false;
    for (int j = tid; j < count; j += kKeepThreads) {
      const int at = path[j];
      bad |= at < j || at >= T || (j > 0 && at <= path[j - 1]);
    }
    if (__syncthreads_or(bad)) err = TS_ERR_INVALID_ARG;
  }
  if (lead && tid == 0) {
    if (err) set_error(a.status, err);
    if (a.new_lens) a.new_lens[b] = err ? n : n - T + count;
  }
  if (err) return;
  const int first = n - T, ps = 1 << a.page_shift;
  // this thread's piece of a row: K or V, head, 16 bytes of it (4-bit pools: then the scales, 2 bytes each)
  constexpr int ES = kType == TS_KV_F32 ? 4 : 2;
  const int pieces = kType == TS_KV_Q4 ? a.D / 32 + a.D / 64 : a.D * ES / 16;
  const int i = blockIdx.y * kKeepThreads + tid;
  const bool mine = i < 2 * a.HKV * pieces;
  const int isv = i / (a.HKV * pieces), g = i / pieces % a.HKV, piece = i % pieces;
  unsigned char* pool = a.pool[isv & 1] + blockIdx.z * a.layer_bytes;
  int64_t head;                                                  // bytes of a head in its page, of a token in it
  int token, off;
  if (kType == TS_KV_Q4) {
    head = q4_block_bytes(a.D);
    if (piece < a.D / 32) {
      token = 32;
      off = piece / 2 * 512 + piece % 2 * 16;
    } else {
      token = 2;
      off = q4_code_bytes(a.D) + (piece - a.D / 32) * 32;
    }
  } else {
    token = a.D * ES;
    head = (int64_t)ps * token;
    off = piece * 16;
  }
  const bool whole = kType != TS_KV_Q4 || token == 32;           // 16 bytes, else 2
  auto address = [&](int64_t place) {
    return pool + ((place >> a.page_shift) * a.HKV + g) * head + (place & (ps - 1)) * token + off;
  };
  for (int j0 = 0; j0 < count; j0 += kKeepRows) {
    const int rows = min(kKeepRows, count - j0);
    __syncthreads();
    for (int j = tid; j < rows; j += kKeepThreads) {
      int64_t place[2];
      for (int e = 0; e < 2; ++e) {
        const int pos = first + (e ? j0 + j : path[j0 + j]);
        const int page = a.page_table[(int64_t)b * a.pt_stride + (pos >> a.page_shift)];
        place[e] = page < 0 || page >= a.num_pages ? -1 : ((int64_t)page << a.page_shift) + (pos & (ps - 1));
      }
      const bool bad = place[0] < 0 || place[1] < 0;
      if (bad && lead) set_error(a.status, TS_ERR_PAGE_OOB);
      s_src[j] = bad || path[j0 + j] == j0 + j ? -1 : place[0];  // (a row that stays where it is)
      s_dst[j] = place[1];
    }
    __syncthreads();
    if (!mine) continue;
    for (int j = 0; j < rows; j += kKeepBatch) {
      uint4 v[kKeepBatch];
#pragma unroll
      for (int k = 0; k < kKeepBatch; ++k) {
        const int64_t src = j + k < rows ? s_src[j + k] : -1;
        if (src < 0) continue;
        if (whole)
          v[k] = *reinterpret_cast<const uint4*>(address(src));
        else
          v[k].x = *reinterpret_cast<const uint16_t*>(address(src));
      }
#pragma unroll
      for (int k = 0; k < kKeepBatch; ++k) {
        if (j + k >= rows || s_src[j + k] < 0) continue;
        if (whole)
          *reinterpret_cast<uint4*>(address(s_dst[j + k])) = v[k];
        else
          *reinterpret_cast<uint16_t*>(address(s_dst[j + k])) = (uint16_t)v[k].x;
      }
    }
  }
}

ts_status run_append(ts_ctx* ctx, const RowsArgs& a, cudaStream_t s) {
  const int grid = (a.total + a.rows_per_cta - 1) / a.rows_per_cta;
  ctx->kernels += 1;
#define TS_APPEND_Q4(NB_, ROWS_) \
  if (a.D == 64 * NB_ && a.rows_per_cta == ROWS_) append_q4_kernel<NB_, ROWS_><<<grid, rows_threads(ROWS_), 0, s>>>(a);
  if (ctx->cfg.kv_dtype == TS_KV_Q4) {
    TS_APPEND_Q4(1, 1) TS_APPEND_Q4(1, kRowsPerCta) TS_APPEND_Q4(2, 1) TS_APPEND_Q4(2, kRowsPerCta)
  } else
#undef TS_APPEND_Q4
    append_rows_kernel<<<grid, rows_threads(a.rows_per_cta), 0, s>>>(a, a.D * (ctx->cfg.kv_dtype == TS_KV_BF16 ? 2 : 4));
  return cuda_status(cudaGetLastError());
}

}  // namespace

ts_status launch_append_q4(ts_ctx* ctx, const void* k_new, const void* v_new, const int32_t* page_table,
                           const int32_t* seq_lens, int B, void* k_pool, void* v_pool, cudaStream_t s) {
  RowsArgs a = rows_args(ctx, B, B, page_table, k_pool, v_pool);
  a.seq_lens = seq_lens;
  a.src[0] = static_cast<const unsigned char*>(k_new);
  a.src[1] = static_cast<const unsigned char*>(v_new);
  a.src_stride[0] = a.src_stride[1] = (int64_t)a.HKV * a.D * 2;
  return run_append(ctx, a, s);
}

ts_status launch_append_prompt(ts_ctx* ctx, const AppendPromptCall& c, cudaStream_t s) {
  if (c.total == 0) return TS_OK;
  RowsArgs a = rows_args(ctx, c.B, c.total, c.page_table, c.k_pool, c.v_pool);
  const int64_t es = ctx->cfg.kv_dtype == TS_KV_F32 ? 4 : 2;
  a.cu = c.cu_rows;
  a.starts = c.starts;
  a.src[0] = static_cast<const unsigned char*>(c.k);
  a.src[1] = static_cast<const unsigned char*>(c.v);
  a.src_stride[0] = c.k_stride * es;
  a.src_stride[1] = c.v_stride * es;
  return run_append(ctx, a, s);
}

ts_status launch_read_kv(ts_ctx* ctx, const int32_t* cu_rows, const int32_t* starts, int B, int total,
                         const int32_t* page_table, const void* k_pool, const void* v_pool, float* k_out, float* v_out,
                         cudaStream_t s) {
  if (total == 0) return TS_OK;
  RowsArgs a = rows_args(ctx, B, total, page_table, const_cast<void*>(k_pool), const_cast<void*>(v_pool));
  a.cu = cu_rows;
  a.starts = starts;
  a.dst[0] = k_out;
  a.dst[1] = v_out;
  const int grid = (total + a.rows_per_cta - 1) / a.rows_per_cta;
  ctx->kernels += 1;
#define TS_READ_ROWS(TYPE_, ROWS_)                                      \
  if (ctx->cfg.kv_dtype == TYPE_ && a.rows_per_cta == ROWS_) \
    read_rows_kernel<TYPE_, ROWS_><<<grid, rows_threads(ROWS_), 0, s>>>(a);
  TS_READ_ROWS(TS_KV_Q4, 1) TS_READ_ROWS(TS_KV_Q4, kRowsPerCta)
  TS_READ_ROWS(TS_KV_BF16, 1) TS_READ_ROWS(TS_KV_BF16, kRowsPerCta)
  TS_READ_ROWS(TS_KV_F32, 1) TS_READ_ROWS(TS_KV_F32, kRowsPerCta)
#undef TS_READ_ROWS
  return cuda_status(cudaGetLastError());
}

ts_status launch_keep_rows(ts_ctx* ctx, const KeepCall& c, cudaStream_t s) {
  const ts_config& cfg = ctx->cfg;
  KeepArgs a{c.path, c.path_stride, c.count, c.cu_rows, c.B, c.total, c.seq_lens, c.page_table, cfg.max_pages_per_seq,
             ctx->page_shift, cfg.num_pages, ctx->max_tokens, cfg.n_kv_heads, cfg.head_dim,
             {static_cast<unsigned char*>(c.k_pool), static_cast<unsigned char*>(c.v_pool)}, c.layer_bytes, c.new_lens,
             ctx->status};
  const int d = cfg.head_dim;
  const int pieces = 2 * cfg.n_kv_heads * (cfg.kv_dtype == TS_KV_Q4 ? d / 32 + d / 64 : d * (cfg.kv_dtype == TS_KV_F32 ? 4 : 2) / 16);
  const dim3 grid(c.B, (pieces + kKeepThreads - 1) / kKeepThreads, c.layers);
  ctx->kernels += 1;
  switch (cfg.kv_dtype) {
    case TS_KV_F32: keep_rows_kernel<TS_KV_F32><<<grid, kKeepThreads, 0, s>>>(a); break;
    case TS_KV_BF16: keep_rows_kernel<TS_KV_BF16><<<grid, kKeepThreads, 0, s>>>(a); break;
    default: keep_rows_kernel<TS_KV_Q4><<<grid, kKeepThreads, 0, s>>>(a);
  }
  return cuda_status(cudaGetLastError());
}

}  // namespace ts
