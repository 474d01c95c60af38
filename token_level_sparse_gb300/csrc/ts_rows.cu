// Rows into and out of the paged pools: packed K and V rows of whole prompts (ts_append_prompt),
// one token per sequence into a 4-bit pool (ts_append_kv), and rows read back as fp32 values
// (ts_read_kv).
//
// Packed row r belongs to sequence b with cu[b] <= r < cu[b + 1] and goes to position
// starts[b] + r - cu[b]. A CTA takes a few neighbouring rows: it looks up their page and slot once,
// then its threads move 16 bytes (or, into and out of 4-bit blocks, 8 elements) each. Every byte is
// read and written once, so the copies are bound by memory; eight lanes share one 4-bit group
// of 64 elements, whose 32 code bytes of neighbouring tokens are contiguous in the block.
#include "ts_q4.cuh"

namespace ts {
namespace {

// Rows of a CTA: four, whose codes are 128 contiguous bytes, or one where there are few rows, so that a decode
// step's rows do not queue behind one another. 33,122 rows written and read back: 89.5 us with four rows
// and 128 threads, 92.5 with 64 threads, 94.7 with 16 rows and 256 threads, 120 with two rows. Eight rows, one to a
// CTA, written and read back: 4.6 us with 256 threads, 4.8 with 128.
constexpr int kRowsPerCta = 4;
__host__ __device__ constexpr int rows_threads(int rows) { return rows == 1 ? 256 : 128; }

struct RowsArgs {
  const int32_t* cu;           // [B + 1]; null: one row per sequence, at position seq_lens[b] - 1
  const int32_t* starts;       // [B] or null (0)
  const int32_t* seq_lens;     // with cu == null
  int B, total, rows_per_cta;
  const int32_t* page_table;
  int pt_stride, page_shift;
  int64_t num_pages;
  int max_tokens;
  int HKV, D;
  const unsigned char* src[2]; // K and V rows, bytes
  int64_t src_stride[2];       // bytes between rows
  unsigned char* pool[2];
  float* dst[2];               // ts_read_kv: [total][H_kv][d]
  int* status;
};

// Place of the CTA's rows: page * page size + slot, or -1 (no such position; recorded).
__device__ __forceinline__ void place_rows(const RowsArgs& a, int64_t* place) {
  // the boundaries of up to 256 sequences in shared memory: one read instead of one per step of the search
  __shared__ int32_t s_cu[257];
  const int32_t* cu = a.cu;
  if (a.cu && a.B <= 256) {
    for (int b = threadIdx.x; b <= a.B; b += blockDim.x) s_cu[b] = a.cu[b];
    __syncthreads();
    cu = s_cu;
  }
  if (a.cu && blockIdx.x == 0) {
    // the boundaries: ascending, from 0, within the rows that there are
    for (int b = threadIdx.x; b <= a.B; b += blockDim.x) {
      const int v = cu[b];
      if (v > a.total || (b == 0 ? v != 0 : v < cu[b - 1])) set_error(a.status, TS_ERR_SEQ_LEN);
    }
  }
  if ((int)threadIdx.x < a.rows_per_cta) {
    const int64_t r = (int64_t)blockIdx.x * a.rows_per_cta + threadIdx.x;
    int64_t at = -1;
    if (r < a.total) {
      int b = (int)r;
      int64_t pos = -1;
      bool inside = true;
      if (a.cu) {
        int lo = 0, hi = a.B;              // the last b with cu[b] <= r
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (cu[mid] <= r) lo = mid; else hi = mid;
        }
        b = lo;
        // rows behind the last sequence stay as they are, so do those of one that ends beyond the rows
        inside = cu[b] >= 0 && r >= cu[b] && r < cu[b + 1] && cu[b + 1] <= a.total;
        const int start = a.starts ? a.starts[b] : 0;
        pos = start < 0 ? -1 : start + (r - cu[b]);
      } else {
        pos = (int64_t)a.seq_lens[b] - 1;
      }
      if (inside) {
        if (pos < 0 || pos >= a.max_tokens) {
          set_error(a.status, TS_ERR_SEQ_LEN);
        } else {
          const int page = a.page_table[(size_t)b * a.pt_stride + (pos >> a.page_shift)];
          if (page < 0 || (int64_t)page >= a.num_pages)
            set_error(a.status, TS_ERR_PAGE_OOB);
          else
            at = ((int64_t)page << a.page_shift) + (pos & ((1 << a.page_shift) - 1));
        }
      }
    }
    place[threadIdx.x] = at;
  }
  __syncthreads();
}

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

// 4-bit pools. Eight lanes quantise one group of 64 elements: scale = bf16(max|x| / 7), code =
// 8 + round(x / scale), ties to even. A scale of zero gives zeros; a group with a NaN or an infinity
// reads back as NaN: its scale is not finite and its codes stand for zero.
//
// The bits are those of exact arithmetic, without a division: x and the scale s have 8 significant bits
// each, so a quotient that is not halfway between two codes is at least 2^-9 away from it (numerator
// and denominator of the difference are whole numbers below 2^9 of one unit), and likewise max|x| / 7
// lies 2^-12 away from any midpoint of bf16. A product with 1/7 that is right to 2^-22 therefore rounds
// to the right scale. A quotient x r, r near 1/s, is off by less than 2^-19, and is rounded twice: to a
// multiple of 2^-10 (by a sum with 1.5 2^13), which makes a quotient halfway between codes exact and leaves
// every other one on its side of halfway, then to a whole number, ties to even (by a sum with 1.5 2^23).
// Scales near or below the smallest normal number have fewer bits and take the divisions instead.
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
      const uint32_t in[4] = {raw[k].x, raw[k].y, raw[k].z, raw[k].w};
      // the largest magnitude by its bits, two at a time: ordered like the values, with infinities and NaN on top
      uint32_t mb = 0u;
#pragma unroll
      for (int e = 0; e < 4; ++e) mb = __vmaxu2(mb, in[e] & 0x7fff7fffu);
#pragma unroll
      for (int d = 4; d >= 1; d >>= 1) mb = __vmaxu2(mb, __shfl_xor_sync(peers, mb, d));
      const float top = bf16_bits_f(max(mb & 0xffffu, mb >> 16));
      __nv_bfloat16 sb;
      uint32_t w;
      if (top >= 0x1p-100f && top < INFINITY) {
        sb = __float2bfloat16_rn(top * (1.f / 7.f));
        const float s = __bfloat162float(sb);
        float rs;
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(rs) : "f"(s));
        const uint64_t r2 = pack_f2(rs, rs), fine = pack_f2(12288.f, 12288.f),
                       whole = pack_f2(12582920.f - 12288.f, 12582920.f - 12288.f), one = pack_f2(1.f, 1.f);
        uint32_t u[4];                   // two codes in the low byte
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint64_t x = pack_f2(__uint_as_float(in[e] << 16), __uint_as_float(in[e] & 0xffff0000u));
          // 1.5 2^23 + 8 + the rounded quotient: the code in the low byte, since |q| < 7.1 (s >= top / 7 (1 - 2^-8))
          float lo, hi;
          unpack_f2(fma_f2(fma_f2(x, r2, fine), one, whole), lo, hi);
          u[e] = __float_as_uint(hi) * 16u + __float_as_uint(lo);
        }
        w = __byte_perm(__byte_perm(u[0], u[1], 0x0040), __byte_perm(u[2], u[3], 0x0040), 0x5410);
      } else {
        sb = __float2bfloat16_rn(__fdiv_rn(top, 7.f));
        const float s = __bfloat162float(sb);
        const bool live = s > 0.f && s < INFINITY;
        w = 0u;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float x = __uint_as_float(e & 1 ? in[e >> 1] & 0xffff0000u : in[e >> 1] << 16);
          const int q = live ? max(-7, min(7, __float2int_rn(__fdiv_rn(x, s)))) : 0;
          w |= (uint32_t)(q + 8) << (4 * e);
        }
      }
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

RowsArgs base_args(ts_ctx* ctx, int B, int total, const int32_t* page_table, void* k_pool, void* v_pool) {
  const ts_config& c = ctx->cfg;
  RowsArgs a{};
  a.B = B;
  a.total = total;
  a.rows_per_cta = total >= 2 * ctx->num_sms ? kRowsPerCta : 1;
  a.page_table = page_table;
  a.pt_stride = c.max_pages_per_seq;
  a.page_shift = ctx->page_shift;
  a.num_pages = c.num_pages;
  a.max_tokens = ctx->max_tokens;
  a.HKV = c.n_kv_heads;
  a.D = c.head_dim;
  a.pool[0] = static_cast<unsigned char*>(k_pool);
  a.pool[1] = static_cast<unsigned char*>(v_pool);
  a.status = ctx->status;
  return a;
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
  RowsArgs a = base_args(ctx, B, B, page_table, k_pool, v_pool);
  a.seq_lens = seq_lens;
  a.src[0] = static_cast<const unsigned char*>(k_new);
  a.src[1] = static_cast<const unsigned char*>(v_new);
  a.src_stride[0] = a.src_stride[1] = (int64_t)a.HKV * a.D * 2;
  return run_append(ctx, a, s);
}

ts_status launch_append_prompt(ts_ctx* ctx, const AppendPromptCall& c, cudaStream_t s) {
  if (c.total == 0) return TS_OK;
  RowsArgs a = base_args(ctx, c.B, c.total, c.page_table, c.k_pool, c.v_pool);
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
  RowsArgs a = base_args(ctx, B, total, page_table, const_cast<void*>(k_pool), const_cast<void*>(v_pool));
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

}  // namespace ts
