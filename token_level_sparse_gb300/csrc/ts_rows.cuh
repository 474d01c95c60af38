// What the kernels share that move rows into and out of the paged pools: where packed rows go, and the
// quantisation of a row's 64 elements.
#pragma once

#include "ts_q4.cuh"

namespace ts {

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
__device__ __forceinline__ uint32_t q4_quantise8(const uint4& raw, unsigned peers, __nv_bfloat16& sb) {
  const uint32_t in[4] = {raw.x, raw.y, raw.z, raw.w};
  // the largest magnitude by its bits, two at a time: ordered like the values, with infinities and NaN on top
  uint32_t mb = 0u;
#pragma unroll
  for (int e = 0; e < 4; ++e) mb = __vmaxu2(mb, in[e] & 0x7fff7fffu);
#pragma unroll
  for (int d = 4; d >= 1; d >>= 1) mb = __vmaxu2(mb, __shfl_xor_sync(peers, mb, d));
  const float top = bf16_bits_f(max(mb & 0xffffu, mb >> 16));
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
  return w;
}

inline RowsArgs rows_args(ts_ctx* ctx, int B, int total, const int32_t* page_table, void* k_pool, void* v_pool) {
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

}  // namespace ts
