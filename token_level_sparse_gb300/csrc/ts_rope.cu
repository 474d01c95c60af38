// Rotary positions: rows of heads turned by their positions (ts_rotate), and K rows turned on their way into the
// paged pools, with V beside them and the queries of the same rows (ts_append_rotated).
//
//   y1 = a (x1 cos t - x2 sin t),   y2 = a (x2 cos t + x1 sin t),   t = pos f_i
//
// for the r/2 pairs of the first r elements of a head: (i, i + r/2), or (2i, 2i + 1). The rest of a head passes as it is.
//
// Angles: f_i / 2pi is held as a 64-bit fraction of a turn, and pos times it, modulo 2^64, is the angle modulo a turn,
// exactly: far positions cost nothing and lose nothing (fp32 products of a position near 10^6 are off by up to 0.03
// radians), and negative positions turn back. The top 32 bits (2^-32 of a turn is
// cut off) go to sincospif as one fp32 number, whose rounding is what is left: up to 2^-26 of a turn, near half a turn.
//
// Every byte is read and written once, so this is bound by memory. A thread holds 8 elements of a head (16 bytes of
// bf16), the same 8 of one row for all the heads that it goes through, so that their cosines and sines stay in
// registers. The other half of its pairs is in its own 8 elements (neighbouring pairs), or in those of another lane of
// the head's 8 or 16 (pairs r/2 apart): a shuffle where r/2 is a multiple of 8, else single elements through shared memory.
// A head lies inside one warp, which has read all of it before it writes: rows may be turned in place.
//
// Measured, bf16, heads of 128: 33,122 rows of 32 heads turned 92 us, 5.9 TB/s read and written; the same rows with K and V of 8
// heads appended 137 us, 5.9 TB/s; eight single rows 4.5 and 8 us on the device (look-ups, one after another).
#include <cmath>
#include <new>

#include "ts_rows.cuh"

namespace ts {
namespace {

// Threads of a CTA, for four rows or (few rows) one. 33,122 rows of 32 heads of 128, bf16 in and out: 92.7 us with 64 threads,
// 12 CTAs to an SM and the next heads loaded before these are turned; 96 with 128 threads and 6 CTAs, 121 with 256; 156 without the
// loads ahead.
__host__ __device__ constexpr int rope_threads(int rows) { return rows == 1 ? 256 : 64; }
__host__ __device__ constexpr int rope_ctas(int rows) { return rows == 1 ? 2 : 12; }

struct RopeArgs {
  RowsArgs rows;                   // places of the rows, pools (src and dst: K and V rows); total
  const int32_t* positions;
  const unsigned char* q;          // rows that are turned and written to q_out; null: none
  int64_t q_stride;                // bytes
  unsigned char* q_out;
  int64_t q_out_stride;            // bytes
  int q_heads, q_out_f32;
  int r, pairs;                    // elements turned; neighbouring pairs
  float factor;
  uint64_t turns[64];              // f_i / 2pi as a fraction of 2^64
};

__device__ __forceinline__ uint4 shfl4(const uint4& v, int from) {
  return make_uint4(__shfl_sync(kFull, v.x, from), __shfl_sync(kFull, v.y, from), __shfl_sync(kFull, v.z, from),
                    __shfl_sync(kFull, v.w, from));
}

// 8 elements of a row, as they are
template <typename T>
struct Raw8;
template <>
struct Raw8<__nv_bfloat16> {
  uint4 a;
  __device__ __forceinline__ void load(const unsigned char* p) { a = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void get(float (&x)[8]) const { KV<__nv_bfloat16>::unpack(a, x); }
  // those of lane `from`
  __device__ __forceinline__ Raw8 of(int from) const {
    Raw8 o;
    o.a = shfl4(a, from);
    return o;
  }
};
template <>
struct Raw8<float> {
  uint4 a, b;
  __device__ __forceinline__ void load(const unsigned char* p) {
    a = *reinterpret_cast<const uint4*>(p);
    b = *reinterpret_cast<const uint4*>(p + 16);
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    KV<float>::unpack(a, x);
    KV<float>::unpack(b, x + 4);
  }
  __device__ __forceinline__ Raw8 of(int from) const {
    Raw8 o;
    o.a = shfl4(a, from);
    o.b = shfl4(b, from);
    return o;
  }
};

__device__ __forceinline__ uint4 to_bf16(const float (&x)[8]) {
  return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
}

__device__ __forceinline__ void store_f32(unsigned char* p, const float (&x)[8]) {
  *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
  *reinterpret_cast<float4*>(p + 16) = make_float4(x[4], x[5], x[6], x[7]);
}

// kPairs 0: neighbours; 1: r/2 apart, a multiple of 8; 2: r/2 apart, any
template <typename T, int D, int ROWS, int kPairs, bool kQ4>
__global__ void __launch_bounds__(rope_threads(ROWS), rope_ctas(ROWS)) rope_kernel(const __grid_constant__ RopeArgs a) {
  constexpr int ES = (int)sizeof(T), THREADS = rope_threads(ROWS);
  constexpr int CPR = D / 8, GROUPS = THREADS / CPR;              // lanes of a head; heads at once
  constexpr int BATCH = ES == 4 || kQ4 ? 2 : 4;                   // heads under way, and as many ahead (more spills)
  static_assert(GROUPS % ROWS == 0 && 32 % CPR == 0, "a head in a warp, a row to a thread");
  __shared__ int64_t s_place[kRowsPerCta];
  __shared__ float s_cos[ROWS][64], s_sin[ROWS][64];
  __shared__ float s_x[kPairs == 2 ? THREADS * 8 : 1];
  const int tid = threadIdx.x, c = tid % CPR, grp = tid / CPR, row = grp % ROWS, half = a.r / 2;
  const int64_t r = (int64_t)blockIdx.x * ROWS + row;
  const bool live = r < a.rows.total;
  const bool into = a.rows.pool[0] != nullptr;
  const int n_kv = into ? a.rows.HKV : 0, n_q = a.q ? a.q_heads : 0, n = 2 * n_kv + n_q;
  constexpr int STEP = GROUPS / ROWS;

  auto source = [&](int h) -> const unsigned char* {
    if (h < n_q) return a.q + r * a.q_stride + ((int64_t)h * D + c * 8) * ES;
    h -= n_q;
    const int isv = h >= n_kv;
    return a.rows.src[isv] + r * a.rows.src_stride[isv] + ((int64_t)(h - isv * n_kv) * D + c * 8) * ES;
  };
  Raw8<T> raw[BATCH], next[BATCH];
  auto load = [&](int h0, Raw8<T> (&to)[BATCH]) {
#pragma unroll
    for (int k = 0; k < BATCH; ++k)
      if (live && h0 + k * STEP < n) to[k].load(source(h0 + k * STEP));
  };
  load(grp / ROWS, raw);           // on their way while angles and places are found

  for (int i = tid; i < ROWS * half; i += THREADS) {
    const int rr = i / half, p = i - rr * half;
    const int64_t at = (int64_t)blockIdx.x * ROWS + rr;
    if (at < a.rows.total) {
      const uint64_t turn = (uint64_t)(int64_t)a.positions[at] * a.turns[p];
      float sn, cs;
      sincospif((float)(int32_t)(turn >> 32) * 0x1p-31f, &sn, &cs);
      s_cos[rr][p] = cs * a.factor;
      s_sin[rr][p] = sn * a.factor;
    }
  }
  int64_t place = -1;
  if (into) {
    place_rows(a.rows, s_place);   // (ends with a barrier)
    place = s_place[row];
  } else {
    __syncthreads();
  }
  // this thread's cosines and signed sines: y = x cs + partner sn; elements behind r: 1 and 0
  float cs[8], sn[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int i = c * 8 + e;
    cs[e] = 1.f;
    sn[e] = 0.f;
    if (i < a.r) {
      const int p = kPairs == 0 ? i >> 1 : (i < half ? i : i - half);
      const float s = s_sin[row][p];
      cs[e] = s_cos[row][p];
      sn[e] = kPairs == 0 ? (e & 1 ? s : -s) : (i < half ? -s : s);
    }
  }
  const int64_t page = place >> a.rows.page_shift;
  const int ps = 1 << a.rows.page_shift, slot = (int)(place & (ps - 1));
  for (int h0 = grp / ROWS; h0 - grp / ROWS < n; h0 += BATCH * STEP) {     // (the same count in every thread)
    load(h0 + BATCH * STEP, next);
#pragma unroll
    for (int k = 0; k < BATCH; ++k) {
      const int h = h0 + k * STEP;
      const bool have = live && h < n;
      const bool is_q = h < n_q;
      const int hk = h - n_q, isv = hk >= n_kv, g = hk - (isv ? n_kv : 0);
      float x[8] = {}, y[8];
      if (have) raw[k].get(x);
      if (kPairs == 0) {
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = fmaf(x[e ^ 1], sn[e], x[e] * cs[e]);
      } else if (kPairs == 1) {
        // (what lanes behind r make of this is not used)
        float other[8];
        raw[k].of((tid & 31) + (c * 8 < half ? half / 8 : (c * 8 < a.r ? -half / 8 : 0))).get(other);
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = fmaf(other[e], sn[e], x[e] * cs[e]);
      } else {
        float* mine = s_x + tid * 8;
        __syncwarp();
#pragma unroll
        for (int e = 0; e < 8; ++e) mine[e] = x[e];
        __syncwarp();
        const float* head = s_x + (tid - c) * 8;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int i = c * 8 + e;
          const float other = i < a.r ? head[i < half ? i + half : i - half] : 0.f;
          y[e] = fmaf(other, sn[e], x[e] * cs[e]);
        }
      }
      // what is not turned keeps its bits: elements behind r, and V
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (c * 8 + e >= a.r || (!is_q && isv)) y[e] = x[e];
      if (is_q) {
        if (have) {
          unsigned char* out = a.q_out + r * a.q_out_stride + ((int64_t)h * D + c * 8) * (a.q_out_f32 ? 4 : 2);
          if (a.q_out_f32)
            store_f32(out, y);
          else
            *reinterpret_cast<uint4*>(out) = to_bf16(y);
        }
      } else if constexpr (kQ4) {
        __nv_bfloat16 sb;
        const uint32_t w = q4_quantise8(to_bf16(y), 0xffu << (tid & 24), sb);
        if (have && place >= 0) {
          const int nb = c >> 3;
          unsigned char* base = a.rows.pool[isv] + (page * a.rows.HKV + g) * q4_block_bytes(D);
          *reinterpret_cast<uint32_t*>(base + nb * 512 + slot * 32 + (c & 7) * 4) = w;
          if ((c & 7) == 0) *reinterpret_cast<__nv_bfloat16*>(base + q4_code_bytes(D) + nb * 32 + slot * 2) = sb;
        }
      } else if (have && place >= 0) {
        unsigned char* out = a.rows.pool[isv] + (((page * a.rows.HKV + g) * ps + slot) * D + c * 8) * ES;
        if constexpr (ES == 4)
          store_f32(out, y);
        else
          *reinterpret_cast<uint4*>(out) = isv ? raw[k].a : to_bf16(y);
      }
    }
#pragma unroll
    for (int k = 0; k < BATCH; ++k) raw[k] = next[k];
  }
}

template <typename T, int D, int ROWS, bool kQ4>
void pick(const RopeArgs& a, int grid, cudaStream_t s) {
  if (a.pairs)
    rope_kernel<T, D, ROWS, 0, kQ4><<<grid, rope_threads(ROWS), 0, s>>>(a);
  else if (a.r % 16 == 0)
    rope_kernel<T, D, ROWS, 1, kQ4><<<grid, rope_threads(ROWS), 0, s>>>(a);
  else
    rope_kernel<T, D, ROWS, 2, kQ4><<<grid, rope_threads(ROWS), 0, s>>>(a);
}

template <typename T, bool kQ4>
ts_status run_rope(ts_ctx* ctx, const RopeArgs& a, cudaStream_t s) {
  const int rows = a.rows.rows_per_cta, grid = (a.rows.total + rows - 1) / rows;
  ctx->kernels += 1;
  if (a.rows.D == 64) {
    if (rows == 1) pick<T, 64, 1, kQ4>(a, grid, s); else pick<T, 64, kRowsPerCta, kQ4>(a, grid, s);
  } else {
    if (rows == 1) pick<T, 128, 1, kQ4>(a, grid, s); else pick<T, 128, kRowsPerCta, kQ4>(a, grid, s);
  }
  return cuda_status(cudaGetLastError());
}

void set_rope(RopeArgs& a, const ts_rope* rope) {
  a.r = rope->rot_dim;
  a.pairs = rope->interleaved;
  a.factor = rope->factor;
  for (int i = 0; i < 64; ++i) a.turns[i] = rope->turns[i];
}

}  // namespace

ts_status launch_rotate(ts_ctx* ctx, const ts_rope* rope, const RotateCall& c, cudaStream_t s) {
  if (c.total == 0) return TS_OK;
  RopeArgs a{};
  a.rows = rows_args(ctx, 1, c.total, nullptr, nullptr, nullptr);
  a.positions = c.positions;
  const int64_t es = c.dtype == TS_KV_F32 ? 4 : 2, eo = c.out_dtype == TS_KV_F32 ? 4 : 2;
  a.q = static_cast<const unsigned char*>(c.x);
  a.q_stride = c.stride * es;
  a.q_out = static_cast<unsigned char*>(c.out);
  a.q_out_stride = c.out_stride * eo;
  a.q_heads = c.heads;
  a.q_out_f32 = c.out_dtype == TS_KV_F32;
  set_rope(a, rope);
  return c.dtype == TS_KV_F32 ? run_rope<float, false>(ctx, a, s) : run_rope<__nv_bfloat16, false>(ctx, a, s);
}

ts_status launch_append_rotated(ts_ctx* ctx, const ts_rope* rope, const AppendPromptCall& c, const RotateCall& q,
                                cudaStream_t s) {
  if (c.total == 0) return TS_OK;
  RopeArgs a{};
  a.rows = rows_args(ctx, c.B, c.total, c.page_table, c.k_pool, c.v_pool);
  const int64_t es = ctx->cfg.kv_dtype == TS_KV_F32 ? 4 : 2;
  a.rows.cu = c.cu_rows;
  a.rows.starts = c.starts;
  a.rows.src[0] = static_cast<const unsigned char*>(c.k);
  a.rows.src[1] = static_cast<const unsigned char*>(c.v);
  a.rows.src_stride[0] = c.k_stride * es;
  a.rows.src_stride[1] = c.v_stride * es;
  a.positions = q.positions;
  a.q = static_cast<const unsigned char*>(q.x);
  a.q_stride = q.stride * es;
  a.q_out = static_cast<unsigned char*>(q.out);
  a.q_out_stride = q.out_stride * (q.out_dtype == TS_KV_F32 ? 4 : 2);
  a.q_heads = ctx->cfg.n_q_heads;
  a.q_out_f32 = q.out_dtype == TS_KV_F32;
  set_rope(a, rope);
  switch (ctx->cfg.kv_dtype) {
    case TS_KV_F32: return run_rope<float, false>(ctx, a, s);
    case TS_KV_BF16: return run_rope<__nv_bfloat16, false>(ctx, a, s);
    default: return run_rope<__nv_bfloat16, true>(ctx, a, s);
  }
}

}  // namespace ts
