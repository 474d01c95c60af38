// The 4-bit paged cache: block format, code arithmetic and the tensor-core pieces that the
// score and the attention over it share.
//
// One (page, KV head) block holds 16 rows of d elements:
//   codes  [d/64][16 tokens][32 bytes]   byte j: element 2j in the low half, 2j + 1 in the high
//   scales [d/64][16 tokens] bf16
// so 16 (d/2 + d/32) bytes, a multiple of 16 (1088 at d = 128). A code u stands for (u - 8) s with
// the scale s of its 64 elements. The 32-byte pieces of one token are the pieces a warp reads:
//  * scores: lane (g, t) takes bytes 8t .. 8t + 7 of token g, so 8 tokens x 4 lanes are 256
//    contiguous bytes;
//  * outputs: lane (g, t) takes word g of token t, so 4 tokens x 8 lanes are 128 contiguous bytes.
//
// Both products run as m16n8k16 with the query heads as the 16 rows: rows 0..7 hold the high part
// of 8 heads' queries (or weights) and rows 8..15 the low part of the same heads, so one
// instruction takes both parts of a split fp32 operand and a lane adds the two results it already
// holds. Codes are exact in fp16 and bf16, their products with either part are exact in fp32.
#pragma once

#include <cuda_fp16.h>

#include "ts_common.cuh"

namespace ts {

constexpr int kQ4Group = 64;   // elements that share a scale

__host__ __device__ constexpr int q4_code_bytes(int d) { return kPage * d / 2; }
__host__ __device__ constexpr int q4_block_bytes(int d) { return kPage * (d / 2 + d / 32); }

// D (16x8, fp32) += A (16x16) B (16x8): lane (g = lane / 4, t = lane % 4) holds A rows g, g + 8 and
// D rows g, g + 8 at columns 2t, 2t + 1, and column g of B.
__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t h2_bits(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }
__device__ __forceinline__ uint32_t b2_bits(__nv_bfloat162 h) { return *reinterpret_cast<uint32_t*>(&h); }
__device__ __forceinline__ __half2 bits_h2(uint32_t u) { return *reinterpret_cast<__half2*>(&u); }
__device__ __forceinline__ __nv_bfloat162 bits_b2(uint32_t u) { return *reinterpret_cast<__nv_bfloat162*>(&u); }
__device__ __forceinline__ float bf16_bits_f(uint32_t u) { return __uint_as_float(u << 16); }

// (x & m) | k in one instruction
__device__ __forceinline__ uint32_t and_or(uint32_t x, uint32_t m, uint32_t k) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(x), "r"(m), "r"(k));
  return r;
}

// The eight codes of a word as four fp16 pairs, pair i = codes (i, i + 4), each minus 8, exactly:
// a code in the low mantissa bits of 1024 is 1024 + u, four bits higher it is 1024 + 16 u.
__device__ __forceinline__ void q4_pairs_f16(uint32_t w, uint32_t (&p)[4]) {
  const __half2 m1032 = __half2half2(__ushort_as_half(0xe408));            // -1032
  const __half2 r16 = __half2half2(__ushort_as_half(0x2c00));              // 1 / 16
  const __half2 m72 = __half2half2(__ushort_as_half(0xd480));              // -(1024 / 16 + 8)
  const uint32_t h = w >> 8;
  p[0] = h2_bits(__hadd2(bits_h2(and_or(w, 0x000f000fu, 0x64006400u)), m1032));
  p[1] = h2_bits(__hfma2(bits_h2(and_or(w, 0x00f000f0u, 0x64006400u)), r16, m72));
  p[2] = h2_bits(__hadd2(bits_h2(and_or(h, 0x000f000fu, 0x64006400u)), m1032));
  p[3] = h2_bits(__hfma2(bits_h2(and_or(h, 0x00f000f0u, 0x64006400u)), r16, m72));
}

// Codes j of two words of four codes each (one token in the low half, one in the high), minus 8, as
// a bf16 pair: a code in the low mantissa bits of 128 is 128 + u.
__device__ __forceinline__ uint32_t q4_pair_bf16(uint32_t ab, int j) {
  const __nv_bfloat162 m136 = bits_b2(0xc308c308u);                        // -136
  return b2_bits(__hadd2(bits_b2(and_or(ab >> (4 * j), 0x000f000fu, 0x43004300u)), m136));
}

// The queries of up to 8 heads as the A operand of the scores: element pairs in the order that
// q4_pairs_f16 gives the codes. A head's queries are scaled by a power of two so that the largest
// lies in [2^14, 2^15), then split into two fp16 terms (hi + lo within 2^-22 of the largest
// relative to it); inv undoes the scaling.
template <int NB>
struct Q4Query {
  uint32_t a[NB][4][4];
  float inv;
};

template <int NB>
__device__ __forceinline__ void q4_load_query(Q4Query<NB>& f, const float* q, bool live, int t) {
  float x[NB][16];
  float mx = 0.f;
#pragma unroll
  for (int nb = 0; nb < NB; ++nb)
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      x[nb][i] = live ? q[nb * 64 + 16 * t + i] : 0.f;
      mx = fmaxf(mx, fabsf(x[nb][i]));
    }
  mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 1));
  mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 2));
  const int ex = (int)(__float_as_uint(mx) >> 23) - 127;                   // mx < 2^(ex + 1)
  const int sh = max(-126, min(126, 14 - ex));
  const float mul = __uint_as_float((uint32_t)(127 + sh) << 23);
  f.inv = __uint_as_float((uint32_t)(127 - sh) << 23);
#pragma unroll
  for (int nb = 0; nb < NB; ++nb)
#pragma unroll
    for (int ks = 0; ks < 4; ++ks)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int i = 8 * (ks >> 1) + 2 * (ks & 1) + h;
        const float x0 = x[nb][i] * mul, x1 = x[nb][i + 4] * mul;
        const __half2 hi = __floats2half2_rn(x0, x1);
        const float2 hf = __half22float2(hi);
        f.a[nb][ks][2 * h] = h2_bits(hi);
        f.a[nb][ks][2 * h + 1] = h2_bits(__floats2half2_rn(x0 - hf.x, x1 - hf.y));
      }
}

// Raw products of 16 tokens with the heads: kw[u][nb] are this lane's 8 bytes of token (u, g).
// dot[2u + x] is head g against this lane's token x of tile u; ks[nb][2u + x] its scales.
template <int NB>
__device__ __forceinline__ void q4_scores(const Q4Query<NB>& f, const uint2 (&kw)[2][NB], const float (&ks)[NB][4],
                                          float (&dot)[4]) {
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    float d0 = 0.f, d1 = 0.f;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      float c[4] = {0.f, 0.f, 0.f, 0.f};
      uint32_t p0[4], p1[4];
      q4_pairs_f16(kw[u][nb].x, p0);
      q4_pairs_f16(kw[u][nb].y, p1);
      mma_f16(c, f.a[nb][0], p0[0], p0[1]);
      mma_f16(c, f.a[nb][1], p0[2], p0[3]);
      mma_f16(c, f.a[nb][2], p1[0], p1[1]);
      mma_f16(c, f.a[nb][3], p1[2], p1[3]);
      d0 = fmaf(c[0] + c[2], ks[nb][2 * u], d0);
      d1 = fmaf(c[1] + c[3], ks[nb][2 * u + 1], d1);
    }
    dot[2 * u] = d0;
    dot[2 * u + 1] = d1;
  }
}

// Running softmax state of up to 8 heads in one warp: m is head g's maximum (the same in the four
// lanes of a head), l this lane's own part of the sum, o the outputs (high-part rows in elements 0,
// 1 of each tile, low-part rows in 2, 3); column n of tile j is element 64 nb + 8 n + j.
template <int NB>
struct Q4State {
  float m, l;
  float o[NB][8][4];
  __device__ __forceinline__ void reset() {
    m = -INFINITY;
    l = 0.f;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[nb][j][e] = 0.f;
  }
};

// Adds 16 tokens: x[i] are base-2 logits of this lane's tokens (-inf: not attended), vw[i][nb] word
// g of token i's codes, vs[nb][i] its scales. The maximum moves only when a logit passes it by more
// than 2^8, so most units cost no shuffle and no rescaling; weights stay below 2^8.
template <int NB>
__device__ __forceinline__ void q4_accumulate(Q4State<NB>& s, const float (&x)[4], const uint32_t (&vw)[4][NB],
                                              const float (&vs)[NB][4]) {
  const float mx = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
  if (__any_sync(kFull, mx > s.m + 8.f)) {
    float mn = fmaxf(s.m, mx);
    mn = fmaxf(mn, __shfl_xor_sync(kFull, mn, 1));
    mn = fmaxf(mn, __shfl_xor_sync(kFull, mn, 2));
    const float f = s.m == mn ? 1.f : ex2(s.m - mn);
    s.m = mn;
    s.l *= f;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) s.o[nb][j][e] *= f;
  }
  float p[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    p[i] = x[i] == -INFINITY ? 0.f : ex2(x[i] - s.m);
    s.l += p[i];
  }
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    // a token that is not attended may lie in a slot never written: its scale is not used
    float w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = x[i] == -INFINITY ? 0.f : p[i] * vs[nb][i];
    uint32_t a[4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const __nv_bfloat162 hi = __floats2bfloat162_rn(w[2 * h], w[2 * h + 1]);
      const float2 hf = __bfloat1622float2(hi);
      a[2 * h] = b2_bits(hi);
      a[2 * h + 1] = b2_bits(__floats2bfloat162_rn(w[2 * h] - hf.x, w[2 * h + 1] - hf.y));
    }
    const uint32_t ab0 = __byte_perm(vw[0][nb], vw[1][nb], 0x5410), ab1 = __byte_perm(vw[0][nb], vw[1][nb], 0x7632);
    const uint32_t cd0 = __byte_perm(vw[2][nb], vw[3][nb], 0x5410), cd1 = __byte_perm(vw[2][nb], vw[3][nb], 0x7632);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      mma_bf16(s.o[nb][j], a, q4_pair_bf16(ab0, j), q4_pair_bf16(cd0, j));
      mma_bf16(s.o[nb][4 + j], a, q4_pair_bf16(ab1, j), q4_pair_bf16(cd1, j));
    }
  }
}

}  // namespace ts
