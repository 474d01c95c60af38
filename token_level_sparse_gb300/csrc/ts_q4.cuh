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
// Both products run as m16n8k16 with the unpacked codes as the 16-row operand (16 tokens, or 16
// elements of the values) and the heads as its 8 columns: column 2h holds the high part of head h's
// query (or weight), column 2h + 1 the low part. One instruction so takes both parts of a split fp32
// operand for four heads, and the two results of a head lie in one lane: lane (g, t) holds head t's
// scores of tokens g and g + 8, its maximum, its sum and its outputs. Codes are exact in fp16 and their
// products with either part exact in fp32.
#pragma once

#include <cfloat>
#include <cuda_fp16.h>

#include "ts_common.cuh"

namespace ts {

__host__ __device__ constexpr int q4_code_bytes(int d) { return kPage * d / 2; }
__host__ __device__ constexpr int q4_block_bytes(int d) { return kPage * (d / 2 + d / 32); }

// D (16x8, fp32) += A (16x16) B (16x8): lane (g = lane / 4, t = lane % 4) holds rows g, g + 8 of A,
// column g of B and rows g, g + 8 of D at columns 2t, 2t + 1. Volatile, as every instruction that a whole
// warp executes together has to be: the compiler may otherwise move it into a branch that only some
// lanes take.
__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t h2_bits(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }
__device__ __forceinline__ __half2 bits_h2(uint32_t u) { return *reinterpret_cast<__half2*>(&u); }
__device__ __forceinline__ float bf16_bits_f(uint32_t u) { return __uint_as_float(u << 16); }

// (x & m) | k in one instruction
__device__ __forceinline__ uint32_t and_or(uint32_t x, uint32_t m, uint32_t k) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(x), "r"(m), "r"(k));
  return r;
}

// The eight codes of a word as four fp16 pairs, pair i = codes (i, i + 4), each minus 8, exactly:
// a code in the low mantissa bits of 1024 is 1024 + u, four bits higher it is 1024 + 16 u. (The bits alone, as
// numbers below 2^-14, with 8 times the queries' sum taken off the products, are 4 instructions fewer and made
// the attention 3% faster, but the tensor cores cut the larger sums off: scores lost a bit.)
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

// Transposes an 8x8 matrix of 16-bit elements held as (row g, columns 2t, 2t + 1).
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

// The queries of up to 4 NT heads as the column operand of the scores: element pairs in the order that
// q4_pairs_f16 gives the codes. A head's queries are scaled by a power of two so that the largest
// lies in [2^14, 2^15), then split into two fp16 terms (hi + lo within 2^-22 of the element, or
// 2^-39 of the largest); inv undoes the scaling for the head whose scores this lane holds.
template <int NB, int NT>
struct Q4Query {
  uint32_t b[NT][NB][4][2];
  float inv[NT];
};

// q: 4 NT rows of 64 NB floats in shared memory, zeros where there is no head.
template <int NB, int NT>
__device__ __forceinline__ void q4_load_query(Q4Query<NB, NT>& f, const float* q, int lane) {
  const int g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const float* row = q + (4 * nt + (g >> 1)) * (NB * 64);
    float x[NB][16];
    float mx = 0.f;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 v = *reinterpret_cast<const float4*>(row + nb * 64 + 16 * t + 4 * i);
        x[nb][4 * i] = v.x;
        x[nb][4 * i + 1] = v.y;
        x[nb][4 * i + 2] = v.z;
        x[nb][4 * i + 3] = v.w;
        mx = fmaxf(fmaxf(mx, fmaxf(fabsf(v.x), fabsf(v.y))), fmaxf(fabsf(v.z), fabsf(v.w)));
      }
    mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 1));
    mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 2));
    const int ex = (int)(__float_as_uint(mx) >> 23) - 127;                 // mx < 2^(ex + 1)
    const int sh = max(-126, min(126, 14 - ex));
    const float mul = __uint_as_float((uint32_t)(127 + sh) << 23);
    f.inv[nt] = __shfl_sync(kFull, __uint_as_float((uint32_t)(127 - sh) << 23), 8 * t);
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int ks = 0; ks < 4; ++ks)
#pragma unroll
        for (int i2 = 0; i2 < 2; ++i2) {
          const int i = 8 * (ks >> 1) + 2 * (ks & 1) + i2;
          const float x0 = x[nb][i] * mul, x1 = x[nb][i + 4] * mul;
          const __half2 hi = __floats2half2_rn(x0, x1);
          const float2 hf = __half22float2(hi);
          f.b[nt][nb][ks][i2] = h2_bits((g & 1) ? __floats2half2_rn(x0 - hf.x, x1 - hf.y) : hi);
        }
  }
}

// Products of 16 tokens with the heads: kw[u][nb] are this lane's 8 bytes of token (u, g), ks[nb][u]
// that token's scale. dot[nt][u] is head 4 nt + t against token (u, g).
template <int NB, int NT>
__device__ __forceinline__ void q4_scores(const Q4Query<NB, NT>& f, const uint2 (&kw)[2][NB], const float (&ks)[NB][2],
                                          float (&dot)[NT][2]) {
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    uint32_t p[2][2][4];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      q4_pairs_f16(kw[u][nb].x, p[u][0]);
      q4_pairs_f16(kw[u][nb].y, p[u][1]);
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int k4 = 0; k4 < 4; ++k4) {
        const int x = k4 >> 1, i = 2 * (k4 & 1);
        const uint32_t a[4] = {p[0][x][i], p[1][x][i], p[0][x][i + 1], p[1][x][i + 1]};
        mma_f16(c, a, f.b[nt][nb][k4][0], f.b[nt][nb][k4][1]);
      }
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const float d = c[2 * u] + c[2 * u + 1];
        dot[nt][u] = nb == 0 ? d * ks[nb][u] : fmaf(d, ks[nb][u], dot[nt][u]);
      }
    }
  }
}

__device__ __forceinline__ int exponent(float x) { return (int)(__float_as_uint(x) >> 23 & 255u) - 127; }
__device__ __forceinline__ float power_of_two(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }   // -127: 0

// Running softmax state of 4 NT heads in one warp, for head 4 nt + t: m what its logits are taken against (their
// maximum rounded down, raised now and then; the same in the eight lanes of a head), l this lane's own part of its
// sum, o its outputs times sc, a power of two of its own for each 64 elements (high parts in elements 0 and 2, low
// parts in 1 and 3): tile j, rows g and g + 8, are elements 64 nb + 8 g + j and + 4.
//
// A weight times its value's scale enters its product as two fp16 terms. sc keeps the largest such term so far
// between 2^6 and 2^13, so that a term is held within 2^-22 of itself, or within 2^-31 of the largest of the same
// 64 elements. It begins as far up as weights below 2^9 allow and comes down to the first terms that there are
// (however late: rows of zeros say nothing about the size of the others) and to any that pass 2^13. Where m rises by a
// whole number, sc rises with it: the sums stay as they are, and the terms behind, which weigh that much more, find
// the unit right for them or bring it down again. Groups do not share sc, so that one whose values are large, or
// not finite, takes nothing from the others.
//
// The tensor cores cut their sums off rather than round them: over a few hundred steps in one accumulator
// that is 3e-6 of an output. So the sums go over to rows in shared memory every kQ4Flush stages, added
// there with rounding, and begin again at zero.
constexpr int kQ4Flush = 16;
constexpr int kQ4MaxUnit = 119;   // largest exponent of sc: weights of 2^8 times sc are finite
// What a head's sums in shared memory count in: the maximum and the powers of two that they belong to.
template <int NB>
struct Q4Unit {
  float m, sc[NB];
};

template <int NB, int NT>
struct Q4State {
  float m[NT], l[NT], sc[NT][NB];
  float o[NT][NB][4][4];
  __device__ __forceinline__ void reset() {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m[nt] = -INFINITY;
      l[nt] = 0.f;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        sc[nt][nb] = power_of_two(kQ4MaxUnit);
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[nt][nb][j][e] = 0.f;
      }
    }
  }
  __device__ __forceinline__ void join_lanes() {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      l[nt] += __shfl_xor_sync(kFull, l[nt], 4);
      l[nt] += __shfl_xor_sync(kFull, l[nt], 8);
      l[nt] += __shfl_xor_sync(kFull, l[nt], 16);
    }
  }
  // Moves the sums over to rows [head][64 NB] (in shared memory, this warp's own), whose units are kept in
  // units[head]. first: there is nothing in the rows yet.
  __device__ __forceinline__ void flush(float* rows, Q4Unit<NB>* units, bool first, int lane) {
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      Q4Unit<NB>& unit = units[4 * nt + t];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        // (sc rises no further than m, so that f is at most 1)
        float f = 0.f;
        if (!first) {
          const int rise = unit.m == m[nt] ? 0 : (int)fminf(m[nt] - unit.m, 1000.f);
          f = power_of_two(max(-127, exponent(sc[nt][nb]) - exponent(unit.sc[nb]) - rise));
        }
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          float4* row = reinterpret_cast<float4*>(rows + (4 * nt + t) * (NB * 64) + nb * 64 + 8 * g + 4 * r);
          float4 v = make_float4(o[nt][nb][0][2 * r] + o[nt][nb][0][2 * r + 1], o[nt][nb][1][2 * r] + o[nt][nb][1][2 * r + 1],
                                 o[nt][nb][2][2 * r] + o[nt][nb][2][2 * r + 1], o[nt][nb][3][2 * r] + o[nt][nb][3][2 * r + 1]);
          if (!first) {
            const float4 w = *row;
            v = make_float4(fmaf(w.x, f, v.x), fmaf(w.y, f, v.y), fmaf(w.z, f, v.z), fmaf(w.w, f, v.w));
          }
          *row = v;
#pragma unroll
          for (int j = 0; j < 4; ++j) o[nt][nb][j][2 * r] = o[nt][nb][j][2 * r + 1] = 0.f;
        }
      }
      __syncwarp();
      if (g == 0) {
        unit.m = m[nt];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) unit.sc[nb] = sc[nt][nb];
      }
    }
    __syncwarp();
  }
};

// Moves the maxima up for 16 P tokens with base-2 logits x[page][nt][u] (-inf: not attended), where a logit
// passes its head's by more than 8: most calls cost one vote and no rescaling, and weights are 2^8 at most.
// Whole numbers, so that what they change by is a power of two.
template <int NB, int NT, int P>
__device__ __forceinline__ void q4_raise_max(Q4State<NB, NT>& s, const float (&x)[P][NT][2]) {
  float top[NT];
  bool grow = false;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    top[nt] = fmaxf(x[0][nt][0], x[0][nt][1]);
#pragma unroll
    for (int pg = 1; pg < P; ++pg) top[nt] = fmaxf(top[nt], fmaxf(x[pg][nt][0], x[pg][nt][1]));
    grow |= top[nt] > s.m[nt] + 8.f;
  }
  if (__any_sync(kFull, grow)) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float mn = fmaxf(s.m[nt], floorf(top[nt]));
      mn = fmaxf(mn, __shfl_xor_sync(kFull, mn, 4));
      mn = fmaxf(mn, __shfl_xor_sync(kFull, mn, 8));
      mn = fmaxf(mn, __shfl_xor_sync(kFull, mn, 16));
      const int rise = s.m[nt] == mn ? 0 : (int)fminf(mn - s.m[nt], 1000.f);
      s.l[nt] *= power_of_two(max(-127, -rise));
      s.m[nt] = mn;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        const int was = exponent(s.sc[nt][nb]), up = min(rise, kQ4MaxUnit - was);
        s.sc[nt][nb] = power_of_two(was + up);
        const float f = power_of_two(max(-127, up - rise));            // (1 but at the end of sc's range)
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) s.o[nt][nb][j][e] *= f;
      }
    }
  }
}

// Weight of a base-2 logit x against m (neither -inf against -inf nor a masked place has any: 0, not NaN).
__device__ __forceinline__ float q4_weight(float x, float m) { return ex2(x - fmaxf(m, -FLT_MAX)); }

// Adds 16 tokens whose logits x[nt][u] (head 4 nt + t, token (u, g)) the maxima already cover: vs[nb][u]
// are that token's value scales, vw[i][nb] word g of the codes of token (i / 2, 2t + i % 2). kMasked: some
// tokens may not be attended (x = -inf).
//
// Where a term passes 2^13, the new sc comes from the exponents of weights and scales, and the terms are formed
// again from both: one in the old unit may have passed fp32. Terms that are not finite have no say in it.
template <int NB, int NT, bool kMasked>
__device__ __forceinline__ void q4_accumulate(Q4State<NB, NT>& s, const float (&x)[NT][2], const uint32_t (&vw)[4][NB],
                                              const float (&vs)[NB][2]) {
  float p[NT][2], w[NT][NB][2], top = 0.f;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const bool out = kMasked && x[nt][u] == -INFINITY;
      p[nt][u] = q4_weight(x[nt][u], s.m[nt]);
      s.l[nt] += p[nt][u];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        // a token that is not attended may lie in a slot never written: its scale is not used
        w[nt][nb][u] = out ? 0.f : p[nt][u] * s.sc[nt][nb] * vs[nb][u];
        top = fmaxf(top, fabsf(w[nt][nb][u]));
      }
    }
  }
  if (__any_sync(kFull, top > 8192.f)) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        // the largest term lies in [2^e, 2^(e + 2))
        int e = -1000;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const float v = fabsf(vs[nb][u]);
          if (p[nt][u] > 0.f && v > 0.f && v < INFINITY) e = max(e, exponent(p[nt][u]) + exponent(v));
        }
        e = max(e, __shfl_xor_sync(kFull, e, 4));
        e = max(e, __shfl_xor_sync(kFull, e, 8));
        e = max(e, __shfl_xor_sync(kFull, e, 16));
        const int was = exponent(s.sc[nt][nb]);
        if (e + was > 11) {
          const int to = max(-126, 6 - e);                           // the largest term to [2^6, 2^8)
          const float f = power_of_two(max(-127, to - was));
          s.sc[nt][nb] = power_of_two(to);
#pragma unroll
          for (int u = 0; u < 2; ++u) w[nt][nb][u] = kMasked && x[nt][u] == -INFINITY ? 0.f : p[nt][u] * s.sc[nt][nb] * vs[nb][u];
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) s.o[nt][nb][j][i] *= f;
        }
      }
    }
  }
  uint32_t b[NT][NB][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        // high and low part of one weight side by side, then across: a lane's tokens become another's columns
        const float hi = __half2float(__float2half_rn(w[nt][nb][u]));
        b[nt][nb][u] = movmatrix_trans(h2_bits(__floats2half2_rn(hi, w[nt][nb][u] - hi)));
      }
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    uint32_t ab0[4], ab1[4], cd0[4], cd1[4];
    q4_pairs_f16(__byte_perm(vw[0][nb], vw[1][nb], 0x5410), ab0);
    q4_pairs_f16(__byte_perm(vw[0][nb], vw[1][nb], 0x7632), ab1);
    q4_pairs_f16(__byte_perm(vw[2][nb], vw[3][nb], 0x5410), cd0);
    q4_pairs_f16(__byte_perm(vw[2][nb], vw[3][nb], 0x7632), cd1);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t a[4] = {ab0[j], ab1[j], cd0[j], cd1[j]};
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) mma_f16(s.o[nt][nb][j], a, b[nt][nb][0], b[nt][nb][1]);
    }
  }
}

}  // namespace ts
