// Causal attention of whole prompts, packed one behind another, with grouped heads.
//
//   s[r][j] = scale <q_r, k_j>,  j <= r       out_r = sum_j 2^(s' - m) v_j / sum_j 2^(s' - m)
//
// with s' = s log2(e) and m a running maximum of the row. 4 d H n^2 / 2 operations for a prompt of
// n tokens against 2 d (2 H + 2 H_kv) n bytes: bound by the tensor cores from a few hundred tokens
// on, so both products run on tcgen05 with their accumulators in tensor memory and the softmax works
// beside them.
//
// A tile is 128 query rows of one KV head: 128 / G tokens with all G query heads of the group, row
// = token * G + head, so a key tile in shared memory serves the whole group and a short prompt fills
// a tile sooner. A CTA works on a block of two neighbouring tiles, which share every key and value
// tile of 128 tokens:
//   warp 8     loads: the two query tiles, then K and V tiles (TMA, 128-byte swizzle, two slots each)
//   warp 9     products: S_i(j+1) = Q_i K(j+1)^T is issued behind O_i += P_i(j) V(j), so the tensor
//              cores have the other tile's products to do while one tile's softmax runs
//   warps 0-3  softmax of tile 0, a thread per row: scores from tensor memory, weights back over them
//   warps 4-7  the same of tile 1
// The running maximum moves only when a score passes it by 2^8: weights and sums stay below 2^8 times
// their number, far inside fp32, and the accumulators are rescaled a handful of times per row. The
// softmax warps do that themselves, in between two products of their tile.
//
// Masked places hold what they hold. A score behind the diagonal is replaced before it is used. A
// value behind the diagonal meets a weight of zero in the product, which is not enough for a NaN or
// an infinity, so in the tiles on the diagonal (and past the sequence's end, where the next
// sequence's rows are) such values are taken out of the tile in shared memory, noted per column with
// their first row, and put back into the outputs of the rows that see them.
//
// Blocks of all sequences are dealt out heaviest first (a block's work grows with its place in its
// sequence), so the grid drains evenly.
#include <cmath>
#include <cuda.h>
#include <cudaTypedefs.h>

#include "ts_tc.cuh"

namespace ts {
namespace {

constexpr int kPrRows = 128;     // query rows of a tile
constexpr int kPrKeys = 128;     // tokens of a key tile
constexpr int kPrSoftmaxWarps = 8;
constexpr int kPrThreads = (kPrSoftmaxWarps + 4) * 32;   // three warpgroups; two warps of the third idle
// Registers a thread: 168 at launch (65536 / 384); the softmax warpgroups hold a row of 128 scores and
// take what the third gives up: 2 * 208 + 88 = 3 * 168.
constexpr int kPrSoftmaxRegs = 208, kPrOtherRegs = 88;
static_assert(2 * kPrSoftmaxRegs + kPrOtherRegs <= 3 * 168, "register shares");
constexpr int kPrNone = 0x7fffffff;

struct PromptArgs {
  CUtensorMap q, k, v;           // [rows][heads][d] each
  const int32_t* cu;
  int B, total;
  int H, HKV, G;
  int tokens;                    // tokens of a tile: 128 / G
  float scale2;                  // |scale| log2(e)
  int negate;                    // scale < 0: the products are taken with -Q
  __nv_bfloat16* out;
  int64_t out_stride;
  float* lse;
  int* status;
  uint64_t wait_ns;
};

template <int D>
struct PrShape {
  static constexpr int HALVES = D / 64;
  static constexpr int QT = kPrRows * D * 2;    // bytes of a query tile
  static constexpr int KT = kPrKeys * D * 2;    // bytes of a key or value tile
  static constexpr int SMEM = 2 * QT + 4 * KT + 1024;
  static constexpr uint32_t TMEM_COLS = 512;
  static constexpr uint32_t S_COL = 0, O_COL = 256;   // tile i: S at 128 i (weights over its first 64), O at 256 + 128 i
};

__device__ __forceinline__ void add2(float& a, float& b, float x, float y) {
  uint64_t s = pack_f2(a, b), t = pack_f2(x, y), r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(s), "l"(t));
  unpack_f2(r, a, b);
}

__device__ __forceinline__ float pr_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Sequence and block of item t (one warp; the same in every lane): items in order of descending
// block number over all sequences. False past the last one. Sequences whose boundaries are not
// ascending inside [0, total] have no blocks.
__device__ __forceinline__ int seq_blocks(const PromptArgs& a, int b, int block) {
  const int s0 = a.cu[b], s1 = a.cu[b + 1];
  return (s0 < 0 || s1 < s0 || s1 > a.total) ? 0 : (s1 - s0 + block - 1) / block;
}

__device__ __forceinline__ int64_t blocks_from(const PromptArgs& a, int block, int mine, int level, int lane) {
  int64_t n = max(0, mine - level);
  for (int b = lane + 32; b < a.B; b += 32) n += max(0, seq_blocks(a, b, block) - level);
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) n += __shfl_xor_sync(kFull, n, d);
  return n;
}

__device__ __forceinline__ bool find_item(const PromptArgs& a, int64_t t, int block, int lane, int& seq, int& blk) {
  const int mine = lane < a.B ? seq_blocks(a, lane, block) : 0;
  int most = mine;
  for (int b = lane + 32; b < a.B; b += 32) most = max(most, seq_blocks(a, b, block));
  most = __reduce_max_sync(kFull, most);
  if (a.B == 1) {
    seq = 0;
    blk = most - 1 - (int)t;
    return t < most;
  }
  if (t >= blocks_from(a, block, mine, 0, lane)) return false;
  int lo = 0, hi = most;             // blocks at level lo or above: more than t; at hi: not
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (blocks_from(a, block, mine, mid, lane) > t) lo = mid; else hi = mid;
  }
  int rank = (int)(t - blocks_from(a, block, mine, lo + 1, lane));
  blk = lo;
  for (int b0 = 0; b0 < a.B; b0 += 32) {
    const bool has = (b0 == 0 ? mine : (b0 + lane < a.B ? seq_blocks(a, b0 + lane, block) : 0)) > lo;
    const unsigned m = __ballot_sync(kFull, has);
    if (rank < __popc(m)) {
      seq = b0 + (int)__fns(m, 0, rank + 1);
      return true;
    }
    rank -= __popc(m);
  }
  return false;
}

template <int D>
__global__ void __launch_bounds__(kPrThreads, 1) prompt_kernel(const __grid_constant__ PromptArgs a) {
  using S = PrShape<D>;
  extern __shared__ unsigned char dsm_raw[];
  unsigned char* base = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(dsm_raw) + 1023) & ~(uintptr_t)1023);
  unsigned char* sQ = base;                // two query tiles
  unsigned char* sK = sQ + 2 * S::QT;      // two key slots
  unsigned char* sV = sK + 2 * S::KT;      // two value slots
  __shared__ __align__(8) uint64_t q_full, k_full[2], k_empty[2], v_full[2], v_empty[2], v_clean[2], s_full[2],
      p_ready[2], o_done[2];
  __shared__ uint32_t s_tmem;
  __shared__ int s_item[3];                // found, sequence, block
  __shared__ int s_first[3][D];            // first row of a column's NaN, +inf, -inf behind the diagonal's start
  __shared__ int s_odd;                    // any of them

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int kv = blockIdx.x % a.HKV;
  const int block = 2 * a.tokens;

  if (warp == kPrSoftmaxWarps) {
    int seq = 0, blk = 0;
    const bool found = find_item(a, blockIdx.x / a.HKV, block, lane, seq, blk);
    if (lane == 0) {
      s_item[0] = found;
      s_item[1] = seq;
      s_item[2] = blk;
      // warps that look through the value tiles: those of a tile past the sequence's end wait for no
      // scores, so nothing would keep them in step with the value slots
      const bool second = found && blk * block + a.tokens < a.cu[seq + 1] - a.cu[seq];
      for (int i = 0; i < 2; ++i) mbar_init(&v_clean[i], second ? kPrSoftmaxWarps : kPrSoftmaxWarps / 2);
      mbar_fence_init();
    }
    if (blockIdx.x == 0)
      for (int b = lane; b <= a.B; b += 32) {
        const int v = a.cu[b];
        if (v > a.total || (b == 0 ? v != 0 : v < a.cu[b - 1])) set_error(a.status, TS_ERR_SEQ_LEN);
      }
  }
  if (warp == kPrSoftmaxWarps + 1) {
    tmem_alloc(&s_tmem, S::TMEM_COLS);
    tmem_relinquish();
  }
  if (tid == 0) {
    mbar_init(&q_full, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&k_full[i], 1);
      mbar_init(&k_empty[i], 1);
      mbar_init(&v_full[i], 1);
      mbar_init(&v_empty[i], 1);
      mbar_init(&s_full[i], 1);
      mbar_init(&p_ready[i], kPrSoftmaxWarps / 2);
      mbar_init(&o_done[i], 1);
    }
    mbar_fence_init();
    s_odd = 0;
  }
  for (int i = tid; i < 3 * D; i += kPrThreads) (&s_first[0][0])[i] = kPrNone;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;

  if (s_item[0]) {
    const int seq = s_item[1], blk = s_item[2];
    const int row0 = a.cu[seq], n = a.cu[seq + 1] - row0;
    const int i0 = blk * block;                                   // first token of the block
    // key tiles of each query tile (0: the tile lies past the sequence), and the first one masked
    int nt[2];
    for (int i = 0; i < 2; ++i) {
      const int first = i0 + i * a.tokens;
      nt[i] = first < n ? (min(first + a.tokens, n) + kPrKeys - 1) / kPrKeys : 0;
    }
    const int ntiles = max(nt[0], nt[1]);
    const int masked_from = (i0 + 1) / kPrKeys;                   // tile j holds a key past token i0: 128 j + 127 > i0

    if (warp >= kPrSoftmaxWarps) {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kPrOtherRegs));
      if (warp == kPrSoftmaxWarps) {
      // ---------------------------------------------------------------- loads
      if (lane == 0) {
        bool ok = true;
        int kn = 0, vn = 0;
        mbar_arrive_expect_tx(&q_full, (uint32_t)(2 * S::HALVES * a.G * a.tokens * 128));
        for (int i = 0; i < 2; ++i)
          for (int h = 0; h < S::HALVES; ++h)
            tma_load_3d(sQ + i * S::QT + h * (kPrRows * 128), &a.q, h * 64, kv * a.G, row0 + i0 + i * a.tokens, &q_full);
        for (int j = 0; j < ntiles && ok; ++j) {
          const int s = j & 1;
          if (j >= 2) ok = mbar_wait(&k_empty[s], ((j >> 1) - 1) & 1, a.wait_ns);
          if (ok) {
            mbar_arrive_expect_tx(&k_full[s], S::KT);
            for (int h = 0; h < S::HALVES; ++h)
              tma_load_3d(sK + s * S::KT + h * (kPrKeys * 128), &a.k, h * 64, kv, row0 + j * kPrKeys, &k_full[s]);
            ++kn;
            if (j >= 2) ok = mbar_wait(&v_empty[s], ((j >> 1) - 1) & 1, a.wait_ns);
          }
          if (ok) {
            mbar_arrive_expect_tx(&v_full[s], S::KT);
            for (int h = 0; h < S::HALVES; ++h)
              tma_load_3d(sV + s * S::KT + h * (kPrKeys * 128), &a.v, h * 64, kv, row0 + j * kPrKeys, &v_full[s]);
            ++vn;
          }
        }
        if (!ok) set_error(a.status, TS_ERR_TIMEOUT);
        // nothing may still be landing when the CTA exits
        if (!mbar_wait(&q_full, 0, a.wait_ns)) set_error(a.status, TS_ERR_TIMEOUT);
        for (int j = max(0, kn - 2); j < kn; ++j) mbar_wait(&k_full[j & 1], (j >> 1) & 1, a.wait_ns);
        for (int j = max(0, vn - 2); j < vn; ++j) mbar_wait(&v_full[j & 1], (j >> 1) & 1, a.wait_ns);
      }
      __syncwarp();
      } else if (warp == kPrSoftmaxWarps + 1) {
      // ------------------------------------------------------------- products
      if (lane == 0) {
        const uint32_t idesc_s = idesc_bf16_f32(kPrRows, kPrKeys) | (a.negate ? 1u << 13 : 0u);   // bit 13: -A
        constexpr uint32_t idesc_o = idesc_bf16_f32_bmn(kPrRows, D);
        const uint32_t q0 = smem_addr(sQ), k0 = smem_addr(sK), v0 = smem_addr(sV);
        auto scores = [&](int i, int j) {
          const uint32_t kt = k0 + (j & 1) * S::KT, qt = q0 + i * S::QT;
#pragma unroll
          for (int h = 0; h < S::HALVES; ++h)
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
              umma_bf16(tmem + S::S_COL + 128 * i, sdesc_sw128(qt + h * (kPrRows * 128) + ks * 32),
                        sdesc_sw128(kt + h * (kPrKeys * 128) + ks * 32), idesc_s, (h | ks) != 0);
          umma_commit(&s_full[i]);
        };
        bool ok = mbar_wait(&q_full, 0, a.wait_ns) && mbar_wait(&k_full[0], 0, a.wait_ns);
        if (ok) {
          tc_fence_after();
          for (int i = 0; i < 2; ++i)
            if (nt[i] > 0) scores(i, 0);
          umma_commit(&k_empty[0]);
        }
        for (int j = 0; j < ntiles && ok; ++j) {
          const int s = j & 1, s1 = (j + 1) & 1;
          ok = mbar_wait(&v_full[s], (j >> 1) & 1, a.wait_ns);
          if (ok && j >= masked_from) ok = mbar_wait(&v_clean[s], ((j >> 1) - (masked_from + (s ^ (masked_from & 1))) / 2) & 1, a.wait_ns);
          if (ok && j + 1 < ntiles) ok = mbar_wait(&k_full[s1], ((j + 1) >> 1) & 1, a.wait_ns);
          for (int i = 0; i < 2 && ok; ++i) {
            if (j >= nt[i]) continue;
            ok = mbar_wait(&p_ready[i], j & 1, a.wait_ns);
            if (!ok) break;
            tc_fence_after();
            const uint32_t vt = v0 + s * S::KT;
#pragma unroll
            for (int ks = 0; ks < kPrKeys / 16; ++ks)
              umma_bf16_ts(tmem + S::O_COL + 128 * i, tmem + S::S_COL + 128 * i + 8 * ks,
                           sdesc_sw128_mn(vt + ks * 2048, kPrKeys * 128, 1024), idesc_o, (j | ks) != 0);
            umma_commit(&o_done[i]);
            if (j + 1 < nt[i]) scores(i, j + 1);
          }
          if (ok) {
            umma_commit(&v_empty[s]);
            if (j + 1 < ntiles) umma_commit(&k_empty[s1]);
          }
        }
        if (!ok) set_error(a.status, TS_ERR_TIMEOUT);
      }
      __syncwarp();
      }
    } else if (nt[warp >> 2] > 0) {
      asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kPrSoftmaxRegs));
      // -------------------------------------------------------------- softmax
      const int i = warp >> 2;                                    // tile
      const int share = S::KT / (nt[1] > 0 ? kPrSoftmaxWarps : kPrSoftmaxWarps / 2);   // bytes of a value tile to look through
      const int row = 32 * (warp & 3) + lane;
      const int first = i0 + i * a.tokens;                        // first token of the tile
      const int tok = first + row / a.G, head = kv * a.G + row % a.G;
      const bool real = row < a.tokens * a.G && tok < n;
      const uint32_t lane_off = (uint32_t)(32 * (warp & 3)) << 16;
      const uint32_t tS = tmem + S::S_COL + 128 * i + lane_off, tO = tmem + S::O_COL + 128 * i + lane_off;
      float m2 = -INFINITY, la = 0.f, lb = 0.f;                   // running maximum (base 2) and two halves of the sum
      bool ok = true;
      for (int j = 0; j < ntiles && ok; ++j) {
        if (j >= masked_from) {
          // this warp's part of the value tile: what is not finite from token i0 on comes out
          ok = mbar_wait(&v_full[j & 1], (j >> 1) & 1, a.wait_ns);
          if (!__all_sync(kFull, ok)) break;
          unsigned char* vt = sV + (j & 1) * S::KT + warp * share;
          uint32_t odd = 0u;
#pragma unroll 4
          for (int c = 0; c < share / 512; ++c) {
            const uint4 w = lds128(vt + c * 512 + lane * 16);
            odd |= ((w.x & 0x7f807f80u) + 0x00800080u) | ((w.y & 0x7f807f80u) + 0x00800080u) |
                   ((w.z & 0x7f807f80u) + 0x00800080u) | ((w.w & 0x7f807f80u) + 0x00800080u);
          }
          if (odd & 0x80008000u) {
            for (int c = 0; c < share / 512; ++c) {
              const int off = warp * share + c * 512 + lane * 16;        // byte in the tile
              const int r = (off % (kPrKeys * 128)) / 128, key = j * kPrKeys + r;
              const int col0 = off / (kPrKeys * 128) * 64 + (((off / 16) % 8) ^ (r & 7)) * 8;
              if (key <= i0) continue;                            // every row of the block sees it
              uint16_t* e16 = reinterpret_cast<uint16_t*>(sV + (j & 1) * S::KT + off);
              for (int e = 0; e < 8; ++e) {
                const uint32_t u = e16[e];
                if ((u & 0x7f80u) != 0x7f80u) continue;
                atomicMin(&s_first[(u & 0x7fu) ? 0 : (u >> 15 ? 2 : 1)][col0 + e], key);
                e16[e] = 0;
                s_odd = 1;
              }
            }
          }
          fence_proxy_async();
          __syncwarp();
          if (lane == 0) mbar_arrive(&v_clean[j & 1]);
        }
        if (j >= nt[i]) continue;
        ok = mbar_wait(&s_full[i], j & 1, a.wait_ns);
        if (!__all_sync(kFull, ok)) break;
        tc_fence_after();
        uint32_t u[128];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld_x32(tS + 32 * c, u + 32 * c);
        tmem_wait_ld();
        float* x = reinterpret_cast<float*>(u);
        if (j * kPrKeys + kPrKeys - 1 > first) {                  // the tile holds keys that a row may not see
          const int lim = tok - j * kPrKeys;
#pragma unroll
          for (int c = 0; c < 128; ++c) x[c] = c <= lim ? x[c] : -INFINITY;
        }
        float mx = x[0], my = x[1];
#pragma unroll
        for (int c = 2; c < 128; c += 2) {
          mx = fmaxf(mx, x[c]);
          my = fmaxf(my, x[c + 1]);
        }
        // rows that are no query of the sequence (their operands may be anything) move no maximum
        const float top = real ? fmaxf(mx, my) * a.scale2 : -INFINITY;
        if (__any_sync(kFull, top > m2 + 8.f)) {
          const float mn = fmaxf(m2, top);
          const float f = mn == m2 ? 1.f : pr_ex2(m2 - mn);
          m2 = mn;
          la *= f;
          lb *= f;
          if (j > 0) {
            // the tile's last product must be in before its accumulators are rescaled
            ok = mbar_wait(&o_done[i], (j - 1) & 1, a.wait_ns);
            if (!__all_sync(kFull, ok)) break;
            tc_fence_after();
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
              uint32_t o[32];
              tmem_ld_x32(tO + 32 * c, o);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
              tmem_st_x32(tO + 32 * c, o);
            }
          }
        }
        const float ms = m2 == -INFINITY ? 0.f : -m2;             // nothing seen yet: every weight is zero
        const uint64_t sc = pack_f2(a.scale2, a.scale2), mm = pack_f2(ms, ms);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t p[32];
#pragma unroll
          for (int c = 0; c < 32; ++c) {
            const int e = 64 * h + 2 * c;
            float y0, y1;
            unpack_f2(fma_f2(pack_f2(x[e], x[e + 1]), sc, mm), y0, y1);
            y0 = pr_ex2(y0);
            y1 = pr_ex2(y1);
            add2(la, lb, y0, y1);
            p[c] = pack_bf16(y0, y1);
          }
          tmem_st_x32(tS + 32 * h, p);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_ready[i]);
      }
      // ---- outputs
      if (__all_sync(kFull, ok)) {
        ok = mbar_wait(&o_done[i], (nt[i] - 1) & 1, a.wait_ns);
        // what the value tiles held is known once every warp has looked through the last of them
        for (int j = max(masked_from, ntiles - 2); j < ntiles; ++j)
          ok = ok && mbar_wait(&v_clean[j & 1], ((j >> 1) - (masked_from + ((j & 1) ^ (masked_from & 1))) / 2) & 1, a.wait_ns);
        if (__all_sync(kFull, ok)) {
          tc_fence_after();
          const float l = la + lb, inv = 1.f / l;
          __nv_bfloat16* dst = a.out + (int64_t)(row0 + tok) * a.out_stride + (int64_t)head * D;
          const bool odd = s_odd != 0;
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            uint32_t o[32];
            tmem_ld_x32(tO + 32 * c, o);
            tmem_wait_ld();
            if (odd) {
#pragma unroll
              for (int e = 0; e < 32; ++e) {
                const int col = 32 * c + e;
                const bool pos = tok >= s_first[1][col], neg = tok >= s_first[2][col];
                float add = pos ? INFINITY : 0.f;
                if (neg) add += -INFINITY;
                if (tok >= s_first[0][col]) add = NAN;
                o[e] = __float_as_uint(__uint_as_float(o[e]) + add);
              }
            }
            if (real) {
              uint4* d4 = reinterpret_cast<uint4*>(dst + 32 * c);
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                uint32_t w[4];
#pragma unroll
                for (int z = 0; z < 4; ++z)
                  w[z] = pack_bf16(__uint_as_float(o[8 * e + 2 * z]) * inv, __uint_as_float(o[8 * e + 2 * z + 1]) * inv);
                d4[e] = make_uint4(w[0], w[1], w[2], w[3]);
              }
            }
          }
          if (real && a.lse) a.lse[(int64_t)(row0 + tok) * a.H + head] = (m2 + log2f(l)) * 0.6931471805599453f;
        }
      }
      if (!ok && lane == 0) set_error(a.status, TS_ERR_TIMEOUT);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kPrSoftmaxWarps + 1) {
    tc_fence_after();
    tmem_dealloc(tmem, S::TMEM_COLS);
  }
}

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
  static const PFN_cuTensorMapEncodeTiled_v12000 encode = [] {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q{};
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      fn = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  }();
  return encode;
}

// bf16 [rows][heads][d] with `stride` elements between rows, boxes of 64 elements x bh heads x bt rows.
bool rows_map(CUtensorMap* map, const void* p, int64_t rows, int heads, int d, int64_t stride, int bh, int bt) {
  const auto encode = tensor_map_encoder();
  if (!encode) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)rows};
  const cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)stride * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)bh, (cuuint32_t)bt};
  const cuuint32_t estr[3] = {1, 1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(p), dims, strides, box, estr,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D>
ts_status run_prompt(ts_ctx* ctx, const PromptArgs& a, int64_t grid, cudaStream_t s) {
  if (!ensure_smem<prompt_kernel<D>>((size_t)PrShape<D>::SMEM, ctx->device)) return TS_ERR_CUDA;
  ProfScope ps(ctx, TS_PROF_ATTEND, s);
  ctx->kernels += 1;
  prompt_kernel<D><<<(unsigned)grid, kPrThreads, PrShape<D>::SMEM, s>>>(a);
  return cuda_status(cudaGetLastError());
}

}  // namespace

bool prompt_supported(const ts_config& c) {
  return (c.kv_dtype == TS_KV_BF16 || c.kv_dtype == TS_KV_Q4) && (c.head_dim == 64 || c.head_dim == 128) &&
         c.n_q_heads / c.n_kv_heads <= 16;
}

ts_status launch_prompt_attend(ts_ctx* ctx, const PromptCall& c, cudaStream_t s) {
  if (c.total == 0) return TS_OK;
  const ts_config& cfg = ctx->cfg;
  PromptArgs a{};
  a.cu = c.cu_rows;
  a.B = c.B;
  a.total = c.total;
  a.H = cfg.n_q_heads;
  a.HKV = cfg.n_kv_heads;
  a.G = a.H / a.HKV;
  a.tokens = kPrRows / a.G;
  a.scale2 = std::fabs(c.scale) * 1.4426950408889634f;
  a.negate = c.scale < 0.f;
  a.out = static_cast<__nv_bfloat16*>(c.out);
  a.out_stride = c.out_stride;
  a.lse = c.lse;
  a.status = ctx->status;
  a.wait_ns = ctx->wait_ns;
  if (!rows_map(&a.q, c.q, c.total, a.H, cfg.head_dim, c.q_stride, a.G, a.tokens) ||
      !rows_map(&a.k, c.k, c.total, a.HKV, cfg.head_dim, c.k_stride, 1, kPrKeys) ||
      !rows_map(&a.v, c.v, c.total, a.HKV, cfg.head_dim, c.v_stride, 1, kPrKeys))
    return TS_ERR_CUDA;
  // a sequence has at most one block that is not full
  const int64_t grid = ((int64_t)c.total / (2 * a.tokens) + (c.B < c.total ? c.B : c.total)) * a.HKV;
  if (grid > 0x7fffffff) return TS_ERR_SHAPE;
  return cfg.head_dim == 64 ? run_prompt<64>(ctx, a, grid, s) : run_prompt<128>(ctx, a, grid, s);
}

}  // namespace ts
