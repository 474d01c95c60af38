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
// a tile sooner. An item of work is a block of two neighbouring tiles, which share every key and value
// tile of 128 tokens. One CTA per SM goes through its items, the roles each at their own pace:
//   warp 8      loads: the two query tiles of an item, then its K and V tiles (TMA, 128-byte swizzle, two
//               slots each, running on across items)
//   warp 9      products: S_i(j+1) = Q_i K(j+1)^T is issued behind O_i += P_i(j) V(j), so the tensor
//               cores have the other tile's products to do while one tile's softmax runs
//   warp 10     finds the next items
//   warp 11     looks through the value tiles on the diagonal (below)
//   warps 0-3   softmax of tile 0, a thread per row: scores from tensor memory, weights back over them; at
//               the end of an item its outputs, while the next item is loaded and its first scores taken
//   warps 4-7   the same of tile 1
// The running maximum is taken anew only in tiles where the sum of the weights against the old one passes
// 2^14: weights and sums stay far inside fp32 (and bf16 has the same relative error everywhere), most tiles
// need no pass over the scores for a maximum, and the accumulators are rescaled a handful of times per row.
// The softmax warps do that themselves, in between two products of their tile.
//
// A weight enters its product as one bf16 number (the sum takes it unrounded). That is the largest error there is
// beside the rounding of the outputs: rms 2.0e-3 of the outputs against 1.6e-3 for their rounding alone, with nine
// ragged prompts. A second bf16 term leaves 1.6e-3, but the tensor cores are what binds: 138 us in place of 98 for
// those, 7.75 ms in place of 5.40 for 32,771 tokens.
//
// Masked places hold what they hold. A score behind the diagonal is replaced before it is used. A
// value behind the diagonal meets a weight of zero in the product, which is not enough for a NaN or
// an infinity, so in the tiles on the diagonal (and past the sequence's end, where the next
// sequence's rows are) such values are taken out of the tile in shared memory, noted per column with
// their first row, and put back into the outputs of the rows that see them.
//
// Items are numbered heaviest first over all sequences (a block's work grows with its place in its
// sequence) and dealt out to the CTAs forth and back, so that they end together.
//
// Measured: 32,771 tokens, 32 heads over 8 of 128: 5.3 ms, 1.65 PFLOP/s (the products; power); nine
// prompts of 7615 tokens together, 28 heads over 4: 97 us, 1.16 PFLOP/s; 48 prompts of 16,437 tokens, 8
// heads over 4 of 64: 29 us, where an item has two or three key tiles and what binds is the softmax of a
// tile (1850 cycles, where one in the middle of a long prompt takes 1100) and an item's outputs (2400
// cycles). Writing outputs by tiled copies instead of stores, and leaving out weights right
// of the diagonal, measured the same (97.1 and 28.5 us; 97.0 and 28.8 us).
#include <cmath>

#include "ts_flash.cuh"

namespace ts {
namespace {

constexpr int kPrRows = 128;     // query rows of a tile
constexpr int kPrKeys = 128;     // tokens of a key tile
constexpr int kPrSoftmaxWarps = 8;
constexpr int kPrThreads = (kPrSoftmaxWarps + 4) * 32;   // three warpgroups
// Registers a thread: 168 at launch (65536 / 384); the softmax warpgroups hold a row of 128 scores and
// take what the third gives up: 2 * 208 + 88 = 3 * 168 (at 72 the products' warp spilled).
constexpr int kPrSoftmaxRegs = 208, kPrOtherRegs = 88;
static_assert(2 * kPrSoftmaxRegs + kPrOtherRegs <= 3 * 168, "register shares");
constexpr float kPrMaxSum = 16384.f;   // of a tile's weights against a maximum taken earlier
constexpr uint16_t kPrNone = 0xffff;

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
  static constexpr int STAGE = 32 * 128;        // bytes of a softmax warp's output staging: 32 rows of 64 columns
  static constexpr int SMEM = 2 * QT + 4 * KT + kPrSoftmaxWarps * STAGE + 1024;
  static_assert(SMEM + 2048 <= 227 * 1024, "shared memory of an SM");
  static constexpr uint32_t TMEM_COLS = 512;
  static constexpr uint32_t S_COL = 0, O_COL = 256;   // tile i: S at 128 i (weights over its first 64), O at 256 + 128 i
};

// Blocks of sequence b; sequences whose boundaries are not ascending inside [0, total] have none.
__device__ __forceinline__ int seq_blocks(const PromptArgs& a, int b, int block) {
  const int s0 = a.cu[b], s1 = a.cu[b + 1];
  return (s0 < 0 || s1 < s0 || s1 > a.total) ? 0 : (s1 - s0 + block - 1) / block;
}

// Numbers the blocks of all sequences in order of descending place in their sequence (one warp; results the
// same in every lane). The blocks of the first 128 sequences stay in registers.
struct BlockOrder {
  int n[4], start[4];
  int most;       // blocks of the longest sequence
  int all;        // blocks

  __device__ __forceinline__ void init(const PromptArgs& a, int block, int lane) {
    most = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int b = lane + 32 * k;
      n[k] = b < a.B ? seq_blocks(a, b, block) : 0;
      start[k] = b < a.B ? a.cu[b] : 0;
      most = max(most, n[k]);
    }
    for (int b = lane + 128; b < a.B; b += 32) most = max(most, seq_blocks(a, b, block));
    most = __reduce_max_sync(kFull, most);
    all = from(a, block, 0, lane);
  }
  // number of blocks at place `level` of their sequence or behind it
  __device__ __forceinline__ int from(const PromptArgs& a, int block, int level, int lane) const {
    int c = max(0, n[0] - level);
    if (a.B > 32) c += max(0, n[1] - level) + max(0, n[2] - level) + max(0, n[3] - level);
    for (int b = lane + 128; b < a.B; b += 32) c += max(0, seq_blocks(a, b, block) - level);
    return __reduce_add_sync(kFull, c);
  }
  // block t < all: its sequence and place. `hi`: a level that block t is below (most at first,
  // afterwards one above an earlier block's place).
  __device__ __forceinline__ void find(const PromptArgs& a, int block, int t, int& hi, int lane, int& seq, int& blk) const {
    int lo = 0;
    while (hi - lo > 1) {            // from(lo) > t >= from(hi)
      const int mid = (lo + hi) >> 1;
      if (from(a, block, mid, lane) > t) lo = mid; else hi = mid;
    }
    blk = lo;
    hi = lo + 1;
    int rank = t - from(a, block, lo + 1, lane);
    for (int b0 = 0; b0 < a.B; b0 += 32) {
      const int mine = b0 < 128 ? (b0 == 0 ? n[0] : b0 == 32 ? n[1] : b0 == 64 ? n[2] : n[3])
                                : (b0 + lane < a.B ? seq_blocks(a, b0 + lane, block) : 0);
      const unsigned m = __ballot_sync(kFull, mine > lo);
      if (rank < __popc(m)) {
        // the lane with `rank` set bits below its own
        const unsigned at = __ballot_sync(kFull, mine > lo && __popc(m & ((1u << lane) - 1u)) == rank);
        seq = b0 + __ffs(at) - 1;
        return;
      }
      rank -= __popc(m);
    }
  }
};

// a[i] = min(a[i], v) between threads (shared memory; for the rare values that are not finite).
__device__ __forceinline__ void min_u16(uint16_t* a, int i, int v) {
  unsigned* word = reinterpret_cast<unsigned*>(a + (i & ~1));
  const int sh = 16 * (i & 1);
  unsigned old = *reinterpret_cast<volatile unsigned*>(word);
  while ((int)(old >> sh & 0xffffu) > v) {
    const unsigned seen = atomicCAS(word, old, (old & ~(0xffffu << sh)) | ((unsigned)v << sh));
    if (seen == old) break;
    old = seen;
  }
}

struct PromptItem {
  int found, row0, n, i0, kv;   // first packed row and length of the sequence, first token of the block
};

template <int D>
__global__ void __launch_bounds__(kPrThreads, 1) prompt_kernel(const __grid_constant__ PromptArgs a) {
  using S = PrShape<D>;
  extern __shared__ unsigned char dsm_raw[];
  unsigned char* base = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(dsm_raw) + 1023) & ~(uintptr_t)1023);
  unsigned char* sQ = base;                // two query tiles
  unsigned char* sK = sQ + 2 * S::QT;      // two key slots
  unsigned char* sV = sK + 2 * S::KT;      // two value slots
  unsigned char* sO = sV + 2 * S::KT;      // output staging, one area per softmax warp
  __shared__ __align__(8) uint64_t q_full, q_empty, k_full[2], k_empty[2], v_full[2], v_empty[2], v_clean[2], s_full[2],
      p_ready[2], o_done[2], item_full[2], item_empty[2], item_clean[2], drained;
  __shared__ uint32_t s_tmem;
  __shared__ PromptItem s_item[2];
  // what value tiles held that is not finite, per item slot: first row of a column's NaN, +inf, -inf, counted
  // from the first masked key tile
  __shared__ __align__(4) uint16_t s_first[2][3][D];
  __shared__ int s_odd[2];                 // any of them

  const int tid = threadIdx.x, warp = __shfl_sync(kFull, tid >> 5, 0), lane = tid & 31;
  const int block = 2 * a.tokens;
  const uint64_t settle = a.wait_ns > kWaitLimitNs ? a.wait_ns : kWaitLimitNs;   // for what is in flight at the end

  if (warp == kPrSoftmaxWarps + 1) {
    tmem_alloc(&s_tmem, S::TMEM_COLS);
    tmem_relinquish();
  }
  if (tid == 0) {
    mbar_init(&q_full, 1);
    mbar_init(&q_empty, 1);
    mbar_init(&drained, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&k_full[i], 1);
      mbar_init(&k_empty[i], 1);
      mbar_init(&v_full[i], 1);
      mbar_init(&v_empty[i], 2);           // the products and the look through
      mbar_init(&v_clean[i], 1);
      mbar_init(&s_full[i], 1);
      mbar_init(&p_ready[i], kPrSoftmaxWarps / 2);
      mbar_init(&o_done[i], 1);
      mbar_init(&item_full[i], 1);
      mbar_init(&item_empty[i], kPrSoftmaxWarps + 3);
      mbar_init(&item_clean[i], 1);
      s_odd[i] = 0;
    }
    mbar_fence_init();
  }
  for (int i = tid; i < 2 * 3 * D; i += kPrThreads) (&s_first[0][0][0])[i] = kPrNone;
  tc_fence_before();
  BlockOrder order;                        // (of warp 10, its loads under way before the others are set up)
  if (warp == kPrSoftmaxWarps + 2) order.init(a, block, lane);
  if (warp == kPrSoftmaxWarps && lane == 0) {
    prefetch_tmap(&a.q);
    prefetch_tmap(&a.k);
    prefetch_tmap(&a.v);
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;

  // Item k of this CTA is in slot k % 2. From it every role derives the same: key tiles of the two query
  // tiles (0: the tile lies past the sequence), the number of key tiles, the first one that holds a key past
  // the block's first token (128 j + 127 > i0).
  auto read_item = [&](int k, PromptItem& it, int (&nt)[2], int& ntiles, int& masked_from) -> bool {
    if (!mbar_wait(&item_full[k & 1], (k >> 1) & 1, a.wait_ns)) return false;
    it = s_item[k & 1];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int first = it.i0 + i * a.tokens;
      nt[i] = first < it.n ? (min(first + a.tokens, it.n) + kPrKeys - 1) / kPrKeys : 0;
    }
    ntiles = max(nt[0], nt[1]);
    masked_from = (it.i0 + 1) / kPrKeys;
    return true;
  };
  PromptItem it;
  int nt[2], ntiles, masked_from;

  if (warp >= kPrSoftmaxWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kPrOtherRegs));
    if (warp == kPrSoftmaxWarps) {
      // ---------------------------------------------------------------- loads
      if (lane == 0) {
        bool ok = true;
        int items = 0, kn = 0, vn = 0;                            // loaded so far: items' queries, K tiles, V tiles
        for (;;) {
          ok = read_item(items, it, nt, ntiles, masked_from);
          if (!ok) break;
          mbar_arrive(&item_empty[items & 1]);
          if (!it.found) break;
          if (items > 0) ok = mbar_wait(&q_empty, (items - 1) & 1, a.wait_ns);
          if (!ok) break;
          mbar_arrive_expect_tx(&q_full, (uint32_t)(2 * S::HALVES * a.G * a.tokens * 128));
          for (int i = 0; i < 2; ++i)
            for (int h = 0; h < S::HALVES; ++h)
              tma_load_3d(sQ + i * S::QT + h * (kPrRows * 128), &a.q, h * 64, it.kv * a.G, it.row0 + it.i0 + i * a.tokens,
                          &q_full);
          ++items;
          for (int j = 0; j < ntiles && ok; ++j) {
            int s = kn & 1;
            if (kn >= 2) ok = mbar_wait(&k_empty[s], ((kn >> 1) - 1) & 1, a.wait_ns);
            if (!ok) break;
            mbar_arrive_expect_tx(&k_full[s], S::KT);
            for (int h = 0; h < S::HALVES; ++h)
              tma_load_3d(sK + s * S::KT + h * (kPrKeys * 128), &a.k, h * 64, it.kv, it.row0 + j * kPrKeys, &k_full[s]);
            ++kn;
            s = vn & 1;
            if (vn >= 2) ok = mbar_wait(&v_empty[s], ((vn >> 1) - 1) & 1, a.wait_ns);
            if (!ok) break;
            mbar_arrive_expect_tx(&v_full[s], S::KT);
            for (int h = 0; h < S::HALVES; ++h)
              tma_load_3d(sV + s * S::KT + h * (kPrKeys * 128), &a.v, h * 64, it.kv, it.row0 + j * kPrKeys, &v_full[s]);
            ++vn;
          }
          if (!ok) break;
        }
        if (!ok) set_error(a.status, TS_ERR_TIMEOUT);
        // nothing may still be landing when the CTA exits, however short the limit was that a role gave up at
        if (items > 0) mbar_wait(&q_full, (items - 1) & 1, settle);
        for (int j = max(0, kn - 2); j < kn; ++j) mbar_wait(&k_full[j & 1], (j >> 1) & 1, settle);
        for (int j = max(0, vn - 2); j < vn; ++j) mbar_wait(&v_full[j & 1], (j >> 1) & 1, settle);
      }
      __syncwarp();
    } else if (warp == kPrSoftmaxWarps + 1) {
      // ------------------------------------------------------------- products
      // The whole warp goes through the loop and one lane issues: with descriptors built by one diverged
      // thread an instruction took 115 cycles to issue where the tensor cores need 64.
      const uint32_t idesc_s = idesc_bf16_f32(kPrRows, kPrKeys) | (a.negate ? 1u << 13 : 0u);   // bit 13: -A
      constexpr uint32_t idesc_o = idesc_bf16_f32_bmn(kPrRows, D);
      const uint64_t dq = sdesc_sw128(smem_addr(sQ)), dk = sdesc_sw128(smem_addr(sK));
      const uint64_t dv = sdesc_sw128_mn(smem_addr(sV), kPrKeys * 128, 1024);
      const uint32_t q_lo = (uint32_t)dq, k_lo = (uint32_t)dk, v_lo = (uint32_t)dv;
      const uint32_t qk_hi = (uint32_t)(dq >> 32), v_hi = (uint32_t)(dv >> 32);
      auto scores = [&](int i, int slot) {
        const uint32_t ql = q_lo + i * (S::QT >> 4), kl = k_lo + slot * (S::KT >> 4);
        if (elect_one()) {
#pragma unroll
          for (int h = 0; h < S::HALVES; ++h)
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
              umma_bf16(tmem + S::S_COL + 128 * i, sdesc_from(ql + ((h * (kPrRows * 128) + ks * 32) >> 4), qk_hi),
                        sdesc_from(kl + ((h * (kPrKeys * 128) + ks * 32) >> 4), qk_hi), idesc_s, (h | ks) != 0);
          umma_commit(&s_full[i]);
        }
        __syncwarp();
      };
      auto commit = [&](uint64_t* bar) {
        if (elect_one()) umma_commit(bar);
        __syncwarp();
      };
      auto wait = [&](uint64_t* bar, uint32_t parity) -> bool { return __all_sync(kFull, mbar_wait(bar, parity, a.wait_ns)); };
      bool ok = true;
      int kt = 0;                                                 // key tiles of the items before
      uint32_t clean_par = 0u, p_par = 0u;                        // parities of the next waits, by slot and by tile
      for (int k = 0;; ++k) {
        ok = __all_sync(kFull, read_item(k, it, nt, ntiles, masked_from));
        if (!ok) break;
        const bool found = __shfl_sync(kFull, it.found, 0) != 0;
#pragma unroll
        for (int i = 0; i < 2; ++i) nt[i] = __shfl_sync(kFull, nt[i], 0);
        ntiles = max(nt[0], nt[1]);
        masked_from = __shfl_sync(kFull, masked_from, 0);
        if (lane == 0) mbar_arrive(&item_empty[k & 1]);
        __syncwarp();
        if (!found) break;
        ok = wait(&q_full, k & 1) && wait(&k_full[kt & 1], (kt >> 1) & 1);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int i = 0; i < 2; ++i)
          if (nt[i] > 0) scores(i, kt & 1);
        commit(&k_empty[kt & 1]);
        if (ntiles == 1) commit(&q_empty);
        for (int j = 0; j < ntiles && ok; ++j) {
          const int g = kt + j, s = g & 1, s1 = s ^ 1;
          ok = wait(&v_full[s], (g >> 1) & 1);
          if (ok && j >= masked_from) {
            ok = wait(&v_clean[s], (clean_par >> s) & 1u);
            clean_par ^= 1u << s;
          }
          if (ok && j + 1 < ntiles) ok = wait(&k_full[s1], ((g + 1) >> 1) & 1);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            if (!ok || j >= nt[i]) continue;
            const uint32_t vl = v_lo + s * (S::KT >> 4);
            ok = wait(&p_ready[i], (p_par >> i) & 1u);
            if (!ok) continue;
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
              for (int ks = 0; ks < kPrKeys / 16; ++ks)
                umma_bf16_ts(tmem + S::O_COL + 128 * i, tmem + S::S_COL + 128 * i + 8 * ks,
                             sdesc_from(vl + ((ks * 2048) >> 4), v_hi), idesc_o, (j | ks) != 0);
              umma_commit(&o_done[i]);
            }
            __syncwarp();
            p_par ^= 1u << i;
            if (j + 1 < nt[i]) scores(i, s1);
          }
          if (ok) {
            commit(&v_empty[s]);
            if (j + 1 < ntiles) commit(&k_empty[s1]);
            if (j + 2 == ntiles) commit(&q_empty);
          }
        }
        if (!ok) break;
        kt += ntiles;
      }
      if (!ok && lane == 0) set_error(a.status, TS_ERR_TIMEOUT);
      // no product may be under way when tensor memory is given back
      commit(&drained);
      mbar_wait(&drained, 0, settle);
      __syncwarp();
    } else if (warp == kPrSoftmaxWarps + 2) {
      // ---------------------------------------------------------------- items
      if (blockIdx.x == 0)
        for (int b = lane; b <= a.B; b += 32) {
          const int v = a.cu[b];
          if (v > a.total || (b == 0 ? v != 0 : v < a.cu[b - 1])) set_error(a.status, TS_ERR_SEQ_LEN);
        }
      int level = order.most;
      bool found = true;
      for (int k = 0; found; ++k) {
        const int64_t t = (int64_t)k * gridDim.x + (k & 1 ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
        int seq = 0, blk = 0;
        found = t < (int64_t)order.all * a.HKV;
        if (found) order.find(a, block, (int)(t / a.HKV), level, lane, seq, blk);
        const int row0 = seq < 128 ? __shfl_sync(kFull, seq < 32 ? order.start[0] : seq < 64 ? order.start[1] : seq < 96 ? order.start[2] : order.start[3], seq & 31)
                                   : a.cu[seq];
        const int end = a.cu[seq + 1];
        if (k >= 2 && !mbar_wait(&item_empty[k & 1], ((k >> 1) - 1) & 1, a.wait_ns)) {
          set_error(a.status, TS_ERR_TIMEOUT);
          break;
        }
        if (s_odd[k & 1]) {
          for (int i = lane; i < 3 * D; i += 32) (&s_first[k & 1][0][0])[i] = kPrNone;
          __syncwarp();
          if (lane == 0) s_odd[k & 1] = 0;
        }
        __syncwarp();
        if (lane == 0) {
          s_item[k & 1] = PromptItem{found, row0, end - row0, blk * block, (int)(t % a.HKV)};
          mbar_arrive(&item_full[k & 1]);
        }
        __syncwarp();
      }
    } else {
      // --------------------------------------------- what is not finite behind the diagonal
      bool ok = true;
      int kt = 0;
      for (int k = 0;; ++k) {
        ok = __all_sync(kFull, read_item(k, it, nt, ntiles, masked_from));
        if (!ok || !it.found) break;
        for (int j = 0; j < ntiles && ok; ++j) {
          const int vs = (kt + j) & 1;
          ok = __all_sync(kFull, mbar_wait(&v_full[vs], ((kt + j) >> 1) & 1, a.wait_ns));
          if (!ok) break;
          if (j >= masked_from) {
            // the values of rows behind token i0 that are not finite come out of the tile
            unsigned char* vt = sV + vs * S::KT;
            uint32_t odd = 0u;
#pragma unroll 8
            for (int c = 0; c < S::KT / 512; ++c) {
              const uint4 w = lds128(vt + c * 512 + lane * 16);
              odd |= ((w.x & 0x7f807f80u) + 0x00800080u) | ((w.y & 0x7f807f80u) + 0x00800080u) |
                     ((w.z & 0x7f807f80u) + 0x00800080u) | ((w.w & 0x7f807f80u) + 0x00800080u);
            }
            if (odd & 0x80008000u) {
              for (int off = lane * 16; off < S::KT; off += 512) {               // byte in the tile
                const int r = (off % (kPrKeys * 128)) / 128, key = j * kPrKeys + r;
                const int col0 = off / (kPrKeys * 128) * 64 + (((off / 16) % 8) ^ (r & 7)) * 8;
                if (key <= it.i0) continue;                       // every row of the block sees it
                uint16_t* e16 = reinterpret_cast<uint16_t*>(vt + off);
                for (int e = 0; e < 8; ++e) {
                  const uint32_t u = e16[e];
                  if ((u & 0x7f80u) != 0x7f80u) continue;
                  min_u16(s_first[k & 1][(u & 0x7fu) ? 0 : (u >> 15 ? 2 : 1)], col0 + e, key - masked_from * kPrKeys);
                  e16[e] = 0;
                  s_odd[k & 1] = 1;
                }
              }
            }
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) mbar_arrive(&v_clean[vs]);
          }
          // (also for the tiles not looked at: so this warp never falls a round behind the value slots)
          if (lane == 0) mbar_arrive(&v_empty[vs]);
          __syncwarp();
        }
        if (!ok) break;
        kt += ntiles;
        if (lane == 0) {
          mbar_arrive(&item_clean[k & 1]);
          mbar_arrive(&item_empty[k & 1]);
        }
        __syncwarp();
      }
      if (!ok && lane == 0) set_error(a.status, TS_ERR_TIMEOUT);
    }
  } else {
    // ---------------------------------------------------------------- softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kPrSoftmaxRegs));
    const int i = warp >> 2;                                      // tile
    const int row = 32 * (warp & 3) + lane;
    const uint32_t inv_g = 65536u / (uint32_t)a.G + 1u;           // r / G = (r inv_g) >> 16 for r < 128, G <= 16
    const uint32_t lane_off = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t tS = tmem + S::S_COL + 128 * i + lane_off, tO = tmem + S::O_COL + 128 * i + lane_off;
    bool ok = true;
    uint32_t s_par = 0u;                                          // parity of the next score tile
    for (int k = 0; ok; ++k) {
      ok = __all_sync(kFull, read_item(k, it, nt, ntiles, masked_from));
      if (!ok || !it.found) break;
      const int mine = __shfl_sync(kFull, i == 0 ? nt[0] : nt[1], 0), slot = k & 1;
      if (mine > 0) {                                             // (else the tile lies past the sequence's end)
        const int first = it.i0 + i * a.tokens;                   // first token of the tile
        const int row_tok = (int)((uint32_t)row * inv_g >> 16), tok = first + row_tok;
        const bool real = row_tok < a.tokens && tok < it.n;
        float mx = -INFINITY, la = 0.f, lb = 0.f;                 // running maximum (unscaled) and two halves of the sum
        for (int j = 0; j < mine; ++j) {
          ok = __all_sync(kFull, mbar_wait(&s_full[i], s_par, a.wait_ns));
          if (!ok) break;
          tc_fence_after();
          // Weights against the maximum that the row has, which covers most tiles. Where their sum says that
          // it does not (and in the first tile, which has none), the scores, still in tensor memory, are read
          // again and the maximum is taken first.
          uint32_t p[64];
          float ta, tb, m2 = mx * a.scale2;
          bool over = real;                                       // this row needs its maximum (in a pass that takes it)
          for (bool raise = j == 0;; raise = true) {
            uint32_t u[128];
#pragma unroll
            for (int c = 0; c < 4; ++c) tmem_ld_x32(tS + 32 * c, u + 32 * c);
            tmem_wait_ld();
            float* x = reinterpret_cast<float*>(u);
            if (j * kPrKeys + kPrKeys - 1 > first) {              // the tile holds keys that a row may not see
              const int lim = tok - j * kPrKeys;                  // ascending with the lanes
              const int low = __shfl_sync(kFull, lim, 0);
#pragma unroll
              for (int c0 = 0; c0 < 128; c0 += 32) {
                if (low < c0 + 31) {                              // (else every row of the warp sees these 32)
#pragma unroll
                  for (int c = c0; c < c0 + 32; ++c) x[c] = c <= lim ? x[c] : -INFINITY;
                }
              }
            }
            if (raise) {
              float ma = x[0], mb = x[1];
#pragma unroll
              for (int c = 2; c < 128; c += 2) {
                ma = fmaxf(ma, x[c]);
                mb = fmaxf(mb, x[c + 1]);
              }
              // each row by itself, so that no row's bits depend on another's: rows that do not need it keep their
              // maximum, as do rows that are no query of the sequence (their operands may be anything)
              const float mn = over ? fmaxf(mx, fmaxf(ma, mb)) : mx, n2 = mn * a.scale2;
              // from the reference that the row's weights had to the one that they get (far maxima: the exact product)
              const float d = far(m2) ? (far(n2) ? (mx - mn) * a.scale2 : fmaf(mx, a.scale2, -n2))
                                      : (far(n2) ? -fmaf(mn, a.scale2, -m2) : m2 - n2);
              const float f = mn == mx ? 1.f : pr_ex2(d);
              mx = mn;
              m2 = n2;
              la *= f;
              lb *= f;
              if (j > 0) {
                // the tile's last product must be in before its accumulators are rescaled
                ok = __all_sync(kFull, mbar_wait(&o_done[i], s_par ^ 1u, a.wait_ns));
                if (!ok) break;
                tc_fence_after();
                // (rare, and the scores hold most registers: eight columns at a time)
#pragma unroll 1
                for (int c = 0; c < D; c += 8) {
                  float o[8];
                  tmem_ld_x8(tO + c, o);
                  tmem_wait_ld();
#pragma unroll
                  for (int e = 0; e < 8; ++e) o[e] *= f;
                  tmem_st_x8(tO + c, o);
                }
              }
            }
            float ms = m2 == -INFINITY ? 0.f : -m2;               // nothing seen yet: every weight is zero
            if (raise && __any_sync(kFull, far(m2) && m2 != -INFINITY)) {
              const bool shift = far(m2) && m2 != -INFINITY;
              const float off = shift ? mx : 0.f;
              ms = shift ? 0.f : ms;
#pragma unroll
              for (int c = 0; c < 128; c += 2) add2(x[c], x[c + 1], -off, -off);
            }
            const uint64_t sc = pack_f2(a.scale2, a.scale2), mm = pack_f2(ms, ms);
            ta = tb = 0.f;
#pragma unroll
            for (int c = 0; c < 64; ++c) {
              float y0, y1;
              unpack_f2(fma_f2(pack_f2(x[2 * c], x[2 * c + 1]), sc, mm), y0, y1);
              y0 = pr_ex2(y0);
              y1 = pr_ex2(y1);
              add2(ta, tb, y0, y1);
              p[c] = pack_bf16(y0, y1);
            }
            if (raise) break;
            over = real && (!(ta + tb <= kPrMaxSum) || far(m2));
            if (!__any_sync(kFull, over)) break;
          }
          if (!ok) break;
          la += ta;
          lb += tb;
          tmem_st_x32(tS, p);
          tmem_st_x32(tS + 32, p + 32);
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&p_ready[i]);
          s_par ^= 1u;
        }
        // ---- outputs
        if (ok) ok = __all_sync(kFull, mbar_wait(&o_done[i], s_par ^ 1u, a.wait_ns));
        if (ok) ok = __all_sync(kFull, mbar_wait(&item_clean[slot], (k >> 1) & 1, a.wait_ns));
        if (ok) {
          tc_fence_after();
          const float l = la + lb, inv = 1.f / l;
          const bool odd = s_odd[slot] != 0;
          const int row0 = s_item[slot].row0, head = s_item[slot].kv * a.G + row - row_tok * a.G;
          if (real && a.lse) a.lse[(int64_t)(row0 + tok) * a.H + head] = (mx * a.scale2 + log2f(l)) * 0.6931471805599453f;
          // this lane's output row; a null pointer where it is none
          const uint64_t dst = real ? reinterpret_cast<uint64_t>(a.out + (int64_t)(row0 + tok) * a.out_stride + (int64_t)head * D) : 0u;
          unsigned char* stage = sO + warp * S::STAGE;
#pragma unroll 1
          for (int h = 0; h < S::HALVES; ++h) {
            // 64 columns of 32 rows through this warp's staging area (swizzled like the operands), so that a
            // store covers whole 128-byte pieces of four rows instead of 16 bytes of 32
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              uint32_t o[32];
              tmem_ld_x32(tO + 64 * h + 32 * c, o);
              tmem_wait_ld();
              if (odd) {
#pragma unroll
                for (int e = 0; e < 32; ++e) {
                  const int col = 64 * h + 32 * c + e;
                  const int at = tok - masked_from * kPrKeys;      // (below 4 tiles: kPrNone is never reached)
                  float add = at >= s_first[slot][1][col] ? INFINITY : 0.f;
                  if (at >= s_first[slot][2][col]) add += -INFINITY;
                  if (at >= s_first[slot][0][col]) add = NAN;
                  o[e] = __float_as_uint(__uint_as_float(o[e]) + add);
                }
              }
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                uint32_t w[4];
#pragma unroll
                for (int z = 0; z < 4; ++z)
                  w[z] = pack_bf16(__uint_as_float(o[8 * e + 2 * z]) * inv, __uint_as_float(o[8 * e + 2 * z + 1]) * inv);
                *reinterpret_cast<uint4*>(stage + lane * 128 + (((4 * c + e) ^ (lane & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
              }
            }
            __syncwarp();
#pragma unroll
            for (int r4 = 0; r4 < 8; ++r4) {
              const int rl = 4 * r4 + (lane >> 3), c16 = lane & 7;
              const uint64_t to = __shfl_sync(kFull, dst, rl);
              const uint4 v = lds128(stage + rl * 128 + ((c16 ^ (rl & 7)) << 4));
              if (to) *reinterpret_cast<uint4*>(to + 128 * h + c16 * 16) = v;
            }
            __syncwarp();
          }
          // the accumulators have been read before the next item's weights let a product write them
          tc_fence_before();
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&item_empty[slot]);
    }
    if (!ok && lane == 0) set_error(a.status, TS_ERR_TIMEOUT);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kPrSoftmaxWarps + 1) {
    tc_fence_after();
    tmem_dealloc(tmem, S::TMEM_COLS);
  }
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
  // a sequence has at most one block that is not full; one CTA per SM where there are that many
  const int64_t items = ((int64_t)c.total / (2 * a.tokens) + (c.B < c.total ? c.B : c.total)) * a.HKV;
  const int64_t grid = items < ctx->num_sms ? items : ctx->num_sms;
  return cfg.head_dim == 64 ? run_prompt<64>(ctx, a, grid, s) : run_prompt<128>(ctx, a, grid, s);
}

}  // namespace ts
