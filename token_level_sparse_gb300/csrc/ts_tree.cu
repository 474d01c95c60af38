// Attention of drafted tokens over a paged cache: the last T cached tokens of a sequence are the nodes of a tree of drafts
// (or the newest tokens of a sequence); each sees the whole prefix and those of the T that its mask names, or
// that come before it.
//
//   s[r][j] = scale <q_r, k_j>      out_r = sum_j 2^(s' - m) v_j / sum_j 2^(s' - m)      (seen j; s' = s log2(e))
//
// Every K and V row is needed once per KV head, 4 d bytes, for 4 d G T operations: bound by memory up to G T of
// about 256 rows, by the tensor cores from there on. Both products run on tcgen05 with their accumulators in tensor
// memory, as for whole prompts (the softmax with its running maximum is the same), and K and V come page by page.
//
// A tile is 128 query rows of one KV head: 128 / G tokens with all G query heads of the group; a block is two
// neighbouring tiles, which share every key and value tile of 128 tokens. The key tiles of all blocks of all KV heads and
// sequences, one behind another, are dealt to one CTA per SM in contiguous shares of equal work, whatever the lengths are. A
// share that begins or ends inside a block leaves its sums in fp32 (unnormalised, with maximum and sum), and a second kernel
// joins them, in order: the same bits every time. Roles of a CTA:
//   warp 8      loads: the query tiles of an item, then K and V pages (TMA, 128-byte swizzle) into a ring of tiles
//   warp 9      products: S = Q K^T, O += P V
//   warp 10     finds the items of the share
//   warp 11     looks through the value tiles that hold drafts or end the sequence (below)
//   warps 0-3   softmax of tile 0, a thread per row; outputs
//   warps 4-7   the same of tile 1. Where a block has one tile they have nothing to do, and tile 0 uses both score
//               buffers in turn, so that the next scores are there when a softmax ends.
//
// Masked places hold what they hold: a score that is not seen is replaced before it is used. A value that is not
// finite would reach other rows through a weight of zero, so among the drafts (and behind the sequence's end, where a page may
// never have been written) such values come out of the tile in shared memory, their tokens are noted, and the rows that see
// them get them back in the outputs, read from the pool.
//
// A weight enters its product as one bf16 number (the sum takes it unrounded), as in the prompt attention: the largest
// error beside the rounding of the outputs, 2.3e-3 of them where their rounding alone leaves 1.7e-3.
//
// Measured, 32 heads over 8 of 128: up to 32 drafts over 262,144 tokens 168 us, 6.4 TB/s (memory); 64 drafts 211 us, 1.3
// PFLOP/s (a key tile's chain of scores, softmax, outputs, 3200 cycles, of which the tensor cores work 2050); 64 over 131,057
// 121 us, of which the join is 12. One-token pages: 826 us, as each of a tile's 256 copies moves 128 bytes (822 with one draft); d 64,
// 8 heads over 4, 262,144 tokens: 76 us with 64 drafts, 101 with 128. Key tiles of 64 tokens with two score buffers to a query
// tile let those overlap better, but each change from one kind of product to the other costs the tensor cores about 150 cycles,
// and twice as many cost more (128).
#include <cmath>

#include "ts_flash.cuh"

namespace ts {
namespace {

constexpr int kTrRows = 128;     // query rows of a tile
constexpr int kTrKeys = 128;     // tokens of a key tile
constexpr int kTrSoftmaxWarps = 8;
constexpr int kTrThreads = (kTrSoftmaxWarps + 4) * 32;
// Registers a thread: 168 at launch (65536 / 384), shared out as in the prompt attention.
constexpr int kTrSoftmaxRegs = 208, kTrOtherRegs = 88;
static_assert(2 * kTrSoftmaxRegs + kTrOtherRegs <= 3 * 168, "register shares");
// What is kept per key tile, for the last eight: the ring holds a value tile that is in use and SLOTS - 1 tiles behind it, every
// second one keys, so nothing is more than six key tiles ahead of anything.
constexpr int kTrRing = 8;
constexpr float kTrMaxSum = 16384.f;   // of a tile's weights against a maximum taken earlier

constexpr int kJoinParts = 256;  // CTAs of a call, at most

struct TreeArgs {
  CUtensorMap q, k, v;           // q [rows][heads][d]; k, v [pages][heads * page size][d]
  const int32_t* cu;
  const int32_t* seq_lens;
  const int32_t* page_table;
  int pt_stride, page_shift;
  int64_t num_pages;
  int max_tokens;
  const uint32_t* mask;          // or null: causal
  int mask_words;
  const __nv_bfloat16* v_pool;
  int B, total;
  int H, HKV, G;
  int tokens;                    // tokens of a tile: 128 / G
  float scale2;                  // |scale| log2(e)
  int negate;                    // scale < 0: the products are taken with -Q
  __nv_bfloat16* out;
  int64_t out_stride;
  float* lse;
  float* part_o;                 // [2 slots per CTA][d / 4][256 rows][4]
  float2* part_ml;               // [2 slots per CTA][256 rows]: maximum (unscaled), sum
  int* status;
  uint64_t wait_ns;
};

template <int D>
struct TrShape {
  static constexpr int HALVES = D / 64;
  static constexpr int QT = kTrRows * D * 2;    // bytes of a query tile
  static constexpr int KT = kTrKeys * D * 2;    // bytes of a key or value tile
  static constexpr int SLOTS = D == 128 ? 5 : 10;   // key and value tiles under way or in use
  static constexpr int SMEM = 2 * QT + SLOTS * KT + 1024;
  static_assert(SMEM + 1536 <= 227 * 1024, "shared memory of an SM");
  static constexpr uint32_t TMEM_COLS = 512;
  // score buffer x at 128 x (weights over its first 64 columns): tile x's, or in a block with one tile the one of every
  // second key tile; outputs of tile i at 256 + 128 i
  static constexpr uint32_t S_COL = 0, O_COL = 256;
};

// Work is counted per key tile: one of a block with two tiles takes longer, 262,144 tokens of 8 KV heads with G 4 201 to 211 us
// (33 to 64 drafts) where a block with one tile takes 168 (up to 32); more in one batch, where those wait less for memory. A block
// (its queries, first softmax and outputs) counts as four units beside its tiles, what two key tiles of a block with one
// tile count or one and a third of a block with two. Set by timings of 16-token pages with d 128 and G 4 and 7; the same for
// the others, where only how even the shares are hangs on it.
constexpr int kTrPair = 3, kTrSingle = 2, kTrBlock = 4;

// A sequence's work: its KV heads one behind another, of each the blocks, of each the key tiles.
struct TreeSeq {
  int row0, T, n;                // first packed row, drafts, cached tokens (drafts among them)
  int blocks, tiles;             // blocks of drafts, key tiles of a block
  int last;                      // work of a key tile of the last block (of the others: kTrPair)
  int err;
  // of a block that is not the last one, and of a KV head
  __device__ __forceinline__ int64_t block() const { return kTrBlock + (int64_t)kTrPair * tiles; }
  __device__ __forceinline__ int64_t head() const { return blocks > 0 ? block() * (blocks - 1) + kTrBlock + (int64_t)last * tiles : 0; }
};

__device__ __forceinline__ TreeSeq tree_seq(const TreeArgs& a, int b) {
  TreeSeq s;
  s.row0 = a.cu[b];
  const int end = a.cu[b + 1];
  s.T = end - s.row0;
  s.n = a.seq_lens[b];
  const bool rows_ok = s.row0 >= 0 && end >= s.row0 && end <= a.total && (b != 0 || s.row0 == 0);
  const bool ok = rows_ok && s.T <= kMaxTree && (!a.mask || s.T <= 32 * a.mask_words) && s.n >= s.T && s.n <= a.max_tokens;
  s.err = ok ? 0 : TS_ERR_SEQ_LEN;
  s.blocks = ok ? (s.T + 2 * a.tokens - 1) / (2 * a.tokens) : 0;
  s.tiles = ok ? (s.n + kTrKeys - 1) / kTrKeys : 0;
  s.last = s.T - (s.blocks - 1) * 2 * a.tokens > a.tokens ? kTrPair : kTrSingle;
  return s;
}

// Running sums over the lanes.
__device__ __forceinline__ int64_t warp_scan_ll(int64_t x, int lane) {
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t o = __shfl_up_sync(kFull, x, d);
    if (lane >= d) x += o;
  }
  return x;
}

// Where the share of CTA c begins, and whose share a place is in. A key tile belongs to the share that its beginning lies
// in (a share may have none).
__device__ __forceinline__ int64_t share_begin(int64_t work, int ctas, int c) { return work * c / ctas; }
__device__ __forceinline__ int share_of(int64_t work, int ctas, int64_t at) { return (int)(((at + 1) * ctas - 1) / work); }
// The first of `tiles` key tiles, beginning at `at` and every `per` from there on, that begins at a place or behind it.
__device__ __forceinline__ int first_tile(int64_t at, int per, int tiles, int64_t place) {
  return place <= at ? 0 : (int)min((int64_t)tiles, (place - at + per - 1) / per);
}

// Places in the ring of an item's key tile j and value tile j, counted from its first: K(0), K(1), V(0), K(2), V(1), ...
__device__ __forceinline__ uint32_t key_load(int j) { return j == 0 ? 0u : 2u * (uint32_t)j - 1u; }
__device__ __forceinline__ uint32_t value_load(int j, int nt) { return (uint32_t)min(2 * j + 2, 2 * nt - 1); }

struct TreeItem {
  int found, row0, T, n, i0;     // sequence; first token (among the drafts) of the block
  int b, kv, j0, j1;             // key tiles [j0, j1) of the block
  int slot;                      // where the sums go; -1: the whole block, outputs
};

// Exponent from reference (ma, a2) to (mb, b2), maxima unscaled and scaled: by the numbers that the weights were taken
// against where fp32 holds those, else from the exact product.
__device__ __forceinline__ float from_to(float ma, float a2, float mb, float b2, float scale2) {
  return far(a2) ? (far(b2) ? (ma - mb) * scale2 : fmaf(ma, scale2, -b2)) : (far(b2) ? -fmaf(mb, scale2, -a2) : a2 - b2);
}

// Which of the 32 tokens from draft k on (k may lie before the first) draft `tok`, packed row `row`, sees.
__device__ __forceinline__ uint32_t seen_bits(const TreeArgs& a, int row, int tok, int T, int k) {
  uint32_t m;
  if (a.mask) {
    const uint32_t* words = a.mask + (int64_t)row * a.mask_words;
    const int at = k >> 5, last = (T + 31) >> 5;                  // (an arithmetic shift)
    const uint32_t lo = at >= 0 && at < last ? words[at] : (at < 0 ? 0xffffffffu : 0u);
    const uint32_t hi = at + 1 >= 0 && at + 1 < last ? words[at + 1] : (at + 1 < 0 ? 0xffffffffu : 0u);
    m = __funnelshift_r(lo, hi, k & 31);
  } else {
    const int lim = tok - k;                   // the last seen bit
    m = lim < 0 ? 0u : (lim >= 31 ? 0xffffffffu : (2u << lim) - 1u);
  }
  const int left = T - k;                      // bits before the sequence's end
  return left >= 32 ? m : left <= 0 ? 0u : m & ((1u << left) - 1u);
}

template <int D>
__global__ void __launch_bounds__(kTrThreads, 1) tree_kernel(const __grid_constant__ TreeArgs a) {
  using S = TrShape<D>;
  extern __shared__ unsigned char dsm_raw[];
  unsigned char* base = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(dsm_raw) + 1023) & ~(uintptr_t)1023);
  unsigned char* sQ = base;                // two query tiles
  unsigned char* sKV = sQ + 2 * S::QT;     // key and value tiles, a ring in the order of their use
  __shared__ __align__(8) uint64_t q_full, q_empty, full[S::SLOTS], empty[S::SLOTS], v_clean[kTrRing], s_full[3], p_ready[3],
      o_done[3], item_full[2], item_empty[2], item_clean[2], drained;
  __shared__ uint32_t s_tmem;
  __shared__ TreeItem s_item[2];
  __shared__ uint32_t s_odd[2][kMaxTree / 32];   // drafts whose values are not all finite, per item slot
  __shared__ int s_any_odd[2];
  // keys of a tile whose page lies outside the pool, and whether there are any
  __shared__ uint32_t s_bad[kTrRing][4];
  __shared__ uint32_t s_any_bad[kTrRing];

  const int tid = threadIdx.x, warp = __shfl_sync(kFull, tid >> 5, 0), lane = tid & 31;
  const uint64_t settle = a.wait_ns > kWaitLimitNs ? a.wait_ns : kWaitLimitNs;   // for what is in flight at the end

  if (warp == kTrSoftmaxWarps + 1) {
    tmem_alloc(&s_tmem, S::TMEM_COLS);
    tmem_relinquish();
  }
  if (tid == 0) {
    mbar_init(&q_full, 1);
    mbar_init(&q_empty, 1);
    mbar_init(&drained, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&item_full[i], 1);
      mbar_init(&item_empty[i], kTrSoftmaxWarps + 3);
      mbar_init(&item_clean[i], 1);
      s_any_odd[i] = 0;
    }
    for (int i = 0; i < S::SLOTS; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 2);             // the products and the look through
    }
    for (int i = 0; i < kTrRing; ++i) mbar_init(&v_clean[i], 1);
    for (int i = 0; i < 3; ++i) {          // tile 0, tile 1, and every second key tile of a block with one tile
      mbar_init(&s_full[i], 1);
      mbar_init(&p_ready[i], kTrSoftmaxWarps / 2);
      mbar_init(&o_done[i], 1);
    }
    mbar_fence_init();
  }
  if (tid < 2 * (kMaxTree / 32)) (&s_odd[0][0])[tid] = 0u;
  tc_fence_before();
  if (warp == kTrSoftmaxWarps && lane == 0) {
    prefetch_tmap(&a.q);
    prefetch_tmap(&a.k);
    prefetch_tmap(&a.v);
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // the join may set itself up where there is room

  // Item k of this CTA is in slot k % 2. From it every role derives the same: whether the block has a second tile, the
  // first key tile that holds drafts (or what is behind the sequence).
  auto read_item = [&](int k, TreeItem& it, bool& two, int& drafts_from) -> bool {
    if (!mbar_wait(&item_full[k & 1], (k >> 1) & 1, a.wait_ns)) return false;
    it = s_item[k & 1];
    two = it.i0 + a.tokens < it.T;
    drafts_from = (it.n - it.T) / kTrKeys;
    return true;
  };
  TreeItem it;
  bool two;
  int drafts_from;

  if (warp >= kTrSoftmaxWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kTrOtherRegs));
    if (warp == kTrSoftmaxWarps) {
      // ---------------------------------------------------------------- loads
      bool ok = true;
      int items = 0, kt = 0;                                      // loaded so far: items' queries, key tiles
      uint32_t loads = 0;                                         // ... tiles of the ring
      uint32_t slot = 0, phase = 0;                               // where the next one goes
      const int ps = 1 << a.page_shift;
      const int tile_shift = ps == 1 ? 7 : 3;                     // log2 of a tile's pages
      const int per = ps == 1 ? 1 : 4, words = ps == 1 ? 4 : 1;
      auto all = [&](bool x) -> bool { return __all_sync(kFull, x); };
      for (;;) {
        ok = all(read_item(items, it, two, drafts_from));
        if (!ok) break;
        __syncwarp();
        if (lane == 0) mbar_arrive(&item_empty[items & 1]);
        if (!it.found) break;
        const int32_t* pages = a.page_table + (int64_t)it.b * a.pt_stride;
        const int n_pages = (it.n + ps - 1) >> a.page_shift;
        // The pages of `per` tiles at a time, one to a lane (four where a page holds one token, for a single tile); -1, whose
        // copy is filled with zeros, behind the sequence and for what is no page of the pool (`out`: those).
        int page[4], ahead[4];
        unsigned out[4] = {0u, 0u, 0u, 0u};
        auto fetch = [&](int j, int (&p)[4]) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int at = (j << tile_shift) + lane + 32 * k;
            p[k] = k < words && at < n_pages ? pages[at] : -1;
          }
        };
        auto vet = [&](int j) {
          unsigned any = 0u;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const bool there = k < words && (j << tile_shift) + lane + 32 * k < n_pages;
            const bool bad = there && (page[k] < 0 || (int64_t)page[k] >= a.num_pages);
            if (bad) page[k] = -1;
            out[k] = __ballot_sync(kFull, bad);
            any |= out[k];
          }
          if (any && lane == 0) set_error(a.status, TS_ERR_PAGE_OOB);
        };
        // which keys of tile `in` of those at hand its pages leave out
        auto note = [&](int in) {
          if (lane == 0) {
            const int r = kt & (kTrRing - 1);
            const unsigned m = out[0] >> (8 * in);                // eight pages, two to a word
            uint32_t any = 0u;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              const uint32_t bad = ps == 1 ? out[w] : (m >> (2 * w) & 1u ? 0xffffu : 0u) | (m >> (2 * w + 1) & 1u ? 0xffff0000u : 0u);
              s_bad[r][w] = bad;
              any |= bad;
            }
            s_any_bad[r] = any;
          }
          ++kt;
        };
        // a tile's pages: the same in every lane, or (pages of one token) a lane's own four
        auto pick = [&](int in, int (&p)[8]) {
#pragma unroll
          for (int k = 0; k < 8; ++k) p[k] = ps == 1 ? page[k & 3] : __shfl_sync(kFull, page[0], 8 * in + k);
        };
        auto load = [&](const CUtensorMap* map, const int (&p)[8]) -> bool {
          if (loads >= S::SLOTS && !all(mbar_wait(&empty[slot], phase ^ 1u, a.wait_ns))) return false;
          unsigned char* dst = sKV + slot * S::KT;
          if (ps != 1) {
            // (one lane of a converged warp, operands the same in all of them)
            if (elect_one()) {
              mbar_arrive_expect_tx(&full[slot], S::KT);
#pragma unroll
              for (int h = 0; h < S::HALVES; ++h)
#pragma unroll
                for (int k = 0; k < 8; ++k)
                  tma_load_3d(dst + h * (kTrKeys * 128) + k * 2048, map, h * 64, it.kv * kPage, p[k], &full[slot]);
            }
          } else {
            if (lane == 0) mbar_arrive_expect_tx(&full[slot], S::KT);
            __syncwarp();
#pragma unroll
            for (int k = 0; k < 4 * S::HALVES; ++k)
              tma_load_3d(dst + (k >> 2) * (kTrKeys * 128) + (lane + 32 * (k & 3)) * 128, map, (k >> 2) * 64, it.kv, p[k & 3],
                          &full[slot]);
          }
          __syncwarp();
          ++loads;
          if (++slot == S::SLOTS) {
            slot = 0;
            phase ^= 1u;
          }
          return true;
        };
        fetch(it.j0, page);
        if (it.j0 + per < it.j1) fetch(it.j0 + per, ahead);
        if (items > 0) ok = all(mbar_wait(&q_empty, (items - 1) & 1, a.wait_ns));
        if (!ok) break;
        const int tiles_q = two ? 2 : 1;
        if (lane == 0) {
          mbar_arrive_expect_tx(&q_full, (uint32_t)(tiles_q * S::HALVES * a.G * a.tokens * 128));
          for (int i = 0; i < tiles_q; ++i)
            for (int h = 0; h < S::HALVES; ++h)
              tma_load_3d(sQ + i * S::QT + h * (kTrRows * 128), &a.q, h * 64, it.kv * a.G, it.row0 + it.i0 + i * a.tokens,
                          &q_full);
        }
        ++items;
        vet(it.j0);
        int in = 0, at = it.j0;                                   // the next tile and its place among the pages at hand
        auto get = [&](int (&p)[8]) {
          if (in == per) {
            in = 0;
#pragma unroll
            for (int k = 0; k < 4; ++k) page[k] = ahead[k];
            if (at + per < it.j1) fetch(at + per, ahead);
            vet(at);
          }
          note(in);
          pick(in, p);
          ++in;
          ++at;
        };
        int p0[8], p1[8];
        get(p0);
        ok = load(&a.k, p0);
        for (int j = it.j0; j < it.j1 && ok; ++j) {               // K(j + 1), V(j)
          if (j + 1 < it.j1) {
            get(p1);
            ok = load(&a.k, p1);
            if (!ok) break;
          }
          ok = load(&a.v, p0);
#pragma unroll
          for (int k = 0; k < 8; ++k) p0[k] = p1[k];
        }
        if (!ok) break;
      }
      if (!ok && lane == 0) set_error(a.status, TS_ERR_TIMEOUT);
      // nothing may still be landing when the CTA exits, however short the limit was that a role gave up at
      if (items > 0) mbar_wait(&q_full, (items - 1) & 1, settle);
      for (uint32_t l = loads > S::SLOTS ? loads - S::SLOTS : 0u; l < loads; ++l)
        mbar_wait(&full[l % S::SLOTS], (l / S::SLOTS) & 1, settle);
      __syncwarp();
    } else if (warp == kTrSoftmaxWarps + 1) {
      // ------------------------------------------------------------- products
      // (the whole warp goes through the loop and one lane issues, with descriptors in uniform registers)
      const uint32_t idesc_s = idesc_bf16_f32(kTrRows, kTrKeys) | (a.negate ? 1u << 13 : 0u);   // bit 13: -A
      constexpr uint32_t idesc_o = idesc_bf16_f32_bmn(kTrRows, D);
      const uint64_t dq = sdesc_sw128(smem_addr(sQ)), dk = sdesc_sw128(smem_addr(sKV));
      const uint64_t dv = sdesc_sw128_mn(smem_addr(sKV), kTrKeys * 128, 1024);
      const uint32_t q_lo = (uint32_t)dq, k_lo = (uint32_t)dk, v_lo = (uint32_t)dv;
      const uint32_t qk_hi = (uint32_t)(dq >> 32), v_hi = (uint32_t)(dv >> 32);
      // (by one lane) scores of query tile i and the key tile in a slot, into the buffer of barrier x
      auto scores = [&](int i, uint32_t slot, int x) {
        const uint32_t ql = q_lo + i * (S::QT >> 4), kl = k_lo + slot * (S::KT >> 4);
#pragma unroll
        for (int h = 0; h < S::HALVES; ++h)
#pragma unroll
          for (int ks = 0; ks < 4; ++ks)
            umma_bf16(tmem + S::S_COL + (x ? 128 : 0), sdesc_from(ql + ((h * (kTrRows * 128) + ks * 32) >> 4), qk_hi),
                      sdesc_from(kl + ((h * (kTrKeys * 128) + ks * 32) >> 4), qk_hi), idesc_s, (h | ks) != 0);
        umma_commit(&s_full[x]);
      };
      // (by one lane) the outputs of tile i take the weights of the buffer of barrier x
      auto outputs = [&](int i, uint32_t slot, int x, bool more) {
        const uint32_t vl = v_lo + slot * (S::KT >> 4);
#pragma unroll
        for (int ks = 0; ks < kTrKeys / 16; ++ks)
          umma_bf16_ts(tmem + S::O_COL + 128 * i, tmem + S::S_COL + (x ? 128 : 0) + 8 * ks, sdesc_from(vl + ((ks * 2048) >> 4), v_hi),
                       idesc_o, more || ks != 0);
        umma_commit(&o_done[x]);
      };
      auto commit = [&](uint64_t* bar) {
        if (elect_one()) umma_commit(bar);
        __syncwarp();
      };
      auto wait = [&](uint64_t* bar, uint32_t parity) -> bool { return __all_sync(kFull, mbar_wait(bar, parity, a.wait_ns)); };
      bool ok = true;
      int kt = 0;                                                 // key tiles of the items before
      uint32_t clean_par = 0u, p_par = 0u;                        // parities of the next waits, by key tile and by barrier
      auto come = [&](uint32_t l) -> bool { return mbar_wait(&full[l % S::SLOTS], (l / S::SLOTS) & 1, a.wait_ns); };
      for (int k = 0;; ++k) {
        ok = __all_sync(kFull, read_item(k, it, two, drafts_from));
        if (!ok) break;
        const bool found = __shfl_sync(kFull, it.found, 0) != 0, pair = __shfl_sync(kFull, two ? 1 : 0, 0) != 0;
        const int nt = __shfl_sync(kFull, it.j1 - it.j0, 0), look = __shfl_sync(kFull, drafts_from - it.j0, 0);
        if (lane == 0) mbar_arrive(&item_empty[k & 1]);
        __syncwarp();
        if (!found) break;
        const uint32_t l0 = 2u * (uint32_t)kt;                    // the item's first tile of the ring
        const int tiles = pair ? 2 : 1;
        const int ahead = pair ? 1 : 2;                           // key tiles whose scores are taken before the first outputs
        ok = wait(&q_full, k & 1);
        for (int j = 0; j < min(ahead, nt) && ok; ++j) {
          const uint32_t l = l0 + key_load(j);
          ok = __all_sync(kFull, come(l));
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
            for (int i = 0; i < tiles; ++i) scores(i, l % S::SLOTS, pair ? i : 2 * j);
            umma_commit(&empty[l % S::SLOTS]);
            if (j + 1 == nt) umma_commit(&q_empty);
          }
          __syncwarp();
        }
        if (!ok) break;
        for (int j = 0; j < nt && ok; ++j) {                      // outputs of key tile j, scores of the one that is ahead
          const uint32_t vl = l0 + value_load(j, nt), kl = l0 + key_load(j + ahead);
          const int g = (kt + j) & (kTrRing - 1);
          const bool next = j + ahead < nt;
          bool here = come(vl);
          if (j >= look) {
            here = here && mbar_wait(&v_clean[g], (clean_par >> g) & 1u, a.wait_ns);
            clean_par ^= 1u << g;
          }
          for (int i = 0; i < tiles && ok; ++i) {
            const int x = pair ? i : 2 * (j & 1);
            here = mbar_wait(&p_ready[x], (p_par >> x) & 1u, a.wait_ns) && here;
            p_par ^= 1u << x;
            ok = __all_sync(kFull, here);
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) {
              outputs(i, vl % S::SLOTS, x, j != 0);
              if (i + 1 == tiles) umma_commit(&empty[vl % S::SLOTS]);
            }
            __syncwarp();
            if (!next) continue;
            if (i == 0) {
              ok = __all_sync(kFull, come(kl));
              if (!ok) break;
              tc_fence_after();
            }
            if (elect_one()) {
              scores(i, kl % S::SLOTS, x);
              if (i + 1 == tiles) {
                umma_commit(&empty[kl % S::SLOTS]);
                if (j + ahead + 1 == nt) umma_commit(&q_empty);
              }
            }
            __syncwarp();
          }
        }
        if (!ok) break;
        kt += nt;
      }
      if (!ok && lane == 0) set_error(a.status, TS_ERR_TIMEOUT);
      // no product may be under way when tensor memory is given back
      commit(&drained);
      mbar_wait(&drained, 0, settle);
      __syncwarp();
    } else if (warp == kTrSoftmaxWarps + 2) {
      // ---------------------------------------------------------------- items
      int64_t work = 0, tiles_all = 0;
      for (int b0 = 0; b0 < a.B; b0 += 32) {
        const int b = b0 + lane;
        TreeSeq s{};
        if (b < a.B) s = tree_seq(a, b);
        const int64_t run = work + warp_scan_ll(s.head() * a.HKV, lane);
        if (blockIdx.x == 0 && s.err) set_error(a.status, s.err);
        work = __shfl_sync(kFull, run, 31);
        tiles_all += __shfl_sync(kFull, warp_scan_ll((int64_t)s.blocks * s.tiles, lane), 31) * a.HKV;
      }
      const int ctas = (int)min((int64_t)gridDim.x, tiles_all);
      int64_t t = 0, e = 0;
      if (work > 0 && (int)blockIdx.x < ctas) {
        t = share_begin(work, ctas, blockIdx.x);
        e = share_begin(work, ctas, blockIdx.x + 1);
      }
      int b0 = 0;                                                 // the sequences looked at: 32 from b0 on
      int64_t before = 0;                                         // tiles of the sequences before them
      bool found = true;
      for (int k = 0; found; ++k) {
        found = t < e;
        TreeItem item{};
        if (found) {
          for (;;) {                                              // the sequence and the block that place t is in
            const int b = b0 + lane;
            TreeSeq s{};
            if (b < a.B) s = tree_seq(a, b);
            const int64_t w = s.head() * a.HKV, run = warp_scan_ll(w, lane);
            const unsigned m = __ballot_sync(kFull, before + run > t);
            if (!m) {
              before += __shfl_sync(kFull, run, 31);
              b0 += 32;
              if (b0 < a.B) continue;
              found = false;                                      // (not reached: t lies below the work)
              break;
            }
            const int src = __ffs(m) - 1;
            const int64_t start = before + __shfl_sync(kFull, run - w, src), head = __shfl_sync(kFull, s.head(), src);
            const int tiles = __shfl_sync(kFull, s.tiles, src), blocks = __shfl_sync(kFull, s.blocks, src);
            const int last = __shfl_sync(kFull, s.last, src);
            const int64_t in = (t - start) % head, one = kTrBlock + (int64_t)kTrPair * tiles;
            const int kv = (int)((t - start) / head), block = (int)min(in / one, (int64_t)blocks - 1);
            const int per = block + 1 < blocks ? kTrPair : last;  // work of a key tile
            const int64_t at = t - in + block * one + kTrBlock;   // where the block's key tiles begin
            const int j0 = first_tile(at, per, tiles, t), j1 = first_tile(at, per, tiles, e);
            t = at + (int64_t)per * tiles;                        // the next block
            if (j0 >= j1) {                                       // (no key tile of this one begins in the share)
              if (t < e) continue;
              found = false;
              break;
            }
            item.row0 = __shfl_sync(kFull, s.row0, src);
            item.T = __shfl_sync(kFull, s.T, src);
            item.n = __shfl_sync(kFull, s.n, src);
            item.b = b0 + src;
            item.kv = kv;
            item.i0 = block * 2 * a.tokens;
            item.j0 = j0;
            item.j1 = j1;
            // (one block at most comes from an earlier share, one at most goes on in a later one)
            item.slot = j0 == 0 && j1 == tiles ? -1 : 2 * (int)blockIdx.x + (j0 == 0 ? 1 : 0);
            break;
          }
        }
        item.found = found;
        if (k >= 2 && !__all_sync(kFull, mbar_wait(&item_empty[k & 1], ((k >> 1) - 1) & 1, a.wait_ns))) {
          if (lane == 0) set_error(a.status, TS_ERR_TIMEOUT);
          break;
        }
        if (s_any_odd[k & 1]) {
          if (lane < kMaxTree / 32) s_odd[k & 1][lane] = 0u;
          __syncwarp();
          if (lane == 0) s_any_odd[k & 1] = 0;
        }
        __syncwarp();
        if (lane == 0) {
          s_item[k & 1] = item;
          mbar_arrive(&item_full[k & 1]);
        }
        __syncwarp();
      }
    } else {
      // ----------------------------------- values that are not finite among the drafts and behind them
      bool ok = true;
      int kt = 0;                                                 // key tiles of the items before
      uint32_t slot = 0, phase = 0;                               // the next tile of the ring
      for (int k = 0;; ++k) {
        ok = __all_sync(kFull, read_item(k, it, two, drafts_from));
        if (!ok || !it.found) break;
        // every tile of the ring in turn, keys too: a parity tells a phase only from its neighbours
        const int nt = it.j1 - it.j0;
        for (int m = 0; m < 2 * nt && ok; ++m) {
          ok = __all_sync(kFull, mbar_wait(&full[slot], phase, a.wait_ns));
          if (!ok) break;
          const bool value = m == 2 * nt - 1 || (m >= 2 && m % 2 == 0);
          const int j = it.j0 + (m == 2 * nt - 1 ? nt - 1 : m / 2 - 1);
          if (value && j >= drafts_from) {
            unsigned char* vt = sKV + slot * S::KT;
            uint32_t odd = 0u;
#pragma unroll 8
            for (int c = 0; c < S::KT / 512; ++c) {
              const uint4 w = lds128(vt + c * 512 + lane * 16);
              odd |= ((w.x & 0x7f807f80u) + 0x00800080u) | ((w.y & 0x7f807f80u) + 0x00800080u) |
                     ((w.z & 0x7f807f80u) + 0x00800080u) | ((w.w & 0x7f807f80u) + 0x00800080u);
            }
            if (odd & 0x80008000u) {
              for (int off = lane * 16; off < S::KT; off += 512) {               // byte in the tile
                const int r = (off % (kTrKeys * 128)) / 128, at = j * kTrKeys + r - (it.n - it.T);
                if (at < 0) continue;                             // every row sees it
                uint16_t* e16 = reinterpret_cast<uint16_t*>(vt + off);
                for (int e = 0; e < 8; ++e) {
                  if ((e16[e] & 0x7f80u) != 0x7f80u) continue;
                  e16[e] = 0;
                  if (at < it.T) {
                    atomicOr(&s_odd[k & 1][at >> 5], 1u << (at & 31));
                    s_any_odd[k & 1] = 1;
                  }
                }
              }
            }
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) mbar_arrive(&v_clean[(kt + j - it.j0) & (kTrRing - 1)]);
          }
          if (lane == 0) mbar_arrive(&empty[slot]);
          __syncwarp();
          if (++slot == S::SLOTS) {
            slot = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        kt += nt;
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
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kTrSoftmaxRegs));
    const int i = warp >> 2;                                      // tile
    const int row = 32 * (warp & 3) + lane;
    const uint32_t inv_g = 65536u / (uint32_t)a.G + 1u;           // r / G = (r inv_g) >> 16 for r < 128, G <= 16
    const uint32_t lane_off = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t tO = tmem + S::O_COL + 128 * i + lane_off;
    bool ok = true;
    uint32_t s_par = 0u, o_par = 0u;                              // parities of the next scores and outputs, by barrier
    int kt = 0;                                                   // key tiles of the items before
    for (int k = 0; ok; ++k) {
      ok = __all_sync(kFull, read_item(k, it, two, drafts_from));
      if (!ok || !it.found) break;
      const int slot = k & 1, nt = __shfl_sync(kFull, it.j1 - it.j0, 0);
      const bool pair = __shfl_sync(kFull, two ? 1 : 0, 0) != 0;
      if (i == 0 || pair) {
        const int first = it.i0 + i * a.tokens;                   // first draft of the tile
        const int row_tok = (int)((uint32_t)row * inv_g >> 16), tok = first + row_tok;
        const bool real = row_tok < a.tokens && tok < it.T;
        const bool idle = !__any_sync(kFull, real);               // no row of this warp is a query: it only keeps step
        const int d0 = it.n - it.T;                               // first draft's position
        const int packed = it.row0 + (real ? tok : 0);
        float mx = -INFINITY, la = 0.f, lb = 0.f;                 // running maximum (unscaled) and two halves of the sum
        int x = i;
        for (int j = 0; j < nt; ++j) {
          // the outputs before these went to the same barrier where the block has two tiles, else to the other one
          const int before = x, key0 = (it.j0 + j) * kTrKeys;
          x = pair ? i : 2 * (j & 1);
          const uint32_t tS = tmem + S::S_COL + (x ? 128 : 0) + lane_off;
          ok = __all_sync(kFull, mbar_wait(&s_full[x], (s_par >> x) & 1u, a.wait_ns));
          if (!ok) break;
          tc_fence_after();
          s_par ^= 1u << x;
          if (!idle) {
            // what is not seen in this tile: drafts, what is behind the sequence, pages outside the pool
            const int ring = (kt + j) & (kTrRing - 1);
            const bool any_bad = s_any_bad[ring] != 0u;
            if (key0 + kTrKeys > d0 || any_bad) {
              // (rare: such scores are replaced in tensor memory, before and apart from what most tiles go through)
#pragma unroll 1
              for (int w = 0; w < 4; ++w) {
                const uint32_t m = seen_bits(a, packed, tok, it.T, key0 + 32 * w - d0) & ~(any_bad ? s_bad[ring][w] : 0u);
                if (!__any_sync(kFull, m != 0xffffffffu)) continue;
                uint32_t u[32];
                tmem_ld_x32(tS + 32 * w, u);
                tmem_wait_ld();
#pragma unroll
                for (int c = 0; c < 32; ++c) u[c] = m >> c & 1u ? u[c] : 0xff800000u;
                tmem_st_x32(tS + 32 * w, u);
              }
              tmem_wait_st();
            }
            // Weights against the maximum that the row has, which covers most tiles. Where their sum says that
            // it does not (and in the first tile, which has none), the scores, still in tensor memory, are read
            // again and the maximum is taken first.
            uint32_t p[kTrKeys / 2];
            float ta, tb, m2 = mx * a.scale2;
            bool over = real;                                     // this row needs its maximum (in a pass that takes it)
            for (bool raise = j == 0;; raise = true) {
              if (raise) {
                float ma = -INFINITY, mb = -INFINITY;
#pragma unroll 1
                for (int c0 = 0; c0 < kTrKeys; c0 += 32) {
                  uint32_t u[32];
                  tmem_ld_x32(tS + c0, u);
                  tmem_wait_ld();
#pragma unroll
                  for (int c = 0; c < 32; c += 2) {
                    ma = fmaxf(ma, __uint_as_float(u[c]));
                    mb = fmaxf(mb, __uint_as_float(u[c + 1]));
                  }
                }
                // each row by itself, so that no row's bits depend on another's: rows that do not need it keep their
                // maximum, as do rows that are no query of the sequence (their operands may be anything)
                const float mn = over ? fmaxf(mx, fmaxf(ma, mb)) : mx, n2 = mn * a.scale2;
                const float f = mn == mx ? 1.f : pr_ex2(from_to(mx, m2, mn, n2, a.scale2));
                mx = mn;
                m2 = n2;
                la *= f;
                lb *= f;
                if (j > 0) {
                  // the last product must be in before its accumulators are rescaled
                  ok = __all_sync(kFull, mbar_wait(&o_done[before], (o_par >> before & 1u) ^ 1u, a.wait_ns));
                  if (!ok) break;
                  tc_fence_after();
                  // (rare: eight columns at a time)
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
              float ms = m2 == -INFINITY ? 0.f : -m2;             // nothing seen yet: every weight is zero
              const bool shift = far(m2) && m2 != -INFINITY;
              const bool shifts = raise && __any_sync(kFull, shift);
              if (shifts && shift) ms = 0.f;
              const float off = shifts && shift ? mx : 0.f;
              const uint64_t sc = pack_f2(a.scale2, a.scale2), mm = pack_f2(ms, ms);
              ta = tb = 0.f;
              // 64 scores at a time, so that they and the weights fit the registers
#pragma unroll
              for (int c0 = 0; c0 < kTrKeys; c0 += 64) {
                uint32_t u[64];
                tmem_ld_x32(tS + c0, u);
                tmem_ld_x32(tS + c0 + 32, u + 32);
                tmem_wait_ld();
                float* y = reinterpret_cast<float*>(u);
                if (shifts) {
#pragma unroll
                  for (int c = 0; c < 64; c += 2) add2(y[c], y[c + 1], -off, -off);
                }
#pragma unroll
                for (int c = 0; c < 32; ++c) {
                  float y0, y1;
                  unpack_f2(fma_f2(pack_f2(y[2 * c], y[2 * c + 1]), sc, mm), y0, y1);
                  y0 = pr_ex2(y0);
                  y1 = pr_ex2(y1);
                  add2(ta, tb, y0, y1);
                  p[c0 / 2 + c] = pack_bf16(y0, y1);
                }
              }
              if (raise) break;
              over = real && (!(ta + tb <= kTrMaxSum) || far(m2));
              if (!__any_sync(kFull, over)) break;
            }
            if (!ok) break;
            la += ta;
            lb += tb;
            tmem_st_x32(tS, p);
            tmem_st_x32(tS + 32, p + 32);
            tmem_wait_st();
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&p_ready[x]);
          o_par ^= 1u << x;
        }
        // ---- outputs
        if (ok) ok = __all_sync(kFull, mbar_wait(&o_done[x], (o_par >> x & 1u) ^ 1u, a.wait_ns));
        if (ok) ok = __all_sync(kFull, mbar_wait(&item_clean[slot], (k >> 1) & 1, a.wait_ns));
        if (ok && !idle) {
          tc_fence_after();
          const float l = la + lb;
          const int head = it.kv * a.G + row - row_tok * a.G;
          // values that are not finite, of the drafts that the row sees, for columns [col, col + 32)
          const bool odd = s_any_odd[slot] != 0;
          auto put_back = [&](int col, uint32_t (&o)[32]) {
            for (int t = it.j0 * kTrKeys > d0 ? it.j0 * kTrKeys - d0 : 0; t < min(it.T, it.j1 * kTrKeys - d0); ++t) {
              if (!(s_odd[slot][t >> 5] >> (t & 31) & 1u)) continue;
              if (!real || !(seen_bits(a, packed, tok, it.T, t) & 1u)) continue;
              const int pos = d0 + t, ps = 1 << a.page_shift;
              const int page = a.page_table[(int64_t)it.b * a.pt_stride + (pos >> a.page_shift)];
              const __nv_bfloat16* v = a.v_pool + ((((int64_t)page * a.HKV + it.kv) << a.page_shift) + (pos & (ps - 1))) * D + col;
              for (int e = 0; e < 32; ++e) {
                const float y = __bfloat162float(v[e]);
                if (!isfinite(y)) {
#pragma unroll
                  for (int z = 0; z < 32; ++z)
                    if (z == e) o[z] = __float_as_uint(__uint_as_float(o[z]) + y);
                }
              }
            }
          };
          if (it.slot >= 0) {
            // sums of a part of the block: 16 bytes of 32 neighbouring rows side by side
            const int at = 128 * i + row;
            if (real) a.part_ml[(int64_t)it.slot * 256 + at] = make_float2(mx, l);
            float4* dst = reinterpret_cast<float4*>(a.part_o) + (int64_t)it.slot * (D / 4) * 256 + at;
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
              uint32_t o[32];
              tmem_ld_x32(tO + 32 * c, o);
              tmem_wait_ld();
              if (odd) put_back(32 * c, o);
#pragma unroll
              for (int e = 0; e < 8; ++e)
                if (real)
                  dst[(int64_t)(8 * c + e) * 256] = make_float4(__uint_as_float(o[4 * e]), __uint_as_float(o[4 * e + 1]),
                                                                __uint_as_float(o[4 * e + 2]), __uint_as_float(o[4 * e + 3]));
            }
          } else {
            const float inv = l > 0.f || l != l ? 1.f / l : 0.f;  // (a row that sees nothing: zeros)
            if (real && a.lse)
              a.lse[(int64_t)packed * a.H + head] = l == 0.f ? -INFINITY : (mx * a.scale2 + log2f(l)) * 0.6931471805599453f;
            unsigned char* dst = reinterpret_cast<unsigned char*>(a.out + (int64_t)packed * a.out_stride + (int64_t)head * D);
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
              uint32_t o[32];
              tmem_ld_x32(tO + 32 * c, o);
              tmem_wait_ld();
              if (odd) put_back(32 * c, o);
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                uint32_t w[4];
#pragma unroll
                for (int z = 0; z < 4; ++z)
                  w[z] = pack_bf16(__uint_as_float(o[8 * e + 2 * z]) * inv, __uint_as_float(o[8 * e + 2 * z + 1]) * inv);
                if (real) *reinterpret_cast<uint4*>(dst + 64 * c + 16 * e) = make_uint4(w[0], w[1], w[2], w[3]);
              }
            }
          }
          // the accumulators have been read before the next item's weights let a product write them
          tc_fence_before();
        }
      }
      kt += nt;
      __syncwarp();
      if (lane == 0) mbar_arrive(&item_empty[slot]);
    }
    if (!ok && lane == 0) set_error(a.status, TS_ERR_TIMEOUT);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kTrSoftmaxWarps + 1) {
    tc_fence_after();
    tmem_dealloc(tmem, S::TMEM_COLS);
  }
}

// Joins the sums of blocks that several CTAs had parts of: eight rows of one to a CTA at a time (neighbouring rows of a block:
// heads, then drafts), whose sums lie side by side; a thread per row, four columns and every second part. Bound by
// latency (which blocks, factors and parts together, sums), then by the parts read from L2.
constexpr int kJoinRows = 8, kJoinGroups = 2, kJoinBatch = 6;
constexpr float kNoPart = -1.f;  // in place of a sum or a factor, which are not negative

// A block that several CTAs have parts of, by the CTA that its first key tile lies with.
struct TreeJoin {
  int64_t at;                    // where its key tiles begin
  int row0, drafts, kv;          // its rows
  int parts;                     // CTAs from this one to the one that its last key tile lies with; 0: no such block
  int per, tiles;                // work of a key tile, key tiles
};

template <int D>
__global__ void __launch_bounds__(kJoinRows * D / 4 * kJoinGroups, 256 / D) join_kernel(const __grid_constant__ TreeArgs a, int grid) {
  constexpr int COLS = D / 4;
  __shared__ int s_upto[kJoinParts];                              // pieces of the blocks up to that of each CTA
  __shared__ TreeJoin s_join[kJoinParts];
  __shared__ TreeSeq s_seq[32];
  __shared__ int64_t s_end[32];                                   // work up to a sequence's end
  __shared__ int64_t s_work;
  __shared__ int s_ctas;
  __shared__ float s_f[kJoinRows][kJoinParts];
  __shared__ float s_inv[kJoinRows];
  __shared__ float4 s_acc[kJoinGroups - 1][kJoinRows * COLS];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int row = tid % kJoinRows, col = tid / kJoinRows % COLS, grp = tid / (kJoinRows * COLS);
  // ---- which blocks: a thread per CTA (256 of each), all from lengths and boundaries, while the other kernel runs
  if (warp == 0) {
    int64_t work = 0, tiles_all = 0;
    for (int b0 = 0; b0 < a.B; b0 += 32) {
      TreeSeq s{};
      if (b0 + lane < a.B) s = tree_seq(a, b0 + lane);
      work = __shfl_sync(kFull, work + warp_scan_ll(s.head() * a.HKV, lane), 31);
      tiles_all += __shfl_sync(kFull, warp_scan_ll((int64_t)s.blocks * s.tiles, lane), 31) * a.HKV;
    }
    if (lane == 0) {
      s_work = work;
      s_ctas = (int)min((int64_t)grid, tiles_all);
    }
  }
  __syncthreads();
  const int64_t work = s_work;
  const int ctas = s_ctas;
  TreeJoin mine{};
  const int64_t begin = tid < ctas ? share_begin(work, ctas, tid) : 0, end = tid < ctas ? share_begin(work, ctas, tid + 1) : 0;
  int64_t before = 0;
  for (int b0 = 0; b0 < a.B; b0 += 32) {
    if (warp == 0) {
      TreeSeq s{};
      if (b0 + lane < a.B) s = tree_seq(a, b0 + lane);
      s_seq[lane] = s;
      s_end[lane] = before + warp_scan_ll(s.head() * a.HKV, lane);
    }
    __syncthreads();
    const int64_t last = end - 1;                                 // the block that the share's last place is in
    if (tid < ctas && last >= before && last < s_end[31]) {
      int b = 0;
      while (s_end[b] <= last) ++b;
      const TreeSeq s = s_seq[b];
      const int64_t start = b ? s_end[b - 1] : before, in = (last - start) % s.head();
      const int block = (int)min(in / s.block(), (int64_t)s.blocks - 1);
      mine.kv = (int)((last - start) / s.head());
      mine.per = block + 1 < s.blocks ? kTrPair : s.last;
      mine.tiles = s.tiles;
      mine.at = last - in + block * s.block() + kTrBlock;
      mine.row0 = s.row0 + block * 2 * a.tokens;
      mine.drafts = min(s.T - block * 2 * a.tokens, 2 * a.tokens);
      const int64_t final = mine.at + (int64_t)mine.per * (s.tiles - 1);
      mine.parts = mine.at >= begin && mine.at < end && final >= end ? share_of(work, ctas, final) - tid + 1 : 0;
    }
    before = s_end[31];
    __syncthreads();
  }
  if (tid < kJoinParts) {
    s_join[tid] = mine;
    s_upto[tid] = mine.parts ? (mine.drafts * a.G + kJoinRows - 1) / kJoinRows : 0;
  }
  __syncthreads();
  if (warp == 0) {
    int sum = 0;
    for (int c = lane; c < kJoinParts; c += 32) {
      int run = s_upto[c];
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int x = __shfl_up_sync(kFull, run, d);
        if (lane >= d) run += x;
      }
      s_upto[c] = sum + run;
      sum += __shfl_sync(kFull, run, 31);
    }
  }
  __syncthreads();
  asm volatile("griddepcontrol.wait;" ::: "memory");
  for (int piece = blockIdx.x; piece < s_upto[kJoinParts - 1]; piece += gridDim.x) {
    int c = 0;
    for (int hi = kJoinParts - 1; c < hi;) {                            // the first CTA with more pieces up to it
      const int mid = (c + hi) >> 1;
      if (s_upto[mid] > piece) hi = mid; else c = mid + 1;
    }
    const TreeJoin& jn = s_join[c];
    const int rows = jn.drafts * a.G, r0 = (piece - (c ? s_upto[c - 1] : 0)) * kJoinRows, parts = jn.parts;
    auto slot_of = [&](int k) { return 2 * (c + k) + (k == 0 ? 1 : 0); };
    auto place = [&](int r) { return r / a.G / a.tokens * 128 + r / a.G % a.tokens * a.G + r % a.G; };
    const float4* src = reinterpret_cast<const float4*>(a.part_o) + (int64_t)col * 256 + place(min(r0 + row, rows - 1));
    float4 o[kJoinBatch];
    auto load = [&](int k0) {
#pragma unroll
      for (int e = 0; e < kJoinBatch; ++e) {
        const int k = k0 + e * kJoinGroups;
        if (k < parts) o[e] = src[(int64_t)slot_of(k) * COLS * 256];
      }
    };
    load(grp);
    if (warp < kJoinRows && r0 + warp < rows) {
      // every part's factor, and the row's sum: a warp per row, a lane per part. A part that saw a number that is none has a
      // sum that is none (its maximum passes it over), which is its factor too; kNoPart: a CTA in between that had no key tile.
      const int r = r0 + warp;
      const float2* ml = a.part_ml + place(r);
      float M = -INFINITY, total = 0.f;
      auto part = [&](int k) {
        const int j0 = first_tile(jn.at, jn.per, jn.tiles, share_begin(work, ctas, c + k));
        const int j1 = first_tile(jn.at, jn.per, jn.tiles, share_begin(work, ctas, c + k + 1));
        return j0 < j1 ? ml[(int64_t)slot_of(k) * 256] : make_float2(-INFINITY, kNoPart);
      };
      for (int k = lane; k < parts; k += 32) {
        const float2 x = part(k);
        M = fmaxf(M, x.y == 0.f || x.y == kNoPart ? -INFINITY : x.x);
      }
      M = warp_max(M);
      const float M2 = M * a.scale2;
      for (int k = lane; k < parts; k += 32) {
        const float2 x = part(k);
        const float f = x.y == 0.f || x.y == kNoPart || x.y != x.y
                            ? x.y
                            : (x.x == M ? 1.f : pr_ex2(from_to(x.x, x.x * a.scale2, M, M2, a.scale2)));
        s_f[warp][k] = f;
        if (f != kNoPart) total = fmaf(f, x.y, total);
      }
      total = warp_sum(total);
      if (lane == 0) {
        s_inv[warp] = total == 0.f ? 0.f : 1.f / total;
        if (a.lse)
          a.lse[(int64_t)(jn.row0 + r / a.G) * a.H + jn.kv * a.G + r % a.G] =
              total == 0.f ? -INFINITY : (M2 + log2f(total)) * 0.6931471805599453f;
      }
    }
    __syncthreads();
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k0 = grp; k0 < parts; k0 += kJoinBatch * kJoinGroups) {
      if (k0 != grp) load(k0);
#pragma unroll
      for (int e = 0; e < kJoinBatch; ++e) {
        const int k = k0 + e * kJoinGroups;
        const float f = k < parts && r0 + row < rows ? s_f[row][k] : kNoPart;
        if (f != kNoPart) {                                       // (a value that is not finite shows however little it weighs)
          acc.x = fmaf(f, o[e].x, acc.x);
          acc.y = fmaf(f, o[e].y, acc.y);
          acc.z = fmaf(f, o[e].z, acc.z);
          acc.w = fmaf(f, o[e].w, acc.w);
        }
      }
    }
    if (grp > 0) s_acc[grp - 1][tid % (kJoinRows * COLS)] = acc;
    __syncthreads();
    if (grp == 0 && r0 + row < rows) {
#pragma unroll
      for (int g = 0; g < kJoinGroups - 1; ++g) {
        const float4 x = s_acc[g][tid];
        acc.x += x.x;
        acc.y += x.y;
        acc.z += x.z;
        acc.w += x.w;
      }
      const float inv = s_inv[row];
      const int r = r0 + row;
      __nv_bfloat16* out = a.out + (int64_t)(jn.row0 + r / a.G) * a.out_stride + (int64_t)(jn.kv * a.G + r % a.G) * D + col * 4;
      *reinterpret_cast<uint2*>(out) = make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
    }
    __syncthreads();
  }
}

// bf16 [pages][heads * page size][d] in boxes of 64 elements x one page of one head.
bool pages_map(CUtensorMap* map, const void* pool, int64_t pages, int rows, int d, int page_size) {
  const auto encode = tensor_map_encoder();
  if (!encode) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)rows, (cuuint64_t)pages};
  const cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)rows * d * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)page_size, 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(pool), dims, strides, box, estr,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D>
ts_status run_tree(ts_ctx* ctx, const TreeArgs& a, cudaStream_t s) {
  if (!ensure_smem<tree_kernel<D>>((size_t)TrShape<D>::SMEM, ctx->device)) return TS_ERR_CUDA;
  ProfScope ps(ctx, TS_PROF_ATTEND, s);
  ctx->kernels += 2;
  const int grid = ctx->num_sms < kJoinParts ? ctx->num_sms : kJoinParts;
  tree_kernel<D><<<grid, kTrThreads, TrShape<D>::SMEM, s>>>(a);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_status(e);
  return cuda_status(launch_behind(join_kernel<D>, dim3((unsigned)(2 * grid)), kJoinRows * D / 4 * kJoinGroups, s, a, grid));
}

}  // namespace

bool tree_supported(const ts_config& c) {
  return c.kv_dtype == TS_KV_BF16 && (c.head_dim == 64 || c.head_dim == 128) && c.n_q_heads / c.n_kv_heads <= 16;
}

int64_t tree_part_slots(int num_sms) { return 2 * (int64_t)num_sms; }

ts_status launch_tree_attend(ts_ctx* ctx, const TreeCall& c, cudaStream_t s) {
  if (c.total == 0) return TS_OK;
  const ts_config& cfg = ctx->cfg;
  TreeArgs a{};
  a.cu = c.cu_rows;
  a.seq_lens = c.seq_lens;
  a.page_table = c.page_table;
  a.pt_stride = cfg.max_pages_per_seq;
  a.page_shift = ctx->page_shift;
  a.num_pages = cfg.num_pages;
  a.max_tokens = ctx->max_tokens;
  a.mask = reinterpret_cast<const uint32_t*>(c.mask);
  a.mask_words = c.mask_words;
  a.v_pool = static_cast<const __nv_bfloat16*>(c.v_pool);
  a.B = c.B;
  a.total = c.total;
  a.H = cfg.n_q_heads;
  a.HKV = cfg.n_kv_heads;
  a.G = a.H / a.HKV;
  a.tokens = kTrRows / a.G;
  a.scale2 = std::fabs(c.scale) * 1.4426950408889634f;
  a.negate = c.scale < 0.f;
  a.out = static_cast<__nv_bfloat16*>(c.out);
  a.out_stride = c.out_stride;
  a.lse = c.lse;
  a.part_o = ctx->tree_part_o;
  a.part_ml = ctx->tree_part_ml;
  a.status = ctx->status;
  a.wait_ns = ctx->wait_ns;
  const int ps = 1 << ctx->page_shift, rows = a.HKV * ps;
  if (!rows_map(&a.q, c.q, c.total, a.H, cfg.head_dim, c.q_stride, a.G, a.tokens) ||
      !pages_map(&a.k, c.k_pool, cfg.num_pages, rows, cfg.head_dim, ps) ||
      !pages_map(&a.v, c.v_pool, cfg.num_pages, rows, cfg.head_dim, ps))
    return TS_ERR_CUDA;
  return cfg.head_dim == 64 ? run_tree<64>(ctx, a, s) : run_tree<128>(ctx, a, s);
}

}  // namespace ts
