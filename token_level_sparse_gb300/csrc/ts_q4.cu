// Score and attention over a 4-bit paged cache (TS_KV_Q4; block format and tensor-core pieces in
// ts_q4.cuh).
//
//   l[h][i] = scale <q_h, (u_i - 8) s_i>      out_h = sum_i softmax_i(l[h]) (u'_i - 8) s'_i
//
// Both read every block of a sequence once and nothing else of size, so they are bound by the
// stream of 4-bit blocks (68 bytes per row of 128) as long as the arithmetic keeps up: the codes
// are unpacked in registers (9 instructions for 8 codes) and multiplied on the tensor cores.
//
// scan_kernel (whole sequences): a CTA owns a group of up to 4 head sets (a head set: up to 4 query
// heads of one KV head, or up to 8 where there are more than 4 to a KV head) and a share of the batch's
// pages. Its warps are shared out over the head sets and take the pages in turn, each with a ring of
// blocks of its own in shared memory that it fills with bulk copies several pages ahead: no warp waits
// for another one inside a sequence. At the end of a sequence's part of the range the warps of a head
// set join their states, and q4_merge_kernel joins the parts of a sequence in CTA order. Every sum
// has a fixed order.
//
// gather_kernel (a list of tokens): 16 listed tokens per step straight from global memory; the list
// is split over CTAs and joined by the same merge.
#include <algorithm>
#include <cmath>
#include <utility>

#include "ts_q4.cuh"

namespace ts {
namespace {

constexpr int kScorePages = 4;                  // pages of a stage of the score (4 against 2: 79 against 85 us, 898K tokens)
constexpr int kScanSeqs = 512;                  // sequences whose page counts a scan CTA keeps in shared memory
constexpr int kQ4Sets = 4;                      // head sets of a CTA, at most
constexpr int kGatherWarps = 6;
constexpr int kGatherCtas = 2;                  // gather CTAs per SM
constexpr float kLog2e = 1.4426950408889634f;

struct Q4Args {
  const float* q;                // [B][H][d]
  const unsigned char* k_pool;   // [num_pages][H_kv][block]
  const unsigned char* v_pool;
  const int32_t* page_table;
  int pt_stride;
  int64_t num_pages;
  const int32_t* seq_lens;
  const uint8_t* skip;           // score only: sequences left out
  int max_tokens;
  int B, H, HKV, G;
  int sets_per_kv;               // head sets of one KV head: ceil(G / set_heads)
  int set_heads;                 // 4 or 8
  int n_groups;                  // groups of kQ4Sets head sets
  int ctas;                      // CTAs per group
  float scale;                   // base 2 (times log2 e), but natural for the scores that no softmax follows
  float* logits;                 // score, in units of scale: H max_tokens to a sequence, head h of token i at
  int64_t head_stride, page_stride;   // h head_stride + i / 16 page_stride + i % 16
  float* part_o;                 // [slot][H][d]: a part's own outputs, divided by its sum
  float2* part_ml;               // [H][slots]: max and sum of 2^(x - max)
  int64_t slots;
  int* status;
};

// Programmatic dependent launch: the scan lets the kernel behind it start its own set-up as SMs become
// free, and that kernel waits for the scan's results (and all that came before) where it needs them.
__device__ __forceinline__ void launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_primary() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

__device__ __forceinline__ int seq_pages(const Q4Args& a, int b) {
  if (a.skip && a.skip[b]) return 0;
  const int n = a.seq_lens[b];
  return (n < 0 || n > a.max_tokens) ? 0 : (n + kPage - 1) / kPage;
}

// Outputs are divided by their sums in every join, before they are added up: sums of weights times values may pass
// fp32 where the values themselves do not. (No token: a sum and outputs of zero.)
__device__ __forceinline__ float reciprocal(float sum) { return sum != 0.f ? 1.f / sum : 0.f; }

// Weight of a part with maximum m in a join with maximum M. Equal maxima weigh 1 also where both are
// -inf: an empty part brings zeros, a part of NaN logits brings its NaN.
__device__ __forceinline__ float part_weight(float m, float M) { return m == M ? 1.f : ex2(m - M); }

// How the pages of the batch are shared out over the CTAs of a group. Two ways:
//  * each sequence gets CTAs of its own, one for every `chunk` pages (4 at least: about a page for every
//    warp of a head set), so that no CTA has parts of two sequences;
//  * the pages of all sequences, one behind another, are cut into equal contiguous ranges.
// A CTA that ends one sequence and begins another pays for both beginnings and ends, 6 us where a page takes
// 0.26 us; rounding up to whole CTAs costs up to chunk - total / ctas pages. The first way is taken where
// that is below 24 pages, and there are more CTAs than sequences.
constexpr int kScanSlack = 24;

struct Q4Share {
  int64_t total, before;    // pages of the batch, and of the sequences before the one asked for
  int ctas, chunk;          // chunk 0: equal ranges
  int first;                // chunk > 0: first CTA of the sequence asked for

  __device__ __forceinline__ int live() const {
    const int64_t want = (total + 3) / 4;
    return (int)(want < 1 ? 1 : (want < ctas ? want : ctas));
  }
};

// (one warp; the same in every lane) pages(b): pages of sequence b
template <typename Pages>
__device__ __forceinline__ Q4Share share_pages(const Q4Args& a, int upto, int lane, Pages pages) {
  int64_t t = 0, u = 0;
  for (int b = lane; b < a.B; b += 32) {
    const int n = pages(b);
    t += n;
    if (b < upto) u += n;
  }
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) {
    t += __shfl_xor_sync(kFull, t, d);
    u += __shfl_xor_sync(kFull, u, d);
  }
  Q4Share sh{t, u, a.ctas, 0, 0};
  if (a.ctas > a.B) {
    const int64_t room = a.ctas - a.B, chunk = max((int64_t)4, (t + room - 1) / room);   // sum of ceil(pages / chunk) <= ctas
    if (chunk * a.ctas < t + (int64_t)kScanSlack * a.ctas) {
      sh.chunk = (int)chunk;
      int f = 0;
      for (int b = lane; b < upto; b += 32) f += (pages(b) + sh.chunk - 1) / sh.chunk;
      sh.first = __reduce_add_sync(kFull, f);
    }
  }
  return sh;
}

// The pages left to a CTA: `left` of them, from page `page` of sequence `b` on.
struct Q4Range {
  int b, page, left;
};

template <typename Pages>
__device__ __forceinline__ bool next_part(const Q4Args& a, Q4Range& r, Pages pages, int& b, int& p0, int& p1) {
  while (r.left > 0 && r.b < a.B) {
    const int np = pages(r.b);
    b = r.b++;
    p0 = r.page;
    r.page = 0;
    if (p0 < np) {
      p1 = min(np, p0 + r.left);
      r.left -= p1 - p0;
      return true;
    }
  }
  return false;
}

// The range of one of `ctas` equal shares.
template <typename Pages>
__device__ __forceinline__ Q4Range equal_range(const Q4Args& a, int64_t total, int cta, int ctas, Pages pages) {
  int64_t at = total * cta / ctas;
  Q4Range r{0, 0, (int)(total * (cta + 1) / ctas - at)};
  while (r.b < a.B && at >= pages(r.b)) at -= pages(r.b++);
  r.page = (int)at;
  return r;
}

// The range of CTA `cta` of a scan (every thread of a warp; all the same).
template <typename Pages>
__device__ __forceinline__ Q4Range cta_range(const Q4Args& a, const Q4Share& sh, int cta, Pages pages) {
  if (sh.chunk == 0) return cta < sh.live() ? equal_range(a, sh.total, cta, sh.live(), pages) : Q4Range{0, 0, 0};
  int c = cta;
  for (int b = 0; b < a.B; ++b) {
    const int np = pages(b), f = (np + sh.chunk - 1) / sh.chunk;
    if (c < f) {
      const int at = (int)((int64_t)np * c / f);
      return Q4Range{b, at, (int)((int64_t)np * (c + 1) / f) - at};
    }
    c -= f;
  }
  return Q4Range{0, 0, 0};
}

// Shape of a scan CTA (one per SM). The attention has as many warps as the registers of one lane's state
// allow. The score has 16, so that the logits of a whole stage stay in registers. Each warp's ring has
// stages of two pages' blocks of K and V, or four of K, which share the cost of a wait and of a round of
// copies; a stage in flight per warp is twice what one SM's share of HBM bandwidth needs to cover a
// microsecond.
template <int NB, int NT, bool kAttend>
struct Q4Ring {
  static constexpr int WARPS = kAttend ? (NT == 1 ? 20 : 12) : 16;
  static constexpr int BLK = q4_block_bytes(NB * 64);
  static constexpr int OPS = kAttend ? 2 : 1;                      // blocks of a page
  static constexpr int PAGES = kAttend ? 2 : kScorePages;          // pages of a stage
  static constexpr int STAGE = PAGES * OPS * BLK;                  // [page][K, V][block]
  static constexpr int STAGES = kAttend ? (NT == 1 ? 2 : 3) : 8 / kScorePages;
  static constexpr int BYTES = STAGES * STAGE;
  static constexpr int QUERY = kQ4Sets * 4 * NT * NB * 64 * 4;     // the CTA's queries, behind the rings
  static constexpr int ROWS = kAttend ? 4 * NT * NB * 64 * 4 : 0;  // one warp's output sums, behind the queries
  static constexpr int SMEM = WARPS * (BYTES + ROWS) + QUERY;
  static_assert(SMEM + 4096 <= 227 * 1024, "shared memory of an SM");
  static_assert(BLK % 16 == 0, "bulk copies");
};

// kAttend: attention partials; otherwise logits and (max, sum exp) partials.
//
// Measured: attention of four sequences, 954K tokens, 32 heads over 8 of 128: 202 us, 5.1 TB/s of blocks;
// what binds is instruction issue (72% of the slots; the tensor pipe 27%). 28 heads over 4: 159 us, 3.3 TB/s;
// a block has twice the products and exponentials, on 12 warps (registers): issue 56%, tensor 35%. Scores of eight
// sequences, 898K tokens, 28 heads over 4: 74 us, 3.3 TB/s of blocks and 1.4 TB/s of logits; issue 56%, the
// rest waits for the tensor and integer pipes, which the unpacking and the products take in turn.
template <int NB, int NT, bool kAttend>
__global__ void __launch_bounds__(Q4Ring<NB, NT, kAttend>::WARPS * 32, 1) scan_kernel(const __grid_constant__ Q4Args a) {
  using R = Q4Ring<NB, NT, kAttend>;
  constexpr int D = NB * 64, CODES = q4_code_bytes(D);
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ __align__(8) uint64_t full[R::WARPS][R::STAGES];
  __shared__ float2 s_ml[R::WARPS][4 * NT];
  __shared__ Q4Unit<NB> s_units[kAttend ? R::WARPS : 1][4 * NT];
  __shared__ int s_pages[kScanSeqs];
  __shared__ Q4Range s_left;           // the CTA's pages that no part has been made of yet
  __shared__ int s_part[4];            // the part at work: is there one, sequence, first page, end

  // (values that are the same in a whole warp pass through a shuffle where they steer loops, so that
  // the compiler knows and needs no divergence handling there)
  const int tid = threadIdx.x, warp = __shfl_sync(kFull, tid >> 5, 0), lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int group = blockIdx.x % a.n_groups, cta = blockIdx.x / a.n_groups;
  const int set0 = group * kQ4Sets, nsets = min(kQ4Sets, a.HKV * a.sets_per_kv - set0);
  const int per_set = R::WARPS / nsets;                            // (some warps may be left over)
  launch_dependents();

  for (int b = tid; b < min(a.B, kScanSeqs); b += R::WARPS * 32) s_pages[b] = seq_pages(a, b);
  if (blockIdx.x == 0)
    for (int b = tid; b < a.B; b += R::WARPS * 32) {
      const int n = a.seq_lens[b];
      if (!(a.skip && a.skip[b]) && (n < 0 || n > a.max_tokens)) set_error(a.status, TS_ERR_SEQ_LEN);
    }
  if (lane == 0) {
    for (int s = 0; s < R::STAGES; ++s) mbar_init(&full[warp][s], 1);
    mbar_fence_init();
  }
  __syncthreads();
  // (the share and its parts are kept in shared memory by one thread: registers are short in the loop)
  auto pages = [&](int b) { return b < kScanSeqs ? s_pages[b] : seq_pages(a, b); };
  auto make_part = [&]() {
    int b = 0, p0 = 0, p1 = 0;
    s_part[0] = next_part(a, s_left, pages, b, p0, p1);
    s_part[1] = b;
    s_part[2] = p0;
    s_part[3] = p1;
  };
  if (warp == 0) {
    const Q4Range r = cta_range(a, share_pages(a, 0, lane, pages), cta, pages);
    if (lane == 0) {
      s_left = r;
      make_part();
    }
  }
  __syncthreads();

  const int hs = warp / per_set, j = warp % per_set;
  const bool works = hs < nsets;
  const int set = set0 + (works ? hs : 0);
  const int kv = set / a.sets_per_kv, head0 = kv * a.G + (set % a.sets_per_kv) * (4 * NT);
  const int nh = min(4 * NT, a.G - (set % a.sets_per_kv) * (4 * NT));   // heads of this set
  unsigned char* ring = smem + (size_t)warp * R::BYTES;
  float* sq = reinterpret_cast<float*>(smem + R::WARPS * R::BYTES);   // [sets][4 NT][D]
  float* sums = reinterpret_cast<float*>(smem + R::WARPS * R::BYTES + R::QUERY + warp * R::ROWS);   // [4 NT][D]
  uint64_t* bars = full[warp];
  uint32_t phases = 0u;                                            // bit s: parity of the stage's next wait
  bool ok = works;
  while (s_part[0]) {
    const int b = __shfl_sync(kFull, s_part[1], 0), p0 = __shfl_sync(kFull, s_part[2], 0),
              p1 = __shfl_sync(kFull, s_part[3], 0), n = __shfl_sync(kFull, a.seq_lens[b], 0);
    // this warp's pages: p0 + j, p0 + j + per_set, ...; lane i holds the id of the next 32 to copy
    const int32_t* pt = a.page_table + (size_t)b * a.pt_stride;
    const int mine = ok && p0 + j < p1 ? (p1 - p0 - j + per_set - 1) / per_set : 0;
    const int stages = (mine + R::PAGES - 1) / R::PAGES;
    int ids = 0, copied = 0, cs = 0;                               // stages copied so far, the next one's slot
    uint32_t lost = 0u;                                            // bit PAGES s + p: page p of slot s has no block
    // lane (page, operand) copies one block. The score's blocks are streamed through L2 (evict first): its
    // logits are read again by the votes and should stay there
    const unsigned char* pool = R::OPS == 2 && (lane & 1) ? a.v_pool : a.k_pool;
    const uint64_t policy = l2_evict_first_policy();
    auto copy_next = [&]() {
      if (copied >= stages) return;
      const int in_ids = (copied * R::PAGES) & 31;
      if (in_ids == 0) {
        const int i = copied * R::PAGES + lane;
        ids = -1;
        if (i < mine) {
          ids = pt[p0 + j + i * per_set];
          if (ids < 0 || (int64_t)ids >= a.num_pages) {
            set_error(a.status, TS_ERR_PAGE_OOB);
            ids = -1;
          }
        }
      }
      const int page = __shfl_sync(kFull, ids, in_ids + (lane / R::OPS & (R::PAGES - 1)));
      const bool in = lane < R::PAGES * R::OPS && page >= 0;       // (pages past the last one have no id)
      const unsigned good = __ballot_sync(kFull, in);
      if (lane == 0) mbar_arrive_expect_tx(&bars[cs], (uint32_t)__popc(good) * R::BLK);
      __syncwarp();
      if (in) {
        const unsigned char* src = pool + ((size_t)page * a.HKV + kv) * R::BLK;
        if (kAttend)
          bulk_g2s(ring + cs * R::STAGE + lane * R::BLK, src, R::BLK, &bars[cs]);
        else
          bulk_g2s_hint(ring + cs * R::STAGE + lane * R::BLK, src, R::BLK, &bars[cs], policy);
      }
      static_assert(R::OPS == 1 || R::PAGES == 2, "bits of the pages");
      constexpr unsigned kAll = (1u << R::PAGES) - 1u;
      const unsigned there = R::OPS == 1 ? good : ((good & 1u) | (good >> 1 & 2u));
      lost = (lost & ~(kAll << (R::PAGES * cs))) | ((~there & kAll) << (R::PAGES * cs));
      ++copied;
      cs = cs + 1 == R::STAGES ? 0 : cs + 1;
    };
    for (int i = 0; i < R::STAGES; ++i) copy_next();
    // the queries of all head sets, once for the CTA, while the first blocks are on their way
    for (int i = tid; i < nsets * 4 * NT * D; i += R::WARPS * 32) {
      const int e = i % D, h = i / D, in_set = h % (4 * NT), gs = set0 + h / (4 * NT);
      const int in_kv = gs % a.sets_per_kv * (4 * NT) + in_set;
      sq[i] = in_kv < a.G ? a.q[((size_t)b * a.H + gs / a.sets_per_kv * a.G + in_kv) * D + e] : 0.f;
    }
    __syncthreads();
    Q4Query<NB, NT> f;
    q4_load_query<NB, NT>(f, sq + (works ? hs : 0) * (4 * NT * D), lane);
    float mul[NT];
    Q4State<NB, NT> st;                                            // (the score uses its m and l alone)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) mul[nt] = a.scale * f.inv[nt];
    st.reset();
    int s = 0, left = n - (p0 + j) * kPage;                        // tokens of the sequence from this page on
    int done = 0;
    // the place in the page of token (u, c): the attention wants lane t's value rows, tokens (u, 2t)
    // and (u, 2t + 1), in different banks; the score wants neighbours for its stores
    auto token = [&](int u, int c) { return kAttend ? 8 * u + 4 * (c & 1) + (c >> 1) : 8 * u + c; };
    // where this lane's logits go, for head t of the set; 4 heads on for the next tile of heads
    float* row = a.logits + (size_t)b * a.H * a.max_tokens + (size_t)(head0 + t) * a.head_stride +
                 (size_t)(p0 + j) * a.page_stride + g;
    const size_t row_step = (size_t)per_set * a.page_stride, tile_step = (size_t)4 * a.head_stride;
    for (; done < stages; ++done) {
      ok = __all_sync(kFull, mbar_wait(&bars[s], (phases >> s) & 1u));
      if (!ok) {
        set_error(a.status, TS_ERR_TIMEOUT);
        break;
      }
      phases ^= 1u << s;
      // both pages of the stage together; one that does not exist, or has no block, has no tokens
      float x[R::PAGES][NT][2];
      int limit[R::PAGES];
      bool whole = true;
#pragma unroll
      for (int pg = 0; pg < R::PAGES; ++pg) {
        limit[pg] = (lost >> (R::PAGES * s + pg)) & 1u ? 0 : left - pg * per_set * kPage;
        whole &= limit[pg] >= kPage;
        const unsigned char* kb = ring + s * R::STAGE + pg * (R::OPS * R::BLK);
        uint2 kw[2][NB];
        float ks[NB][2];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            kw[u][nb] = *reinterpret_cast<const uint2*>(kb + nb * 512 + token(u, g) * 32 + t * 8);
            ks[nb][u] = bf16_bits_f(*reinterpret_cast<const uint16_t*>(kb + CODES + nb * 32 + token(u, g) * 2));
          }
        q4_scores<NB, NT>(f, kw, ks, x[pg]);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int u = 0; u < 2; ++u) x[pg][nt][u] *= mul[nt];
      }
      if (!whole) {
#pragma unroll
        for (int pg = 0; pg < R::PAGES; ++pg)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int u = 0; u < 2; ++u) x[pg][nt][u] = token(u, g) < limit[pg] ? x[pg][nt][u] : -INFINITY;
      }
      q4_raise_max<NB, NT, R::PAGES>(st, x);
      if constexpr (kAttend) {
#pragma unroll
        for (int pg = 0; pg < R::PAGES; ++pg) {
          const unsigned char* vb = ring + s * R::STAGE + pg * (R::OPS * R::BLK) + R::BLK;
          uint32_t vw[4][NB];
          float vs[NB][2];
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              vw[e][nb] = *reinterpret_cast<const uint32_t*>(vb + nb * 512 + token(e >> 1, 2 * t + (e & 1)) * 32 + g * 4);
#pragma unroll
            for (int u = 0; u < 2; ++u)
              vs[nb][u] = bf16_bits_f(*reinterpret_cast<const uint16_t*>(vb + CODES + nb * 32 + token(u, g) * 2));
          }
          if (pg == R::PAGES - 1) {
            __syncwarp();                                          // every lane has read the stage
            copy_next();
          }
          if (whole)
            q4_accumulate<NB, NT, false>(st, x[pg], vw, vs);
          else
            q4_accumulate<NB, NT, true>(st, x[pg], vw, vs);
        }
      } else {
        __syncwarp();
        copy_next();
#pragma unroll
        for (int pg = 0; pg < R::PAGES; ++pg) {
          const bool there = done * R::PAGES + pg < mine;          // (a page without a block has logits of -inf)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            st.l[nt] += q4_weight(x[pg][nt][0], st.m[nt]) + q4_weight(x[pg][nt][1], st.m[nt]);
            if (there && 4 * nt + t < nh) {
              row[nt * tile_step + pg * row_step] = x[pg][nt][0];
              row[nt * tile_step + pg * row_step + 8] = x[pg][nt][1];
            }
          }
        }
        row += R::PAGES * row_step;
      }
      if (kAttend && done % kQ4Flush == kQ4Flush - 1) st.flush(sums, s_units[warp], done < kQ4Flush, lane);
      left -= R::PAGES * per_set * kPage;
      s = s + 1 == R::STAGES ? 0 : s + 1;
    }
    if (!ok && works) {
      // a wait ran out: what was copied ahead lands before the ring is used for anything else
      for (; done < copied; ++done) {
        mbar_wait(&bars[s], (phases >> s) & 1u);
        s = s + 1 == R::STAGES ? 0 : s + 1;
      }
    }
    // the next sequence's copies begin at stage 0 again
    // ---- the warps of a head set join their states
    st.join_lanes();
    if (g == 0) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) s_ml[warp][4 * nt + t] = make_float2(st.m[nt], st.l[nt]);
    }
    __syncthreads();
    float fac[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float M = -INFINITY, L = 0.f;
      for (int w = 0; w < (works ? per_set : 0); ++w) M = fmaxf(M, s_ml[hs * per_set + w][4 * nt + t].x);
      for (int w = 0; w < (works ? per_set : 0); ++w) {
        const float2 ml = s_ml[hs * per_set + w][4 * nt + t];
        L += ml.y * part_weight(ml.x, M);
      }
      fac[nt] = part_weight(st.m[nt], M) * reciprocal(L);
      if (works && j == 0 && g == 0 && 4 * nt + t < nh)
        a.part_ml[(int64_t)(head0 + 4 * nt + t) * a.slots + cta + b] = make_float2(M, L);
    }
    if constexpr (kAttend) {
      st.flush(sums, s_units[warp], done < kQ4Flush, lane);
      // each warp's own factors: from its maximum to the set's and divided by the sum, and out of its powers of two
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
        if (g == 0) {
          s_units[warp][4 * nt + t].m = fac[nt];
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) s_units[warp][4 * nt + t].sc[nb] = __uint_as_float((254u << 23) - __float_as_uint(st.sc[nt][nb]));
        }
      __syncthreads();
      if (works) {
        float* po = a.part_o + ((int64_t)(cta + b) * a.H + head0) * D;
        const float* rows = reinterpret_cast<const float*>(smem + R::WARPS * R::BYTES + R::QUERY) + hs * per_set * (4 * NT * D);
        for (int i = j * 32 + lane; i < nh * D; i += per_set * 32) {
          float acc = 0.f;
          for (int w = 0; w < per_set; ++w) {
            const Q4Unit<NB>& f = s_units[hs * per_set + w][i / D];
            acc = fmaf(rows[w * (4 * NT * D) + i] * f.m, f.sc[i % D / 64], acc);
          }
          po[i] = acc;
        }
      }
    }
    if (tid == 0) make_part();                                     // (every warp has read the old one)
    __syncthreads();
  }
}

// The parts of a sequence's scan that exist: slots [first, first + count).
template <typename Pages>
__device__ __forceinline__ void scan_slots(const Q4Args& a, int b, int lane, Pages pages, int64_t& first, int& count) {
  const Q4Share sh = share_pages(a, b, lane, pages);
  const int np = pages(b);
  count = 0;
  first = 0;
  if (np == 0) return;
  if (sh.chunk > 0) {
    first = sh.first + b;
    count = (np + sh.chunk - 1) / sh.chunk;
    return;
  }
  const int nc = sh.live();
  const int c0 = (int)(((sh.before + 1) * nc - 1) / sh.total), c1 = (int)(((sh.before + np) * nc - 1) / sh.total);
  first = c0 + b;
  count = c1 - c0 + 1;
}

// Joins the parts of (head, sequence) in slot order. splits > 0: the gather's parts, splits per
// sequence; otherwise the scan's. Bound by the latency of its loads, all of which a thread has under way at
// once up to eight parts (7 us for 38 parts of 32 heads in four sequences, begun while the scan ends).
constexpr int kMaxParts = 512;   // of one sequence
template <int D>
__global__ void __launch_bounds__(1024, 1) q4_merge_kernel(const __grid_constant__ Q4Args a, int splits, float* out,
                                                        float* lse) {
  constexpr int ROWS = 1024 / D;   // parts added at once
  const int h = blockIdx.x, b = blockIdx.y, tid = threadIdx.x, e = tid % D, row = tid / D;
  __shared__ float s_o[ROWS][D];
  __shared__ float2 s_ml[kMaxParts];
  int64_t first;
  int count;
  if (splits > 0) {
    first = (int64_t)b * splits;
    count = splits;
  } else {
    scan_slots(a, b, tid & 31, [&](int i) { return seq_pages(a, i); }, first, count);
  }
  wait_for_primary();
  // the outputs of a thread's first parts are on their way while the sums are joined
  constexpr int BATCH = 8;
  const float* po = a.part_o + (first * a.H + h) * D + e;
  float x[BATCH];
  auto load = [&](int i0) {
#pragma unroll
    for (int k = 0; k < BATCH; ++k) x[k] = i0 + k * ROWS < count ? __ldcg(po + (size_t)(i0 + k * ROWS) * a.H * D) : 0.f;
  };
  for (int i = tid; i < count; i += blockDim.x) s_ml[i] = __ldcg(a.part_ml + h * a.slots + first + i);
  load(row);
  __syncthreads();
  // every warp the same maximum and sum
  float M = -INFINITY, L = 0.f;
  for (int i = tid & 31; i < count; i += 32) M = fmaxf(M, s_ml[i].x);
  M = warp_max(M);
  for (int i = tid & 31; i < count; i += 32) L = fmaf(part_weight(s_ml[i].x, M), s_ml[i].y, L);
  L = warp_sum(L);
  const float inv = reciprocal(L);
  float o = 0.f;
  for (int i0 = row; i0 < count; i0 += BATCH * ROWS) {
    if (i0 != row) load(i0);
#pragma unroll
    for (int k = 0; k < BATCH; ++k)
      if (i0 + k * ROWS < count) {
        const float2 ml = s_ml[i0 + k * ROWS];
        o = fmaf(part_weight(ml.x, M) * ml.y * inv, x[k], o);
      }
  }
  s_o[row][e] = o;
  __syncthreads();
  if (row != 0) return;
  float O = 0.f;
#pragma unroll
  for (int i = 0; i < ROWS; ++i) O += s_o[i][e];
  out[((size_t)b * a.H + h) * D + e] = O;
  // (a sum of NaN, of a NaN among the rows, is not an empty sequence)
  if (lse && e == 0) lse[(size_t)b * a.H + h] = L != 0.f ? (M + log2f(L)) * 0.6931471805599453f : -INFINITY;
}

// The head soft vote from the scan's base-2 logits and parts: v_i = sum_h 2^(l_hi - M_h) / Z_h. Like the
// scan, a CTA takes an even, contiguous share of the batch's pages; for each sequence in it its warps
// first join the heads' parts (the same in every CTA), then a warp sums a page at a time: lane (head, quad)
// every eighth head of four tokens, and then across the lanes. The logits of a page lie together, so a load
// of the warp is 512 contiguous bytes, four of which are under way per page. Measured: 101 MB of logits,
// 27 us, 3.7 TB/s, more than half of them out of L2.
constexpr int kVoteThreads = 512;
constexpr int kVoteHeads = 256;

__global__ void __launch_bounds__(kVoteThreads, 2) q4_vote_kernel(const __grid_constant__ Q4Args a, float* vote,
                                                                  int64_t vote_stride) {
  constexpr int WARPS = kVoteThreads / 32, BATCH = 4;
  __shared__ float2 s_mz[kVoteHeads];
  __shared__ int s_pages[kScanSeqs];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, quad = lane & 3, h8 = lane >> 2;
  for (int b = tid; b < min(a.B, kScanSeqs); b += kVoteThreads) s_pages[b] = seq_pages(a, b);
  __syncthreads();
  auto pages = [&](int i) { return i < kScanSeqs ? s_pages[i] : seq_pages(a, i); };
  Q4Range r = equal_range(a, share_pages(a, 0, lane, pages).total, blockIdx.x, gridDim.x, pages);
  int b, p0, p1;
  wait_for_primary();
  while (next_part(a, r, pages, b, p0, p1)) {
    const int n = a.seq_lens[b];
    const float* logits = a.logits + (size_t)b * a.H * a.max_tokens + 4 * quad;
    // heads h8 + 8 (k0 .. k0 + 3) of this lane's four tokens of page pg
    auto load = [&](float4 (&x)[BATCH], int pg, int k0) {
#pragma unroll
      for (int k = 0; k < BATCH; ++k) {
        const int h = h8 + 8 * (k0 + k);
        x[k] = pg < p1 && h < a.H
                   ? __ldcg(reinterpret_cast<const float4*>(logits + (size_t)pg * a.page_stride + (size_t)h * a.head_stride))
                   : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
      }
    };
    float4 x[BATCH];
    load(x, p0 + warp, 0);                         // on their way while the statistics are joined
    int64_t first;
    int count;
    scan_slots(a, b, lane, pages, first, count);
    __syncthreads();                               // the last sequence's statistics are done with
    for (int h = warp; h < a.H; h += WARPS) {
      constexpr int FIRST = 5;                     // parts of a lane under way at once
      const float2* ml = a.part_ml + h * a.slots + first;
      float2 y[FIRST];
#pragma unroll
      for (int k = 0; k < FIRST; ++k) y[k] = lane + 32 * k < count ? ml[lane + 32 * k] : make_float2(-INFINITY, 0.f);
      float M = -INFINITY;
#pragma unroll
      for (int k = 0; k < FIRST; ++k) M = fmaxf(M, y[k].x);
      for (int i = lane + 32 * FIRST; i < count; i += 32) M = fmaxf(M, ml[i].x);
      M = warp_max(M);
      KahanF z;
#pragma unroll
      for (int k = 0; k < FIRST; ++k) z.add(y[k].y * part_weight(y[k].x, M));
      for (int i = lane + 32 * FIRST; i < count; i += 32) z.add(ml[i].y * part_weight(ml[i].x, M));
      const float Z = warp_sum_comp(z.s, -z.c);
      // a sequence none of whose pages is in the pool has logits of -inf alone and a sum of zero: votes of zero
      if (lane == 0) s_mz[h] = Z == 0.f ? make_float2(0.f, 0.f) : make_float2(M, 1.f / Z);
    }
    __syncthreads();
    for (int pg = p0 + warp; pg < p1; pg += WARPS) {
      float acc[4] = {0.f, 0.f, 0.f, 0.f};
      float4 next[BATCH];
      load(next, pg + WARPS, 0);
      for (int k0 = 0; 8 * k0 < a.H; k0 += BATCH) {
        if (k0 > 0) load(x, pg, k0);
#pragma unroll
        for (int k = 0; k < BATCH; ++k) {
          const int h = h8 + 8 * (k0 + k);
          if (h >= a.H) continue;
          const float2 mz = s_mz[h];
          acc[0] = fmaf(ex2(x[k].x - mz.x), mz.y, acc[0]);
          acc[1] = fmaf(ex2(x[k].y - mz.x), mz.y, acc[1]);
          acc[2] = fmaf(ex2(x[k].z - mz.x), mz.y, acc[2]);
          acc[3] = fmaf(ex2(x[k].w - mz.x), mz.y, acc[3]);
        }
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        acc[e] += __shfl_xor_sync(kFull, acc[e], 4);
        acc[e] += __shfl_xor_sync(kFull, acc[e], 8);
        acc[e] += __shfl_xor_sync(kFull, acc[e], 16);
      }
      // lane (h8 = e, quad) writes token 4 quad + e
      const float v = h8 == 0 ? acc[0] : h8 == 1 ? acc[1] : h8 == 2 ? acc[2] : acc[3];
      const int i = pg * kPage + 4 * quad + h8;
      if (h8 < 4 && i < n) vote[(size_t)b * vote_stride + i] = v;
#pragma unroll
      for (int k = 0; k < BATCH; ++k) x[k] = next[k];
    }
  }
}

struct Q4GatherArgs {
  const int32_t* idx;     // [B][idx_stride]
  int64_t idx_stride;
  const int32_t* count;   // [B]
  int splits;
};

// CTA (split, head set, sequence): a contiguous part of the index list, 16 tokens per warp and step. Bound by
// a chain of latencies (list, page id, row), so the list is spread over as many CTAs as fit at once and
// the next step's ids are looked up early: 2564 of 131,057 tokens, 32 heads over 8: 9.3 us from cold caches, the
// merge, begun meanwhile, 5.7. Two CTAs of six warps to an SM: over the same inputs again and again, with merge,
// that list takes 9.2 us and one of 20,000 17.3 (four CTAs of four warps: 10.3 and 18.4; two of eight, as far as
// the registers allow: 9.6 and 16.8, but eight lists of 10,000 with 28 heads over 4 58 in place of 47).
template <int NB, int NT>
__global__ void __launch_bounds__(kGatherWarps * 32, kGatherCtas) gather_kernel(const __grid_constant__ Q4Args a,
                                                                                  const __grid_constant__ Q4GatherArgs ga) {
  constexpr int D = NB * 64, BLK = q4_block_bytes(D), CODES = q4_code_bytes(D);
  __shared__ __align__(16) float merge[kGatherWarps][4 * NT][D];
  __shared__ __align__(16) float sq[4 * NT * D];
  __shared__ float2 s_ml[kGatherWarps][4 * NT];
  __shared__ Q4Unit<NB> s_units[kGatherWarps][4 * NT];
  const int split = blockIdx.x, set = blockIdx.y, b = blockIdx.z;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int kv = set / a.sets_per_kv, head0 = kv * a.G + (set % a.sets_per_kv) * (4 * NT);
  const int nh = min(4 * NT, a.G - (set % a.sets_per_kv) * (4 * NT));
  const int cnt = (int)min((int64_t)max(ga.count[b], 0), ga.idx_stride);
  const int units = (cnt + 15) / 16;
  const int u0 = (int)((int64_t)units * split / ga.splits), u1 = (int)((int64_t)units * (split + 1) / ga.splits);
  const int32_t* ib = ga.idx + (size_t)b * ga.idx_stride;
  const int32_t* pt = a.page_table + (size_t)b * a.pt_stride;

  launch_dependents();
  // lane i looks up list entry i (of 16) of a step: its row in the pool, -1 where there is none. The next
  // step's entries are looked up while one step's rows are on their way.
  auto listed = [&](int u) -> int64_t {
    const int at = u * 16 + (lane & 15);
    if (u >= u1 || at >= cnt) return -1;
    const int tk = ib[at];
    int page = -1;
    if (tk >= 0 && tk < a.max_tokens) page = pt[tk / kPage];
    if (page >= 0 && (int64_t)page < a.num_pages) return ((int64_t)page * a.HKV + kv) * kPage + tk % kPage;
    set_error(a.status, TS_ERR_PAGE_OOB);
    return -1;
  };
  int64_t mine = listed(u0 + warp);
  for (int i = tid; i < 4 * NT * D; i += kGatherWarps * 32)
    sq[i] = i / D < nh ? a.q[((size_t)b * a.H + head0) * D + i] : 0.f;
  __syncthreads();
  Q4Query<NB, NT> f;
  q4_load_query<NB, NT>(f, sq, lane);
  float mul[NT];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) mul[nt] = a.scale * f.inv[nt];
  Q4State<NB, NT> st;
  st.reset();
  int steps = 0;
  bool flushed = false;
  for (int u = u0 + warp; u < u1; u += kGatherWarps) {
    uint2 kw[2][NB];
    float ks[NB][2], vs[NB][2], x[1][NT][2];
    uint32_t vw[4][NB];
    bool in[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int64_t row = __shfl_sync(kFull, mine, 8 * i + g);
      in[i] = row >= 0;
      const size_t blk = in[i] ? (size_t)(row / kPage) * BLK : 0;
      const int slot = in[i] ? (int)(row % kPage) : 0;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        const size_t so = blk + CODES + nb * 32 + slot * 2;
        kw[i][nb] = in[i] ? *reinterpret_cast<const uint2*>(a.k_pool + blk + nb * 512 + slot * 32 + t * 8) : make_uint2(0u, 0u);
        ks[nb][i] = in[i] ? bf16_bits_f(*reinterpret_cast<const uint16_t*>(a.k_pool + so)) : 0.f;
        vs[nb][i] = in[i] ? bf16_bits_f(*reinterpret_cast<const uint16_t*>(a.v_pool + so)) : 0.f;
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t row = __shfl_sync(kFull, mine, 8 * (i >> 1) + 2 * t + (i & 1));
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
        vw[i][nb] = row < 0 ? 0u
                            : *reinterpret_cast<const uint32_t*>(a.v_pool + (size_t)(row / kPage) * BLK + nb * 512 +
                                                                 (row % kPage) * 32 + g * 4);
    }
    mine = listed(u + kGatherWarps);
    q4_scores<NB, NT>(f, kw, ks, x[0]);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 2; ++i) x[0][nt][i] = in[i] ? x[0][nt][i] * mul[nt] : -INFINITY;
    q4_raise_max<NB, NT, 1>(st, x);
    q4_accumulate<NB, NT, true>(st, x[0], vw, vs);
    if (++steps % (2 * kQ4Flush) == 0) {
      st.flush(&merge[warp][0][0], s_units[warp], !flushed, lane);
      flushed = true;
    }
  }
  st.join_lanes();
  if (g == 0) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) s_ml[warp][4 * nt + t] = make_float2(st.m[nt], st.l[nt]);
  }
  st.flush(&merge[warp][0][0], s_units[warp], !flushed, lane);
  __syncthreads();
  const int64_t slot = (int64_t)b * ga.splits + split;
  // a thread to each (warp, head): the warp's factor in the head's part
  if (tid < kGatherWarps * 4 * NT) {
    const int w = tid / (4 * NT), hg = tid % (4 * NT);
    float M = -INFINITY, L = 0.f;
#pragma unroll
    for (int i = 0; i < kGatherWarps; ++i) M = fmaxf(M, s_ml[i][hg].x);
#pragma unroll
    for (int i = 0; i < kGatherWarps; ++i) L = fmaf(part_weight(s_ml[i][hg].x, M), s_ml[i][hg].y, L);
    s_units[w][hg].m = part_weight(s_ml[w][hg].x, M) * reciprocal(L);
    if (w == 0 && hg < nh) a.part_ml[(head0 + hg) * a.slots + slot] = make_float2(M, L);
  }
  __syncthreads();
  for (int i = tid; i < nh * D; i += kGatherWarps * 32) {
    const int hg = i / D;
    float O = 0.f;
#pragma unroll
    for (int w = 0; w < kGatherWarps; ++w)
      O = fmaf(merge[w][hg][i % D] * s_units[w][hg].m, __uint_as_float((254u << 23) - __float_as_uint(s_units[w][hg].sc[i % D / 64])), O);
    a.part_o[(slot * a.H + head0) * D + i] = O;
  }
}

Q4Args make_args(ts_ctx* ctx, const float* q, const void* k_pool, const void* v_pool, const int32_t* page_table,
                 const int32_t* seq_lens, int B, float scale) {
  const ts_config& c = ctx->cfg;
  Q4Args a{};
  a.q = q;
  a.k_pool = static_cast<const unsigned char*>(k_pool);
  a.v_pool = static_cast<const unsigned char*>(v_pool);
  a.page_table = page_table;
  a.pt_stride = c.max_pages_per_seq;
  a.num_pages = c.num_pages;
  a.seq_lens = seq_lens;
  a.max_tokens = ctx->max_tokens;
  a.B = B;
  a.H = c.n_q_heads;
  a.HKV = c.n_kv_heads;
  a.G = a.H / a.HKV;
  a.set_heads = a.G <= 4 ? 4 : 8;
  a.sets_per_kv = (a.G + a.set_heads - 1) / a.set_heads;
  a.n_groups = (a.HKV * a.sets_per_kv + kQ4Sets - 1) / kQ4Sets;
  a.ctas = ctx->num_sms / a.n_groups;
  a.ctas = std::max(1, std::min(a.ctas, kMaxParts));
  a.scale = scale;
  a.logits = ctx->logits;
  a.part_o = ctx->q4_part_o;
  a.part_ml = ctx->q4_part_ml;
  a.slots = q4_part_slots(c, ctx->num_sms);
  a.status = ctx->status;
  return a;
}

// Launches `kernel` as a dependent of the kernel before it in the stream (see launch_dependents).
template <typename... Params, typename... Args>
cudaError_t launch_behind(void (*kernel)(Params...), dim3 grid, int threads, cudaStream_t s, Args&&... args) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t lc = {};
  lc.gridDim = grid;
  lc.blockDim = dim3(threads);
  lc.stream = s;
  lc.attrs = attr;
  lc.numAttrs = 1;
  return cudaLaunchKernelEx(&lc, kernel, std::forward<Args>(args)...);
}

template <int NB, int NT>
ts_status run_attend(ts_ctx* ctx, const Q4Args& a, float* out, float* lse, cudaStream_t s) {
  constexpr size_t smem = Q4Ring<NB, NT, true>::SMEM;
  if (!ensure_smem<scan_kernel<NB, NT, true>>(smem, ctx->device)) return TS_ERR_CUDA;
  ProfScope ps(ctx, TS_PROF_ATTEND, s);
  ctx->kernels += 2;
  scan_kernel<NB, NT, true><<<a.ctas * a.n_groups, Q4Ring<NB, NT, true>::WARPS * 32, smem, s>>>(a);
  const cudaError_t e = cudaGetLastError();
  return cuda_status(e != cudaSuccess ? e : launch_behind(q4_merge_kernel<NB * 64>, dim3(a.H, a.B), 1024, s, a, 0, out, lse));
}

template <int NB, int NT>
ts_status run_scan(ts_ctx* ctx, const Q4Args& a, cudaStream_t s) {
  constexpr size_t smem = Q4Ring<NB, NT, false>::SMEM;
  if (!ensure_smem<scan_kernel<NB, NT, false>>(smem, ctx->device)) return TS_ERR_CUDA;
  ProfScope ps(ctx, TS_PROF_SCORE, s);
  ctx->kernels += 1;
  scan_kernel<NB, NT, false><<<a.ctas * a.n_groups, Q4Ring<NB, NT, false>::WARPS * 32, smem, s>>>(a);
  return cuda_status(cudaGetLastError());
}

template <int NB, int NT>
ts_status run_gather(ts_ctx* ctx, const Q4Args& a, const Q4GatherArgs& ga, float* out, float* lse, cudaStream_t s) {
  ProfScope ps(ctx, TS_PROF_ATTEND, s);
  ctx->kernels += 2;
  gather_kernel<NB, NT><<<dim3(ga.splits, a.HKV * a.sets_per_kv, a.B), kGatherWarps * 32, 0, s>>>(a, ga);
  const cudaError_t e = cudaGetLastError();
  return cuda_status(e != cudaSuccess ? e : launch_behind(q4_merge_kernel<NB * 64>, dim3(a.H, a.B), 1024, s, a, ga.splits, out, lse));
}

}  // namespace

// (64-element blocks of a head, column tiles of a head set)
#define TS_Q4_DISPATCH(FN, ...)                                                                   \
  (ctx->cfg.head_dim == 64 ? (a.set_heads == 4 ? FN<1, 1>(__VA_ARGS__) : FN<1, 2>(__VA_ARGS__)) \
                           : (a.set_heads == 4 ? FN<2, 1>(__VA_ARGS__) : FN<2, 2>(__VA_ARGS__)))

bool q4_supported(const ts_config& c) {
  return c.kv_dtype == TS_KV_Q4 && c.page_size == kPage && (c.head_dim == 64 || c.head_dim == 128) &&
         c.n_q_heads / c.n_kv_heads <= 16;
}

// Parts of any call: a scan has at most one per CTA and one more per sequence, a gather at most
// kGatherCtas num_sms, or one per sequence.
int64_t q4_part_slots(const ts_config& c, int num_sms) { return kGatherCtas * (int64_t)num_sms + c.max_batch; }

ts_status launch_attend_q4(ts_ctx* ctx, const AttendCall& c, const int32_t* seq_lens, cudaStream_t s) {
  Q4Args a = make_args(ctx, c.q, c.k_pool, c.v_pool, c.page_table, seq_lens, c.B, c.scale * kLog2e);
  if (!c.idx) return TS_Q4_DISPATCH(run_attend, ctx, a, c.out, c.lse, s);
  // as many CTAs as fit the GPU at once, but no more than have a step for each of their warps: every part
  // costs the merge
  const int sets = a.HKV * a.sets_per_kv * a.B, fit = kGatherCtas * ctx->num_sms / sets;
  const int64_t full = (c.idx_stride + 16 * kGatherWarps - 1) / (16 * kGatherWarps);
  const int splits = (int)std::max<int64_t>(1, std::min<int64_t>(std::min(fit, kAttnMaxSplits), full));
  Q4GatherArgs ga{c.idx, c.idx_stride, c.count, splits};
  return TS_Q4_DISPATCH(run_gather, ctx, a, ga, c.out, c.lse, s);
}

ts_status launch_score_q4(ts_ctx* ctx, const ScoreCall& c, cudaStream_t s) {
  const bool soft = c.fn == TS_SCORE_HEAD_SOFT_VOTE;
  Q4Args a = make_args(ctx, c.q, c.k_pool, nullptr, c.page_table, c.seq_lens, c.B, soft ? c.scale * kLog2e : c.scale);
  a.skip = c.skip;
  // for the votes page by page, so that what is written and read together lies together; the other
  // selection functions read [B][H][max_tokens]
  a.head_stride = soft ? kPage : a.max_tokens;
  a.page_stride = soft ? (int64_t)kPage * a.H : kPage;
  const ts_status st = TS_Q4_DISPATCH(run_scan, ctx, a, s);
  if (st != TS_OK || !soft) return st;   // the other selection functions rank the natural logits themselves
  ProfScope ps(ctx, TS_PROF_VOTE, s);
  ctx->kernels += 1;
  return cuda_status(launch_behind(q4_vote_kernel, dim3(2 * ctx->num_sms), kVoteThreads, s, a, c.vote, c.vote_stride));
}

}  // namespace ts
