// Score and attention over a 4-bit paged cache (TS_KV_Q4; block format and tensor-core pieces in
// ts_q4.cuh).
//
//   l[h][i] = scale <q_h, (u_i - 8) s_i>      out_h = sum_i softmax_i(l[h]) (u'_i - 8) s'_i
//
// Both read every block of a sequence once and nothing else of size, so they are bound by the
// stream of 4-bit blocks (68 bytes per row of 128) as long as the arithmetic keeps up: the codes
// are unpacked in registers (9 instructions for 8 codes) and multiplied on the tensor cores.
//
// scan_kernel (whole sequences): a CTA owns a group of up to 4 head sets (a head set: up to 8 query
// heads of one KV head) and an even share of all pages of the batch, as one contiguous range. A
// producer warp streams its pages' blocks through a ring in shared memory with bulk copies; 12
// consumer warps, 12 / sets of them per head set, take the pages in turn. At the end of a
// sequence's part of the range the warps of a head set join their states, and q4_merge_kernel
// joins the parts of a sequence in CTA order. Every sum has a fixed order.
//
// gather_kernel (a list of tokens): 16 listed tokens per step straight from global memory; the list
// is split over CTAs and joined by the same merge.
#include <algorithm>
#include <cmath>

#include "ts_q4.cuh"

namespace ts {
namespace {

constexpr int kQ4Warps = 12;                    // consumer warps: a multiple of 1, 2, 3 and 4 head sets
constexpr int kQ4Threads = (kQ4Warps + 1) * 32;
constexpr int kQ4Sets = 4;                      // head sets of a CTA, at most
constexpr int kQ4MaxStages = 32;
constexpr int kQ4RingBytes = 144 * 1024;
constexpr int kGatherWarps = 4;

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
  int sets_per_kv;               // head sets of one KV head: ceil(G / 8)
  int n_groups;                  // groups of kQ4Sets head sets
  int ctas;                      // CTAs per group
  float scale;
  float* logits;                 // score: [B][H][max_tokens]
  float* part_o;                 // [slot][H][d]
  float2* part_ml;               // [slot][H]: max and sum (base 2 for attention, natural for the score)
  int* status;
};

__device__ __forceinline__ int seq_pages(const Q4Args& a, int b) {
  if (a.skip && a.skip[b]) return 0;
  const int n = a.seq_lens[b];
  return (n < 0 || n > a.max_tokens) ? 0 : (n + kPage - 1) / kPage;
}

// CTAs of a group that get pages: a share is at least one page for every warp of a head set, so a
// short batch does not spread over CTAs whose merge would cost more than their pages.
__device__ __forceinline__ int live_ctas(int64_t total, int ctas) {
  const int64_t want = (total + 2) / 3;
  return (int)(want < 1 ? 1 : (want < ctas ? want : ctas));
}

// Weight of a part with maximum m in a join with maximum M. Equal maxima weigh 1 also where both are
// -inf: an empty part brings zeros, a part of NaN logits brings its NaN.
template <bool kBase2>
__device__ __forceinline__ float part_weight(float m, float M) {
  return m == M ? 1.f : (kBase2 ? ex2(m - M) : expf(m - M));
}

// Total pages of the batch and of the sequences before `upto` (one warp; the same in every lane).
__device__ __forceinline__ void count_pages(const Q4Args& a, int upto, int lane, int64_t& total, int64_t& before) {
  int64_t t = 0, u = 0;
  for (int b = lane; b < a.B; b += 32) {
    const int n = seq_pages(a, b);
    t += n;
    if (b < upto) u += n;
  }
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) {
    t += __shfl_xor_sync(kFull, t, d);
    u += __shfl_xor_sync(kFull, u, d);
  }
  total = t;
  before = u;
}

// The part of one CTA's page range that lies in one sequence.
struct Q4Range {
  int64_t at, end;   // pages of the batch left to this CTA
  int b;             // sequence of `at`
  int64_t b0;        // first page of sequence b in the batch
};

__device__ __forceinline__ bool next_part(const Q4Args& a, Q4Range& r, int& b, int& p0, int& p1) {
  while (r.at < r.end && r.b < a.B) {
    const int np = seq_pages(a, r.b);
    if (r.at < r.b0 + np) {
      b = r.b;
      p0 = (int)(r.at - r.b0);
      p1 = (int)min((int64_t)np, r.end - r.b0);
      r.at = r.b0 + p1;
      return true;
    }
    r.b0 += np;
    ++r.b;
  }
  return false;
}

// kAttend: attention partials; otherwise logits and (max, sum exp) partials.
template <int NB, bool kAttend>
__global__ void __launch_bounds__(kQ4Threads, 1) scan_kernel(const __grid_constant__ Q4Args a) {
  constexpr int D = NB * 64;
  constexpr int BLK = q4_block_bytes(D), CODES = q4_code_bytes(D);
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ __align__(8) uint64_t full[kQ4MaxStages], empty[kQ4MaxStages];
  __shared__ int s_valid[kQ4MaxStages];
  __shared__ float2 s_ml[kQ4Warps][8];
  __shared__ Q4Range s_range;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int group = blockIdx.x % a.n_groups, cta = blockIdx.x / a.n_groups;
  const int set0 = group * kQ4Sets, nsets = min(kQ4Sets, a.HKV * a.sets_per_kv - set0);
  const int kv0 = set0 / a.sets_per_kv, nkv = (set0 + nsets - 1) / a.sets_per_kv - kv0 + 1;
  const int per_set = kQ4Warps / nsets;
  const int operand = nkv * BLK;                                   // bytes of one page's K (or V) of this group
  const int stage_bytes = (kAttend ? 2 : 1) * operand;
  const int nst = min(kQ4MaxStages, kQ4RingBytes / stage_bytes);

  if (warp == 0) {
    // this CTA's pages of the batch and the sequence they begin in
    int64_t total, before;
    count_pages(a, 0, lane, total, before);
    if (lane == 0) {
      const int nc = live_ctas(total, a.ctas);
      Q4Range r;
      r.at = cta < nc ? total * cta / nc : 0;
      r.end = cta < nc ? total * (cta + 1) / nc : 0;
      r.b = 0;
      r.b0 = 0;
      s_range = r;
      for (int s = 0; s < nst; ++s) {
        mbar_init(&full[s], 1);
        mbar_init(&empty[s], nsets);
      }
      mbar_fence_init();
    }
    if (cta == 0 && group == 0)
      for (int b = lane; b < a.B; b += 32) {
        const int n = a.seq_lens[b];
        if (!(a.skip && a.skip[b]) && (n < 0 || n > a.max_tokens)) set_error(a.status, TS_ERR_SEQ_LEN);
      }
  }
  __syncthreads();
  Q4Range r = s_range;
  int b, p0, p1, it = 0;                                           // it: pages of this CTA so far

  if (warp == kQ4Warps) {
    // ---- producer: 32 page ids at a time, then one bulk copy per page and operand
    bool ok = true;
    while (ok && next_part(a, r, b, p0, p1)) {
      for (int c0 = p0; c0 < p1 && ok; c0 += 32) {
        const int mine = c0 + lane < p1 ? a.page_table[(size_t)b * a.pt_stride + c0 + lane] : 0;
        for (int j = 0; j < min(32, p1 - c0); ++j, ++it) {
          const int page = __shfl_sync(kFull, mine, j);
          const int s = it % nst;
          int fine = 1;
          if (lane == 0) {
            if (it >= nst) fine = mbar_wait(&empty[s], ((it / nst) - 1) & 1);
            if (fine) {
              const bool in = page >= 0 && (int64_t)page < a.num_pages;
              s_valid[s] = in;
              if (in) {
                unsigned char* dst = smem + (size_t)s * stage_bytes;
                const size_t off = ((size_t)page * a.HKV + kv0) * BLK;
                mbar_arrive_expect_tx(&full[s], (uint32_t)stage_bytes);
                bulk_g2s(dst, a.k_pool + off, (uint32_t)operand, &full[s]);
                if (kAttend) bulk_g2s(dst + operand, a.v_pool + off, (uint32_t)operand, &full[s]);
              } else {
                set_error(a.status, TS_ERR_PAGE_OOB);
                mbar_arrive(&full[s]);
              }
            }
          }
          if (!__shfl_sync(kFull, fine, 0)) {
            if (lane == 0) set_error(a.status, TS_ERR_TIMEOUT);
            ok = false;
            break;
          }
        }
      }
    }
    // no copy may still be landing when the CTA exits
    if (lane == 0)
      for (int i = max(0, it - nst); i < it; ++i)
        if (!mbar_wait(&full[i % nst], (i / nst) & 1)) set_error(a.status, TS_ERR_TIMEOUT);
    return;
  }

  // ---- consumers: warp -> (head set, pages it = j mod per_set)
  const int hs = warp / per_set, j = warp % per_set;
  const bool works = hs < nsets;
  const int set = set0 + (works ? hs : 0);
  const int kv = set / a.sets_per_kv, head0 = kv * a.G + (set % a.sets_per_kv) * 8;
  const int nh = min(8, a.G - (set % a.sets_per_kv) * 8);          // heads of this set
  float* merge = reinterpret_cast<float*>(smem + kQ4RingBytes);    // [warps][8][D]
  bool ok = works;
  while (next_part(a, r, b, p0, p1)) {
    const int n = a.seq_lens[b];
    Q4Query<NB> f;
    q4_load_query<NB>(f, a.q + ((size_t)b * a.H + head0 + (g < nh ? g : 0)) * D, g < nh, t);
    const float mul = a.scale * f.inv * (kAttend ? 1.4426950408889634f : 1.f);
    Q4State<NB> st;
    st.reset();
    float m = -INFINITY, l = 0.f;                                  // the score's running (max, sum exp) of this lane
    for (int p = p0; p < p1; ++p, ++it) {
      if (it % per_set != j || !ok) continue;
      const int s = it % nst;
      if (!mbar_wait(&full[s], (it / nst) & 1)) {
        set_error(a.status, TS_ERR_TIMEOUT);
        ok = false;
        continue;
      }
      const unsigned char* kb = smem + (size_t)s * stage_bytes + (kv - kv0) * BLK;
      const bool valid = s_valid[s] != 0;
      uint2 kw[2][NB];
      float ks[NB][4];
      // token (tile u, column c) of the 16: the attention wants lane t's four tokens to be t + 4 i
      // (its V rows then fall in different banks), the score wants neighbours for its stores
      auto token = [&](int u, int c) { return kAttend ? 8 * u + 4 * (c & 1) + (c >> 1) : 8 * u + c; };
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
        for (int u = 0; u < 2; ++u)
          kw[u][nb] = *reinterpret_cast<const uint2*>(kb + nb * 512 + token(u, g) * 32 + t * 8);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          ks[nb][i] = bf16_bits_f(
              *reinterpret_cast<const uint16_t*>(kb + CODES + nb * 32 + token(i >> 1, 2 * t + (i & 1)) * 2));
      }
      float x[4];
      q4_scores<NB>(f, kw, ks, x);
      const int left = valid ? n - p * kPage : 0;                  // tokens of the sequence in this page
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = token(i >> 1, 2 * t + (i & 1)) < left ? x[i] * mul : -INFINITY;
      if constexpr (kAttend) {
        const unsigned char* vb = kb + operand;
        uint32_t vw[4][NB];
        float vs[NB][4];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int tk = token(i >> 1, 2 * t + (i & 1));
            vw[i][nb] = *reinterpret_cast<const uint32_t*>(vb + nb * 512 + tk * 32 + g * 4);
            vs[nb][i] = bf16_bits_f(*reinterpret_cast<const uint16_t*>(vb + CODES + nb * 32 + tk * 2));
          }
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[s]);
        q4_accumulate<NB>(st, x, vw, vs);
      } else {
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[s]);
        const float mn = fmaxf(m, fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])));
        l *= m == mn ? 1.f : expf(m - mn);
#pragma unroll
        for (int i = 0; i < 4; ++i) l += x[i] == -INFINITY ? 0.f : expf(x[i] - mn);
        m = mn;
        if (g < nh) {
          float* row = a.logits + ((size_t)b * a.H + head0 + g) * a.max_tokens + p * kPage + 2 * t;
#pragma unroll
          for (int u = 0; u < 2; ++u) *reinterpret_cast<float2*>(row + 8 * u) = make_float2(x[2 * u], x[2 * u + 1]);
        }
      }
    }
    // ---- the warps of a head set join their states (named barrier of the consumers)
    if constexpr (kAttend) {
      l = st.l;
      m = st.m;
    } else {
      const float m1 = fmaxf(m, __shfl_xor_sync(kFull, m, 1));
      const float mn = fmaxf(m1, __shfl_xor_sync(kFull, m1, 2));
      l *= m == mn ? 1.f : expf(m - mn);
      m = mn;
    }
    l += __shfl_xor_sync(kFull, l, 1);
    l += __shfl_xor_sync(kFull, l, 2);
    if (t == 0) s_ml[warp][g] = make_float2(m, l);
    asm volatile("bar.sync 1, %0;" ::"n"(kQ4Warps * 32) : "memory");
    float M = -INFINITY, L = 0.f;
    if (works) {
      for (int w = 0; w < per_set; ++w) M = fmaxf(M, s_ml[hs * per_set + w][g].x);
      for (int w = 0; w < per_set; ++w) {
        const float2 ml = s_ml[hs * per_set + w][g];
        L += ml.y * part_weight<kAttend>(ml.x, M);
      }
      const int64_t slot = cta + b;
      if (j == 0 && t == 0 && g < nh) a.part_ml[slot * a.H + head0 + g] = make_float2(M, L);
    }
    if constexpr (kAttend) {
      if (works) {
        const float fac = part_weight<true>(st.m, M);
        float* mg = merge + ((size_t)warp * 8 + g) * D;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            float4 lo, hi;
            lo.x = (st.o[nb][0][q] + st.o[nb][0][q + 2]) * fac;
            lo.y = (st.o[nb][1][q] + st.o[nb][1][q + 2]) * fac;
            lo.z = (st.o[nb][2][q] + st.o[nb][2][q + 2]) * fac;
            lo.w = (st.o[nb][3][q] + st.o[nb][3][q + 2]) * fac;
            hi.x = (st.o[nb][4][q] + st.o[nb][4][q + 2]) * fac;
            hi.y = (st.o[nb][5][q] + st.o[nb][5][q + 2]) * fac;
            hi.z = (st.o[nb][6][q] + st.o[nb][6][q + 2]) * fac;
            hi.w = (st.o[nb][7][q] + st.o[nb][7][q + 2]) * fac;
            float4* dst = reinterpret_cast<float4*>(mg + nb * 64 + 8 * (2 * t + q));
            dst[0] = lo;
            dst[1] = hi;
          }
      }
      asm volatile("bar.sync 1, %0;" ::"n"(kQ4Warps * 32) : "memory");
      if (works) {
        float* po = a.part_o + ((int64_t)(cta + b) * a.H + head0) * D;
        const float* mg = merge + (size_t)hs * per_set * 8 * D;
        for (int i = j * 32 + lane; i < nh * D; i += per_set * 32) {
          float acc = 0.f;
          for (int w = 0; w < per_set; ++w) acc += mg[(size_t)w * 8 * D + i];
          po[i] = acc;
        }
      }
    }
    asm volatile("bar.sync 1, %0;" ::"n"(kQ4Warps * 32) : "memory");   // joined: the areas may be reused
  }
}

// The parts of a sequence's scan that exist: slots [first, first + count).
__device__ __forceinline__ void scan_slots(const Q4Args& a, int b, int lane, int64_t& first, int& count) {
  int64_t total, before;
  count_pages(a, b, lane, total, before);
  const int np = seq_pages(a, b);
  count = 0;
  first = 0;
  if (np == 0) return;
  const int nc = live_ctas(total, a.ctas);
  const int c0 = (int)(((before + 1) * nc - 1) / total), c1 = (int)(((before + np) * nc - 1) / total);
  first = c0 + b;
  count = c1 - c0 + 1;
}

// Joins the parts of (head, sequence) in slot order. splits > 0: the gather's parts, splits per
// sequence; otherwise the scan's.
constexpr int kMaxParts = 512;   // of one sequence
template <int D>
__global__ void __launch_bounds__(1024) q4_merge_kernel(const __grid_constant__ Q4Args a, int splits, float* out,
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
    scan_slots(a, b, tid & 31, first, count);
  }
  for (int i = tid; i < count; i += blockDim.x) s_ml[i] = __ldcg(a.part_ml + (first + i) * a.H + h);
  __syncthreads();
  float M = -INFINITY;
  for (int i = 0; i < count; ++i) M = fmaxf(M, s_ml[i].x);
  float o = 0.f;
  const float* po = a.part_o + (first * a.H + h) * D + e;
#pragma unroll 4
  for (int i = row; i < count; i += ROWS)
    o = fmaf(part_weight<true>(s_ml[i].x, M), __ldcg(po + (size_t)i * a.H * D), o);
  s_o[row][e] = o;
  __syncthreads();
  if (row != 0) return;
  float O = 0.f, L = 0.f;
#pragma unroll
  for (int i = 0; i < ROWS; ++i) O += s_o[i][e];
  for (int i = 0; i < count; ++i) L = fmaf(part_weight<true>(s_ml[i].x, M), s_ml[i].y, L);
  const bool some = L != 0.f;   // true for NaN: a NaN among the rows is not an empty sequence
  out[((size_t)b * a.H + h) * D + e] = some ? O / L : 0.f;
  if (lse && e == 0) lse[(size_t)b * a.H + h] = some ? (M + log2f(L)) * 0.6931471805599453f : -INFINITY;
}

// (max, 1 / sum) of each head over the whole sequence, from the scan's parts.
__global__ void q4_stats_kernel(const __grid_constant__ Q4Args a, float2* stats) {
  const int b = blockIdx.x;
  int64_t first;
  int count;
  scan_slots(a, b, threadIdx.x & 31, first, count);
  for (int h = threadIdx.x; h < a.H; h += blockDim.x) {
    const float2* ml = a.part_ml + first * a.H + h;
    float M = -INFINITY;
    for (int i = 0; i < count; ++i) M = fmaxf(M, ml[(size_t)i * a.H].x);
    KahanF z;
    for (int i = 0; i < count; ++i) {
      const float2 x = ml[(size_t)i * a.H];
      z.add(x.y * part_weight<false>(x.x, M));
    }
    stats[(size_t)b * a.H + h] = make_float2(M, 1.f / (z.s - z.c));
  }
}

struct Q4GatherArgs {
  const int32_t* idx;     // [B][idx_stride]
  int64_t idx_stride;
  const int32_t* count;   // [B]
  int splits;
};

// CTA (split, head set, sequence): a contiguous part of the index list, 16 tokens per warp and step.
template <int NB>
__global__ void __launch_bounds__(kGatherWarps * 32) gather_kernel(const __grid_constant__ Q4Args a,
                                                                   const __grid_constant__ Q4GatherArgs ga) {
  constexpr int D = NB * 64;
  constexpr int BLK = q4_block_bytes(D), CODES = q4_code_bytes(D);
  __shared__ __align__(16) float merge[kGatherWarps][8][D];
  __shared__ float2 s_ml[kGatherWarps][8];
  const int split = blockIdx.x, set = blockIdx.y, b = blockIdx.z;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int kv = set / a.sets_per_kv, head0 = kv * a.G + (set % a.sets_per_kv) * 8;
  const int nh = min(8, a.G - (set % a.sets_per_kv) * 8);
  const int cnt = (int)min((int64_t)max(ga.count[b], 0), ga.idx_stride);
  const int units = (cnt + 15) / 16;
  const int u0 = (int)((int64_t)units * split / ga.splits), u1 = (int)((int64_t)units * (split + 1) / ga.splits);
  const int32_t* ib = ga.idx + (size_t)b * ga.idx_stride;
  const int32_t* pt = a.page_table + (size_t)b * a.pt_stride;

  Q4Query<NB> f;
  q4_load_query<NB>(f, a.q + ((size_t)b * a.H + head0 + (g < nh ? g : 0)) * D, g < nh, t);
  const float mul = a.scale * f.inv * 1.4426950408889634f;
  Q4State<NB> st;
  st.reset();
  for (int u = u0 + warp; u < u1; u += kGatherWarps) {
    // lane i holds list entry i (of 16) as its block offset and slot; -1 where there is none
    int64_t mine = -1;
    const int at = u * 16 + (lane & 15);
    if (at < cnt) {
      const int tk = ib[at];
      int page = -1;
      if (tk >= 0 && tk < a.max_tokens) page = pt[tk / kPage];
      if (page >= 0 && (int64_t)page < a.num_pages)
        mine = ((int64_t)page * a.HKV + kv) * kPage + tk % kPage;      // row number in the pool
      else
        set_error(a.status, TS_ERR_PAGE_OOB);
    }
    uint2 kw[2][NB];
    float ks[NB][4], vs[NB][4], x[4];
    uint32_t vw[4][NB];
    int64_t own[4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int64_t row = __shfl_sync(kFull, mine, 8 * i + g);
      const unsigned char* kb = a.k_pool + (row < 0 ? 0 : (row / kPage) * BLK + (row % kPage) * 32);
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
        kw[i][nb] = row < 0 ? make_uint2(0u, 0u) : *reinterpret_cast<const uint2*>(kb + nb * 512 + t * 8);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      own[i] = __shfl_sync(kFull, mine, 8 * (i >> 1) + 2 * t + (i & 1));
      const size_t blk = own[i] < 0 ? 0 : (size_t)(own[i] / kPage) * BLK;
      const int slot = own[i] < 0 ? 0 : (int)(own[i] % kPage);
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        const size_t so = blk + CODES + nb * 32 + slot * 2;
        ks[nb][i] = own[i] < 0 ? 0.f : bf16_bits_f(*reinterpret_cast<const uint16_t*>(a.k_pool + so));
        vs[nb][i] = own[i] < 0 ? 0.f : bf16_bits_f(*reinterpret_cast<const uint16_t*>(a.v_pool + so));
        vw[i][nb] = own[i] < 0 ? 0u : *reinterpret_cast<const uint32_t*>(a.v_pool + blk + nb * 512 + slot * 32 + g * 4);
      }
    }
    q4_scores<NB>(f, kw, ks, x);
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = own[i] < 0 ? -INFINITY : x[i] * mul;
    q4_accumulate<NB>(st, x, vw, vs);
  }
  float l = st.l;
  l += __shfl_xor_sync(kFull, l, 1);
  l += __shfl_xor_sync(kFull, l, 2);
  if (t == 0) s_ml[warp][g] = make_float2(st.m, l);
#pragma unroll
  for (int nb = 0; nb < NB; ++nb)
#pragma unroll
    for (int q = 0; q < 2; ++q)
#pragma unroll
      for (int jj = 0; jj < 8; ++jj)
        merge[warp][g][nb * 64 + 8 * (2 * t + q) + jj] = st.o[nb][jj][q] + st.o[nb][jj][q + 2];
  __syncthreads();
  const int64_t slot = (int64_t)b * ga.splits + split;
  for (int i = tid; i < nh * D; i += kGatherWarps * 32) {
    const int hg = i / D;
    float M = -INFINITY, L = 0.f, O = 0.f;
#pragma unroll
    for (int w = 0; w < kGatherWarps; ++w) M = fmaxf(M, s_ml[w][hg].x);
#pragma unroll
    for (int w = 0; w < kGatherWarps; ++w) {
      const float wt = part_weight<true>(s_ml[w][hg].x, M);
      L = fmaf(wt, s_ml[w][hg].y, L);
      O = fmaf(wt, merge[w][hg][i % D], O);
    }
    a.part_o[(slot * a.H + head0) * D + i] = O;
    if (i % D == 0) a.part_ml[slot * a.H + head0 + hg] = make_float2(M, L);
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
  a.sets_per_kv = (a.G + 7) / 8;
  a.n_groups = (a.HKV * a.sets_per_kv + kQ4Sets - 1) / kQ4Sets;
  a.ctas = ctx->num_sms / a.n_groups;
  a.ctas = std::max(1, std::min(a.ctas, kMaxParts));
  a.scale = scale;
  a.logits = ctx->logits;
  a.part_o = ctx->q4_part_o;
  a.part_ml = ctx->q4_part_ml;
  a.status = ctx->status;
  return a;
}

template <int NB>
ts_status run_attend(ts_ctx* ctx, const Q4Args& a, float* out, float* lse, cudaStream_t s) {
  constexpr size_t smem = kQ4RingBytes + (size_t)kQ4Warps * 8 * NB * 64 * sizeof(float);
  if (!ensure_smem<scan_kernel<NB, true>>(smem, ctx->device)) return TS_ERR_CUDA;
  ProfScope ps(ctx, TS_PROF_ATTEND, s);
  ctx->kernels += 2;
  scan_kernel<NB, true><<<a.ctas * a.n_groups, kQ4Threads, smem, s>>>(a);
  q4_merge_kernel<NB * 64><<<dim3(a.H, a.B), 1024, 0, s>>>(a, 0, out, lse);
  return cuda_status(cudaGetLastError());
}

template <int NB>
ts_status run_scan(ts_ctx* ctx, const Q4Args& a, cudaStream_t s) {
  if (!ensure_smem<scan_kernel<NB, false>>((size_t)kQ4RingBytes, ctx->device)) return TS_ERR_CUDA;
  ProfScope ps(ctx, TS_PROF_SCORE, s);
  ctx->kernels += 2;
  scan_kernel<NB, false><<<a.ctas * a.n_groups, kQ4Threads, kQ4RingBytes, s>>>(a);
  q4_stats_kernel<<<a.B, 256, 0, s>>>(a, ctx->stats);
  return cuda_status(cudaGetLastError());
}

template <int NB>
ts_status run_gather(ts_ctx* ctx, const Q4Args& a, const Q4GatherArgs& ga, float* out, float* lse, cudaStream_t s) {
  ProfScope ps(ctx, TS_PROF_ATTEND, s);
  ctx->kernels += 2;
  gather_kernel<NB><<<dim3(ga.splits, a.HKV * a.sets_per_kv, a.B), kGatherWarps * 32, 0, s>>>(a, ga);
  q4_merge_kernel<NB * 64><<<dim3(a.H, a.B), 1024, 0, s>>>(a, ga.splits, out, lse);
  return cuda_status(cudaGetLastError());
}

}  // namespace

bool q4_supported(const ts_config& c) {
  return c.kv_dtype == TS_KV_Q4 && c.page_size == kPage && (c.head_dim == 64 || c.head_dim == 128) &&
         c.n_q_heads / c.n_kv_heads <= 16;
}

// Parts of any call: a scan has at most one per CTA and one more per sequence, a gather at most
// 2 num_sms + B (splits below rounds up once per sequence).
int64_t q4_part_slots(const ts_config& c, int num_sms) { return 2 * (int64_t)num_sms + c.max_batch; }

int q4_gather_splits(const ts_config& c, int num_sms, int B) {
  const int sets = c.n_kv_heads * ((c.n_q_heads / c.n_kv_heads + 7) / 8);
  const int s = (2 * num_sms + sets * B - 1) / (sets * B);
  return s < 1 ? 1 : (s > kAttnMaxSplits ? kAttnMaxSplits : s);
}

ts_status launch_attend_q4(ts_ctx* ctx, const AttendCall& c, const int32_t* seq_lens, cudaStream_t s) {
  Q4Args a = make_args(ctx, c.q, c.k_pool, c.v_pool, c.page_table, seq_lens, c.B, c.scale);
  if (!c.idx) return ctx->cfg.head_dim == 64 ? run_attend<1>(ctx, a, c.out, c.lse, s) : run_attend<2>(ctx, a, c.out, c.lse, s);
  Q4GatherArgs ga{c.idx, c.idx_stride, c.count, q4_gather_splits(ctx->cfg, ctx->num_sms, c.B)};
  return ctx->cfg.head_dim == 64 ? run_gather<1>(ctx, a, ga, c.out, c.lse, s)
                                 : run_gather<2>(ctx, a, ga, c.out, c.lse, s);
}

ts_status launch_score_q4(ts_ctx* ctx, const ScoreCall& c, cudaStream_t s) {
  Q4Args a = make_args(ctx, c.q, c.k_pool, nullptr, c.page_table, c.seq_lens, c.B, c.scale);
  a.skip = c.skip;
  return ctx->cfg.head_dim == 64 ? run_scan<1>(ctx, a, s) : run_scan<2>(ctx, a, s);
}

}  // namespace ts
