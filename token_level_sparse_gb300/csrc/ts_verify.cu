// Which drafted tokens of a tree the target keeps, and the token behind them (ts_verify_tree).
//
// At a node with target distribution p and draft distribution q the children are tried in order. A child x is taken
// where u q(x) Z < r(x) W; else, r being the residual, its mass moves on:
//
//   r_0 = p, Z_0 = 1, W_0 = 1      r_k = max(r_(k-1) - Z_(k-1) q / W_(k-1), 0),  Z_k = sum r_k
//
// (W: what is left of the draft's mass, 1 throughout where siblings are drawn independently). Z_k is not divided out, so
// the residual is r_k = max(p - c_k q, 0) with c_k = c_(k-1) + Z_(k-1) / W_(k-1): one number per node, and every
// element is formed from p and q alone. With no child left a token is drawn from r: the first whose running sum passes
// u Z. Drafts without probabilities stand for a q of 1 at each child: refused ones are taken out of p.
//
// What it reads is small (the last node's rows of p and q, and once more for every refused child that has a sibling behind it),
// and a chain of dependent steps, so it is bound by latency. A cluster of CTAs takes a sequence, a slice of the
// vocabulary each. The first warp of the first CTA walks: p(x) and q(x) of all nodes are fetched beforehand, side by side, so
// its steps run in shared memory, and tells the others what to sum (a message in their shared memory, a cluster
// barrier on either side). Nobody else decides anything, so all of them always agree on the next barrier.
//
// Sums decide whole numbers, so they are held in pairs of floats (p - c q exactly, c in two floats), warps and CTAs in fp64,
// all in a fixed order: off by 2^-44 of the sum as a rule, by n^2 2^-49 < 2^-33 at most, n <= 256 elements to a lane, and by 2^-45
// of the sums of p and c q, which may nearly cancel. FP64 throughout would be the slower pipe by far (sixteen warps that
// scanned 128 sums in fp64 took 8 us). Entries that are NaN or negative count as zero.
//
// Measured: a chain of 6 over 32,001 tokens 13 us (1 for the nodes, 2 for the walk, 1.7 for a sweep, 2 to find the part and 2 the
// token, cluster barriers of 0.5); 32 trees of up to 64 nodes over 128,256 tokens 53 us, as long as the one with most
// refusals takes, 6 us for each sweep of its rows.
#include <cooperative_groups.h>
#include <math_constants.h>

#include "ts_common.cuh"

namespace ts {
namespace {

namespace cg = cooperative_groups;

constexpr int kVfThreads = 512;
constexpr int kVfWarps = kVfThreads / 32;
constexpr int kVfCluster = 8;          // CTAs of a sequence, at most (the portable size)
constexpr int kVfSlice = 1 << 17;      // vocabulary of a CTA, at most

struct VerifyArgs {
  const int32_t* tokens;
  const int32_t* parents;
  const int32_t* cu;
  int B, total, V;
  const float* target;
  int64_t target_stride;
  const float* draft;                  // or null
  int64_t draft_stride;
  const float* u;
  const float* u_next;
  int distinct;
  int32_t* path;
  int64_t path_stride;
  int32_t* count;
  int32_t* next;
  int* status;
};

enum { kVfSum = 0, kVfDraw = 1, kVfEnd = 2 };

struct Order {                         // what the walk asks of every CTA
  int what;
  int node;                            // the node whose rows are meant (in its sequence)
  int masked;                          // drafts without probabilities: its children are taken out
  double c;
};

// max(p - c q, 0) as a pair of floats; entries that are NaN or negative count as zero. The product and the differences are
// rounded each by itself: a multiply-add in the place of one would leave e out or in twice, up to 2^-24 of c q.
__device__ __forceinline__ void residual(float p, float q, float ch, float cl, float& hi, float& lo) {
  q = fmaxf(q, 0.f);
  const float h = __fmul_rn(ch, q), e = fmaf(ch, q, -h);             // c_hi q exactly
  const float s = __fsub_rn(p, h), t = __fsub_rn(__fsub_rn(p, s), h);   // p - h exactly, where it is not negative (so p is the larger)
  const float l = fmaf(-cl, q, t - e);
  const bool some = s + l > 0.f;
  hi = some ? s : 0.f;
  lo = some ? l : 0.f;
}

// A sum as a pair of floats, s + c, to which pairs are added (the part of an addition that s does not hold goes to c).
struct PairSum {
  float s = 0.f, c = 0.f;
  __device__ __forceinline__ void add(float hi, float lo) {
    float t, e;
    two_sum(s, hi, t, e);              // (one addition on the way from one s to the next)
    s = t;
    c += e + lo;
  }
  __device__ __forceinline__ double value() const { return (double)s + (double)c; }
};

// Vocabulary of a warp: whole 512-byte pieces, so that aligned rows are read 16 bytes a lane.
__host__ __device__ inline int warp_part(int V, int ctas) {
  const int warps = ctas * kVfWarps;
  return ((V + warps - 1) / warps + 127) / 128 * 128;
}

__global__ void __launch_bounds__(kVfThreads, 2) verify_kernel(const __grid_constant__ VerifyArgs a) {
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank(), ctas = (int)cluster.num_blocks();
  cluster.barrier_arrive();            // shared memory of another CTA may be written once that CTA runs (waited for below)
  const int b = blockIdx.x / ctas, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  extern __shared__ unsigned s_gone[];                          // bit per token of the slice (drafts without probabilities)
  __shared__ int s_parent[kMaxTree], s_token[kMaxTree];
  __shared__ float s_u[kMaxTree], s_p[kMaxTree], s_q[kMaxTree];
  __shared__ Order s_order;
  __shared__ float2 s_part[kVfCluster * kVfWarps];              // (of the first CTA) sums by CTA and warp, as pairs
  __shared__ double s_before, s_t;                              // the draw: what lies before the part that holds the token,
  __shared__ int s_from;                                        // the number that is passed, and the part
  __shared__ int s_found;

  const int first = a.cu[b], end = a.cu[b + 1];
  const bool fine = first >= 0 && end >= first && end <= a.total && end - first <= kMaxTree && (b != 0 || first == 0);
  const int T = fine ? end - first : 0;
  if (rank == 0 && tid == 0 && !fine) set_error(a.status, TS_ERR_SEQ_LEN);

  // the slice, and this warp's part of it
  const int part = warp_part(a.V, ctas), slice = kVfWarps * part, v0 = min(a.V, rank * slice), v1 = min(a.V, v0 + slice);
  const int w0 = min(v1, v0 + warp * part), w1 = min(v1, w0 + part);

  if (rank == 0) {
    for (int i = tid; i < T; i += kVfThreads) {
      const int par = i ? a.parents[first + i] : -1, tok = i ? a.tokens[first + i] : -1;
      const bool ok = i == 0 || (par >= 0 && par < i && tok >= 0 && tok < a.V);
      if (!ok) set_error(a.status, TS_ERR_INVALID_ARG);
      const bool use = ok && i > 0;
      s_parent[i] = use ? par : -2;
      s_token[i] = use ? tok : -1;
      s_u[i] = use ? a.u[first + i] : 0.f;
      s_p[i] = use ? a.target[(int64_t)(first + par) * a.target_stride + tok] : 0.f;
      s_q[i] = use && a.draft ? a.draft[(int64_t)(first + par) * a.draft_stride + tok] : 0.f;
    }
    __syncthreads();
  }

  // state of the walk (first warp of the first CTA; the same in every lane)
  int cur = 0, at = 1, kept = T > 0 ? 1 : 0;
  double c = 0., Z = 1., W = 1.;
  bool stale = false;                  // Z is that of an earlier c
  int draws = 0;
  if (rank == 0 && warp == 0 && lane == 0 && T > 0) {
    if (a.path_stride > 0) a.path[(int64_t)b * a.path_stride] = 0;
  }
  int token = -1;

  cluster.barrier_wait(cg::cluster_group::arrival_token());       // (the nodes were fetched meanwhile)
  for (;;) {
    if (rank == 0 && warp == 0) {
      Order o{kVfEnd, cur, 0, 0.};
      if (T > 0) {
        o.what = kVfDraw;
        // children of cur from node `at` on
        while (at < T) {
          const int i = at + lane;
          const unsigned m = __ballot_sync(kFull, i < T && s_parent[i] == cur);
          if (!m) {
            at += 32;
            continue;
          }
          const int x = at + __ffs(m) - 1;
          if (a.draft && stale) {      // its test needs the sum of the residual
            o.what = kVfSum;
            at = x;
            break;
          }
          at = x + 1;
          const double u = s_u[x];
          bool yes;
          double px = fmaxf(s_p[x], 0.f);
          if (a.draft) {
            const double qx = fmaxf(s_q[x], 0.f);
            const double r = fmax(px - c * qx, 0.);
            yes = W > 0. && u * qx * Z < r * W;
            if (!yes) {
              if (W > 0.) c += Z / W;
              if (a.distinct) W -= qx;
              stale = true;
            }
          } else {
            // a token that an earlier child had is gone
            bool dup = false;
            for (int j = cur + 1 + lane; j < x; j += 32) dup |= s_parent[j] == cur && s_token[j] == s_token[x];
            if (__any_sync(kFull, dup)) px = 0.;
            yes = u * Z < px;
            if (!yes) Z -= px;
          }
          if (yes) {
            if (lane == 0 && kept < a.path_stride) a.path[(int64_t)b * a.path_stride + kept] = x;
            ++kept;
            cur = x;
            c = 0.;
            Z = W = 1.;
            stale = false;
          }
        }
        o.node = cur;
        o.masked = a.draft == nullptr && draws == 0;
        o.c = draws == 0 ? c : 0.;     // nothing left of the residual: the second draw is from p itself
      }
      if (lane < ctas) *cluster.map_shared_rank(&s_order, lane) = o;
    }
    cluster.sync();
    const Order o = s_order;
    if (o.what == kVfEnd) break;
    // ---- sums of this warp's part
    const float* p = a.target + (int64_t)(first + o.node) * a.target_stride;
    const bool with_q = a.draft != nullptr && o.c != 0.;
    const float* q = with_q ? a.draft + (int64_t)(first + o.node) * a.draft_stride : p;
    const float ch = with_q ? (float)o.c : 0.f, cl = with_q ? (float)(o.c - (double)ch) : 0.f;
    if (o.masked) {
      for (int i = tid; i < (slice + 31) / 32; i += kVfThreads) s_gone[i] = 0u;
      __syncthreads();
      for (int i = o.node + 1 + tid; i < T; i += kVfThreads) {
        const int tok = a.tokens[first + i];
        if (a.parents[first + i] == o.node && tok >= v0 && tok < v1) atomicOr(&s_gone[(tok - v0) >> 5], 1u << ((tok - v0) & 31));
      }
      __syncthreads();
    }
    auto entry = [&](int i, float pv, float qv, float& hi, float& lo) {
      residual(pv, qv, ch, cl, hi, lo);
      if (o.masked && (s_gone[(i - v0) >> 5] >> ((i - v0) & 31) & 1u)) hi = lo = 0.f;
    };
    PairSum held_here;
    auto add = [&](int i, float pv, float qv) {
      float x, y;
      entry(i, pv, qv, x, y);
      held_here.add(x, y);
    };
    const bool aligned = ((reinterpret_cast<uintptr_t>(p) | reinterpret_cast<uintptr_t>(q)) & 15) == 0;
    if (aligned) {
      constexpr int UN = 4;            // 16-byte loads of either row under way
      for (int i0 = w0 + 4 * lane; i0 < w1; i0 += 128 * UN) {
        float4 pv[UN], qv[UN];
#pragma unroll
        for (int k = 0; k < UN; ++k) {
          const int i = i0 + 128 * k;
          pv[k] = qv[k] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (i + 3 < w1) {
            pv[k] = __ldg(reinterpret_cast<const float4*>(p + i));
            if (with_q) qv[k] = __ldg(reinterpret_cast<const float4*>(q + i));
          }
        }
#pragma unroll
        for (int k = 0; k < UN; ++k) {
          const int i = i0 + 128 * k;
          if (i + 3 < w1) {
            add(i, pv[k].x, qv[k].x);
            add(i + 1, pv[k].y, qv[k].y);
            add(i + 2, pv[k].z, qv[k].z);
            add(i + 3, pv[k].w, qv[k].w);
          } else {
            for (int l = i; l < w1; ++l) add(l, p[l], with_q ? q[l] : 0.f);   // (the vocabulary's last elements)
          }
        }
      }
    } else {
      constexpr int UN = 8;
      for (int i0 = w0 + lane; i0 < w1; i0 += 32 * UN) {
        float pv[UN], qv[UN];
#pragma unroll
        for (int k = 0; k < UN; ++k) {
          const int i = i0 + 32 * k;
          pv[k] = i < w1 ? __ldg(p + i) : 0.f;
          qv[k] = i < w1 && with_q ? __ldg(q + i) : 0.f;
        }
#pragma unroll
        for (int k = 0; k < UN; ++k)
          if (i0 + 32 * k < w1) add(i0 + 32 * k, pv[k], qv[k]);
      }
    }
    // (pairs of floats down to one per warp: sixteen warps' sums in fp64 would queue for its pipe for microseconds)
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1)
      held_here.add(__shfl_xor_sync(kFull, held_here.s, d), __shfl_xor_sync(kFull, held_here.c, d));
    if (lane == 0) *cluster.map_shared_rank(&s_part[rank * kVfWarps + warp], 0) = make_float2(held_here.s, held_here.c);
    if (tid == 0) s_found = -1;
    cluster.sync();
    if (o.what == kVfSum) {
      if (rank == 0 && warp == 0) {
        double s = 0.;
        for (int k = lane; k < ctas * kVfWarps; k += 32) s += (double)s_part[k].x + (double)s_part[k].y;
#pragma unroll
        for (int d = 16; d >= 1; d >>= 1) s += __shfl_xor_sync(kFull, s, d);
        Z = s;
        stale = false;
      }
      continue;
    }
    // ---- the draw: a warp of every CTA finds from all sums the part that holds the token
    if (warp == 0) {
      const float2* parts = cluster.map_shared_rank(&s_part[0], 0);
      const int n = ctas * kVfWarps;
      // running sums over the parts: a lane takes PL neighbours
      constexpr int PL = kVfCluster * kVfWarps / 32;
      float2 pair[PL];
#pragma unroll
      for (int k = 0; k < PL; ++k) pair[k] = PL * lane + k < n ? parts[PL * lane + k] : make_float2(0.f, 0.f);
      double held[PL], lane_sum = 0.;
#pragma unroll
      for (int k = 0; k < PL; ++k) {
        held[k] = (double)pair[k].x + (double)pair[k].y;
        lane_sum += held[k];
      }
      double run = lane_sum;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const double o2 = __shfl_up_sync(kFull, run, d);
        if (lane >= d) run += o2;
      }
      const double all = __shfl_sync(kFull, run, 31), t = (double)a.u_next[b] * all;
      // the first part that holds something and whose running sum passes t; where rounding leaves none, the last that does
      double at_part = run - lane_sum;
      int mine_over = -1, mine_some = -1;
#pragma unroll
      for (int k = 0; k < PL; ++k) {
        if (held[k] > 0.) {
          mine_some = k;
          if (mine_over < 0 && at_part + held[k] > t) mine_over = k;
        }
        if (mine_over < 0 && k + 1 < PL) at_part += held[k];
      }
      const unsigned over = __ballot_sync(kFull, mine_over >= 0), some = __ballot_sync(kFull, mine_some >= 0);
      const int l = over ? __ffs(over) - 1 : 31 - __clz(some);
      if (some && lane == l) {
        s_from = PL * l + (over ? mine_over : mine_some);
        s_before = at_part;
        s_t = over ? t : CUDART_INF;                              // (not passed: the part's last element that holds something)
      }
      if (!some && lane == 0) s_from = -1;
    }
    __syncthreads();
    if (s_from == rank * kVfWarps + warp) {
      const double before = s_before, t = s_t;
      // a lane takes neighbouring elements: its sum, the sums of the lanes before it
      const int len = part / 32, e0 = min(w1, w0 + lane * len), e1 = min(w1, e0 + len);   // (a multiple of 4)
      PairSum piece;
      bool any = false;
      constexpr int UN = 8;
      for (int i0 = e0; i0 < e1; i0 += UN) {
        __align__(16) float pv[UN], qv[UN];
#pragma unroll
        for (int k = 0; k < UN; k += 4) {
          if (aligned && i0 + k + 3 < e1) {
            *reinterpret_cast<float4*>(pv + k) = *reinterpret_cast<const float4*>(p + i0 + k);
            if (with_q) *reinterpret_cast<float4*>(qv + k) = *reinterpret_cast<const float4*>(q + i0 + k);
          } else {
#pragma unroll
            for (int l = k; l < k + 4; ++l) {
              pv[l] = i0 + l < e1 ? p[i0 + l] : 0.f;
              qv[l] = i0 + l < e1 && with_q ? q[i0 + l] : 0.f;
            }
          }
        }
#pragma unroll
        for (int k = 0; k < UN; ++k) {
          if (!with_q) qv[k] = 0.f;
          if (i0 + k >= e1) continue;
          float x, y;
          entry(i0 + k, pv[k], qv[k], x, y);
          piece.add(x, y);
          any |= x + y > 0.f;
        }
      }
      const double sum = piece.value();
      double run = sum;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const double o2 = __shfl_up_sync(kFull, run, d);
        if (lane >= d) run += o2;
      }
      const unsigned over = __ballot_sync(kFull, any && before + run > t);
      const unsigned some = __ballot_sync(kFull, any);
      if (some) {
        // then the whole warp goes through the elements of one of them, 32 at a time
        const int owner = over ? __ffs(over) - 1 : 31 - __clz(some);
        const int f0 = __shfl_sync(kFull, e0, owner), f1 = __shfl_sync(kFull, e1, owner);
        double acc = __shfl_sync(kFull, before + (run - sum), owner);
        int pick = -1;
        for (int i0 = f0; i0 < f1; i0 += 32) {
          const int i = i0 + lane;
          float x = 0.f, y = 0.f;
          if (i < f1) entry(i, p[i], with_q ? q[i] : 0.f, x, y);
          const double v = (double)x + (double)y;
          double upto = v;
#pragma unroll
          for (int d = 1; d < 32; d <<= 1) {
            const double o2 = __shfl_up_sync(kFull, upto, d);
            if (lane >= d) upto += o2;
          }
          const unsigned held = __ballot_sync(kFull, v > 0.), passed1 = __ballot_sync(kFull, v > 0. && acc + upto > t);
          if (held) pick = i0 + (passed1 ? __ffs(passed1) - 1 : 31 - __clz(held));
          if (passed1) break;
          acc += __shfl_sync(kFull, upto, 31);
        }
        if (lane < ctas) *cluster.map_shared_rank(&s_found, lane) = pick;
      }
    }
    cluster.sync();
    ++draws;
    token = s_found;
    if (token >= 0 || draws == 2) break;
  }
  if (rank == 0) {
    if (warp == 0 && lane == 0) {
      a.count[b] = kept;
      a.next[b] = token;
      if (kept > a.path_stride) set_error(a.status, TS_ERR_CAPACITY);
      s_found = kept;
    }
    __syncthreads();
    for (int64_t i = s_found + tid; i < a.path_stride; i += kVfThreads) a.path[(int64_t)b * a.path_stride + i] = -1;
  }
}

}  // namespace

ts_status launch_verify(ts_ctx* ctx, const VerifyCall& c, cudaStream_t s) {
  VerifyArgs a{c.tokens, c.parents, c.cu_rows, c.B, c.total, c.vocab, c.target, c.target_stride, c.draft, c.draft_stride,
               c.u, c.u_next, c.distinct, c.path, c.path_stride, c.count, c.next, ctx->status};
  int ctas = 1;
  while (ctas < kVfCluster && (c.vocab > kVfSlice * ctas || c.vocab >= 2048 * ctas)) ctas *= 2;
  const size_t smem = c.draft ? 0 : (size_t)kVfWarps * warp_part(c.vocab, ctas) / 8;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)ctas;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3((unsigned)(c.B * ctas));
  lc.blockDim = dim3(kVfThreads);
  lc.dynamicSmemBytes = smem;
  lc.stream = s;
  lc.attrs = attr;
  lc.numAttrs = 1;
  ctx->kernels += 1;
  return cuda_status(cudaLaunchKernelEx(&lc, verify_kernel, a));
}

}  // namespace ts
