// Losses over the head's per-token cross-entropies ce[t] = -log p(token t), and
// their gradients with respect to ce:
//
// Policy loss (clipped ratio with a KL term to a reference).  Per counted token
//   D = ce_old - ce,  r = exp(D),  d = ce - ce_ref,
//   l = max(-A r, -A clip(r, 1 - lo, 1 + hi)) + k (exp(d) - 1 - d),
//   dl/dce = A r [the first term is not clipped] + k (exp(d) - 1),
// weighted 1 / tokens, 1 / (sequences * tokens of the sequence) or 1.
//
// Preference loss.  Sequences 0..N-1 are chosen, N..2N-1 rejected; with
// s = sum over a sequence's counted tokens of (ce_ref - ce) (or their mean) and
// D = s_chosen - s_rejected,
//   sigmoid  l = (1 - e) log(1 + exp(-h)) + e log(1 + exp(h)),  h = beta D - margin
//   hinge    l = max(0, 1 - h)
//   squared  l = (D - 1 / (2 beta))^2
// averaged over the pairs; every counted token of a sequence gets the slope.
//
// One launch does the whole call: the phases (counts and sums per sequence;
// per-pair or per-sequence factors; gradients; the loss) meet at a barrier of
// all its blocks, so there is no counter to clear and no second launch: one
// block up to kOneBlock tokens, one cluster of up to 16 with the cluster's
// hardware barrier up to kOneCluster, above that a cooperative grid of up to
// one block per SM.  Each warp owns a contiguous run of tokens, cut at sequence
// boundaries; the piece of a sequence in a later warp's run goes to that warp's
// slot and the pieces are added in run order, so results do not depend on
// timing.  What bounds it: launch, barrier and load latency; at 10^6 tokens the
// fp64 arithmetic is about a third.
//
// All sums, log-ratios and exponentials are fp64: a log-ratio decides on which
// side of a clipping border a token lies, exp(d) - 1 - d is of second order in
// d, and a loss of normalised advantages is a small difference of large sums.
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "device.cuh"
#include "handle.h"

namespace cg = cooperative_groups;

namespace archead {

namespace {

constexpr int kLossThreads = 1024, kLossWarps = kLossThreads / 32;
constexpr int kLossMaxBlocks = 160;   // of the cooperative grid (one per SM, 148 here)
constexpr int kMaxUnits = kLossWarps * kLossMaxBlocks;
constexpr int kGroup = 128;           // tokens of a warp iteration: four consecutive ones per lane
constexpr int kOneBlock = kLossWarps * kGroup, kOneCluster = 16 * kOneBlock;

struct TokenArgs {
  const float* ce;
  const float* ce_ref;        // or null
  const uint8_t* mask;        // or null
  const int32_t* cu;          // [S + 1], or null: one sequence of T tokens
  int32_t T, S, unit;         // unit: tokens per warp, 32, 64 or a multiple of kGroup
  int32_t vec;                // every token array is 16-byte (mask: 4-byte) aligned
  float* grad;
  double* seg_sum;            // [S] sum of a sequence's first piece
  double* open_sum;           // [units] sum of the piece a unit begins with
  int32_t* seg_n;             // the same for counted tokens
  int32_t* open_n;
  float* coef;                // [S] gradient of a sequence's tokens (preference loss)
  double* each;               // [S] 1 / counted tokens (policy loss)
  double* part;               // [blocks][4] sums of a block
  int32_t* part_n;            // [blocks][2]
};

struct PolicyArgs {
  TokenArgs a;
  const float* old;
  const float* adv;
  double border_hi, border_lo, clip_hi, clip_lo, kl, scale;   // log borders; 1 + hi, 1 - lo
  int32_t reduction, per_sequence;
  float* loss;
  float* stats;
};

struct PreferenceArgs {
  TokenArgs a;
  double beta, margin, smooth, scale;
  int32_t N, kind, average;
  float* loss;
  float* rewards;             // [2][N]
};

__device__ __forceinline__ int cu_at(const TokenArgs& a, int s) {
  if (a.cu == nullptr) return s == 0 ? 0 : a.T;
  return min(max(__ldg(a.cu + s), 0), a.T);
}

// The last s in [0, S] with cu[s] <= t, -1 if there is none (cu[S] ends the last
// sequence); the same t in every lane, 32 probes a round.
__device__ __forceinline__ int seq_of_warp(const TokenArgs& a, int t, int lane) {
  int lo = 0, hi = a.S;
  for (;;) {
    const int step = (hi - lo + 32) / 32, at = lo + lane * step;
    const int n = __popc(__ballot_sync(0xffffffffu, at <= hi && cu_at(a, min(at, a.S)) <= t));
    if (n == 0) return lo - 1;
    lo += (n - 1) * step;
    if (step == 1) return lo;
    hi = min(hi, lo + step - 1);
  }
}

// The same per lane, from `from` on (whose offset is <= t): doubling steps, then
// halving ones.
__device__ __forceinline__ int seq_from(const TokenArgs& a, int t, int from) {
  if (from < 0) {
    if (cu_at(a, 0) > t) return -1;
    from = 0;
  }
  int step = 1;
  while (from + step <= a.S && cu_at(a, from + step) <= t) {
    from += step;
    step *= 2;
  }
  for (step /= 2; step > 0; step /= 2)
    if (from + step <= a.S && cu_at(a, from + step) <= t) from += step;
  return from;
}

__device__ __forceinline__ void load4(const float* p, int t, int T, bool vec, float (&v)[4]) {
  if (vec && t + 3 < T) {
    const float4 x = *reinterpret_cast<const float4*>(p + t);
    v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = t + i < T ? p[t + i] : 0.f;
  }
}
__device__ __forceinline__ void store4(float* p, int t, int T, bool vec, const float (&v)[4]) {
  if (vec && t + 3 < T) {
    *reinterpret_cast<float4*>(p + t) = make_float4(v[0], v[1], v[2], v[3]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (t + i < T) p[t + i] = v[i];
  }
}
// Bit i: token t + i counts.
__device__ __forceinline__ uint32_t keep4(const TokenArgs& a, int t) {
  uint32_t k = 0;
  if (a.mask == nullptr) {
#pragma unroll
    for (int i = 0; i < 4; ++i) k |= (t + i < a.T ? 1u : 0u) << i;
  } else if (a.vec && t + 3 < a.T) {
    const uchar4 m = *reinterpret_cast<const uchar4*>(a.mask + t);
    k = (m.x ? 1u : 0u) | (m.y ? 2u : 0u) | (m.z ? 4u : 0u) | (m.w ? 8u : 0u);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) k |= (t + i < a.T && a.mask[t + i] ? 1u : 0u) << i;
  }
  return k;
}

__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ int warp_sum(int v) { return __reduce_add_sync(0xffffffffu, v); }

// exp(x), exp(x) - 1 and exp(x) - 1 - x without their cancellation: the argument less
// a multiple n of log 2 (one fused step; the constant is off by up to 2^-54, which
// moves the value by n 2^-54, 2^-44 at |x| = 700), then the Taylor series up to f^10.
// What that leaves out is below 2^-41 of exp(x), 2^-40 of exp(x) - 1 and 2^-37 of
// exp(x) - 1 - x, for |f| <= log(2) / 2.
__device__ __forceinline__ double exp_k3(double x, double& m1, double& k3) {
  double r;
  if (fabs(x) < 700.0) {
    const double n = rint(x * 1.4426950408889634);
    const double f = fma(-n, 0.69314718055994531, x);
    double q = 1.0 / 3628800.0;
    q = fma(q, f, 1.0 / 362880.0);
    q = fma(q, f, 1.0 / 40320.0);
    q = fma(q, f, 1.0 / 5040.0);
    q = fma(q, f, 1.0 / 720.0);
    q = fma(q, f, 1.0 / 120.0);
    q = fma(q, f, 1.0 / 24.0);
    q = fma(q, f, 1.0 / 6.0);
    q = fma(q, f, 0.5);
    q = q * f * f;
    if (n == 0.0) {
      k3 = q;
      m1 = f + q;
      return 1.0 + m1;
    }
    r = (1.0 + (f + q)) * __hiloint2double((1023 + static_cast<int>(n)) << 20, 0);
  } else {
    r = exp(x);   // overflow, underflow, NaN
  }
  m1 = r - 1.0;   // (not k3 + x: of a large -x nothing of it would be left, of an infinite one NaN)
  k3 = x > 700.0 ? m1 : m1 - x;   // (x is less than half an ulp there, and infinity less infinity NaN)
  return r;
}

// Sums and counts of the pieces of sequences in this warp's run of tokens.
// kSum: also the sum of (ce_ref - ce).  A group inside one sequence adds to
// per-lane sums; one with boundaries goes 32 tokens at a time through a
// segmented scan (the same steps however many sequences begin in it).
template <bool kSum>
__device__ void walk_segments(const TokenArgs& a, int unit, int lane) {
  const int u0 = unit * a.unit, u1 = min(u0 + a.unit, a.T);
  if (u0 >= u1) return;
  int s = seq_of_warp(a, u0, lane);   // -1: before the first sequence, S: after the last
  int cs = 0, ce = 0;                 // of s, where it is one
  double sum = 0.0;
  int n = 0;                          // of s so far, per lane
  auto enter = [&]() {
    if (s >= 0 && s < a.S) {
      cs = cu_at(a, s);
      ce = cu_at(a, s + 1);
    }
  };
  auto put = [&](int seq, int begin, double v, int c) {
    if (begin >= u0) {
      if constexpr (kSum) a.seg_sum[seq] = v;
      a.seg_n[seq] = c;
    } else {
      if constexpr (kSum) a.open_sum[unit] = v;
      a.open_n[unit] = c;
    }
  };
  enter();
  for (int g = u0; g < u1; g += kGroup) {
    const int t = g + 4 * lane, g1 = min(g + kGroup, u1);
    if (s >= 0 && s < a.S && cs <= g && ce >= g1) {
      const uint32_t keep = keep4(a, t);
      float x[4], y[4] = {0.f, 0.f, 0.f, 0.f};
      if constexpr (kSum) {
        load4(a.ce, t, a.T, a.vec, x);
        if (a.ce_ref != nullptr) load4(a.ce_ref, t, a.T, a.vec, y);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (t + i < g1 && (keep >> i & 1u)) {
          if constexpr (kSum) sum += static_cast<double>(y[i]) - static_cast<double>(x[i]);
          ++n;
        }
      }
      if (ce > g1) continue;   // (the common case: goes on in the next group or run)
      if constexpr (kSum) sum = warp_sum(sum);
      n = warp_sum(n);
      if (lane == 0) put(s, cs, sum, n);
      sum = 0.0;
      n = 0;
      s = seq_from(a, g1, s);
      enter();
      continue;
    }
    // What s has so far, in every lane.
    double run = kSum ? warp_sum(sum) : 0.0;
    int run_n = warp_sum(n), run_s = s;
    double val[4];
    bool cnt[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {   // all loads of the group first
      const int tt = g + 32 * i + lane;
      cnt[i] = tt < g1 && (a.mask == nullptr || a.mask[tt] != 0);
      val[i] = 0.0;
      if constexpr (kSum)
        if (tt < g1) val[i] = (a.ce_ref != nullptr ? static_cast<double>(a.ce_ref[tt]) : 0.0) - static_cast<double>(a.ce[tt]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int h = g + 32 * i, tt = h + lane;
      if (h >= g1) break;
      int q = -1, qs = 0, qe = 0;
      if (tt < g1) {
        q = seq_from(a, tt, run_s);
        if (q >= a.S) q = -1;
        if (q >= 0) {
          qs = cu_at(a, q);
          qe = cu_at(a, q + 1);
          if (tt >= qe) q = -1;
        }
      }
      const bool counts = q >= 0 && cnt[i];
      double v = counts ? val[i] : 0.0;
      int c = counts ? 1 : 0;
      const int before = __shfl_up_sync(0xffffffffu, q, 1), after = __shfl_down_sync(0xffffffffu, q, 1);
      bool head = lane == 0 || q != before;
      const bool tail = lane == 31 || q != after;
#pragma unroll
      for (int o = 1; o < 32; o *= 2) {
        const int cc = __shfl_up_sync(0xffffffffu, c, o);
        const bool hh = __shfl_up_sync(0xffffffffu, head ? 1 : 0, o) != 0;
        double vv = 0.0;
        if constexpr (kSum) vv = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o && !head) {
          if constexpr (kSum) v += vv;
          c += cc;
          head = hh;
        }
      }
      if (q >= 0 && q == run_s) {   // begun before these 32
        if constexpr (kSum) v += run;
        c += run_n;
      }
      const bool ends = q >= 0 && tt + 1 >= qe;
      if (tail && ends) put(q, qs, v, c);
      // the sequence of the last token goes on, or nothing does
      const int last = min(31, g1 - 1 - h);
      const bool on = __shfl_sync(0xffffffffu, q >= 0 && !ends ? 1 : 0, last) != 0;
      const int lq = __shfl_sync(0xffffffffu, q, last);
      if constexpr (kSum) run = on ? __shfl_sync(0xffffffffu, v, last) : 0.0;
      run_n = on ? __shfl_sync(0xffffffffu, c, last) : 0;
      if (lq >= 0) run_s = lq;
    }
    s = seq_from(a, g1, run_s);
    enter();
    sum = lane == 0 ? run : 0.0;
    n = lane == 0 ? run_n : 0;
  }
  if (s >= 0 && s < a.S && cs < u1 && ce > u1) {   // unfinished at the end of the run
    if constexpr (kSum) sum = warp_sum(sum);
    n = warp_sum(n);
    if (lane == 0) put(s, cs, sum, n);
  }
}

// Counted tokens (and the sum) of sequence s, from its pieces, by one warp.
template <bool kSum>
__device__ __forceinline__ int sequence_total(const TokenArgs& a, int s, int lane, double& sum) {
  const int cs = cu_at(a, s), ce = cu_at(a, s + 1);
  sum = 0.0;
  if (ce <= cs) return 0;
  const int ua = cs / a.unit, ub = (ce - 1) / a.unit;
  int n = 0;
#pragma unroll 4
  for (int u = ua + 1 + lane; u <= ub; u += 32) {
    if constexpr (kSum) sum += a.open_sum[u];
    n += a.open_n[u];
  }
  if (lane == 0) {
    if constexpr (kSum) sum += a.seg_sum[s];
    n += a.seg_n[s];
  }
  if constexpr (kSum) sum = warp_sum(sum);
  return warp_sum(n);
}

// The same for a sequence per lane (-1: none): the lane adds the pieces of a
// short one, the warp together those of a long one.
template <bool kSum>
__device__ __forceinline__ int lane_total(const TokenArgs& a, int s, int lane, double& sum) {
  constexpr int kAlone = 8;
  int n = 0, ua = 0, ub = -1;
  sum = 0.0;
  if (s >= 0) {
    const int cs = cu_at(a, s), ce = cu_at(a, s + 1);
    if (ce > cs) {
      ua = cs / a.unit;
      ub = (ce - 1) / a.unit;
    }
  }
  const bool together = ub - ua > kAlone;
  if (ub >= ua && !together) {
    if constexpr (kSum) sum = a.seg_sum[s];
    n = a.seg_n[s];
    for (int u = ua + 1; u <= ub; ++u) {
      if constexpr (kSum) sum += a.open_sum[u];
      n += a.open_n[u];
    }
  }
  for (uint32_t todo = __ballot_sync(0xffffffffu, together); todo != 0; todo &= todo - 1) {
    const int who = __ffs(todo) - 1;
    double v;
    const int c = sequence_total<kSum>(a, __shfl_sync(0xffffffffu, s, who), lane, v);
    if (lane == who) {
      sum = v;
      n = c;
    }
  }
  return n;
}

// Walks a run in groups and hands each lane's four tokens their sequence (-1:
// in none); `body(t, seq[4])`.
template <class F>
__device__ __forceinline__ void for_tokens(const TokenArgs& a, int unit, int lane, F body) {
  const int u0 = unit * a.unit, u1 = min(u0 + a.unit, a.T);
  if (u0 >= u1) return;
  int s = seq_of_warp(a, u0, lane);
  for (int g = u0; g < u1; g += kGroup) {
    const int t = g + 4 * lane;
    int q[4];
    const int next = s < a.S ? cu_at(a, s + 1) : a.T + 1;   // (s = -1: the first sequence's begin)
    const int g1 = min(g + kGroup, u1);
    if (next >= g1) {
#pragma unroll
      for (int i = 0; i < 4; ++i) q[i] = s >= 0 && s < a.S ? s : -1;
    } else {
      int from = s;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        int z = seq_from(a, min(t + i, g1 - 1), from);
        from = z;
        if (z >= a.S || (z >= 0 && t + i >= cu_at(a, z + 1))) z = -1;
        q[i] = z;
      }
      s = __shfl_sync(0xffffffffu, from, 31);
    }
    if (t < g1) body(t, q);   // (a run is a multiple of four tokens)
  }
}

// Barrier of all blocks of the launch, with their writes before it visible after
// it: of one block, of one cluster, of a cooperative grid.
enum MeetKind { kMeetBlock, kMeetCluster, kMeetGrid };
template <MeetKind kMeet>
__device__ __forceinline__ void meet() {
  if constexpr (kMeet == kMeetBlock) __syncthreads();
  else if constexpr (kMeet == kMeetCluster) cg::this_cluster().sync();
  else cg::this_grid().sync();
}

// Sums over the warps of this block, in warp order, of N values that lane 0 of
// each holds -> part[block].
template <int N>
__device__ __forceinline__ void block_sums(const TokenArgs& a, const double (&v)[N], int warp, int lane) {
  __shared__ double sums[kLossWarps][N];
  if (lane == 0)
#pragma unroll
    for (int i = 0; i < N; ++i) sums[warp][i] = v[i];
  __syncthreads();
  if (threadIdx.x < N) {
    double x = 0.0;
    for (int w = 0; w < kLossWarps; ++w) x += sums[w][threadIdx.x];
    a.part[4 * blockIdx.x + threadIdx.x] = x;
  }
}
// The sum of value i over all blocks, by one warp (the same order every time).
__device__ __forceinline__ double all_blocks(const TokenArgs& a, int i, int lane) {
  double x = 0.0;
  for (int b = lane; b < gridDim.x; b += 32) x += __ldcg(a.part + 4 * b + i);
  return warp_sum(x);
}

}  // namespace

template <MeetKind kMeet>
__global__ void __launch_bounds__(kLossThreads, 1) policy_loss_kernel(const PolicyArgs p) {
  __shared__ int count[2], counts[2];   // counted tokens, sequences with any: this block's share, of all
  const TokenArgs& a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int unit = blockIdx.x * kLossWarps + warp, units = gridDim.x * kLossWarps;
  if (threadIdx.x < 2) count[threadIdx.x] = 0;
  __syncthreads();
  const bool by_sequence = p.reduction == ARCHEAD_REDUCE_SEQUENCES;
  if (a.mask != nullptr && by_sequence) {
    walk_segments<false>(a, unit, lane);
    meet<kMeet>();
  }
  int total = 0, alive = 0;
  if (by_sequence) {
    const int each = min(32, (a.S + units - 1) / units);   // sequences of a warp at a time
    for (int s0 = each * unit; s0 < a.S; s0 += each * units) {
      const int s = lane < each && s0 + lane < a.S ? s0 + lane : -1;
      double unused;
      int n = 0;
      if (a.mask != nullptr) n = lane_total<false>(a, s, lane, unused);
      else if (s >= 0) n = max(0, cu_at(a, s + 1) - cu_at(a, s));
      if (s >= 0) a.each[s] = n > 0 ? 1.0 / n : 0.0;
      total += n;
      alive += n > 0 ? 1 : 0;
    }
    total = warp_sum(total);
    alive = warp_sum(alive);
  } else if (a.mask != nullptr) {
    const int b = max(unit * a.unit, cu_at(a, 0)), e = min(min((unit + 1) * a.unit, a.T), cu_at(a, a.S));
    for (int t = unit * a.unit + 4 * lane; t < e; t += kGroup) {
      const uint32_t k = keep4(a, t);
#pragma unroll
      for (int i = 0; i < 4; ++i) total += (k >> i & 1u) && t + i >= b && t + i < e ? 1 : 0;
    }
    total = warp_sum(total);
  } else if (unit == 0) {
    total = max(0, cu_at(a, a.S) - cu_at(a, 0));
  }
  if (lane == 0 && (total != 0 || alive != 0)) {   // (integers: the order of the adds is free)
    atomicAdd(&count[0], total);
    atomicAdd(&count[1], alive);
  }
  __syncthreads();
  if (threadIdx.x < 2) a.part_n[2 * blockIdx.x + threadIdx.x] = count[threadIdx.x];
  meet<kMeet>();
  if (warp < 2) {
    int n = 0;
    for (int b = lane; b < gridDim.x; b += 32) n += __ldcg(a.part_n + 2 * b + warp);
    n = warp_sum(n);
    if (lane == 0) counts[warp] = n;
  }
  __syncthreads();
  total = counts[0];
  const double all = p.reduction == ARCHEAD_REDUCE_SUM ? p.scale
                     : by_sequence                     ? p.scale / max(counts[1], 1)
                                                       : p.scale / max(total, 1);
  double loss = 0.0, cut_n = 0.0, kl_old = 0.0, kl_ref = 0.0;
  for_tokens(a, unit, lane, [&](int t, const int (&q)[4]) {
    if (t >= a.T) return;
    const uint32_t keep = keep4(a, t);
    float x[4], o[4], r[4], A[4], g[4];
    load4(a.ce, t, a.T, a.vec, x);
    load4(p.old, t, a.T, a.vec, o);
    if (a.ce_ref != nullptr) load4(a.ce_ref, t, a.T, a.vec, r);
    if (!p.per_sequence) load4(p.adv, t, a.T, a.vec, A);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      g[i] = 0.f;
      if (q[i] < 0 || !(keep >> i & 1u)) continue;
      const double adv = p.per_sequence ? __ldg(p.adv + q[i]) : A[i];
      const double w = by_sequence ? all * a.each[q[i]] : all;
      const double D = static_cast<double>(o[i]) - static_cast<double>(x[i]);
      double m1, k3;
      const double ratio = exp_k3(D, m1, k3);
      const bool cut = adv > 0.0 ? D > p.border_hi : adv < 0.0 && D < p.border_lo;
      const double gain = adv == 0.0 && ratio == ratio ? 0.0 : adv * ratio;   // (0 times a ratio that overflowed would be NaN)
      double l = cut ? -adv * (adv > 0.0 ? p.clip_hi : p.clip_lo) : -gain, dl = cut ? 0.0 : gain;
      cut_n += cut ? 1.0 : 0.0;
      kl_old += k3;
      if (a.ce_ref != nullptr) {
        const double d = static_cast<double>(x[i]) - static_cast<double>(r[i]);
        double k;
        exp_k3(d, m1, k);
        kl_ref += k;
        if (p.kl != 0.0) {   // (0 times an infinite divergence would be NaN)
          l = fma(p.kl, k, l);
          dl = fma(p.kl, m1, dl);
        }
      }
      loss = fma(w, l, loss);
      g[i] = static_cast<float>(w * dl);
    }
    store4(a.grad, t, a.T, a.vec, g);
  });
  block_sums<4>(a, {warp_sum(loss), warp_sum(cut_n), warp_sum(kl_old), warp_sum(kl_ref)}, warp, lane);
  meet<kMeet>();
  if (blockIdx.x == 0 && warp < 4) {
    const double v = all_blocks(a, warp, lane);
    if (lane == 0) {
      if (warp == 0) *p.loss = static_cast<float>(v);
      else p.stats[warp - 1] = static_cast<float>(v / max(total, 1));
    }
  }
}

template <MeetKind kMeet>
__global__ void __launch_bounds__(kLossThreads, 1) preference_loss_kernel(const PreferenceArgs p) {
  const TokenArgs& a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int unit = blockIdx.x * kLossWarps + warp, units = gridDim.x * kLossWarps;
  walk_segments<true>(a, unit, lane);
  meet<kMeet>();
  double loss = 0.0;
  const int each = min(32, (p.N + units - 1) / units);   // pairs of a warp at a time
  for (int i0 = each * unit; i0 < p.N; i0 += each * units) {
    const int i = lane < each && i0 + lane < p.N ? i0 + lane : -1;
    double sc, sr;
    const int nc = lane_total<true>(a, i, lane, sc), nr = lane_total<true>(a, i < 0 ? -1 : p.N + i, lane, sr);
    if (i < 0) continue;
    const double fc = p.average ? 1.0 / max(nc, 1) : 1.0, fr = p.average ? 1.0 / max(nr, 1) : 1.0;
    sc *= fc;
    sr *= fr;
    double slope;   // d l / d D
    if (p.kind == ARCHEAD_PREFERENCE_SQUARED) {
      const double m = sc - sr - 0.5 / p.beta;
      loss += m * m;
      slope = 2.0 * m;
    } else {
      const double h = p.beta * (sc - sr) - p.margin;
      if (p.kind == ARCHEAD_PREFERENCE_HINGE) {
        loss += h < 1.0 ? 1.0 - h : h == h ? 0.0 : h;
        slope = h < 1.0 ? -p.beta : h == h ? 0.0 : h;
      } else {
        const double e = exp(-fabs(h)), up = 1.0 / (1.0 + e), lo = e / (1.0 + e);   // sigmoid(|h|), sigmoid(-|h|)
        const double l1 = log1p(e);
        loss += (1.0 - p.smooth) * (l1 + fmax(-h, 0.0));
        if (p.smooth != 0.0) loss += p.smooth * (l1 + fmax(h, 0.0));   // (0 times infinity is no loss)
        const double s_pos = h >= 0.0 ? up : lo, s_neg = h >= 0.0 ? lo : up;        // sigmoid(h), sigmoid(-h)
        slope = p.beta * (p.smooth * s_pos - (1.0 - p.smooth) * s_neg);
      }
    }
    const double f = p.scale / p.N;
    a.coef[i] = static_cast<float>(-slope * fc * f);
    a.coef[p.N + i] = static_cast<float>(slope * fr * f);
    p.rewards[i] = static_cast<float>(p.beta * sc);
    p.rewards[p.N + i] = static_cast<float>(p.beta * sr);
  }
  block_sums<1>(a, {warp_sum(loss)}, warp, lane);
  meet<kMeet>();
  for_tokens(a, unit, lane, [&](int t, const int (&q)[4]) {
    if (t >= a.T) return;
    const uint32_t keep = keep4(a, t);
    float g[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) g[i] = q[i] >= 0 && (keep >> i & 1u) ? a.coef[q[i]] : 0.f;
    store4(a.grad, t, a.T, a.vec, g);
  });
  if (blockIdx.x == 0 && warp == 0) {
    const double v = all_blocks(a, 0, lane);
    if (lane == 0) *p.loss = static_cast<float>(p.N > 0 ? v * p.scale / p.N : 0.0);
  }
}

namespace {

constexpr int kMaxTokens = 1 << 20;

bool aligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

// Workspace: pieces per sequence and per unit, factors per sequence.
struct LossLayout {
  size_t seg_sum, open_sum, seg_n, open_n, coef, each, part, part_n, total;
};
LossLayout loss_layout(int S) {
  LossLayout o{};
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t r = at;
    at += round_up(bytes, 256);
    return r;
  };
  const size_t s = S > 0 ? S : 1;
  o.seg_sum = take(s * 8);
  o.open_sum = take(kMaxUnits * 8);
  o.seg_n = take(s * 4);
  o.open_n = take(kMaxUnits * 4);
  o.coef = take(s * 4);
  o.each = take(s * 8);
  o.part = take(kLossMaxBlocks * 32);
  o.part_n = take(kLossMaxBlocks * 8);
  o.total = at;
  return o;
}

// Blocks of a call: a warp's run is one group of tokens while that many fit.
int loss_blocks(int T, int* blocks) {
  *blocks = 1;
  while (*blocks < 16 && T > *blocks * kOneBlock) *blocks *= 2;
  if (T <= kOneCluster) return ARCHEAD_OK;
  int dev = -1, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return set_cuda_error(e);
  *blocks = std::max(16, std::min(sms, kLossMaxBlocks));
  return ARCHEAD_OK;
}

void token_args(TokenArgs& a, const float* ce, const float* ce_ref, const uint8_t* mask, const int32_t* cu, int T, int S,
                float* grad, void* ws, int blocks) {
  const LossLayout o = loss_layout(S);
  uint8_t* w = static_cast<uint8_t*>(ws);
  a.ce = ce;
  a.ce_ref = ce_ref;
  a.mask = mask;
  a.cu = cu;
  a.T = T;
  a.S = S;
  // whole groups, or a part of one so that few tokens still spread over the warps
  const int per = (T + blocks * kLossWarps - 1) / (blocks * kLossWarps);
  a.unit = per <= 32 ? 32 : per <= 64 ? 64 : static_cast<int>(round_up(per, kGroup));
  a.vec = aligned(ce, 16) && aligned(ce_ref, 16) && aligned(mask, 4) && aligned(grad, 16) ? 1 : 0;
  a.grad = grad;
  a.seg_sum = reinterpret_cast<double*>(w + o.seg_sum);
  a.open_sum = reinterpret_cast<double*>(w + o.open_sum);
  a.seg_n = reinterpret_cast<int32_t*>(w + o.seg_n);
  a.open_n = reinterpret_cast<int32_t*>(w + o.open_n);
  a.coef = reinterpret_cast<float*>(w + o.coef);
  a.each = reinterpret_cast<double*>(w + o.each);
  a.part = reinterpret_cast<double*>(w + o.part);
  a.part_n = reinterpret_cast<int32_t*>(w + o.part_n);
}

template <class Args>
struct LossKernels {
  void (*block)(Args);
  void (*cluster)(Args);
  void (*grid)(Args);
};
constexpr LossKernels<PolicyArgs> kPolicy{policy_loss_kernel<kMeetBlock>, policy_loss_kernel<kMeetCluster>,
                                          policy_loss_kernel<kMeetGrid>};
constexpr LossKernels<PreferenceArgs> kPreference{preference_loss_kernel<kMeetBlock>, preference_loss_kernel<kMeetCluster>,
                                                  preference_loss_kernel<kMeetGrid>};

template <class Args>
int launch_loss(const LossKernels<Args>& kernels, const Args& args, int blocks, archead_stream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(kLossThreads);
  cfg.stream = reinterpret_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  void (*kernel)(Args) = kernels.block;
  cudaError_t e = cudaSuccess;
  if (blocks > 16) {
    kernel = kernels.grid;
    attr[0].id = cudaLaunchAttributeCooperative;
    attr[0].val.cooperative = 1;
  } else if (blocks > 1) {
    kernel = kernels.cluster;
    // clusters of more than 8 blocks are opted into (per context, so at every call)
    if (blocks > 8) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = blocks;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  }
  cfg.attrs = attr;
  cfg.numAttrs = blocks > 1 ? 1 : 0;
  if (e == cudaSuccess) e = cudaLaunchKernelEx(&cfg, kernel, args);
  return e == cudaSuccess ? ARCHEAD_OK : set_cuda_error(e);
}

}  // namespace

}  // namespace archead

using namespace archead;

extern "C" ARCHEAD_API size_t archead_loss_workspace_bytes(int32_t n_sequences) {
  if (n_sequences < 0 || n_sequences > 2 * kMaxTokens) return 0;
  return loss_layout(n_sequences).total;
}

extern "C" ARCHEAD_API int archead_policy_loss(const float* ce, const float* ce_old, const float* advantages,
                                               const float* ce_ref, const uint8_t* mask, const int32_t* cu_seqlens,
                                               int32_t T, int32_t n_sequences, const archead_policy_options* options,
                                               float* loss, float* grad_ce, float* stats, void* workspace,
                                               size_t workspace_bytes, archead_stream_t stream) {
  if (options == nullptr || loss == nullptr || stats == nullptr || workspace == nullptr) return ARCHEAD_EINVAL;
  if (T < 0 || T > kMaxTokens || n_sequences < 0 || n_sequences > 2 * kMaxTokens) return ARCHEAD_EINVAL;
  if (T > 0 && (ce == nullptr || ce_old == nullptr || grad_ce == nullptr)) return ARCHEAD_EINVAL;
  if (cu_seqlens == nullptr && n_sequences != 1) return ARCHEAD_EINVAL;
  const archead_policy_options& o = *options;
  if (!(o.clip_low >= 0.0 && o.clip_low <= 1.0) || !(o.clip_high >= 0.0) || !std::isfinite(o.kl_coef) ||
      !std::isfinite(o.scale))
    return ARCHEAD_EINVAL;
  if (o.reduction < ARCHEAD_REDUCE_TOKENS || o.reduction > ARCHEAD_REDUCE_SUM) return ARCHEAD_EINVAL;
  if (o.advantage_per != ARCHEAD_PER_TOKEN && o.advantage_per != ARCHEAD_PER_SEQUENCE) return ARCHEAD_EINVAL;
  const bool per_sequence = o.advantage_per == ARCHEAD_PER_SEQUENCE;
  if (advantages == nullptr && (per_sequence ? n_sequences : T) > 0) return ARCHEAD_EINVAL;
  const void* words[] = {ce, ce_old, advantages, ce_ref, cu_seqlens, loss, grad_ce, stats};
  for (const void* q : words)
    if (!aligned(q, 4)) return ARCHEAD_EALIGN;
  if (!aligned(workspace, 256)) return ARCHEAD_EALIGN;
  if (workspace_bytes < loss_layout(n_sequences).total) return ARCHEAD_ENOMEM;
  int blocks = 1;
  const int rc = loss_blocks(T, &blocks);
  if (rc != ARCHEAD_OK) return rc;
  PolicyArgs p{};
  token_args(p.a, ce, ce_ref, mask, cu_seqlens, T, n_sequences, grad_ce, workspace, blocks);
  if (!aligned(ce_old, 16) || (!per_sequence && !aligned(advantages, 16))) p.a.vec = 0;
  p.old = ce_old;
  p.adv = advantages;
  p.border_hi = std::log1p(o.clip_high);
  p.border_lo = std::log1p(-o.clip_low);
  p.clip_hi = 1.0 + o.clip_high;
  p.clip_lo = 1.0 - o.clip_low;
  p.kl = o.kl_coef;
  p.scale = o.scale;
  p.reduction = o.reduction;
  p.per_sequence = per_sequence ? 1 : 0;
  p.loss = loss;
  p.stats = stats;
  return launch_loss(kPolicy, p, blocks, stream);
}

extern "C" ARCHEAD_API int archead_preference_loss(const float* ce, const float* ce_ref, const uint8_t* mask,
                                                   const int32_t* cu_seqlens, int32_t T, int32_t n_pairs,
                                                   const archead_preference_options* options, float* loss,
                                                   float* grad_ce, float* rewards, void* workspace,
                                                   size_t workspace_bytes, archead_stream_t stream) {
  if (options == nullptr || loss == nullptr || workspace == nullptr || cu_seqlens == nullptr) return ARCHEAD_EINVAL;
  if (T < 0 || T > kMaxTokens || n_pairs < 0 || n_pairs > kMaxTokens) return ARCHEAD_EINVAL;
  if (T > 0 && (ce == nullptr || grad_ce == nullptr)) return ARCHEAD_EINVAL;
  if (n_pairs > 0 && rewards == nullptr) return ARCHEAD_EINVAL;
  const archead_preference_options& o = *options;
  if (!(o.beta > 0.0) || !std::isfinite(o.beta) || !std::isfinite(o.margin) || !std::isfinite(o.scale))
    return ARCHEAD_EINVAL;
  if (o.kind < ARCHEAD_PREFERENCE_SIGMOID || o.kind > ARCHEAD_PREFERENCE_SQUARED) return ARCHEAD_EINVAL;
  if (!(o.label_smoothing >= 0.0 && o.label_smoothing <= 0.5)) return ARCHEAD_EINVAL;
  if (o.label_smoothing != 0.0 && o.kind != ARCHEAD_PREFERENCE_SIGMOID) return ARCHEAD_EINVAL;
  if (o.margin != 0.0 && o.kind == ARCHEAD_PREFERENCE_SQUARED) return ARCHEAD_EINVAL;
  const void* words[] = {ce, ce_ref, cu_seqlens, loss, grad_ce, rewards};
  for (const void* q : words)
    if (!aligned(q, 4)) return ARCHEAD_EALIGN;
  if (!aligned(workspace, 256)) return ARCHEAD_EALIGN;
  if (workspace_bytes < loss_layout(2 * n_pairs).total) return ARCHEAD_ENOMEM;
  int blocks = 1;
  const int rc = loss_blocks(T, &blocks);
  if (rc != ARCHEAD_OK) return rc;
  PreferenceArgs p{};
  token_args(p.a, ce, ce_ref, mask, cu_seqlens, T, 2 * n_pairs, grad_ce, workspace, blocks);
  p.beta = o.beta;
  p.margin = o.margin;
  p.smooth = o.label_smoothing;
  p.scale = o.scale;
  p.N = n_pairs;
  p.kind = o.kind;
  p.average = o.average != 0;
  p.loss = loss;
  p.rewards = rewards;
  return launch_loss(kPreference, p, blocks, stream);
}
