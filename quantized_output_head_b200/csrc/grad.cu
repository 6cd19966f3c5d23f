// Gradient of the cross-entropy with respect to the hidden states, through the
// packed head (ARCHead paper, §3.2 Eq. 7; the head itself is frozen).
//
// With y[t] = W h[t] over all rows of the head, lse[t] its log-sum-exp and
// g[t] = dLoss / dce[t], ce[t] = lse[t] - y[t, target[t]]:
//   dh[t,:] = g[t] sum_v (p[t,v] - [v = target[t]]) W[v,:],   p = exp(y - lse).
// W is never formed.  With W~ the concatenated packed operand of the
// tensor-core forward (tc_params.h; columns residual | core | correction)
//   y = 2^-c_t X W~^T,        G = p, but 0 at the target's row,
//   dX = G W~ + (p[target] - 1) W~[target]   (one row of d + r_c' + r_r' columns),
//   dh = g ( dX_res + dX_core (s_R R) + dX_corr (s_B B) ),
// so the low-rank factors are applied once per token, not once per row.
//
// The recomputed logits carry the forward's rounding (up to ~1e-2 where y is
// large), the given lse that of whichever kernel made it; a row that holds most
// of the mass would get all of their difference.  So the probabilities are
// normalised by their own sum S[t] = Rest[t] + p[t,target], Rest[t] = sum_v G[t,v],
// after the fact:
//   sum_v (p / S - [v = target]) W[v] = (G W) / S - (Rest / S) W[target].
// No term cancels: with the target's p - 1 inside G, its coefficient 1 - p of a
// confident token would be a difference of terms of size |S - 1| that are rounded
// to fp16 (rows of 1 - p = 1e-5 were 45 % off with lse off by 1e-2).
// On a vocabulary shard S is not known: lse is taken as it is, and the coefficient
// is p - 1, from y - lse in one rounding.  Of a sure token it is as good as y and
// lse agree, so a shard's logits come from the kernels that gave its lse: the
// activation kernel's z at every token count, and on heads that the tensor-core
// forward does not take the decode kernel's logits, 8 tokens a pass (rows of
// 1 - p = 1e-2 were up to 39 % off with the fp16 rows' logits there, 0.06 % now).
//
// Many tokens: the vocabulary is walked in chunks of rows.  Per chunk
//   1. dequant_rows_kernel   W~ of the chunk, fp16, in the workspace
//   2. gemm softmax          G of the chunk, fp16
//   3. gemm accumulate       dX += G W~, fp32
// and after the last chunk
//   4. dx_kernel             dX / S - (Rest / S) W~[target], its low-rank
//      columns to fp16; lowrank_rows_kernel: [s_R R | s_B B], fp16
//   5. gemm finish           dh from dX_res + dz [s_R R | s_B B].
// Few tokens: G from the forward kernels, gw_kernel for G W~, then 4 and 5; up to
// 8 tokens finish_few_kernel in place of 5.
//
// Roundings to fp16: W~ entries (2^-11 relative, as in the forward), G (2^-11,
// stored times 2^15 so that a probability keeps its full precision down to
// 2^-29), dX of the low-rank columns and the rows of R and B (for dh; z takes them
// exactly).  fp16 because the tensor cores take no operand of more than 11 bits
// (tf32 has the same 11, at half the rate; bf16 has 8), and a second fp16 term
// for the rest of each operand would double the products for bits that the bf16
// result drops.  All are independent from entry to entry, so the sum's error
// stays near 2^-12 of its own size, below the bf16 rounding of the result; sums
// are fp32.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "device.cuh"
#include "handle.h"
#include "tcgen05.cuh"

namespace archead {

namespace {

constexpr int kGradTokens = 4096;     // tokens of one pass over the head
// Vocabulary rows of one pass: as many as keep the W~ chunk and the G chunk near
// these sizes, evened out over the passes (4096 tokens of 151936 x 4096, 4672
// columns: 35,840 rows fit, five passes of 30,464).  Fewer passes re-read and
// re-write dX less often and leave fewer part-filled rounds of tiles: 29, 17, 9 and
// 5 passes took 9.1, 8.5, 8.2 and 7.9 ms for the chunks' kernels there.
constexpr size_t kGradWBytes = size_t(320) << 20, kGradGBytes = size_t(512) << 20;
constexpr int kGradScale = kTcGradScale;   // G is stored times 2^15

// ------------------------------------------------------------ packed -> fp16
struct DequantParams {
  const uint8_t* mtiles;
  uint16_t* out;              // [rows][Kc]
  int32_t mt0, n_mt;          // m-tiles [mt0, mt0 + n_mt)
  int32_t Kc, n_res, n_L, n_A, n_ks, g_log2;
  uint32_t off_res, off_Lnib, off_Lhi, off_A, off_sres, off_sL, off_sA, mblk_bytes;
  float sc_res, sc_L, sc_A;
};

__device__ __forceinline__ uint32_t ldg32(const uint8_t* p) { return __ldg(reinterpret_cast<const uint32_t*>(p)); }
// (Packed codes are read once: they take no line of L1.)
__device__ __forceinline__ uint4 ldg128(const uint8_t* p) {
  uint4 v;
  asm("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

// Scale pair (rows gr, gr + 8) times 2^e, as two half2 (s, s).
__device__ __forceinline__ void scales_of(uint32_t bits, float mul, uint32_t& s0, uint32_t& s1) {
  const float2 f = half2_bits_to_float2(bits);
  s0 = pack_half2(f.x * mul, f.x * mul);
  s1 = pack_half2(f.y * mul, f.y * mul);
}

// One warp per (m-tile, 64-column k-step): each lane unpacks its fragments of
// four k16 steps, applies the scale (the one rounding) and writes 8 bytes per
// row and step, in the column order of the activation operand.
__global__ void __launch_bounds__(256) dequant_rows_kernel(const DequantParams p) {
  const int lane = threadIdx.x & 31;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  if (item >= static_cast<int64_t>(p.n_mt) * p.n_ks) return;
  const int mt = static_cast<int>(item / p.n_ks), ks = static_cast<int>(item % p.n_ks);
  const uint8_t* blk = p.mtiles + static_cast<size_t>(p.mt0 + mt) * p.mblk_bytes;
  const int gr = lane >> 2, cc = lane & 3;
  uint32_t a[4][4], s0[4], s1[4];
  if (ks < p.n_res) {
    const uint4 c = ldg128(blk + p.off_res + ks * kResChunkBytes + lane * 16);
    const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
    for (int st = 0; st < 4; ++st) {
      scales_of(ldg32(blk + p.off_sres + ((ks * 64 + st * 16) >> p.g_log2) * kSresGroupBytes + gr * 4), p.sc_res, s0[st],
                s1[st]);
      unpack_int4_signed(w[st], a[st]);
    }
  } else if (ks < p.n_res + p.n_L) {
    const int c = ks - p.n_res;
    const uint4 n = ldg128(blk + p.off_Lnib + c * kLNibChunkBytes + lane * 16);
    const uint32_t hb = ldg32(blk + p.off_Lhi + c * kLHiChunkBytes + lane * 4);
    unpack_int5_signed<0>(n.x, hb, a[0]);
    unpack_int5_signed<1>(n.y, hb, a[1]);
    unpack_int5_signed<2>(n.z, hb, a[2]);
    unpack_int5_signed<3>(n.w, hb, a[3]);
    scales_of(ldg32(blk + p.off_sL + gr * 4), p.sc_L, s0[0], s1[0]);
#pragma unroll
    for (int st = 1; st < 4; ++st) {
      s0[st] = s0[0];
      s1[st] = s1[0];
    }
  } else {
    const int c = 2 * (ks - p.n_res - p.n_L);
    const uint4 c0 = ldg128(blk + p.off_A + c * kAChunkBytes + lane * 16);
    unpack_int8_signed(c0.x, c0.y, a[0]);
    unpack_int8_signed(c0.z, c0.w, a[1]);
    if (c + 1 < p.n_A) {
      const uint4 c1 = ldg128(blk + p.off_A + (c + 1) * kAChunkBytes + lane * 16);
      unpack_int8_signed(c1.x, c1.y, a[2]);
      unpack_int8_signed(c1.z, c1.w, a[3]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) a[2][i] = a[3][i] = 0u;
    }
    scales_of(ldg32(blk + p.off_sA + gr * 4), p.sc_A, s0[0], s1[0]);
#pragma unroll
    for (int st = 1; st < 4; ++st) {
      s0[st] = s0[0];
      s1[st] = s1[0];
    }
  }
  uint16_t* row0 = p.out + static_cast<size_t>(mt * kMT + gr) * p.Kc + ks * 64 + 4 * cc;
  uint16_t* row1 = row0 + static_cast<size_t>(8) * p.Kc;
#pragma unroll
  for (int st = 0; st < 4; ++st) {
    *reinterpret_cast<uint2*>(row0 + st * 16) = make_uint2(hmul2_bits(a[st][0], s0[st]), hmul2_bits(a[st][2], s0[st]));
    *reinterpret_cast<uint2*>(row1 + st * 16) = make_uint2(hmul2_bits(a[st][1], s1[st]), hmul2_bits(a[st][3], s1[st]));
  }
}

// Rows of [s_R R | s_B B] times 2^rho, fp16 [Kz'][d]; row e holds the low-rank
// index at position e of the operand order.
struct LowrankParams {
  const int8_t* R;
  const uint16_t* s_R;
  const int8_t* B;
  const uint16_t* s_B;
  uint16_t* out;
  uint16_t* out_perm;         // or null: [Kz'][2 d], columns in the operand order: the rows, then what fp16 left of them
  uint32_t* header;           // 64 words of the workspace: status, tickets
  int32_t d, rcp, rrp, Kz, g_B;
  float mul_c, mul_r;
};
// (For z a row is the sum of two fp16 ones: a code times an fp16 scale has at most 19
// bits, so the pair is exact and z is as good as the forward's activation kernel's.
// The rounded rows alone move the logits by up to 2^-11 of their size.)
// A thread per 8 columns; the first block also clears the workspace header.
__global__ void __launch_bounds__(256) lowrank_rows_kernel(const LowrankParams p) {
  if (blockIdx.x == 0 && threadIdx.x < 64) p.header[threadIdx.x] = 0u;
  const int per = p.d / 8, i = blockIdx.x * 256 + threadIdx.x;
  const int e = i / per, j = (i - e * per) * 8;
  if (e >= p.Kz) return;
  const int k = (e & ~15) + tc_kcol(e & 15);
  const bool core = k < p.rcp;
  uint32_t o[4] = {0u, 0u, 0u, 0u}, left[4] = {0u, 0u, 0u, 0u};
  if (core || k - p.rcp < p.rrp) {
    const int r = core ? k : k - p.rcp;
    const uint2 codes = __ldg(reinterpret_cast<const uint2*>((core ? p.R : p.B) + static_cast<size_t>(r) * p.d + j));
    const int8_t* c8 = reinterpret_cast<const int8_t*>(&codes);
    const uint16_t* sb = core ? nullptr : p.s_B + static_cast<size_t>(r) * (p.d / p.g_B);
    const float mul = core ? __half2float(__ushort_as_half(p.s_R[r])) * p.mul_c : p.mul_r;
#pragma unroll
    for (int c = 0; c < 8; c += 2) {
      float v[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        v[h] = static_cast<float>(c8[c + h]) * mul;
        if (!core) v[h] *= __half2float(__ushort_as_half(sb[(j + c + h) / p.g_B]));
      }
      o[c / 2] = pack_half2(v[0], v[1]);
      const float2 f = half2_bits_to_float2(o[c / 2]);
      left[c / 2] = pack_half2(v[0] - f.x, v[1] - f.y);
    }
  }
  *reinterpret_cast<uint4*>(p.out + static_cast<size_t>(e) * p.d + j) = make_uint4(o[0], o[1], o[2], o[3]);
  if (p.out_perm != nullptr) {
    uint16_t* row = p.out_perm + static_cast<size_t>(e) * 2 * p.d + (j & ~15);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      *reinterpret_cast<uint32_t*>(row + tc_kpos((j & 15) + 2 * c)) = o[c];
      *reinterpret_cast<uint32_t*>(row + p.d + tc_kpos((j & 15) + 2 * c)) = left[c];
    }
  }
}

// The h columns of X, and 2^-c_t, where the activation kernel is not used (many
// tokens; heads with g_B not a multiple of 64, which it does not take); the z
// columns come from a product with the rows of R and B as pairs of fp16 rows (1769 x 2176 with
// 512 + 512 rows, g_B = 32, 2708 tokens: 0.18 ms for the whole gradient; with the
// decode path's z kernel, 8 tokens a pass over R and B, 2.4).  One block per token.
struct XParams {
  const uint16_t* hidden;
  uint16_t* xop;
  float* cinv;
  int32_t d, Kc, alpha, mseg;
};
__global__ void __launch_bounds__(128) x_hidden_kernel(const XParams p) {
  __shared__ uint32_t part[4];
  const int t = blockIdx.x;
  const uint16_t* h = p.hidden + static_cast<size_t>(t) * p.d;
  uint32_t m = 0;
  for (int j = threadIdx.x; j < p.d; j += 128) m = max(m, static_cast<uint32_t>(h[j]) & 0x7FFFu);   // |bf16| orders like its bits
  m = __reduce_max_sync(0xffffffffu, m);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = m;
  __syncthreads();
  m = max(max(part[0], part[1]), max(part[2], part[3]));
  int E = 0;
  if (m != 0) frexpf(__uint_as_float(m << 16), &E);   // max|h_t| < 2^E
  E = max(E, kMinExp);
  if (threadIdx.x == 0) p.cinv[t] = ldexpf(1.f, E - kScaleExp - p.mseg);
  const float s = ldexpf(1.f, kScaleExp - E + p.mseg - p.alpha);
  for (int e = threadIdx.x; e < p.d; e += 128) {
    const int k = (e & ~15) + tc_kcol(e & 15);
    p.xop[static_cast<size_t>(t) * p.Kc + e] =
        __half_as_ushort(__float2half_rn(__uint_as_float(static_cast<uint32_t>(h[k]) << 16) * s));
  }
}

// Four operand columns from 4 q on of row `row` of an m-tile block, times the
// segment's 2^alpha|beta|gamma (fp32, exact).
__device__ __forceinline__ float4 packed_row4(const DequantParams& p, const uint8_t* blk, int row, int q) {
  const int ks = q >> 4, st = (q >> 2) & 3, cc = q & 3, gr = row & 7, up = row >> 3;
  const int lane = 4 * gr + cc;
  uint32_t a[4];
  uint32_t sbits;
  float mul;
  if (ks < p.n_res) {
    unpack_int4_signed(ldg32(blk + p.off_res + ks * kResChunkBytes + lane * 16 + st * 4), a);
    sbits = ldg32(blk + p.off_sres + ((ks * 64 + st * 16) >> p.g_log2) * kSresGroupBytes + gr * 4);
    mul = p.sc_res;
  } else if (ks < p.n_res + p.n_L) {
    const int c = ks - p.n_res;
    const uint32_t w = ldg32(blk + p.off_Lnib + c * kLNibChunkBytes + lane * 16 + st * 4);
    const uint32_t hb = ldg32(blk + p.off_Lhi + c * kLHiChunkBytes + lane * 4);
    if (st == 0) unpack_int5_signed<0>(w, hb, a);
    else if (st == 1) unpack_int5_signed<1>(w, hb, a);
    else if (st == 2) unpack_int5_signed<2>(w, hb, a);
    else unpack_int5_signed<3>(w, hb, a);
    sbits = ldg32(blk + p.off_sL + gr * 4);
    mul = p.sc_L;
  } else {
    const int c = 2 * (ks - p.n_res - p.n_L) + (st >> 1);
    if (c >= p.n_A) return make_float4(0.f, 0.f, 0.f, 0.f);
    const uint8_t* at = blk + p.off_A + c * kAChunkBytes + lane * 16 + (st & 1) * 8;
    unpack_int8_signed(ldg32(at), ldg32(at + 4), a);
    sbits = ldg32(blk + p.off_sA + gr * 4);
    mul = p.sc_A;
  }
  const float2 s2 = half2_bits_to_float2(sbits);
  const float s = (up ? s2.y : s2.x) * mul;
  const float2 lo = half2_bits_to_float2(a[up]), hi = half2_bits_to_float2(a[2 + up]);
  return make_float4(lo.x * s, lo.y * s, hi.x * s, hi.y * s);
}

constexpr int kGwCols = 256, kGwChunks = kGwCols / 64;   // column block of gw_kernel
// Row splits of the column blocks: the first `res` blocks are residual alone,
// then come `rest` with core, correction or mixed chunks (the last may be short).
struct GwSplits {
  int32_t res, rest, s_res, s_rest, s_last;
};
__host__ __device__ __forceinline__ int gw_splits(const GwSplits& g, int block) {
  return block < g.res ? g.s_res : block + 1 < g.res + g.rest ? g.s_rest : g.s_last;
}

// Blocks of 1024 (or 256) columns per token: Rest from the tiles' partial sums (in a
// fixed order), then dX (added over the K splits) / S - (Rest / S) W~[target]; the
// residual columns stay fp32 in the first split's place, the low-rank ones become
// the fp16 operand dz [T][Kz'].  Latency is all there is to it at few tokens: the
// loads are issued in batches, a token's partial sums lie side by side, and the
// target's row is read before the wait (16 tokens of 262144 x 2560: 21 -> 6 us).
struct DxParams {
  DequantParams rows;
  const float* ssum;          // [tokens][ssum_pitch], n_ssum of them used
  const float* ltgt;          // [tokens]: log of the target's probability
  const float* grad;
  const int32_t* targets;
  float* dx;
  size_t split_stride;
  uint16_t* dz;
  int32_t n_ssum, ssum_pitch, Kc, d, V, row0, whole;   // whole: all rows of the vocabulary are here
  int32_t splits;                                  // partial dX of every column, or (0) by
  GwSplits gw;
};
// Up to kDxWaysTokens tokens the partial dX of a column are added by 4 threads
// (whole gradient: 16 tokens of 8000 x 512 41.1 us with one, 37.6 with 4; 64 tokens
// of 65531 x 1024 69.3 and 66.2, of 32003 x 2048 81.6 and 80.4; but 128 tokens of
// 32003 x 2048 100.6 and 103, each block adding up S anew).
constexpr int kDxWays = 4, kDxWaysTokens = 64;
template <int kWays>
__global__ void __launch_bounds__(256) dx_kernel(const DxParams p) {
  constexpr int kCols = 256 / kWays;                  // float4 columns of a block
  __shared__ float part[8];
  __shared__ float4 sums[kWays > 1 ? 256 : 1];
  // What the call was given may be read before the wait: the call's first kernel
  // is not a dependent launch.
  const int t = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int way = threadIdx.x / kCols, q = blockIdx.y * kCols + threadIdx.x % kCols;
  const bool in = q < p.Kc / 4, out = in && way == 0, live = p.grad[t] != 0.f;   // (else its row of dX is zero, S has no meaning)
  const int target = live ? p.targets[t] - p.row0 : -1;
  const bool here = target >= 0 && target < p.V;   // (of these rows)
  float4 w = make_float4(0.f, 0.f, 0.f, 0.f);
  if (out && here)
    w = packed_row4(p.rows, p.rows.mtiles + static_cast<size_t>(target / kMT) * p.rows.mblk_bytes, target % kMT, q);
  grid_dependency_wait();
  grid_launch_dependents();
  float4* dx = reinterpret_cast<float4*>(p.dx + static_cast<size_t>(t) * p.Kc) + q;
  uint2* dz = reinterpret_cast<uint2*>(p.dz + static_cast<size_t>(t) * (p.Kc - p.d) + 4 * q - p.d);
  if (!live) {
    if (out && 4 * q >= p.d) *dz = make_uint2(0u, 0u);
    return;
  }
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  if (in) {
    const int n = p.splits > 0 ? p.splits : gw_splits(p.gw, 4 * q / kGwCols);
#pragma unroll 8
    for (int s = way; s < n; s += kWays) {
      const float4 x = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(dx) + s * p.split_stride);
      v = make_float4(v.x + x.x, v.y + x.y, v.z + x.z, v.w + x.w);
    }
  }
  if constexpr (kWays > 1) {
    sums[threadIdx.x] = v;
    __syncthreads();
#pragma unroll
    for (int i = 1; i < kWays; ++i) {
      const float4 x = sums[i * kCols + threadIdx.x % kCols];
      v = make_float4(v.x + x.x, v.y + x.y, v.z + x.z, v.w + x.w);
    }
  }
  const float own = here ? p.ltgt[t] : 0.f;
  float r = 1.f, c = here ? expm1f(own) : 0.f;
  if (p.whole) {
    const float* parts = p.ssum + static_cast<size_t>(t) * p.ssum_pitch;
    float s = 0.f;
#pragma unroll 4
    for (int i = threadIdx.x; i < p.n_ssum / 4; i += 256) {
      const float4 x = reinterpret_cast<const float4*>(parts)[i];
      s += (x.x + x.y) + (x.z + x.w);
    }
    if (threadIdx.x < p.n_ssum % 4) s += parts[p.n_ssum - 1 - threadIdx.x];
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane == 0) part[warp] = s;
    __syncthreads();
    s = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) s += part[i];
    r = 1.f / (s + expf(own));
    c = -s * r;
  }
  if (!out) return;
  c *= static_cast<float>(1 << kGradScale);
  v = make_float4(fmaf(c, w.x, v.x * r), fmaf(c, w.y, v.y * r), fmaf(c, w.z, v.z * r), fmaf(c, w.w, v.w * r));
  if (4 * q < p.d) {
    *dx = v;
  } else {
    constexpr float kInv = 1.f / (1 << kGradScale);
    *dz = make_uint2(pack_half2(v.x * kInv, v.y * kInv), pack_half2(v.z * kInv, v.w * kInv));
  }
}

// Launch as a programmatic dependent of the stream's previous kernel: the new
// grid's blocks may be set up while it drains, and each waits for its end
// (griddepcontrol.wait) before it touches memory that others write or read.
template <class... Params, class... Args>
cudaError_t launch_after(void (*kernel)(Params...), dim3 grid, int threads, size_t smem, cudaStream_t stream,
                         const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// -------------------------------------------------------------------- gemm
// D[256 tokens x 256 columns] tiles of A B, A [tokens][K] fp16 K-major, B fp16
// either [columns][K] (softmax, lowrank) or [K][columns] (accumulate, finish), by TMA in
// k-steps of 64, on pairs of CTAs: each holds the A rows of its 128 tokens and
// half of B's columns, one tcgen05.mma of the leader multiplies both (the tensor
// cores read their shared-memory operands at about 64 bytes a clock and SM; alone,
// a CTA's 128 x 256 tile needs 96 for the full rate).  A pair walks its units (K
// split, token tile, column tile); in each CTA warp 0 issues the copies, which
// count on the leader's barrier, warp 1 of the leader the MMAs, warps 2-9 empty
// one of two TMEM accumulators while the next fills.
constexpr int kGM = 256, kGN = 256, kGStages = 6, kGEpi = 8, kGWarps = 2 + kGEpi;
constexpr uint32_t kGABytes = kGM / 2 * 128, kGBBytes = kGN / 2 * 128, kGStageBytes = kGABytes + kGBBytes;
constexpr uint32_t kGBarOff = kGStages * kGStageBytes;
constexpr uint32_t kGTileOff = kGBarOff + 256;       // 32 x 33 words per epilogue warp
constexpr uint32_t kGSmem = kGTileOff + kGEpi * 32 * 33 * 4 + 1024;
constexpr uint32_t kGTmem = 512;

enum GemmMode { kSoftmax, kLowrank, kAccumulate, kFinish };
constexpr bool gemm_b_mn(GemmMode m) { return m == kAccumulate || m == kFinish; }   // B stored [K][columns]

struct GemmParams {
  int32_t M, N;                        // tokens; columns of this product
  int32_t n_k, n_mt, splits;
  int32_t n_full, n_half;              // units of 256 columns; of the last 128 or fewer
  int32_t half0, half_pairs;           // pairs that take the half units
  uint32_t* status;
  const float* grad;                   // [M]
  const int32_t* targets;              // [M]
  int32_t row0, v_total;
  // softmax
  const float* cinv;                   // [M]
  const float* lse;                    // [M]
  uint16_t* G;                         // [M][pitch]
  int32_t pitch, v0, V;                // first row of the chunk, rows of the head
  float* ssum;                         // [tokens][ssum_pitch]: sums of G over half a tile's rows
  int32_t ssum_pitch;
  float* ltgt;                         // [tokens]: y - lse of the target's row
  uint16_t* x;                         // lowrank: z columns of X, [M][Kc]
  // accumulate / finish
  float* dx;                           // [splits][M][Kc]
  size_t split_stride;
  int32_t Kc, first;
  void* out;                           // finish: [M][N]
  int32_t out_f32;
  float mul_acc, mul_dx;
};

struct GemmSmem {
  uint32_t stages, full, empty, accf, acce;   // addresses
  uint32_t* tmem;
  int* abort_flag;
  uint32_t* tile;
};

__device__ __forceinline__ bool aborted(int* flag) { return *reinterpret_cast<volatile int*>(flag) != 0; }

// Bounded, warp-uniform wait; on expiry raises the status and the abort flag.
__device__ __forceinline__ bool warp_wait(int* abort_flag, uint32_t bar, uint32_t parity, uint32_t* status) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  bool ok = !aborted(abort_flag) && mbar_wait(bar, parity);
  ok = __all_sync(0xffffffffu, ok);
  if (!ok && (threadIdx.x & 31) == 0 && !aborted(abort_flag)) {
    *reinterpret_cast<volatile int*>(abort_flag) = 1;
    atomicOr(status, static_cast<uint32_t>(ARCHEAD_STATUS_WAIT_TIMEOUT));
  }
  return ok;
}
__device__ __forceinline__ bool g_wait(const GemmSmem& s, uint32_t bar, uint32_t parity, uint32_t* status) {
  return warp_wait(s.abort_flag, bar, parity, status);
}

// The i-th unit of a pair: first its share of the full ones (round robin), then
// of the half ones.
struct GemmUnit {
  int m, n, k0, k1, split;
  int cols;     // 256 or 128, half of them in each CTA
};
__device__ __forceinline__ bool g_unit(const GemmParams& p, int pair, int pairs, int i, GemmUnit& r) {
  int u = pair + i * pairs, n_full_t = p.N / kGN;
  const int mine = (p.n_full - pair + pairs - 1) / pairs;
  r.cols = kGN;
  if (i >= mine) {
    const int h = pair - p.half0 + (i - mine) * p.half_pairs;
    if (pair < p.half0 || pair >= p.half0 + p.half_pairs || h >= p.n_half) return false;
    r.split = h / p.n_mt;
    r.m = h - r.split * p.n_mt;
    r.n = n_full_t;
    r.cols = kGN / 2;
  } else {
    if (p.n_half == 0 && p.N % kGN != 0) ++n_full_t;   // a last tile of more than 128 columns counts as full
    const int tiles = p.n_mt * n_full_t;
    r.split = u / tiles;
    const int rest = u - r.split * tiles;
    r.n = rest / p.n_mt;
    r.m = rest - r.n * p.n_mt;
  }
  r.k0 = static_cast<int>(static_cast<int64_t>(p.n_k) * r.split / p.splits);
  r.k1 = static_cast<int>(static_cast<int64_t>(p.n_k) * (r.split + 1) / p.splits);
  return true;
}

template <GemmMode kMode>
__device__ void g_tma_warp(const GemmParams& p, const GemmSmem& sm, const CUtensorMap* ma, const CUtensorMap* mb,
                           int pair, int pairs, int rank) {
  int s = 0, issued = 0;
  uint32_t ph = 0;
  bool ok = true;
  GemmUnit w;
  for (int i = 0; ok && g_unit(p, pair, pairs, i, w); ++i) {
    const int n0 = w.n * kGN + rank * (w.cols / 2);
    const int nb = w.cols / 128;   // 64-column boxes of B (stored [K][columns])
    const uint32_t bytes = 2 * (kGABytes + (gemm_b_mn(kMode) ? nb * 8192u : kGBBytes));   // of both CTAs
    for (int k = w.k0; k < w.k1; ++k) {
      ok = g_wait(sm, sm.empty + 8 * s, ph ^ 1u, p.status);
      if (!ok) break;
      if (elect_one()) {
        const uint32_t a = sm.stages + s * kGStageBytes, b = a + kGABytes;
        const uint32_t bar = cluster_addr(sm.full + 8 * s, 0);   // the leader's
        if (rank == 0) mbar_arrive_expect_tx(sm.full + 8 * s, bytes);
        // (z: the same h times the rows, then times what fp16 left of them)
        const int ka = kMode == kLowrank && k >= p.n_k / 2 ? k - p.n_k / 2 : k;
        tma_load_2d_pair(a, ma, ka * 64, w.m * kGM + rank * (kGM / 2), bar);
        if constexpr (!gemm_b_mn(kMode)) {
          tma_load_2d_pair(b, mb, k * 64, n0, bar);
        } else {
          for (int e = 0; e < nb; ++e) tma_load_2d_pair(b + e * 8192u, mb, n0 + 64 * e, k * 64, bar);
        }
      }
      __syncwarp();
      ++issued;
      if (++s == kGStages) {
        s = 0;
        ph ^= 1u;
      }
    }
  }
  if (!ok && rank == 0) {
    // Copies still in flight land before the pair's shared memory goes away.
    const int back = min(issued, kGStages);
    for (int i = 1; i <= back; ++i) {
      const int at = issued - i;
      mbar_wait(sm.full + 8 * (at % kGStages), (at / kGStages) & 1u);
    }
  }
}

// The whole warp walks the k-steps and one elected lane issues.  Issuing a
// tcgen05.mma costs mostly the instructions that prepare its operands, so each
// is an immediate offset from running values that advance by constants.
template <GemmMode kMode>
__device__ void g_mma_warp(const GemmParams& p, const GemmSmem& sm, uint32_t tmem_base, int pair, int pairs) {
  constexpr bool kMn = gemm_b_mn(kMode);
  constexpr uint32_t kBStep = kMn ? 128u : 2u;   // descriptor units per K = 16
  constexpr uint32_t kStep = kGStageBytes >> 4;
  constexpr uint32_t kDesc = tc_idesc_f16(kGM, kGN) | (kMn ? kTcIdescBmn : 0u);
  constexpr uint32_t kHalfDesc = tc_idesc_f16(kGM, kGN / 2) | (kMn ? kTcIdescBmn : 0u);
  const uint64_t ad0 = smem_desc_k128(sm.stages);
  const uint64_t bd0 = kMn ? smem_desc_mn128(sm.stages + kGABytes, 8192u) : smem_desc_k128(sm.stages + kGABytes);
  uint64_t a = ad0, b = bd0;
  uint32_t full = sm.full, empty = sm.empty, ph = 0, aph = 1, d = tmem_base, accf = sm.accf, acce = sm.acce;
  int s = 0;
  GemmUnit w;
  for (int i = 0; g_unit(p, pair, pairs, i, w); ++i) {
    if (!g_wait(sm, acce, aph, p.status)) return;
    tc_fence_after();
    const uint32_t idesc = w.cols == kGN ? kDesc : kHalfDesc;
    uint32_t acc = 0;
    for (int k = w.k0; k < w.k1; ++k) {
      if (!g_wait(sm, full, ph, p.status)) return;
      tc_fence_after();
      if (elect_one()) {
        tc_mma_ss_pair(d, a, b, idesc, acc);
        tc_mma_ss_pair(d, a + 2, b + kBStep, idesc, 1u);
        tc_mma_ss_pair(d, a + 4, b + 2 * kBStep, idesc, 1u);
        tc_mma_ss_pair(d, a + 6, b + 3 * kBStep, idesc, 1u);
        tc_commit_pair(empty);
      }
      __syncwarp();
      acc = 1;
      if (++s == kGStages) {
        s = 0;
        ph ^= 1u;
        a = ad0;
        b = bd0;
        full = sm.full;
        empty = sm.empty;
      } else {
        a += kStep;
        b += kStep;
        full += 8;
        empty += 8;
      }
    }
    if (elect_one()) tc_commit_pair(accf);
    __syncwarp();
    // the other accumulator
    if (d == tmem_base) {
      d += kGN;
      accf += 8;
      acce += 8;
    } else {
      d = tmem_base;
      accf = sm.accf;
      acce = sm.acce;
      aph ^= 1u;
    }
  }
}

__device__ __forceinline__ float grad_nan() { return __int_as_float(0x7fc00000); }

// Columns in pieces of 32.  A lane holds one token's row of the accumulator; G
// and dX cross the warp through a padded tile, so that a load or store touches a
// few whole row segments and not 16 bytes of 32 rows.
template <GemmMode kMode>
__device__ void g_epilogue(const GemmParams& p, const GemmSmem& sm, uint32_t tmem_base, int lane, int pair, int pairs,
                           int rank) {
  const int ew = (threadIdx.x >> 5) - 2, q = (ew + 2) & 3, half = ew >> 2;   // TMEM lane quarter, half of the columns
  uint32_t* tile = sm.tile + ew * (32 * 33);
  bool ok = true;
  GemmUnit w;
  for (int i = 0; g_unit(p, pair, pairs, i, w); ++i) {
    const uint32_t acc = i & 1;
    const int t0 = w.m * kGM + rank * (kGM / 2) + 32 * q, t = t0 + lane, n0 = w.n * kGN;
    const int ncol = min((half + 1) * (w.cols / 2), p.N - n0), nrow = min(32, p.M - t0);
    const bool live = t < p.M;
    float g = 0.f, cinv = 0.f, lse = 0.f;
    int target = -1;
    if (live && (kMode == kSoftmax || kMode == kFinish)) {
      g = p.grad[t];
      target = p.targets[t];
      if constexpr (kMode == kSoftmax) {
        cinv = p.cinv[t];
        lse = p.lse[t];
      }
    }
    if (ok) ok = g_wait(sm, sm.accf + 8 * acc, (i >> 1) & 1, p.status);
    if (ok && nrow > 0) {
      tc_fence_after();
      const uint32_t taddr = tmem_base + (static_cast<uint32_t>(32 * q) << 16) + acc * kGN;
      if constexpr (kMode == kFinish) {
        if (live && g != 0.f && (target < 0 || target >= p.v_total)) {
          g = grad_nan();
          if (w.n == 0) atomicOr(p.status, static_cast<uint32_t>(ARCHEAD_STATUS_BAD_TARGET));
        }
      }
      // probabilities come out of the exponential times 2^15
      const float k2 = cinv * 1.44269504f, l2 = lse * 1.44269504f - static_cast<float>(kGradScale);
      float ssum = 0.f;
      for (int c0 = half * (w.cols / 2); c0 < ncol; c0 += 32) {
        uint32_t r[32];
        tmem_ld_32x32b_x32(taddr + c0, r);
        tmem_ld_wait();
        if constexpr (kMode == kSoftmax) {
          // columns are vocabulary rows of the chunk; a token without a
          // gradient gets zeros (its lse and target may be anything)
          const int tl = target - p.row0 - p.v0 - n0 - c0, left = p.V - p.v0 - n0 - c0;
          const bool own = g != 0.f && tl >= 0 && tl < 32, any = __any_sync(0xffffffffu, own) != 0;
          if (any) {   // in one rounding: on a shard exp(y - lse) - 1 is taken of it
            float acc_t = 0.f;
#pragma unroll
            for (int c = 0; c < 32; ++c)
              if (c == tl) acc_t = __uint_as_float(r[c]);
            if (own) p.ltgt[t] = fmaf(acc_t, cinv, -lse);
          }
          float x[32];
#pragma unroll
          for (int c = 0; c < 32; ++c) x[c] = exp2_approx(fmaf(__uint_as_float(r[c]), k2, -l2));
#pragma unroll
          for (int c = 0; c < 32; ++c)
            if (g == 0.f) x[c] = 0.f;
          if (left < 32) {
#pragma unroll
            for (int c = 0; c < 32; ++c)
              if (c >= left) x[c] = 0.f;
          }
          if (any) {
#pragma unroll
            for (int c = 0; c < 32; ++c)
              if (c == tl) x[c] = 0.f;
          }
#pragma unroll
          for (int c = 0; c < 32; c += 4) ssum += (x[c] + x[c + 1]) + (x[c + 2] + x[c + 3]);
#pragma unroll
          for (int c = 0; c < 32; c += 2) tile[lane * 17 + c / 2] = pack_half2(x[c], x[c + 1]);
          __syncwarp();
          // 16-byte runs: four of a row's 64 bytes, eight rows at a time
#pragma unroll
          for (int it = 0; it < 4; ++it) {
            const int row = 8 * it + (lane >> 2), v = lane & 3;
            if (row < nrow && c0 + 8 * v < ncol) {
              const uint32_t* src = tile + row * 17 + 4 * v;
              *reinterpret_cast<uint4*>(p.G + static_cast<size_t>(t0 + row) * p.pitch + n0 + c0 + 8 * v) =
                  make_uint4(src[0], src[1], src[2], src[3]);
            }
          }
        } else if constexpr (kMode == kLowrank) {
          // z columns of X
          if (live) {
            uint4* dst = reinterpret_cast<uint4*>(p.x + static_cast<size_t>(t) * p.Kc + n0 + c0);
#pragma unroll
            for (int v = 0; v < 4; ++v) {
              uint32_t o[4];
#pragma unroll
              for (int e = 0; e < 4; ++e)
                o[e] = pack_half2(__uint_as_float(r[8 * v + 2 * e]) * p.mul_acc, __uint_as_float(r[8 * v + 2 * e + 1]) * p.mul_acc);
              dst[v] = make_uint4(o[0], o[1], o[2], o[3]);
            }
          }
        } else if constexpr (kMode == kAccumulate) {
          const bool none = w.k0 == w.k1;   // a split without rows in a short chunk
#pragma unroll
          for (int c = 0; c < 32; ++c) tile[lane * 33 + c] = none ? 0u : r[c];
          __syncwarp();
          float* dst = p.dx + w.split * p.split_stride + static_cast<size_t>(t0) * p.Kc + n0 + c0 + lane;
          float old[32];
          if (!p.first) {
#pragma unroll
            for (int row = 0; row < 32; ++row) old[row] = row < nrow ? dst[static_cast<size_t>(row) * p.Kc] : 0.f;
          }
#pragma unroll
          for (int row = 0; row < 32; ++row) {
            if (row < nrow) {
              const float x = __uint_as_float(tile[row * 33 + lane]);
              dst[static_cast<size_t>(row) * p.Kc] = p.first ? x : old[row] + x;
            }
          }
        } else {
          if (live) {
            // row segments of 128 bytes and more, lane by lane (through the tile
            // this took half as long again: both ways cross it)
            float x[32];
            const float4* src = reinterpret_cast<const float4*>(p.dx + static_cast<size_t>(t) * p.Kc + n0 + c0);
#pragma unroll
            for (int c = 0; c < 32; ++c) x[c] = p.n_k > 0 ? __uint_as_float(r[c]) * p.mul_acc : 0.f;
#pragma unroll
            for (int v = 0; v < 8; ++v) {
              const float4 y = src[v];
              const float z[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
              for (int e = 0; e < 4; ++e) {   // dX is in the operand order
                const int at = 4 * v + e, c = (at & 16) + tc_kcol(at & 15);
                x[c] = fmaf(z[e], p.mul_dx, x[c]);
              }
            }
#pragma unroll
            for (int c = 0; c < 32; ++c) x[c] = g == 0.f ? 0.f : x[c] * g;
            if (p.out_f32) {
              float4* dst = reinterpret_cast<float4*>(static_cast<float*>(p.out) + static_cast<size_t>(t) * p.N + n0 + c0);
#pragma unroll
              for (int v = 0; v < 8; ++v) dst[v] = make_float4(x[4 * v], x[4 * v + 1], x[4 * v + 2], x[4 * v + 3]);
            } else {
              uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + static_cast<size_t>(t) * p.N + n0 + c0);
#pragma unroll
              for (int v = 0; v < 4; ++v) {
                uint32_t o[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const __nv_bfloat162 b = __floats2bfloat162_rn(x[8 * v + 2 * e], x[8 * v + 2 * e + 1]);
                  o[e] = *reinterpret_cast<const uint32_t*>(&b);
                }
                dst[v] = make_uint4(o[0], o[1], o[2], o[3]);
              }
            }
          }
        }
        __syncwarp();
      }
      if (kMode == kSoftmax && live)
        p.ssum[static_cast<size_t>(t) * p.ssum_pitch + 2 * (p.v0 / kGN + w.n) + half] = ssum * (1.f / (1 << kGradScale));
      tc_fence_before();
    }
    __syncwarp();
    if (lane == 0) mbar_arrive_cluster(cluster_addr(sm.acce + 8 * acc, 0));
  }
}

template <GemmMode kMode>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kGWarps * 32, 1)
    grad_gemm_kernel(const GemmParams p, const __grid_constant__ CUtensorMap ma, const __grid_constant__ CUtensorMap mb) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  GemmSmem sm;
  sm.stages = smem_addr(base);
  sm.full = sm.stages + kGBarOff;
  sm.empty = sm.full + 8 * kGStages;
  sm.accf = sm.empty + 8 * kGStages;
  sm.acce = sm.accf + 16;
  sm.tmem = reinterpret_cast<uint32_t*>(base + kGBarOff + 16 * kGStages + 32);
  sm.abort_flag = reinterpret_cast<int*>(sm.tmem + 1);
  sm.tile = reinterpret_cast<uint32_t*>(base + kGTileOff);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int pair = blockIdx.x / 2, pairs = gridDim.x / 2, rank = blockIdx.x & 1;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kGStages; ++s) {
      mbar_init(sm.full + 8 * s, 1);
      mbar_init(sm.empty + 8 * s, 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(sm.accf + 8 * a, 1);
      mbar_init(sm.acce + 8 * a, 2 * kGEpi);   // the epilogue warps of both CTAs
    }
    *sm.abort_flag = 0;
    mbar_fence_init();
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_addr(sm.tmem), kGTmem);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();   // both CTAs' barriers are set up
  tc_fence_after();
  const uint32_t tmem_base = *sm.tmem;
  grid_dependency_wait();
  grid_launch_dependents();
  if (warp == 0) g_tma_warp<kMode>(p, sm, &ma, &mb, pair, pairs, rank);
  else if (warp == 1) {
    if (rank == 0) g_mma_warp<kMode>(p, sm, tmem_base, pair, pairs);
  } else g_epilogue<kMode>(p, sm, tmem_base, lane, pair, pairs, rank);
  tc_fence_before();
  __syncthreads();
  cluster_sync();   // nothing of the pair still reads, writes or signals the other CTA
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, kGTmem);
  }
}

template <GemmMode kMode>
cudaError_t launch_gemm(GemmParams& p, const CUtensorMap& ma, const CUtensorMap& mb, int num_sms, cudaStream_t stream) {
  const int rest = p.N % kGN, pairs = num_sms / 2;
  const bool half = rest != 0 && rest <= kGN / 2;
  p.n_mt = (p.M + kGM - 1) / kGM;
  p.n_full = p.splits * p.n_mt * (p.N / kGN + (rest != 0 && !half ? 1 : 0));
  p.n_half = half ? p.splits * p.n_mt : 0;
  const int grid = std::min(p.n_full + p.n_half, pairs);
  // The half units go to the pairs that the last round of full ones leaves idle,
  // two each, if they fit there; else to all.
  p.half0 = p.n_full % grid;
  p.half_pairs = grid - p.half0;
  if (p.n_half > 2 * p.half_pairs) {
    p.half0 = 0;
    p.half_pairs = grid;
  }
  return launch_after(grad_gemm_kernel<kMode>, dim3(2 * grid), kGWarps * 32, kGSmem, stream, p, ma, mb);
}

// ------------------------------------------------------- few tokens: G, G W~
// The order in which gw_kernel loads G: pieces of 32 tokens x 128 rows of the head
// (8 KB), in a piece 16-byte runs of 8 rows, the 32 tokens of a run side by side, so
// that a warp's load of one run per lane (= token) is 512 contiguous bytes.  (Read
// row by row, 16 bytes of 32 rows per load, G cost gw_kernel 37 of 161 us at 64
// tokens.)  The tensor-core forward writes it from its epilogue; for the few tokens
// of the decode kernel g_kernel makes it from the logits (fp32 [T][V]): one block
// per piece, one warp per token, with the token's sum of G and, where the target is
// one of the rows, its y - lse; the piece's other tokens are zeros.
struct GParams {
  const float* y;
  const float* lse;
  const float* grad;
  const int32_t* targets;
  uint4* G;                   // [k-step][16][32]
  float* ssum;                // [T][ssum_pitch], one per k-step
  float* ltgt;                // [T]
  int32_t T, V, row0, ssum_pitch;   // T <= kDecodeTokens
};
constexpr int kGwRows = 128, kGwMt = kGwRows / kMT;   // rows and m-tiles of a k-step
static_assert(kTcMinTokens <= kDecodeTokens + 1, "a token per warp of g_kernel");
__global__ void __launch_bounds__(32 * kDecodeTokens) g_kernel(const GParams p) {
  __shared__ __align__(16) uint16_t piece[kGwRows / 8][kDecodeTokens][8];
  grid_dependency_wait();
  grid_launch_dependents();
  const int t = threadIdx.x >> 5, lane = threadIdx.x & 31, v0 = blockIdx.x * kGwRows;
  const bool live = t < p.T && p.grad[t] != 0.f;   // (its lse and target may be anything otherwise)
  const float lse = live ? p.lse[t] : 0.f;
  const int target = live ? p.targets[t] - p.row0 : -1;
  const float* y = p.y + static_cast<size_t>(t) * p.V;
  float sum = 0.f;
#pragma unroll
  for (int e = 0; e < kGwRows / 32; ++e) {
    const int v = v0 + 32 * e + lane;
    float x = live && v < p.V ? __expf(y[v] - lse) : 0.f;
    if (live && v == target) {
      if (v < p.V) p.ltgt[t] = y[v] - lse;
      x = 0.f;
    }
    sum += x;
    piece[4 * e + (lane >> 3)][t][lane & 7] = __half_as_ushort(__float2half_rn(x * static_cast<float>(1 << kGradScale)));
  }
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0 && t < p.T) p.ssum[static_cast<size_t>(t) * p.ssum_pitch + blockIdx.x] = sum;
  __syncthreads();
  uint4* dst = p.G + static_cast<size_t>(blockIdx.x) * (kGwRows / 8 * 32);
  for (int i = threadIdx.x; i < kGwRows / 8 * 32; i += blockDim.x)
    dst[i] = lane < kDecodeTokens ? *reinterpret_cast<const uint4*>(piece[i >> 5][lane]) : make_uint4(0u, 0u, 0u, 0u);
}

// dX = G W~ for up to 128 tokens, the packed rows dequantised on the way:
// D[128 tokens x 256 columns of W~] in TMEM, A = 128 columns of G in TMEM, B = a
// 128-row x 256-column tile of W~ as the dequantising warps leave it in shared
// memory (rows of 64 columns, so MN-major: the transpose costs nothing).  A CTA
// owns one block of 256 columns and a range of vocabulary rows, writes one
// partial dX, and dx_kernel adds the partials of a column's CTAs in order.
//   warps 0-15  dequantise: set w / 8 takes every second tile, a warp one 16-row
//               m-tile of it, its packed bytes loaded one of its tiles early
//               straight into registers (one 16-byte load per lane and 64
//               columns: nothing to copy, wait for or re-read).
//   warps 16-19 G: the 32 tokens of their TMEM lane quarter, a k-step ahead in
//               registers; warp 19 also issues the MMAs (as a duty of warps 0-15
//               G cost the schedulers of the first quarters two thirds more
//               instructions than the others).
// Afterwards warps 0-15 write the accumulator.
// What set the shape: the tensor cores read shared-memory operands at about 64
// bytes a clock, so G sits in TMEM (with both operands in shared memory a tile
// took nearly twice its clocks of math); a barrier round (wait, fence, commit)
// and the issue of an MMA cost the MMA warp about 450 and 48 clocks, so a tile is
// 8 MMAs of 256 columns (with 128 columns, 840 clocks a tile for 512 of math).
constexpr int kGwWarps = 20, kGwSets = 2, kGwStages = 3, kGwBufs = 4;
constexpr int kGwMma = kGwWarps - 1;                  // the warp that issues the MMAs
constexpr uint32_t kGwHalf = kGwRows * 128;           // 128 rows x 64 columns of fp16
constexpr uint32_t kGwTile = kGwChunks * kGwHalf;
constexpr uint32_t kGwBarOff = kGwStages * kGwTile;
constexpr uint32_t kGwSmem = kGwBarOff + 512 + 1024;

struct GwParams {
  DequantParams rows;
  const uint4* G;              // in that order, zeros past the last row of the head
  int32_t T;
  int32_t n_mtiles, nk;        // k-steps of kGwRows rows
  int32_t chunks;              // 64-column chunks in all
  GwSplits splits;
  float* dx;                   // [split][T][Kc]
  size_t split_stride;
  uint32_t* status;
};

// Packed bytes of two 64-column chunks of one m-tile, as one lane holds them:
// codes; fifth bits (core: x.x) or the second half (correction); scale pairs.
// GP: scale groups per 128 residual columns (8, 4, 2; 1 for groups of 128 and more).
template <int GP>
struct RawPair {
  static constexpr int kPer = GP < 2 ? 1 : GP / 2;   // groups per chunk
  uint4 c[2], x[2];
  uint32_t s[2 * kPer];
};

__device__ __forceinline__ void sts128(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}

// A chunk's 16 rows x 64 columns into the swizzled tile: lane (gr, cc) holds 16
// columns of rows gr and gr + 8, stored as columns 16 cc .. 16 cc + 15 (32
// contiguous bytes of each row; the order is undone when dX is written).
template <int GP>
__device__ __forceinline__ void store_chunk(const DequantParams& p, const RawPair<GP>& r, int ks, int ch, uint32_t lo, uint32_t hi) {
  constexpr int kPer = RawPair<GP>::kPer;
  uint32_t a[4][4], s0[4], s1[4];
  if (ks < p.n_res) {
    const uint32_t w[4] = {r.c[ch].x, r.c[ch].y, r.c[ch].z, r.c[ch].w};
#pragma unroll
    for (int st = 0; st < 4; ++st) {
      unpack_int4_signed(w[st], a[st]);
      if (st % (4 / kPer) == 0) scales_of(r.s[ch * kPer + st * kPer / 4], p.sc_res, s0[st], s1[st]);
      else s0[st] = s0[st - 1], s1[st] = s1[st - 1];
    }
  } else {
    if (ks < p.n_res + p.n_L) {
      unpack_int5_signed<0>(r.c[ch].x, r.x[ch].x, a[0]);
      unpack_int5_signed<1>(r.c[ch].y, r.x[ch].x, a[1]);
      unpack_int5_signed<2>(r.c[ch].z, r.x[ch].x, a[2]);
      unpack_int5_signed<3>(r.c[ch].w, r.x[ch].x, a[3]);
      scales_of(r.s[ch * kPer], p.sc_L, s0[0], s1[0]);
    } else {
      unpack_int8_signed(r.c[ch].x, r.c[ch].y, a[0]);
      unpack_int8_signed(r.c[ch].z, r.c[ch].w, a[1]);
      if (2 * (ks - p.n_res - p.n_L) + 1 < p.n_A) {
        unpack_int8_signed(r.x[ch].x, r.x[ch].y, a[2]);
        unpack_int8_signed(r.x[ch].z, r.x[ch].w, a[3]);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) a[2][i] = a[3][i] = 0u;
      }
      scales_of(r.s[ch * kPer], p.sc_A, s0[0], s1[0]);
    }
#pragma unroll
    for (int st = 1; st < 4; ++st) s0[st] = s0[0], s1[st] = s1[0];
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t at = (h ? hi : lo) + ch * kGwHalf;
    const int i = 2 * h, j = 2 * h + 1;
    sts128(at, hmul2_bits(a[i][0], s0[i]), hmul2_bits(a[i][2], s0[i]), hmul2_bits(a[j][0], s0[j]), hmul2_bits(a[j][2], s0[j]));
    sts128(at + 1024u, hmul2_bits(a[i][1], s1[i]), hmul2_bits(a[i][3], s1[i]), hmul2_bits(a[j][1], s1[j]),
           hmul2_bits(a[j][3], s1[j]));
  }
}

// The common case, both chunks residual.
template <int GP>
__device__ __forceinline__ void store_pair(const RawPair<GP>& r, float sc, uint32_t lo, uint32_t hi) {
  uint32_t s0 = 0, s1 = 0;
#pragma unroll
  for (int ch = 0; ch < 2; ++ch) {
    const uint32_t w[4] = {r.c[ch].x, r.c[ch].y, r.c[ch].z, r.c[ch].w};
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t up[4], dn[4];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int st = 2 * h + e, step = 4 * ch + st;
        if (step * GP % 8 == 0) scales_of(r.s[GP < 2 ? 0 : step * GP / 8], sc, s0, s1);
        uint32_t a[4];
        unpack_int4_signed(w[st], a);
        up[2 * e] = hmul2_bits(a[0], s0);
        up[2 * e + 1] = hmul2_bits(a[2], s0);
        dn[2 * e] = hmul2_bits(a[1], s1);
        dn[2 * e + 1] = hmul2_bits(a[3], s1);
      }
      const uint32_t at = (h ? hi : lo) + ch * kGwHalf;
      sts128(at, up[0], up[1], up[2], up[3]);
      sts128(at + 1024u, dn[0], dn[1], dn[2], dn[3]);
    }
  }
}

template <int GP>
__global__ void __launch_bounds__(kGwWarps * 32, 1) gw_kernel(const GwParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t tiles = smem_addr(base);
  const uint32_t wfull = tiles + kGwBarOff, wempty = wfull + 8 * kGwStages, gfull = wempty + 8 * kGwStages,
                 gempty = gfull + 8 * kGwBufs, done = gempty + 8 * kGwBufs;
  uint32_t* tmem = reinterpret_cast<uint32_t*>(base + kGwBarOff + 16 * kGwStages + 16 * kGwBufs + 8);
  int* flag = reinterpret_cast<int*>(tmem + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kGwStages; ++s) {
      mbar_init(wfull + 8 * s, 8);
      mbar_init(wempty + 8 * s, 1);
    }
    for (int s = 0; s < kGwBufs; ++s) {
      mbar_init(gfull + 8 * s, (p.T + 31) / 32);
      mbar_init(gempty + 8 * s, 1);
    }
    mbar_init(done, 1);
    *flag = 0;
    mbar_fence_init();
  }
  if (warp == kGwMma) {
    tmem_alloc(smem_addr(tmem), kGTmem);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *tmem;
  grid_dependency_wait();
  grid_launch_dependents();

  // This CTA: column block, its chunks, its k-steps.
  const GwSplits& g = p.splits;
  int block, split = blockIdx.x;
  if (split < g.res * g.s_res) {
    block = split / g.s_res;
    split -= block * g.s_res;
  } else {
    split -= g.res * g.s_res;
    block = min(split / g.s_rest, g.rest - 1);
    split -= block * g.s_rest;
    block += g.res;
  }
  const int splits = gw_splits(g, block);
  const int c0 = block * kGwChunks, nc = min(kGwChunks, p.chunks - c0);
  const int k0 = static_cast<int>(static_cast<int64_t>(p.nk) * split / splits);
  const int k1 = static_cast<int>(static_cast<int64_t>(p.nk) * (split + 1) / splits);
  const int steps = k1 - k0;

  if (warp < 16) {
    const int set = warp >> 3, j = warp & 7;
    const int gr = lane >> 2, cc = lane & 3;
    // byte offsets of this lane inside a tile: row 16 j + gr, 16-byte pieces 2 cc and 2 cc + 1 (swizzled by the row)
    const uint32_t row = tiles + static_cast<uint32_t>((16 * j + gr) * 128);
    const uint32_t o_lo = row + static_cast<uint32_t>(((2 * cc) ^ gr) * 16);
    const uint32_t o_hi = row + static_cast<uint32_t>(((2 * cc + 1) ^ gr) * 16);

    // The next tile's packed bytes, two pairs of chunks.  Every load has its own
    // register and at most a predicate: a load under a branch that others share a
    // register with would have to land before the branch ends.
    constexpr int kPer = RawPair<GP>::kPer;
    RawPair<GP> raw[2];
    uint32_t code_off[kGwChunks], scale_off[kGwChunks];
#pragma unroll
    for (int ch = 0; ch < kGwChunks; ++ch) {
      const int ks = min(c0 + ch, p.chunks - 1), kc = ks - p.rows.n_res, ka = 2 * (kc - p.rows.n_L);
      code_off[ch] = lane * 16 + (kc < 0 ? p.rows.off_res + ks * kResChunkBytes
                                         : ka < 0 ? p.rows.off_Lnib + kc * kLNibChunkBytes : p.rows.off_A + ka * kAChunkBytes);
      scale_off[ch] = gr * 4 + (kc < 0 ? p.rows.off_sres + ((ks * 64) >> p.rows.g_log2) * kSresGroupBytes
                                       : ka < 0 ? p.rows.off_sL : p.rows.off_sA);
    }
    int pk = k0 + set;
    const uint8_t* pm = p.rows.mtiles + static_cast<size_t>(kGwMt * pk + j) * p.rows.mblk_bytes;
    const size_t next_k = static_cast<size_t>(kGwSets * kGwMt) * p.rows.mblk_bytes;
    auto load = [&](RawPair<GP>& r, int i) {
      // (past the end of the rows: any valid bytes)
      const uint8_t* m = pk < k1 && kGwMt * pk + j < p.n_mtiles ? pm : p.rows.mtiles;
#pragma unroll
      for (int ch = 0; ch < 2; ++ch) {
        const int e = 2 * i + ch, ks = min(c0 + e, p.chunks - 1), kc = ks - p.rows.n_res, ka = 2 * (kc - p.rows.n_L);
        r.c[ch] = ldg128(m + code_off[e]);
#pragma unroll
        for (int q = 0; q < kPer; ++q) r.s[ch * kPer + q] = ldg32(m + scale_off[e] + (kc < 0 ? q * kSresGroupBytes : 0));
        if (kc >= 0 && ka < 0) r.x[ch].x = ldg32(m + p.rows.off_Lhi + (code_off[e] - p.rows.off_Lnib) / 4);
        if (ka >= 0 && ka + 1 < p.rows.n_A) r.x[ch] = ldg128(m + code_off[e] + kAChunkBytes);
      }
    };
    load(raw[0], 0);
    load(raw[1], 1);
    int s = set;
    uint32_t ph = 1;
    for (int k = k0 + set; k < k1; k += kGwSets) {
      if (!warp_wait(flag, wempty + 8 * s, ph, p.status)) break;
      pk += kGwSets;
      pm += next_k;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t lo = o_lo + s * kGwTile + 2 * i * kGwHalf, hi = o_hi + s * kGwTile + 2 * i * kGwHalf;
        const int c = c0 + 2 * i;
        if (kGwMt * k + j >= p.n_mtiles) {   // rows past the last m-tile
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            sts128(lo + h * kGwHalf, 0u, 0u, 0u, 0u);
            sts128(lo + h * kGwHalf + 1024u, 0u, 0u, 0u, 0u);
            sts128(hi + h * kGwHalf, 0u, 0u, 0u, 0u);
            sts128(hi + h * kGwHalf + 1024u, 0u, 0u, 0u, 0u);
          }
        } else if (c + 1 < p.rows.n_res) {
          store_pair<GP>(raw[i], p.rows.sc_res, lo, hi);
        } else {
          if (c < p.chunks) store_chunk<GP>(p.rows, raw[i], c, 0, lo, hi);
          if (c + 1 < p.chunks) store_chunk<GP>(p.rows, raw[i], c + 1, 1, lo, hi);
        }
        load(raw[i], i);
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive(wfull + 8 * s);
      s += kGwSets;
      if (s >= kGwStages) {
        s -= kGwStages;
        ph ^= 1u;
      }
    }
    // The accumulator: lane quarter w % 4 (tokens), every fourth piece of 32
    // columns.  A lane's 32 columns are two runs of the dequantising lanes' 16:
    // float4 (h, st) of them is operand columns 16 st + 4 (2 half + h) of the chunk.
    const int quarter = warp & 3;
    if (warp_wait(flag, done, 0u, p.status) && 32 * quarter < p.T) {
      tc_fence_after();
      const int t = 32 * quarter + lane;
      float* dx = p.dx + split * p.split_stride + static_cast<size_t>(t) * p.rows.Kc + c0 * 64;
      for (int piece = warp >> 2; piece < 2 * nc; piece += 4) {
        uint32_t r[32];
        tmem_ld_32x32b_x32(tbase + (static_cast<uint32_t>(32 * quarter) << 16) + 32 * piece, r);
        tmem_ld_wait();
        if (t < p.T) {
          float* dst = dx + (piece >> 1) * 64 + (piece & 1) * 8;
#pragma unroll
          for (int st = 0; st < 4; ++st)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int i = 16 * h + 4 * st;
              *reinterpret_cast<float4*>(dst + 16 * st + 4 * h) =
                  make_float4(__uint_as_float(r[i]), __uint_as_float(r[i + 1]), __uint_as_float(r[i + 2]), __uint_as_float(r[i + 3]));
            }
        }
        __syncwarp();
      }
      tc_fence_before();
    }
  } else {
    // G of this warp's 32 tokens: 128 rows of a k-step are 16 runs of 8, one
    // 16-byte load each, 64 TMEM columns.
    const int q = warp & 3;
    const bool has_g = 32 * q < p.T;
    const int nq = (p.T + 31) / 32;
    const uint4* gsrc = p.G + (static_cast<size_t>(k0) * nq + q) * (kGwRows / 8 * 32) + lane;
    const uint32_t gdst = tbase + (static_cast<uint32_t>(32 * q) << 16) + kGwCols;
    int gi = 0;
    uint32_t gv[4][16];
    auto g_load = [&]() {
      if (gi < steps) {
        const uint4* src = gsrc + static_cast<size_t>(gi) * nq * (kGwRows / 8 * 32);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const uint4 x = __ldg(src + 32 * i);
          uint32_t* v = &gv[i >> 2][4 * (i & 3)];
          v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
        }
      }
    };
    auto g_put = [&]() {   // k-step gi
      const int s = gi & (kGwBufs - 1);
      if (!warp_wait(flag, gempty + 8 * s, ((gi / kGwBufs) & 1) ^ 1, p.status)) return false;
      tc_fence_after();
#pragma unroll
      for (int i = 0; i < 4; ++i) tmem_st_32x32b_x16(gdst + (kGwRows / 2) * s + 16 * i, gv[i]);
      ++gi;
      g_load();
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(gfull + 8 * s);
      return true;
    };
    if (has_g) g_load();
    if (warp != kGwMma) {
      if (has_g)
        while (gi < steps && g_put()) {}
    } else {
      // (running values and immediate offsets only, as in g_mma_warp)
      const uint64_t bd0 = smem_desc_mn128(tiles, kGwHalf);
      const uint32_t idesc = tc_idesc_f16(128, 64 * nc) | kTcIdescBmn;
      const uint32_t a0 = tbase + kGwCols;
      uint64_t bd = bd0;
      uint32_t ad = a0, wf = wfull, we = wempty, wph = 0, gf = gfull, ge = gempty, gph = 0;
      uint32_t acc = 0;
      bool ok = !has_g || g_put();
      for (int k = 0; k < steps && ok; ++k) {
        ok = warp_wait(flag, gf, gph, p.status) && warp_wait(flag, wf, wph, p.status);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
          tc_mma_ts(tbase, ad, bd, idesc, acc);
          tc_mma_ts(tbase, ad + 8, bd + 128, idesc, 1u);
          tc_mma_ts(tbase, ad + 16, bd + 256, idesc, 1u);
          tc_mma_ts(tbase, ad + 24, bd + 384, idesc, 1u);
          tc_mma_ts(tbase, ad + 32, bd + 512, idesc, 1u);
          tc_mma_ts(tbase, ad + 40, bd + 640, idesc, 1u);
          tc_mma_ts(tbase, ad + 48, bd + 768, idesc, 1u);
          tc_mma_ts(tbase, ad + 56, bd + 896, idesc, 1u);
          tc_commit(we);
          tc_commit(ge);
        }
        __syncwarp();
        acc = 1;
        bd += kGwTile >> 4;
        wf += 8;
        we += 8;
        if (wf == wempty) {   // the ring wraps
          bd = bd0;
          wf = wfull;
          we = wempty;
          wph ^= 1u;
        }
        ad += kGwRows / 2;
        gf += 8;
        ge += 8;
        if (gf == gempty) {
          ad = a0;
          gf = gfull;
          ge = gempty;
          gph ^= 1u;
        }
        // its own share of the next k-step, when this one's MMAs are queued
        if (has_g && gi < steps) ok = g_put();
      }
      if (ok && elect_one()) tc_commit(done);
      __syncwarp();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kGwMma) {
    tc_fence_after();
    tmem_dealloc(tbase, kGTmem);
  }
}

// dh of up to kDecodeTokens tokens from dX_res + dz [s_R R | s_B B], the int8
// codes as they are.  A block owns 64 columns; 32 half warps take every 32nd row,
// 8 rows in flight, the first ones before the wait (they are weights), and their
// sums meet in shared memory in a fixed order.  The tensor-core product's set-up
// and its fp16 rows of R and B are most of its time here: the whole gradient of
// one token of 32003 x 2048 took 70.7 us with it, 64.8 so; of 8000 x 512 45.2 and
// 38.4; 8 tokens of 8000 x 512 55.5 and 50.6.
struct FinishFewParams {
  const int8_t* R;
  const uint16_t* s_R;
  const int8_t* B;
  const uint16_t* s_B;
  const uint16_t* dz;         // [T][Kz], operand order
  const float* dx;            // [T][Kc], operand order
  const float* grad;
  const int32_t* targets;
  void* out;
  uint32_t* status;
  int32_t T, d, Kc, Kz, rcp, rrp, g_B, v_total, out_f32;
  float mul_c, mul_r, mul_dx;
};
constexpr int kFinishChunk = 512, kFinishRows = 8;   // dz columns in shared memory; rows in flight

// Four columns of the low-rank row at position e of the operand order.
__device__ __forceinline__ float4 lowrank_row4(const FinishFewParams& p, int e, int j) {
  const int k = (e & ~15) + tc_kcol(e & 15);
  const bool core = k < p.rcp;
  const int r = core ? k : k - p.rcp;
  if (e >= p.Kz || (!core && r >= p.rrp)) return make_float4(0.f, 0.f, 0.f, 0.f);
  const char4 c = __ldg(reinterpret_cast<const char4*>((core ? p.R : p.B) + static_cast<size_t>(r) * p.d + j));
  float4 s;
  if (core) {
    s.x = s.y = s.z = s.w = __half2float(__ushort_as_half(__ldg(p.s_R + r))) * p.mul_c;
  } else {
    const uint16_t* sb = p.s_B + static_cast<size_t>(r) * (p.d / p.g_B);
    const auto at = [&](int col) { return __half2float(__ushort_as_half(__ldg(sb + col / p.g_B))) * p.mul_r; };
    s.x = at(j);
    s.y = s.z = s.w = s.x;
    if (p.g_B % 4 != 0) {
      s.y = at(j + 1);
      s.z = at(j + 2);
      s.w = at(j + 3);
    }
  }
  return make_float4(c.x * s.x, c.y * s.y, c.z * s.z, c.w * s.w);
}

template <int TT>
__global__ void __launch_bounds__(512) finish_few_kernel(const FinishFewParams p) {
  __shared__ __align__(16) float sh[16 * TT * 64];     // dz of a chunk, then the warps' sums
  static_assert(kFinishChunk <= 16 * 64, "dz of a chunk fits");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, slot = threadIdx.x >> 4;
  const int j0 = blockIdx.x * 64, j = j0 + 4 * (lane & 15);
  // this thread's result: token t, column j0 + col
  const int t = threadIdx.x >> 6, col = threadIdx.x & 63;
  const bool mine = t < TT && t < p.T;
  const float g = mine ? p.grad[t] : 0.f;
  const int target = mine ? p.targets[t] : -1;
  float4 w[kFinishRows], next[kFinishRows];
#pragma unroll
  for (int i = 0; i < kFinishRows; ++i) w[i] = lowrank_row4(p, slot + 32 * i, j);
  grid_dependency_wait();
  const float res = mine ? p.dx[static_cast<size_t>(t) * p.Kc + j0 + (col & ~15) + tc_kpos(col & 15)] : 0.f;
  float acc[TT][4] = {};
  for (int c0 = 0; c0 < p.Kz; c0 += kFinishChunk) {
    const int n = min(kFinishChunk, p.Kz - c0);
    if (c0 > 0) __syncthreads();
#pragma unroll
    for (int tt = 0; tt < TT; ++tt)
      for (int e = threadIdx.x; e < n; e += 512)
        sh[e * TT + tt] = tt < p.T ? __half2float(__ushort_as_half(p.dz[static_cast<size_t>(tt) * p.Kz + c0 + e])) : 0.f;
    __syncthreads();
    for (int b = 0; b < n; b += 32 * kFinishRows) {
#pragma unroll
      for (int i = 0; i < kFinishRows; ++i) next[i] = lowrank_row4(p, c0 + b + slot + 32 * (kFinishRows + i), j);
#pragma unroll
      for (int i = 0; i < kFinishRows; ++i) {
        const int e = b + slot + 32 * i;
        if (e < n) {
#pragma unroll
          for (int tt = 0; tt < TT; ++tt) {
            const float z = sh[e * TT + tt];
            acc[tt][0] = fmaf(z, w[i].x, acc[tt][0]);
            acc[tt][1] = fmaf(z, w[i].y, acc[tt][1]);
            acc[tt][2] = fmaf(z, w[i].z, acc[tt][2]);
            acc[tt][3] = fmaf(z, w[i].w, acc[tt][3]);
          }
        }
        w[i] = next[i];
      }
    }
  }
  __syncthreads();
#pragma unroll
  for (int tt = 0; tt < TT; ++tt) {
#pragma unroll
    for (int c = 0; c < 4; ++c) acc[tt][c] += __shfl_xor_sync(0xffffffffu, acc[tt][c], 16);
    if (lane < 16)
      *reinterpret_cast<float4*>(sh + (warp * TT + tt) * 64 + 4 * lane) =
          make_float4(acc[tt][0], acc[tt][1], acc[tt][2], acc[tt][3]);
  }
  __syncthreads();
  if (!mine) return;
  float x = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) x += sh[(i * TT + t) * 64 + col];
  x = g == 0.f ? 0.f : fmaf(res, p.mul_dx, x) * g;
  if (g != 0.f && (target < 0 || target >= p.v_total)) {
    x = grad_nan();
    if (j0 + col == 0) atomicOr(p.status, static_cast<uint32_t>(ARCHEAD_STATUS_BAD_TARGET));
  }
  const size_t at = static_cast<size_t>(t) * p.d + j0 + col;
  if (p.out_f32) static_cast<float*>(p.out)[at] = x;
  else static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16(x);
}

// -------------------------------------------------------------------- host
// Few tokens: the packed rows are dequantised inside the second product,
// kFewPass tokens a pass over the head.  One such pass beats the chunks of W~ at
// any head size; two do while the fp16 rows of the head are more than one chunk
// (151936 x 4096: 0.78 ms at 129 tokens, 1.0 at 256, against 1.1; with the rows
// in one chunk, 65531 x 1024: 160 to 198 us against 142).
constexpr int kFewPass = 128;

// Many tokens of a whole head with low-rank rows: z by a product with the rows of R and B
// (pairs of fp16 rows) from this many tokens on, below by the activation kernel,
// which has one launch less (whole gradient, 151936 x 4096: 1024 tokens 2.94
// against 2.97 ms, 4096 tokens 9.65 against 9.83 ms; 32003 x 2048: 1024 tokens 374
// against 371 us, 4096 1179 against 1225).
constexpr int kOwnXTokens = 1024;

// Work split of gw_kernel.
struct GwPlan {
  int chunks, nk, grid;
  GwSplits s;
};
GwPlan gw_plan(const archead_handle& h) {
  GwPlan g{};
  g.chunks = tc_kc(h.L) / 64;
  g.nk = (h.L.n_mtiles + kGwMt - 1) / kGwMt;
  const int blocks = (g.chunks + kGwChunks - 1) / kGwChunks, last = g.chunks - (blocks - 1) * kGwChunks;
  g.s.res = h.L.n_res / kGwChunks;
  g.s.rest = blocks - g.s.res;
  // Row splits in proportion to a block's cost, so that the CTAs end together
  // (measured at 151936 x 4096, 64 tokens: 0.91 us a tile of residual columns,
  // 1.2 of INT5 codes, which take more unpacking, 0.72 of a single chunk, which
  // has the same barriers).
  const double rest = 1.25, tail = g.s.rest > 0 ? 0.65 + 0.15 * last : 0.0;
  const double total = g.s.res + rest * std::max(0, g.s.rest - 1) + tail;
  const auto share = [&](double cost) { return std::max(1, std::min(g.nk, static_cast<int>(h.num_sms * cost / total))); };
  g.s.s_res = share(1.0);
  g.s.s_rest = share(rest);
  g.s.s_last = share(tail);
  g.grid = g.s.res * g.s.s_res + (g.s.rest > 0 ? (g.s.rest - 1) * g.s.s_rest + g.s.s_last : 0);
  return g;
}

// K splits (of a chunk's rows) of the accumulation: the fewest that keep the
// pairs busy.  Rounds of units over the pairs, a last column tile of 128 or fewer
// being half a unit, per split; each further split has to save 3% for its
// partial dX.
int accumulate_splits(int tokens, int Kc, int chunk, int pairs) {
  const int mt = (tokens + kGM - 1) / kGM, rest = Kc % kGN;
  const bool half = rest != 0 && rest <= kGN / 2;
  const int full1 = mt * (Kc / kGN + (rest != 0 && !half ? 1 : 0)), half1 = half ? mt : 0;
  int best = 1;
  double best_cost = 1e30;
  for (int s = 1; s <= 8 && s * 256 <= chunk; ++s) {
    const int full = s * full1, rounds = (full + pairs - 1) / pairs, idle = rounds * pairs - full;
    const double cost = (rounds + (s * half1 > 2 * idle ? 0.5 : 0.0)) / s * (1.0 + 0.03 * (s - 1));
    if (cost < best_cost) {
      best_cost = cost;
      best = s;
    }
  }
  return best;
}

struct GradLayout {
  bool few, direct;                // direct: so few that the last product takes R and B as they are
  bool own_x;                      // X by x_hidden_kernel and a product
  int tokens, chunk, splits, Kz;   // tokens and vocabulary rows per pass; partial dX (K splits)
  int pitch, n_ssum;
  size_t fwd, logits, cinv, ssum, ltgt, xop, w, g, dx, dz, rb, rbp, total;
};

GradLayout grad_layout(const archead_handle& h, int T) {
  const Layout& L = h.L;
  GradLayout o{};
  const int Kc = tc_kc(L);
  o.Kz = Kc - L.d;
  size_t at = 256;
  auto take = [&](size_t bytes) {
    const size_t r = at;
    at += round_up(bytes, 256);
    return r;
  };
  const bool whole = h.v_total == L.V;
  const size_t rows = std::max<size_t>(4096, std::min(kGradWBytes / (2 * Kc), kGradGBytes / (2 * std::min(T, kGradTokens))));
  // (without the tensor-core forward a pass of its logits takes 8 tokens)
  o.few = h.tc_ok ? T <= kFewPass || (T <= 2 * kFewPass && static_cast<size_t>(L.Vp) > rows) : T <= kDecodeTokens || !whole;
  const int pass = h.tc_ok ? kFewPass : kDecodeTokens, passes = (T + pass - 1) / pass;
  const size_t t = o.few ? (T + passes - 1) / passes : std::min(T, kGradTokens);
  o.tokens = static_cast<int>(t);
  o.direct = t <= kDecodeTokens;
  if (o.few) {
    // The forward call's workspace comes first: its header is this one's.
    o.fwd = ws_layout(h, o.tokens).total;
    at = round_up(o.fwd, 256);
    o.n_ssum = (L.n_mtiles + kGwMt - 1) / kGwMt;
    if (!use_tc(h, o.tokens)) o.logits = take(t * L.V * 4);
    const GwPlan g = gw_plan(h);
    o.splits = std::max(g.s.s_res, std::max(g.s.s_rest, g.s.s_last));
  } else {
    const int n_chunks = static_cast<int>((L.Vp + rows - 1) / rows);
    o.chunk = static_cast<int>(round_up((L.Vp + n_chunks - 1) / n_chunks, kGN));
    o.pitch = o.chunk + 64;   // (a power of two between G's rows would send a whole box to one memory channel)
    o.n_ssum = 2 * ((L.Vp + kGN - 1) / kGN);
    o.splits = accumulate_splits(o.tokens, Kc, o.chunk, h.num_sms / 2);
    o.own_x = !h.tc_ok || (whole && o.Kz > 0 && t >= kOwnXTokens);
    o.cinv = take(t * 4);
    o.xop = take(t * Kc * 2);
    o.w = take(static_cast<size_t>(o.chunk) * Kc * 2);
  }
  o.ssum = take(t * (o.few ? 4 * o.n_ssum : round_up(o.n_ssum, 4)) * 4);
  o.ltgt = take(t * 4);
  o.g = take(o.few ? static_cast<size_t>(o.n_ssum) * kGwRows * round_up(t, 32) * 2 : t * o.pitch * 2);
  o.dx = take(static_cast<size_t>(o.splits) * t * Kc * 4);
  o.dz = take(t * o.Kz * 2);
  if (!o.direct) o.rb = take(static_cast<size_t>(o.Kz) * L.d * 2);
  if (o.own_x) o.rbp = take(static_cast<size_t>(o.Kz) * L.d * 4);
  o.total = at;
  return o;
}

DequantParams dequant_params(const archead_handle& h, uint16_t* out) {
  const Layout& L = h.L;
  DequantParams dq{};
  dq.mtiles = h.arena;
  dq.out = out;
  dq.Kc = tc_kc(L);
  dq.n_res = L.n_res;
  dq.n_L = L.n_L;
  dq.n_A = L.n_A;
  dq.n_ks = dq.Kc / 64;
  while ((1 << dq.g_log2) < L.g) ++dq.g_log2;
  dq.off_res = L.off_res;
  dq.off_Lnib = L.off_Lnib;
  dq.off_Lhi = L.off_Lhi;
  dq.off_A = L.off_A;
  dq.off_sres = L.off_sres;
  dq.off_sL = L.off_sL;
  dq.off_sA = L.off_sA;
  dq.mblk_bytes = L.mblk_bytes;
  dq.sc_res = std::ldexp(1.f, h.tc_alpha);
  dq.sc_L = std::ldexp(1.f, h.tc_beta);
  dq.sc_A = std::ldexp(1.f, h.tc_gamma);
  return dq;
}

struct GradCall {
  const archead_handle& h;
  const GradLayout& o;
  uint8_t* wb;
  cudaStream_t stream;
  int sigma;                  // dz carries 2^beta (2^gamma), the rows of R (B) 2^rho: both meet in 2^sigma
};

// X and 2^-c_t of one pass's tokens.
cudaError_t grad_activations(const GradCall& c, const uint16_t* hidden, GemmParams p) {
  const archead_handle& h = c.h;
  const Layout& L = h.L;
  const int T = p.M, Kc = tc_kc(L);
  uint16_t* xop = reinterpret_cast<uint16_t*>(c.wb + c.o.xop);
  float* cinv = reinterpret_cast<float*>(c.wb + c.o.cinv);
  if (!c.o.own_x) {
    ActParams ap = act_params(h);
    ap.hidden = hidden;
    ap.status = p.status;
    ap.xop = xop;
    ap.cinv = cinv;
    ap.T = T;
    ap.zpart = reinterpret_cast<float*>(c.wb + c.o.dx);   // dX is written later
    ap.zticket = reinterpret_cast<uint32_t*>(c.wb + kActTicketOff);
    return launch_act_prep(ap, act_prep_splits(T, L.d, Kc, h.num_sms, c.o.dz - c.o.dx), c.stream);
  }
  x_hidden_kernel<<<T, 128, 0, c.stream>>>(XParams{hidden, xop, cinv, L.d, Kc, h.tc_alpha, h.tc_mseg});
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || c.o.Kz == 0) return e;
  // z = h [R | B]^T: the operand's h carries 2^(c_t - alpha), the rows 2^(sigma - beta|gamma)
  CUtensorMap mx, mr;
  e = tc_encode_map(&mx, xop, L.d, T, Kc, kGM / 2);
  if (e == cudaSuccess) e = tc_encode_map(&mr, reinterpret_cast<const uint16_t*>(c.wb + c.o.rbp), 2 * L.d, c.o.Kz, 2 * L.d, kGN / 2);
  if (e != cudaSuccess) return e;
  p.N = c.o.Kz;
  p.n_k = 2 * L.d / 64;
  p.splits = 1;
  p.x = xop + L.d;
  p.mul_acc = std::ldexp(1.f, h.tc_alpha - c.sigma);
  return launch_gemm<kLowrank>(p, mx, mr, h.num_sms, c.stream);
}

// The rows of R and B for the last product; the header cleared (status word,
// tickets of the activation kernel).
int grad_lowrank(const GradCall& c) {
  const Layout& L = c.h.L;
  if (c.o.Kz == 0 || c.o.direct) {
    const cudaError_t e = cudaMemsetAsync(c.wb, 0, 256, c.stream);
    return e == cudaSuccess ? ARCHEAD_OK : set_cuda_error(e);
  }
  LowrankParams lp{reinterpret_cast<const int8_t*>(c.h.arena + L.off_R),
                   reinterpret_cast<const uint16_t*>(c.h.arena + L.off_sR),
                   reinterpret_cast<const int8_t*>(c.h.arena + L.off_B),
                   reinterpret_cast<const uint16_t*>(c.h.arena + L.off_sB),
                   reinterpret_cast<uint16_t*>(c.wb + c.o.rb),
                   c.o.rbp != 0 ? reinterpret_cast<uint16_t*>(c.wb + c.o.rbp) : nullptr,
                   reinterpret_cast<uint32_t*>(c.wb), L.d, L.rcp, L.rrp, c.o.Kz, L.g_B,
                   std::ldexp(1.f, c.sigma - c.h.tc_beta), std::ldexp(1.f, c.sigma - c.h.tc_gamma)};
  lowrank_rows_kernel<<<(c.o.Kz * (L.d / 8) + 255) / 256, 256, 0, c.stream>>>(lp);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? ARCHEAD_OK : set_cuda_error(e);
}

// dX -> dh of one pass's tokens.
int grad_finish(const GradCall& c, GemmParams& p, int n_ssum, int splits, const GwSplits& gw) {
  const Layout& L = c.h.L;
  const int Kc = tc_kc(L), Kz = c.o.Kz, nt = p.M;
  uint16_t* dz = reinterpret_cast<uint16_t*>(c.wb + c.o.dz);
  DxParams dp{dequant_params(c.h, nullptr), p.ssum, p.ltgt, p.grad, p.targets, p.dx, p.split_stride, dz, n_ssum, p.ssum_pitch, Kc, L.d,
              L.V, c.h.row0, c.h.v_total == L.V ? 1 : 0, splits, gw};
  const bool ways = nt <= kDxWaysTokens;
  const auto dx = ways ? dx_kernel<kDxWays> : dx_kernel<1>;
  const int cols = ways ? 1024 / kDxWays : 1024;
  cudaError_t e = launch_after(dx, dim3(nt, (Kc + cols - 1) / cols), 256, 0, c.stream, dp);
  if (e == cudaSuccess && c.o.direct) {
    const FinishFewParams f{reinterpret_cast<const int8_t*>(c.h.arena + L.off_R),
                            reinterpret_cast<const uint16_t*>(c.h.arena + L.off_sR),
                            reinterpret_cast<const int8_t*>(c.h.arena + L.off_B),
                            reinterpret_cast<const uint16_t*>(c.h.arena + L.off_sB),
                            dz, p.dx, p.grad, p.targets, p.out, p.status, nt, L.d, Kc, Kz, L.rcp, L.rrp, L.g_B, p.v_total,
                            p.out_f32, std::ldexp(1.f, -c.h.tc_beta), std::ldexp(1.f, -c.h.tc_gamma),
                            std::ldexp(1.f, -kGradScale - c.h.tc_alpha)};
    const auto kernel = nt == 1 ? finish_few_kernel<1> : nt == 2 ? finish_few_kernel<2>
                        : nt <= 4 ? finish_few_kernel<4> : finish_few_kernel<8>;
    e = launch_after(kernel, dim3(L.d / 64), 512, 0, c.stream, f);
    return e == cudaSuccess ? ARCHEAD_OK : set_cuda_error(e);
  }
  CUtensorMap mz{}, mr{};
  if (e == cudaSuccess && Kz > 0) {
    e = tc_encode_map(&mz, dz, Kz, nt, Kz, kGM / 2);
    if (e == cudaSuccess) e = tc_encode_map(&mr, reinterpret_cast<const uint16_t*>(c.wb + c.o.rb), L.d, Kz, L.d, 64);
  }
  if (e != cudaSuccess) return set_cuda_error(e);
  p.N = L.d;
  p.n_k = Kz / 64;
  p.splits = 1;
  p.mul_acc = std::ldexp(1.f, -c.sigma);
  p.mul_dx = std::ldexp(1.f, -kGradScale - c.h.tc_alpha);
  e = launch_gemm<kFinish>(p, mz, mr, c.h.num_sms, c.stream);
  return e == cudaSuccess ? ARCHEAD_OK : set_cuda_error(e);
}

// Few tokens: the forward kernels' logits, G, then G W~ from the packed rows.
int grad_few(const GradCall& c, const uint16_t* hidden, GemmParams& p) {
  const archead_handle& h = c.h;
  const Layout& L = h.L;
  const int T = p.M;
  int n_ssum = c.o.n_ssum;
  cudaError_t e;
  if (use_tc(h, T)) {
    n_ssum *= 4;
    p.ssum_pitch = n_ssum;
    const int rc = forward_tc_grad(h, hidden, T, p.targets, p.lse, p.grad, p.G, p.ssum, p.ltgt, c.wb, c.stream);
    if (rc != ARCHEAD_OK) return rc;
  } else {
    float* logits = reinterpret_cast<float*>(c.wb + c.o.logits);
    const int rc = forward_logits(h, hidden, T, logits, c.wb, c.o.fwd, c.stream);
    if (rc != ARCHEAD_OK) return rc;
    GParams gp{logits, p.lse, p.grad, p.targets, reinterpret_cast<uint4*>(p.G), p.ssum, p.ltgt, T, L.V, h.row0, p.ssum_pitch};
    e = launch_after(g_kernel, dim3(c.o.n_ssum), 32 * kDecodeTokens, 0, c.stream, gp);
    if (e != cudaSuccess) return set_cuda_error(e);
  }
  const GwPlan g = gw_plan(h);
  GwParams w{};
  w.rows = dequant_params(h, nullptr);
  w.G = reinterpret_cast<const uint4*>(p.G);
  w.T = T;
  w.n_mtiles = L.n_mtiles;
  w.nk = g.nk;
  w.chunks = g.chunks;
  w.splits = g.s;
  w.dx = p.dx;
  w.split_stride = p.split_stride;
  w.status = p.status;
  const int gl = w.rows.g_log2;
  const auto kernel = gl >= 7 ? gw_kernel<1> : gl == 6 ? gw_kernel<2> : gl == 5 ? gw_kernel<4> : gw_kernel<8>;
  e = launch_after(kernel, dim3(g.grid), kGwWarps * 32, kGwSmem, c.stream, w);
  if (e != cudaSuccess) return set_cuda_error(e);
  return grad_finish(c, p, n_ssum, 0, g.s);
}

// Many tokens: chunk by chunk through the dequantised rows.
int grad_many(const GradCall& c, const uint16_t* hidden, GemmParams& p) {
  const archead_handle& h = c.h;
  const Layout& L = h.L;
  const GradLayout& o = c.o;
  const int Kc = tc_kc(L), nt = p.M;
  uint16_t* w = reinterpret_cast<uint16_t*>(c.wb + o.w);
  cudaError_t e = grad_activations(c, hidden, p);
  if (e != cudaSuccess) return set_cuda_error(e);
  DequantParams dq = dequant_params(h, w);
  p.cinv = reinterpret_cast<const float*>(c.wb + o.cinv);
  const uint16_t* xop = reinterpret_cast<const uint16_t*>(c.wb + o.xop);
  CUtensorMap mx, mg, mwk, mwn;
  for (int v0 = 0; v0 < L.Vp; v0 += o.chunk) {
    const int rows = std::min(o.chunk, L.Vp - v0);
    dq.mt0 = v0 / kMT;
    dq.n_mt = rows / kMT;
    const int64_t items = static_cast<int64_t>(dq.n_mt) * dq.n_ks;
    dequant_rows_kernel<<<static_cast<unsigned>((items + 7) / 8), 256, 0, c.stream>>>(dq);
    e = cudaGetLastError();
    if (e == cudaSuccess) e = tc_encode_map(&mx, xop, Kc, nt, Kc, kGM / 2);
    if (e == cudaSuccess) e = tc_encode_map(&mg, p.G, rows, nt, o.pitch, kGM / 2);
    if (e == cudaSuccess) e = tc_encode_map(&mwk, w, Kc, rows, Kc, kGN / 2);
    if (e == cudaSuccess) e = tc_encode_map(&mwn, w, Kc, rows, Kc, 64);
    if (e != cudaSuccess) return set_cuda_error(e);
    p.v0 = v0;
    p.N = rows;
    p.n_k = Kc / 64;
    p.splits = 1;
    e = launch_gemm<kSoftmax>(p, mx, mwk, h.num_sms, c.stream);
    if (e != cudaSuccess) return set_cuda_error(e);
    p.N = Kc;
    p.n_k = (rows + 63) / 64;
    p.splits = o.splits;
    p.first = v0 == 0;
    e = launch_gemm<kAccumulate>(p, mg, mwn, h.num_sms, c.stream);
    if (e != cudaSuccess) return set_cuda_error(e);
  }
  return grad_finish(c, p, o.n_ssum, o.splits, GwSplits{});
}

int grad_launch(const archead_handle& h, const GradLayout& o, const uint16_t* hidden, int T, const int32_t* targets,
                const float* lse, const float* grad, void* out, bool out_f32, uint8_t* wb, cudaStream_t stream) {
  const Layout& L = h.L;
  GradCall c{h, o, wb, stream, L.r_c > 0 ? h.tc_beta + h.tc_rho_c : 1 << 20};
  if (L.r_r > 0) c.sigma = std::min(c.sigma, h.tc_gamma + h.tc_rho_r);
  if (o.Kz == 0) c.sigma = 0;
  int rc = grad_lowrank(c);
  for (int t0 = 0; t0 < T && rc == ARCHEAD_OK; t0 += o.tokens) {
    const int nt = std::min(o.tokens, T - t0);
    const size_t first = static_cast<size_t>(t0) * L.d;
    GemmParams p{};
    p.M = nt;
    p.status = reinterpret_cast<uint32_t*>(wb + 4);
    p.grad = grad + t0;
    p.targets = targets + t0;
    p.row0 = h.row0;
    p.v_total = h.v_total;
    p.lse = lse + t0;
    p.G = reinterpret_cast<uint16_t*>(wb + o.g);
    p.pitch = o.pitch;
    p.V = L.V;
    p.ssum = reinterpret_cast<float*>(wb + o.ssum);
    p.ssum_pitch = static_cast<int32_t>(round_up(o.n_ssum, 4));   // 16-byte rows
    p.ltgt = reinterpret_cast<float*>(wb + o.ltgt);
    p.dx = reinterpret_cast<float*>(wb + o.dx);
    p.Kc = tc_kc(L);
    p.split_stride = static_cast<size_t>(nt) * p.Kc;
    p.out = static_cast<uint8_t*>(out) + first * (out_f32 ? 4 : 2);
    p.out_f32 = out_f32 ? 1 : 0;
    rc = o.few ? grad_few(c, hidden + first, p) : grad_many(c, hidden + first, p);
  }
  return rc;
}

constexpr int kMaxTokens = 1 << 20;

// Shared-memory limits of the kernels, at a head's first gradient call: at its
// construction they would load a dozen kernels for programs that only infer (whose
// first head took 15 ms in place of 9).  Calls that race set them twice.
cudaError_t grad_set_attributes(const archead_handle& h) {
  if (__atomic_load_n(&h.grad_ready, __ATOMIC_ACQUIRE) != 0) return cudaSuccess;
  cudaError_t e = h.tc_ok ? tc_set_grad_attributes() : cudaSuccess;
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(grad_gemm_kernel<kSoftmax>, cudaFuncAttributeMaxDynamicSharedMemorySize, kGSmem);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(grad_gemm_kernel<kLowrank>, cudaFuncAttributeMaxDynamicSharedMemorySize, kGSmem);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(grad_gemm_kernel<kAccumulate>, cudaFuncAttributeMaxDynamicSharedMemorySize, kGSmem);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(grad_gemm_kernel<kFinish>, cudaFuncAttributeMaxDynamicSharedMemorySize, kGSmem);
  for (const void* k : {reinterpret_cast<const void*>(&gw_kernel<1>), reinterpret_cast<const void*>(&gw_kernel<2>),
                        reinterpret_cast<const void*>(&gw_kernel<4>), reinterpret_cast<const void*>(&gw_kernel<8>)})
    if (e == cudaSuccess) e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kGwSmem);
  if (e == cudaSuccess) __atomic_store_n(&h.grad_ready, 1, __ATOMIC_RELEASE);
  return e;
}

}  // namespace

}  // namespace archead

using namespace archead;

extern "C" ARCHEAD_API size_t archead_grad_workspace_bytes(const archead_handle* handle, int32_t T) {
  if (handle == nullptr || T <= 0 || T > kMaxTokens) return 0;
  return grad_layout(*handle, T).total;
}

extern "C" ARCHEAD_API int archead_grad_hidden(const archead_handle* handle, const uint16_t* hidden, int32_t T,
                                               const int32_t* targets, const float* lse, const float* grad_ce,
                                               void* grad_hidden, int32_t grad_dtype, void* workspace,
                                               size_t workspace_bytes, archead_stream_t stream) {
  if (handle == nullptr || hidden == nullptr || targets == nullptr || lse == nullptr || grad_ce == nullptr ||
      grad_hidden == nullptr || workspace == nullptr)
    return ARCHEAD_EINVAL;
  if (T <= 0 || T > kMaxTokens) return ARCHEAD_EINVAL;
  if (grad_dtype != ARCHEAD_GRAD_BF16 && grad_dtype != ARCHEAD_GRAD_F32) return ARCHEAD_EINVAL;
  auto aligned = [](const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; };
  if (!aligned(hidden, 16) || !aligned(grad_hidden, 16) || !aligned(workspace, 256) || !aligned(targets, 4) ||
      !aligned(lse, 4) || !aligned(grad_ce, 4))
    return ARCHEAD_EALIGN;
  const GradLayout o = grad_layout(*handle, T);
  if (workspace_bytes < o.total) return ARCHEAD_ENOMEM;
  int dev = -1;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return set_cuda_error(e);
  if (dev != handle->device) return ARCHEAD_EINVAL;
  e = grad_set_attributes(*handle);
  if (e != cudaSuccess) return set_cuda_error(e);
  return grad_launch(*handle, o, hidden, T, targets, lse, grad_ce, grad_hidden, grad_dtype == ARCHEAD_GRAD_F32,
                     static_cast<uint8_t*>(workspace), reinterpret_cast<cudaStream_t>(stream));
}
