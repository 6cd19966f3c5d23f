// Gradient of the cross-entropy with respect to the hidden states, through the
// packed head (ARCHead paper, §3.2 Eq. 7; the head itself is frozen).
//
// With y[t] = W h[t] over all rows of the head, lse[t] its log-sum-exp and
// g[t] = dLoss / dce[t], ce[t] = lse[t] - y[t, target[t]]:
//   G[t,v]  = exp(y[t,v] - lse[t]) - [v = target[t]]
//   dh[t,:] = g[t] sum_v G[t,v] W[v,:].
// W is never formed.  With W~ the concatenated packed operand of the
// tensor-core forward (tc_params.h; columns residual | core | correction)
//   y = 2^-c_t X W~^T,        dX = G W~   (one row of d + r_c' + r_r' columns),
//   dh = g ( dX_res + dX_core (s_R R) + dX_corr (s_B B) ),
// so the low-rank factors are applied once per token, not once per row.
//
// The recomputed logits carry the forward's rounding (up to ~1e-2 where y is
// large), the given lse that of whichever kernel made it; a row that holds most
// of the mass would get all of their difference.  So the probabilities are
// normalised by their own sum S[t] = sum_v exp(y[t,v] - lse[t]), after the fact:
//   sum_v (exp(y - lse) / S - [v = target]) W[v] = (G W) / S + (1/S - 1) W[target].
// (On a vocabulary shard S is not known and lse is taken as it is.)
//
// The vocabulary is walked in chunks of at most kGradChunk rows.  Per chunk
//   1. dequant_rows_kernel   W~ of the chunk, fp16, in the workspace
//   2. gemm softmax          G of the chunk, fp16
//   3. gemm accumulate       dX += G W~, fp32
// and after the last chunk
//   4. dx_kernel             dX / S + (1/S - 1) W~[target], its low-rank
//      columns to fp16; lowrank_rows_kernel: [s_R R | s_B B], fp16
//   5. gemm finish           dh from dX_res + dz [s_R R | s_B B].
//
// Roundings to fp16: W~ entries (2^-11 relative, as in the forward), G (2^-11,
// stored times 2^15 so that a probability keeps its full precision down to
// 2^-29), dX of the low-rank columns and the rows of R and B.  All are
// independent from entry to entry, so the sum's error stays near 2^-12 of its
// own size, below the bf16 rounding of the result; sums are fp32.
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

constexpr int kGradChunk = 16384;     // vocabulary rows of one pass (W~ chunk: 153 MB at 4672 columns)
constexpr int kGradTokens = 4096;     // tokens of one pass over the head
constexpr int kGradScale = 15;        // G is stored times 2^15

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
__device__ __forceinline__ uint4 ldg128(const uint8_t* p) { return __ldg(reinterpret_cast<const uint4*>(p)); }

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
  int32_t d, rcp, rrp, Kz, g_B;
  float mul_c, mul_r;
};
__global__ void __launch_bounds__(256) lowrank_rows_kernel(const LowrankParams p) {
  const int e = blockIdx.x;
  const int k = (e & ~15) + tc_kcol(e & 15);
  uint16_t* out = p.out + static_cast<size_t>(e) * p.d;
  for (int j = threadIdx.x; j < p.d; j += blockDim.x) {
    float v = 0.f;
    if (k < p.rcp) {
      v = static_cast<float>(p.R[static_cast<size_t>(k) * p.d + j]) * __half2float(__ushort_as_half(p.s_R[k])) * p.mul_c;
    } else if (k - p.rcp < p.rrp) {
      const int r = k - p.rcp;
      v = static_cast<float>(p.B[static_cast<size_t>(r) * p.d + j]) *
          __half2float(__ushort_as_half(p.s_B[static_cast<size_t>(r) * (p.d / p.g_B) + j / p.g_B])) * p.mul_r;
    }
    out[j] = __half_as_ushort(__float2half_rn(v));
  }
}

// X of heads whose z the activation kernel does not compute (g_B not a multiple
// of 64), from the decode prologue's z pairs.
struct XParams {
  const uint16_t* hidden;
  const uint16_t* zhi;
  const uint16_t* zlo;
  const int32_t* escale;
  uint16_t* xop;
  float* cinv;
  int32_t d, rcp, Kz, Kc, alpha, beta, gamma, mseg, e_B;
};
__global__ void __launch_bounds__(256) x_from_z_kernel(const XParams p) {
  const int t = blockIdx.x, E = p.escale[t];
  if (threadIdx.x == 0) p.cinv[t] = ldexpf(1.f, E - kScaleExp - p.mseg);
  const float sh = ldexpf(1.f, kScaleExp - E + p.mseg - p.alpha);
  const float sc = ldexpf(1.f, p.e_B + p.mseg - p.beta), sr = ldexpf(1.f, p.e_B + p.mseg - p.gamma);
  for (int e = threadIdx.x; e < p.Kc; e += blockDim.x) {
    const int k = (e & ~15) + tc_kcol(e & 15);
    float v = 0.f;
    if (k < p.d) {
      v = __uint_as_float(static_cast<uint32_t>(p.hidden[static_cast<size_t>(t) * p.d + k]) << 16) * sh;
    } else if (k - p.d < p.Kz) {
      const size_t i = static_cast<size_t>(t) * p.Kz + (k - p.d);
      const float z = __half2float(__ushort_as_half(p.zhi[i])) + __half2float(__ushort_as_half(p.zlo[i]));
      v = z * (k - p.d < p.rcp ? sc : sr);
    }
    p.xop[static_cast<size_t>(t) * p.Kc + e] = __half_as_ushort(__float2half_rn(v));
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

// Blocks of 1024 columns per token: S from the tiles' partial sums (in a fixed order), then
// dX (added over the K splits) / S + (1/S - 1) W~[target]; the residual columns
// stay fp32 in the first split's place, the low-rank ones become the fp16
// operand dz [T][Kz'].
struct DxParams {
  DequantParams rows;
  const float* ssum;          // [n_ssum][tokens]
  const float* grad;
  const int32_t* targets;
  float* dx;
  size_t split_stride;
  uint16_t* dz;
  int32_t n_ssum, tokens, Kc, d, V, row0, whole;   // whole: all rows of the vocabulary are here
  int32_t splits, splits_last, last;               // partial dX of columns below `last`, and of the rest
};
__global__ void __launch_bounds__(256) dx_kernel(const DxParams p) {
  __shared__ float part[8];
  const int t = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int q0 = blockIdx.y * blockDim.x + threadIdx.x, dq = gridDim.y * blockDim.x;
  if (p.grad[t] == 0.f) {     // its row of dX is zero, S has no meaning
    for (int q = q0; q < (p.Kc - p.d) / 4; q += dq)
      *reinterpret_cast<uint2*>(p.dz + static_cast<size_t>(t) * (p.Kc - p.d) + 4 * q) = make_uint2(0u, 0u);
    return;
  }
  float r = 1.f;
  if (p.whole) {
    float s = 0.f;
    for (int i = threadIdx.x; i < p.n_ssum; i += blockDim.x) s += p.ssum[static_cast<size_t>(i) * p.tokens + t];
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane == 0) part[warp] = s;
    __syncthreads();
    s = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) s += part[w];
    r = 1.f / s;
  }
  const int target = p.targets[t] - p.row0;
  const bool has = p.whole && target >= 0 && target < p.V;
  const float c = (r - 1.f) * static_cast<float>(1 << kGradScale);
  const uint8_t* blk = p.rows.mtiles + static_cast<size_t>(has ? target / kMT : 0) * p.rows.mblk_bytes;
  float* dx = p.dx + static_cast<size_t>(t) * p.Kc;
  for (int q = q0; q < p.Kc / 4; q += dq) {
    float4 v = reinterpret_cast<const float4*>(dx)[q];
    const int n = 4 * q < p.last ? p.splits : p.splits_last;
    for (int s = 1; s < n; ++s) {
      const float4 x = reinterpret_cast<const float4*>(dx + s * p.split_stride)[q];
      v = make_float4(v.x + x.x, v.y + x.y, v.z + x.z, v.w + x.w);
    }
    float4 w = make_float4(0.f, 0.f, 0.f, 0.f);
    if (has) w = packed_row4(p.rows, blk, target % kMT, q);
    v = make_float4(fmaf(c, w.x, v.x * r), fmaf(c, w.y, v.y * r), fmaf(c, w.z, v.z * r), fmaf(c, w.w, v.w * r));
    if (4 * q < p.d) {
      reinterpret_cast<float4*>(dx)[q] = v;
    } else {
      constexpr float kInv = 1.f / (1 << kGradScale);
      *reinterpret_cast<uint2*>(p.dz + static_cast<size_t>(t) * (p.Kc - p.d) + 4 * q - p.d) =
          make_uint2(pack_half2(v.x * kInv, v.y * kInv), pack_half2(v.z * kInv, v.w * kInv));
    }
  }
}

// -------------------------------------------------------------------- gemm
// D[128 tokens x 256 columns] tiles of A B, A [tokens][K] fp16 K-major, B fp16
// either [columns][K] (softmax) or [K][columns] (accumulate, finish), by TMA in
// k-steps of 64.  One CTA per SM walks its units (K split, token tile, column
// tile); warp 0 issues the copies, warp 1 the MMAs, warps 2-5 empty one of two
// TMEM accumulators while the next fills.
constexpr int kGM = 128, kGN = 256, kGStages = 4, kGWarps = 6;
constexpr uint32_t kGABytes = kGM * 128, kGBBytes = kGN * 128, kGStageBytes = kGABytes + kGBBytes;
constexpr uint32_t kGBarOff = kGStages * kGStageBytes;
constexpr uint32_t kGSmem = kGBarOff + 256 + 1024;
constexpr uint32_t kGTmem = 512;

enum GemmMode { kSoftmax, kAccumulate, kFinish };

struct GemmParams {
  int32_t M, N;                        // tokens; columns of this product
  int32_t n_k, n_mt, n_nt, splits, n_units;
  uint32_t* status;
  const float* grad;                   // [M]
  const int32_t* targets;              // [M]
  int32_t row0, v_total;
  // softmax
  const float* cinv;                   // [M]
  const float* lse;                    // [M]
  uint16_t* G;                         // [M][pitch]
  int32_t pitch, v0, V;                // first row of the chunk, rows of the head
  float* ssum;                         // [tiles][tokens]: sums of exp(y - lse) over the tile's rows
  int32_t tokens;
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

struct GemmUnit {
  int m, n, k0, k1, split;
};
__device__ __forceinline__ GemmUnit g_unit(const GemmParams& p, int u) {
  GemmUnit r;
  const int tiles = p.n_mt * p.n_nt;
  r.split = u / tiles;
  const int rest = u - r.split * tiles;
  r.n = rest / p.n_mt;
  r.m = rest - r.n * p.n_mt;
  r.k0 = static_cast<int>(static_cast<int64_t>(p.n_k) * r.split / p.splits);
  r.k1 = static_cast<int>(static_cast<int64_t>(p.n_k) * (r.split + 1) / p.splits);
  return r;
}

template <GemmMode kMode>
__device__ void g_tma_warp(const GemmParams& p, const GemmSmem& sm, const CUtensorMap* ma, const CUtensorMap* mb) {
  int s = 0, issued = 0;
  uint32_t ph = 0;
  bool ok = true;
  for (int u = blockIdx.x; ok && u < p.n_units; u += gridDim.x) {
    const GemmUnit w = g_unit(p, u);
    const int nb = (min(kGN, p.N - w.n * kGN) + 63) / 64;   // 64-column blocks of B (stored [K][columns])
    for (int k = w.k0; k < w.k1; ++k) {
      ok = g_wait(sm, sm.empty + 8 * s, ph ^ 1u, p.status);
      if (!ok) break;
      if (elect_one()) {
        const uint32_t bar = sm.full + 8 * s, a = sm.stages + s * kGStageBytes, b = a + kGABytes;
        mbar_arrive_expect_tx(bar, kGABytes + (kMode == kSoftmax ? kGBBytes : nb * 8192u));
        tma_load_2d(a, ma, k * 64, w.m * kGM, bar);
        if constexpr (kMode == kSoftmax) {
          tma_load_2d(b, mb, k * 64, w.n * kGN, bar);
        } else {
          for (int i = 0; i < nb; ++i) tma_load_2d(b + i * 8192u, mb, w.n * kGN + 64 * i, k * 64, bar);
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
  if (!ok) {
    // Copies still in flight land before the block's shared memory goes away.
    const int back = min(issued, kGStages);
    for (int i = 1; i <= back; ++i) {
      const int at = issued - i;
      mbar_wait(sm.full + 8 * (at % kGStages), (at / kGStages) & 1u);
    }
  }
}

template <GemmMode kMode>
__device__ void g_mma_warp(const GemmParams& p, const GemmSmem& sm, uint32_t tmem_base) {
  constexpr bool kMn = kMode != kSoftmax;
  const uint64_t ad0 = smem_desc_k128(sm.stages);
  const uint64_t bd0 = kMn ? smem_desc_mn128(sm.stages + kGABytes, 8192u) : smem_desc_k128(sm.stages + kGABytes);
  constexpr uint32_t kBStep = kMn ? 128u : 2u;   // descriptor units per K = 16
  int s = 0, i = 0;
  uint32_t ph = 0;
  for (int u = blockIdx.x; u < p.n_units; u += gridDim.x, ++i) {
    const GemmUnit w = g_unit(p, u);
    const uint32_t acc = i & 1;
    if (!g_wait(sm, sm.acce + 8 * acc, ((i >> 1) & 1) ^ 1, p.status)) return;
    tc_fence_after();
    const int ncol = (min(kGN, p.N - w.n * kGN) + 15) & ~15;
    const uint32_t idesc = tc_idesc_f16(kGM, ncol) | (kMn ? kTcIdescBmn : 0u);
    const uint32_t d = tmem_base + acc * kGN;
    for (int k = w.k0; k < w.k1; ++k) {
      if (!g_wait(sm, sm.full + 8 * s, ph, p.status)) return;
      tc_fence_after();
      if (elect_one()) {
        const uint64_t a = ad0 + static_cast<uint64_t>(s) * (kGStageBytes >> 4);
        const uint64_t b = bd0 + static_cast<uint64_t>(s) * (kGStageBytes >> 4);
        tc_mma_ss(d, a, b, idesc, k != w.k0);
        tc_mma_ss(d, a + 2, b + kBStep, idesc, 1u);
        tc_mma_ss(d, a + 4, b + 2 * kBStep, idesc, 1u);
        tc_mma_ss(d, a + 6, b + 3 * kBStep, idesc, 1u);
        tc_commit(sm.empty + 8 * s);
      }
      __syncwarp();
      if (++s == kGStages) {
        s = 0;
        ph ^= 1u;
      }
    }
    if (elect_one()) tc_commit(sm.accf + 8 * acc);
    __syncwarp();
  }
}

__device__ __forceinline__ float grad_nan() { return __int_as_float(0x7fc00000); }

// Lane = token row, columns in pieces of 32.
template <GemmMode kMode>
__device__ void g_epilogue(const GemmParams& p, const GemmSmem& sm, uint32_t tmem_base, int lane) {
  const int q = (threadIdx.x >> 5) & 3;
  bool ok = true;
  int i = 0;
  for (int u = blockIdx.x; u < p.n_units; u += gridDim.x, ++i) {
    const GemmUnit w = g_unit(p, u);
    const uint32_t acc = i & 1;
    const int t = w.m * kGM + 32 * q + lane, n0 = w.n * kGN;
    const int ncol = min(kGN, p.N - n0);
    const bool live = t < p.M;
    float g = 0.f, cinv = 0.f, lse = 0.f;
    int target = -1;
    if (live && kMode != kAccumulate) {
      g = p.grad[t];
      target = p.targets[t];
      if constexpr (kMode == kSoftmax) {
        cinv = p.cinv[t];
        lse = p.lse[t];
      }
    }
    if (ok) ok = g_wait(sm, sm.accf + 8 * acc, (i >> 1) & 1, p.status);
    if (ok) {
      tc_fence_after();
      const uint32_t taddr = tmem_base + (static_cast<uint32_t>(32 * q) << 16) + acc * kGN;
      if constexpr (kMode == kFinish) {
        if (live && g != 0.f && (target < 0 || target >= p.v_total)) {
          g = grad_nan();
          if (w.n == 0) atomicOr(p.status, static_cast<uint32_t>(ARCHEAD_STATUS_BAD_TARGET));
        }
      }
      float ssum = 0.f;
      for (int c0 = 0; c0 < ncol; c0 += 32) {
        uint32_t r[32];
        tmem_ld_32x32b_x32(taddr + c0, r);
        tmem_ld_wait();
        if (!live) {
          // a row past the last token
        } else if constexpr (kMode == kSoftmax) {
          // columns are vocabulary rows of the chunk; a token without a
          // gradient gets zeros (its lse and target may be anything)
          const int tl = target - p.row0 - p.v0 - n0 - c0;
          uint32_t o[16];
#pragma unroll
          for (int c = 0; c < 32; c += 2) {
            float e[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              float x = __expf(fmaf(__uint_as_float(r[c + h]), cinv, -lse));
              if (g == 0.f || p.v0 + n0 + c0 + c + h >= p.V) x = 0.f;
              ssum += x;
              e[h] = (x - (g != 0.f && c + h == tl ? 1.f : 0.f)) * static_cast<float>(1 << kGradScale);
            }
            o[c / 2] = pack_half2(e[0], e[1]);
          }
          uint4* dst = reinterpret_cast<uint4*>(p.G + static_cast<size_t>(t) * p.pitch + n0 + c0);
#pragma unroll
          for (int v = 0; v < 4; ++v)
            if (c0 + 8 * v < ncol) dst[v] = make_uint4(o[4 * v], o[4 * v + 1], o[4 * v + 2], o[4 * v + 3]);
        } else if constexpr (kMode == kAccumulate) {
          float4* dst = reinterpret_cast<float4*>(p.dx + w.split * p.split_stride + static_cast<size_t>(t) * p.Kc + n0 + c0);
#pragma unroll
          for (int v = 0; v < 8; ++v) {
            float4 x = make_float4(__uint_as_float(r[4 * v]), __uint_as_float(r[4 * v + 1]),
                                   __uint_as_float(r[4 * v + 2]), __uint_as_float(r[4 * v + 3]));
            if (w.k0 == w.k1) x = make_float4(0.f, 0.f, 0.f, 0.f);   // a split without rows in a short chunk
            if (!p.first) {
              const float4 y = dst[v];
              x = make_float4(x.x + y.x, x.y + y.y, x.z + y.z, x.w + y.w);
            }
            dst[v] = x;
          }
        } else {
          float x[32];
#pragma unroll
          for (int c = 0; c < 32; ++c) x[c] = p.n_k > 0 ? __uint_as_float(r[c]) * p.mul_acc : 0.f;
          const float4* src = reinterpret_cast<const float4*>(p.dx + static_cast<size_t>(t) * p.Kc + n0 + c0);
#pragma unroll
          for (int v = 0; v < 8; ++v) {
            const float4 y = src[v];
            const float z[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
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
        __syncwarp();
      }
      if (kMode == kSoftmax && live) p.ssum[static_cast<size_t>(p.v0 / kGN + w.n) * p.tokens + t] = ssum;
      tc_fence_before();
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(sm.acce + 8 * acc);
  }
}

template <GemmMode kMode>
__global__ void __launch_bounds__(kGWarps * 32, 1)
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
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kGStages; ++s) {
      mbar_init(sm.full + 8 * s, 1);
      mbar_init(sm.empty + 8 * s, 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(sm.accf + 8 * a, 1);
      mbar_init(sm.acce + 8 * a, 4);
    }
    *sm.abort_flag = 0;
    mbar_fence_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_addr(sm.tmem), kGTmem);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *sm.tmem;
  if (warp == 0) g_tma_warp<kMode>(p, sm, &ma, &mb);
  else if (warp == 1) g_mma_warp<kMode>(p, sm, tmem_base);
  else g_epilogue<kMode>(p, sm, tmem_base, lane);
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, kGTmem);
  }
}

template <GemmMode kMode>
cudaError_t launch_gemm(GemmParams& p, const CUtensorMap& ma, const CUtensorMap& mb, int num_sms, cudaStream_t stream) {
  p.n_mt = (p.M + kGM - 1) / kGM;
  p.n_nt = (p.N + kGN - 1) / kGN;
  p.n_units = p.splits * p.n_mt * p.n_nt;
  grad_gemm_kernel<kMode><<<std::min(p.n_units, num_sms), kGWarps * 32, kGSmem, stream>>>(p, ma, mb);
  return cudaGetLastError();
}

// ------------------------------------------------------- few tokens: G, G W~
// G from the forward kernels' logits (fp32 [T][V]): one block per (token, piece
// of kGPiece rows), with the piece's sum of exp(y - lse).
constexpr int kGPiece = 2048;
struct GParams {
  const float* y;
  const float* lse;
  const float* grad;
  const int32_t* targets;
  uint16_t* G;                // [T][pitch]
  float* ssum;                // [pieces][T]
  int32_t T, V, Vp, row0, pitch;
};
__global__ void __launch_bounds__(256) g_kernel(const GParams p) {
  __shared__ float part[8];
  const int t = blockIdx.y, v0 = blockIdx.x * kGPiece, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool live = p.grad[t] != 0.f;   // (its lse and target may be anything otherwise)
  const float lse = live ? p.lse[t] : 0.f;
  const int target = live ? p.targets[t] - p.row0 : -1;
  const float* y = p.y + static_cast<size_t>(t) * p.V;
  uint16_t* G = p.G + static_cast<size_t>(t) * p.pitch;
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < kGPiece / 512; ++i) {
    const int v = v0 + 512 * i + 2 * threadIdx.x;
    if (v >= p.Vp) break;
    float x[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      x[e] = live && v + e < p.V ? __expf(y[v + e] - lse) : 0.f;
      sum += x[e];
      if (live && v + e == target) x[e] -= 1.f;
    }
    constexpr float k = 1 << kGradScale;
    *reinterpret_cast<uint32_t*>(G + v) = pack_half2(x[0] * k, x[1] * k);
  }
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) part[warp] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) s += part[w];
    p.ssum[static_cast<size_t>(blockIdx.x) * p.T + t] = s;
  }
}

// dX = G W~ for up to 256 tokens, the packed rows dequantised on the way:
// D[column of W~][token], A = the 64-row x 256-column tile of W~ as the
// dequantising warps leave it in shared memory (rows of 64 columns, so
// MN-major: the transpose costs nothing), B = 64 columns of G by TMA.  A CTA
// owns `nb` column blocks of 256 (2 nb accumulators of N TMEM columns fill the
// 512) and a range of vocabulary rows, writes one partial dX, and dx_kernel adds
// the partials of a column's CTAs in order.
//   warps 0-15  dequantise: set w / 8 takes every second tile; a warp one 16-row
//               m-tile x 128 columns of it, its packed bytes loaded kGwAhead
//               tiles early straight into registers (one 16-byte load per lane
//               and 64 columns: nothing to copy, wait for or re-read).
//   warp 16     TMA of G        warp 17  MMA
// Afterwards warps 0-15 write the accumulators.
constexpr int kGwWarps = 18, kGwStages = 4, kGwMaxN = 256, kGwAhead = 2;
constexpr uint32_t kGwTile = 256 * 128;        // 64 rows x 256 columns of fp16
constexpr uint32_t kGwGOff = kGwStages * kGwTile;
constexpr uint32_t kGwSmemMax = 231424;        // 226 KB: with the 1 KB of alignment all a block may have

struct GwParams {
  DequantParams rows;
  int32_t n_mtiles, nk;        // k-steps of 64 rows
  int32_t T, N;                // tokens; rounded up to 16
  int32_t nb, chunks;          // column blocks of 256 per CTA; 64-column chunks in all
  int32_t full, s_full, s_last;   // groups of nb whole blocks; row splits of those and of the last group
  int32_t gstages;
  uint32_t g_bytes, bar_off;
  float* dx;                   // [split][T][Kc]
  size_t split_stride;
  uint32_t* status;
};

// Packed bytes of one 64-column chunk, as one lane holds them.
template <int GM>
struct RawChunk {
  uint4 c, x;                  // codes; fifth bits (core: x.x) or the second half (correction)
  uint32_t s[1 << GM];         // scale pairs
};

template <int GM>
__device__ __forceinline__ void load_chunk(const DequantParams& p, const uint8_t* blk, int ks, int lane, RawChunk<GM>& r) {
  const int gr = lane >> 2;
  if (ks < p.n_res) {
    r.c = ldg128(blk + p.off_res + ks * kResChunkBytes + lane * 16);
    const uint8_t* s = blk + p.off_sres + ((ks * 64) >> p.g_log2) * kSresGroupBytes + gr * 4;
#pragma unroll
    for (int g = 0; g < (1 << GM); ++g) r.s[g] = ldg32(s + g * kSresGroupBytes);
  } else if (ks < p.n_res + p.n_L) {
    const int c = ks - p.n_res;
    r.c = ldg128(blk + p.off_Lnib + c * kLNibChunkBytes + lane * 16);
    r.x.x = ldg32(blk + p.off_Lhi + c * kLHiChunkBytes + lane * 4);
    r.s[0] = ldg32(blk + p.off_sL + gr * 4);
  } else {
    const int c = 2 * (ks - p.n_res - p.n_L);
    r.c = ldg128(blk + p.off_A + c * kAChunkBytes + lane * 16);
    if (c + 1 < p.n_A) r.x = ldg128(blk + p.off_A + (c + 1) * kAChunkBytes + lane * 16);
    r.s[0] = ldg32(blk + p.off_sA + gr * 4);
  }
}

__device__ __forceinline__ void sts128(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}

// A chunk's 16 rows x 64 columns into the swizzled tile: lane (gr, cc) holds 16
// columns of rows gr and gr + 8, stored as columns 16 cc .. 16 cc + 15 (32
// contiguous bytes of each row; the order is undone when dX is written).
template <int GM>
__device__ __forceinline__ void store_chunk(const DequantParams& p, const RawChunk<GM>& r, int ks, uint32_t lo, uint32_t hi) {
  uint32_t a[4][4], s0[4], s1[4];
  if (ks < p.n_res) {
    const uint32_t w[4] = {r.c.x, r.c.y, r.c.z, r.c.w};
#pragma unroll
    for (int st = 0; st < 4; ++st) {
      unpack_int4_signed(w[st], a[st]);
      if (st % (4 >> GM) == 0) scales_of(r.s[st >> (2 - GM)], p.sc_res, s0[st], s1[st]);
      else s0[st] = s0[st - 1], s1[st] = s1[st - 1];
    }
  } else {
    if (ks < p.n_res + p.n_L) {
      unpack_int5_signed<0>(r.c.x, r.x.x, a[0]);
      unpack_int5_signed<1>(r.c.y, r.x.x, a[1]);
      unpack_int5_signed<2>(r.c.z, r.x.x, a[2]);
      unpack_int5_signed<3>(r.c.w, r.x.x, a[3]);
      scales_of(r.s[0], p.sc_L, s0[0], s1[0]);
    } else {
      unpack_int8_signed(r.c.x, r.c.y, a[0]);
      unpack_int8_signed(r.c.z, r.c.w, a[1]);
      if (2 * (ks - p.n_res - p.n_L) + 1 < p.n_A) {
        unpack_int8_signed(r.x.x, r.x.y, a[2]);
        unpack_int8_signed(r.x.z, r.x.w, a[3]);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) a[2][i] = a[3][i] = 0u;
      }
      scales_of(r.s[0], p.sc_A, s0[0], s1[0]);
    }
#pragma unroll
    for (int st = 1; st < 4; ++st) s0[st] = s0[0], s1[st] = s1[0];
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t at = h ? hi : lo;
    const int i = 2 * h, j = 2 * h + 1;
    sts128(at, hmul2_bits(a[i][0], s0[i]), hmul2_bits(a[i][2], s0[i]), hmul2_bits(a[j][0], s0[j]), hmul2_bits(a[j][2], s0[j]));
    sts128(at + 1024u, hmul2_bits(a[i][1], s1[i]), hmul2_bits(a[i][3], s1[i]), hmul2_bits(a[j][1], s1[j]),
           hmul2_bits(a[j][3], s1[j]));
  }
}

template <int GM>
__global__ void __launch_bounds__(kGwWarps * 32, 1) gw_kernel(const GwParams p, const __grid_constant__ CUtensorMap mg) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t tiles = smem_addr(base), gtiles = tiles + kGwGOff;
  const uint32_t wfull = tiles + p.bar_off, wempty = wfull + 8 * kGwStages, gfull = wempty + 8 * kGwStages,
                 gempty = gfull + 32, done = gempty + 32;
  uint32_t* tmem = reinterpret_cast<uint32_t*>(base + p.bar_off + 16 * kGwStages + 72);
  int* flag = reinterpret_cast<int*>(tmem + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kGwStages; ++s) {
      mbar_init(wfull + 8 * s, 8);
      mbar_init(wempty + 8 * s, 1);
    }
    for (int s = 0; s < 4; ++s) {
      mbar_init(gfull + 8 * s, 1);
      mbar_init(gempty + 8 * s, 1);
    }
    mbar_init(done, 1);
    *flag = 0;
    mbar_fence_init();
  }
  if (warp == 17) {
    tmem_alloc(smem_addr(tmem), kGTmem);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *tmem;

  // This CTA: column group, its chunks and blocks, its k-steps.
  const int u = blockIdx.x;
  const bool whole = u < p.full * p.s_full;
  const int group = whole ? u / p.s_full : p.full;
  const int split = whole ? u - group * p.s_full : u - p.full * p.s_full, splits = whole ? p.s_full : p.s_last;
  const int c0 = group * p.nb * 4, nc = min(4 * p.nb, p.chunks - c0), nbl = (nc + 3) / 4;
  const int k0 = static_cast<int>(static_cast<int64_t>(p.nk) * split / splits);
  const int k1 = static_cast<int>(static_cast<int64_t>(p.nk) * (split + 1) / splits);

  if (warp < 16) {
    const int set = warp >> 3, j = warp & 3, half = (warp >> 2) & 1, total = (k1 - k0) * nbl;
    const int gr = lane >> 2, cc = lane & 3;
    // byte offsets of this lane inside a tile: row 16 j + gr, 16-byte pieces 2 cc and 2 cc + 1 (swizzled by the row)
    const uint32_t row = static_cast<uint32_t>((16 * j + gr) * 128) + half * 16384u;
    const uint32_t o_lo = row + static_cast<uint32_t>(((2 * cc) ^ gr) * 16), o_hi = row + static_cast<uint32_t>(((2 * cc + 1) ^ gr) * 16);
    RawChunk<GM> raw[kGwAhead][2];
    int pit = set, pk = k0 + set / nbl, pb = set % nbl;   // the tile to load next
    auto load = [&](RawChunk<GM> (&r)[2]) {
      const int mt = 4 * pk + j, c = 4 * pb + 2 * half;
      if (pit < total && mt < p.n_mtiles) {
        const uint8_t* blk = p.rows.mtiles + static_cast<size_t>(mt) * p.rows.mblk_bytes;
        if (c < nc) load_chunk<GM>(p.rows, blk, c0 + c, lane, r[0]);
        if (c + 1 < nc) load_chunk<GM>(p.rows, blk, c0 + c + 1, lane, r[1]);
      }
      pit += 2;
      pb += 2;
      while (pb >= nbl) {
        pb -= nbl;
        ++pk;
      }
    };
#pragma unroll
    for (int i = 0; i < kGwAhead; ++i) load(raw[i]);
    int k = k0 + set / nbl, b = set % nbl;
    bool ok = true;
    for (int it = set; it < total && ok;) {
#pragma unroll
      for (int i = 0; i < kGwAhead; ++i) {
        if (it >= total || !ok) break;
        const int s = it & (kGwStages - 1), c = 4 * b + 2 * half;
        ok = warp_wait(flag, wempty + 8 * s, ((it / kGwStages) & 1) ^ 1, p.status);
        if (!ok) break;
        const uint32_t tile = tiles + s * kGwTile;
        if (4 * k + j < p.n_mtiles) {
          if (c < nc) store_chunk<GM>(p.rows, raw[i][0], c0 + c, tile + o_lo, tile + o_hi);
          if (c + 1 < nc) store_chunk<GM>(p.rows, raw[i][1], c0 + c + 1, tile + o_lo + 8192u, tile + o_hi + 8192u);
        } else {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            sts128(tile + o_lo + h * 8192u, 0u, 0u, 0u, 0u);
            sts128(tile + o_lo + h * 8192u + 1024u, 0u, 0u, 0u, 0u);
            sts128(tile + o_hi + h * 8192u, 0u, 0u, 0u, 0u);
            sts128(tile + o_hi + h * 8192u + 1024u, 0u, 0u, 0u, 0u);
          }
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive(wfull + 8 * s);
        load(raw[i]);
        it += 2;
        b += 2;
        while (b >= nbl) {
          b -= nbl;
          ++k;
        }
      }
    }
    // The accumulators: lane quarter w % 4 (columns of W~), every fourth block
    // of 128 columns, 16 tokens at a time.
    if (warp_wait(flag, done, 0u, p.status)) {
      tc_fence_after();
      const int q = warp & 3, m = 32 * q + lane, at = m & 63;
      // the column's place in the operand order
      const int pos = (m & 64) + ((at >> 2) & 3) * 16 + (at >> 4) * 4 + (at & 3);
      float* dx = p.dx + split * p.split_stride + c0 * 64;
      for (int blk = warp >> 2; 2 * blk < nc; blk += 4) {
        for (int t0 = 0; t0 < p.T; t0 += 16) {
          uint32_t r[16];
          tmem_ld_32x32b_x16(tbase + (static_cast<uint32_t>(32 * q) << 16) + blk * p.N + t0, r);
          tmem_ld_wait();
          if (2 * blk + (m >> 6) < nc) {
#pragma unroll
            for (int i = 0; i < 16; ++i)
              if (t0 + i < p.T) dx[static_cast<size_t>(t0 + i) * p.rows.Kc + blk * 128 + pos] = __uint_as_float(r[i]);
          }
          __syncwarp();
        }
      }
      tc_fence_before();
    }
  } else if (warp == 16) {
    int issued = 0;
    bool ok = true;
    for (int k = k0; k < k1 && ok; ++k, ++issued) {
      const int s = issued % p.gstages;
      ok = warp_wait(flag, gempty + 8 * s, ((issued / p.gstages) & 1) ^ 1, p.status);
      if (!ok) break;
      if (elect_one()) {
        mbar_arrive_expect_tx(gfull + 8 * s, p.g_bytes);
        tma_load_2d(gtiles + s * p.g_bytes, &mg, k * 64, 0, gfull + 8 * s);
      }
      __syncwarp();
    }
    if (!ok) {
      // Copies still in flight land before the block's shared memory goes away.
      const int back = min(issued, p.gstages);
      for (int i = 1; i <= back; ++i) mbar_wait(gfull + 8 * ((issued - i) % p.gstages), ((issued - i) / p.gstages) & 1u);
    }
  } else {
    const uint32_t idesc = tc_idesc_f16(128, p.N) | kTcIdescAmn;
    const uint64_t ad0 = smem_desc_mn128(tiles, 8192u), bd0 = smem_desc_k128(gtiles);
    bool ok = true;
    int it = 0;
    for (int k = k0; k < k1 && ok; ++k) {
      const int gs = (k - k0) % p.gstages;
      ok = warp_wait(flag, gfull + 8 * gs, ((k - k0) / p.gstages) & 1, p.status);
      if (!ok) break;
      const uint64_t bd = bd0 + static_cast<uint64_t>(gs) * (p.g_bytes >> 4);
      for (int b = 0; b < nbl; ++b, ++it) {
        const int s = it & (kGwStages - 1);
        ok = warp_wait(flag, wfull + 8 * s, (it / kGwStages) & 1, p.status);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
          const uint64_t a = ad0 + static_cast<uint64_t>(s) * (kGwTile >> 4);
          const uint32_t d = tbase + 2 * b * p.N;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            if (4 * b + 2 * i < nc) {
#pragma unroll
              for (int e = 0; e < 4; ++e)
                tc_mma_ss(d + i * p.N, a + i * 1024 + e * 128, bd + 2 * e, idesc, (k != k0 || e != 0) ? 1u : 0u);
            }
          }
          tc_commit(wempty + 8 * s);
          if (b == nbl - 1) tc_commit(gempty + 8 * gs);
        }
        __syncwarp();
      }
    }
    if (ok && elect_one()) tc_commit(done);
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 17) {
    tc_fence_after();
    tmem_dealloc(tbase, kGTmem);
  }
}

// -------------------------------------------------------------------- host
constexpr int kFewTokens = 128;   // up to here the packed rows are dequantised inside the second product

// Work split of gw_kernel.
struct GwPlan {
  int N, nb, chunks, full, s_full, s_last, nk;
};
GwPlan gw_plan(const archead_handle& h, int T) {
  GwPlan g{};
  g.N = (T + 15) / 16 * 16;
  g.chunks = tc_kc(h.L) / 64;
  g.nk = (h.L.n_mtiles + 3) / 4;
  // As many column blocks as the TMEM holds (G is read once per group), fewer
  // where the head is too small to give every SM a few tiles.
  for (g.nb = kGwMaxN / g.N; g.nb > 1; --g.nb)
    if (static_cast<int64_t>((g.chunks + 4 * g.nb - 1) / (4 * g.nb)) * g.nk >= 8 * h.num_sms) break;
  g.full = g.chunks / (4 * g.nb);
  const int rest = g.chunks - g.full * 4 * g.nb;
  const auto share = [&](int c) {
    return std::max(1, std::min(g.nk, static_cast<int>(static_cast<int64_t>(h.num_sms) * c / g.chunks)));
  };
  g.s_full = g.full > 0 ? share(4 * g.nb) : 0;
  g.s_last = rest > 0 ? share(rest) : 0;
  return g;
}

struct GradLayout {
  bool few;
  int tokens, chunk, splits, Kz;   // tokens and vocabulary rows per pass; partial dX (K splits)
  int pitch, n_ssum;
  size_t fwd, logits, cinv, ssum, xop, w, g, dx, dz, rb, escale, zhi, zlo, total;
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
  o.few = T <= kFewTokens;
  const size_t t = o.few ? T : std::min(T, kGradTokens);
  o.tokens = static_cast<int>(t);
  if (o.few) {
    // The forward call's workspace comes first: its header is this one's.
    o.fwd = ws_layout(h, T).total;
    at = round_up(o.fwd, 256);
    o.pitch = static_cast<int>(round_up(L.Vp, 64));
    o.n_ssum = (L.Vp + kGPiece - 1) / kGPiece;
    o.logits = take(t * L.V * 4);
    const GwPlan g = gw_plan(h, T);
    o.splits = std::max(g.s_full, g.s_last);
  } else {
    const int n_chunks = (L.Vp + kGradChunk - 1) / kGradChunk;
    o.chunk = static_cast<int>(round_up((L.Vp + n_chunks - 1) / n_chunks, kGN));
    o.pitch = o.chunk;
    o.n_ssum = (L.Vp + kGN - 1) / kGN;
    // Few tiles: the accumulation splits its K (the rows of a chunk) so that
    // every SM has a unit; the splits are added in order at the end.
    const int tiles = ((o.tokens + kGM - 1) / kGM) * ((Kc + kGN - 1) / kGN);
    o.splits = std::max(1, std::min(h.num_sms / tiles, o.chunk / 256));
    o.cinv = take(t * 4);
    o.xop = take(t * Kc * 2);
    o.w = take(static_cast<size_t>(o.chunk) * Kc * 2);
  }
  o.ssum = take(o.n_ssum * t * 4);
  o.g = take(t * o.pitch * 2);
  o.dx = take(static_cast<size_t>(o.splits) * t * Kc * 4);
  o.dz = take(t * o.Kz * 2);
  o.rb = take(static_cast<size_t>(o.Kz) * L.d * 2);
  if (!o.few && !h.tc_ok) {
    o.escale = take(t * 4);
    o.zhi = take(t * L.Kz * 2);
    o.zlo = take(t * L.Kz * 2);
  }
  o.total = at;
  return o;
}

// X and 2^-c_t of one pass's tokens.
cudaError_t grad_activations(const archead_handle& h, const GradLayout& o, const uint16_t* hidden, int T, uint8_t* wb,
                             cudaStream_t stream) {
  const Layout& L = h.L;
  uint32_t* status = reinterpret_cast<uint32_t*>(wb + 4);
  if (h.tc_ok) {
    ActParams ap = act_params(h);
    ap.hidden = hidden;
    ap.status = status;
    ap.xop = reinterpret_cast<uint16_t*>(wb + o.xop);
    ap.cinv = reinterpret_cast<float*>(wb + o.cinv);
    ap.T = T;
    ap.zpart = reinterpret_cast<float*>(wb + o.dx);   // dX is written later
    ap.zticket = reinterpret_cast<uint32_t*>(wb + kActTicketOff);
    return launch_act_prep(ap, act_prep_splits(T, L.d, ap.Kc, h.num_sms, o.dz - o.dx), stream);
  }
  PrologueParams pp{};
  pp.hidden = hidden;
  pp.R = reinterpret_cast<const int8_t*>(h.arena + L.off_R);
  pp.s_R = reinterpret_cast<const uint16_t*>(h.arena + L.off_sR);
  pp.B = reinterpret_cast<const int8_t*>(h.arena + L.off_B);
  pp.s_B = reinterpret_cast<const uint16_t*>(h.arena + L.off_sB);
  pp.zhi = reinterpret_cast<uint16_t*>(wb + o.zhi);
  pp.zlo = reinterpret_cast<uint16_t*>(wb + o.zlo);
  pp.escale = reinterpret_cast<int32_t*>(wb + o.escale);
  pp.counter = reinterpret_cast<uint32_t*>(wb);
  pp.status = status;
  pp.e_B = h.e_B;
  pp.T = T;
  pp.d = L.d;
  pp.rcp = L.rcp;
  pp.rrp = L.rrp;
  pp.Kz = L.Kz;
  pp.g_B = L.g_B;
  pp.V = L.V;
  pp.v_total = h.v_total;
  cudaError_t e = launch_prologue(pp, stream);
  if (e != cudaSuccess) return e;
  XParams xp{hidden, pp.zhi, pp.zlo, pp.escale, reinterpret_cast<uint16_t*>(wb + o.xop),
             reinterpret_cast<float*>(wb + o.cinv), L.d, L.rcp, L.Kz, tc_kc(L), h.tc_alpha, h.tc_beta, h.tc_gamma,
             h.tc_mseg, h.e_B};
  x_from_z_kernel<<<T, 256, 0, stream>>>(xp);
  return cudaGetLastError();
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

// The rows of R and B for the last product.
int grad_lowrank(const GradCall& c) {
  const Layout& L = c.h.L;
  if (c.o.Kz == 0) return ARCHEAD_OK;
  LowrankParams lp{reinterpret_cast<const int8_t*>(c.h.arena + L.off_R),
                   reinterpret_cast<const uint16_t*>(c.h.arena + L.off_sR),
                   reinterpret_cast<const int8_t*>(c.h.arena + L.off_B),
                   reinterpret_cast<const uint16_t*>(c.h.arena + L.off_sB),
                   reinterpret_cast<uint16_t*>(c.wb + c.o.rb), L.d, L.rcp, L.rrp, c.o.Kz, L.g_B,
                   std::ldexp(1.f, c.sigma - c.h.tc_beta), std::ldexp(1.f, c.sigma - c.h.tc_gamma)};
  lowrank_rows_kernel<<<c.o.Kz, 256, 0, c.stream>>>(lp);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? ARCHEAD_OK : set_cuda_error(e);
}

// dX -> dh of one pass's tokens.
int grad_finish(const GradCall& c, GemmParams& p, int splits, int splits_last, int last) {
  const Layout& L = c.h.L;
  const int Kc = tc_kc(L), Kz = c.o.Kz, nt = p.M;
  uint16_t* dz = reinterpret_cast<uint16_t*>(c.wb + c.o.dz);
  DxParams dp{dequant_params(c.h, nullptr), p.ssum, p.grad, p.targets, p.dx, p.split_stride, dz, c.o.n_ssum, nt, Kc, L.d,
              L.V, c.h.row0, c.h.v_total == L.V ? 1 : 0, splits, splits_last, last};
  dx_kernel<<<dim3(nt, (Kc + 1023) / 1024), 256, 0, c.stream>>>(dp);
  cudaError_t e = cudaGetLastError();
  CUtensorMap mz{}, mr{};
  if (e == cudaSuccess && Kz > 0) {
    e = tc_encode_map(&mz, dz, Kz, nt, Kz, kGM);
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
  float* logits = reinterpret_cast<float*>(c.wb + c.o.logits);
  const int rc = forward_logits(h, hidden, T, logits, c.wb, c.o.fwd, c.stream);
  if (rc != ARCHEAD_OK) return rc;
  GParams gp{logits, p.lse, p.grad, p.targets, p.G, p.ssum, T, L.V, L.Vp, h.row0, c.o.pitch};
  g_kernel<<<dim3(c.o.n_ssum, T), 256, 0, c.stream>>>(gp);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return set_cuda_error(e);
  const GwPlan g = gw_plan(h, T);
  GwParams w{};
  w.rows = dequant_params(h, nullptr);
  w.n_mtiles = L.n_mtiles;
  w.nk = g.nk;
  w.T = T;
  w.N = g.N;
  w.nb = g.nb;
  w.chunks = g.chunks;
  w.full = g.full;
  w.s_full = g.s_full;
  w.s_last = g.s_last;
  w.g_bytes = static_cast<uint32_t>(g.N) * 128u;
  w.gstages = static_cast<int>(std::min<uint32_t>(4, (kGwSmemMax - kGwGOff - 256) / w.g_bytes));
  w.bar_off = kGwGOff + w.gstages * w.g_bytes;
  w.dx = p.dx;
  w.split_stride = p.split_stride;
  w.status = p.status;
  CUtensorMap mg;
  e = tc_encode_map(&mg, p.G, L.Vp, T, c.o.pitch, g.N);
  if (e != cudaSuccess) return set_cuda_error(e);
  const int grid = g.full * g.s_full + g.s_last;
  const uint32_t smem = w.bar_off + 256 + 1024;
  if (w.rows.g_log2 >= 6) gw_kernel<0><<<grid, kGwWarps * 32, smem, c.stream>>>(w, mg);
  else if (w.rows.g_log2 == 5) gw_kernel<1><<<grid, kGwWarps * 32, smem, c.stream>>>(w, mg);
  else gw_kernel<2><<<grid, kGwWarps * 32, smem, c.stream>>>(w, mg);
  e = cudaGetLastError();
  if (e != cudaSuccess) return set_cuda_error(e);
  return grad_finish(c, p, g.s_full, g.s_last, g.full * g.nb * 256);
}

// Many tokens: chunk by chunk through the dequantised rows.
int grad_many(const GradCall& c, const uint16_t* hidden, GemmParams& p) {
  const archead_handle& h = c.h;
  const Layout& L = h.L;
  const GradLayout& o = c.o;
  const int Kc = tc_kc(L), nt = p.M;
  uint16_t* w = reinterpret_cast<uint16_t*>(c.wb + o.w);
  cudaError_t e = grad_activations(h, o, hidden, nt, c.wb, c.stream);
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
    if (e == cudaSuccess) e = tc_encode_map(&mx, xop, Kc, nt, Kc, kGM);
    if (e == cudaSuccess) e = tc_encode_map(&mg, p.G, rows, nt, o.pitch, kGM);
    if (e == cudaSuccess) e = tc_encode_map(&mwk, w, Kc, rows, Kc, kGN);
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
  return grad_finish(c, p, o.splits, o.splits, Kc);
}

int grad_launch(const archead_handle& h, const GradLayout& o, const uint16_t* hidden, int T, const int32_t* targets,
                const float* lse, const float* grad, void* out, bool out_f32, uint8_t* wb, cudaStream_t stream) {
  const Layout& L = h.L;
  GradCall c{h, o, wb, stream, L.r_c > 0 ? h.tc_beta + h.tc_rho_c : 1 << 20};
  if (L.r_r > 0) c.sigma = std::min(c.sigma, h.tc_gamma + h.tc_rho_r);
  if (o.Kz == 0) c.sigma = 0;
  // The header: status word, tickets of the activation kernel.
  const cudaError_t e = cudaMemsetAsync(wb, 0, 256, stream);
  if (e != cudaSuccess) return set_cuda_error(e);
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
    p.tokens = nt;
    p.dx = reinterpret_cast<float*>(wb + o.dx);
    p.Kc = tc_kc(L);
    p.split_stride = static_cast<size_t>(nt) * p.Kc;
    p.out = out_f32 ? static_cast<void*>(static_cast<float*>(out) + first) : static_cast<void*>(static_cast<uint16_t*>(out) + first);
    p.out_f32 = out_f32 ? 1 : 0;
    rc = o.few ? grad_few(c, hidden + first, p) : grad_many(c, hidden + first, p);
  }
  return rc;
}

constexpr int kMaxTokens = 1 << 20;

}  // namespace

cudaError_t grad_set_attributes() {
  cudaError_t e = cudaFuncSetAttribute(grad_gemm_kernel<kSoftmax>, cudaFuncAttributeMaxDynamicSharedMemorySize, kGSmem);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(grad_gemm_kernel<kAccumulate>, cudaFuncAttributeMaxDynamicSharedMemorySize, kGSmem);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(grad_gemm_kernel<kFinish>, cudaFuncAttributeMaxDynamicSharedMemorySize, kGSmem);
  for (const void* k : {reinterpret_cast<const void*>(&gw_kernel<0>), reinterpret_cast<const void*>(&gw_kernel<1>),
                        reinterpret_cast<const void*>(&gw_kernel<2>)})
    if (e == cudaSuccess) e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kGwSmemMax + 1024);
  return e;
}

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
  return grad_launch(*handle, o, hidden, T, targets, lse, grad_ce, grad_hidden, grad_dtype == ARCHEAD_GRAD_F32,
                     static_cast<uint8_t*>(workspace), reinterpret_cast<cudaStream_t>(stream));
}
