// Products grouped by expert over ragged row segments (gfx950): the linear
// layers of a mixture of experts and their gradients, whose weight gradients
// are the gradient list of the owner-local Muon step.
//
// Rows of the activations are sorted by expert; expert e owns the rows
// offsets[e] <= r < offsets[e + 1] (device int32, read by the kernels, so no
// call waits for them).  With W_e stored out x in (n x k), row-major, stacked:
//   forward          Y[r]  = X[r] W_e^T              (reduction over k)
//   input gradient   dX[r] = dY[r] W_e               (reduction over n)
//   weight gradient  dW_e  = beta dW_e + sum_r dY[r]^T X[r]
// All three are C[p][q] = sum_t P[p][t] Q[q][t] with fp32 accumulation; they
// differ in which operand is contiguous along t.
#pragma once

#include "common.hpp"
#include "ns_gemm.hpp"

namespace mfsdp {

enum GroupMode { kGroupFwd = 0, kGroupDgrad = 1, kGroupWgrad = 2 };

struct GroupArgs {
  const void* p;         // fwd: X, dgrad: dY, wgrad: dY
  const void* q;         // fwd, dgrad: W; wgrad: X (or its int8 codes)
  const uint8_t* qs;     // wgrad from a checkpoint: exponent bytes, else null
  void* out;             // Y, dX or dW
  const int32_t* off;    // experts + 1 row offsets
  int64_t ldp, ldq, ldo; // row strides in elements (ldq: wgrad's X only)
  int32_t experts, rows; // rows: rows of the activations (offsets are clamped to it)
  int32_t n, k;
  float beta;            // wgrad
  int32_t out_f32;       // wgrad: dW is fp32 whatever the operands' type
};

// Columns of an activation row that share one checkpoint scale.
constexpr int kCkptBlock = 128;

// 2^(b - 127) for an exponent byte 1 <= b <= 254; NaN for 255, the mark of a
// block that held an infinity or a NaN.
__device__ __forceinline__ float ckpt_scale(uint32_t b) {
  return b == 255u ? __uint_as_float(0x7fc00000u) : __uint_as_float(b << 23);
}

// Segment of expert e, clamped to the rows that exist: a decreasing pair is
// an empty segment.
__device__ __forceinline__ void group_segment(const GroupArgs& g, int e, int& lo, int& hi) {
  lo = min(max(g.off[e], 0), g.rows);
  hi = max(min(max(g.off[e + 1], 0), g.rows), lo);
}

// Which (expert, row tile, column tile) the b-th workgroup of a forward or
// input-gradient launch takes: expert e has ceil(rows_e / bp) * nq tiles.
// Lane l sums the tiles of experts [l*c, (l+1)*c), one scan over the wave
// gives every lane its first tile and the total, and the lane whose range
// holds the tile walks its experts.  Every wave does this for itself, with no
// barrier.  Tiles are dealt so that each XCD runs a contiguous range of them
// (xcd_remap over the number of tiles that there really are: the grid only
// bounds it).  Returns false when there is no such tile.  Row tiles run
// fastest within bands of kGroupBand, so that the workgroups an XCD runs
// together share weight panels.
constexpr int kGroupBand = 8;

__device__ __forceinline__ bool group_find(const GroupArgs& g, int b, int bp, int nq, int& expert,
                                           int& ti, int& tj) {
  const int lane = threadIdx.x & 63;
  const int c = (g.experts + 63) >> 6;
  const int e0 = min(lane * c, g.experts), e1 = min(e0 + c, g.experts);
  int sum = 0;
  for (int e = e0; e < e1; ++e) {
    int lo, hi;
    group_segment(g, e, lo, hi);
    sum += (hi - lo + bp - 1) / bp;
  }
  int incl = sum;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int v = __shfl_up(incl, d, 64);
    if (lane >= d) incl += v;
  }
  const int total = __builtin_amdgcn_readlane(incl, 63) * nq;
  if (b >= total) return false;
  const int want = xcd_remap(b, total);
  int at = (incl - sum) * nq;
  int fe = -1, fl = 0, fr = 0;
  if (want >= at && want < incl * nq) {
    for (int e = e0; e < e1; ++e) {
      int lo, hi;
      group_segment(g, e, lo, hi);
      const int np = (hi - lo + bp - 1) / bp;
      if (want < at + np * nq) {
        fe = e;
        fl = want - at;
        fr = np;
        break;
      }
      at += np * nq;
    }
  }
  const int src = __builtin_ctzll(__ballot(fe >= 0));
  expert = __builtin_amdgcn_readlane(fe, src);
  const int local = __builtin_amdgcn_readlane(fl, src);
  const int np = __builtin_amdgcn_readlane(fr, src);
  const int band = local / (kGroupBand * nq), r = local - band * (kGroupBand * nq);
  const int in_band = min(kGroupBand, np - band * kGroupBand);
  ti = band * kGroupBand + r % in_band;
  tj = r / in_band;
  return true;
}

// C tile element (p, q) of an MFMA block computed as Q-fragment x P-fragment:
// lane l and register r hold p = l % 32 and q = (r / 4) * 8 + (l / 32) * 4 +
// r % 4, four consecutive q per four registers.
__device__ __forceinline__ int acc_q(int r, int lhalf) { return (r >> 2) * 8 + lhalf * 4 + (r & 3); }

// The kernel for every alignment, stride and width: 64 x 64 tiles, four waves
// of one 32 x 32 MFMA block each, operands loaded element by element (lanes
// along whichever axis is contiguous) and stored to LDS with t contiguous.
// It takes the shapes that the 16-byte DMA kernel cannot (rows that do not
// start on 16 bytes, widths off a multiple of 16 bytes).
template <class E, int MODE, bool CKPT>
__global__ __launch_bounds__(256) void grouped_any_kernel(GroupArgs g) {
  using S = typename E::storage_t;
  constexpr int V = E::kVec;
  constexpr int BK = 4 * V;          // 32 bf16 or 16 fp32 per step: 64 bytes
  constexpr int PITCH = BK + V;      // 80 bytes: 16-byte aligned, spreads the banks
  constexpr int B = 64;
  constexpr int N_LD = B * BK / 256;
  __shared__ __align__(16) S sp[B * PITCH];
  __shared__ __align__(16) S sq[B * PITCH];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int lrow = lane & 31, lhalf = lane >> 5;

  int e, ti, tj, lo, hi;
  if (MODE == kGroupWgrad) {
    const int tq = (g.k + B - 1) / B, tp = (g.n + B - 1) / B;
    const int t = xcd_remap(blockIdx.x, gridDim.x);
    e = t / (tp * tq);
    ti = t / tq % tp;
    tj = t % tq;
  } else {
    const int nq = ((MODE == kGroupFwd ? g.n : g.k) + B - 1) / B;
    if (!group_find(g, blockIdx.x, B, nq, e, ti, tj)) return;
  }
  group_segment(g, e, lo, hi);
  const size_t wsize = static_cast<size_t>(g.n) * g.k;
  // strides of P and Q along p / q (s?) and along t (t?)
  const S* P = static_cast<const S*>(g.p);
  const S* Q = static_cast<const S*>(g.q);
  const int8_t* Qc = static_cast<const int8_t*>(g.q);
  int64_t ps, pt, qs, qt;
  int np, nq, R;
  if (MODE == kGroupWgrad) {
    P += lo * g.ldp;
    Q += lo * g.ldq;
    Qc += lo * g.ldq;
    ps = 1; pt = g.ldp; qs = 1; qt = g.ldq;
    np = g.n; nq = g.k; R = hi - lo;
  } else {
    P += lo * g.ldp;
    Q += e * wsize;
    ps = g.ldp; pt = 1;
    np = hi - lo;
    if (MODE == kGroupFwd) {
      qs = g.k; qt = 1; nq = g.n; R = g.k;
    } else {
      qs = 1; qt = g.k; nq = g.k; R = g.n;
    }
  }
  const int p0 = ti * B, q0 = tj * B;
  f32x16_t acc = f32x16_t{};
  const int wp = (wave >> 1) * 32, wq = (wave & 1) * 32;
  S rp[N_LD], rq[N_LD];
  constexpr bool kPT = MODE == kGroupWgrad, kQT = MODE != kGroupFwd;
  auto coord = [&](int j, bool along_t, int& i, int& t) {
    const int u = tid + 256 * j;
    if (along_t) { t = u % BK; i = u / BK; } else { i = u % B; t = u / B; }
  };
  auto load = [&](int t0) {
#pragma unroll
    for (int j = 0; j < N_LD; ++j) {
      int i, t;
      coord(j, !kPT, i, t);
      rp[j] = p0 + i < np && t0 + t < R ? P[(p0 + i) * ps + (t0 + t) * pt] : S(0);
      coord(j, !kQT, i, t);
      const bool in = q0 + i < nq && t0 + t < R;
      if constexpr (CKPT) {
        const int col = q0 + i;
        const int nb = (g.k + kCkptBlock - 1) / kCkptBlock;
        rq[j] = in ? E::from_f32(Qc[col + (t0 + t) * qt] *
                                 ckpt_scale(g.qs[static_cast<size_t>(lo + t0 + t) * nb + col / kCkptBlock]))
                   : S(0);
      } else {
        rq[j] = in ? Q[(q0 + i) * qs + (t0 + t) * qt] : S(0);
      }
    }
  };
  if (R > 0) load(0);
  for (int t0 = 0; t0 < R; t0 += BK) {
    __syncthreads();
#pragma unroll
    for (int j = 0; j < N_LD; ++j) {
      int i, t;
      coord(j, !kPT, i, t);
      sp[i * PITCH + t] = rp[j];
      coord(j, !kQT, i, t);
      sq[i * PITCH + t] = rq[j];
    }
    __syncthreads();
    if (t0 + BK < R) load(t0 + BK);
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const int c = (2 * s + lhalf) * V;
      const uint4 fp = *reinterpret_cast<const uint4*>(sp + (wp + lrow) * PITCH + c);
      const uint4 fq = *reinterpret_cast<const uint4*>(sq + (wq + lrow) * PITCH + c);
      Mma<E>::run(acc, fq, fp);
    }
  }
  const int p = p0 + wp + lrow;
  if (p >= np) return;
#pragma unroll
  for (int r = 0; r < 16; ++r) {
    const int q = q0 + wq + acc_q(r, lhalf);
    if (q >= nq) continue;
    if (MODE == kGroupWgrad) {
      const size_t at = e * wsize + static_cast<size_t>(p) * g.k + q;
      if (g.out_f32) {
        float* o = static_cast<float*>(g.out) + at;
        *o = g.beta == 0.f ? acc[r] : fmaf(g.beta, *o, acc[r]);
      } else {
        S* o = static_cast<S*>(g.out) + at;
        *o = E::from_f32(g.beta == 0.f ? acc[r] : fmaf(g.beta, E::to_f32(*o), acc[r]));
      }
    } else {
      static_cast<S*>(g.out)[(lo + p) * g.ldo + q] = E::from_f32(acc[r]);
    }
  }
}

}  // namespace mfsdp
