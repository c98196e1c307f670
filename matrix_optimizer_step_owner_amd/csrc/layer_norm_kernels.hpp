// Layer norm and its gradients (gfx950), for rows of d values in fp32 arithmetic:
//
//   m = mean(x) (0 if not centred), v = mean((x - m)^2), r = 1 / sqrt(v + eps)
//   xh = (x - m) r,   y = xh w + b
//   g = dy w,  dx = r (g - xh mean(g xh) - mean(g))     (the last if centred)
//   dw = beta dw + sum_rows dy xh,   db = beta db + sum_rows dy
//
// The gradient reads x and dy once: m and r are computed again from the row
// that is at hand, so the forward keeps nothing.  The sums over rows are those
// of each workgroup's rows, in their order, and then of the workgroups' in
// theirs, in two launches: no atomics, equal inputs give equal bits.
//
// One workgroup takes one row at a time, UPT units of 16 bytes per thread in
// registers (UPT = 0: rows that do not fit, read again from the caches).  Bound
// by HBM.
#pragma once

#include "common.hpp"
#include "exchange_kernels.hpp"

namespace mfsdp {

struct NormArgs {
  const void* x;         // rows x d, row stride ldx
  const void* dy;        // rows x d, row stride ldy
  const void* w;         // d, fp32 or bf16
  const void* b;         // d, the type of w, or null
  void* out;             // y or dx, row stride ldo
  float* part;           // [groups][dbias ? 2 : 1][d] partial sums
  float* dw;             // d
  float* db;             // d, or null
  int64_t ldx, ldy, ldo;
  int32_t rows, d;
  int32_t centered, w_bf16;
  int32_t groups;        // workgroups of the gradient
  float eps, beta;
};

constexpr int kNormThreadsMax = 512;

// Sum over the workgroup, on every thread; `part` is used twice in turn.
template <int N>
__device__ __forceinline__ void norm_sum(float (&v)[N], float (*part)[N]) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = warp_sum(v[i]);
  if (waves == 1) return;
  __syncthreads();
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) part[wave][i] = v[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    float s = 0.f;
    for (int w = 0; w < waves; ++w) s += part[w][i];
    v[i] = s;
  }
}

// V values of a weight (or bias) from column c on, `left` of them.
template <int V>
__device__ __forceinline__ void norm_weight(const void* w, int bf, int c, int left, float (&v)[V]) {
#pragma unroll
  for (int i = 0; i < V; ++i) v[i] = 0.f;
  if (!w) return;
  if (left >= V) {
    if (bf) {
      const uint16_t* p = static_cast<const uint16_t*>(w) + c;
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] = bf16_to_f32(p[i]);
    } else {
      const float* p = static_cast<const float*>(w) + c;
#pragma unroll
      for (int i = 0; i < V; i += 4) {
        const uint4 t = load16_any(p + i);
        float f[4];
        Vec16<ElemF32>::unpack(t, f);
#pragma unroll
        for (int q = 0; q < 4; ++q) v[i + q] = f[q];
      }
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < V; ++i)
    if (i < left) v[i] = bf ? bf16_to_f32(static_cast<const uint16_t*>(w)[c + i]) : static_cast<const float*>(w)[c + i];
}

// First column of this thread's u-th unit.
template <int V>
__device__ __forceinline__ int norm_col(int u) {
  return (u * static_cast<int>(blockDim.x) + static_cast<int>(threadIdx.x)) * V;
}

// One row: in registers, or (UPT = 0) where it lies.
template <class E, int UPT>
struct NormRow {
  using S = typename E::storage_t;
  static constexpr int V = E::kVec;
  uint4 raw[UPT > 0 ? UPT : 1];
  const S* p;
  int d;
  __device__ __forceinline__ void load(const S* row, int d_) {
    p = row;
    d = d_;
    if constexpr (UPT > 0) {
#pragma unroll
      for (int u = 0; u < UPT; ++u) raw[u] = fetch(u);
    }
  }
  __device__ __forceinline__ uint4 fetch(int u) const {
    const int c = norm_col<V>(u);
    return c < d ? unit_load<E>(p + c, d - c) : make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void get(int u, float (&v)[V]) const {
    if constexpr (UPT > 0) Vec16<E>::unpack(raw[u], v);
    else Vec16<E>::unpack(fetch(u), v);
  }
};

// f(u) for this thread's units.
template <int UPT, int V, class F>
__device__ __forceinline__ void norm_units(int d, F&& f) {
  if constexpr (UPT > 0) {
#pragma unroll
    for (int u = 0; u < UPT; ++u) f(u);
  } else {
    for (int u = 0; norm_col<V>(u) < d; ++u) f(u);
  }
}

// Mean and 1 / sqrt(variance + eps).  Two sums: the squares' deviations are
// taken from the mean itself, so a large mean costs no digits.
template <class E, int UPT>
__device__ __forceinline__ void norm_stats(const NormArgs& a, const NormRow<E, UPT>& x, float (*part)[1],
                                           float& mean, float& r) {
  constexpr int V = E::kVec;
  mean = 0.f;
  float s[1] = {0.f};
  if (a.centered) {
    norm_units<UPT, V>(a.d, [&](int u) {
      float v[V];
      x.get(u, v);
#pragma unroll
      for (int i = 0; i < V; ++i) s[0] += v[i];
    });
    norm_sum<1>(s, part);
    mean = s[0] / static_cast<float>(a.d);
  }
  s[0] = 0.f;
  norm_units<UPT, V>(a.d, [&](int u) {
    float v[V];
    x.get(u, v);
    const int left = a.d - norm_col<V>(u);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float c = i < left ? v[i] - mean : 0.f;
      s[0] = fmaf(c, c, s[0]);
    }
  });
  norm_sum<1>(s, part);
  r = 1.f / sqrtf(s[0] / static_cast<float>(a.d) + a.eps);
}

template <class E, int UPT>
__global__ __launch_bounds__(kNormThreadsMax) void layer_norm_kernel(NormArgs a) {
  using S = typename E::storage_t;
  constexpr int V = E::kVec;
  __shared__ float part[kNormThreadsMax / 64][1];
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    NormRow<E, UPT> x;
    x.load(static_cast<const S*>(a.x) + row * a.ldx, a.d);
    float mean, r;
    norm_stats<E, UPT>(a, x, part, mean, r);
    S* y = static_cast<S*>(a.out) + row * a.ldo;
    norm_units<UPT, V>(a.d, [&](int u) {
      const int c = norm_col<V>(u), left = a.d - c;
      if (left <= 0) return;
      float v[V], w[V], b[V];
      x.get(u, v);
      norm_weight<V>(a.w, a.w_bf16, c, left, w);
      norm_weight<V>(a.b, a.w_bf16, c, left, b);
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] = fmaf((v[i] - mean) * r, w[i], b[i]);
      unit_store<E>(y + c, left, Vec16<E>::pack(v));
    });
  }
}

template <class E, int UPT>
__global__ __launch_bounds__(kNormThreadsMax) void layer_norm_grad_kernel(NormArgs a) {
  using S = typename E::storage_t;
  constexpr int V = E::kVec;
  constexpr int N = UPT > 0 ? UPT : 1;
  __shared__ float part1[kNormThreadsMax / 64][1];
  __shared__ float part2[kNormThreadsMax / 64][2];
  const int sums = a.db ? 2 : 1;
  float* pw = a.part + static_cast<size_t>(blockIdx.x) * sums * a.d;
  float* pb = pw + a.d;
  float w[N][V], accw[N][V], accb[N][V];
#pragma unroll
  for (int u = 0; u < N; ++u) {
    if constexpr (UPT > 0) norm_weight<V>(norm_col<V>(u) < a.d ? a.w : nullptr, a.w_bf16, norm_col<V>(u), a.d - norm_col<V>(u), w[u]);
#pragma unroll
    for (int i = 0; i < V; ++i) accw[u][i] = accb[u][i] = 0.f;
  }
  const float inv = 1.f / static_cast<float>(a.d);
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    NormRow<E, UPT> x, dy;
    x.load(static_cast<const S*>(a.x) + row * a.ldx, a.d);
    dy.load(static_cast<const S*>(a.dy) + row * a.ldy, a.d);
    float mean, r;
    norm_stats<E, UPT>(a, x, part1, mean, r);
    float c[2] = {0.f, 0.f};    // sums of g and g xh
    auto weight = [&](int u, float (&v)[V]) {
      if constexpr (UPT > 0) {
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = w[u][i];
      } else {
        norm_weight<V>(a.w, a.w_bf16, norm_col<V>(u), a.d - norm_col<V>(u), v);
      }
    };
    norm_units<UPT, V>(a.d, [&](int u) {
      float xv[V], gv[V], wv[V];
      x.get(u, xv);
      dy.get(u, gv);
      weight(u, wv);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float g = gv[i] * wv[i], xh = (xv[i] - mean) * r;     // past the row dy is 0
        c[0] += g;
        c[1] = fmaf(g, xh, c[1]);
      }
    });
    norm_sum<2>(c, part2);
    const float c0 = a.centered ? c[0] * inv : 0.f, c1 = c[1] * inv;
    S* dx = static_cast<S*>(a.out) + row * a.ldo;
    const bool first = row == blockIdx.x;
    norm_units<UPT, V>(a.d, [&](int u) {
      const int col = norm_col<V>(u), left = a.d - col;
      if (left <= 0) return;
      float xv[V], gv[V], wv[V], o[V], dw[V];
      x.get(u, xv);
      dy.get(u, gv);
      weight(u, wv);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float xh = (xv[i] - mean) * r;
        o[i] = r * (fmaf(-xh, c1, gv[i] * wv[i]) - c0);
        dw[i] = gv[i] * xh;
      }
      unit_store<E>(dx + col, left, Vec16<E>::pack(o));
      if constexpr (UPT > 0) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          accw[u][i] += dw[i];
          accb[u][i] += gv[i];
        }
      } else {    // this thread's own columns of the partial sums
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (i < left) {
            pw[col + i] = first ? dw[i] : pw[col + i] + dw[i];
            if (a.db) pb[col + i] = first ? gv[i] : pb[col + i] + gv[i];
          }
      }
    });
  }
  if constexpr (UPT > 0) {
#pragma unroll
    for (int u = 0; u < N; ++u) {
      const int col = norm_col<V>(u);
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (col + i < a.d) {
          pw[col + i] = accw[u][i];
          if (a.db) pb[col + i] = accb[u][i];
        }
    }
  }
}

// dw = beta dw + sum over the workgroups' partial sums: 64 columns of one of the
// two per workgroup, kNormSlices waves each with its own contiguous part.
constexpr int kNormSlices = 16;

__global__ __launch_bounds__(64 * kNormSlices) void layer_norm_sum_kernel(NormArgs a) {
  __shared__ float part[kNormSlices][64];
  const int lane = threadIdx.x & 63, slice = threadIdx.x >> 6;
  const int sums = a.db ? 2 : 1, blocks = (a.d + 63) / 64;
  const int which = blockIdx.x / blocks, c = blockIdx.x % blocks * 64 + lane;
  const int per = (a.groups + kNormSlices - 1) / kNormSlices;
  const int g0 = min(slice * per, a.groups), g1 = min(g0 + per, a.groups);
  float s = 0.f;
  if (c < a.d) {
    const float* p = a.part + static_cast<size_t>(which) * a.d + c;
#pragma unroll 8
    for (int g = g0; g < g1; ++g) s += p[static_cast<size_t>(g) * sums * a.d];
  }
  part[slice][lane] = s;
  __syncthreads();
  if (slice > 0 || c >= a.d) return;
  for (int q = 1; q < kNormSlices; ++q) s += part[q][lane];
  float* out = (which ? a.db : a.dw) + c;
  *out = a.beta != 0.f ? fmaf(a.beta, *out, s) : s;
}

}  // namespace mfsdp
