// Rows to their experts' order and back (gfx950), by the plan of a routing:
// place[t][j] is the row of token t's j-th choice, or outside [0, rows) where
// it has none.
//
//   dispatch          out[place[t][j]] = x[t]
//   combine           y[t] = beta y[t] + sum_j w[t][j] h[place[t][j]]   (w = 1: dispatch's gradient)
//   combine gradient  dh[place[t][j]] = w[t][j] dy[t],  dw[t][j] = <dy[t], h[place[t][j]]>
//
// All of them go token by token, so that a token's own row is read or written
// once whatever k is, and rows of no choice are neither read nor written.  They
// are bound by HBM: 8192 tokens of 4096 bf16, k = 8, take 105 us to dispatch (5.8
// TB/s), 113 to combine (5.3) and 206 for the combine's gradient (5.5).  A unit is
// 16 bytes of a row, at any alignment of elements; the last of a row may hold fewer.
#pragma once

#include "common.hpp"
#include "grouped_kernels.hpp"

namespace mfsdp {

constexpr int kExchangeFlight = 8;    // rows of one token in flight

struct ExchangeArgs {
  const void* x;          // dispatch: x; combine: h; gradient: h
  const void* dy;         // gradient: dy
  const int32_t* place;   // tokens x k
  const float* weights;   // tokens x k, or null
  void* out;              // dispatch: rows; combine: y; gradient: dh
  float* dw;              // gradient: tokens x k
  int64_t ldx, ldy, ldo;
  int32_t tokens, rows, k, d;
  int32_t tpt;            // threads per token, up to 256; in the gradient 64, 128 or 256
  int32_t chunks;         // workgroups per token (dispatch, combine)
  float beta;
};

// Streamed load of 16 bytes at any element.
__device__ __forceinline__ uint4 load16_stream(const void* p) {
  const u32x4_t v = __builtin_nontemporal_load((const MFSDP_GLOBAL u32x4_el_t*)(p));
  return make_uint4(v.x, v.y, v.z, v.w);
}

// 16 bytes of E from p on, of which `left` elements exist (others 0).  (STREAM as an
// argument would be lost: the compiler merges two loads that differ in it alone.)
template <class E, bool STREAM = false>
__device__ __forceinline__ uint4 unit_load(const typename E::storage_t* p, int left) {
  using S = typename E::storage_t;
  if constexpr (STREAM) {
    if (left >= E::kVec) return load16_stream(p);
  } else {
    if (left >= E::kVec) return load16_any(p);
  }
  S v[E::kVec];
#pragma unroll
  for (int i = 0; i < E::kVec; ++i) v[i] = i < left ? gld<S>(p + i) : S(0);
  uint4 r;
  __builtin_memcpy(&r, v, 16);
  return r;
}

template <class E>
__device__ __forceinline__ void unit_store(typename E::storage_t* p, int left, const uint4& v) {
  using S = typename E::storage_t;
  if (left >= E::kVec) {
    stream16_any(p, v);
    return;
  }
  S s[E::kVec];
  __builtin_memcpy(s, &v, 16);
#pragma unroll
  for (int i = 0; i < E::kVec; ++i)
    if (i < left) gst<S>(p + i, s[i]);
}

// Token and first unit of this thread: 256 / tpt tokens per workgroup, or
// several workgroups per token.
struct ExchangeUnit {
  int64_t t;
  int u, step;
  __device__ __forceinline__ explicit ExchangeUnit(const ExchangeArgs& a) {
    const int per = 256 / a.tpt;
    const int64_t b = blockIdx.x / a.chunks;
    t = static_cast<int>(threadIdx.x) < per * a.tpt ? b * per + threadIdx.x / a.tpt : a.tokens;   // none
    u = static_cast<int>(blockIdx.x % a.chunks) * a.tpt + static_cast<int>(threadIdx.x % a.tpt);
    step = a.chunks * a.tpt;
  }
};

template <class E>
__global__ __launch_bounds__(256) void dispatch_kernel(ExchangeArgs a) {
  using S = typename E::storage_t;
  constexpr int V = E::kVec;
  const ExchangeUnit at(a);
  if (at.t >= a.tokens) return;
  const S* x = static_cast<const S*>(a.x) + at.t * a.ldx;
  const int32_t* place = a.place + at.t * a.k;
  const int units = (a.d + V - 1) / V;
  for (int u = at.u; u < units; u += at.step) {
    const uint4 v = unit_load<E>(x + u * V, a.d - u * V);
    for (int j = 0; j < a.k; ++j) {
      const int r = place[j];
      if (r >= 0 && r < a.rows) unit_store<E>(static_cast<S*>(a.out) + r * a.ldo + u * V, a.d - u * V, v);
    }
  }
}

// STREAM: experts' rows past what the last-level cache holds pass the L2s by: 8192
// tokens of 4096 bf16, k = 8 (537 MB) 119 -> 113 us, its gradient 232 -> 208; with k
// = 2 (134 MB) 41 -> 52 and 58 -> 72.
template <class E, bool STREAM>
__global__ __launch_bounds__(256) void combine_kernel(ExchangeArgs a) {
  using S = typename E::storage_t;
  constexpr int V = E::kVec;
  const ExchangeUnit at(a);
  if (at.t >= a.tokens) return;
  const int32_t* place = a.place + at.t * a.k;
  const float* w = a.weights ? a.weights + at.t * a.k : nullptr;
  S* y = static_cast<S*>(a.out) + at.t * a.ldo;
  const int units = (a.d + V - 1) / V;
  for (int u = at.u; u < units; u += at.step) {
    const int left = a.d - u * V;
    float acc[V];
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = 0.f;
    for (int j0 = 0; j0 < a.k; j0 += kExchangeFlight) {
      uint4 raw[kExchangeFlight];
      float wj[kExchangeFlight];
#pragma unroll
      for (int j = 0; j < kExchangeFlight; ++j) {
        const int r = j0 + j < a.k ? place[j0 + j] : -1;
        const bool on = r >= 0 && r < a.rows;
        wj[j] = on ? (w ? w[j0 + j] : 1.f) : 0.f;
        raw[j] = make_uint4(0, 0, 0, 0);
        if (on) raw[j] = unit_load<E, STREAM>(static_cast<const S*>(a.x) + r * a.ldx + u * V, left);
      }
#pragma unroll
      for (int j = 0; j < kExchangeFlight; ++j) {
        float v[V];
        Vec16<E>::unpack(raw[j], v);
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] = fmaf(wj[j], v[i], acc[i]);
      }
    }
    if (a.beta != 0.f) {
      float old[V];
      Vec16<E>::unpack(unit_load<E>(y + u * V, left), old);
#pragma unroll
      for (int i = 0; i < V; ++i) acc[i] = fmaf(a.beta, old[i], acc[i]);
    }
    unit_store<E>(y + u * V, left, Vec16<E>::pack(acc));
  }
}

// One token per tpt threads: the inner products are sums over its whole row,
// added in fp32 by thread, by wave (a tree) and by waves in their order.
template <class E, bool STREAM>
__global__ __launch_bounds__(256) void combine_grad_kernel(ExchangeArgs a) {
  using S = typename E::storage_t;
  constexpr int V = E::kVec;
  __shared__ float part[4][kExchangeFlight];
  const ExchangeUnit at(a);
  const bool on_t = at.t < a.tokens;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int units = on_t ? (a.d + V - 1) / V : 0;
  const int64_t t = on_t ? at.t : 0;
  const S* dy = static_cast<const S*>(a.dy) + t * a.ldy;
  for (int j0 = 0; j0 < a.k; j0 += kExchangeFlight) {
    int r[kExchangeFlight];
    float w[kExchangeFlight], dot[kExchangeFlight];
#pragma unroll
    for (int j = 0; j < kExchangeFlight; ++j) {
      const int row = j0 + j < a.k ? a.place[t * a.k + j0 + j] : -1;
      r[j] = row >= 0 && row < a.rows ? row : -1;
      w[j] = r[j] >= 0 ? a.weights[t * a.k + j0 + j] : 0.f;
      dot[j] = 0.f;
    }
    for (int u = at.u; u < units; u += at.step) {
      const int left = a.d - u * V;
      uint4 raw[kExchangeFlight];
      const uint4 g = unit_load<E>(dy + u * V, left);
#pragma unroll
      for (int j = 0; j < kExchangeFlight; ++j) {
        raw[j] = make_uint4(0, 0, 0, 0);
        if (r[j] >= 0) raw[j] = unit_load<E, STREAM>(static_cast<const S*>(a.x) + r[j] * a.ldx + u * V, left);
      }
      float gv[V];
      Vec16<E>::unpack(g, gv);
#pragma unroll
      for (int j = 0; j < kExchangeFlight; ++j) {
        if (r[j] < 0) continue;
        float h[V], o[V];
        Vec16<E>::unpack(raw[j], h);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          dot[j] = fmaf(gv[i], h[i], dot[j]);
          o[i] = w[j] * gv[i];
        }
        unit_store<E>(static_cast<S*>(a.out) + r[j] * a.ldo + u * V, left, Vec16<E>::pack(o));
      }
    }
#pragma unroll
    for (int j = 0; j < kExchangeFlight; ++j) dot[j] = warp_sum(dot[j]);
    const int waves = a.tpt / 64, first = wave / waves * waves;
    if (waves > 1) {
      __syncthreads();      // the sums of the choices before have been read
      if (lane == 0) {
#pragma unroll
        for (int j = 0; j < kExchangeFlight; ++j) part[wave][j] = dot[j];
      }
      __syncthreads();
    }
    if (wave == first && lane < kExchangeFlight && on_t && j0 + lane < a.k) {
      float s = 0.f;
      if (waves > 1) {
        for (int q = 0; q < waves; ++q) s += part[first + q][lane];
      } else {
#pragma unroll
        for (int j = 0; j < kExchangeFlight; ++j)
          if (lane == j) s = dot[j];
      }
      a.dw[t * a.k + j0 + lane] = s;
    }
  }
}

}  // namespace mfsdp
