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
// Rows of up to 2048 units of 16 bytes stay in registers, UPT units per thread of L
// lanes of a wave (64 / L rows to a wave) or, L = 0, of a workgroup.  Each takes
// many rows and loads the next one while it adds up this one.  Wider rows are read again
// from the caches, and the sums over rows by a kernel over columns.
//
// Bound by HBM, and close to it by the vector units: a value costs some 14
// instructions of four cycles in the gradient, which 16 values per lane, their
// deviations kept, and two sums of two values per row (instead of three) leave it.
// 16384 rows of 5120 bf16 take 56 us forward (6.0 TB/s) and 97 to 101 for the gradients
// (5.2, the partial sums' 21 MB among the bytes), two launches in a row; one by one,
// in a profile, 82 and 5.
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
  float* stats;          // [rows][2] mean and 1 / sqrt(variance + eps), of wide rows
  float* dw;             // d
  float* db;             // d, or null
  int64_t ldx, ldy, ldo;
  int32_t rows, d;
  int32_t centered, w_bf16;
  int32_t groups;        // waves or workgroups that rows are dealt to
  float eps, beta;
};

constexpr int kNormThreadsMax = 512;

// First column of this thread's u-th unit.
template <int L, int V>
__device__ __forceinline__ int norm_col(int u) {
  const int threads = L ? L : static_cast<int>(blockDim.x), own = L ? static_cast<int>(threadIdx.x) % L : static_cast<int>(threadIdx.x);
  return (u * threads + own) * V;
}

// Rows: the first of this group of threads (a wave, or a workgroup), and this
// thread's among those that the group takes at once.
template <int L>
struct NormRows {
  static constexpr int AT_ONCE = L ? 64 / L : 1;
  int group, sub;
  int64_t step;
  __device__ __forceinline__ explicit NormRows(const NormArgs& a) {
    group = L ? static_cast<int>(blockIdx.x) * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) : static_cast<int>(blockIdx.x);
    sub = L ? static_cast<int>(threadIdx.x & 63) / L : 0;
    step = static_cast<int64_t>(a.groups) * AT_ONCE;
  }
};

// Sum over each L neighbouring lanes, on all of them.
template <int L>
__device__ __forceinline__ float lanes_sum(float v) {
  if constexpr (L == 64) return wave_sum(v);
  auto add = [&](uint32_t w) { v += __uint_as_float(w); };
  auto bits = [&] { return static_cast<int>(__float_as_uint(v)); };
  add(static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(bits(), 0xb1, 0xf, 0xf, true)));    // neighbours
  add(static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(bits(), 0x4e, 0xf, 0xf, true)));    // pairs
  add(static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(bits(), 0x141, 0xf, 0xf, true)));   // mirrors of 8
  if constexpr (L >= 16) add(static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(bits(), 0x140, 0xf, 0xf, true)));   // of 16
  if constexpr (L >= 32) v += __shfl_xor(v, 16, 64);
  return v;
}

// LDS of a row's sums; rows have two sets in turn.
struct NormParts {
  float2 p[2][2][kNormThreadsMax / 64];
};

// Two sums over a row's threads, on all of them.  One barrier: each pair of a row has
// LDS of its own, and rows have two sets in turn, so that a slow wave's reads are
// behind it before they are written again.  The barrier waits for LDS alone:
// __syncthreads would also wait for the next row's loads and this one's stores.
template <int L>
__device__ __forceinline__ void norm_sum(float& v0, float& v1, float2* part) {
  if constexpr (L != 0) {
    v0 = lanes_sum<L>(v0);
    v1 = lanes_sum<L>(v1);
    return;
  }
  v0 = wave_sum(v0);
  v1 = wave_sum(v1);
  const int waves = blockDim.x >> 6;
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = make_float2(v0, v1);
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
  v0 = v1 = 0.f;
  for (int w = 0; w < waves; ++w) {
    const float2 t = part[w];
    v0 += t.x;
    v1 += t.y;
  }
}

// V values of a weight (or bias) from column c on; 0 past the row, and without one.
template <int V>
__device__ __forceinline__ void norm_weight(const void* w, int bf, int c, int d, float (&v)[V]) {
#pragma unroll
  for (int i = 0; i < V; ++i) v[i] = 0.f;
  if (!w || c >= d) return;
  if (c + V <= d && !bf) {
#pragma unroll
    for (int i = 0; i < V; i += 4) {
      float f[4];
      Vec16<ElemF32>::unpack(load16_any(static_cast<const float*>(w) + c + i), f);
#pragma unroll
      for (int q = 0; q < 4; ++q) v[i + q] = f[q];
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < V; ++i)
    if (c + i < d) v[i] = bf ? bf16_to_f32(static_cast<const uint16_t*>(w)[c + i]) : static_cast<const float*>(w)[c + i];
}

// One row in registers.  FULL: the threads' units are exactly the row; else some
// threads' last unit is not, or not wholly, the row's (the host chooses the number
// of threads so).
template <class E, int UPT, int L, bool FULL>
struct NormRow {
  using S = typename E::storage_t;
  static constexpr int V = E::kVec;
  uint4 raw[UPT];
  __device__ __forceinline__ void load(const S* row, int d) {
#pragma unroll
    for (int u = 0; u < UPT; ++u) {
      const int c = norm_col<L, V>(u);
      if (FULL || u + 1 < UPT) raw[u] = load16_any(row + c);
      else raw[u] = c < d ? unit_load<E>(row + c, d - c) : make_uint4(0, 0, 0, 0);
    }
  }
  __device__ __forceinline__ void get(int u, float (&v)[V]) const { Vec16<E>::unpack(raw[u], v); }
};

// A deviation, 0 past the row (not FULL, of the last unit).
template <int UPT, int V, int L, bool FULL>
struct NormKeep {
  int left;
  __device__ __forceinline__ explicit NormKeep(int d) { left = d - norm_col<L, V>(UPT - 1); }
  __device__ __forceinline__ float operator()(int u, int i, float v) const { return FULL || u + 1 < UPT || i < left ? v : 0.f; }
};

template <class E, int UPT, int L, bool FULL>
__global__ __launch_bounds__(L ? 256 : kNormThreadsMax) void layer_norm_kernel(NormArgs a) {
  using S = typename E::storage_t;
  constexpr int V = E::kVec;
  __shared__ NormParts parts;
  const NormRows<L> at(a);
  if (L && at.group >= a.groups) return;
  NormRow<E, UPT, L, FULL> x;
  // rows of one wave's lanes end together: past the last, it is read again
  auto fetch = [&](int64_t row) { x.load(static_cast<const S*>(a.x) + min(row, static_cast<int64_t>(a.rows) - 1) * a.ldx, a.d); };
  int64_t row0 = static_cast<int64_t>(at.group) * at.AT_ONCE;
  fetch(row0 + at.sub);
  float w[UPT][V], b[UPT][V];
#pragma unroll
  for (int u = 0; u < UPT; ++u) {
    norm_weight<V>(a.w, a.w_bf16, norm_col<L, V>(u), a.d, w[u]);
    norm_weight<V>(a.b, a.w_bf16, norm_col<L, V>(u), a.d, b[u]);
  }
  const NormKeep<UPT, V, L, FULL> keep(a.d);
  const float inv = 1.f / static_cast<float>(a.d);
  int set = 0;
  for (; row0 < a.rows; row0 += at.step, set ^= 1) {
    const int64_t row = row0 + at.sub;
    float xc[UPT][V], s = 0.f, none = 0.f;
#pragma unroll
    for (int u = 0; u < UPT; ++u) {
      x.get(u, xc[u]);
#pragma unroll
      for (int i = 0; i < V; ++i) s += xc[u][i];
    }
    if (row0 + at.step < a.rows) fetch(row + at.step);
    float mean = 0.f;
    if (a.centered) {
      norm_sum<L>(s, none, parts.p[set][0]);
      mean = s * inv;
    }
    float q = 0.f;
#pragma unroll
    for (int u = 0; u < UPT; ++u)
#pragma unroll
      for (int i = 0; i < V; ++i) {
        xc[u][i] = keep(u, i, xc[u][i] - mean);
        q = fmaf(xc[u][i], xc[u][i], q);
      }
    norm_sum<L>(q, none, parts.p[set][1]);
    const float r = rsqrtf(q * inv + a.eps);
    if (L && row >= a.rows) continue;
    S* y = static_cast<S*>(a.out) + row * a.ldo;
#pragma unroll
    for (int u = 0; u < UPT; ++u) {
      const int c = norm_col<L, V>(u);
#pragma unroll
      for (int i = 0; i < V; ++i) xc[u][i] = fmaf(xc[u][i] * r, w[u][i], b[u][i]);
      if (FULL || u + 1 < UPT) unit_store<E>(y + c, V, Vec16<E>::pack(xc[u]));
      else if (c < a.d) unit_store<E>(y + c, a.d - c, Vec16<E>::pack(xc[u]));
    }
  }
}

// Each group of threads that takes rows (a workgroup, or a wave) has partial sums
// of its own.
template <class E, int UPT, int L, bool FULL>
__global__ __launch_bounds__(L ? 256 : kNormThreadsMax) void layer_norm_grad_kernel(NormArgs a) {
  using S = typename E::storage_t;
  constexpr int V = E::kVec;
  __shared__ NormParts parts;
  const NormRows<L> at(a);
  if (L && at.group >= a.groups) return;
  NormRow<E, UPT, L, FULL> x, dy;
  auto fetch = [&](int64_t row) {
    row = min(row, static_cast<int64_t>(a.rows) - 1);
    x.load(static_cast<const S*>(a.x) + row * a.ldx, a.d);
    dy.load(static_cast<const S*>(a.dy) + row * a.ldy, a.d);
  };
  int64_t row0 = static_cast<int64_t>(at.group) * at.AT_ONCE;
  fetch(row0 + at.sub);
  float w[UPT][V], accw[UPT][V], accb[UPT][V];
#pragma unroll
  for (int u = 0; u < UPT; ++u) {
    norm_weight<V>(a.w, a.w_bf16, norm_col<L, V>(u), a.d, w[u]);
#pragma unroll
    for (int i = 0; i < V; ++i) accw[u][i] = accb[u][i] = 0.f;
  }
  const NormKeep<UPT, V, L, FULL> keep(a.d);
  const float inv = 1.f / static_cast<float>(a.d);
  int set = 0;
  for (; row0 < a.rows; row0 += at.step, set ^= 1) {
    const int64_t row = row0 + at.sub;
    float xc[UPT][V], dv[UPT][V], s = 0.f, c0 = 0.f;
#pragma unroll
    for (int u = 0; u < UPT; ++u) {
      x.get(u, xc[u]);
      dy.get(u, dv[u]);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        s += xc[u][i];
        c0 = fmaf(dv[u][i], w[u][i], c0);
      }
    }
    if (row0 + at.step < a.rows) fetch(row + at.step);
    float mean = 0.f;
    if (a.centered) {
      norm_sum<L>(s, c0, parts.p[set][0]);
      mean = s * inv;
      c0 *= inv;
    } else {
      c0 = 0.f;
    }
    float q = 0.f, c1 = 0.f;      // sums of xc^2 and of g xc
#pragma unroll
    for (int u = 0; u < UPT; ++u)
#pragma unroll
      for (int i = 0; i < V; ++i) {
        xc[u][i] = keep(u, i, xc[u][i] - mean);
        q = fmaf(xc[u][i], xc[u][i], q);
        c1 = fmaf(dv[u][i] * w[u][i], xc[u][i], c1);
      }
    norm_sum<L>(q, c1, parts.p[set][1]);
    const float r = rsqrtf(q * inv + a.eps);
    if (L && row >= a.rows) continue;       // (the last round: nothing follows)
    // dx = r g - r c0 - xc r^3 mean(g xc)
    const float k0 = -r * c0, k1 = -r * (r * (r * (c1 * inv)));    // (r^3 alone may leave fp32's range)
    S* dx = static_cast<S*>(a.out) + row * a.ldo;
#pragma unroll
    for (int u = 0; u < UPT; ++u) {
      const int c = norm_col<L, V>(u);
      float o[V];
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float rd = r * dv[u][i];
        o[i] = fmaf(xc[u][i], k1, fmaf(rd, w[u][i], k0));
        accw[u][i] = fmaf(rd, xc[u][i], accw[u][i]);
        accb[u][i] += dv[u][i];
      }
      if (FULL || u + 1 < UPT) unit_store<E>(dx + c, V, Vec16<E>::pack(o));
      else if (c < a.d) unit_store<E>(dx + c, a.d - c, Vec16<E>::pack(o));
    }
  }
  if constexpr (L != 0 && L < 64) {   // the wave's rows, in a tree
#pragma unroll
    for (int u = 0; u < UPT; ++u)
#pragma unroll
      for (int i = 0; i < V; ++i)
#pragma unroll
        for (int d = L; d < 64; d *= 2) {
          accw[u][i] += __shfl_xor(accw[u][i], d, 64);
          accb[u][i] += __shfl_xor(accb[u][i], d, 64);
        }
    if (at.sub > 0) return;
  }
  float* pw = a.part + static_cast<size_t>(at.group) * (a.db ? 2 : 1) * a.d;
#pragma unroll
  for (int u = 0; u < UPT; ++u) {
    const int c = norm_col<L, V>(u);
#pragma unroll
    for (int h = 0; h < V; h += 4) {
      const float fw[4] = {accw[u][h], accw[u][h + 1], accw[u][h + 2], accw[u][h + 3]};
      const float fb[4] = {accb[u][h], accb[u][h + 1], accb[u][h + 2], accb[u][h + 3]};
      if (!FULL && c + h >= a.d) continue;
      if (FULL || c + h + 4 <= a.d) {
        store16_any(pw + c + h, Vec16<ElemF32>::pack(fw));
        if (a.db) store16_any(pw + a.d + c + h, Vec16<ElemF32>::pack(fb));
      } else {
        for (int i = 0; c + h + i < a.d; ++i) {
          pw[c + h + i] = fw[i];
          if (a.db) pw[a.d + c + h + i] = fb[i];
        }
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Rows that do not fit: one workgroup per row, each pass reads it again (2000 rows
// of 24576 bf16: gradients 137 us, where the bytes would take 57).
// ---------------------------------------------------------------------------
// f(c, x, dy) for this thread's units of a row.
template <class E, class F>
__device__ __forceinline__ void norm_wide(const typename E::storage_t* x, const typename E::storage_t* dy, int d, F&& f) {
  constexpr int V = E::kVec;
  for (int c = static_cast<int>(threadIdx.x) * V; c < d; c += static_cast<int>(blockDim.x) * V) {
    float xv[V], gv[V];
    Vec16<E>::unpack(unit_load<E>(x + c, d - c), xv);
    if (dy) Vec16<E>::unpack(unit_load<E>(dy + c, d - c), gv);
    f(c, xv, gv);
  }
}

template <class E, bool GRAD>
__global__ __launch_bounds__(kNormThreadsMax) void layer_norm_wide_kernel(NormArgs a) {
  using S = typename E::storage_t;
  constexpr int V = E::kVec;
  __shared__ NormParts parts;
  const float inv = 1.f / static_cast<float>(a.d);
  int set = 0;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, set ^= 1) {
    const S* x = static_cast<const S*>(a.x) + row * a.ldx;
    const S* dy = GRAD ? static_cast<const S*>(a.dy) + row * a.ldy : nullptr;
    float s = 0.f, c0 = 0.f, mean = 0.f;
    if (a.centered) {
      norm_wide<E>(x, dy, a.d, [&](int c, const float (&xv)[V], const float (&gv)[V]) {
        float w[V];
        if (GRAD) norm_weight<V>(a.w, a.w_bf16, c, a.d, w);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          s += xv[i];
          if (GRAD) c0 = fmaf(gv[i], w[i], c0);
        }
      });
      norm_sum<0>(s, c0, parts.p[set][0]);
      mean = s * inv;
      c0 *= inv;
    }
    float q = 0.f, c1 = 0.f;
    norm_wide<E>(x, dy, a.d, [&](int c, const float (&xv)[V], const float (&gv)[V]) {
      float w[V];
      if (GRAD) norm_weight<V>(a.w, a.w_bf16, c, a.d, w);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float xc = c + i < a.d ? xv[i] - mean : 0.f;
        q = fmaf(xc, xc, q);
        if (GRAD) c1 = fmaf(gv[i] * w[i], xc, c1);
      }
    });
    norm_sum<0>(q, c1, parts.p[set][1]);
    const float r = rsqrtf(q * inv + a.eps);
    const float k0 = -r * c0, k1 = -r * (r * (r * (c1 * inv)));
    S* out = static_cast<S*>(a.out) + row * a.ldo;
    norm_wide<E>(x, dy, a.d, [&](int c, const float (&xv)[V], const float (&gv)[V]) {
      float w[V], o[V];
      norm_weight<V>(a.w, a.w_bf16, c, a.d, w);
      if constexpr (GRAD) {
#pragma unroll
        for (int i = 0; i < V; ++i) o[i] = fmaf(xv[i] - mean, k1, fmaf(r * gv[i], w[i], k0));
      } else {
        float b[V];
        norm_weight<V>(a.b, a.w_bf16, c, a.d, b);
#pragma unroll
        for (int i = 0; i < V; ++i) o[i] = fmaf((xv[i] - mean) * r, w[i], b[i]);
      }
      unit_store<E>(out + c, a.d - c, Vec16<E>::pack(o));
    });
    if (GRAD && threadIdx.x == 0) {
      a.stats[2 * row] = mean;
      a.stats[2 * row + 1] = r;
    }
  }
}

// Partial sums over rows by columns: a workgroup takes 256 units of a group's rows.
template <class E>
__global__ __launch_bounds__(256) void layer_norm_columns_kernel(NormArgs a, int blocks) {
  using S = typename E::storage_t;
  constexpr int V = E::kVec, F = 4;       // rows in flight
  const int group = static_cast<int>(blockIdx.x) / blocks;
  const int c = (static_cast<int>(blockIdx.x) % blocks * 256 + static_cast<int>(threadIdx.x)) * V;
  if (c >= a.d) return;
  const int64_t per = (a.rows + a.groups - 1) / a.groups;
  const int64_t r0 = group * per, r1 = min(r0 + per, static_cast<int64_t>(a.rows));
  float accw[V], accb[V];
#pragma unroll
  for (int i = 0; i < V; ++i) accw[i] = accb[i] = 0.f;
  for (int64_t r = r0; r < r1; r += F) {
    uint4 x[F], dy[F];
#pragma unroll
    for (int j = 0; j < F; ++j) {
      const int64_t row = min(r + j, r1 - 1);
      x[j] = unit_load<E>(static_cast<const S*>(a.x) + row * a.ldx + c, a.d - c);
      dy[j] = unit_load<E>(static_cast<const S*>(a.dy) + row * a.ldy + c, a.d - c);
    }
#pragma unroll
    for (int j = 0; j < F; ++j) {
      if (r + j >= r1) break;
      const float mean = a.stats[2 * (r + j)], rs = a.stats[2 * (r + j) + 1];
      float xv[V], gv[V];
      Vec16<E>::unpack(x[j], xv);
      Vec16<E>::unpack(dy[j], gv);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        accw[i] = fmaf(gv[i] * rs, xv[i] - mean, accw[i]);
        accb[i] += gv[i];
      }
    }
  }
  float* pw = a.part + static_cast<size_t>(group) * (a.db ? 2 : 1) * a.d + c;
#pragma unroll
  for (int i = 0; i < V; ++i)
    if (c + i < a.d) {
      pw[i] = accw[i];
      if (a.db) pw[a.d + i] = accb[i];
    }
}

// dw = beta dw + sum over the groups' partial sums: 64 columns of one of the two
// per workgroup, kNormSlices waves each with its own contiguous part.
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
