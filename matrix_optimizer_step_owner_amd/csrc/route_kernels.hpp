// Routing of tokens to experts (gfx950): the chosen experts and their weights,
// the logits' gradient, the plan that sorts rows by expert, the balance bias.
//
// One wave takes one token.  Lane l holds the PER consecutive experts from
// l * PER on, so that the order of lanes is the order of experts and the first
// lane of a ballot is the lowest index among equals.  A round of the choice is
// the largest key in a wave (six DPP steps on order-preserving integers), one
// ballot, and the winner's key set to 0.
//
// Which experts are chosen is decided as in exact arithmetic.  Without a bias
// and groups the order of scores is that of the logits, and no score is needed.
// Otherwise keys are scores in fp32, and whatever they leave open -- neighbours
// in the chosen order, the last chosen and any other, or the border between
// groups, nearer than the rounding of both -- sends the token through the same choice in fp64.  That is one
// token in some hundred; fp64 for all of them would double the time.
#pragma once

#include "common.hpp"
#include "grouped_kernels.hpp"

namespace mfsdp {

constexpr int kRouteExpertsMax = 1024;
constexpr int kRouteChosenMax = 32;
constexpr int kRouteGroupsMax = 64;
constexpr float kRouteTiny = 1e-20f;

struct RouteArgs {
  const void* logits;     // tokens x n, row stride ld
  const float* bias;      // n, or null
  const uint8_t* mask;    // tokens, 0: padding; or null
  int32_t* chosen;        // tokens x k
  float* weights;         // tokens x k
  int64_t ld;
  int32_t tokens, n, k;
  int32_t groups, top, group_size;
  int32_t sigmoid, renorm;
  float scale;
};

// Order-preserving integers of floats: 0 is "not there", 1 a NaN (behind -inf).
__device__ __forceinline__ uint32_t route_key(float v) {
  const uint32_t u = __float_as_uint(v + 0.f);    // one zero
  return v != v ? 1u : u ^ (static_cast<int32_t>(u) < 0 ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ uint64_t route_key(double v) {
  const uint64_t u = static_cast<uint64_t>(__double_as_longlong(v + 0.0));
  return v != v ? 1ull : u ^ (static_cast<int64_t>(u) < 0 ? ~0ull : 1ull << 63);
}
__device__ __forceinline__ float route_value(uint32_t k) {
  if (k <= 1u) return __uint_as_float(0x7fc00000u);
  return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}
__device__ __forceinline__ double route_value(uint64_t k) {
  if (k <= 1ull) return __longlong_as_double(0x7ff8000000000000ll);
  return __longlong_as_double(static_cast<int64_t>(k >> 63 ? k ^ (1ull << 63) : ~k));
}

// Largest value in the wave, on every lane (as a scalar).
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t dpp_or0(uint32_t v) {
  return static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), CTRL, ROWS, 0xf, false));
}
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  v = max(v, dpp_or0<0x111, 0xf>(v));   // row_shr:1, :2, :4, :8
  v = max(v, dpp_or0<0x112, 0xf>(v));
  v = max(v, dpp_or0<0x114, 0xf>(v));
  v = max(v, dpp_or0<0x118, 0xf>(v));
  v = max(v, dpp_or0<0x142, 0xa>(v));   // row_bcast:15, :31
  v = max(v, dpp_or0<0x143, 0xc>(v));
  return static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(v), 63));
}
__device__ __forceinline__ uint64_t wave_max(uint64_t v) {
  const uint32_t hi = wave_max(static_cast<uint32_t>(v >> 32));
  const uint32_t lo = wave_max(static_cast<uint32_t>(v >> 32) == hi ? static_cast<uint32_t>(v) : 0u);
  return static_cast<uint64_t>(hi) << 32 | lo;
}

// PER elements from p + lane * PER on, those before n; others as `fill`.
template <class E, int PER>
__device__ __forceinline__ void route_load(const typename E::storage_t* p, int first, int n, float fill,
                                           float (&v)[PER]) {
  using S = typename E::storage_t;
  S raw[PER];
  if (first + PER <= n) {
    if constexpr (PER * sizeof(S) % 16 == 0) {
#pragma unroll
      for (int i = 0; i < PER; i += 16 / static_cast<int>(sizeof(S))) {
        const uint4 t = load16_any(p + first + i);
        __builtin_memcpy(raw + i, &t, 16);
      }
    } else {
#pragma unroll
      for (int i = 0; i < PER; ++i) raw[i] = gld<S>(p + first + i);
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) v[i] = E::to_f32(raw[i]);
  } else {
#pragma unroll
    for (int i = 0; i < PER; ++i) v[i] = first + i < n ? E::to_f32(gld<S>(p + first + i)) : fill;
  }
}

// Score of one expert; top and sum are the row's (softmax).
__device__ __forceinline__ float route_score(float x, int sigmoid, float top, float sum) {
  return sigmoid ? 1.f / (1.f + expf(-x)) : expf(x - top) / sum;
}

// Largest logit and sum of exp(x - largest) of a row (softmax).
template <int PER>
__device__ __forceinline__ void route_softmax(const float (&x)[PER], int first, int n, float& top, float& sum) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i)
    if (first + i < n) m = max(m, route_key(x[i]));
  top = route_value(wave_max(m));
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < PER; ++i)
    if (first + i < n) s += expf(x[i] - top);
  sum = warp_sum(s);
}

// Groups: returns the bits of those that stay.  vk: keys of score + bias, 0
// where there is no expert.  `close`: the border between the last group that
// stays and the first that does not is nearer than the sums' rounding.
template <int PER, class V, class K>
__device__ __forceinline__ uint64_t route_groups(const RouteArgs& a, const K (&vk)[PER], const int (&gid)[PER],
                                                 int lane, bool& close) {
  V mine = V(0);
  for (int g = 0; g < a.groups; ++g) {
    K best = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (gid[i] == g) best = max(best, vk[i]);
    const K one = wave_max(best);
    const int owner = __builtin_ctzll(__ballot(best == one));
    // second: the owner leaves out its first one that is equal
    K next = 0;
    bool skip = lane == owner;
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (gid[i] == g) {
        if (skip && vk[i] == one) skip = false;
        else next = max(next, vk[i]);
      }
    const K two = wave_max(next);
    V sum = route_value(one);
    if (a.group_size > 1) sum += route_value(two);
    if (lane == g) mine = sum;
  }
  const K key = lane < a.groups ? route_key(mine) : K(0);
  int rank = 0;
  for (int g = 0; g < a.groups; ++g) {
    K other;
    if constexpr (sizeof(K) == 8)
      other = static_cast<uint64_t>(static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(key >> 32), g))) << 32 |
              static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(key), g));
    else
      other = static_cast<K>(__builtin_amdgcn_readlane(static_cast<int>(key), g));
    rank += other > key || (other == key && g < lane) ? 1 : 0;
  }
  const bool stays = lane < a.groups && rank < a.top;
  if constexpr (sizeof(K) == 4) {
    if (a.top < a.groups) {
      // each of a sum's two keys is off by at most 33 * 2^-23 (s (|x - top| + 32)
      // is under 33) and half a step of itself
      const float out = route_value(wave_max(stays || lane >= a.groups ? 0u : key));
      const float in = route_value(~wave_max(stays ? ~key : 0u));
      const float tol = 0x1p-23f * (132.f + 8.f * (fabsf(in) + fabsf(out)));
      close = !(in - out > tol);
    }
  }
  return __ballot(stays);
}

// The k largest keys in order, lane j receiving expert j (others -1); their keys
// are set to 0.
template <int PER, class K>
__device__ __forceinline__ int route_pick(K (&key)[PER], int first, int k, int lane) {
  int mine = -1;
  for (int j = 0; j < k; ++j) {
    K best = key[0];
#pragma unroll
    for (int i = 1; i < PER; ++i) best = max(best, key[i]);
    const K m = wave_max(best);
    if (m == 0) break;
    const int owner = __builtin_ctzll(__ballot(best == m));
    int at = 0;
#pragma unroll
    for (int i = PER - 1; i >= 0; --i)
      if (key[i] == m) at = i;
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (lane == owner && i == at) key[i] = 0;
    const int e = __builtin_amdgcn_readlane(first + at, owner);
    if (lane == j) mine = e;
  }
  return mine;
}

template <class E, int PER>
__global__ __launch_bounds__(256) void route_kernel(RouteArgs a) {
  using S = typename E::storage_t;
  const int lane = threadIdx.x & 63;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6);
  if (t >= a.tokens) return;
  int32_t* chosen = a.chosen + t * a.k;
  float* weights = a.weights + t * a.k;
  if (a.mask && a.mask[t] == 0) {
    if (lane < a.k) {
      chosen[lane] = -1;
      weights[lane] = 0.f;
    }
    return;
  }
  const S* row = static_cast<const S*>(a.logits) + t * a.ld;
  const int first = lane * PER;
  float x[PER];
  route_load<E, PER>(row, first, a.n, 0.f, x);
  float top = 0.f, sum = 1.f;
  if (!a.sigmoid) route_softmax<PER>(x, first, a.n, top, sum);

  uint32_t key[PER];
  int mine;
  if (!a.bias && a.groups == 1) {
#pragma unroll
    for (int i = 0; i < PER; ++i) key[i] = first + i < a.n ? route_key(x[i]) : 0u;
    mine = route_pick<PER>(key, first, a.k, lane);
  } else {
    float b[PER];
    int gid[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      b[i] = 0.f;
      gid[i] = (first + i) / a.group_size;
    }
    if (a.bias) route_load<ElemF32, PER>(a.bias, first, a.n, 0.f, b);
#pragma unroll
    for (int i = 0; i < PER; ++i)
      key[i] = first + i < a.n ? route_key(route_score(x[i], a.sigmoid, top, sum) + b[i]) : 0u;
    bool close = false;
    uint64_t stay = 1;
    if (a.groups > 1) {
      stay = route_groups<PER, float>(a, key, gid, lane, close);
#pragma unroll
      for (int i = 0; i < PER; ++i)
        if (!(stay >> gid[i] & 1) || first + i >= a.n) key[i] = 0;
    }
    if (!a.bias) {   // within the groups the logits decide
#pragma unroll
      for (int i = 0; i < PER; ++i)
        if (key[i]) key[i] = route_key(x[i]);
      mine = route_pick<PER>(key, first, a.k, lane);
    } else {
      mine = route_pick<PER>(key, first, a.k, lane);
      // neighbours in the order: their keys' rounding against their distance
      const float mx = mine >= 0 ? E::to_f32(gld<S>(row + mine)) : 0.f;
      const float mb = mine >= 0 ? gld<float>(a.bias + mine) : 0.f;
      const float ms = route_score(mx, a.sigmoid, top, sum), mk = ms + mb;
      auto rounding = [&](float score, float xi, float k) {
        return 0x1p-23f * (score * (32.f + (a.sigmoid ? 0.f : fabsf(xi - top))) + 2.f * fabsf(k));
      };
      const float off = rounding(ms, mx, mk);
      const float ox = __shfl_down(mx, 1, 64), ob = __shfl_down(mb, 1, 64), ok = __shfl_down(mk, 1, 64);
      const float tol = off + __shfl_down(off, 1, 64);
      bool open = lane + 1 < a.k && !(mk - ok > tol) && !(ox == mx && ob == mb);
      // the last against all that were not chosen: the next of them alone would
      // not do, as one that is equal to the last hides others behind it
      auto last = [&](float v) { return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), a.k - 1)); };
      const float lx = last(mx), lb = last(mb), lk = last(mk), lo = last(off);
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        if (key[i] == 0) continue;
        const float ki = route_value(key[i]);
        open = open || (!(lk - ki > lo + rounding(fabsf(ki - b[i]), x[i], ki)) && !(x[i] == lx && b[i] == lb));
      }
      close = close || __ballot(open) != 0;
    }
    if (__builtin_expect(__ballot(close) != 0, 0)) {
      double d[PER], dtop = 0.0, dsum = 1.0;
      if (!a.sigmoid) {
        dtop = top;
        double s = 0.0;
#pragma unroll
        for (int i = 0; i < PER; ++i)
          if (first + i < a.n) s += exp(static_cast<double>(x[i]) - dtop);
        dsum = warp_sum(s);
      }
      uint64_t dk[PER];
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const double v = a.sigmoid ? 1.0 / (1.0 + exp(-static_cast<double>(x[i]))) : exp(static_cast<double>(x[i]) - dtop) / dsum;
        d[i] = v + static_cast<double>(b[i]);
        dk[i] = first + i < a.n ? route_key(d[i]) : 0ull;
      }
      if (a.groups > 1) {
        bool none = false;
        stay = route_groups<PER, double>(a, dk, gid, lane, none);
      }
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        if (!(stay >> gid[i] & 1) || first + i >= a.n) dk[i] = 0;
        else if (!a.bias) dk[i] = route_key(x[i]);
      }
      mine = route_pick<PER>(dk, first, a.k, lane);
    }
  }

  const bool on = lane < a.k;
  const float s = on ? route_score(E::to_f32(gld<S>(row + max(mine, 0))), a.sigmoid, top, sum) : 0.f;
  const float total = a.renorm ? warp_sum(s) + kRouteTiny : 1.f;
  if (on) {
    chosen[lane] = mine;
    weights[lane] = a.scale * s / total;
  }
}

// ---------------------------------------------------------------------------
// Gradient of the weights by the logits
// ---------------------------------------------------------------------------
struct RouteGradArgs {
  const float* dw;        // tokens x k
  const void* logits;     // tokens x n, row stride ld
  const int32_t* chosen;  // tokens x k; outside [0, n): none
  void* out;              // tokens x n, row stride ldo
  int64_t ld, ldo;
  int32_t tokens, n, k;
  int32_t sigmoid, renorm;
  float scale;
};

// With s the chosen scores, g the weights' gradient and D = sum s + 1e-20:
//   ds_j = scale / D (g_j - sum_i g_i s_i / D)     (scale g_j if not renormalised)
//   softmax  dx_e = p_e (ds_e - sum_j ds_j s_j)    ds_e = 0 where not chosen
//   sigmoid  dx_e = ds_e s_e (1 - s_e)
template <class E, int PER>
__global__ __launch_bounds__(256) void route_grad_kernel(RouteGradArgs a) {
  using S = typename E::storage_t;
  const int lane = threadIdx.x & 63;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6);
  if (t >= a.tokens) return;
  const S* row = static_cast<const S*>(a.logits) + t * a.ld;
  S* out = static_cast<S*>(a.out) + t * a.ldo;
  const int first = lane * PER;
  int e = lane < a.k ? a.chosen[t * a.k + lane] : -1;
  if (e >= a.n) e = -1;
  const bool on = e >= 0;
  float dx[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) dx[i] = 0.f;
  if (__ballot(on) != 0) {    // a padded token's logits are not read
    const float xe = on ? E::to_f32(gld<S>(row + e)) : 0.f;
    const float g = on ? a.dw[t * a.k + lane] : 0.f;
    float x[PER], top = 0.f, sum = 1.f;
    if (!a.sigmoid) {
      route_load<E, PER>(row, first, a.n, 0.f, x);
      route_softmax<PER>(x, first, a.n, top, sum);
    }
    const float s = on ? route_score(xe, a.sigmoid, top, sum) : 0.f;
    float ds = a.scale * g;
    if (a.renorm) {
      const float d = warp_sum(s) + kRouteTiny;
      ds = a.scale / d * (g - warp_sum(g * s) / d);
    }
    if (!on) ds = 0.f;
    float c = 0.f;
    if (a.sigmoid) {
      const float q = expf(-fabsf(xe));         // s (1 - s), no difference
      ds *= q / ((1.f + q) * (1.f + q));
    } else {
      c = warp_sum(ds * s);
    }
    for (int j = 0; j < a.k; ++j) {             // an expert that is named twice adds up
      const int ej = __builtin_amdgcn_readlane(e, j);
      const float dj = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(ds), j));
#pragma unroll
      for (int i = 0; i < PER; ++i)
        if (ej == first + i) dx[i] += dj;
    }
    if (!a.sigmoid) {
#pragma unroll
      for (int i = 0; i < PER; ++i) dx[i] = expf(x[i] - top) / sum * (dx[i] - c);
    }
  }
  if (first + PER <= a.n && PER % E::kVec == 0) {
#pragma unroll
    for (int i = 0; i < PER; i += E::kVec) {
      float v[E::kVec];
#pragma unroll
      for (int q = 0; q < E::kVec; ++q) v[q] = dx[(i + q) % PER];
      store16_any(out + first + i, Vec16<E>::pack(v));
    }
  } else {
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (first + i < a.n) gst<S>(out + first + i, E::from_f32(dx[i]));
  }
}

// ---------------------------------------------------------------------------
// Plan: a stable counting sort of (token, choice) by expert
// ---------------------------------------------------------------------------
constexpr int kPlanThreads = 1024;
constexpr int kPlanWaves = kPlanThreads / 64;
constexpr int kPlanBinsMax = kRouteExpertsMax;
constexpr int kPlanSmall = 8192;       // slots that one workgroup takes alone

struct PlanArgs {
  const int32_t* chosen;   // n slots; outside [0, experts): no row
  int32_t* offsets;        // experts + 1
  int32_t* place;          // n
  uint32_t* hist;          // [blocks][experts]
  int32_t n, experts;
  int32_t bits;            // of an expert's number
  int32_t per_block;       // slots per workgroup, a multiple of kPlanThreads
};

__device__ __forceinline__ uint32_t plan_expert(const PlanArgs& a, int i) {
  const int e = a.chosen[i];
  return e >= 0 && e < a.experts ? static_cast<uint32_t>(e) : 0xffffffffu;
}

__global__ __launch_bounds__(kPlanThreads) void plan_hist_kernel(PlanArgs a) {
  __shared__ uint32_t h[kPlanBinsMax];
  for (int b = threadIdx.x; b < a.experts; b += kPlanThreads) h[b] = 0;
  __syncthreads();
  const int i0 = blockIdx.x * a.per_block, i1 = min(i0 + a.per_block, a.n);
  for (int i = i0 + threadIdx.x; i < i1; i += kPlanThreads) {
    const uint32_t e = plan_expert(a, i);
    if (e != 0xffffffffu) atomicAdd(&h[e], 1u);
  }
  __syncthreads();
  for (int b = threadIdx.x; b < a.experts; b += kPlanThreads)
    a.hist[static_cast<size_t>(blockIdx.x) * a.experts + b] = h[b];
}

// Rows of this workgroup's slots.  base: first row of each expert's slots here.
// Each wave takes a contiguous part; counts per wave give its own first rows,
// and within 64 slots the lower lanes with the same expert are counted by
// ballots over the bits of its number.  Counts are sums of whole numbers: the
// order in which they are added does not show.
__device__ __forceinline__ void plan_place(const PlanArgs& a, int i0, int i1, const uint32_t* base,
                                           uint32_t (*cnt)[kPlanBinsMax]) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int per_wave = (i1 - i0 + kPlanThreads - 1) / kPlanThreads * 64;
  const int w0 = min(i0 + wave * per_wave, i1), w1 = min(w0 + per_wave, i1);
  for (int b = lane; b < a.experts; b += 64) cnt[wave][b] = 0;
  __syncthreads();
  for (int i = w0 + lane; i < w1; i += 64) {
    const uint32_t e = plan_expert(a, i);
    if (e != 0xffffffffu) atomicAdd(&cnt[wave][e], 1u);
  }
  __syncthreads();
  for (int b = threadIdx.x; b < a.experts; b += kPlanThreads) {
    uint32_t at = base[b];
#pragma unroll
    for (int w = 0; w < kPlanWaves; ++w) {
      const uint32_t c = cnt[w][b];
      cnt[w][b] = at;
      at += c;
    }
  }
  __syncthreads();
  for (int i = w0; i < w1; i += 64) {
    const bool in = i + lane < w1;
    const uint32_t e = in ? plan_expert(a, i + lane) : 0xffffffffu;
    const bool on = e != 0xffffffffu;
    uint64_t same = __ballot(on);
    for (int b = 0; b < a.bits; ++b) {
      const uint64_t m = __ballot(e >> b & 1);
      same &= e >> b & 1 ? m : ~m;
    }
    int row = -1;
    if (on) {
      const uint32_t rank = __popcll(same & ((uint64_t(1) << lane) - 1));
      const uint32_t at = cnt[wave][e] + rank;
      row = static_cast<int>(at);
      // the highest lane of each expert moves the wave's place on, behind the
      // reads above (one wave, LDS operations in order)
      if (rank + 1 == static_cast<uint32_t>(__popcll(same))) cnt[wave][e] = at + 1;
    }
    if (in) a.place[i + lane] = row;
    __builtin_amdgcn_wave_barrier();
  }
}

// Exclusive scan of tot[0 .. experts) into base, plus add; one expert a thread.
__device__ __forceinline__ uint32_t plan_scan(const uint32_t* tot, const uint32_t* add, uint32_t* base, int experts,
                                              uint32_t* wave_sum, int32_t* offsets) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, b = threadIdx.x;
  const uint32_t t = b < experts ? tot[b] : 0;
  uint32_t incl = t;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const uint32_t v = __shfl_up(incl, d, 64);
    if (lane >= d) incl += v;
  }
  if (lane == 63) wave_sum[wave] = incl;
  __syncthreads();
  uint32_t before = incl - t;
  for (int w = 0; w < wave; ++w) before += wave_sum[w];
  if (b < experts) {
    base[b] = before + add[b];
    if (offsets) {
      offsets[b] = static_cast<int32_t>(before);
      if (b == experts - 1) offsets[experts] = static_cast<int32_t>(before + t);
    }
  }
  __syncthreads();
  return before;
}
static_assert(kPlanBinsMax <= kPlanThreads, "plan_scan takes one expert per thread");

// One workgroup for all slots (SMALL), or the second of two launches.
template <bool SMALL>
__global__ __launch_bounds__(kPlanThreads) void plan_place_kernel(PlanArgs a) {
  __shared__ uint32_t base[kPlanBinsMax], tot[kPlanBinsMax], add[kPlanBinsMax];
  __shared__ uint32_t cnt[kPlanWaves][kPlanBinsMax];
  __shared__ uint32_t wave_sum[kPlanWaves];
  if constexpr (SMALL) {
    for (int b = threadIdx.x; b < a.experts; b += kPlanThreads) tot[b] = add[b] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < a.n; i += kPlanThreads) {
      const uint32_t e = plan_expert(a, i);
      if (e != 0xffffffffu) atomicAdd(&tot[e], 1u);
    }
  } else {
    for (int b = threadIdx.x; b < a.experts; b += kPlanThreads) {
      uint32_t t = 0, before = 0;
      for (unsigned w = 0; w < gridDim.x; ++w) {
        const uint32_t c = a.hist[static_cast<size_t>(w) * a.experts + b];
        if (w < blockIdx.x) before += c;
        t += c;
      }
      tot[b] = t;
      add[b] = before;
    }
  }
  __syncthreads();
  plan_scan(tot, add, base, a.experts, wave_sum, blockIdx.x == 0 ? a.offsets : nullptr);
  const int i0 = SMALL ? 0 : blockIdx.x * a.per_block;
  plan_place(a, i0, SMALL ? a.n : min(i0 + a.per_block, a.n), base, cnt);
}

// ---------------------------------------------------------------------------
// Balance: bias[e] += rate * sign(mean count - count[e])
// ---------------------------------------------------------------------------
struct BalanceArgs {
  float* bias;
  const void* counts;    // int32 or int64
  int32_t n, wide;
  float rate;
};

__global__ __launch_bounds__(256) void route_balance_kernel(BalanceArgs a) {
  __shared__ int64_t part[4];
  auto count = [&](int e) -> int64_t {
    return a.wide ? static_cast<const int64_t*>(a.counts)[e] : static_cast<const int32_t*>(a.counts)[e];
  };
  int64_t sum = 0;
  for (int e = threadIdx.x; e < a.n; e += 256) sum += count(e);
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) sum += __shfl_xor(sum, d, 64);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = sum;
  __syncthreads();
  sum = part[0] + part[1] + part[2] + part[3];
  for (int e = threadIdx.x; e < a.n; e += 256) {
    const int64_t d = sum - count(e) * a.n;    // in whole numbers: no rounding decides
    if (d != 0) a.bias[e] += d > 0 ? a.rate : -a.rate;
  }
}

}  // namespace mfsdp
