// Routing of tokens to experts (gfx950): the chosen experts and their weights,
// the logits' gradient, the plan that sorts rows by expert, the balance bias.
//
// One wave takes one token.  Lane l holds the PER consecutive experts from
// l * PER on, so that the order of lanes is the order of experts and the first
// lane of a ballot is the lowest index among equals.  A round of the choice is
// the largest of the lanes' first keys (six DPP steps on order-preserving
// integers), one ballot, and the winner's sorted list moved up.
//
// Which experts are chosen is decided as in exact arithmetic.  Without a bias
// and groups the order of scores is that of the logits, and no score is needed.
// Otherwise keys are scores in fp32, and whatever they leave open -- neighbours
// in the chosen order, the last chosen and any other, or the border between
// groups, nearer than the rounding of both -- sends the token through the same
// choice in fp64: of 256 experts in eight groups, k = 8, normal logits, 6 tokens of
// a thousand with sigmoid scores, 2 with softmax.
//
// Bound by the vector units, some 470 instructions of four cycles per token:
// 32771 tokens of 256 experts, k = 8, 18 us by the logits alone, 22 with sigmoid
// scores and a bias, 29 with eight groups (single launches in a profile 32); the bytes
// would take 7.
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
  int32_t lanes;          // lanes of a group, if that is a power of two, else 0
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

// n / d to little more than half a step, 1 where n == d: the hardware's reciprocal
// (off by a step) and one Newton step.  For 1e-20 <= d < 2^20 and 0 <= n <= d.
__device__ __forceinline__ float route_quotient(float n, float d) {
  const float r = __builtin_amdgcn_rcpf(d), q = n * r;
  return fmaf(fmaf(-q, d, n), r, q);
}

// Score of one expert; top and sum are the row's largest logit and the sum of its
// exponentials (softmax).  A sigmoid by its smaller side's exponential, which has a
// digit wherever the score has one.
__device__ __forceinline__ float route_score(float x, int sigmoid, float top, float sum) {
  const float e = expf(sigmoid ? -fabsf(x) : x - top);
  return route_quotient(sigmoid && x >= 0.f ? 1.f : e, sigmoid ? 1.f + e : sum);
}

// exp(x) by the hardware's 2^x: relatively off by (|x| + 2) 2^-23, a fifth of the
// instructions.  For keys, sums and gradients; the weights' scores are taken from
// expf.  Quotients in these are products with the hardware's reciprocal, one step off.
__device__ __forceinline__ float route_exp(float x) { return __builtin_amdgcn_exp2f(x * 1.44269504f); }

// Largest logit and sum of exp(x - largest) of a row (softmax); x becomes the
// exponentials.
template <int PER>
__device__ __forceinline__ void route_softmax(float (&x)[PER], int first, int n, float& top, float& sum) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i)
    if (first + i < n) m = max(m, route_key(x[i]));
  top = route_value(wave_max(m));
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    x[i] = first + i < n ? route_exp(x[i] - top) : 0.f;
    s += x[i];
  }
  sum = wave_sum(s);
}

// Distance within which fp32 keys do not decide, for keys of size `key`.  A
// softmax's score is off by (|x - top| + 32) 2^-23 of itself (the sum's 22 additions
// and its terms' own rounding among them) and s |x - top| is under 1/e; a sigmoid's by
// less than 8 2^-23.  `most` bounds the scores.  Twice that for two of them, and
// their additions' rounding.
__device__ __forceinline__ float route_doubt(float most, float key) {
  return 0x1p-22f * (34.f * most + 1.f + 2.f * fabsf(key));
}

// Two largest keys of a lane's own.
template <int PER, class K>
__device__ __forceinline__ void route_two(const K (&k)[PER], K& one, K& two) {
  one = k[0];
  two = 0;
#pragma unroll
  for (int i = 1; i < PER; ++i) {
    two = max(two, min(one, k[i]));
    one = max(one, k[i]);
  }
}

// The same lane's value, LANES / 2 further in its row of LANES, for LANES <= 16 as a
// mirror: callers hold the same in both halves' lanes.
template <int LANES>
__device__ __forceinline__ uint32_t route_swap(uint32_t v) {
  if constexpr (LANES == 2) return static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(v), 0xb1, 0xf, 0xf, true));
  if constexpr (LANES == 4) return static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(v), 0x4e, 0xf, 0xf, true));
  if constexpr (LANES == 8) return static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(v), 0x141, 0xf, 0xf, true));
  if constexpr (LANES == 16) return static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(v), 0x140, 0xf, 0xf, true));
  return static_cast<uint32_t>(__shfl_xor(static_cast<int>(v), LANES / 2, 64));
}
template <int LANES>
__device__ __forceinline__ uint64_t route_swap(uint64_t v) {
  return static_cast<uint64_t>(route_swap<LANES>(static_cast<uint32_t>(v >> 32))) << 32 | route_swap<LANES>(static_cast<uint32_t>(v));
}

// Groups: which of this lane's experts stay, as bits.  vk: keys of score + bias, 0
// where there is no expert.  `close`: the border between the last group that
// stays and the first that does not is nearer than `doubt` says of the sums.
template <int PER, class V, class K>
__device__ __forceinline__ uint32_t route_groups(const RouteArgs& a, const K (&vk)[PER], int lane, float most,
                                                 bool& close) {
  const int first = lane * PER;
  int step;       // lanes between the first lanes of groups; group g's sum is with lane g * step
  V mine = V(0);
  if (a.lanes > 0) {
    // a group is a.lanes lanes, a power of two up to 32 (there are two groups at least):
    // their two largest by exchanges
    K one, two;
    route_two<PER, K>(vk, one, two);
    auto merge = [&](auto lanes_c) {
      constexpr int L = decltype(lanes_c)::value;
      if (a.lanes < L) return;
      const K o1 = route_swap<L>(one), o2 = route_swap<L>(two);
      two = max(max(two, o2), min(one, o1));
      one = max(one, o1);
    };
    merge(std::integral_constant<int, 2>{});
    merge(std::integral_constant<int, 4>{});
    merge(std::integral_constant<int, 8>{});
    merge(std::integral_constant<int, 16>{});
    merge(std::integral_constant<int, 32>{});
    mine = route_value(one);
    if (a.group_size > 1) mine += route_value(two);
    step = a.lanes;
  } else {
    for (int g = 0; g < a.groups; ++g) {
      const int lo = g * a.group_size, hi = lo + a.group_size;
      K in[PER], one, two;
#pragma unroll
      for (int i = 0; i < PER; ++i) in[i] = first + i >= lo && first + i < hi ? vk[i] : K(0);
      route_two<PER, K>(in, one, two);
      const K best = wave_max(one);
      const int owner = __builtin_ctzll(__ballot(one == best));
      const K next = wave_max(lane == owner ? two : one);
      V sum = route_value(best);
      if (a.group_size > 1) sum += route_value(next);
      if (lane == g) mine = sum;
    }
    step = 1;
  }
  // how many groups are before a lane's own (and where it has none, before none)
  const K key = route_key(mine);
  const int own = lane / step;
  const bool group = lane < a.groups * step;
  int rank = 0;
  bool stays;
  if constexpr (sizeof(K) == 8) {
    for (int g = 0; g < a.groups; ++g) {
      const int at = g * step;
      const K other = static_cast<uint64_t>(static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(key >> 32), at))) << 32 |
                      static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(key), at));
      rank += other > key || (other == key && g < own) ? 1 : 0;
    }
    stays = group && rank < a.top;
  } else {
    // equal sums at the border show as too many that stay: fp64 then
    for (int g = 0, at = 0; g < a.groups; ++g, at += step)
      rank += static_cast<K>(__builtin_amdgcn_readlane(static_cast<int>(key), at)) > key ? 1 : 0;
    stays = group && rank < a.top;
    if (a.top < a.groups) {
      const float out = route_value(wave_max(group && !stays ? key : 0u));
      const float in = route_value(~wave_max(stays ? ~key : 0u));
      close = __popcll(__ballot(stays)) != a.top * step || !(in - out > 2.f * route_doubt(most, fabsf(in) + fabsf(out)));
    }
  }
  if (a.lanes > 0) return stays ? 0xffffffffu : 0u;
  const uint64_t bits = __ballot(stays);
  uint32_t mask = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i)
    mask |= first + i < a.n ? static_cast<uint32_t>(bits >> ((first + i) / a.group_size) & 1) << i : 0u;
  return mask;
}

// The k largest keys in order, lane j receiving expert j (others -1).  A lane's keys
// are lists of up to four, each sorted first, with their places, by rank, as the
// digits of one word (of equal keys the lower place is first): a round then compares
// the lists' heads alone, and the list that the winner is of moves up by one.  (One
// search per round over eight unsorted keys: 32768 x 512, k = 10, 40 us; one sorted
// list of eight 64; two of four 34.)  On return key[0] is the largest that a lane
// has left.
template <int PER, class K>
__device__ __forceinline__ int route_pick(K (&key)[PER], int k, int lane) {
  constexpr int W = PER < 4 ? PER : 4, LISTS = PER / W;
  int mine = -1;
  uint32_t digits[LISTS];
#pragma unroll
  for (int l = 0; l < LISTS; ++l) {
    K(&at)[W] = *reinterpret_cast<K(*)[W]>(&key[l * W]);
    int rank[W];
#pragma unroll
    for (int i = 0; i < W; ++i) rank[i] = i;
#pragma unroll
    for (int i = 0; i < W; ++i)
#pragma unroll
      for (int q = i + 1; q < W; ++q) {
        const int after = at[i] < at[q] ? 1 : 0;
        rank[i] += after;
        rank[q] -= after;
      }
    digits[l] = 0;
#pragma unroll
    for (int i = 0; i < W; ++i) digits[l] |= static_cast<uint32_t>(l * W + i) << (4 * rank[i]);
#pragma unroll
    for (int end = W - 1; end > 0; --end)
#pragma unroll
      for (int i = 0; i < end; ++i) {
        const K hi = max(at[i], at[i + 1]);
        at[i + 1] = min(at[i], at[i + 1]);
        at[i] = hi;
      }
  }
  auto head = [&] {
    K h = key[0];
#pragma unroll
    for (int l = 1; l < LISTS; ++l) h = max(h, key[l * W]);
    return h;
  };
  for (int j = 0; j < k; ++j) {
    const K h = head(), m = wave_max(h);
    const int owner = __builtin_ctzll(__ballot(h == m));
    uint64_t left = uint64_t(1) << owner;     // of the owner's lists, the first with it
    int place = 0;
#pragma unroll
    for (int l = 0; l < LISTS; ++l) {
      const uint64_t of = LISTS == 1 ? left : left & __ballot(key[l * W] == m);
      left &= ~of;
      const bool won = __builtin_amdgcn_inverse_ballot_w64(of);    // no comparison per lane
      const int digit = __builtin_amdgcn_readlane(static_cast<int>(digits[l]), owner) & 15;
      if (LISTS == 1 || of) place = digit;
#pragma unroll
      for (int i = 0; i < W; ++i) key[l * W + i] = won ? (i + 1 < W ? key[l * W + (i + 1) % W] : K(0)) : key[l * W + i];
      digits[l] = won ? digits[l] >> 4 : digits[l];
    }
    const int e = owner * PER + place;
    mine = __builtin_amdgcn_inverse_ballot_w64(uint64_t(1) << j) ? e : mine;
  }
  key[0] = head();
  return mine;
}

// The choice in fp64, where fp32 leaves it open.
template <class E, int PER>
__device__ __forceinline__ int route_exact(const RouteArgs& a, const typename E::storage_t* row, float top, int lane) {
  const int first = lane * PER;
  float x[PER], b[PER];
  route_load<E, PER>(row, first, a.n, 0.f, x);
#pragma unroll
  for (int i = 0; i < PER; ++i) b[i] = 0.f;
  if (a.bias) route_load<ElemF32, PER>(a.bias, first, a.n, 0.f, b);
  const double dtop = top;
  double sum = 1.0;
  if (!a.sigmoid) {
    double s = 0.0;
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (first + i < a.n) s += exp(static_cast<double>(x[i]) - dtop);
    sum = warp_sum(s);
  }
  uint64_t key[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const double s = a.sigmoid ? 1.0 / (1.0 + exp(-static_cast<double>(x[i]))) : exp(static_cast<double>(x[i]) - dtop) / sum;
    key[i] = first + i < a.n ? route_key(s + static_cast<double>(b[i])) : 0ull;
  }
  uint32_t stay = 0xffffffffu;
  bool none = false;
  if (a.groups > 1) stay = route_groups<PER, double, uint64_t>(a, key, lane, 0.f, none);
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    if (!(stay >> i & 1)) key[i] = 0;
    else if (!a.bias && key[i]) key[i] = route_key(x[i]);
  }
  return route_pick<PER, uint64_t>(key, a.k, lane);
}

template <class E, int PER>
__global__ __launch_bounds__(256) void route_kernel(RouteArgs a) {
  using S = typename E::storage_t;
  const int lane = threadIdx.x & 63;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
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
  const bool on = lane < a.k;
  float top = 0.f, sum = 1.f;
  uint32_t key[PER];
  int mine;
  float mx;
  if (!a.bias) {      // the logits decide (within the groups)
#pragma unroll
    for (int i = 0; i < PER; ++i) key[i] = first + i < a.n ? route_key(x[i]) : 0u;
  }
  if (!a.sigmoid) route_softmax<PER>(x, first, a.n, top, sum);     // x: exponentials
  bool close = false;
  if (!a.bias && a.groups == 1) {
    mine = route_pick<PER, uint32_t>(key, a.k, lane);
    mx = on ? E::to_f32(gld<S>(row + mine)) : 0.f;
  } else {
    const float most = a.sigmoid ? 1.f : __builtin_amdgcn_rcpf(sum);
    float v[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) v[i] = 0.f;
    if (a.bias) route_load<ElemF32, PER>(a.bias, first, a.n, 0.f, v);
    uint32_t vk[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      v[i] += a.sigmoid ? __builtin_amdgcn_rcpf(1.f + route_exp(-x[i])) : x[i] * most;
      vk[i] = first + i < a.n ? route_key(v[i]) : 0u;
    }
    if (a.groups > 1) {
      const uint32_t stay = route_groups<PER, float, uint32_t>(a, vk, lane, most, close);
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        if (a.bias) vk[i] = stay >> i & 1 ? vk[i] : 0u;
        else key[i] = stay >> i & 1 ? key[i] : 0u;
      }
    }
    if (!a.bias) {
      mine = route_pick<PER, uint32_t>(key, a.k, lane);
      mx = on ? E::to_f32(gld<S>(row + mine)) : 0.f;
    } else {
      mine = route_pick<PER, uint32_t>(vk, a.k, lane);
      // neighbours in the order, unless they are equal, and the last against
      // what is left
      mx = on ? E::to_f32(gld<S>(row + mine)) : 0.f;
      const float mb = on ? gld<float>(a.bias + mine) : 0.f;
      const float mk = (a.sigmoid ? __builtin_amdgcn_rcpf(1.f + route_exp(-mx)) : route_exp(mx - top) * most) + mb;
      const float doubt = route_doubt(most, mk);
      // every lane takes part in these, before any of them can leave
      const float nk = wave_next(mk), nx = wave_next(mx), nb = wave_next(mb);
      auto last = [&](float q) { return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(q), a.k - 1)); };
      const float lk = last(mk), ld = last(doubt);
      const bool order = (lane + 1 < a.k) & !(mk - nk > doubt) & !((nx == mx) & (nb == mb));
      const bool rest = (vk[0] != 0) & !(lk - route_value(vk[0]) > ld);
      close = __ballot(order | rest) != 0 || close;
    }
  }
  if (__builtin_expect(close, 0)) {
    mine = route_exact<E, PER>(a, row, top, lane);
    mx = on ? E::to_f32(gld<S>(row + mine)) : 0.f;
  }

  const float s = on ? route_score(mx, a.sigmoid, top, sum) : 0.f;
  const float part = a.renorm ? route_quotient(s, wave_sum(s) + kRouteTiny) : s;
  if (on) {
    chosen[lane] = mine;
    weights[lane] = a.scale * part;
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
// Bound by HBM, 5.2 TB/s: 32771 tokens of 256 experts fp32, k = 8, 13.3 us.  The
// chosen experts' terms reach the lanes that hold them
// through LDS (a loop over them, which experts that are named twice still take,
// was 40% of the instructions).
template <class E, int PER>
__global__ __launch_bounds__(256) void route_grad_kernel(RouteGradArgs a) {
  using S = typename E::storage_t;
  __shared__ __align__(16) float term[4][64 * PER];
  __shared__ int tag[4][64 * PER];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t t = static_cast<int64_t>(blockIdx.x) * 4 + wave;
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
    float x[PER], top = 0.f, inv = 1.f;
    if (!a.sigmoid) {
      route_load<E, PER>(row, first, a.n, 0.f, x);
      route_softmax<PER>(x, first, a.n, top, inv);      // x: exponentials
      inv = __builtin_amdgcn_rcpf(inv);
    }
    const float q = route_exp(a.sigmoid ? -fabsf(xe) : xe - top), r = __builtin_amdgcn_rcpf(1.f + q);
    const float s = !on ? 0.f : !a.sigmoid ? q * inv : xe >= 0.f ? r : q * r;
    float ds = a.scale * g;
    if (a.renorm) {
      const float d = __builtin_amdgcn_rcpf(wave_sum(s) + kRouteTiny);
      ds = a.scale * d * (g - wave_sum(g * s) * d);
    }
    if (!on) ds = 0.f;
    float c = 0.f;
    if (a.sigmoid) ds *= q * r * r;             // s (1 - s), no difference
    else c = wave_sum(ds * s);
    // one wave's own part of LDS: its operations are in order
#pragma unroll
    for (int i = 0; i < PER; ++i) term[wave][first + i] = 0.f;
    if (on) tag[wave][e] = lane;
    __builtin_amdgcn_wave_barrier();
    if (on) term[wave][e] = ds;
    const bool twice = on && tag[wave][e] != lane;
    __builtin_amdgcn_wave_barrier();
    if (__builtin_expect(__ballot(twice) == 0, 1)) {
#pragma unroll
      for (int i = 0; i < PER; ++i) dx[i] = term[wave][first + i];
    } else {
      for (int j = 0; j < a.k; ++j) {           // an expert that is named twice adds up
        const int ej = __builtin_amdgcn_readlane(e, j);
        const float dj = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(ds), j));
#pragma unroll
        for (int i = 0; i < PER; ++i)
          if (ej == first + i) dx[i] += dj;
      }
    }
    if (!a.sigmoid) {
#pragma unroll
      for (int i = 0; i < PER; ++i) dx[i] = x[i] * inv * (dx[i] - c);
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
// Plan: a stable counting sort of (token, choice) by expert.  Bound by latency: two
// launches, each a few dependent trips to memory (262168 choices of 256 experts
// 9.8 us, 2^21 of them 18).
// ---------------------------------------------------------------------------
constexpr int kPlanThreads = 1024;
constexpr int kPlanWaves = kPlanThreads / 64;
constexpr int kPlanBinsMax = kRouteExpertsMax;
constexpr int kPlanSmall = 8 * kPlanThreads;    // slots that one workgroup takes alone: 4096 take 5.9 us, 8192 9.5, 16396 14; two launches 10.1

struct PlanArgs {
  const int32_t* chosen;   // n slots; outside [0, experts): no row
  int32_t* offsets;        // experts + 1
  int32_t* place;          // n
  uint32_t* hist;          // [blocks][pitch]: counts of each expert
  int32_t n, experts;
  int32_t pitch;           // experts, a multiple of four
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
    a.hist[static_cast<size_t>(blockIdx.x) * a.pitch + b] = h[b];
}

// Rows of a workgroup's slots: each wave takes a contiguous part, counts of each
// wave's own give its first rows, and within 64 slots the lower lanes with the
// same expert are counted by ballots over the bits of its number.  Counts are sums
// of whole numbers: the order in which they are added does not show.
__device__ __forceinline__ int plan_wave_slots(int slots) { return (slots + kPlanThreads - 1) / kPlanThreads * 64; }

// cnt: from counts of each wave to its first rows; base: the workgroup's.
__device__ __forceinline__ void plan_first_rows(const PlanArgs& a, const uint32_t* base, uint32_t (*cnt)[kPlanBinsMax]) {
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
}

// The 64 slots from i on, of experts e, the wave's part ending at w1.
__device__ __forceinline__ void plan_round(const PlanArgs& a, int i, int w1, uint32_t e, uint32_t* cnt) {
  const int lane = threadIdx.x & 63;
  const bool on = e != 0xffffffffu;
  const uint64_t there = __ballot(on);
  uint32_t lo = static_cast<uint32_t>(there), hi = static_cast<uint32_t>(there >> 32);
  for (int b = 0; b < a.bits; ++b) {
    const uint32_t bit = 0u - (e >> b & 1);       // all of it or none
    const uint64_t m = __ballot(bit);
    lo &= ~(bit ^ static_cast<uint32_t>(m));
    hi &= ~(bit ^ static_cast<uint32_t>(m >> 32));
  }
  int row = -1;
  if (on) {
    const uint32_t rank = __builtin_amdgcn_mbcnt_hi(hi, __builtin_amdgcn_mbcnt_lo(lo, 0));
    const uint32_t at = cnt[e] + rank;
    row = static_cast<int>(at);
    // the highest lane of each expert moves the wave's place on, behind the
    // reads above (one wave, LDS operations in order)
    if (rank + 1 == static_cast<uint32_t>(__popc(lo) + __popc(hi))) cnt[e] = at + 1;
  }
  if (i + lane < w1) a.place[i + lane] = row;
  __builtin_amdgcn_wave_barrier();
}

// Exclusive scan of tot[0 .. experts) into base, plus add; one expert a thread.
__device__ __forceinline__ void plan_scan(const uint32_t* tot, const uint32_t* add, uint32_t* base, int experts,
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
}
static_assert(kPlanBinsMax <= kPlanThreads, "plan_scan takes one expert per thread");

// The second of two launches.
__global__ __launch_bounds__(kPlanThreads) void plan_place_kernel(PlanArgs a) {
  __shared__ uint32_t base[kPlanBinsMax], tot[kPlanBinsMax], add[kPlanBinsMax];
  __shared__ uint32_t cnt[kPlanWaves][kPlanBinsMax];
  __shared__ uint32_t wave_sum[kPlanWaves];
  // every workgroup adds up all counts: four experts a thread, as many threads per
  // four as there are, eight loads of each in flight
  for (int b = threadIdx.x; b < a.experts; b += kPlanThreads) tot[b] = add[b] = 0;
  __syncthreads();
  const int wide = (a.pitch / 4 + 63) & ~63, slices = kPlanThreads / wide;
  const int b = threadIdx.x % wide * 4, blocks = static_cast<int>(gridDim.x), here = static_cast<int>(blockIdx.x);
  const int slice = __builtin_amdgcn_readfirstlane(threadIdx.x / wide);     // whole waves: addresses and ends are scalars
  if (b < a.experts && slice < slices) {
    uint32_t t[4] = {}, before[4] = {};
    for (int w = slice; w < blocks; w += 8 * slices) {
      uint4 c[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) c[i] = gld<uint4>(a.hist + static_cast<size_t>(min(w + i * slices, blocks - 1)) * a.pitch + b);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int at = w + i * slices;
        const uint32_t v[4] = {c[i].x, c[i].y, c[i].z, c[i].w};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          if (at < blocks) t[q] += v[q];
          if (at < here) before[q] += v[q];
        }
      }
    }
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (b + q < a.experts) {
        atomicAdd(&tot[b + q], t[q]);
        atomicAdd(&add[b + q], before[q]);
      }
  }
  __syncthreads();
  plan_scan(tot, add, base, a.experts, wave_sum, blockIdx.x == 0 ? a.offsets : nullptr);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int i0 = blockIdx.x * a.per_block, i1 = min(i0 + a.per_block, a.n), per_wave = plan_wave_slots(i1 - i0);
  const int w0 = min(i0 + wave * per_wave, i1), w1 = min(w0 + per_wave, i1);
  for (int b = lane; b < a.experts; b += 64) cnt[wave][b] = 0;
  __syncthreads();
  for (int i = w0 + lane; i < w1; i += 64) {
    const uint32_t e = plan_expert(a, i);
    if (e != 0xffffffffu) atomicAdd(&cnt[wave][e], 1u);
  }
  __syncthreads();
  plan_first_rows(a, base, cnt);
  auto fetch = [&](int i) { return i + lane < w1 ? plan_expert(a, i + lane) : 0xffffffffu; };
  uint32_t next = fetch(w0);
  for (int i = w0; i < w1; i += 64) {
    const uint32_t e = next;
    next = fetch(i + 64);
    plan_round(a, i, w1, e, cnt[wave]);
  }
}

// One workgroup for all slots, which stay in registers: read once, counted once.
__global__ __launch_bounds__(kPlanThreads) void plan_small_kernel(PlanArgs a) {
  constexpr int ROUNDS = kPlanSmall / kPlanThreads;
  __shared__ uint32_t base[kPlanBinsMax], tot[kPlanBinsMax], add[kPlanBinsMax];
  __shared__ uint32_t cnt[kPlanWaves][kPlanBinsMax];
  __shared__ uint32_t wave_sum[kPlanWaves];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int per_wave = plan_wave_slots(a.n), w0 = min(wave * per_wave, a.n), w1 = min(w0 + per_wave, a.n);
  uint32_t e[ROUNDS];
#pragma unroll
  for (int r = 0; r < ROUNDS; ++r) e[r] = w0 + 64 * r + lane < w1 ? plan_expert(a, w0 + 64 * r + lane) : 0xffffffffu;
  for (int b = lane; b < a.experts; b += 64) cnt[wave][b] = 0;
  __syncthreads();
#pragma unroll
  for (int r = 0; r < ROUNDS; ++r)
    if (e[r] != 0xffffffffu) atomicAdd(&cnt[wave][e[r]], 1u);
  __syncthreads();
  for (int b = threadIdx.x; b < a.experts; b += kPlanThreads) {
    uint32_t t = 0;
#pragma unroll
    for (int w = 0; w < kPlanWaves; ++w) t += cnt[w][b];
    tot[b] = t;
    add[b] = 0;
  }
  __syncthreads();
  plan_scan(tot, add, base, a.experts, wave_sum, a.offsets);
  plan_first_rows(a, base, cnt);
#pragma unroll
  for (int r = 0; r < ROUNDS; ++r)
    if (w0 + 64 * r < w1) plan_round(a, w0 + 64 * r, w1, e[r], cnt[wave]);
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
