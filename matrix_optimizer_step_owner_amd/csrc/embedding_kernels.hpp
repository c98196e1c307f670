// Embedding rows of a list of tokens and the table's gradient (gfx950).
//
//   lookup    out[i] = scale * table[token_i], rounded once
//   gradient  grad[v] = beta * grad[v] + scale * sum_{i: token_i = v} dY[i]
//
// A token outside [0, vocab) stands for padding: its row is zero and it adds
// nothing.  The gradient is the dense fp32 segment of a packed AdamW tail.  It
// is a sum over the tokens in sorted order, never of atomics: positions are
// sorted by token (a stable radix sort, so equal tokens keep their order), one
// workgroup per block of table rows adds each row's positions one after the
// other, and a row with more than kEmbRun positions is first summed in chunks
// of kEmbRun sorted positions by workgroups of their own, so that a frequent
// token does not hold up one workgroup.  Results depend on nothing but the
// inputs.
#pragma once

#include "common.hpp"
#include "ns_gemm.hpp"

namespace mfsdp {

// ---------------------------------------------------------------------------
// Lookup
// ---------------------------------------------------------------------------
struct EmbArgs {
  const void* table;     // vocab x d, contiguous
  const void* tokens;    // int32 or int64
  void* out;             // tokens x d, row stride ldo
  int64_t n_tokens, vocab, ldo;
  int32_t d;
  int32_t tok64;
  int32_t chunks;        // workgroups per token (wide rows), or 0
  int32_t per_wg;        // tokens per workgroup (narrow rows)
  float scale;
};

__device__ __forceinline__ int64_t emb_token(const void* tokens, int tok64, int64_t i) {
  return tok64 ? static_cast<const int64_t*>(tokens)[i] : static_cast<const int32_t*>(tokens)[i];
}

// A unit is eight columns of one row on the vector path (rows of both sides
// start on 16 bytes, d a multiple of eight), one column otherwise.
// Bound by HBM: each row is read once and written once.
template <class ET, class EO, bool VEC>
__global__ __launch_bounds__(256) void embedding_kernel(EmbArgs a) {
  using T = typename ET::storage_t;
  using O = typename EO::storage_t;
  constexpr int W = VEC ? 8 : 1;
  const int units = a.d / W;
  int64_t i;
  int u;
  if (a.chunks) {
    i = blockIdx.x / a.chunks;
    u = static_cast<int>(blockIdx.x % a.chunks) * 256 + threadIdx.x;
  } else {
    const int t = threadIdx.x / units;
    i = static_cast<int64_t>(blockIdx.x) * a.per_wg + t;
    u = threadIdx.x - t * units;
    if (t >= a.per_wg) return;
  }
  if (i >= a.n_tokens || u >= units) return;
  const int64_t tok = emb_token(a.tokens, a.tok64, i);
  const bool in = tok >= 0 && tok < a.vocab;
  O* dst = static_cast<O*>(a.out) + i * a.ldo + u * W;
  const T* src = static_cast<const T*>(a.table) + (in ? tok : 0) * a.d + u * W;
  if constexpr (VEC) {
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (in) {
      load8<ET>(src, v);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] *= a.scale;
    }
    store8<EO>(dst, v);
  } else {
    *dst = EO::from_f32(in ? ET::to_f32(*src) * a.scale : 0.f);
  }
}

// ---------------------------------------------------------------------------
// Stable radix sort of (token, position)
// ---------------------------------------------------------------------------
constexpr int kSortThreads = 256;
constexpr int kSortWaves = kSortThreads / 64;
constexpr int kSortBitsMax = 9;                       // digit bits of one pass
constexpr int kSortBinsMax = 1 << kSortBitsMax;

struct SortArgs {
  const void* tokens;      // first pass: keys come from here
  const uint32_t* key_in;  // later passes
  const uint32_t* pos_in;
  uint32_t* key_out;
  uint32_t* pos_out;
  uint32_t* hist;          // [blocks][bins]
  int64_t vocab;
  int32_t n, tok64, first;
  int32_t per_block;       // keys per workgroup, a multiple of kSortThreads
  int32_t shift, bits;
};

// Key of position i: its token, or vocab (sorted last) for padding.
__device__ __forceinline__ uint32_t sort_key(const SortArgs& s, int i) {
  if (!s.first) return s.key_in[i];
  const int64_t t = emb_token(s.tokens, s.tok64, i);
  return static_cast<uint32_t>(t >= 0 && t < s.vocab ? t : s.vocab);
}

__global__ __launch_bounds__(kSortThreads) void sort_hist_kernel(SortArgs s) {
  __shared__ uint32_t h[kSortBinsMax];
  const int bins = 1 << s.bits;
  for (int b = threadIdx.x; b < bins; b += kSortThreads) h[b] = 0;
  __syncthreads();
  const int64_t i0 = static_cast<int64_t>(blockIdx.x) * s.per_block;
  const int i1 = static_cast<int>(min(i0 + s.per_block, static_cast<int64_t>(s.n)));
  for (int64_t i = i0 + threadIdx.x; i < i1; i += kSortThreads)
    atomicAdd(&h[(sort_key(s, static_cast<int>(i)) >> s.shift) & (bins - 1)], 1u);
  __syncthreads();
  for (int b = threadIdx.x; b < bins; b += kSortThreads)
    s.hist[static_cast<size_t>(blockIdx.x) * bins + b] = h[b];
}

// One pass over one workgroup's keys [i0, i1): each wave takes a contiguous
// quarter, so that order is kept.  base[] holds where each bin of this
// workgroup starts in the output; the per-wave counts then give each wave its
// start, and within 64 keys a lane's place is the number of lower lanes with
// the same digit (bits ballots).
__device__ __forceinline__ void sort_scatter(const SortArgs& s, int i0, int i1,
                                             const uint32_t* base,
                                             uint32_t (*cnt)[kSortBinsMax]) {
  const int bins = 1 << s.bits;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int per_wave = ((i1 - i0 + kSortThreads - 1) / kSortThreads) * 64;
  const int w0 = min(i0 + wave * per_wave, i1), w1 = min(w0 + per_wave, i1);
  for (int b = threadIdx.x; b < kSortWaves * bins; b += kSortThreads)
    cnt[b >> s.bits][b & (bins - 1)] = 0;
  __syncthreads();
  for (int i = w0 + lane; i < w1; i += 64)
    atomicAdd(&cnt[wave][(sort_key(s, i) >> s.shift) & (bins - 1)], 1u);
  __syncthreads();
  for (int b = threadIdx.x; b < bins; b += kSortThreads) {
    uint32_t at = base[b];
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) {
      const uint32_t c = cnt[w][b];
      cnt[w][b] = at;
      at += c;
    }
  }
  __syncthreads();
  for (int i = w0; i < w1; i += 64) {
    const bool on = i + lane < w1;
    const uint32_t key = on ? sort_key(s, i + lane) : 0;
    const uint32_t pos = on ? (s.first ? static_cast<uint32_t>(i + lane) : s.pos_in[i + lane]) : 0;
    const uint32_t d = (key >> s.shift) & (bins - 1);
    uint64_t same = __ballot(on);
    for (int b = 0; b < s.bits; ++b) {
      const uint64_t m = __ballot((d >> b) & 1);
      same &= (d >> b) & 1 ? m : ~m;
    }
    if (on) {
      const uint32_t rank = __popcll(same & ((uint64_t(1) << lane) - 1));
      const uint32_t at = cnt[wave][d] + rank;
      s.key_out[at] = key;
      s.pos_out[at] = pos;
      // the highest lane of each digit moves the wave's place on; its read of
      // the count above is ordered before this write, as are the others'
      // (one wave, LDS operations in order)
      if (rank + 1 == static_cast<uint32_t>(__popcll(same))) cnt[wave][d] = at + 1;
    }
    __builtin_amdgcn_wave_barrier();
  }
}

// Exclusive scan of tot[0..bins) into base[], plus add[]; kSortThreads threads.
__device__ __forceinline__ void sort_scan(const uint32_t* tot, const uint32_t* add, uint32_t* base,
                                          int bins, uint32_t* wave_sum) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int b0 = 2 * threadIdx.x;   // kSortBinsMax = 2 * kSortThreads
  const uint32_t t0 = b0 < bins ? tot[b0] : 0, t1 = b0 + 1 < bins ? tot[b0 + 1] : 0;
  uint32_t incl = t0 + t1;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const uint32_t v = __shfl_up(incl, d, 64);
    if (lane >= d) incl += v;
  }
  if (lane == 63) wave_sum[wave] = incl;
  __syncthreads();
  uint32_t before = incl - t0 - t1;
  for (int w = 0; w < wave; ++w) before += wave_sum[w];
  if (b0 < bins) base[b0] = before + add[b0];
  if (b0 + 1 < bins) base[b0 + 1] = before + t0 + add[b0 + 1];
  __syncthreads();
}
static_assert(kSortBinsMax == 2 * kSortThreads, "sort_scan takes two bins per thread");

__global__ __launch_bounds__(kSortThreads) void sort_scatter_kernel(SortArgs s) {
  __shared__ uint32_t base[kSortBinsMax], tot[kSortBinsMax], add[kSortBinsMax];
  __shared__ uint32_t cnt[kSortWaves][kSortBinsMax];
  __shared__ uint32_t wave_sum[kSortWaves];
  const int bins = 1 << s.bits;
  for (int b = threadIdx.x; b < bins; b += kSortThreads) {
    uint32_t t = 0, before = 0;
    for (unsigned w = 0; w < gridDim.x; ++w) {
      const uint32_t c = s.hist[static_cast<size_t>(w) * bins + b];
      if (w < blockIdx.x) before += c;
      t += c;
    }
    tot[b] = t;
    add[b] = before;
  }
  __syncthreads();
  sort_scan(tot, add, base, bins, wave_sum);
  const int64_t i0 = static_cast<int64_t>(blockIdx.x) * s.per_block;
  const int i1 = static_cast<int>(min(i0 + s.per_block, static_cast<int64_t>(s.n)));
  sort_scatter(s, static_cast<int>(i0), i1, base, cnt);
}

// A list that one workgroup sorts: every pass in one launch, between the two
// pairs of buffers; the last pass writes key_out / pos_out.
struct SortSmallArgs {
  SortArgs s;              // key_out, pos_out: the sorted list
  uint32_t *key_tmp, *pos_tmp;
  int32_t key_bits, passes;
};

__global__ __launch_bounds__(kSortThreads) void sort_small_kernel(SortSmallArgs a) {
  __shared__ uint32_t base[kSortBinsMax], tot[kSortBinsMax], add[kSortBinsMax];
  __shared__ uint32_t cnt[kSortWaves][kSortBinsMax];
  __shared__ uint32_t wave_sum[kSortWaves];
  for (int p = 0; p < a.passes; ++p) {
    SortArgs s = a.s;
    s.first = p == 0;
    s.shift = p * s.bits;
    const bool to_out = ((a.passes - 1 - p) & 1) == 0;   // the last pass ends in key_out
    s.key_out = to_out ? a.s.key_out : a.key_tmp;
    s.pos_out = to_out ? a.s.pos_out : a.pos_tmp;
    s.key_in = to_out ? a.key_tmp : a.s.key_out;
    s.pos_in = to_out ? a.pos_tmp : a.s.pos_out;
    const int bins = 1 << s.bits;
    for (int b = threadIdx.x; b < bins; b += kSortThreads) tot[b] = add[b] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < s.n; i += kSortThreads)
      atomicAdd(&tot[(sort_key(s, i) >> s.shift) & (bins - 1)], 1u);
    __syncthreads();
    sort_scan(tot, add, base, bins, wave_sum);
    sort_scatter(s, 0, s.n, base, cnt);
    __threadfence_block();
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------
// Sums over the sorted list
// ---------------------------------------------------------------------------
constexpr int kEmbRun = 64;       // longest run that one workgroup adds alone
constexpr int kEmbRows = 32;      // table rows per workgroup

struct EmbGradArgs {
  const void* dy;          // tokens x d, row stride ld
  const uint32_t* key;     // sorted tokens (padding: vocab, last)
  const uint32_t* pos;     // their positions
  float* part;             // [chunks of kEmbRun sorted positions][2][d]
  float* grad;             // vocab x d
  int64_t vocab, ld;
  int32_t n, d;
  float scale, beta;
};

// First sorted index whose key is >= v.
__device__ __forceinline__ int emb_lower(const uint32_t* key, int n, int64_t v) {
  int lo = 0, hi = n;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (static_cast<int64_t>(key[mid]) < v) lo = mid + 1; else hi = mid;
  }
  return lo;
}

// Sum of dY over sorted positions [b, e), W columns from c, in order.
template <class E, int W>
__device__ __forceinline__ void emb_sum(const EmbGradArgs& a, int b, int e, int c, float (&acc)[W]) {
  using S = typename E::storage_t;
  const S* dy = static_cast<const S*>(a.dy) + c;
  int i = b;
  auto add = [&](int j) {
    float v[W];
    const S* p = dy + a.pos[j] * a.ld;
    if constexpr (W == 8) load8<E>(p, v); else v[0] = E::to_f32(*p);
#pragma unroll
    for (int k = 0; k < W; ++k) acc[k] += v[k];
  };
  for (; i + 4 <= e; i += 4) {
    add(i);
    add(i + 1);
    add(i + 2);
    add(i + 3);
  }
  for (; i < e; ++i) add(i);
}

// Partial sums of the runs longer than kEmbRun: workgroup (chunk, columns).
// Such a run covers the first or the last position of every chunk it meets,
// so a chunk has at most two partial rows: slot 0 for the run at its first
// position, slot 1 for another one at its last.
template <class E, int W>
__global__ __launch_bounds__(256) void emb_partial_kernel(EmbGradArgs a, int col_wgs) {
  const int chunk = blockIdx.x / col_wgs;
  const int c = (static_cast<int>(blockIdx.x % col_wgs) * 256 + static_cast<int>(threadIdx.x)) * W;
  const int b = chunk * kEmbRun, e = min(b + kEmbRun, a.n);
  __shared__ int lim[4];
  const uint32_t kf = a.key[b], kl = a.key[e - 1];
  if (threadIdx.x < 4)
    lim[threadIdx.x] = emb_lower(a.key, a.n, static_cast<int64_t>(threadIdx.x < 2 ? kf : kl) + (threadIdx.x & 1));
  __syncthreads();
  if (c >= a.d) return;
#pragma unroll
  for (int slot = 0; slot < 2; ++slot) {
    const int r0 = lim[2 * slot], r1 = lim[2 * slot + 1];
    const uint32_t k = slot ? kl : kf;
    if (r1 - r0 <= kEmbRun || static_cast<int64_t>(k) >= a.vocab || (slot && kl == kf)) continue;
    float acc[W] = {};
    emb_sum<E, W>(a, max(r0, b), min(r1, e), c, acc);
    float* o = a.part + (static_cast<size_t>(chunk) * 2 + slot) * a.d + c;
#pragma unroll
    for (int k2 = 0; k2 < W; k2 += W == 8 ? 4 : 1) {
      if constexpr (W == 8) gst<float4>(o + k2, make_float4(acc[k2], acc[k2 + 1], acc[k2 + 2], acc[k2 + 3]));
      else o[k2] = acc[k2];
    }
  }
}

// Table rows: workgroup (kEmbRows rows, columns).  Bound by HBM: dY is read
// once and every gradient row written once (beta = 0: rows without a token
// are zeroed here, beta = 1: they are not touched).
template <class E, int W>
__global__ __launch_bounds__(256) void emb_rows_kernel(EmbGradArgs a, int col_wgs) {
  const int64_t v0 = static_cast<int64_t>(blockIdx.x / col_wgs) * kEmbRows;
  const int c = (static_cast<int>(blockIdx.x % col_wgs) * 256 + static_cast<int>(threadIdx.x)) * W;
  const int rows = static_cast<int>(min(static_cast<int64_t>(kEmbRows), a.vocab - v0));
  __shared__ int start[kEmbRows + 1];
  if (threadIdx.x <= static_cast<unsigned>(rows))
    start[threadIdx.x] = emb_lower(a.key, a.n, v0 + threadIdx.x);
  __syncthreads();
  if (c >= a.d) return;
  for (int r = 0; r < rows; ++r) {
    const int b = start[r], e = start[r + 1];
    if (b == e && a.beta == 1.f) continue;
    float acc[W] = {};
    if (e - b <= kEmbRun) {
      emb_sum<E, W>(a, b, e, c, acc);
    } else {
      for (int chunk = b / kEmbRun; chunk <= (e - 1) / kEmbRun; ++chunk) {
        const int slot = chunk * kEmbRun >= b ? 0 : 1;
        const float* p = a.part + (static_cast<size_t>(chunk) * 2 + slot) * a.d + c;
#pragma unroll
        for (int k = 0; k < W; ++k) acc[k] += p[k];
      }
    }
    float* o = a.grad + (v0 + r) * a.d + c;
    if constexpr (W == 8) {
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
      if (a.beta != 0.f) {
        x = gld<float4>(o);
        y = gld<float4>(o + 4);
        x = make_float4(a.beta * x.x, a.beta * x.y, a.beta * x.z, a.beta * x.w);
        y = make_float4(a.beta * y.x, a.beta * y.y, a.beta * y.z, a.beta * y.w);
      }
      gst<float4>(o, make_float4(fmaf(a.scale, acc[0], x.x), fmaf(a.scale, acc[1], x.y),
                                 fmaf(a.scale, acc[2], x.z), fmaf(a.scale, acc[3], x.w)));
      gst<float4>(o + 4, make_float4(fmaf(a.scale, acc[4], y.x), fmaf(a.scale, acc[5], y.y),
                                     fmaf(a.scale, acc[6], y.z), fmaf(a.scale, acc[7], y.w)));
    } else {
      *o = fmaf(a.scale, acc[0], a.beta == 0.f ? 0.f : a.beta * *o);
    }
  }
}

}  // namespace mfsdp
