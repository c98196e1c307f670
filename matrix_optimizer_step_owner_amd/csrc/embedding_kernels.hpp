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
//
// Both are bound by HBM.  Lookup of 32768 rows of 4096 bf16 values: 76 us.
// Gradient of the same list on a table of 100000 rows (1.64 GB written, 0.27
// read): 416 us, of it 32 for the two passes of the sort, 25 for the partial
// sums and 350 for the rows; filling the gradient with zeros alone takes 238.
#pragma once

#include <type_traits>

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

// W consecutive elements as loaded, and as floats.  Loads and conversions are
// kept apart, so that several loads can be in flight before the first is waited
// for.
typedef uint32_t u32x2v_t __attribute__((ext_vector_type(2)));
template <class E, int W>
struct EmbRaw {
  static constexpr int kBytes = W * (16 / E::kVec);
  typename std::conditional<
      W == 1, typename E::storage_t,
      typename std::conditional<kBytes == 8, u32x2v_t, u32x4_t>::type>::type r;
  __device__ __forceinline__ void load(const typename E::storage_t* p) { r = gld<decltype(r)>(p); }
  __device__ __forceinline__ void get(float (&v)[W]) const {
    if constexpr (W == 1) {
      v[0] = E::to_f32(r);
    } else {
#pragma unroll
      for (int i = 0; i < W; ++i) {
        if constexpr (E::kVec == 8)
          v[i] = __uint_as_float(i & 1 ? r[i >> 1] & 0xffff0000u : r[i >> 1] << 16);
        else
          v[i] = __uint_as_float(r[i]);
      }
    }
  }
  // streamed store of W values, rounded to the type
  __device__ __forceinline__ static void put(typename E::storage_t* p, const float (&v)[W]) {
    if constexpr (W == 1) {
      gst<typename E::storage_t>(p, E::from_f32(v[0]));
    } else {
      decltype(EmbRaw::r) o;
#pragma unroll
      for (int i = 0; i < kBytes / 4; ++i) {
        if constexpr (E::kVec == 8) o[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
        else o[i] = __float_as_uint(v[i]);
      }
      __builtin_nontemporal_store(o, (MFSDP_GLOBAL decltype(o)*)(p));
    }
  }
};

// A unit is W columns of one row: 16 bytes of the output, where rows of both
// sides start on whole units, one column otherwise.  Bound by HBM: each row is read and
// written once (rows of frequent tokens come from the caches, which the
// streamed output leaves to them).
template <class ET, class EO, bool VEC>
__global__ __launch_bounds__(256) void embedding_kernel(EmbArgs a) {
  using T = typename ET::storage_t;
  using O = typename EO::storage_t;
  constexpr int W = VEC ? EO::kVec : 1;
  constexpr int PART = W < ET::kVec ? W : ET::kVec;   // columns of one load
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
  float v[W] = {};
  if (tok >= 0 && tok < a.vocab) {
    EmbRaw<ET, PART> raw[W / PART];
#pragma unroll
    for (int p = 0; p < W / PART; ++p)
      raw[p].load(static_cast<const T*>(a.table) + tok * a.d + u * W + p * PART);
#pragma unroll
    for (int p = 0; p < W / PART; ++p) {
      float x[PART];
      raw[p].get(x);
#pragma unroll
      for (int e = 0; e < PART; ++e) v[p * PART + e] = x[e] * a.scale;
    }
  }
  EmbRaw<EO, W>::put(static_cast<O*>(a.out) + i * a.ldo + u * W, v);
}

// ---------------------------------------------------------------------------
// Stable radix sort of (token, position)
// ---------------------------------------------------------------------------
constexpr int kSortThreads = 1024;
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
// part, so that order is kept.  base[] holds where each bin of this
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

// Exclusive scan of tot[0..bins) into base[], plus add[]; one bin per thread.
__device__ __forceinline__ void sort_scan(const uint32_t* tot, const uint32_t* add, uint32_t* base,
                                          int bins, uint32_t* wave_sum) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int b = threadIdx.x;
  const uint32_t t = b < bins ? tot[b] : 0;
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
  if (b < bins) base[b] = before + add[b];
  __syncthreads();
}
static_assert(kSortBinsMax <= kSortThreads, "sort_scan takes one bin per thread");

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
constexpr int kEmbRows = 4;       // table rows per workgroup

struct EmbGradArgs {
  const void* dy;          // tokens x d, row stride ld
  const uint32_t* key;     // sorted tokens (padding: vocab, last)
  const uint32_t* pos;     // their positions
  float* part;             // [chunks of kEmbRun sorted positions][2][d]
  int32_t* begin;          // first sorted index of each block of kEmbRows table rows, and n
  float* grad;             // vocab x d
  int64_t vocab, ld;
  int64_t block0;          // first block of table rows of this launch
  int32_t n, d;
  int32_t tpr;             // threads per row: 64, 128 or 256
  float scale, beta;
};

// First sorted index in [lo, hi) whose key is >= v.
__device__ __forceinline__ int emb_lower(const uint32_t* key, int lo, int hi, int64_t v) {
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (static_cast<int64_t>(key[mid]) < v) lo = mid + 1; else hi = mid;
  }
  return lo;
}

// Columns of one thread: kEmbGroups groups of W, a.tpr * W apart, so that a
// wave's accesses are contiguous (W = 4: 8 bytes of bf16 read, 16 of fp32
// written per lane).  a.tpr threads, whole waves, take one row, so that rows
// narrower than a workgroup are taken several at once.
constexpr int kEmbGroups = 2;
constexpr int kEmbFlight = 8;   // rows' loads in flight

// Columns of this thread's groups: first column, or 0 where there is none (a
// load takes no branch: it would be waited for before the next is issued).
struct EmbCols {
  int c[kEmbGroups];
  bool on[kEmbGroups];
  __device__ __forceinline__ EmbCols(int d, int wg, int t, int tpr, int w) {
#pragma unroll
    for (int q = 0; q < kEmbGroups; ++q) {
      const int col = ((wg * kEmbGroups + q) * tpr + t) * w;
      on[q] = t < tpr && col < d;
      c[q] = on[q] ? col : 0;
    }
  }
};

// Adds rows i = b .. e - 1 at row_of(i) to acc, in order, with F rows' loads in
// flight.  Called by whole waves: row_of may exchange lanes.
template <class E, int W, int F, class RowOf>
__device__ __forceinline__ void emb_sum(int b, int e, const EmbCols& cols, RowOf row_of,
                                        float (&acc)[kEmbGroups][W]) {
  for (int i = b; i < e; i += F) {
    EmbRaw<E, W> raw[F][kEmbGroups];
#pragma unroll
    for (int j = 0; j < F; ++j) {
      const typename E::storage_t* p = row_of(min(i + j, e - 1));
#pragma unroll
      for (int q = 0; q < kEmbGroups; ++q) raw[j][q].load(p + cols.c[q]);
    }
#pragma unroll
    for (int j = 0; j < F; ++j)
      if (i + j < e) {
#pragma unroll
        for (int q = 0; q < kEmbGroups; ++q) {
          float v[W];
          raw[j][q].get(v);
#pragma unroll
          for (int k = 0; k < W; ++k) acc[q][k] += v[k];
        }
      }
  }
}

// Partial sums of the runs longer than kEmbRun: workgroup (chunk, columns).
// Such a run covers the first or the last position of every chunk it meets,
// so a chunk has at most two partial rows: slot 0 for the run at its first
// position, slot 1 for another one at its last.  Each wave holds the chunk's 64
// keys, one a lane, and finds both runs' ends by a ballot; one key 64 places
// away then tells whether a run is that long.  The workgroups behind those find
// where each block of table rows begins in the sorted list, so that the next
// kernel's many workgroups do not each search the whole list.
template <class E, int W>
__global__ __launch_bounds__(256) void emb_partial_kernel(EmbGradArgs a, int chunks, int col_wgs) {
  static_assert(kEmbRun == 64, "one key per lane");
  const int chunk = blockIdx.x / col_wgs;
  if (chunk >= chunks) {
    const int64_t i = (static_cast<int64_t>(blockIdx.x) - static_cast<int64_t>(chunks) * col_wgs) * 256 + threadIdx.x;
    const int64_t blocks = (a.vocab + kEmbRows - 1) / kEmbRows;
    if (i <= blocks) a.begin[i] = emb_lower(a.key, 0, a.n, min(i * kEmbRows, a.vocab));
    return;
  }
  const int lane = threadIdx.x & 63;
  const int b = chunk * kEmbRun, e = min(b + kEmbRun, a.n);
  const bool in = b + lane < e;
  const uint32_t key = in ? a.key[b + lane] : 0xffffffffu;   // no token's key
  const uint32_t kf = __shfl(key, 0, 64), kl = __shfl(key, e - b - 1, 64);
  const uint32_t pos = in ? a.pos[b + lane] : 0;
  const int end0 = b + __popcll(__ballot(key == kf));        // of the first position's run, in the chunk
  const int beg1 = e - __popcll(__ballot(key == kl));        // of the last one's
  // longer than 64: 64 places before its last known (or after its first) it goes on
  const bool hot0 = (end0 == e && e < a.n && a.key[e] == kf) ||
                    (end0 > kEmbRun && a.key[end0 - 1 - kEmbRun] == kf);
  const bool hot1 = kl != kf && beg1 + kEmbRun < a.n && a.key[beg1 + kEmbRun] == kl;
  const EmbCols cols(a.d, blockIdx.x % col_wgs, threadIdx.x, a.tpr, W);
  using S = typename E::storage_t;
#pragma unroll
  for (int slot = 0; slot < 2; ++slot) {
    if (!(slot ? hot1 : hot0) || static_cast<int64_t>(slot ? kl : kf) >= a.vocab) continue;
    float acc[kEmbGroups][W] = {};
    emb_sum<E, W, kEmbFlight>(
        slot ? beg1 : b, slot ? e : end0, cols,
        [&](int i) { return static_cast<const S*>(a.dy) + static_cast<int64_t>(__shfl(pos, i - b, 64)) * a.ld; }, acc);
    float* o = a.part + (static_cast<size_t>(chunk) * 2 + slot) * a.d;
#pragma unroll
    for (int q = 0; q < kEmbGroups; ++q)
      if (cols.on[q]) {
#pragma unroll
        for (int x = 0; x < W; ++x) o[cols.c[q] + x] = acc[q][x];
      }
  }
}

// Table rows: workgroup (kEmbRows rows, columns).  Bound by HBM: dY is read once
// and every gradient row written once (beta = 0: rows without a token are
// zeroed here, beta = 1: they are not touched).  Up to 64 keys of the block's
// list sit one a lane, so that each row's part of it comes from two ballots.
template <class E, int W>
__global__ __launch_bounds__(256) void emb_rows_kernel(EmbGradArgs a, int col_wgs) {
  using S = typename E::storage_t;
  const int64_t block = a.block0 + blockIdx.x / col_wgs;
  const int64_t v0 = block * kEmbRows;
  const int lane = threadIdx.x & 63;
  const int sub = threadIdx.x / a.tpr;
  const EmbCols cols(a.d, blockIdx.x % col_wgs, threadIdx.x % a.tpr, a.tpr, W);
  const int rows = static_cast<int>(min(static_cast<int64_t>(kEmbRows), a.vocab - v0));
  const int lb = a.n == 0 ? 0 : a.begin[block], le = a.n == 0 ? 0 : a.begin[block + 1];
  if (W == 4 && lb == le && a.beta == 0.f) {   // no token here: one contiguous stretch of zeros
    float* o = a.grad + v0 * a.d;
    const int64_t n4 = static_cast<int64_t>(rows) * a.d / 4;
    for (int64_t i = static_cast<int64_t>(blockIdx.x % col_wgs) * 256 + threadIdx.x; i < n4; i += 256 * col_wgs)
      gst_stream(o + 4 * i, make_uint4(0, 0, 0, 0));
    return;
  }
  const bool held = le - lb <= 64;
  const uint32_t key = held && lb + lane < le ? a.key[lb + lane] : 0xffffffffu;
  const uint32_t pos = held && lb + lane < le ? a.pos[lb + lane] : 0;
  for (int r = sub; r < rows; r += 256 / a.tpr) {   // one row per wave: every branch is uniform
    const uint32_t v = static_cast<uint32_t>(v0 + r);
    int b = lb, e = lb;
    if (le > lb) {
      if (held) {
        b = lb + __popcll(__ballot(key < v));
        e = lb + __popcll(__ballot(key <= v));
      } else {
        b = emb_lower(a.key, lb, le, v);
        e = emb_lower(a.key, b, le, static_cast<int64_t>(v) + 1);
      }
    }
    if (b == e && a.beta == 1.f) continue;
    float acc[kEmbGroups][W] = {};
    if (e - b > kEmbRun) {   // partial rows of the chunks it meets
      emb_sum<ElemF32, W, kEmbFlight>(
          b / kEmbRun, (e - 1) / kEmbRun + 1, cols,
          [&](int i) { return a.part + (static_cast<size_t>(i) * 2 + (i * kEmbRun >= b ? 0 : 1)) * a.d; }, acc);
    } else if (e > b) {
      emb_sum<E, W, kEmbFlight>(
          b, e, cols,
          [&](int i) {
            const uint32_t at = held ? static_cast<uint32_t>(__shfl(pos, i - lb, 64)) : a.pos[i];
            return static_cast<const S*>(a.dy) + static_cast<int64_t>(at) * a.ld;
          },
          acc);
    }
    float* o = a.grad + (v0 + r) * a.d;
#pragma unroll
    for (int q = 0; q < kEmbGroups; ++q) {
      if (!cols.on[q]) continue;
      float* oq = o + cols.c[q];
      float out[W] = {};
      if (a.beta != 0.f) {
        EmbRaw<ElemF32, W> old;
        old.load(oq);
        old.get(out);
      }
#pragma unroll
      for (int x = 0; x < W; ++x) out[x] = fmaf(a.scale, acc[q][x], a.beta != 0.f ? a.beta * out[x] : 0.f);
      EmbRaw<ElemF32, W>::put(oq, out);
    }
  }
}

}  // namespace mfsdp
