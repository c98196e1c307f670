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
// differ in which operand is contiguous along t, and are one kernel template
// (grouped_tile_kernel): a workgroup computes one C tile, MFMA fragments read
// from LDS panels that arrive by 16-byte DMA a step or more ahead, or, where
// rows do not start on 16 bytes, through registers.
//
// What bounds them, in bf16:
//   - long segments: MFMA issue and the power of it.  8 experts of 14336 x 4096,
//     16384 rows: forward 1.06-1.10, input gradient 1.05 and weight gradient
//     1.16 PFLOP/s (0.95-0.97 from 8-bit codes), 57-64% of the MFMA cycles at 1.7-1.8 GHz;
//     one expert of 4096 x 4096 with 8192 rows 1.22-1.32.  The difference is
//     workgroups that wait for the last round of tiles, tiles that a segment
//     fills in part, and each tile's start and end, which nothing covers at
//     one workgroup per CU.
//   - 256 small experts (512 x 1536) of about 128 rows: HBM.  110, 121 and 110
//     us: 4.4 to 4.9 TB/s, where a plain copy moves 5.1.
//   - few rows: the weights' stream, 5.5-7.1 TB/s; the smallest calls, the
//     latency of a dozen steps (7.6 us).
//   - weight gradients that add to a bf16 dW (beta != 0): its elements, read and
//     written one by one; 256 experts 515 us, where the bytes take 185.
// fp32 runs the same tiles on 32x32x2 MFMAs, 133-139 TFLOP/s.
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
  int32_t stream;        // output rows are whole 128-byte lines
  int32_t stream_w;      // fwd: the weights in use are more than the L2s hold
  int32_t out_f32;       // wgrad: dW is fp32 whatever the operands' type
  int32_t part_rows;     // wgrad: segments are cut into parts of so many rows, 0: they are not
  int32_t parts_max;     // parts that there is room for
  float* part;           // wgrad in parts: [parts][n][k], summed by a second kernel
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

struct GroupSpan {
  int expert;   // whose tile it is
  int local;    // tile number within the expert
  int rows;     // row tiles of the expert
  int first;    // row tiles of the experts before it
};

__device__ __forceinline__ bool group_span(const GroupArgs& g, int b, int bp, int nq, GroupSpan& out) {
  const int lane = threadIdx.x & 63;
  const int c = (g.experts + 63) >> 6;
  const int e0 = min(lane * c, g.experts), e1 = min(e0 + c, g.experts);
  int64_t sum = 0;
  for (int e = e0; e < e1; ++e) {
    int lo, hi;
    group_segment(g, e, lo, hi);
    sum += (hi - lo + bp - 1) / bp;
  }
  int64_t incl = sum;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int64_t v = __shfl_up(incl, d, 64);
    if (lane >= d) incl += v;
  }
  // No more tiles than the grid has (the host bounds it by what ordered offsets
  // can give; others give wrong results, not accesses outside).
  const int total = static_cast<int>(min(__shfl(incl, 63, 64) * nq, static_cast<int64_t>(gridDim.x)));
  if (b >= total) return false;
  const int want = xcd_remap(b, total);
  int64_t at = incl - sum;
  int fe = -1, fl = 0, fr = 0, ff = 0;
  if (want >= at * nq && want < incl * nq) {
    for (int e = e0; e < e1; ++e) {
      int lo, hi;
      group_segment(g, e, lo, hi);
      const int np = (hi - lo + bp - 1) / bp;
      if (want < (at + np) * nq) {
        fe = e;
        fl = static_cast<int>(want - at * nq);
        fr = np;
        ff = static_cast<int>(at);
        break;
      }
      at += np;
    }
  }
  const uint64_t found = __ballot(fe >= 0);
  if (found == 0) return false;
  const int src = __builtin_ctzll(found);
  out.expert = __builtin_amdgcn_readlane(fe, src);
  out.local = __builtin_amdgcn_readlane(fl, src);
  out.rows = __builtin_amdgcn_readlane(fr, src);
  out.first = __builtin_amdgcn_readlane(ff, src);
  return true;
}

__device__ __forceinline__ bool group_find(const GroupArgs& g, int b, int bp, int nq, int& expert,
                                           int& ti, int& tj, bool& alone) {
  GroupSpan s;
  if (!group_span(g, b, bp, nq, s)) return false;
  expert = s.expert;
  alone = s.rows == 1 && g.stream_w;
  const int band = s.local / (kGroupBand * nq), r = s.local - band * (kGroupBand * nq);
  const int in_band = min(kGroupBand, s.rows - band * kGroupBand);
  ti = band * kGroupBand + r % in_band;
  tj = r / in_band;
  return true;
}

// C tile element (p, q) of an MFMA block computed as Q-fragment x P-fragment:
// lane l and register r hold p = l % 32 and q = (r / 4) * 8 + (l / 32) * 4 +
// r % 4, four consecutive q per four registers.
__device__ __forceinline__ int acc_q(int r, int lhalf) { return (r >> 2) * 8 + lhalf * 4 + (r & 3); }

// Tile BP x BQ of C by WP x WQ waves, each TP x TQ MFMA blocks of 32 x 32.  A
// step is 64 * U bytes of t per row (32 U bf16, 16 U fp32), 2 U sub-steps of
// one MFMA depth, kept in STAGES LDS buffers.  KS > 1: KS such sets of waves
// share a step's sub-steps, and their sums are added at the end.
template <int BP_, int BQ_, int WP_, int WQ_, int U_, int STAGES_, int KS_ = 1, int OCC_ = 2>
struct GroupTile {
  static constexpr int BP = BP_, BQ = BQ_, WP = WP_, WQ = WQ_, U = U_, STAGES = STAGES_, KS = KS_;
  static constexpr int OCC = OCC_;   // waves per SIMD that registers must leave room for
  static constexpr int WAVES = WP * WQ * KS, THREADS = 64 * WAVES;
  static constexpr int TP = BP / WP / 32, TQ = BQ / WQ / 32;
  static constexpr int SLOTS = TP * TQ;              // MFMA blocks per wave and sub-step
  static constexpr int SUBS = 2 * U;
  static constexpr int PP = BP * U / 16 / WAVES;     // 1 KB pieces per wave and step, P panel
  static constexpr int QP = BQ * U / 16 / WAVES;     // ... Q panel
  static constexpr int STAGE_BYTES = (BP + BQ) * 64 * U;
  static_assert(PP * 16 * WAVES == BP * U && QP * 16 * WAVES == BQ * U, "whole pieces");
  static_assert(TP * 32 * WP == BP && TQ * 32 * WQ == BQ && SUBS % KS == 0, "whole blocks");
  static_assert(STAGES >= 2, "one buffer fills while another is read");
  // A buffer's refill is issued over the SUBS * SLOTS MFMA slots that follow
  // the barrier behind its last read: slots 0 .. SLOTS - 1 are the last
  // sub-step of that step, the others the next step up to its barrier.
  // slot_of(q) spreads the pieces, so that requests do not queue up in front of
  // the MFMAs; with two buffers they have to arrive by that next barrier and
  // go out in the first half.
  static constexpr int WINDOW = STAGES == 2 ? SUBS * SLOTS / 2 : SUBS * SLOTS;
  template <int N>
  static constexpr int slot_of(int q) { return q * WINDOW / N; }
  template <int N>
  static constexpr int early() {                      // pieces of the last sub-step
    int n = 0;
    for (int q = 0; q < N; ++q) n += slot_of<N>(q) < SLOTS ? 1 : 0;
    return n;
  }
};

// How a tile's operands reach LDS.
enum GroupLoad {
  kLoadDma = 0,      // 16-byte DMA: rows start on 16 bytes, widths are whole 16-byte pieces
  kLoadDmaCkpt = 1,  // the same, Q as int8 codes (k a multiple of 16, bf16)
  kLoadReg = 2,      // through registers, any alignment and width
  kLoadRegCkpt = 3   // the same, Q as int8 codes
};

// 16 bytes of bf16 or fp32 elements, 8 and 4 bytes of codes, at any element.
typedef u32x4_t u32x4_el_t __attribute__((aligned(2)));
typedef unsigned int u32x2_t __attribute__((ext_vector_type(2)));
typedef u32x2_t u32x2_b_t __attribute__((aligned(1)));
typedef uint32_t u32_b_t __attribute__((aligned(1)));

__device__ __forceinline__ uint4 load16_any(const void* p) {
  const u32x4_t v = *(const MFSDP_GLOBAL u32x4_el_t*)(p);
  return make_uint4(v.x, v.y, v.z, v.w);
}

__device__ __forceinline__ void store16_any(void* p, const uint4& v) {
  *(MFSDP_GLOBAL u32x4_el_t*)(p) = u32x4_t{v.x, v.y, v.z, v.w};
}

// Streamed store.  Outputs whose rows are whole 128-byte lines are streamed:
// the weight gradients of 256 experts (403 MB) took 134 us with plain stores
// and 107 us so, and products whose outputs fit the L2s measured the same
// either way.  Others are not: lines that two workgroups share then reach HBM
// in pieces (11 gradients of 6144 x 5608: 212 us plain, 367 us streamed).
__device__ __forceinline__ void stream16_any(void* p, const uint4& v) {
  __builtin_nontemporal_store(u32x4_t{v.x, v.y, v.z, v.w}, (MFSDP_GLOBAL u32x4_el_t*)(p));
}

// load8 and store8 at any element.
template <class E>
__device__ __forceinline__ void load8_any(const typename E::storage_t* p, float (&v)[8]) {
  Raw8 r;
  r.a = load16_any(p);
  r.b = E::kVec == 4 ? load16_any(p + 4) : make_uint4(0, 0, 0, 0);
  unpack_raw8<E>(r, v);
}

template <class E>
__device__ __forceinline__ void store8_any(typename E::storage_t* p, const float (&v)[8]) {
  if constexpr (E::kVec == 8) {
    store16_any(p, Vec16<E>::pack(v));
  } else {
    const float a[4] = {v[0], v[1], v[2], v[3]}, b[4] = {v[4], v[5], v[6], v[7]};
    store16_any(p, Vec16<E>::pack(a));
    store16_any(p + 4, Vec16<E>::pack(b));
  }
}

// One wave-wide global -> LDS copy of 64 x 16 bytes: lane l's bytes at
// base + voff land at lds + 16 * l.  The buffer's range check turns the
// offset kDmaNone into zeros, which is how rows and columns outside the
// operand are filled.  Inline assembly for the reason given at lds_dma16; no
// output register, and the kernel waits with vmcnt before the barrier that
// publishes the data.
typedef uint32_t u32x4s_t __attribute__((ext_vector_type(4)));
constexpr uint32_t kDmaNone = 0x80000000u;

__device__ __forceinline__ u32x4s_t dma_buffer(const char* base) {
  const uint64_t b = reinterpret_cast<uintptr_t>(base);
  u32x4s_t r;
  r[0] = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(b));
  r[1] = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(b >> 32)) & 0xffffu;   // stride 0
  r[2] = 0x7fffffffu;    // bytes: every valid offset is below (checked on the host)
  r[3] = 0x00020000u;    // untyped 32-bit data
  return r;
}

__device__ __forceinline__ void lds_dma16_buf(uint32_t lds, uint32_t voff, u32x4s_t buf) {
  const uint32_t ulds = static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(lds));
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
               :: "s"(ulds), "v"(voff), "s"(buf) : "memory", "m0");
}

// The same for data that no other workgroup reads (streamed).
__device__ __forceinline__ void lds_dma16_buf_nt(uint32_t lds, uint32_t voff, u32x4s_t buf) {
  const uint32_t ulds = static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(lds));
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen nt lds"
               :: "s"(ulds), "v"(voff), "s"(buf) : "memory", "m0");
}

// 16-byte chunk swizzle of a K-contiguous panel row of 64 * U bytes: the 16 rows
// that a fragment read touches at one chunk cover all 16 chunks of the 256-byte
// bank row.
template <int U>
__device__ __forceinline__ int rswz(int row) {
  return U == 1 ? (row >> 2) & 3 : U == 2 ? (row >> 1) & 7 : row & 15;
}

// 16-byte chunk swizzle of a panel read along t (row of B elements per t): the
// four rows that one transposing read touches land in four 64-byte windows of
// the 256-byte bank row.
template <int B>
__device__ __forceinline__ int tswz(int kk) {
  return B >= 128 ? 4 * (kk & 3) : 4 * ((kk >> 1) & 1);
}

// Which (expert, row tile, column tile) workgroup b of a weight gradient takes.
// Tiles of one expert go in chunks of up to 32 (a band of eight by four, which
// share panels) to the XCDs in turn: experts differ in length, and an XCD
// that held whole experts would finish long after another.  False if b is one
// of the places that the last chunks leave empty.
struct WgradOrder {
  int tp, tq, per, chunks, size;   // tiles, chunks per expert, tiles per chunk
  __host__ __device__ WgradOrder(int n, int k, int bp, int bq) {
    tp = (n + bp - 1) / bp;
    tq = (k + bq - 1) / bq;
    per = tp * tq;
    chunks = (per + 31) / 32;
    size = (per + chunks - 1) / chunks;
  }
  __host__ __device__ int64_t blocks(int64_t experts) const {
    return (experts * chunks + kXcds - 1) / kXcds * kXcds * size;
  }
};

__device__ __forceinline__ bool wgrad_find(const GroupArgs& g, int b, int bp, int bq, int& expert,
                                           int& ti, int& tj) {
  const WgradOrder o(g.n, g.k, bp, bq);
  const int x = b % kXcds, i = b / kXcds;
  const int j = i / o.size;
  const int chunk = j * kXcds + x;
  expert = chunk / o.chunks;
  const int local = (chunk - expert * o.chunks) * o.size + i - j * o.size;
  if (expert >= g.experts || local >= o.per) return false;
  const int band = local / (kGroupBand * o.tq), r = local - band * (kGroupBand * o.tq);
  const int in_band = min(kGroupBand, o.tp - band * kGroupBand);
  ti = band * kGroupBand + r % in_band;
  tj = r / in_band;
  return true;
}

// The same where segments are cut into parts of g.part_rows rows: workgroup b
// takes tile b' % tiles of part b' / tiles, parts counted over all experts, and
// b' dealt so that an XCD runs neighbours.  `part` is the part's number over
// all experts, lo and hi its rows.
__device__ __forceinline__ bool wgrad_find_part(const GroupArgs& g, int b, int bp, int bq, int& part,
                                                int& lo, int& hi, int& ti, int& tj) {
  const int tq = (g.k + bq - 1) / bq, tiles = (g.n + bp - 1) / bp * tq;
  GroupSpan s;
  if (!group_span(g, b, g.part_rows, tiles, s)) return false;
  part = s.first + s.local / tiles;
  const int tile = s.local % tiles;
  ti = tile / tq;
  tj = tile % tq;
  group_segment(g, s.expert, lo, hi);
  lo += s.local / tiles * g.part_rows;
  hi = min(hi, lo + g.part_rows);
  return true;
}

// CKPT: Q is the int8 checkpoint of X.  Its codes arrive by DMA one step ahead
// of P, 32 rows of BQ bytes per step, and while step t is multiplied every
// thread turns 16 codes of step t + 1 into bf16 (exact: seven bits of
// magnitude and a power of two) in one of two panels that the fragments are
// then read from as from X itself: each code is converted once, where a
// conversion of the fragments would do it for every wave row.  The scales of
// kCkptSteps steps at a time wait in LDS as floats, two such groups in turn.
constexpr int kCkptSteps = 16;

template <class E, int MODE, class C, int LOAD>
__global__ __launch_bounds__(C::THREADS, C::OCC) void grouped_tile_kernel(GroupArgs g) {
  constexpr bool CKPT = LOAD == kLoadDmaCkpt;
  constexpr bool kReg = LOAD == kLoadReg || LOAD == kLoadRegCkpt;
  constexpr bool kCodes = LOAD == kLoadDmaCkpt || LOAD == kLoadRegCkpt;
  static_assert(!kCodes || MODE == kGroupWgrad, "checkpoint form");
  static_assert(!CKPT || (E::kVec == 8 && C::U == 1 && C::KS == 1), "checkpoint form");
  using S = typename E::storage_t;
  constexpr int V = E::kVec;
  constexpr int BK = 4 * V * C::U;
  constexpr int ROW = 64 * C::U;               // bytes of a K-contiguous panel row
  constexpr bool kPT = MODE == kGroupWgrad;    // P, Q read along t
  constexpr bool kQT = MODE != kGroupFwd;
  constexpr int TP = C::TP, TQ = C::TQ;
  // Stages: P panel, then Q panel; with CKPT P panel, then codes, and behind
  // the stages two Q panels and two groups of scales.
  constexpr int kQCodes = C::BQ * 32;                       // bytes of one step's codes
  constexpr int kStage = CKPT ? C::BP * ROW + kQCodes : C::STAGE_BYTES;
  constexpr int kStagesEnd = C::STAGES * kStage;
  constexpr int kQPanel = C::BQ * ROW;
  constexpr int kScaleCols = C::BQ < kCkptBlock ? 1 : C::BQ / kCkptBlock;
  constexpr int kScaleGroup = kCkptSteps * 32 * kScaleCols;  // floats
  constexpr int kLds = CKPT ? kStagesEnd + 2 * kQPanel + 2 * kScaleGroup * 4 : kStagesEnd;
  constexpr int QPW = CKPT ? kQCodes / 1024 / C::WAVES : C::QP;   // DMA pieces per wave
  constexpr int PIECES = C::PP + QPW;
  static_assert(!CKPT || (QPW * 1024 * C::WAVES == kQCodes && kQCodes == 16 * C::THREADS),
                "16 codes per thread and step");
  __shared__ __align__(16) char lds[kLds];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  constexpr int kTileWaves = C::WP * C::WQ;
  const int tw = wave % kTileWaves, ks = wave / kTileWaves;   // wave of the tile, set of waves
  const int wp = tw / C::WQ, wq = tw % C::WQ;
  const int lrow = lane & 31, lhalf = lane >> 5;

  // ---- tile and operands ----------------------------------------------------
  int e, ti, tj, lo, hi;
  const size_t wsize = static_cast<size_t>(g.n) * g.k;
  const bool split = MODE == kGroupWgrad && g.part_rows > 0;
  // An expert with one row tile of few rows: its weights are read by this column
  // of tiles alone, and streamed if they would not stay in the L2s (eight 14336 x 4096 experts, 16 rows: 145 ->
  // 131 us; not where a panel row is less than two lines, as in the input
  // gradient: one expert there 36 -> 59 us).
  constexpr bool kAlone = MODE == kGroupFwd && C::KS > 1;
  bool alone = false;
  if (split) {
    if (!wgrad_find_part(g, blockIdx.x, C::BP, C::BQ, e, lo, hi, ti, tj)) return;   // e: the part
  } else {
    if (MODE == kGroupWgrad) {
      if (!wgrad_find(g, blockIdx.x, C::BP, C::BQ, e, ti, tj)) return;
    } else {
      const int nq = ((MODE == kGroupFwd ? g.n : g.k) + C::BQ - 1) / C::BQ;
      if (!group_find(g, blockIdx.x, C::BP, nq, e, ti, tj, alone)) return;
    }
    group_segment(g, e, lo, hi);
  }
  const int p0 = ti * C::BP, q0 = tj * C::BQ;
  const S* P = static_cast<const S*>(g.p) + lo * g.ldp;
  const S* Q = static_cast<const S*>(g.q);
  int64_t ldq;
  int np, nq, R;
  if (MODE == kGroupWgrad) {
    if (!kCodes) Q += lo * g.ldq;
    ldq = g.ldq;
    np = g.n; nq = g.k; R = hi - lo;
  } else {
    Q += e * wsize;
    ldq = g.k;
    np = hi - lo;
    nq = MODE == kGroupFwd ? g.n : g.k;
    R = MODE == kGroupFwd ? g.k : g.n;
  }
  P += kPT ? p0 : p0 * g.ldp;
  Q += kQT ? q0 : q0 * ldq;
  const int prem = np - p0, qrem = nq - q0;    // rows / columns of the tile that exist

  // ---- DMA: this wave's pieces of a step -------------------------------------
  // K-contiguous panel: 16 / U rows x 64 U bytes per piece, chunk c of row r at
  // r * 64 U + (c ^ rswz(r)) * 16.  Panel read along t: BK rows of B elements,
  // chunk c of row kk at kk * B * size + (c ^ tswz(kk)) * 16.  voff is the
  // lane's byte offset from the step's base, klim the first t (from the step's
  // own) that the chunk holds: at or past the end of t it loads zeros, as do
  // chunks outside the tile's rows and columns.
  // kLoadReg: the columns of a chunk that exist are counted too (cnt), and a
  // chunk that reaches past the row loads them one by one.
  uint32_t voff[PIECES];
  int klim[PIECES], cnt[PIECES];
  auto setup = [&](int q, int piece, bool along, int64_t ld, int rem, int width) {
    if (!along) {
      const int row = piece * (16 / C::U) + lane / (4 * C::U), c = (lane & (4 * C::U - 1)) ^ rswz<C::U>(row);
      voff[q] = static_cast<uint32_t>((row * ld + c * V) * static_cast<int64_t>(sizeof(S)));
      klim[q] = row < rem ? c * V : 0x7fffffff;
      cnt[q] = V;
    } else {
      const int pitch = width * static_cast<int>(sizeof(S));
      const int at = piece * 1024 + lane * 16;
      const int kk = at / pitch, pc = at % pitch / 16;
      const int c = V == 8 ? pc ^ (width >= 128 ? 4 * (kk & 3) : 4 * ((kk >> 1) & 1)) : pc;
      voff[q] = static_cast<uint32_t>((kk * ld + c * V) * static_cast<int64_t>(sizeof(S)));
      klim[q] = c * V < rem ? kk : 0x7fffffff;
      cnt[q] = min(V, rem - c * V);
      if (LOAD == kLoadRegCkpt && q >= C::PP) voff[q] = static_cast<uint32_t>(kk * ld + c * V);
    }
  };
#pragma unroll
  for (int q = 0; q < C::PP; ++q) setup(q, wave * C::PP + q, kPT, g.ldp, prem, C::BP);
#pragma unroll
  for (int q = 0; q < QPW; ++q) {
    if constexpr (CKPT) {   // codes: rows of BQ bytes, 16 columns per lane
      const int at = (wave * QPW + q) * 1024 + lane * 16;
      const int kk = at / C::BQ, col = at % C::BQ;
      voff[C::PP + q] = static_cast<uint32_t>(kk * ldq + col);
      klim[C::PP + q] = col < qrem ? kk : 0x7fffffff;
    } else {
      setup(C::PP + q, wave * QPW + q, kQT, ldq, qrem, C::BQ);
    }
  }
  const char* pbase = reinterpret_cast<const char*>(P);
  const char* qbase = kCodes ? static_cast<const char*>(g.q) + lo * g.ldq + q0
                           : reinterpret_cast<const char*>(Q);
  const int64_t pstep = (kPT ? g.ldp : 1) * static_cast<int64_t>(BK * sizeof(S));
  const int64_t qstep = (kQT ? ldq : 1) * static_cast<int64_t>(BK * (kCodes ? 1 : sizeof(S)));
  const uint32_t lds0 = lds_addr(lds);
  // Next step to fetch: pbase / qbase point at it, `left` values of t remain
  // from it on.  With CKPT qbase and qleft are one step further on.
  int left = R, qleft = R;
  auto dma_piece = [&](uint32_t stage, int q) {
    const bool is_p = q < C::PP;
    uint32_t at = lds0 + stage;
    if (CKPT && !is_p) at = lds0 + (stage + kStage == kStagesEnd ? 0 : stage + kStage);
    at += is_p ? (wave * C::PP + q) * 1024 : C::BP * ROW + (wave * QPW + q - C::PP) * 1024;
    const uint32_t off = klim[q] < (is_p ? left : qleft) ? voff[q] : kDmaNone;
    if (kAlone && !is_p && alone)
      lds_dma16_buf_nt(at, off, dma_buffer(qbase));
    else
      lds_dma16_buf(at, off, dma_buffer(is_p ? pbase : qbase));
  };
  auto dma_next = [&] {
    pbase += pstep;
    qbase += qstep;
    left -= BK;
    qleft -= BK;
  };

  // kLoadReg: this thread's chunks of the next step, in registers (codes are
  // converted on the way).
  uint4 stash[kReg ? PIECES : 1];
  auto reg_load = [&] {
#pragma unroll
    for (int q = 0; q < PIECES; ++q) {
      const bool is_p = q < C::PP;
      const bool along = is_p ? kPT : kQT;
      const int n = klim[q] >= left ? 0 : along ? cnt[q] : min(left - klim[q], V);
      const char* src = (is_p ? pbase : qbase) + voff[q];
      uint4 v = make_uint4(0, 0, 0, 0);
      if (LOAD == kLoadRegCkpt && !is_p) {
        uint32_t w[2] = {0, 0};
        float s = 0.f;
        if (n > 0) {
          const int nb = (g.k + kCkptBlock - 1) / kCkptBlock;
          const int row = R - left + klim[q], col = q0 + static_cast<int>(voff[q] - klim[q] * ldq);
          s = ckpt_scale(gld<uint8_t>(g.qs + static_cast<size_t>(lo + row) * nb + col / kCkptBlock));
        }
        if (n == V && V == 8) {
          const u32x2_t t = *(const MFSDP_GLOBAL u32x2_b_t*)(src);
          w[0] = t.x;
          w[1] = t.y;
        } else if (n == V) {
          w[0] = *(const MFSDP_GLOBAL u32_b_t*)(src);
        } else {
          for (int i = 0; i < n; ++i)
            w[i >> 2] |= static_cast<uint32_t>(gld<uint8_t>(src + i)) << (8 * (i & 3));
        }
        float f[V];
#pragma unroll
        for (int i = 0; i < V; ++i)
          f[i] = static_cast<float>(static_cast<int8_t>(w[i >> 2] >> (8 * (i & 3)))) * (i < n ? s : 0.f);
        v = Vec16<E>::pack(f);
      } else if (n == V) {
        v = load16_any(src);
      } else if (n > 0) {
        S x[V];
#pragma unroll
        for (int i = 0; i < V; ++i) x[i] = i < n ? gld<S>(src + i * sizeof(S)) : S(0);
        __builtin_memcpy(&v, x, 16);
      }
      stash[q] = v;
    }
  };
  auto reg_store = [&](uint32_t stage) {
#pragma unroll
    for (int q = 0; q < PIECES; ++q) {
      const int piece = q < C::PP ? wave * C::PP + q : wave * QPW + q - C::PP;
      *reinterpret_cast<uint4*>(lds + stage + (q < C::PP ? 0 : C::BP * ROW) + piece * 1024 + lane * 16) = stash[q];
    }
  };

  // ---- fragments ---------------------------------------------------------------
  // Lane l holds, for sub-step s, the 16-byte slice 2s + l/32 of t of row l%32
  // of each 32-row block.
  constexpr int kPR = kPT && V == 8 ? 2 : 1, kQR = kQT && V == 8 ? 2 : 1;   // reads per fragment
  constexpr int kReads = TP * kPR + TQ * kQR;
  auto frag = [&](const char* panel, auto along_c, auto width_c, int s, int base, int half, uint4& f) {
    constexpr bool along = decltype(along_c)::value;
    constexpr int width = decltype(width_c)::value;
    if constexpr (!along) {
      const int row = base + lrow, c = 2 * s + lhalf;
      f = *reinterpret_cast<const uint4*>(panel + row * ROW + ((c ^ rswz<C::U>(row)) << 4));
    } else if constexpr (V == 8) {
      // transposing read: in each group of 16 lanes, lane i points at row
      // kk + i/4, columns n + 4 (i%4) .. + 4, and receives column i at rows
      // kk .. kk + 3
      const int il = lane & 15;
      const int n = base + 16 * ((lane >> 4) & 1) + 4 * (il & 3);
      const int kk = 16 * s + 8 * lhalf + 4 * half + (il >> 2);
      const int byte = kk * (width * 2) + (((n >> 3) ^ tswz<width>(kk)) << 4) + ((n & 7) << 1);
      const v4i16_t t = __builtin_amdgcn_ds_read_tr16_b64_v4i16((MFSDP_LDS v4i16_t*)(panel + byte));
      const uint2 w = __builtin_bit_cast(uint2, t);
      if (half == 0) {
        f.x = w.x;
        f.y = w.y;
      } else {
        f.z = w.x;
        f.w = w.y;
      }
    } else {
      const float* pf = reinterpret_cast<const float*>(panel);
      const int kk = 4 * (2 * s + lhalf), n = base + lrow;
      f = make_uint4(__float_as_uint(pf[(kk + 0) * width + n]), __float_as_uint(pf[(kk + 1) * width + n]),
                     __float_as_uint(pf[(kk + 2) * width + n]), __float_as_uint(pf[(kk + 3) * width + n]));
    }
  };
  uint4 fp[2][TP], fq[2][TQ];
  using PT_c = std::integral_constant<bool, kPT>;
  using QT_c = std::integral_constant<bool, kQT>;
  using PW_c = std::integral_constant<int, C::BP>;
  using QW_c = std::integral_constant<int, C::BQ>;
  auto read_piece = [&](uint32_t stage, uint32_t qpanel, int s, int r, uint4 (&a)[TP], uint4 (&b)[TQ]) {
    const char* base = lds + stage;
    if (r < TP * kPR) {
      frag(base, PT_c{}, PW_c{}, s, (wp * TP + r / kPR) * 32, r % kPR, a[r / kPR]);
    } else {
      const int j = r - TP * kPR;
      frag(CKPT ? lds + kStagesEnd + qpanel : base + C::BP * ROW, QT_c{}, QW_c{}, s, (wq * TQ + j / kQR) * 32, j % kQR, b[j / kQR]);
    }
  };

  f32x16_t acc[TP][TQ];
#pragma unroll
  for (int i = 0; i < TP; ++i)
#pragma unroll
    for (int j = 0; j < TQ; ++j) acc[i][j] = f32x16_t{};

  // fp32: the blocks' sums are moved to a second set every kFlush steps, so that
  // a long sum is a sum of sums of 512 values and its rounding does not grow
  // with its whole length.  A set of waves adds BK / KS values of each step.
  constexpr int kFlush = 512 * C::KS / BK;
  static_assert(kFlush * BK == 512 * C::KS, "whole steps");
  constexpr bool kTwoSums = V == 4;
  f32x16_t acc2[kTwoSums ? TP : 1][kTwoSums ? TQ : 1];
  if constexpr (kTwoSums) {
#pragma unroll
    for (int i = 0; i < TP; ++i)
#pragma unroll
      for (int j = 0; j < TQ; ++j) acc2[i][j] = f32x16_t{};
  }
  auto flush = [&](int t) {
    if constexpr (kTwoSums) {
      if (__builtin_expect(t % kFlush != kFlush - 1, 1)) return;
      // Keeps this a branch: as selects in every step, behind a wait for the
      // MFMAs, it cost 13-20% (16 x 1024 x 2048 x 2048 fp32: 106 -> 129 us).
      asm volatile("");
#pragma unroll
      for (int i = 0; i < TP; ++i)
#pragma unroll
        for (int j = 0; j < TQ; ++j) {
          acc2[i][j] += acc[i][j];
          acc[i][j] = f32x16_t{};
        }
    }
  };

  // ---- main loop ------------------------------------------------------------------
  // Step t computes on stage t % STAGES.  Each sub-step reads the fragments of
  // the next one; before the last, whose fragments have then been read, the
  // waves wait until step t + 1 has landed (only later steps' pieces may be in
  // flight) and until their own reads are done (lgkmcnt), and meet a barrier:
  // behind it the last sub-step reads step t + 1's first fragments, and the
  // stage of step t is free for the DMA of step t + STAGES.  Steps past the end
  // load zeros and are never multiplied.
  const int nk = (R + BK - 1) / BK;

  // CKPT: this thread's 16 codes of a step are row crow, columns ccol..; the
  // scales of group j (steps kCkptSteps * j on) go to half j & 1.
  const int crow = tid * 16 / C::BQ, ccol = tid * 16 % C::BQ;
  float* const scale_lds = reinterpret_cast<float*>(lds + kStagesEnd + 2 * kQPanel);
  constexpr int kScaleLd = CKPT ? kScaleGroup / C::THREADS : 1;
  float sc[kScaleLd];
  auto scales_load = [&](int j) {
    const int nb = (g.k + kCkptBlock - 1) / kCkptBlock;
#pragma unroll
    for (int i = 0; i < kScaleLd; ++i) {
      const int u = tid + i * C::THREADS;
      const int row = j * (kCkptSteps * 32) + u / kScaleCols, blk = q0 / kCkptBlock + u % kScaleCols;
      sc[i] = row < R && blk < nb
                  ? ckpt_scale(gld<uint8_t>(g.qs + static_cast<size_t>(lo + row) * nb + blk)) : 0.f;
    }
  };
  auto scales_store = [&](int j) {
#pragma unroll
    for (int i = 0; i < kScaleLd; ++i) scale_lds[(j & 1) * kScaleGroup + tid + i * C::THREADS] = sc[i];
  };
  // Step t's codes, kept in `stage`, in five pieces: the reads, then four codes
  // each, spread over the MFMA slots of a sub-step.
  uint4 codes;
  float scale;
  uint32_t half[4];
  auto convert = [&](uint32_t stage, int t, int piece) {
    if (piece == 0) {
      codes = *reinterpret_cast<const uint4*>(lds + stage + C::BP * ROW + tid * 16);
      scale = scale_lds[((t / kCkptSteps) & 1) * kScaleGroup +
                        (t % kCkptSteps * 32 + crow) * kScaleCols + ccol / kCkptBlock];
      return;
    }
    const uint32_t w = piece == 1 ? codes.x : piece == 2 ? codes.y : piece == 3 ? codes.z : codes.w;
    float v[4];
#pragma unroll
    for (int b = 0; b < 4; ++b) v[b] = static_cast<float>(static_cast<int8_t>(w >> (8 * b))) * scale;
    const int at = (piece - 1) & 1 ? 2 : 0;
    half[at] = pack_bf16x2(v[0], v[1]);
    half[at + 1] = pack_bf16x2(v[2], v[3]);
    if (at) {
      char* panel = lds + kStagesEnd + (t & 1) * kQPanel + crow * (C::BQ * 2);
      *reinterpret_cast<uint4*>(panel + (((ccol / 8 + (piece >> 2)) ^ tswz<C::BQ>(crow)) << 4)) =
          make_uint4(half[0], half[1], half[2], half[3]);
    }
  };
  // slot of a sub-step in which a piece goes
  auto convert_slot = [](int piece) { return piece == 0 ? 0 : 1 + piece * (C::SLOTS - 1) / 5; };

  if constexpr (kReg || C::KS > 1) {
    // One barrier per step: behind it every wave has read the step before, whose
    // buffer the loads refill, and this step is there.
    constexpr int kSubs = C::SUBS / C::KS;      // of this set of waves
    auto multiply = [&](uint32_t stage) {
#pragma unroll
      for (int i = 0; i < kSubs; ++i) {
#pragma unroll
        for (int r = 0; r < kReads; ++r) read_piece(stage, 0, ks * kSubs + i, r, fp[i & 1], fq[i & 1]);
#pragma unroll
        for (int x = 0; x < C::SLOTS; ++x)
          Mma<E>::run(acc[x / TQ][x % TQ], fq[i & 1][x % TQ], fp[i & 1][x / TQ]);
      }
    };
    if constexpr (kReg) {
      static_assert(C::STAGES == 2, "two buffers behind the registers");
      if (nk > 0) {
        reg_load();
        reg_store(0);
        dma_next();
      }
      uint32_t cur = 0;
#pragma unroll 1
      for (int t = 0; t < nk; ++t) {
        if (t + 1 < nk) reg_load();
        __syncthreads();
        multiply(cur);
        flush(t);
        cur ^= kStage;
        if (t + 1 < nk) reg_store(cur);
        dma_next();
      }
    } else if (nk > 0) {
#pragma unroll
      for (int s = 0; s < C::STAGES - 1; ++s) {
#pragma unroll
        for (int q = 0; q < PIECES; ++q) dma_piece(s * kStage, q);
        dma_next();
      }
      uint32_t cur = 0, fill = kStagesEnd - kStage;
#pragma unroll 1
      for (int t = 0; t < nk; ++t) {
        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier"
                     :: "n"((C::STAGES - 2) * PIECES) : "memory");
#pragma unroll
        for (int q = 0; q < PIECES; ++q) dma_piece(fill, q);
        dma_next();
        multiply(cur);
        flush(t);
        fill = cur;
        cur = cur + kStage == kStagesEnd ? 0 : cur + kStage;
      }
    }
  } else if (nk > 0) {
    if constexpr (CKPT) {   // codes of step 0, then one step ahead of P
      scales_load(0);
      scales_store(0);
#pragma unroll
      for (int q = C::PP; q < PIECES; ++q) dma_piece(kStagesEnd - kStage, q);
      qbase += qstep;
      qleft -= BK;
    }
#pragma unroll
    for (int s = 0; s < C::STAGES - 1; ++s) {
#pragma unroll
      for (int q = 0; q < PIECES; ++q) dma_piece(s * kStage, q);
      dma_next();
    }
    uint32_t cur = 0, fill = kStagesEnd - kStage;
    constexpr int kEarly = C::template early<PIECES>();
    static_assert(!CKPT || kEarly <= C::PP, "the codes behind step 0's may only follow their conversion");
#pragma unroll
    for (int q = 0; q < kEarly; ++q) dma_piece(fill, q);
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier"
                 :: "n"((C::STAGES - 2) * PIECES + kEarly) : "memory");
    if constexpr (CKPT) {
#pragma unroll
      for (int i = 0; i < 5; ++i) convert(0, 0, i);
      asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    }
    // A wave whose rows or columns the tile does not have only moves data: its
    // share of the SIMD is the other waves' (16 x 24576 x 5632 x 2048 forward:
    // 547 -> 536 us).  Not in weight gradients, whose tiles are seldom cut: 110
    // -> 114 us on 256 x 32771 x 512 x 1536.
    const bool idle = MODE != kGroupWgrad && (wp * TP * 32 >= prem || wq * TQ * 32 >= qrem);
    if (idle) {
#pragma unroll 1
      for (int t = 0; t < nk; ++t) {
#pragma unroll
        for (int q = kEarly; q < PIECES; ++q) dma_piece(fill, q);
        dma_next();
        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier"
                     :: "n"((C::STAGES - 2) * PIECES) : "memory");
#pragma unroll
        for (int q = 0; q < kEarly; ++q) dma_piece(cur, q);
        fill = cur;
        cur = cur + kStage == kStagesEnd ? 0 : cur + kStage;
      }
    }
    const int steps = idle ? 0 : nk;
    uint32_t qcur = 0;
#pragma unroll
    for (int r = 0; r < kReads; ++r) read_piece(0, 0, 0, r, fp[0], fq[0]);
#pragma unroll 1
    for (int t = 0; t < steps; ++t) {
      const uint32_t nxt = cur + kStage == kStagesEnd ? 0 : cur + kStage;
      if constexpr (CKPT) {
        // the next group's scales: loaded at the start of a group, stored half
        // way, read from the last conversion of the group on
        if (t % kCkptSteps == 0) scales_load(t / kCkptSteps + 1);
        if (t % kCkptSteps == kCkptSteps / 2) scales_store(t / kCkptSteps + 1);
      }
#pragma unroll
      for (int sub = 0; sub < C::SUBS; ++sub) {
        constexpr int kLast = C::SUBS - 1;
#pragma unroll
        for (int x = 0; x < C::SLOTS; ++x) {
          Mma<E>::run(acc[x / TQ][x % TQ], fq[sub & 1][x % TQ], fp[sub & 1][x / TQ]);
#pragma unroll
          for (int r = x; r < kReads; r += C::SLOTS) {
            if (sub < kLast) read_piece(cur, qcur, sub + 1, r, fp[(sub + 1) & 1], fq[(sub + 1) & 1]);
            else read_piece(nxt, qcur ^ kQPanel, 0, r, fp[0], fq[0]);
          }
#pragma unroll
          for (int q = 0; q < PIECES; ++q)
            if (C::template slot_of<PIECES>(q) == (sub == kLast ? x : (sub + 1) * C::SLOTS + x))
              dma_piece(sub == kLast ? cur : fill, q);
          if constexpr (CKPT) {
#pragma unroll
            for (int i = 0; i < 5; ++i)
              if (sub == 0 && x == convert_slot(i)) convert(nxt, t + 1, i);
          }
          __builtin_amdgcn_sched_barrier(0);
        }
        if (sub == kLast - 1) {
          dma_next();
          asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier"
                       :: "n"((C::STAGES - 2) * PIECES) : "memory");
        }
      }
      flush(t);
      fill = cur;
      cur = nxt;
      qcur ^= kQPanel;
    }
  }
  // every DMA has landed and every fragment is read before the stages are reused
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");

  if constexpr (kTwoSums) {
#pragma unroll
    for (int i = 0; i < TP; ++i)
#pragma unroll
      for (int j = 0; j < TQ; ++j) acc[i][j] += acc2[i][j];
  }
  if constexpr (C::KS > 1) {   // the other sets' sums, in their order
    constexpr int kBlock = 64 * 16;   // floats of one MFMA block
    float* sums = reinterpret_cast<float*>(lds);
    static_assert((C::KS - 1) * kTileWaves * C::SLOTS * kBlock * 4 <= kLds, "sums fit");
    auto at = [&](int set, int x, int r) {
      return ((set * kTileWaves + tw) * C::SLOTS + x) * kBlock + r * 64 + lane;
    };
    if (ks > 0) {
#pragma unroll
      for (int x = 0; x < C::SLOTS; ++x)
#pragma unroll
        for (int r = 0; r < 16; ++r) sums[at(ks - 1, x, r)] = acc[x / TQ][x % TQ][r];
    }
    __syncthreads();
    if (ks > 0) return;
#pragma unroll
    for (int s = 0; s < C::KS - 1; ++s)
#pragma unroll
      for (int x = 0; x < C::SLOTS; ++x)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[x / TQ][x % TQ][r] += sums[at(s, x, r)];
    // this wave's staging below may overlap sums that another wave still reads
    static_assert((C::KS - 1) * kTileWaves * C::SLOTS * kBlock * 4 <= kLds / 2,
                  "staging behind the sums");
  }

  // ---- epilogue -------------------------------------------------------------------
  // 32 rows of each row of waves at a time go through LDS (lane l holds row
  // l % 32 and four consecutive columns per four registers), and every wave
  // then stores some of those rows over the tile's whole width: a store covers
  // 512 bytes of a row or more where the tile is 256 wide, so that lines are
  // written whole wherever the rows start.
  constexpr int COLS = TQ * 32;
  const float beta = split ? 0.f : g.beta;
  const bool out_f32 = V == 4 || (MODE == kGroupWgrad && (split || g.out_f32));
  const bool f32 = out_f32 || (MODE == kGroupWgrad && beta != 0.f);
  const int prow0 = wp * TP * 32;
  char* out;
  int64_t ldo;
  if (MODE == kGroupWgrad) {
    ldo = g.k;
    out = split ? reinterpret_cast<char*>(g.part) : static_cast<char*>(g.out);
    out += (e * wsize + p0 * ldo + q0) * (out_f32 ? 4 : 2);
  } else {
    ldo = g.ldo;
    out = static_cast<char*>(g.out) + ((lo + p0) * ldo + q0) * static_cast<int64_t>(sizeof(S));
  }
  // stream_c: whether stores are streamed.  Two copies of the loops, chosen once:
  // the compiler would merge two stores that differ in that alone.
  auto write = [&](auto stream_c, auto f32_c) {
    constexpr bool kStream = decltype(stream_c)::value, kF32 = decltype(f32_c)::value;
    constexpr int ES = kF32 ? 4 : 2;                 // bytes of a staged value
    constexpr int GROUPS = C::BQ * ES / 16;          // 16-byte pieces per row
    constexpr int RPP = 64 / GROUPS;                 // rows per pass of a wave
    constexpr int PITCH = C::BQ * ES + 16;
    constexpr int BLOCK = C::WP * 32 * PITCH;
    constexpr int kSpace = C::KS > 1 ? kLds / 2 : kLds;
    constexpr int BUFS = C::TP > 1 && 2 * BLOCK <= kSpace ? 2 : 1;
    static_assert(BLOCK <= kSpace && RPP >= 1 && 32 / C::WQ % RPP == 0, "staging fits");
    char* stage = lds + (kLds - kSpace) + wp * (32 * PITCH);
#pragma unroll
    for (int i = 0; i < TP; ++i) {
      char* mine = stage + (BUFS == 2 ? (i & 1) * BLOCK : 0);
      if (BUFS == 1 && i > 0) __syncthreads();       // the rows before have been read
#pragma unroll
      for (int j = 0; j < TQ; ++j)
#pragma unroll
        for (int r = 0; r < 16; r += 4) {
          char* at = mine + lrow * PITCH + (wq * COLS + j * 32 + acc_q(r, lhalf)) * ES;
          if constexpr (kF32)
            *reinterpret_cast<float4*>(at) = make_float4(acc[i][j][r], acc[i][j][r + 1], acc[i][j][r + 2], acc[i][j][r + 3]);
          else
            *reinterpret_cast<uint2*>(at) =
                make_uint2(pack_bf16x2(acc[i][j][r], acc[i][j][r + 1]), pack_bf16x2(acc[i][j][r + 2], acc[i][j][r + 3]));
        }
      __syncthreads();
#pragma unroll
      for (int r0 = 0; r0 < 32 / C::WQ; r0 += RPP) {
        const int row = wq * (32 / C::WQ) + r0 + lane / GROUPS, q = lane % GROUPS * (16 / ES);
        const uint4 raw = *reinterpret_cast<const uint4*>(mine + row * PITCH + q * ES);
        const int p = prow0 + i * 32 + row;
        if (p >= prem || q >= qrem) continue;
        if constexpr (!kF32) {
          uint16_t* o = reinterpret_cast<uint16_t*>(out) + p * ldo + q;
          if (q + 8 <= qrem) {
            if constexpr (kStream) stream16_any(o, raw);
            else store16_any(o, raw);
          } else {
            const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
            for (int k = 0; k < 8; ++k)
              if (q + k < qrem) o[k] = static_cast<uint16_t>(w[k >> 1] >> (16 * (k & 1)));
          }
        } else {
          float v[4];
          Vec16<ElemF32>::unpack(raw, v);
          if (out_f32) {
            float* o = reinterpret_cast<float*>(out) + p * ldo + q;
            if (q + 4 <= qrem) {
              if (MODE == kGroupWgrad && beta != 0.f) {
                float old[4];
                Vec16<ElemF32>::unpack(load16_any(o), old);
#pragma unroll
                for (int k = 0; k < 4; ++k) v[k] = fmaf(beta, old[k], v[k]);
              }
              if constexpr (kStream) stream16_any(o, Vec16<ElemF32>::pack(v));
              else store16_any(o, Vec16<ElemF32>::pack(v));
            } else {
#pragma unroll
              for (int k = 0; k < 4; ++k)
                if (q + k < qrem) o[k] = MODE == kGroupWgrad && beta != 0.f ? fmaf(beta, o[k], v[k]) : v[k];
            }
          } else {   // beta * dW + sum in bf16
            uint16_t* o = reinterpret_cast<uint16_t*>(out) + p * ldo + q;
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (q + k < qrem) o[k] = f32_to_bf16_rne(fmaf(beta, bf16_to_f32(o[k]), v[k]));
          }
        }
      }
    }
  };
  using yes = std::integral_constant<bool, true>;
  using no = std::integral_constant<bool, false>;
  const bool stream = g.stream && !split;
  if constexpr (V == 8) {
    if (!f32) {
      if (stream) write(yes{}, no{});
      else write(no{}, no{});
      return;
    }
  }
  if constexpr (V == 4 || MODE == kGroupWgrad) {
    if (stream) write(yes{}, yes{});
    else write(no{}, yes{});
  }
}

// Sum of the parts of each expert's weight gradient, in their order:
// dW = beta dW + sum_s part[s].  One workgroup takes 2048 elements of one
// expert.
template <class EO>
__global__ __launch_bounds__(256) void grouped_sum_kernel(GroupArgs g, int per_expert) {
  using O = typename EO::storage_t;
  const int e = blockIdx.x / per_expert;
  const size_t wsize = static_cast<size_t>(g.n) * g.k;
  // parts of the experts before this one: each wave adds them up for itself
  int64_t first = 0;
  for (int i = threadIdx.x & 63; i < e; i += 64) {
    int lo, hi;
    group_segment(g, i, lo, hi);
    first += (hi - lo + g.part_rows - 1) / g.part_rows;
  }
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) first += __shfl_xor(first, d, 64);
  first = min(first, static_cast<int64_t>(g.parts_max));
  int lo, hi;
  group_segment(g, e, lo, hi);
  const int parts = min((hi - lo + g.part_rows - 1) / g.part_rows, g.parts_max - static_cast<int>(first));
  const size_t i = static_cast<size_t>(blockIdx.x % per_expert) * 2048 + threadIdx.x * 8;
  if (i >= wsize) return;
  O* out = static_cast<O*>(g.out) + e * wsize + i;
  const float* part = g.part + first * wsize + i;
  float v[8] = {};
  if (i + 8 <= wsize) {
#pragma unroll 4
    for (int s = 0; s < parts; ++s) {
      float p[8];
      load8_any<ElemF32>(part + s * wsize, p);
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] += p[k];
    }
    if (g.beta != 0.f) {
      float old[8];
      load8_any<EO>(out, old);
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = fmaf(g.beta, old[k], v[k]);
    }
    store8_any<EO>(out, v);
  } else {
    for (int k = 0; k < 8 && i + k < wsize; ++k) {
      float x = 0.f;
      for (int s = 0; s < parts; ++s) x += part[s * wsize + k];
      out[k] = EO::from_f32(g.beta != 0.f ? fmaf(g.beta, EO::to_f32(out[k]), x) : x);
    }
  }
}

}  // namespace mfsdp
