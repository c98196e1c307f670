// Host side of the operators that make the gradients of the owner-local step:
// products grouped by expert, 8-bit activation checkpoints and the embedding
// with its gradient.  Included once, by mfsdp.hip, after its helpers (fail,
// launch, check_aliasing); every launch takes its sizes from the arguments
// alone and its offsets and tokens from device memory, so all of these calls
// can be captured into a graph.
#pragma once

namespace {

// A buffer of rows: `width` bytes each, `pitch` bytes apart.
struct Extent {
  uintptr_t lo, hi;
  size_t pitch, width;
  const char* what;
};

void add_rows(std::vector<Extent>* list, const void* p, int64_t rows, int64_t cols, int64_t ld,
              size_t es, const char* what) {
  if (rows < 1 || cols < 1) return;
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  const size_t pitch = static_cast<size_t>(ld) * es, width = static_cast<size_t>(cols) * es;
  list->push_back({lo, lo + (rows - 1) * pitch + width, pitch, width, what});
}

void add_bytes(std::vector<Extent>* list, const void* p, size_t nb, const char* what) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  if (nb) list->push_back({lo, lo + nb, nb, nb, what});
}

bool overlap(const Extent& a, const Extent& b) {
  if (a.hi <= b.lo || b.hi <= a.lo) return false;
  if (a.pitch != b.pitch) return true;
  // columns of one wider buffer: apart if each row's part is
  const size_t d = a.lo < b.lo ? (b.lo - a.lo) % a.pitch : (a.pitch - (a.lo - b.lo) % a.pitch) % a.pitch;
  return !(d >= a.width && d + b.width <= a.pitch);
}

// The outputs must be disjoint from the inputs and from each other; inputs may
// overlap one another.
mfsdp_status_t check_outputs(const std::vector<Extent>& outs, const std::vector<Extent>& ins) {
  for (size_t i = 0; i < outs.size(); ++i) {
    for (size_t j = i + 1; j < outs.size(); ++j)
      if (overlap(outs[i], outs[j]))
        return fail(MFSDP_ERR_ALIAS, "%s overlaps %s", outs[i].what, outs[j].what);
    for (const Extent& in : ins)
      if (overlap(outs[i], in))
        return fail(MFSDP_ERR_ALIAS, "%s overlaps %s", outs[i].what, in.what);
  }
  return MFSDP_OK;
}

// ---------------------------------------------------------------------------
// Products grouped by expert
// ---------------------------------------------------------------------------
// n, k and strides: 128 rows of fp32 lie within the kernels' 32-bit byte offsets
constexpr int64_t kGroupDimMax = int64_t(1) << 22;
constexpr int64_t kGroupRowsMax = int64_t(1) << 30;
constexpr int64_t kGroupExpertsMax = int64_t(1) << 20;

// Upper bound of the row tiles of height bp: every expert with rows adds at
// most one that is not full.
int64_t group_tiles_max(int64_t rows, int64_t experts, int64_t bp) {
  return (rows + std::min(rows, experts) * (bp - 1)) / bp;
}

// Workgroups of a launch: a grid has fewer than 2^32 threads along x.
constexpr int64_t kGroupBlocksMax = (int64_t(1) << 23) - 1;   // of 512 threads
constexpr int64_t kBlocksMax = (int64_t(1) << 24) - 1;        // of 256

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Workgroups of one launch with tiles of bp x bq.
int64_t group_blocks(const GroupArgs& g, int mode, int bp, int bq) {
  if (mode == kGroupWgrad && g.part_rows > 0)
    return group_tiles_max(g.rows, g.experts, g.part_rows) * ceil_div(g.n, bp) * ceil_div(g.k, bq);
  if (mode == kGroupWgrad) return WgradOrder(g.n, g.k, bp, bq).blocks(g.experts);
  return group_tiles_max(g.rows, g.experts, bp) * ceil_div(mode == kGroupFwd ? g.n : g.k, bq);
}

template <class E, int MODE, class C, int LOAD>
hipError_t launch_tile(const GroupArgs& g, hipStream_t stream) {
  const dim3 grid(static_cast<unsigned>(group_blocks(g, MODE, C::BP, C::BQ)));
  return launch(MFSDP_KERNEL_GROUPED, stream, [&] {
    grouped_tile_kernel<E, MODE, C, LOAD><<<grid, dim3(C::THREADS), 0, stream>>>(g);
  });
}

// Tiles.  Measured in us, bf16 unless said, experts x rows x n x k:
using TileWgrad = GroupTile<256, 256, 2, 4, 1, 4>;        // both panels read along t
using TileWgradSquare = GroupTile<128, 128, 2, 2, 1, 4>;  // two workgroups per CU
using TileLarge = GroupTile<256, 256, 2, 4, 2, 2>;        // whole 128-byte lines of t per row
using TileWide = GroupTile<128, 256, 2, 4, 2, 3>;
using TilePair = GroupTile<128, 256, 2, 2, 1, 3>;         // two workgroups per CU
using TileSquare = GroupTile<128, 128, 2, 2, 2, 2>;       // two workgroups per CU, through registers
using TileSmall = GroupTile<64, 256, 1, 4, 1, 4>;         // two workgroups per CU
using TileRows = GroupTile<32, 64, 1, 2, 4, 3, 4>;        // two workgroups per CU
using TileFew = GroupTile<32, 32, 1, 1, 8, 3, 8>;
using TileRowsReg = GroupTile<32, 64, 1, 2, 4, 2, 4>;
using TileF32 = GroupTile<128, 128, 2, 2, 1, 4>;

// Weight gradients: 256 x 256 tiles where n and k fill more than half of one and
// there are enough for the 256 CUs, or where long segments can be cut into
// enough parts; 128 x 128 tiles otherwise, two workgroups per CU.  Both sides:
// 256 x 32771 x 512 x 1536 113 us with the large, 134 with the small ones; 8 x
// 2048 x 1536 x 1024 16 either way; 256 x 131072 x 1536 x 160 133 and 167; 256 x
// 32768 x 192 x 192 14 either way; 64 x 16384 x 128 x 2048 28 and 24; 256 x 32768
// x 64 x 64 12 and 8.  Parts have a fixed number of rows, so that experts of
// different lengths give equal work; a second kernel sums them (4 x 32768 x 512
// x 512: 207 us whole, 62 in equal numbers of parts per expert, 42 so).  The
// choice depends on the sizes alone.
struct WgradPlan {
  bool large;
  int32_t part_rows;   // 0: whole segments
  int32_t parts_max;
  size_t bytes;        // of the parts
};

WgradPlan wgrad_plan(int64_t experts, int64_t rows, int64_t n, int64_t k, bool bf) {
  WgradPlan p{};
  if (experts == 0) return p;
  const int64_t large = ceil_div(n, 256) * ceil_div(k, 256);
  const int64_t square = ceil_div(n, 128) * ceil_div(k, 128);
  p.large = bf && n > 128 && k > 128 && experts * large >= 192;
  if (p.large || rows == 0) return p;
  // a part: as many rows as leave two 128 x 128 tiles (one 256 x 256) per CU,
  // each expert's last part, which is not full, among them; and enough rows to
  // be worth its sum
  const bool wide = bf && n >= 256 && k >= 256;
  const int64_t tiles = wide ? large : square;
  const int64_t room = wide ? 256 : 512, want = std::max(room - experts * tiles, room / 4);
  const int64_t len = std::max<int64_t>(bf ? 128 : 64, round_up(ceil_div(rows * tiles, want), 64));
  if (rows < len * experts * 5 / 4) return p;
  p.large = wide;
  p.part_rows = static_cast<int32_t>(len);
  p.parts_max = static_cast<int32_t>(group_tiles_max(rows, experts, len));
  p.bytes = static_cast<size_t>(p.parts_max) * n * k * 4;
  return p;
}

// The kernels by name.  The rules below choose one from sizes, types and
// alignment; launches and mfsdp_grouped_linear_tile both go by them.
enum GroupKernel {
  kUseLarge, kUseWide, kUsePair, kUseSmall, kUseRows, kUseFew, kUseF32,   // forward, input gradient
  kUseSquareReg, kUseRowsReg,                                             // ... through registers
  kUseWgrad, kUseWgradSquare, kUseWgradF32, kUseWgradReg                  // weight gradient
};

struct GroupShape {
  int32_t rows, cols, threads, wave_sets;
  bool dma;
};

template <class C>
constexpr GroupShape shape_of(bool dma) {
  return {C::BP, C::BQ, C::THREADS, C::KS, dma};
}

GroupShape group_shape(GroupKernel u) {
  switch (u) {
    case kUseLarge: return shape_of<TileLarge>(true);
    case kUseWide: return shape_of<TileWide>(true);
    case kUsePair: return shape_of<TilePair>(true);
    case kUseSmall: return shape_of<TileSmall>(true);
    case kUseRows: return shape_of<TileRows>(true);
    case kUseFew: return shape_of<TileFew>(true);
    case kUseF32: case kUseWgradF32: return shape_of<TileF32>(true);
    case kUseRowsReg: return shape_of<TileRowsReg>(false);
    case kUseWgrad: return shape_of<TileWgrad>(true);
    case kUseWgradSquare: return shape_of<TileWgradSquare>(true);
    case kUseSquareReg: case kUseWgradReg: break;
  }
  return shape_of<TileSquare>(false);
}

// Weight gradient.
GroupKernel wgrad_kernel(bool bf, bool dma, bool large) {
  return !dma ? kUseWgradReg : !bf ? kUseWgradF32 : large ? kUseWgrad : kUseWgradSquare;
}

// Forward and input gradient.  Rows per expert (known on the host only on
// average) decide the tile's height, the number of tiles whether there are
// enough of that size for the 256 CUs.
GroupKernel rows_kernel(int mode, const GroupArgs& g, bool bf, bool dma) {
  const int64_t experts = std::min<int64_t>(g.experts, g.rows);
  const int64_t per = g.rows / experts;
  const int64_t width = mode == kGroupFwd ? g.n : g.k, depth = mode == kGroupFwd ? g.k : g.n;
  auto tiles = [&](int64_t bp, int64_t bq) {   // an expert with few rows has one row tile
    const int64_t high = per < bp / 2 ? experts : g.rows / bp + experts / 2 + 1;
    return high * ceil_div(width, bq);
  };
  // Under two tiles of 64 columns per four CUs, 32 columns and eight sets of
  // waves: 256 x 8 x 512 x 1536 8.5 -> 7.2 us (fp32 21.0 -> 13.2), but with
  // 224 tiles, 1 x 1 x 14336 x 4096, 22.0 -> 24.5.
  const GroupKernel few_rows = mode == kGroupFwd && tiles(32, 64) <= 128 ? kUseFew : kUseRows;
  // Through registers: 7 x 2049 x 513 x 257 8.9 (few rows' tile) and 11.8 us,
  // its input gradient 10.0 and 21.2 (fp32 19 and 54); 8 x 8192 x 2047 x 2049
  // 244 and 138 us.
  if (!dma) return per <= 48 || tiles(128, 128) < 128 ? kUseRowsReg : kUseSquareReg;
  // fp32: 16 x 1024 x 2048 x 2048 114 (few rows) and 252 us; 64 x 8192 x 2048
  // x 1024 398 and 387; 1 x 8192 x 4096 x 4096 2427 and 1994 us.
  if (!bf) return per <= 96 || tiles(128, 128) < 192 ? few_rows : kUseF32;
  // Forward of 32 x 1024 x 2048 x 2048: 51 us, 67 and more with taller tiles;
  // its input gradient, whose narrow tiles read the weights in 128-byte pieces,
  // 61, and 50 with taller ones.
  if ((mode == kGroupFwd && per <= 40) || tiles(64, 256) < 128) return few_rows;
  // 64 x 1024 x 1024 x 2048, input gradient: 48 (64 rows) and 50 us
  // (128 rows).
  if (per <= 24 || tiles(128, 256) < 100) return kUseSmall;
  // 16 x 24576 x 5632 x 2048: 532 (256 rows) and 576 us (128 rows); 64 x 8192
  // x 2048 x 1024, 128 rows per expert: 89 and 69 us.
  if (per >= 320 && tiles(256, 256) >= 256) return kUseLarge;
  // Short sums leave a tile's start and end uncovered unless two workgroups
  // share a CU: 256 x 32771 x 512 x 1536, input gradient (depth 512): 118
  // (pair) and 136 us; forward (depth 1536): 130 and 109 us.
  return depth < 1024 && tiles(128, 256) >= 512 ? kUsePair : kUseWide;
}

template <class E, int LOAD>
hipError_t launch_wgrad(const GroupArgs& g, GroupKernel use, hipStream_t stream) {
  hipError_t e;
  if constexpr (LOAD == kLoadReg || LOAD == kLoadRegCkpt)
    e = launch_tile<E, kGroupWgrad, TileSquare, LOAD>(g, stream);
  else if constexpr (E::kVec == 4)
    e = launch_tile<E, kGroupWgrad, TileF32, LOAD>(g, stream);
  else
    e = use == kUseWgrad
            ? launch_tile<E, kGroupWgrad, TileWgrad, LOAD>(g, stream)
            : launch_tile<E, kGroupWgrad, TileWgradSquare, LOAD>(g, stream);
  if (e != hipSuccess || g.part_rows == 0) return e;
  const int64_t per = ceil_div(static_cast<int64_t>(g.n) * g.k, 2048);
  const dim3 grid(static_cast<unsigned>(g.experts * per));
  return launch(MFSDP_KERNEL_GROUPED, stream, [&] {
    if (E::kVec == 8 && !g.out_f32)
      grouped_sum_kernel<ElemBF16><<<grid, dim3(256), 0, stream>>>(g, static_cast<int>(per));
    else
      grouped_sum_kernel<ElemF32><<<grid, dim3(256), 0, stream>>>(g, static_cast<int>(per));
  });
}

template <class E, int MODE>
hipError_t launch_rows(const GroupArgs& g, GroupKernel use, hipStream_t stream) {
  switch (use) {
    case kUseRows: return launch_tile<E, MODE, TileRows, kLoadDma>(g, stream);
    case kUseRowsReg: return launch_tile<E, MODE, TileRowsReg, kLoadReg>(g, stream);
    case kUseSquareReg: return launch_tile<E, MODE, TileSquare, kLoadReg>(g, stream);
    default: break;
  }
  if constexpr (MODE == kGroupFwd)
    if (use == kUseFew) return launch_tile<E, MODE, TileFew, kLoadDma>(g, stream);
  if constexpr (E::kVec == 4) {
    if (use == kUseF32) return launch_tile<E, MODE, TileF32, kLoadDma>(g, stream);
  } else {
    switch (use) {
      case kUseLarge: return launch_tile<E, MODE, TileLarge, kLoadDma>(g, stream);
      case kUseWide: return launch_tile<E, MODE, TileWide, kLoadDma>(g, stream);
      case kUsePair: return launch_tile<E, MODE, TilePair, kLoadDma>(g, stream);
      case kUseSmall: return launch_tile<E, MODE, TileSmall, kLoadDma>(g, stream);
      default: break;
    }
  }
  return hipErrorInvalidValue;   // no kernel of this type and direction
}

template <class E>
hipError_t launch_grouped(int mode, const GroupArgs& g, GroupKernel use, hipStream_t stream) {
  if (mode == kGroupFwd) return launch_rows<E, kGroupFwd>(g, use, stream);
  if (mode == kGroupDgrad) return launch_rows<E, kGroupDgrad>(g, use, stream);
  const bool dma = use != kUseWgradReg;
  if (!g.qs) return dma ? launch_wgrad<E, kLoadDma>(g, use, stream) : launch_wgrad<E, kLoadReg>(g, use, stream);
  if constexpr (E::kVec == 8)
    if (dma) return launch_wgrad<E, kLoadDmaCkpt>(g, use, stream);
  return launch_wgrad<E, kLoadRegCkpt>(g, use, stream);
}

// Whether operands can go to LDS by 16-byte DMA, rows starting on 16 bytes: they
// have a whole number of 16-byte pieces, and 256 of them lie within 2^31 bytes
// (`widest`: the largest width or stride).
bool group_dma(int mode, bool codes, bool bf, int64_t n, int64_t k, int64_t widest) {
  const int64_t es = bf ? 2 : 4, v = 16 / es;
  return (!codes || (bf && k % 16 == 0)) && k % v == 0 && (n % v == 0 || mode == kGroupFwd) &&
         widest * es < (int64_t(1) << 23);
}

GroupKernel group_kernel(int mode, const GroupArgs& g, bool bf, bool dma, const WgradPlan& plan) {
  return mode == kGroupWgrad ? wgrad_kernel(bf, dma, plan.large) : rows_kernel(mode, g, bf, dma);
}

// Whether the launches' grids hold the call: its tiles (of forward and input
// gradient through registers as many as 32 x 64 ones would be, whichever of the
// two kernels runs) and the 2048-element pieces of a sum of parts.
bool group_fits(int mode, const GroupArgs& g, GroupKernel use) {
  const GroupShape s = group_shape(use);
  const bool reg = mode != kGroupWgrad && !s.dma;
  const int64_t blocks = reg ? group_blocks(g, mode, 32, 64) : group_blocks(g, mode, s.rows, s.cols);
  const int64_t sums = g.part_rows ? g.experts * ceil_div(static_cast<int64_t>(g.n) * g.k, 2048) : 0;
  return blocks <= kGroupBlocksMax && sums <= kBlocksMax;
}

mfsdp_status_t grouped_sizes(int64_t experts, int64_t rows, int64_t n, int64_t k,
                             mfsdp_dtype_t dtype) {
  if (dtype != MFSDP_DTYPE_F32 && dtype != MFSDP_DTYPE_BF16)
    return fail(MFSDP_ERR_UNSUPPORTED, "unsupported dtype %d", (int)dtype);
  if (experts < 0 || rows < 0 || n < 1 || k < 1)
    return fail(MFSDP_ERR_INVALID_ARGUMENT,
                "experts=%lld rows=%lld n=%lld k=%lld: counts must be >= 0, widths >= 1",
                (long long)experts, (long long)rows, (long long)n, (long long)k);
  if (experts > kGroupExpertsMax || rows > kGroupRowsMax || n > kGroupDimMax || k > kGroupDimMax)
    return fail(MFSDP_ERR_UNSUPPORTED, "a size exceeds the kernels' indexing");
  return MFSDP_OK;
}

// Checks what the three products share, chooses the kernel and launches.
mfsdp_status_t grouped_impl(int mode, const void* p, int64_t ldp, const void* q, int64_t ldq,
                            const uint8_t* qs, const int32_t* offsets, int64_t experts,
                            int64_t rows, int64_t n, int64_t k, mfsdp_dtype_t dtype, void* out,
                            int64_t ldo, mfsdp_dtype_t out_dtype, float beta, void* workspace,
                            size_t workspace_bytes, hipStream_t stream) {
  g_last_error.clear();
  mfsdp_status_t st = grouped_sizes(experts, rows, n, k, dtype);
  if (st != MFSDP_OK) return st;
  if (out_dtype != dtype && out_dtype != MFSDP_DTYPE_F32)
    return fail(MFSDP_ERR_UNSUPPORTED, "unsupported gradient dtype %d", (int)out_dtype);
  if (!finite(beta)) return fail(MFSDP_ERR_INVALID_ARGUMENT, "non-finite beta");
  const int64_t np = mode == kGroupFwd ? k : n;                           // width of P's rows
  const int64_t no = mode == kGroupFwd ? n : k;                           // width of the output's
  if (ldp < np || (mode == kGroupWgrad ? ldq < k : ldo < no))
    return fail(MFSDP_ERR_INVALID_ARGUMENT, "a row stride is smaller than the row");
  if (ldp > kGroupDimMax || ldq > kGroupDimMax || ldo > kGroupDimMax)
    return fail(MFSDP_ERR_UNSUPPORTED, "a size exceeds the kernels' indexing");
  if (experts == 0 || (rows == 0 && mode != kGroupWgrad)) return MFSDP_OK;
  if (!out || !offsets || (rows > 0 && (!p || !q)) || (mode != kGroupWgrad && !q))
    return fail(MFSDP_ERR_INVALID_ARGUMENT, "null pointer");
  const size_t es = elem_size(dtype), eo = elem_size(out_dtype);
  if (!aligned(p, es) || (!qs && !aligned(q, es)) || !aligned(out, eo) || !aligned(offsets, 4))
    return fail(MFSDP_ERR_INVALID_ARGUMENT, "a buffer is not aligned to its elements");
  const bool bf = dtype == MFSDP_DTYPE_BF16;
  const WgradPlan plan = mode == kGroupWgrad ? wgrad_plan(experts, rows, n, k, bf) : WgradPlan{};
  const size_t need = plan.bytes;
  if (need) {
    if (!workspace) return fail(MFSDP_ERR_WORKSPACE, "workspace is null");
    if (!aligned(workspace, kWsAlign))
      return fail(MFSDP_ERR_WORKSPACE, "workspace must be %zu-byte aligned", kWsAlign);
    if (workspace_bytes < need)
      return fail(MFSDP_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", workspace_bytes, need);
  }
  {
    std::vector<Extent> ins, outs;
    const size_t wb = static_cast<size_t>(experts) * n * k;
    if (need) add_bytes(&outs, workspace, need, "workspace");
    add_bytes(&ins, offsets, static_cast<size_t>(experts + 1) * 4, "offsets");
    add_rows(&ins, p, rows, np, ldp, es, mode == kGroupFwd ? "x" : "dy");
    if (mode == kGroupWgrad) {
      add_rows(&ins, q, rows, k, ldq, qs ? 1 : es, qs ? "codes" : "x");
      if (qs)
        add_bytes(&ins, qs, static_cast<size_t>(rows) * ((k + kCkptBlock - 1) / kCkptBlock),
                  "scales");
      add_bytes(&outs, out, wb * eo, "dw");
    } else {
      add_bytes(&ins, q, wb * es, "weight");
      add_rows(&outs, out, rows, no, ldo, es, mode == kGroupFwd ? "y" : "dx");
    }
    st = check_outputs(outs, ins);
    if (st != MFSDP_OK) return st;
  }

  GroupArgs g{};
  g.p = p;
  g.q = q;
  g.qs = qs;
  g.out = out;
  g.off = offsets;
  g.ldp = ldp;
  g.ldq = ldq;
  g.ldo = ldo;
  g.experts = static_cast<int32_t>(experts);
  g.rows = static_cast<int32_t>(rows);
  g.n = static_cast<int32_t>(n);
  g.k = static_cast<int32_t>(k);
  g.beta = beta;
  g.out_f32 = out_dtype == MFSDP_DTYPE_F32 ? 1 : 0;
  g.part_rows = plan.part_rows;
  g.parts_max = plan.parts_max;
  g.part = static_cast<float*>(workspace);
  g.stream = aligned(out, 128) && (mode == kGroupWgrad ? k : ldo) * static_cast<int64_t>(eo) % 128 == 0;
  // eight L2s of 4 MB
  g.stream_w = std::min(experts, rows) * n * k * static_cast<int64_t>(es) > (int64_t(32) << 20);
  const int64_t v = 16 / static_cast<int64_t>(es);
  const bool dma = aligned(p, 16) && aligned(q, 16) && ldp % v == 0 && ldq % v == 0 &&
                   group_dma(mode, qs != nullptr, bf, n, k, std::max({n, k, ldp, ldq}));
  const GroupKernel use = group_kernel(mode, g, bf, dma, plan);
  if (!group_fits(mode, g, use)) return fail(MFSDP_ERR_UNSUPPORTED, "too many tiles");
  const hipError_t e = bf ? launch_grouped<ElemBF16>(mode, g, use, stream)
                          : launch_grouped<ElemF32>(mode, g, use, stream);
  if (e != hipSuccess) return fail(MFSDP_ERR_HIP, "grouped launch: %s", hipGetErrorString(e));
  return MFSDP_OK;
}

// ---------------------------------------------------------------------------
// 8-bit activation checkpoints
// ---------------------------------------------------------------------------
mfsdp_status_t ckpt_impl(bool quantize, void* x, int64_t ld, int8_t* codes, uint8_t* scales,
                         int64_t rows, int64_t k, mfsdp_dtype_t dtype, hipStream_t stream) {
  g_last_error.clear();
  if (dtype != MFSDP_DTYPE_F32 && dtype != MFSDP_DTYPE_BF16)
    return fail(MFSDP_ERR_UNSUPPORTED, "unsupported dtype %d", (int)dtype);
  if (rows < 0 || k < 1 || ld < k)
    return fail(MFSDP_ERR_INVALID_ARGUMENT, "rows=%lld k=%lld ld=%lld", (long long)rows,
                (long long)k, (long long)ld);
  if (rows > kGroupRowsMax || k > kGroupDimMax || ld > kGroupDimMax)
    return fail(MFSDP_ERR_UNSUPPORTED, "a size exceeds the kernels' indexing");
  if (rows == 0) return MFSDP_OK;
  if (!x || !codes || !scales) return fail(MFSDP_ERR_INVALID_ARGUMENT, "null pointer");
  const size_t es = elem_size(dtype);
  if (!aligned(x, es))
    return fail(MFSDP_ERR_INVALID_ARGUMENT, "a buffer is not aligned to its elements");
  CkptArgs a{};
  a.ld = ld;
  a.k = static_cast<int32_t>(k);
  a.nb = static_cast<int32_t>((k + kCkptBlock - 1) / kCkptBlock);
  a.vec = aligned(x, 16) && (ld * static_cast<int64_t>(es)) % 16 == 0 && k % 8 == 0 &&
          aligned(codes, 8);
  {
    std::vector<Extent> xs, cs;
    add_rows(&xs, x, rows, k, ld, es, "x");
    add_bytes(&cs, codes, static_cast<size_t>(rows) * k, "codes");
    add_bytes(&cs, scales, static_cast<size_t>(rows) * a.nb, "scales");
    const mfsdp_status_t st = quantize ? check_outputs(cs, xs) : check_outputs(xs, cs);
    if (st != MFSDP_OK) return st;
  }
  const int64_t most = kBlocksMax * 16 * kCkptUnits / a.nb;   // rows of one launch
  hipError_t e = hipSuccess;
  for (int64_t r = 0; r < rows && e == hipSuccess; r += most) {
    a.x = static_cast<char*>(x) + r * ld * static_cast<int64_t>(es);
    a.codes = codes + r * k;
    a.scales = scales + r * a.nb;
    a.units = static_cast<uint32_t>(std::min(most, rows - r) * a.nb);
    const dim3 grid(static_cast<unsigned>(ceil_div(a.units, 16 * kCkptUnits))), wg(256);
    e = launch(MFSDP_KERNEL_CKPT, stream, [&] {
      if (quantize) {
        if (dtype == MFSDP_DTYPE_BF16) ckpt_quantize_kernel<ElemBF16><<<grid, wg, 0, stream>>>(a);
        else ckpt_quantize_kernel<ElemF32><<<grid, wg, 0, stream>>>(a);
      } else {
        if (dtype == MFSDP_DTYPE_BF16) ckpt_restore_kernel<ElemBF16><<<grid, wg, 0, stream>>>(a);
        else ckpt_restore_kernel<ElemF32><<<grid, wg, 0, stream>>>(a);
      }
    });
  }
  if (e != hipSuccess) return fail(MFSDP_ERR_HIP, "checkpoint launch: %s", hipGetErrorString(e));
  return MFSDP_OK;
}

// ---------------------------------------------------------------------------
// Embedding
// ---------------------------------------------------------------------------
constexpr int64_t kEmbVocabMax = (int64_t(1) << 31) - 1;
constexpr int64_t kEmbTokensMax = int64_t(1) << 28;

template <class ET, class EO>
hipError_t launch_embedding(const EmbArgs& a, bool vec, int64_t blocks, hipStream_t stream) {
  return launch(MFSDP_KERNEL_EMBED, stream, [&] {
    const dim3 grid(static_cast<unsigned>(blocks)), wg(256);
    if (vec) embedding_kernel<ET, EO, true><<<grid, wg, 0, stream>>>(a);
    else embedding_kernel<ET, EO, false><<<grid, wg, 0, stream>>>(a);
  });
}

mfsdp_status_t embedding_impl(const void* table, mfsdp_dtype_t table_dtype, int64_t vocab,
                              int64_t d, const void* tokens, int token_bytes, int64_t n_tokens,
                              float scale, void* out, int64_t ldo, mfsdp_dtype_t out_dtype,
                              hipStream_t stream) {
  g_last_error.clear();
  for (mfsdp_dtype_t dt : {table_dtype, out_dtype})
    if (dt != MFSDP_DTYPE_F32 && dt != MFSDP_DTYPE_BF16)
      return fail(MFSDP_ERR_UNSUPPORTED, "unsupported dtype %d", (int)dt);
  if (token_bytes != 4 && token_bytes != 8)
    return fail(MFSDP_ERR_UNSUPPORTED, "tokens of %d bytes: 4 or 8 are taken", token_bytes);
  if (vocab < 1 || d < 1 || n_tokens < 0 || ldo < d)
    return fail(MFSDP_ERR_INVALID_ARGUMENT, "vocab=%lld d=%lld tokens=%lld ldo=%lld",
                (long long)vocab, (long long)d, (long long)n_tokens, (long long)ldo);
  if (!finite(scale)) return fail(MFSDP_ERR_INVALID_ARGUMENT, "non-finite scale");
  if (vocab > kEmbVocabMax || d > kGroupDimMax || ldo > kGroupDimMax || n_tokens > kEmbTokensMax)
    return fail(MFSDP_ERR_UNSUPPORTED, "a size exceeds the kernels' indexing");
  if (n_tokens == 0) return MFSDP_OK;
  if (!table || !tokens || !out) return fail(MFSDP_ERR_INVALID_ARGUMENT, "null pointer");
  const size_t et = elem_size(table_dtype), eo = elem_size(out_dtype);
  if (!aligned(table, et) || !aligned(out, eo) || !aligned(tokens, token_bytes))
    return fail(MFSDP_ERR_INVALID_ARGUMENT, "a buffer is not aligned to its elements");
  {
    std::vector<Extent> ins, outs;
    add_bytes(&ins, table, static_cast<size_t>(vocab) * d * et, "table");
    add_bytes(&ins, tokens, static_cast<size_t>(n_tokens) * token_bytes, "tokens");
    add_rows(&outs, out, n_tokens, d, ldo, eo, "out");
    const mfsdp_status_t st = check_outputs(outs, ins);
    if (st != MFSDP_OK) return st;
  }
  EmbArgs a{};
  a.table = table;
  a.vocab = vocab;
  a.ldo = ldo;
  a.d = static_cast<int32_t>(d);
  a.tok64 = token_bytes == 8;
  a.scale = scale;
  const int64_t w = 16 / static_cast<int64_t>(eo);
  const bool vec = d % w == 0 && aligned(table, std::min<size_t>(w * et, 16)) && aligned(out, 16) &&
                   ldo % w == 0;
  const int64_t units = vec ? d / w : d;
  int64_t most;   // tokens of one launch
  if (units > 128) {
    a.chunks = static_cast<int32_t>((units + 255) / 256);
    most = kBlocksMax / a.chunks;
  } else {
    a.per_wg = static_cast<int32_t>(256 / units);
    most = kBlocksMax * a.per_wg;
  }
  const bool tb = table_dtype == MFSDP_DTYPE_BF16, ob = out_dtype == MFSDP_DTYPE_BF16;
  hipError_t e = hipSuccess;
  for (int64_t t0 = 0; t0 < n_tokens && e == hipSuccess; t0 += most) {
    a.tokens = static_cast<const char*>(tokens) + t0 * token_bytes;
    a.out = static_cast<char*>(out) + t0 * ldo * static_cast<int64_t>(eo);
    a.n_tokens = std::min(most, n_tokens - t0);
    const int64_t blocks = a.chunks ? a.n_tokens * a.chunks : ceil_div(a.n_tokens, a.per_wg);
    e = tb ? (ob ? launch_embedding<ElemBF16, ElemBF16>(a, vec, blocks, stream)
                 : launch_embedding<ElemBF16, ElemF32>(a, vec, blocks, stream))
           : (ob ? launch_embedding<ElemF32, ElemBF16>(a, vec, blocks, stream)
                 : launch_embedding<ElemF32, ElemF32>(a, vec, blocks, stream));
  }
  if (e != hipSuccess) return fail(MFSDP_ERR_HIP, "embedding launch: %s", hipGetErrorString(e));
  return MFSDP_OK;
}

// Workspace of an embedding gradient: two (key, position) lists, the digit
// counts of the sort and the partial rows of long runs.
struct EmbPlan {
  size_t key0, pos0, key1, pos1, hist, begin, part, total;
  int32_t key_bits, bits, passes, per_block, blocks;
};

// Lists up to this length are sorted by one workgroup in one launch.
constexpr int64_t kSortSmall = 4096;

EmbPlan emb_plan(int64_t n, int64_t vocab, int64_t d) {
  EmbPlan p{};
  p.key_bits = 1;
  while ((int64_t(1) << p.key_bits) <= vocab) ++p.key_bits;    // keys are 0..vocab
  p.passes = (p.key_bits + kSortBitsMax - 1) / kSortBitsMax;
  p.bits = (p.key_bits + p.passes - 1) / p.passes;
  // at most 512 workgroups: each reads the digit counts of all of them
  const int64_t per = std::max<int64_t>(2048, (n + 511) / 512);
  p.per_block = static_cast<int32_t>(round_up(per, kSortThreads));
  p.blocks = n <= kSortSmall ? 1 : static_cast<int32_t>((n + p.per_block - 1) / p.per_block);
  size_t off = 0;
  auto take = [&](size_t nb) {
    const size_t at = off;
    off = align_up(off + nb, kWsAlign);
    return at;
  };
  const size_t list = static_cast<size_t>(n) * 4;
  p.key0 = take(list);
  p.pos0 = take(list);
  p.key1 = take(list);
  p.pos1 = take(list);
  p.hist = take(p.blocks > 1 ? (static_cast<size_t>(p.blocks) << p.bits) * 4 : 0);
  p.begin = take((static_cast<size_t>(vocab + kEmbRows - 1) / kEmbRows + 1) * 4);
  p.part = take(n > kEmbRun ? static_cast<size_t>((n + kEmbRun - 1) / kEmbRun) * 2 * d * 4 : 0);
  p.total = off;
  return p;
}

mfsdp_status_t emb_grad_sizes(int64_t n_tokens, int64_t vocab, int64_t d) {
  if (vocab < 1 || d < 1 || n_tokens < 0)
    return fail(MFSDP_ERR_INVALID_ARGUMENT, "vocab=%lld d=%lld tokens=%lld", (long long)vocab,
                (long long)d, (long long)n_tokens);
  if (vocab > kEmbVocabMax || d > kGroupDimMax || n_tokens > kEmbTokensMax)
    return fail(MFSDP_ERR_UNSUPPORTED, "a size exceeds the kernels' indexing");
  return MFSDP_OK;
}

template <class E, int W>
hipError_t launch_emb_sums(const EmbGradArgs& a, hipStream_t stream) {
  const int64_t col_wgs = ceil_div(a.d, static_cast<int64_t>(a.tpr) * W * kEmbGroups);
  const int64_t row_blocks = ceil_div(a.vocab, kEmbRows);
  if (a.n > 0) {   // partial sums of long runs (if there can be any), row block bounds
    const int64_t chunks = a.n > kEmbRun ? ceil_div(a.n, kEmbRun) : 0;
    const int64_t blocks = chunks * col_wgs + ceil_div(row_blocks + 1, 256);
    const hipError_t e = launch(MFSDP_KERNEL_EMBED_GRAD, stream, [&] {
      emb_partial_kernel<E, W><<<dim3(static_cast<unsigned>(blocks)), dim3(256), 0, stream>>>(
          a, static_cast<int>(chunks), static_cast<int>(col_wgs));
    });
    if (e != hipSuccess) return e;
  }
  const int64_t most = kBlocksMax / col_wgs;   // row blocks of one launch
  for (int64_t b = 0; b < row_blocks; b += most) {
    EmbGradArgs part = a;
    part.block0 = b;
    const int64_t blocks = std::min(most, row_blocks - b) * col_wgs;
    const hipError_t e = launch(MFSDP_KERNEL_EMBED_GRAD, stream, [&] {
      emb_rows_kernel<E, W><<<dim3(static_cast<unsigned>(blocks)), dim3(256), 0, stream>>>(
          part, static_cast<int>(col_wgs));
    });
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

mfsdp_status_t embedding_grad_impl(const void* dy, int64_t ld, mfsdp_dtype_t dtype,
                                   const void* tokens, int token_bytes, int64_t n_tokens,
                                   int64_t vocab, int64_t d, float scale, float beta, float* grad,
                                   void* workspace, size_t workspace_bytes, hipStream_t stream) {
  g_last_error.clear();
  if (dtype != MFSDP_DTYPE_F32 && dtype != MFSDP_DTYPE_BF16)
    return fail(MFSDP_ERR_UNSUPPORTED, "unsupported dtype %d", (int)dtype);
  if (token_bytes != 4 && token_bytes != 8)
    return fail(MFSDP_ERR_UNSUPPORTED, "tokens of %d bytes: 4 or 8 are taken", token_bytes);
  mfsdp_status_t st = emb_grad_sizes(n_tokens, vocab, d);
  if (st != MFSDP_OK) return st;
  if (ld < d) return fail(MFSDP_ERR_INVALID_ARGUMENT, "a row stride is smaller than the row");
  if (ld > kGroupDimMax) return fail(MFSDP_ERR_UNSUPPORTED, "a size exceeds the kernels' indexing");
  if (!finite(scale) || !finite(beta))
    return fail(MFSDP_ERR_INVALID_ARGUMENT, "non-finite scale or beta");
  if (!grad || (n_tokens > 0 && (!dy || !tokens)))
    return fail(MFSDP_ERR_INVALID_ARGUMENT, "null pointer");
  const size_t es = elem_size(dtype);
  if ((n_tokens > 0 && (!aligned(dy, es) || !aligned(tokens, token_bytes))) || !aligned(grad, 4))
    return fail(MFSDP_ERR_INVALID_ARGUMENT, "a buffer is not aligned to its elements");
  const EmbPlan p = emb_plan(n_tokens, vocab, d);
  if (n_tokens > 0) {
    if (!workspace) return fail(MFSDP_ERR_WORKSPACE, "workspace is null");
    if (!aligned(workspace, kWsAlign))
      return fail(MFSDP_ERR_WORKSPACE, "workspace must be %zu-byte aligned", kWsAlign);
    if (workspace_bytes < p.total)
      return fail(MFSDP_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", workspace_bytes,
                  p.total);
  }
  {
    std::vector<Extent> ins, outs;
    add_rows(&ins, dy, n_tokens, d, ld, es, "dy");
    add_bytes(&ins, tokens, static_cast<size_t>(n_tokens) * token_bytes, "tokens");
    add_bytes(&outs, grad, static_cast<size_t>(vocab) * d * 4, "grad");
    if (n_tokens > 0) add_bytes(&outs, workspace, p.total, "workspace");
    st = check_outputs(outs, ins);
    if (st != MFSDP_OK) return st;
  }
  const bool vec = d % 4 == 0 && aligned(grad, 16) && aligned(dy, 4 * es) && ld % 4 == 0;
  const int64_t cols = vec ? 4 : 1;
  int32_t tpr = 64;
  while (tpr < 256 && tpr * cols * kEmbGroups < d) tpr *= 2;
  const int64_t col_wgs = ceil_div(d, tpr * cols * kEmbGroups);
  if (ceil_div(n_tokens, kEmbRun) * col_wgs + ceil_div(vocab, kEmbRows) / 256 + 2 > kBlocksMax)
    return fail(MFSDP_ERR_UNSUPPORTED, "too many rows");

  char* ws = static_cast<char*>(workspace);
  EmbGradArgs a{};
  a.dy = dy;
  a.grad = grad;
  a.vocab = vocab;
  a.ld = ld;
  a.n = static_cast<int32_t>(n_tokens);
  a.d = static_cast<int32_t>(d);
  a.tpr = tpr;
  a.scale = scale;
  a.beta = beta;
  hipError_t e = hipSuccess;
  if (n_tokens > 0) {
    uint32_t* key[2] = {reinterpret_cast<uint32_t*>(ws + p.key0), reinterpret_cast<uint32_t*>(ws + p.key1)};
    uint32_t* pos[2] = {reinterpret_cast<uint32_t*>(ws + p.pos0), reinterpret_cast<uint32_t*>(ws + p.pos1)};
    SortArgs s{};
    s.tokens = tokens;
    s.vocab = vocab;
    s.n = a.n;
    s.tok64 = token_bytes == 8;
    s.per_block = p.per_block;
    s.bits = p.bits;
    int at = 0;   // list that holds the result
    if (p.blocks == 1) {
      SortSmallArgs sm{};
      sm.s = s;
      sm.s.key_out = key[0];
      sm.s.pos_out = pos[0];
      sm.key_tmp = key[1];
      sm.pos_tmp = pos[1];
      sm.key_bits = p.key_bits;
      sm.passes = p.passes;
      e = launch(MFSDP_KERNEL_EMBED_GRAD, stream, [&] {
        sort_small_kernel<<<dim3(1), dim3(kSortThreads), 0, stream>>>(sm);
      });
    } else {
      const dim3 grid(static_cast<unsigned>(p.blocks)), wg(kSortThreads);
      s.hist = reinterpret_cast<uint32_t*>(ws + p.hist);
      for (int q = 0; q < p.passes && e == hipSuccess; ++q) {
        s.first = q == 0;
        s.shift = q * p.bits;
        s.key_in = key[at];
        s.pos_in = pos[at];
        at ^= 1;
        s.key_out = key[at];
        s.pos_out = pos[at];
        e = launch(MFSDP_KERNEL_EMBED_GRAD, stream,
                   [&] { sort_hist_kernel<<<grid, wg, 0, stream>>>(s); });
        if (e == hipSuccess)
          e = launch(MFSDP_KERNEL_EMBED_GRAD, stream,
                     [&] { sort_scatter_kernel<<<grid, wg, 0, stream>>>(s); });
      }
    }
    if (e != hipSuccess) return fail(MFSDP_ERR_HIP, "sort launch: %s", hipGetErrorString(e));
    a.key = key[at];
    a.pos = pos[at];
    a.part = reinterpret_cast<float*>(ws + p.part);
    a.begin = reinterpret_cast<int32_t*>(ws + p.begin);
  }
  if (dtype == MFSDP_DTYPE_BF16)
    e = vec ? launch_emb_sums<ElemBF16, 4>(a, stream) : launch_emb_sums<ElemBF16, 1>(a, stream);
  else
    e = vec ? launch_emb_sums<ElemF32, 4>(a, stream) : launch_emb_sums<ElemF32, 1>(a, stream);
  if (e != hipSuccess)
    return fail(MFSDP_ERR_HIP, "embedding gradient launch: %s", hipGetErrorString(e));
  return MFSDP_OK;
}

// No C++ exception crosses the ABI.
template <class F>
mfsdp_status_t guarded(F&& f) {
  try {
    return f();
  } catch (const std::exception& ex) {
    return fail(MFSDP_ERR_UNSUPPORTED, "host exception: %s", ex.what());
  }
}

}  // namespace

extern "C" {

mfsdp_status_t mfsdp_grouped_linear(const void* x, int64_t ld_x, const void* weight,
                                    const int32_t* offsets, int64_t n_experts, int64_t rows,
                                    int64_t n, int64_t k, mfsdp_dtype_t dtype, void* y,
                                    int64_t ld_y, hipStream_t stream) {
  return guarded([&] {
    return grouped_impl(kGroupFwd, x, ld_x, weight, 0, nullptr, offsets, n_experts, rows, n, k,
                        dtype, y, ld_y, dtype, 0.f, nullptr, 0, stream);
  });
}

mfsdp_status_t mfsdp_grouped_linear_dgrad(const void* dy, int64_t ld_dy, const void* weight,
                                          const int32_t* offsets, int64_t n_experts, int64_t rows,
                                          int64_t n, int64_t k, mfsdp_dtype_t dtype, void* dx,
                                          int64_t ld_dx, hipStream_t stream) {
  return guarded([&] {
    return grouped_impl(kGroupDgrad, dy, ld_dy, weight, 0, nullptr, offsets, n_experts, rows, n, k,
                        dtype, dx, ld_dx, dtype, 0.f, nullptr, 0, stream);
  });
}

mfsdp_status_t mfsdp_grouped_linear_wgrad_workspace_size(int64_t n_experts, int64_t rows,
                                                         int64_t n, int64_t k,
                                                         mfsdp_dtype_t dtype, size_t* out_bytes) {
  return guarded([&]() -> mfsdp_status_t {
    g_last_error.clear();
    if (!out_bytes) return fail(MFSDP_ERR_INVALID_ARGUMENT, "out_bytes is null");
    const mfsdp_status_t st = grouped_sizes(n_experts, rows, n, k, dtype);
    if (st != MFSDP_OK) return st;
    *out_bytes = wgrad_plan(n_experts, rows, n, k, dtype == MFSDP_DTYPE_BF16).bytes;
    return MFSDP_OK;
  });
}

mfsdp_status_t mfsdp_grouped_linear_wgrad(const void* dy, int64_t ld_dy, const void* x,
                                          int64_t ld_x, const int32_t* offsets, int64_t n_experts,
                                          int64_t rows, int64_t n, int64_t k, mfsdp_dtype_t dtype,
                                          void* dw, mfsdp_dtype_t dw_dtype, float beta,
                                          void* workspace, size_t workspace_bytes,
                                          hipStream_t stream) {
  return guarded([&] {
    return grouped_impl(kGroupWgrad, dy, ld_dy, x, ld_x, nullptr, offsets, n_experts, rows, n, k,
                        dtype, dw, 0, dw_dtype, beta, workspace, workspace_bytes, stream);
  });
}

mfsdp_status_t mfsdp_grouped_linear_wgrad_ckpt(const void* dy, int64_t ld_dy, const int8_t* codes,
                                               const uint8_t* scales, const int32_t* offsets,
                                               int64_t n_experts, int64_t rows, int64_t n,
                                               int64_t k, mfsdp_dtype_t dtype, void* dw,
                                               mfsdp_dtype_t dw_dtype, float beta,
                                               void* workspace, size_t workspace_bytes,
                                               hipStream_t stream) {
  return guarded([&]() -> mfsdp_status_t {
    if (!scales && rows > 0 && n_experts > 0) {
      g_last_error.clear();
      return fail(MFSDP_ERR_INVALID_ARGUMENT, "null pointer");
    }
    return grouped_impl(kGroupWgrad, dy, ld_dy, codes, k, scales, offsets, n_experts, rows, n, k,
                        dtype, dw, 0, dw_dtype, beta, workspace, workspace_bytes, stream);
  });
}

mfsdp_status_t mfsdp_grouped_linear_tile(mfsdp_grouped_product_t product, int64_t n_experts,
                                         int64_t rows, int64_t n, int64_t k, mfsdp_dtype_t dtype,
                                         int rows_aligned, mfsdp_grouped_tile_t* out) {
  return guarded([&]() -> mfsdp_status_t {
    g_last_error.clear();
    if (!out || product < MFSDP_GROUPED_FORWARD || product > MFSDP_GROUPED_WGRAD_CKPT)
      return fail(MFSDP_ERR_INVALID_ARGUMENT, "product %d, out %p", (int)product, (void*)out);
    mfsdp_status_t st = grouped_sizes(n_experts, rows, n, k, dtype);
    if (st != MFSDP_OK) return st;
    *out = mfsdp_grouped_tile_t{};
    const bool codes = product == MFSDP_GROUPED_WGRAD_CKPT, bf = dtype == MFSDP_DTYPE_BF16;
    const int mode = codes ? kGroupWgrad : static_cast<int>(product);
    if (n_experts == 0 || (rows == 0 && mode != kGroupWgrad)) return MFSDP_OK;   // no launch
    GroupArgs g{};
    g.experts = static_cast<int32_t>(n_experts);
    g.rows = static_cast<int32_t>(rows);
    g.n = static_cast<int32_t>(n);
    g.k = static_cast<int32_t>(k);
    const WgradPlan plan = mode == kGroupWgrad ? wgrad_plan(n_experts, rows, n, k, bf) : WgradPlan{};
    g.part_rows = plan.part_rows;
    const bool dma = rows_aligned && group_dma(mode, codes, bf, n, k, std::max(n, k));
    const GroupKernel use = group_kernel(mode, g, bf, dma, plan);
    if (!group_fits(mode, g, use)) return fail(MFSDP_ERR_UNSUPPORTED, "too many tiles");
    const GroupShape s = group_shape(use);
    out->rows = s.rows;
    out->cols = s.cols;
    out->threads = s.threads;
    out->wave_sets = s.wave_sets;
    out->lds_dma = s.dma ? 1 : 0;
    out->part_rows = plan.part_rows;
    out->workgroups = group_blocks(g, mode, s.rows, s.cols);
    return MFSDP_OK;
  });
}

mfsdp_status_t mfsdp_ckpt_quantize(const void* x, int64_t ld_x, int64_t rows, int64_t k,
                                   mfsdp_dtype_t dtype, int8_t* codes, uint8_t* scales,
                                   hipStream_t stream) {
  return guarded([&] {
    return ckpt_impl(true, const_cast<void*>(x), ld_x, codes, scales, rows, k, dtype, stream);
  });
}

mfsdp_status_t mfsdp_ckpt_restore(const int8_t* codes, const uint8_t* scales, int64_t rows,
                                  int64_t k, mfsdp_dtype_t dtype, void* x, int64_t ld_x,
                                  hipStream_t stream) {
  return guarded([&] {
    return ckpt_impl(false, x, ld_x, const_cast<int8_t*>(codes), const_cast<uint8_t*>(scales),
                     rows, k, dtype, stream);
  });
}

mfsdp_status_t mfsdp_embedding(const void* table, mfsdp_dtype_t table_dtype, int64_t vocab,
                               int64_t d, const void* tokens, int token_bytes, int64_t n_tokens,
                               float scale, void* out, int64_t ld_out, mfsdp_dtype_t out_dtype,
                               hipStream_t stream) {
  return guarded([&] {
    return embedding_impl(table, table_dtype, vocab, d, tokens, token_bytes, n_tokens, scale, out,
                          ld_out, out_dtype, stream);
  });
}

mfsdp_status_t mfsdp_embedding_grad_workspace_size(int64_t n_tokens, int64_t vocab, int64_t d,
                                                   size_t* out_bytes) {
  return guarded([&]() -> mfsdp_status_t {
    g_last_error.clear();
    if (!out_bytes) return fail(MFSDP_ERR_INVALID_ARGUMENT, "out_bytes is null");
    const mfsdp_status_t st = emb_grad_sizes(n_tokens, vocab, d);
    if (st == MFSDP_OK) *out_bytes = n_tokens > 0 ? emb_plan(n_tokens, vocab, d).total : 0;
    return st;
  });
}

mfsdp_status_t mfsdp_embedding_grad(const void* dy, int64_t ld_dy, mfsdp_dtype_t dtype,
                                    const void* tokens, int token_bytes, int64_t n_tokens,
                                    int64_t vocab, int64_t d, float scale, float beta, float* grad,
                                    void* workspace, size_t workspace_bytes, hipStream_t stream) {
  return guarded([&] {
    return embedding_grad_impl(dy, ld_dy, dtype, tokens, token_bytes, n_tokens, vocab, d, scale,
                               beta, grad, workspace, workspace_bytes, stream);
  });
}

}  // extern "C"
