// Host side of the operators around the experts' products: routing and its
// plan, the exchange of rows, layer norm, products in 8-bit floats.  Included
// once, by mfsdp.hip, behind grads_host.hpp, whose helpers it uses.  Every
// launch takes its sizes from the arguments alone; experts, rows and offsets
// stay on the device, so all of these calls can be captured into a graph.
#pragma once

namespace {

// The buffers of one call, on the stack: a call of a few microseconds should
// not spend one of them on allocating lists.
struct Buffers {
  Extent list[12];
  int n = 0, outs = 0;     // the first `outs` are written
  void rows(const void* p, int64_t rows, int64_t cols, int64_t ld, size_t es, const char* what) {
    if (rows < 1 || cols < 1 || !p) return;
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    const size_t pitch = static_cast<size_t>(ld) * es, width = static_cast<size_t>(cols) * es;
    list[n++] = {lo, lo + (rows - 1) * pitch + width, pitch, width, what};
  }
  void bytes(const void* p, size_t nb, const char* what) {
    if (!nb || !p) return;
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    list[n++] = {lo, lo + nb, nb, nb, what};
  }
  void outputs_end() { outs = n; }
  mfsdp_status_t check() const {
    for (int i = 0; i < outs; ++i)
      for (int j = i + 1; j < n; ++j)
        if (overlap(list[i], list[j]))
          return fail(MFSDP_ERR_ALIAS, "%s overlaps %s", list[i].what, list[j].what);
    return MFSDP_OK;
  }
};

bool known_dtype(mfsdp_dtype_t dt) { return dt == MFSDP_DTYPE_F32 || dt == MFSDP_DTYPE_BF16; }

mfsdp_status_t bad_dtype(mfsdp_dtype_t dt) {
  return fail(MFSDP_ERR_UNSUPPORTED, "unsupported dtype %d", (int)dt);
}

mfsdp_status_t null_pointer() { return fail(MFSDP_ERR_INVALID_ARGUMENT, "null pointer"); }

mfsdp_status_t misaligned() {
  return fail(MFSDP_ERR_INVALID_ARGUMENT, "a buffer is not aligned to its elements");
}

mfsdp_status_t too_large() { return fail(MFSDP_ERR_UNSUPPORTED, "a size exceeds the kernels' indexing"); }

mfsdp_status_t launched(hipError_t e, const char* what) {
  return e == hipSuccess ? MFSDP_OK : fail(MFSDP_ERR_HIP, "%s launch: %s", what, hipGetErrorString(e));
}

mfsdp_status_t check_workspace(const void* workspace, size_t have, size_t need) {
  if (!need) return MFSDP_OK;
  if (!workspace) return fail(MFSDP_ERR_WORKSPACE, "workspace is null");
  if (!aligned(workspace, kWsAlign))
    return fail(MFSDP_ERR_WORKSPACE, "workspace must be %zu-byte aligned", kWsAlign);
  if (have < need) return fail(MFSDP_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", have, need);
  return MFSDP_OK;
}

// ---------------------------------------------------------------------------
// Routing
// ---------------------------------------------------------------------------
constexpr int64_t kRouteTokensMax = int64_t(1) << 25;    // four to a workgroup, under 2^24 of them
constexpr int64_t kRouteSlotsMax = int64_t(1) << 30;

mfsdp_status_t route_sizes(int64_t tokens, int64_t n, int64_t k) {
  if (tokens < 0 || n < 1 || k < 1 || k > n)
    return fail(MFSDP_ERR_INVALID_ARGUMENT, "tokens=%lld experts=%lld k=%lld: 1 <= k <= experts", (long long)tokens,
                (long long)n, (long long)k);
  if (n > kRouteExpertsMax || k > kRouteChosenMax)
    return fail(MFSDP_ERR_UNSUPPORTED, "experts=%lld k=%lld: at most %d and %d are taken", (long long)n, (long long)k,
                kRouteExpertsMax, kRouteChosenMax);
  if (tokens >= kRouteTokensMax || tokens * k > kRouteSlotsMax) return too_large();
  return MFSDP_OK;
}

template <class F>
hipError_t launch_per_expert(int64_t n, F&& f) {    // experts of one lane
  if (n <= 64) return f(std::integral_constant<int, 1>{});
  if (n <= 128) return f(std::integral_constant<int, 2>{});
  if (n <= 256) return f(std::integral_constant<int, 4>{});
  if (n <= 512) return f(std::integral_constant<int, 8>{});
  return f(std::integral_constant<int, 16>{});
}

mfsdp_status_t route_impl(const void* logits, int64_t ld, const float* bias, const uint8_t* mask, int64_t tokens,
                          int64_t n, int64_t k, mfsdp_dtype_t dtype, int scores, int64_t groups, int64_t top_groups,
                          int renormalize, float scale, int32_t* experts, float* weights, hipStream_t stream) {
  g_last_error.clear();
  if (!known_dtype(dtype)) return bad_dtype(dtype);
  mfsdp_status_t st = route_sizes(tokens, n, k);
  if (st != MFSDP_OK) return st;
  if (scores != MFSDP_ROUTE_SOFTMAX && scores != MFSDP_ROUTE_SIGMOID)
    return fail(MFSDP_ERR_INVALID_ARGUMENT, "scores=%d", scores);
  if (groups < 1 || n % groups != 0 || top_groups < 1 || top_groups > groups || k > n / groups * top_groups)
    return fail(MFSDP_ERR_INVALID_ARGUMENT, "groups=%lld top_groups=%lld: groups divide the experts, and those that stay hold k",
                (long long)groups, (long long)top_groups);
  if (groups > kRouteGroupsMax) return fail(MFSDP_ERR_UNSUPPORTED, "groups=%lld: at most %d are taken", (long long)groups, kRouteGroupsMax);
  if (ld < n) return fail(MFSDP_ERR_INVALID_ARGUMENT, "a row stride is smaller than the row");
  if (ld > kGroupDimMax) return too_large();
  if (!finite(scale)) return fail(MFSDP_ERR_INVALID_ARGUMENT, "non-finite scale");
  if (tokens == 0) return MFSDP_OK;
  if (!logits || !experts || !weights) return null_pointer();
  const size_t es = elem_size(dtype);
  if (!aligned(logits, es) || !aligned(experts, 4) || !aligned(weights, 4) || (bias && !aligned(bias, 4))) return misaligned();
  Buffers b;
  b.bytes(experts, static_cast<size_t>(tokens * k) * 4, "experts");
  b.bytes(weights, static_cast<size_t>(tokens * k) * 4, "weights");
  b.outputs_end();
  b.rows(logits, tokens, n, ld, es, "logits");
  b.bytes(bias, static_cast<size_t>(n) * 4, "bias");
  b.bytes(mask, static_cast<size_t>(tokens), "mask");
  st = b.check();
  if (st != MFSDP_OK) return st;
  RouteArgs a{};
  a.logits = logits;
  a.bias = bias;
  a.mask = mask;
  a.chosen = experts;
  a.weights = weights;
  a.ld = ld;
  a.tokens = static_cast<int32_t>(tokens);
  a.n = static_cast<int32_t>(n);
  a.k = static_cast<int32_t>(k);
  a.groups = static_cast<int32_t>(groups);
  a.top = static_cast<int32_t>(top_groups);
  a.group_size = static_cast<int32_t>(n / groups);
  a.sigmoid = scores == MFSDP_ROUTE_SIGMOID;
  a.renorm = renormalize != 0;
  a.scale = scale;
  const dim3 grid(static_cast<unsigned>(ceil_div(tokens, 4))), wg(256);
  const hipError_t e = launch_per_expert(n, [&](auto per) {
    constexpr int PER = decltype(per)::value;
    const int lanes = a.group_size % PER == 0 ? a.group_size / PER : 0;
    a.lanes = lanes > 0 && (lanes & (lanes - 1)) == 0 ? lanes : 0;
    return launch(MFSDP_KERNEL_ROUTE, stream, [&] {
      if (dtype == MFSDP_DTYPE_BF16) route_kernel<ElemBF16, PER><<<grid, wg, 0, stream>>>(a);
      else route_kernel<ElemF32, PER><<<grid, wg, 0, stream>>>(a);
    });
  });
  return launched(e, "routing");
}

mfsdp_status_t route_grad_impl(const float* dweights, const void* logits, int64_t ld, const int32_t* experts,
                               int64_t tokens, int64_t n, int64_t k, mfsdp_dtype_t dtype, int scores, int renormalize,
                               float scale, void* dlogits, int64_t ldd, hipStream_t stream) {
  g_last_error.clear();
  if (!known_dtype(dtype)) return bad_dtype(dtype);
  mfsdp_status_t st = route_sizes(tokens, n, k);
  if (st != MFSDP_OK) return st;
  if (scores != MFSDP_ROUTE_SOFTMAX && scores != MFSDP_ROUTE_SIGMOID)
    return fail(MFSDP_ERR_INVALID_ARGUMENT, "scores=%d", scores);
  if (ld < n || ldd < n) return fail(MFSDP_ERR_INVALID_ARGUMENT, "a row stride is smaller than the row");
  if (ld > kGroupDimMax || ldd > kGroupDimMax) return too_large();
  if (!finite(scale)) return fail(MFSDP_ERR_INVALID_ARGUMENT, "non-finite scale");
  if (tokens == 0) return MFSDP_OK;
  if (!dweights || !logits || !experts || !dlogits) return null_pointer();
  const size_t es = elem_size(dtype);
  if (!aligned(logits, es) || !aligned(dlogits, es) || !aligned(experts, 4) || !aligned(dweights, 4)) return misaligned();
  Buffers b;
  b.rows(dlogits, tokens, n, ldd, es, "dlogits");
  b.outputs_end();
  b.rows(logits, tokens, n, ld, es, "logits");
  b.bytes(experts, static_cast<size_t>(tokens * k) * 4, "experts");
  b.bytes(dweights, static_cast<size_t>(tokens * k) * 4, "dweights");
  st = b.check();
  if (st != MFSDP_OK) return st;
  RouteGradArgs a{};
  a.dw = dweights;
  a.logits = logits;
  a.chosen = experts;
  a.out = dlogits;
  a.ld = ld;
  a.ldo = ldd;
  a.tokens = static_cast<int32_t>(tokens);
  a.n = static_cast<int32_t>(n);
  a.k = static_cast<int32_t>(k);
  a.sigmoid = scores == MFSDP_ROUTE_SIGMOID;
  a.renorm = renormalize != 0;
  a.scale = scale;
  const dim3 grid(static_cast<unsigned>(ceil_div(tokens, 4))), wg(256);
  const hipError_t e = launch_per_expert(n, [&](auto per) {
    constexpr int PER = decltype(per)::value;
    return launch(MFSDP_KERNEL_ROUTE, stream, [&] {
      if (dtype == MFSDP_DTYPE_BF16) route_grad_kernel<ElemBF16, PER><<<grid, wg, 0, stream>>>(a);
      else route_grad_kernel<ElemF32, PER><<<grid, wg, 0, stream>>>(a);
    });
  });
  return launched(e, "routing gradient");
}

struct RoutePlanSizes {
  int32_t per_block, blocks;
  size_t bytes;
};

RoutePlanSizes route_plan_sizes(int64_t slots, int64_t n) {
  RoutePlanSizes p{};
  // at most 256 workgroups: each reads the counts of all of them (2^21 choices of
  // 256 experts 19 us, 24 with 512)
  p.per_block = static_cast<int32_t>(round_up(std::max<int64_t>(2048, ceil_div(slots, 256)), kPlanThreads));
  p.blocks = slots <= kPlanSmall ? 1 : static_cast<int32_t>(ceil_div(slots, p.per_block));
  p.bytes = p.blocks > 1 ? static_cast<size_t>(p.blocks) * round_up(n, 4) * 4 : 0;
  return p;
}

// k may pass the number of experts here: a plan of any list is taken.
mfsdp_status_t route_plan_args(int64_t tokens, int64_t k, int64_t n) {
  if (tokens < 0 || n < 1 || k < 1)
    return fail(MFSDP_ERR_INVALID_ARGUMENT, "tokens=%lld experts=%lld k=%lld", (long long)tokens, (long long)n, (long long)k);
  if (n > kRouteExpertsMax || k > kRouteChosenMax || tokens > kRouteSlotsMax || tokens * k > kRouteSlotsMax) return too_large();
  return MFSDP_OK;
}

mfsdp_status_t route_plan_impl(const int32_t* experts, int64_t tokens, int64_t k, int64_t n, int32_t* offsets,
                               int32_t* place, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  g_last_error.clear();
  mfsdp_status_t st = route_plan_args(tokens, k, n);
  if (st != MFSDP_OK) return st;
  const int64_t slots = tokens * k;
  if (!offsets || (slots > 0 && (!experts || !place))) return null_pointer();
  if (!aligned(offsets, 4) || !aligned(experts, 4) || !aligned(place, 4)) return misaligned();
  const RoutePlanSizes p = route_plan_sizes(slots, n);
  st = check_workspace(workspace, workspace_bytes, p.bytes);
  if (st != MFSDP_OK) return st;
  Buffers b;
  b.bytes(offsets, static_cast<size_t>(n + 1) * 4, "offsets");
  b.bytes(place, static_cast<size_t>(slots) * 4, "place");
  if (p.bytes) b.bytes(workspace, p.bytes, "workspace");
  b.outputs_end();
  b.bytes(experts, static_cast<size_t>(slots) * 4, "experts");
  st = b.check();
  if (st != MFSDP_OK) return st;
  PlanArgs a{};
  a.chosen = experts;
  a.offsets = offsets;
  a.place = place;
  a.hist = static_cast<uint32_t*>(workspace);
  a.n = static_cast<int32_t>(slots);
  a.experts = static_cast<int32_t>(n);
  a.pitch = static_cast<int32_t>(round_up(n, 4));
  while ((int64_t(1) << a.bits) < n) ++a.bits;
  a.per_block = p.per_block;
  const dim3 grid(static_cast<unsigned>(p.blocks)), wg(kPlanThreads);
  hipError_t e;
  if (p.blocks == 1) {
    e = launch(MFSDP_KERNEL_ROUTE, stream, [&] { plan_small_kernel<<<grid, wg, 0, stream>>>(a); });
  } else {
    e = launch(MFSDP_KERNEL_ROUTE, stream, [&] { plan_hist_kernel<<<grid, wg, 0, stream>>>(a); });
    if (e == hipSuccess)
      e = launch(MFSDP_KERNEL_ROUTE, stream, [&] { plan_place_kernel<<<grid, wg, 0, stream>>>(a); });
  }
  return launched(e, "routing plan");
}

mfsdp_status_t route_balance_impl(float* bias, const void* counts, int count_bytes, int64_t n, float rate, hipStream_t stream) {
  g_last_error.clear();
  if (count_bytes != 4 && count_bytes != 8)
    return fail(MFSDP_ERR_UNSUPPORTED, "counts of %d bytes: 4 or 8 are taken", count_bytes);
  if (n < 1 || !finite(rate)) return fail(MFSDP_ERR_INVALID_ARGUMENT, "experts=%lld, or a non-finite rate", (long long)n);
  if (n > kRouteExpertsMax) return too_large();
  if (!bias || !counts) return null_pointer();
  if (!aligned(bias, 4) || !aligned(counts, count_bytes)) return misaligned();
  Buffers b;
  b.bytes(bias, static_cast<size_t>(n) * 4, "bias");
  b.outputs_end();
  b.bytes(counts, static_cast<size_t>(n) * count_bytes, "counts");
  const mfsdp_status_t st = b.check();
  if (st != MFSDP_OK) return st;
  BalanceArgs a{bias, counts, static_cast<int32_t>(n), count_bytes == 8, rate};
  const hipError_t e = launch(MFSDP_KERNEL_ROUTE, stream, [&] { route_balance_kernel<<<dim3(1), dim3(256), 0, stream>>>(a); });
  return launched(e, "routing balance");
}

// ---------------------------------------------------------------------------
// Exchange of rows
// ---------------------------------------------------------------------------
enum ExchangeMode { kDispatch, kCombine, kCombineGrad };

mfsdp_status_t exchange_impl(ExchangeMode mode, const void* x, int64_t ldx, const void* dy, int64_t ldy,
                             const int32_t* place, const float* weights, int64_t tokens, int64_t k, int64_t rows,
                             int64_t d, mfsdp_dtype_t dtype, float beta, void* out, int64_t ldo, float* dw,
                             hipStream_t stream) {
  g_last_error.clear();
  if (!known_dtype(dtype)) return bad_dtype(dtype);
  if (tokens < 0 || k < 1 || rows < 0 || d < 1)
    return fail(MFSDP_ERR_INVALID_ARGUMENT, "tokens=%lld k=%lld rows=%lld d=%lld", (long long)tokens, (long long)k,
                (long long)rows, (long long)d);
  if (ldx < d || ldo < d || (mode == kCombineGrad && ldy < d))
    return fail(MFSDP_ERR_INVALID_ARGUMENT, "a row stride is smaller than the row");
  if (!finite(beta)) return fail(MFSDP_ERR_INVALID_ARGUMENT, "non-finite beta");
  if (tokens > kRouteSlotsMax || k > kRouteChosenMax || tokens * k > kRouteSlotsMax || rows > kGroupRowsMax ||
      d > kGroupDimMax || ldx > kGroupDimMax || ldo > kGroupDimMax || ldy > kGroupDimMax)
    return too_large();
  if (tokens == 0) return MFSDP_OK;
  const bool grad = mode == kCombineGrad;
  const void* token_rows = mode == kDispatch ? x : grad ? dy : out;      // tokens x d
  const void* expert_rows = mode == kDispatch ? out : x;                  // rows x d
  if (!place || !token_rows || (rows > 0 && (!expert_rows || !out)) || (grad && (!weights || !dw))) return null_pointer();
  const size_t es = elem_size(dtype);
  if (!aligned(x, es) || !aligned(out, es) || !aligned(dy, es) || !aligned(place, 4) || !aligned(weights, 4) || !aligned(dw, 4))
    return misaligned();
  const size_t slots = static_cast<size_t>(tokens * k);
  Buffers b;
  b.rows(out, mode == kCombine ? tokens : rows, d, ldo, es, mode == kDispatch ? "out" : grad ? "dh" : "y");
  if (grad) b.bytes(dw, slots * 4, "dweights");
  b.outputs_end();
  b.rows(x, mode == kDispatch ? tokens : rows, d, ldx, es, mode == kDispatch ? "x" : "h");
  if (grad) b.rows(dy, tokens, d, ldy, es, "dy");
  b.bytes(place, slots * 4, "place");
  b.bytes(weights, slots * 4, "weights");
  const mfsdp_status_t st = b.check();
  if (st != MFSDP_OK) return st;
  ExchangeArgs a{};
  a.ldx = ldx;
  a.ldy = ldy;
  a.ldo = ldo;
  a.rows = static_cast<int32_t>(rows);
  a.k = static_cast<int32_t>(k);
  a.d = static_cast<int32_t>(d);
  a.beta = beta;
  const int64_t units = ceil_div(d, 16 / static_cast<int64_t>(es));
  if (grad) {     // whole waves
    a.chunks = 1;
    a.tpt = 64;
    while (a.tpt < 256 && a.tpt * 2 < units) a.tpt *= 2;
  } else {
    a.chunks = static_cast<int32_t>(ceil_div(units, 256));
    a.tpt = static_cast<int32_t>(ceil_div(units, a.chunks));
  }
  // more than the 256 MB of the last-level cache, and lines that rows do not share
  const bool streamed_rows = std::min(rows, tokens * k) * d * static_cast<int64_t>(es) > (int64_t(1) << 28) &&
                             aligned(x, 64) && ldx * es % 64 == 0;
  const int64_t per = 256 / a.tpt, most = kBlocksMax / a.chunks * per;    // tokens of one launch
  hipError_t e = hipSuccess;
  for (int64_t t0 = 0; t0 < tokens && e == hipSuccess; t0 += most) {
    const size_t slot = static_cast<size_t>(t0 * k);
    auto at = [&](const void* p, int64_t ld) { return p ? static_cast<const char*>(p) + t0 * ld * static_cast<int64_t>(es) : nullptr; };
    a.x = mode == kDispatch ? at(x, ldx) : x;
    a.dy = at(dy, ldy);
    a.out = mode == kCombine ? const_cast<char*>(at(out, ldo)) : out;
    a.place = place + slot;
    a.weights = weights ? weights + slot : nullptr;
    a.dw = dw ? dw + slot : nullptr;
    a.tokens = static_cast<int32_t>(std::min(most, tokens - t0));
    const dim3 grid(static_cast<unsigned>(ceil_div(a.tokens, per) * a.chunks)), wg(256);
    e = launch(MFSDP_KERNEL_EXCHANGE, stream, [&] {
      auto go = [&](auto elem, auto streamed) {
        using E = decltype(elem);
        constexpr bool STREAM = decltype(streamed)::value;
        if (mode == kDispatch) dispatch_kernel<E><<<grid, wg, 0, stream>>>(a);
        else if (mode == kCombine) combine_kernel<E, STREAM><<<grid, wg, 0, stream>>>(a);
        else combine_grad_kernel<E, STREAM><<<grid, wg, 0, stream>>>(a);
      };
      auto type = [&](auto streamed) { dtype == MFSDP_DTYPE_BF16 ? go(ElemBF16{}, streamed) : go(ElemF32{}, streamed); };
      if (mode != kDispatch && streamed_rows) type(std::integral_constant<bool, true>{});
      else type(std::integral_constant<bool, false>{});
    });
  }
  return launched(e, "exchange");
}

// ---------------------------------------------------------------------------
// Layer norm
// ---------------------------------------------------------------------------
struct NormPlan {
  int upt, threads;     // units of 16 bytes per thread (0: read again), threads of a workgroup
  int lanes;            // of a wave per row, 0: a workgroup
  bool full;            // the threads' units are exactly the row
  int64_t groups;       // waves or workgroups that the rows are dealt to
};

NormPlan norm_plan(int64_t rows, int64_t d, bool bf, bool grad) {
  const int64_t v = bf ? 8 : 4, units = ceil_div(d, v);
  NormPlan p{};
  if (units <= 2 * 64) {
    p.upt = units <= 64 ? 1 : 2;
    p.lanes = units <= 8 ? 8 : units <= 16 ? 16 : units <= 32 ? 32 : 64;
    p.threads = 256;
  } else {
    p.upt = units <= 2 * kNormThreadsMax ? 2 : units <= 4 * kNormThreadsMax ? 4 : 0;
    p.threads = p.upt ? static_cast<int>(round_up(ceil_div(units, p.upt), 64)) : kNormThreadsMax;
  }
  p.full = p.upt && d == (p.lanes ? p.lanes : p.threads) * p.upt * v;
  // The gradient: as many workgroups per CU as make eight waves.  Fewer leave loads
  // and additions uncovered, more add partial sums: 16384 x 5120 bf16 121, 98 and
  // 115 us with one, two and three; 16384 x 4096 96, 72 and 73; 32768 x 2048 98, 72
  // and 80 with two, four and eight; 4096 x 16384 82 and 97 with one and two.
  // Wide rows: some thousand workgroups of 256 units of columns.
  if (!p.upt) p.groups = std::max<int64_t>(16, 1024 / ceil_div(units, 256));
  else if (p.lanes || !grad) p.groups = 2048;
  else p.groups = 256 * ceil_div(8, p.threads / 64);
  if (p.lanes) {    // waves, of eight rounds at least: 32768 x 128 bf16 15 us with 1024, 19 with 2048; 524288 x 128 113 and 84
    const int64_t rounds = ceil_div(rows, 64 / p.lanes);
    p.groups = std::min<int64_t>(grad ? ceil_div(rounds, 8) : rounds, p.groups);
  } else {
    p.groups = std::min(rows, p.groups);
  }
  return p;
}

mfsdp_status_t norm_sizes(int64_t rows, int64_t d, mfsdp_dtype_t dtype) {
  if (!known_dtype(dtype)) return bad_dtype(dtype);
  if (rows < 0 || d < 1) return fail(MFSDP_ERR_INVALID_ARGUMENT, "rows=%lld d=%lld", (long long)rows, (long long)d);
  if (rows > kGroupRowsMax || d > kGroupDimMax) return too_large();
  return MFSDP_OK;
}

size_t norm_part_bytes(const NormPlan& p, int64_t d, bool bias) {
  return align_up(static_cast<size_t>(p.groups) * (bias ? 2 : 1) * d * 4, kWsAlign);
}

size_t norm_workspace(const NormPlan& p, int64_t rows, int64_t d, bool bias) {
  return norm_part_bytes(p, d, bias) + (p.upt ? 0 : static_cast<size_t>(rows) * 8);
}

template <class E, int UPT, int L, bool FULL>
void launch_norm(const NormArgs& a, const NormPlan& p, bool grad, hipStream_t stream) {
  const dim3 grid(static_cast<unsigned>(L ? ceil_div(p.groups, 4) : p.groups)), wg(static_cast<unsigned>(p.threads));
  if (grad) layer_norm_grad_kernel<E, UPT, L, FULL><<<grid, wg, 0, stream>>>(a);
  else layer_norm_kernel<E, UPT, L, FULL><<<grid, wg, 0, stream>>>(a);
}

template <class E>
hipError_t launch_norm(const NormArgs& a, const NormPlan& p, bool grad, hipStream_t stream) {
  if (p.upt == 0) {
    // under 2^32 threads of a launch; a workgroup takes further rows in turn
    const dim3 grid(static_cast<unsigned>(std::min<int64_t>(a.rows, int64_t(1) << 22))), wg(kNormThreadsMax);
    hipError_t e = launch(MFSDP_KERNEL_LAYER_NORM, stream, [&] {
      if (grad) layer_norm_wide_kernel<E, true><<<grid, wg, 0, stream>>>(a);
      else layer_norm_wide_kernel<E, false><<<grid, wg, 0, stream>>>(a);
    });
    if (e != hipSuccess || !grad) return e;
    const int blocks = static_cast<int>(ceil_div(a.d, 256 * E::kVec));
    const dim3 columns(static_cast<unsigned>(p.groups * blocks));
    return launch(MFSDP_KERNEL_LAYER_NORM, stream,
                  [&] { layer_norm_columns_kernel<E><<<columns, dim3(256), 0, stream>>>(a, blocks); });
  }
  return launch(MFSDP_KERNEL_LAYER_NORM, stream, [&] {
    auto go = [&](auto upt, auto lanes) {
      constexpr int UPT = decltype(upt)::value, L = decltype(lanes)::value;
      if (p.full) launch_norm<E, UPT, L, true>(a, p, grad, stream);
      else launch_norm<E, UPT, L, false>(a, p, grad, stream);
    };
    using std::integral_constant;
    const integral_constant<int, 0> all;
    const integral_constant<int, 1> one;
    const integral_constant<int, 2> two;
    switch (p.lanes) {
      case 0: p.upt == 2 ? go(two, all) : go(integral_constant<int, 4>{}, all); break;
      case 8: go(one, integral_constant<int, 8>{}); break;
      case 16: go(one, integral_constant<int, 16>{}); break;
      case 32: go(one, integral_constant<int, 32>{}); break;
      default: p.upt == 1 ? go(one, integral_constant<int, 64>{}) : go(two, integral_constant<int, 64>{});
    }
  });
}

// grad: dy is given, out is dx.
mfsdp_status_t norm_impl(bool grad, const void* dy, int64_t ldy, const void* x, int64_t ldx, const void* weight,
                         const void* bias, mfsdp_dtype_t weight_dtype, int64_t rows, int64_t d, mfsdp_dtype_t dtype,
                         int centered, float eps, float beta, void* out, int64_t ldo, float* dweight, float* dbias,
                         void* workspace, size_t workspace_bytes, hipStream_t stream) {
  g_last_error.clear();
  mfsdp_status_t st = norm_sizes(rows, d, dtype);
  if (st != MFSDP_OK) return st;
  if (!known_dtype(weight_dtype)) return bad_dtype(weight_dtype);
  if (ldx < d || ldo < d || (grad && ldy < d))
    return fail(MFSDP_ERR_INVALID_ARGUMENT, "a row stride is smaller than the row");
  if (ldx > kGroupDimMax || ldo > kGroupDimMax || ldy > kGroupDimMax) return too_large();
  if (!finite(eps) || eps < 0.f || !finite(beta)) return fail(MFSDP_ERR_INVALID_ARGUMENT, "eps must be finite and >= 0, beta finite");
  if (rows == 0 && !grad) return MFSDP_OK;
  if (!weight || (grad && !dweight) || (rows > 0 && (!x || !out || (grad && !dy)))) return null_pointer();
  const size_t es = elem_size(dtype), ew = elem_size(weight_dtype);
  if (!aligned(x, es) || !aligned(dy, es) || !aligned(out, es) || !aligned(weight, ew) || !aligned(bias, ew) ||
      !aligned(dweight, 4) || !aligned(dbias, 4))
    return misaligned();
  const bool bf = dtype == MFSDP_DTYPE_BF16;
  const NormPlan p = norm_plan(rows, d, bf, grad);
  const size_t need = grad ? norm_workspace(p, rows, d, dbias != nullptr) : 0;
  st = check_workspace(workspace, workspace_bytes, need);
  if (st != MFSDP_OK) return st;
  Buffers b;
  b.rows(out, rows, d, ldo, es, grad ? "dx" : "y");
  if (grad) {
    b.bytes(dweight, static_cast<size_t>(d) * 4, "dweight");
    b.bytes(dbias, static_cast<size_t>(d) * 4, "dbias");
    b.bytes(workspace, need, "workspace");
  }
  b.outputs_end();
  b.rows(x, rows, d, ldx, es, "x");
  if (grad) b.rows(dy, rows, d, ldy, es, "dy");
  b.bytes(weight, static_cast<size_t>(d) * ew, "weight");
  b.bytes(bias, static_cast<size_t>(d) * ew, "bias");
  st = b.check();
  if (st != MFSDP_OK) return st;
  NormArgs a{};
  a.x = x;
  a.dy = dy;
  a.w = weight;
  a.b = bias;
  a.out = out;
  a.part = static_cast<float*>(workspace);
  a.stats = a.part ? a.part + norm_part_bytes(p, d, dbias != nullptr) / 4 : nullptr;
  a.dw = dweight;
  a.db = dbias;
  a.ldx = ldx;
  a.ldy = ldy;
  a.ldo = ldo;
  a.rows = static_cast<int32_t>(rows);
  a.d = static_cast<int32_t>(d);
  a.centered = centered != 0;
  a.w_bf16 = weight_dtype == MFSDP_DTYPE_BF16;
  a.groups = static_cast<int32_t>(p.groups);
  a.eps = eps;
  a.beta = beta;
  hipError_t e = hipSuccess;
  if (rows > 0) e = bf ? launch_norm<ElemBF16>(a, p, grad, stream) : launch_norm<ElemF32>(a, p, grad, stream);
  if (grad && e == hipSuccess) {
    const dim3 grid(static_cast<unsigned>(ceil_div(d, 64) * (dbias ? 2 : 1)));
    e = launch(MFSDP_KERNEL_LAYER_NORM, stream, [&] { layer_norm_sum_kernel<<<grid, dim3(64 * kNormSlices), 0, stream>>>(a); });
  }
  return launched(e, "layer norm");
}

// ---------------------------------------------------------------------------
// Products in 8-bit floats
// ---------------------------------------------------------------------------
constexpr int64_t kScaledDimMax = kGroupDimMax - kScaledBlock;    // rows of codes are filled up

mfsdp_status_t scaled_quantize_impl(const void* x, int64_t ld, int64_t rows, int64_t k, mfsdp_dtype_t dtype,
                                    uint8_t* codes, uint8_t* scales, hipStream_t stream) {
  g_last_error.clear();
  if (!known_dtype(dtype)) return bad_dtype(dtype);
  if (rows < 0 || k < 1 || ld < k)
    return fail(MFSDP_ERR_INVALID_ARGUMENT, "rows=%lld k=%lld ld=%lld", (long long)rows, (long long)k, (long long)ld);
  if (rows > kGroupRowsMax || k > kScaledDimMax || ld > kGroupDimMax) return too_large();
  if (rows == 0) return MFSDP_OK;
  if (!x || !codes || !scales) return null_pointer();
  const size_t es = elem_size(dtype);
  if (!aligned(x, es)) return misaligned();
  if (!aligned(codes, 16)) return fail(MFSDP_ERR_INVALID_ARGUMENT, "codes must be 16-byte aligned");
  const int64_t nb = ceil_div(k, kScaledBlock);
  Buffers b;
  b.bytes(codes, static_cast<size_t>(rows) * nb * kScaledBlock, "codes");
  b.bytes(scales, static_cast<size_t>(rows) * nb, "scales");
  b.outputs_end();
  b.rows(x, rows, k, ld, es, "x");
  const mfsdp_status_t st = b.check();
  if (st != MFSDP_OK) return st;
  ScaledQuantArgs a{};
  a.ld = ld;
  a.k = static_cast<int32_t>(k);
  a.nb = static_cast<int32_t>(nb);
  const int64_t most = kBlocksMax * 16 * kScaledUnits / nb;   // rows of one launch
  hipError_t e = hipSuccess;
  for (int64_t r = 0; r < rows && e == hipSuccess; r += most) {
    a.x = static_cast<const char*>(x) + r * ld * static_cast<int64_t>(es);
    a.codes = codes + r * nb * kScaledBlock;
    a.scales = scales + r * nb;
    a.units = static_cast<uint32_t>(std::min(most, rows - r) * nb);
    const dim3 grid(static_cast<unsigned>(ceil_div(a.units, 16 * kScaledUnits))), wg(256);
    e = launch(MFSDP_KERNEL_SCALED, stream, [&] {
      if (dtype == MFSDP_DTYPE_BF16) scaled_quantize_kernel<ElemBF16><<<grid, wg, 0, stream>>>(a);
      else scaled_quantize_kernel<ElemF32><<<grid, wg, 0, stream>>>(a);
    });
  }
  return launched(e, "8-bit float");
}

mfsdp_status_t scaled_weight_impl(const void* w, int64_t experts, int64_t n, int64_t k, mfsdp_dtype_t dtype,
                                  uint8_t* codes, uint8_t* scales, uint8_t* tcodes, uint8_t* tscales, hipStream_t stream) {
  g_last_error.clear();
  if (!known_dtype(dtype)) return bad_dtype(dtype);
  if (experts < 0 || n < 1 || k < 1)
    return fail(MFSDP_ERR_INVALID_ARGUMENT, "experts=%lld n=%lld k=%lld", (long long)experts, (long long)n, (long long)k);
  if (experts > kGroupExpertsMax || n > kScaledDimMax || k > kScaledDimMax) return too_large();
  if (!codes != !scales || !tcodes != !tscales || (!codes && !tcodes))
    return fail(MFSDP_ERR_INVALID_ARGUMENT, "codes and scales come together, of one copy or both");
  if (experts == 0) return MFSDP_OK;
  if (!w) return null_pointer();
  const size_t es = elem_size(dtype);
  if (!aligned(w, es)) return misaligned();
  if (!aligned(codes, 16) || !aligned(tcodes, 16)) return fail(MFSDP_ERR_INVALID_ARGUMENT, "codes must be 16-byte aligned");
  const int64_t nb = ceil_div(n, kScaledBlock), kb = ceil_div(k, kScaledBlock);
  const size_t blocks = static_cast<size_t>(experts) * nb * kb;
  Buffers b;
  b.bytes(codes, static_cast<size_t>(experts) * n * kb * kScaledBlock, "codes");
  b.bytes(scales, blocks, "scales");
  b.bytes(tcodes, static_cast<size_t>(experts) * k * nb * kScaledBlock, "transposed codes");
  b.bytes(tscales, blocks, "transposed scales");
  b.outputs_end();
  b.bytes(w, static_cast<size_t>(experts) * n * k * es, "weight");
  const mfsdp_status_t st = b.check();
  if (st != MFSDP_OK) return st;
  ScaledWeightArgs a{};
  a.w = w;
  a.codes = codes;
  a.scales = scales;
  a.tcodes = tcodes;
  a.tscales = tscales;
  a.n = static_cast<int32_t>(n);
  a.k = static_cast<int32_t>(k);
  a.nb = static_cast<int32_t>(nb);
  a.kb = static_cast<int32_t>(kb);
  hipError_t e = hipSuccess;
  a.tiles = static_cast<int64_t>(blocks);
  const int64_t most = kBlocksMax / kScaledBlocks * kScaledBlocks;    // blocks of one launch (under 2^32 threads)
  for (int64_t t = 0; t < a.tiles && e == hipSuccess; t += most) {
    a.tile0 = t;
    const dim3 grid(static_cast<unsigned>(ceil_div(std::min(most, a.tiles - t), kScaledBlocks))), wg(256 * kScaledBlocks);
    e = launch(MFSDP_KERNEL_SCALED, stream, [&] {
      if (dtype == MFSDP_DTYPE_BF16) scaled_weight_kernel<ElemBF16><<<grid, wg, 0, stream>>>(a);
      else scaled_weight_kernel<ElemF32><<<grid, wg, 0, stream>>>(a);
    });
  }
  return launched(e, "8-bit float matrices");
}

// Tiles.  scaled_kernel chooses among them; the times at its rule are in us, of
// experts x rows x n x k.
using ScaledLarge = ScaledTile<256, 256, 2, 4, 2, 2>;
using ScaledPair = ScaledTile<128, 128, 2, 2, 2, 2>;         // two workgroups per CU
using ScaledRows = ScaledTile<32, 64, 1, 2, 4, 3, 4, 4>;     // two workgroups per CU
using ScaledFew = ScaledTile<32, 32, 1, 1, 4, 3, 4, 4>;

template <class C>
hipError_t launch_scaled(const ScaledArgs& a, int64_t workgroups, hipStream_t stream) {
  const dim3 grid(static_cast<unsigned>(workgroups));
  return launch(MFSDP_KERNEL_SCALED, stream, [&] { scaled_tile_kernel<C><<<grid, dim3(C::THREADS), 0, stream>>>(a); });
}

enum ScaledKernel { kScaledLarge, kScaledPair, kScaledRows, kScaledFew };

// Row tiles are estimated from the mean of the experts that have rows.
ScaledKernel scaled_kernel(int64_t experts, int64_t rows, int64_t n, int64_t k) {
  const int64_t used = std::min(experts, rows), per = rows / used;
  auto tiles = [&](int64_t bp, int64_t bq) {
    return static_cast<double>(std::max(used, rows / bp + used / 2) * ceil_div(n, bq));
  };
  // One row tile of 32 x 64 per expert reads each weight once.  Up to three tiles
  // per CU: 1 x 64 x 14336 x 4096 21 against 34 us with 128 x 128, 8 x 128 x 4096 x
  // 4096 30 and 39.  More of them where few rows wait for long rows of weights: 8
  // x 128 x 14336 x 4096 90 and 113, 256 x 256 x 512 x 1536 30 and 36; but 32 x 256
  // x 2048 x 2048 32 and 28.  32 x 32 where there are few: 1 x 16 x 4096 x 4096 10.3
  // against 11.5.
  const double narrow = per < 32 ? static_cast<double>(used * ceil_div(n, 64)) : tiles(32, 64);
  if (narrow <= 768 || (per < 32 && (per <= 4 || k >= 4096))) return narrow <= 128 ? kScaledFew : kScaledRows;
  // Rounds of the 256 CUs, in the time of one of 256 x 256: one of two 128 x 128
  // per CU takes 0.72, and half of a further one overlaps (1 x 2048 x 4096 x 4096 47
  // and 36, 1 x 1024 x 14336 x 4096 53 and 65, 32 x 6144 x 2048 x 2048 53 and 39).
  // Few rows fill large tiles unevenly: 256 x 32771 x 512 x 1536 61 and 51 with
  // segments that differ by half, 48 and 51 with nearly equal ones.
  const double large = std::ceil(tiles(256, 256) / 256) * (per < 256 ? 1.3 : 1.0);
  const double pairs = tiles(128, 128) / 512, small = 0.72 * (pairs <= 1 ? 1 : pairs + 0.45);
  if (large > small) return kScaledPair;
  return kScaledLarge;
}

GroupShape scaled_shape(ScaledKernel u) {
  switch (u) {
    case kScaledLarge: return shape_of<ScaledLarge>(true);
    case kScaledPair: return shape_of<ScaledPair>(true);
    case kScaledRows: return shape_of<ScaledRows>(true);
    case kScaledFew: break;
  }
  return shape_of<ScaledFew>(true);
}

// The kernel that a product's sizes take and its workgroups (0: no launch), or why
// they are refused.
mfsdp_status_t scaled_choose(int64_t experts, int64_t rows, int64_t n, int64_t k, ScaledKernel* use, int64_t* workgroups) {
  *workgroups = 0;
  const mfsdp_status_t st = grouped_sizes(experts, rows, n, k, MFSDP_DTYPE_BF16);
  if (st != MFSDP_OK) return st;
  if (n > kScaledDimMax || k > kScaledDimMax) return too_large();
  if (experts == 0 || rows == 0) return MFSDP_OK;
  *use = scaled_kernel(experts, rows, n, round_up(k, kScaledBlock));
  const GroupShape s = scaled_shape(*use);
  const int64_t tiles = group_tiles_max(rows, experts, s.rows) * ceil_div(n, s.cols);
  if (tiles > kGroupBlocksMax) return fail(MFSDP_ERR_UNSUPPORTED, "too many tiles");
  *workgroups = tiles;
  return MFSDP_OK;
}

mfsdp_status_t scaled_linear_impl(const uint8_t* codes, const uint8_t* scales, const uint8_t* wcodes,
                                  const uint8_t* wscales, const int32_t* offsets, int64_t experts, int64_t rows,
                                  int64_t n, int64_t k, void* y, int64_t ldy, hipStream_t stream) {
  g_last_error.clear();
  ScaledKernel use{};
  int64_t workgroups;
  mfsdp_status_t st = scaled_choose(experts, rows, n, k, &use, &workgroups);
  if (st != MFSDP_OK) return st;
  if (ldy > kGroupDimMax) return too_large();
  if (ldy < n) return fail(MFSDP_ERR_INVALID_ARGUMENT, "a row stride is smaller than the row");
  if (workgroups == 0) return MFSDP_OK;
  if (!codes || !scales || !wcodes || !wscales || !offsets || !y) return null_pointer();
  if (!aligned(y, 2) || !aligned(offsets, 4)) return misaligned();
  if (!aligned(codes, 16) || !aligned(wcodes, 16)) return fail(MFSDP_ERR_INVALID_ARGUMENT, "codes must be 16-byte aligned");
  const int64_t nb = ceil_div(n, kScaledBlock), kb = ceil_div(k, kScaledBlock), depth = kb * kScaledBlock;
  Buffers b;
  b.rows(y, rows, n, ldy, 2, "y");
  b.outputs_end();
  b.bytes(codes, static_cast<size_t>(rows) * depth, "codes");
  b.bytes(scales, static_cast<size_t>(rows) * kb, "scales");
  b.bytes(wcodes, static_cast<size_t>(experts) * n * depth, "weight codes");
  b.bytes(wscales, static_cast<size_t>(experts) * nb * kb, "weight scales");
  b.bytes(offsets, static_cast<size_t>(experts + 1) * 4, "offsets");
  st = b.check();
  if (st != MFSDP_OK) return st;
  ScaledArgs a{};
  a.g.p = codes;
  a.g.q = wcodes;
  a.g.out = y;
  a.g.off = offsets;
  a.g.ldp = a.g.ldq = depth;
  a.g.ldo = ldy;
  a.g.experts = static_cast<int32_t>(experts);
  a.g.rows = static_cast<int32_t>(rows);
  a.g.n = static_cast<int32_t>(n);
  a.g.k = static_cast<int32_t>(depth);
  a.ps = scales;
  a.qs = wscales;
  a.kb = static_cast<int32_t>(kb);
  a.nb = static_cast<int32_t>(nb);
  a.g.stream = aligned(y, 128) && ldy * 2 % 128 == 0;
  hipError_t e = hipErrorInvalidValue;
  switch (use) {
    case kScaledLarge: e = launch_scaled<ScaledLarge>(a, workgroups, stream); break;
    case kScaledPair: e = launch_scaled<ScaledPair>(a, workgroups, stream); break;
    case kScaledRows: e = launch_scaled<ScaledRows>(a, workgroups, stream); break;
    case kScaledFew: e = launch_scaled<ScaledFew>(a, workgroups, stream); break;
  }
  return launched(e, "8-bit float product");
}

}  // namespace

extern "C" {

mfsdp_status_t mfsdp_route(const void* logits, int64_t ld_logits, const float* bias, const uint8_t* mask,
                           int64_t tokens, int64_t n_experts, int64_t k, mfsdp_dtype_t dtype,
                           mfsdp_route_score_t scores, int64_t groups, int64_t top_groups, int renormalize,
                           float scale, int32_t* experts, float* weights, hipStream_t stream) {
  return guarded([&] {
    return route_impl(logits, ld_logits, bias, mask, tokens, n_experts, k, dtype, scores, groups, top_groups,
                      renormalize, scale, experts, weights, stream);
  });
}

mfsdp_status_t mfsdp_route_grad(const float* dweights, const void* logits, int64_t ld_logits, const int32_t* experts,
                                int64_t tokens, int64_t n_experts, int64_t k, mfsdp_dtype_t dtype,
                                mfsdp_route_score_t scores, int renormalize, float scale, void* dlogits,
                                int64_t ld_dlogits, hipStream_t stream) {
  return guarded([&] {
    return route_grad_impl(dweights, logits, ld_logits, experts, tokens, n_experts, k, dtype, scores, renormalize,
                           scale, dlogits, ld_dlogits, stream);
  });
}

mfsdp_status_t mfsdp_route_plan_workspace_size(int64_t tokens, int64_t k, int64_t n_experts, size_t* out_bytes) {
  return guarded([&]() -> mfsdp_status_t {
    g_last_error.clear();
    if (!out_bytes) return fail(MFSDP_ERR_INVALID_ARGUMENT, "out_bytes is null");
    const mfsdp_status_t st = route_plan_args(tokens, k, n_experts);
    if (st == MFSDP_OK) *out_bytes = route_plan_sizes(tokens * k, n_experts).bytes;
    return st;
  });
}

mfsdp_status_t mfsdp_route_plan(const int32_t* experts, int64_t tokens, int64_t k, int64_t n_experts,
                                int32_t* offsets, int32_t* place, void* workspace, size_t workspace_bytes,
                                hipStream_t stream) {
  return guarded([&] {
    return route_plan_impl(experts, tokens, k, n_experts, offsets, place, workspace, workspace_bytes, stream);
  });
}

mfsdp_status_t mfsdp_route_balance(float* bias, const void* counts, int count_bytes, int64_t n_experts, float rate,
                                   hipStream_t stream) {
  return guarded([&] { return route_balance_impl(bias, counts, count_bytes, n_experts, rate, stream); });
}

mfsdp_status_t mfsdp_route_dispatch(const void* x, int64_t ld_x, const int32_t* place, int64_t tokens, int64_t k,
                                    int64_t rows, int64_t d, mfsdp_dtype_t dtype, void* out, int64_t ld_out,
                                    hipStream_t stream) {
  return guarded([&] {
    return exchange_impl(kDispatch, x, ld_x, nullptr, 0, place, nullptr, tokens, k, rows, d, dtype, 0.f, out, ld_out,
                         nullptr, stream);
  });
}

mfsdp_status_t mfsdp_route_combine(const void* h, int64_t ld_h, const int32_t* place, const float* weights,
                                   int64_t tokens, int64_t k, int64_t rows, int64_t d, mfsdp_dtype_t dtype,
                                   float beta, void* y, int64_t ld_y, hipStream_t stream) {
  return guarded([&] {
    return exchange_impl(kCombine, h, ld_h, nullptr, 0, place, weights, tokens, k, rows, d, dtype, beta, y, ld_y,
                         nullptr, stream);
  });
}

mfsdp_status_t mfsdp_route_combine_grad(const void* dy, int64_t ld_dy, const void* h, int64_t ld_h,
                                        const int32_t* place, const float* weights, int64_t tokens, int64_t k,
                                        int64_t rows, int64_t d, mfsdp_dtype_t dtype, void* dh, int64_t ld_dh,
                                        float* dweights, hipStream_t stream) {
  return guarded([&] {
    return exchange_impl(kCombineGrad, h, ld_h, dy, ld_dy, place, weights, tokens, k, rows, d, dtype, 0.f, dh, ld_dh,
                         dweights, stream);
  });
}

mfsdp_status_t mfsdp_layer_norm(const void* x, int64_t ld_x, const void* weight, const void* bias,
                                mfsdp_dtype_t weight_dtype, int64_t rows, int64_t d, mfsdp_dtype_t dtype,
                                int centered, float eps, void* y, int64_t ld_y, hipStream_t stream) {
  return guarded([&] {
    return norm_impl(false, nullptr, 0, x, ld_x, weight, bias, weight_dtype, rows, d, dtype, centered, eps, 0.f, y,
                     ld_y, nullptr, nullptr, nullptr, 0, stream);
  });
}

mfsdp_status_t mfsdp_layer_norm_grad_workspace_size(int64_t rows, int64_t d, mfsdp_dtype_t dtype, int with_bias,
                                                    size_t* out_bytes) {
  return guarded([&]() -> mfsdp_status_t {
    g_last_error.clear();
    if (!out_bytes) return fail(MFSDP_ERR_INVALID_ARGUMENT, "out_bytes is null");
    const mfsdp_status_t st = norm_sizes(rows, d, dtype);
    if (st == MFSDP_OK) *out_bytes = rows ? norm_workspace(norm_plan(rows, d, dtype == MFSDP_DTYPE_BF16, true), rows, d, with_bias != 0) : 0;
    return st;
  });
}

mfsdp_status_t mfsdp_layer_norm_grad(const void* dy, int64_t ld_dy, const void* x, int64_t ld_x, const void* weight,
                                     mfsdp_dtype_t weight_dtype, int64_t rows, int64_t d, mfsdp_dtype_t dtype,
                                     int centered, float eps, float beta, void* dx, int64_t ld_dx, float* dweight,
                                     float* dbias, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  return guarded([&] {
    return norm_impl(true, dy, ld_dy, x, ld_x, weight, nullptr, weight_dtype, rows, d, dtype, centered, eps, beta, dx,
                     ld_dx, dweight, dbias, workspace, workspace_bytes, stream);
  });
}

mfsdp_status_t mfsdp_scaled_quantize(const void* x, int64_t ld_x, int64_t rows, int64_t k, mfsdp_dtype_t dtype,
                                     uint8_t* codes, uint8_t* scales, hipStream_t stream) {
  return guarded([&] { return scaled_quantize_impl(x, ld_x, rows, k, dtype, codes, scales, stream); });
}

mfsdp_status_t mfsdp_scaled_quantize_weight(const void* weight, int64_t n_experts, int64_t n, int64_t k,
                                            mfsdp_dtype_t dtype, uint8_t* codes, uint8_t* scales, uint8_t* tcodes,
                                            uint8_t* tscales, hipStream_t stream) {
  return guarded([&] {
    return scaled_weight_impl(weight, n_experts, n, k, dtype, codes, scales, tcodes, tscales, stream);
  });
}

mfsdp_status_t mfsdp_scaled_linear(const uint8_t* codes, const uint8_t* scales, const uint8_t* weight_codes,
                                   const uint8_t* weight_scales, const int32_t* offsets, int64_t n_experts,
                                   int64_t rows, int64_t n, int64_t k, void* y, int64_t ld_y, hipStream_t stream) {
  return guarded([&] {
    return scaled_linear_impl(codes, scales, weight_codes, weight_scales, offsets, n_experts, rows, n, k, y,
                              ld_y, stream);
  });
}

mfsdp_status_t mfsdp_scaled_linear_tile(int64_t n_experts, int64_t rows, int64_t n, int64_t k,
                                        mfsdp_grouped_tile_t* out) {
  return guarded([&]() -> mfsdp_status_t {
    g_last_error.clear();
    if (!out) return fail(MFSDP_ERR_INVALID_ARGUMENT, "out is null");
    ScaledKernel use{};
    int64_t workgroups;
    const mfsdp_status_t st = scaled_choose(n_experts, rows, n, k, &use, &workgroups);
    if (st != MFSDP_OK) return st;
    *out = mfsdp_grouped_tile_t{};
    if (workgroups == 0) return MFSDP_OK;   // no launch
    const GroupShape s = scaled_shape(use);
    out->rows = s.rows;
    out->cols = s.cols;
    out->threads = s.threads;
    out->wave_sets = s.wave_sets;
    out->lds_dma = 1;
    out->workgroups = workgroups;
    return MFSDP_OK;
  });
}

}  // extern "C"
