"""The gradient operators on the GPU against plain float64 forms (grads_ref.py,
where the bounds are derived): products grouped by expert with their gradients,
8-bit checkpoints, the embedding and its gradient, and a run of them together
with the Muon step and the AdamW tail.
"""

import numpy as np
import pytest
import torch

import matrix_optimizer_step_owner_amd as mf
import grads_ref as ref
import oracle
from gpu_helpers import ADAMW_TOL, f64 as np64, muon_hparams, rel

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
DEV = torch.device("cuda:0")
NAN = float("nan")


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def rand(shape, dtype, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std).to(dtype)


def strided(t, pad):
    """t on the GPU as columns of a wider matrix of NaN."""
    if pad == 0:
        return t.to(DEV)
    wide = torch.full((t.shape[0], t.shape[1] + 2 * pad), NAN, dtype=t.dtype, device=DEV)
    wide[:, pad:pad + t.shape[1]] = t.to(DEV)
    return wide[:, pad:pad + t.shape[1]]


def offsets_of(counts, lead=0):
    return torch.tensor(np.concatenate([[0], np.cumsum(counts)]) + lead, dtype=torch.int32)


# (rows of each expert, rows before the first, rows after the last)
ROUTES = {
    "one row": ([1], 0, 0),
    "one expert": ([300], 0, 0),
    "empty ones": ([0, 5, 0, 0, 64, 1, 0], 3, 2),
    "none": ([0, 0, 0], 2, 1),
    "two short": ([60, 60], 0, 0),
    "tiny": ([1, 2, 0, 1, 1, 3, 1, 0, 1], 0, 0),
    "mixed": ([33, 127, 0, 128, 129, 255, 256, 257, 31, 32], 0, 5),
    "skewed": ([1500, 3, 0, 40], 1, 0),
    "parts": ([1300, 0, 900, 37], 0, 3),           # weight gradients summed in parts
    "long one": ([5003], 2, 0),
    "five": ([300, 0, 70, 513, 40], 0, 0),
    "many": ([(7 * i * i) % 23 for i in range(200)], 0, 0),
}
# n, k, columns before and after each activation row (strides)
WIDTHS = {
    "whole": (256, 512, 0),
    "narrow": (64, 64, 8),
    "ragged": (328, 200, 16),
    "odd": (131, 77, 0),
    "odd stride": (96, 160, 3),
    "one": (1, 1, 0),
    "short": (8, 40, 0),
    "long": (40, 1032, 8),
    "big": (1496, 2000, 8),                        # several tiles each way
}
GROUPED = [("one row", "whole"), ("one expert", "whole"), ("empty ones", "ragged"), ("none", "whole"), ("tiny", "whole"),
           ("tiny", "odd"), ("mixed", "whole"), ("mixed", "ragged"), ("mixed", "odd"), ("mixed", "odd stride"), ("skewed", "ragged"),
           ("skewed", "long"), ("many", "narrow"), ("many", "odd"), ("empty ones", "one"), ("mixed", "short"), ("one row", "long"),
           ("tiny", "long"), ("parts", "whole"), ("parts", "narrow"), ("parts", "odd"), ("long one", "narrow"), ("long one", "ragged"),
           ("five", "big"), ("many", "ragged"), ("two short", "big"), ("parts", "ragged")]


def setup(route, width, dtype, seed=0):
    counts, lead, tail = ROUTES[route]
    n, k, pad = WIDTHS[width]
    rows = sum(counts) + lead + tail
    off = offsets_of(counts, lead)
    x, dy = rand((rows, k), dtype, seed), rand((rows, n), dtype, seed + 1)
    for t in (x, dy):       # rows of no expert must not be read
        t[:lead] = NAN
        t[rows - tail:] = NAN
    w = rand((len(counts), n, k), dtype, seed + 2, 0.05)
    return x, dy, w, off, n, k, pad


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("route,width", GROUPED)
def test_grouped_linear(route, width, dtype):
    x, _, w, off, n, k, pad = setup(route, width, dtype)
    out = strided(torch.full((x.shape[0], n), 7.0, dtype=dtype), pad)
    got = mf.grouped_linear(strided(x, pad), w.to(DEV), off.to(DEV), out=out)
    assert got is out
    y, mag, on = ref.linear(x, w, off)
    assert torch.equal(got[~on.to(DEV)], torch.full_like(got[~on.to(DEV)], 7.0)), "rows of no expert were written"
    assert ref.worst(got[on.to(DEV)], y[on], ref.half_step(dtype) * y[on].abs() + k * ref.U * mag[on]) <= 1.0
    if pad:   # what lies between the rows
        wide = out._base
        assert torch.isnan(wide[:, :pad]).all() and torch.isnan(wide[:, pad + n:]).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("route,width", GROUPED)
def test_grouped_dgrad(route, width, dtype):
    _, dy, w, off, n, k, pad = setup(route, width, dtype, 10)
    out = strided(torch.full((dy.shape[0], k), 7.0, dtype=dtype), pad)
    got = mf.grouped_linear_dgrad(strided(dy, pad), w.to(DEV), off.to(DEV), out=out)
    dx, mag, on = ref.dgrad(dy, w, off)
    assert torch.equal(got[~on.to(DEV)], torch.full_like(got[~on.to(DEV)], 7.0)), "rows of no expert were written"
    assert ref.worst(got[on.to(DEV)], dx[on], ref.half_step(dtype) * dx[on].abs() + n * ref.U * mag[on]) <= 1.0
    if pad:
        wide = out._base
        assert torch.isnan(wide[:, :pad]).all() and torch.isnan(wide[:, pad + k:]).all()


def wgrad_bound(dw, mag, terms, old, beta, out_dtype):
    """The sum's bound, one rounding of beta*old + sum in fp32 and one to the type."""
    return (ref.half_step(out_dtype) + ref.U) * (dw + beta * old).abs() + (terms[:, None, None] + 1) * ref.U * (mag + abs(beta) * old.abs())


@pytest.mark.parametrize("ckpt", [False, True])
@pytest.mark.parametrize("dtype,out_dtype", [(BF, BF), (BF, F32), (F32, F32)])
@pytest.mark.parametrize("route,width", GROUPED)
def test_grouped_wgrad(route, width, dtype, out_dtype, ckpt):
    x, dy, w, off, n, k, pad = setup(route, width, dtype, 20)
    if ckpt:
        codes, scales = ref.ckpt_quantize(x)
        x = torch.from_numpy(ref.ckpt_restore(codes, scales))
        codes, scales = torch.from_numpy(codes).to(DEV), torch.from_numpy(scales).to(DEV)
    dw, mag, terms = ref.wgrad(dy, x, off)
    for beta in (0.0, 1.0, -0.5):
        old = rand(w.shape, out_dtype, 30)
        grad = old.to(DEV) if beta else torch.full(w.shape, NAN, dtype=out_dtype, device=DEV)
        old = ref.f64(old) if beta else torch.zeros(w.shape, dtype=torch.float64)
        dyg = strided(dy, pad)
        if ckpt:
            got = mf.grouped_linear_wgrad_ckpt(dyg, codes, scales, off.to(DEV), grad, beta=beta)
        else:
            got = mf.grouped_linear_wgrad(dyg, strided(x, pad), off.to(DEV), grad, beta=beta)
        assert got is grad
        assert ref.worst(got, dw + beta * old, wgrad_bound(dw, mag, terms, old, beta, out_dtype)) <= 1.0


@pytest.mark.parametrize("dtype", [BF, F32])
def test_segments_do_not_touch(dtype):
    # infinities and NaN in one expert's rows and weights stay in its results
    counts = [40, 70, 90, 33]
    off = offsets_of(counts)
    n, k = 64, 128
    x, dy, w = rand((sum(counts), k), dtype, 1), rand((sum(counts), n), dtype, 2), rand((4, n, k), dtype, 3)
    clean = [mf.grouped_linear(x.to(DEV), w.to(DEV), off.to(DEV)), mf.grouped_linear_dgrad(dy.to(DEV), w.to(DEV), off.to(DEV)),
             mf.grouped_linear_wgrad(dy.to(DEV), x.to(DEV), off.to(DEV), torch.zeros(4, n, k, dtype=dtype, device=DEV))]
    xb, dyb, wb = x.clone(), dy.clone(), w.clone()
    xb[40:110], dyb[40:110], wb[1] = float("inf"), NAN, NAN
    bad = [mf.grouped_linear(xb.to(DEV), wb.to(DEV), off.to(DEV)), mf.grouped_linear_dgrad(dyb.to(DEV), wb.to(DEV), off.to(DEV)),
           mf.grouped_linear_wgrad(dyb.to(DEV), xb.to(DEV), off.to(DEV), torch.zeros(4, n, k, dtype=dtype, device=DEV))]
    for i in (0, 1):
        assert torch.equal(clean[i][:40], bad[i][:40]) and torch.equal(clean[i][110:], bad[i][110:])
        assert torch.isnan(bad[i][40:110]).all()
    others = [0, 2, 3]
    assert torch.equal(clean[2][others], bad[2][others]) and torch.isnan(bad[2][1]).all()


def test_wrong_offsets_stay_inside():
    # offsets outside [0, rows] are clamped and a decreasing pair is empty: the
    # rows that remain are right
    x, w = rand((50, 64), BF, 1).to(DEV), rand((4, 32, 64), BF, 2).to(DEV)
    off = torch.tensor([-5, 20, 10, 30, 1000], dtype=torch.int32, device=DEV)
    dy = rand((50, 32), BF, 3).to(DEV)
    grad = torch.full((4, 32, 64), NAN, dtype=F32, device=DEV)
    mf.grouped_linear_wgrad(dy, x, off, grad)
    for e, (lo, hi) in enumerate([(0, 20), (20, 20), (10, 30), (30, 50)]):
        want = ref.f64(dy[lo:hi]).t() @ ref.f64(x[lo:hi])
        mag = ref.f64(dy[lo:hi]).abs().t() @ ref.f64(x[lo:hi]).abs()
        assert ref.worst(grad[e], want, ref.half_step(F32) * want.abs() + 51 * ref.U * mag + 1e-300) <= 1.0


def test_disordered_offsets_end():
    # up and down again for every expert: far more tiles, and parts of the
    # weight gradient, than ordered offsets can give.  The calls return, what
    # lies behind the outputs stays as it was, and the next call is right.
    rows, n, k, experts = 3000, 64, 64, 40
    x, dy = rand((rows, k), BF, 1).to(DEV), rand((rows, n), BF, 2).to(DEV)
    w = rand((experts, n, k), BF, 3).to(DEV)
    off = torch.tensor([0, rows] * (experts // 2) + [0], dtype=torch.int32, device=DEV)
    outs = [torch.full((rows + 64, n), 7.0, dtype=BF, device=DEV), torch.full((rows + 64, k), 7.0, dtype=BF, device=DEV),
            torch.full((experts + 1, n, k), 7.0, device=DEV)]
    two = torch.tensor([0, rows, 0, rows], dtype=torch.int32, device=DEV)
    few = torch.full((4, n, k), 7.0, device=DEV)
    mf.grouped_linear(x, w, off, out=outs[0][:rows])
    mf.grouped_linear_dgrad(dy, w, off, out=outs[1][:rows])
    mf.grouped_linear_wgrad(dy, x, off, outs[2][:experts])
    mf.grouped_linear_wgrad(dy, x, two, few[:3])       # in parts
    torch.cuda.synchronize()
    assert all((o[rows:] == 7.0).all() for o in outs[:2]) and (outs[2][experts] == 7.0).all() and (few[3] == 7.0).all()
    good = offsets_of([rows // experts] * experts)
    y, mag, _ = ref.linear(x, w, good)
    assert ref.worst(mf.grouped_linear(x, w, good.to(DEV)), y, ref.half_step(BF) * y.abs() + k * ref.U * mag) <= 1.0


def test_no_rows():
    w, off = rand((3, 16, 24), BF, 1).to(DEV), torch.zeros(4, dtype=torch.int32, device=DEV)
    x, dy = torch.empty(0, 24, dtype=BF, device=DEV), torch.empty(0, 16, dtype=BF, device=DEV)
    assert mf.grouped_linear(x, w, off).shape == (0, 16) and mf.grouped_linear_dgrad(dy, w, off).shape == (0, 24)
    grad = torch.full((3, 16, 24), NAN, device=DEV)
    assert not mf.grouped_linear_wgrad(dy, x, off, grad).any()
    assert torch.equal(mf.grouped_linear_wgrad(dy, x, off, grad + 2.0, beta=0.5), torch.ones_like(grad))
    codes, scales = mf.ckpt_quantize(x)
    assert codes.shape == (0, 24) and scales.shape == (0, 1) and mf.ckpt_restore(codes, scales).shape == (0, 24)
    assert not mf.grouped_linear_wgrad_ckpt(dy, codes, scales, off, grad).any()


@pytest.mark.parametrize("dtype,k", [(BF, 4096), (BF, 4104), (F32, 4096)])
def test_large_weights_few_rows(dtype, k):
    # weights of 69 MB and more: more than the L2s hold, read by one tile column each
    n, counts = 2056, [1, 0, 2, 40, 1]
    off = offsets_of(counts)
    x, dy, w = rand((44, k), dtype, 1), rand((44, n), dtype, 2), rand((5, n, k), dtype, 3, 0.05)
    y, mag, _ = ref.linear(x, w, off)
    assert ref.worst(mf.grouped_linear(x.to(DEV), w.to(DEV), off.to(DEV)), y, ref.half_step(dtype) * y.abs() + k * ref.U * mag) <= 1.0
    dx, mag, _ = ref.dgrad(dy, w, off)
    assert ref.worst(mf.grouped_linear_dgrad(dy.to(DEV), w.to(DEV), off.to(DEV)), dx, ref.half_step(dtype) * dx.abs() + n * ref.U * mag) <= 1.0


def test_far_rows():
    # byte offsets of rows and weights past 32 bits: 80000 rows of 32768 bf16
    # values, the last few of them in use (rows behind the first 65536 start
    # past 4 GiB)
    rows, ld, n, k = 80000, 32768, 64, 128
    buf = torch.empty(rows, ld, dtype=BF, device=DEV)
    x, dy = buf[:, :k], buf[:, k:k + n]
    xs, dys = rand((500, k), BF, 1), rand((500, n), BF, 2)
    x[-500:], dy[-500:] = xs.to(DEV), dys.to(DEV)
    off = torch.tensor([rows - 500, rows - 300, rows], dtype=torch.int32)
    small = off - (rows - 500)
    w = rand((2, n, k), BF, 3)
    out = buf[:, 1024:1024 + n]
    mf.grouped_linear(x, w.to(DEV), off.to(DEV), out=out)
    y, mag, _ = ref.linear(xs, w, small)
    assert ref.worst(out[-500:], y, ref.half_step(BF) * y.abs() + k * ref.U * mag) <= 1.0
    grad = torch.empty(2, n, k, device=DEV)
    mf.grouped_linear_wgrad(dy, x, off.to(DEV), grad)
    dw, mag, terms = ref.wgrad(dys, xs, small)
    assert ref.worst(grad, dw, wgrad_bound(dw, mag, terms, torch.zeros_like(dw), 0.0, F32)) <= 1.0
    codes, scales = mf.ckpt_quantize(x[-500:])
    cr, sr = ref.ckpt_quantize(xs)
    assert np.array_equal(codes.cpu().numpy(), cr) and np.array_equal(scales.cpu().numpy(), sr)
    t = torch.full((rows,), -1, device=DEV)
    t[-500:] = torch.arange(500, device=DEV) % 7
    g = mf.embedding_grad(x, t, torch.empty(9, k, device=DEV))
    gr, mag, terms = ref.embedding_grad(xs, torch.arange(500) % 7, 9, 1.0)
    assert ref.worst(g, gr, (terms[:, None] + 2) * ref.U * mag) <= 1.0
    mf.embedding(g, t, out=buf[:, 2048:2048 + k])
    want = ref.embedding(g.cpu(), torch.arange(500) % 7, 1.0)
    assert ref.worst(buf[-500:, 2048:2048 + k], want, ref.half_step(BF) * (1 + 2 ** -20) * want.abs()) <= 1.0
    assert not buf[:rows - 500:997, 2048:2048 + k].any()


def test_timing_kinds():
    x, w, off = rand((10, 16), BF, 1).to(DEV), rand((2, 8, 16), BF, 2).to(DEV), offsets_of([4, 6]).to(DEV)
    mf.timing.enable(True)
    try:
        mf.timing.reset()
        mf.grouped_linear(x, w, off)
        mf.ckpt_restore(*mf.ckpt_quantize(x))
        t = torch.zeros(10, dtype=torch.int64, device=DEV)
        mf.embedding(x, t)
        mf.embedding_grad(x, t, torch.empty(3, 16, device=DEV))
        counts = [mf.timing.read(kind)[1] for kind in ("grouped", "ckpt", "embed", "embed_grad")]
        assert counts[:3] == [1, 2, 1] and counts[3] >= 2
    finally:
        mf.timing.enable(False)
        mf.timing.reset()


def test_gradients_against_differences():
    # the product is linear in x and in W: f = sum(G * Y) changes by exactly
    # <dX, h> when x does by h.  Both sides carry the forward product's fp32
    # error: k * 2^-23 * sum |G||x||W|, twice, and the gradient's own.
    counts = [30, 0, 65, 5]
    off, n, k = offsets_of(counts), 48, 80
    x, h, G = rand((100, k), F32, 1), rand((100, k), F32, 2), rand((100, n), F32, 3)
    w, hw = rand((4, n, k), F32, 4, 0.1), rand((4, n, k), F32, 5, 0.1)
    offd = off.to(DEV)

    def f(xx, ww):
        return float((ref.f64(mf.grouped_linear(xx.to(DEV), ww.to(DEV), offd)) * ref.f64(G)).sum())

    def size(xx, ww):
        return float((ref.linear(xx, ww, off)[1] * ref.f64(G).abs()).sum())

    dx = ref.f64(mf.grouped_linear_dgrad(G.to(DEV), w.to(DEV), offd))
    dw = ref.f64(mf.grouped_linear_wgrad(G.to(DEV), x.to(DEV), offd, torch.zeros(4, n, k, device=DEV)))
    tol = (n + k + 102) * 2 * ref.U      # every sum's length, each side
    assert abs(f(x + h, w) - f(x, w) - float((dx * ref.f64(h)).sum())) <= tol * (size(x, w) + size(x + h, w) + size(h, w))
    assert abs(f(x, w + hw) - f(x, w) - float((dw * ref.f64(hw)).sum())) <= tol * (size(x, w) + size(x, w + hw) + size(x, hw))


# ---------------------------------------------------------------------------
# 8-bit checkpoints
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,k,pad", [(1, 1, 0), (3, 128, 0), (5, 129, 0), (64, 1000, 8), (33, 300, 0), (7, 96, 3), (200, 512, 0), (2, 5000, 16)])
def test_ckpt(rows, k, pad, dtype):
    x = rand((rows, k), F32, 1) * torch.exp(3 * rand((rows, 1), F32, 2))
    x[:, k // 2] *= 40.0
    x[rows // 2, : k // 3] = 0.0
    x = x.to(dtype)
    codes, scales = mf.ckpt_quantize(strided(x, pad))
    cr, sr = ref.ckpt_quantize(x)
    assert np.array_equal(codes.cpu().numpy(), cr) and np.array_equal(scales.cpu().numpy(), sr)
    want = torch.from_numpy(ref.ckpt_restore(cr, sr))
    for out_dtype in (BF, F32):
        assert torch.equal(ref.f64(mf.ckpt_restore(codes, scales, out_dtype)), want)   # exact in both
        out = strided(torch.zeros(rows, k, dtype=out_dtype), pad)
        mf.ckpt_restore(codes, scales, out=out)
        assert torch.equal(ref.f64(out), want)
    # half a step of 2^e at most
    step = torch.from_numpy(np.repeat(np.ldexp(1.0, sr.astype(int) - 127), 128, axis=1)[:, :k])
    assert bool(((want - ref.f64(x)).abs() <= step / 2).all())


def test_ckpt_borders_and_specials():
    tiny = 2.0 ** -126
    rows = [[127.0], [127.5], [128.0], [254.0], [255.0], [0.5, -127.0], [1.5, 2.5, -0.5, 127.0], [0.0], [-0.0], [tiny], [tiny / 4, -tiny / 2],
            [127 * tiny], [128 * tiny], [3.3e38, 1.0], [-3.4028235e38], [float("inf"), 1.0], [1.0, NAN], [-float("inf")]]
    for dtype in (F32, BF):
        x = torch.zeros(len(rows), 130)
        for i, r in enumerate(rows):
            x[i, : len(r)] = torch.tensor(r)
        x[:, 128] = 1.0      # the second block of each row stands for itself
        x = x.to(dtype)
        codes, scales = mf.ckpt_quantize(x.to(DEV))
        cr, sr = ref.ckpt_quantize(x)
        assert np.array_equal(scales.cpu().numpy(), sr), np.argwhere(scales.cpu().numpy() != sr)
        assert np.array_equal(codes.cpu().numpy(), cr)
        back = ref.f64(mf.ckpt_restore(codes, scales, F32)).numpy()
        assert np.array_equal(back, ref.ckpt_restore(cr, sr), equal_nan=True)
        assert np.isnan(back[-1, :128]).all() and (back[-1, 128] == 1.0)


# ---------------------------------------------------------------------------
# Embedding
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("tdt,odt", [(BF, BF), (F32, BF), (BF, F32), (F32, F32)])
@pytest.mark.parametrize("vocab,d,n,pad", [(10, 8, 1, 0), (100, 64, 33, 8), (1000, 300, 70, 0), (50, 2056, 9, 0), (7, 5000, 3, 0), (64, 1, 300, 0),
                                           (300, 96, 40, 3)])
def test_embedding(vocab, d, n, pad, tdt, odt):
    table = rand((vocab, d), tdt, 1)
    t = torch.randint(0, vocab, (n,), generator=torch.Generator().manual_seed(2))
    t[n // 2] = vocab - 1
    if n > 2:
        t[0], t[1] = -1, vocab      # padding on both sides of the table
    for tok in (t, t.to(torch.int32)):
        out = strided(torch.full((n, d), 5.0, dtype=odt), pad)
        mf.embedding(table.to(DEV), tok.to(DEV), scale=1.7, out=out)
        want = ref.embedding(table, tok, 1.7)
        # one fp32 product, one rounding to the type
        assert ref.worst(out, want, (ref.half_step(F32) + ref.half_step(odt) * (1 + 2 ** -20)) * want.abs()) <= 1.0
    if n % 3 == 0:
        got = mf.embedding(table.to(DEV), t.view(3, -1).to(DEV), dtype=odt)
        assert got.shape == (3, n // 3, d) and torch.equal(got.view(n, d), mf.embedding(table.to(DEV), t.to(DEV), dtype=odt))
    far = torch.tensor([2 ** 40, -2 ** 40, 2 ** 32], device=DEV)    # beyond 32 bits: padding, not a wrapped row
    assert not mf.embedding(table.to(DEV), far).any()


def tokens_of(kind, n, vocab, seed):
    g = torch.Generator().manual_seed(seed)
    if kind == "uniform":
        return torch.randint(0, vocab, (n,), generator=g)
    if kind == "one":
        return torch.full((n,), vocab // 2)
    if kind == "padding":
        return torch.full((n,), -1)
    u = torch.rand(n, generator=g, dtype=torch.float64)
    t = (torch.exp(u * np.log(vocab)).long() - 1).clamp(max=vocab - 1)
    t[torch.rand(n, generator=g) < 0.1] = vocab + 3
    return t


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("kind", ["uniform", "one", "zipf", "padding"])
@pytest.mark.parametrize("n,vocab,d,pad", [(1, 5, 8, 0), (64, 30, 16, 0), (65, 30, 16, 8), (1000, 600, 72, 0), (700, 33, 35, 0), (4096, 100, 8, 0),
                                           (4097, 70000, 8, 0), (9001, 300, 24, 3), (20000, 5000, 40, 0)])
def test_embedding_grad(n, vocab, d, pad, kind, dtype):
    t = tokens_of(kind, n, vocab, n + vocab)
    dy = rand((n, d), dtype, 3)
    dy[(t < 0) | (t >= vocab)] = NAN        # rows of padding must not be read
    g, mag, terms = ref.embedding_grad(dy, t, vocab, 1.3)
    mag = torch.nan_to_num(mag)
    for beta in (0.0, 1.0, 0.25):
        old = rand((vocab, d), F32, 4)
        grad = old.to(DEV) if beta else torch.full((vocab, d), NAN, device=DEV)
        old = ref.f64(old) if beta else torch.zeros(vocab, d, dtype=torch.float64)
        got = mf.embedding_grad(strided(dy, pad), t.to(DEV), grad, scale=1.3, beta=beta)
        assert got is grad
        bound = (terms[:, None] + 2) * ref.U * mag + 2 * ref.U * (beta * old.abs())
        assert ref.worst(got, g + beta * old, bound) <= 1.0
        if beta == 1.0:
            assert torch.equal(got.cpu()[terms == 0], old[terms == 0].float())
    # the same inputs give the same bits, with 32-bit tokens too
    one = mf.embedding_grad(strided(dy, pad), t.to(DEV), torch.zeros(vocab, d, device=DEV))
    two = mf.embedding_grad(strided(dy, pad), t.to(torch.int32).to(DEV), torch.zeros(vocab, d, device=DEV))
    assert torch.equal(one, two)


def test_embedding_grad_without_tokens():
    grad = torch.ones(10, 8, device=DEV)
    dy, t = torch.zeros(0, 8, dtype=BF, device=DEV), torch.zeros(0, dtype=torch.int64, device=DEV)
    assert torch.equal(mf.embedding_grad(dy, t, grad, beta=1.0), torch.ones(10, 8, device=DEV))
    assert not mf.embedding_grad(dy, t, grad).any()
    assert mf.embedding(torch.ones(4, 8, device=DEV), t).shape == (0, 8)


def test_embedding_gradient_against_differences():
    # linear in the table: sum(G * out) changes by <grad, h> when the table does by h
    t = torch.tensor([3, 1, 3, 3, 0, -1, 6, 1], device=DEV)
    table, h, G = rand((7, 16), F32, 1).to(DEV), rand((7, 16), F32, 2).to(DEV), rand((8, 16), F32, 3).to(DEV)
    grad = mf.embedding_grad(G, t, torch.empty(7, 16, device=DEV), scale=0.7)
    f = lambda tb: ref.f64(mf.embedding(tb, t, scale=0.7)) * ref.f64(G)
    got = float((f(table + h) - f(table)).sum())
    size = float(f(table.abs() + h.abs()).abs().sum())
    assert abs(got - float((ref.f64(grad) * ref.f64(h)).sum())) <= 16 * ref.U * size


# ---------------------------------------------------------------------------
# Streams, graphs, runs together
# ---------------------------------------------------------------------------
def train_step(s):
    """Embedding, an 8-bit checkpoint, experts, and every gradient."""
    h = mf.embedding(s["table"], s["tokens"], scale=2.0, dtype=BF)
    codes, scales = mf.ckpt_quantize(h)
    y = mf.grouped_linear(h, s["w"], s["off"])
    dh = mf.grouped_linear_dgrad(y, s["w"], s["off"])        # dY = Y: the gradient of sum(Y^2) / 2
    mf.grouped_linear_wgrad_ckpt(y, codes, scales, s["off"], s["dw"])
    mf.grouped_linear_wgrad(y, h, s["off"], s["dw2"], beta=0.5)
    mf.embedding_grad(dh, s["tokens"], s["dtable"], scale=2.0)
    return y, dh


def train_state(seed, n=300, vocab=40, d=96, nn=64, counts=(100, 0, 170, 30)):
    return {"table": rand((vocab, d), F32, seed).to(DEV), "tokens": tokens_of("uniform", n, vocab, seed).to(DEV),
            "w": rand((len(counts), nn, d), BF, seed + 1, 0.1).to(DEV), "off": offsets_of(counts).to(DEV),
            "dw": torch.zeros(len(counts), nn, d, dtype=BF, device=DEV), "dw2": torch.zeros(len(counts), nn, d, device=DEV),
            "dtable": torch.zeros(vocab, d, device=DEV)}


def results(s, y, dh):
    return [t.clone() for t in (y, dh, s["dw"], s["dw2"], s["dtable"])]


def test_graph_replays_follow_the_inputs():
    s = train_state(1)
    train_step(s)                       # loads the kernels
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph, second = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            y, dh = train_step(s)
        s2 = train_state(2)
        with torch.cuda.graph(second, stream=side):     # a second graph beside it
            y2, dh2 = train_step(s2)
    torch.cuda.synchronize()
    for k, counts in enumerate([(100, 0, 170, 30), (1, 1, 1, 297), (0, 0, 300, 0), (75, 75, 75, 75)]):
        new = train_state(10 + k, counts=counts)
        for name in ("table", "tokens", "w", "off"):
            s[name].copy_(new[name])
        for name in ("dw2",):
            s[name].zero_()
        graph.replay()
        second.replay()
        graph_out = None
        torch.cuda.synchronize()
        graph_out = results(s, y, dh)
        eager = results(new, *train_step(new))
        torch.cuda.synchronize()
        for a, b in zip(graph_out, eager):
            assert torch.equal(a, b), k
    s2e = train_state(2)
    want = results(s2e, *train_step(s2e))
    got = results(s2, y2, dh2)
    for i in (0, 1, 2, 4):      # dw2 adds up over the replays
        assert torch.equal(got[i], want[i])


def test_side_streams():
    # two streams at once, each with its own workspace, give what one gives
    states = [train_state(5, n=9000, vocab=3000, counts=(4000, 0, 4999, 1)), train_state(6)]
    want = []
    for s in states:
        want.append(results(s, *train_step(s)))
        s["dw2"].zero_()
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream(), torch.cuda.Stream()], [None, None]
    for i, s in enumerate(states):
        with torch.cuda.stream(streams[i]):
            y, dh = train_step(s)
            got[i] = (y, dh)
    torch.cuda.synchronize()
    for i, s in enumerate(states):
        for a, b in zip(results(s, *got[i]), want[i]):
            assert torch.equal(a, b)


def test_together_with_the_step():
    # embedding -> experts -> gradients -> Muon on the experts' matrices and
    # AdamW on the table's packed segment
    s = train_state(7, n=500, vocab=60, d=128, nn=96, counts=(200, 0, 260, 40))
    table0, w0 = s["table"].clone(), s["w"].clone()
    packed, (at,) = mf.tail_pack([s["table"].view(-1)])
    s["table"] = packed[at:at + 60 * 128].view(60, 128)
    gpacked = torch.zeros_like(packed)
    s["dtable"] = gpacked[at:at + 60 * 128].view(60, 128)
    y, dh = train_step(s)
    # gradients against the formulas, each from what the step before it gave
    h = mf.embedding(table0, s["tokens"], scale=2.0, dtype=BF)
    cr, sr = ref.ckpt_quantize(h)
    dw, mag, terms = ref.wgrad(y, torch.from_numpy(ref.ckpt_restore(cr, sr)), s["off"])
    assert ref.worst(s["dw"], dw, wgrad_bound(dw, mag, terms, torch.zeros_like(dw), 0.0, BF)) <= 1.0
    g, mag, terms = ref.embedding_grad(dh, s["tokens"], 60, 2.0)
    assert ref.worst(s["dtable"], g, (terms[:, None] + 2) * ref.U * mag) <= 1.0
    # The step on them: the views of the stacked weights and gradients give bit
    # for bit what separate matrices of the same values give.  (The bars of
    # the step's own oracle tests are for gradients of full rank.  This one,
    # W H^T H over 60 different rows of H, has rank 60 at most: its 36 zero
    # singular values hold bf16 rounding, which five iterations raise by up to
    # 3.4445^5 = 485, so 64-bit and bf16 results may differ there by design.)
    hp = muon_hparams()
    W, G = list(s["w"]), list(s["dw"])
    M, U = [torch.zeros_like(v) for v in W], [torch.empty(v.shape, device=DEV) for v in W]
    Wc, Gc = [v.clone() for v in w0], [v.clone() for v in G]
    Mc, Uc = [torch.zeros_like(v) for v in W], [torch.empty(v.shape, device=DEV) for v in W]
    mf.MuonStep(W, G, M, update_out=U).step(lr=hp["lr"], beta=hp["beta"], weight_decay=hp["weight_decay"])
    mf.muon_step(Wc, Gc, Mc, update_out=Uc, lr=hp["lr"], beta=hp["beta"], weight_decay=hp["weight_decay"])
    p0 = np64(packed)
    m, v = torch.zeros_like(packed), torch.zeros_like(packed)
    mf.adamw_tail(packed, gpacked, m, v, lr=0.01, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.01, step=1)
    torch.cuda.synchronize()
    for e in range(4):
        assert torch.equal(W[e], Wc[e]) and torch.equal(M[e], Mc[e]) and torch.equal(U[e], Uc[e])
        assert torch.isfinite(W[e]).all() and (e == 1 or not torch.equal(W[e], w0[e]))
    assert not s["dw"][1].any() and not U[1].any()          # expert 1 had no rows
    pr, _, _ = oracle.adamw_tail(p0, np64(gpacked), np.zeros_like(p0), np.zeros_like(p0), lr=0.01, beta1=0.9, beta2=0.95,
                                 eps=1e-8, weight_decay=0.01, step=1)
    assert rel(np64(packed), pr) <= ADAMW_TOL
    assert not torch.equal(s["table"], table0)
