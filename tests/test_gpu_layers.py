"""Routing, the exchange of rows, layer norm and 8-bit float products on the GPU
against plain float64 forms (layers_ref.py, where the bounds are derived), each
at the sizes, masks and values where it can go wrong.
"""

import numpy as np
import pytest
import torch

import grads_ref as gref
import layers_ref as ref
import matrix_optimizer_step_owner_amd as mf
from test_gpu_grads import BF, DEV, F32, NAN, ROUTES, _need_gpu, offsets_of, rand, strided  # noqa: F401

pytestmark = pytest.mark.gpu
INF = float("inf")


# ---------------------------------------------------------------------------
# Routing
# ---------------------------------------------------------------------------
# tokens, experts, k, groups, groups that stay, columns before and after a row
ROUTINGS = [(1, 1, 1, 1, 1, 0), (1, 256, 8, 8, 4, 0), (5, 7, 3, 1, 1, 3), (33, 60, 4, 1, 1, 0), (130, 64, 6, 8, 3, 8), (70, 65, 2, 5, 2, 1),
            (64, 128, 8, 4, 4, 0), (17, 160, 6, 8, 3, 0), (200, 256, 8, 8, 4, 0), (50, 384, 8, 1, 1, 0), (40, 512, 10, 16, 5, 4), (9, 1000, 32, 10, 7, 0),
            (21, 1024, 1, 64, 1, 0), (12, 40, 32, 1, 1, 0), (6, 32, 32, 1, 1, 0), (16, 12, 4, 12, 4, 0), (31, 48, 2, 2, 1, 5)]


def logits_of(tokens, n, dtype, seed):
    return (rand((tokens, n), F32, seed, 2.0) + rand((n,), F32, seed + 1)).to(dtype)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("tokens,n,k,groups,top,pad", ROUTINGS)
def test_route(tokens, n, k, groups, top, pad, biased, kind, dtype):
    x = logits_of(tokens, n, dtype, tokens + n)
    bias = rand((n,), F32, 5, 0.05) if biased else None
    mask = torch.rand(tokens, generator=torch.Generator().manual_seed(3)) < 0.8 if tokens > 1 else None
    if mask is not None:
        x[~mask] = NAN          # not read
    for renormalize, scale in ((True, 1.0), (False, 2.5)):
        e, w = mf.route(strided(x, pad), k, scores=kind, bias=None if bias is None else bias.to(DEV), groups=groups, top_groups=top,
                        renormalize=renormalize, scale=scale, mask=None if mask is None else mask.to(DEV))
        xr = torch.nan_to_num(x)
        want, ww, bound = ref.route(xr, k, kind, bias, groups, top, renormalize, scale, mask)
        assert e.dtype == torch.int32 and torch.equal(e.cpu().long(), want)
        assert ref.f64(w).sub(ww).abs().le(bound).all()


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,top", [(1, 1), (4, 2)])
def test_near_and_equal_keys(kind, groups, top):
    # keys that fp32 cannot tell apart, and keys that are equal: 64 bits decide,
    # then the index
    tokens, n, k = 300, 64, 7
    g = torch.Generator().manual_seed(1)
    base = torch.randn(tokens, 1, generator=g).repeat(1, n)
    step = torch.randint(-2, 3, (tokens, n), generator=g).float() * 2.0 ** -23
    for x in (base, base * (1 + step), torch.randint(-2, 3, (tokens, n), generator=g).float()):
        for bias in (None, torch.zeros(n), torch.randint(-2, 3, (n,), generator=g).float() * 2.0 ** -25, torch.randint(0, 2, (n,), generator=g).float()):
            e, w = mf.route(x.to(DEV), k, scores=kind, bias=None if bias is None else bias.to(DEV), groups=groups, top_groups=top)
            want, ww, bound = ref.route(x, k, kind, bias, groups, top)
            told = ~ref.undecided(x, kind, bias, groups, top)       # (x1, b1), (x2, b2) against (x1, b2), (x2, b1)
            assert torch.equal(e.cpu().long()[told], want[told]) and int(told.sum()) >= 200
            assert ref.f64(w)[told].sub(ww[told]).abs().le(bound[told]).all()


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("n,k,groups,top", [(250, 20, 1, 1), (256, 32, 8, 3), (500, 32, 1, 1), (512, 20, 16, 4), (1000, 32, 1, 1), (1024, 9, 4, 1)])
def test_equal_keys_of_a_lane(n, k, groups, top, kind):
    # many equal keys in each lane's lists, whatever their order
    g = torch.Generator().manual_seed(n)
    x = torch.randint(-2, 3, (200, n), generator=g).float()
    x[100:] = torch.where(torch.rand(100, n, generator=g) < 0.9, x[100:, :1], x[100:])
    for bias in (None, torch.randint(0, 2, (n,), generator=g).float()):
        e, w = mf.route(x.to(DEV), k, scores=kind, bias=None if bias is None else bias.to(DEV), groups=groups, top_groups=top)
        want, ww, bound = ref.route(x, k, kind, bias, groups, top)
        told = ~ref.undecided(x, kind, bias, groups, top)
        assert torch.equal(e.cpu().long()[told], want[told]) and int(told.sum()) >= 100
        assert ref.f64(w)[told].sub(ww[told]).abs().le(bound[told]).all()


def test_trading_bias():
    # a bias that makes up for the score to the last bits of fp32: what the
    # scores round to would choose otherwise
    n = 128
    x = torch.linspace(-4, 4, n).repeat(50, 1) + rand((50, 1), F32, 2)
    s = torch.sigmoid(x[0].double())
    bias = (0.75 - s).float()
    e, _ = mf.route(x.to(DEV), 16, scores="sigmoid", bias=bias.to(DEV), groups=8, top_groups=4)
    assert torch.equal(e.cpu().long(), ref.route(x, 16, "sigmoid", bias, 8, 4)[0])


def test_route_specials():
    # infinities, the type's lowest value and NaN: experts stay different and in range
    low = torch.finfo(F32).min
    n = 64
    rows = [torch.full((n,), -INF), torch.full((n,), low), torch.full((n,), NAN), torch.zeros(n), torch.full((n,), 1e4)]
    x = torch.stack(rows + [torch.linspace(-3, 3, n).where(torch.arange(n) % 3 > 0, torch.tensor(v)) for v in (-INF, INF, NAN, low)])
    x[3, 5], x[3, 6] = -0.0, 0.0
    for kind in ("softmax", "sigmoid"):
        for bias in (None, torch.linspace(0, 1, n), torch.full((n,), -INF).where(torch.arange(n) < 60, torch.tensor(0.0))):
            for groups, top in ((1, 1), (8, 3)):
                e, w = mf.route(x.to(DEV), 8, scores=kind, bias=None if bias is None else bias.to(DEV), groups=groups, top_groups=top)
                e = e.cpu()
                assert ((e >= 0) & (e < n)).all() and all(len(set(r.tolist())) == 8 for r in e)
    # masked experts (bias -inf) are chosen last, in the order of their index
    e, _ = mf.route(torch.zeros(1, n, device=DEV), 8, bias=torch.full((n,), -INF).where(torch.arange(n) < 60, torch.tensor(0.0)).to(DEV))
    assert e.tolist() == [[60, 61, 62, 63, 0, 1, 2, 3]]
    # the largest finite logits overflow no score
    e, w = mf.route(torch.full((2, n), 3e38, device=DEV), 4)
    assert e.tolist() == [[0, 1, 2, 3]] * 2 and torch.equal(w, torch.full((2, 4), 0.25, device=DEV))
    # NaN is behind everything, -inf included
    y = torch.full((1, n), -INF)
    y[0, 0] = NAN
    assert mf.route(y.to(DEV), 3)[0].tolist() == [[1, 2, 3]]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("tokens,n,k,groups,top,pad", ROUTINGS)
def test_route_grad(tokens, n, k, groups, top, pad, kind, dtype):
    x = logits_of(tokens, n, dtype, tokens + n)
    e = ref.route(x, k, kind)[0].to(torch.int32)
    if tokens > 2:
        e[1] = -1
        x[1] = NAN              # a token without experts is not read
        e[2, 0] = n             # an expert that is not there
        if k > 1:
            e[2, -1] = e[2, 1]  # one that is named twice
    dw = rand((tokens, k), F32, 9)
    for renormalize, scale in ((True, 1.0), (False, 2.5), (True, 0.0)):
        out = strided(torch.full((tokens, n), 7.0, dtype=dtype), pad)
        got = mf.route_grad(dw.to(DEV), strided(x, pad), e.to(DEV), scores=kind, renormalize=renormalize, scale=scale, out=out)
        assert got is out
        want, bound = ref.route_grad(dw, torch.nan_to_num(x), e, kind, renormalize, scale)
        assert ref.f64(got).sub(want).abs().le(bound + ref.half_step(dtype) * want.abs()).all()
        if pad:
            assert torch.isnan(out._base[:, :pad]).all() and torch.isnan(out._base[:, pad + n:]).all()


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
def test_route_gradient_against_differences(kind, renormalize):
    # the weights' change along a direction, chosen experts unchanged: differences
    # in 64 bits of the plain form at the kernel's own choice
    x, k = logits_of(6, 20, F32, 4), 4
    e, w = mf.route(x.to(DEV), k, scores=kind, renormalize=renormalize, scale=1.5)
    dw, h = rand((6, k), F32, 1), rand((6, 20), F32, 2).double()
    grad = ref.f64(mf.route_grad(dw.to(DEV), x.to(DEV), e, scores=kind, renormalize=renormalize, scale=1.5))

    def f(x):
        s = ref.scores(x, kind)[0].gather(1, e.cpu().long())
        return float((dw.double() * 1.5 * (s / (s.sum(1, keepdim=True) + 1e-20) if renormalize else s)).sum())
    t = 1e-5
    slope = (f(x.double() + t * h) - f(x.double() - t * h)) / (2 * t)
    # the differences: third derivatives of size under 10 |h|^3 |dw| times t^2, and 64-bit rounding over t
    size = float(dw.abs().sum()) * 1.5
    assert abs(slope - float((grad * h).sum())) <= size * (10 * 20 * 64 * t * t + 1e-15 / t + 400 * ref.U * 20)


@pytest.mark.parametrize("tokens,k,n", [(0, 1, 4), (1, 1, 1), (3, 2, 5), (64, 1, 64), (65, 3, 7), (768, 8, 256), (769, 8, 256), (1000, 8, 256), (1024, 8, 256), (1025, 8, 256), (2000, 6, 60),
                                        (5000, 8, 1024), (40000, 8, 33), (9000, 1, 1), (300000, 2, 128), (700, 32, 40)])
@pytest.mark.parametrize("kind", ["even", "one", "none", "wild"])
def test_plan(tokens, k, n, kind):
    g = torch.Generator().manual_seed(tokens + n)
    e = torch.randint(0, n, (tokens, k), generator=g, dtype=torch.int32)
    if kind == "one":
        e[:] = n - 1
    elif kind == "none":
        e[:] = -1
    elif kind == "wild":        # numbers outside are no choice
        e = torch.where(torch.rand(tokens, k, generator=g) < 0.3, torch.randint(-2 ** 31, 2 ** 31 - 1, (tokens, k), generator=g).to(torch.int32), e)
    p = mf.route_plan(e.to(DEV), n)
    off, place = ref.plan(e, n)
    assert torch.equal(p.offsets.cpu().long(), off) and torch.equal(p.place.cpu().long(), place)


@pytest.mark.parametrize("counts", [[5], [3, 3, 3], [0, 0, 9, 1], [2 ** 40, 2 ** 40 + 1, 2 ** 40 + 2], list(range(1000))])
def test_balance(counts):
    c = torch.tensor(counts)
    b = rand((len(counts),), F32, 1)
    sign = torch.sign(torch.tensor([sum(counts) - v * len(counts) for v in counts], dtype=torch.float64))
    want = b + (0.001 * sign).float()
    for dt in (torch.int64, torch.int32):
        if max(counts) < 2 ** 31:
            got = b.to(DEV)
            assert mf.route_balance(got, c.to(dt).to(DEV), 0.001) is got
            assert torch.equal(got.cpu(), want)
    got = b.to(DEV)
    assert torch.equal(mf.route_balance(got, c.to(DEV), 0.001).cpu(), want)


# ---------------------------------------------------------------------------
# Exchange
# ---------------------------------------------------------------------------
def plan_of(tokens, k, n, seed, drop=0.2):
    g = torch.Generator().manual_seed(seed)
    e = torch.stack([torch.randperm(n, generator=g)[:k] for _ in range(tokens)]).to(torch.int32) if tokens else torch.zeros(0, k, dtype=torch.int32)
    e[torch.rand(tokens, generator=g) < drop] = -1
    return ref.plan(e, n)[1].to(torch.int32)


# tokens, k, experts, d, columns before and after
EXCHANGES = [(1, 1, 1, 1, 0), (1, 8, 16, 512, 0), (5, 2, 4, 7, 0), (33, 3, 5, 64, 8), (64, 8, 32, 129, 0), (40, 1, 3, 1000, 3), (70, 9, 12, 520, 0),
             (10, 32, 40, 96, 1), (7, 6, 8, 4096, 8), (12, 4, 4, 5003, 0), (300, 8, 64, 256, 0), (9, 2, 2, 8200, 16)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("tokens,k,n,d,pad", EXCHANGES)
def test_dispatch_and_combine(tokens, k, n, d, pad, dtype):
    place = plan_of(tokens, k, n, 3)
    rows = tokens * k
    x, h, w = rand((tokens, d), dtype, 1), rand((rows, d), dtype, 2), rand((tokens, k), F32, 4)
    row, on = ref.held(place, rows)
    used = torch.zeros(rows, dtype=torch.bool)
    used[row[on]] = True
    h[~used] = NAN              # rows of no choice are not read
    out = strided(torch.full((rows, d), 7.0, dtype=dtype), pad)
    got = mf.route_dispatch(strided(x, pad), place.to(DEV), out=out)
    want = torch.full((rows, d), 7.0, dtype=dtype)
    t, _ = on.nonzero(as_tuple=True)
    want[row[on]] = x[t]
    assert got is out and torch.equal(got.cpu(), want)
    if pad:
        assert torch.isnan(out._base[:, :pad]).all() and torch.isnan(out._base[:, pad + d:]).all()
    for weights in (w, None):
        for beta in (0.0, 1.0, -0.5):
            old = rand((tokens, d), dtype, 6)
            y = strided(old if beta else torch.full((tokens, d), NAN, dtype=dtype), pad)
            got = mf.route_combine(strided(h, pad), place.to(DEV), None if weights is None else weights.to(DEV), beta=beta, out=y)
            v, mag = ref.combine(torch.nan_to_num(h), place, weights)
            v, mag = (v + beta * ref.f64(old), mag + abs(beta) * ref.f64(old).abs()) if beta else (v, mag)
            assert got is y and gref.worst(got, v, ref.half_step(dtype) * v.abs() + (k + 2) * ref.U * mag) <= 1.0
    assert torch.equal(mf.route_combine(h.to(DEV), place.to(DEV), w.to(DEV)), mf.route_combine(strided(h, pad), place.to(DEV), w.to(DEV)))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("tokens,k,n,d,pad", EXCHANGES)
def test_combine_grad(tokens, k, n, d, pad, dtype):
    place = plan_of(tokens, k, n, 3)
    rows = tokens * k
    dy, h, w = rand((tokens, d), dtype, 1), rand((rows, d), dtype, 2), rand((tokens, k), F32, 4)
    dh, has, dw, mag = ref.combine_grad(dy, h, place, w)
    h[~has] = NAN
    out = strided(torch.full((rows, d), 7.0, dtype=dtype), pad)
    got, gw = mf.route_combine_grad(strided(dy, pad), strided(h, pad), place.to(DEV), w.to(DEV), dh=out)
    assert got is out
    has = has.to(DEV)
    assert torch.equal(got[~has], torch.full_like(got[~has], 7.0))
    want = dh[has.cpu()]
    assert gref.worst(got[has], want, (ref.half_step(dtype) + ref.U) * want.abs()) <= 1.0
    assert gref.worst(gw, dw, ref.row_terms(d) * ref.U * mag + 1e-38) <= 1.0
    if pad:
        assert torch.isnan(out._base[:, :pad]).all() and torch.isnan(out._base[:, pad + d:]).all()


def test_places_outside():
    # rows outside the buffer are none, whatever the number
    place = torch.tensor([[0, -1], [5, 6], [2 ** 31 - 1, -2 ** 31], [1, 3]], dtype=torch.int32, device=DEV)
    x, w = rand((4, 40), F32, 1).to(DEV), rand((4, 2), F32, 2).to(DEV)
    out = mf.route_dispatch(x, place, out=torch.zeros(6, 40, device=DEV))
    assert torch.equal(out[0], x[0]) and torch.equal(out[5], x[1]) and torch.equal(out[1], x[3]) and torch.equal(out[3], x[3])
    assert not out[2].any() and not out[4].any()
    y = mf.route_combine(out, place)
    assert torch.equal(y[0], x[0]) and torch.equal(y[1], x[1]) and not y[2].any() and torch.equal(y[3], 2 * x[3])
    dh, dw = mf.route_combine_grad(x, out, place, w, dh=torch.zeros(6, 40, device=DEV))
    assert dw[0, 1] == 0 and dw[1, 1] == 0 and not dw[2].any() and not dh[2].any() and not dh[4].any()


def test_exchange_against_differences():
    # bilinear in h and w, linear in x: changes along a direction are the gradients'
    place = plan_of(30, 3, 6, 5)
    pg = place.to(DEV)
    h, a, w, b, G = rand((90, 48), F32, 1), rand((90, 48), F32, 2), rand((30, 3), F32, 3), rand((30, 3), F32, 4), rand((30, 48), F32, 5)
    dh, dw = mf.route_combine_grad(G.to(DEV), h.to(DEV), pg, w.to(DEV), dh=torch.zeros(90, 48, device=DEV))
    f = lambda h, w: float((ref.f64(mf.route_combine(h.to(DEV), pg, w.to(DEV))) * G.double()).sum())
    size = lambda h, w: float((ref.combine(h, place, w)[1] * G.double().abs()).sum())
    tol = 2 * (3 + 48 / 64 + 40) * ref.U
    assert abs(f(h + a, w) - f(h, w) - float((ref.f64(dh) * a.double()).sum())) <= tol * (size(h, w) + size(h + a, w) + size(a, w))
    assert abs(f(h, w + b) - f(h, w) - float((ref.f64(dw) * b.double()).sum())) <= tol * (size(h, w) + size(h, w + b) + size(h, b))
    x = rand((30, 48), F32, 6)
    xs = mf.route_dispatch(x.to(DEV), pg, out=torch.zeros(90, 48, device=DEV))
    dx = mf.route_combine(a.to(DEV), pg)
    left, right = ref.f64(xs) * a.double(), x.double() * ref.f64(dx)
    assert abs(float(left.sum() - right.sum())) <= 5 * ref.U * float(left.abs().sum())


# ---------------------------------------------------------------------------
# Layer norm
# ---------------------------------------------------------------------------
NORMS = [(1, 1, 0), (3, 2, 0), (5, 7, 0), (2, 64, 8), (33, 129, 0), (70, 300, 3), (9, 512, 0), (600, 96, 0), (1030, 513, 0), (17, 1537, 0), (7, 2048, 8),
         (5, 4096, 0), (4, 5120, 0), (3, 8192, 0), (3, 8200, 1), (2, 16384, 0), (2, 16392, 0), (700, 40, 0), (2, 40000, 8)]


def activations(rows, d, dtype, seed):
    x = rand((rows, d), F32, seed) * torch.exp(rand((rows, 1), F32, seed + 1)) + rand((rows, 1), F32, seed + 2, 3.0)
    x[:, d // 2] *= 20.0
    return x.to(dtype)


@pytest.mark.parametrize("dtype,wdt", [(BF, F32), (BF, BF), (F32, F32), (F32, BF)])
@pytest.mark.parametrize("centered", [True, False])
@pytest.mark.parametrize("rows,d,pad", NORMS)
def test_layer_norm(rows, d, pad, centered, dtype, wdt):
    x, w, b = activations(rows, d, dtype, 1), rand((d,), F32, 5).to(wdt), rand((d,), F32, 6).to(wdt)
    for bias in (b, None):
        out = strided(torch.zeros(rows, d, dtype=dtype), pad)
        got = mf.layer_norm(strided(x, pad), w.to(DEV), None if bias is None else bias.to(DEV), eps=1e-4, centered=centered, out=out)
        y, bound = ref.norm(x, w, bias, 1e-4, centered)
        assert got is out and gref.worst(got, y, bound + ref.half_step(dtype) * y.abs() + 1e-30) <= 1.0
        if pad:
            assert torch.isnan(out._base[:, :pad]).all() and torch.isnan(out._base[:, pad + d:]).all()


@pytest.mark.parametrize("dtype,wdt", [(BF, F32), (BF, BF), (F32, F32), (F32, BF)])
@pytest.mark.parametrize("centered", [True, False])
@pytest.mark.parametrize("rows,d,pad", NORMS)
def test_layer_norm_grad(rows, d, pad, centered, dtype, wdt):
    x, dy, w = activations(rows, d, dtype, 1), rand((rows, d), dtype, 2), rand((d,), F32, 5).to(wdt)
    (dx, bx), (dw, bw), (db, bb) = ref.norm_grad(dy, x, w, 1e-4, centered)
    for beta in (0.0, 1.0, -0.5):
        old = [rand((d,), F32, 7), rand((d,), F32, 8)]
        gw, gb = (o.to(DEV) if beta else torch.full((d,), NAN, device=DEV) for o in old)
        out = strided(torch.zeros(rows, d, dtype=dtype), pad)
        with_bias = beta != 1.0
        got = mf.layer_norm_grad(strided(dy, pad), strided(x, pad), w.to(DEV), gw, gb if with_bias else None, eps=1e-4, centered=centered, beta=beta, out=out)
        assert got is out and gref.worst(got, dx, bx + ref.half_step(dtype) * dx.abs() + 1e-30) <= 1.0
        for g, o, v, bound, on in ((gw, old[0], dw, bw, True), (gb, old[1], db, bb, with_bias)):
            if on:
                o = beta * ref.f64(o) if beta else torch.zeros(d, dtype=torch.float64)
                assert gref.worst(g, v + o, bound + 2 * ref.U * (v.abs() + o.abs()) + 1e-30) <= 1.0
        if pad:
            assert torch.isnan(out._base[:, :pad]).all() and torch.isnan(out._base[:, pad + d:]).all()
    # the same inputs give the same bits
    again = [torch.zeros(d, device=DEV) for _ in range(4)]
    a = mf.layer_norm_grad(dy.to(DEV), x.to(DEV), w.to(DEV), again[0], again[1])
    b = mf.layer_norm_grad(dy.to(DEV), x.to(DEV), w.to(DEV), again[2], again[3])
    assert torch.equal(a, b) and torch.equal(again[0], again[2]) and torch.equal(again[1], again[3])


def test_norm_of_constant_and_large_rows():
    # no variance: only the bias is left; a large mean costs no digits of the deviations
    x = torch.full((3, 100), 5.0, device=DEV)
    b = rand((100,), F32, 1).to(DEV)
    assert torch.equal(mf.layer_norm(x, torch.ones(100, device=DEV), b), b.expand(3, 100))
    assert not mf.layer_norm(torch.zeros(2, 9, device=DEV), torch.ones(9, device=DEV), centered=False).any()
    x = 1000.0 + rand((4, 256), F32, 2)
    y, bound = ref.norm(x, torch.ones(256), None, 1e-5, True)
    assert gref.worst(mf.layer_norm(x.to(DEV), torch.ones(256, device=DEV)), y, bound + ref.half_step(F32) * y.abs()) <= 1.0
    # a row's NaN and infinities stay in it
    x = rand((3, 64), F32, 3)
    x[1, 5], x[2, 7] = NAN, INF
    y = mf.layer_norm(x.to(DEV), torch.ones(64, device=DEV))
    assert torch.isfinite(y[0]).all() and torch.isnan(y[1]).all() and torch.isnan(y[2, 7])


@pytest.mark.parametrize("centered", [True, False])
@pytest.mark.parametrize("d", [40, 3000, 9000])     # lanes, a workgroup, rows that are read again
@pytest.mark.parametrize("power", [-45, 45])
def test_norm_of_tiny_and_huge_rows(power, d, centered):
    # without eps, a row's size leaves the result; its cube is outside fp32's range
    x, dy, w = (rand((3, d), F32, 1).double() * 2.0 ** power).float(), rand((3, d), F32, 2), 1 + rand((d,), F32, 3, 0.1)
    y, bound = ref.norm(x, w, None, 0.0, centered)
    assert gref.worst(mf.layer_norm(x.to(DEV), w.to(DEV), eps=0.0, centered=centered), y, bound + ref.half_step(F32) * y.abs()) <= 1.0
    (dx, bx), (dw, bw), _ = ref.norm_grad(dy, x, w, 0.0, centered)
    g = torch.zeros(d, device=DEV)
    got = mf.layer_norm_grad(dy.to(DEV), x.to(DEV), w.to(DEV), g, eps=0.0, centered=centered)
    assert gref.worst(got, dx, bx + ref.half_step(F32) * dx.abs()) <= 1.0 and gref.worst(g, dw, bw + ref.U * dw.abs()) <= 1.0


def test_norm_gradient_without_rows():
    x, w = torch.zeros(0, 8, dtype=BF, device=DEV), torch.ones(8, device=DEV)
    g, b = torch.full((8,), 2.0, device=DEV), torch.full((8,), NAN, device=DEV)
    assert mf.layer_norm(x, w).shape == (0, 8)
    mf.layer_norm_grad(x, x, w, g, beta=0.5)
    mf.layer_norm_grad(x, x, w, torch.zeros(8, device=DEV), b)
    assert torch.equal(g, torch.ones(8, device=DEV)) and not b.any()


@pytest.mark.parametrize("centered", [True, False])
def test_norm_gradient_against_differences(centered):
    x, w, b, G = activations(8, 50, F32, 1), rand((50,), F32, 4), rand((50,), F32, 5), rand((8, 50), F32, 6)
    hx, hw, hb = rand((8, 50), F32, 7).double(), rand((50,), F32, 8).double(), rand((50,), F32, 9).double()
    gw, gb = torch.empty(50, device=DEV), torch.empty(50, device=DEV)
    dx = mf.layer_norm_grad(G.to(DEV), x.to(DEV), w.to(DEV), gw, gb, centered=centered)
    f = lambda x, w, b: float((ref.norm(x, w, b, 1e-5, centered)[0] * G.double()).sum())
    t = 1e-5
    X, W, B = x.double(), w.double(), b.double()
    for h, grad, g in ((hx, dx, lambda t: f(X + t * hx, W, B)), (hw, gw, lambda t: f(X, W + t * hw, B)), (hb, gb, lambda t: f(X, W, B + t * hb))):
        slope, terms = (g(t) - g(-t)) / (2 * t), (ref.f64(grad) * h).abs()
        assert abs(slope - float((ref.f64(grad) * h).sum())) <= 1e-6 * float(terms.sum() + 1)


# ---------------------------------------------------------------------------
# 8-bit floats
# ---------------------------------------------------------------------------
def codes_of(t):
    return ref.f64(t.float()).numpy()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,k,pad", [(1, 1, 0), (3, 128, 0), (5, 129, 0), (64, 1000, 8), (33, 300, 0), (7, 96, 3), (200, 512, 0), (2, 5000, 16)])
def test_scaled_quantize(rows, k, pad, dtype):
    x = rand((rows, k), F32, 1) * torch.exp(3 * rand((rows, 1), F32, 2))
    x[:, k // 2] *= 40.0
    x[rows // 2, : k // 3] = 0.0
    x = x.to(dtype)
    codes, scales = mf.scaled_quantize(strided(x, pad))
    cr, sr = ref.scaled_rows(x)
    assert np.array_equal(scales.cpu().numpy(), sr) and np.array_equal(codes_of(codes), cr)


def test_scaled_borders_and_specials():
    tiny = 2.0 ** -126
    rows = [[448.0], [449.0], [464.0], [465.0], [1.75], [1.7500001], [0.5, -448.0], [17.0, 19.0, 21.0, 256.0], [0.0], [-0.0, 1.0], [tiny], [tiny / 4, -tiny / 2],
            [448 * tiny], [449 * tiny], [3.3e38, 1.0], [-3.4028235e38], [INF, 1.0], [1.0, NAN], [-INF], [256.0, 2.0 ** -9, 2.0 ** -10, 3 * 2.0 ** -10, 2.0 ** -6]]
    for dtype in (F32, BF):
        x = torch.zeros(len(rows), 130)
        for i, r in enumerate(rows):
            x[i, : len(r)] = torch.tensor(r)
        x[:, 128] = 1.0
        x = x.to(dtype)
        codes, scales = mf.scaled_quantize(x.to(DEV))
        cr, sr = ref.scaled_rows(x)
        assert np.array_equal(scales.cpu().numpy(), sr), np.argwhere(scales.cpu().numpy() != sr)
        assert np.array_equal(codes_of(codes), cr, equal_nan=True), np.argwhere(codes_of(codes) != cr)


def test_every_rounding():
    # all bf16 values between two powers of two and their neighbourhood below, in one block scale
    v = torch.arange(0, 0x43e1, dtype=torch.int32).to(torch.int16).view(BF).float()      # 0 .. 448 + a step
    v = v[v <= 448.0]
    v = torch.cat([v, torch.zeros(-v.numel() % 127)]).view(-1, 127)
    x = torch.cat([v, torch.full((v.shape[0], 1), 448.0)], 1)       # 2^0 in every block
    codes, scales = mf.scaled_quantize(x.to(DEV))
    assert (scales == 127).all() and np.array_equal(codes_of(codes), ref.e4m3(x.double().numpy()))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("e,n,k", [(1, 1, 1), (3, 128, 128), (2, 129, 127), (4, 64, 300), (2, 300, 520), (5, 7, 1000)])
def test_scaled_weights(e, n, k, dtype):
    w = (rand((e, n, k), F32, 1, 0.05) * torch.exp(2 * rand((e, 1, k), F32, 2))).to(dtype)
    codes, scales, tcodes, tscales = mf.scaled_quantize_weight(w.to(DEV), both=True)
    cr, sr = ref.scaled_matrices(w)
    assert np.array_equal(scales.cpu().numpy(), sr) and np.array_equal(codes_of(codes), cr)
    ct, st = ref.scaled_matrices(w.transpose(1, 2).contiguous())
    assert np.array_equal(tscales.cpu().numpy(), st) and np.array_equal(codes_of(tcodes), ct)
    one = mf.scaled_quantize_weight(w.to(DEV))
    assert len(one) == 2 and torch.equal(one[0].view(torch.uint8), codes.view(torch.uint8)) and torch.equal(one[1], scales)


SCALED = [("one row", 256, 512, 0), ("one expert", 256, 512, 0), ("empty ones", 328, 200, 8), ("none", 64, 128, 0), ("tiny", 131, 77, 0), ("mixed", 256, 512, 8),
          ("mixed", 131, 300, 3), ("skewed", 328, 200, 0), ("many", 64, 64, 0), ("five", 1496, 2000, 8), ("two short", 40, 1032, 0), ("tiny", 1, 1, 0),
          ("long one", 72, 130, 0), ("one row", 4097, 640, 0)]


@pytest.mark.parametrize("route,n,k,pad", SCALED)
def test_scaled_linear(route, n, k, pad):
    counts, lead, tail = ROUTES[route]
    rows = sum(counts) + lead + tail
    off = offsets_of(counts, lead)
    x, w = rand((rows, k), BF, 1), rand((len(counts), n, k), BF, 2, 0.05)
    x[:lead], x[rows - tail:] = NAN, NAN        # not read
    (cr, sr), (cw, sw) = ref.scaled_rows(x), ref.scaled_matrices(w)
    out = strided(torch.full((rows, n), 7.0, dtype=BF), pad)
    got = mf.scaled_linear(*mf.scaled_quantize(x.to(DEV)), *mf.scaled_quantize_weight(w.to(DEV)), off.to(DEV), out=out)
    assert got is out
    xv, wv = ref.rows_values(cr, sr), ref.matrices_values(cw, sw)
    y, _, on = gref.linear(xv, wv, off)
    assert torch.equal(got[~on.to(DEV)], torch.full_like(got[~on.to(DEV)], 7.0)), "rows of no expert were written"
    assert gref.worst(got[on.to(DEV)], y[on], (ref.half_step(BF) * y.abs() + (1 + 2 ** -8) * ref.product_bound(xv, wv, off))[on]) <= 1.0
    if pad:
        assert torch.isnan(out._base[:, :pad]).all() and torch.isnan(out._base[:, pad + n:]).all()


def test_scaled_input_gradient():
    counts, n, k = [33, 0, 200, 7], 200, 328
    off = offsets_of(counts)
    dy, w = rand((240, n), BF, 1), rand((4, n, k), BF, 2, 0.05)
    _, _, tcodes, tscales = mf.scaled_quantize_weight(w.to(DEV), both=True)
    dx = mf.scaled_linear(*mf.scaled_quantize(dy.to(DEV)), tcodes, tscales, off.to(DEV))
    wt = ref.matrices_values(*ref.scaled_matrices(w))[:, :, :k].transpose(1, 2).contiguous()
    dyv = ref.rows_values(*ref.scaled_rows(dy))[:, :n]
    y, _, _ = gref.linear(dyv, wt, off)
    assert dx.shape == (240, k) and gref.worst(dx, y, ref.half_step(BF) * y.abs() + (1 + 2 ** -8) * ref.product_bound(dyv, wt, off)) <= 1.0


def test_scaled_segments_do_not_touch():
    # an expert's infinities and NaN reach its own results alone, and all of a row's where they are in it
    counts = [40, 70, 90, 33]
    off = offsets_of(counts).to(DEV)
    n, k = 160, 256
    x, w = rand((233, k), BF, 1), rand((4, n, k), BF, 2, 0.05)
    clean = mf.scaled_linear(*mf.scaled_quantize(x.to(DEV)), *mf.scaled_quantize_weight(w.to(DEV)), off)
    xb, wb = x.clone(), w.clone()
    xb[45, 130], wb[3, 140, 5] = INF, NAN
    y = mf.scaled_linear(*mf.scaled_quantize(xb.to(DEV)), *mf.scaled_quantize_weight(wb.to(DEV)), off)
    bad = torch.zeros(233, n, dtype=torch.bool, device=DEV)
    bad[45], bad[200:, 128:] = True, True
    assert torch.isnan(y[bad]).all() and torch.equal(y[~bad], clean[~bad])


def test_scaled_wide_exponents():
    # blocks whose powers lie far apart: the scales of each block count, in every direction
    x = rand((130, 640), F32, 1) * torch.exp2(torch.randint(-40, 40, (130, 5), generator=torch.Generator().manual_seed(2)).float()).repeat_interleave(128, 1)
    w = rand((1, 260, 640), F32, 3)
    w *= torch.exp2(torch.randint(-30, 30, (1, 3, 5), generator=torch.Generator().manual_seed(4)).float()).repeat_interleave(128, 1)[:, :260].repeat_interleave(128, 2)
    got = mf.scaled_linear(*mf.scaled_quantize(x.to(DEV)), *mf.scaled_quantize_weight(w.to(DEV)), offsets_of([130]).to(DEV))
    xv, wv = ref.rows_values(*ref.scaled_rows(x)), ref.matrices_values(*ref.scaled_matrices(w))
    y, _, _ = gref.linear(xv, wv, offsets_of([130]))
    assert gref.worst(got, y, ref.half_step(BF) * y.abs() + (1 + 2 ** -8) * ref.product_bound(xv, wv, offsets_of([130]))) <= 1.0
