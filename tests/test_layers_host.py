"""Refusals of routing, the exchange of rows, layer norm and the 8-bit float
products, and their host arithmetic, without a GPU: every call here returns
before anything is enqueued, so its pointers are never read.
"""

import ctypes
import os

import numpy as np
import pytest
import torch

import layers_ref as ref
import matrix_optimizer_step_owner_amd as mf
from matrix_optimizer_step_owner_amd import _lib

pytestmark = pytest.mark.skipif(not os.path.exists(_lib.LIB_PATH), reason="libmfsdp.so not built")

A = 1 << 40            # addresses that are never read, 1 GiB apart
GB = 1 << 30
P = [A + i * GB for i in range(8)]
BF, F32 = _lib.DTYPE_BF16, _lib.DTYPE_F32
OK, INVALID, UNSUPPORTED, WORKSPACE, ALIAS = 0, 1, 2, 3, 4
NAN, INF = float("nan"), float("inf")


def call(name, order, base, over):
    a = {**base, **over}
    assert set(a) == set(order), set(a) ^ set(order)
    return getattr(_lib.load(), name)(*[a[k] for k in order], None)


ROUTE = dict(x=P[0], ld=64, bias=P[1], mask=P[2], t=100, n=64, k=4, dt=BF, sc=0, g=8, top=2, re=1, s=1.0, e=P[3], w=P[4])


@pytest.mark.parametrize("over,want", [
    (dict(t=0), OK), (dict(t=0, x=None, e=None, w=None), OK), (dict(t=-1), INVALID), (dict(n=0), INVALID), (dict(k=0), INVALID), (dict(k=65), INVALID),
    (dict(ld=63), INVALID), (dict(sc=2), INVALID), (dict(sc=-1), INVALID), (dict(g=0), INVALID), (dict(g=7), INVALID), (dict(top=0), INVALID),
    (dict(top=9), INVALID), (dict(k=17), INVALID), (dict(s=NAN), INVALID), (dict(s=INF), INVALID), (dict(x=None), INVALID), (dict(e=None), INVALID),
    (dict(w=None), INVALID), (dict(x=P[0] + 1), INVALID), (dict(bias=P[1] + 2), INVALID), (dict(e=P[3] + 2), INVALID), (dict(dt=5), UNSUPPORTED),
    (dict(n=1025, ld=1025, g=1, top=1), UNSUPPORTED), (dict(k=33, g=1, top=1), UNSUPPORTED), (dict(n=1000, ld=1000, g=100, top=100), UNSUPPORTED),
    (dict(t=1 << 25), UNSUPPORTED), (dict(ld=(1 << 22) + 1), UNSUPPORTED), (dict(e=P[0]), ALIAS), (dict(w=P[0] + 99 * 128 + 124), ALIAS),
    (dict(w=P[3]), ALIAS), (dict(e=P[1]), ALIAS), (dict(e=P[2]), ALIAS),
])
def test_route_refusals(over, want):
    assert call("mfsdp_route", list(ROUTE), ROUTE, over) == want


GRAD = dict(dw=P[0], x=P[1], ld=64, e=P[2], t=100, n=64, k=4, dt=BF, sc=1, re=1, s=1.0, out=P[3], ldo=64)


@pytest.mark.parametrize("over,want", [
    (dict(t=0), OK), (dict(t=-1), INVALID), (dict(k=65), INVALID), (dict(ld=63), INVALID), (dict(ldo=63), INVALID), (dict(sc=3), INVALID),
    (dict(s=NAN), INVALID), (dict(dw=None), INVALID), (dict(x=None), INVALID), (dict(e=None), INVALID), (dict(out=None), INVALID),
    (dict(out=P[3] + 1), INVALID), (dict(dt=9), UNSUPPORTED), (dict(k=33), UNSUPPORTED), (dict(out=P[1]), ALIAS), (dict(out=P[0]), ALIAS), (dict(out=P[2]), ALIAS),
])
def test_route_grad_refusals(over, want):
    assert call("mfsdp_route_grad", list(GRAD), GRAD, over) == want


PLAN = dict(e=P[0], t=100000, k=4, n=64, off=P[1], place=P[2], ws=P[3], wsb=1 << 20)


@pytest.mark.parametrize("over,want", [
    (dict(t=-1), INVALID), (dict(k=0), INVALID), (dict(n=0), INVALID), (dict(off=None), INVALID), (dict(e=None), INVALID), (dict(place=None), INVALID),
    (dict(e=P[0] + 1), INVALID), (dict(n=1025), UNSUPPORTED), (dict(k=33), UNSUPPORTED), (dict(t=(1 << 28) + 1), UNSUPPORTED), (dict(t=1 << 62), UNSUPPORTED),
    (dict(ws=None), WORKSPACE), (dict(ws=P[3] + 128), WORKSPACE), (dict(wsb=1000), WORKSPACE), (dict(place=P[0]), ALIAS), (dict(off=P[2] + 64), ALIAS),
    (dict(ws=P[0]), ALIAS),
])
def test_route_plan_refusals(over, want):
    assert call("mfsdp_route_plan", list(PLAN), PLAN, over) == want


def size_of(name, *args):
    out = ctypes.c_size_t(7)
    return getattr(_lib.load(), name)(*args, ctypes.byref(out)), out.value


def test_workspace_sizes():
    assert size_of("mfsdp_route_plan_workspace_size", 0, 1, 1) == (OK, 0) and size_of("mfsdp_route_plan_workspace_size", 512, 8, 256) == (OK, 0)
    st, need = size_of("mfsdp_route_plan_workspace_size", 32768, 8, 256)
    assert st == OK and 0 < need <= 512 * 256 * 4
    assert size_of("mfsdp_route_plan_workspace_size", -1, 1, 1)[0] == INVALID and size_of("mfsdp_route_plan_workspace_size", 1, 33, 64)[0] == UNSUPPORTED
    assert _lib.load().mfsdp_route_plan_workspace_size(1, 1, 1, None) == INVALID
    assert size_of("mfsdp_layer_norm_grad_workspace_size", 0, 64, BF, 1) == (OK, 0)
    one, two = (size_of("mfsdp_layer_norm_grad_workspace_size", 16384, 5120, BF, b)[1] for b in (0, 1))
    assert 0 < one < two <= 2 * 2048 * 5120 * 4
    assert size_of("mfsdp_layer_norm_grad_workspace_size", -1, 64, BF, 1)[0] == INVALID
    assert size_of("mfsdp_layer_norm_grad_workspace_size", 1, 64, 7, 1)[0] == UNSUPPORTED
    assert _lib.load().mfsdp_layer_norm_grad_workspace_size(1, 1, BF, 0, None) == INVALID


@pytest.mark.parametrize("over,want", [
    (dict(n=0), INVALID), (dict(rate=NAN), INVALID), (dict(b=None), INVALID), (dict(c=None), INVALID), (dict(b=P[0] + 2), INVALID), (dict(c=P[1] + 4, cb=8), INVALID),
    (dict(cb=2), UNSUPPORTED), (dict(n=1025), UNSUPPORTED), (dict(c=P[0]), ALIAS),
])
def test_balance_refusals(over, want):
    base = dict(b=P[0], c=P[1], cb=4, n=64, rate=0.1)
    assert call("mfsdp_route_balance", list(base), base, over) == want


DISPATCH = dict(x=P[0], ldx=40, place=P[1], t=10, k=2, rows=20, d=40, dt=BF, out=P[2], ldo=40)
COMBINE = dict(h=P[0], ldh=40, place=P[1], w=P[3], t=10, k=2, rows=20, d=40, dt=BF, beta=0.0, y=P[2], ldy=40)
COMBINE_GRAD = dict(dy=P[4], lddy=40, h=P[0], ldh=40, place=P[1], w=P[3], t=10, k=2, rows=20, d=40, dt=BF, dh=P[2], lddh=40, dw=P[5])


@pytest.mark.parametrize("over,want", [
    (dict(t=0), OK), (dict(t=-1), INVALID), (dict(k=0), INVALID), (dict(rows=-1), INVALID), (dict(d=0), INVALID), (dict(ldx=39), INVALID), (dict(ldo=39), INVALID),
    (dict(x=None), INVALID), (dict(place=None), INVALID), (dict(out=None), INVALID), (dict(x=P[0] + 1), INVALID), (dict(place=P[1] + 2), INVALID),
    (dict(dt=4), UNSUPPORTED), (dict(k=33), UNSUPPORTED), (dict(ldx=(1 << 22) + 1), UNSUPPORTED), (dict(rows=(1 << 30) + 1), UNSUPPORTED), (dict(t=1 << 62, k=2), UNSUPPORTED),
    (dict(out=P[0]), ALIAS), (dict(out=P[1]), ALIAS), (dict(out=P[0] + 9 * 80 + 78), ALIAS),
])
def test_dispatch_refusals(over, want):
    assert call("mfsdp_route_dispatch", list(DISPATCH), DISPATCH, over) == want


@pytest.mark.parametrize("over,want", [
    (dict(t=0), OK), (dict(ldh=39), INVALID), (dict(ldy=39), INVALID), (dict(beta=NAN), INVALID), (dict(h=None), INVALID), (dict(y=None), INVALID),
    (dict(w=P[3] + 2), INVALID), (dict(dt=4), UNSUPPORTED), (dict(y=P[0]), ALIAS), (dict(y=P[3]), ALIAS), (dict(y=P[1]), ALIAS),
])
def test_combine_refusals(over, want):
    assert call("mfsdp_route_combine", list(COMBINE), COMBINE, over) == want


@pytest.mark.parametrize("over,want", [
    (dict(t=0), OK), (dict(lddy=39), INVALID), (dict(lddh=39), INVALID), (dict(w=None), INVALID), (dict(dw=None), INVALID), (dict(dy=None), INVALID),
    (dict(h=None), INVALID), (dict(dh=None), INVALID), (dict(dh=P[0]), ALIAS), (dict(dh=P[4]), ALIAS), (dict(dw=P[3]), ALIAS), (dict(dw=P[2]), ALIAS),
])
def test_combine_grad_refusals(over, want):
    assert call("mfsdp_route_combine_grad", list(COMBINE_GRAD), COMBINE_GRAD, over) == want


NORM = dict(x=P[0], ldx=40, w=P[1], b=P[2], wdt=F32, rows=10, d=40, dt=BF, c=1, eps=1e-5, y=P[3], ldy=40)
NORM_GRAD = dict(dy=P[4], lddy=40, x=P[0], ldx=40, w=P[1], wdt=F32, rows=10, d=40, dt=BF, c=1, eps=1e-5, beta=0.0, dx=P[3], lddx=40, dw=P[5], db=P[6], ws=P[7], wsb=1 << 20)


@pytest.mark.parametrize("over,want", [
    (dict(rows=0), OK), (dict(rows=-1), INVALID), (dict(d=0), INVALID), (dict(ldx=39), INVALID), (dict(ldy=39), INVALID), (dict(eps=-1.0), INVALID),
    (dict(eps=NAN), INVALID), (dict(x=None), INVALID), (dict(w=None), INVALID), (dict(y=None), INVALID), (dict(w=P[1] + 2), INVALID), (dict(b=P[2] + 1), INVALID),
    (dict(dt=4), UNSUPPORTED), (dict(wdt=4), UNSUPPORTED), (dict(d=(1 << 22) + 1, ldx=1 << 23, ldy=1 << 23), UNSUPPORTED), (dict(rows=(1 << 30) + 1), UNSUPPORTED),
    (dict(y=P[0]), ALIAS), (dict(y=P[1]), ALIAS), (dict(y=P[2]), ALIAS),
])
def test_norm_refusals(over, want):
    assert call("mfsdp_layer_norm", list(NORM), NORM, over) == want


@pytest.mark.parametrize("over,want", [
    (dict(rows=-1), INVALID), (dict(lddy=39), INVALID), (dict(lddx=39), INVALID), (dict(beta=INF), INVALID), (dict(dy=None), INVALID), (dict(dw=None), INVALID),
    (dict(dx=None), INVALID), (dict(dw=P[5] + 2), INVALID), (dict(db=P[6] + 2), INVALID), (dict(ws=None), WORKSPACE), (dict(ws=P[7] + 16), WORKSPACE),
    (dict(wsb=100), WORKSPACE), (dict(dx=P[4]), ALIAS), (dict(dx=P[0]), ALIAS), (dict(dw=P[6]), ALIAS), (dict(ws=P[5]), ALIAS), (dict(dw=P[1]), ALIAS),
    (dict(db=P[3]), ALIAS),
])
def test_norm_grad_refusals(over, want):
    assert call("mfsdp_layer_norm_grad", list(NORM_GRAD), NORM_GRAD, over) == want


@pytest.mark.parametrize("over,want", [
    (dict(rows=0), OK), (dict(rows=-1), INVALID), (dict(k=0), INVALID), (dict(ld=39), INVALID), (dict(x=None), INVALID), (dict(c=None), INVALID), (dict(s=None), INVALID),
    (dict(c=P[1] + 8), INVALID), (dict(x=P[0] + 1), INVALID), (dict(dt=2), UNSUPPORTED), (dict(k=1 << 22, ld=1 << 22), UNSUPPORTED), (dict(c=P[0]), ALIAS),
    (dict(s=P[1] + 100), ALIAS), (dict(s=P[0] + 2), ALIAS),
])
def test_scaled_quantize_refusals(over, want):
    base = dict(x=P[0], ld=40, rows=10, k=40, dt=BF, c=P[1], s=P[2])
    assert call("mfsdp_scaled_quantize", list(base), base, over) == want


@pytest.mark.parametrize("over,want", [
    (dict(e=0), OK), (dict(e=-1), INVALID), (dict(n=0), INVALID), (dict(w=None), INVALID), (dict(c=None), INVALID), (dict(ts=None), INVALID),
    (dict(c=None, s=None, tc=None, ts=None), INVALID), (dict(tc=P[3] + 8), INVALID), (dict(dt=2), UNSUPPORTED), (dict(n=1 << 22), UNSUPPORTED),
    (dict(c=P[0]), ALIAS), (dict(tc=P[1]), ALIAS), (dict(ts=P[2]), ALIAS),
])
def test_scaled_weight_refusals(over, want):
    base = dict(w=P[0], e=3, n=50, k=40, dt=BF, c=P[1], s=P[2], tc=P[3], ts=P[4])
    assert call("mfsdp_scaled_quantize_weight", list(base), base, over) == want


@pytest.mark.parametrize("over,want", [
    (dict(e=0), OK), (dict(rows=0), OK), (dict(e=-1), INVALID), (dict(n=0), INVALID), (dict(k=0), INVALID), (dict(ldy=49), INVALID), (dict(c=None), INVALID),
    (dict(s=None), INVALID), (dict(wc=None), INVALID), (dict(ws=None), INVALID), (dict(off=None), INVALID), (dict(y=None), INVALID), (dict(c=P[0] + 8), INVALID),
    (dict(wc=P[2] + 4), INVALID), (dict(y=P[5] + 1), INVALID), (dict(off=P[4] + 2), INVALID), (dict(k=1 << 22), UNSUPPORTED), (dict(e=(1 << 20) + 1), UNSUPPORTED),
    (dict(rows=1 << 30, n=4000000, ldy=4000000, k=1), UNSUPPORTED), (dict(y=P[0]), ALIAS), (dict(y=P[3]), ALIAS), (dict(y=P[4]), ALIAS),
])
def test_scaled_linear_refusals(over, want):
    base = dict(c=P[0], s=P[1], wc=P[2], ws=P[3], off=P[4], e=3, rows=10, n=50, k=40, y=P[5], ldy=50)
    assert call("mfsdp_scaled_linear", list(base), base, over) == want


def tile(e, rows, n, k):
    t = _lib.MfsdpGroupedTile()
    st = _lib.load().mfsdp_scaled_linear_tile(e, rows, n, k, ctypes.byref(t))
    return st, t.rows, t.cols, t.wave_sets, t.workgroups


def test_scaled_tiles():
    # the kernels that the GPU tests and the measured cases mean
    assert tile(256, 8, 512, 1536) == (OK, 32, 32, 4, 8 * 16) and tile(8, 128, 14336, 4096)[1:4] == (32, 64, 4)
    assert tile(256, 32771, 512, 1536)[1:4] == (128, 128, 1) and tile(8, 16384, 14336, 4096)[1:4] == (256, 256, 1)
    from test_gpu_layers_calls import TILES
    for shape, counts, n, k in TILES:
        assert tile(len(counts), sum(counts), n, k)[1:3] == shape, (shape, counts, n, k)
    assert {t[0] for t in TILES} == {(32, 32), (32, 64), (128, 128), (256, 256)}
    assert tile(0, 5, 1, 1) == (OK, 0, 0, 0, 0) and tile(-1, 5, 1, 1)[0] == INVALID
    assert _lib.load().mfsdp_scaled_linear_tile(1, 1, 1, 1, None) == INVALID


def test_python_checks():
    x, i = torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32)
    c = torch.zeros(4, 128, dtype=torch.float8_e4m3fn)
    for f in (lambda: mf.route(x, 2), lambda: mf.route_grad(x, x, i), lambda: mf.route_plan(i, 4), lambda: mf.route_balance(x[0], x[0], 0.1),
              lambda: mf.route_dispatch(x, i), lambda: mf.route_combine(x, i), lambda: mf.route_combine_grad(x, x, i, x), lambda: mf.layer_norm(x, x[0]),
              lambda: mf.layer_norm_grad(x, x, x[0], x[0]), lambda: mf.scaled_quantize(x), lambda: mf.scaled_quantize_weight(x[None]),
              lambda: mf.scaled_linear(c, i, c[None], i, i)):
        with pytest.raises(ValueError, match="GPU"):
            f()
    for f in (lambda: mf.route([1.0], 1), lambda: mf.layer_norm(3, x), lambda: mf.scaled_quantize(None), lambda: mf.route_plan([[0]], 2)):
        with pytest.raises(TypeError, match="must be a tensor"):
            f()


# the references themselves, by other means
def test_reference_rounding():
    g = np.random.RandomState(0)
    v = np.concatenate([g.uniform(-448, 448, 2000), g.uniform(-2.0 ** -5, 2.0 ** -5, 2000), [448.0, 17.0, 19.0, 2.0 ** -10, 3 * 2.0 ** -10, 0.0, -0.0]])
    every = np.sort(np.concatenate([[m * 2.0 ** -9 for m in range(8)], [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8) if (e, m) != (15, 7)]]))
    got = np.abs(ref.e4m3(v))
    near = np.abs(np.abs(v)[:, None] - every[None])
    assert np.isin(got, every).all() and np.array_equal(np.abs(got - np.abs(v)), near.min(1))
    assert np.array_equal(ref.e4m3(v), torch.tensor(v).float().to(torch.float8_e4m3fn).double().numpy()) or (torch.tensor(v).float().double().numpy() != v).any()


@pytest.mark.parametrize("top", [448.0, 449.0, 1.75, 1.76, 0.0, 3.4e38, 2.0 ** -126, 449 * 2.0 ** -126, 1.0])
def test_reference_exponent(top):
    e = -126
    while top > 448.0 * 2.0 ** e:
        e += 1
    assert int(ref.scaled_exponent(np.float64(top))) == e


def test_reference_choice():
    # by sorting (key, -index) pairs one row at a time
    g = torch.Generator().manual_seed(1)
    x = torch.randint(-3, 4, (40, 24), generator=g).float()
    bias = torch.randint(0, 3, (24,), generator=g).float() / 4
    for groups, top in ((1, 1), (6, 2), (4, 4)):
        got = ref.route(x, 5, "sigmoid", bias, groups, top)[0]
        s = torch.sigmoid(x.double()) + bias.double()
        for t in range(40):
            size = 24 // groups
            sums = [sum(sorted((float(v) for v in s[t, i * size:(i + 1) * size]), reverse=True)[:2]) for i in range(groups)]
            stay = sorted(range(groups), key=lambda i: (-sums[i], i))[:top]
            order = sorted((e for e in range(24) if e // size in stay), key=lambda e: (-float(s[t, e]), e))
            assert got[t].tolist() == order[:5]


SCALED_LINEAR = dict(c=P[0], s=P[1], wc=P[2], ws=P[3], off=P[4], e=3, rows=0, n=50, k=40, y=P[5], ldy=1 << 22)


@pytest.mark.parametrize("e,rows,n,k,want", [
    (3, 0, (1 << 22) - 128, 40, OK), (3, 0, (1 << 22) - 127, 40, UNSUPPORTED), (3, 0, 50, (1 << 22) - 127, UNSUPPORTED), (0, 5, 50, 1 << 22, UNSUPPORTED),
    (1, 10, 1 << 22, 40, UNSUPPORTED), (1, 1 << 30, 4000000, 1, UNSUPPORTED), (1 << 20, 1 << 30, 128, 128, UNSUPPORTED), ((1 << 20) + 1, 0, 1, 1, UNSUPPORTED),
    (3, -1, 50, 40, INVALID), (3, 0, 0, 40, INVALID),
])
def test_scaled_tile_query_refuses_what_the_product_does(e, rows, n, k, want):
    assert tile(e, rows, n, k)[0] == want
    assert call("mfsdp_scaled_linear", list(SCALED_LINEAR), SCALED_LINEAR, dict(e=e, rows=rows, n=n, k=k)) == want
    if want != OK:      # and leaves what it was given
        t = _lib.MfsdpGroupedTile(rows=7, workgroups=9)
        assert _lib.load().mfsdp_scaled_linear_tile(e, rows, n, k, ctypes.byref(t)) == want and (t.rows, t.workgroups) == (7, 9)
