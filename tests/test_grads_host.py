"""Refusals of the gradient operators (products grouped by expert, 8-bit
checkpoints, embedding) and their host arithmetic, without a GPU: every call
here returns before anything is enqueued, so its pointers are never read.
"""

import ctypes
import os

import pytest
import torch

import grads_ref as ref
import matrix_optimizer_step_owner_amd as mf
from matrix_optimizer_step_owner_amd import _lib

pytestmark = pytest.mark.skipif(not os.path.exists(_lib.LIB_PATH), reason="libmfsdp.so not built")

A = 1 << 40            # addresses that are never read, 1 GiB apart
GB = 1 << 30
X, W, OFF, Y, WS = A, A + GB, A + 2 * GB, A + 3 * GB, A + 4 * GB
BF, F32 = _lib.DTYPE_BF16, _lib.DTYPE_F32
OK, INVALID, UNSUPPORTED, WORKSPACE, ALIAS = 0, 1, 2, 3, 4


def fwd(x=X, ldx=64, w=W, off=OFF, e=4, rows=100, n=32, k=64, dt=BF, y=Y, ldy=32, name="mfsdp_grouped_linear"):
    return getattr(_lib.load(), name)(x, ldx, w, off, e, rows, n, k, dt, y, ldy, None)


def wgrad(dy=X, lddy=32, x=W, ldx=64, off=OFF, e=4, rows=100, n=32, k=64, dt=BF, dw=Y, dwt=BF, beta=0.0, ws=None, wsb=0):
    return _lib.load().mfsdp_grouped_linear_wgrad(dy, lddy, x, ldx, off, e, rows, n, k, dt, dw, dwt, beta, ws, wsb, None)


def wgrad_ckpt(codes=W, scales=WS, rows=100, e=4, dt=BF, dwt=BF, beta=0.0, dw=Y):
    return _lib.load().mfsdp_grouped_linear_wgrad_ckpt(X, 32, codes, scales, OFF, e, rows, 32, 64, dt, dw, dwt, beta, None, 0, None)


@pytest.mark.parametrize("over,want", [
    (dict(e=0), OK), (dict(rows=0), OK), (dict(e=0, x=None, w=None, off=None, y=None), OK),
    (dict(e=-1), INVALID), (dict(rows=-1), INVALID), (dict(n=0), INVALID), (dict(k=0), INVALID),
    (dict(ldx=63), INVALID), (dict(ldy=31), INVALID),
    (dict(x=None), INVALID), (dict(w=None), INVALID), (dict(off=None), INVALID), (dict(y=None), INVALID),
    (dict(x=X + 1), INVALID), (dict(off=OFF + 2), INVALID), (dict(y=Y + 2, dt=F32), INVALID),
    (dict(dt=7), UNSUPPORTED), (dict(k=(1 << 24) + 1, ldx=(1 << 24) + 1), UNSUPPORTED),
    (dict(rows=(1 << 30) + 1), UNSUPPORTED), (dict(e=(1 << 20) + 1), UNSUPPORTED),
    (dict(rows=1 << 28, n=64, ldy=64, k=1, ldx=1, x=A, w=A + 8 * GB, off=A + 9 * GB, y=A + 16 * GB), UNSUPPORTED),   # 2^23 tiles
    (dict(y=X), ALIAS), (dict(y=W + 64), ALIAS), (dict(y=OFF), ALIAS),
    (dict(y=X + 99 * 128 + 126), ALIAS),      # the last element of x
    # columns of one buffer of 100 values a row: x has 64, y the 32 from column 63 on, or from 69 with a row's end in the next
    (dict(ldx=100, ldy=100, y=X + 2 * 63), ALIAS), (dict(ldx=100, ldy=100, y=X + 2 * 69), ALIAS), (dict(ldx=100, ldy=100, y=X - 2 * 31), ALIAS),
])
def test_grouped_linear_refusals(over, want):
    assert fwd(**over) == want


@pytest.mark.parametrize("over,want", [
    (dict(ldx=31), INVALID), (dict(ldy=63), INVALID), (dict(y=None), INVALID), (dict(dt=2), UNSUPPORTED),
    (dict(y=X), ALIAS),
])
def test_dgrad_refusals(over, want):
    base = dict(ldx=32, ldy=64, name="mfsdp_grouped_linear_dgrad")
    assert fwd(**{**base, **over}) == want


@pytest.mark.parametrize("over,want", [
    (dict(e=0), OK), (dict(lddy=31), INVALID), (dict(ldx=63), INVALID), (dict(dw=None), INVALID),
    (dict(dy=None), INVALID), (dict(x=None), INVALID), (dict(beta=float("nan")), INVALID),
    (dict(beta=float("inf")), INVALID), (dict(dt=F32, dwt=BF), UNSUPPORTED), (dict(dwt=5), UNSUPPORTED),
    (dict(dw=X), ALIAS), (dict(dw=W), ALIAS), (dict(dw=OFF), ALIAS),
])
def test_wgrad_refusals(over, want):
    assert wgrad(**over) == want


@pytest.mark.parametrize("over,want", [
    (dict(e=0), OK), (dict(codes=None), INVALID), (dict(scales=None), INVALID), (dict(dt=9), UNSUPPORTED),
    (dict(dw=W), ALIAS), (dict(dw=WS), ALIAS),
])
def test_wgrad_ckpt_refusals(over, want):
    assert wgrad_ckpt(**over) == want


@pytest.mark.parametrize("over,want", [
    (dict(rows=0), OK), (dict(rows=-1), INVALID), (dict(k=0), INVALID), (dict(ld=63), INVALID),
    (dict(x=None), INVALID), (dict(codes=None), INVALID), (dict(scales=None), INVALID), (dict(x=X + 1), INVALID),
    (dict(dt=3), UNSUPPORTED), (dict(k=(1 << 24) + 1, ld=1 << 25), UNSUPPORTED),
    (dict(codes=X), ALIAS), (dict(scales=W), ALIAS), (dict(scales=X + 4), ALIAS),
])
def test_ckpt_refusals(over, want):
    a = {**dict(x=X, ld=64, rows=10, k=64, dt=BF, codes=W, scales=Y), **over}
    lib = _lib.load()
    assert lib.mfsdp_ckpt_quantize(a["x"], a["ld"], a["rows"], a["k"], a["dt"], a["codes"], a["scales"], None) == want
    # restoring writes x and only reads codes and scales, which may be anything
    if over != dict(scales=W):
        assert lib.mfsdp_ckpt_restore(a["codes"], a["scales"], a["rows"], a["k"], a["dt"], a["x"], a["ld"], None) == want


@pytest.mark.parametrize("over,want", [
    (dict(nt=0), OK), (dict(nt=-1), INVALID), (dict(vocab=0), INVALID), (dict(d=0), INVALID), (dict(ldo=7), INVALID),
    (dict(table=None), INVALID), (dict(tokens=None), INVALID), (dict(out=None), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(tokens=W + 4, tb=8), INVALID), (dict(tb=2), UNSUPPORTED), (dict(tdt=4), UNSUPPORTED), (dict(odt=4), UNSUPPORTED),
    (dict(vocab=1 << 31), UNSUPPORTED), (dict(nt=(1 << 28) + 1), UNSUPPORTED), (dict(out=X), ALIAS), (dict(out=W), ALIAS),
])
def test_embedding_refusals(over, want):
    a = {**dict(table=X, tdt=BF, vocab=50, d=8, tokens=W, tb=8, nt=20, scale=1.0, out=Y, ldo=8, odt=BF), **over}
    assert _lib.load().mfsdp_embedding(a["table"], a["tdt"], a["vocab"], a["d"], a["tokens"], a["tb"], a["nt"], a["scale"],
                                       a["out"], a["ldo"], a["odt"], None) == want


def wgrad_ws(e, rows, n, k, dt=BF):
    out = ctypes.c_size_t(7)
    return _lib.load().mfsdp_grouped_linear_wgrad_workspace_size(e, rows, n, k, dt, ctypes.byref(out)), out.value


def test_wgrad_workspace():
    assert wgrad_ws(0, 0, 1, 1) == (OK, 0) and wgrad_ws(256, 32768, 512, 1536) == (OK, 0) and wgrad_ws(4, 100, 32, 64) == (OK, 0)
    assert wgrad_ws(-1, 0, 1, 1)[0] == INVALID and wgrad_ws(1, 1, 0, 1)[0] == INVALID and wgrad_ws(1, 1, 1, 1, 5)[0] == UNSUPPORTED
    assert _lib.load().mfsdp_grouped_linear_wgrad_workspace_size(1, 1, 1, 1, BF, None) == INVALID
    # two small matrices with many rows are summed in parts
    st, need = wgrad_ws(2, 10000, 32, 64)
    assert st == OK and need > 0 and need % (32 * 64 * 4) == 0
    args = dict(e=2, rows=10000, dw=A + 8 * GB)
    assert wgrad(**args) == WORKSPACE and wgrad(**args, ws=WS + 16, wsb=need) == WORKSPACE and wgrad(**args, ws=WS, wsb=need - 1) == WORKSPACE
    assert wgrad(**args, ws=X, wsb=need) == ALIAS and wgrad(**args, ws=args["dw"], wsb=need) == ALIAS


def emb_ws(nt, vocab, d):
    out = ctypes.c_size_t(0)
    return _lib.load().mfsdp_embedding_grad_workspace_size(nt, vocab, d, ctypes.byref(out)), out.value


@pytest.mark.parametrize("over,want", [
    (dict(nt=-1), INVALID), (dict(vocab=0), INVALID), (dict(ld=7), INVALID), (dict(dy=None), INVALID),
    (dict(tokens=None), INVALID), (dict(grad=None), INVALID), (dict(grad=Y + 2), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(beta=float("nan")), INVALID), (dict(tb=1), UNSUPPORTED),
    (dict(dt=6), UNSUPPORTED), (dict(vocab=1 << 31), UNSUPPORTED), (dict(ws=None), WORKSPACE),
    (dict(ws=WS + 128), WORKSPACE), (dict(short=1), WORKSPACE), (dict(grad=X), ALIAS), (dict(grad=WS), ALIAS),
    (dict(ws=X), ALIAS), (dict(ws=W), ALIAS),
])
def test_embedding_grad_refusals(over, want):
    a = {**dict(dy=X, ld=8, dt=BF, tokens=W, tb=8, nt=200, vocab=50, d=8, scale=1.0, beta=0.0, grad=Y, ws=WS, short=0), **over}
    st, need = emb_ws(200, 50, 8)
    assert st == OK
    assert _lib.load().mfsdp_embedding_grad(a["dy"], a["ld"], a["dt"], a["tokens"], a["tb"], a["nt"], a["vocab"], a["d"],
                                            a["scale"], a["beta"], a["grad"], a["ws"], need - a["short"], None) == want


def test_embedding_grad_workspace_size():
    assert emb_ws(0, 50, 8) == (OK, 0)
    st, nb = emb_ws(32768, 100000, 4096)
    # two lists of (token, position), two fp32 rows per 64 positions, an index per
    # four table rows, and little more (digit counts)
    want = 4 * 32768 * 4 + 2 * 512 * 4096 * 4 + 25001 * 4
    assert st == OK and want <= nb <= want + (1 << 17)
    assert emb_ws(-1, 50, 8)[0] == INVALID and emb_ws(1, 0, 8)[0] == INVALID and emb_ws(1, 1 << 31, 8)[0] == UNSUPPORTED
    assert _lib.load().mfsdp_embedding_grad_workspace_size(1, 2, 3, None) == INVALID


def test_python_checks():
    x, w, off = torch.zeros(4, 8), torch.zeros(2, 3, 8), torch.zeros(3, dtype=torch.int32)
    codes, scales = torch.zeros(4, 8, dtype=torch.int8), torch.zeros(4, 1, dtype=torch.uint8)
    for call in (lambda: mf.grouped_linear(x, w, off), lambda: mf.grouped_linear_dgrad(x, w, off),
                 lambda: mf.grouped_linear_wgrad(x, x, off, w), lambda: mf.ckpt_quantize(x), lambda: mf.ckpt_restore(codes, scales),
                 lambda: mf.grouped_linear_wgrad_ckpt(x, codes, scales, off, w), lambda: mf.embedding(x, off),
                 lambda: mf.embedding_grad(x, off, x)):
        with pytest.raises(ValueError, match="GPU"):
            call()
    with pytest.raises(TypeError, match="tensor"):
        mf.grouped_linear([1.0], w, off)


def test_row_strides():
    from matrix_optimizer_step_owner_amd.grads import _rows
    t = torch.zeros(6, 10)
    assert _rows(t, "t") == 10 and _rows(t[:, :4], "t") == 10 and _rows(t[::2], "t") == 20
    assert _rows(t[:1, :4], "t") == 4 and _rows(t[:0, :4], "t") == 4
    assert _rows(t[:, :1], "t") == 10
    for bad in (t.t(), t[:1].expand(5, 10), t[:, ::2]):
        with pytest.raises(ValueError):
            _rows(bad, "t")
    with pytest.raises(ValueError, match="shape"):
        _rows(t, "t", (6, 9))


@pytest.mark.parametrize("top", [127.0, 127.5, 128.0, 254.0, 254.01, 1.0, 63.5, 0.0, 3.4e38, 2.0 ** -126, 128 * 2.0 ** -126])
def test_checkpoint_exponent_of_the_reference(top):
    # the plain form's exponent is the smallest e in [-126, 121] with top <= 127 * 2^e, by trying them
    e = -126
    while top > 127.0 * 2.0 ** e and e < 121:
        e += 1
    codes, scales = ref.ckpt_quantize(torch.tensor([[top, 0.0]], dtype=torch.float64))
    assert int(scales[0, 0]) == e + 127 and abs(codes[0, 0] * 2.0 ** e - top) <= 2.0 ** (e if top > 127.5 * 2.0 ** 121 else e - 1)
