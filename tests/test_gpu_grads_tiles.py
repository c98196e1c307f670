"""Every kernel of the expert products on the GPU, at sizes that the library's
own rule sends there (grads_tiles.py), against the plain float64 forms.
"""

import pytest
import torch

import grads_ref as ref
import grads_tiles as gt
import matrix_optimizer_step_owner_amd as mf
from test_gpu_grads import BF, DEV, F32, NAN, _need_gpu, offsets_of, rand, strided, wgrad_bound  # noqa: F401

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": BF, "fp32": F32}


@pytest.mark.parametrize("case", gt.ROWS_CASES, ids=gt.name)
def test_rows(case):
    product, dtype, counts, width, depth, pad, kernel = case
    assert gt.rows_kernel(case) == kernel
    dt = DTYPES[dtype]
    rows = sum(counts)
    off = offsets_of(counts)
    a = rand((rows, depth), dt, 1)
    forward = product == gt.FWD
    w = rand((len(counts), width, depth) if forward else (len(counts), depth, width), dt, 2, 0.05)
    out = strided(torch.full((rows, width), NAN, dtype=dt), pad)
    call, plain = (mf.grouped_linear, ref.linear) if forward else (mf.grouped_linear_dgrad, ref.dgrad)
    got = call(strided(a, pad), w.to(DEV), off.to(DEV), out=out)
    y, mag, on = plain(a, w, off)
    assert on.all()
    assert ref.worst(got, y, ref.half_step(dt) * y.abs() + depth * ref.U * mag) <= 1.0
    if pad:   # what lies between the rows
        wide = out._base
        assert torch.isnan(wide[:, :pad]).all() and torch.isnan(wide[:, pad + width:]).all()


@pytest.mark.parametrize("case", gt.WGRAD_CASES, ids=gt.name)
def test_weight_gradients(case):
    product, dtype, counts, n, k, kernel, parts = case
    assert gt.wgrad_kernel(case) == (kernel, parts)
    dt = DTYPES[dtype]
    rows = sum(counts)
    off = offsets_of(counts)
    # activations whose rows differ in size, so that each has scales of its own
    x = rand((rows, k), F32, 1)
    x = (x * torch.exp2(torch.arange(rows) % 13 - 6.0)[:, None]).to(dt)
    dy = rand((rows, n), dt, 2)
    codes = None
    if product == gt.CKPT:
        cr, sr = ref.ckpt_quantize(x)
        x = torch.from_numpy(ref.ckpt_restore(cr, sr))
        codes, scales = torch.from_numpy(cr).to(DEV), torch.from_numpy(sr).to(DEV)
    dw, mag, terms = ref.wgrad(dy, x, off)
    for beta in (0.0, 1.0):
        old = rand((len(counts), n, k), dt, 3)
        grad = old.to(DEV) if beta else torch.full(old.shape, NAN, dtype=dt, device=DEV)
        old = ref.f64(old) if beta else torch.zeros(old.shape, dtype=torch.float64)
        if codes is None:
            mf.grouped_linear_wgrad(dy.to(DEV), x.to(DEV), off.to(DEV), grad, beta=beta)
        else:
            mf.grouped_linear_wgrad_ckpt(dy.to(DEV), codes, scales, off.to(DEV), grad, beta=beta)
        assert ref.worst(grad, dw + beta * old, wgrad_bound(dw, mag, terms, old, beta, dt)) <= 1.0
