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


# (product, depth, kernel): kernels whose sets of waves share each step
LONG_SUMS = [(gt.FWD, 1 << 20, gt.FEW), (gt.FWD, (1 << 20) + 1, gt.ROWS_REG), (gt.DGRAD, 1 << 20, gt.ROWS),
             (gt.DGRAD, (1 << 20) + 1, gt.ROWS_REG)]


@pytest.mark.parametrize("product,depth,kernel", LONG_SUMS)
def test_long_fp32_sums(product, depth, kernel):
    # A sum in fp32 is a sum of sums of 512 values, so its error does not grow
    # with its whole length: 512 additions within a run, one for each run of a
    # set of waves, one for each set.  All products are 1 + 2^-10: a single long
    # chain loses that fraction at every addition once it has passed 2^14.
    width = 8
    n, k = (width, depth) if product == gt.FWD else (depth, width)
    t = gt.tile(product, 1, 3, n, k, "fp32", gt.aligned("fp32", depth, k))[1]
    assert (t.rows, t.cols, t.threads, t.wave_sets, t.lds_dma) == kernel
    a = torch.ones(3, depth, device=DEV)
    w = torch.full((1, n, k), 1.0 + 2.0 ** -10, device=DEV)
    off = torch.tensor([0, 3], dtype=torch.int32, device=DEV)
    got = (mf.grouped_linear if product == gt.FWD else mf.grouped_linear_dgrad)(a, w, off)
    want = torch.full((3, width), depth * (1.0 + 2.0 ** -10), dtype=torch.float64)
    additions = 512 + -(-depth // (512 * t.wave_sets)) + t.wave_sets + 2
    assert ref.worst(got, want, (ref.half_step(F32) + additions * ref.U) * want) <= 1.0
