"""The weights of chosen experts where a rounding more than the formula's shows: one
expert alone, scores down to the smallest numbers, large factors.
"""

import pytest
import torch

import layers_ref as ref
import matrix_optimizer_step_owner_amd as mf
from test_gpu_grads import BF, DEV, F32, _need_gpu, rand  # noqa: F401
from test_gpu_layers import logits_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("n,groups,top,biased", [(1, 1, 1, False), (8, 1, 1, True), (60, 1, 1, False), (256, 8, 4, True), (1000, 10, 7, False)])
def test_one_expert_alone_has_the_factor(n, groups, top, biased, kind, dtype):
    # s / (s + 1e-20) is 1 in fp32 for every score from 2^-41 on
    x, bias = logits_of(3000, n, dtype, n), rand((n,), F32, 5, 0.05).to(DEV) if biased else None
    for scale in (1.0, 2.5, 0.1):
        _, w = mf.route(x.to(DEV), 1, scores=kind, bias=bias, groups=groups, top_groups=top, scale=scale)
        assert torch.equal(w, torch.full_like(w, scale))


def test_scores_of_every_size():
    # a sigmoid in fp32: the exponential is off by two half steps, then a sum (below
    # 1 / 2 it passes through once more) and a quotient, each half a step, in terms
    # of its own size; below 2^-126 numbers are whole multiples of 2^-149
    x = torch.linspace(-103.0, 103.0, 4001).view(-1, 1)
    _, w = mf.route(x.to(DEV), 1, scores="sigmoid", renormalize=False)
    want = ref.scores(x, "sigmoid")[0]
    assert (ref.f64(w) - want).abs().le(4 * ref.U * want + 2.0 ** -149).all()
    # a softmax's: its exponential's argument is rounded too, |x - top| half steps
    x = torch.stack([torch.zeros(4001), torch.linspace(-103.0, 0.0, 4001)], 1)
    e, w = mf.route(x.to(DEV), 2, renormalize=False)
    s, _ = ref.scores(x, "softmax")
    want = s.gather(1, e.cpu().long())
    off = (x - x.amax(1, keepdim=True)).gather(1, e.cpu().long()).abs().double()
    # the sum's exponentials are the hardware's, off by (|x| + 2) U of terms whose size falls faster
    assert (ref.f64(w) - want).abs().le((off / 2 + 8) * ref.U * want + 2.0 ** -149).all()


@pytest.mark.parametrize("kind,low", [("sigmoid", -100.0), ("sigmoid", -60.0), ("softmax", 0.0)])
def test_large_factors(kind, low):
    # scale * s / (sum + 1e-20): scale / (sum + 1e-20) alone may pass fp32's range
    x = torch.full((5, 16), low)
    _, w = mf.route(x.to(DEV), 4, scores=kind, scale=1e30)
    _, want, _ = ref.route(x, 4, kind, scale=1e30)
    # as above, and denormal scores' own steps
    assert (ref.f64(w) - want).abs().le(16 * ref.U * want + 2.0 ** -149 / 1e-20 * 1e30 * 8).all()
    assert torch.isfinite(w).all()
