"""The order of the chosen experts where one pair of neighbours alone is too near for
fp32, at each place among them: the pair's order has to be that of 64 bits, with
no other pair near that would send the token there.
"""

import pytest
import torch

import layers_ref as ref
import matrix_optimizer_step_owner_amd as mf
from test_gpu_grads import DEV, _need_gpu  # noqa: F401

pytestmark = pytest.mark.gpu

FAR = 2.0 ** -16        # what fp32 tells apart: its keys are off by under 2^-17 (34 scores of 2^-22 and the key's own rounding)


def one_near_pair(kind, tokens, n, k, j, groups, top, shift):
    """(logits, bias): keys of `shift` and more, far from one another but for the
    chosen ones at places j and j + 1, which are equal before the logits are rounded.
    The last expert takes what is left of a softmax's sum, and is behind all."""
    g = torch.Generator().manual_seed(1000 * n + 10 * k + j)
    unit = 0.9 if kind == "sigmoid" else 4.0 / n        # a softmax's scores sum: 4 (0.05 + 0.95 / 7), and the last one
    bias = (unit * (0.08 * torch.rand(n, generator=g) - 0.04) + shift).float()
    bias[-1] = shift - 5.0
    b = bias.double()
    level = (torch.stack([torch.randperm(n, generator=g) for _ in range(tokens)]) + 0.25 * torch.rand(tokens, n, generator=g)) / n
    key = shift + unit * (0.05 + 0.95 * (level.double() if kind == "sigmoid" else level.double() ** 6))
    key[:, -1] = shift - 4.5
    chosen = ref.order(torch.where(groups_that_stay(key, groups, top), key, torch.tensor(float("nan"), dtype=torch.float64)))[:, :k]
    key.scatter_(1, chosen[:, j + 1:j + 2], key.gather(1, chosen[:, j:j + 1]))
    s = key - b
    if kind == "sigmoid":
        x = torch.log(s / (1 - s))
    else:
        s[:, -1] = 1 - s[:, :-1].sum(1)
        x = torch.log(s)
    return x.float(), bias


def groups_that_stay(key, groups, top):
    t, n = key.shape
    two = key.view(t, groups, -1).topk(2, 2)[0].sum(2)
    stay = torch.zeros(two.shape, dtype=torch.bool).scatter_(1, ref.order(two)[:, :top], True)
    return stay.repeat_interleave(n // groups, 1)


def only_pair(x, bias, kind, k, j, groups, top):
    """Rows where the pair is near, and neither another pair, nor the last chosen and
    the next, nor the border between groups."""
    key = ref.scores(x, kind)[0] + bias.double()
    stay = groups_that_stay(key, groups, top)
    v = torch.where(stay, key, torch.tensor(-float("inf"), dtype=torch.float64)).sort(1, descending=True)[0][:, :k + 1]
    gap = v[:, :-1] - v[:, 1:]
    near = gap < 2.0 ** -24
    alone = near[:, j] & (near.sum(1) == 1) & ((gap > FAR).sum(1) == gap.shape[1] - 1)
    if groups > top:
        two = key.view(*key.shape[:1], groups, -1).topk(2, 2)[0].sum(2).sort(1, descending=True)[0]
        alone &= two[:, top - 1] - two[:, top] > 4 * FAR
    return alone


PLACES = [(2, 0), (3, 0), (3, 1), (8, 0), (8, 3), (8, 5), (8, 6), (32, 0), (32, 17), (32, 30)]


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("n,groups,top,shift", [(64, 1, 1, 0.0), (64, 1, 1, -2.0), (200, 1, 1, 0.0), (256, 8, 4, 0.0), (256, 8, 4, -2.0), (512, 4, 2, 0.0)])
@pytest.mark.parametrize("k,j", PLACES)
def test_one_near_pair(k, j, n, groups, top, shift, kind):
    x, bias = one_near_pair(kind, 400, n, k, j, groups, top, shift)
    alone = only_pair(x, bias, kind, k, j, groups, top)
    assert int(alone.sum()) >= 200
    e, w = mf.route(x.to(DEV), k, scores=kind, bias=bias.to(DEV), groups=groups, top_groups=top)
    want, ww, bound = ref.route(x, k, kind, bias, groups, top)
    assert torch.equal(e.cpu().long()[alone], want[alone])
    assert ref.f64(w)[alone].sub(ww[alone]).abs().le(bound[alone]).all()


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("k,j", PLACES)
def test_zero_beside_a_tiny_logit(k, j, kind):
    # without a bias' help: logit 0 at a lower index than one of 2^-30, which is larger
    n = 64
    x = torch.full((n, n), -3.0) - 0.05 * torch.arange(n)
    for t in range(n):
        at = torch.randperm(n, generator=torch.Generator().manual_seed(t))[:j + 2]
        low, high = sorted(at[:2].tolist())
        x[t, at[2:]] = 1.0 + 0.05 * torch.arange(j).float()
        x[t, low], x[t, high] = 0.0, 2.0 ** -30
    e, _ = mf.route(x.to(DEV), k, scores=kind, bias=torch.zeros(n, device=DEV))
    assert torch.equal(e.cpu().long(), ref.route(x, k, kind, torch.zeros(n))[0])
