"""Sizes that routing refuses are refused before anything is allocated for them."""

import pytest
import torch

import matrix_optimizer_step_owner_amd as mf
from test_gpu_grads import DEV, _need_gpu  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("k", [-1, 0, 65, 10 ** 12])
def test_numbers_of_choices(k):
    x = torch.zeros(1000, 64, device=DEV)
    before = torch.cuda.max_memory_allocated()
    with pytest.raises(mf.MfsdpError, match="INVALID|UNSUPPORTED"):
        mf.route(x, k)
    assert torch.cuda.max_memory_allocated() - before <= 1 << 20


@pytest.mark.parametrize("n", [-10 ** 12, -1, 0, 1025, 10 ** 12])
def test_numbers_of_experts(n):
    e = torch.zeros(1000, 4, dtype=torch.int32, device=DEV)
    before = torch.cuda.max_memory_allocated()
    with pytest.raises(mf.MfsdpError, match="INVALID|UNSUPPORTED"):
        mf.route_plan(e, n)
    assert torch.cuda.max_memory_allocated() - before <= 1 << 20
