"""Which kernel an expert product takes (host arithmetic, no GPU): the sizes of
the GPU tests reach the kernels that they name, and the query's refusals.
"""

import os

import pytest

import grads_tiles as gt
from matrix_optimizer_step_owner_amd import _lib

pytestmark = pytest.mark.skipif(not os.path.exists(_lib.LIB_PATH), reason="libmfsdp.so not built")


@pytest.mark.parametrize("case", gt.ROWS_CASES, ids=gt.name)
def test_forward_and_input_gradient_kernels(case):
    assert gt.rows_kernel(case) == case[-1]


@pytest.mark.parametrize("case", gt.WGRAD_CASES, ids=gt.name)
def test_weight_gradient_kernels(case):
    assert gt.wgrad_kernel(case) == case[-2:]


def test_every_kernel_is_reached():
    # bf16 forward and input gradient have eight kernels each (few rows: nine
    # with the forward's), fp32 four (five), weight gradients three
    reached = {(c[0], c[1], c[-1]) for c in gt.ROWS_CASES}
    for p in (gt.FWD, gt.DGRAD):
        few = {gt.FEW} if p == gt.FWD else set()
        assert {k for q, d, k in reached if (q, d) == (p, "bf16")} == {gt.LARGE, gt.WIDE, gt.PAIR, gt.SMALL, gt.ROWS, gt.SQUARE_REG,
                                                                       gt.ROWS_REG} | few
        assert {k for q, d, k in reached if (q, d) == (p, "fp32")} == {gt.SQUARE, gt.ROWS, gt.SQUARE_REG, gt.ROWS_REG} | few
    for p in (gt.WGRAD, gt.CKPT):
        assert {c[-2] for c in gt.WGRAD_CASES if c[0] == p} == {gt.LARGE, gt.SQUARE, gt.SQUARE_REG}


def test_refusals():
    ok, invalid, unsupported = 0, 1, 2
    assert gt.tile(4, 1, 1, 1, 1, "bf16")[0] == invalid and gt.tile(-1, 1, 1, 1, 1, "bf16")[0] == invalid
    assert gt.tile(gt.FWD, -1, 1, 1, 1, "bf16")[0] == invalid and gt.tile(gt.FWD, 1, 1, 0, 1, "bf16")[0] == invalid
    assert gt.tile(gt.FWD, 1, 1, 1, 1, 9)[0] == unsupported and gt.tile(gt.FWD, 1, (1 << 30) + 1, 1, 1, "bf16")[0] == unsupported
    assert _lib.load().mfsdp_grouped_linear_tile(0, 1, 1, 1, 1, _lib.DTYPE_BF16, 1, None) == invalid
    for args in ((gt.FWD, 0, 100, 64, 64), (gt.DGRAD, 4, 0, 64, 64), (gt.WGRAD, 0, 100, 64, 64)):
        status, t = gt.tile(*args, "bf16")
        assert status == ok and (t.rows, t.cols, t.threads, t.workgroups) == (0, 0, 0, 0)
    status, t = gt.tile(gt.WGRAD, 3, 0, 64, 64, "bf16")     # beta * dW, without rows
    assert status == ok and t.workgroups >= 3


def test_tile_limits():
    # counted in the tiles that the call would run: 2^23 of 256 x 256 outputs
    # here, 34 GB of bf16 in 32 x 64 ones
    status, t = gt.tile(gt.FWD, 1, 131072, 131200, 64, "bf16")
    assert status == 0 and (t.rows, t.cols, t.workgroups) == (256, 256, 512 * 513)
    status, t = gt.tile(gt.DGRAD, 1, 131072, 64, 131200, "bf16")
    assert status == 0 and (t.rows, t.cols, t.workgroups) == (256, 256, 512 * 513)
    assert gt.tile(gt.FWD, 1, 1 << 30, 1 << 22, 64, "bf16")[0] == 2       # 2^36 of them
    # operands through registers: in 32 x 64 outputs
    assert gt.tile(gt.FWD, 1, 1 << 28, 64, 1, "bf16")[0] == 2 and gt.tile(gt.FWD, 1, 1 << 27, 64, 1, "bf16")[0] == 0
    assert gt.tile(gt.WGRAD, 1 << 20, 1 << 20, 400, 400, "bf16")[0] == 0 and gt.tile(gt.WGRAD, 1 << 20, 1 << 20, 400, 400, "fp32")[0] == 2


@pytest.mark.parametrize("product", [gt.WGRAD, gt.CKPT])
@pytest.mark.parametrize("n,k,side", [(64, 64, 128), (128, 128, 128), (64, 512, 128), (2048, 128, 128), (96, 1536, 128), (136, 144, 256),
                                      (512, 192, 256), (160, 1536, 256), (512, 1536, 256)])
def test_large_weight_gradient_tiles_have_outputs(product, n, k, side):
    # 256 x 256 tiles, however many there are, only where n and k fill more than
    # half of one
    status, t = gt.tile(product, 256, 32768, n, k, "bf16")
    assert status == 0 and (t.rows, t.cols, t.lds_dma) == (side, side, 1)
