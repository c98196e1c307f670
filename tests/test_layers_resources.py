"""Resource guards of the gfx950 kernels of routing, the exchange of rows, layer
norm and 8-bit float products (host-side compile, no GPU): nothing in scratch, no
spills, and LDS for as many workgroups per CU as the tiles count on.
"""

from test_build_resources import device_build, kernel_usage, pytestmark  # noqa: F401

KERNELS = {"route_kernel": 10, "route_grad_kernel": 10, "plan_hist_kernel": 1, "plan_place_kernel": 1, "plan_small_kernel": 1, "route_balance_kernel": 1, "dispatch_kernel": 2,
           "combine_kernel": 4, "combine_grad_kernel": 4, "layer_norm_kernel": 20, "layer_norm_grad_kernel": 20, "layer_norm_wide_kernel": 4,
           "layer_norm_columns_kernel": 2, "layer_norm_sum_kernel": 1, "scaled_quantize_kernel": 2, "scaled_weight_kernel": 2, "scaled_tile_kernel": 4}


def test_no_scratch(device_build):
    _, remarks = device_build
    usage = kernel_usage(remarks)
    for name, least in KERNELS.items():
        found = {k: v for k, v in usage.items() if name in k}
        assert len(found) >= least, (name, sorted(usage))
        for k, v in found.items():
            assert v.get("ScratchSize", 0) == 0 and v.get("VGPRs Spill", 0) == 0, (k, v)
            assert v.get("LDS Size", 0) <= 160 * 1024, (k, v)


def test_two_workgroups_fit(device_build):
    _, remarks = device_build
    for k, v in kernel_usage(remarks).items():
        if "scaled_tile_kernel" in k and "Li256ELi256E" not in k:
            assert 2 * v["LDS Size"] <= 160 * 1024, (k, v)
