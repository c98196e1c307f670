"""Resource guards of the gradient operators' gfx950 kernels (host-side compile,
no GPU): accumulators, fragments and loads in flight stay in registers (no
scratch, no spills), and the tiles that count on two workgroups per CU leave
room for both in its 160 KB of LDS.
"""

from test_build_resources import device_build, kernel_usage, pytestmark  # noqa: F401

KERNELS = {"grouped_tile_kernel": 1, "grouped_sum_kernel": 2, "ckpt_quantize_kernel": 2, "ckpt_restore_kernel": 2,
           "embedding_kernel": 8, "sort_hist_kernel": 1, "sort_scatter_kernel": 1, "sort_small_kernel": 1, "emb_partial_kernel": 4,
           "emb_rows_kernel": 4}


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
    # tiles of four waves (and of eight over 32 x 64): two workgroups per CU
    _, remarks = device_build
    usage = kernel_usage(remarks)
    pairs = {k: v for k, v in usage.items() if "grouped_tile_kernel" in k and "Li256ELi256E" not in k and "Li128ELi256ELi2ELi4E" not in k
             and "Li32ELi32E" not in k}
    assert len(pairs) >= 10, sorted(usage)
    for k, v in pairs.items():
        assert 2 * v["LDS Size"] <= 160 * 1024, (k, v)
