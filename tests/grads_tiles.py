"""Sizes that reach each kernel of the expert products, and the kernel that each
is meant to reach, so that a change of the rules cannot drop one unseen.
"""

import ctypes

from matrix_optimizer_step_owner_amd import _lib

FWD, DGRAD, WGRAD, CKPT = 0, 1, 2, 3
CODES = {"bf16": _lib.DTYPE_BF16, "fp32": _lib.DTYPE_F32}

# (outputs of a workgroup, its threads, sets of waves, by LDS DMA)
LARGE = (256, 256, 512, 1, 1)
WIDE = (128, 256, 512, 1, 1)
PAIR = (128, 256, 256, 1, 1)
SMALL = (64, 256, 256, 1, 1)
ROWS = (32, 64, 512, 4, 1)
FEW = (32, 32, 512, 8, 1)
SQUARE = (128, 128, 256, 1, 1)
SQUARE_REG = (128, 128, 256, 1, 0)
ROWS_REG = (32, 64, 512, 4, 0)

# Segments end inside tiles, some within a tile's first 32 rows; widths leave
# some waves of the last tile a few columns and others none; depths end inside
# a step.  Each is (product, dtype, rows of each expert, output width, depth,
# columns before and after each activation row, kernel): `width` and `depth`
# are n and k of the forward and k and n of the input gradient.
RAGGED4 = (701, 0, 130, 769)
RAGGED20 = tuple((173 * i * i) % 563 for i in range(19)) + (903,)
LONG4 = (2305, 1, 1282, 2412)
ROWS_CASES = [
    (p, d, c, w, t, pad, kernel)
    for p in (FWD, DGRAD)
    for d, c, w, t, pad, kernel in [
        ("bf16", LONG4, 2568, 328, 8, LARGE),
        ("bf16", LONG4, 2696, 1032, 0, LARGE),
        ("bf16", RAGGED4, 1928, 1032, 8, WIDE),
        ("bf16", RAGGED4, 1992, 72, 0, WIDE),
        ("bf16", RAGGED20, 2312, 264, 8, PAIR),
        ("bf16", RAGGED20, 2184, 1016, 0, PAIR),
        ("bf16", (577, 423), 1800, 520, 8, SMALL),
        ("bf16", (20, 0, 33, 64, 1, 20, 22, 19, 1), 1000, 2056, 8, ROWS),
        ("fp32", RAGGED4, 1928, 1036, 4, SQUARE),
        ("fp32", LONG4, 1156, 260, 0, SQUARE),
        ("fp32", (20, 0, 33, 64, 1, 20, 22, 19, 1), 1000, 2052, 4, ROWS),
        ("bf16", RAGGED4, 2001, 1031, 0, SQUARE_REG),
        ("bf16", RAGGED4, 1930, 264, 3, SQUARE_REG),
        ("fp32", RAGGED4, 2001, 1031, 3, SQUARE_REG),
        ("bf16", (20, 0, 33, 5), 1001, 333, 1, ROWS_REG),
        ("fp32", (20, 0, 33, 5), 1001, 333, 1, ROWS_REG),
    ]
] + [
    (FWD, "bf16", (5, 0, 3), 200, 1032, 8, FEW),
    (FWD, "fp32", (5, 0, 35), 200, 1036, 4, FEW),
]

# (product, dtype, rows of each expert, n, k, kernel, in parts).  Steps have 32
# rows, and 16 of them share a group of scales in one half of their buffer: the
# long segments run through four groups.
WGRAD_CASES = [
    (p, d, c, n, k, kernel, parts)
    for p in (WGRAD, CKPT)
    for d, c, n, k, kernel, parts in [
        ("bf16", (1700, 37, 0, 513, 260, 1), 1800, 1040, LARGE, False),
        ("bf16", (1700,) + tuple((31 * i) % 97 for i in range(99)), 120, 112, SQUARE, False),
        ("bf16", (100003, 0, 37600), 200, 208, SQUARE, True),
        ("bf16", (20011, 31, 9000), 520, 272, LARGE, True),
        ("bf16", (1700, 37, 0, 513), 331, 205, SQUARE_REG, True),
        ("fp32", (1700, 37, 0, 513, 260, 1), 1160, 1040, SQUARE if p == WGRAD else SQUARE_REG, False),
    ]
]


def tile(product, experts, rows, n, k, dtype, rows_aligned=True):
    out = _lib.MfsdpGroupedTile()
    status = _lib.load().mfsdp_grouped_linear_tile(product, experts, rows, n, k, CODES.get(dtype, dtype), int(rows_aligned),
                                                   ctypes.byref(out))
    return status, out


def aligned(dtype, *widths):
    return all(w * (2 if dtype == "bf16" else 4) % 16 == 0 for w in widths)


def rows_kernel(case):
    """What the library chooses for one of ROWS_CASES."""
    product, dtype, counts, width, depth, pad, _ = case
    n, k = (width, depth) if product == FWD else (depth, width)
    # the activation's rows and the weights'
    status, t = tile(product, len(counts), sum(counts), n, k, dtype, aligned(dtype, depth + 2 * pad, pad, k))
    assert status == 0
    return t.rows, t.cols, t.threads, t.wave_sets, t.lds_dma


def wgrad_kernel(case):
    product, dtype, counts, n, k, _, _ = case
    status, t = tile(product, len(counts), sum(counts), n, k, dtype, aligned(dtype, n, k))
    assert status == 0
    return (t.rows, t.cols, t.threads, t.wave_sets, t.lds_dma), t.part_rows > 0


def name(case):
    product, dtype, counts = case[:3]
    kernel = next(c for c in case if isinstance(c, tuple) and c is not counts)
    return "-".join([("forward", "dgrad", "wgrad", "wgrad_ckpt")[product], dtype, "x".join(map(str, kernel[:2])),
                     f"{kernel[2]}t", "dma" if kernel[4] else "reg", "x".join(str(v) for v in case[3:5])])
