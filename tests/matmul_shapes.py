"""Sizes of the block-scaled product that reach each of its kernels:
(kernel, rows per group or None, rows without groups, columns, k).  What they
reach is checked by test_matmul_shapes.py, what it computes by
test_gpu_fp8_ops.py."""

NAMES = ["16x64", "16x16", "32x32", "far 64x256", "256x256", "128x256", "64x256", "64x128", "64x64"]   # in MatmulShape's order

CASES = [
    ("16x64", [3, 0, 5, 1, 2, 0, 4, 1, 0, 9], 0, 200, 392),
    ("16x64", [1, 2, 0, 3], 0, 130, 2056),
    ("16x16", None, 13, 200, 392),
    ("16x16", None, 16, 70, 4100),
    ("32x32", None, 29, 200, 392),
    ("64x64", None, 300, 600, 392),       # four blocks a step: one step, several and a part of one
    ("64x64", None, 130, 200, 1160),
    ("64x64", None, 70, 130, 512),
    ("64x128", None, 700, 3000, 392),
    ("64x128", None, 40, 200, 100),       # no whole block
    ("64x128", [70, 0, 1, 64, 130, 5], 0, 300, 520),
    ("64x256", None, 2100, 1000, 3080),
    ("64x256", [5] * 100 + [0, 64, 65, 1, 0] * 5 + [3] * 5, 0, 256, 3850),
    ("128x256", None, 1900, 3000, 392),
    ("128x256", None, 2700, 1500, 128),
    ("128x256", [900, 0, 129, 64, 600, 128, 1], 0, 3000, 392),
    ("256x256", None, 2900, 3000, 392),
    ("256x256", None, 2900, 3000, 128),
    ("256x256", None, 2900, 3000, 100),
    ("256x256", [1500, 129, 0, 1, 900, 128, 257, 60], 0, 3000, 256),
]
