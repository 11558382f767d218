"""Which kernel a block-scaled product goes to (host code alone, built with
g++, no GPU): the sizes that the GPU tests use reach every one."""

import ctypes
import os
import shutil
import subprocess

import pytest

import matmul_shapes
from rl_weight_refit_amd import binding as B

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def shape(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ not available")
    lib = str(tmp_path_factory.mktemp("shape") / "matmul_shape.so")
    r = subprocess.run([gxx, "-std=c++17", "-Wall", "-shared", "-fPIC", "-I", os.path.join(ROOT, "include"),
                        "-I", os.path.join(ROOT, "rl_weight_refit_amd", "csrc"),
                        os.path.join(ROOT, "tests", "fuzz", "matmul_shape.cpp"), "-o", lib], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
    f = ctypes.CDLL(lib).matmul_shape
    return lambda mm, gathered: matmul_shapes.NAMES[f(ctypes.byref(mm), gathered)]


def test_sizes_reach_their_kernels(shape):
    for name, groups, M, N, K in matmul_shapes.CASES:
        m = sum(groups) if groups else M
        for out in ("bf16", "f16", "f32"):
            for b_rows in (128, 1):
                for index in (0, 300):
                    mm = B.Fp8Matmul(m, N, K, out, groups=len(groups or []), a_rows=index or m, b_block_rows=b_rows,
                                     a_stride=-(-K // 16) * 16, b_stride=-(-K // 16) * 16)
                    assert shape(mm, index > 0) == name, (name, m, N, K, out, b_rows, index)


def test_every_kernel_is_reached():
    dense, grouped = ({c[0] for c in matmul_shapes.CASES if (c[1] is not None) == g} for g in (False, True))
    assert dense | grouped == set(matmul_shapes.NAMES) - {"far 64x256"}
    assert grouped == {"16x64", "64x128", "64x256", "128x256", "256x256"}   # the others never take groups here


def test_operands_beyond_32_bit_offsets(shape):
    """The sizes of test_gpu_ops_far.py, and the last ones that 32 bits reach."""
    far = lambda M, gathered=0, **kw: shape(B.Fp8Matmul(M, 300, 408, "bf16", a_rows=gathered or M, b_block_rows=1, **kw),
                                            gathered > 0) == "far 64x256"
    assert far(700, 4200, a_stride=1 << 20) and not far(700, 4095, a_stride=1 << 20) and far(700, 4096, a_stride=1 << 20)
    assert far(150, a_stride=1 << 25) and far(150, a_stride=1 << 24) and not far(150, a_stride=(1 << 24) - 16)
    assert far(320, b_stride=1 << 25) and not far(320, b_stride=(1 << 24) - 16)
    assert far(150, a_scale_stride=1 << 23) and far(320, b_scale_stride=1 << 22)
    assert not far(30, a_stride=1 << 25)   # few rows stream b
    # strides of a single row mean nothing
    one = B.Fp8Matmul(500, 1, 408, "bf16", a_rows=1, a_stride=1 << 60, a_scale_stride=1 << 60, b_stride=1 << 60, b_scale_stride=1 << 60)
    assert shape(one, True) != "far 64x256"
