"""First use of the operators around the products inside a stream capture, in
a process of its own, and the kernels that only some shapes reach."""
import os
import subprocess
import sys

import pytest

from dense_gemm_engineering_bf16_b200 import gemm as G
from test_rmsnorm_gpu import run_back, run_norm
from test_w4_gpu import run as run_w4

pytestmark = pytest.mark.gpu


def test_first_use_inside_a_capture_is_refused():
    child = os.path.join(os.path.dirname(os.path.abspath(__file__)), "operators_capture_child.py")
    r = subprocess.run([sys.executable, child], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("ok"), r.stdout + r.stderr


@pytest.mark.parametrize("yt", [G.OUT_F32, G.OUT_BF16])
@pytest.mark.parametrize("ht", [G.OUT_F32, G.OUT_BF16])
@pytest.mark.parametrize("dt", [G.OUT_F32, G.OUT_BF16])
@pytest.mark.parametrize("K", [700, 8201, 12000, 14999])
def test_back_rows_of_four_eights_per_thread(K, yt, ht, dt):
    """Long rows, with the residual's gradient staged or read directly, and an odd end."""
    run_back(5, K, yt, ht, dt, seed=K)
    run_back(310, K, yt, ht, dt, seed=K, in_place="dR" if yt == dt else None)


@pytest.mark.parametrize("M,K", [(297, 8192), (400, 8193), (600, 4100), (297, 16384)])
@pytest.mark.parametrize("xt", [G.OUT_F32, G.OUT_BF16])
def test_norm_many_long_rows(M, K, xt):
    run_norm(M, K, xt, G.OUT_F32, mx=K % 32 == 0, seed=M)
    run_norm(M, K, xt, G.OUT_BF16, mx=K % 32 == 0, seed=M + 1, in_place=True)


@pytest.mark.parametrize("M", [17, 24, 25, 32, 33, 40, 48, 49, 64, 100])
@pytest.mark.parametrize("group", [32, 256])
def test_w4_every_batch_class(M, group):
    run_w4(M, 390, 2336, group, seed=M)
    run_w4(M, 130, 1056, group, zeros=False, ct=G.OUT_BF16, seed=M + 1)
    run_w4(M, 64, 736, group, seed=M + 2, ints=True)


def test_w4_scales_at_the_ends_of_their_range():
    """Weights go through the product over 64; tiny and huge scales come back exactly."""
    import numpy as np
    import torch
    from operator_refs import Buffer
    from test_w4_gpu import operands, reference
    for e in (-100, 100):
        A, B, S, Z = operands(4, 70, 256, 64, True, 11, ints=True)
        S.t[:] = (S.t.double() * 2.0 ** e).bfloat16()
        C = Buffer(4, 70, torch.float32)
        G.gemm_bf16_w4(A.ptr, B.ptr, S.ptr, Z.ptr, C.ptr, 4, 70, 256, A.ld, B.ld, S.ld, C.ld, 64)
        assert np.array_equal(C.f64(), reference(A, B, S, Z, 64, 256)[0])
