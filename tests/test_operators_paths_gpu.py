"""Kernels of the operators that only some combinations of size and type reach."""
import numpy as np
import pytest
import torch

from dense_gemm_engineering_bf16_b200 import gemm as G
from operator_refs import BF16, F32, normal
from test_mxfp8_quantize_gpu import run as run_quantize
from test_rmsnorm_gpu import run_back

pytestmark = pytest.mark.gpu


def many_rows():
    """Rows from which the K-major bf16 quantiser takes eight eights per thread."""
    return 16 * torch.cuda.get_device_properties(0).multi_processor_count


@pytest.mark.parametrize("K", [32, 288, 2048, 2080, 16416])
@pytest.mark.parametrize("extra", [-1, 0, 5])
def test_quantize_many_bf16_rows(K, extra):
    M = many_rows() + extra
    if K == 16416 and extra == -1:
        M //= 2                                   # long rows on the other variant too
    x = normal(K + extra, M, K, 1.0)
    x[3, 1], x[M - 1, K - 1], x[M // 2, :32] = float("nan"), -float("inf"), 0.0
    run_quantize(x, BF16, G.KMAJOR)


@pytest.mark.parametrize("yt,ht,dt", [(F32, BF16, BF16), (BF16, F32, BF16), (BF16, BF16, F32), (F32, F32, F32)])
@pytest.mark.parametrize("K", [5, 90, 128, 250, 256, 300, 512])
def test_back_rows_of_one_warp_share_a_block(K, yt, ht, dt):
    """Several rows per block (more rows than SMs), one warp each, with fp32
    operands: the threads' elements lie in two groups."""
    for M in (297, 1000):
        run_back(M, K, yt, ht, dt, residual=M == 1000, seed=K + M)


@pytest.mark.parametrize("K", [13304, 13312, 13313, 13320, 16384])
@pytest.mark.parametrize("dt", [F32, BF16])
def test_back_fp32_rows_on_both_sides_of_shared_memory(K, dt):
    """With dy and h in fp32, two rows fit into shared memory up to 13312
    elements; longer ones take the kernel with two passes over a row."""
    run_back(4, K, F32, F32, dt, seed=K)
    run_back(301, K, F32, F32, dt, residual=False, seed=K + 1)


def test_back_rows_on_both_sides_of_two_eights_per_thread():
    for K in (8184, 8192, 8193, 8200):
        a = run_back(200, K, BF16, BF16, BF16, seed=K)
        b = run_back(200, K, BF16, BF16, BF16, seed=K)
        assert all(np.array_equal(x.f64(), y.f64()) for x, y in zip(a, b))
