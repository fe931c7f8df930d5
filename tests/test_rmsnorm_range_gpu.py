"""gemm_rmsnorm_backward at the ends of the range of its operands, against its
formula in 64 bits: products of intermediate values must not leave fp32's range
where the gradients themselves are in it.

Tolerances count roundings, u = 2^-24 each.  n = h rstd takes one, g = dy w
one, a term g n of the row's sum three in all, the sum itself depth(K) =
44 + K / 1024 additions, the mean, rstd and h two or three more: with ten to
spare, (depth + 10) u of the sum of magnitudes, and 4 u of g.  A term of dw takes two
roundings and at most M + 40 additions.
"""
import numpy as np
import pytest
import torch

from dense_gemm_engineering_bf16_b200 import gemm as G
from operator_refs import F32, TINY, U32, Buffer, normal, rmsnorm_reference
from test_rmsnorm_gpu import depth

pytestmark = pytest.mark.gpu
SIZES = [(3, 96), (300, 200), (3, 700), (310, 3000), (3, 9000), (3, 20001)]


def check(M, K, h, dy, eps):
    """Forward (which gives rstd) and backward on fp32 operands."""
    H, dY = Buffer(M, K, torch.float32, fill=h), Buffer(M, K, torch.float32, fill=dy)
    w = (1 + 0.3 * normal(7, 1, K))[0].cuda()
    Y, RS = Buffer(M, K, torch.bfloat16), Buffer(1, M, torch.float32)
    dH, dW = Buffer(M, K, torch.float32), Buffer(1, K, torch.float32)
    ws = torch.empty(G.gemm_rmsnorm_backward_workspace(M, K), dtype=torch.uint8, device="cuda")
    G.gemm_rmsnorm(H.ptr, None, None, w, Y.ptr, None, None, RS.ptr, M, K, H.ld, 0, 0, Y.ld, 0, F32, F32, eps)
    G.gemm_rmsnorm_backward(dY.ptr, H.ptr, w, RS.ptr, None, dH.ptr, dW.ptr, ws, M, K, dY.ld, H.ld, 0, dH.ld, F32, F32,
                            F32)
    torch.cuda.synchronize()
    y, rs = rmsnorm_reference(H.f64(), w.double().cpu().numpy(), eps)
    got = RS.f64()[0]
    assert np.all(np.isfinite(got)) and np.all(np.abs(got - rs) <= 1e-3 * rs)   # subnormal squares keep few bits
    rs = got[:, None]                                        # the backward pass takes it as given
    n, g = H.f64() * rs, dY.f64() * w.double().cpu().numpy()
    mean = (g * n).mean(axis=1, keepdims=True)
    want = rs * (g - n * mean)
    tol = rs * (np.abs(g) * 4 * U32 + np.abs(n) * np.abs(g * n).mean(axis=1, keepdims=True) * (depth(K) + 10) * U32)
    assert np.all(np.abs(dH.f64() - want) <= tol + np.abs(want) * 3 * U32 + TINY)
    s = np.abs(dY.f64() * n).sum(axis=0)
    assert np.all(np.abs(dW.f64()[0] - (dY.f64() * n).sum(axis=0)) <= s * (M + 42) * U32 + TINY)


@pytest.mark.parametrize("M,K", SIZES)
def test_rows_of_zeros_under_a_subnormal_eps(M, K):
    """rstd is above 2^64, its square above fp32's range; dh = rstd dy w."""
    h = normal(1, M, K) * 1e-3
    h[::2] = 0
    check(M, K, h, normal(2, M, K), 1e-39)


@pytest.mark.parametrize("M,K", SIZES)
@pytest.mark.parametrize("h_scale,dy_scale,eps", [(1e16, 1e23, 1e-5), (1e-18, 1e-22, 1e-38)])
def test_products_of_the_gradient_and_the_row_out_of_range(M, K, h_scale, dy_scale, eps):
    """dy h is above fp32's largest value, or among its subnormals, where dy (h
    rstd) is neither."""
    check(M, K, normal(3, M, K) * h_scale, normal(4, M, K) * dy_scale, eps)
