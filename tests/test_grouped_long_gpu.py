"""Grouped products and gradients whose reductions are longer than the tensor
core sums by itself, up to the largest accepted.  Ones and small integers at
places that are known: every partial sum is exact, so results are exact too."""
import pytest
import torch

from dense_gemm_engineering_bf16_b200 import gemm as G

from operator_refs import BF16, F32, TORCH

pytestmark = pytest.mark.gpu
MOST = (1 << 31) - 1


def ends_of(sizes):
    return torch.tensor(sizes, dtype=torch.int64).cumsum(0).to(torch.int32).cuda()


@pytest.mark.parametrize("layout", [G.KMAJOR, G.MNMAJOR])
@pytest.mark.parametrize("d_type,beta", [(BF16, 0.0), (BF16, 1.0), (F32, 0.0)])
def test_gradient_of_experts_past_a_million_rows(d_type, beta, layout):
    """Several segments, then experts without rows and with a few, for the same CTAs."""
    sizes = [(1 << 20) + 9, 0, 3 << 20, 5, (1 << 20) - 1, 1 << 20] + [0] * 300 + [7] * 300 + [(2 << 20) + 33]
    M, N, K = sum(sizes), 8, 16
    dc, a = (torch.ones(M, n, device="cuda").bfloat16() for n in (N, K))
    high, wide = (N, K) if layout == G.KMAJOR else (K, N)
    db = torch.full((len(sizes), high, wide), 64.0, dtype=TORCH[d_type], device="cuda")
    G.gemm_bf16_grouped_wgrad(dc, a, ends_of(sizes), db, len(sizes), M, N, K, N, K, wide, high * wide, d_type, layout, beta)
    G.gemm_check_device_status()
    want = (torch.tensor(sizes, device="cuda") + 64.0 * beta).to(TORCH[d_type])
    assert torch.equal(db, want[:, None, None].expand_as(db))


@pytest.mark.parametrize("c_type", [BF16, F32])
def test_rows_past_a_million_products(c_type):
    """More tiles than a split of K leaves clusters for."""
    N, K = 128 * 80, (1 << 20) + 72
    a = torch.ones(3, K, dtype=torch.bfloat16, device="cuda")
    b = torch.ones(N, K, dtype=torch.bfloat16, device="cuda")
    b[:, K - 1], b[5, 1 << 20] = 4.0, 9.0
    c = torch.empty(3, N, dtype=TORCH[c_type], device="cuda")
    G.gemm_bf16_grouped(a, b, ends_of([3]), c, 1, 3, N, K, K, K, 0, N, c_type)
    G.gemm_check_device_status()
    want = torch.full((3, N), K + 3.0, device="cuda")
    want[:, 5] += 8
    assert torch.equal(c, want.to(TORCH[c_type]))


def test_rows_of_the_longest_reduction():
    """K = 2^31 - 1, split over a cluster: shares end at the ends of their type."""
    a = torch.zeros(1, MOST + 1, dtype=torch.bfloat16, device="cuda")
    b = torch.zeros(2, MOST + 1, dtype=torch.bfloat16, device="cuda")
    at = [0, 63, 64, (1 << 28) - 1, 1 << 28, (1 << 30) + 5, 7 * (1 << 28), MOST - 64, MOST - 1]
    a[0, at] = torch.arange(1.0, 1.0 + len(at), device="cuda").bfloat16()
    b[0, at], b[1, at[-1]] = 1.0, 3.0
    a[0, MOST] = b[:, MOST] = float("nan")            # of the pitch
    for c_type in (BF16, F32):
        c = torch.empty(1, 8, dtype=TORCH[c_type], device="cuda")
        G.gemm_bf16_grouped(a, b, ends_of([1]), c, 1, 1, 2, MOST, MOST + 1, MOST + 1, 0, 8, c_type)
        G.gemm_check_device_status()
        assert c[0, :2].tolist() == [45.0, 27.0]


@pytest.mark.parametrize("d_type", [BF16, F32])
def test_gradient_of_an_expert_past_2_to_the_30_rows(d_type):
    """One expert with more than 2^30 rows, and later ones on the same CTA with one each."""
    first, N, K, E = (1 << 30) + 100, 8, 8, 300
    M = first + E - 1
    dc, a = (torch.zeros(M, n, dtype=torch.bfloat16, device="cuda") for n in (N, K))
    at = [0, (1 << 20) - 1, 1 << 20, (1 << 29) + 3, (1 << 30) - 1, 1 << 30, (1 << 30) + 63, (1 << 30) + 64, first - 1]
    dc[at, 0] = 1.0
    a[at, 0] = torch.arange(1.0, 1.0 + len(at), device="cuda").bfloat16()
    a[at, 3] = 2.0
    dc[first:], a[first:] = 1.0, 5.0
    db = torch.empty(E, N, K, dtype=TORCH[d_type], device="cuda")
    G.gemm_bf16_grouped_wgrad(dc, a, ends_of([first] + [1] * (E - 1)), db, E, M, N, K, N, K, K, N * K, d_type)
    G.gemm_check_device_status()
    assert db[0, 0].tolist() == [45.0, 0.0, 0.0, 18.0, 0.0, 0.0, 0.0, 0.0]
    assert not bool(db[0, 1:].any()) and bool((db[1:] == 5.0).all())
