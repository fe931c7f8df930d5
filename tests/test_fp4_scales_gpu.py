"""gemm_fp4 under scales of its matrices whose product fp32 does not hold: the
sums times both scales, as far as the result itself is in range.

Codes and block scales of one or a power of two, so that sums and results are
exact: the only roundings are those of results below fp32's normal range."""
import numpy as np
import pytest
import torch

from dense_gemm_engineering_bf16_b200 import gemm as G

from operator_refs import BF16, F32, TORCH

pytestmark = pytest.mark.gpu
NV = G.FP4_NV
ROWS = [1, 40, 90, 1100]        # K split over clusters, whole, single CTAs, pairs


def run(M, ga, gb, c_type, block=448.0, N=1100, K=1024, zeros=False):
    """Ones (code 2) with block scales `block`; A's row 0 zero where asked for."""
    a, b = (torch.full((n, K // 2), 0x22, dtype=torch.uint8, device="cuda") for n in (M, N))
    if zeros:
        a[0] = 0
    byte = int(torch.tensor([block]).to(torch.float8_e4m3fn).view(torch.uint8))
    sa, sb = (torch.full((G.gemm_fp4_scale_bytes(n, K, NV),), byte, dtype=torch.uint8, device="cuda") for n in (M, N))
    ga, gb = (torch.tensor([g], device="cuda", dtype=torch.float32) if g is not None else None for g in (ga, gb))
    c = torch.full((M, 1104), 7.0, dtype=TORCH[c_type], device="cuda")
    G.gemm_fp4(a, sa, ga, b, sb, gb, c, M, N, K, K // 2, K // 2, 1104, NV, c_type)
    G.gemm_check_device_status()
    assert bool((c[:, N:] == 7.0).all())
    return c[:, :N]


@pytest.mark.parametrize("c_type", [F32, BF16])
@pytest.mark.parametrize("M", ROWS)
@pytest.mark.parametrize("ea,eb", [(-80, -80), (-100, -40), (-26, -100), (-63, -63), (-63, -64), (-100, -100), (70, 70),
                                   (100, 27), (64, 64), (100, -100), (-100, 100), (100, 100), (0, -100), (100, 0)])
def test_scales_at_the_ends_of_their_range(ea, eb, M, c_type):
    """Block scales of 2^-9 .. 2^8 around them; K ones: 2^(10 + 2 block + ea + eb)."""
    for block in (2.0 ** 8, 1.0, 2.0 ** -9):
        got = run(M, 2.0 ** ea, 2.0 ** eb, c_type, block).double()
        exact = 2.0 ** (10 + 2 * np.log2(block) + ea + eb)
        want = torch.tensor([exact], dtype=torch.float64).to(torch.float32).to(TORCH[c_type]).double().item()
        assert bool((got == want).all()), (block, got[0, 0].item(), want)


@pytest.mark.parametrize("M", ROWS)
@pytest.mark.parametrize("g", [2.0 ** -100, 2.0 ** -80, 2.0 ** -64, 2.0 ** 64, 2.0 ** 70, 2.0 ** 100])
def test_rows_of_zeros_stay_zero(g, M):
    for c_type in (F32, BF16):
        got = run(M, g, g, c_type, zeros=True)
        assert bool((got[0] == 0).all())


@pytest.mark.parametrize("M", ROWS)
def test_ordinary_scales_are_multiplied_first(M):
    """Bit for bit: the product of the scales in fp32, then the sum times it."""
    for ga, gb in ((0.0081, 0.0021), (None, 3.7), (-0.3, None), (1e-17, 1e-17), (1e18, 1e17), (0.0, 0.5)):
        got = run(M, ga, gb, F32, 1.125)
        alpha = np.float32(1.0 if ga is None else ga) * np.float32(1.0 if gb is None else gb)
        want = np.float32(1024 * 1.125 ** 2) * alpha
        assert bool((got == float(want)).all())
