"""Arguments that no word of gemm_call holds are refused as the library's own
refusals are: GemmError, or with check=False its status.  Nothing is launched."""
import numpy as np
import pytest
import torch

from dense_gemm_engineering_bf16_b200 import gemm as G

INVALID = 1


def wgrad(M=0, beta=0.0, **k):
    """No rows and no columns: nothing to do where the arguments are numbers."""
    return G.gemm_bf16_grouped_wgrad(None, None, None, None, 1, M, 0, 0, 0, 0, 0, 0, beta=beta, stream=0, **k)


@pytest.mark.parametrize("beta", [1e39, -1e300, 10 ** 400, 1j, "1", None])
def test_a_beta_that_fp32_does_not_hold(beta):
    with pytest.raises(G.GemmError) as e:
        wgrad(beta=beta)
    assert e.value.status == INVALID
    assert wgrad(beta=beta, check=False) == INVALID


@pytest.mark.parametrize("beta", [0, 1, True, 3e38, float("inf"), float("nan"), np.float64(0.5), np.float32(2), torch.tensor(0.25)])
def test_a_beta_that_it_holds(beta):
    assert wgrad(beta=beta) == 0


@pytest.mark.parametrize("M", [1 << 63, -(1 << 63) - 1, 10 ** 30, 2.0, "8", None, torch.tensor([1, 2]), torch.tensor(2.5)])
def test_a_size_that_is_no_64_bit_number(M):
    with pytest.raises(G.GemmError) as e:
        wgrad(M=M)
    assert e.value.status == INVALID
    assert wgrad(M=M, check=False) == INVALID


@pytest.mark.parametrize("M", [0, np.int32(0), np.int64(0), torch.tensor(0), False])
def test_a_size_that_is_one(M):
    assert wgrad(M=M) == 0
