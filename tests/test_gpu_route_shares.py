"""lora_moe_route: renormalised weights of experts whose scores are too small for fp32, which a bias has chosen."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from test_gpu_route import check, logits

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,E,k", [(5, 4, 2), (300, 64, 8), (9, 250, 8), (2500, 256, 8), (40, 1000, 32)])
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_shares_of_small_scores(T, E, k, sigmoid, dtype):
    """Logits up to some 400 below the largest, in any order of the biases: scores of 2^-126 to 2^-500, alone and beside others."""
    x = logits(T, E, E, dtype, spread=100.0)
    bias = 10.0 * torch.randn(E, generator=torch.Generator().manual_seed(E))
    check(x, k, sigmoid, bias, renormalize=True)
    check(x, k, sigmoid, bias, renormalize=True, scale=2.5)
    check(x, k, sigmoid, bias)
    check(x - 200.0, k, sigmoid, bias, renormalize=True)
    check(x, k, sigmoid, None, renormalize=True)
    x[:, ::2] = -np.inf
    check(x, k, sigmoid, bias, renormalize=True)


@pytest.mark.parametrize("sigmoid", [False, True])
def test_a_mask_of_the_lowest_number(sigmoid):
    """Masked experts fill the last places, with no share."""
    x = logits(6, 40, 3)
    x[:, 3:] = torch.finfo(torch.float32).min
    check(x, 5, sigmoid, None, renormalize=True)
    check(x, 5, sigmoid, torch.zeros(40), renormalize=True)
    x[:] = torch.finfo(torch.float32).min
    check(x, 5, True, None, renormalize=True)  # nothing has a score
