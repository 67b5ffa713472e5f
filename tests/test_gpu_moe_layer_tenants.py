"""lora_moe_layer: what one adapter's weights hold shows in its own tokens alone."""
import math

import pytest

torch = pytest.importorskip("torch")

from moe_layer_util import Layer
from test_gpu_moe_layer_sums import set_adapters

pytestmark = pytest.mark.gpu

BAD = 1  # the adapter whose weights are not finite


def make(T, K, shared, rank, n13=2):
    layer = Layer(T, 3, K, 72, 136, adapters=3, rank=rank, shared=shared, n13=n13, seed=T + rank)
    idx = torch.arange(T) % 4 - 1  # all three adapters and none side by side
    return layer.batch(idx=idx.to(torch.int32)), idx


@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("tensor", ["a13", "b13", "a2", "b2"])
@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("T,K,rank", [(4, 2, 8), (45, 2, 40), (300, 1, 8)])
def test_other_tokens_stay_as_they_are(value, tensor, shared, T, K, rank):
    layer, idx = make(T, K, shared, rank)
    clean = layer.call().clone()
    layer.check()
    w = getattr(layer, tensor)
    w[BAD, ..., 3, 5] = value
    w[BAD, ..., -1, -1] = value
    set_adapters(layer)
    got = layer.call()[:T]
    mine = (idx == BAD).cuda()
    assert torch.equal(got[~mine], clean[:T][~mine])
    if tensor == "b2":  # rows of B are columns of the result
        bad = torch.zeros(72, dtype=torch.bool)
        bad[3] = bad[71] = True
        assert not torch.any(torch.isfinite(got[mine][:, bad]))
        assert torch.equal(got[mine][:, ~bad], clean[:T][mine][:, ~bad])
    else:
        assert not torch.any(torch.isfinite(got[mine]))


@pytest.mark.parametrize("n13", [1, 2])
def test_gate_and_up_in_one_slice_or_two(n13):
    layer, idx = make(30, 2, False, 16, n13)
    clean = layer.call().clone()
    layer.b13[BAD, :, 100, 7] = math.inf
    layer.b13[BAD, :, 136 + 9, 2] = math.nan
    set_adapters(layer)
    got = layer.call()[:30]
    mine = (idx == BAD).cuda()
    assert torch.equal(got[~mine], clean[:30][~mine])
    assert not torch.any(torch.isfinite(got[mine]))
