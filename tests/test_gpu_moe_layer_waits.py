"""lora_moe_layer when its waits run out: no fault is provoked, the waits are only made short."""
import pytest

torch = pytest.importorskip("torch")

from heterogeneous_adapters_lora_gb300 import lora as L
from moe_layer_util import Layer

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("limit", [-1, 1, 3])
@pytest.mark.parametrize("adapters", [0, 3])
def test_waits_that_give_up(limit, adapters):
    """Either the result is right or the status says that it is not, and the next call is whole again."""
    layer = Layer(70, 8, 2, 1032, 520, adapters=adapters, rank=16, seed=2)
    want = layer.call().clone()
    layer.check()
    times = 0
    for _ in range(6):
        layer.status.zero_()
        L.lora_set_spin_limit(limit)
        try:
            layer.call()
            torch.cuda.synchronize()
        finally:
            L.lora_set_spin_limit(1 << 20)
        if int(layer.status):
            assert int(layer.status) == L.CODE["LORA_ERR_TIMEOUT"]
            times += 1
        else:
            assert torch.equal(layer.out, want)
        layer.status.zero_()
        layer.out.fill_(7.0)
        assert torch.equal(layer.call(), want)
        assert int(layer.status) == 0
    assert times or limit > 0  # with no poll at all some waits are not over when they are asked


def test_no_status_word():
    layer = Layer(20, 4, 2, 264, 136, adapters=2, rank=8, seed=3)
    want = layer.call().clone()
    word, layer.status = layer.status, None
    L.lora_set_spin_limit(-1)
    try:
        layer.call()
        torch.cuda.synchronize()
    finally:
        L.lora_set_spin_limit(1 << 20)
    layer.status = word
    assert torch.equal(layer.call(), want) and int(word) == 0
