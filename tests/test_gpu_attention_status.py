"""The status word of an attention plan: what a step found stays until it is read."""
import pytest

torch = pytest.importorskip("torch")

from heterogeneous_adapters_lora_gb300 import lora as L
from attn_util import Batch

pytestmark = pytest.mark.gpu

INDEX = L.CODE["LORA_ERR_DEVICE_INDEX"]


def batch(seed=40):
    return Batch([3, 1], [40, 9], heads=(4, 2, 64), page=16, seed=seed, poison=0.5).upload()


def status(b):
    return L.lora_attn_get_status(b.plan)


def test_an_index_outside_the_cache_outlives_the_next_steps():
    b = batch()
    good = b.dtable.clone()
    b.dtable[0, 0] = 1 << 20
    b.run()
    b.dtable.copy_(good)
    for _ in range(3):  # later steps are laid out and run well
        b.build()
        b.run()
    assert status(b) == INDEX
    assert status(b) == 0
    b.check()


def test_bad_lengths_outlive_the_next_steps():
    b = batch()
    b.dkv[0] = -1
    b.build()
    b.dkv[0] = 40
    b.build()
    b.run()
    assert status(b) == INDEX
    b.check()  # also asserts that the word is clear now


@pytest.mark.parametrize("fill", [0x00, 0x09, 0x08, 0xFF])
def test_a_fresh_plan_has_none(fill):
    """Whatever its memory held before: not built yet, and after its first build."""
    b = batch()
    b.plan_buf.fill_(fill)
    size = b.plan_buf.numel()
    L.lora_attn_plan_bind(b.plan, b.desc(), b.plan_buf, size, 4, 2, 0)
    assert status(b) == 0
    b.build()
    assert status(b) == 0
    b.run()
    b.check()


def test_bound_again_over_an_unread_error():
    b = batch()
    b.dkv[0] = -1
    b.build()
    b.dkv[0] = 40
    L.lora_attn_plan_bind(b.plan, b.desc(), b.plan_buf, b.plan_buf.numel(), 4, 2, 0)
    assert status(b) == 0
    b.build()
    b.run()
    b.check()


def test_a_captured_first_build_does_not_clear_at_every_replay():
    b = batch()
    L.lora_attn_plan_bind(b.plan, b.desc(), b.plan_buf, b.plan_buf.numel(), 4, 2, 0)
    good = b.dtable.clone()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        b.build()
        b.run()
    b.dtable[1, 0] = -5
    g.replay()
    b.dtable.copy_(good)
    g.replay()
    g.replay()
    assert status(b) == INDEX
    g.replay()
    assert status(b) == 0
    b.check()
