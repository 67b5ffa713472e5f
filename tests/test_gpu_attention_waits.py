"""The attention calls when their waits run out: no fault is provoked, the waits are only made short."""
import pytest

torch = pytest.importorskip("torch")

from heterogeneous_adapters_lora_gb300 import lora as L
from attn_util import Batch

pytestmark = pytest.mark.gpu

BATCHES = {
    "prompts": (([300, 5, 1], [300, 5, 70]), dict(heads=(8, 2, 128))),
    "paged chunks": (([130, 40], [900, 2000]), dict(heads=(14, 2, 64), page=16)),
    "single tokens": (([1] * 60, [40 * i + 1 for i in range(60)]), dict(heads=(8, 2, 128), page=16)),
    "prefixes": (([1] * 40 + [9], list(range(40)) + [20]), dict(heads=(4, 2, 64), page=32, groups=[0, 30, 41],
                                                                prefix_lens=[700, 90])),
    # each CTA has one item of 16 blocks: the warps of its other slot wait for the next unit for
    # more than 10 us, longer than a few polls (1.5 us each at most)
    "one item a CTA": (([1] * 19, [2000 + i for i in range(19)]), dict(heads=(32, 8, 128), page=16)),
}


@pytest.mark.parametrize("limit", [-1, 1])
@pytest.mark.parametrize("name", list(BATCHES))
def test_waits_that_give_up(name, limit):
    """The call ends, the status says so, and the next calls on the same plan and workspace are whole."""
    a, kw = BATCHES[name]
    b = Batch(*a, seed=31, **kw).upload()
    ref = b.reference()
    b.run()
    b.check(ref)
    seen = set()
    for _ in range(3):
        L.lora_set_spin_limit(limit)
        try:
            b.run()
            seen.add(L.lora_attn_get_status(b.plan))
        finally:
            L.lora_set_spin_limit(1 << 20)
        b.out.fill_(7.0)
        b.run()
        b.check(ref)
    assert seen <= {0, L.CODE["LORA_ERR_TIMEOUT"]}
    if name == "one item a CTA":
        assert seen == {L.CODE["LORA_ERR_TIMEOUT"]}
