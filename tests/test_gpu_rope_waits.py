"""lora_qk_norm_rope when its waits for copies run out: no fault is provoked, the waits are only made short."""
import pytest

torch = pytest.importorskip("torch")

from heterogeneous_adapters_lora_gb300 import lora as L
from test_gpu_rope import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("limit", [-1, 1, 2])
@pytest.mark.parametrize("heads", [(8, 2, 128), (32, 8, 128)])
def test_waits_that_give_up(limit, heads):
    """Every token is either done right or left alone, the status says so, and the next call is whole again."""
    c = Case(6000, heads=heads, max_pos=500, seed=12)
    whole = [x.clone() for x in (c.run().q, c.k, c.v)]
    c.check()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    L.lora_set_spin_limit(limit)
    try:
        c.run(status)
    finally:
        L.lora_set_spin_limit(1 << 20)
    places = c.slots.long().cuda()
    kept = torch.all(c.q == 7.0, 1)
    for got, want, at in ((c.q, whole[0], None), (c.k, whole[1], places), (c.v, whole[2], places)):
        if at is not None:
            got, want = got[at], want[at]
        assert torch.equal(got[~kept], want[~kept])
        assert torch.all(got[kept] == 7.0)
    assert int(status) == (L.CODE["LORA_ERR_TIMEOUT"] if kept.any() else 0)
    status.zero_()
    c.run(status).check()
    assert int(status) == 0


def test_waits_that_give_up_at_once():
    """With no poll at all some rows are not there yet when their CTA asks for them."""
    c = Case(4000, heads=(32, 8, 128), max_pos=500, seed=13)
    want = c.run().q.clone()
    c.check()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    times = 0
    for _ in range(10):
        status.zero_()
        L.lora_set_spin_limit(-1)
        try:
            c.run(status)
        finally:
            L.lora_set_spin_limit(1 << 20)
        kept = torch.all(c.q == 7.0, 1)
        assert int(status) == (L.CODE["LORA_ERR_TIMEOUT"] if kept.any() else 0)
        assert torch.equal(c.q[~kept], want[~kept])
        times += bool(kept.any())
        assert torch.equal(c.run().q, want)
    assert times
