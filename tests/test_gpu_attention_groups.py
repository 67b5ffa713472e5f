"""Groups without sequences: more groups than sequences, and steps in which no group has any."""
import os

import pytest

torch = pytest.importorskip("torch")

from heterogeneous_adapters_lora_gb300 import lora as L
from attn_util import Batch


def desc():
    return L.AttnDesc(n_q_heads=4, n_kv_heads=2, head_dim=64, page_size=16, causal=1, scale=0.125)


def test_plans_may_hold_more_groups_than_sequences():
    if not os.path.exists(L.LIB_PATH):
        from heterogeneous_adapters_lora_gb300 import build
        build.build()
    sizes = [L.lora_attn_plan_bytes(desc(), 8, 2, g) for g in (2, 3, 64)]
    assert 0 < sizes[0] < sizes[1] < sizes[2]
    assert L.lora_attn_plan_bytes(desc(), 8, 2, -1) == 0
    assert L.lora_attn_plan_bytes(desc(), 8, 0, 3) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("q,own,groups,prefix", [([1], [5], [0, 0, 1, 1], [7, 30, 9]), ([3], [40], [0, 0, 0, 0, 1], [200, 1, 0, 130]),
                                                 ([1, 1], [0, 20], [0, 1, 1, 1, 1, 2], [64, 9, 8, 7, 0])])
def test_more_groups_than_sequences(q, own, groups, prefix):
    b = Batch(q, own, heads=(4, 2, 64), page=16, groups=groups, prefix_lens=prefix, seed=50).upload()
    b.run()
    b.check()


@pytest.mark.gpu
def test_a_step_without_sequences():
    """A server's groups stay when none of them has a request: nothing is written, and the next step is whole."""
    b = Batch([1, 4], [9, 30], heads=(4, 2, 64), page=16, groups=[0, 1, 2], prefix_lens=[40, 7], seed=51).upload()
    starts = torch.zeros(3, dtype=torch.int32, device="cuda")
    for cu in (b.dcu, None):
        L.lora_attn_build_plan(b.plan, 0, 0, cu, None, 2, starts, b.dpl, 0, 40)
        b.run()
        assert torch.all(b.out == 7.0) and L.lora_attn_get_status(b.plan) == 0
    b.build()
    b.run()
    b.check()
