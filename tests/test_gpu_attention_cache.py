"""Caches without rows: whatever a table says, keys and values count as zeros and the status tells of it."""
import pytest

torch = pytest.importorskip("torch")

from heterogeneous_adapters_lora_gb300 import lora as L
from attn_util import Batch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("page,entry", [(0, 0), (0, -3), (0, -128), (16, 0), (16, -1), (128, 0)])
@pytest.mark.parametrize("prefix", [False, True])
def test_no_rows_at_all(page, entry, prefix):
    """n_rows 0 with buffers of known contents behind it: none of them may enter the result."""
    kw = dict(groups=[0, 3], prefix_lens=[40]) if prefix else {}
    b = Batch([1, 1, 30], [40, 5, 40], heads=(4, 2, 64), page=page, seed=30, poison=0.5, **kw).upload()
    b.dk.fill_(1.0)
    b.dv.fill_(3.0)
    b.dtable.fill_(entry)
    args = [b.plan, b.dq, b.dq.stride(0), b.dk, b.dk.stride(0), b.dv, b.dv.stride(0), 0, b.dtable, b.dtable.stride(0)]
    rest = [b.out, b.out.stride(0), b.ws, b.ws_bytes]
    if prefix:
        L.lora_prefix_attention(*args, b.dtable[b.n:], b.dtable.stride(0), *rest)
    else:
        L.lora_prompt_attention(*args, *rest)
    assert L.lora_attn_get_status(b.plan) == L.CODE["LORA_ERR_DEVICE_INDEX"]
    assert torch.all(b.out == 0)
