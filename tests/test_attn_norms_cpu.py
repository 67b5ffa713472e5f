"""That the checks of attention see what they are for: mistakes planted in the reference."""
import pytest

torch = pytest.importorskip("torch")

from attn_norms import NORM, norm_errors, single_out
from attn_util import Batch


def batch(**kw):
    return Batch([1], [20000], heads=(4, 2, 128), page=64, seed=12, **kw)


def without(b, keys):
    """The reference's output with some keys of the first sequence left out, rounded to bf16."""
    stays = torch.ones(b.kv_lens[0], dtype=torch.bool)
    stays[keys] = False
    rows, n = b.place[0], b.kv_lens[0]
    b.place[0], b.kv_lens[0] = rows[stays], int(stays.sum())
    out = b.reference()[0]
    b.place[0], b.kv_lens[0] = rows, n
    return out.to(torch.bfloat16).double()


@pytest.mark.parametrize("block", [0, 1, 77, 155, 156])
def test_a_lost_block_shows(block):
    b = batch()
    ref = b.reference()[0]
    assert torch.all(norm_errors(ref.to(torch.bfloat16).double(), ref) <= NORM)
    lost = without(b, slice(128 * block, min(20000, 128 * block + 128)))
    assert torch.any(norm_errors(lost, ref) > NORM)


@pytest.mark.parametrize("key", [0, 127, 128, 9983, 9984, 19967, 19968, 19999])
def test_a_lost_key_at_a_boundary_shows(key):
    b = single_out(batch())
    ref, mag = b.reference()
    bound = (2.0 ** -8 + 2.0 ** -10) * mag + 2.0 ** -8 * ref.abs() + 1e-30
    assert torch.equal(ref, mag)
    lost = without(b, [key])
    assert torch.any((lost - ref).abs() > bound)


def test_a_part_of_wrong_weight_shows():
    """Two halves of the keys joined with one half's statistics 5% too large."""
    b = batch()
    ref = b.reference()[0]
    first, second = without(b, slice(10000, 20000)), without(b, slice(0, 10000))
    q, k = b.q[:1, :512].double().view(4, 128), b.k[b.place[0], :256].double().view(-1, 2, 128)
    w = torch.exp(torch.einsum("hgd,jhd->hgj", q.view(2, 2, 128), k) * b.scale).view(4, -1)
    wa, wb = w[:, :10000].sum(1)[None, :, None], w[:, 10000:].sum(1)[None, :, None]
    assert torch.all(norm_errors((first * wa + second * wb) / (wa + wb), ref) <= NORM)
    assert torch.any(norm_errors((first * wa * 1.05 + second * wb) / (wa * 1.05 + wb), ref) > NORM)
