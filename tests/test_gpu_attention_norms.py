"""Attention by norms of each token's head, and by keys beside the boundaries of blocks, ranges and parts."""
import pytest

torch = pytest.importorskip("torch")

from attn_norms import check_norms, single_out
from attn_util import Batch

pytestmark = pytest.mark.gpu

BATCHES = {
    "few tokens, many keys": (([1, 2], [20000, 9000]), dict(heads=(4, 2, 128), page=64)),
    "single tokens": (([1] * 20, [128 * i + (i % 3) - 1 if i else 1 for i in range(20)]), dict(heads=(8, 2, 128), page=16)),
    "single tokens, one head a key": (([1] * 9, [700 * i + 3 for i in range(9)]), dict(heads=(4, 4, 64), page=32)),
    "a prompt": (([1100], [1100]), dict(heads=(4, 1, 128))),
    "prompts": (([40, 300, 129], [40, 300, 129]), dict(heads=(6, 2, 64))),
    "chunks": (([100, 37], [3000, 1500]), dict(heads=(7, 1, 128), page=16)),
    "one prefix": (([1] * 70, list(range(70))), dict(heads=(8, 2, 64), page=32, groups=[0, 70], prefix_lens=[2900])),
    "prefixes": (([1] * 30, [11 * i for i in range(30)]), dict(heads=(4, 1, 128), page=16, groups=[0, 1, 12, 12, 30],
                                                               prefix_lens=[513, 1290, 64, 127])),
    "prompts behind prefixes": (([50, 1, 200, 3], [50, 400, 200, 90]),
                                dict(heads=(4, 2, 64), page=16, groups=[0, 2, 4], prefix_lens=[900, 257])),
    "not causal": (([90, 5], [1500, 700]), dict(heads=(4, 2, 64), causal=0)),
}


@pytest.mark.parametrize("name", list(BATCHES))
def test_norms(name):
    a, kw = BATCHES[name]
    b = Batch(*a, seed=70, **kw).upload()
    b.run()
    check_norms(b)


@pytest.mark.parametrize("name", list(BATCHES))
def test_keys_beside_boundaries(name):
    a, kw = BATCHES[name]
    b = single_out(Batch(*a, seed=71, **kw)).upload()
    b.run()
    b.check()
