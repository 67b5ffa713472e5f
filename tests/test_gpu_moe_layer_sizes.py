"""lora_moe_layer at the sizes it is meant for, against the formula in 64 bits with a tolerance that is a small part of the result.

moe_layer_util's bound adds up absolute values and so grows with the sizes until it allows anything; here sums are taken to
lose what sums of such numbers do.
"""
import pytest

torch = pytest.importorskip("torch")

from heterogeneous_adapters_lora_gb300 import lora as L
from moe_layer_util import Layer

pytestmark = pytest.mark.gpu


def formula(layer, adapters=True):
    """out [T][D] in 64 bits, on the GPU; `adapters` False: without their part."""
    T, K, D, F = layer.T, layer.K, layer.D, layer.F
    x = layer.x[:, :D].cuda().double()
    ids = layer.ids.long()
    out = torch.zeros(T, D, dtype=torch.float64, device="cuda")

    def on(t):
        return t.cuda().double()

    slots = torch.full((T,), -1) if layer.idx is None or not adapters else layer.idx.long()
    for e in range(layer.E):
        at = (ids == e).nonzero()
        if not len(at):
            continue
        t, k = at[:, 0], at[:, 1]
        td = t.cuda()
        gu = x[td] @ on(layer.w13[e, :, :D]).T
        keep = []
        for a in slots[t].unique().tolist():
            if not 0 <= a < layer.adapters or layer.ranks[a] == 0:
                continue
            m = (slots[t] == a).nonzero()[:, 0].cuda()
            r, s, near = layer.ranks[a], layer.scales[a], 0 if layer.shared else e
            b13 = on(layer.b13[a, e, :, :r])
            for j in range(2):
                v = s * (x[td][m] @ on(layer.a13[a, near, j if layer.n13 == 2 else 0, :r]).T)
                gu[m, j * F:(j + 1) * F] += v @ b13[j * F:(j + 1) * F].T
            keep.append((a, m, r, s, near))
        g = gu[:, :F]
        if layer.gelu:
            h = 0.5 * g * (1 + torch.tanh((2 / torch.pi) ** 0.5 * (g + 0.044715 * g ** 3))) * gu[:, F:]
        else:
            h = g * torch.sigmoid(g) * gu[:, F:]
        y = h @ on(layer.w2[e, :, :F]).T
        for a, m, r, s, near in keep:
            y[m] += s * ((h[m] @ on(layer.a2[a, e, :r]).T) @ on(layer.b2[a, near, :, :r]).T)
        w = torch.ones(len(t)) if layer.weights is None else layer.weights[t, k]
        out.index_add_(0, td, w.cuda().double()[:, None] * y)
    return out


def fits(got, want):
    """Whether each number and all of them together are as near as the roundings allow.

    The result's own rounding: 2^-8 of it at most, a third of that squared on average.  A sum of n products is taken by sixteens,
    of which each may cut 2^-23 of the sum so far: n / 16 2^-23, 2^-15 of the numbers' size for 4096 of them.  h is a product
    of two such and, where all are cut alike, off by 3 2^-15, W2 h and the adapters' parts by another 2^-15: below 2^-12 of what a
    row's numbers are like.
    """
    rms = want.square().mean(1, keepdim=True).sqrt()
    off = (got - want).abs()
    each = bool((off <= 2.0 ** -8 * want.abs() + 2.0 ** -12 * rms).all())
    return each and bool(off.square().mean().sqrt() <= (2.0 ** -8 / 3 ** 0.5 + 2.0 ** -12) * want.square().mean().sqrt())


CASES = {
    # 512 pairs over 64 experts, outer tensors shared: several CTAs for a set of slots, units cut
    "shared_64": dict(T=64, E=64, K=8, D=2048, F=1408, adapters=8, rank=16, shared=True),
    # groups of 32 and more pairs with K loops of 32 and 22 blocks
    "batch_256": dict(T=256, E=64, K=8, D=2048, F=1408, adapters=8, rank=16),
    "bare_256": dict(T=256, E=32, K=8, D=2048, F=1408),
    # few large experts, adapters of rank 64 beside shorter ones
    "large_experts": dict(T=96, E=8, K=2, D=2048, F=4096, adapters=4, rank=64, ranks=(64, 9, 0, 33)),
    "one_large_expert": dict(T=200, E=2, K=1, D=4096, F=2048, adapters=3, rank=16, gelu=True),
    # more than 256 pairs and few experts, shared and not, one w13 slice and two
    "shared_300": dict(T=300, E=5, K=2, D=1040, F=520, adapters=3, rank=16, shared=True),
    "shared_one_slice": dict(T=150, E=3, K=2, D=1032, F=264, adapters=4, rank=136, ranks=(136, 7, 64, 129), shared=True, n13=1),
    "one_slice": dict(T=150, E=3, K=2, D=1032, F=264, adapters=4, rank=136, ranks=(136, 7, 64, 129), n13=1),
    # a set of slots for several adapters: more slots than tokens
    "more_slots_than_tokens": dict(T=2, E=4, K=2, D=1024, F=264, adapters=7, rank=16, shared=True),
    "more_slots_than_many_tokens": dict(T=140, E=4, K=2, D=520, F=264, adapters=150, rank=8, shared=True),
    "decode_16": dict(T=16, E=64, K=8, D=2048, F=1408, adapters=8, rank=16),
}


@pytest.mark.parametrize("name", CASES)
def test_against_the_formula(name):
    c = dict(CASES[name])
    layer = Layer(seed=len(name), **c)
    got = layer.call()[:layer.T].double()
    again = layer.call()[:layer.T].double()
    assert int(layer.status) == 0
    want = formula(layer)
    assert fits(got, want)
    assert torch.equal(got, again)
    # what a tolerance that is too wide would let pass
    assert not fits(torch.zeros_like(want), want)
    assert not fits(0.99 * want, want)
    if layer.adapters:
        assert not fits(formula(layer, adapters=False), want)
    if name == "more_slots_than_tokens":
        for idx in ([0, 2], [6, 4], [3, 5], [1, 1]):
            layer.batch(idx=torch.tensor(idx, dtype=torch.int32))
            assert fits(layer.call()[:2].double(), formula(layer))


def test_one_group_of_every_size():
    """A unit that CTAs share, adapters in two lots of 32, 1 to 64 pairs of one expert and more."""
    layer = Layer(140, 1, 1, 2048, 264, adapters=3, rank=24, ranks=(24, 10, 17), seed=3)
    for n in (1, 7, 8, 9, 31, 32, 33, 40, 63, 64, 65, 96, 97, 128, 129, 140):
        ids = torch.full((140, 1), -1, dtype=torch.int32)
        ids[:n] = 0
        layer.batch(ids=ids)
        got = layer.call()[:140].double()
        assert torch.all(got[n:] == 0)
        assert fits(got[:n], formula(layer)[:n])
