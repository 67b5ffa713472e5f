"""lora_moe_layer: what its products leave enters the products behind them with all bits of fp32.

Every result here is the difference of two sums that agree in their first 12 bits and are themselves exact in fp32, so what is
left of it in the result shows the bits that the sums were held with.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from heterogeneous_adapters_lora_gb300 import lora as L
from moe_layer_util import Layer, act

pytestmark = pytest.mark.gpu


def set_adapters(layer):
    """The pool's adapters as the layer's host tensors are now."""
    outer, n13, w = 1 if layer.shared else layer.E, layer.n13, 2 * layer.F // layer.n13
    for a, r in enumerate(layer.ranks):
        A = [layer.a13[a, :, j, :r].contiguous().cuda() for j in range(n13)] + [layer.a2[a, :, :r].contiguous().cuda()]
        B = [layer.b13[a, :, j * w:(j + 1) * w, :r].contiguous().cuda() for j in range(n13)] + [layer.b2[a, :, :, :r].contiguous().cuda()]
        L.lora_set_moe(layer.pool, a, r, layer.scales[a], A, [outer] * n13 + [layer.E], B, [layer.E] * n13 + [outer])
        torch.cuda.synchronize()


def pairs_of(n, far):
    """Places (i, j) of the numbers that nearly agree: neighbours, or half of all places apart."""
    return (np.arange(n // 2), np.arange(n // 2) + n // 2) if far else (np.arange(0, n, 2), np.arange(1, n, 2))


# where the two numbers meet: h in W2; A13 x in B13; h in A2; A2 h in B2
@pytest.mark.parametrize("what", ["w2", "b13", "a2", "b2"])
@pytest.mark.parametrize("far", [False, True])
@pytest.mark.parametrize("T", [5, 40])
@pytest.mark.parametrize("shared", [False, True])
def test_differences(what, far, T, shared):
    if what == "w2" and shared:
        pytest.skip("has no adapters")
    D, F, R, E = 200, 136, 24, 2
    g = torch.Generator().manual_seed(T + 2 * far)
    layer = Layer(T, E, 1, D, F, adapters=0 if what == "w2" else 2, rank=R, scales=[1.0, 1.0], shared=shared, seed=T, p_none=0.0,
                  with_weights=False)
    # x: numbers of 8 bits in [1, 2); the last column 2^-12 of such, what two numbers differ by, the one before it 2^-8 of such, in both
    # of them, the third last what the gate takes
    x = (128 + torch.randint(0, 128, (T, D), generator=g)).double() / 128
    x[:, D - 1] *= 2.0 ** -12
    x[:, D - 2] *= 2.0 ** -8
    first, second = pairs_of(F if what in ("w2", "a2", "b2") else R, far)
    n = len(first)
    w13, w2 = torch.zeros(E, 2 * F, D, dtype=torch.float64), torch.zeros(E, D, F, dtype=torch.float64)
    w13[:, :F, D - 3] = 1.0                                   # one gate for all of h
    xs = x.numpy()
    gate = act(xs[:, D - 3], False)[:, None]
    both, tiny = xs[:, D - 2:D - 1], xs[:, D - 1:]
    if layer.adapters:
        for v in (layer.a13, layer.b13, layer.a2, layer.b2):
            v.zero_()
    if what == "b13":
        for r in range(n):                                    # v = x[r] + the column for both, and with the last column
            layer.a13[:, :, 1, first[r], [r, D - 2]] = 1.0
            layer.a13[:, :, 1, second[r], [r, D - 2]] = 1.0
            layer.a13[:, :, 1, second[r], D - 1] = 1.0
        at = np.arange(F) % n
        for f in range(F):
            layer.b13[:, :, F + f, first[at[f]]] = -1.0
            layer.b13[:, :, F + f, second[at[f]]] = 1.0
        for d in range(D):
            w2[:, d, d % F] = 1.0
        want = np.broadcast_to(gate * tiny, (T, D))
        largest = gate * (xs[:, np.arange(D) % F % n] + both)
    else:
        for i in range(n):                                    # u = x[i] + the column for both, and with the last column
            w13[:, F + first[i], [i, D - 2]] = 1.0
            w13[:, F + second[i], [i, D - 2]] = 1.0
            w13[:, F + second[i], D - 1] = 1.0
        if what == "w2":
            at = np.arange(D) % n
            for d in range(D):
                w2[:, d, first[at[d]]] = -1.0
                w2[:, d, second[at[d]]] = 1.0
        elif what == "a2":
            pair = np.arange(R) * 5 % n                       # rank r takes the difference of pair 5 r
            for r in range(R):
                layer.a2[:, :, r, first[pair[r]]] = -1.0
                layer.a2[:, :, r, second[pair[r]]] = 1.0
            at = pair[np.arange(D) % R]
            for d in range(D):
                layer.b2[:, :, d, d % R] = 1.0
        else:
            one, two = pairs_of(R, far)                       # rank `one` takes h of `first`, `two` of `second`
            for r in range(R // 2):
                layer.a2[:, :, one[r], first[r]] = layer.a2[:, :, two[r], second[r]] = 1.0
            at = np.arange(D) % (R // 2)
            for d in range(D):
                layer.b2[:, :, d, one[at[d]]] = -1.0
                layer.b2[:, :, d, two[at[d]]] = 1.0
        want = np.broadcast_to(gate * tiny, (T, D))
        largest = gate * (xs[:, at] + both)
    if layer.adapters:
        set_adapters(layer)
    layer.batch(x=x.to(torch.bfloat16), w13=w13.to(torch.bfloat16), w2=w2.to(torch.bfloat16))
    got = layer.call()[:T].double().cpu().numpy()
    # the result's own rounding; each of the two numbers rounded once or twice to 24 bits (2^-24 of it each time, up to 2^-23
    # in a sum that cuts), and their sum over parts: 10 such steps of the larger one
    off = np.abs(got - want)
    assert np.all(off <= 2.0 ** -8 * np.abs(want) + 10 * 2.0 ** -24 * largest), float((off / (np.abs(want))).max())
