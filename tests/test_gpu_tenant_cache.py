"""The example's steps against the layer's formulas: queries, keys and values from the hidden states, at positions and
cache rows counted here, and attention over the keys of each request in the order in which they came."""
import copy

import pytest

torch = pytest.importorskip("torch")

from attn_norms import NORM, norm_errors
from test_gpu_tenant_prefixes import example

pytestmark = pytest.mark.gpu

# Base output, delta and their sum are rounded to bf16 (2^-8 each of terms up to 1.3 times the sum's size here),
# and the normed and rotated head once more: four times 2^-8 of a head's norm.
QKV = 4 * 2.0 ** -8


class Steps:
    """Runs the example and checks every step; `later` and `below` plant a wrong position or row in the reference."""

    def __init__(self, later=0, below=0, **kw):
        self.later, self.below = later, below
        self.keys, self.count = {}, 0  # by the pages of a request or prefix: its (k, v) so far
        m = example()
        whole = self

        class Batch(m.Batch):
            def __init__(self, seqs, page, prefixes=None):
                self.asked = copy.deepcopy(seqs), copy.deepcopy(prefixes)
                super().__init__(seqs, page, prefixes)

        class Layer(m.Layer):
            def step(self, batch, x):
                self.x = x.clone()
                return super().step(batch, x)

        m.Batch, m.Layer = Batch, Layer
        self.y = m.run(visit=lambda layer, batch: whole.check(layer, batch), **kw)

    def qkv(self, layer, x, adapters):
        W = layer.qkv.W.double().cpu()
        y = x @ W.T
        for a in set(adapters):
            mine = [t for t, b in enumerate(adapters) if b == a]
            A, B = layer.qkv.keep[6 * a:6 * a + 3], layer.qkv.keep[6 * a + 3:6 * a + 6]
            y[mine] += torch.cat([x[mine] @ p.double().cpu().T @ q.double().cpu().T for p, q in zip(A, B)], 1)
        return y

    def turned(self, z, weight, at):
        d = z.shape[-1]
        z = z / (z.pow(2).mean(-1, keepdim=True) + 1e-6).sqrt() * weight.double().cpu()
        ang = torch.tensor(at, dtype=torch.float64)[:, None, None] * 10000.0 ** (-torch.arange(0, d, 2, dtype=torch.float64) / d)
        a, b = z[..., :d // 2], z[..., d // 2:]
        return torch.cat([a * ang.cos() - b * ang.sin(), b * ang.cos() + a * ang.sin()], -1)

    def check(self, layer, batch):
        hq, hkv, d, page = layer.hq, layer.hkv, layer.d, layer.page
        seqs, prefixes = batch.asked
        ahead = [p for p in prefixes for _ in range(p[2])] if prefixes else [([], 0, 0)] * len(seqs)
        tokens = [(s, p, i) for s, p in zip(seqs, ahead) for i in range(s["past"], s["past"] + s["n"])]
        rows = torch.tensor([s["pages"][i // page] * page + i % page + self.below for s, _, i in tokens])
        rows %= layer.k.shape[0]
        at = [p[1] + i + self.later for _, p, i in tokens]
        y = self.qkv(layer, layer.x.double().cpu(), [s["adapter"] for s, _, _ in tokens])
        q, k, v = (z.view(len(tokens), -1, d) for z in y.split([hq * d, hkv * d, hkv * d], 1))
        got_k, got_v = (z.cpu()[rows].double().view(-1, hkv, d) for z in (layer.k, layer.v))
        got_q = layer.q.double().cpu().view(-1, hq, d)
        assert torch.all(norm_errors(got_q, self.turned(q, layer.q_w, at)) <= QKV)
        assert torch.all(norm_errors(got_k, self.turned(k, layer.k_w, at)) <= QKV)
        assert torch.all(norm_errors(got_v, v) <= QKV)
        # every key and value as it came, whatever the cache's tables say later
        for t, (s, _, i) in enumerate(tokens):
            mine = self.keys.setdefault(tuple(s["pages"]), [])
            assert len(mine) == i
            mine.append((got_k[t], got_v[t]))
        out = layer.out.double().cpu().view(-1, hq, d)
        for t, (s, p, i) in enumerate(tokens):
            seen = (self.keys[tuple(p[0])] if p[1] else []) + self.keys[tuple(s["pages"])][:i + 1]
            assert len(seen) == p[1] + i + 1
            kk, vv = (torch.stack([x[n] for x in seen]).repeat_interleave(hq // hkv, 1) for n in (0, 1))
            w = torch.softmax(torch.einsum("hd,jhd->hj", got_q[t], kk) * d ** -0.5, -1)
            assert torch.all(norm_errors(out[t], torch.einsum("hj,jhd->hd", w, vv)) <= NORM)
        self.count += 1


@pytest.mark.parametrize("heads,page", [((8, 2, 64), 16), ((4, 4, 128), 32)])
def test_every_step_from_the_hidden_states(heads, page):
    s = Steps(heads=heads, page=page, hidden=256, requests=7)
    assert s.count == 5 and torch.all(torch.isfinite(s.y.float()))


@pytest.mark.parametrize("planted", [dict(later=1), dict(later=-1), dict(below=1)])
def test_a_wrong_place_shows(planted):
    with pytest.raises(AssertionError):
        Steps(heads=(8, 2, 64), page=16, hidden=256, requests=3, **planted)
