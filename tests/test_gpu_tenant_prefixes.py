"""The example that runs the LoRA layers, norms with rotation, cache and attention together."""
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")

from heterogeneous_adapters_lora_gb300 import lora as L

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    spec = importlib.util.spec_from_file_location("tenant_prefixes", os.path.join(ROOT, "examples", "tenant_prefixes.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("heads,page", [((8, 2, 64), 16), ((4, 4, 128), 32)])
def test_layer_steps(heads, page):
    """Every step's attention against a 64-bit one over the cache as the step left it: keys and values read
    through the tables, a tenant's prefix ahead of each of its requests."""
    steps = []

    def visit(layer, b):
        hq, hkv, d = heads
        k, v = layer.k.double().cpu().view(-1, hkv, d), layer.v.double().cpu().view(-1, hkv, d)
        q, out = layer.q.double().cpu().view(-1, hq, d), layer.out.double().cpu().view(-1, hq, d)
        cu, kv, table = b.cu_q.tolist(), b.kv_len.tolist(), b.table.cpu()
        rows_of = lambda line, n: line.long()[torch.arange(n) // page] * page + torch.arange(n) % page  # noqa: E731
        for s in range(b.n):
            rows, ahead = rows_of(table[s], kv[s]), 0
            if b.groups:
                g = max(i for i in range(b.groups) if b.group_start[i] <= s and b.group_start[i + 1] > s)
                ahead = int(b.prefix_len[g])
                rows = torch.cat([rows_of(b.prefix_table.cpu()[g], ahead), rows])
            n = cu[s + 1] - cu[s]
            kk, vv = (x[rows].repeat_interleave(hq // hkv, 1) for x in (k, v))
            score = torch.einsum("ihd,jhd->hij", q[cu[s]:cu[s + 1]], kk) * d ** -0.5
            j, i = torch.arange(ahead + kv[s]), torch.arange(n)
            score[:, j[None, :] > (ahead + kv[s] - n + i)[:, None]] = -float("inf")
            p = torch.softmax(score, -1)
            ref, mag = torch.einsum("hij,jhd->ihd", p, vv), torch.einsum("hij,jhd->ihd", p, vv.abs())
            bound = (2.0 ** -8 + 2.0 ** -10) * mag + 2.0 ** -8 * ref.abs() + 1e-30
            assert torch.all((out[cu[s]:cu[s + 1]] - ref).abs() <= bound)
        steps.append(b.tokens)

    y = example().run(heads=heads, page=page, hidden=256, visit=visit)
    assert len(steps) == 5 and steps[-1] == y.shape[0]
    assert torch.all(torch.isfinite(y.float()))


def test_steps_are_repeatable():
    m = example()
    a, b = m.run(hidden=256), m.run(hidden=256)
    assert torch.equal(a, b)
