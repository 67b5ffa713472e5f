"""What an attention plan lays out, read back from its arrays: every tile of queries meets every block of its keys once,
partial results lie apart, and nothing exceeds what the plan and the workspace have room for."""
import random

import pytest

torch = pytest.importorskip("torch")

from heterogeneous_adapters_lora_gb300 import lora as L

pytestmark = pytest.mark.gpu

BLOCK, ROWS, SHORT = 128, 128, 16  # keys of a block, rows of a tile, own keys that the join takes
GUARD = 256


class Plan:
    def __init__(self, heads, q, kv, starts=None, prefix=(), causal=1):
        hq, hkv = heads
        desc = L.AttnDesc(n_q_heads=hq, n_kv_heads=hkv, head_dim=64, page_size=16, causal=causal, scale=1.0)
        caps = (max(1, sum(q)), len(q), len(prefix))
        size = L.lora_attn_plan_bytes(desc, *caps)
        self.buf = torch.full((size + GUARD,), 0xA5, dtype=torch.uint8, device="cuda")
        self.plan = L.AttnPlan()
        L.lora_attn_plan_bind(self.plan, desc, self.buf, size, *caps)
        cu = [0]
        for n in q:
            cu.append(cu[-1] + n)
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        self.keep = [i32(x) for x in (cu, kv, starts or [0], list(prefix) or [0])]
        g = len(prefix)
        L.lora_attn_build_plan(self.plan, len(q), cu[-1], self.keep[0], self.keep[1], g, self.keep[2] if g else None,
                               self.keep[3] if g else None, max(kv), max(prefix) if g else 0)
        assert L.lora_attn_get_status(self.plan) == 0
        words = self.buf[:size].cpu().numpy().view("int32")
        at = lambda p: (p - self.buf.data_ptr()) // 4  # noqa: E731
        c = words[at(self.plan.counters):][:8]
        self.n_items, self.n_part, self.n_tiles, _, self.n_units, self.n_joins = c[:6].tolist()
        take = lambda p, n, w: words[at(p):][:n * w].reshape(n, w).tolist()  # noqa: E731
        p = self.plan
        assert self.n_items <= p.max_items and self.n_units <= self.n_items
        assert self.n_tiles <= p.max_tiles and self.n_part <= p.max_part and self.n_joins <= caps[0]
        self.items, self.units = take(p.items, self.n_items, 8), take(p.units, self.n_units, 16)
        self.joins = take(p.joins, self.n_joins, 12)
        assert torch.all(self.buf[size:] == 0xA5)
        self.check(hq // hkv, cu, kv, starts, prefix, causal)

    def check(self, group, cu, kv, starts, prefix, causal):
        tpi = 2 * (ROWS // group)
        problems = [(-1 - g, cu[starts[g]], cu[starts[g + 1]], p, 0, False) for g, p in enumerate(prefix)]
        for b, k in enumerate(kv):
            g = max((x for x in range(len(prefix)) if starts[x] <= b < starts[x + 1]), default=None)
            problems.append((b, cu[b], cu[b + 1], k, causal, g is not None and prefix[g] > 0))
        want, tiles, joined = {}, 0, set()
        for prob, a, z, keys, ordered, behind in problems:
            for t0 in range(a, z, tpi):
                n = min(tpi, z - t0)
                tiles += 1
                seen = min(keys, keys - (z - a) + (t0 - a) + n) if ordered else keys
                blocks = max(0, -(-seen // BLOCK))
                if prob >= 0 and prefix and z - a == 1 and keys <= SHORT:
                    joined.add(t0)
                    continue
                if blocks or (prob >= 0 and not behind):
                    want[prob, t0] = n, blocks, keys, keys - (z - a) + (t0 - a) + 1 if ordered else keys, prob < 0 or behind
        assert tiles == self.n_tiles
        got = {}
        for it in self.items:
            got.setdefault((it[2], it[0]), []).append(it)
        assert set(got) == set(want)
        rows = []
        for key, its in got.items():
            n, blocks, keys, lim, behind = want[key]
            its.sort(key=lambda x: x[3])
            assert its[0][3] == 0 and its[-1][4] == blocks
            assert all(x[4] == y[3] for x, y in zip(its, its[1:])) and all(x[3] < x[4] for x in its if blocks)
            for it in its:
                assert it[1] == n and it[5] == keys and it[6] == lim
                if len(its) > 1 or behind:
                    rows.append((it[7], n))
                    joined.update(range(it[0], it[0] + n))
                else:
                    assert it[7] == -1
        rows.sort()
        assert all(a + n <= b for (a, n), (b, _) in zip(rows, rows[1:]))
        assert not rows or (rows[0][0] >= 0 and rows[-1][0] + rows[-1][1] <= self.n_part)
        alone = sorted(x for u in self.units for x in (u[:8], u[8:]) if x[1])
        assert alone == sorted(self.items)
        assert sorted(j[0] for j in self.joins) == sorted(joined)


HEADS = [(32, 8), (28, 4), (16, 16), (8, 1), (128, 1), (40, 40), (6, 2), (192, 192), (640, 320), (5, 1)]


@pytest.mark.parametrize("heads", HEADS)
def test_layouts(heads):
    r = random.Random(heads[0] * 1000 + heads[1])
    some = lambda lo, hi: int(round(lo * (hi / lo) ** r.random()))  # noqa: E731
    for turn in range(12):
        n = some(1, 300)
        kind = r.choice(["tokens", "chunks", "mixed"])
        q = [1 if kind == "tokens" else r.choice([0, 1, some(1, 900)]) if kind == "mixed" else some(1, 400) for _ in range(n)]
        if sum(q) == 0:
            q[0] = 3
        longest = r.choice([10, 200, 3000, 40000])
        kv = [r.choice([0, some(1, longest), some(1, longest)]) for _ in range(n)]
        starts, prefix = None, ()
        if r.random() < 0.6:
            g = some(1, n)
            starts = [0] + sorted(r.randint(0, n) for _ in range(g - 1)) + [n]
            prefix = [r.choice([0, some(1, 8000)]) for _ in range(g)]
        Plan(heads, q, kv, starts, prefix, causal=r.choice([1, 1, 0]))


@pytest.mark.parametrize("heads", [(32, 8), (1, 1), (128, 1), (320, 320)])
def test_long_ranges(heads):
    """One token or a few over very many keys, alone and beside short ones."""
    Plan(heads, [1], [1 << 24])
    Plan(heads, [1, 1, 300], [1 << 24, 5, 300])
    Plan(heads, [1] * 40, [17] * 40, [0, 40], [1 << 22])
    Plan(heads, [700], [1 << 20])
