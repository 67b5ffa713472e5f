"""The next token of a row of logits (lora_sample) against the formula in 64 bits."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from heterogeneous_adapters_lora_gb300 import lora as L

pytestmark = pytest.mark.gpu

BF16_MAX = float(torch.finfo(torch.bfloat16).max)


def reference_row(x, temperature, top_k, top_p, min_p, u):
    live = np.flatnonzero(x > -np.inf)  # neither -inf nor NaN
    if not live.size:
        return -1, -math.inf
    x = np.minimum(x[live], BF16_MAX) + 0.0
    greedy = not temperature > 0
    order = np.argsort(-x, kind="stable")
    z = (x[order] - x[order[0]]) / (1.0 if greedy else float(temperature))
    p = np.exp(z)
    total = math.fsum(p)
    left = len(p)
    if top_k > 0:
        left = min(left, int(top_k))
    mass = np.cumsum(p[:left])
    if top_p < 1:
        left = min(left, int(np.searchsorted(mass, max(0.0, float(top_p)) * mass[-1], side="left")) + 1)
    if min_p > 0:
        left = max(1, min(left, int(np.count_nonzero(p >= float(min_p)))))
    if greedy:
        left = 1
    u = 0.0 if not u > 0 else min(float(u), 1 - 2.0 ** -24)
    at = min(left - 1, int(np.searchsorted(mass[:left], u * mass[left - 1], side="right")))
    return int(live[order[at]]), float(z[at]) - math.log(total)


def check(x, temperature=None, top_k=None, top_p=None, min_p=None, uniform=None, pad=0, vocab=None):
    """x: [T][V] bf16 on the host; parameters: lists of T, or None."""
    T, V = x.shape
    vocab = V if vocab is None else vocab
    ld = (V + 7) // 8 * 8 + pad
    buf = torch.full((T, ld), 99.0, dtype=torch.bfloat16)
    buf[:, :V] = x
    buf = buf.cuda()
    dev = [None if v is None else torch.tensor(v, dtype=torch.int32 if i == 1 else torch.float32, device="cuda")
           for i, v in enumerate((temperature, top_k, top_p, min_p, uniform))]
    tokens = torch.full((T + 1,), 77, dtype=torch.int32, device="cuda")
    logprobs = torch.full((T + 1,), 77.0, device="cuda")
    L.lora_sample(buf, ld, T, vocab, *dev, tokens, logprobs)
    alone = torch.full((T,), 77, dtype=torch.int32, device="cuda")
    L.lora_sample(buf, ld, T, vocab, *dev, alone, None)
    assert torch.equal(alone, tokens[:T]) and int(tokens[T]) == 77 and float(logprobs[T]) == 77.0
    host = x[:, :vocab].double().numpy()
    given = [None if v is None else v.cpu().numpy() for v in dev]
    for t in range(T):
        args = [d if g is None else g[t] for g, d in zip(given, (1.0, 0, 1.0, 0.0, 0.0))]
        token, logprob = reference_row(host[t], *args)
        assert int(tokens[t]) == token, (t, args)
        got = float(logprobs[t])
        if not math.isfinite(logprob):
            assert got == logprob
        else:
            # the distance to the largest logit, rounded twice (2^-23 of it), and the logarithm of the sum: the sum's rounding
            # (2^-24), log's ulp and a multiple of ln 2 (at most 19 of them, rounded) and their sums, 2^-20 in all
            assert abs(got - logprob) <= 2.0 ** -20 + 2.0 ** -22 * abs(logprob)


def rows(T, V, seed, spread=2.5):
    return (spread * torch.randn(T, V, generator=torch.Generator().manual_seed(seed))).to(torch.bfloat16)


def uniform(T, seed=0):
    return torch.rand(T, generator=torch.Generator().manual_seed(1000 + seed)).tolist()


@pytest.mark.parametrize("V", [1, 2, 7, 8, 9, 255, 256, 257, 4095, 32007, 128256, 257024])
def test_temperature_alone(V):
    check(rows(5, V, V), [0.7, 1.0, 1.3, 0.0, 5.0], uniform=uniform(5, V), pad=8 * (V % 3))


@pytest.mark.parametrize("V", [9, 1000, 50257])
def test_top_k(V):
    T = 12
    check(rows(T, V, V), [1.0] * T, [0, 1, 2, 3, 5, 8, 40, 999, 1000, 50256, 50257, 2 ** 31 - 1], uniform=uniform(T, V))
    check(rows(2, V, V), [1.0] * 2, [-1, -2 ** 31], uniform=uniform(2, V))


@pytest.mark.parametrize("V", [9, 1000, 50257])
def test_top_p(V):
    p = [1.0, 0.999999, 0.95, 0.5, 0.1, 1e-6, 0.0, -1.0, 2.0, math.nan, 1e-30, 0.9]
    check(rows(len(p), V, V), None, None, p, None, uniform(len(p), V))


@pytest.mark.parametrize("V", [9, 1000, 50257])
def test_min_p(V):
    p = [0.0, 1.0, 0.5, 0.05, 1e-3, 1e-9, 1e-30, -1.0, 2.0, math.nan]
    check(rows(len(p), V, V), None, None, None, p, uniform(len(p), V))


@pytest.mark.parametrize("seed", range(4))
def test_all_filters(seed):
    T, r = 64, np.random.RandomState(seed)
    x = rows(T, 20011, seed, [1.0, 2.5, 8.0, 0.01][seed])
    check(x, r.choice([0.0, 0.5, 1.0, 2.0], T).tolist(), r.choice([0, 1, 10, 500, 15000], T).tolist(),
          r.choice([1.0, 0.95, 0.6], T).tolist(), r.choice([0.0, 0.02, 0.3], T).tolist(), r.rand(T).tolist())


def test_numbers_at_the_ends_and_outside():
    u = [0.0, 2.0 ** -24, 1 - 2.0 ** -24, 1.0, 7.0, -1.0, math.nan, 1e-38, math.inf, -math.inf]
    check(rows(len(u), 3001, 1), uniform=u)
    check(rows(len(u), 3001, 1), top_k=[5] * len(u), uniform=u)


def test_nothing_given_is_the_first_column_of_the_order():
    check(rows(3, 501, 2))


def test_temperatures():
    t = [0.0, -1.0, math.nan, math.inf, 1e-3, 1e-9, 1e3, 1e9]
    check(rows(len(t), 2049, 3), t, uniform=uniform(len(t)))


def test_equal_logits():
    """Ties by index, and prefixes that end inside of them: weights of exactly 1, so the borders are exact."""
    x = torch.zeros(10, 64, dtype=torch.bfloat16)
    x[1::2] = -0.0
    x[2, 32:] = -100.0
    u = [i / 10 for i in range(10)]
    check(x, uniform=u)
    check(x, top_k=[1, 2, 3, 4, 5, 31, 32, 33, 63, 64], uniform=u)
    check(x, top_p=[0.5, 0.25, 0.125, 1 / 64, 3 / 64, 63 / 64, 0.75, 0.015, 0.016, 0.3], uniform=u)
    check(x, top_k=[8] * 10, top_p=[0.5, 0.25, 0.125, 0.126, 0.124, 0.875, 0.75, 0.99, 0.01, 0.3], uniform=u)
    check(x, min_p=[1.0] * 10, uniform=u)
    wide = torch.zeros(2, 200000, dtype=torch.bfloat16)  # more equals than 16 bits count
    check(wide, uniform=[0.123456, 0.999])


def test_masked_columns():
    x = rows(9, 5003, 4)
    x[0] = -math.inf
    x[1] = math.nan
    x[2, 1:] = -math.inf
    x[3, ::2] = -math.inf
    x[4, ::3] = math.nan
    x[5, :4000] = torch.finfo(torch.bfloat16).min
    x[6] = torch.finfo(torch.bfloat16).min
    x[7, 100] = math.inf
    x[8, 10:20] = math.inf
    u = uniform(9)
    check(x, uniform=u)
    check(x, [0.0] * 9, uniform=u)
    check(x, [2.0] * 9, [7] * 9, [0.9] * 9, [0.1] * 9, u)


@pytest.mark.parametrize("spread,temperature", [(1e-8, 1e-8), (1e-12, 1.0), (1e4, 1e4), (1e4, 1.0), (1e30, 1e30), (200.0, 300.0),
                                                (3e38, 1e38), (3e38, math.inf), (1e-30, 1e-25), (1e30, 1e-30), (1e-38, 1e-40)])
def test_other_magnitudes(spread, temperature):
    """Logits outside of the range that is counted at once: the same answers."""
    x = rows(6, 3001, 11, spread)
    x[2, :1500] *= 1e-6
    x[3, 7] = 0.0
    x[4, 10] = 40.0
    t = [temperature] * 6
    check(x, t, uniform=uniform(6))
    check(x, t, [0, 3, 100, 1000, 2999, 1], uniform=uniform(6, 1))
    check(x, t, [0, 0, 1000, 0, 0, 5], [0.9, 0.5, 0.99, 0.1, 1.0, 0.7], [0.0, 0.0, 0.0, 0.3, 0.01, 0.0], uniform(6, 2))


def test_logarithm_of_a_share_that_is_nearly_all():
    """One logit above the others: -log(1 + e) for small e, not the logarithm of a rounded sum."""
    x = torch.zeros(4, 999, dtype=torch.bfloat16)
    x[:, 500] = torch.tensor([16.0, 20.0, 28.0, 40.0], dtype=torch.bfloat16)
    buf, tokens, logprobs = torch.zeros(4, 1000, dtype=torch.bfloat16, device="cuda"), torch.zeros(4, dtype=torch.int32, device="cuda"), torch.zeros(4, device="cuda")
    buf[:, :999] = x.cuda()
    L.lora_sample(buf, 1000, 4, 999, None, None, None, None, None, tokens, logprobs)
    assert tokens.tolist() == [500] * 4
    for got, a in zip(logprobs.tolist(), (16.0, 20.0, 28.0, 40.0)):
        want = -math.log1p(998 * math.exp(-a))
        # the sum is rounded to fp32 (2^-24), ldexp and the signs are exact, log1p is off by at most 2 ulp (2^-22).  The weights
        # exp(-a) 2^62 are integers, each off by less than 1: at 28 of 3188704 (2^-21), at 40 of 19.6 (1 / 19)
        assert abs(got - want) <= (2.0 ** -21 + (1 / 19 if a == 40.0 else 2.0 ** -20)) * abs(want)


def test_columns_behind_the_vocabulary_take_no_part():
    x = rows(4, 1000, 5)
    x[:, 700:] = 50.0
    for vocab in (1, 8, 699, 700):
        check(x, uniform=uniform(4), vocab=vocab)


def test_no_rows():
    L.lora_sample(torch.zeros(8, dtype=torch.bfloat16, device="cuda"), 8, 0, 8, None, None, None, None, None, None, None)


def test_captured_and_replayed_on_another_stream():
    x = rows(7, 3001, 6)
    buf = torch.zeros(7, 3008, dtype=torch.bfloat16, device="cuda")
    u = torch.zeros(7, device="cuda")
    tokens = torch.zeros(7, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        L.lora_sample(buf, 3008, 7, 3001, None, None, None, None, u, tokens, None)
    for seed in (1, 2):
        x = rows(7, 3001, seed)
        buf[:, :3001] = x.cuda()
        u.copy_(torch.tensor(uniform(7, seed)))
        graph.replay()
        torch.cuda.synchronize()
        want = [reference_row(x[t].double().numpy(), 1.0, 0, 1.0, 0.0, float(u[t]))[0] for t in range(7)]
        assert tokens.tolist() == want
