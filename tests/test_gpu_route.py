"""The router's choice (lora_moe_route) against the formula in 64 bits."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from heterogeneous_adapters_lora_gb300 import lora as L

pytestmark = pytest.mark.gpu

F32_MAX = float(np.finfo(np.float32).max)


def reference(x, k, sigmoid, bias, renormalize, scale):
    """ids and weights of logits x [T][E] in 64 bits."""
    x = np.asarray(x, np.float64)
    live = x > -np.inf  # not NaN either
    x = np.where(live, np.minimum(x, F32_MAX), -np.inf)
    with np.errstate(over="ignore", invalid="ignore", divide="ignore"):
        if sigmoid:
            score = 1 / (1 + np.exp(-x))
        else:
            top = x.max(1, keepdims=True)
            score = np.exp(x - np.where(top > -np.inf, top, 0))
            score /= score.sum(1, keepdims=True)
        by = np.where(live, score + np.asarray(bias, np.float64) if bias is not None else x, -np.inf)
    by = np.where(np.isnan(by), -np.inf, by)
    order = np.argsort(-by, axis=1, kind="stable")[:, :k]
    rows = np.arange(len(x))[:, None]
    there = by[rows, order] > -np.inf
    ids = np.where(there, order, -1)
    w = np.where(there, score[rows, order], 0.0)
    if renormalize:
        total = w.sum(1, keepdims=True)
        w = np.where(total > 0, w / np.where(total > 0, total, 1), 0)
    return ids.astype(np.int32), w * scale


def route(x, k, sigmoid=False, bias=None, renormalize=False, scale=1.0, pad=0, stream=None):
    T, E = x.shape
    wide = x.dtype == torch.float32
    buf = torch.full((T, E + pad), 50.0, dtype=x.dtype, device="cuda")
    buf[:, :E] = x.cuda()
    d = L.RouteDesc(n_experts=E, top_k=k, scoring=int(sigmoid), renormalize=int(renormalize), logits_f32=int(wide), scale=scale)
    ids = torch.full((T, k), 77, dtype=torch.int32, device="cuda")
    w = torch.full((T, k), 77.0, device="cuda")
    L.lora_moe_route(d, buf, E + pad, T, None if bias is None else bias.cuda(), ids, w, stream)
    return ids.cpu().numpy(), w.cpu().numpy()


def check(x, k, sigmoid=False, bias=None, renormalize=False, scale=1.0, pad=0):
    ids, w = route(x, k, sigmoid, bias, renormalize, scale, pad)
    want, ww = reference(x.double().numpy(), k, sigmoid, None if bias is None else bias.numpy(), renormalize, scale)
    assert np.array_equal(ids, want)
    # a score is off by at most 1.1e-5 of itself (the rounding of a logit minus the largest, up to 104 of them, exp's 2 ulp,
    # and a sum of up to 1024 terms), its quotient by a sum of such twice that; scores below the
    # smallest normal number may vanish
    assert np.all(np.abs(w - ww) <= 2.2e-5 * np.abs(ww) + 1.2e-38 * abs(scale))


def logits(T, E, seed, dtype=torch.float32, spread=1.0):
    return (spread * torch.randn(T, E, generator=torch.Generator().manual_seed(seed))).to(dtype)


@pytest.mark.parametrize("E,k", [(1, 1), (2, 2), (31, 3), (32, 32), (33, 1), (64, 8), (65, 8), (256, 8), (257, 9), (1024, 32)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("sigmoid", [False, True])
def test_sizes(E, k, dtype, sigmoid):
    x = logits(37, E, E + k, dtype)
    bias = 0.1 * torch.randn(E, generator=torch.Generator().manual_seed(5))
    for b in (None, bias):
        check(x, k, sigmoid, b, renormalize=E % 2 == 0, scale=2.5 if E % 3 == 0 else 1.0, pad=E % 5)


@pytest.mark.parametrize("T", [0, 1, 3, 4, 5, 1001])
def test_tokens(T):
    check(logits(T, 48, T), 6, renormalize=True)


def test_equal_logits_go_to_the_lower_id():
    x = torch.zeros(3, 70)
    x[1, 40:] = 1.0
    x[2, ::2] = -0.0
    for bias in (None, torch.zeros(70)):
        check(x, 8, bias=bias)
        check(x, 8, True, bias)


def test_masked_experts_leave_places_empty():
    x = logits(6, 40, 3)
    x[0, 3:] = -np.inf          # three are left for five places
    x[1, :] = -np.inf           # none
    x[2, 5] = np.nan
    x[3, 7] = np.inf
    x[4, ::2] = torch.finfo(torch.float32).min
    x[5, :] = np.nan
    bias = torch.zeros(40)
    bias[1] = -np.inf           # nor are those chosen whose bias masks them
    bias[2] = np.nan
    for b in (None, bias):
        for sigmoid in (False, True):
            for renormalize in (False, True):
                check(x, 5, sigmoid, b, renormalize)


def test_biased_scores_closer_than_fp32_tells():
    """Neighbours that differ by 1e-9 of a score: the order is that of the exact sums."""
    g = torch.Generator().manual_seed(2)
    x = torch.randn(200, 64, generator=g)
    x[:, 32:] = x[:, :32] + 1e-7 * torch.randn(200, 32, generator=g)
    for sigmoid in (False, True):
        check(x, 8, sigmoid, torch.zeros(64))
    base = torch.randn(64, generator=g)  # biases that cancel the scores up to their own rounding
    score = torch.sigmoid(base.double())
    check(base[None].repeat(3, 1), 8, True, (0.5 - score).float())
    check(base[None].repeat(3, 1), 8, False, (0.5 - torch.softmax(base.double(), 0)).float())


def test_far_logits():
    x = logits(50, 64, 9, spread=300.0)
    check(x, 8)
    check(x, 8, False, 0.01 * torch.randn(64, generator=torch.Generator().manual_seed(1)))
    check(x, 8, True, None, True)


def test_captured_and_replayed_on_another_stream():
    x = logits(9, 64, 4).cuda()
    d = L.RouteDesc(n_experts=64, top_k=8, scale=1.0, logits_f32=1)
    ids, w = torch.zeros(9, 8, dtype=torch.int32, device="cuda"), torch.zeros(9, 8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            L.lora_moe_route(d, x, 64, 9, None, ids, w)
    for seed in (5, 6):
        x.copy_(logits(9, 64, seed))
        graph.replay()
        torch.cuda.synchronize()
        assert np.array_equal(ids.cpu().numpy(), reference(x.cpu().numpy(), 8, False, None, False, 1.0)[0])


@pytest.mark.parametrize("E,k", [(200, 8), (254, 32), (1000, 32), (256, 12)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T", [40, 2500])
def test_favourites_of_one_lane_and_equals_everywhere(T, E, k, dtype):
    """More candidates than lanes, all of them in one or two lanes, and borders that fall between equals."""
    x = logits(T, E, E, dtype, spread=0.1)
    x[:8, 40:48] += 5.0                # neighbours, in one lane
    x[8:16, E - 12:] += 5.0
    x[16:24] = (x[16:24] * 20).round() / 2   # many equals
    x[24] = 1.0
    x[25, ::2] = -np.inf
    x[26, 3:] = -np.inf
    x[27] = -1e30
    x[T - 28:] = x[:28].clone()
    bias = 0.1 * torch.randn(E, generator=torch.Generator().manual_seed(6))
    big = bias.clone()
    big[::3] = -1e9
    big[5] = 3e38
    endless = bias.clone()
    endless[7] = endless[9] = np.inf
    for sigmoid in (False, True):
        for b in (None, bias, torch.zeros(E), big, endless):
            check(x, k, sigmoid, b, renormalize=True)
