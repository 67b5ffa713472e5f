"""A layer of experts for a few tokens (lora_moe_layer) against the formula in 64 bits."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from heterogeneous_adapters_lora_gb300 import lora as L
from moe_layer_util import Layer

pytestmark = pytest.mark.gpu


def run(*args, **kw):
    layer = Layer(*args, **kw)
    layer.call()
    layer.check()
    assert int(layer.status) == 0
    return layer


@pytest.mark.parametrize("T,E,K,D,F", [(1, 1, 1, 8, 8), (1, 4, 2, 64, 64), (3, 8, 2, 512, 256), (2, 3, 1, 72, 136), (5, 6, 3, 1040, 272),
                                       (17, 8, 4, 128, 120), (33, 4, 2, 264, 1032), (1, 16, 8, 2048, 1408)])
@pytest.mark.parametrize("gelu", [False, True])
def test_without_adapters(T, E, K, D, F, gelu):
    run(T, E, K, D, F, gelu=gelu, seed=T + D)


@pytest.mark.parametrize("rank,ranks", [(1, None), (8, None), (16, None), (24, (24, 9, 16, 0)), (64, (64, 1, 33, 8)), (256, (256, 3, 100, 77))])
@pytest.mark.parametrize("shared", [False, True])
def test_adapters(rank, ranks, shared):
    run(13, 6, 3, 136, 208, adapters=4, rank=rank, ranks=ranks, shared=shared, seed=rank)


@pytest.mark.parametrize("n13", [1, 2])
def test_gate_and_up_in_one_slice_or_two(n13):
    run(9, 4, 2, 256, 128, adapters=3, rank=16, n13=n13, seed=n13)


@pytest.mark.parametrize("T", [1, 2, 7, 8, 9, 15, 16, 17, 63, 64, 65, 130])
def test_one_expert_takes_every_token(T):
    run(T, 1, 1, 128, 64, adapters=2, rank=8, seed=T)


@pytest.mark.parametrize("T,E,K", [(100, 2, 2), (40, 3, 3), (300, 5, 2), (128, 1, 32), (128, 40, 32), (600, 7, 2)])
def test_many_pairs_of_an_expert(T, E, K):
    run(T, E, K, 64, 72, adapters=3, rank=8, seed=T)


def test_one_rank_slice_of_every_size():
    for F in (8, 56, 64, 72, 120, 128, 136, 248, 256, 264):
        run(3, 2, 1, 80, F, adapters=2, rank=8, seed=F)
    for D in (8, 56, 64, 72, 120, 128, 136, 248, 256, 264, 520):
        run(3, 2, 1, D, 80, adapters=2, rank=8, seed=D)


@pytest.mark.parametrize("T,E,K,adapters", [(1, 1024, 32, 2), (9, 300, 4, 3), (130, 200, 1, 0)])
def test_many_experts(T, E, K, adapters):
    run(T, E, K, 64, 40, adapters=adapters, rank=8, seed=E)


def test_padded_rows():
    run(11, 4, 2, 200, 104, adapters=2, rank=16, pads=(8, 16, 24, 40), seed=3)


def test_no_routing_weights():
    run(6, 4, 2, 64, 64, adapters=2, rank=8, with_weights=False)


def test_the_same_expert_twice():
    layer = Layer(5, 4, 3, 96, 80, adapters=2, rank=8, seed=8)
    ids = layer.ids.clone()
    ids[:, 1] = ids[:, 0]
    ids[4] = 2
    layer.batch(ids=ids).call()
    layer.check()


def test_experts_and_slots_that_are_none():
    layer = Layer(12, 4, 3, 96, 80, adapters=2, rank=8, seed=9)
    ids, idx = layer.ids.clone(), layer.idx.clone()
    ids[0] = -1  # a token without experts
    ids[3, 1] = -1
    idx[:] = torch.tensor([0, 1] * 6)
    idx[5] = -1
    layer.batch(ids=ids, idx=idx).call()
    layer.check()
    assert torch.all(layer.out[0, :96] == 0)
    assert int(layer.status) == 0
    for bad in (4, 1000, -2, -2 ** 31):
        wrong = ids.clone()
        wrong[7, 2] = bad
        layer.status.zero_()
        layer.batch(ids=wrong).call()
        layer.check()
        assert int(layer.status) == L.CODE["LORA_ERR_DEVICE_INDEX"]
    for bad in (2, -2, 2 ** 31 - 1):
        wrong = idx.clone()
        wrong[6] = bad
        layer.status.zero_()
        layer.batch(ids=ids, idx=wrong).call()
        layer.check()
        assert int(layer.status) == L.CODE["LORA_ERR_DEVICE_INDEX"]
    nobody = torch.full_like(ids, -1)
    layer.batch(ids=nobody, idx=idx).call()
    layer.check()


def test_no_adapter_at_all():
    layer = Layer(7, 4, 2, 64, 64, adapters=2, rank=8, p_none=1.1)
    layer.call()
    layer.check()
    L.lora_reset(layer.pool, 0)
    layer.ranks[0] = 0
    layer.batch(idx=torch.tensor([0, 1, 0, 1, -1, 0, 1], dtype=torch.int32)).call()
    layer.check()


def test_no_tokens():
    layer = Layer(0, 4, 2, 64, 64)
    layer.call()
    layer.check()


def test_smaller_batches_in_one_workspace():
    big = Layer(40, 6, 2, 136, 72, adapters=3, rank=8, seed=1, max_tokens=64)
    small = Layer(3, 6, 2, 136, 72, adapters=3, rank=8, seed=2, max_tokens=64)
    small.ws = big.ws
    for layer in (big, small, big, small, small):
        layer.out.fill_(7.0)
        layer.call()
        layer.check()


def test_same_result_every_time():
    layer = Layer(50, 6, 3, 520, 264, adapters=3, rank=16, seed=4)
    first = layer.call().clone()
    for _ in range(5):
        assert torch.equal(layer.call(), first)


def test_not_a_number_stays_with_its_token():
    layer = Layer(9, 3, 2, 72, 64, adapters=2, rank=8, seed=6)
    x = layer.x.clone()
    x[4, 3] = float("nan")
    x[6, 0] = float("inf")
    clean = layer.call().clone()
    layer.batch(x=x).call()
    others = [t for t in range(9) if t not in (4, 6)]
    assert torch.equal(layer.out[others], clean[others])
    assert torch.all(torch.isnan(layer.out[4, :72]))
    assert not torch.any(torch.isfinite(layer.out[6, :72]))


@pytest.mark.parametrize("adapters", [0, 2])
def test_infinite_h_is_infinite_in_the_result(adapters):
    """act(g) u beyond fp32 for one token, weights above 0: infinity, as the formula in fp32 has it, not NaN."""
    layer = Layer(5, 2, 2, 72, 64, adapters=adapters, rank=8, seed=7)
    x, tiny = layer.x.clone(), 2.0 ** -20
    x[3] = 1e25
    values = dict(x=x, w13=layer.w13.abs() + tiny, w2=layer.w2.abs() + tiny)
    if adapters:
        values["idx"] = torch.tensor([0, 1, 0, -1, 1], dtype=torch.int32)
    layer.batch(**values).call()
    assert torch.all(layer.out[3, :72] == float("inf"))
    assert torch.all(torch.isfinite(layer.out[[0, 1, 2, 4], :72]))


def test_captured_with_another_workspace_and_replayed():
    layer = Layer(10, 4, 2, 128, 72, adapters=2, rank=8, seed=10)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        layer.call()
    for seed in (1, 2, 3):
        g = torch.Generator().manual_seed(seed)
        layer.batch(x=torch.randn(10, 128, generator=g).to(torch.bfloat16), ids=torch.randint(-1, 4, (10, 2), generator=g).to(torch.int32))
        layer.out.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        layer.check()


def test_two_graphs_and_eager_calls_share_a_workspace():
    """Replayed in turn on one stream, with an eager call of a third batch between them."""
    a, b, c = (Layer(T, 6, 2, 264, 136, adapters=2, rank=8, seed=30 + T, max_tokens=48) for T in (5, 48, 1))
    b.ws = c.ws = a.ws
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs = []
    for layer in (a, b):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=side):
            layer.call()
    for _ in range(3):
        for layer in (a, b, c):
            layer.out.fill_(7.0)
        graphs[1].replay()
        graphs[0].replay()
        c.call()
        graphs[1].replay()
        torch.cuda.synchronize()
        for layer in (a, b, c):
            layer.check()


def test_every_pair_for_one_expert_of_many():
    """All the pairs a call takes, for one of 200 experts, and shares of groups of every size."""
    layer = Layer(512, 200, 8, 72, 136, adapters=3, rank=8, seed=12)
    ids = torch.full_like(layer.ids, 137)
    layer.batch(ids=ids).call()
    layer.check()
    ids[:, 1:] = -1
    ids[::3, 1] = 5
    layer.batch(ids=ids).call()
    layer.check()


def test_two_layers_on_two_streams():
    layers = [Layer(20, 6, 2, 264, 136, adapters=2, rank=8, seed=20 + i) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in layers]
    torch.cuda.synchronize()
    for _ in range(5):
        for layer, s in zip(layers, streams):
            layer.call(s)
    torch.cuda.synchronize()
    for layer in layers:
        layer.check()


def test_large_layer_of_one_token_and_of_many():
    """The 64 experts of 2048 and 1408 with adapters of rank 16."""
    for T in (1, 4):
        run(T, 64, 8, 2048, 1408, adapters=8, rank=16, seed=T)
