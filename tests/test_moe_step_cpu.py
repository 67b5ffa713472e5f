"""What the calls around a layer of experts refuse: on the host, before anything is launched."""
import ctypes

import pytest

from heterogeneous_adapters_lora_gb300 import lora as L

AT = 1 << 20  # an aligned address that nothing reads


@pytest.fixture(scope="module", autouse=True)
def lib():
    import os
    if not os.path.exists(L.LIB_PATH):
        from heterogeneous_adapters_lora_gb300 import build
        build.build()
    return L.lib()


def refused(code, call, *args):
    with pytest.raises(L.LoraError) as e:
        call(*args, stream=0)
    assert e.value.name == code


def route_args(**change):
    d = dict(n_experts=8, top_k=2, scoring=0, renormalize=0, logits_f32=1, scale=1.0)
    a = dict(logits=AT, ld=8, T=3, bias=AT, ids=AT, w=AT)
    for k, v in change.items():
        (d if k in d else a)[k] = v
    return [L.RouteDesc(**d), a["logits"], a["ld"], a["T"], a["bias"], a["ids"], a["w"]]


@pytest.mark.parametrize("change", [
    dict(n_experts=0), dict(n_experts=1025), dict(top_k=0), dict(top_k=9), dict(n_experts=64, ld=64, top_k=33), dict(scoring=2),
    dict(renormalize=-1), dict(logits_f32=2), dict(scale=float("nan")), dict(scale=float("inf")), dict(ld=7), dict(T=-1),
    dict(logits=None), dict(logits=AT + 2), dict(logits=AT + 1, logits_f32=0), dict(bias=AT + 2), dict(ids=None), dict(ids=AT + 1),
    dict(w=None), dict(w=AT + 2)])
def test_route(change):
    refused("LORA_ERR_INVALID_ARG", L.lora_moe_route, *route_args(**change))


def test_no_tokens_need_no_buffers():
    L.lora_moe_route(*route_args(T=0, logits=None, bias=None, ids=None, w=None), stream=0)
    L.lora_sample(None, 8, 0, 8, None, None, None, None, None, None, None, stream=0)
    L.lora_moe_layer(*layer_args(T=0, x=None, ids=None, w=None, w13=None, w2=None, out=None, ws=None, ws_bytes=0), stream=0)


def sample_args(**change):
    a = dict(logits=AT, ld=64, T=3, vocab=60, temperature=AT, top_k=AT, top_p=AT, min_p=AT, uniform=AT, tokens=AT, logprobs=AT)
    a.update(change)
    return list(a.values())


@pytest.mark.parametrize("code,change", [
    ("LORA_ERR_SHAPE", dict(vocab=0)), ("LORA_ERR_SHAPE", dict(vocab=257025, ld=257032)), ("LORA_ERR_INVALID_ARG", dict(ld=56)),
    ("LORA_ERR_INVALID_ARG", dict(ld=65)), ("LORA_ERR_INVALID_ARG", dict(T=-1)), ("LORA_ERR_INVALID_ARG", dict(logits=None)),
    ("LORA_ERR_INVALID_ARG", dict(logits=AT + 8)), ("LORA_ERR_INVALID_ARG", dict(tokens=None)),
    *[("LORA_ERR_INVALID_ARG", {k: AT + 2}) for k in ("temperature", "top_k", "top_p", "min_p", "uniform", "tokens", "logprobs")]])
def test_sample(code, change):
    refused(code, L.lora_sample, *sample_args(**change))


def layer_args(**change):
    d = dict(n_experts=8, top_k=2, d_model=64, d_mlp=32, activation=0)
    a = dict(pool=None, idx=None, x=AT, ldx=64, T=3, ids=AT, w=AT, w13=AT, ld13=64, w2=AT, ld2=32, out=AT, ldo=64, status=AT, ws=AT,
             ws_bytes=1 << 40)
    for k, v in change.items():
        (d if k in d else a)[k] = v
    return [L.MoELayerDesc(**d), *a.values()]


@pytest.mark.parametrize("code,change", [
    *[("LORA_ERR_INVALID_ARG", c) for c in (
        dict(n_experts=0), dict(n_experts=1025), dict(top_k=0), dict(top_k=33), dict(d_model=0), dict(d_model=60), dict(d_mlp=0),
        dict(d_mlp=20), dict(d_model=65544, ldx=65544, ld13=65544, ldo=65544), dict(activation=2), dict(activation=-1), dict(T=-1),
        dict(ldx=56), dict(ldx=68), dict(ld13=56), dict(ld13=65), dict(ld2=24), dict(ld2=36), dict(ldo=56), dict(ldo=66),
        dict(x=None), dict(x=AT + 8), dict(ids=None), dict(ids=AT + 2), dict(w=AT + 1), dict(w13=None), dict(w13=AT + 4),
        dict(w2=None), dict(w2=AT + 2), dict(out=None), dict(out=AT + 8), dict(status=AT + 2), dict(idx=AT), dict(ws=None),
        dict(ws=AT + 8))],
    ("LORA_ERR_CAPACITY", dict(ws_bytes=0)), ("LORA_ERR_CAPACITY", dict(T=2049)), ("LORA_ERR_CAPACITY", dict(T=2 ** 31 - 1, top_k=32))])
def test_layer(code, change):
    refused(code, L.lora_moe_layer, *layer_args(**change))


def test_layer_workspace():
    d = L.MoELayerDesc(n_experts=8, top_k=2, d_model=64, d_mlp=32)
    sizes = [L.lora_moe_layer_workspace_bytes(d, None, t) for t in (0, 1, 100, 2048)]
    assert 0 < sizes[0] <= sizes[1] <= sizes[2] <= sizes[3]
    assert L.lora_moe_layer_workspace_bytes(d, None, 2049) == 0
    assert L.lora_moe_layer_workspace_bytes(d, None, -1) == 0
    assert L.lora_moe_layer_workspace_bytes(L.MoELayerDesc(n_experts=8, top_k=2, d_model=60, d_mlp=32), None, 1) == 0
    assert L.lib().lora_moe_layer_workspace_bytes(ctypes.POINTER(L.MoELayerDesc)(), None, 1) == 0
    refused("LORA_ERR_CAPACITY", L.lora_moe_layer, *layer_args(ws_bytes=L.lora_moe_layer_workspace_bytes(d, None, 3) - 1))
