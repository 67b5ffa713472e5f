"""The rest of a decode step around the LoRA layers, as measured work.

Three operators, each over the range a serving program calls it with:

route   the router's choice: scores of the experts' logits, the k best of a token and their weights
        (``lora_moe_route``)
layer   a whole layer of experts for a few tokens: the products of the chosen experts' weights, the
        deltas of the tokens' adapters, the activation between them and the weighted sum
        (``lora_moe_layer``)
sample  the next tokens of a batch from its logits: temperature, top-k, top-p and min-p of each
        request, and a random number of each (``lora_sample``)

Activations, weights and logits of the vocabulary are bf16, logits of a router fp32 or bf16, weights
of chosen experts, random numbers and log probabilities fp32.
"""
import math

import torch

own = False

GELU_IN, GELU_CUBE = 0.7978845608028654, 0.044715  # tanh form: sqrt(2 / pi) and the cube's factor


# ------------------------------------------------------------------ cases

def _named(name, c):
    return {"name": name, **c} if name else c


def _route(name, tokens, experts, top_k, sigmoid, bias, renormalize, wide):
    return _named(name, {"op": "route", "tokens": tokens, "experts": experts, "top_k": top_k, "sigmoid": sigmoid, "bias": bias,
                         "renormalize": renormalize, "wide": wide})


def _layer(name, tokens, experts, top_k, d_model, d_mlp, adapters=0, rank=0, shared=False, ranks="one", gelu=False, dropped=0.0, hot=0.0):
    return _named(name, {"op": "layer", "tokens": tokens, "experts": experts, "top_k": top_k, "d_model": d_model, "d_mlp": d_mlp,
                         "adapters": adapters, "rank": rank, "shared": shared, "ranks": ranks, "gelu": gelu, "dropped": dropped, "hot": hot})


def _sample(name, rows, vocab, filters, masked=0.0, spread=2.5):
    return _named(name, {"op": "sample", "rows": rows, "vocab": vocab, "filters": filters, "masked": masked, "spread": spread})


def listed():
    return [
        # one request generating: the smallest call
        _route("route_token", 1, 64, 8, False, False, False, True),
        # the prefill batch of 7995 tokens, scores with a bias that balances the experts
        _route("route_prefill", 7995, 256, 8, True, True, True, False),
        # a small layer without adapters: latency counts
        _layer("layer_small", 3, 8, 2, 512, 256),
        # one request generating, 64 experts with adapters of rank 16
        _layer("layer_token", 1, 64, 8, 2048, 1408, 8, 16),
        # a small decode batch
        _layer("layer_decode", 16, 64, 8, 2048, 1408, 8, 16),
        # odd sizes, ranks of different lengths, pairs that were dropped, an expert that most tokens choose
        _layer("layer_ragged", 37, 6, 3, 1040, 272, 4, 24, False, "mixed", True, 0.05, 3.0),
        # the layout whose outer adapter tensors are shared by the experts
        _layer("layer_shared", 64, 64, 8, 2048, 1408, 8, 16, True),
        # the decode batch of 256 tokens
        _layer("layer_batch", 256, 64, 8, 2048, 1408, 8, 16),
        # one request with a small vocabulary
        _sample("sample_row", 1, 32007, "mixed"),
        # the decode batch of 256 requests, filters of each its own, a grammar's mask on some
        _sample("sample_batch", 256, 128256, "mixed", 0.1),
        # temperature alone: the whole vocabulary takes part
        _sample("sample_free", 64, 128256, "none", 0.0, 1.5),
        # the largest vocabulary, the shortest prefix that holds a share of the mass
        _sample("sample_wide", 17, 257024, "top_p"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "layer", "layer", "sample", "sample"])
    if op == "route":
        experts = _log_int(rng, 2, 256)
        sigmoid = rng.random() < 0.5
        return _route(None, _log_int(rng, 1, 7900), experts, rng.randint(1, min(8, experts)), sigmoid, sigmoid and rng.random() < 0.7,
                      rng.random() < 0.6, rng.random() < 0.5)
    if op == "layer":
        experts = _log_int(rng, 2, 64)
        adapters = rng.choice([0, rng.randint(1, 8), rng.randint(1, 8)])
        rank = rng.choice([8, 16, 16, 24, 32]) if adapters else 0
        return _layer(None, _log_int(rng, 1, 120 if rank > 16 else 250), experts, rng.randint(1, min(8, experts)), 8 * _log_int(rng, 16, 256),
                      8 * _log_int(rng, 8, 176), adapters, rank, adapters > 0 and rng.random() < 0.4, rng.choice(["one", "mixed"]),
                      rng.random() < 0.3, rng.choice([0.0, 0.05]), rng.choice([0.0, 0.0, 3.0]))
    rows = _log_int(rng, 1, 256)
    vocab = _log_int(rng, 500, min(257024, 256 * 128256 // rows))
    return _sample(None, rows, vocab, rng.choice(["none", "top_k", "top_p", "min_p", "mixed"]), rng.choice([0.0, 0.1]), rng.uniform(1.0, 4.0))


def work(case):
    c = case
    if c["op"] == "route":
        n = c["tokens"] * c["experts"]
        return {"bytes": n * (4 if c["wide"] else 2) + (4 * c["experts"] if c["bias"] else 0) + 8 * c["tokens"] * c["top_k"], "flops": 8 * n}
    if c["op"] == "sample":
        n = c["rows"] * c["vocab"]
        return {"bytes": 2 * n + 28 * c["rows"], "flops": 8 * n}
    t, k, e, d, f = c["tokens"], c["top_k"], c["experts"], c["d_model"], c["d_mlp"]
    # the experts, and the (adapter, expert) pairs, that a batch of that many tokens is expected to meet
    experts = e * (1 - (1 - k / e) ** t)
    bytes_ = experts * 3 * f * d * 2 + 2 * t * d * 2 + 8 * t * k
    flops = 6 * t * k * f * d
    if c["adapters"]:
        keys = c["adapters"] * e * (1 - (1 - 0.9 * k / (e * c["adapters"])) ** t)
        outer = c["adapters"] * (1 - (1 - 0.9 / c["adapters"]) ** t) if c["shared"] else keys
        mean = c["rank"] * (0.6 if c["ranks"] == "mixed" else 1.0)
        bytes_ += mean * 2 * (outer * 3 * d + keys * 3 * f)
        flops += 0.9 * t * k * mean * 6 * (f + d)
    return {"bytes": int(bytes_), "flops": int(flops)}


# ------------------------------------------------------------------ inputs

def _rand(gen, std, *shape):
    return (std * torch.randn(*shape, generator=gen, device="cuda")).to(torch.bfloat16)


def _pick(gen, rows, choices, dtype):
    at = torch.randint(0, len(choices), (rows,), generator=gen, device="cuda")
    return torch.tensor(choices, dtype=dtype, device="cuda")[at]


class _Pool:
    """An adapter pool that goes with the state that holds it."""

    def __init__(self, s):
        from heterogeneous_adapters_lora_gb300 import lora
        c = s["case"]
        self.lora = lora
        self.handle = lora.lora_pool_create(lora.PoolDesc(
            max_loras=c["adapters"], max_rank=c["rank"], num_experts=c["experts"], d_model=c["d_model"], d_mlp=c["d_mlp"], n_w13_slices=2,
            w13_slice_width=c["d_mlp"], shared_outer=int(c["shared"])))
        e, f = c["experts"], c["d_mlp"]
        outer = 1 if c["shared"] else e
        for a, (r, scale) in enumerate(zip(s["ranks"], s["scales"])):
            if r == 0:
                continue
            gate, up = (s["a13"][a, :, j, :r].contiguous() for j in (0, 1))
            gate_b, up_b = (s["b13"][a, :, j * f:(j + 1) * f, :r].contiguous() for j in (0, 1))
            lora.lora_set_moe(self.handle, a, r, scale, [gate, up, s["a2"][a, :, :r].contiguous()], [outer, outer, e],
                              [gate_b, up_b, s["b2"][a, :, :, :r].contiguous()], [e, e, outer])

    def __del__(self):
        self.lora.lora_pool_destroy(self.handle)


def _prepare_layer(s, gen):
    c = s["case"]
    t, e, k, d, f = c["tokens"], c["experts"], c["top_k"], c["d_model"], c["d_mlp"]
    s["x"] = _rand(gen, 1.0, t, d)
    s["w13"] = _rand(gen, d ** -0.5, e, 2 * f, d)
    s["w2"] = _rand(gen, f ** -0.5, e, d, f)
    logits = torch.randn(t, e, generator=gen, device="cuda")
    logits[:, 0] += c["hot"]
    weight, ids = torch.topk(torch.softmax(logits, 1), k, dim=1)
    gone = torch.rand(t, k, generator=gen, device="cuda") < c["dropped"]
    s["ids"] = torch.where(gone, -1, ids).to(torch.int32)
    s["weights"] = (weight / weight.sum(1, keepdim=True)).contiguous()
    s["out"] = torch.zeros(t, d, dtype=torch.bfloat16, device="cuda")
    n, r = c["adapters"], c["rank"]
    s["idx"] = None
    if n:
        outer = 1 if c["shared"] else e
        s["ranks"] = [r if c["ranks"] == "one" else (r, r * 3 // 8, r * 2 // 3, r // 3)[a % 4] for a in range(n)]
        s["scales"] = [(2.0, 1.0, 0.5)[a % 3] for a in range(n)]
        s["scale"] = torch.tensor(s["scales"], device="cuda")
        live = torch.arange(r, device="cuda")[None, :] < torch.tensor(s["ranks"], device="cuda")[:, None]
        s["a13"] = _rand(gen, d ** -0.5, n, outer, 2, r, d) * live[:, None, None, :, None]
        s["b13"] = _rand(gen, 0.5 * r ** -0.5, n, e, 2 * f, r) * live[:, None, None, :]
        s["a2"] = _rand(gen, f ** -0.5, n, e, r, f) * live[:, None, :, None]
        s["b2"] = _rand(gen, 0.5 * r ** -0.5, n, outer, d, r) * live[:, None, None, :]
        idx = torch.randint(0, n, (t,), generator=gen, device="cuda")
        s["idx"] = torch.where(torch.rand(t, generator=gen, device="cuda") < 0.1, -1, idx).to(torch.int32)
    if own:  # the pool that holds the adapters, and the workspace a program keeps
        from heterogeneous_adapters_lora_gb300 import lora
        s["pool"] = _Pool(s) if n else None
        s["handle"] = s["pool"].handle if n else None
        s["desc"] = lora.MoELayerDesc(n_experts=e, top_k=k, d_model=d, d_mlp=f, activation=int(c["gelu"]))
        s["ws_bytes"] = lora.lora_moe_layer_workspace_bytes(s["desc"], s["handle"], t)
        s["ws"] = torch.empty(s["ws_bytes"], dtype=torch.uint8, device="cuda")
        lora.lora_workspace_init(s["ws"], s["ws_bytes"])


def _prepare_sample(s, gen):
    c = s["case"]
    n, v = c["rows"], c["vocab"]
    x = c["spread"] * torch.randn(n, (v + 7) // 8 * 8, generator=gen, device="cuda")
    # a few candidates stand out, as they do behind a prompt
    some = torch.randint(0, v, (n, 40), generator=gen, device="cuda")
    x.scatter_add_(1, some, 4 * torch.rand(n, 40, generator=gen, device="cuda") * c["spread"])
    if c["masked"]:
        rows = torch.rand(n, 1, generator=gen, device="cuda") < c["masked"]
        x.masked_fill_(rows & (torch.rand(x.shape, generator=gen, device="cuda") < 0.9), -math.inf)
        x[:, :2] = 0.0
    s["logits"] = x.to(torch.bfloat16)
    mixed = c["filters"] == "mixed"
    f32, i32 = torch.float32, torch.int32
    s["temperature"] = _pick(gen, n, [0.0, 0.6, 0.8, 1.0, 1.3] if mixed else [0.7, 1.0, 1.2], f32)
    s["top_k"] = _pick(gen, n, [0, 1, 20, 50, 1000] if mixed else [40, 100], i32) if mixed or c["filters"] == "top_k" else None
    s["top_p"] = _pick(gen, n, [1.0, 0.95, 0.9, 0.5], f32) if mixed or c["filters"] == "top_p" else None
    s["min_p"] = _pick(gen, n, [0.0, 0.0, 0.02, 0.1] if mixed else [0.05, 0.1], f32) if mixed or c["filters"] == "min_p" else None
    s["uniform"] = torch.rand(n, generator=gen, device="cuda")
    s["tokens"] = torch.zeros(n, dtype=i32, device="cuda")
    s["logprobs"] = torch.zeros(n, dtype=f32, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = {"case": case}
    if case["op"] == "layer":
        _prepare_layer(s, gen)
    elif case["op"] == "sample":
        _prepare_sample(s, gen)
    else:
        t, e, k = case["tokens"], case["experts"], case["top_k"]
        s["logits"] = torch.randn(t, e, generator=gen, device="cuda").to(torch.float32 if case["wide"] else torch.bfloat16)
        s["bias"] = 0.1 * torch.randn(e, generator=gen, device="cuda") if case["bias"] else None
        s["ids"] = torch.zeros(t, k, dtype=torch.int32, device="cuda")
        s["weights"] = torch.zeros(t, k, dtype=torch.float32, device="cuda")
        if own:
            from heterogeneous_adapters_lora_gb300 import lora
            s["desc"] = lora.RouteDesc(n_experts=e, top_k=k, scoring=int(case["sigmoid"]), renormalize=int(case["renormalize"]),
                                       logits_f32=int(case["wide"]), scale=1.0)
    return s


# ------------------------------------------------------------------ plain forms

def _plain_route(s):
    c = s["case"]
    x = s["logits"].double()  # choices next to a border
    score = torch.sigmoid(x) if c["sigmoid"] else torch.softmax(x, 1)
    by = score + s["bias"].double() if c["bias"] else (score if c["sigmoid"] else x)
    ids = torch.sort(by, dim=1, descending=True, stable=True).indices[:, :c["top_k"]]
    w = score.gather(1, ids)
    if c["renormalize"]:
        w = w / w.sum(1, keepdim=True)
    return {"ids": ids.to(torch.int32), "weights": w.float()}


def _act(x, gelu):
    if gelu:
        return 0.5 * x * (1 + torch.tanh(GELU_IN * (x + GELU_CUBE * x * x * x)))
    return x / (1 + torch.exp(-x))


def _plain_layer(s):
    c = s["case"]
    t, e, k, f = c["tokens"], c["experts"], c["top_k"], c["d_mlp"]
    x = s["x"].float()
    there = s["ids"] >= 0
    ids = s["ids"].long().clamp(min=0)
    w = s["weights"] * there
    few = t * k <= e
    token = torch.arange(t, device=x.device)[:, None].expand(t, k)
    if few:  # the chosen experts' weights
        gu = torch.matmul(s["w13"][ids].float(), x[:, None, :, None])[..., 0]
    else:  # every expert for every token, then the chosen ones
        gu = torch.matmul(x, s["w13"].float().transpose(1, 2))[ids, token]
    if c["adapters"]:
        a = s["idx"].long()
        scale = torch.where(a >= 0, s["scale"][a.clamp(min=0)], 0.0)[:, None, None]
        slot = a.clamp(min=0)[:, None].expand(t, k)
        outer = torch.zeros_like(ids) if c["shared"] else ids
        v = torch.matmul(s["a13"][slot, outer].float(), x[:, None, None, :, None])[..., 0] * scale[..., None]
        b = s["b13"][slot, ids].float().view(t, k, 2, f, -1)
        gu = gu + torch.matmul(b, v[..., None])[..., 0].reshape(t, k, 2 * f)
    h = _act(gu[..., :f], c["gelu"]) * gu[..., f:]
    if few:
        out = (torch.matmul(s["w2"][ids].float(), h[..., None])[..., 0] * w[..., None]).sum(1)
    else:
        spread = torch.zeros(e, t, f, device=x.device)
        spread.index_put_((ids, token), h * w[..., None], accumulate=True)
        out = torch.matmul(spread, s["w2"].float().transpose(1, 2)).sum(0)
    if c["adapters"]:
        v = torch.matmul(s["a2"][slot, ids].float(), h[..., None])[..., 0] * scale * w[..., None]
        out = out + torch.matmul(s["b2"][slot, outer].float(), v[..., None])[..., 0].sum(1)
    return out.to(torch.bfloat16)


def _plain_sample(s):
    c = s["case"]
    v = c["vocab"]
    x = s["logits"][:, :v].double() + 0.0  # in 64 bits: long sums, and numbers next to a border of theirs
    greedy = s["temperature"] <= 0
    top = x.amax(1, keepdim=True)
    none = top == -math.inf
    z = (x - torch.where(none, 0.0, top)) / torch.where(greedy, 1.0, s["temperature"]).double()[:, None]
    log_total = torch.where(none, 1.0, z.exp().sum(1, keepdim=True)).log()
    order = torch.sort(x, dim=1, descending=True, stable=True).indices
    w = z.gather(1, order).exp()
    mass = w.cumsum(1)
    keep = torch.full_like(order[:, :1], v)
    if s["top_k"] is not None:
        keep = torch.where(s["top_k"] > 0, s["top_k"].clamp(max=v), v).long()[:, None]
    if s["top_p"] is not None:
        share = s["top_p"].double()[:, None]
        short = (mass < share * mass.gather(1, keep - 1)).sum(1, keepdim=True) + 1
        keep = torch.where(share >= 1, keep, torch.minimum(keep, short))
    if s["min_p"] is not None:
        keep = torch.minimum(keep, (w >= s["min_p"].double()[:, None]).sum(1, keepdim=True))
    keep = torch.where(greedy[:, None], 1, keep.clamp(min=1))
    target = s["uniform"].double()[:, None] * mass.gather(1, keep - 1)
    at = torch.minimum((mass <= target).sum(1, keepdim=True), keep - 1)
    token = order.gather(1, at)
    logprob = z.gather(1, token) - log_total
    return {"tokens": torch.where(none, -1, token)[:, 0].to(torch.int32), "logprobs": logprob[:, 0].float()}


def run(state):
    s = state
    c = s["case"]
    if not own:
        return {"route": _plain_route, "layer": _plain_layer, "sample": _plain_sample}[c["op"]](s)
    from heterogeneous_adapters_lora_gb300 import lora
    if c["op"] == "route":
        lora.lora_moe_route(s["desc"], s["logits"], s["logits"].stride(0), c["tokens"], s["bias"], s["ids"], s["weights"])
        return {"ids": s["ids"], "weights": s["weights"]}
    if c["op"] == "sample":
        lora.lora_sample(s["logits"], s["logits"].stride(0), c["rows"], c["vocab"], s["temperature"], s["top_k"], s["top_p"], s["min_p"],
                         s["uniform"], s["tokens"], s["logprobs"])
        return {"tokens": s["tokens"], "logprobs": s["logprobs"]}
    lora.lora_moe_layer(s["desc"], s["handle"], s["idx"], s["x"], s["x"].stride(0), c["tokens"], s["ids"], s["weights"], s["w13"],
                        s["w13"].stride(1), s["w2"], s["w2"].stride(1), s["out"], s["out"].stride(0), None, s["ws"], s["ws_bytes"])
    return s["out"]


# ------------------------------------------------------------------ in 64 bits

def _exact_route(s):
    c = s["case"]
    x = s["logits"].cpu().numpy().astype("float64") if c["wide"] else s["logits"].float().cpu().numpy().astype("float64")
    import numpy as np
    score = 1 / (1 + np.exp(-x)) if c["sigmoid"] else np.exp(x - x.max(1, keepdims=True))
    if not c["sigmoid"]:
        score /= score.sum(1, keepdims=True)
    by = score + s["bias"].cpu().numpy().astype("float64") if c["bias"] else score.copy()
    rows = np.arange(len(x))
    ids = np.zeros((len(x), c["top_k"]), np.int32)
    for j in range(c["top_k"]):
        ids[:, j] = by.argmax(1)
        by[rows, ids[:, j]] = -np.inf
    w = score[rows[:, None], ids]
    return {"ids": ids, "weights": w / w.sum(1, keepdims=True) if c["renormalize"] else w}


def _exact_layer(s):
    c = s["case"]
    t, d, f = c["tokens"], c["d_model"], c["d_mlp"]
    out = torch.zeros(t, d, dtype=torch.float64, device="cuda")
    x = s["x"].double()
    for e in range(c["experts"]):
        rows, place = torch.nonzero(s["ids"] == e, as_tuple=True)
        if not len(rows):
            continue
        gu = x[rows] @ s["w13"][e].double().T
        near = 0 if c["shared"] else e
        slots = s["idx"][rows].tolist() if c["adapters"] else []
        for i, a in enumerate(slots):
            if a >= 0:
                for j in (0, 1):
                    v = s["a13"][a, near, j].double() @ x[rows[i]] * s["scales"][a]
                    gu[i, j * f:(j + 1) * f] += s["b13"][a, e, j * f:(j + 1) * f].double() @ v
        g, u = gu[:, :f], gu[:, f:]
        if c["gelu"]:
            h = g * 0.5 * (1 + torch.tanh(math.sqrt(2 / math.pi) * (g + GELU_CUBE * g.pow(3)))) * u
        else:
            h = g * torch.sigmoid(g) * u
        y = h @ s["w2"][e].double().T
        for i, a in enumerate(slots):
            if a >= 0:
                y[i] += s["b2"][a, near].double() @ (s["a2"][a, e].double() @ h[i]) * s["scales"][a]
        out.index_add_(0, rows, y * s["weights"][rows, place].double()[:, None])
    return out


def _exact_sample(s):
    import numpy as np
    c = s["case"]
    x = s["logits"][:, :c["vocab"]].float().cpu().numpy().astype("float64")
    given = {k: None if s[k] is None else s[k].cpu().numpy() for k in ("temperature", "top_k", "top_p", "min_p", "uniform")}
    tokens, logprobs = [], []
    for i, row in enumerate(x):
        order = np.argsort(-row, kind="stable")
        temperature = float(given["temperature"][i])
        p = np.exp((row[order] - row[order[0]]) / (temperature if temperature > 0 else 1.0))
        total = math.fsum(p)
        left = len(p)
        if given["top_k"] is not None and given["top_k"][i] > 0:
            left = min(left, int(given["top_k"][i]))
        mass = np.cumsum(p[:left])
        if given["top_p"] is not None and given["top_p"][i] < 1:
            left = min(left, int(np.searchsorted(mass, float(given["top_p"][i]) * mass[-1], side="left")) + 1)
        if given["min_p"] is not None:
            left = max(1, min(left, int(np.count_nonzero(p >= float(given["min_p"][i])))))
        if temperature <= 0:
            left = 1
        at = min(left - 1, int(np.searchsorted(mass[:left], float(given["uniform"][i]) * mass[left - 1], side="right")))
        tokens.append(int(order[at]))
        logprobs.append(math.log(p[at]) - math.log(total))
    return {"tokens": np.array(tokens, np.int32), "logprobs": np.array(logprobs)}


def exact(case, seed):
    s = prepare(case, seed)
    return {"route": _exact_route, "layer": _exact_layer, "sample": _exact_sample}[case["op"]](s)
