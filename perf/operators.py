"""The attention block between a LoRA QKV layer and a LoRA output layer, as measured work.

Three operators of that block, each over the range a serving program calls it with:

rope    norms of queries and keys per head with the position rotation in the same pass, read from
        the packed QKV output; keys and values go to their rows of the cache
        (``lora_qk_norm_rope``)
prompt  causal attention over packed sequences of different lengths with grouped heads: whole
        prompts, chunks of prompts behind cached keys, and single tokens (``lora_prompt_attention``)
prefix  attention for a batch whose requests share long prefixes (a tenant's common instructions),
        each prefix's part computed once for all its requests (``lora_prefix_attention``)

All tensors are bf16; weights of the norms are bf16, the table of cosines and sines is fp32.
A plan of an attention batch depends on the lengths alone and is built once for all the layers of a
step, so it is part of the state, as the workspace is.
"""
import math
import random

import torch

own = False

EPS = 1e-6
MAX_POS = 16384

# (query heads, key/value heads, head size)
HEADS = [(32, 8, 128), (32, 8, 128), (16, 16, 64), (28, 4, 128), (40, 8, 128), (8, 1, 64), (24, 8, 96)]


# ------------------------------------------------------------------ cases

def _heads(hq, hkv, d):
    return {"heads": hq, "kv_heads": hkv, "head_dim": d}


def _rope(name, tokens, heads, rot, interleaved, cache):
    c = {"op": "rope", "tokens": tokens, **_heads(*heads), "rot_dim": rot, "interleaved": interleaved, "cache": cache}
    return {"name": name, **c} if name else c


def _prompt(name, seqs, q, past, heads, page, lens):
    c = {"op": "prompt", "seqs": seqs, "q_lo": q[0], "q_hi": q[1], "past_lo": past[0], "past_hi": past[1],
         **_heads(*heads), "page": page, "lens": lens}
    return {"name": name, **c} if name else c


def _prefix(name, seqs, groups, prefix, mine, heads, page, lens):
    c = {"op": "prefix", "seqs": seqs, "groups": groups, "prefix_lo": prefix[0], "prefix_hi": prefix[1],
         "own_lo": mine[0], "own_hi": mine[1], **_heads(*heads), "page": page, "lens": lens}
    return {"name": name, **c} if name else c


def listed():
    h = (32, 8, 128)  # the QKV layer of 4096 inputs and outputs of 4096, 1024 and 1024
    return [
        # one request generating: the smallest call of a layer
        _rope("rope_token", 1, h, 128, False, True),
        # the decode batch of 256 tokens, keys and values into a paged cache
        _rope("rope_decode", 256, h, 128, False, True),
        # a prefill batch of 7995 tokens, results beside the input
        _rope("rope_prefill", 7995, h, 128, False, False),
        # smaller heads with half of each rotated, pairs side by side
        _rope("rope_partial", 2049, (16, 16, 64), 32, True, True),
        # a few short prompts: latency counts
        _prompt("prompt_short", 8, (5, 64), (0, 0), h, 0, 1),
        # the prefill batch of requests of mixed lengths, packed
        _prompt("prompt_mixed", 12, (33, 2048), (0, 0), h, 0, 2),
        # one long prompt
        _prompt("prompt_long", 1, (7995, 7995), (0, 0), h, 0, 3),
        # chunks of prompts behind keys already in a paged cache
        _prompt("prompt_chunks", 6, (100, 512), (300, 7000), (28, 4, 128), 16, 4),
        # a decode step: single tokens over histories of different lengths
        _prompt("prompt_tokens", 64, (1, 1), (20, 4000), h, 16, 5),
        # a handful of requests behind one common instruction
        _prefix("prefix_few", 4, 1, (1000, 1000), (1, 40), h, 16, 6),
        # the decode batch of 256, all behind one long prefix
        _prefix("prefix_batch", 256, 1, (8190, 8190), (1, 500), h, 16, 7),
        # the decode batch over 32 adapters, each with a prefix of its own
        _prefix("prefix_tenants", 256, 32, (100, 2000), (1, 800), h, 32, 8),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "prompt", "prefix"])
    heads = rng.choice(HEADS)
    lens = rng.randrange(1 << 20)
    if op == "rope":
        rot = rng.choice([heads[2], heads[2] // 2])
        return _rope(None, _log_int(rng, 1, 7900), heads, rot, rng.random() < 0.3, rng.random() < 0.6)
    page = rng.choice([16, 32, 64])
    if op == "prefix":
        seqs = _log_int(rng, 2, 250)
        groups = 1 if rng.random() < 0.5 else _log_int(rng, 1, seqs)
        longest = _log_int(rng, 64, 8000 if groups == 1 else 2000)
        return _prefix(None, seqs, groups, (max(1, longest // 8), longest), (1, _log_int(rng, 8, 500)), heads, page, lens)
    kind = rng.choice(["packed", "chunks", "tokens"])
    if kind == "tokens":
        return _prompt(None, _log_int(rng, 1, 64), (1, 1), (0, _log_int(rng, 30, 4000)), heads, page, lens)
    if kind == "chunks":
        return _prompt(None, _log_int(rng, 1, 6), (1, _log_int(rng, 16, 512)), (0, _log_int(rng, 100, 7000)), heads, page, lens)
    seqs = _log_int(rng, 1, 32)
    total = _log_int(rng, 8 * seqs, 6000 if seqs == 1 or seqs > 8 else 3000)
    mean = total // seqs
    return _prompt(None, seqs, (max(1, mean // 4), mean if seqs == 1 else 2 * mean), (0, 0), heads, 0, lens)


def _lengths(case):
    """What a batch is made of: per sequence (queries, keys of its own), per group (first sequence, prefix)."""
    r = random.Random(case["lens"])
    n = case["seqs"]
    if case["op"] == "prompt":
        q = [_log_int(r, case["q_lo"], case["q_hi"]) for _ in range(n)]
        kv = [x + r.randint(case["past_lo"], case["past_hi"]) for x in q]
        return q, kv, [], []
    q = [1] * n
    kv = [r.randint(case["own_lo"], case["own_hi"]) for _ in range(n)]
    g = case["groups"]
    starts = [0] + sorted(r.sample(range(1, n), g - 1)) + [n]
    prefix = [r.randint(case["prefix_lo"], case["prefix_hi"]) for _ in range(g)]
    return q, kv, starts, prefix


def work(case):
    hq, hkv, d = case["heads"], case["kv_heads"], case["head_dim"]
    if case["op"] == "rope":
        t = case["tokens"]
        row = (hq + 2 * hkv) * d * 2
        table = min(t, MAX_POS) * case["rot_dim"] * 4 if case["rot_dim"] else 0
        return {"bytes": 2 * t * row + table + 4 * t + (4 * t if case["cache"] else 0) + 4 * d,
                "flops": t * (hq + hkv) * (4 * d + 3 * case["rot_dim"])}
    q, kv, starts, prefix = _lengths(case)
    pairs = sum(sum(max(0, k - n + 1 + i) for i in range(n)) for n, k in zip(q, kv))
    pairs += sum(p * (b - a) for a, b, p in zip(starts, starts[1:], prefix))
    rows = sum(kv) + sum(prefix)
    return {"bytes": 2 * sum(q) * hq * d * 2 + 2 * rows * hkv * d * 2, "flops": 4 * pairs * hq * d}


# ------------------------------------------------------------------ inputs

def _rand(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda").to(torch.bfloat16)


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _cache_places(gen, lens, page, spare):
    """Pages given out in no order: (int32 table [n][widest], rows of the whole cache)."""
    need = [-(-x // page) for x in lens]
    wide = max(1, max(need))
    total = sum(need) + spare
    order = torch.randperm(total, generator=gen, device="cuda").to(torch.int32)
    first = torch.tensor([0] + need, device="cuda").cumsum(0)[:-1]
    idx = (first[:, None] + torch.arange(wide, device="cuda")[None, :]).clamp_(max=total - 1)
    return order[idx], total * page


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    hq, hkv, d = case["heads"], case["kv_heads"], case["head_dim"]
    s = {"case": case, "scale": 1.0 / math.sqrt(d)}
    if case["op"] == "rope":
        t, rot = case["tokens"], case["rot_dim"]
        s["qkv"] = _rand(gen, t, (hq + 2 * hkv) * d)
        s["q_weight"] = (1 + 0.1 * torch.randn(d, generator=gen, device="cuda")).to(torch.bfloat16)
        s["k_weight"] = (1 + 0.1 * torch.randn(d, generator=gen, device="cuda")).to(torch.bfloat16)
        s["positions"] = torch.randint(0, MAX_POS, (t,), generator=gen, device="cuda", dtype=torch.int32)
        freq = 10000.0 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)
        ang = torch.arange(MAX_POS, device="cuda", dtype=torch.float64)[:, None] * freq
        s["cos_sin"] = torch.cat([ang.cos(), ang.sin()], 1).float()
        rows = t + (t // 8 + 16 if case["cache"] else 0)
        s["slots"] = torch.randperm(rows, generator=gen, device="cuda")[:t].to(torch.int32) if case["cache"] else None
        s["q_out"] = torch.zeros(t, hq * d, dtype=torch.bfloat16, device="cuda")
        s["k_out"] = torch.zeros(rows, hkv * d, dtype=torch.bfloat16, device="cuda")
        s["v_out"] = torch.zeros(rows, hkv * d, dtype=torch.bfloat16, device="cuda")
        if own:  # the fixed shape of the layer, as the library takes it
            from heterogeneous_adapters_lora_gb300 import lora
            s["desc"] = lora.RopeDesc(n_q_heads=hq, n_kv_heads=hkv, head_dim=d, rot_dim=rot,
                                      interleaved=int(case["interleaved"]), max_pos=MAX_POS, eps=EPS)
        return s
    q, kv, starts, prefix = _lengths(case)
    t, page = sum(q), case["page"]
    cu = [0]
    for x in q:
        cu.append(cu[-1] + x)
    s["cu_q"], s["kv_len"] = _i32(cu), _i32(kv)
    s["max_q"], s["max_kv"] = max(q), max(kv)
    s["group_start"] = _i32(starts) if prefix else None
    s["prefix_len"] = _i32(prefix) if prefix else None
    s["max_prefix"] = max(prefix) if prefix else 0
    if page:
        s["q"] = _rand(gen, t, hq * d)
        table, rows = _cache_places(gen, kv + prefix, page, 7)
        s["k"], s["v"] = _rand(gen, rows, hkv * d), _rand(gen, rows, hkv * d)
        s["table"], s["prefix_table"] = table[:len(kv)], table[len(kv):] if prefix else None
    else:  # the packed QKV output itself: keys and values where the layer wrote them
        qkv = _rand(gen, t, (hq + 2 * hkv) * d)
        s["q"], s["k"], s["v"] = qkv.split([hq * d, hkv * d, hkv * d], dim=1)
        s["table"], s["prefix_table"] = s["cu_q"][:-1].reshape(-1, 1), None
    s["out"] = torch.zeros(t, hq * d, dtype=torch.bfloat16, device="cuda")
    if own:  # the plan of the batch (one for all layers of a step) and the workspace a program keeps
        from heterogeneous_adapters_lora_gb300 import lora
        desc = lora.AttnDesc(n_q_heads=hq, n_kv_heads=hkv, head_dim=d, page_size=page, causal=1, scale=s["scale"])
        n, g = len(kv), len(prefix)
        s["plan"] = lora.AttnPlan()
        size = lora.lora_attn_plan_bytes(desc, t, n, g)
        s["plan_buf"] = torch.empty(size, dtype=torch.uint8, device="cuda")
        lora.lora_attn_plan_bind(s["plan"], desc, s["plan_buf"], size, t, n, g)
        lora.lora_attn_build_plan(s["plan"], n, t, s["cu_q"], s["kv_len"], g, s["group_start"], s["prefix_len"],
                                  s["max_kv"], s["max_prefix"])
        s["ws_bytes"] = lora.lora_attn_workspace_bytes(s["plan"])
        s["ws"] = torch.empty(s["ws_bytes"], dtype=torch.uint8, device="cuda")
        lora.lora_workspace_init(s["ws"], s["ws_bytes"])
    return s


# ------------------------------------------------------------------ plain forms

def _norm_rope(x, weight, cos, sin, rot, interleaved):
    x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight
    r, rest = x[..., :rot], x[..., rot:]
    a, b = (r[..., 0::2], r[..., 1::2]) if interleaved else (r[..., :rot // 2], r[..., rot // 2:])
    p, q = a * cos - b * sin, b * cos + a * sin
    r = torch.stack([p, q], -1).flatten(-2) if interleaved else torch.cat([p, q], -1)
    return torch.cat([r, rest], -1)


def _plain_rope(s):
    c = s["case"]
    hq, hkv, d, rot = c["heads"], c["kv_heads"], c["head_dim"], c["rot_dim"]
    t = s["qkv"].shape[0]
    q, k, v = s["qkv"].split([hq * d, hkv * d, hkv * d], dim=1)
    cs = s["cos_sin"][s["positions"].long()][:, None, :]
    cos, sin = cs[..., :rot // 2], cs[..., rot // 2:]
    q = _norm_rope(q.float().view(t, hq, d), s["q_weight"].float(), cos, sin, rot, c["interleaved"])
    k = _norm_rope(k.float().view(t, hkv, d), s["k_weight"].float(), cos, sin, rot, c["interleaved"])
    s["q_out"].copy_(q.view(t, -1))
    if s["slots"] is None:
        s["k_out"].copy_(k.view(t, -1))
        s["v_out"].copy_(v)
    else:
        s["k_out"][s["slots"].long()] = k.view(t, -1).to(torch.bfloat16)
        s["v_out"][s["slots"].long()] = v
    return {"q": s["q_out"], "k": s["k_out"], "v": s["v_out"]}


def _rows(table, page, n):
    """Row of every logical key: [sequences][n]."""
    j = torch.arange(n, device=table.device)
    if not page:
        return table.long() + j
    return table.long()[:, (j // page).clamp(max=table.shape[1] - 1)] * page + j % page


def _plain_attention(s):
    c = s["case"]
    hq, hkv, d, page = c["heads"], c["kv_heads"], c["head_dim"], c["page"]
    g, cu, kv = hq // hkv, s["cu_q"].long(), s["kv_len"].long()
    n, t, dev = kv.shape[0], s["q"].shape[0], s["q"].device
    q_len = cu[1:] - cu[:-1]
    i = torch.arange(s["max_q"], device=dev)
    j = torch.arange(s["max_kv"], device=dev)
    # a query sees the keys up to its own place, which ends with the sequence's last key
    seen = j[None, None, :] <= (kv - q_len)[:, None, None] + i[None, :, None]
    seen = seen & (j[None, None, :] < kv[:, None, None])
    rows = _rows(s["table"], page, s["max_kv"])
    if s["prefix_len"] is not None:
        starts = s["group_start"].long()
        group = torch.searchsorted(starts, torch.arange(n, device=dev), right=True) - 1
        jp = torch.arange(s["max_prefix"], device=dev)
        ahead = (jp[None, :] < s["prefix_len"].long()[group][:, None])[:, None, :].expand(n, s["max_q"], -1)
        seen = torch.cat([ahead, seen], 2)
        rows = torch.cat([_rows(s["prefix_table"], page, s["max_prefix"])[group], rows], 1)
    rows = rows.clamp(max=s["k"].shape[0] - 1)
    take = (cu[:-1, None] + i).clamp(max=t - 1)
    q = s["q"][take].float().view(n, -1, hkv, g, d).permute(0, 2, 3, 1, 4).reshape(n, hkv, -1, d)
    k = s["k"][rows].float().view(n, -1, hkv, d).permute(0, 2, 3, 1)
    v = s["v"][rows].float().view(n, -1, hkv, d).transpose(1, 2)
    score = torch.matmul(q, k).mul_(s["scale"]).view(n, hkv, g, s["max_q"], -1)
    score.masked_fill_(~seen[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    p = score.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(n, hkv, g * s["max_q"], -1), v).view(n, hkv, g, s["max_q"], d)
    o = o / torch.where(total == 0, 1.0, total)
    seq = torch.repeat_interleave(torch.arange(n, device=dev), q_len, output_size=t)
    return o[seq, :, :, torch.arange(t, device=dev) - cu[seq]].reshape(t, hq * d).to(torch.bfloat16)


def run(state):
    s = state
    op = s["case"]["op"]
    if not own:
        return _plain_rope(s) if op == "rope" else _plain_attention(s)
    from heterogeneous_adapters_lora_gb300 import lora
    if op == "rope":
        t = s["qkv"].shape[0]
        lora.lora_qk_norm_rope(s["desc"], s["qkv"], s["qkv"].stride(0), t, s["q_weight"], s["k_weight"], s["positions"],
                               s["cos_sin"], s["q_out"], s["q_out"].stride(0), s["k_out"], s["k_out"].stride(0),
                               s["v_out"], s["v_out"].stride(0), s["slots"], s["k_out"].shape[0], None)
        return {"q": s["q_out"], "k": s["k_out"], "v": s["v_out"]}
    q, k, v, out, table = s["q"], s["k"], s["v"], s["out"], s["table"]
    if op == "prompt":
        lora.lora_prompt_attention(s["plan"], q, q.stride(0), k, k.stride(0), v, v.stride(0), k.shape[0], table,
                                   table.stride(0), out, out.stride(0), s["ws"], s["ws_bytes"])
    else:
        lora.lora_prefix_attention(s["plan"], q, q.stride(0), k, k.stride(0), v, v.stride(0), k.shape[0], table,
                                   table.stride(0), s["prefix_table"], s["prefix_table"].stride(0), out, out.stride(0),
                                   s["ws"], s["ws_bytes"])
    return out


# ------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    hq, hkv, d = case["heads"], case["kv_heads"], case["head_dim"]
    if case["op"] == "rope":
        t, rot = case["tokens"], case["rot_dim"]
        x = s["qkv"].double().view(t, hq + 2 * hkv, d)
        out = x.clone()
        for first, count, w in ((0, hq, s["q_weight"]), (hq, hkv, s["k_weight"])):
            y = x[:, first:first + count]
            y = y / (y.pow(2).sum(-1, keepdim=True) / d + EPS).sqrt() * w.double()
            out[:, first:first + count] = y
            cs = s["cos_sin"].double()[s["positions"].long()]
            for m in range(rot // 2):
                a, b = (2 * m, 2 * m + 1) if case["interleaved"] else (m, m + rot // 2)
                co, si = cs[:, m, None], cs[:, rot // 2 + m, None]
                out[:, first:first + count, a] = y[..., a] * co - y[..., b] * si
                out[:, first:first + count, b] = y[..., a] * si + y[..., b] * co
        rows = s["k_out"].shape[0]
        place = s["slots"].long() if s["slots"] is not None else torch.arange(t, device="cuda")
        k = torch.zeros(rows, hkv * d, dtype=torch.float64, device="cuda")
        v = torch.zeros_like(k)
        k[place] = out[:, hq:hq + hkv].reshape(t, -1)
        v[place] = out[:, hq + hkv:].reshape(t, -1)
        return {"q": out[:, :hq].reshape(t, -1), "k": k, "v": v}
    q_lens, kv, starts, prefix = _lengths(case)
    page, g = case["page"], hq // hkv
    out = torch.empty(sum(q_lens), hq, d, dtype=torch.float64, device="cuda")

    def places(table, b, n):
        j = torch.arange(n, device="cuda")
        return table[b].long()[j // page] * page + j % page if page else table[b, 0].long() + j

    at = 0
    for b, (n, m) in enumerate(zip(q_lens, kv)):
        rows, ahead = places(s["table"], b, m), 0
        if prefix:
            mine = max(x for x in range(len(prefix)) if starts[x] <= b)
            ahead = prefix[mine]
            rows = torch.cat([places(s["prefix_table"], mine, ahead), rows])
        last = ahead + m - n + torch.arange(n, device="cuda")
        hidden = torch.arange(ahead + m, device="cuda")[None, :] > last[:, None]
        k = s["k"][rows].double().view(-1, hkv, d)
        v = s["v"][rows].double().view(-1, hkv, d)
        for h in range(hq):
            score = s["q"][at:at + n, h * d:(h + 1) * d].double() @ k[:, h // g].T / math.sqrt(d)
            score[hidden] = -math.inf
            out[at:at + n, h] = torch.softmax(score, -1) @ v[:, h // g]
        at += n
    return out.view(-1, hq * d)
