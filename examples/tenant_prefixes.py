"""One attention layer of a server whose tenants each have an adapter and a common instruction.

Every tenant's instruction (prefix) goes through the layer once, with the tenant's adapter, and its keys and
values stay in the paged cache.  Requests come in groups by tenant: first their own prompts, then one token at
a time, always behind the tenant's prefix, whose keys are read once for all the tenant's requests.

    x -> lora_linear_apply (QKV) -> lora_qk_norm_rope -> lora_prompt_attention / lora_prefix_attention
      -> lora_linear_apply (output)

Run on a GPU: ``python examples/tenant_prefixes.py``.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from heterogeneous_adapters_lora_gb300 import lora as L  # noqa: E402


class LoraLinear:
    """A base weight with a pool of adapters: y = x W^T + the row's adapter's delta."""

    def __init__(self, in_dim, out_dims, adapters, rank, max_tokens, gen):
        d = L.PoolDesc(max_loras=adapters, max_rank=rank, in_dim=in_dim, n_slices=len(out_dims))
        for j, o in enumerate(out_dims):
            d.out_dims[j] = o
        self.in_dim, self.out = in_dim, sum(out_dims)
        self.pool = L.lora_pool_create(d)
        self.keep = []
        for a in range(adapters):
            A = [_normal(gen, rank, in_dim, std=in_dim ** -0.5) for _ in out_dims]
            B = [_normal(gen, o, rank, std=0.3) for o in out_dims]
            L.lora_set(self.pool, a, rank, 1.0, A, B)
            self.keep += A + B
        self.W = _normal(gen, self.out, in_dim, std=in_dim ** -0.5)
        self.ws_bytes = L.lora_workspace_bytes(self.pool, max_tokens, 1)
        self.ws = torch.zeros(self.ws_bytes, dtype=torch.uint8, device="cuda")

    def __call__(self, meta, x):
        y = torch.empty(x.shape[0], self.out, dtype=torch.bfloat16, device="cuda")
        L.lora_linear_apply(self.pool, meta, x, x.stride(0), self.W, self.in_dim, None, y, y.stride(0), self.ws,
                            self.ws_bytes)
        return y

    def close(self):
        torch.cuda.synchronize()
        L.lora_pool_destroy(self.pool)


def _normal(gen, *shape, std=1.0):
    return (torch.randn(*shape, generator=gen, device="cuda") * std).to(torch.bfloat16)


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


class Layer:
    def __init__(self, hidden, heads, adapters, rank, pages, page_size, max_tokens, max_seqs, max_pos=4096, seed=0):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)
        self.hidden, (self.hq, self.hkv, self.d) = hidden, heads
        self.page = page_size
        self.qkv = LoraLinear(hidden, [self.hq * self.d, self.hkv * self.d, self.hkv * self.d], adapters, rank, max_tokens,
                              gen)
        self.proj = LoraLinear(self.hq * self.d, [hidden], adapters, rank, max_tokens, gen)
        nbytes = L.lora_meta_bytes(max_tokens, adapters)
        self.meta, self.meta_buf = L.Meta(), torch.empty(nbytes, dtype=torch.uint8, device="cuda")
        L.lora_meta_bind(self.meta, self.meta_buf, nbytes, max_tokens, adapters)
        # norms, rotation, cache
        self.rope = L.RopeDesc(n_q_heads=self.hq, n_kv_heads=self.hkv, head_dim=self.d, rot_dim=self.d, interleaved=0,
                               max_pos=max_pos, eps=1e-6)
        self.q_w, self.k_w = (1 + 0.1 * _normal(gen, self.d), 1 + 0.1 * _normal(gen, self.d))
        ang = (torch.arange(max_pos, device="cuda")[:, None] *
               10000.0 ** (-torch.arange(0, self.d, 2, device="cuda") / self.d))
        self.cos_sin = torch.cat([ang.cos(), ang.sin()], 1).float()
        self.k = torch.zeros(pages * page_size, self.hkv * self.d, dtype=torch.bfloat16, device="cuda")
        self.v = torch.zeros_like(self.k)
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        # plans and their workspace
        self.attn = L.AttnDesc(n_q_heads=self.hq, n_kv_heads=self.hkv, head_dim=self.d, page_size=page_size, causal=1,
                               scale=self.d ** -0.5)
        self.caps = (max_tokens, max_seqs, max_seqs)
        size = L.lora_attn_plan_bytes(self.attn, *self.caps)
        self.plan, self.plan_buf = L.AttnPlan(), torch.empty(size, dtype=torch.uint8, device="cuda")
        L.lora_attn_plan_bind(self.plan, self.attn, self.plan_buf, size, *self.caps)
        self.ws_bytes = L.lora_attn_workspace_bytes(self.plan)
        self.ws = torch.empty(self.ws_bytes, dtype=torch.uint8, device="cuda")
        L.lora_workspace_init(self.ws, self.ws_bytes)

    def step(self, batch, x):
        """The layer on one batch (a Batch): hidden states in, hidden states out."""
        T = x.shape[0]
        # once per step, for all layers
        L.lora_build_meta(self.qkv.pool, batch.adapter, T, None, 1, self.meta)
        L.lora_attn_build_plan(self.plan, batch.n, T, batch.cu_q, batch.kv_len, batch.groups, batch.group_start,
                               batch.prefix_len, batch.max_kv, batch.max_prefix)
        # per layer
        qkv = self.qkv(self.meta, x)
        self.q = torch.empty(T, self.hq * self.d, dtype=torch.bfloat16, device="cuda")
        L.lora_qk_norm_rope(self.rope, qkv, qkv.stride(0), T, self.q_w, self.k_w, batch.position, self.cos_sin, self.q,
                            self.q.stride(0), self.k, self.k.stride(0), self.v, self.v.stride(0), batch.slot,
                            self.k.shape[0], self.status)
        self.out = torch.empty_like(self.q)
        args = [self.plan, self.q, self.q.stride(0), self.k, self.k.stride(0), self.v, self.v.stride(0),
                self.k.shape[0], batch.table, batch.table.stride(0)]
        rest = [self.out, self.out.stride(0), self.ws, self.ws_bytes]
        if batch.groups:
            L.lora_prefix_attention(*args, batch.prefix_table, batch.prefix_table.stride(0), *rest)
        else:
            L.lora_prompt_attention(*args, *rest)
        return self.proj(self.meta, self.out)

    def close(self):
        assert int(self.status) == 0 and L.lora_attn_get_status(self.plan) == 0
        self.qkv.close()
        self.proj.close()


class Batch:
    """Sequences (pages, keys before this step, queries of this step, adapter), by tenant behind its prefix."""

    def __init__(self, seqs, page, prefixes=None):
        # seqs: list of dicts(pages, past, n, adapter); prefixes: list of (pages, length, number of seqs)
        self.n = len(seqs)
        wide = max(len(s["pages"]) for s in seqs)
        ahead = [0] * self.n
        if prefixes:
            ahead = [p[1] for p in prefixes for _ in range(p[2])]
            wide = max([wide] + [len(p[0]) for p in prefixes])
        fill = lambda pages: list(pages) + [0] * (wide - len(pages))  # noqa: E731
        cu, pos, slot, adapter = [0], [], [], []
        for s, before in zip(seqs, ahead):
            cu.append(cu[-1] + s["n"])
            for i in range(s["past"], s["past"] + s["n"]):
                pos.append(before + i)
                slot.append(s["pages"][i // page] * page + i % page)
            adapter += [s["adapter"]] * s["n"]
        self.cu_q, self.position, self.slot, self.adapter = _i32(cu), _i32(pos), _i32(slot), _i32(adapter)
        self.kv_len = _i32([s["past"] + s["n"] for s in seqs])
        self.max_kv = max(s["past"] + s["n"] for s in seqs)
        self.table = _i32([fill(s["pages"]) for s in seqs])
        self.tokens = cu[-1]
        self.groups, self.max_prefix = 0, 0
        self.group_start = self.prefix_len = self.prefix_table = None
        if prefixes:
            starts = [0]
            for p in prefixes:
                starts.append(starts[-1] + p[2])
            self.groups, self.max_prefix = len(prefixes), max(p[1] for p in prefixes)
            self.group_start, self.prefix_len = _i32(starts), _i32([p[1] for p in prefixes])
            self.prefix_table = _i32([fill(p[0]) for p in prefixes])


def run(tenants=4, requests=12, prefix=(96, 160), prompt=(5, 40), new_tokens=3, hidden=512, heads=(8, 2, 64), rank=8,
        page=16, seed=0, visit=None):
    """Prefixes, prompts and `new_tokens` single-token steps; visit(layer, batch) after each step."""
    rng = torch.Generator().manual_seed(seed)
    rand = lambda lo, hi: int(torch.randint(lo, hi + 1, (1,), generator=rng))  # noqa: E731
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    free = torch.randperm(4096, generator=rng).tolist()
    take = lambda n: [free.pop() for _ in range(n)]  # noqa: E731
    layer = Layer(hidden, heads, tenants, rank, 4096, page, 4096, 256, seed=seed)

    def step(batch):
        y = layer.step(batch, _normal(gen, batch.tokens, hidden))
        if visit:
            visit(layer, batch)
        return y

    # the tenants' prefixes, packed into one batch
    lens = [rand(*prefix) // page * page for _ in range(tenants)]
    prefixes = [take(n // page) for n in lens]
    step(Batch([dict(pages=p, past=0, n=n, adapter=a) for a, (p, n) in enumerate(zip(prefixes, lens))], page))
    # requests by tenant: prompts, then single tokens
    owner = sorted(rand(0, tenants - 1) for _ in range(requests))
    counts = [owner.count(a) for a in range(tenants)]
    shared = [(prefixes[a], lens[a], counts[a]) for a in range(tenants)]
    seqs = []
    for a in owner:
        n = rand(*prompt)
        seqs.append(dict(pages=take(-(-(n + new_tokens) // page)), past=0, n=n, adapter=a))
    y = step(Batch(seqs, page, shared))
    for _ in range(new_tokens):
        for s in seqs:
            s["past"], s["n"] = s["past"] + s["n"], 1
        y = step(Batch(seqs, page, shared))
    layer.close()
    return y


if __name__ == "__main__":
    y = run()
    print("hidden states of the last step:", tuple(y.shape), "rms %.3f" % y.float().square().mean().sqrt())
