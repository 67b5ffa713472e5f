"""Batches and 64-bit references of the attention tests."""
import numpy as np
import torch

from heterogeneous_adapters_lora_gb300 import lora as L


def bf16(x):
    return x.to(torch.bfloat16)


class Batch:
    """A batch in a cache whose every row that no sequence owns holds NaN (or what `poison` says)."""

    def __init__(self, q_lens, kv_lens, heads=(4, 2, 64), page=0, causal=1, groups=None, prefix_lens=None, seed=0,
                 q_pad=0, kv_pad=0, out_pad=0, scale=None, spare=3, poison=float("nan"), first_row=0, device="cuda",
                 spread=1.0):
        self.q_lens, self.kv_lens = list(q_lens), list(kv_lens)
        self.hq, self.hkv, self.d = heads
        self.page, self.causal = page, causal
        self.groups, self.prefix_lens = groups, list(prefix_lens or [])
        self.scale = scale if scale is not None else self.d ** -0.5
        g = torch.Generator().manual_seed(seed)
        T = sum(self.q_lens)
        lens = self.kv_lens + self.prefix_lens
        if page:
            need = [-(-x // page) for x in lens]
            wide = max([1] + need) + 1
            total = sum(need) + spare
            order = torch.randperm(total, generator=g) + first_row // page
            table = torch.full((len(lens), wide), -77, dtype=torch.int32)  # never to be read past a length
            at = 0
            for b, n in enumerate(need):
                table[b, :n] = order[at:at + n].to(torch.int32)
                at += n
            rows = total * page
        else:
            starts, at = [], 5
            for x in lens:
                starts.append(at)
                at += x + spare
            table = torch.tensor(starts, dtype=torch.int32).reshape(-1, 1) + first_row
            rows = at + 2
        self.rows, self.first_row = rows + first_row, first_row
        kc, qc = self.hkv * self.d, self.hq * self.d
        self.k = torch.full((rows, kc + kv_pad), poison, dtype=torch.bfloat16)
        self.v = torch.full((rows, kc + kv_pad), poison, dtype=torch.bfloat16)
        self.q = torch.full((max(T, 1), qc + q_pad), float("nan"), dtype=torch.bfloat16)
        self.q[:T, :qc] = bf16(spread * torch.randn(T, qc, generator=g))
        self.table_host = table
        self.place = []  # local row (without first_row) of every key of every table line
        for b, n in enumerate(lens):
            j = torch.arange(n)
            r = table[b].long()[j // page] * page + j % page if page else table[b, 0].long() + j
            r = r - first_row
            self.k[r, :kc] = bf16(spread * torch.randn(n, kc, generator=g))
            self.v[r, :kc] = bf16(torch.randn(n, kc, generator=g))
            self.place.append(r)
        n = len(self.kv_lens)
        self.device = device
        self.cu = torch.tensor(np.concatenate([[0], np.cumsum(self.q_lens)]), dtype=torch.int32)
        self.T, self.out_pad, self.n = T, out_pad, n

    def reference(self):
        """(out, sum_j p_j |v_j|) in float64, [T][hq][d]."""
        out = torch.zeros(self.T, self.hq, self.d, dtype=torch.float64)
        mag = torch.zeros_like(out)
        g = self.hq // self.hkv
        kc, qc = self.hkv * self.d, self.hq * self.d
        for b in range(self.n):
            nq, nk = self.q_lens[b], self.kv_lens[b]
            rows, ahead = self.place[b], 0
            if self.groups is not None:
                mine = max(x for x in range(len(self.prefix_lens)) if self.groups[x] <= b and self.groups[x + 1] > b)
                ahead = self.prefix_lens[mine]
                rows = torch.cat([self.place[self.n + mine], rows])
            t0 = int(self.cu[b])
            q = self.q[t0:t0 + nq, :qc].double().view(nq, self.hq, self.d)
            k = self.k[rows, :kc].double().view(-1, self.hkv, self.d).repeat_interleave(g, 1)
            v = self.v[rows, :kc].double().view(-1, self.hkv, self.d).repeat_interleave(g, 1)
            for i in range(nq):
                see = ahead + (max(0, min(nk, nk - nq + i + 1)) if self.causal else nk)
                if see == 0:
                    continue
                s = torch.einsum("hd,jhd->hj", q[i], k[:see]) * self.scale
                p = torch.softmax(s, -1)
                out[t0 + i] = torch.einsum("hj,jhd->hd", p, v[:see])
                mag[t0 + i] = torch.einsum("hj,jhd->hd", p, v[:see].abs())
        return out, mag

    def desc(self):
        return L.AttnDesc(n_q_heads=self.hq, n_kv_heads=self.hkv, head_dim=self.d, page_size=self.page,
                          causal=self.causal, scale=self.scale)

    def upload(self, spare_tokens=0, spare_seqs=0):
        dev = self.device
        self.dq = self.q.to(dev)
        self.dk, self.dv = self.k.to(dev), self.v.to(dev)
        self.dtable = self.table_host.to(dev)
        self.dcu = self.cu.to(dev)
        self.dkv = torch.tensor(self.kv_lens, dtype=torch.int32, device=dev)
        g = len(self.prefix_lens)
        self.dgs = torch.tensor(self.groups, dtype=torch.int32, device=dev) if g else None
        self.dpl = torch.tensor(self.prefix_lens, dtype=torch.int32, device=dev) if g else None
        caps = (max(1, self.T) + spare_tokens, max(1, self.n) + spare_seqs, g + (spare_seqs if g else 0))
        self.plan = L.AttnPlan()
        size = L.lora_attn_plan_bytes(self.desc(), *caps)
        assert size > 0
        self.plan_buf = torch.empty(size, dtype=torch.uint8, device=dev)
        L.lora_attn_plan_bind(self.plan, self.desc(), self.plan_buf, size, *caps)
        self.ws_bytes = L.lora_attn_workspace_bytes(self.plan)
        self.ws = torch.empty(self.ws_bytes, dtype=torch.uint8, device=dev)
        L.lora_workspace_init(self.ws, self.ws_bytes)
        self.out = torch.full((max(1, self.T), self.hq * self.d + self.out_pad), 7.0, dtype=torch.bfloat16, device=dev)
        self.build()
        return self

    def build(self, **kw):
        g = len(self.prefix_lens)
        L.lora_attn_build_plan(self.plan, self.n, self.T, self.dcu, self.dkv, g, self.dgs, self.dpl,
                               max(self.kv_lens + [0]), max(self.prefix_lens + [0]), **kw)

    def run(self, plan=None, **kw):
        plan = plan or self.plan
        a = [plan, self.dq, self.dq.stride(0), self.dk, self.dk.stride(0), self.dv, self.dv.stride(0),
             self.dk.shape[0], self.dtable, self.dtable.stride(0)]
        b = [self.out, self.out.stride(0), self.ws, self.ws_bytes]
        if self.prefix_lens:
            L.lora_prefix_attention(*a, self.dtable[self.n:], self.dtable.stride(0), *b, **kw)
        else:
            L.lora_prompt_attention(*a, *b, **kw)
        return self.out

    def check(self, ref=None):
        """Bounds, element by element.  A probability is rounded to bf16 once for its product with v (at most
        2^-8 of it), the result once more (2^-8 of it); scores and sums in fp32 and the approximate exponential
        are given 2^-10 of sum p |v|."""
        out, mag = ref if ref is not None else self.reference()
        got = self.out[:self.T].float().cpu().double()
        qc = self.hq * self.d
        if self.out_pad:
            assert torch.all(got[:, qc:] == 7.0)
        got = got[:, :qc].reshape(self.T, self.hq, self.d)
        bound = (2.0 ** -8 + 2.0 ** -10) * mag + 2.0 ** -8 * out.abs() + 1e-30
        bad = ~((got - out).abs() <= bound)
        assert not bad.any(), (f"{int(bad.sum())} of {bad.numel()} values off, first at {bad.nonzero()[0].tolist()}: "
                               f"{got[bad][0].item()} for {out[bad][0].item()}")
        assert L.lora_attn_get_status(self.plan) == 0
