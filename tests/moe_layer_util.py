"""A layer of experts with adapters: inputs, the formula in 64 bits, and how far fp32 sums may be from it."""
import numpy as np
import torch

from heterogeneous_adapters_lora_gb300 import lora as L


def act(g, gelu):
    if gelu:
        return 0.5 * g * (1 + np.tanh(np.sqrt(2 / np.pi) * (g + 0.044715 * g ** 3)))
    return g / (1 + np.exp(-g))


def _normal(gen, std, *shape):
    return (std * torch.randn(*shape, generator=gen)).to(torch.bfloat16)


class Layer:
    """Weights, adapters and a batch on the GPU; `reference` works on copies of them."""

    def __init__(self, T, E, K, D, F, adapters=0, rank=0, ranks=None, scales=None, shared=False, n13=2, gelu=False, seed=0,
                 pads=(0, 0, 0, 0), p_none=0.1, max_tokens=None, with_weights=True):
        g = torch.Generator().manual_seed(seed)
        self.T, self.E, self.K, self.D, self.F, self.gelu, self.shared = T, E, K, D, F, gelu, shared
        self.x = _normal(g, 1.0, T, D + pads[0])
        self.w13 = _normal(g, D ** -0.5, E, 2 * F, D + pads[1])
        self.w2 = _normal(g, F ** -0.5, E, D, F + pads[2])
        self.ids = torch.stack([torch.randperm(E, generator=g)[:K] if K <= E else torch.randint(0, E, (K,), generator=g)
                                for _ in range(T)]).to(torch.int32) if T else torch.zeros(0, K, dtype=torch.int32)
        self.weights = torch.rand(T, K, generator=g) if with_weights else None
        self.pad_out = pads[3]
        self.adapters, self.pool, self.idx = adapters, None, None
        if adapters:
            outer = 1 if shared else E
            self.ranks = [rank] * adapters if ranks is None else list(ranks)
            self.scales = [1.0 + 0.5 * a for a in range(adapters)] if scales is None else list(scales)
            self.a13 = _normal(g, D ** -0.5, adapters, outer, n13, rank, D)
            self.b13 = _normal(g, 0.5 * rank ** -0.5, adapters, E, 2 * F, rank)
            self.a2 = _normal(g, F ** -0.5, adapters, E, rank, F)
            self.b2 = _normal(g, 0.5 * rank ** -0.5, adapters, outer, D, rank)
            self.n13 = n13
            idx = torch.randint(0, adapters, (T,), generator=g)
            idx[torch.rand(T, generator=g) < p_none] = -1
            self.idx = idx.to(torch.int32)
            self.pool = L.lora_pool_create(L.PoolDesc(max_loras=adapters, max_rank=rank, num_experts=E, d_model=D, d_mlp=F, n_w13_slices=n13,
                                                      w13_slice_width=2 * F // n13, shared_outer=int(shared)))
            keep = []
            for a, r in enumerate(self.ranks):
                if r == 0:
                    continue
                A = [self.a13[a, :, j, :r].contiguous().cuda() for j in range(n13)] + [self.a2[a, :, :r].contiguous().cuda()]
                w = 2 * F // n13
                B = [self.b13[a, :, j * w:(j + 1) * w, :r].contiguous().cuda() for j in range(n13)]
                B.append(self.b2[a, :, :, :r].contiguous().cuda())
                L.lora_set_moe(self.pool, a, r, self.scales[a], A, [outer] * n13 + [E], B, [E] * n13 + [outer])
                keep += A + B
            torch.cuda.synchronize()
        self.desc = L.MoELayerDesc(n_experts=E, top_k=K, d_model=D, d_mlp=F, activation=int(gelu))
        self.ws_bytes = L.lora_moe_layer_workspace_bytes(self.desc, self.pool, T if max_tokens is None else max_tokens)
        self.ws = torch.zeros(self.ws_bytes, dtype=torch.uint8, device="cuda")
        self.dev = {k: None if v is None else v.cuda() for k, v in
                    {"x": self.x, "w13": self.w13, "w2": self.w2, "ids": self.ids, "weights": self.weights, "idx": self.idx}.items()}
        self.out = torch.full((T + 1, D + pads[3]), 7.0, dtype=torch.bfloat16, device="cuda")
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def close(self):
        if self.pool:
            L.lora_pool_destroy(self.pool)
            self.pool = None

    def __del__(self):
        self.close()

    def batch(self, **values):
        """Other rows, ids, weights or slots (host tensors of the same shapes)."""
        for k, v in values.items():
            setattr(self, k, v)
            self.dev[k].copy_(v)
        return self

    def call(self, stream=None):
        d = self.dev
        L.lora_moe_layer(self.desc, self.pool, d["idx"], d["x"], d["x"].stride(0), self.T, d["ids"], d["weights"], d["w13"],
                         d["w13"].stride(1), d["w2"], d["w2"].stride(1), self.out, self.out.stride(0), self.status, self.ws, self.ws_bytes,
                         stream)
        return self.out

    def reference(self):
        """(out in 64 bits, bound of the error of fp32 sums with h in two bf16 before the last rounding)."""
        T, K, D, F = self.T, self.K, self.D, self.F
        x = self.x[:, :D].double().numpy()
        out, bound = np.zeros((T, D)), np.zeros((T, D))
        step = 2.0 ** -23  # of a sum: one step of it for each addition, whichever way it is rounded
        for t in range(T):
            a = -1 if self.idx is None else int(self.idx[t])
            if not 0 <= a < self.adapters or self.ranks[a] == 0:
                a = -1
            for k in range(K):
                e = int(self.ids[t, k])
                if not 0 <= e < self.E:
                    continue
                w13, w2 = self.w13[e, :, :D].double().numpy(), self.w2[e, :, :F].double().numpy()
                gu = w13 @ x[t]
                off = (D + 4) * step * (np.abs(w13) @ np.abs(x[t]))
                if a >= 0:
                    r, s, near = self.ranks[a], self.scales[a], 0 if self.shared else e
                    b13 = self.b13[a, e, :, :r].double().numpy()
                    for j in range(2):
                        A = self.a13[a, near, j if self.n13 == 2 else 0, :r].double().numpy()
                        part = slice(j * F, (j + 1) * F)
                        gu[part] += s * (b13[part] @ (A @ x[t]))
                        off[part] += (D + r + 8) * step * s * (np.abs(b13[part]) @ (np.abs(A) @ np.abs(x[t])))
                g, u = gu[:F], gu[F:]
                ag = act(g, self.gelu)
                h = ag * u
                # |act'| <= 1.13; act itself is off by a few steps of |g|
                dh = (1.13 * off[:F] + 8 * step * np.abs(g)) * (np.abs(u) + off[F:]) + np.abs(ag) * off[F:] + 2 * step * np.abs(h)
                h_off = dh + 2.0 ** -16 * np.abs(h)
                y = w2 @ h
                dy = np.abs(w2) @ (h_off + (F + 4) * step * np.abs(h))
                if a >= 0:
                    A, B = self.a2[a, e, :r].double().numpy(), self.b2[a, near, :, :r].double().numpy()
                    y += s * (B @ (A @ h))
                    dy += s * (np.abs(B) @ (np.abs(A) @ (h_off + (F + r + 8) * step * np.abs(h))))
                w = 1.0 if self.weights is None else float(self.weights[t, k])
                out[t] += w * y
                bound[t] += abs(w) * (dy + (K + 2) * step * np.abs(y))
        return out, bound

    def check(self, out=None):
        got = (self.out if out is None else out).float().cpu().double().numpy()
        assert np.all(got[self.T:] == 7.0) and np.all(got[:, self.D:] == 7.0)  # nothing beside the rows
        want, bound = self.reference()
        got = got[:self.T, :self.D]
        off = np.abs(got - want)
        assert np.all(off <= 2.0 ** -8 * np.abs(want) + 1.01 * bound), float((off / (2.0 ** -8 * np.abs(want) + bound)).max())
        return self
