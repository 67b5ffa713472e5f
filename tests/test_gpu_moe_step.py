"""The rest of a decode step as it is used: router's choice, the experts with their adapters, lm_head with LoRA, the next tokens."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from heterogeneous_adapters_lora_gb300 import harness as H
from heterogeneous_adapters_lora_gb300 import lora as L
from moe_layer_util import Layer
from test_gpu_route import reference as route_reference
from test_gpu_sample import reference_row

pytestmark = pytest.mark.gpu


class Step:
    """route -> layer -> lora_logits_apply -> sample over one batch; the router and the lm_head's base product are the caller's."""

    def __init__(self, T, V=2000, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.layer = Layer(T, 8, 2, 256, 128, adapters=3, rank=8, seed=seed)
        self.T, self.V, self.W = T, V, (V + 7) // 8 * 8
        self.gate = torch.randn(256, 8, generator=g).cuda() / 16
        self.head = (torch.randn(256, self.W, generator=g) / 8).to(torch.bfloat16).cuda()
        d = L.PoolDesc(max_loras=3, max_rank=8, in_dim=256, n_slices=1, is_lm_head=1)
        d.out_dims[0] = self.W
        self.pool = L.lora_pool_create(d)
        self.keep = []
        for a in range(3):
            A, B = (torch.randn(8, 256, generator=g) / 16).to(torch.bfloat16).cuda(), torch.randn(self.W, 8, generator=g).to(torch.bfloat16).cuda()
            L.lora_set(self.pool, a, 8, 1.0, [A], [B])
            self.keep += [A, B]
        self.meta = H.MetaBuffer(T, 3)
        self.ws_bytes = L.lora_workspace_bytes(self.pool, T, 1)
        self.ws = torch.zeros(self.ws_bytes, dtype=torch.uint8, device="cuda")
        self.route = L.RouteDesc(n_experts=8, top_k=2, logits_f32=1, renormalize=1, scale=1.0)
        self.temperature = torch.rand(T, generator=g).cuda() + 0.5
        self.top_k = torch.randint(1, 100, (T,), generator=g).to(torch.int32).cuda()
        self.top_p = torch.full((T,), 0.95, device="cuda")
        self.uniform = torch.rand(T, generator=g).cuda()
        self.scores = torch.zeros(T, 8, device="cuda")
        self.base = torch.zeros(T, self.W, dtype=torch.bfloat16, device="cuda")
        self.logits = torch.zeros(T, self.W, dtype=torch.bfloat16, device="cuda")
        self.tokens = torch.zeros(T, dtype=torch.int32, device="cuda")
        self.logprobs = torch.zeros(T, device="cuda")

    def run(self):
        y, T = self.layer, self.T
        torch.matmul(y.dev["x"].float(), self.gate, out=self.scores)
        L.lora_moe_route(self.route, self.scores, 8, T, None, y.dev["ids"], y.dev["weights"])
        out = y.call()[:T]
        torch.matmul(out, self.head, out=self.base)
        L.lora_build_meta(self.pool, y.dev["idx"], T, None, 1, self.meta.meta)
        L.lora_logits_apply(self.pool, self.meta.meta, out, out.stride(0), self.base, self.W, self.W, None, self.logits, self.W, self.V, 1.0,
                            self.ws, self.ws_bytes)
        L.lora_sample(self.logits, self.W, T, self.V, self.temperature, self.top_k, self.top_p, None, self.uniform, self.tokens, self.logprobs)

    def check(self):
        torch.cuda.synchronize()
        y = self.layer
        ids, w = route_reference(self.scores.cpu().numpy(), 2, False, None, True, 1.0)
        assert np.array_equal(y.dev["ids"].cpu().numpy(), ids)
        assert np.allclose(y.dev["weights"].cpu().numpy(), w, rtol=2.2e-5)
        y.x, y.ids, y.weights, y.idx = (y.dev[k].cpu() for k in ("x", "ids", "weights", "idx"))
        y.check()
        x = self.logits[:, :self.V].cpu().double().numpy()
        for t in range(self.T):
            token, logprob = reference_row(x[t], float(self.temperature[t]), int(self.top_k[t]), float(self.top_p[t]), 0.0,
                                           float(self.uniform[t]))
            assert int(self.tokens[t]) == token
            assert abs(float(self.logprobs[t]) - logprob) <= 2.0 ** -20 + 2.0 ** -22 * abs(logprob)

    def close(self):
        L.lora_pool_destroy(self.pool)
        self.layer.close()


@pytest.mark.parametrize("T", [1, 6, 40])
def test_step(T):
    s = Step(T, seed=T)
    s.run()
    s.check()
    s.close()


def test_steps_from_a_graph():
    s = Step(12, seed=3)
    s.run()  # the library GEMM of the test's own products is looked up outside of the capture
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        s.run()
    for seed in (7, 8, 9):
        g = torch.Generator().manual_seed(seed)
        s.layer.dev["x"].copy_(torch.randn(12, 256, generator=g))
        s.layer.dev["idx"].copy_(torch.randint(-1, 3, (12,), generator=g))
        s.uniform.copy_(torch.rand(12, generator=g))
        graph.replay()
        s.check()
    s.close()
