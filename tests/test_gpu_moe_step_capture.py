"""The first calls of a process are captured ones: what is looked up once does not disturb a capture."""
import os
import subprocess
import sys

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

PROGRAM = """
import torch
from heterogeneous_adapters_lora_gb300 import lora as L
from moe_layer_util import Layer

layer = Layer(3, 8, 2, 264, 136, adapters=2, rank=8, seed=1)
scores = torch.randn(3, 8, device="cuda")
logits = torch.randn(3, 50000, device="cuda").to(torch.bfloat16)
tokens = torch.zeros(3, dtype=torch.int32, device="cuda")
route = L.RouteDesc(n_experts=8, top_k=2, logits_f32=1, renormalize=1, scale=1.0)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    L.lora_moe_route(route, scores, 8, 3, None, layer.dev["ids"], layer.dev["weights"])
    layer.call()
    L.lora_sample(logits, 50000, 3, 50000, None, None, None, None, None, tokens, None)
graph.replay()
torch.cuda.synchronize()
layer.ids, layer.weights = layer.dev["ids"].cpu(), layer.dev["weights"].cpu()
layer.check()
assert torch.equal(layer.ids, torch.sort(scores, 1, descending=True).indices[:, :2].int().cpu())
assert tokens.tolist() == logits.float().cpu().numpy().argmax(1).tolist()  # the first of equal ones
"""


def test_first_calls_are_captured():
    here = os.path.dirname(os.path.abspath(__file__))
    env = dict(os.environ, PYTHONPATH=os.pathsep.join([os.path.dirname(here), here, os.environ.get("PYTHONPATH", "")]))
    done = subprocess.run([sys.executable, "-c", PROGRAM], env=env, capture_output=True, text=True, timeout=300)
    assert done.returncode == 0, done.stderr
