"""The first call of a process may be a captured one: the per-request operators look
up what they need of the device without touching the stream under capture."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CODE = """
import torch
from speculative_decoding_spec_gb300 import binding, synth
g = torch.Generator(device="cuda").manual_seed(1)
M, V, K, r = 9, 50001, 512, 16
x = torch.randn((M, V), generator=g, device="cuda") * 2
u = torch.rand(M, generator=g, device="cuda")
p = torch.full((M,), 0.9, device="cuda")
d = torch.zeros((3, 2), dtype=torch.int32, device="cuda")
w = {name: synth.make_matrix(g, name, 1, 768, K, 0.02, "cuda") for name in ("bf16", "q4_0")}
h = torch.randn((M, K), generator=g, device="cuda")
lora = binding.Lora((torch.randn((3, r, K), generator=g, device="cuda") * 0.05).bfloat16(),
                    (torch.randn((3, 768, r), generator=g, device="cuda") * 0.1).bfloat16())
ids = (torch.arange(M, device="cuda") %% 4 - 1).to(torch.int32)
calls = {"sample": lambda: binding.spec_sample(x, u), "sample_p": lambda: binding.spec_sample(x, u, None, None, p),
         "accept": lambda: binding.spec_accept_sampled(x, d, u, None, None, p),
         "lora_bf16": lambda: (binding.spec_linear_lora(w["bf16"], h, lora, ids),),
         "lora_q4_0": lambda: (binding.spec_linear_lora(w["q4_0"], h, lora, ids),)}
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = calls[%r]()
graph.replay()
torch.cuda.synchronize()
want = calls[%r]()
assert all(torch.equal(a, b) for a, b in zip(got, want))
print("same")
"""


@pytest.mark.parametrize("call", ["sample", "sample_p", "accept", "lora_bf16", "lora_q4_0"])
def test_first_call_is_captured(call):
    r = subprocess.run([sys.executable, "-c", CODE % (call, call)], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "same" in r.stdout, r.stdout + r.stderr
