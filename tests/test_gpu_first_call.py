"""The operators around the projections as the first calls of a process, inside a graph capture."""
import subprocess
import sys

import pytest

from conftest import ROOT

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

pytestmark = pytest.mark.gpu

HEAD = """
import torch
import skinny_bf16_split_gb300 as dep
def check(call):
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        out = call()
    graph.replay()
    torch.cuda.synchronize()
    got = [t.clone() for t in out]
    want = call()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
"""
CALLS = {
    "norm": """
x = torch.randn(5, 1000, device="cuda").bfloat16()
check(lambda: dep.add_rms_norm(x, quant="int8"))
""",
    "delta tokens": """
q, k, v = (torch.randn(3, 2, 64, device="cuda").bfloat16() for _ in range(3))
g, beta, S = -torch.rand(3, 2, device="cuda"), torch.rand(3, 2, device="cuda"), torch.zeros(3, 2, 64, 64, device="cuda")
So = torch.empty_like(S)
check(lambda: (dep.gated_delta_rule(q, k, v, g, beta, S, So, n_seq=3, l2norm=True), So))
""",
    "delta chunks": """
q, k, v = (torch.randn(40, 2, 64, device="cuda").bfloat16() for _ in range(3))
g, beta, S = -torch.rand(40, 2, device="cuda"), torch.rand(40, 2, device="cuda"), torch.zeros(1, 2, 64, 64, device="cuda")
So = torch.empty_like(S)
check(lambda: (dep.gated_delta_rule(q, k, v, g, beta, S, So, l2norm=True), So))
""",
    "int8": """
w = torch.randint(-127, 128, (4096, 4096), dtype=torch.int8, device="cuda")
x = torch.randint(-127, 128, (100, 4096), dtype=torch.int8, device="cuda")
p = dep.Int8Projection(w, torch.rand(4096, device="cuda"))
xs = torch.rand(100, device="cuda")
check(lambda: [p.run(x[:n], xs[:n]) for n in (1, 4, 20, 100)])
""",
}


@pytest.mark.parametrize("name", list(CALLS))
def test_first_call_of_a_process_can_be_captured(dep, name):
    r = subprocess.run([sys.executable, "-c", HEAD + CALLS[name]], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
