"""The attention core's operators as the first calls of a process, inside a graph capture."""
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

pytestmark = pytest.mark.gpu

CALLS = {
    "rotate": """
q, k = torch.randn(5, 8, 128, device="cuda").bfloat16(), torch.randn(5, 2, 128, device="cuda").bfloat16()
pos, freqs = torch.arange(5, device="cuda", dtype=torch.int32), dep.rotary_freqs(128)[0]
check(lambda: dep.norm_rotate(q, k, pos, freqs, norm=True))
""",
    "append": """
k, v = torch.randn(5, 2, 64, device="cuda").bfloat16(), torch.randn(5, 2, 64, device="cuda").bfloat16()
kc, vc = torch.zeros(3, 16, 2, 64, device="cuda").bfloat16(), torch.zeros(3, 16, 2, 64, device="cuda").bfloat16()
slots = torch.arange(20, 25, device="cuda", dtype=torch.int32)
check(lambda: (dep.append_kv(k, v, kc, vc, slots), kc, vc)[1:])
""",
    "attention": """
for d in (64, 128):
    q = torch.randn(7, 12, d, device="cuda").bfloat16()
    kc, vc = torch.randn(70, 16, 2, d, device="cuda").bfloat16(), torch.randn(70, 16, 2, d, device="cuda").bfloat16()
    table = torch.randperm(70, device="cuda").int().view(1, 70)
    lens = torch.tensor([1100], device="cuda", dtype=torch.int32)
    check(lambda: [dep.paged_attention(q, kc, vc, table, lens)])
""",
}


@pytest.mark.parametrize("name", list(CALLS))
def test_first_call_of_a_process_can_be_captured(dep, name):
    import subprocess
    import sys

    from conftest import ROOT
    from test_gpu_first_call import HEAD
    r = subprocess.run([sys.executable, "-c", HEAD + CALLS[name]], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
