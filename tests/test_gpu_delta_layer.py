"""The layer of examples/delta_layer.py: norm, int8 projections and delta rule together."""
import os
import sys

import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module")
def example(dep):
    import delta_layer
    return delta_layer


# The output's rounding (2^-8), and one step of y's 8 bits, 1/127 of a row's largest value, which a
# rounding of the delta rule's output can move: about a quarter of that of a typical value, over sqrt(12).
OUT = 2.0 ** -8 + 4 / 127 / 12 ** 0.5


def close(got, want):
    assert (got.double() - want).norm() <= OUT * want.norm()


@pytest.mark.parametrize("hidden,heads,dim", [(256, 8, 64), (512, 16, 128)])
def test_prompts_then_decode(example, hidden, heads, dim):
    layer = example.DeltaLayer(hidden, heads, dim, slots=6)
    lengths, slots = [37, 1, 20], torch.tensor([3, 0, 5], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 37, 38, 58], dtype=torch.int32, device="cuda")
    x, r = example.tokens(58, hidden, 1)
    want, S = layer.reference(x, r, torch.zeros(3, heads, dim, dim, device="cuda"), lengths)
    close(layer.forward(x, r, slots, cu), want)
    for step in range(3):
        x, r = example.tokens(3, hidden, 2 + step)
        before = r.clone()
        want, S = layer.reference(x, r, S, [1, 1, 1])
        close(layer.forward(x, r, slots), want)
        assert torch.equal(r, (x.float() + before.float()).bfloat16())
    assert not layer.state[[1, 2, 4]].any()
    assert (layer.state[[3, 0, 5]].double() - S).norm() <= 1e-2 * S.norm()  # inputs in BF16, off by roundings


def test_step_as_a_graph(example):
    layer = example.DeltaLayer(256, 8, 64, slots=4)
    slots = torch.arange(4, dtype=torch.int32, device="cuda")
    x, r = example.tokens(4, 256, 7)
    r0 = r.clone()
    want = layer.forward(x, r, slots).clone()
    S1 = layer.state.clone()
    layer.state.zero_()
    r.copy_(r0)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer.forward(x, r, slots)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(layer.state, S1)
