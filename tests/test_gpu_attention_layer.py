"""The layer of examples/attention_layer.py: norm, int8 projections, rotation, cache and attention together."""
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
    import attention_layer
    return attention_layer


# The output's rounding (2^-8), and one step of y's 8 bits, 1/127 of a row's largest value, which a rounding of
# the attention's output can move: about a quarter of that of a typical value, over sqrt(12).
OUT = 2.0 ** -8 + 4 / 127 / 12 ** 0.5


def close(got, want):
    assert (got.double() - want).norm() <= OUT * want.norm()


@pytest.mark.parametrize("hidden,heads,kv,dim,page", [(256, 8, 2, 64, 16), (512, 16, 16, 128, 24), (256, 24, 1, 128, 5)])
def test_prompts_decode_and_drafts(example, hidden, heads, kv, dim, page):
    layer = example.AttentionLayer(hidden, heads, kv, dim, pages=90, page_size=page, factor=2.0, original=32)
    pages = example.Pages(90, page, 30)
    lengths = [37, 1, 40]
    x, r = example.tokens(78, hidden, 1)
    place = example.i32([j for n in lengths for j in range(n)])
    want, past = layer.reference(x, r, place, [None] * 3, lengths)
    close(layer.forward(x, r, place, **pages.extend(dict(enumerate(lengths)))), want)
    for step in range(3):
        x, r = example.tokens(3, hidden, 2 + step)
        before = r.clone()
        place = example.i32([n + step for n in lengths])
        want, past = layer.reference(x, r, place, past, [1, 1, 1])
        close(layer.forward(x, r, place, **pages.extend({0: 1, 1: 1, 2: 1})), want)
        assert torch.equal(r, (x.float() + before.float()).bfloat16())
    # trees of five for two of the sequences, twice: what is dropped leaves nothing behind
    tree = torch.tensor([0b1, 0b11, 0b101, 0b1101, 0b10001] * 2, device="cuda")
    depth = [0, 1, 1, 2, 1]
    for step in range(2):
        x, r = example.tokens(10, hidden, 9 + step)
        place = example.i32([lengths[s] + 3 + j for s in (0, 2) for j in depth])
        want, _ = layer.reference(x, r, place, [past[0], past[2]], [5, 5], tree)
        close(layer.forward(x, r, place, **pages.extend({0: 5, 2: 5}), tree=tree), want)
        for s in (0, 2):
            pages.drop(s, 5)


def test_a_path_of_a_tree_is_what_decoding_it_gives(example):
    layer = example.AttentionLayer(256, 8, 2, 64, pages=40, page_size=16)
    pages = example.Pages(40, 16, 12)
    x, r = example.tokens(50, 256, 1)
    layer.forward(x, r, example.i32(list(range(50))), **pages.extend({0: 50}))
    x, r = example.tokens(6, 256, 2)
    tree = torch.tensor([0b1, 0b11, 0b101, 0b1011, 0b10101, 0b101011], device="cuda")  # 0-1-3-5 and 0-2-4
    depth = example.i32([50, 51, 51, 52, 52, 53])
    drafted = layer.forward(x, r.clone(), depth, **pages.extend({0: 6}), tree=tree)
    pages.drop(0, 6)
    for i, node in enumerate((0, 1, 3, 5)):
        one = layer.forward(x[node: node + 1], r[node: node + 1].clone(), example.i32([50 + i]), **pages.extend({0: 1}))
        close(one, drafted[node: node + 1].double())


def test_step_as_a_graph(example):
    layer = example.AttentionLayer(256, 8, 2, 64, pages=40, page_size=16)
    pages = example.Pages(40, 16, 6)
    x, r = example.tokens(60, 256, 5)
    layer.forward(x, r, example.i32(list(range(30)) * 2), **pages.extend({0: 30, 1: 30}))
    x, r = example.tokens(2, 256, 7)
    r0, at, place = r.clone(), pages.extend({0: 1, 1: 1}), example.i32([30, 30])
    want = layer.forward(x, r, place, **at).clone()
    r.copy_(r0)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer.forward(x, r, place, **at)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
