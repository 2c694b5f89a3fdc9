"""Attention where sequences share pages, heads share rows, and trees have more tokens than a word names."""
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from test_gpu_attention import NAN, Case, rnd  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [16, 5])
def test_sequences_that_share_pages(dep, d, page):
    """A prefix that all have, each with new tokens of its own behind it."""
    prefix, n = 6 * page, 3
    c = Case([(n, prefix)] * 5, 12, 2, d, page, seed=1)
    for s in range(1, 5):
        c.table[s, :6] = c.table[0, :6]
        c.keys[s][:prefix], c.values[s][:prefix] = c.keys[0][:prefix], c.values[0][:prefix]
    c.fill()
    c.check(c.run(dep))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [16, 64, 5])
def test_heads_that_share_rows(dep, d, page):
    """Caches expanded over the heads, and over the pages: strides of zero."""
    hk = 4
    c = Case([(1, 400), (20, 90)], 8, hk, d, page, seed=2)
    one = [torch.full((c.k.shape[0], page, 1, d), NAN, device="cuda", dtype=torch.bfloat16) for _ in range(2)]
    for s in range(2):
        c.keys[s], c.values[s] = (x[:, :1].expand(-1, hk, -1) for x in (c.keys[s], c.values[s]))
        at = torch.arange(c.lens[s], device="cuda")
        pg = c.table[s].long()[at // page]
        one[0][pg, at % page], one[1][pg, at % page] = c.keys[s][:, :1], c.values[s][:, :1]
    c.k, c.v = (x.expand(-1, -1, hk, -1) for x in one)
    c.check(c.run(dep))
    # every page the same
    c = Case([(1, 7 * page - 1)], 8, hk, d, page, seed=3)
    k, v = rnd(8, page, hk, d).bfloat16(), rnd(9, page, hk, d).bfloat16()
    c.keys[0], c.values[0] = k.repeat(7, 1, 1), v.repeat(7, 1, 1)
    pages = c.k.shape[0]
    c.k, c.v = k[None].expand(pages, -1, -1, -1), v[None].expand(pages, -1, -1, -1)
    c.check(c.run(dep))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [16, 5])
def test_trees_past_the_words(dep, d, page):
    """Tokens from the 64th on are seen by none, and see what their words name."""
    for seqs in ([(70, 100), (130, 0), (64, 5), (1, 40)], [(300, 1000)], [(65, 0), (66, 62)]):
        c = Case(seqs, 12, 2, d, page, tree=True, seed=len(seqs))
        for s, n in enumerate(c.new):  # what lies there does not matter
            at = c.lens[s] - n + 64
            if n > 64:
                c.keys[s][at:], c.values[s][at:] = NAN, NAN
        c.fill()
        got = c.run(dep)
        for s, n in enumerate(c.new):
            if n > 64:
                at = c.lens[s] - n + 64
                c.keys[s][at:], c.values[s][at:] = 0, 0
        c.check(got)


def test_a_table_that_names_a_page_twice(dep):
    c = Case([(2, 158)], 8, 2, 128, 16, seed=4)
    c.table[0, 3] = c.table[0, 7]
    c.keys[0][48:64], c.values[0][48:64] = c.keys[0][112:128], c.values[0][112:128]
    c.check(c.run(dep))
