"""Attention where values are not finite, in every form that an item takes; and long contexts by the norm of the error."""
import math

import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from attention_norm import norm_error, norm_limit  # noqa: E402
from test_gpu_attention import INF, NAN, Case  # noqa: E402

pytestmark = pytest.mark.gpu

FORMS = {
    "items whole in a block": dict(seqs=[(3, 20 + i % 9) for i in range(400)], hq=12, hk=2),
    "one tile": dict(seqs=[(3, 20), (64, 0)], hq=4, hk=1),
    "cut": dict(seqs=[(6, 3000)], hq=12, hk=1),
    "two tiles of rows": dict(seqs=[(20, 300), (20, 30)], hq=24, hk=2),
    "two tiles of rows, whole": dict(seqs=[(18, 100 + i) for i in range(200)], hq=24, hk=2),
    "three blocks of rows": dict(seqs=[(50, 70)], hq=13, hk=1),
}


@pytest.mark.parametrize("form", list(FORMS))
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [16, 5])
@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("what", [NAN, INF, -INF])
def test_values_that_only_some_rows_see(dep, form, d, page, tree, what):
    c = Case(d=d, page=page, tree=tree, seed=3, **FORMS[form])
    want, lse = c.run(dep).clone(), c.lse.clone()
    for s, n in enumerate(c.new):
        c.values[s][c.lens[s] - n + n // 2, 0, 1::5] = what
    c.fill()
    got = c.run(dep)
    assert torch.equal(c.lse, lse)
    G, hit = c.hq // c.hk, torch.zeros(d, dtype=torch.bool, device="cuda")
    hit[1::5] = True
    assert torch.equal(got[:, G:], want[:, G:]) and torch.equal(got[:, :, ~hit], want[:, :, ~hit])
    see = torch.zeros(c.T, dtype=torch.bool, device="cuda")
    for s, n in enumerate(c.new):
        see[c.first[s]: c.first[s] + n] = c.seen(s)[:, c.lens[s] - n + n // 2]
    assert see.any() and not see.all()
    assert torch.equal(got[~see], want[~see])
    seen = got[see][:, :G][:, :, hit]
    assert (seen.isnan() if math.isnan(what) else seen == what).all()


@pytest.mark.parametrize("what", [NAN, INF])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("tree", [False, True])
def test_values_behind_scores_of_minus_infinity(dep, what, d, tree):
    """A token whose scores are all minus infinity has zeros, whatever the values are; others are as they were."""
    c = Case([(1, 0), (3, 0), (2, 150), (30, 0)], 12, 2, d, 16, tree=tree, seed=4)
    if tree:
        c.tree[...] = -1
    c.q[...] = c.q.abs().clamp(min=0.01)
    want, lse = c.run(dep).clone(), c.lse.clone()
    for s in (0, 1, 3):
        c.keys[s][:, 0, 0] = -INF
        c.values[s][:, 0, ::2] = what
    c.fill()
    got = c.run(dep)
    for s, n in enumerate(c.new):
        rows = slice(c.first[s], c.first[s] + n)
        if s == 2:
            assert torch.equal(got[rows], want[rows]) and torch.equal(c.lse[rows], lse[rows])
        else:
            assert (got[rows, :6] == 0).all() and (c.lse[rows, :6] == -INF).all()
            assert torch.equal(got[rows, 6:], want[rows, 6:]) and torch.equal(c.lse[rows, 6:], lse[rows, 6:])


@pytest.mark.parametrize("power,seqs,tree", [
    (125, [(1, 511), (1, 7), (1, 999)], False), (125, [(20, 300), (64, 600)], True), (125, [(300, 100), (40, 700)], False),
    (116, [(1, 40018), (1, 3000)], False), (116, [(16, 30003)], True), (-100, [(1, 511), (3, 40000)], False),
])
@pytest.mark.parametrize("d", [64, 128])
def test_values_up_to_the_ends_of_their_range(dep, power, seqs, tree, d):
    """The sums before the division stay in FP32 wherever those of exp(score - maximum) do."""
    c = Case(seqs, 12, 2, d, 16, tree=tree, seed=6)
    for s in range(len(seqs)):
        c.values[s] = ((1 + c.values[s].float().abs() % 1) * 2.0 ** power).bfloat16()
    c.fill()
    c.check(c.run(dep))


LONG = [
    ([(1, 5000)], 12, 1, 128, 64, False), ([(1, 40018)], 12, 1, 128, 64, False), ([(1, 70001)], 12, 1, 64, 64, False),
    ([(1, 131071)], 24, 2, 128, 64, False), ([(1, 131071)], 24, 2, 64, 128, False), ([(16, 40003)], 24, 2, 128, 128, True),
    ([(16, 20003)], 24, 2, 64, 128, True), ([(64, 9000), (64, 8000)], 24, 2, 128, 64, True),
    ([(1, 30000), (1, 5), (1, 12000), (1, 7777)], 24, 2, 128, 16, False), ([(300, 9000), (40, 20000)], 6, 1, 64, 24, False),
    ([(1, 20000), (3, 7000)], 16, 2, 128, 5, False), ([(130, 9000)], 6, 2, 128, 64, False),
]


@pytest.mark.parametrize("seqs,hq,hk,d,page,tree", LONG)
def test_long_contexts_by_the_norm(dep, seqs, hq, hk, d, page, tree):
    c = Case(seqs, hq, hk, d, page, tree=tree, seed=11)
    got = c.run(dep)
    for s, n in enumerate(c.new):
        if c.lens[s] < 1000:
            continue
        f, see = c.first[s], c.seen(s)
        for h in range(hq):
            k, v = (x[:, h // (hq // hk)].double() for x in (c.keys[s], c.values[s]))
            want = (c.q[f: f + n, h].double() @ k.T * c.scale).masked_fill(~see, -INF).softmax(-1) @ v
            error = norm_error(got[f: f + n, h].double(), want)
            assert error <= norm_limit(n * d), (s, h, error)
