"""Attention with scores of any size: finite ones far outside the range of the exponential."""
import math

import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from test_gpu_attention import INF, Case  # noqa: E402

pytestmark = pytest.mark.gpu

SHAPES = {
    "one": dict(seqs=[(1, 300), (1, 5)], hq=12, hk=2, page=16),
    "long": dict(seqs=[(1, 40019)], hq=12, hk=1, page=64),
    "causal": dict(seqs=[(70, 200), (3, 140), (1, 0)], hq=6, hk=2, page=16),
    "tree": dict(seqs=[(20, 150), (64, 30)], hq=24, hk=2, page=16, tree=True),
    "copies": dict(seqs=[(5, 400)], hq=8, hk=2, page=5),
}


def far(shape, d, top, sign):
    """Scores sign * j * top / 256, j whole numbers of 128 to 255: exact in FP32, and so far apart that of a row's
    positions only those of the highest score count, each as much as another."""
    c = Case(d=d, scale=2.0 ** -4, seed=d, **SHAPES[shape])
    a = round(math.log2(top) + 4 - 8)  # of q times the unit of k
    g = torch.Generator(device="cuda").manual_seed(7)
    c.q[...] = 0
    c.q[..., 3] = sign * 2.0 ** (a - a // 2)
    for s, n in enumerate(c.lens):
        c.keys[s] = torch.zeros_like(c.keys[s])
        c.keys[s][..., 3] = torch.randint(128, 256, (n, c.hk), generator=g, device="cuda") * 2.0 ** (a // 2)
    c.fill()
    return c


@pytest.mark.parametrize("shape", list(SHAPES))
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("power", [20, 24, 27, 28, 29, 31, 34, 40, 60, 100])
def test_scores_beyond_the_exponential(dep, shape, d, sign, power):
    c = far(shape, d, 2.0 ** power, sign)
    got = c.run(dep)
    for s, n in enumerate(c.new):
        f, G = c.first[s], c.hq // c.hk
        see = c.seen(s)
        for h in range(c.hq):
            x = (c.q[f: f + n, h].double() @ c.keys[s][:, h // G].double().T * c.scale).masked_fill(~see, -INF)
            top = x.amax(-1, keepdim=True)
            p = ((x == top) & see).double()
            count = p.sum(-1, keepdim=True)
            p = p / count.clamp(min=1)
            v = c.values[s][:, h // G].double()
            # o: its rounding and P's (2^-8 each at most, P's the same for all), sums of FP32
            bound = 2.0 ** -8 * (p @ v).abs() + (2.0 ** -8 + 2.0 ** -20) * (p @ v.abs()) + 1e-38
            assert ((got[f: f + n, h].double() - p @ v).abs() <= bound).all(), (s, h)
            # lse: the factor log2 e, its product with the score, ln 2 and the last product, 2^-24 each
            lse = (top + count.log())[:, 0]
            g = c.lse[f: f + n, h].double()
            assert torch.where(count[:, 0] == 0, g == -INF, (g - lse).abs() <= 2.0 ** -22 * lse.abs()).all(), (s, h)


@pytest.mark.parametrize("shape", list(SHAPES))
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("power", [10, 16, 20, 22])
def test_small_differences_of_large_scores(dep, shape, d, power):
    """2^power + small whole numbers, exact in FP32: the differences alone count."""
    c = Case(d=d, scale=1.0, seed=d, **SHAPES[shape])
    g = torch.Generator(device="cuda").manual_seed(8)
    c.q[...] = 0
    c.q[..., 1] = 2.0 ** (power // 2)
    c.q[..., 2] = 1
    for s, n in enumerate(c.lens):
        c.keys[s] = torch.zeros_like(c.keys[s])
        c.keys[s][..., 1] = 2.0 ** (power - power // 2)
        c.keys[s][..., 2] = torch.randint(-3, 4, (n, c.hk), generator=g, device="cuda")
    c.fill()
    got = c.run(dep)
    for s, n in enumerate(c.new):
        f, G = c.first[s], c.hq // c.hk
        see = c.seen(s)
        for h in range(c.hq):
            x = (c.q[f: f + n, h].double() @ c.keys[s][:, h // G].double().T).masked_fill(~see, -INF)
            lse = x.logsumexp(-1)
            p = torch.where(see & (lse > -INF)[:, None], (x - lse[:, None]).exp(), 0.0)
            v = c.values[s][:, h // G].double()
            # o: its rounding and that of every p, 2^-8 each; the products and sums of FP32
            bound = 2.0 ** -8 * (p @ v).abs() + (2.0 ** -8 + 2.0 ** -18) * (p @ v.abs()) + 1e-38
            assert ((got[f: f + n, h].double() - p @ v).abs() <= bound).all(), (s, h)
            gl = c.lse[f: f + n, h].double()
            assert torch.where(lse == -INF, gl == -INF, (gl - lse).abs() <= 2.0 ** -22 * lse.abs()).all(), (s, h)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("context", [0, 100, 40000])
def test_log_sum_exp_near_zero(dep, d, context):
    """Sums of almost one: their logarithm is as exact as FP32 numbers next to one are."""
    c = Case([(1, context), (3, 0)], 4, 2, d, 16, scale=0.125, seed=5)
    length = context + 1
    c.q[...] = 0
    c.q[..., 0] = 1.0
    # exact scores: -8 ln(length) times the scale, as near as BF16 comes to it
    for s, n in enumerate(c.lens):
        c.keys[s] = torch.zeros_like(c.keys[s])
        c.keys[s][..., 0] = -8 * math.log(length if s == 0 else 1)
    c.fill()
    c.run(dep)
    for s, n in enumerate(c.new):
        see = c.seen(s)
        x = (c.q[c.first[s]: c.first[s] + n, 0].double() @ c.keys[s][:, 0].double().T * c.scale).masked_fill(~see, -INF)
        # the score's product with log2 e, twenty of its size at most, the sum (of equal terms, added pairwise and in turn: 2^-17
        # of it at this length), the logarithm and its products
        limit = 2.0 ** -22 * x.masked_fill(~see, 0).abs().amax(-1) + 2.0 ** -24 * 2 * (1 + see.sum(-1) / 64) + 2.0 ** -22
        got = c.lse[c.first[s]: c.first[s] + n].double()
        assert ((got - x.logsumexp(-1)[:, None]).abs() <= limit[:, None]).all(), (got, x.logsumexp(-1))
