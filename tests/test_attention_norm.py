"""The norm's limit for attention over long contexts: it passes what BF16 rounds, and sees a lost or misplaced part."""
import pytest

torch = pytest.importorskip("torch")

from attention_norm import norm_error, norm_limit  # noqa: E402


def attention(length, d, rows, seed):
    g = torch.Generator().manual_seed(seed)
    q, k, v = (torch.randn(n, d, generator=g).bfloat16().double() for n in (rows, length, length))
    return q @ k.T * d ** -0.5, v


@pytest.mark.parametrize("length", [5000, 40019])
@pytest.mark.parametrize("d", [64, 128])
def test_what_rounding_costs_is_within_the_limit(length, d):
    for seed in range(3):
        x, v = attention(length, d, 6, seed)
        want = x.softmax(-1) @ v
        p = x.exp()
        got = ((p.bfloat16().double() @ v) / p.sum(-1, keepdim=True)).bfloat16().double()
        for row in range(6):  # one token's head at a time, the fewest elements
            assert norm_error(got[row], want[row]) <= norm_limit(d)


@pytest.mark.parametrize("length", [5000, 40019])
@pytest.mark.parametrize("mistake", ["a tile's values lost", "a tile twice", "two tiles' values exchanged", "a block's share lost",
                                     "a part's sum lost", "a part of another head"])
def test_a_mistake_is_seen(length, mistake):
    x, v = attention(length, 128, 12, 1)
    p, want = x.softmax(-1), x.softmax(-1) @ v
    a, b, share = slice(1280, 1408), slice(2560, 2688), slice(1280, 1280 + length // 87)
    if mistake == "a tile's values lost":
        got = want - p[:, a] @ v[a]
    elif mistake == "a tile twice":
        got = want + p[:, a] @ v[a]
    elif mistake == "two tiles' values exchanged":
        got = want + (p[:, a] - p[:, b]) @ (v[b] - v[a])
    elif mistake == "a block's share lost":
        got = want - p[:, share] @ v[share]
    elif mistake == "a part's sum lost":
        got = want / (1 - p[:, share].sum(-1, keepdim=True))
    else:
        got = want - p[:, share] @ v[share] + (p[:, share] @ v[share]).roll(1, 0)
    for row in range(12):
        assert norm_error(got[row], want[row]) > norm_limit(128), row
