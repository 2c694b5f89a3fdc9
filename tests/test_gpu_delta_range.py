"""The gated delta rule at the ends of its ranges: values far from one, tokens of very different
size, infinities and NaN, decays above one, many sequences; and its precision on ordinary ones.

Tolerances.  o is rounded once to BF16 (2^-8 of the value).  Before that every operand of a
product keeps 2^-22 of itself or more, and FP32 sums half a step each.  An output is a sum over a
row of the state, whose terms may cancel, and the row carries errors of what it held lately, so what such
roundings leave is counted against |S_row| |q|, the largest of the last sixteen tokens (a chunk): a sum of dk
terms with independent errors of 2^-22 is off by 2^-22 |S_row| |q| / sqrt(dk), states add up over a dozen
chunks, and the largest of some 10^5 outputs is five times the usual: 2^-19 allows two to four times that.  Where other
tokens of the chunk are far larger, an output may have lost 2^-10 of itself.
A state adds such errors up over its chunks of 16 tokens like a random walk: 2^-19 sqrt(1 + T / 16) of
its norm, the largest of the last sixteen tokens, for each sequence and head."""
import math

import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

pytestmark = pytest.mark.gpu


def make(T, hq, hv, dk, dv, channel, seed=0, rate=1.0):
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    q, k, v = rnd(T, hq, dk).bfloat16(), rnd(T, hq, dk).bfloat16(), rnd(T, hv, dv).bfloat16()
    lg = -torch.nn.functional.softplus(rnd(T, hv, dk) if channel else rnd(T, hv)) * rate
    return [q, k, v, lg, torch.sigmoid(rnd(T, hv))]


def states(n, hv, dv, dk, seed=1):
    return torch.randn(n, hv, dv, dk, generator=torch.Generator().manual_seed(seed))


def definition(q, k, v, g, beta, S, lengths, l2norm=True):
    """In float64, token by token: o, the final states, |S_row| |q| for each output and |S| for each state
    (the largest of the last sixteen tokens)."""
    dk = q.shape[2]
    q, k, v, g, beta, S = (t.double() for t in (q, k, v, g, beta, S))
    rep = v.shape[1] // q.shape[1]
    if l2norm:
        q, k = (t / (t.pow(2).sum(-1, keepdim=True) + 1e-6).sqrt() for t in (q, k))
    q, k = q.repeat_interleave(rep, 1) * dk ** -0.5, k.repeat_interleave(rep, 1)
    a = g.exp() if g.dim() == 3 else g.exp()[..., None]
    o, S = torch.zeros(v.shape, dtype=torch.float64), S.clone()
    size, norm = torch.zeros_like(o), torch.zeros(S.shape[:2], dtype=torch.float64)
    t = 0
    for s, n in enumerate(lengths):
        rows = [size_of(S[s])]
        for _ in range(n):
            St = S[s] * a[t][:, None, :]
            u = beta[t][:, None] * (v[t] - torch.einsum("hvk,hk->hv", St, k[t]))
            S[s] = St + u[:, :, None] * k[t][:, None, :]
            o[t] = torch.einsum("hvk,hk->hv", S[s], q[t])
            rows = rows[-16:] + [size_of(S[s])]
            size[t] = torch.stack(rows).amax(0) * size_of(q[t])[:, None]
            t += 1
        norm[s] = size_of(torch.stack(rows)).amax(0)
    return o, S, size, norm


def size_of(t):
    """Norm over the last dimension, infinities and NaN left out, of values whose squares may pass float64."""
    t = torch.where(torch.isfinite(t), t, 0.0)
    top = t.abs().amax(-1).clamp(min=1e-300)
    return (t / top[..., None]).norm(dim=-1) * top


def call(dep, a, S, lengths=None, l2norm=True, tokenwise=False, monkeypatch=None):
    if tokenwise:
        monkeypatch.setattr(dep._binding, "dep_delta_workspace", lambda args: 0)
    a = [t.cuda() for t in a]
    cu = torch.tensor([0] + list(lengths)).cumsum(0).int().cuda() if lengths else None
    S = S.cuda()
    o = dep.gated_delta_rule(*a, S, cu_seqlens=cu, l2norm=l2norm)
    return o.double().cpu(), S.double().cpu()


def close(o, S, want_o, want_S, size, norm, T):
    finite = torch.isfinite(want_o)
    assert torch.equal(torch.isfinite(o), finite), "outputs that are not finite, in other places"
    w, d = torch.where(finite, want_o, 0.0), torch.where(finite, o - want_o, 0.0).abs()
    bad = ~(d <= (2.0 ** -8 + 2.0 ** -10) * w.abs() + 2.0 ** -19 * size)
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:4].tolist(), float(d[bad].max()), float(w.abs()[bad].max()))
    finite = torch.isfinite(want_S)
    assert torch.equal(torch.isfinite(S), finite), "states that are not finite, in other places"
    err = size_of(torch.where(finite, S - want_S, 0.0).flatten(2))
    assert (err <= 2.0 ** -19 * math.sqrt(1 + T / 16) * norm).all(), float((err / norm.clamp(min=1e-300)).max())


@pytest.fixture(params=["chunks", "tokens"])
def way(request, monkeypatch):
    return dict(tokenwise=request.param == "tokens", monkeypatch=monkeypatch)


@pytest.mark.parametrize("channel", [True, False])
@pytest.mark.parametrize("rate", [1.0, 0.05])
@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 64), (128, 64), (64, 48)])
@pytest.mark.parametrize("T", [8, 40, 200])
def test_precision(dep, way, T, dk, dv, rate, channel):
    a, S = make(T, 2, 4, dk, dv, channel, seed=T + dk, rate=rate), states(1, 4, dv, dk)
    close(*call(dep, a, S, **way), *definition(*a, S, [T]), T)


@pytest.mark.parametrize("channel", [True, False])
@pytest.mark.parametrize("power", [-85, -80, -60, -40, 40, 100])
def test_values_far_from_one(dep, way, power, channel):
    """States and v of one size: o and the states are linear in them."""
    a, S = make(70, 2, 2, 128, 64, channel, seed=5, rate=0.1), states(1, 2, 64, 128) * 2.0 ** power
    a[2] = (a[2].float() * 2.0 ** power).bfloat16()
    close(*call(dep, a, S, **way), *definition(*a, S, [70]), 70)


@pytest.mark.parametrize("power", [-85, -60, -40, 40, 100])
def test_states_alone_far_from_one(dep, way, power):
    a, S = make(70, 2, 2, 128, 64, True, seed=6, rate=0.01), states(1, 2, 64, 128) * 2.0 ** power
    a[2].zero_()
    close(*call(dep, a, S, **way), *definition(*a, S, [70]), 70)


@pytest.mark.parametrize("start", [0.0, 2.0 ** -85, 2.0 ** -70, 1.0])
@pytest.mark.parametrize("size", [1e36, 1e25, 1e-25])
def test_states_and_values_of_different_size(dep, way, start, size):
    a, S = make(70, 2, 2, 128, 64, True, seed=7, rate=0.1), states(1, 2, 64, 128) * start
    a[2] = (a[2].float() * size).bfloat16()
    if start == 1.0 and size < 1:
        a[3] *= 0.1  # (what v brings is then below the state's precision)
    close(*call(dep, a, S, **way), *definition(*a, S, [70]), 70)


@pytest.mark.parametrize("orders", [3, 6, 12])
@pytest.mark.parametrize("rising", [True, False])
@pytest.mark.parametrize("zero", [True, False])
def test_keys_of_different_norm(dep, way, zero, rising, orders):
    """Without normalisation, k's norm runs over `orders` orders of magnitude within each chunk."""
    T, d = 48, 64
    a, S = make(T, 2, 2, d, d, True, seed=8, rate=0.1), states(1, 2, d, d)
    i = torch.arange(T) % 16 / 15
    f = 10.0 ** (-orders * (1 - i if rising else i))
    a[1] = (a[1].float() / math.sqrt(d) * f[:, None, None]).bfloat16()
    if zero:
        S.zero_()
    close(*call(dep, a, S, l2norm=False, **way), *definition(*a, S, [T], l2norm=False), T)


@pytest.mark.parametrize("channel", [True, False])
@pytest.mark.parametrize("power", [-60, -20, 30, 55])
def test_norm_of_large_and_small_queries_and_keys(dep, way, power, channel):
    """With normalisation: up to |q|, |k| of 2^60 the unit vectors, down to zeros, where 1e-6 takes over."""
    a, S = make(40, 2, 2, 128, 64, channel, seed=15), states(1, 2, 64, 128)
    a[0], a[1] = ((t.float() * 2.0 ** power).bfloat16() for t in a[:2])
    close(*call(dep, a, S, **way), *definition(*a, S, [40]), 40)


@pytest.mark.parametrize("power", [10, 25, 35, 60])
@pytest.mark.parametrize("at", [5, 16, 31])
def test_a_token_of_another_size(dep, way, at, power):
    """One token's v, far larger than all others in some value channels: those before it keep their outputs."""
    T, d = 48, 128
    a, S = make(T, 2, 2, d, d, False, seed=9, rate=0.1), 0.01 * states(1, 2, d, d)
    a[2][at, :, ::3] *= 2.0 ** power
    close(*call(dep, a, S, **way), *definition(*a, S, [T]), T)


@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("where", ["q", "k", "v", "v all", "beta", "g"])
@pytest.mark.parametrize("at", [0, 5, 15, 30, 39])
@pytest.mark.parametrize("channel", [True, False])
def test_infinities_and_nans_reach_later_tokens_only(dep, way, channel, at, where, value):
    lengths, d = (40, 9), 64
    a, S = make(49, 2, 2, d, d, channel, seed=10, rate=0.1), states(2, 2, d, d)
    if where == "q":
        a[0][at, 0, 3] = value
    elif where == "k":
        a[1][at, 0, 3] = value
    elif where == "v":
        a[2][at, 0, 5:8] = value
    elif where == "v all":
        a[2][at] = value
    elif where == "beta":
        a[4][at, 0] = value
    else:
        a[3][at, 0] = value
    want = a.copy()
    want[3] = torch.where(want[3] > 0, 0.0, want[3])  # a decay is at most one
    close(*call(dep, a, S, lengths, **way), *definition(*want, S, lengths), 40)


@pytest.mark.parametrize("chunks", [1, 2, 3])
def test_causal_in_passes_over_a_small_workspace(dep, monkeypatch, chunks):
    lengths, hv, d = (40, 0, 90, 7), 2, 64
    T, n = sum(lengths), len(lengths)
    a, S = make(T, hv, hv, d, d, True, seed=16, rate=0.1), states(n, hv, d, d)
    a[2][21, 0, 9], a[2][100, 1, 5], a[2][60] = math.nan, math.inf, a[2][60] * 2.0 ** 40
    chunk = dep.dep_delta_workspace(dep.dep_delta_args_t(tokens=T, n_seq=n, Hv=hv, Dk=d)) // (T // 16 + n)
    monkeypatch.setattr(dep._binding, "dep_delta_workspace", lambda args: chunks * chunk)
    close(*call(dep, a, S, lengths), *definition(*a, S, lengths), 90)


@pytest.mark.parametrize("channel", [True, False])
@pytest.mark.parametrize("power", [-30, 0, 30, 60])
@pytest.mark.parametrize("at", [0, 3, 15, 16, 20, 31, 33])
def test_a_decay_to_nothing_forgets(dep, way, at, power, channel):
    """After it everything is as from an empty state, however large the state was."""
    T, d = 40, 64
    a, S = make(T, 2, 2, d, d, channel, seed=17, rate=0.1), states(1, 2, d, d) * 2.0 ** power
    a[3][at] = -math.inf
    o, S = call(dep, a, S, **way)
    close(o[at:], S, *definition(*(t[at:] for t in a), torch.zeros(1, 2, d, d), [T - at]), T - at)


def test_an_infinite_state_stays_in_its_row(dep, way):
    a, S = make(40, 1, 2, 64, 64, True, seed=11), states(1, 2, 64, 64)
    S[0, 1, 7, 3], S[0, 0, 20, 20] = math.inf, math.nan
    close(*call(dep, a, S, **way), *definition(*a, S, [40]), 40)


@pytest.mark.parametrize("channel", [True, False])
def test_decays_above_one_count_as_one(dep, way, channel):
    a, S = make(50, 2, 2, 64, 64, channel, seed=12), states(1, 2, 64, 64)
    a[3][::3] = 0.5
    a[3][1] = 80.0
    want = a.copy()
    want[3] = want[3].clamp(max=0)
    close(*call(dep, a, S, **way), *definition(*want, S, [50]), 50)


@pytest.mark.parametrize("channel", [True, False])
@pytest.mark.parametrize("l2norm", [True, False])
@pytest.mark.parametrize("zeros", ["q", "k", "v", "beta", "all"])
def test_tokens_of_zeros(dep, way, zeros, l2norm, channel):
    """Some tokens, some value channels, and a whole chunk are zero."""
    T, d = 60, 64
    a, S = make(T, 2, 2, d, d, channel, seed=13), torch.zeros(1, 2, d, d)
    if not l2norm:  # beta |k|^2 below 2, where the rule contracts
        a[1] = (a[1].float() / math.sqrt(d)).bfloat16()
    for i, name in enumerate(("q", "k", "v", "", "beta")):
        if zeros in (name, "all"):
            a[i][0:3] = 0
            a[i][16:32] = 0
            a[i][40] = 0
    a[2][..., 5] = 0
    close(*call(dep, a, S, l2norm=l2norm, **way), *definition(*a, S, [T], l2norm=l2norm), T)


@pytest.mark.parametrize("n", [31, 33, 64, 100, 257, 300, 1100])
@pytest.mark.parametrize("channel", [True, False])
def test_many_sequences(dep, n, channel):
    """Ragged ones, empty ones among them, by chunks."""
    g = torch.Generator().manual_seed(n)
    lengths = torch.randint(0, 24, (n,), generator=g).tolist()
    lengths[0], lengths[-1], lengths[n // 2] = 40, 19, 0
    T = sum(lengths)
    assert T >= 8 * n
    a, S = make(T, 1, 1, 64, 16, channel, seed=n), states(n, 1, 16, 64)
    close(*call(dep, a, S, lengths), *definition(*a, S, lengths), 40)


@pytest.mark.parametrize("table", [(3, 20, 33), (0, 0, 1), (7, 7, 50), (49, 50, 50)])
def test_tokens_of_no_sequence_keep_their_outputs(dep, way, table):
    T, d = 50, 64
    a, S = make(T, 2, 2, d, d, False, seed=14), states(2, 2, d, d)
    if way["tokenwise"]:
        way["monkeypatch"].setattr(dep._binding, "dep_delta_workspace", lambda args: 0)
    out, Sd = torch.full((T, 2, d), 7.0, dtype=torch.bfloat16, device="cuda"), S.cuda()
    cu = torch.tensor(table, dtype=torch.int32, device="cuda")
    dep.gated_delta_rule(*[t.cuda() for t in a], Sd, cu_seqlens=cu, l2norm=True, out=out)
    out = out.double().cpu()
    first, end = table[0], table[2]
    assert (out[:first] == 7).all() and (out[end:] == 7).all()
    lengths = [table[1] - first, end - table[1]]
    close(out[first:end], Sd.double().cpu(), *definition(*(t[first:end] for t in a), S, lengths), 50)
