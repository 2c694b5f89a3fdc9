"""The gated delta rule against its definition, token by token in 64 bits."""
import math

import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

pytestmark = pytest.mark.gpu


def make(T, hq, hv, dk, dv, channel, seed=0, rate=1.0, packed=True):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    if packed:  # columns of one projection's output
        a = rnd(T, 2 * hq * dk + hv * dv + 8).bfloat16()
        q, k, v = (t for t in a[:, : 2 * hq * dk + hv * dv].split([hq * dk, hq * dk, hv * dv], 1))
        q, k, v = q.unflatten(1, (hq, dk)), k.unflatten(1, (hq, dk)), v.unflatten(1, (hv, dv))
    else:
        q, k, v = rnd(T, hq, dk).bfloat16(), rnd(T, hq, dk).bfloat16(), rnd(T, hv, dv).bfloat16()
    lg = -torch.nn.functional.softplus(rnd(T, hv, dk) if channel else rnd(T, hv)) * rate
    return q, k, v, lg, torch.sigmoid(rnd(T, hv))


def definition(q, k, v, g, beta, S, lengths, scale, l2norm, slots=None):
    """(o, final states) in float64 on the host; S: [n_states, Hv, Dv, Dk]."""
    q, k, v, g, beta, S = (t.detach().double().cpu() for t in (q, k, v, g, beta, S))
    hv, rep = v.shape[1], v.shape[1] // q.shape[1]
    if l2norm:
        q, k = (t / (t.pow(2).sum(-1, keepdim=True) + 1e-6).sqrt() for t in (q, k))
    q, k = q.repeat_interleave(rep, 1) * scale, k.repeat_interleave(rep, 1)
    a = g.exp() if g.dim() == 3 else g.exp()[..., None]
    o, S = torch.zeros(v.shape, dtype=torch.float64), S.clone()
    t = 0
    for s, n in enumerate(lengths):
        i = s if slots is None else slots[s]
        for _ in range(n):
            if 0 <= i < len(S):
                St = S[i] * a[t][:, None, :]
                u = beta[t][:, None] * (v[t] - torch.einsum("hvk,hk->hv", St, k[t]))
                S[i] = St + u[:, :, None] * k[t][:, None, :]
                o[t] = torch.einsum("hvk,hk->hv", S[i], q[t])
            t += 1
    return o, S


def close(o, S, want_o, want_S, T, dk):
    """States: FP32 sums of dk products over T tokens, half a step each, adding up like a random
    walk, four times that.  o: its rounding, and two operands rounded to 11 bits in the last product
    (eight times the root mean square of such an error)."""
    d = (S.double().cpu() - want_S).norm() / max(want_S.norm(), 1e-30)
    assert d <= 2.0 ** -22 * math.sqrt(dk * (T + 1)), float(d)
    if want_o.numel():
        d = (o.double().cpu() - want_o).abs()
        rms = want_o.pow(2).mean().sqrt()
        bad = ~(d <= 2.0 ** -8 * want_o.abs() + 8 * 2.0 ** -11 * rms)
        assert not bad.any(), (int(bad.sum()), bad.nonzero()[:4].tolist(), float(d.max()))


def run_case(dep, lengths, hq, hv, dk, dv, channel, l2norm=True, seed=0, rate=1.0, zero=False, use_cu=True, scale=None):
    T = sum(lengths)
    a = make(T, hq, hv, dk, dv, channel, seed, rate)
    if not l2norm:  # keep beta |k|^2 below 2, where the rule contracts
        a = (a[0], (a[1].float() / math.sqrt(dk)).bfloat16(), *a[2:])
    n = len(lengths)
    S = torch.randn(n, hv, dv, dk, device="cuda", generator=torch.Generator(device="cuda").manual_seed(seed + 1))
    cu = torch.tensor([0] + list(lengths)).cumsum(0).int().cuda() if use_cu else None
    S0 = torch.zeros_like(S) if zero else S.clone()
    out = torch.full((T, hv, dv), float("nan"), dtype=torch.bfloat16, device="cuda")
    Sout = torch.full_like(S, float("nan"))
    dep.gated_delta_rule(*a, None if zero else S, Sout, cu_seqlens=cu, n_seq=n, l2norm=l2norm, out=out, scale=scale)
    torch.cuda.synchronize()
    if not zero:
        assert torch.equal(S, S0)
    want = definition(*a, S0, lengths, dk ** -0.5 if scale is None else scale, l2norm)
    close(out, Sout, *want, max(lengths), dk)


@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 64), (64, 128), (128, 64), (128, 16), (64, 48), (128, 256), (64, 208)])
@pytest.mark.parametrize("channel", [True, False])
@pytest.mark.parametrize("lengths", [(1,), (1, 1, 1), (2, 2), (17,), (64, 1, 0, 33)])
def test_matches_definition(dep, dk, dv, channel, lengths):
    run_case(dep, lengths, 2, 4, dk, dv, channel, seed=dk + dv + len(lengths))


@pytest.mark.parametrize("n", [1, 2, 3, 4, 5, 7, 8, 9, 15, 16, 17, 31, 32, 33, 47, 48, 49, 63, 64, 65, 96, 127, 128, 129, 200])
@pytest.mark.parametrize("channel", [True, False])
def test_every_length(dep, n, channel):
    run_case(dep, (n,), 1, 2, 128, 128, channel, seed=n)
    run_case(dep, (n, n + 1), 2, 2, 64, 64, channel, seed=n, zero=True)


@pytest.mark.parametrize("hq,hv", [(1, 1), (1, 5), (3, 3), (2, 8), (4, 4)])
def test_head_layouts(dep, hq, hv):
    run_case(dep, (3, 40), hq, hv, 128, 128, True, seed=hv)
    run_case(dep, (1, 1), hq, hv, 64, 128, False, seed=hv)


@pytest.mark.parametrize("channel", [True, False])
def test_equal_lengths_without_a_table(dep, channel):
    run_case(dep, (4, 4, 4), 2, 2, 128, 128, channel, use_cu=False)
    run_case(dep, (50, 50), 2, 2, 128, 128, channel, use_cu=False)
    run_case(dep, (70,), 2, 2, 128, 128, channel, use_cu=False, scale=0.3)


@pytest.mark.parametrize("n", [1, 5, 80])
def test_without_normalisation(dep, n):
    run_case(dep, (n, n), 2, 2, 128, 128, True, l2norm=False)
    run_case(dep, (n,), 2, 2, 64, 64, False, l2norm=False)


@pytest.mark.parametrize("rate", [0.0, 1e-3, 20.0, 300.0])
def test_decays_from_none_to_total(dep, rate):
    """Decays from 1 to below the smallest FP32 number within one token."""
    run_case(dep, (70,), 2, 2, 128, 128, True, rate=rate, seed=3)
    run_case(dep, (70,), 2, 2, 64, 64, False, rate=rate, seed=4)


@pytest.mark.parametrize("lengths", [(3,), (90, 20)])
@pytest.mark.parametrize("channel", [True, False])
def test_minus_infinity_empties_the_state(dep, lengths, channel):
    T, hq, hv, d = sum(lengths), 2, 2, 128
    a = make(T, hq, hv, d, d, channel, seed=6)
    a[3][T // 2] = -math.inf
    a[3][0, 0] = -math.inf
    S = torch.randn(len(lengths), hv, d, d, device="cuda")
    cu = torch.tensor([0] + list(lengths)).cumsum(0).int().cuda()
    want = definition(*a, S, lengths, d ** -0.5, True)
    out = dep.gated_delta_rule(*a, S, cu_seqlens=cu, l2norm=True)
    close(out, S, *want, max(lengths), d)


def test_writing_nothing_and_everything(dep):
    """beta = 0 leaves only the decay; beta = 1 with repeated keys overwrites what a key holds."""
    T, hv, d = 60, 2, 128
    q, k, v, g, beta = make(T, hv, hv, d, d, True, seed=7)
    beta[:30], beta[30:] = 0, 1
    k = k.clone()
    k[30:] = k[30:31]
    g[30:] = 0
    S = torch.randn(1, hv, d, d, device="cuda")
    want = definition(q, k, v, g, beta, S, (T,), d ** -0.5, True)
    out = dep.gated_delta_rule(q, k, v, g, beta, S, l2norm=True)
    close(out, S, *want, T, d)


@pytest.mark.parametrize("tokens", [1, 3, 40])
def test_slots_and_padding(dep, tokens):
    """States in places of a pool; sequences in no place give zeros and leave the pool alone."""
    hv, d, slots = 3, 64, [4, -1, 0, 7, 2]
    n, T = len(slots), len(slots) * tokens
    a = make(T, hv, hv, d, d, True, seed=8)
    S = torch.randn(6, hv, d, d, device="cuda")
    want = definition(*a, S, [tokens] * n, d ** -0.5, True, slots)
    out = torch.full((T, hv, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    before = S.clone()
    dep.gated_delta_rule(*a, S, n_seq=n, l2norm=True, out=out, slots=torch.tensor(slots, dtype=torch.int32, device="cuda"))
    close(out, S, *want, tokens, d)
    for i in (1, 3, 5):
        assert torch.equal(S[i], before[i])
    assert (out[tokens:2 * tokens] == 0).all() and (out[3 * tokens:4 * tokens] == 0).all()


def test_table_values_are_clipped_to_the_tensors(dep):
    """A table that runs past the tokens (or backwards) reads and writes nothing outside."""
    hv, d, T = 2, 64, 40
    a = make(T, hv, hv, d, d, False, seed=9)
    S = torch.randn(3, hv, d, d, device="cuda")
    before = S.clone()
    buf = torch.full((T + 20, hv, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    cu = torch.tensor([-5, 20, 10, 1000], dtype=torch.int32, device="cuda")
    dep.gated_delta_rule(*a, S, cu_seqlens=cu, l2norm=True, out=buf[:T])
    torch.cuda.synchronize()
    assert buf[T:].isnan().all() and torch.equal(S[1], before[1])
    want = definition(*(t[:20] for t in a), before[:1], (20,), d ** -0.5, True)
    assert (S[:1].double().cpu() - want[1]).norm() <= 1e-5 * want[1].norm()


def test_long_sequence_and_split_calls_agree(dep):
    """One call over a long sequence, and the same tokens in pieces that end inside a chunk."""
    T, hv, d = 1000, 2, 128
    a = make(T, hv, hv, d, d, True, seed=10, rate=0.05)
    S1 = torch.zeros(1, hv, d, d, device="cuda")
    S2 = S1.clone()
    o1 = dep.gated_delta_rule(*a, S1, l2norm=True)
    o2 = torch.empty_like(o1)
    cuts = [0, 1, 38, 39, 430, 999, 1000]
    for i, j in zip(cuts, cuts[1:]):
        dep.gated_delta_rule(*(t[i:j] for t in a), S2, l2norm=True, out=o2[i:j])
    want = definition(*a, torch.zeros(1, hv, d, d), (T,), d ** -0.5, True)
    close(o1, S1, *want, T, d)
    close(o2, S2, *want, T, d)


def test_more_tokens_and_states_than_32_bits_of_bytes(dep):
    """The last of so many states that their offset in elements passes 2^31."""
    hv, d = 16, 128
    n = (2 ** 31) // (hv * d * d) + 2
    S = torch.zeros(n, hv, d, d, device="cuda")
    S[-1] = torch.randn(hv, d, d, device="cuda")
    a = make(41, hv, hv, d, d, False, seed=12)
    slots = torch.tensor([n - 1, 0], dtype=torch.int32, device="cuda")
    first = S[-1:].clone()
    cu = torch.tensor([0, 1, 41], dtype=torch.int32, device="cuda")
    out = dep.gated_delta_rule(*a, S, cu_seqlens=cu, slots=slots, l2norm=True)
    both = torch.cat([S[-1:], S[:1]])
    want = definition(*a, torch.cat([first, torch.zeros_like(first)]), (1, 40), d ** -0.5, True)
    close(out, both, *want, 40, d)
    assert not S[1:-1].any()


@pytest.mark.parametrize("tokens", [1, 100])
def test_same_bits_again_in_a_graph_and_on_another_stream(dep, tokens):
    hv, d, n = 4, 128, 3
    a = make(n * tokens, hv, hv, d, d, True, seed=13)
    S = torch.randn(n, hv, d, d, device="cuda")
    So, out = torch.empty_like(S), torch.empty(n * tokens, hv, d, dtype=torch.bfloat16, device="cuda")
    call = lambda **k: dep.gated_delta_rule(*a, S, So, n_seq=n, l2norm=True, out=out, **k)  # noqa: E731
    call()
    want = out.clone(), So.clone()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    out.zero_(), So.zero_()
    side.wait_stream(torch.cuda.current_stream())
    call(stream=side)
    side.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(So, want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    out.zero_(), So.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(So, want[1])


@pytest.mark.parametrize("channel,dk", [(True, 128), (False, 64)])
def test_workspaces_of_any_size(dep, monkeypatch, channel, dk):
    """The same bits from one pass over all chunks and from many, down to one chunk a pass; token by
    token without a workspace."""
    lengths, hv = (40, 0, 17, 1, 90, 33), 4
    T, n = sum(lengths), len(lengths)
    a = make(T, 2, hv, dk, 128, channel, seed=11)
    S = torch.randn(n + 1, hv, 128, dk, device="cuda", generator=torch.Generator(device="cuda").manual_seed(12))
    cu = torch.tensor([0] + list(lengths)).cumsum(0).int().cuda()
    slots = torch.tensor([3, 0, 6, 9, 1, 2], dtype=torch.int32, device="cuda")  # sequence 3 is padding
    size = dep.dep_delta_workspace(dep.dep_delta_args_t(tokens=T, n_seq=n, Hv=hv, Dk=dk))
    chunk = size // (T // 16 + n)
    assert size == chunk * (T // 16 + n) > 0

    def run(size, in_place):
        monkeypatch.setattr(dep._binding, "dep_delta_workspace", lambda args: size)
        start, end = S.clone(), torch.full_like(S, 7.0)
        end = start if in_place else end
        out = dep.gated_delta_rule(*a, start, end, cu_seqlens=cu, slots=slots, l2norm=True)
        return out, end

    for in_place in (False, True):
        out, end = run(size, in_place)
        for part in (size - 16, 7 * chunk, 3 * chunk + 16, 2 * chunk, chunk):
            o, e = run(part, in_place)
            assert torch.equal(o, out) and torch.equal(e, end), part
    o, e = run(0, True)
    want = definition(*a, S, lengths, dk ** -0.5, True, slots.tolist())
    for got in ((out, end), (o, e)):
        close(*got, *want, max(lengths), dk)


def test_python_refusals(dep):
    a = make(4, 2, 2, 64, 64, False)
    S = torch.zeros(1, 2, 64, 64, device="cuda")
    ok = dict(state=S)
    for change in (dict(state=None), dict(state=S.double()), dict(state=S[:, :1]), dict(n_seq=3),
                   dict(cu_seqlens=torch.tensor([0, 4], device="cuda")), dict(slots=torch.zeros(2, dtype=torch.int32, device="cuda")),
                   dict(out=torch.zeros(4, 2, 64, device="cuda")), dict(state_out=torch.zeros(2, 2, 64, 64, device="cuda"))):
        with pytest.raises((ValueError, dep.DepError)):
            dep.gated_delta_rule(*a, **{**ok, **change})
    with pytest.raises(ValueError):
        dep.gated_delta_rule(a[0], a[1], a[2], a[3][:, :1], a[4], S)
    with pytest.raises(dep.DepError) as e:  # 16-byte loads
        dep.gated_delta_rule(a[0].contiguous().flatten()[4:388].view(3, 2, 64), a[1][:3], a[2][:3], a[3][:3], a[4][:3], S)
    assert e.value.status == dep.DEP_ERR_MISALIGNED
