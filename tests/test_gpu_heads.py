"""Norm and rotation of heads, and appending to a paged cache, against the definition in 64 bits."""
import math

import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

pytestmark = pytest.mark.gpu
NAN = float("nan")


def rnd(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")


def definition(x, positions, freqs, interleaved, amplitude, norm, weight, eps, first):
    """(y, the size that FP32's errors are relative to) of [T, heads, D] in float64."""
    x = x.double()
    if norm:
        x = x / (x.pow(2).mean(-1, keepdim=True) + eps).sqrt()
        if weight is not None:
            x = x * weight.double()
    y, size = x.clone(), x.abs()
    if freqs is not None:
        r = freqs.numel()
        i = torch.arange(r, device=x.device)
        a, b = (first + 2 * i, first + 2 * i + 1) if interleaved else (first + i, first + r + i)
        u = positions.double()[:, None, None] * freqs
        y[..., a] = amplitude * (x[..., a] * u.cos() - x[..., b] * u.sin())
        y[..., b] = amplitude * (x[..., b] * u.cos() + x[..., a] * u.sin())
        size = size.clone()
        size[..., a] = size[..., b] = abs(amplitude) * torch.hypot(x[..., a], x[..., b])
    return y, size


def close(got, want, size):
    """The rounding to BF16 (half a step, 2^-8 of the value) and FP32's errors: the sum of squares and
    about sixteen roundings of at most 2^-23 of the pair's size each, the angle's 2^-23."""
    d = (got.double() - want).abs()
    bad = ~(d <= 2.0 ** -8 * want.abs() + 2.0 ** -18 * size + 2.0 ** -133)
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:3].tolist(), float(d.max()))


def rotate_case(dep, T, hq, hk, d, rot, first=0, interleaved=False, norm=True, weights=True, amplitude=1.0, eps=1e-6,
                in_place=False, seed=0, base=1e4, top=1 << 20):
    packed = rnd(seed, T, (hq + 2 * hk) * d + 8).bfloat16()
    q, k = packed[:, : hq * d].unflatten(1, (hq, d)), packed[:, hq * d: (hq + hk) * d].unflatten(1, (hk, d))
    qw, kw = ((1 + 0.3 * rnd(seed + i, d)).bfloat16() if norm and weights else None for i in (1, 2))
    freqs = dep.rotary_freqs(rot, base)[0] if rot else None
    pos = torch.randint(-top // 8, top, (T,), device="cuda", dtype=torch.int32) if rot else None
    want = [definition(x, pos, freqs, interleaved, amplitude, norm, w, eps, first) for x, w in ((q, qw), (k, kw))]
    rest = packed[:, (hq + hk) * d:].clone()
    kw_ = dict(interleaved=interleaved, amplitude=amplitude, norm=norm, q_weight=qw, k_weight=kw, eps=eps, first=first)
    if in_place:
        got = dep.norm_rotate(q, k, pos, freqs, q_out=q, k_out=k, **kw_)
    else:
        before = packed.clone()
        out = torch.full((T, (hq + hk) * d + 16), NAN, device="cuda", dtype=torch.bfloat16)
        qo, ko = out[:, : hq * d].unflatten(1, (hq, d)), out[:, hq * d: (hq + hk) * d].unflatten(1, (hk, d))
        got = dep.norm_rotate(q, k, pos, freqs, q_out=qo, k_out=ko, **kw_)
        assert torch.equal(packed, before) and out[:, (hq + hk) * d:].isnan().all()
    assert torch.equal(packed[:, (hq + hk) * d:], rest)
    for g, w in zip(got, want):
        close(g, *w)


@pytest.mark.parametrize("d,rot,first", [(128, 128, 0), (64, 64, 0), (80, 32, 0), (96, 96, 0), (256, 256, 0), (128, 64, 64),
                                         (72, 40, 16), (8, 8, 0), (248, 8, 240), (128, 0, 0), (16, 8, 8), (192, 64, 128)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [False, True])
def test_matches_definition(dep, d, rot, first, interleaved, norm):
    rotate_case(dep, 37, 6, 2, d, rot, first, interleaved, norm, seed=d + rot)


@pytest.mark.parametrize("T,hq,hk", [(1, 1, 1), (1, 96, 8), (2, 33, 1), (300, 14, 14), (5000, 3, 1), (4097, 96, 8)])
def test_sizes(dep, T, hq, hk):
    rotate_case(dep, T, hq, hk, 128, 128, seed=T)


@pytest.mark.parametrize("interleaved", [False, True])
def test_in_place(dep, interleaved):
    rotate_case(dep, 129, 12, 4, 128, 96, 16, interleaved, in_place=True, weights=False, amplitude=1.25)


def test_q_alone_and_new_outputs(dep):
    q = rnd(1, 5, 3, 64).bfloat16()
    pos, freqs = torch.arange(5, device="cuda", dtype=torch.int32), dep.rotary_freqs(64)[0]
    close(dep.norm_rotate(q, None, pos, freqs), *definition(q, pos, freqs, False, 1.0, False, None, 0, 0))
    empty = dep.norm_rotate(q[:0], q[:0], pos[:0], freqs)
    assert empty[0].shape == (0, 3, 64) and empty[1].shape == (0, 3, 64)


def test_far_positions(dep):
    """Angles at the ends of the positions' range: 64-bit fractions of a turn against exact integers."""
    freqs = dep.rotary_freqs(64, 5e5)[0]
    pos = torch.tensor([2 ** 31 - 1, -(2 ** 31), 2 ** 30 + 12345, 0, -1], dtype=torch.int32, device="cuda")
    q = torch.zeros(5, 1, 64, device="cuda", dtype=torch.bfloat16)
    q[..., :32] = 1
    got = dep.norm_rotate(q, None, pos, freqs)
    from fractions import Fraction
    pi = Fraction(3141592653589793238462643383279502884197169399375105820974944592307816406286, 10 ** 75)
    for t in range(5):
        for i in range(32):
            u = Fraction(int(pos[t])) * Fraction(float(freqs[i])) / (2 * pi) % 1
            want = torch.tensor([math.cos(2 * math.pi * float(u)), math.sin(2 * math.pi * float(u))])
            d = (got[t, 0, [i, i + 32]].cpu().double() - want).abs()
            # 2^-53 of f / 2 pi (below 1/6) times 2^31 positions: 2^-24 of a turn; then as in close()
            assert (d <= 2.0 ** -8 * want.abs() + 2.0 ** -18 + 2 * math.pi * 2.0 ** -24).all(), (t, i, d)


@pytest.mark.parametrize("exponent", [126, 100, 60, 57, 0, -40, -60, -100, -126, -133])
@pytest.mark.parametrize("eps", [1e-6, 0.0])
def test_norm_over_the_range(dep, exponent, eps):
    """Heads whose squares leave FP32's range, beside ordinary ones."""
    q = rnd(3, 9, 5, 128).bfloat16()
    if exponent < -120:
        q = torch.where(q.abs() < 0.5, 1.0, q.sign()).bfloat16()
    q[1::2] = torch.ldexp(q[1::2].double(), torch.tensor(exponent, device="cuda")).clamp(-3.38e38, 3.38e38).bfloat16()
    if eps == 0.0:
        assert q.abs().amax(-1).gt(0).all()
    w = (1 + 0.3 * rnd(4, 128)).bfloat16()
    got = dep.norm_rotate(q, None, None, None, norm=True, q_weight=w, eps=eps)
    close(got, *definition(q, None, None, False, 1.0, True, w, eps, 0))


def test_infinities_and_nan_stay_in_their_head(dep):
    q = rnd(5, 4, 6, 64).bfloat16()
    clean = dep.norm_rotate(q, None, None, None, norm=True)
    q[1, 2, 5], q[2, 3, 63] = math.inf, NAN
    got = dep.norm_rotate(q, None, None, None, norm=True)
    touched = torch.zeros(4, 6, dtype=torch.bool, device="cuda")
    touched[1, 2] = touched[2, 3] = True
    assert torch.equal(got[~touched], clean[~touched]) and got[1, 2, 5].isnan() and got[2, 3].isnan().all()
    assert (got[1, 2, :5] == 0).all()


def test_rotary_freqs(dep):
    f, a = dep.rotary_freqs(128, 10000.0, device="cpu")
    assert a == 1.0 and f.dtype == torch.float64 and f[0] == 1.0 and abs(float(f[-1]) - 10000 ** (-126 / 128)) < 1e-15
    g, a = dep.rotary_freqs(128, 10000.0, factor=8, device="cpu")
    assert a == 1.0 and torch.equal(g, f / 8)
    g, a = dep.rotary_freqs(128, 10000.0, factor=8, original=4096, device="cpu")
    assert abs(a - (0.1 * math.log(8) + 1)) < 1e-15
    turns = 4096 * f / (2 * math.pi)
    assert torch.equal(g[turns > 40], f[turns > 40]) and torch.equal(g[turns < 0.8], f[turns < 0.8] / 8)
    assert (g <= f).all() and (g >= f / 8).all()
    for bad in (dict(rot=7), dict(rot=64, base=1.0), dict(rot=64, factor=0.5), dict(rot=64, original=0),
                dict(rot=64, fast=1.0, slow=2.0)):
        with pytest.raises(ValueError):
            dep.rotary_freqs(**bad)


# ---- the cache -------------------------------------------------------------------------------

def cache(pages, page, heads, d, layout, seed=0):
    """k and v: apart by token or by head, two halves of one tensor, or the two interleaved row by row."""
    if layout == "token":
        return tuple(rnd(seed + i, pages, page, heads, d).bfloat16() for i in (0, 1))
    if layout == "head":
        return tuple(rnd(seed + i, pages, heads, page, d).bfloat16().transpose(1, 2) for i in (0, 1))
    if layout == "paired":
        both = rnd(seed, pages, 2, page, heads, d).bfloat16()
        return both[:, 0], both[:, 1]
    both = rnd(seed, pages, page, heads, 2 * d).bfloat16()
    return both[..., :d], both[..., d:]


def append_case(dep, T, hq, hk, d, page, layout, rot=None, norm=True, interleaved=False, first=0, seed=0, pages=None):
    pages = -(-T // page) + 2 if pages is None else pages
    packed = rnd(seed, T, (hq + 2 * hk) * d).bfloat16()
    q, k, v = packed.split([hq * d, hk * d, hk * d], 1)
    q, k, v = q.unflatten(1, (hq, d)) if hq else None, k.unflatten(1, (hk, d)), v.unflatten(1, (hk, d))
    kc, vc = cache(pages, page, hk, d, layout, seed + 10)
    slots = torch.randperm(pages * page, device="cuda")[:T].int()
    slots[::7] = -1
    if T > 3:
        slots[3] = pages * page
    rot = d if rot is None else rot
    freqs, amplitude = dep.rotary_freqs(rot, 1e4, factor=4, original=64) if rot else (None, 1.0)
    pos = torch.randint(0, 1 << 20, (T,), device="cuda", dtype=torch.int32) if rot else None
    qw, kw = ((1 + 0.3 * rnd(seed + i, d)).bfloat16() if norm else None for i in (1, 2))
    want_k, want_v, size = kc.double(), vc.double(), kc.double().abs()
    y, s = definition(k, pos, freqs, interleaved, amplitude, norm, kw, 1e-5, first)
    live = [t for t, i in enumerate(slots.tolist()) if 0 <= i < pages * page]
    at = slots[live].long()
    want_k[at // page, at % page], want_v[at // page, at % page], size[at // page, at % page] = y[live], v[live].double(), s[live]
    got = dep.append_kv(k, v, kc, vc, slots, pos, freqs, interleaved=interleaved, amplitude=amplitude, norm=norm,
                        k_weight=kw, eps=1e-5, first=first, q=q, q_weight=qw if hq else None)
    close(kc, want_k, size)
    assert torch.equal(vc.double(), want_v)
    untouched = torch.ones(pages, page, dtype=torch.bool, device="cuda")
    untouched[at // page, at % page] = False
    assert torch.equal(kc.double()[untouched], want_k[untouched])
    if hq:
        close(got, *definition(q, pos, freqs, interleaved, amplitude, norm, qw, 1e-5, first))
    else:
        assert got is None


@pytest.mark.parametrize("layout", ["token", "head", "paired", "rows"])
@pytest.mark.parametrize("T,page", [(1, 1), (5, 16), (64, 24), (777, 5), (1500, 64)])
@pytest.mark.parametrize("hq", [0, 6])
def test_append(dep, layout, T, page, hq):
    append_case(dep, T, hq, 2, 128, page, layout, seed=T)


@pytest.mark.parametrize("d,rot,first,interleaved,norm", [(64, 64, 0, True, True), (80, 32, 8, False, False), (256, 128, 0, False, True),
                                                         (128, 0, 0, False, False), (64, 0, 0, False, True)])
def test_append_forms(dep, d, rot, first, interleaved, norm):
    append_case(dep, 100, 4, 4, d, 16, "token", rot, norm, interleaved, first)


def test_append_all_padding(dep):
    k, v, q = rnd(1, 4, 2, 64).bfloat16(), rnd(2, 4, 2, 64).bfloat16(), rnd(3, 4, 2, 64).bfloat16()
    kc, vc = cache(3, 8, 2, 64, "token")
    before = kc.clone(), vc.clone()
    slots = torch.tensor([-1, 24, -(2 ** 31), 2 ** 31 - 1], device="cuda", dtype=torch.int32)
    got = dep.append_kv(k, v, kc, vc, slots, q=q, norm=True)
    assert torch.equal(kc, before[0]) and torch.equal(vc, before[1])
    close(got, *definition(q, None, None, False, 1.0, True, None, 1e-6, 0))
    # a cache of no pages
    got = dep.append_kv(k, v, kc[:0], vc[:0], slots, q=q, norm=True)
    close(got, *definition(q, None, None, False, 1.0, True, None, 1e-6, 0))
    assert dep.append_kv(k, v, kc[:0], vc[:0], slots) is None
    assert dep.append_kv(k[:0], v[:0], kc, vc, slots[:0]) is None and torch.equal(kc, before[0])


def test_append_past_32_bits(dep):
    """A cache of more than 2^32 bytes and 2^31 elements."""
    pages, page, hk, d = 33000, 64, 8, 128
    kc = torch.empty(pages, page, hk, d, device="cuda", dtype=torch.bfloat16)
    vc = torch.empty_like(kc)
    k, v = rnd(1, 3, hk, d).bfloat16(), rnd(2, 3, hk, d).bfloat16()
    slots = torch.tensor([pages * page - 1, 32767 * 64 + 63, 32768 * 64], device="cuda", dtype=torch.int32)
    dep.append_kv(k, v, kc, vc, slots)
    for t, i in enumerate(slots.tolist()):
        assert torch.equal(kc[i // page, i % page], k[t]) and torch.equal(vc[i // page, i % page], v[t])


def test_streams_and_graphs(dep):
    q, k, v = (rnd(i, 50, 4, 128).bfloat16() for i in range(3))
    kc, vc = cache(4, 16, 4, 128, "token")
    slots = torch.randperm(64, device="cuda")[:50].int()
    pos, freqs = torch.arange(50, device="cuda", dtype=torch.int32), dep.rotary_freqs(128)[0]
    want_q, want_k = dep.norm_rotate(q, k, pos, freqs, norm=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = dep.append_kv(k, v, kc, vc, slots, pos, freqs, norm=True, q=q, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want_q) and torch.equal(kc.view(64, 4, 128)[slots.long()], want_k)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = dep.append_kv(k, v, kc, vc, slots, pos, freqs, norm=True, q=q)
        rot = dep.norm_rotate(q, k, pos, freqs)
    kc.zero_()
    q.copy_(k)
    slots.copy_(slots.flip(0))
    pos.add_(7)
    graph.replay()
    assert torch.equal(out, dep.norm_rotate(q, None, pos, freqs, norm=True))
    assert torch.equal(kc.view(64, 4, 128)[slots.long()], dep.norm_rotate(k, None, pos, freqs, norm=True))
    assert torch.equal(rot[0], dep.norm_rotate(q, None, pos, freqs))
