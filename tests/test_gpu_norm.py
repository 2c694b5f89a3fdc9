"""RMS norm with the residual's addition and an 8-bit output, against its
definition in 64 bits: whole numbers and stored sums equal, the rest within the
roundings that the kernel makes."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

pytestmark = pytest.mark.gpu

EPS = 1e-6
# relative error of 1/rms: the longest chain of FP32 additions (64 of a thread, 5 + 32 of the block),
# then a division, a square root and a reciprocal, half a step (2^-24) each, halved by the root or not
RSTD = 2.0 ** -24 * (64 + 37 + 8)


def inputs(rows, cols, seed=0, residual=True):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(rows, cols, generator=g, device="cuda").bfloat16()
    r = (4 * torch.randn(rows, cols, generator=g, device="cuda")).bfloat16() if residual else None
    w = (1 + 0.2 * torch.randn(cols, generator=g, device="cuda")).bfloat16()
    return x, r, w


def reference(x, r, w, fmt, norm=True):
    """(values, scales, h): float64 on the host."""
    h = x if r is None else (x.float() + r.float()).bfloat16()
    hd = h.double().cpu().numpy()
    p = hd * (w.double().cpu().numpy() if w is not None else 1.0)
    rstd = 1.0 / np.sqrt((hd * hd).mean(1, keepdims=True) + EPS) if norm else np.ones((len(hd), 1))
    if fmt is None:
        return p * rstd, None, h
    if fmt == "int8":
        top = np.abs(p).max(1, keepdims=True)
        with np.errstate(invalid="ignore", divide="ignore"):
            q = np.where(top > 0, np.rint(127 * p / top), 0)
        return q, (top * rstd / 127)[:, 0], h
    rows, cols = p.shape
    pad = np.pad(p, ((0, 0), (0, -cols % 128))).reshape(rows, -1, 128)
    top = np.abs(pad).max(2, keepdims=True)
    with np.errstate(invalid="ignore", divide="ignore"):
        ratio = np.where(top > 0, 448 * pad / top, 0).reshape(rows, -1)[:, :cols]
    return e4m3(ratio), top[..., 0] * rstd / 448, h


def e4m3(v):
    """Nearest e4m3 value, ties to even, of doubles up to 448."""
    a = np.abs(v)
    e = np.floor(np.log2(np.maximum(a, 2.0 ** -9)))
    e = np.where(np.ldexp(1.0, e.astype(int)) > a, e - 1, e)
    step = np.ldexp(1.0, (np.maximum(e, -6) - 3).astype(int))
    return np.copysign(np.rint(a / step) * step, v)


def check(dep, x, r, w, fmt, norm=True, **kw):
    before = None if r is None else r.clone()
    want, scale, h = reference(x, r, w, fmt, norm)
    if norm:
        got = dep.add_rms_norm(x, w, r, eps=EPS, quant=fmt, **kw)
    else:
        got = dep.quantize_rows(x, quant=fmt, **kw)
    torch.cuda.synchronize()
    if r is not None:
        stored = kw.get("residual_out", r)
        assert torch.equal(stored.view(torch.int16), h.view(torch.int16))
        if "residual_out" in kw:
            assert torch.equal(r, before)
    if fmt is None:
        y = got.double().cpu().numpy()
        assert np.all(np.abs(y - want) <= np.abs(want) * (2.0 ** -8 * (1 + RSTD) + RSTD + 2.0 ** -23))
        return got
    q, s = got
    np.testing.assert_array_equal(q.float().cpu().numpy(), want.astype(np.float32))
    s = s.double().cpu().numpy()
    assert s.shape == scale.shape
    assert np.all(np.abs(s - scale) <= np.abs(scale) * (RSTD + 2.0 ** -22))
    return got


SHAPES = [(1, 7168), (3, 1), (2, 7), (5, 8), (4, 127), (9, 128), (1, 129), (7, 256), (17, 1000), (3, 1024), (2, 1032),
          (5, 4096), (3, 5001), (2, 8192), (2, 12288), (3, 12289), (2, 16392), (1, 65536), (33, 64)]


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("fmt", [None, "int8", "e4m3"])
def test_norm_matches_definition(dep, rows, cols, fmt):
    check(dep, *inputs(rows, cols, seed=cols), fmt)
    x, _, w = inputs(rows, cols, seed=cols + 1)
    check(dep, x, None, w, fmt)


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_quantize_matches_definition(dep, rows, cols, fmt):
    x, _, _ = inputs(rows, cols, seed=cols)
    check(dep, x, None, None, fmt, norm=False)


@pytest.mark.parametrize("fmt", [None, "int8", "e4m3"])
@pytest.mark.parametrize("offset,extra", [(0, 8), (1, 3), (8, 0), (3, 5), (0, 1)])
def test_strided_and_shifted_rows(dep, fmt, offset, extra):
    rows, cols = 6, 1048
    big = [torch.full((rows, cols + offset + extra), float("nan"), device="cuda").bfloat16() for _ in range(3)]
    x, r, w = inputs(rows, cols, seed=5)
    views = [b[:, offset:offset + cols] for b in big]
    views[0].copy_(x)
    views[1].copy_(r)
    check(dep, views[0], views[1], w, fmt, residual_out=views[2])
    for b in big:  # nothing outside the rows was written
        assert torch.isnan(b[:, :offset]).all() and torch.isnan(b[:, offset + cols:]).all()


@pytest.mark.parametrize("fmt", [None, "int8", "e4m3"])
@pytest.mark.parametrize("cols", [257, 1018, 1023, 2047, 2050, 8185, 8191, 16383, 16386, 65535])
def test_contiguous_rows_of_odd_length(dep, fmt, cols):
    """Every row starts at another place of a 16-byte granule."""
    check(dep, *inputs(9, cols, seed=cols), fmt)


@pytest.mark.parametrize("fmt", [None, "int8", "e4m3"])
def test_longest_rows_out_of_line(dep, fmt):
    x, r, w = inputs(3, 65536, seed=15)
    views = []
    for a, off in ((x, 7), (r, 7), (w.unsqueeze(0), 3)):
        b = torch.zeros(a.shape[0], 65536 + 9, device="cuda").bfloat16()
        b[:, off:off + 65536] = a
        views.append(b[:, off:off + 65536])
    check(dep, views[0], views[1], views[2][0], fmt, residual_out=torch.empty_like(x))


@pytest.mark.parametrize("fmt", [None, "int8", "e4m3"])
def test_output_rows_keep_their_surroundings(dep, fmt):
    rows, cols = 5, 333
    dt = {None: torch.bfloat16, "int8": torch.int8, "e4m3": torch.float8_e4m3fn}[fmt]
    raw = torch.full((rows, cols + 9), 0x55 if fmt else 0x5555, dtype=torch.uint8 if fmt else torch.int16, device="cuda")
    out = raw.view(dt)[:, 4:4 + cols]
    x, r, w = inputs(rows, cols, seed=6)
    check(dep, x, r, w, fmt, out=out)
    assert (raw[:, :4] == raw[0, 0]).all() and (raw[:, 4 + cols:] == raw[0, 0]).all()


def test_in_place_output(dep):
    x, r, w = inputs(40, 2048, seed=7)
    want = dep.add_rms_norm(x.clone(), w, r.clone())
    got = dep.add_rms_norm(x, w, r, out=x)
    assert got.data_ptr() == x.data_ptr() and torch.equal(got, want)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_ties_round_to_even(dep, fmt):
    """Small whole numbers over a largest value that makes many quotients exact ties."""
    g = torch.Generator(device="cuda").manual_seed(11)
    x = torch.randint(-254, 255, (64, 1536), generator=g, device="cuda").float().bfloat16()
    x[:, ::128] = 254.0
    check(dep, x, None, None, fmt, norm=False)
    w = torch.full((1536,), 0.5, device="cuda").bfloat16()
    check(dep, x, None, w, fmt)


@pytest.mark.parametrize("cols", [320, 321, 4096])
def test_wide_range_of_values(dep, cols):
    """Magnitudes over sixty powers of two, in x and in the weight."""
    g = torch.Generator(device="cuda").manual_seed(12)
    e = torch.randint(-30, 30, (16, cols), generator=g, device="cuda").float()
    x = (torch.randn(16, cols, generator=g, device="cuda") * torch.exp2(e)).bfloat16()
    w = torch.exp2(torch.randint(-8, 8, (cols,), generator=g, device="cuda").float()).bfloat16()
    for fmt in (None, "int8", "e4m3"):
        check(dep, x, None, w, fmt)


@pytest.mark.parametrize("fmt", [None, "int8", "e4m3"])
@pytest.mark.parametrize("cols", [200, 2000])
def test_empty_rows_and_special_values(dep, fmt, cols):
    x, _, w = inputs(6, cols, seed=13)
    x[1] = 0
    x[2] = 1e-36  # below the smallest quotient: stored as zeros
    x[3, 5] = float("inf")
    x[4, 7] = float("nan")
    clean = [0, 5]
    got = dep.add_rms_norm(x, w, None, eps=EPS, quant=fmt)
    alone = dep.add_rms_norm(x[clean].contiguous(), w, None, eps=EPS, quant=fmt)
    if fmt is None:
        assert torch.equal(got[clean], alone)
        assert (got[1] == 0).all() and (got[4].isnan()).all() and got[3, 5].isnan()
        return
    q, s = got
    assert torch.equal(q[clean].view(torch.uint8), alone[0].view(torch.uint8)) and torch.equal(s[clean], alone[1])
    for row in (1, 2):
        assert (q[row].float() == 0).all() and (s[row] == 0).all()
    bad = ~torch.isfinite(s.reshape(6, -1))
    assert not bad[clean].any() and not bad[1].any() and bad[3].any() and bad[4].any()


def test_same_bits_in_a_graph_and_on_another_stream(dep):
    x, r, w = inputs(65, 3000, seed=14)
    ro, out, sc = torch.empty_like(r), torch.empty(65, 3000, dtype=torch.int8, device="cuda"), torch.empty(65, device="cuda")
    call = lambda **k: dep.add_rms_norm(x, w, r, quant="int8", residual_out=ro, out=out, out_scale=sc, **k)  # noqa: E731
    call()
    want = out.clone(), sc.clone()
    torch.cuda.synchronize()
    out.zero_(), sc.zero_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    call(stream=side)
    side.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(sc, want[1])
    out.zero_(), sc.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(sc, want[1])


def test_python_refusals(dep):
    x, r, w = inputs(4, 64)
    for kw in (dict(quant="int4"), dict(residual_out=r), dict(out_scale=torch.zeros(4, device="cuda")),
               dict(out=torch.zeros(4, 63, device="cuda", dtype=torch.bfloat16)),
               dict(quant="e4m3", out_scale=torch.zeros(4, device="cuda")), dict(residual=r.float())):
        with pytest.raises(ValueError):
            dep.add_rms_norm(x, w, **kw)
    with pytest.raises(ValueError):
        dep.add_rms_norm(x.t(), None)
    with pytest.raises(ValueError):
        dep.add_rms_norm(x, w[:60])
    assert dep.add_rms_norm(x[:0], w).shape == (0, 64)
