"""The norm and the 8-bit rows over all of BF16's range: values next to its largest,
whose products and squares pass FP32's, and the smallest."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

pytestmark = pytest.mark.gpu

LARGEST = float(torch.finfo(torch.bfloat16).max)


def e4m3(v):
    """Nearest e4m3 value, ties to even, of doubles up to 448."""
    a = np.abs(v)
    e = np.floor(np.log2(np.maximum(a, 2.0 ** -9)))
    e = np.where(np.ldexp(1.0, e.astype(int)) > a, e - 1, e)
    step = np.ldexp(1.0, (np.maximum(e, -6) - 3).astype(int))
    return np.copysign(np.rint(a / step) * step, v)


def quantised(p, fmt):
    """(q, P) of rows p in 64 bits; P for each row, or for each group of 128 columns."""
    rows, cols = p.shape
    if fmt == "int8":
        top = np.abs(p).max(1)
        return np.rint(127 * p / top[:, None]), top
    pad = np.pad(p, ((0, 0), (0, -cols % 128))).reshape(rows, -1, 128)
    top = np.abs(pad).max(2)
    return e4m3((448 * pad / top[..., None]).reshape(rows, -1)[:, :cols]), top


def rows_up_to(top, rows, cols, seed=0):
    """Normal rows whose largest value in every group of 128 columns is about `top`, with the fractions
    1, 1/2, -1/4, -1 of it at the start of each."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols, generator=g, dtype=torch.float64).clamp(-3, 3) * (top / 4)
    for c in range(0, cols, 128):
        n = min(4, cols - c)
        x[:, c:c + n] = torch.tensor([top, top / 2, -top / 4, -top], dtype=torch.float64)[:n]
    return x.clamp(-LARGEST, LARGEST).bfloat16()


TOPS = [2.0 ** -100, 1.1 * 2.0 ** -99, 2.0 ** -80, 1e30, 7e35, 9e35, 1e36, 2.6e36, 2.9e36, 1e37, 1e38, 1.7e38, LARGEST]


@pytest.mark.parametrize("top", TOPS)
@pytest.mark.parametrize("cols", [5, 128, 1000, 1024, 5001, 7168, 40000])
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_rows_up_to_the_largest_value(dep, fmt, cols, top):
    """The 8-bit values of the exact quotients; scales P / 127 and P / 448, one division in FP32
    (half a step of 2^-23, and one more for the constant's)."""
    x = rows_up_to(top, 3, cols, seed=cols)
    x[1] = (x[1].double() * (2.0 ** -90 if top > 1 else 2.0 ** 90)).bfloat16()  # an ordinary row beside them
    q, scale = dep.quantize_rows(x.cuda(), quant=fmt)
    want, P = quantised(x.double().numpy(), fmt)
    np.testing.assert_array_equal(q.float().cpu().numpy(), want.astype(np.float32))
    s, want_s = scale.double().cpu().numpy(), P / (127 if fmt == "int8" else 448)
    assert np.all(np.abs(s - want_s) <= 2.0 ** -23 * want_s)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_large_weights(dep, fmt):
    """p = h * weight beyond 2^121, from a weight of that size."""
    rows, cols = 3, 1160
    x = rows_up_to(3.0, rows, cols, seed=1)
    w = torch.full((cols,), 2.0 ** 124).bfloat16()
    q, _ = dep.add_rms_norm(x.cuda(), w.cuda(), quant=fmt)
    want, _ = quantised(x.double().numpy() * 2.0 ** 124, fmt)
    np.testing.assert_array_equal(q.float().cpu().numpy(), want.astype(np.float32))


def test_infinities_and_nans_show_in_the_scale(dep):
    x = rows_up_to(2.0, 4, 300, seed=2)
    x[1, 7], x[2, 9] = float("inf"), float("nan")
    x = x.cuda()
    for fmt in ("int8", "e4m3"):
        _, s = dep.quantize_rows(x, quant=fmt)
        s = s.view(4, -1).cpu()
        assert torch.isfinite(s[0]).all() and torch.isfinite(s[3]).all()
        assert not torch.isfinite(s[1, 0]) and torch.isnan(s[2, 0])


# relative error of 1/rms: the longest chain of FP32 additions (64 of a thread, 5 + 32 of the block), then a
# division, a square root and a reciprocal, half a step (2^-24) each
RSTD = 2.0 ** -24 * (64 + 37 + 8)


@pytest.mark.parametrize("size", [1e10, 1e19, 3e19, 1e25, 1e30, 1e37])
@pytest.mark.parametrize("cols", [8, 129, 1000, 1024, 5001, 7168, 16384, 40000])
@pytest.mark.parametrize("fmt", [None, "int8", "e4m3"])
def test_norm_of_rows_whose_squares_pass_fp32(dep, fmt, cols, size):
    """y = h / rms(h) * w is of ordinary size however large h is."""
    g = torch.Generator().manual_seed(cols)
    x = (torch.randn(3, cols, generator=g, dtype=torch.float64) * size).bfloat16()
    r = (torch.randn(3, cols, generator=g, dtype=torch.float64) * size).bfloat16()
    x[1], r[1] = torch.randn(cols, generator=g).bfloat16(), torch.randn(cols, generator=g).bfloat16()
    w = (1 + 0.2 * torch.randn(cols, generator=g)).bfloat16()
    h = (x.float() + r.float()).bfloat16()
    rd = r.cuda()
    got = dep.add_rms_norm(x.cuda(), w.cuda(), rd, quant=fmt)
    assert torch.equal(rd.cpu().view(torch.int16), h.view(torch.int16))
    hd = h.double().numpy()
    p, rstd = hd * w.double().numpy(), 1 / np.sqrt((hd * hd).mean(1, keepdims=True) + 1e-6)
    if fmt is None:
        y, want = got.double().cpu().numpy(), p * rstd
        assert np.all(np.abs(y - want) <= np.abs(want) * (2.0 ** -8 * (1 + RSTD) + RSTD + 2.0 ** -23))
        return
    q, s = got
    want, P = quantised(p, fmt)
    np.testing.assert_array_equal(q.float().cpu().numpy(), want.astype(np.float32))
    want_s = P * (rstd[:, 0] if fmt == "int8" else rstd) / (127 if fmt == "int8" else 448)
    s = s.double().cpu().numpy()
    assert np.all(np.abs(s - want_s) <= np.abs(want_s) * (RSTD + 2.0 ** -22))


@pytest.mark.parametrize("size", [1e-10, 1e-17, 1e-20, 1e-30, 1e-37])
@pytest.mark.parametrize("cols", [8, 1000, 5001, 7168, 40000])
def test_norm_of_tiny_rows_without_eps(dep, cols, size):
    g = torch.Generator().manual_seed(cols)
    x = (torch.randn(3, cols, generator=g, dtype=torch.float64) * size).bfloat16()
    x[1] = torch.randn(cols, generator=g).bfloat16()
    hd = x.double().numpy()
    y = dep.add_rms_norm(x.cuda(), eps=0.0).double().cpu().numpy()
    want = hd / np.sqrt((hd * hd).mean(1, keepdims=True))
    assert np.all(np.abs(y - want) <= np.abs(want) * (2.0 ** -8 * (1 + RSTD) + RSTD + 2.0 ** -23))


def test_an_infinity_in_a_norm(dep):
    """rms is infinite: zeros, and a NaN (infinity over infinity) where the infinity stood."""
    x = rows_up_to(2.0, 2, 300, seed=3)
    x[1, 7] = float("inf")
    y = dep.add_rms_norm(x.cuda()).cpu()
    assert torch.isfinite(y[0]).all() and torch.isnan(y[1, 7])
    y[1, 7] = 0
    assert not y[1].any()
