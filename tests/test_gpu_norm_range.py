"""The norm and the 8-bit rows over all of BF16's range."""
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
