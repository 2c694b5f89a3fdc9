"""The projection with 8-bit integers on both sides, against exact integer sums."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

pytestmark = pytest.mark.gpu


def make(B, N, K, seed=0, low=-128):
    rng = np.random.default_rng(seed)
    x = rng.integers(low, 128, (B, K), dtype=np.int64)
    w = rng.integers(low, 128, (N, K), dtype=np.int64)
    xs = rng.uniform(0.5, 2.0, B).astype(np.float32)
    ws = (rng.uniform(0.5, 2.0, N) / 1000).astype(np.float32)
    return x, w, xs, ws


def sums(x, w):
    """Exact integer sums (products of halves stay below 2^53 in float64)."""
    return x.astype(np.float64) @ w.astype(np.float64).T


def dev(a, dtype):
    return torch.from_numpy(np.ascontiguousarray(a)).to(dtype).cuda()


def check(y, x, w, xs, ws):
    """Three FP32 roundings (the sum, the scales' product, their product) and one to BF16."""
    want = sums(x, w) * xs[:, None].astype(np.float64) * ws.astype(np.float64)
    got = y.double().cpu().numpy()
    assert got.shape == want.shape
    bad = ~(np.abs(got - want) <= np.abs(want) * (2.0 ** -8 + 2.0 ** -21))
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist())


def run(dep, x, w, xs, ws, max_rows=None):
    p = dep.Int8Projection(dev(w, torch.int8), dev(ws, torch.float32), max_rows=max_rows or len(x))
    out = torch.full((len(x), len(w)), float("nan"), dtype=torch.bfloat16, device="cuda")
    try:
        p.run(dev(x, torch.int8), dev(xs, torch.float32), out=out)
        torch.cuda.synchronize()
        assert dep.dep_int8_device_status(p.plan) == 0
    finally:
        p.close()
    return out


@pytest.mark.parametrize("B", [1, 2, 3, 7, 8, 9, 16, 17, 32, 33, 64, 65, 100, 128, 129, 200, 256, 257, 300])
@pytest.mark.parametrize("N,K", [(333, 1008), (1000, 4096)])
def test_batches(dep, B, N, K):
    a = make(B, N, K, seed=B)
    check(run(dep, *a), *a)


@pytest.mark.parametrize("B", [66, 95, 96, 97, 130, 191, 192, 193])
@pytest.mark.parametrize("N,K", [(700, 2000), (2311, 7168), (20480, 1040)])
def test_widths_between_powers_of_two(dep, B, N, K):
    a = make(B, N, K, seed=B + 1)
    check(run(dep, *a), *a)


@pytest.mark.parametrize("most", [96, 130, 256])
def test_narrower_batches_of_one_plan(dep, most):
    """Every kernel that batches up to a plan's rows reach, in its workspace."""
    x, w, xs, ws = make(most, 1500, 4000, seed=most)
    p = dep.Int8Projection(dev(w, torch.int8), dev(ws, torch.float32), max_rows=most)
    for B in (most, 5, 20, 60, 90, 96, 1):
        out = p.run(dev(x[:B], torch.int8), dev(xs[:B], torch.float32))
        check(out, x[:B], w, xs[:B], ws)
    assert dep.dep_int8_device_status(p.plan) == 0
    p.close()


@pytest.mark.parametrize("N,K", [(1, 16), (1, 4096), (7, 32), (64, 48), (127, 64), (128, 80), (129, 128), (130, 1024),
                                 (255, 1040), (2311, 3056), (5, 20000), (20000, 64), (300, 131056)])
@pytest.mark.parametrize("B", [1, 5, 37])
def test_shapes(dep, N, K, B):
    a = make(B, N, K, seed=N + K)
    check(run(dep, *a), *a)


@pytest.mark.parametrize("B", [3, 16, 70, 150, 256])
def test_extreme_values_sum_exactly(dep, B):
    """Sums far past 2^24 that cancel to small numbers: exact only in integers."""
    N, K = 200, 8192
    x = np.full((B, K), -128, dtype=np.int64)
    w = np.full((N, K), -128, dtype=np.int64)
    w[:, K // 2:] = 127  # K/2 (16384 - 16256): cancels to 2^19
    w[np.arange(N), np.arange(N) * 7] += 1  # one step of 128 less in each row, at another place
    x[:, 0] = np.arange(B) % 127
    xs, ws = np.ones(B, np.float32), np.ones(N, np.float32)
    check(run(dep, x, w, xs, ws), x, w, xs, ws)
    w2 = np.full((N, K), -128, dtype=np.int64)  # 2^27: the largest sums
    check(run(dep, x, w2, xs, ws), x, w2, xs, ws)
    # 2048 products of 2^14, 4096 of -2^13 and a one: sums of 1, which 24 bits lose on the way
    w3 = np.zeros((N, K), dtype=np.int64)
    w3[:, :2048], w3[:, 2048:6144], w3[:, 7000] = -128, 64, 1
    x3 = np.full((B, K), -128, dtype=np.int64)
    x3[:, 6144:] = 0
    x3[:, 7000] = 1
    assert np.all(sums(x3, w3) == 1)
    check(run(dep, x3, w3, xs, ws), x3, w3, xs, ws)


def test_wider_batches_than_the_plan(dep):
    a = make(150, 300, 512, seed=3)
    check(run(dep, *a, max_rows=20), *a)


@pytest.mark.parametrize("N,K", [(14560, 7168), (7168, 12288)])
@pytest.mark.parametrize("B", [1, 16, 64, 256])
def test_layer_shapes(dep, N, K, B):
    g = torch.Generator(device="cuda").manual_seed(B)
    x = torch.randint(-128, 128, (B, K), generator=g, device="cuda", dtype=torch.int8)
    w = torch.randint(-128, 128, (N, K), generator=g, device="cuda", dtype=torch.int8)
    xs = torch.rand(B, generator=g, device="cuda") + 0.5
    ws = (torch.rand(N, generator=g, device="cuda") + 0.5) / 1000
    p = dep.Int8Projection(w, ws, max_rows=B)
    out = p.run(x, xs)
    want = (x.double() @ w.double().t()) * xs.double()[:, None] * ws.double()
    assert ((out.double() - want).abs() <= want.abs() * (2.0 ** -8 + 2.0 ** -21)).all()
    first = out.clone()
    for _ in range(5):  # the same bits from run to run
        assert torch.equal(p.run(x, xs, out=out), first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p.run(x, xs, out=out)
        p.run(x, xs, out=out)
    out.zero_()
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, first) and dep.dep_int8_device_status(p.plan) == 0
    assert dep.dep_int8_plan_workspace(p.plan) > 0


def test_one_plan_serves_smaller_batches_in_turn(dep):
    N, K = 1000, 2048
    x, w, xs, ws = make(256, N, K, seed=9)
    p = dep.Int8Projection(dev(w, torch.int8), dev(ws, torch.float32), max_rows=256)
    side = torch.cuda.Stream()
    for B in (256, 1, 40, 3, 129, 0, 17):
        xd, sd = dev(x[:B], torch.int8), dev(xs[:B], torch.float32)
        side.wait_stream(torch.cuda.current_stream())
        y = p.run(xd, sd, stream=side)
        side.synchronize()
        if B:
            check(y, x[:B], w, xs[:B], ws)


def test_special_scales(dep):
    x, w, xs, ws = make(4, 40, 256, seed=10)
    xs[1], xs[2], ws[3] = 0.0, np.inf, np.nan
    y = run(dep, x, w, xs, ws)
    assert y[:, 3].isnan().all() and (y[1, 4:] == 0).all() and not torch.isfinite(y[2]).any()
    assert torch.isfinite(y[0, 4:]).all()


def test_refusals(dep):
    x, w, xs, ws = make(4, 48, 64, seed=2)
    xd, wd, xsd, wsd = dev(x, torch.int8), dev(w, torch.int8), dev(xs, torch.float32), dev(ws, torch.float32)
    plan = dep.dep_int8_plan(48, 64, 4)
    buf = torch.zeros(4 * 48 + 8, dtype=torch.bfloat16, device="cuda")
    y = buf[: 4 * 48]
    try:
        def status(*a):
            with pytest.raises(dep.DepError) as e:
                dep.dep_int8_run(*a)
            return e.value.status
        assert status(plan, xd, xsd, wd, wsd, buf[1:], 4) == dep.DEP_ERR_MISALIGNED
        assert status(plan, xd, None, wd, wsd, y, 4) == dep.DEP_ERR_INVALID_ARG
        assert status(plan, xd, xsd, wd, wsd, y, -1) == dep.DEP_ERR_INVALID_ARG
        assert status(plan, xd, xsd, wd, wsd, wd, 4) == dep.DEP_ERR_INVALID_ARG
        dep.dep_int8_run(plan, xd, xsd, wd, wsd, y, 0)
    finally:
        dep.dep_int8_plan_destroy(plan)
    p = dep.Int8Projection(wd, wsd)
    for bad in (lambda: p.run(xd.float(), xsd), lambda: p.run(xd, xsd[:3]), lambda: p.run(xd[:, :32], xsd),
                lambda: p.run(xd, xsd, out=torch.zeros(4, 47, device="cuda", dtype=torch.bfloat16)),
                lambda: dep.Int8Projection(wd.t(), wsd), lambda: dep.Int8Projection(wd, wsd[:5])):
        with pytest.raises(ValueError):
            bad()
    p.close()
    p.close()
