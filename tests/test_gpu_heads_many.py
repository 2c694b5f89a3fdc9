"""Norm and rotation with many tasks for each warp: through shared memory where that pays, in registers elsewhere."""
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from test_gpu_heads import NAN, rnd, rotate_case  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("T,hq,hk,d,rot,interleaved", [
    (2300, 96, 8, 128, 128, False), (6700, 64, 8, 64, 64, False), (7001, 61, 10, 64, 64, False), (2300, 97, 7, 128, 128, False),
    (2300, 96, 8, 128, 128, True), (2300, 96, 8, 128, 64, False), (2300, 96, 8, 96, 96, False), (1200, 96, 8, 256, 256, False),
    (2300, 96, 8, 128, 0, False), (9001, 20, 4, 64, 64, False),
])
def test_many_tasks(dep, T, hq, hk, d, rot, interleaved, norm):
    rotate_case(dep, T, hq, hk, d, rot, interleaved=interleaved, norm=norm, seed=T + d)


def test_many_tasks_in_place(dep):
    rotate_case(dep, 2300, 96, 8, 128, 128, in_place=True)
    rotate_case(dep, 7001, 61, 10, 64, 64, in_place=True)


@pytest.mark.parametrize("hq,hk,d,T", [(96, 8, 128, 2300), (64, 8, 64, 7000)])
def test_appending_gives_the_same_bits(dep, hq, hk, d, T):
    """With and without the values among a warp's tasks; some tokens are padding."""
    packed = rnd(T, T, (hq + 2 * hk) * d).bfloat16()
    q, k, v = (x.unflatten(1, (-1, d)) for x in packed.split([hq * d, hk * d, hk * d], 1))
    freqs, pos = dep.rotary_freqs(d)[0], torch.arange(T, device="cuda", dtype=torch.int32) * 7
    qw, kw = ((1 + 0.3 * rnd(i, d)).bfloat16() for i in (1, 2))
    want = dep.norm_rotate(q, k, pos, freqs, norm=True, q_weight=qw, k_weight=kw)
    pages = -(-T // 16) + 1
    slots = torch.randperm(pages * 16, device="cuda")[:T].int()
    slots[::50] = -1
    kc, vc = (torch.full((pages, 16, hk, d), NAN, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    got = dep.append_kv(k, v, kc, vc, slots, pos, freqs, norm=True, k_weight=kw, q=q, q_weight=qw)
    assert torch.equal(got, want[0])
    live = slots >= 0
    at = slots[live].long()
    assert torch.equal(kc.flatten(0, 1)[at], want[1][live]) and torch.equal(vc.flatten(0, 1)[at], v[live])
    left = torch.ones(pages * 16, dtype=torch.bool, device="cuda")
    left[at] = False
    assert kc.flatten(0, 1)[left].isnan().all() and vc.flatten(0, 1)[left].isnan().all()
