"""The 8-bit integer projection's argument checks on batches whose sizes pass 32 bits."""
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B", [2 ** 29, 2 ** 30])
def test_overlap_is_refused_where_the_output_passes_32_bits(dep, B):
    """y [B, 1] of 2 GiB and more, inside x [B, 16]; nothing is launched."""
    x = torch.empty(B, 16, dtype=torch.int8, device="cuda")
    xs = torch.empty(B, device="cuda")
    w, ws = torch.zeros(1, 16, dtype=torch.int8, device="cuda"), torch.zeros(1, device="cuda")
    y = x.view(-1)[16 * B - 2 * B:].view(torch.bfloat16).view(B, 1)
    plan = dep.dep_int8_plan(1, 16, 256)
    try:
        with pytest.raises(dep.DepError) as e:
            dep.dep_int8_run(plan, x, xs, w, ws, y, B)
        assert e.value.status == dep.DEP_ERR_INVALID_ARG
    finally:
        dep.dep_int8_plan_destroy(plan)
