"""Attention's waits run out: the kernel returns, says so, and leaves nothing behind that a later call meets."""
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from test_gpu_attention import Case  # noqa: E402

pytestmark = pytest.mark.gpu

CASES = {
    "long": dict(seqs=[(1, 70001)], hq=12, hk=1, d=128, page=64),
    "long, 64 channels": dict(seqs=[(1, 150001)], hq=12, hk=1, d=64, page=64),
    "ragged": dict(seqs=[(1, 700 * i % 9000) for i in range(60)], hq=24, hk=2, d=128, page=16, gap=(3, 2)),
    "trees": dict(seqs=[(30, 9000), (30, 12000), (64, 0)], hq=24, hk=2, d=128, page=16, tree=True),
    "trees, 64 channels": dict(seqs=[(30, 20000), (30, 12000), (64, 0)], hq=24, hk=2, d=64, page=64, tree=True),
    "causal": dict(seqs=[(300, 500), (150, 3000)], hq=24, hk=2, d=64, page=24),
    "copies": dict(seqs=[(1, 40000), (5, 30000)], hq=8, hk=2, d=128, page=5),
}


def arguments(dep, c, status):
    """c's call, with a workspace of its own."""
    out, lse = torch.full((c.T, c.hq, c.d), 7.0, device="cuda", dtype=torch.bfloat16), torch.full((c.T, c.hq), 7.0, device="cuda")
    args = dep.dep_attention_args_t(
        q=c.q.data_ptr(), k_cache=c.k.data_ptr(), v_cache=c.v.data_ptr(), page_table=c.table.data_ptr(), kv_lens=c.kv.data_ptr(),
        cu_seqlens=c.cu.data_ptr(), tree=c.tree.data_ptr() if c.tree is not None else 0, o=out.data_ptr(), lse=lse.data_ptr(),
        q_stride=c.q.stride(0), o_stride=out.stride(0), k_page_stride=c.k.stride(0), k_slot_stride=c.k.stride(1),
        k_head_stride=c.k.stride(2), v_page_stride=c.v.stride(0), v_slot_stride=c.v.stride(1), v_head_stride=c.v.stride(2),
        table_stride=c.table.stride(0), tokens=c.T, n_pages=c.k.shape[0], n_seq=len(c.lens), Hq=c.hq, Hk=c.hk, D=c.d,
        page_size=c.page, table_width=c.table.shape[1], scale=c.scale, status=status.data_ptr())
    work = torch.zeros(dep.dep_attention_workspace(args), dtype=torch.uint8, device="cuda")
    args.workspace, args.workspace_bytes = work.data_ptr(), work.numel()
    return args, out, lse, work


@pytest.mark.parametrize("code", ["PRODUCER", "CONSUMER", "MMA", "EPILOGUE"])
@pytest.mark.parametrize("case", list(CASES))
def test_a_wait_that_runs_out(dep, case, code):
    c = Case(seed=2, **CASES[case])
    want = c.run(dep).clone()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    args, out, lse, work = arguments(dep, c, status)
    row = torch.zeros(c.T, dtype=torch.bool, device="cuda")  # of a sequence
    for f, n in zip(c.first, c.new):
        row[f: f + n] = True
    dep.dep_attention_selftest_timeout(args, getattr(dep, "DEP_DEV_TIMEOUT_" + code))
    torch.cuda.synchronize()
    if (case, code) == ("causal", "PRODUCER"):
        # 568 tiles and 176 units of the items' own, 744 on 152 SMs: five a block at most, and a ring holds five tiles of 64
        # channels, so no block ever waits for a slot
        assert status.item() == 0 and torch.equal(out, want)
    else:
        assert 1 <= status.item() <= 4
        # rows are complete or NaN, and some are; those of no sequence are left
        gone = out.isnan().all(-1) & lse.isnan()
        assert gone.any() and (out[~row] == 7).all() and (lse[~row] == 7).all()
        assert (gone[row] | ((out == want).all(-1) & (lse == c.lse))[row]).all()
    # the same arguments and workspace once more, without a wait that is held up
    status.zero_()
    dep.dep_paged_attention(args)
    torch.cuda.synchronize()
    assert status.item() == 0 and torch.equal(out[row], want[row]) and torch.equal(lse[row], c.lse[row])


def test_the_rows_tell_without_a_status_word(dep):
    c = Case([(1, 9000), (2, 300)], 12, 2, 128, 16)
    args, out, lse, work = arguments(dep, c, torch.zeros(1, dtype=torch.int32, device="cuda"))
    args.status = None
    dep.dep_attention_selftest_timeout(args, dep.DEP_DEV_TIMEOUT_EPILOGUE)
    torch.cuda.synchronize()
    assert out.isnan().all() and lse.isnan().all()


def test_a_wait_that_is_not_needed(dep):
    """Calls of one tile never wait for a free slot: they end as ever."""
    c = Case([(1, 100), (1, 20)], 4, 2, 128, 16)
    want = c.run(dep).clone()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    args, out, lse, work = arguments(dep, c, status)
    dep.dep_attention_selftest_timeout(args, dep.DEP_DEV_TIMEOUT_PRODUCER)
    torch.cuda.synchronize()
    assert status.item() == 0 and torch.equal(out, want) and torch.equal(lse, c.lse)
