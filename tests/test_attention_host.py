"""Refusals of the attention core's operators: host checks, no GPU.

Every call here is refused before anything is launched, so made-up addresses of
the right alignment stand for device memory."""
import ctypes

import pytest

A = 1 << 20  # an address; tensors below are placed megabytes apart
INF = float("inf")


def heads_args(dep, append=False, **kw):
    base = dict(q=A, k=2 * A, q_weight=4 * A, k_weight=5 * A, freqs=6 * A, positions=7 * A, q_out=8 * A, q_stride=256,
                k_stride=128, q_out_stride=256, tokens=5, Hq=4, Hk=2, D=64, rot=64, first=0, flags=2, eps=1e-6,
                amplitude=1.0, page_size=16)
    if append:
        base.update(v=3 * A, v_stride=128, slots=9 * A, k_cache=16 * A, v_cache=32 * A, n_pages=8, k_page_stride=2048,
                    k_slot_stride=128, k_head_stride=64, v_page_stride=2048, v_slot_stride=128, v_head_stride=64)
    else:
        base.update(k_out=10 * A, k_out_stride=128)
    base.update(kw)
    return dep.dep_heads_args_t(**base)


BOTH = [
    (dict(tokens=-1), "INVALID_ARG"), (dict(Hq=-1), "INVALID_ARG"), (dict(Hk=-1), "INVALID_ARG"), (dict(D=0), "INVALID_ARG"),
    (dict(rot=-8), "INVALID_ARG"), (dict(first=-8), "INVALID_ARG"), (dict(first=8), "INVALID_ARG"),  # past the head's end
    (dict(flags=4), "INVALID_ARG"), (dict(eps=-1.0), "INVALID_ARG"), (dict(eps=float("nan")), "INVALID_ARG"),
    (dict(eps=INF), "INVALID_ARG"), (dict(amplitude=INF), "INVALID_ARG"), (dict(flags=0), "INVALID_ARG"),  # weights, no norm
    (dict(q=None), "INVALID_ARG"), (dict(q_out=None), "INVALID_ARG"), (dict(k=None), "INVALID_ARG"),
    (dict(freqs=None), "INVALID_ARG"), (dict(positions=None), "INVALID_ARG"),
    (dict(q_stride=248), "INVALID_ARG"), (dict(k_stride=120), "INVALID_ARG"), (dict(q_out_stride=8), "INVALID_ARG"),
    (dict(D=68, rot=0), "UNSUPPORTED"), (dict(rot=20), "UNSUPPORTED"), (dict(rot=32, first=4), "UNSUPPORTED"),
    (dict(D=264, q_stride=2048, q_out_stride=2048, k_stride=2048), "UNSUPPORTED"),
    (dict(Hq=1 << 26, q_stride=1 << 40, q_out_stride=1 << 40), "UNSUPPORTED"),
    (dict(q=A + 8), "MISALIGNED"), (dict(k_stride=132), "MISALIGNED"), (dict(q_weight=4 * A + 8), "MISALIGNED"),
    (dict(freqs=6 * A + 4), "MISALIGNED"), (dict(positions=7 * A + 2), "MISALIGNED"), (dict(q_out=8 * A + 2), "MISALIGNED"),
    (dict(q_out=A + 128), "INVALID_ARG"),                     # q's own rows, shifted
    (dict(q_out=A, q_out_stride=264), "INVALID_ARG"),         # spaced otherwise
    (dict(q_out=2 * A), "INVALID_ARG"), (dict(q_out=4 * A), "INVALID_ARG"), (dict(q_out=6 * A), "INVALID_ARG"),
    (dict(q_out=7 * A), "INVALID_ARG"),
]


@pytest.mark.parametrize("append", [False, True])
@pytest.mark.parametrize("change,status", BOTH)
def test_heads_refusals(dep, append, change, status):
    call = dep.dep_append_kv if append else dep.dep_norm_rotate
    if append and change == dict(D=264, q_stride=2048, q_out_stride=2048, k_stride=2048):
        change = dict(change, v_stride=2048)
    with pytest.raises(dep.DepError) as e:
        call(heads_args(dep, append, **change), 0)
    assert e.value.status == getattr(dep, "DEP_ERR_" + status)


@pytest.mark.parametrize("change,status", [
    (dict(Hq=0, q=None, q_out=None), "INVALID_ARG"), (dict(k_out=None), "INVALID_ARG"), (dict(Hk=0), "INVALID_ARG"),
    (dict(v=3 * A), "INVALID_ARG"), (dict(slots=3 * A), "INVALID_ARG"), (dict(k_cache=3 * A), "INVALID_ARG"),
    (dict(k_out_stride=64), "INVALID_ARG"), (dict(k_out=10 * A + 8), "MISALIGNED"), (dict(k_out=8 * A), "INVALID_ARG"),
    (dict(k_out=A), "INVALID_ARG"), (dict(k_out=2 * A, k_out_stride=136), "INVALID_ARG"),
])
def test_rotate_refusals(dep, change, status):
    with pytest.raises(dep.DepError) as e:
        dep.dep_norm_rotate(heads_args(dep, **change), 0)
    assert e.value.status == getattr(dep, "DEP_ERR_" + status)


@pytest.mark.parametrize("change,status", [
    (dict(Hk=0), "INVALID_ARG"), (dict(v=None), "INVALID_ARG"), (dict(slots=None), "INVALID_ARG"),
    (dict(k_cache=None), "INVALID_ARG"), (dict(v_cache=None), "INVALID_ARG"), (dict(n_pages=-1), "INVALID_ARG"),
    (dict(page_size=0), "INVALID_ARG"), (dict(k_out=10 * A), "INVALID_ARG"), (dict(v_stride=64), "INVALID_ARG"),
    (dict(Hq=0), "INVALID_ARG"), (dict(n_pages=1 << 40), "UNSUPPORTED"),
    (dict(slots=9 * A + 2), "MISALIGNED"), (dict(v_cache=32 * A + 8), "MISALIGNED"), (dict(k_slot_stride=132), "MISALIGNED"),
    (dict(k_head_stride=-64), "INVALID_ARG"),
    (dict(k_slot_stride=0), "INVALID_ARG"), (dict(k_page_stride=1024), "INVALID_ARG"),  # rows that share bytes
    (dict(v_head_stride=56), "INVALID_ARG"),
    (dict(v_cache=16 * A), "INVALID_ARG"), (dict(v_cache=16 * A + 256), "INVALID_ARG"),  # the same cache, and one slot on
    (dict(k_cache=2 * A), "INVALID_ARG"), (dict(v_cache=3 * A), "INVALID_ARG"), (dict(k_cache=A - 4096), "INVALID_ARG"),
    (dict(k_cache=9 * A), "INVALID_ARG"), (dict(v_cache=8 * A), "INVALID_ARG"),
])
def test_append_refusals(dep, change, status):
    with pytest.raises(dep.DepError) as e:
        dep.dep_append_kv(heads_args(dep, True, **change), 0)
    assert e.value.status == getattr(dep, "DEP_ERR_" + status)


def test_heads_nothing_to_do(dep):
    dep.dep_norm_rotate(heads_args(dep, tokens=0), 0)
    dep.dep_append_kv(heads_args(dep, True, tokens=0), 0)
    dep.dep_append_kv(heads_args(dep, True, Hq=0, q=None, q_out=None, q_weight=None, n_pages=0, k_cache=None, v_cache=None), 0)
    assert dep.lib().dep_norm_rotate(None, None) == dep.lib().dep_append_kv(None, None) == dep.DEP_ERR_INVALID_ARG


def attention_args(dep, **kw):
    base = dict(q=A, k_cache=16 * A, v_cache=32 * A, page_table=3 * A, kv_lens=4 * A, cu_seqlens=5 * A, tree=6 * A,
                o=7 * A, lse=8 * A, q_stride=256, o_stride=256, k_page_stride=2048, k_slot_stride=128, k_head_stride=64,
                v_page_stride=2048, v_slot_stride=128, v_head_stride=64, table_stride=4, tokens=6, n_pages=8, n_seq=3, Hq=4,
                Hk=2, D=64, page_size=16, table_width=4, scale=0.125)
    base.update(kw)
    args = dep.dep_attention_args_t(**base)
    if "workspace" not in kw and "workspace_bytes" not in kw and args.Hq > 0 and args.Hk > 0 and args.n_seq >= 0 and args.tokens >= 0:
        args.workspace, args.workspace_bytes = 64 * A, dep.dep_attention_workspace(args)
    return args


@pytest.mark.parametrize("change,status", [
    (dict(tokens=-1), "INVALID_ARG"), (dict(n_seq=-1), "INVALID_ARG"), (dict(Hq=0), "INVALID_ARG"), (dict(Hk=0), "INVALID_ARG"),
    (dict(Hq=3), "INVALID_ARG"), (dict(page_size=0), "INVALID_ARG"), (dict(table_width=-1), "INVALID_ARG"),
    (dict(n_pages=-1), "INVALID_ARG"), (dict(scale=-1.0), "INVALID_ARG"), (dict(scale=INF), "INVALID_ARG"),
    (dict(scale=float("nan")), "INVALID_ARG"), (dict(scale=3e38), "INVALID_ARG"), (dict(n_seq=0), "INVALID_ARG"), (dict(tokens=7, cu_seqlens=None), "INVALID_ARG"),
    (dict(D=96, q_stride=512, o_stride=512), "UNSUPPORTED"), (dict(D=256, q_stride=1024, o_stride=1024), "UNSUPPORTED"),
    (dict(table_width=1 << 30, table_stride=1 << 30), "UNSUPPORTED"), (dict(n_pages=1 << 40), "UNSUPPORTED"),
    (dict(q=None), "INVALID_ARG"), (dict(o=None), "INVALID_ARG"), (dict(kv_lens=None), "INVALID_ARG"),
    (dict(page_table=None), "INVALID_ARG"), (dict(k_cache=None), "INVALID_ARG"), (dict(v_cache=None), "INVALID_ARG"),
    (dict(q_stride=248), "INVALID_ARG"), (dict(o_stride=248), "INVALID_ARG"), (dict(table_stride=3), "INVALID_ARG"),
    (dict(k_page_stride=-2048), "INVALID_ARG"),
    (dict(q=A + 8), "MISALIGNED"), (dict(o_stride=260), "MISALIGNED"), (dict(v_head_stride=68), "MISALIGNED"),
    (dict(tree=6 * A + 4), "MISALIGNED"), (dict(lse=8 * A + 2), "MISALIGNED"), (dict(kv_lens=4 * A + 2), "MISALIGNED"),
    (dict(cu_seqlens=5 * A + 1), "MISALIGNED"), (dict(page_table=3 * A + 2), "MISALIGNED"),
    (dict(o=A), "INVALID_ARG"), (dict(o=16 * A + 2048), "INVALID_ARG"), (dict(o=32 * A), "INVALID_ARG"),
    (dict(lse=7 * A + 64), "INVALID_ARG"), (dict(lse=3 * A), "INVALID_ARG"), (dict(lse=6 * A), "INVALID_ARG"),
    (dict(o=4 * A), "INVALID_ARG"), (dict(lse=5 * A), "INVALID_ARG"),
    (dict(n_seq=(1 << 31) - 1), "UNSUPPORTED"), (dict(tokens=1 << 30), "UNSUPPORTED"),
    (dict(status=9 * A + 2), "MISALIGNED"), (dict(status=7 * A), "INVALID_ARG"), (dict(status=8 * A), "INVALID_ARG"),
    (dict(workspace=64 * A, workspace_bytes=100), "INVALID_ARG"), (dict(workspace=None, workspace_bytes=1 << 28), "INVALID_ARG"),
    (dict(workspace=64 * A + 8, workspace_bytes=1 << 28), "MISALIGNED"), (dict(workspace=A, workspace_bytes=1 << 28), "INVALID_ARG"),
])
def test_attention_refusals(dep, change, status):
    with pytest.raises(dep.DepError) as e:
        dep.dep_paged_attention(attention_args(dep, **change), 0)
    assert e.value.status == getattr(dep, "DEP_ERR_" + status)


def test_attention_workspace_size(dep):
    size = lambda **kw: dep.dep_attention_workspace(attention_args(dep, workspace=64 * A, **kw))  # noqa: E731
    assert size(tokens=0) == 0
    assert size(tokens=1) < size(tokens=2) < size(tokens=127) < size(tokens=128) == size(tokens=1 << 20)  # 256 rows of an item at most
    assert size(tokens=1, n_seq=1) == size(tokens=1, n_seq=1000) and size(tokens=64, D=128) > size(tokens=64, D=64)
    assert size(tokens=1 << 20, D=128) < 64 << 20


def test_attention_nothing_to_do(dep):
    dep.dep_paged_attention(attention_args(dep, tokens=0, n_seq=0), 0)
    dep.dep_paged_attention(attention_args(dep, tokens=0), 0)
    assert dep.lib().dep_paged_attention(None, None) == dep.DEP_ERR_INVALID_ARG
    assert dep.lib().dep_attention_workspace(None, ctypes.byref(ctypes.c_int64())) == dep.DEP_ERR_INVALID_ARG
    assert dep.lib().dep_attention_workspace(ctypes.byref(attention_args(dep)), None) == dep.DEP_ERR_INVALID_ARG
    for bad in (dict(tokens=-1), dict(n_seq=-1), dict(Hq=0), dict(Hk=0)):
        with pytest.raises(dep.DepError):
            dep.dep_attention_workspace(attention_args(dep, workspace=64 * A, **bad))


def test_python_entry_points_refuse(dep):
    torch = pytest.importorskip("torch")
    h = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    cache = torch.zeros(3, 16, 4, 64, dtype=torch.bfloat16)
    i32 = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        dep.norm_rotate(h)
    with pytest.raises(ValueError):
        dep.append_kv(h, h, cache, cache, i32)
    with pytest.raises(ValueError):
        dep.paged_attention(h, cache, cache, i32[:, None], i32)


def test_arguments_that_a_field_does_not_hold(dep):
    """Sizes past their field's width are refused, not cut off to its bits."""
    from skinny_bf16_split_gb300 import _binding as b
    for cls, fill in ((dep.dep_heads_args_t, b._heads_args), (dep.dep_attention_args_t, b._attention_args)):
        names = [n for n, _ in cls._fields_]
        args = fill(*range(1, len(names) + 1))
        assert [getattr(args, n) for n in names] == list(range(1, len(names) + 1))
        for name, kind in cls._fields_:
            for value in {ctypes.c_int32: ((1 << 32) + 16, -(1 << 31) - 1), ctypes.c_int64: (1 << 63,),
                          ctypes.c_uint32: (1 << 32, -1), ctypes.c_float: (), ctypes.c_void_p: ()}[kind]:
                with pytest.raises(ValueError):
                    fill(*(value if n == name else 0 for n in names))
