"""Refusals of the operators around the projections: host checks, no GPU.

Every call here is refused before anything is launched, so made-up addresses of
the right alignment stand for device memory."""
import ctypes

import pytest

A = 1 << 20  # an address; tensors below are placed megabytes apart


def norm_args(dep, **kw):
    base = dict(x=A, residual=2 * A, weight=3 * A, residual_out=2 * A, out=4 * A, scale=None, x_stride=64,
                residual_stride=64, residual_out_stride=64, out_stride=64, rows=4, cols=64, quant=dep.DEP_QUANT_NONE,
                eps=1e-6)
    base.update(kw)
    return dep.dep_norm_args_t(**base)


@pytest.mark.parametrize("change,status", [
    (dict(rows=-1), "INVALID_ARG"), (dict(cols=0), "INVALID_ARG"), (dict(quant=3), "INVALID_ARG"),
    (dict(quant=-1), "INVALID_ARG"), (dict(eps=-1.0), "INVALID_ARG"), (dict(eps=float("nan")), "INVALID_ARG"),
    (dict(x=None), "INVALID_ARG"), (dict(out=None), "INVALID_ARG"), (dict(residual=None), "INVALID_ARG"),
    (dict(residual_out=None), "INVALID_ARG"), (dict(x_stride=63), "INVALID_ARG"),
    (dict(out_stride=63), "INVALID_ARG"), (dict(residual_stride=8), "INVALID_ARG"),
    (dict(scale=9 * A), "INVALID_ARG"),                       # scales without an 8-bit format
    (dict(quant=1), "INVALID_ARG"),                           # and the reverse
    (dict(x=A + 1), "MISALIGNED"), (dict(out=4 * A + 1), "MISALIGNED"),
    (dict(cols=65537, x_stride=65537, residual_stride=65537, residual_out_stride=65537, out_stride=65537),
     "UNSUPPORTED"),
    (dict(out=A + 2), "INVALID_ARG"),                         # rows shifted over x's
    (dict(out=2 * A), "INVALID_ARG"),                         # over the residual
    (dict(out=3 * A), "INVALID_ARG"),                         # over the weight
    (dict(residual_out=A), "INVALID_ARG"),                    # over x
    (dict(residual_out_stride=80), "INVALID_ARG"),            # the residual's rows, spaced otherwise
    (dict(quant=1, scale=5 * A, out=A), "INVALID_ARG"),       # 8-bit rows over x
    (dict(quant=1, scale=4 * A + 64), "INVALID_ARG"),         # scales inside the output
    (dict(quant=2, scale=5 * A + 2), "MISALIGNED"),
])
def test_norm_refusals(dep, change, status):
    with pytest.raises(dep.DepError) as e:
        dep.dep_add_rms_norm(norm_args(dep, **change), 0)
    assert e.value.status == getattr(dep, "DEP_ERR_" + status)


def test_norm_nothing_to_do(dep):
    dep.dep_add_rms_norm(norm_args(dep, rows=0), 0)
    assert dep.lib().dep_add_rms_norm(None, None) == dep.DEP_ERR_INVALID_ARG


@pytest.mark.parametrize("change", [dict(), dict(residual=2 * A, residual_out=2 * A), dict(weight=3 * A),
                                    dict(quant=0, scale=None)])
def test_quantize_refuses_what_belongs_to_the_norm(dep, change):
    kw = dict(residual=None, residual_out=None, weight=None, quant=1, scale=5 * A)
    if not change:
        kw["scale"] = None
    kw.update(change)
    with pytest.raises(dep.DepError) as e:
        dep.dep_quantize_rows(norm_args(dep, **kw), 0)
    assert e.value.status == dep.DEP_ERR_INVALID_ARG


def delta_args(dep, **kw):
    M = 64 * A
    base = dict(q=A, k=2 * A, v=3 * A, g=4 * A, beta=5 * A, state_in=M, state_out=M, o=6 * A, cu_seqlens=None,
                slots=None, q_stride=128, k_stride=128, v_stride=256, g_stride=4, beta_stride=4, o_stride=256, tokens=6,
                n_states=3, n_seq=3, Hq=2, Hv=4, Dk=64, Dv=64, flags=0, scale=0.125)
    base.update(kw)
    return dep.dep_delta_args_t(**base)


@pytest.mark.parametrize("change,status", [
    (dict(tokens=-1), "INVALID_ARG"), (dict(n_seq=-1), "INVALID_ARG"), (dict(Hq=0), "INVALID_ARG"),
    (dict(Hq=3), "INVALID_ARG"), (dict(flags=4), "INVALID_ARG"), (dict(tokens=7), "INVALID_ARG"),
    (dict(n_seq=0), "INVALID_ARG"), (dict(n_states=2), "INVALID_ARG"), (dict(state_out=None), "INVALID_ARG"),
    (dict(q=None), "INVALID_ARG"), (dict(beta=None), "INVALID_ARG"), (dict(o=None), "INVALID_ARG"),
    (dict(q_stride=120), "INVALID_ARG"), (dict(v_stride=248), "INVALID_ARG"), (dict(beta_stride=3), "INVALID_ARG"),
    (dict(flags=1), "INVALID_ARG"),                            # per-channel decays need 4 * 64 columns
    (dict(Dk=96), "UNSUPPORTED"), (dict(Dv=24), "UNSUPPORTED"), (dict(Dv=272, v_stride=1088, o_stride=1088), "UNSUPPORTED"),
    (dict(Dv=8), "UNSUPPORTED"),
    (dict(q=A + 8), "MISALIGNED"), (dict(k_stride=132), "MISALIGNED"), (dict(state_in=64 * A + 4), "MISALIGNED"),
    (dict(g=4 * A + 2), "MISALIGNED"), (dict(cu_seqlens=7 * A + 2), "MISALIGNED"), (dict(slots=7 * A + 1), "MISALIGNED"),
    (dict(flags=1, g_stride=258), "MISALIGNED"),
    (dict(o=3 * A), "INVALID_ARG"), (dict(o=64 * A), "INVALID_ARG"),  # over v, over the states
    (dict(state_out=64 * A + 65536), "INVALID_ARG"),           # states that overlap by a part
])
def test_delta_refusals(dep, change, status):
    with pytest.raises(dep.DepError) as e:
        dep.dep_delta_rule(delta_args(dep, **change), 0)
    assert e.value.status == getattr(dep, "DEP_ERR_" + status)


@pytest.mark.parametrize("change,status", [
    (dict(workspace_bytes=-1), "INVALID_ARG"), (dict(workspace_bytes=64), "INVALID_ARG"),
    (dict(workspace=80 * A + 8, workspace_bytes=64), "MISALIGNED"),
    (dict(workspace=A, workspace_bytes=64), "INVALID_ARG"),              # over q
    (dict(workspace=6 * A - 64, workspace_bytes=128), "INVALID_ARG"),    # reaches into o
    (dict(workspace=64 * A + 1024, workspace_bytes=64), "INVALID_ARG"),  # among the states
])
def test_delta_workspace_refusals(dep, change, status):
    with pytest.raises(dep.DepError) as e:
        dep.dep_delta_rule(delta_args(dep, **change), 0)
    assert e.value.status == getattr(dep, "DEP_ERR_" + status)


def test_delta_workspace_size(dep):
    size = lambda **kw: dep.dep_delta_workspace(delta_args(dep, **kw))  # noqa: E731
    assert size(tokens=64, n_seq=64) == 0 and size(tokens=0, n_seq=0) == 0
    one = size(tokens=48, n_seq=1) // 4  # 48 tokens may touch four chunks
    assert one > 0 and size(tokens=480, n_seq=2, Hv=4) == 32 * one and size(tokens=48, n_seq=1, Hv=8) == 8 * one
    assert one < size(tokens=48, n_seq=1, Dk=128) // 4 and size(tokens=1 << 30, n_seq=1) <= 2 << 30
    assert size(tokens=1 << 30, n_seq=1, Hv=1 << 20) == (1 << 20) * one // 4 > 2 << 30
    for args in (delta_args(dep, tokens=-1), delta_args(dep, n_seq=-1), delta_args(dep, Hv=0)):
        with pytest.raises(dep.DepError):
            dep.dep_delta_workspace(args)


def test_delta_nothing_to_do(dep):
    dep.dep_delta_rule(delta_args(dep, tokens=0, n_seq=0), 0)
    assert dep.lib().dep_delta_rule(None, None) == dep.DEP_ERR_INVALID_ARG


@pytest.mark.parametrize("N,K,rows,status", [(0, 64, 1, "INVALID_ARG"), (8, 8, 1, "INVALID_ARG"),
                                             (8, 64, 0, "INVALID_ARG"), (8, 72, 1, "MISALIGNED"),
                                             (8, 131072, 1, "UNSUPPORTED")])
def test_int8_plan_refusals(dep, N, K, rows, status):
    with pytest.raises(dep.DepError) as e:
        dep.dep_int8_plan(N, K, rows)
    assert e.value.status == getattr(dep, "DEP_ERR_" + status)


def test_int8_null_arguments(dep):
    L = dep.lib()
    assert L.dep_int8_plan(8, 64, 1, None) == dep.DEP_ERR_INVALID_ARG
    assert L.dep_int8_run(None, A, A, A, A, A, 1, None) == dep.DEP_ERR_INVALID_ARG
    assert L.dep_int8_plan_workspace(None, ctypes.byref(ctypes.c_size_t())) == dep.DEP_ERR_INVALID_ARG
    assert L.dep_int8_device_status(None, None, ctypes.byref(ctypes.c_int32())) == dep.DEP_ERR_INVALID_ARG
    L.dep_int8_plan_destroy(None)


def test_python_entry_points_refuse_host_tensors(dep):
    torch = pytest.importorskip("torch")
    x = torch.zeros(2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        dep.add_rms_norm(x)
    with pytest.raises(ValueError):
        dep.quantize_rows(x, quant=None)
    with pytest.raises(ValueError):
        dep.gated_delta_rule(x, x, x, x, x, x)
    with pytest.raises(ValueError):
        dep.Int8Projection(torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4))
