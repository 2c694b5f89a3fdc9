"""Refusals of the attention's give-up self-test: host checks, no GPU."""
import pytest

from test_attention_host import A, attention_args


@pytest.mark.parametrize("code", [0, 5, -1])
def test_selftest_refusals(dep, code):
    with pytest.raises(dep.DepError) as e:
        dep.dep_attention_selftest_timeout(attention_args(dep), code, 0)
    assert e.value.status == dep.DEP_ERR_INVALID_ARG


@pytest.mark.parametrize("change,status", [(dict(tokens=-1), "INVALID_ARG"), (dict(D=96, q_stride=512, o_stride=512), "UNSUPPORTED"),
                                           (dict(q=A + 8), "MISALIGNED"), (dict(o=A), "INVALID_ARG")])
def test_selftest_refuses_what_the_call_refuses(dep, change, status):
    with pytest.raises(dep.DepError) as e:
        dep.dep_attention_selftest_timeout(attention_args(dep, **change), dep.DEP_DEV_TIMEOUT_MMA, 0)
    assert e.value.status == getattr(dep, "DEP_ERR_" + status)


def test_selftest_of_nothing(dep):
    dep.dep_attention_selftest_timeout(attention_args(dep, tokens=0), dep.DEP_DEV_TIMEOUT_MMA, 0)
    assert dep.lib().dep_attention_selftest_timeout(None, 1, None) == dep.DEP_ERR_INVALID_ARG
