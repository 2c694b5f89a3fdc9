"""Sizes at the ends of what the attention's arithmetic holds: host checks, no GPU."""
import pytest

from test_attention_host import A, attention_args

FAR = dict(workspace=64 * A, workspace_bytes=1 << 40)


@pytest.mark.parametrize("change", [
    # a token's heads past 2^31 channels
    dict(tokens=1, n_seq=1, Hq=1 << 25, q_stride=1 << 31, o_stride=1 << 31, lse=None),
    dict(tokens=3, Hq=(1 << 24) + 2, D=128, q_stride=1 << 40, o_stride=1 << 40),
    dict(tokens=1, n_seq=1, Hq=(1 << 31) - (1 << 14), q_stride=1 << 40, o_stride=1 << 40),
    # rows past 2^31, up to where their number passes 64 bits
    dict(tokens=1 << 30), dict(tokens=1 << 60, Hq=16, q_stride=1024, o_stride=1024), dict(tokens=(1 << 62) + 1),
    dict(tokens=1 << 62, Hq=4, Hk=4), dict(tokens=(1 << 63) - 1),
])
def test_sizes_that_32_bits_do_not_hold(dep, change):
    with pytest.raises(dep.DepError) as e:
        dep.dep_paged_attention(attention_args(dep, **{**FAR, "cu_seqlens": 1 << 50, **change}), 0)
    assert e.value.status == dep.DEP_ERR_UNSUPPORTED


@pytest.mark.parametrize("tokens", [1 << 31, 1 << 56, 1 << 62, (1 << 63) - 1])
@pytest.mark.parametrize("Hq", [2, 1 << 30])
def test_workspace_of_any_number_of_tokens(dep, tokens, Hq):
    size = lambda t: dep.dep_attention_workspace(attention_args(dep, tokens=t, Hq=Hq, Hk=2, **FAR))  # noqa: E731
    assert size(tokens) == size(1 << 20) > size(1) - 1 > 0
