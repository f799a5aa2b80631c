"""The limits that include/gdr.h states for linear attention and the group norm:
taken up to them, GDR_ERR_UNSUPPORTED past them (shape part only, on the CPU)."""

import pytest

from tests.test_linear_abi import bwd, fwd, norm, prob, query

FORWARD, BACKWARD, NORM = ("gdr_linear_forward_workspace", "gdr_linear_backward_workspace",
                           "gdr_group_norm_backward_workspace")
TOP = (1 << 31) - 1


@pytest.mark.parametrize("kw", [dict(B=64, T=1 << 22, Hk=16, Hv=32), dict(B=1, T=TOP, Hk=2, Hv=2),
                                dict(B=1, T=TOP // 2, Hk=16, Hv=16, Dk=16, Dv=16), dict(B=60000, T=35000, Hk=1, Hv=1)])
def test_forward_counts_tokens_not_heads(kw):
    """Only the VJP's partial rows have a place for every key head's token."""
    assert query(FORWARD, prob(**kw))[0] == 0
    assert fwd(prob(**kw), ragged=True, q=None) == 1 and fwd(prob(**kw), q=None) == 1  # past the shape's checks


@pytest.mark.parametrize("kw", [dict(B=2, T=1 << 30, Hk=1, Hv=1), dict(B=1, T=TOP + 1, Hk=1, Hv=1),
                                dict(B=65535, T=TOP, Hk=1, Hv=1)])
def test_forward_past_its_tokens(kw):
    assert query(FORWARD, prob(**kw)) == (3, 12345) and fwd(prob(**kw)) == 3


def test_backward_counts_its_heads():
    assert query(BACKWARD, prob(B=1, T=TOP // 2, Hk=2, Hv=2))[0] == 0
    assert query(BACKWARD, prob(B=1, T=TOP // 2 + 1, Hk=2, Hv=2)) == (3, 12345)
    assert bwd(prob(B=64, T=1 << 22, Hk=16, Hv=32)) == 3


def test_states_and_rows():
    assert query(FORWARD, prob(B=65535, Hk=1, Hv=1, T=1))[0] == 0 and query(FORWARD, prob(B=65536, Hk=1, Hv=1))[0] == 3
    # B Hv (2 ceil(Dk / 64) + ceil(Dv / 64)) up to 2^22
    assert query(FORWARD, prob(B=1 << 14, Hk=64, Hv=64, Dk=64, Dv=128, T=1))[0] == 0
    assert query(FORWARD, prob(B=(1 << 14) + 1, Hk=64, Hv=64, Dk=64, Dv=128, T=1))[0] == 3
    # a row of 2^22 elements, q's and k's or v's
    assert query(FORWARD, prob(B=1, Hk=1 << 14, Hv=1 << 14, Dk=256, Dv=64, T=1))[0] == 0
    assert query(FORWARD, prob(B=1, Hk=1, Hv=(1 << 14) + 1, Dk=16, Dv=256, T=1))[0] == 3


def test_norm():
    assert query(NORM, norm(rows=1 << 40))[0] == 0 and query(NORM, norm(rows=(1 << 40) + 1))[0] == 3
    assert query(NORM, norm(groups=65535, channels=64))[0] == 0 and query(NORM, norm(groups=65536, channels=8))[0] == 3
    assert query(NORM, norm(groups=1 << 13, channels=512))[0] == 0
    assert query(NORM, norm(groups=(1 << 13) + 1, channels=512))[0] == 3
    assert query(NORM, norm(x_row=1 << 22))[0] == 0 and query(NORM, norm(z_row=(1 << 22) + 8))[0] == 3
