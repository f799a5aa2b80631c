"""Views that the operators beside the delta rule take and refuse: rows may lie
apart, but each has its own storage.  A row of an expanded tensor has not, and
its distance, 0, must not be taken for that of dense rows."""

import pytest
import torch

import gated_delta_rule_54_amd as gdr
from gated_delta_rule_54_amd import linear as L

BF, F = torch.bfloat16, torch.float32


def shared_rows(device="cpu"):
    one = torch.zeros(1, 1, 4, 64, dtype=BF, device=device)
    return (one.expand(8, 1, 4, 64),                                        # one token's query for eight sequences
            one.expand(1, 100, 4, 64), one.expand(3, 100, 4, 64), one[0].expand(7, 4, 64),
            torch.zeros(2, 5, 1, 64, dtype=BF, device=device)[:, :1].expand(2, 5, 1, 64),
            torch.zeros(1000, dtype=BF, device=device).as_strided((5, 4, 64), (128, 64, 1)))  # rows that overlap


def test_rows_without_storage_of_their_own_are_refused():
    for t in shared_rows():
        with pytest.raises(ValueError, match="strides"):
            L._row_stride(t, "q")


def test_expanded_axes_of_one_row_or_none_are_dense():
    assert L._row_stride(torch.zeros(1, 1, 4, 64).expand(1, 1, 4, 64), "q") == 0
    assert L._row_stride(torch.zeros(1, 1, 4, 64).expand(8, 1, 4, 64)[:1], "q") == 0
    assert L._row_stride(torch.zeros(1, 1, 4, 64).expand(0, 5, 4, 64), "q") == 0
    assert L._row_stride(torch.zeros(6, 1, 64)[::2], "x") == 128


@pytest.mark.gpu
def test_calls_refuse_expanded_operands():
    """Every operand that may be strided, before anything is launched."""
    dense = torch.zeros(8, 1, 4, 64, dtype=BF, device="cuda")
    for bad in shared_rows("cuda")[:1]:
        for i in range(3):
            qkv = [dense] * 3
            qkv[i] = bad
            with pytest.raises(ValueError, match="strides"):
                gdr.gdr_linear_forward(*qkv)
            with pytest.raises(ValueError, match="strides"):
                gdr.gdr_linear_backward(*qkv, None, None, dense)
        with pytest.raises(ValueError, match="strides"):
            gdr.gdr_group_norm_forward(bad)
        with pytest.raises(ValueError, match="strides"):
            gdr.gdr_group_norm_forward(dense, z=bad)
        with pytest.raises(ValueError, match="strides"):
            gdr.gdr_group_norm_backward(dense, None, None, bad, dense)
    o, _ = gdr.gdr_linear_forward(dense, dense, dense)  # the same call on storage of their own
    assert not o.any()
