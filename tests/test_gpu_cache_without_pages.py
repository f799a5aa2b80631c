"""A cache without a page, or a table without a column: nothing is stored and nothing is
visible, the new tokens' q is turned as ever."""

import pytest
import torch

import gated_delta_rule_54_amd as gdr
from tests.test_gpu_rotary import BF, dev, freqs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("pages,columns", [(0, 3), (0, 0), (2, 0)])
@pytest.mark.parametrize("ragged", [False, True])
def test_no_pages(pages, columns, ragged):
    k, v, q = (torch.randn(1, 10, H, 64, device="cuda").to(BF) for H in (2, 2, 4))
    kc, vc = (torch.full((pages, 16, 2, 64), 7.0, device="cuda", dtype=BF) for _ in "kv")
    B = 2 if ragged else 1
    table = torch.arange(B * columns, dtype=torch.int32, device="cuda").reshape(B, columns)
    lengths = torch.tensor([12, 6][:B], device="cuda")
    f = dev(freqs(64))
    how = dict(cu_seqlens=torch.tensor([0, 4, 10], device="cuda")) if ragged else {}
    got = gdr.gdr_cache_append(k, v, kc, vc, table, lengths, f, q=q, **how)
    place = torch.tensor([[8, 9, 10, 11, 0, 1, 2, 3, 4, 5]], device="cuda") if ragged else torch.arange(2, 12, device="cuda")[None]
    want, _ = gdr.gdr_rotary_forward(q, None, place, f, out_dtype=BF)
    assert torch.equal(got, want)
    assert (kc == 7).all() and (vc == 7).all()
    o, lse = gdr.gdr_cache_attention(got[:, :B].transpose(0, 1).contiguous(), kc, vc, table, lengths)
    assert (o == 0).all() and (lse == -float("inf")).all()
