"""Options of the attention layer's calls that are refused are refused whatever calls
came before: also where they equal an option that a call was planned for."""

import numpy as np
import pytest
import torch

import gated_delta_rule_54_amd as gdr
from tests.test_gpu_rotary import BF

pytestmark = pytest.mark.gpu


def randn(*shape):
    return torch.randn(*shape, device="cuda").to(BF)


def test_options_that_equal_a_planned_one():
    q, k, v, do = randn(1, 9, 4, 32), randn(1, 9, 2, 32), randn(1, 9, 2, 32), randn(1, 9, 4, 32)
    kc, vc = randn(4, 16, 2, 32), randn(4, 16, 2, 32)
    table = torch.arange(4, dtype=torch.int32, device="cuda").reshape(1, 4)
    n = torch.tensor([30], device="cuda")
    cu = torch.tensor([0, 4, 9], device="cuda")
    o, lse = gdr.gdr_attention_forward(q, k, v, window=5, sinks=2)
    forward = lambda **how: gdr.gdr_attention_forward(q, k, v, **how)
    backward = lambda **how: gdr.gdr_attention_backward(q, k, v, o, lse, do, **how)
    token = lambda **how: gdr.gdr_cache_attention(q[:, :1].contiguous(), kc, vc, table, n, **how)
    ragged = lambda **how: gdr.gdr_attention_forward(q, k, v, cu_seqlens=cu, **how)
    calls = [(forward, dict(window=5, sinks=2)), (backward, dict(window=5, sinks=2)),
             (token, dict(window=5, sinks=2, max_len=40)), (ragged, dict(max_seqlen=5))]
    for call, how in calls:
        for _ in range(2):
            for name, x in how.items():
                with pytest.raises(TypeError):
                    call(**dict(how, **{name: float(x)}))
            want = call(**how)
        # an integer of another kind is one
        same = call(**{name: np.int64(x) for name, x in how.items()})
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, same))


def test_lse_of_a_token():
    kc = randn(4, 16, 2, 32)
    table = torch.arange(4, dtype=torch.int32, device="cuda").reshape(1, 4)
    n = torch.tensor([30], device="cuda")
    q = randn(1, 1, 4, 32)
    for bad in (False, 1, "no"):
        with pytest.raises(TypeError, match="lse"):
            gdr.gdr_cache_attention(q, kc, kc, table, n, lse=bad)
    assert gdr.gdr_cache_attention(q, kc, kc, table, n, lse=None)[1] is None
