"""The last rows of a long sequence under a window with fp32 outputs, against the 64-bit
definition of the short sequence that they see (the sinks and the last tokens), under
the bounds of test_gpu_attention: no part of an operand may be missing at far offsets,
where a bound relative to bf16 would not tell."""

import numpy as np
import pytest
import torch

import gated_delta_rule_54_amd as gdr
from tests.test_gpu_attention import bounds, close
from tests.test_gpu_attention_large import randn
from tests.test_gpu_rotary import BF, F, host

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("io", [BF, F])
@pytest.mark.parametrize("D,W,S", [(64, 200, 5), (128, 150, 0), (256, 90, 70)])
def test_last_rows(io, D, W, S):
    T, Hq, Hk = 120_000 + 37, 2, 1
    x = [randn(80 + i, 1, T, H, D, dtype=io) for i, H in enumerate((Hq, Hk, Hk, Hq))]
    q, k, v, do = x
    how = dict(window=W, sinks=S)
    o, lse = gdr.gdr_attention_forward(q, k, v, **how)
    dq, dk, dv = gdr.gdr_attention_backward(q, k, v, o, lse, do, **how)

    def cut(t):
        # places of the cut: sinks, then the last 2 W tokens, of which the last W have
        # every token they see in it
        return host(torch.cat([t[0, :S], t[0, -2 * W:]]))

    res, tol = bounds(*(cut(t) for t in x), cut(o), D ** -0.5, W, S, F)
    for name, t in (("o", o), ("lse", lse), ("dq", dq), ("dk", dk), ("dv", dv)):
        assert np.isfinite(host(t[0, -W:])).all()
        close(name, host(t[0, -W:]), res[name][-W:], tol[name][-W:], F)
