"""dg where the decay's factor is zero: alpha_t <S_{t-1}, dS_t> is exactly 0
there, while the suffix sums that give dg elsewhere leave their rounding."""

import numpy as np
import pytest
import torch

import gated_delta_rule_54_amd as gdr
from tests.test_gpu_linear import ALGOS, BF, F, check, draw, to_dev

pytestmark = pytest.mark.gpu


def dg_of(x, algo, **kw):
    t = to_dev(x, BF)
    return gdr.gdr_linear_backward(t["q"], t["k"], t["v"], t["g"], t["h0"], t["do"], t["dht"], algo=algo, **kw)[3]


@pytest.mark.parametrize("algo", ALGOS)
@pytest.mark.parametrize("low", [-np.inf, -3e4, -104.5, np.finfo(np.float32).min])
def test_zero_at_dropped_states(algo, low):
    x = draw(51, 2, 150, 2, 4, 64, 64)
    at = [0, 37, 63, 64, 100, 149]
    x["g"][:, at, 1:3] = low
    dg = dg_of(x, algo)
    assert (dg[:, at, 1:3] == 0).all()
    assert dg[:, :, 0].count_nonzero() == dg[:, :, 0].numel()
    check(x, BF, F, algo)


@pytest.mark.parametrize("algo", ALGOS)
def test_zero_for_a_head_that_keeps_nothing(algo):
    x = draw(52, 2, 90, 2, 4, 64, 64, gate="head")
    x["g"][[1, 3]] = -np.inf, -200.0
    dg = dg_of(x, algo)
    assert dg[1] == 0 and dg[3] == 0 and dg[0] != 0 and dg[2] != 0
    check(x, BF, F, algo)


@pytest.mark.parametrize("algo", ALGOS)
def test_zero_in_a_ragged_batch(algo):
    x = draw(53, 1, 120, 2, 2, 64, 64, state=False)
    x["g"][:, [0, 30, 50, 51]] = -np.inf
    cu = torch.tensor([10, 30, 30, 51, 110], device="cuda")
    dg = dg_of(x, algo, cu_seqlens=cu)
    assert (dg[:, [30, 50, 51]] == 0).all() and dg[:, [10, 29, 31, 109]].all()
