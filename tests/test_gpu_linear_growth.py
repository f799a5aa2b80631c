"""Gates above 0: growth of up to 2^48 over the tokens of a chunk, with decays
far below fp32's least value between, keeps every term (include/gdr.h)."""

import numpy as np
import pytest

from tests.test_gpu_linear import ALGOS, BF, F, check, draw

pytestmark = pytest.mark.gpu

LN2 = float(np.log(2.0))


@pytest.mark.parametrize("algo", ALGOS)
@pytest.mark.parametrize("io", [BF, F])
@pytest.mark.parametrize("steps", [((16, 3.0), (16, -9.5), (16, 2.9), (16, -3.0)), ((8, 5.9), (9, -20.0), (8, 5.9), (40, 0.0)),
                                   ((1, 47.0), (1, -150.0), (14, 0.0), (1, 47.0), (1, -149.0), (30, 0.5), (13, -1.2)),
                                   ((64, 0.74), (64, -0.74))])
def test_growth_within_a_chunk(algo, io, steps):
    log2 = np.concatenate([np.full(n, r) for n, r in steps])
    # up to 2^48 over any run of a chunk's tokens: what the test is for
    for c in (32, 64):
        for i in range(0, len(log2), c):
            s = np.concatenate([[0.0], np.cumsum(log2[i:i + c])])
            assert max(s[b] - s[:b + 1].min() for b in range(len(s))) <= 48.0
    x = draw(71, 1, len(log2), 2, 2, 64, 64, io, state=False)
    x["g"][:] = (LN2 * log2)[None, :, None].astype(np.float32)
    check(x, io, F, algo)
