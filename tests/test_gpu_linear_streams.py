"""Calls at once on two streams, from one thread and from two: each gives the
bits it gives alone."""

import threading

import pytest
import torch

import gated_delta_rule_54_amd as gdr
from tests.test_gpu_linear import BF, draw, to_dev

pytestmark = pytest.mark.gpu


def layer(t, algo):
    rule = t["q"], t["k"], t["v"], t["g"], t["h0"]
    o, ht = gdr.gdr_linear_forward(*rule, algo=algo, out_dtype=BF)
    y = gdr.gdr_group_norm_forward(o, t["w"], None, t["do"], out_dtype=BF)
    do, dz, dw, _ = gdr.gdr_group_norm_backward(o, t["w"], None, t["do"], y, out_dtype=BF)
    return (o, ht, y, do, dz, dw) + gdr.gdr_linear_backward(*rule, do, t["dht"], algo=algo, out_dtype=BF)


@pytest.mark.parametrize("algo", ["sequential", "chunked"])
@pytest.mark.parametrize("threads", [False, True])
def test_two_streams_at_once(algo, threads):
    x = [to_dev(draw(81 + i, 2, 700 - 50 * i, 2, 4, 64, 64), BF) for i in range(2)]
    for t in x:
        t["w"] = 1 + 0.2 * torch.randn(4, 64, device="cuda")
    want = [layer(t, algo) for t in x]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in x]
    got = [[], []]

    def run(i, n):
        with torch.cuda.stream(streams[i]):
            for _ in range(n):
                got[i].append(layer(x[i], algo))

    if threads:
        work = [threading.Thread(target=run, args=(i, 4)) for i in range(2)]
        for w in work:
            w.start()
        for w in work:
            w.join()
    else:
        for _ in range(4):
            run(0, 1)
            run(1, 1)
    torch.cuda.synchronize()
    for i in range(2):
        assert len(got[i]) == 4
        for res in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(res, want[i]))
