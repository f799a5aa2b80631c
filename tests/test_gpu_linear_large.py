"""Linear attention and the group norm where offsets pass 32 bits (elements and
bytes), and a ragged batch captured once and replayed with other offsets.

A decay of e^-1 a token leaves nothing of a token 200 later (e^-200 is below
fp32's least value), so a long sequence's last and first rows are those of the
cuts around them."""

import numpy as np
import pytest
import torch

import gated_delta_rule_54_amd as gdr
from tests.test_gpu_linear import BF, F, draw, to_dev

pytestmark = pytest.mark.gpu

T, HK, HV, D = 1_100_000, 1, 32, 128  # v, o, dv: 4.5e9 elements
END, NEAR = 300, 64


def randn(seed, *shape):
    """bf16 of no more memory than the result's and a piece's."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.empty(shape, dtype=BF, device="cuda")
    for piece in x.view(-1).split(1 << 28):
        piece.copy_(torch.randn(piece.numel(), device="cuda", generator=g))
    return x


def same(name, a, b):
    """fp32 sums cut otherwise, rounded once to bf16: the next value at most,
    and where terms cancel, 2^-16 of what is there."""
    a, b = a.float(), b.float()
    assert torch.isfinite(a).all(), name
    assert ((a - b).abs() <= 2.0 ** -7 * b.abs() + 2.0 ** -16 * b.abs().max()).all(), name


def test_linear_past_32_bits():
    k, v = randn(1, 1, T, HK, D), randn(2, 1, T, HV, D)
    q = randn(3, 1, T, HK, D)
    g = torch.full((1, T, HV), -1.0, device="cuda")
    for algo in ("chunked", "auto"):
        o, ht = gdr.gdr_linear_forward(q, k, v, g, algo=algo, out_dtype=BF)
        cut = [a[:, -END:].contiguous() for a in (q, k, v, g)]
        o1, ht1 = gdr.gdr_linear_forward(*cut, algo="chunked", out_dtype=BF)
        same("o", o[:, -NEAR:], o1[:, -NEAR:])
        assert ((ht - ht1).abs() <= 2.0 ** -16 * ht1.abs().max()).all()
    do = o.copy_(v)  # of o's memory
    dq, dk, dv, dg, _ = gdr.gdr_linear_backward(q, k, v, g, None, do, out_dtype=BF)
    one = gdr.gdr_linear_backward(*cut, None, do[:, -END:].contiguous(), algo="chunked", out_dtype=BF)
    for name, a, b in zip(("dq", "dk", "dv"), (dq, dk, dv), one):
        same(name, a[:, -NEAR:], b[:, -NEAR:])
    first = gdr.gdr_linear_backward(*(a[:, :END].contiguous() for a in (q, k, v, g)), None, do[:, :END].contiguous(),
                                    algo="chunked", out_dtype=BF)
    for name, a, b in zip(("dq", "dk", "dv"), (dq, dk, dv), first):
        same(name, a[:, :NEAR], b[:, :NEAR])
    assert torch.isfinite(dg).all()


def test_norm_past_32_bits():
    rows = T
    x, z = randn(4, rows, HV, D), randn(5, rows, HV, D)
    w = 1 + 0.1 * torch.randn(HV, D, device="cuda")
    y = gdr.gdr_group_norm_forward(x, w, None, z, center=True, out_dtype=BF)
    e = slice(rows - 50, rows)
    assert torch.equal(y[e], gdr.gdr_group_norm_forward(x[e], w, None, z[e], center=True, out_dtype=BF))
    dy = y.copy_(z)
    dx, dz, dw, _ = gdr.gdr_group_norm_backward(x, w, None, z, dy, center=True, out_dtype=BF)
    one = gdr.gdr_group_norm_backward(x[e], w, None, z[e], dy[e], center=True, out_dtype=BF)
    assert torch.equal(dx[e], one[0]) and torch.equal(dz[e], one[1])
    parts = [gdr.gdr_group_norm_backward(*(a[i:i + 100_000] if a.dim() == 3 else a for a in (x, w)), None,
                                         z[i:i + 100_000], dy[i:i + 100_000], center=True, out_dtype=BF)[2]
             for i in range(0, rows, 100_000)]
    # fp32 over each slot's rows, 64 bits over the slots: random signs, so far below rows 2^-24 of the terms
    assert ((sum(p.double() for p in parts) - dw).abs() <= 1e-4 * dw.abs().max()).all()


@pytest.mark.parametrize("algo", ["sequential", "chunked"])
def test_ragged_graph_replayed_with_other_offsets(algo):
    """Captured with a bound and replayed as the batch's offsets change, to
    empty sequences and uncovered rows too: the eager bits each time."""
    rows, N, bound = 400, 5, 250
    x = draw(61, 1, rows, 2, 4, 64, 64, state=False)
    r = np.random.default_rng(62)
    x["h0"], x["dht"] = (r.standard_normal((N, 4, 64, 64)).astype(np.float32) for _ in range(2))
    t = to_dev(x, BF)
    offsets = [[0, 100, 100, 230, 399, 400], [0, 250, 400, 400, 400, 400], [7, 8, 9, 10, 260, 300], [0, 0, 0, 0, 0, 0]]
    cu = torch.tensor(offsets[0], device="cuda")
    kw = dict(algo=algo, cu_seqlens=cu, max_seqlen=bound)

    def both():
        return (gdr.gdr_linear_forward(t["q"], t["k"], t["v"], t["g"], t["h0"], **kw)
                + gdr.gdr_linear_backward(t["q"], t["k"], t["v"], t["g"], t["h0"], t["do"], t["dht"], **kw))

    both()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res = both()
    for o in offsets[1:] + offsets[:2]:
        cu.copy_(torch.tensor(o))
        for a in res:
            a.fill_(7.0)
        graph.replay()
        want = both()
        torch.cuda.synchronize()
        s = slice(o[0], o[-1])
        for i, (a, b) in enumerate(zip(res, want)):
            if i in (1, 6):  # the states
                assert torch.equal(a, b), (o, i)
            else:
                assert torch.equal(a[:, s], b[:, s]) and (a[:, :o[0]] == 7).all() and (a[:, o[-1]:] == 7).all(), (o, i)
