"""The attention layer where offsets pass 32 bits (elements and bytes), sequences
are long, or many calls share what they can: against cuts whose result is the same.

Under a window a far token's row depends on the last few tokens (and the sinks)
alone, so the last rows of a long sequence are those of a short one with the same
tokens; tolerances are those of sums cut otherwise, 2^-16 of the largest value in
fp32 outputs (see test_gpu_attention), and half a step of bf16 either way."""

import numpy as np
import pytest
import torch

import gated_delta_rule_54_amd as gdr
from tests.test_gpu_rotary import BF, F, close, dev, freqs, host

pytestmark = pytest.mark.gpu


def randn(seed, *shape, dtype=BF):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.empty(shape, dtype=dtype, device="cuda")
    for piece in x.view(-1).split(1 << 28):
        piece.copy_(torch.randn(piece.numel(), device="cuda", generator=g))
    return x


def same(a, b):
    a, b = a.float(), b.float()
    assert torch.isfinite(a).all()
    assert ((a - b).abs() <= 2.0 ** -7 * b.abs() + 2.0 ** -16 * b.abs().max()).all()


def test_attention_past_32_bits():
    """A batch of 2.3e9 elements: its last sequence alone."""
    B, T, Hq, Hk, D = 9, 60_000, 32, 2, 128
    q, k, v = randn(1, B, T, Hq, D), randn(2, B, T, Hk, D), randn(3, B, T, Hk, D)
    how = dict(window=100, sinks=3)
    o, lse = gdr.gdr_attention_forward(q, k, v, out_dtype=BF, **how)
    o1, lse1 = gdr.gdr_attention_forward(q[-1:], k[-1:], v[-1:], out_dtype=BF, **how)
    assert torch.equal(o[-1:], o1) and torch.equal(lse[-1:], lse1)
    do = q  # any gradient
    dq, dk, dv = gdr.gdr_attention_backward(q, k, v, o, lse, do, **how)
    one = gdr.gdr_attention_backward(q[-1:], k[-1:], v[-1:], o1, lse1, do[-1:], **how)
    assert torch.equal(dq[-1:], one[0])
    same(dk[-1:], one[1])
    same(dv[-1:], one[2])


def test_a_long_sequence_under_a_window():
    """300,000 tokens: the last rows against a short sequence of the sinks and the
    last tokens (placed as they lie: the sinks first), and the middle's gradients."""
    T, Hq, Hk, D, W, S = 300_000, 4, 2, 64, 200, 5
    x = [randn(10 + i, 1, T, H, D) for i, H in enumerate((Hq, Hk, Hk, Hq))]
    q, k, v, do = x
    o, lse = gdr.gdr_attention_forward(q, k, v, window=W, sinks=S)
    near = 2 * W
    cut = [torch.cat([t[:, :S], t[:, -near:]], 1) for t in x]
    o1, lse1 = gdr.gdr_attention_forward(*cut[:3], window=W, sinks=S)
    same(o[:, -W:], o1[:, -W:])
    assert ((lse[:, -W:] - lse1[:, -W:]).abs() <= 2.0 ** -16 * (1 + lse1[:, -W:].abs())).all()
    dq, dk, dv = gdr.gdr_attention_backward(q, k, v, o, lse, do, window=W, sinks=S)
    one = gdr.gdr_attention_backward(*cut[:3], o1, lse1, cut[3], window=W, sinks=S)
    same(dq[:, -W:], one[0][:, -W:])
    same(dk[:, -W:], one[1][:, -W:])
    same(dv[:, -W:], one[2][:, -W:])
    # a sink is seen by every token: its gradients from the definition, summed in 64 bits
    for h in range(Hk):
        qs, ds, os_ = (t[0, :, 2 * h:2 * h + 2].double() for t in (q, do, o))
        P = torch.exp(qs @ k[0, :S, h].double().T / 8 - lse[0, :, 2 * h:2 * h + 2].double()[..., None])
        P[:S] *= torch.ones(S, S, device="cuda").tril()[:, None]
        want = torch.einsum("tgs,tgd->sd", P, ds)
        size = torch.einsum("tgs,tgd->sd", P, ds.abs())
        assert ((dv[0, :S, h].double() - want).abs() <= 2.0 ** -13 * size).all()
        dS = P * (ds @ v[0, :S, h].double().T - (ds * os_).sum(-1, keepdim=True))
        want = torch.einsum("tgs,tgd->sd", dS, qs) / 8
        size = torch.einsum("tgs,tgd->sd", dS.abs(), qs.abs()) / 8
        assert ((dk[0, :S, h].double() - want).abs() <= 2.0 ** -13 * size).all()


def test_cache_past_32_bits():
    """A cache of 5.4e9 elements each for keys and values: tokens in its last pages."""
    pages, size, Hk, D = 20_600, 512, 4, 128
    k, v = (torch.zeros(pages, size, Hk, D, dtype=BF, device="cuda") for _ in "kv")
    table = torch.arange(pages - 1, pages - 9, -1, dtype=torch.int32, device="cuda").reshape(2, 4)
    n = torch.tensor([1900, 700], device="cuda")
    f = dev(freqs(D))
    new = randn(20, 2, 700, 8 + 2 * Hk, D)
    q, x, y = new[:, :, :8], new[:, :, 8:8 + Hk], new[:, :, 8 + Hk:]
    qo = gdr.gdr_cache_append(x, y, k, v, table, n, f, q=q)
    near = [c[-8:].clone() for c in (k, v)]
    assert int((k[:-8].view(torch.int16) != 0).sum()) == 0
    small = (table - (pages - 8)).to(torch.int32)
    o, lse = gdr.gdr_cache_attention(qo[:, -1:], k, v, table, n, window=690)
    o1, lse1 = gdr.gdr_cache_attention(qo[:, -1:], *near, small, n, window=690)
    assert torch.equal(o, o1) and torch.equal(lse, lse1) and torch.isfinite(o).all() and (o != 0).any()
    for b, m in ((0, 1900), (1, 700)):
        j = torch.arange(m - 700, m, device="cuda")
        assert torch.equal(v[table[b].long()[j // size], j % size], y[b])
        close(k[table[b].long()[j[::70] // size], j[::70] % size], host(x[b, ::70]), host(j[::70]).astype(np.int64), freqs(D), BF)


def test_a_long_cache_of_short_pages():
    """2^20 tokens in pages of one token."""
    T, Hk, D = 1 << 20, 1, 64
    k, v = randn(30, T, 1, Hk, D), randn(31, T, 1, Hk, D)
    order = torch.randperm(T, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    table = order.to(torch.int32)[None]
    q = randn(32, 1, 1, 4, D)
    n = torch.tensor([T - 5], device="cuda")
    o, lse = gdr.gdr_cache_attention(q, k, v, table, n)
    kk, vv = k[order[:T - 5], 0, 0].double(), v[order[:T - 5], 0, 0].double()
    S = q[0, 0].double() @ kk.T / 8
    want = torch.softmax(S, -1) @ vv
    size = torch.softmax(S, -1) @ vv.abs()
    # sums of 2^20 terms over 256 pieces of 4 waves: 2^10 to a sum, and the scores' error
    assert ((o[0, 0].double() - want).abs() <= 2.0 ** -12 * size).all()
    assert (lse[0, 0].double() - torch.logsumexp(S, -1)).abs().max() <= 2.0 ** -12


def test_rotary_past_32_bits():
    """4.4e9 elements: the last rows."""
    rows, H, D = 1_080_000, 32, 128
    x = randn(40, rows, H, D)
    pos = torch.arange(rows, device="cuda")
    y, _ = gdr.gdr_rotary_forward(x, None, pos, dev(freqs(D)), out_dtype=BF)
    close(y[-5:], host(x[-5:]), np.arange(rows - 5, rows), freqs(D), BF)
    z, _ = gdr.gdr_rotary_backward(y, None, pos, dev(freqs(D)), dq=y)
    assert z is y and ((y[-5:].float() - x[-5:].float()).abs() <= 2.0 ** -6 * x[-5:].float().abs().amax()).all()


def test_rotary_of_many_rows():
    """More rows than a launch of one workgroup for each two can have."""
    rows = 17_000_001
    x = randn(41, rows, 1, 16)
    pos = torch.arange(rows, device="cuda") % 1000
    y, _ = gdr.gdr_rotary_forward(x, None, pos, dev(freqs(16)), out_dtype=BF)
    for at in (slice(0, 9), slice(8388600, 8388620), slice(rows - 9, rows)):
        close(y[at], host(x[at]), host(pos[at]).astype(np.int64), freqs(16), BF)
    small, _ = gdr.gdr_rotary_forward(x[-1000:], None, pos[-1000:], dev(freqs(16)), out_dtype=BF)
    assert torch.equal(y[-1000:], small)


def test_two_graphs_of_one_pool():
    """Two captured training steps and a decoding step that share a memory pool,
    replayed in turn with other inputs and eager calls between."""
    q, k, v, do = (randn(50 + i, 1, 500, H, 64) for i, H in enumerate((4, 2, 2, 4)))
    kc, vc = randn(60, 40, 16, 2, 64), randn(61, 40, 16, 2, 64)
    table = torch.arange(40, dtype=torch.int32, device="cuda").reshape(1, 40)
    n = torch.tensor([600], device="cuda")

    def train(window):
        o, lse = gdr.gdr_attention_forward(q, k, v, window=window, sinks=2)
        return (o, lse) + gdr.gdr_attention_backward(q, k, v, o, lse, do, window=window, sinks=2)

    calls = [lambda: train(60), lambda: train(None), lambda: gdr.gdr_cache_attention(q[:, :1], kc, vc, table, n)]
    for c in calls:
        c()
    torch.cuda.synchronize()
    graphs, pool = [], None
    for c in calls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, pool=pool):
            res = c()
        pool = pool or g.pool()
        graphs.append((g, res))
    for i in range(3):
        for t in (q, k, v, do):
            t.copy_(torch.randn_like(t.float()))
        n.fill_(600 - 250 * i)
        for (g, res), c in zip(graphs, calls):
            g.replay()
            torch.cuda.synchronize()
            got = [r.clone() for r in res]
            assert all(torch.equal(a, b) for a, b in zip(got, c()))
