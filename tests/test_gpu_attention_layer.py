"""The attention layer's operators together, as a model runs them: a prompt's
prefill and decoding over the cache against the whole sequence at once, a training
step through the rotation, and the layer beside a recurrent one.

Tolerance of a row computed in two ways: both are within the tolerances of
test_gpu_attention (o) and test_gpu_cache of the same 64-bit value; with scores of
a few units that is below 2^-13 of the largest |v|, for bf16 keys, stored alike,
as for fp32."""

import numpy as np
import pytest
import torch

import gated_delta_rule_54_amd as gdr
from oracle import attention_oracle as ao
from tests.test_gpu_rotary import BF, F, dev, freqs, host

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("io", [BF, F])
@pytest.mark.parametrize("window,sinks", [(None, 0), (40, 3)])
@pytest.mark.parametrize("heads", [False, True])
def test_prefill_then_tokens(io, window, sinks, heads):
    """17 ragged prompts are appended and attended to; then tokens one by one, the
    cache's layer a captured graph; each row is the row of the whole sequence."""
    Hq, Hk, D, R, size, steps = 4, 2, 64, 32, 16, 6
    r = np.random.default_rng(1)
    prompts = [int(n) for n in r.integers(1, 90, 17)]
    total = [n + steps for n in prompts]
    x = [torch.from_numpy(r.standard_normal((n, Hq + 2 * Hk, D)).astype(np.float32)).to(io) for n in total]
    f = dev(freqs(R))
    most = -(-max(total) // size)
    pages = sum(-(-n // size) for n in total) + 1
    order = iter(r.permutation(pages))
    table = torch.full((17, most), -1, dtype=torch.int32)
    for b, n in enumerate(total):
        for i in range(-(-n // size)):
            table[b, i] = int(next(order))
    table = table.cuda()
    make = lambda: torch.full((pages, Hk, size, D), float("nan"), device="cuda", dtype=io).transpose(1, 2) if heads else \
        torch.full((pages, size, Hk, D), float("nan"), device="cuda", dtype=io)
    kc, vc = make(), make()

    # the whole sequences, without a cache
    cu = dev(np.concatenate([[0], np.cumsum(total)]), torch.int64)
    t = torch.cat(x)[None].cuda()
    pos = torch.cat([torch.arange(n) for n in total])[None].cuda()
    q, k = gdr.gdr_rotary_forward(t[:, :, :Hq], t[:, :, Hq:Hq + Hk], pos, f, out_dtype=io)
    want, lse_want = gdr.gdr_attention_forward(q, k, t[:, :, Hq + Hk:], window=window, sinks=sinks, cu_seqlens=cu,
                                               max_seqlen=max(total))
    rows = [slice(int(cu[b]), int(cu[b + 1])) for b in range(17)]

    # prefill
    cu0 = dev(np.concatenate([[0], np.cumsum(prompts)]), torch.int64)
    p = torch.cat([a[:n] for a, n in zip(x, prompts)])[None].cuda()
    lengths = dev(prompts, torch.int64)
    q0 = gdr.gdr_cache_append(p[:, :, Hq:Hq + Hk], p[:, :, Hq + Hk:], kc, vc, table, lengths, f, q=p[:, :, :Hq],
                              cu_seqlens=cu0, max_seqlen=max(prompts))
    for b, n in enumerate(prompts):
        at = rows[b].start
        assert torch.equal(q0[0, int(cu0[b]):int(cu0[b + 1])], q[0, at:at + n])
        j = torch.arange(n, device="cuda")
        assert torch.equal(kc[table[b].long()[j // size], j % size], k[0, at:at + n])

    # tokens
    step = torch.empty(17, 1, Hq + 2 * Hk, D, device="cuda", dtype=io)

    def layer():
        qs = gdr.gdr_cache_append(step[:, :, Hq:Hq + Hk], step[:, :, Hq + Hk:], kc, vc, table, lengths, f,
                                  q=step[:, :, :Hq])
        return gdr.gdr_cache_attention(qs, kc, vc, table, lengths, window=window, sinks=sinks)

    graph = None
    for s in range(steps):
        lengths += 1
        step.copy_(torch.stack([a[n + s] for a, n in zip(x, prompts)])[:, None])
        if s < 2:
            o, lse = layer()
        else:
            if graph is None:
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph):
                    o, lse = layer()
            graph.replay()
        torch.cuda.synchronize()
        for b, n in enumerate(prompts):
            row = rows[b].start + n + s
            big = float(t[0, rows[b], Hq + Hk:].abs().max())
            assert float((o[b, 0] - want[0, row]).abs().max()) <= 2.0 ** -13 * big
            assert float((lse[b, 0] - lse_want[0, row]).abs().max()) <= 2.0 ** -13


@pytest.mark.parametrize("axes", [1, 3])
def test_training_step_through_the_rotation(axes):
    """Gradients of the raw q and k: rotation, attention, and back, against
    differences of the 64-bit definitions (fp32; the chain's relative error is
    that of its links, below 2^-15 of the gradients' norm)."""
    T, Hq, Hk, D, R = 70, 4, 2, 32, 32
    r = np.random.default_rng(3)
    q, k, v, do = (r.standard_normal(s).astype(np.float32) for s in ((T, Hq, D), (T, Hk, D), (T, Hk, D), (T, Hq, D)))
    pos = np.arange(T) if axes == 1 else r.integers(0, 30, (axes, T))
    sec = None if axes == 1 else (6, 5, 5)
    f = freqs(R)
    how = dict(window=30, sinks=2)
    tp = dev(pos.reshape(pos.shape[:-1] + (1, T)), torch.int64)
    t = [dev(a)[None] for a in (q, k, v, do)]
    qr, kr = gdr.gdr_rotary_forward(t[0], t[1], tp, dev(f), section=sec)
    o, lse = gdr.gdr_attention_forward(qr, kr, t[2], **how)
    dqr, dkr, dv = gdr.gdr_attention_backward(qr, kr, t[2], o, lse, t[3], **how)
    dq, dk = gdr.gdr_rotary_backward(dqr, dkr, tp, dev(f), section=sec, dq=dqr, dk=dkr)
    assert dq is dqr
    rq, rk = ao.rotary(q, pos, f, section=sec), ao.rotary(k, pos, f, section=sec)
    ref = ao.attention_vjp(rq, rk, v, do, D ** -0.5, 30, 2)
    ref = ao.rotary(ref[0], pos, f, section=sec, back=True), ao.rotary(ref[1], pos, f, section=sec, back=True), ref[2]
    for got, want in zip((dq, dk, dv), ref):
        assert np.linalg.norm(host(got)[0] - want) <= 2.0 ** -15 * np.linalg.norm(want)


def test_beside_a_recurrent_layer():
    """A hybrid stack's step in one graph: a linear-attention token and a cached
    attention token from the same projection, replayed as the sequences grow."""
    B, Hk, D, size = 5, 2, 64, 16
    r = np.random.default_rng(4)
    x = dev(r.standard_normal((B, 1, 4 + 2 + 2, D)), BF)
    q, k, v = x[:, :, :4], x[:, :, 4:6], x[:, :, 6:]
    table = torch.arange(B * 4, dtype=torch.int32, device="cuda").reshape(B, 4)
    f = dev(freqs(64))

    def state():
        return (torch.zeros(B, Hk, D, D, device="cuda"), torch.zeros(B * 4, size, Hk, D, device="cuda", dtype=BF),
                torch.zeros(B * 4, size, Hk, D, device="cuda", dtype=BF), torch.zeros(B, dtype=torch.int64, device="cuda"))

    def step(h, kc, vc, n):
        n += 1
        o1, _ = gdr.gdr_linear_forward(k, k, v, None, h, ht=h, out_dtype=BF)
        qs = gdr.gdr_cache_append(k, v, kc, vc, table, n, f, q=q)
        o2, _ = gdr.gdr_cache_attention(qs, kc, vc, table, n, out_dtype=BF, lse=None)
        return o1, o2

    a, b = state(), state()
    step(*state())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        res = step(*a)
    for t in a:
        t.zero_()
    for i in range(40):
        x.copy_(torch.randn_like(x.float()).to(BF))
        g.replay()
        want = step(*b)
        torch.cuda.synchronize()
        assert all(torch.equal(p, w) for p, w in zip(res, want)), i


@pytest.mark.parametrize("io", [BF, F])
def test_last_tokens_of_long_projections(io):
    """One token of each sequence of a long projection: rows far apart."""
    B, T, Hk, D = 3, 9000, 2, 64
    x = torch.randn(B, T, 8, D, device="cuda").to(io)
    kc, vc = (torch.zeros(B * 2, 16, Hk, D, device="cuda", dtype=io) for _ in "kv")
    table = torch.arange(B * 2, dtype=torch.int32, device="cuda").reshape(B, 2)
    n = torch.tensor([17, 3, 32], device="cuda")
    f, last = dev(freqs(D)), x[:, -1:]
    assert last.stride(0) > 1 << 22
    one = [t.clone() for t in (kc, vc)]
    q = gdr.gdr_cache_append(last[:, :, 4:6], last[:, :, 6:], kc, vc, table, n, f, q=last[:, :, :4])
    d = last.contiguous()
    q1 = gdr.gdr_cache_append(d[:, :, 4:6].contiguous(), d[:, :, 6:].contiguous(), *one, table, n, f,
                              q=d[:, :, :4].contiguous())
    assert torch.equal(q, q1) and torch.equal(kc, one[0]) and torch.equal(vc, one[1])
    for a, b in zip(gdr.gdr_cache_attention(last[:, :, :4], kc, vc, table, n),
                    gdr.gdr_cache_attention(d[:, :, :4].contiguous(), kc, vc, table, n)):
        assert torch.equal(a, b)
    y, _ = gdr.gdr_rotary_forward(last[:, :, :4], None, (n - 1)[:, None], f, out_dtype=io)
    assert torch.equal(y, q)


def test_calls_alike_but_for_one_thing():
    """Calls that differ in one shape, stride, type or option, in turn and again: each
    is what it is alone (what a call keeps goes by all of them)."""
    r = torch.Generator(device="cuda").manual_seed(5)
    rn = lambda *s: torch.randn(*s, device="cuda", generator=r)
    q, k, v, do = rn(1, 40, 4, 32), rn(1, 40, 2, 32), rn(1, 40, 2, 32), rn(1, 40, 4, 32)
    wide = rn(1, 40, 3, 32)
    cases = [dict(), dict(window=5), dict(window=5, sinks=1), dict(scale=0.3), dict(sinks=1)]
    seen = []
    for turn in range(2):
        got = []
        for how in cases:
            for kk in (k, wide[:, :, :2]):
                o, lse = gdr.gdr_attention_forward(q, kk, v, **how)
                got += [o, lse, *gdr.gdr_attention_backward(q, kk, v, o, lse, do, **how)]
            o, lse = gdr.gdr_attention_forward(q, k, v, out_dtype=BF, **how)
            got += [o, lse, *gdr.gdr_attention_backward(q, k, v, o, lse, do, **how)]
            assert o.dtype == BF
        seen.append(got)
    assert all(torch.equal(a, b) for a, b in zip(*seen))
    for how, at in zip(cases, range(0, 75, 15)):
        for kk, i in ((k, 0), (wide[:, :, :2], 5)):
            x = [host(t[0]) for t in (q, kk, v)]
            ref, _ = ao.attention(*x, how.get("scale", 32 ** -0.5), how.get("window"), how.get("sinks", 0))
            assert np.abs(host(seen[0][at + i][0]) - ref).max() < 2.0 ** -13 * np.abs(x[2]).max()
    with pytest.raises(ValueError):
        gdr.gdr_attention_forward(q, k, v[:, :39])
    f = dev(freqs(32))
    pos = torch.arange(40, device="cuda")[None]
    a = gdr.gdr_rotary_forward(q, k, pos, f)
    b = gdr.gdr_rotary_forward(q, k, pos, f, adjacent=True)
    c = gdr.gdr_rotary_backward(q, k, pos, f)
    again = gdr.gdr_rotary_forward(q, k, pos, f)
    assert torch.equal(a[0], again[0]) and not torch.equal(a[0], b[0]) and not torch.equal(a[0], c[0])
