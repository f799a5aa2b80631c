"""The paged cache on the GPU: the append, and attention of one token, against
the float64 definitions of oracle/attention_oracle.py.

Tolerances, u = 2^-24.  A score is a sum of D products: off by 2 D u of the sum A
of their absolute values (2: a product and its addition).  It and the maximum
are scaled and subtracted, 4 u of their sizes, and the exponential rounds to 2
units in the last place.  So a weight is off by r = 2 D u A + 4 u (|s| + |m|) + 4 u
of itself, numerator and denominator each; both sum n terms (2 n u), P enters as
24 bits (u), joins scale by exponentials and add (16 u): o is off by (2 r + (2 n
+ 20) u) sum P |v|, lse by r + (2 n + 8) u + u |lse|.  A bf16 output adds 2^-8 of
its value.  Stored keys: see test_gpu_rotary."""

import numpy as np
import pytest
import torch

import gated_delta_rule_54_amd as gdr
from gated_delta_rule_54_amd.synth import round_bf16
from oracle import attention_oracle as ao
from tests.test_gpu_rotary import BF, F, U, dev, freqs, host, pair_sums

pytestmark = pytest.mark.gpu


def randn(r, *shape, io=F):
    x = r.standard_normal(shape).astype(np.float32)
    return round_bf16(x) if io == BF else x


def paged(r, lengths, Hk, D, size, io, heads=False, spare=2, extra=1, bad=()):
    """Caches with a table of pages in random order; what no sequence holds is
    NaN.  bad: (sequence, nth page) that are not there."""
    need = [-(-n // size) for n in lengths]
    pages = sum(need) + spare
    order = list(r.permutation(pages))
    table = np.full((len(lengths), max(need, default=0) + extra), -1, np.int32)
    kc, vc = (np.full((pages, size, Hk, D), np.nan, np.float32) for _ in "kv")
    for b, n in enumerate(lengths):
        for i in range(need[b]):
            page = order.pop()
            table[b, i] = page
            m = min(size, n - i * size)
            kc[page, :m], vc[page, :m] = randn(r, m, Hk, D, io=io), randn(r, m, Hk, D, io=io)
    for j, (b, i) in enumerate(bad):
        table[b, i] = (-1, pages, -2 ** 31, 2 ** 31 - 1)[j % 4]
    on = [dev(c.transpose(0, 2, 1, 3), io).transpose(1, 2) if heads else dev(c, io) for c in (kc, vc)]
    return kc, vc, table, on


def check(lengths, Hq, Hk, D, size=16, io=BF, out=F, heads=False, window=None, sinks=0, scale=None, max_len=None, bad=(),
          seed=1, strided=False):
    r = np.random.default_rng(seed)
    kc, vc, table, (k, v) = paged(r, lengths, Hk, D, size, io, heads, bad=bad)
    B = len(lengths)
    q = randn(r, B, Hq, D, io=io)
    qt = dev(q, io)[:, None]
    if strided:
        row = torch.full((B, 1, Hq + 3, D), float("nan"), device="cuda", dtype=io)
        row[:, :, :Hq] = qt
        qt = row[:, :, :Hq]
    o, lse = gdr.gdr_cache_attention(qt, k, v, dev(table, torch.int32), dev(lengths, torch.int64), scale=scale,
                                     window=window, sinks=sinks, max_len=max_len, out_dtype=out)
    c = D ** -0.5 if scale is None else scale
    ro, rl, got = ao.cache_attention(q, kc, vc, table, lengths, c, window, sinks, max_len)
    assert o.shape == (B, 1, Hq, D) and lse.shape == (B, 1, Hq)
    o, lse = host(o)[:, 0], host(lse)[:, 0]
    for b, at in enumerate(got):
        if not at:
            assert np.all(o[b] == 0) and np.all(np.isneginf(lse[b]))
            continue
        p, s = (list(x) for x in zip(*at))
        n = len(p)
        for h in range(Hq):
            kk, vv = (x[p, s, h // (Hq // Hk)].astype(np.float64) for x in (kc, vc))
            S, A = c * kk @ q[b, h], c * np.abs(kk) @ np.abs(q[b, h])
            rel = np.max(2 * D * U * A + 4 * U * (np.abs(S) + np.abs(S).max()) + 4 * U)
            P = np.exp(S - rl[b, h])
            tol = (2 * rel + (2 * n + 20) * U) * (P @ np.abs(vv))
            if out == BF:
                tol = tol + 2.0 ** -8 * (np.abs(ro[b, h]) + tol)
            assert np.all(np.abs(o[b, h] - ro[b, h]) <= tol), (b, h)
            assert abs(lse[b, h] - rl[b, h]) <= rel + (2 * n + 8) * U + U * abs(rl[b, h]), (b, h)


@pytest.mark.parametrize("D", [16, 48, 64, 80, 128, 144, 192, 256])
@pytest.mark.parametrize("io,out", [(BF, F), (BF, BF), (F, F), (F, BF)])
def test_widths_and_types(D, io, out):
    check([37, 1, 16, 0, 700], 4, 2, D, io=io, out=out)


@pytest.mark.parametrize("Hq,Hk", [(1, 1), (3, 3), (8, 2), (16, 1), (17, 1), (40, 2), (6, 2)])
@pytest.mark.parametrize("io", [BF, F])
def test_head_groups(Hq, Hk, io):
    check([300, 5, 33], Hq, Hk, 64, io=io)


@pytest.mark.parametrize("size", [1, 7, 16, 31, 48, 64, 128, 1024])
@pytest.mark.parametrize("heads", [False, True])
def test_pages(size, heads):
    check([1, size, size + 1, 3 * size - 1, 200], 4, 2, 64, size=size, heads=heads)
    check([1, size, size + 1, 3 * size - 1, 200], 4, 2, 96, size=size, heads=heads, io=F)


@pytest.mark.parametrize("lengths", [[15], [31], [32], [33], [127], [128], [129], [255], [256], [257], [1023], [4097],
                                     [0], [0, 0, 5], [2 ** 14 + 3]])
def test_lengths(lengths):
    check(lengths, 4, 2, 64, size=32)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (31, 0), (32, 4), (100, 77), (257, 1), (699, 1), (700, 3),
                                          (5000, 9), (64, 5000)])
@pytest.mark.parametrize("io", [BF, F])
def test_windows(window, sinks, io):
    check([700, 50, 100, 1, 0, 257], 4, 2, 64, size=48, io=io, window=window, sinks=sinks)


def test_pages_that_are_not_there():
    """Evicted pages (behind the window and in it), whole sequences of them, and
    entries that name no page of the cache."""
    check([200, 64, 100, 20], 4, 2, 64, bad=[(0, 0), (0, 5), (0, 12), (2, 3), (2, 4), (3, 0), (3, 1), (1, 2)])
    check([200, 64, 100, 20], 4, 2, 64, io=F, window=40, sinks=3, bad=[(0, 4), (0, 3), (2, 0), (3, 0), (3, 1)])
    check([5000], 4, 2, 64, size=64, bad=[(0, i) for i in range(0, 70, 3)])


def test_max_len_scale_and_strides():
    check([700, 300, 5], 4, 2, 64, max_len=320, scale=0.03)
    check([700, 300, 5], 4, 2, 128, scale=2.0, strided=True)
    check([700, 300, 5], 8, 2, 64, strided=True, io=F)


def test_many_sequences():
    check(list(np.random.default_rng(9).integers(0, 90, 700)), 2, 1, 32)


@pytest.mark.parametrize("io,D", [(BF, 64), (BF, 256), (F, 48)])
def test_more_sequences_than_the_card_holds_pieces(io, D):
    """Cut, with more pieces than the card holds at once; one sequence far longer than
    the others, and empty ones."""
    r = np.random.default_rng(12)
    lengths = [int(n) for n in r.integers(0, 120, 290)]
    lengths[7], lengths[8:12] = 5000, [0, 64, 65, 0]
    check(lengths, 4, 2, D, io=io)
    check(lengths, 4, 2, D, io=io, window=70, sinks=3)


def test_large_scores():
    """A softmax that is nearly one key: weights over many decades."""
    check([900, 77], 4, 2, 64, scale=3.0, out=BF)
    check([900, 77], 4, 2, 64, scale=3.0, io=F)


def test_infinities_and_nan():
    r = np.random.default_rng(4)
    kc, vc, table, (k, v) = paged(r, [40, 40, 40, 40], 1, 64, 16, F)
    q = randn(r, 4, 1, 64)
    q[:, :, 0] = 1.0

    def at(c, b, j):
        return c[table[b, j // 16], j % 16, 0]

    at(k, 0, 5)[0] = float("inf")    # a score of +Inf
    at(k, 1, 5)[0] = -float("inf")   # a key with no weight
    at(k, 2, 5)[0] = float("nan")
    at(v, 3, 5)[0] = float("nan")
    o, lse = gdr.gdr_cache_attention(dev(q)[:, None], k, v, dev(table, torch.int32), torch.full((4,), 40, device="cuda"))
    o, lse = host(o)[:, 0, 0], host(lse)[:, 0, 0]
    assert np.all(np.isnan(o[0])) and np.all(np.isnan(o[2])) and np.isnan(lse[2])
    assert np.all(np.isfinite(o[1])) and np.isfinite(lse[1])
    assert np.isnan(o[3, 0]) and np.all(np.isfinite(o[3, 1:])) and np.isfinite(lse[3])
    kc[table[1, 0], 5, 0, 0] = -1e30
    ref, rl, _ = ao.cache_attention(q[1:2], kc, vc, table[1:2], [40], 0.125)
    assert np.allclose(o[1], ref[0, 0], atol=1e-4) and abs(lse[1] - rl[0, 0]) < 1e-4
    k[:] = float("-inf")  # no score at all
    o, lse = gdr.gdr_cache_attention(dev(np.abs(q))[:, None], k, v, dev(table, torch.int32),
                                     torch.full((4,), 40, device="cuda"))
    assert torch.all(torch.isneginf(lse)) and torch.all(o[:3] == 0)


@pytest.mark.parametrize("io", [BF, F])
def test_same_bits_twice_replayed_and_elsewhere(io):
    """Twice, on another stream, and from a graph whose lengths, table, q and
    pages change between replays."""
    r = np.random.default_rng(5)
    lengths = [3000, 17, 0, 900]
    _, _, table, (k, v) = paged(r, lengths, 2, 64, 32, io, extra=3)
    q, t, n = dev(randn(r, 4, 1, 8, 64), io), dev(table, torch.int32), dev(lengths, torch.int64)
    call = lambda: gdr.gdr_cache_attention(q, k, v, t, n, window=1000, sinks=4)
    one = call()
    assert all(torch.equal(a, b) for a, b in zip(one, call()))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = gdr.gdr_cache_attention(q, k, v, t, n, window=1000, sinks=4, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(one, other))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        res = call()
    for i in range(4):
        n.copy_(torch.tensor([3000 - 700 * i, 17 - i, 0, 900 - 899 * (i == 2)]))
        q.copy_(torch.randn_like(q.float()).to(io))
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(res, call()))


def test_two_streams_at_once():
    r = np.random.default_rng(6)
    sets = []
    for i in range(2):
        _, _, table, (k, v) = paged(r, [2000 - 500 * i, 90], 2, 64, 16, BF)
        sets.append((dev(randn(r, 2, 1, 4, 64), BF), k, v, dev(table, torch.int32), dev([2000 - 500 * i, 90], torch.int64)))
    want = [gdr.gdr_cache_attention(*s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [[], []]
    for _ in range(5):
        for i in range(2):
            got[i].append(gdr.gdr_cache_attention(*sets[i], stream=streams[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(a, b) for res in got[i] for a, b in zip(res, want[i]))


def test_refusals_of_cache_attention():
    r = np.random.default_rng(7)
    _, _, table, (k, v) = paged(r, [40, 9], 2, 64, 16, BF)
    q, t, n = dev(randn(r, 2, 1, 4, 64), BF), dev(table, torch.int32), dev([40, 9], torch.int64)
    call = gdr.gdr_cache_attention
    for bad in (lambda: call(q[:, 0], k, v, t, n), lambda: call(q[:1], k, v, t, n), lambda: call(q, k, v[:-1], t, n),
                lambda: call(q, k, v, t, n[:1]), lambda: call(q, k, v, t, n, window=0), lambda: call(q, k, v, t, n, sinks=-1),
                lambda: call(q, k, v, t, n, max_len=0), lambda: call(q, k, v, t.cpu(), n),
                lambda: call(q, k, v, t, n, o=torch.empty(2, 1, 4, 32, device="cuda"))):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: call(q.float(), k, v, t, n), lambda: call(q, k, v, t.long(), n), lambda: call(q, k, v, t, n.int()),
                lambda: call(q, k.half(), v.half(), t, n)):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: call(q[:, :, :3], k, v, t, n), lambda: call(q, k, v, t, n, max_len=10 ** 6),
                lambda: call(q, k, v, t, n, scale=0.0)):
        with pytest.raises(gdr.GdrError):
            bad()


# ---- the append -----------------------------------------------------------

def check_append(lengths, new, Hq, Hk, D, R, size=16, io=BF, cd=BF, heads=False, ragged=False, pos=None, bad=(), seed=2,
                 gap=0, T=None, **turn):
    r = np.random.default_rng(seed)
    kc, vc, table, on = paged(r, lengths, Hk, D, size, cd, heads, bad=bad)
    kc, vc = np.nan_to_num(kc, nan=7.0), np.nan_to_num(vc, nan=7.0)
    for c, h in zip(on, (kc, vc)):
        c.copy_(dev(h, cd))
    if ragged:
        cu = np.concatenate([[gap], gap + np.cumsum(new)])
        rows, first = int(cu[-1]) + gap, list(cu[:-1])
    else:
        rows, first = len(new) * new[0], [i * new[0] for i in range(len(new))]
    x = randn(r, rows, Hq + 2 * Hk, D, io=io)
    t = dev(x, io).reshape((1, rows, Hq + 2 * Hk, D) if ragged else (len(new), new[0], Hq + 2 * Hk, D))
    q, k, v = t[:, :, :Hq], t[:, :, Hq:Hq + Hk], t[:, :, Hq + Hk:]
    freq = freqs(R) if R else None
    qo = torch.full(t.shape[:2] + (Hq, D), 5.0, device="cuda", dtype=cd) if Hq else None
    p = None if pos is None else dev(pos.reshape(pos.shape[:-1] + t.shape[:2]), torch.int64)
    got = gdr.gdr_cache_append(k, v, *on, dev(table, torch.int32), dev(lengths, torch.int64),
                               None if freq is None else dev(freq), p, q=q if Hq else None, q_out=qo,
                               cu_seqlens=dev(cu, torch.int64) if ragged else None, max_seqlen=T, **turn)
    assert got is qo
    kept = [(f, n) for f, n in zip(first, new)]
    rk, rv = ao.append(kc, vc, table, lengths, kept, x[:, Hq:Hq + Hk], x[:, Hq + Hk:], freq, pos, **turn)
    far = (max(lengths) if pos is None else int(np.abs(pos).max())) + 1
    # what is stored: turned keys, values as they are (rounded where the cache is narrower)
    sums, _ = ao.append(np.zeros_like(kc), vc, table, lengths, kept, pair_sums(x[:, Hq:Hq + Hk], R, turn.get("adjacent", False)),
                        x[:, Hq + Hk:])
    tol = sums * ((np.pi + 7) * U + 2.0 ** -52 * far)
    rnd = 2.0 ** -8 if cd == BF else 0.0
    changed = np.any(rk != kc, axis=-1, keepdims=True)
    assert np.all(np.abs(host(on[0]) - rk) <= np.where(changed, tol + rnd * (np.abs(rk) + tol), 0.0))
    assert np.array_equal(host(on[1]), host(torch.from_numpy(rv).to(cd)))
    if Hq:
        ref = np.full((rows, Hq, D), 5.0)
        for b, (f, n) in enumerate(kept):
            at = np.arange(lengths[b] - n, lengths[b]) if pos is None else pos[..., f:f + n]
            xq = x[f:f + n, :Hq]
            ref[f:f + n] = xq if freq is None else ao.rotary(xq, at, freq, **turn)
        tol = pair_sums(x[:, :Hq], R, turn.get("adjacent", False)) * ((np.pi + 7) * U + 2.0 ** -52 * far)
        assert np.all(np.abs(host(qo).reshape(ref.shape) - ref) <= tol + rnd * (np.abs(ref) + tol))


@pytest.mark.parametrize("io,cd", [(BF, BF), (F, F), (F, BF), (BF, F)])
@pytest.mark.parametrize("Hq,Hk,D,R", [(4, 2, 64, 64), (1, 1, 16, 16), (3, 3, 96, 32), (8, 2, 256, 64), (0, 2, 128, 128),
                                       (5, 1, 80, 0)])
def test_append_types_and_heads(Hq, Hk, D, R, io, cd):
    check_append([40, 1, 17], [1, 1, 1], Hq, Hk, D, R, io=io, cd=cd)
    check_append([40, 7, 17], [7, 7, 7], Hq, Hk, D, R, io=io, cd=cd, heads=True)


@pytest.mark.parametrize("size", [1, 5, 16, 64])
@pytest.mark.parametrize("gap", [0, 3])
def test_append_ragged(size, gap):
    check_append([40, 0, 17, 300, 64, 1], [40, 0, 5, 299, 64, 1], 4, 2, 64, 32, size=size, ragged=True, gap=gap)


def test_append_many_sequences():
    r = np.random.default_rng(8)
    new = list(r.integers(0, 4, 600))
    check_append([int(n + r.integers(0, 30)) for n in new], new, 2, 1, 32, 32, ragged=True, io=F, cd=F)
    check_append([int(n) for n in r.integers(1, 99, 700)], [1] * 700, 2, 1, 32, 32)


def test_append_positions_and_axes():
    r = np.random.default_rng(9)
    check_append([40, 9], [8, 8], 4, 2, 64, 64, pos=r.integers(0, 100000, 16))
    check_append([40, 9], [8, 8], 4, 2, 64, 64, pos=r.integers(0, 999, (3, 16)), section=(16, 8, 8), cycled=True)
    check_append([40, 9], [8, 8], 4, 2, 64, 48, pos=r.integers(0, 999, (2, 16)), section=(10, 14), adjacent=True)
    check_append([40, 9], [20, 9], 4, 2, 64, 64, pos=r.integers(0, 999, 29), ragged=True)


def test_append_without_a_place():
    """Tokens before the sequence's start, past the table, on pages that are not
    there, and past the bound on new tokens: not stored; q is turned all the same
    where the token is one of the call's."""
    check_append([40, 3, 90], [8, 8, 8], 4, 2, 64, 64, bad=[(0, 2), (2, 5)])
    r = np.random.default_rng(10)
    _, _, table, (k, v) = paged(r, [64, 64], 1, 32, 16, F, extra=0)
    k.zero_(), v.zero_()
    x = dev(randn(r, 2, 20, 1, 32))
    gdr.gdr_cache_append(x, x, k, v, dev(table, torch.int32), dev([74, 5], torch.int64))
    for b, n in ((0, 74), (1, 5)):
        for t in range(20):
            at = n - 20 + t
            if 0 <= at < 64:
                assert torch.equal(v[table[b, at // 16], at % 16], x[b, t])
    assert int((v != 0).any(-1).sum()) == 10 + 5
    k.zero_(), v.zero_()
    cu = dev([0, 12, 20], torch.int64)
    gdr.gdr_cache_append(x[:1], x[:1], k, v, dev(table, torch.int32), dev([12, 8], torch.int64), cu_seqlens=cu, max_seqlen=9)
    assert int((v != 0).any(-1).sum()) == 9 + 8


def test_append_captured_and_replayed():
    """A decoding step whose lengths grow between replays."""
    r = np.random.default_rng(11)
    _, _, table, (k, v) = paged(r, [60, 60, 60], 2, 64, 16, BF)
    k.zero_(), v.zero_()
    k2, v2 = k.clone(), v.clone()
    x, n, t = dev(randn(r, 3, 1, 8, 64), BF), dev([1, 7, 30], torch.int64), dev(table, torch.int32)
    f = dev(freqs(64))
    call = lambda kc, vc: gdr.gdr_cache_append(x[:, :, 4:6], x[:, :, 6:], kc, vc, t, n, f, q=x[:, :, :4])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        q = call(k, v)
    for _ in range(5):
        g.replay()
        torch.cuda.synchronize()
        want = call(k2, v2)
        assert torch.equal(q, want) and torch.equal(k, k2) and torch.equal(v, v2)
        n += 1
        x.copy_(torch.randn_like(x.float()).to(BF))


def test_refusals_of_the_append():
    r = np.random.default_rng(12)
    _, _, table, (k, v) = paged(r, [40, 9], 2, 64, 16, BF)
    x, t, n = dev(randn(r, 2, 3, 2, 64), BF), dev(table, torch.int32), dev([40, 9], torch.int64)
    f = dev(freqs(64))
    call = gdr.gdr_cache_append
    for bad in (lambda: call(x[:1], x[:1], k, v, t, n), lambda: call(x, x[:, :2], k, v, t, n), lambda: call(x[0], x[0], k, v, t, n),
                lambda: call(x, x, k, v, t, n, f, torch.zeros(6, dtype=torch.int64, device="cuda")),
                lambda: call(x, x, k, v, t, n, f, section=(16, 16)), lambda: call(x, x, k, v, t, n, f, q_out=x),
                lambda: call(x, x, k, v, t, n, cu_seqlens=torch.tensor([0, 3, 6], device="cuda")),
                lambda: call(x[:, :1].expand(2, 3, 2, 64), x, k, v, t, n)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        call(x, x.float(), k, v, t, n)
    with pytest.raises(TypeError):
        call(x, x, k, v, t, n, f, q=x, q_out=torch.empty(2, 3, 2, 64, device="cuda"))
