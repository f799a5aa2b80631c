"""Linear attention with a decay for each head on the GPU, against the float64
recurrence of oracle/linear_oracle.py.

Tolerances.  Every result is a sum of products; ``forward_abs`` /
``backward_abs`` give the same sums over absolute values, A.  A sum formed in
fp32 through n roundings is off by at most n 2^-24 A, and, the roundings'
signs being independent, by about sqrt(n) 2^-24 A in the 2-norm; n counts the
products' width, the tokens (each decays and adds: at most 4 roundings) and 64
for exponentials.  A bf16 output is rounded once more (2^-8 of its value) and
may come from matrix-core operands rounded to bf16, one per product (2^-8 A).
"""

import numpy as np
import pytest
import torch

import gated_delta_rule_54_amd as gdr
from gated_delta_rule_54_amd.synth import round_bf16
from oracle import linear_oracle as lo

pytestmark = pytest.mark.gpu

NAMES = ("dq", "dk", "dv", "dg", "dh0")
BF, F = torch.bfloat16, torch.float32


def draw(seed, B, T, Hk, Hv, Dk, Dv, io=BF, gate="token", state=True, strength=1.0):
    r = np.random.default_rng(seed)
    n = lambda *s: r.standard_normal(s).astype(np.float32)
    x = dict(q=n(B, T, Hk, Dk) * Dk ** -0.5, k=n(B, T, Hk, Dk), v=n(B, T, Hv, Dv), do=n(B, T, Hv, Dv))
    x = {a: round_bf16(t) if io == BF else t for a, t in x.items()}
    rate = 2.0 ** -np.linspace(0, 7, Hv).astype(np.float32)
    if gate == "token":
        x["g"] = -(strength * rate * np.logaddexp(0, n(B, T, Hv))).astype(np.float32)
    else:
        x["g"] = -strength * rate if gate == "head" else None
    x["h0"] = 0.5 * n(B, Hv, Dk, Dv) if state else None
    x["dht"] = 0.3 * n(B, Hv, Dk, Dv) if state else None
    return x


def to_dev(x, io):
    return {a: None if t is None else torch.from_numpy(np.ascontiguousarray(t)).cuda().to(
        io if a in ("q", "k", "v", "do") else F) for a, t in x.items()}


def host(t):
    return t.detach().double().cpu().numpy()


def close(name, got, ref, A, n, out):
    got = host(got) if isinstance(got, torch.Tensor) else got
    assert got.shape == ref.shape, name
    if ref.size == 0:
        return
    err = np.abs(got - ref)
    tol = n * 2.0 ** -24 * A + 1e-30
    if out == BF:
        tol = tol + 2.0 ** -8 * (A + np.abs(ref) + tol)
    worst = float(np.max(err / tol))
    print(f"  {name}: {worst:.3f} of the bound, max error {err.max():.2e}")
    assert np.isfinite(got).all() and worst <= 1.0, (name, worst)
    if out == F:
        two = np.linalg.norm(err) / (4 * np.sqrt(n) * 2.0 ** -24 * np.linalg.norm(A) + 1e-30)
        assert two <= 1.0, (name, "2-norm", two)


def check(x, io, out, algo, **kw):
    B, T, Hk, Dk = x["q"].shape
    Dv = x["v"].shape[3]
    t = to_dev(x, io)
    o, ht = gdr.gdr_linear_forward(t["q"], t["k"], t["v"], t["g"], t["h0"], algo=algo, out_dtype=out, **kw)
    got = gdr.gdr_linear_backward(t["q"], t["k"], t["v"], t["g"], t["h0"], t["do"], t["dht"], algo=algo,
                                  out_dtype=out, **kw)
    torch.cuda.synchronize()
    verify(x, out, o, ht, got)


def verify(x, out, o, ht, got):
    T, Dk, Dv = x["q"].shape[1], x["q"].shape[3], x["v"].shape[3]
    group = x["v"].shape[2] // x["q"].shape[2]
    args = x["q"], x["k"], x["v"], x["g"], x["h0"]
    n = max(Dk, Dv) + 4 * T + 64 + group
    ro, rht = lo.forward(*args)
    ao, aht = lo.forward_abs(*args)
    close("o", o, ro, ao, n, out)
    close("ht", ht, rht, aht, n, F)
    ref = lo.backward(*args, x["do"], x["dht"])
    A = lo.backward_abs(*args, x["do"], x["dht"])
    for name, a, r, s in zip(NAMES, got, ref, A):
        if r is None:
            assert a is None
            continue
        close(name, a, r, s, 2 * n if name == "dg" else n, F if name in ("dg", "dh0") else out)


ALGOS = ("sequential", "chunked")


@pytest.mark.parametrize("algo", ALGOS)
@pytest.mark.parametrize("T", [1, 2, 63, 64, 65, 200])
def test_lengths(algo, T):
    check(draw(T, 2, T, 2, 4, 128, 128), BF, BF, algo)


@pytest.mark.parametrize("algo", ALGOS)
@pytest.mark.parametrize("Dk,Dv", [(16, 16), (64, 64), (64, 128), (128, 64), (96, 80), (32, 48), (256, 128), (144, 256)])
def test_widths(algo, Dk, Dv):
    check(draw(Dk + Dv, 1, 97, 2, 2, Dk, Dv), BF, F, algo)


@pytest.mark.parametrize("algo", ALGOS)
@pytest.mark.parametrize("io,out", [(BF, BF), (BF, F), (F, F), (F, BF)])
@pytest.mark.parametrize("gate", ["token", "head", "none"])
def test_types_and_gates(algo, io, out, gate):
    check(draw(5, 2, 131, 2, 2, 64, 64, io, gate, state=gate != "none"), io, out, algo)


@pytest.mark.parametrize("algo", ALGOS)
@pytest.mark.parametrize("Hk,Hv", [(1, 1), (1, 4), (2, 6), (3, 3), (1, 8)])
def test_head_groups(algo, Hk, Hv):
    check(draw(Hv, 1, 70, Hk, Hv, 64, 128), BF, BF, algo)


@pytest.mark.parametrize("algo", ALGOS)
@pytest.mark.parametrize("gate", ["token", "head"])
def test_long(algo, gate):
    """Past several segments of the chunked path, in 32-bit outputs."""
    check(draw(11, 1, 1500, 1, 2, 64, 64, BF, gate), BF, F, algo)


@pytest.mark.parametrize("algo", ALGOS)
@pytest.mark.parametrize("io", [BF, F])
def test_strong_decay_and_resets(algo, io):
    """Gates from nearly zero to far below e^-100, and -Inf (the state is
    dropped) inside a chunk, at its first and at its last token."""
    x = draw(12, 1, 150, 2, 2, 64, 64, io, strength=40.0)
    x["g"][:, [0, 37, 63, 64, 100], 0] = -np.inf
    x["g"][:, 80:90, 1] = -3e4
    check(x, io, F, algo)


@pytest.mark.parametrize("algo", ALGOS)
def test_missing_operands(algo):
    x = draw(13, 2, 77, 2, 2, 64, 64, state=False)
    t = to_dev(x, BF)
    o, ht = gdr.gdr_linear_forward(t["q"], t["k"], t["v"], t["g"], algo=algo, out_dtype=F, ht=None)
    assert ht is None
    got = gdr.gdr_linear_backward(t["q"], t["k"], t["v"], t["g"], None, t["do"], algo=algo, out_dtype=F,
                                  want_dg=False, want_dh0=False)
    assert got[3] is None and got[4] is None
    full = gdr.gdr_linear_backward(t["q"], t["k"], t["v"], t["g"], None, t["do"], algo=algo, out_dtype=F)
    _, ht = gdr.gdr_linear_forward(t["q"], t["k"], t["v"], t["g"], algo=algo, out_dtype=F)
    verify(x, F, o, ht, full)
    verify(x, F, o, ht, got[:3] + full[3:])


@pytest.mark.parametrize("algo", ALGOS)
@pytest.mark.parametrize("io", [BF, F])
def test_strided_rows(algo, io):
    """q, k, v as column ranges of one projection, the v range behind a gap."""
    x = draw(14, 2, 90, 2, 4, 64, 64, io)
    t = to_dev(x, io)
    B, T = 2, 90
    row = torch.full((B, T, 128 + 128 + 32 + 256 + 8), float("nan"), dtype=io, device="cuda")
    views = {"q": row[..., :128].unflatten(-1, (2, 64)), "k": row[..., 128:256].unflatten(-1, (2, 64)),
             "v": row[..., 288:544].unflatten(-1, (4, 64))}
    for n, v in views.items():
        v.copy_(t[n])
    a = dict(algo=algo, out_dtype=F)
    o, ht = gdr.gdr_linear_forward(views["q"], views["k"], views["v"], t["g"], t["h0"], **a)
    got = gdr.gdr_linear_backward(views["q"], views["k"], views["v"], t["g"], t["h0"], t["do"], t["dht"], **a)
    verify(x, F, o, ht, got)
    ro, rht = gdr.gdr_linear_forward(t["q"], t["k"], t["v"], t["g"], t["h0"], **a)
    assert torch.equal(o, ro) and torch.equal(ht, rht)
    # a single token of each sequence: the rows are the batch's
    one = {n: v[:, 5:6] for n, v in views.items()}
    o, _ = gdr.gdr_linear_forward(one["q"], one["k"], one["v"], t["g"][:, 5:6].contiguous(), t["h0"], **a)
    ro, _ = gdr.gdr_linear_forward(*(t[n][:, 5:6].contiguous() for n in ("q", "k", "v", "g")), t["h0"], **a)
    assert torch.equal(o, ro)


@pytest.mark.parametrize("algo", ALGOS)
@pytest.mark.parametrize("io,out,bound", [(BF, BF, None), (BF, F, 400), (F, F, None)])
def test_ragged(algo, io, out, bound):
    """Sequences of 0, 1, 63, 64, 130 and 333 tokens behind 5 uncovered rows
    and before 7: each as a call of its own, the uncovered rows untouched."""
    lens = [0, 1, 63, 64, 130, 0, 333]
    cu = np.concatenate([[5], 5 + np.cumsum(lens)]).astype(np.int64)
    rows, Hk, Hv, Dk, Dv = int(cu[-1]) + 7, 2, 4, 64, 128
    x = draw(15, 1, rows, Hk, Hv, Dk, Dv, io)
    r = np.random.default_rng(16)
    x["h0"], x["dht"] = (r.standard_normal((len(lens), Hv, Dk, Dv)).astype(np.float32) for _ in range(2))
    t = to_dev(x, io)
    for n in ("q", "k", "v", "do"):
        t[n][:, :5], t[n][:, cu[-1]:] = float("nan"), float("nan")
    o = torch.full((1, rows, Hv, Dv), 7.0, dtype=out, device="cuda")
    kw = dict(algo=algo, cu_seqlens=torch.from_numpy(cu).cuda(), max_seqlen=bound)
    _, ht = gdr.gdr_linear_forward(t["q"], t["k"], t["v"], t["g"], t["h0"], o=o, **kw)
    got = gdr.gdr_linear_backward(t["q"], t["k"], t["v"], t["g"], t["h0"], t["do"], t["dht"], out_dtype=out, **kw)
    assert bool((o[:, :5] == 7).all()) and bool((o[:, cu[-1]:] == 7).all())
    for i in range(len(lens)):
        s = slice(cu[i], cu[i + 1])
        one = {n: x[n][:, s] for n in ("q", "k", "v", "g", "do")}
        one.update(h0=x["h0"][i:i + 1], dht=x["dht"][i:i + 1])
        if lens[i] == 0:
            assert torch.equal(ht[i], t["h0"][i]) and torch.equal(got[4][i], t["dht"][i])
            continue
        verify(one, out, o[:, s], ht[i:i + 1], [a[:, s] for a in got[:4]] + [got[4][i:i + 1]])


@pytest.mark.parametrize("algo", ALGOS)
def test_ragged_head_decay(algo):
    lens = [40, 0, 129]
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int64)
    x = draw(17, 1, 169, 2, 2, 64, 64, gate="head", state=False)
    t = to_dev(x, BF)
    got = gdr.gdr_linear_backward(t["q"], t["k"], t["v"], t["g"], None, t["do"], algo=algo, out_dtype=F,
                                  cu_seqlens=torch.from_numpy(cu).cuda())
    ref = A = 0
    for i in range(3):
        s = slice(cu[i], cu[i + 1])
        one = [x[n][:, s] for n in ("q", "k", "v")] + [x["g"], None, x["do"][:, s]]
        ref, A = ref + lo.backward(*one)[3], A + lo.backward_abs(*one)[3]
    close("dg", got[3], ref, A, 2 * (64 + 4 * 169 + 64), F)


@pytest.mark.parametrize("algo", ALGOS)
def test_empty(algo):
    e = lambda *s, dt=BF: torch.zeros(s, dtype=dt, device="cuda")
    h0 = torch.randn(2, 4, 64, 64, device="cuda")
    o, ht = gdr.gdr_linear_forward(e(2, 0, 2, 64), e(2, 0, 2, 64), e(2, 0, 4, 64), e(4, dt=F), h0, algo=algo)
    assert o.shape == (2, 0, 4, 64) and torch.equal(ht, h0)
    _, ht = gdr.gdr_linear_forward(e(2, 0, 2, 64), e(2, 0, 2, 64), e(2, 0, 4, 64), None, algo=algo)
    assert not ht.any()
    got = gdr.gdr_linear_backward(e(2, 0, 2, 64), e(2, 0, 2, 64), e(2, 0, 4, 64), e(4, dt=F), None,
                                  e(2, 0, 4, 64), h0, algo=algo)
    assert torch.equal(got[4], h0) and not got[3].any()
    o, ht = gdr.gdr_linear_forward(e(0, 9, 2, 64), e(0, 9, 2, 64), e(0, 9, 4, 64), e(4, dt=F), algo=algo)
    assert o.shape == (0, 9, 4, 64) and ht.shape == (0, 4, 64, 64)


@pytest.mark.parametrize("T", [1, 3])
def test_decode_in_place(T):
    """Steps that update the state in place, against one call over all
    tokens: the same arithmetic, token by token."""
    x = draw(18, 3, 5 * T, 2, 4, 128, 128)
    t = to_dev(x, BF)
    s = t["h0"].clone()
    for i in range(5):
        c = slice(i * T, (i + 1) * T)
        q, k, v, g = (t[n][:, c].contiguous() for n in ("q", "k", "v", "g"))
        o, ht = gdr.gdr_linear_forward(q, k, v, g, s, ht=s, algo="sequential")
        assert ht is s
        whole, _ = gdr.gdr_linear_forward(*(t[n][:, :(i + 1) * T].contiguous() for n in ("q", "k", "v", "g")),
                                          t["h0"], algo="sequential")
        assert torch.equal(o, whole[:, c])
    args = x["q"], x["k"], x["v"], x["g"], x["h0"]
    close("ht", s, lo.forward(*args)[1], lo.forward_abs(*args)[1], 128 + 20 * T + 64, F)


@pytest.mark.parametrize("algo", ALGOS)
def test_prefill_in_place_then_decode(algo):
    """A long prompt's state written over its initial state, then one token."""
    x = draw(19, 1, 1101, 2, 4, 64, 64)
    t = to_dev(x, BF)
    s = t["h0"].clone()
    p = {n: t[n][:, :1100].contiguous() for n in ("q", "k", "v", "g")}
    gdr.gdr_linear_forward(p["q"], p["k"], p["v"], p["g"], s, ht=s, algo=algo)
    p = {n: t[n][:, 1100:].contiguous() for n in ("q", "k", "v", "g")}
    o, _ = gdr.gdr_linear_forward(p["q"], p["k"], p["v"], p["g"], s, ht=s)
    args = x["q"], x["k"], x["v"], x["g"], x["h0"]
    n = 64 + 4 * 1101 + 64
    close("ht", s, lo.forward(*args)[1], lo.forward_abs(*args)[1], n, F)
    close("o", o, lo.forward(*args)[0][:, 1100:], lo.forward_abs(*args)[0][:, 1100:], n, F)


@pytest.mark.parametrize("algo", ALGOS)
def test_nan_stays_in_its_sequence_and_head(algo):
    x = draw(20, 2, 150, 2, 2, 64, 64)
    t = to_dev(x, BF)
    clean = gdr.gdr_linear_forward(t["q"], t["k"], t["v"], t["g"], t["h0"], algo=algo)
    t["v"][1, 70, 1, 3] = float("nan")
    t["k"][1, 90, 1, 2] = float("inf")
    o, ht = gdr.gdr_linear_forward(t["q"], t["k"], t["v"], t["g"], t["h0"], algo=algo)
    assert torch.equal(o[0], clean[0][0]) and torch.equal(o[1, :, 0], clean[0][1, :, 0])
    assert torch.equal(ht[0], clean[1][0]) and torch.equal(ht[1, 0], clean[1][1, 0])
    assert torch.equal(o[1, :64, 1], clean[0][1, :64, 1])  # chunks before the token
    assert bool(o[1, 70:, 1, 3].isnan().all()) and not bool(ht[1, 1].isfinite().all())


@pytest.mark.parametrize("algo", ALGOS)
def test_same_bits_twice(algo):
    x = draw(21, 2, 700, 2, 4, 128, 64)
    t = to_dev(x, BF)
    runs = []
    for _ in range(2):
        runs.append(gdr.gdr_linear_forward(t["q"], t["k"], t["v"], t["g"], t["h0"], algo=algo)
                    + gdr.gdr_linear_backward(t["q"], t["k"], t["v"], t["g"], t["h0"], t["do"], t["dht"], algo=algo))
    assert all(torch.equal(a, b) for a, b in zip(*runs))


@pytest.mark.parametrize("algo", ALGOS)
def test_graph_replays_and_other_streams(algo):
    """Forward and VJP captured together, replayed with new inputs between
    eager calls, and a call on a side stream: the eager bits each time."""
    x = [to_dev(draw(22 + i, 2, 600, 2, 4, 64, 64), BF) for i in range(4)]
    names = ("q", "k", "v", "g", "h0", "do", "dht")
    buf = {n: x[0][n].clone() for n in names}

    def both(t):
        return (gdr.gdr_linear_forward(t["q"], t["k"], t["v"], t["g"], t["h0"], algo=algo)
                + gdr.gdr_linear_backward(t["q"], t["k"], t["v"], t["g"], t["h0"], t["do"], t["dht"], algo=algo))

    side = torch.cuda.Stream()
    want = [both(t) for t in x]
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(2):
            both(buf)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res = both(buf)
    for i in (1, 2, 3, 1):
        for n in names:
            buf[n].copy_(x[i][n])
        graph.replay()
        both(x[0])
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(res, want[i])), i
    o, ht = gdr.gdr_linear_forward(x[2]["q"], x[2]["k"], x[2]["v"], x[2]["g"], x[2]["h0"], algo=algo, stream=side)
    side.synchronize()
    assert torch.equal(o, want[2][0]) and torch.equal(ht, want[2][1])
