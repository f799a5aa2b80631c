"""How far a NaN of one token reaches in attention and its VJP: the tokens that it is
visible to (or that are visible to it), and those that share a tile of 64 with
them; no others.

The backward is given clean o and lse, so that what it returns shows its own reach.
With bf16 outputs a row's delta is corrected by the sum of its dS, so a row whose
dS are NaN gives NaN to the dk of every key that it sees."""

import numpy as np
import pytest
import torch

import gated_delta_rule_54_amd as gdr
from oracle import attention_oracle as ao
from tests.test_gpu_attention import draw
from tests.test_gpu_rotary import BF, F, dev

pytestmark = pytest.mark.gpu

TILE = 64


def tiles_seen(ok):
    """[T, T]: whether any pair of i's tile and j's is visible."""
    T = len(ok)
    n = -(-T // TILE)
    full = np.zeros((n * TILE, n * TILE), bool)
    full[:T, :T] = ok
    near = full.reshape(n, TILE, n, TILE).any((1, 3))
    return np.repeat(np.repeat(near, TILE, 0), TILE, 1)[:T, :T]


def may_reach(which, t, ok, out):
    """Rows of dq, dk and dv that may be NaN where row t of `which` is."""
    near, own = tiles_seen(ok), np.arange(len(ok)) == t
    if which in ("q", "dout"):
        return own, near[t], near[t]
    # rows that see key t have a NaN dS
    through = ok[ok[:, t]].any(0) if out == BF else own
    return near[:, t], through | own, own


# blocks of 32 queries on a small grid, of 128 where 256 blocks or more (1024 in fp32
# above 64 channels) fill the card
@pytest.mark.parametrize("B", [1, 180])
@pytest.mark.parametrize("window,sinks", [(None, 0), (40, 3)])
@pytest.mark.parametrize("io,out,D", [(BF, F, 64), (BF, BF, 128), (F, F, 64), (F, F, 128), (BF, BF, 256), (F, BF, 256)])
def test_a_token_s_nan_in_the_vjp(io, out, D, window, sinks, B):
    T, Hq, Hk = 300, 4, 2
    how = dict(window=window, sinks=sinks)
    x = draw(70, T, Hq, Hk, D, io)
    t = dict(zip(("q", "k", "v", "dout"), (dev(a, io).expand(B, *a.shape).contiguous() for a in x)))
    o, lse = gdr.gdr_attention_forward(t["q"], t["k"], t["v"], out_dtype=out, **how)
    ok = ao.seen(T, window, sinks)
    for which in t:
        for at in (10, 100, 200, 299):
            bad = dict(t, **{which: t[which].clone()})
            bad[which][0, at, 0, 5] = float("nan")
            grads = gdr.gdr_attention_backward(bad["q"], bad["k"], bad["v"], o, lse, bad["dout"], **how)
            for name, g, may in zip(("dq", "dk", "dv"), grads, may_reach(which, at, ok, out)):
                rows = torch.isnan(g[0]).any(-1)
                own = 0 if which in ("q", "dout") and name == "dq" else slice(0, 2) if name == "dq" else 0
                reached = np.flatnonzero(rows.any(1).cpu().numpy() & ~may)
                assert reached.size == 0, (which, at, name, reached)
                rest = rows.clone()
                rest[:, own] = False  # the head, or the heads that share the key head
                assert not rest.any(), (which, at, name)
                assert not torch.isnan(g[1:]).any(), (which, at, name)
            if which != "v":
                assert torch.isnan(grads[0][0, at, 0]).any()


@pytest.mark.parametrize("B", [1, 180])
@pytest.mark.parametrize("window,sinks", [(None, 0), (40, 3)])
@pytest.mark.parametrize("io,out,D", [(BF, F, 64), (BF, BF, 128), (F, F, 64), (F, F, 128), (BF, BF, 256), (F, BF, 256)])
def test_a_token_s_nan_in_the_forward(io, out, D, window, sinks, B):
    """v: by tiles.  q and k enter scores, which are masked one by one."""
    T, Hq, Hk = 300, 4, 2
    how = dict(window=window, sinks=sinks, out_dtype=out)
    t = dict(zip("qkv", (dev(a, io).expand(B, *a.shape).contiguous() for a in draw(71, T, Hq, Hk, D, io)[:3])))
    ok = ao.seen(T, window, sinks)
    for which in t:
        for at in (10, 100, 200, 299):
            bad = dict(t, **{which: t[which].clone()})
            bad[which][0, at, 0, 5] = float("nan")
            o, lse = gdr.gdr_attention_forward(bad["q"], bad["k"], bad["v"], **how)
            may = {"q": np.arange(T) == at, "k": ok[:, at], "v": tiles_seen(ok)[:, at]}[which]
            must = {"q": np.arange(T) == at, "k": ok[:, at], "v": ok[:, at]}[which]
            heads = 1 if which == "q" else 2
            rows = torch.isnan(o[0, :, :heads]).any(-1).cpu().numpy()
            assert not (rows.any(1) & ~may).any() and rows[must].all(), (which, at)
            nan = torch.isnan(lse[0, :, :heads]).cpu().numpy()
            assert (nan == ((may & (which != "v"))[:, None])).all(), (which, at)
            assert not torch.isnan(o[0, :, heads:]).any() and not torch.isnan(o[1:]).any(), (which, at)
