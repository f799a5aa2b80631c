"""The float64 definitions of linear attention with decay and of the group
norm: gradients against central differences and torch's autograd of the
matrix forms, and closed forms."""

import numpy as np
import pytest
import torch

from oracle import linear_oracle as lo


def draw(seed, B=2, T=5, Hk=2, Hv=4, Dk=3, Dv=4, head=False):
    r = np.random.default_rng(seed)
    n = r.standard_normal
    g = -0.3 * abs(n(Hv) if head else n((B, T, Hv)))
    return dict(q=n((B, T, Hk, Dk)), k=n((B, T, Hk, Dk)), v=n((B, T, Hv, Dv)), g=g, h0=n((B, Hv, Dk, Dv)),
                do=n((B, T, Hv, Dv)), dht=n((B, Hv, Dk, Dv)))


@pytest.mark.parametrize("head", [False, True])
def test_gradients_against_differences(head):
    x = draw(1, head=head)

    def loss(**kw):
        y = dict(x, **kw)
        o, ht = lo.forward(y["q"], y["k"], y["v"], y["g"], y["h0"])
        return (o * x["do"]).sum() + (ht * x["dht"]).sum()

    got = lo.backward(x["q"], x["k"], x["v"], x["g"], x["h0"], x["do"], x["dht"])
    r = np.random.default_rng(2)
    for name, grad in zip(("q", "k", "v", "g", "h0"), got):
        d = r.standard_normal(x[name].shape)
        num = (loss(**{name: x[name] + 1e-6 * d}) - loss(**{name: x[name] - 1e-6 * d})) / 2e-6
        assert abs(num - (grad * d).sum()) < 1e-6 * max(1.0, abs(num)), name


def test_forward_is_the_masked_product():
    """O = (Q K^T o e^{G_t - G_s}, s <= t) V + e^{G_t} Q h0, written densely."""
    x = draw(3)
    o, ht = lo.forward(x["q"], x["k"], x["v"], x["g"], x["h0"])
    B, T, Hv, _ = o.shape
    for b in range(B):
        for h in range(Hv):
            q, k, v, G = x["q"][b, :, h // 2], x["k"][b, :, h // 2], x["v"][b, :, h], np.cumsum(x["g"][b, :, h])
            W = np.tril(np.exp(G[:, None] - G[None, :]))
            np.testing.assert_allclose(o[b, :, h], (q @ k.T * W) @ v + np.exp(G)[:, None] * (q @ x["h0"][b, h]),
                                       rtol=1e-12, atol=1e-12)
            np.testing.assert_allclose(ht[b, h], np.exp(G[-1]) * x["h0"][b, h] + (k * np.exp(G[-1] - G)[:, None]).T @ v,
                                       rtol=1e-12, atol=1e-12)


def test_a_gate_of_minus_infinity_drops_the_state():
    x = draw(4)
    g = x["g"].copy()
    g[:, 2] = -np.inf
    o, ht = lo.forward(x["q"], x["k"], x["v"], g, x["h0"])
    o2, ht2 = lo.forward(x["q"][:, 2:], x["k"][:, 2:], x["v"][:, 2:], x["g"][:, 2:], None)
    np.testing.assert_allclose(o[:, 2:], o2, rtol=1e-12)
    np.testing.assert_allclose(ht, ht2, rtol=1e-12)


def test_chain_identities():
    """dq, dk and dv are chains of the same kind, and dg the suffix sum of
    q . dq - k . dk: what the kernels are built on."""
    x = draw(5, Hk=4)
    dq, dk, dv, dg, dh0 = lo.backward(x["q"], x["k"], x["v"], x["g"], x["h0"], x["do"], x["dht"])
    t = lambda s: np.swapaxes(s, -1, -2)
    cq, last = lo.forward(x["do"], x["v"], x["k"], x["g"], t(x["h0"]))
    np.testing.assert_allclose(cq, dq, rtol=1e-10, atol=1e-12)
    back = np.concatenate([np.zeros_like(x["g"][:, :1]), x["g"][:, :0:-1]], axis=1)
    f = lambda a: a[:, ::-1]
    cv, first = lo.forward(f(x["k"]), f(x["q"]), f(x["do"]), back, x["dht"])
    np.testing.assert_allclose(f(cv), dv, rtol=1e-10, atol=1e-12)
    ck, _ = lo.forward(f(x["v"]), f(x["do"]), f(x["q"]), back, t(x["dht"]))
    np.testing.assert_allclose(f(ck), dk, rtol=1e-10, atol=1e-12)
    np.testing.assert_allclose(np.exp(x["g"][:, 0])[..., None, None] * first, dh0, rtol=1e-10, atol=1e-12)
    e = (x["q"] * dq - x["k"] * dk).sum(-1)
    suffix = np.cumsum(e[:, ::-1], axis=1)[:, ::-1] + (t(last) * x["dht"]).sum((-2, -1))[:, None]
    np.testing.assert_allclose(suffix, dg, rtol=1e-9, atol=1e-10)


@pytest.mark.parametrize("act", ["gate", "silu", "none"])
@pytest.mark.parametrize("center", [False, True])
@pytest.mark.parametrize("shared", [False, True])
def test_norm_against_autograd(act, center, shared):
    r = np.random.default_rng(7)
    x, dy = r.standard_normal((5, 3, 8)), r.standard_normal((5, 3, 8))
    z = r.standard_normal((5, 3, 8)) if act == "gate" else None
    w, b = (r.standard_normal((8,) if shared else (3, 8)) for _ in range(2))
    t = [torch.tensor(a, requires_grad=True) if a is not None else None for a in (x, z, w, b)]
    tx, tz, tw, tb = t
    if center:
        n = torch.nn.functional.layer_norm(tx, (8,), eps=1e-5)
    else:
        n = tx * torch.rsqrt(tx.pow(2).mean(-1, keepdim=True) + 1e-5)
    u = n * tw + tb
    y = u * torch.nn.functional.silu(tz) if act == "gate" else torch.nn.functional.silu(u) if act == "silu" else u
    y.backward(torch.tensor(dy))
    np.testing.assert_allclose(lo.norm_forward(x, w, b, z, center, act == "silu"), y.detach().numpy(), rtol=1e-10)
    got = lo.norm_backward(x, w, b, z, dy, center, act == "silu")
    for a, ref in zip(got, (tx, tz, tw, tb)):
        if ref is not None:
            np.testing.assert_allclose(a, ref.grad.numpy(), rtol=1e-8, atol=1e-10)
