"""Independent float64 definitions of linear attention with a decay for each
head and of the group norm (test infrastructure only; shares nothing with the
HIP path).

The recurrence per batch and value head, S_0 = h0:
    S_t = e^{g_t} S_{t-1} + k_t v_t^T,  o_t = S_t^T q_t,
value head h reading q/k head h / (Hv / Hk).  The VJP stores every state and
sweeps backward; it does not use the chain identities the kernels are built
on.  ``forward_abs`` / ``backward_abs`` are the same sums over absolute
values: what a rounding error of any operand or partial sum is measured by.
"""

import numpy as np


def _f(x):
    return None if x is None else np.asarray(x, dtype=np.float64)


def _decay(g, B, T, Hv):
    if g is None:
        return np.ones((B, T, Hv))
    return np.exp(np.broadcast_to(g, (B, T, Hv)))


def _states(q, k, v, g, h0):
    """All states S_0 .. S_T [T+1, B, Hv, Dk, Dv], heads of k repeated."""
    B, T, Hk, Dk = k.shape
    Hv, Dv = v.shape[2:]
    kk = np.repeat(k, Hv // Hk, axis=2)
    a = _decay(g, B, T, Hv)
    S = np.zeros((T + 1, B, Hv, Dk, Dv))
    if h0 is not None:
        S[0] = h0
    for t in range(T):
        S[t + 1] = np.where(a[:, t, :, None, None] == 0.0, 0.0, a[:, t, :, None, None] * S[t])
        S[t + 1] += kk[:, t, :, :, None] * v[:, t, :, None, :]
    return S, a


def forward(q, k, v, g=None, h0=None):
    """(o [B, T, Hv, Dv], S_T)."""
    q, k, v, g, h0 = _f(q), _f(k), _f(v), _f(g), _f(h0)
    S, _ = _states(q, k, v, g, h0)
    qq = np.repeat(q, v.shape[2] // q.shape[2], axis=2)
    o = np.einsum("bthd,tbhde->bthe", qq, S[1:]) if q.shape[1] else np.zeros_like(v)
    return o, S[-1]


def backward(q, k, v, g, h0, do, dht=None):
    """(dq, dk, dv, dg, dh0) of <do, o> + <dht, S_T>; dg is None without g and
    summed over all tokens for a constant decay per head."""
    q, k, v, g, h0, do, dht = (_f(x) for x in (q, k, v, g, h0, do, dht))
    B, T, Hk, Dk = q.shape
    Hv, Dv = v.shape[2:]
    G = Hv // Hk
    S, a = _states(q, k, v, g, h0)
    qq, kk = np.repeat(q, G, axis=2), np.repeat(k, G, axis=2)
    dq, dk, dv = np.zeros((B, T, Hv, Dk)), np.zeros((B, T, Hv, Dk)), np.zeros_like(v)
    dg = np.zeros((B, T, Hv))
    D = np.zeros((B, Hv, Dk, Dv)) if dht is None else dht.copy()
    for t in reversed(range(T)):
        D = D + qq[:, t, :, :, None] * do[:, t, :, None, :]
        dq[:, t] = np.einsum("bhde,bhe->bhd", S[t + 1], do[:, t])
        dk[:, t] = np.einsum("bhde,bhe->bhd", D, v[:, t])
        dv[:, t] = np.einsum("bhde,bhd->bhe", D, kk[:, t])
        dg[:, t] = a[:, t] * np.einsum("bhde,bhde->bh", S[t], D)
        D = a[:, t, :, None, None] * D
    dq, dk = (x.reshape(B, T, Hk, G, Dk).sum(3) for x in (dq, dk))
    if g is None:
        dg = None
    elif g.ndim == 1:
        dg = dg.sum((0, 1))
    return dq, dk, dv, dg, D


def forward_abs(q, k, v, g=None, h0=None):
    return forward(abs(_f(q)), abs(_f(k)), abs(_f(v)), g, None if h0 is None else abs(_f(h0)))


def backward_abs(q, k, v, g, h0, do, dht=None):
    """The sums of absolute values behind each gradient.  dg's are those of
    dg_t = sum_{r >= t} (q_r . dq_r - k_r . dk_r) + <S_T, dS_T>, the form whose
    terms cancel the most."""
    q, k, v, h0, do, dht = (None if x is None else abs(_f(x)) for x in (q, k, v, h0, do, dht))
    g = _f(g)
    dq, dk, dv, _, dh0 = backward(q, k, v, g, h0, do, dht)
    if g is None:
        return dq, dk, dv, None, dh0
    B, T, Hk, Dk = q.shape
    Hv = v.shape[2]
    row = np.zeros((B, T, Hv))
    qq, kk = np.repeat(q, Hv // Hk, axis=2), np.repeat(k, Hv // Hk, axis=2)
    for h in range(Hv):  # per value head: one head's gradients
        one = backward(qq[:, :, h:h + 1], kk[:, :, h:h + 1], v[:, :, h:h + 1],
                       g[h:h + 1] if g.ndim == 1 else g[:, :, h:h + 1], None if h0 is None else h0[:, h:h + 1],
                       do[:, :, h:h + 1], None if dht is None else dht[:, h:h + 1])
        row[:, :, h] = ((qq[:, :, h] * one[0][:, :, 0]) + (kk[:, :, h] * one[1][:, :, 0])).sum(-1)
    last = forward(q, k, v, g, h0)[1]
    end = 0.0 if dht is None else (last * dht).sum((-2, -1))
    dg = np.cumsum(row[:, ::-1], axis=1)[:, ::-1] + (end if dht is None else end[:, None, :])
    return dq, dk, dv, (dg.sum((0, 1)) if g.ndim == 1 else dg), dh0


# ---- group norm -----------------------------------------------------------

def _sigmoid(x):
    return 1.0 / (1.0 + np.exp(-x))


def norm_forward(x, w=None, b=None, z=None, center=False, silu=False, eps=1e-5):
    x, z = _f(x), _f(z)
    mu = x.mean(-1, keepdims=True) if center else 0.0
    n = (x - mu) / np.sqrt(((x - mu) ** 2).mean(-1, keepdims=True) + eps)
    u = n * (1.0 if w is None else _f(w)) + (0.0 if b is None else _f(b))
    return u * z * _sigmoid(z) if z is not None else u * _sigmoid(u) if silu else u


def norm_backward(x, w, b, z, dy, center=False, silu=False, eps=1e-5):
    """(dx, dz, dw, db) by the chain rule through the Jacobian of n, written
    as the full D x D matrix of each row."""
    x, z, dy = _f(x), _f(z), _f(dy)
    D = x.shape[-1]
    w_ = np.ones(D) if w is None else _f(w)
    mu = x.mean(-1, keepdims=True) if center else 0.0
    sd = np.sqrt(((x - mu) ** 2).mean(-1, keepdims=True) + eps)
    n = (x - mu) / sd
    u = n * w_ + (0.0 if b is None else _f(b))
    dz = None
    if z is not None:
        s = _sigmoid(z)
        dz = dy * u * (s + z * s * (1 - s))
        du = dy * z * s
    elif silu:
        s = _sigmoid(u)
        du = dy * (s + u * s * (1 - s))
    else:
        du = dy
    P = np.eye(D) - (1.0 / D if center else 0.0)
    J = (P - n[..., :, None] * n[..., None, :] / D) / sd[..., None]  # dn_i / dx_j
    dx = np.einsum("...i,...ij->...j", du * w_, J)
    axes = tuple(range(x.ndim - 1 if w_.ndim == 1 else x.ndim - 2))
    return dx, dz, (du * n).sum(axes), du.sum(axes)
