"""Independent float64 definitions of the attention layer's operators (test
infrastructure only; shares nothing with the HIP path): rotary positions, a
paged cache, attention of one token over it, and causal attention with a window
and its VJP.  ``bounds`` arguments give, beside a result, the sums over absolute
values that a rounding error of any operand or partial sum is measured by.
"""

import numpy as np


def _f(x):
    return None if x is None else np.asarray(x, dtype=np.float64)


# ---- rotary positions -----------------------------------------------------

def pair_axis(half, section=None, cycled=False):
    """The axis of each of `half` pairs."""
    if section is None or len(section) == 1:
        return [0] * half
    if not cycled:
        return [a for a, n in enumerate(section) for _ in range(n)]
    axes = len(section)
    return [i % axes if i < axes * section[i % axes] else 0 for i in range(half)]


def rotary(x, pos, freq, section=None, adjacent=False, cycled=False, back=False):
    """x [rows, H, D] turned at pos [rows] or [axes, rows] (Python integers'
    products with freq, reduced modulo a turn)."""
    x, freq = _f(x), np.asarray(freq, np.float32).astype(np.float64)
    half = len(freq)
    pos = np.asarray(pos, dtype=np.int64)
    pos = pos[None] if pos.ndim == 1 else pos
    y = x.copy()
    for i, a in enumerate(pair_axis(half, section, cycled)):
        w = pos[a].astype(np.longdouble) * np.longdouble(freq[i])
        w = np.asarray(np.remainder(w, 2 * np.longdouble(np.pi) + np.longdouble(2.4492935982947064e-16)), np.float64)
        c, s = np.cos(w)[:, None], np.sin(w)[:, None] * (-1 if back else 1)
        p, r = (2 * i, 2 * i + 1) if adjacent else (i, i + half)
        y[..., p] = x[..., p] * c - x[..., r] * s
        y[..., r] = x[..., r] * c + x[..., p] * s
    return y


# ---- attention ------------------------------------------------------------

def seen(T, window=None, sinks=0):
    """[T, T]: whether token i sees token j."""
    i, j = np.arange(T)[:, None], np.arange(T)[None]
    low = j <= i
    return low if window is None else low & ((i - j < window) | (j < sinks))


def _softmax(S, ok):
    S = np.where(ok, S, -np.inf)
    m = S.max(-1, keepdims=True)
    with np.errstate(invalid="ignore"):
        e = np.where(ok, np.exp(S - m), 0.0)
    n = e.sum(-1, keepdims=True)
    return e / n, (m + np.log(n))[..., 0]


def attention(q, k, v, scale, window=None, sinks=0):
    """One sequence: q [T, Hq, D], k, v [T, Hk, D] -> o, lse [T, Hq]."""
    q, k, v = _f(q), _f(k), _f(v)
    T, Hq, D = q.shape
    G = Hq // k.shape[1]
    o, lse = np.zeros_like(q), np.zeros((T, Hq))
    ok = seen(T, window, sinks)
    for h in range(Hq):
        P, lse[:, h] = _softmax(scale * q[:, h] @ k[:, h // G].T, ok)
        o[:, h] = P @ v[:, h // G]
    return o, lse


def attention_vjp(q, k, v, do, scale, window=None, sinks=0):
    """(dq, dk, dv) of <do, o>, by the chain rule through the softmax's Jacobian
    row by row (no delta)."""
    q, k, v, do = _f(q), _f(k), _f(v), _f(do)
    T, Hq, D = q.shape
    G = Hq // k.shape[1]
    dq, dk, dv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    ok = seen(T, window, sinks)
    for h in range(Hq):
        kh = h // G
        P, _ = _softmax(scale * q[:, h] @ k[:, kh].T, ok)
        dP = do[:, h] @ v[:, kh].T
        for i in range(T):
            J = np.diag(P[i, :i + 1]) - np.outer(P[i, :i + 1], P[i, :i + 1])
            dS = J @ dP[i, :i + 1]
            dq[i, h] = scale * dS @ k[:i + 1, kh]
            dk[:i + 1, kh] += scale * np.outer(dS, q[i, h])
        dv[:, kh] += P.T @ do[:, h]
    return dq, dk, dv


# ---- the paged cache ------------------------------------------------------

def append(kc, vc, table, lengths, new, k, v, freq=None, pos=None, **turn):
    """The caches [pages, size, Hk, D] with the new tokens of each sequence:
    new: [(first row, rows)], k, v [rows, Hk, D] (as stored, before rounding)."""
    kc, vc, k, v = _f(kc).copy(), _f(vc).copy(), _f(k), _f(v)
    size = kc.shape[1]
    for b, (row, n) in enumerate(new):
        for t in range(n):
            at = int(lengths[b]) - n + t
            if at < 0 or at // size >= len(table[b]):
                continue
            page = int(table[b][at // size])
            if not 0 <= page < len(kc):
                continue
            p = [at] if pos is None else np.asarray(pos)[..., row + t:row + t + 1]
            kr = k[row + t:row + t + 1]
            kc[page, at % size] = kr[0] if freq is None else rotary(kr, p, freq, **turn)[0]
            vc[page, at % size] = v[row + t]
    return kc, vc


def visible(n, table, size, pages, window=None, sinks=0):
    """(page, slot) of the tokens that the last of n sees, in order."""
    out = []
    for j in range(n):
        if window is not None and n - 1 - j >= window and j >= sinks:
            continue
        page = int(table[j // size])
        if 0 <= page < pages:
            out.append((page, j % size))
    return out


def cache_attention(q, kc, vc, table, lengths, scale, window=None, sinks=0, max_len=None):
    """q [B, Hq, D] -> o, lse, and per query head the visible keys and values."""
    q, kc, vc = _f(q), _f(kc), _f(vc)
    B, Hq, D = q.shape
    Hk = kc.shape[2]
    o, lse, got = np.zeros_like(q), np.full((B, Hq), -np.inf), []
    most = len(table[0]) * kc.shape[1] if B else 0
    for b in range(B):
        n = max(0, min(int(lengths[b]), most if max_len is None else max_len))
        at = visible(n, table[b], kc.shape[1], len(kc), window, sinks)
        got.append(at)
        if not at:
            continue
        p, s = (list(x) for x in zip(*at))
        for h in range(Hq):
            k, v = kc[p, s, h // (Hq // Hk)], vc[p, s, h // (Hq // Hk)]
            P, l1 = _softmax(scale * (k @ q[b, h])[None], np.ones((1, len(p)), bool))
            o[b, h], lse[b, h] = P[0] @ v, l1[0]
    return o, lse, got
