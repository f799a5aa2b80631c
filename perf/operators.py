"""The operators beside the gated delta rule, as they are timed and compared:
linear attention with a decay for each head (forward over prompts, single
tokens, VJP) and the group norm of the heads' outputs with its activation
(forward, VJP).

With ``own`` false, ``run`` computes a case in elementary torch operations in
32 bits (running sums of the decay in 64); with ``own`` true it makes the
library's calls.  ``exact`` gives the same outputs from the definitions, token
by token, in 64 bits.
"""

import math

import numpy as np
import torch

own = False

BF16, F32 = "bf16", "f32"
DT = {BF16: torch.bfloat16, F32: torch.float32}
EPS = 1e-5
CHUNK = 128  # rows of a chunk of the plain form


# ---- the cases ------------------------------------------------------------

def linear(kind, B, T, Hk, Hv, Dk, Dv, io=BF16, out=BF16, gate="token", state=False, lengths=0):
    """One linear-attention case.  gate: "token" (g [B, T, Hv]), "head"
    (g [Hv]); state: h0 given (and dht, for the VJP); lengths: that many
    prompts of unequal length, at most T tokens each, laid end to end."""
    return dict(kind=kind, B=B, T=T, Hk=Hk, Hv=Hv, Dk=Dk, Dv=Dv, io=io, out=out, gate=gate, state=state,
                lengths=lengths)


def norm(kind, rows, G, D, io=BF16, out=BF16, act="gate", center=True, shared=False):
    """One group-norm case: rows of G groups of D channels; act: "gate"
    (times silu(z)), "silu" or "none"; center: subtract the mean; shared: one
    weight of D channels for all groups."""
    return dict(kind=kind, rows=rows, G=G, D=D, io=io, out=out, act=act, center=center, shared=shared)


def listed():
    return [
        # a training batch's forward pass, the shapes of the gated delta rule's benchmark step
        dict(linear("forward", 4, 4096, 16, 32, 128, 128), name="forward B4 T4096"),
        # a ragged prefill of 17 prompts, its states kept for decoding
        dict(linear("forward", 17, 2048, 16, 32, 128, 128, lengths=17), name="forward ragged 17"),
        # one long document through constant decays per head: few rows, a long axis
        dict(linear("forward", 1, 32768, 8, 8, 128, 128, gate="head"), name="forward B1 T32768"),
        # a short odd prompt in 32 bits with unequal head widths, continuing a state
        dict(linear("forward", 2, 333, 4, 4, 64, 128, io=F32, out=F32, state=True), name="forward f32 T333"),
        # serving: one token for each of 8 and of 256 sequences
        dict(linear("forward", 8, 1, 16, 32, 128, 128, state=True), name="token B8"),
        dict(linear("forward", 256, 1, 16, 32, 128, 128, state=True), name="token B256"),
        # the training batch's VJP, and that of a short odd sequence with both end states
        dict(linear("backward", 4, 4096, 16, 32, 128, 128), name="backward B4 T4096"),
        dict(linear("backward", 1, 777, 8, 8, 64, 64, state=True), name="backward B1 T777"),
        # the heads' outputs of the training batch, forward and VJP, gated
        dict(norm("norm", 16384, 32, 128), name="norm 16384 rows"),
        dict(norm("norm_backward", 16384, 32, 128), name="norm backward 16384 rows"),
        # a decoding step's rows; a ragged batch's odd rows with a weight shared by the heads
        dict(norm("norm", 8, 32, 128, center=False, shared=True), name="norm 8 rows"),
        dict(norm("norm_backward", 1237, 24, 96, center=False, shared=True), name="norm backward 1237 rows"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["forward", "forward", "token", "backward", "backward", "norm", "norm_backward"])
    io = rng.choice([BF16, BF16, BF16, F32])
    out = F32 if io == F32 else rng.choice([BF16, BF16, F32])
    if kind in ("norm", "norm_backward"):
        G, D = rng.choice([1, 4, 7, 16, 24, 32]), rng.choice([32, 64, 80, 96, 128, 192, 256, 512])
        rows = _log_int(rng, 1, max(1, min(16384, 16384 * 4096 * (1 if io == F32 else 2) // (4 * G * D))))
        return norm(kind, rows, G, D, io, out, rng.choice(["gate", "gate", "silu", "none"]), rng.random() < 0.5,
                    rng.random() < 0.5)
    group = rng.choice([1, 1, 2, 4])
    Hk = rng.choice([1, 2, 4, 8])
    Hv = Hk * group
    Dk, Dv = rng.choice([(64, 64), (64, 128), (128, 64), (128, 128), (128, 128), (96, 80), (32, 48)])
    gate = rng.choice(["token", "token", "head"])
    state = rng.random() < 0.5
    if kind == "token":
        return linear("forward", _log_int(rng, 1, 256), rng.choice([1, 1, 1, 2, 5]), Hk, Hv, Dk, Dv, io, out, gate,
                      True)
    T = _log_int(rng, 2, 8192 if io == BF16 else 2048)
    B = _log_int(rng, 1, max(1, min(8, 16384 // T)))
    n = rng.choice([0, 0, 0, B]) if B > 1 else 0
    return linear(kind, B, T, Hk, Hv, Dk, Dv, io, out, gate, state, n)


def _lengths(B, T):
    """The lengths of B prompts: from a sixteenth of T to T, the first one T."""
    lens = np.random.default_rng(B * T).integers(max(1, T // 16), T + 1, B)
    lens[0] = T
    return lens


# ---- inputs ---------------------------------------------------------------

def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)

    def randn(*shape):
        return torch.randn(shape, generator=gen, device=dev, dtype=torch.float32)

    s = dict(case=case)
    if case["kind"].startswith("norm"):
        rows, G, D, io = case["rows"], case["G"], case["D"], DT[case["io"]]
        s["x"] = (0.5 * randn(rows, G, D) + 0.1).to(io)
        s["z"] = randn(rows, G, D).to(io) if case["act"] == "gate" else None
        s["w"] = 1 + 0.1 * (randn(D) if case["shared"] else randn(G, D))
        s["b"] = 0.1 * (randn(D) if case["shared"] else randn(G, D)) if case["center"] else None
        if case["kind"] == "norm_backward":
            s["dy"] = randn(rows, G, D).to(io)
        return s
    B, T, Hk, Hv, Dk, Dv, io = (case[n] for n in ("B", "T", "Hk", "Hv", "Dk", "Dv", "io"))
    io = DT[io]
    s["cu"] = None
    rows = (B, T)
    if case["lengths"]:
        cu = np.concatenate([[0], np.cumsum(_lengths(B, T))]).astype(np.int64)
        rows = (1, int(cu[-1]))
        s["cu"] = torch.from_numpy(cu).to(dev)
    # feature maps: silu, and the query's scale folded in
    s["q"] = (torch.nn.functional.silu(randn(*rows, Hk, Dk)) * Dk ** -0.5).to(io)
    s["k"] = torch.nn.functional.silu(randn(*rows, Hk, Dk)).to(io)
    s["v"] = randn(*rows, Hv, Dv).to(io)
    # memories from about two tokens to a few hundred
    rate = -torch.exp2(-8.0 * torch.arange(1, Hv + 1, device=dev, dtype=torch.float32) / Hv)
    s["g"] = rate if case["gate"] == "head" else (rate * torch.nn.functional.softplus(randn(*rows, Hv))).contiguous()
    s["h0"] = 0.5 * randn(B, Hv, Dk, Dv) if case["state"] else None
    if case["kind"] == "backward":
        s["do"] = randn(*rows, Hv, Dv).to(io)
        s["dht"] = 0.1 * randn(B, Hv, Dk, Dv) if case["state"] else None
    else:
        s["ht"] = torch.empty(B, Hv, Dk, Dv, device=dev)
    return s


# ---- the plain form -------------------------------------------------------

def _pad_rows(x, cu, T):
    """[1, rows, ...] -> [N, T, ...] with zeros past each sequence's end."""
    at = cu[:-1, None] + torch.arange(T, device=cu.device)
    ok = at < cu[1:, None]
    y = x[0][at.clamp(max=x.shape[1] - 1)]
    return torch.where(ok.reshape(ok.shape + (1,) * (y.dim() - 2)), y, torch.zeros((), dtype=y.dtype, device=y.device))


def _unpad_rows(x, cu):
    """[N, T, ...] -> [1, rows, ...], the inverse of _pad_rows."""
    ok = torch.arange(x.shape[1], device=cu.device) < (cu[1:] - cu[:-1])[:, None]
    return x[ok][None]


def _decayed(x, y, z, g, h0):
    """out_t = S_t^T x_t with S_t = e^{g_t} S_{t-1} + y_t z_t^T, and the last
    state.  x, y [B, H, T, D1], z [B, H, T, D2], g [B, H, T] (64 bits)."""
    B, H, T, D1 = x.shape
    D2 = z.shape[-1]
    C = min(CHUNK, T)
    N = -(-T // C)
    tail = N * C - T
    pad = torch.nn.functional.pad
    x, y, z = (pad(a, (0, 0, 0, tail)).reshape(B, H, N, C, -1) for a in (x, y, z))
    G = pad(g, (0, tail)).reshape(B, H, N, C).cumsum(-1)
    low = torch.ones(C, C, dtype=torch.bool, device=x.device).tril()
    W = torch.exp((G[..., :, None] - G[..., None, :]).masked_fill(~low, -math.inf)).float()
    inner = ((x @ y.mT) * W) @ z
    end = G[..., -1:]
    S = (y * torch.exp(end - G).float()[..., None]).mT @ z
    L = end[..., 0].cumsum(-1)
    before = torch.ones(N, N, dtype=torch.bool, device=x.device).tril(-1)
    M = torch.exp((L - end[..., 0])[..., :, None] - L[..., None, :])
    M = torch.where(before, M, torch.zeros((), dtype=M.dtype, device=M.device)).float()
    S = S.reshape(B, H, N, D1 * D2)
    last = (torch.exp(L[..., -1:] - L).float()[..., None, :] @ S).reshape(B, H, D1, D2)
    into = M @ S
    if h0 is not None:
        into = into + torch.exp(L - end[..., 0]).float()[..., None] * h0.reshape(B, H, 1, D1 * D2)
        last = last + torch.exp(L[..., -1]).float()[..., None, None] * h0
    out = inner + torch.exp(G).float()[..., None] * (x @ into.reshape(B, H, N, D1, D2))
    return out.reshape(B, H, N * C, D2)[:, :, :T], last


def _heads(s, *names):
    """The named inputs as [B, H, T, D] in 32 bits, keys and queries repeated
    for the value heads that share them, and g as [B, H, T] in 64."""
    case, cu = s["case"], s["cu"]
    Hk, Hv = case["Hk"], case["Hv"]
    got = []
    for n in names:
        x = s[n] if cu is None else _pad_rows(s[n], cu, case["T"])
        x = x.float().transpose(1, 2)
        got.append(x.repeat_interleave(Hv // Hk, 1) if x.shape[1] != Hv else x)
    g = s["g"].double()
    if g.dim() == 1:
        g = g.expand(s["q"].shape[0], s["q"].shape[1], Hv)
    g = g if cu is None else _pad_rows(g, cu, case["T"])
    return got + [g.transpose(1, 2)]


def _rows(x, s, dtype):
    x = x.transpose(1, 2)
    return (x if s["cu"] is None else _unpad_rows(x, s["cu"])).to(dtype).contiguous()


def _plain_forward(s):
    q, k, v, g = _heads(s, "q", "k", "v")
    o, ht = _decayed(q, k, v, g, s["h0"])
    return _rows(o, s, DT[s["case"]["out"]]), ht


def _plain_backward(s):
    case = s["case"]
    q, k, v, do, g = _heads(s, "q", "k", "v", "do")
    h0, dht = s["h0"], s["dht"]
    dq, last = _decayed(do, v, k, g, None if h0 is None else h0.mT)
    # time reversed: the gradient of S_t decays by the NEXT token's factor
    back = torch.cat([torch.zeros_like(g[..., :1]), g.flip(-1)[..., :-1]], -1)
    dv, first = _decayed(k.flip(2), q.flip(2), do.flip(2), back, dht)
    dk, _ = _decayed(v.flip(2), do.flip(2), q.flip(2), back, None if dht is None else dht.mT)
    dv, dk = dv.flip(2), dk.flip(2)
    dg = ((q.double() * dq).sum(-1) - (k.double() * dk).sum(-1)).flip(-1).cumsum(-1).flip(-1)
    if dht is not None:
        dg = dg + (last.mT.double() * dht).sum((-2, -1))[..., None]
    dh0 = torch.exp(g[..., 0]).float()[..., None, None] * first
    B, Hv, T, Dk = dq.shape
    dq, dk = (a.reshape(B, case["Hk"], Hv // case["Hk"], T, Dk).sum(2) for a in (dq, dk))
    out = DT[case["out"]]
    dg = _rows(dg[..., None], s, torch.float64)[..., 0]
    dg = dg.sum((0, 1)) if case["gate"] == "head" else dg
    return tuple(_rows(a, s, out) for a in (dq, dk, dv)) + (dg.float(), dh0)


def _norm_parts(s):
    x = s["x"].float()
    if s["case"]["center"]:
        x = x - x.mean(-1, keepdim=True)
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    u = x * r * s["w"]
    return x * r, r, u if s["b"] is None else u + s["b"]


def _plain_norm(s):
    _, _, u = _norm_parts(s)
    act = s["case"]["act"]
    if act == "gate":
        z = s["z"].float()
        u = u * z * torch.sigmoid(z)
    elif act == "silu":
        u = u * torch.sigmoid(u)
    return u.to(DT[s["case"]["out"]])


def _plain_norm_backward(s):
    case, out = s["case"], DT[s["case"]["out"]]
    n, r, u = _norm_parts(s)
    dy = s["dy"].float()
    res = {}
    du = dy
    if case["act"] == "gate":
        z = s["z"].float()
        g = torch.sigmoid(z)
        du = dy * z * g
        res["dz"] = (dy * u * g * (1 + z * (1 - g))).to(out)
    elif case["act"] == "silu":
        g = torch.sigmoid(u)
        du = dy * g * (1 + u * (1 - g))
    dn = du * s["w"]
    dx = dn - n * (dn * n).mean(-1, keepdim=True)
    if case["center"]:
        dx = dx - dn.mean(-1, keepdim=True)
    res["dx"] = (r * dx).to(out)
    over = (0, 1) if case["shared"] else (0,)
    res["dw"] = (du * n).sum(over, dtype=torch.float64).float()
    if s["b"] is not None:
        res["db"] = du.sum(over, dtype=torch.float64).float()
    return res


# ---- one pass -------------------------------------------------------------

def run(state):
    case = state["case"]
    kind = case["kind"]
    if not own:
        return {"forward": _plain_forward, "backward": _plain_backward, "norm": _plain_norm,
                "norm_backward": _plain_norm_backward}[kind](state)
    import gated_delta_rule_54_amd as gdr
    s, out = state, DT[case["out"]]
    if kind == "forward":
        return gdr.gdr_linear_forward(s["q"], s["k"], s["v"], s["g"], s["h0"], ht=s["ht"], out_dtype=out,
                                      cu_seqlens=s["cu"], max_seqlen=case["T"] if case["lengths"] else None)
    if kind == "backward":
        return gdr.gdr_linear_backward(s["q"], s["k"], s["v"], s["g"], s["h0"], s["do"], s["dht"], out_dtype=out,
                                       cu_seqlens=s["cu"], max_seqlen=case["T"] if case["lengths"] else None)
    how = dict(center=case["center"], silu=case["act"] == "silu", eps=EPS, out_dtype=out)
    if kind == "norm":
        return gdr.gdr_group_norm_forward(s["x"], s["w"], s["b"], s["z"], **how)
    dx, dz, dw, db = gdr.gdr_group_norm_backward(s["x"], s["w"], s["b"], s["z"], s["dy"], **how)
    res = {"dx": dx, "dw": dw}
    if dz is not None:
        res["dz"] = dz
    if db is not None:
        res["db"] = db
    return res


# ---- what a pass cannot do without ----------------------------------------

def work(case):
    size = {BF16: 2, F32: 4}
    i, o = size[case["io"]], size[case["out"]]
    if case["kind"].startswith("norm"):
        n = case["rows"] * case["G"] * case["D"]
        c = 4 * (case["D"] if case["shared"] else case["G"] * case["D"])
        ins, outs = (2 if case["act"] == "gate" else 1), 1
        params = 2 if case["center"] else 1
        if case["kind"] == "norm":
            return {"bytes": n * (ins * i + outs * o) + params * c, "flops": 10 * n}
        return {"bytes": n * ((ins + 1) * i + ins * o) + 2 * params * c, "flops": 25 * n}
    B, T, Hk, Hv, Dk, Dv = (case[n] for n in ("B", "T", "Hk", "Hv", "Dk", "Dv"))
    rows = int(_lengths(B, T).sum()) if case["lengths"] else B * T
    gate = 4 * (Hv if case["gate"] == "head" else rows * Hv)
    st = 4 * B * Hv * Dk * Dv
    qk, vv = rows * Hk * Dk, rows * Hv * Dv
    if case["kind"] == "forward":
        return {"bytes": 2 * qk * i + vv * (i + o) + gate + st * (2 if case["state"] else 1),
                "flops": 4 * rows * Hv * Dk * Dv}
    return {"bytes": 2 * qk * (i + o) + vv * (2 * i + o) + 2 * gate + st * (3 if case["state"] else 1),
            "flops": 10 * rows * Hv * Dk * Dv}


# ---- the definitions, in 64 bits ------------------------------------------

def _recurrence(s):
    """Token by token over one state per sequence and value head: the outputs
    of the forward and, for a VJP case, the gradients."""
    case, cu = s["case"], s["cu"]
    Hk, Hv, T = case["Hk"], case["Hv"], case["T"]
    q, k, v = (s[n].double() for n in ("q", "k", "v"))
    rows = q.shape[1]
    starts = torch.arange(case["B"], device=q.device) * rows if cu is None else cu[:-1]
    lens = torch.full_like(starts, T) if cu is None else cu[1:] - cu[:-1]
    q, k, v = (a.flatten(0, 1) for a in (q, k, v))
    g = s["g"].double()
    a = torch.exp(g.expand(q.shape[0], Hv) if g.dim() == 1 else g.flatten(0, 1))
    head = torch.arange(Hv, device=q.device) // (Hv // Hk)
    S = torch.zeros(case["B"], Hv, case["Dk"], case["Dv"], dtype=torch.float64, device=q.device)
    if s["h0"] is not None:
        S = s["h0"].double()
    back = case["kind"] == "backward"
    do = s["do"].double().flatten(0, 1) if back else None
    o = None if back else torch.zeros_like(v)
    dq = torch.zeros(q.shape[0], Hv, case["Dk"], dtype=torch.float64, device=q.device) if back else None
    uneven = case["lengths"] > 0
    for t in range(T):
        live = (lens > t).nonzero()[:, 0] if uneven else slice(None)
        r = starts[live] + t
        new = a[r][..., None, None] * S[live] + k[r][:, head, :, None] * v[r][:, :, None, :]
        S = S.index_copy(0, live, new) if uneven else new
        if back:
            dq[r] = (new @ do[r][..., None])[..., 0]
        else:
            o[r] = (q[r][:, head][:, :, None, :] @ new)[:, :, 0]
    if not back:
        return o.reshape(s["v"].shape), S
    dk, dv = torch.zeros_like(dq), torch.zeros_like(v)
    dg = torch.zeros_like(a)
    dS = torch.zeros_like(S) if s["dht"] is None else s["dht"].double()
    run_dg = (S * dS).sum((-2, -1))
    for t in reversed(range(T)):
        live = (lens > t).nonzero()[:, 0] if uneven else slice(None)
        r = starts[live] + t
        D = dS[live] + q[r][:, head, :, None] * do[r][:, :, None, :]
        dk[r] = (D @ v[r][..., None])[..., 0]
        dv[r] = (k[r][:, head][:, :, None, :] @ D)[:, :, 0]
        now = run_dg[live] + (q[r][:, head] * dq[r]).sum(-1) - (k[r][:, head] * dk[r]).sum(-1)
        dg[r] = now
        D = a[r][..., None, None] * D
        if uneven:
            run_dg, dS = run_dg.index_copy(0, live, now), dS.index_copy(0, live, D)
        else:
            run_dg, dS = now, D
    dq, dk = (x.reshape(-1, Hk, Hv // Hk, case["Dk"]).sum(2).reshape(s["q"].shape) for x in (dq, dk))
    dg = dg.sum(0) if case["gate"] == "head" else dg.reshape(s["g"].shape)
    return dq, dk, dv.reshape(s["v"].shape), dg, dS


def _norm_exact(s):
    case = s["case"]
    x, w = s["x"].double(), s["w"].double()
    b = 0.0 if s["b"] is None else s["b"].double()
    mu = x.mean(-1, keepdim=True) if case["center"] else 0.0
    sd = torch.sqrt(((x - mu) ** 2).mean(-1, keepdim=True) + EPS)
    hat = (x - mu) / sd
    u = hat * w + b
    z = s["z"].double() if case["act"] == "gate" else None
    if case["kind"] == "norm":
        return u * z / (1 + torch.exp(-z)) if z is not None else u / (1 + torch.exp(-u)) if case["act"] == "silu" else u
    dy, res = s["dy"].double(), {}
    du = dy
    if z is not None:
        e = 1 / (1 + torch.exp(-z))
        du = dy * (z * e)
        res["dz"] = dy * u * (e + z * e * (1 - e))
    elif case["act"] == "silu":
        e = 1 / (1 + torch.exp(-u))
        du = dy * (e + u * e * (1 - e))
    d = du * w
    proj = hat * (d * hat).mean(-1, keepdim=True)
    res["dx"] = (d - proj - (d.mean(-1, keepdim=True) if case["center"] else 0.0)) / sd
    axes = (0, 1) if case["shared"] else (0,)
    res["dw"] = (du * hat).sum(axes)
    if s["b"] is not None:
        res["db"] = du.sum(axes)
    return res


def exact(case, seed):
    s = prepare(case, seed)
    return _norm_exact(s) if case["kind"].startswith("norm") else _recurrence(s)
