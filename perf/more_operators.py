"""The operators of an attention layer beside the recurrences, as they are
timed and compared: rotary positions (forward, VJP), appending keys and values
to a paged cache, attention of one new token over that cache, and causal
attention with a sliding window and first tokens that stay visible (forward,
and a training step's forward with VJP).

With ``own`` false, ``run`` computes a case in elementary torch operations in
32 bits (angles in 64); with ``own`` true it makes the library's calls.
``exact`` gives the same outputs from the definitions in 64 bits.
"""

import math

import numpy as np
import torch

own = False

BF16, F32 = "bf16", "f32"
DT = {BF16: torch.bfloat16, F32: torch.float32}


# ---- the cases ------------------------------------------------------------

def rotary(kind, B, T, Hq, Hk, D, R, io=BF16, out=BF16, axes=1, cycled=False, adjacent=False):
    """Rotary positions of q (Hq heads) and k (Hk) over the first R of D
    channels.  axes: positions a token has (time, height, width); cycled: the
    pairs take the axes in turn; adjacent: pairs are (2i, 2i + 1)."""
    return dict(kind=kind, B=B, T=T, Hq=Hq, Hk=Hk, D=D, R=R, io=io, out=out, axes=axes, cycled=cycled,
                adjacent=adjacent)


def append(B, T, Hq, Hk, D, R, page, io=BF16, heads=False, lengths=0, past=0, axes=1):
    """T new tokens for each of B sequences (lengths: that many prompts of
    unequal length, at most T, laid end to end) behind up to `past` old ones,
    into pages of `page` tokens; heads: pages are laid out head by head."""
    return dict(kind="append", B=B, T=T, Hq=Hq, Hk=Hk, D=D, R=R, page=page, io=io, heads=heads, lengths=lengths,
                past=past, axes=axes)


def decode(B, L, Hq, Hk, D, page, io=BF16, out=BF16, heads=False, window=0, sinks=0, even=False):
    """One new token for each of B sequences of up to L tokens (even: all of
    them L) in pages of `page` tokens."""
    return dict(kind="decode", B=B, L=L, Hq=Hq, Hk=Hk, D=D, page=page, io=io, out=out, heads=heads, window=window,
                sinks=sinks, even=even)


def attention(kind, B, T, Hq, Hk, D, io=BF16, out=BF16, window=0, sinks=0, lengths=0):
    """Causal attention over B sequences of T tokens, or over `lengths` ragged
    ones of at most T; window 0: all earlier tokens."""
    return dict(kind=kind, B=B, T=T, Hq=Hq, Hk=Hk, D=D, io=io, out=out, window=window, sinks=sinks, lengths=lengths)


def listed():
    return [
        # queries and keys of a training batch, the benchmark step's tokens
        dict(rotary("rotary", 4, 4096, 32, 8, 128, 128), name="rotary B4 T4096"),
        # gradients through positions of image patches: three axes in turn, a quarter of a wide head rotated
        dict(rotary("rotary_backward", 1, 2777, 16, 2, 256, 64, axes=3, cycled=True), name="rotary backward axes"),
        # a ragged prefill of 17 prompts into the cache
        dict(append(17, 2048, 32, 8, 128, 128, 64, lengths=17), name="append ragged 17"),
        # a decoding step of 64 sequences, wide heads of which a quarter is rotated
        dict(append(64, 1, 16, 2, 256, 64, 16, past=4096), name="append B64"),
        # decoding: one long document; a batch of unequal lengths; a few short ones in 32 bits with a window
        dict(decode(1, 131072, 32, 8, 128, 64, heads=True, even=True), name="decode B1 L131072"),
        dict(decode(64, 8192, 16, 2, 256, 16), name="decode B64 L8192"),
        dict(decode(3, 777, 6, 2, 96, 16, io=F32, out=F32, window=300, sinks=4), name="decode f32 B3 L777"),
        # the attention layer of the training batch, all earlier tokens visible
        dict(attention("attention", 4, 4096, 32, 8, 128), name="attention B4 T4096"),
        # a ragged prefill through a layer with a window and sinks
        dict(attention("attention", 17, 2048, 16, 4, 64, window=512, sinks=16, lengths=17), name="attention ragged 17"),
        # a short odd prompt in 32 bits
        dict(attention("attention", 2, 333, 6, 2, 96, io=F32, out=F32), name="attention f32 T333"),
        # training: a layer with a window; a short odd sequence with a head for each query head
        dict(attention("train", 2, 4096, 32, 8, 128, window=1024, sinks=4), name="train B2 T4096"),
        dict(attention("train", 1, 777, 8, 8, 80), name="train B1 T777"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["rotary", "rotary_backward", "append", "append", "decode", "decode", "decode", "attention",
                       "attention", "train", "train"])
    io = rng.choice([BF16, BF16, BF16, F32])
    out = F32 if io == F32 else rng.choice([BF16, BF16, BF16, F32])
    D = rng.choice([64, 64, 80, 96, 128, 128, 128, 192, 256])
    Hk = rng.choice([1, 2, 3, 4, 8])
    Hq = Hk * rng.choice([1, 2, 4, 4, 6, 8])
    R = rng.choice([D, D, 32, 64])
    axes = rng.choice([1, 1, 1, 2, 3])
    if kind.startswith("rotary"):
        T = _log_int(rng, 1, 4096)
        return rotary(kind, _log_int(rng, 1, 4), T, min(Hq, 32), Hk, min(D, 128) if T > 1024 else D,
                      min(R, 128) if T > 1024 else R, io, out, axes, rng.random() < 0.5, rng.random() < 0.3)
    page = rng.choice([16, 16, 32, 64, 128, 48])
    heads = rng.random() < 0.5
    if kind == "append":
        if rng.random() < 0.5:
            return append(_log_int(rng, 1, 256), rng.choice([1, 1, 1, 2, 4]), min(Hq, 32), Hk, D, R, page, io, heads, 0,
                          _log_int(rng, 1, 4096), axes)
        B = _log_int(rng, 2, 16)
        return append(B, _log_int(rng, 8, 1024), min(Hq, 32), Hk, D, R, page, io, heads, rng.choice([0, B]),
                      rng.choice([0, 100]), axes)
    window = rng.choice([0, 0, _log_int(rng, 1, 2048)])
    sinks = rng.choice([0, 1, 4, 77]) if window else 0
    if kind == "decode":
        L = _log_int(rng, 1, 65536)
        most = max(1, min(128, (1 << 29) // (L * Hk * D)))
        return decode(_log_int(rng, 1, most), L, min(Hq, 64), Hk, D, page, io, out, heads, window, sinks,
                      rng.random() < 0.3)
    T = _log_int(rng, 2, 4096 if kind == "attention" and io == BF16 else 2048 if io == BF16 else 1024)
    B = _log_int(rng, 1, max(1, min(8, 8192 // T)))
    return attention(kind, B, T, min(Hq, 32), Hk, D, io, out, window, sinks, rng.choice([0, 0, B]) if B > 1 else 0)


def _lengths(B, T):
    """The lengths of B prompts: from a sixteenth of T to T, the first one T."""
    lens = np.random.default_rng(B * T).integers(max(1, T // 16), T + 1, B)
    lens[0] = T
    return lens


def _new(case):
    """New tokens of each sequence."""
    return _lengths(case["B"], case["T"]) if case["lengths"] else np.full(case["B"], case["T"])


def _held(case):
    """Tokens that each sequence of a cache holds (after an append)."""
    if case["kind"] == "decode":
        return np.full(case["B"], case["L"]) if case["even"] else _lengths(case["B"], case["L"])
    old = _lengths(case["B"], case["past"]) if case["past"] else 0
    return _new(case) + old


def _sections(case):
    """Pairs of each axis: the first has what the others leave."""
    half, axes = case["R"] // 2, case["axes"]
    return (half - (axes - 1) * (half // axes),) + (half // axes,) * (axes - 1)


# ---- inputs ---------------------------------------------------------------

def _freq(R, dev):
    return torch.pow(10000.0, -2.0 * torch.arange(R // 2, device=dev, dtype=torch.float64) / R).float()


def _cache(case, s, randn, dev):
    """Paged buffers with room for every sequence, their pages in any order
    and a few of nobody's."""
    B, ps, Hk, D = case["B"], case["page"], case["Hk"], case["D"]
    held = _held(case)
    need = -(-held // ps)
    pages = int(need.sum()) + 3
    order = torch.randperm(pages, generator=s["gen"], device=dev).to(torch.int32)
    table = torch.full((B, int(need.max()) + 1), -1, dtype=torch.int32, device=dev)
    first = torch.from_numpy(np.concatenate([[0], np.cumsum(need)[:-1]])).to(dev)
    at = torch.arange(table.shape[1], device=dev)
    used = at < torch.from_numpy(need).to(dev)[:, None]
    table[used] = order[(first[:, None] + at)[used]]
    s["table"] = table
    s["lens"] = torch.from_numpy(held.astype(np.int64)).to(dev)
    for name in ("kc", "vc"):
        if case["heads"]:
            s[name] = randn(pages, Hk, ps, D).to(DT[case["io"]]).transpose(1, 2)
        else:
            s[name] = randn(pages, ps, Hk, D).to(DT[case["io"]])


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)

    def randn(*shape):
        return torch.randn(shape, generator=gen, device=dev, dtype=torch.float32)

    s = dict(case=case, gen=gen)
    kind, B, Hq, Hk, D = (case[n] for n in ("kind", "B", "Hq", "Hk", "D"))
    io = DT[case["io"]]
    if kind == "decode":
        s["q"] = randn(B, 1, Hq, D).to(io)
        _cache(case, s, randn, dev)
        return s
    s["cu"] = None
    rows = (B, case["T"])
    if case.get("lengths"):
        cu = np.concatenate([[0], np.cumsum(_lengths(B, case["T"]))]).astype(np.int64)
        rows = (1, int(cu[-1]))
        s["cu"] = torch.from_numpy(cu).to(dev)
    # queries, keys and values as column ranges of one projection's rows
    heads = Hq + Hk + (0 if kind.startswith("rotary") else Hk)
    x = randn(*rows, heads, D).to(io)
    s["q"], s["k"], s["v"] = x[..., :Hq, :], x[..., Hq:Hq + Hk, :], x[..., Hq + Hk:, :]
    if kind in ("attention", "train"):
        s["do"] = randn(*rows, Hq, D).to(io) if kind == "train" else None
        return s
    s["freq"] = _freq(case["R"], dev)
    # positions: a token's place in a long context, or frame, row and column of a patch
    shape = rows if case["axes"] == 1 else (case["axes"],) + rows
    s["pos"] = torch.randint(0, 131072 if case["axes"] == 1 else 4096, shape, generator=gen, device=dev)
    if kind == "append":
        _cache(case, s, randn, dev)
        s["pos"] = None if case["axes"] == 1 else s["pos"]  # by default a token's place in its sequence
    return s


# ---- the plain form -------------------------------------------------------

def _pair_axis(case, dev):
    """The axis of each pair."""
    half, axes, sec = case["R"] // 2, case["axes"], _sections(case)
    i = torch.arange(half, device=dev)
    if case.get("cycled"):
        a = i % axes
        return torch.where(i < axes * torch.tensor(sec, device=dev)[a], a, 0)
    return torch.repeat_interleave(torch.arange(axes, device=dev), torch.tensor(sec, device=dev))


def _turns(case, pos, freq):
    """cos and sin of each token and pair, from 64-bit angles: [..., 1, R/2]."""
    p = pos[None] if case["axes"] == 1 else pos
    angle = p[_pair_axis(case, pos.device)].movedim(0, -1).double() * freq.double()
    return torch.cos(angle).float().unsqueeze(-2), torch.sin(angle).float().unsqueeze(-2)


def _rotate(x, cos, sin, case, back=False):
    """x [..., H, D] in 32 bits, its first R channels turned."""
    R = case["R"]
    x = x.float()
    if back:
        sin = -sin
    if case.get("adjacent"):
        a, b = x[..., 0:R:2], x[..., 1:R:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :R // 2], x[..., R // 2:R]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([y, x[..., R:]], -1)


def _plain_rotary(s):
    case = s["case"]
    cos, sin = _turns(case, s["pos"], s["freq"])
    back = case["kind"] == "rotary_backward"
    return tuple(_rotate(s[n], cos, sin, case, back).to(DT[case["out"]]) for n in ("q", "k"))


def _places(s):
    """Sequence and place in it of each new token, in the order of the rows."""
    case, cu, lens = s["case"], s["cu"], s["lens"]
    B, T = case["B"], case["T"]
    if cu is None:
        b = torch.arange(B, device=lens.device)[:, None].expand(B, T)
        return b, lens[:, None] - T + torch.arange(T, device=lens.device)
    row = torch.arange(s["q"].shape[1], device=lens.device)
    b = torch.searchsorted(cu, row, right=True) - 1
    return b[None], (lens[b] - cu[b + 1] + row)[None]


def _plain_append(s):
    case, ps = s["case"], s["case"]["page"]
    b, place = _places(s)
    cos, sin = _turns(case, place if s["pos"] is None else s["pos"], s["freq"])
    page = s["table"][b, place // ps].long()
    s["kc"][page, place % ps] = _rotate(s["k"], cos, sin, case).to(DT[case["io"]])
    s["vc"][page, place % ps] = s["v"]
    return _rotate(s["q"], cos, sin, case).to(DT[case["io"]]), s["kc"], s["vc"]


def _softmax_v(S, seen, v):
    """softmax over the seen keys times v, and the logarithm of the sum."""
    S = S.masked_fill(~seen, -math.inf)
    m = S.amax(-1, keepdim=True)
    P = torch.exp(S - m)
    total = P.sum(-1, keepdim=True)
    return (P @ v) / total, (m + torch.log(total))[..., 0]


def _plain_decode(s):
    case = s["case"]
    B, Hq, Hk, D = (case[n] for n in ("B", "Hq", "Hk", "D"))
    lens = s["lens"][:, None]
    used = s["table"].clamp(min=0).long()
    k, v = (s[n][used].flatten(1, 2).float().transpose(1, 2) for n in ("kc", "vc"))  # [B, Hk, L, D]
    j = torch.arange(k.shape[2], device=k.device)
    seen = j < lens
    if case["window"]:
        seen = seen & ((lens - 1 - j < case["window"]) | (j < case["sinks"]))
    v = v.masked_fill(~seen[:, None, :, None], 0.0)
    q = s["q"].float().reshape(B, Hk, Hq // Hk, D)
    o, lse = _softmax_v((q @ k.mT) * D ** -0.5, seen[:, None, None], v)
    return o.reshape(B, 1, Hq, D).to(DT[case["out"]]), lse.reshape(B, 1, Hq)


def _seen(case, T, dev):
    i, j = torch.arange(T, device=dev)[:, None], torch.arange(T, device=dev)
    low = j <= i
    if not case["window"]:
        return low
    return low & ((i - j < case["window"]) | (j < case["sinks"]))


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


def _grouped(s, name):
    """[B, T, H, D] as [B, Hk, H / Hk, T, D] in 32 bits."""
    x = s[name] if s["cu"] is None else _pad_rows(s[name], s["cu"], s["case"]["T"])
    return x.float().unflatten(2, (s["case"]["Hk"], -1)).permute(0, 2, 3, 1, 4)


def _rows(x, s, dtype):
    x = x.permute(0, 3, 1, 2, 4).flatten(2, 3)
    return (x if s["cu"] is None else _unpad_rows(x, s["cu"])).to(dtype).contiguous()


def _plain_attention(s):
    case, out = s["case"], DT[s["case"]["out"]]
    q, k, v = (_grouped(s, n) for n in ("q", "k", "v"))
    scale = case["D"] ** -0.5
    seen = _seen(case, case["T"], q.device)
    S = (q @ k.mT) * scale
    o, lse = _softmax_v(S, seen, v)
    res = {"o": _rows(o, s, out), "lse": _rows(lse[..., None], s, torch.float32)[..., 0]}
    if case["kind"] == "train":
        do = _grouped(s, "do")
        P = torch.exp(S.masked_fill_(~seen, -math.inf) - lse[..., None])
        res["dv"] = _rows((P.mT @ do).sum(2, keepdim=True), s, out)
        dS = P * (do @ v.mT - (do * o).sum(-1, keepdim=True))
        res["dq"] = _rows((dS @ k) * scale, s, out)
        res["dk"] = _rows((dS.mT @ q).sum(2, keepdim=True) * scale, s, out)
    return res


# ---- one pass -------------------------------------------------------------

def run(state):
    s, case = state, state["case"]
    kind = case["kind"]
    if not own:
        return {"rotary": _plain_rotary, "rotary_backward": _plain_rotary, "append": _plain_append,
                "decode": _plain_decode, "attention": _plain_attention, "train": _plain_attention}[kind](s)
    import gated_delta_rule_54_amd as gdr
    if kind in ("rotary", "rotary_backward"):
        call = gdr.gdr_rotary_forward if kind == "rotary" else gdr.gdr_rotary_backward
        return call(s["q"], s["k"], s["pos"], s["freq"], section=_sections(case) if case["axes"] > 1 else None,
                    cycled=case["cycled"] and case["axes"] > 1, adjacent=case["adjacent"], out_dtype=DT[case["out"]])
    if kind == "append":
        q = gdr.gdr_cache_append(s["k"], s["v"], s["kc"], s["vc"], s["table"], s["lens"], s["freq"], s["pos"],
                                 q=s["q"], section=_sections(case) if case["axes"] > 1 else None,
                                 cu_seqlens=s["cu"], max_seqlen=case["T"] if case["lengths"] else None)
        return q, s["kc"], s["vc"]
    if kind == "decode":
        return gdr.gdr_cache_attention(s["q"], s["kc"], s["vc"], s["table"], s["lens"], window=case["window"] or None,
                                       sinks=case["sinks"], out_dtype=DT[case["out"]])
    how = dict(window=case["window"] or None, sinks=case["sinks"], cu_seqlens=s["cu"],
               max_seqlen=case["T"] if case["lengths"] else None)
    o, lse = gdr.gdr_attention_forward(s["q"], s["k"], s["v"], out_dtype=DT[case["out"]], **how)
    res = {"o": o, "lse": lse}
    if kind == "train":
        res["dq"], res["dk"], res["dv"] = gdr.gdr_attention_backward(s["q"], s["k"], s["v"], o, lse, s["do"], **how)
    return res


# ---- what a pass cannot do without ----------------------------------------

def _visible(case, n):
    """Keys that the token with n of them (its own the last) sees."""
    n = np.asarray(n, dtype=np.float64)
    if not case["window"]:
        return n
    return np.minimum(n, case["window"] + np.minimum(case["sinks"], np.maximum(0, n - case["window"])))


def work(case):
    size = {BF16: 2, F32: 4}
    kind, B, Hq, Hk, D = (case[n] for n in ("kind", "B", "Hq", "Hk", "D"))
    i = size[case["io"]]
    if kind == "decode":
        seen = float(_visible(case, _held(case)).sum())
        return {"bytes": seen * 2 * Hk * D * i + B * Hq * (D * (i + size[case["out"]]) + 4), "flops": seen * 4 * Hq * D}
    rows = int(_new(case).sum()) if case.get("lengths") else B * case["T"]
    if kind in ("rotary", "rotary_backward"):
        n = rows * (Hq + Hk)
        return {"bytes": n * D * (i + size[case["out"]]) + 8 * rows * case["axes"], "flops": 3 * n * case["R"]}
    if kind == "append":
        n = rows * (Hq + 2 * Hk) * D
        return {"bytes": 2 * n * i + (0 if case["axes"] == 1 else 8 * rows * case["axes"]),
                "flops": 3 * rows * (Hq + Hk) * case["R"]}
    o = size[case["out"]]
    pairs = sum(float(_visible(case, np.arange(1, n + 1)).sum()) for n in _new(case))
    q, kv = rows * Hq * D, 2 * rows * Hk * D
    if kind == "attention":
        return {"bytes": q * (i + o) + kv * i + 4 * rows * Hq, "flops": pairs * 4 * Hq * D}
    return {"bytes": q * (2 * i + 2 * o) + kv * (i + o) + 4 * rows * Hq, "flops": pairs * 14 * Hq * D}


# ---- the definitions, in 64 bits ------------------------------------------

def _turned(x, pos, freq, case, sign):
    """x [..., H, D] as complex numbers times e^{i angle}, pair by pair."""
    R, x = case["R"], x.double()
    axis = []
    left = list(_sections(case))
    for i in range(R // 2):
        if case.get("cycled"):
            a = i % case["axes"]
            a = a if left[a] > 0 or a == 0 else 0
        else:
            a = next(n for n, c in enumerate(left) if c > 0)
        left[a] -= 1
        axis.append(a)
    p = pos.double() if case["axes"] > 1 else pos.double()[None]
    angle = torch.stack([p[a] * float(f) for a, f in zip(axis, freq.double().tolist())], -1)[..., None, :]
    near, far = (slice(0, R, 2), slice(1, R, 2)) if case.get("adjacent") else (slice(0, R // 2), slice(R // 2, R))
    z = torch.complex(x[..., near].contiguous(), x[..., far].contiguous())
    z = z * torch.polar(torch.ones_like(angle), sign * angle)
    y = x.clone()
    y[..., near], y[..., far] = z.real, z.imag
    return y


def _exact_append(s):
    case = s["case"]
    kc, vc = s["kc"].double(), s["vc"].double()
    q = torch.empty_like(s["q"], dtype=torch.float64)
    row = 0
    flat = [s[n].flatten(0, 1) for n in ("q", "k", "v")]
    pos = None if s["pos"] is None else s["pos"].flatten(-2)
    q = q.flatten(0, 1)
    for b, (n, held) in enumerate(zip(_new(case).tolist(), _held(case).tolist())):
        at = torch.arange(held - n, held, device=kc.device)
        rows = slice(row, row + n)
        p = at if pos is None else pos[..., rows]
        q[rows] = _turned(flat[0][rows], p, s["freq"], case, 1)
        page = s["table"][b].long()[at // case["page"]]
        kc[page, at % case["page"]] = _turned(flat[1][rows], p, s["freq"], case, 1)
        vc[page, at % case["page"]] = flat[2][rows].double()
        row += n
    return q.reshape(s["q"].shape), kc, vc


def _exact_decode(s):
    case = s["case"]
    B, Hq, Hk, D = (case[n] for n in ("B", "Hq", "Hk", "D"))
    o = torch.zeros(B, 1, Hq, D, dtype=torch.float64, device=s["q"].device)
    lse = torch.full((B, 1, Hq), -math.inf, dtype=torch.float64, device=o.device)
    for b, n in enumerate(_held(case).tolist()):
        j = list(range(n)) if not case["window"] else sorted(
            set(range(min(n, case["sinks"]))) | set(range(max(0, n - case["window"]), n)))
        j = torch.tensor(j, device=o.device)
        page = s["table"][b].long()[j // case["page"]]
        k, v = (s[c][page, j % case["page"]].double() for c in ("kc", "vc"))  # [n, Hk, D]
        for h in range(Hk):
            g = slice(h * (Hq // Hk), (h + 1) * (Hq // Hk))
            w = s["q"][b, 0, g].double() @ k[:, h].T / math.sqrt(D)
            o[b, 0, g] = torch.softmax(w, -1) @ v[:, h]
            lse[b, 0, g] = torch.logsumexp(w, -1)
    return o, lse


def _exact_attention(s):
    case = s["case"]
    Hq, Hk, D = (case[n] for n in ("Hq", "Hk", "D"))
    train = case["kind"] == "train"
    q, k, v = (s[n].flatten(0, 1).double() for n in ("q", "k", "v"))
    res = {"o": torch.empty_like(q), "lse": torch.empty(q.shape[:2], dtype=torch.float64, device=q.device)}
    if train:
        do = s["do"].flatten(0, 1).double()
        res.update(dq=torch.empty_like(q), dk=torch.zeros_like(k), dv=torch.zeros_like(v))
    row, scale = 0, 1 / math.sqrt(D)
    for n in _new(case).tolist():
        i = torch.arange(n, device=q.device)
        far = i[:, None] - i
        hidden = far < 0
        if case["window"]:
            hidden |= (far >= case["window"]) & (i >= case["sinks"])
        r = slice(row, row + n)
        for h in range(Hq):
            m = h // (Hq // Hk)
            w = (q[r, h] @ k[r, m].T * scale).masked_fill_(hidden, -math.inf)
            res["lse"][r, h] = torch.logsumexp(w, -1)
            P = torch.softmax(w, -1)
            res["o"][r, h] = P @ v[r, m]
            if train:
                d = do[r, h]
                res["dv"][r, m] += P.T @ d
                dP = d @ v[r, m].T
                w = P * (dP - (P * dP).sum(-1, keepdim=True)) * scale
                res["dq"][r, h] = w @ k[r, m]
                res["dk"][r, m] += w.T @ q[r, h]
        row += n
    shape = {"o": s["q"], "dq": s["q"], "dk": s["k"], "dv": s["v"]}
    return {n: x.reshape(s["q"].shape[:3] if n == "lse" else shape[n].shape) for n, x in res.items()}


def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] in ("rotary", "rotary_backward"):
        sign = 1 if case["kind"] == "rotary" else -1
        return tuple(_turned(s[n], s["pos"], s["freq"], case, sign) for n in ("q", "k"))
    return {"append": _exact_append, "decode": _exact_decode, "attention": _exact_attention,
            "train": _exact_attention}[case["kind"]](s)
