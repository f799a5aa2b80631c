"""Binding of the attention layer beside the recurrent ones (include/gdr.h):
rotary positions, the append to a paged cache of keys and values, attention of
one new token over it, and causal attention over whole sequences with its VJP.
Argument marshalling only, as in ``linear``.

q, k and v may be column ranges of a wider row, as there; a cache may have any
strides with dense channels.  Every other tensor is contiguous.  Outputs and
workspaces are allocated on the stream the call runs on: the current stream of
the tensors' device, or ``stream``.
"""

import ctypes
import operator

import torch

from .binding import _ragged_dims, lib
from .linear import _check_status, _device, _dtype, _here, _on, _ptr, _raw_stream, _row_stride, _want, _workspace

GDR_ROTARY_ADJACENT, GDR_ROTARY_CYCLED = 1, 2


class GdrRotary(ctypes.Structure):
    _fields_ = [("R", ctypes.c_int32), ("axes", ctypes.c_int32), ("section", ctypes.c_int32 * 4),
                ("flags", ctypes.c_uint32)]


class GdrRotaryProblem(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("Hq", ctypes.c_int32), ("Hk", ctypes.c_int32), ("D", ctypes.c_int32),
                ("io_dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32), ("rot", GdrRotary),
                ("q_row", ctypes.c_int64), ("k_row", ctypes.c_int64),
                ("qo_row", ctypes.c_int64), ("ko_row", ctypes.c_int64)]


class GdrCache(ctypes.Structure):
    _fields_ = [("pages", ctypes.c_int64), ("page_size", ctypes.c_int32), ("Hk", ctypes.c_int32),
                ("D", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("page_stride", ctypes.c_int64), ("token_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64),
                ("max_pages", ctypes.c_int32), ("table_row", ctypes.c_int64)]


class GdrAppendProblem(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int64), ("T", ctypes.c_int64), ("rows", ctypes.c_int64),
                ("Hq", ctypes.c_int32), ("io_dtype", ctypes.c_int32), ("rot", GdrRotary), ("cache", GdrCache),
                ("q_row", ctypes.c_int64), ("k_row", ctypes.c_int64), ("v_row", ctypes.c_int64)]


class GdrCacheAttentionProblem(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int64), ("Hq", ctypes.c_int32), ("out_dtype", ctypes.c_int32), ("cache", GdrCache),
                ("q_row", ctypes.c_int64), ("max_len", ctypes.c_int64), ("window", ctypes.c_int64),
                ("sinks", ctypes.c_int64), ("scale", ctypes.c_float)]


class GdrAttentionProblem(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int64), ("T", ctypes.c_int64),
                ("Hq", ctypes.c_int32), ("Hk", ctypes.c_int32), ("D", ctypes.c_int32),
                ("io_dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32),
                ("window", ctypes.c_int64), ("sinks", ctypes.c_int64), ("scale", ctypes.c_float),
                ("q_row", ctypes.c_int64), ("k_row", ctypes.c_int64), ("v_row", ctypes.c_int64)]


# A call for a few tokens is bound by the host.  What a call works out from its
# operands' shapes, strides, types and devices, and from its options, is kept by these
# (never by a tensor or its address): the checks that passed, the problem, the
# workspace's size.  Integers are kept with their class: 4.0 equals 4, but is refused.
_plans = {}
_MOST = 4096


def _meta(t):
    return None if t is None else (t.shape, t.stride(), t.dtype, t.device)


def _whole(x, name):
    if x is None:
        return None
    try:
        return operator.index(x)
    except TypeError:
        raise TypeError(f"{name} must be an integer, got {x!r}") from None


def _plan(key, make):
    plan = make()
    if len(_plans) >= _MOST:
        _plans.clear()
    _plans[key] = plan
    return plan


# ---- rotary positions -----------------------------------------------------

def _rotary(freq, section, adjacent, cycled, dev):
    """The turn that freq [R / 2] and the axes' sections describe."""
    flags = (GDR_ROTARY_ADJACENT if adjacent else 0) | (GDR_ROTARY_CYCLED if cycled else 0)
    axes = (ctypes.c_int32 * 4)()
    n = 1
    if section is not None:
        n = len(section)
        if not 1 <= n <= 4:
            raise ValueError("section must name the pairs of 1 to 4 axes")
        axes[:n] = [int(s) for s in section]
    if freq is None:
        return GdrRotary(0, 1, axes, 0)
    if freq.dim() != 1:
        raise ValueError("freq must be [R / 2]")
    _want(freq, "freq", tuple(freq.shape), torch.float32, dev)
    if section is not None and sum(section) != freq.numel():
        raise ValueError(f"section must sum to the {freq.numel()} pairs of freq, got {tuple(section)}")
    return GdrRotary(2 * freq.numel(), n, axes, flags)


def _positions(pos, rot, rows, dev):
    shape = rows if rot.axes == 1 else (rot.axes,) + rows
    if pos is not None and rot.axes == 1 and pos.dim() == len(rows) + 1 and pos.shape[0] == 1:
        shape = (1,) + rows
    _want(pos, "pos", shape, torch.int64, dev)


def _heads(t, name):
    if t.dim() < 2:
        raise ValueError(f"{name} must be [..., heads, dim]")
    return tuple(t.shape[:-2]), t.shape[-2], t.shape[-1]


def _turn(entry, q, k, pos, freq, section, adjacent, cycled, out_dtype, q_out, k_out, stream):
    dev = _device(q, "q")
    if not _here(dev, stream):
        with _on(dev, stream):
            return _turn(entry, q, k, pos, freq, section, adjacent, cycled, out_dtype, q_out, k_out, None)
    section = None if section is None else tuple(section)
    key = (entry, _meta(q), _meta(k), _meta(pos), _meta(freq), _meta(q_out), _meta(k_out), section, adjacent, cycled,
           out_dtype)
    plan = _plans.get(key) or _plan(key, lambda: _turn_plan(q, k, pos, freq, section, adjacent, cycled, out_dtype,
                                                            q_out, k_out, dev))
    ref, q_shape, k_shape = plan
    if q_out is None:
        q_out = torch.empty(q_shape, dtype=out_dtype, device=dev)
    if k is not None and k_out is None:
        k_out = torch.empty(k_shape, dtype=out_dtype, device=dev)
    st = getattr(lib(), entry)(ref, q.data_ptr(), _ptr(k), _ptr(pos), _ptr(freq), q_out.data_ptr(), _ptr(k_out),
                               _raw_stream(dev.index))
    if st:
        _check_status(st, entry)
    return q_out, k_out


def _turn_plan(q, k, pos, freq, section, adjacent, cycled, out_dtype, q_out, k_out, dev):
    rows, Hq, D = _heads(q, "q")
    Hk = 0
    if k is not None:
        Hk = k.shape[-2] if k.dim() >= 2 else 0
        _want(k, "k", rows + (Hk, D), q.dtype, dev, False)
    elif k_out is not None:
        raise ValueError("k_out without k")
    rot = _rotary(freq, section, adjacent, cycled, dev)
    if rot.R and pos is None:
        raise ValueError("pos is required")
    _positions(pos, rot, rows, dev)
    dt = out_dtype if q_out is None else q_out.dtype
    for t, name, H in ((q_out, "q_out", Hq), (k_out, "k_out", Hk)):
        if t is not None:
            _want(t, name, rows + (H, D), t.dtype, dev, False)
    if k is not None and (out_dtype if k_out is None else k_out.dtype) != dt:
        raise TypeError(f"q_out is {dt}, k_out {out_dtype if k_out is None else k_out.dtype}")
    n = 1
    for s in rows:
        n *= s
    strides = [0 if t is None else _row_stride(t, name)
               for t, name in ((q, "q"), (k, "k"), (q_out, "q_out"), (k_out, "k_out"))]
    prob = GdrRotaryProblem(n, Hq, Hk, D, _dtype(q.dtype, "q"), _dtype(dt, "q_out"), rot, *strides)
    return ctypes.byref(prob), rows + (Hq, D), rows + (Hk, D)


def gdr_rotary_forward(q, k, pos, freq, *, section=None, adjacent=False, cycled=False, out_dtype=torch.float32,
                       q_out=None, k_out=None, stream=None):
    """Turns pair i of the first R channels of q [..., Hq, D] and k [..., Hk, D]
    (or None) by pos * freq[i].  Returns (q_out, k_out).

    freq: float32 [R / 2].  pos: int64, one for each row (q's leading axes), or
    [axes, ...] with ``section``, the number of pairs that each axis (time,
    height, width) turns: in that order, or in turns with ``cycled``.  Pairs
    are (i, i + R / 2), with ``adjacent`` (2i, 2i + 1).  ``q_out`` and
    ``k_out`` may be tensors to write into (then their dtype is the output's),
    q and k themselves among them."""
    return _turn("gdr_rotary_forward", q, k, pos, freq, section, adjacent, cycled, out_dtype, q_out, k_out, stream)


def gdr_rotary_backward(dq_out, dk_out, pos, freq, *, section=None, adjacent=False, cycled=False,
                        out_dtype=torch.float32, dq=None, dk=None, stream=None):
    """VJP of gdr_rotary_forward: returns (dq, dk) from the gradients of its
    outputs; arguments as there (``dq`` and ``dk`` may be tensors to write
    into, also in place)."""
    return _turn("gdr_rotary_backward", dq_out, dk_out, pos, freq, section, adjacent, cycled, out_dtype, dq, dk,
                 stream)


# ---- the paged cache ------------------------------------------------------

def _cache(k_cache, v_cache, table, lengths, dev):
    if k_cache.dim() != 4:
        raise ValueError("k_cache must be [pages, page_size, Hk, D]")
    pages, size, Hk, D = k_cache.shape
    _want(k_cache, "k_cache", (pages, size, Hk, D), k_cache.dtype, dev, False)
    _want(v_cache, "v_cache", (pages, size, Hk, D), k_cache.dtype, dev, False)
    st = k_cache.stride()
    if st != v_cache.stride():
        raise ValueError(f"k_cache and v_cache must have the same strides, got {st} and {v_cache.stride()}")
    if st[3] != 1 or (0 in st and any(s == 0 and n > 1 for s, n in zip(st, k_cache.shape))):
        raise ValueError(f"a cache must have dense channels and no expanded axes, got strides {st}")
    if table.dim() != 2 or table.dtype != torch.int32:
        raise TypeError("table must be a 2-d int32 device tensor")
    B, most = table.shape
    if table.device != dev:
        raise ValueError(f"table is on {table.device}, expected {dev}")
    row = table.stride(0) if B > 1 else most
    if (most > 1 and table.stride(1) != 1) or row < most:
        raise ValueError("table must have dense rows that do not overlap")
    _want(lengths, "lengths", (B,), torch.int64, dev)
    return GdrCache(pages, size, Hk, D, _dtype(k_cache.dtype, "k_cache"), st[0], st[1], st[2], most, row)


def gdr_cache_append(k, v, k_cache, v_cache, table, lengths, freq=None, pos=None, *, q=None, section=None,
                     adjacent=False, cycled=False, q_out=None, stream=None, cu_seqlens=None, max_seqlen=None):
    """Stores the new tokens' k (turned as by gdr_rotary_forward where ``freq``
    is given) and v [B, T, Hk, D] in the paged cache, and returns the turned q
    [B, T, Hq, D] in the cache's dtype (None without ``q``).

    k_cache, v_cache: [pages, page_size, Hk, D], written in place; table: int32
    [B, max_pages], each sequence's pages in order (an entry outside the cache
    is a page that is not there: nothing is stored to it); lengths: int64 [B],
    the tokens that each sequence holds with the new ones, which are its last.
    ``pos`` (as for gdr_rotary_forward) is by default each token's place in its
    sequence.  No two tokens may go to one place of the cache.  ``cu_seqlens`` /
    ``max_seqlen`` as for ``gdr_forward``: rows that no sequence covers are
    neither read nor written."""
    dev = _device(k, "k")
    if not _here(dev, stream):
        with _on(dev, stream):
            return gdr_cache_append(k, v, k_cache, v_cache, table, lengths, freq, pos, q=q, section=section,
                                    adjacent=adjacent, cycled=cycled, q_out=q_out, cu_seqlens=cu_seqlens,
                                    max_seqlen=max_seqlen)
    if k.dim() != 4:
        raise ValueError("k must be [B, T, Hk, D]")
    dims = k.shape[:2] if cu_seqlens is None else _ragged_dims(k, cu_seqlens, max_seqlen)
    section = None if section is None else tuple(section)
    key = ("append", _meta(k), _meta(v), _meta(k_cache), _meta(v_cache), _meta(table), _meta(lengths), _meta(freq),
           _meta(pos), _meta(q), _meta(q_out), _meta(cu_seqlens), dims, max_seqlen.__class__, section, adjacent, cycled)
    plan = _plans.get(key) or _plan(key, lambda: _append_plan(k, v, k_cache, v_cache, table, lengths, freq, pos, q,
                                                              section, adjacent, cycled, q_out, cu_seqlens, dims, dev))
    ref, shape = plan
    if q is not None and q_out is None:
        q_out = torch.empty(shape, dtype=k_cache.dtype, device=dev)
    args = (lengths.data_ptr(), table.data_ptr(), _ptr(q), k.data_ptr(), v.data_ptr(), _ptr(pos), _ptr(freq),
            _ptr(q_out), k_cache.data_ptr(), v_cache.data_ptr(), _raw_stream(dev.index))
    if cu_seqlens is not None:
        st = lib().gdr_cache_append_varlen(ref, cu_seqlens.data_ptr(), *args)
    else:
        st = lib().gdr_cache_append(ref, *args)
    if st:
        _check_status(st, "gdr_cache_append")
    return q_out


def _append_plan(k, v, k_cache, v_cache, table, lengths, freq, pos, q, section, adjacent, cycled, q_out, cu_seqlens,
                 dims, dev):
    cache = _cache(k_cache, v_cache, table, lengths, dev)
    rows = tuple(k.shape[:2])
    _want(k, "k", rows + (cache.Hk, cache.D), k.dtype, dev, False)
    _want(v, "v", rows + (cache.Hk, cache.D), k.dtype, dev, False)
    Hq = 0
    if q is not None:
        Hq = q.shape[2] if q.dim() == 4 else 0
        _want(q, "q", rows + (Hq, cache.D), k.dtype, dev, False)
        _want(q_out, "q_out", rows + (Hq, cache.D), k_cache.dtype, dev)
    elif q_out is not None:
        raise ValueError("q_out without q")
    rot = _rotary(freq, section, adjacent, cycled, dev)
    if rot.axes > 1 and pos is None:
        raise ValueError("pos is required where there are several axes")
    _positions(pos, rot, rows, dev)
    B, T = dims[0], _whole(dims[1], "max_seqlen")
    if cu_seqlens is not None and not cu_seqlens.is_contiguous():
        raise ValueError("cu_seqlens must be contiguous")
    if B != table.shape[0]:
        raise ValueError(f"table has {table.shape[0]} sequences, the batch {B}")
    prob = GdrAppendProblem(B, min(T, rows[1]), rows[0] * rows[1], Hq, _dtype(k.dtype, "k"), rot, cache,
                            0 if q is None else _row_stride(q, "q"), _row_stride(k, "k"), _row_stride(v, "v"))
    return ctypes.byref(prob), rows + (Hq, cache.D)


def gdr_cache_attention_workspace(prob):
    n = ctypes.c_size_t(0)
    _check_status(lib().gdr_cache_attention_workspace(ctypes.byref(prob), ctypes.byref(n)),
                  "gdr_cache_attention_workspace")
    return n.value


def _span(window, sinks):
    """The window (0: none), both checked."""
    window, sinks = _whole(window, "window"), _whole(sinks, "sinks")
    if window is not None and window < 1:
        raise ValueError("window must be at least 1, or None for all tokens")
    if sinks is None or sinks < 0:
        raise ValueError("sinks must be at least 0")
    return 0 if window is None else window


def _lse_meta(lse):
    if not isinstance(lse, torch.Tensor):
        raise TypeError(f"lse must be True, None or a tensor, got {lse!r}")
    return _meta(lse)


def gdr_cache_attention(q, k_cache, v_cache, table, lengths, *, scale=None, window=None, sinks=0, max_len=None,
                        out_dtype=torch.float32, o=None, lse=True, stream=None):
    """Attention of one new token for each sequence, q [B, 1, Hq, D] in the
    cache's dtype, over the tokens that the cache holds, its own among them (the
    last).  Returns (o, lse): [B, 1, Hq, D] and the softmax sums' logarithms,
    float32 [B, 1, Hq]; a sequence without a visible token gives 0 and -inf.

    k_cache, v_cache, table, lengths: as for gdr_cache_append; tokens of pages
    that are not there are not visible.  With ``window`` only the last so many
    tokens are, and the first ``sinks``.  ``max_len`` bounds the lengths
    (default: what the table holds); a captured call serves any lengths up to
    it.  ``scale``: D ** -0.5 by default.  ``o`` and ``lse`` may be tensors to
    write into, ``lse`` None where it is not wanted."""
    dev = _device(q, "q")
    if not _here(dev, stream):
        with _on(dev, stream):
            return gdr_cache_attention(q, k_cache, v_cache, table, lengths, scale=scale, window=window, sinks=sinks,
                                       max_len=max_len, out_dtype=out_dtype, o=o, lse=lse)
    scale = None if scale is None else float(scale)
    key = ("cache", _meta(q), _meta(k_cache), _meta(v_cache), _meta(table), _meta(lengths), _meta(o),
           lse if lse is None or lse is True else _lse_meta(lse), scale, window, sinks, max_len, window.__class__,
           sinks.__class__, max_len.__class__, out_dtype)
    plan = _plans.get(key) or _plan(key, lambda: _cache_attention_plan(
        q, k_cache, v_cache, table, lengths, scale, window, sinks, max_len, out_dtype, o, lse, dev))
    ref, shape, nws = plan
    if o is None:
        o = torch.empty(shape, dtype=out_dtype, device=dev)
    if lse is True:
        lse = torch.empty(shape[:3], dtype=torch.float32, device=dev)
    ws = _workspace(nws, dev)
    st = lib().gdr_cache_attention(ref, q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), table.data_ptr(),
                                   lengths.data_ptr(), o.data_ptr(), _ptr(lse), _ptr(ws), nws, _raw_stream(dev.index))
    if st:
        _check_status(st, "gdr_cache_attention")
    return o, lse


def _cache_attention_plan(q, k_cache, v_cache, table, lengths, scale, window, sinks, max_len, out_dtype, o, lse, dev):
    if q.dim() != 4:
        raise ValueError("q must be [B, 1, Hq, D]")
    cache = _cache(k_cache, v_cache, table, lengths, dev)
    shape = (table.shape[0], 1, q.shape[2], cache.D)
    _want(q, "q", shape, k_cache.dtype, dev, False)
    if o is not None:
        _want(o, "o", shape, o.dtype, dev)
    if lse is not True:
        _want(lse, "lse", shape[:3], torch.float32, dev)
    window, max_len = _span(window, sinks), _whole(max_len, "max_len")
    if max_len is None:
        max_len = 0
    elif max_len < 1:
        raise ValueError("max_len must be at least 1")
    prob = GdrCacheAttentionProblem(shape[0], shape[2], _dtype(out_dtype if o is None else o.dtype, "out_dtype"), cache,
                                    _row_stride(q, "q"), max_len, window, _whole(sinks, "sinks"),
                                    cache.D ** -0.5 if scale is None else scale)
    return ctypes.byref(prob), shape, gdr_cache_attention_workspace(prob)


# ---- attention over whole sequences ---------------------------------------

def _attention_problem(q, k, v, scale, window, sinks, out_dtype, cu_seqlens, dims):
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("q, k, v must be [B, T, heads, dim]")
    dev = _device(q, "q")
    rows = tuple(q.shape[:2])
    Hq, D = q.shape[2:]
    Hk = k.shape[2]
    _want(k, "k", rows + (Hk, D), q.dtype, dev, False)
    _want(v, "v", rows + (Hk, D), q.dtype, dev, False)
    B, T = rows if cu_seqlens is None else dims
    if cu_seqlens is not None:
        if not cu_seqlens.is_contiguous():
            raise ValueError("cu_seqlens must be contiguous")
        T = min(_whole(T, "max_seqlen"), rows[1])  # no sequence is longer than the batch
    return GdrAttentionProblem(B, T, Hq, Hk, D, _dtype(q.dtype, "q"), _dtype(out_dtype, "out_dtype"),
                               _span(window, sinks), _whole(sinks, "sinks"),
                               D ** -0.5 if scale is None and D else scale or 0.0,
                               _row_stride(q, "q"), _row_stride(k, "k"), _row_stride(v, "v"))


def gdr_attention_forward(q, k, v, *, scale=None, window=None, sinks=0, out_dtype=torch.float32, o=None, stream=None,
                          cu_seqlens=None, max_seqlen=None):
    """Causal attention of q [B, T, Hq, D] over k, v [B, T, Hk, D]: a token sees
    the tokens up to itself, with ``window`` the last so many of them and the
    first ``sinks``.  Returns (o, lse): [B, T, Hq, D], and float32 [B, T, Hq],
    both of which gdr_attention_backward takes.  ``scale``: D ** -0.5 by default;
    ``o`` may be a tensor to write into; ``cu_seqlens`` / ``max_seqlen`` as for
    ``gdr_forward``: rows that no sequence covers are left as they were."""
    dev = _device(q, "q")
    if not _here(dev, stream):
        with _on(dev, stream):
            return gdr_attention_forward(q, k, v, scale=scale, window=window, sinks=sinks, out_dtype=out_dtype, o=o,
                                         cu_seqlens=cu_seqlens, max_seqlen=max_seqlen)
    dims = None if cu_seqlens is None else _ragged_dims(q, cu_seqlens, max_seqlen)
    scale = None if scale is None else float(scale)
    key = ("forward", _meta(q), _meta(k), _meta(v), _meta(o), _meta(cu_seqlens), dims, scale, window, sinks,
           window.__class__, sinks.__class__, max_seqlen.__class__, out_dtype)

    def make():
        if o is not None:
            _want(o, "o", tuple(q.shape), o.dtype, dev)
        return ctypes.byref(_attention_problem(q, k, v, scale, window, sinks, out_dtype if o is None else o.dtype,
                                               cu_seqlens, dims)), tuple(q.shape)

    ref, shape = _plans.get(key) or _plan(key, make)
    if o is None:
        o = torch.empty(shape, dtype=out_dtype, device=dev)
    lse = torch.empty(shape[:3], dtype=torch.float32, device=dev)
    args = (q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(), _raw_stream(dev.index))
    if cu_seqlens is not None:
        st = lib().gdr_attention_forward_varlen(ref, cu_seqlens.data_ptr(), *args)
    else:
        st = lib().gdr_attention_forward(ref, *args)
    if st:
        _check_status(st, "gdr_attention_forward")
    return o, lse


def gdr_attention_backward_workspace(prob, rows):
    """``rows``: token rows of q."""
    n = ctypes.c_size_t(0)
    _check_status(lib().gdr_attention_backward_workspace(ctypes.byref(prob), rows, ctypes.byref(n)),
                  "gdr_attention_backward_workspace")
    return n.value


def gdr_attention_backward(q, k, v, o, lse, dout, *, scale=None, window=None, sinks=0, stream=None, cu_seqlens=None,
                           max_seqlen=None):
    """VJP of gdr_attention_forward for <dout, o>, from its inputs and what it
    returned.  Returns (dq, dk, dv) in o's dtype; rows that no sequence covers
    are not written."""
    dev = _device(q, "q")
    if not _here(dev, stream):
        with _on(dev, stream):
            return gdr_attention_backward(q, k, v, o, lse, dout, scale=scale, window=window, sinks=sinks,
                                          cu_seqlens=cu_seqlens, max_seqlen=max_seqlen)
    dims = None if cu_seqlens is None else _ragged_dims(q, cu_seqlens, max_seqlen)
    scale = None if scale is None else float(scale)
    key = ("backward", _meta(q), _meta(k), _meta(v), _meta(o), _meta(lse), _meta(dout), _meta(cu_seqlens), dims, scale,
           window, sinks, window.__class__, sinks.__class__, max_seqlen.__class__)

    def make():
        prob = _attention_problem(q, k, v, scale, window, sinks, o.dtype, cu_seqlens, dims)
        _want(o, "o", tuple(q.shape), o.dtype, dev)
        _want(lse, "lse", tuple(q.shape[:3]), torch.float32, dev)
        _want(dout, "dout", tuple(q.shape), q.dtype, dev)
        rows = q.shape[0] * q.shape[1]
        return ctypes.byref(prob), rows, gdr_attention_backward_workspace(prob, rows)

    ref, rows, nws = _plans.get(key) or _plan(key, make)
    dq = torch.empty(q.shape, dtype=o.dtype, device=dev)
    dk = torch.empty(k.shape, dtype=o.dtype, device=dev)
    dv = torch.empty(v.shape, dtype=o.dtype, device=dev)
    ws = _workspace(nws, dev)
    args = (q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(), dout.data_ptr(), dq.data_ptr(),
            dk.data_ptr(), dv.data_ptr(), _ptr(ws), nws, _raw_stream(dev.index))
    if cu_seqlens is not None:
        st = lib().gdr_attention_backward_varlen(ref, rows, cu_seqlens.data_ptr(), *args)
    else:
        st = lib().gdr_attention_backward(ref, *args)
    if st:
        _check_status(st, "gdr_attention_backward")
    return dq, dk, dv
