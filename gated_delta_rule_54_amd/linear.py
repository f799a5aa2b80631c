"""Binding of the operators beside the gated delta rule: linear attention with
a decay for each head, and the group norm of the heads' outputs
(include/gdr.h).  Argument marshalling only, as in ``binding``.

q, k, v, x and z may be column ranges of a wider row (a fused projection's
output): the last axes dense, the rows any 16-byte-aligned distance apart that
keeps them disjoint (an expanded tensor is refused).
Every other tensor is contiguous.  Outputs and workspaces are allocated on the
stream the call runs on: the current stream of the tensors' device, or
``stream``.
"""

import contextlib
import ctypes

import torch

from .binding import ALGOS, GDR_BF16, GDR_F32, GDR_OK, GdrError, _ragged_dims, lib

GDR_LINEAR_HEAD_DECAY = 1
GDR_NORM_CENTER, GDR_NORM_SILU, GDR_NORM_SHARED_WEIGHT = 1, 2, 4

_DT = {torch.float32: GDR_F32, torch.bfloat16: GDR_BF16}


class GdrLinearProblem(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int64), ("T", ctypes.c_int64),
                ("Hk", ctypes.c_int32), ("Hv", ctypes.c_int32),
                ("Dk", ctypes.c_int32), ("Dv", ctypes.c_int32),
                ("io_dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32),
                ("flags", ctypes.c_uint32), ("algo", ctypes.c_int32),
                ("q_row", ctypes.c_int64), ("k_row", ctypes.c_int64), ("v_row", ctypes.c_int64)]


class GdrNormProblem(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("groups", ctypes.c_int32), ("channels", ctypes.c_int32),
                ("io_dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32),
                ("flags", ctypes.c_uint32), ("eps", ctypes.c_float),
                ("x_row", ctypes.c_int64), ("z_row", ctypes.c_int64)]


def _dtype(t, name):
    try:
        return _DT[t]
    except KeyError:
        raise TypeError(f"{name} has unsupported dtype {t}") from None


def _ptr(t):
    return None if t is None else t.data_ptr()


def _row_stride(t, name):
    """Elements between the rows of t [..., rows, H, D] whose last two axes
    are dense and whose rows are equally spaced over all leading axes; 0 where
    they follow each other without a gap.  Rows that share storage (an expanded
    tensor's lie 0 elements apart) are refused: 0 says that they are dense."""
    if t.is_contiguous() or t.numel() == 0:
        return 0
    shape, stride = t.shape, t.stride()
    H, D = shape[-2], shape[-1]
    ok = (D == 1 or stride[-1] == 1) and (H == 1 or stride[-2] == D)
    row, n = None, 1
    for s, st in zip(reversed(shape[:-2]), reversed(stride[:-2])):
        if s == 1:
            continue
        if row is None:
            row = st
        ok = ok and st == n * row
        n *= s
    if not ok or (row is not None and row < H * D):
        raise ValueError(f"{name} must have dense last axes and equally spaced rows that do not overlap, "
                         f"got strides {stride}")
    return 0 if row is None or row == H * D else row


def _want(t, name, shape, dtype, dev, contiguous=True):
    if t is None:
        return
    if t.shape == shape and t.dtype == dtype and t.device == dev and (not contiguous or t.is_contiguous()):
        return
    if tuple(t.shape) != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {shape}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != dev:
        raise ValueError(f"{name} is on {t.device}, expected {dev}")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


@contextlib.contextmanager
def _on(dev, stream):
    """The call's stream made current (with its device), as a HIP handle."""
    if stream is None:
        stream = torch.cuda.current_stream(dev)
    elif stream.device != dev:
        raise ValueError(f"stream is on {stream.device}, the tensors on {dev}")
    with torch.cuda.stream(stream):
        yield stream.cuda_stream


def _here(dev, stream):
    """Whether the call runs where torch already is: no context is needed."""
    return stream is None and dev.index == torch.cuda.current_device()


# The current stream's handle, without the Stream object around it where torch
# has a call for that: a call for one token is bound by the host.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda index: torch.cuda.current_stream(index).cuda_stream)


def _check_status(st, where):
    if st != GDR_OK:
        raise GdrError(st, where)


def _device(t, name):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    return t.device


# ---- linear attention -----------------------------------------------------

def _linear_problem(q, k, v, g, h0, out_dtype, algo, cu_seqlens, max_seqlen):
    if q.dim() != 4 or v.dim() != 4:
        raise ValueError("q, k, v must be [B, T, heads, dim]")
    dev = _device(q, "q")
    rows = tuple(q.shape[:2])
    Hk, Dk = q.shape[2:]
    Hv, Dv = v.shape[2:]
    _want(k, "k", rows + (Hk, Dk), q.dtype, dev, False)
    _want(v, "v", rows + (Hv, Dv), q.dtype, dev, False)
    head = g is not None and g.dim() == 1
    _want(g, "g", (Hv,) if head else rows + (Hv,), torch.float32, dev)
    B, T = rows if cu_seqlens is None else _ragged_dims(q, cu_seqlens, max_seqlen)
    if cu_seqlens is not None:
        if not cu_seqlens.is_contiguous():
            raise ValueError("cu_seqlens must be contiguous")
        T = min(T, rows[1])  # no sequence is longer than the batch
    _want(h0, "h0", (B, Hv, Dk, Dv), torch.float32, dev)
    return GdrLinearProblem(B, T, Hk, Hv, Dk, Dv, _dtype(q.dtype, "q"), _dtype(out_dtype, "out_dtype"),
                            GDR_LINEAR_HEAD_DECAY if head else 0, ALGOS[algo], _row_stride(q, "q"),
                            _row_stride(k, "k"), _row_stride(v, "v"))


def gdr_linear_forward_workspace(prob):
    n = ctypes.c_size_t(0)
    _check_status(lib().gdr_linear_forward_workspace(ctypes.byref(prob), ctypes.byref(n)),
                  "gdr_linear_forward_workspace")
    return n.value


def gdr_linear_backward_workspace(prob, rows=None):
    """``rows``: the token rows of a ragged batch, where they are counted."""
    n = ctypes.c_size_t(0)
    if rows is None:
        st = lib().gdr_linear_backward_workspace(ctypes.byref(prob), ctypes.byref(n))
    else:
        st = lib().gdr_linear_backward_varlen_workspace(ctypes.byref(prob), rows, ctypes.byref(n))
    _check_status(st, "gdr_linear_backward_workspace")
    return n.value


def _workspace(nbytes, dev):
    return torch.empty(nbytes, dtype=torch.uint8, device=dev) if nbytes else None


def gdr_linear_forward(q, k, v, g=None, h0=None, *, algo="auto", out_dtype=torch.float32, o=None, ht=True,
                       stream=None, cu_seqlens=None, max_seqlen=None):
    """S_t = exp(g_t) S_{t-1} + k_t v_t^T, o_t = S_t^T q_t.  Returns (o, ht).

    q, k [B, T, Hk, Dk], v [B, T, Hv, Dv]; g [B, T, Hv], [Hv] (a constant
    decay per head) or None (no decay); h0 [B, Hv, Dk, Dv] or None.  ``o`` may
    be a tensor to write into (its dtype is the output's, its memory none of
    the inputs'); ``ht`` is True
    (allocate), None (not wanted) or a tensor, which may be ``h0``.
    ``cu_seqlens`` / ``max_seqlen`` as for ``gdr_forward``: rows that no
    sequence covers are left as they were."""
    dev = _device(q, "q")
    if not _here(dev, stream):
        with _on(dev, stream):
            return gdr_linear_forward(q, k, v, g, h0, algo=algo, out_dtype=out_dtype, o=o, ht=ht,
                                      cu_seqlens=cu_seqlens, max_seqlen=max_seqlen)
    prob = _linear_problem(q, k, v, g, h0, out_dtype if o is None else o.dtype, algo, cu_seqlens, max_seqlen)
    state = (prob.B, prob.Hv, prob.Dk, prob.Dv)
    if o is None:
        o = torch.empty(v.shape, dtype=out_dtype, device=dev)
    else:
        _want(o, "o", tuple(v.shape), o.dtype, dev)
    if ht is True:
        ht = torch.empty(state, dtype=torch.float32, device=dev)
    else:
        _want(ht, "ht", state, torch.float32, dev)
    ws = _workspace(gdr_linear_forward_workspace(prob), dev)
    args = (_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(h0), _ptr(o), _ptr(ht), _ptr(ws),
            0 if ws is None else ws.numel(), _raw_stream(dev.index))
    if cu_seqlens is not None:
        st = lib().gdr_linear_forward_varlen(ctypes.byref(prob), _ptr(cu_seqlens), *args)
    else:
        st = lib().gdr_linear_forward(ctypes.byref(prob), *args)
    _check_status(st, "gdr_linear_forward")
    return o, ht


def gdr_linear_backward(q, k, v, g, h0, dout, dht=None, *, algo="auto", out_dtype=torch.float32, want_dg=True,
                        want_dh0=True, stream=None, cu_seqlens=None, max_seqlen=None):
    """VJP of gdr_linear_forward for <dout, o> + <dht, ht>, from the forward's
    inputs.  Returns (dq, dk, dv, dg, dh0); dg (in g's shape) is None without
    g or ``want_dg``, dh0 without ``want_dh0``."""
    dev = _device(q, "q")
    if not _here(dev, stream):
        with _on(dev, stream):
            return gdr_linear_backward(q, k, v, g, h0, dout, dht, algo=algo, out_dtype=out_dtype, want_dg=want_dg,
                                       want_dh0=want_dh0, cu_seqlens=cu_seqlens, max_seqlen=max_seqlen)
    prob = _linear_problem(q, k, v, g, h0, out_dtype, algo, cu_seqlens, max_seqlen)
    state = (prob.B, prob.Hv, prob.Dk, prob.Dv)
    _want(dout, "dout", tuple(v.shape), q.dtype, dev)
    _want(dht, "dht", state, torch.float32, dev)
    dq = torch.empty(q.shape, dtype=out_dtype, device=dev)
    dk = torch.empty(k.shape, dtype=out_dtype, device=dev)
    dv = torch.empty(v.shape, dtype=out_dtype, device=dev)
    dg = torch.empty(g.shape, dtype=torch.float32, device=dev) if want_dg and g is not None else None
    dh0 = torch.empty(state, dtype=torch.float32, device=dev) if want_dh0 else None
    rows = None if cu_seqlens is None else q.shape[1]
    ws = _workspace(gdr_linear_backward_workspace(prob, rows), dev)
    args = (_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(h0), _ptr(dout), _ptr(dht), _ptr(dq), _ptr(dk), _ptr(dv),
            _ptr(dg), _ptr(dh0), _ptr(ws), 0 if ws is None else ws.numel(),
            _raw_stream(dev.index))
    if cu_seqlens is not None:
        st = lib().gdr_linear_backward_varlen_rows(ctypes.byref(prob), rows, _ptr(cu_seqlens), *args)
    else:
        st = lib().gdr_linear_backward(ctypes.byref(prob), *args)
    _check_status(st, "gdr_linear_backward")
    return dq, dk, dv, dg, dh0


# ---- group norm -----------------------------------------------------------

def _norm_problem(x, weight, bias, z, center, silu, eps, out_dtype):
    if x.dim() < 2:
        raise ValueError("x must be [..., groups, channels]")
    dev = _device(x, "x")
    G, D = x.shape[-2:]
    shared = False
    for t, name in ((weight, "weight"), (bias, "bias")):
        if t is None:
            continue
        if t.dim() == 1:
            shared = True
        _want(t, name, (D,) if shared else (G, D), torch.float32, dev)
    _want(weight, "weight", (D,) if shared else (G, D), torch.float32, dev)
    _want(z, "z", tuple(x.shape), x.dtype, dev, False)
    rows = x.numel() // (G * D) if G * D else 0
    flags = ((GDR_NORM_CENTER if center else 0) | (GDR_NORM_SILU if silu else 0)
             | (GDR_NORM_SHARED_WEIGHT if shared else 0))
    return GdrNormProblem(rows, G, D, _dtype(x.dtype, "x"), _dtype(out_dtype, "out_dtype"), flags, eps,
                          _row_stride(x, "x"), 0 if z is None else _row_stride(z, "z"))


def gdr_group_norm_forward(x, weight=None, bias=None, z=None, *, center=False, silu=False, eps=1e-5,
                           out_dtype=torch.float32, y=None, stream=None):
    """u = weight n + bias with n the normalised groups of x [..., groups,
    channels]; returns u silu(z) with a gate z (x's shape and dtype), silu(u)
    with ``silu``, else u.  ``center`` subtracts the mean (a group norm;
    without it the root mean square's).  weight and bias: float32 [groups,
    channels], or [channels] for all groups, or None.  ``y`` may be a tensor
    to write into, of none of the inputs' memory."""
    dev = _device(x, "x")
    if not _here(dev, stream):
        with _on(dev, stream):
            return gdr_group_norm_forward(x, weight, bias, z, center=center, silu=silu, eps=eps,
                                          out_dtype=out_dtype, y=y)
    prob = _norm_problem(x, weight, bias, z, center, silu, eps, out_dtype if y is None else y.dtype)
    if y is None:
        y = torch.empty(x.shape, dtype=out_dtype, device=dev)
    else:
        _want(y, "y", tuple(x.shape), y.dtype, dev)
    st = lib().gdr_group_norm_forward(ctypes.byref(prob), _ptr(x), _ptr(weight), _ptr(bias), _ptr(z), _ptr(y),
                                      _raw_stream(dev.index))
    _check_status(st, "gdr_group_norm_forward")
    return y


def gdr_group_norm_backward_workspace(prob):
    n = ctypes.c_size_t(0)
    _check_status(lib().gdr_group_norm_backward_workspace(ctypes.byref(prob), ctypes.byref(n)),
                  "gdr_group_norm_backward_workspace")
    return n.value


def gdr_group_norm_backward(x, weight, bias, z, dy, *, center=False, silu=False, eps=1e-5, out_dtype=torch.float32,
                            stream=None):
    """VJP of gdr_group_norm_forward.  Returns (dx, dz, dweight, dbias), None
    for the operands that were None; dweight and dbias are float32."""
    dev = _device(x, "x")
    if not _here(dev, stream):
        with _on(dev, stream):
            return gdr_group_norm_backward(x, weight, bias, z, dy, center=center, silu=silu, eps=eps,
                                           out_dtype=out_dtype)
    prob = _norm_problem(x, weight, bias, z, center, silu, eps, out_dtype)
    _want(dy, "dy", tuple(x.shape), x.dtype, dev)
    dx = torch.empty(x.shape, dtype=out_dtype, device=dev)
    dz = torch.empty(x.shape, dtype=out_dtype, device=dev) if z is not None else None
    dw = torch.empty_like(weight) if weight is not None else None
    db = torch.empty_like(bias) if bias is not None else None
    ws = _workspace(gdr_group_norm_backward_workspace(prob) if dw is not None or db is not None else 0, dev)
    st = lib().gdr_group_norm_backward(ctypes.byref(prob), _ptr(x), _ptr(weight), _ptr(bias), _ptr(z), _ptr(dy),
                                       _ptr(dx), _ptr(dz), _ptr(dw), _ptr(db), _ptr(ws),
                                       0 if ws is None else ws.numel(), _raw_stream(dev.index))
    _check_status(st, "gdr_group_norm_backward")
    return dx, dz, dw, db
