"""CPU checks of the linear attention's and group norm's C entry points and
their binding: bad arguments are refused before anything reaches the GPU."""

import ctypes

import pytest
import torch

import gated_delta_rule_54_amd as gdr
from gated_delta_rule_54_amd import binding as B
from gated_delta_rule_54_amd import linear as L

FAKE = 0x10000  # an aligned address that is never dereferenced
PAST = 1 << 40


def prob(**kw):
    base = dict(B=2, T=100, Hk=2, Hv=4, Dk=64, Dv=128, io_dtype=1, out_dtype=1, flags=0, algo=0, q_row=0, k_row=0,
                v_row=0)
    base.update(kw)
    return L.GdrLinearProblem(**base)


def norm(**kw):
    base = dict(rows=10, groups=4, channels=128, io_dtype=1, out_dtype=1, flags=0, eps=1e-5, x_row=0, z_row=0)
    base.update(kw)
    return L.GdrNormProblem(**base)


def query(name, p):
    n = ctypes.c_size_t(12345)
    return getattr(B.lib(), name)(ctypes.byref(p), ctypes.byref(n)), n.value


def fwd(p, ragged=False, ws=FAKE, nws=PAST, **over):
    a = dict(q=FAKE, k=FAKE, v=FAKE, g=FAKE, h0=None, o=FAKE, ht=None)
    cu = over.pop("cu", FAKE)
    a.update(over)
    if ragged:
        return B.lib().gdr_linear_forward_varlen(ctypes.byref(p), cu, *a.values(), ws, nws, None)
    return B.lib().gdr_linear_forward(ctypes.byref(p), *a.values(), ws, nws, None)


def bwd(p, ragged=False, ws=FAKE, nws=PAST, **over):
    a = dict(q=FAKE, k=FAKE, v=FAKE, g=FAKE, h0=None, dout=FAKE, dht=None, dq=FAKE, dk=FAKE, dv=FAKE, dg=FAKE,
             dh0=None)
    cu = over.pop("cu", FAKE)
    a.update(over)
    if ragged:
        return B.lib().gdr_linear_backward_varlen(ctypes.byref(p), cu, *a.values(), ws, nws, None)
    return B.lib().gdr_linear_backward(ctypes.byref(p), *a.values(), ws, nws, None)


BAD = [
    (dict(Hv=3), 2), (dict(T=-1), 2), (dict(B=-2), 2), (dict(Hk=0), 2), (dict(Dk=0), 2), (dict(Dv=-16), 2),
    (dict(Dk=24), 3), (dict(Dv=272), 3), (dict(io_dtype=2), 3), (dict(out_dtype=-1), 3), (dict(flags=2), 3),
    (dict(algo=3), 3), (dict(algo=-1), 3), (dict(q_row=120), 2), (dict(k_row=-8), 2), (dict(v_row=504), 2),
    (dict(q_row=132), 4), (dict(v_row=(1 << 22) + 8), 3), (dict(B=70000), 3), (dict(T=1 << 31), 3),
    (dict(B=60000, T=60000), 3), (dict(B=60000, Hk=1000, Hv=1000, T=1), 3),
]


@pytest.mark.parametrize("kw,status", BAD)
def test_bad_linear_problems(kw, status):
    p = prob(**kw)
    assert query("gdr_linear_forward_workspace", p) == (status, 12345)
    assert query("gdr_linear_backward_workspace", p) == (status, 12345)
    assert fwd(p, q=None) == status and bwd(p, dq=None) == status


def test_linear_null_arguments():
    for name in ("q", "k", "v", "o"):
        assert fwd(prob(), **{name: None}) == 1
    for name in ("q", "k", "v", "dout", "dq", "dk", "dv"):
        assert bwd(prob(), **{name: None}) == 1
    assert bwd(prob(), g=None) == 1            # dg without g
    assert fwd(prob(), ragged=True, cu=None) == 1 and bwd(prob(), ragged=True, cu=None) == 1
    assert B.lib().gdr_linear_forward(None, *[FAKE] * 8, 0, None) == 1
    assert B.lib().gdr_linear_forward_workspace(None, None) == 1
    assert B.lib().gdr_linear_backward_workspace(ctypes.byref(prob()), None) == 1


def test_linear_alignment():
    for name in ("q", "k", "v", "h0", "o", "ht"):
        assert fwd(prob(), **{name: FAKE + 8}) == 4
    for name in ("q", "dout", "dht", "dq", "dv", "dh0"):
        assert bwd(prob(), **{name: FAKE + 8}) == 4
    assert fwd(prob(), g=FAKE + 2) == 4 and bwd(prob(), dg=FAKE + 2) == 4
    assert fwd(prob(), ragged=True, cu=FAKE + 4) == 4
    assert bwd(prob(), ws=FAKE + 16) == 4


@pytest.mark.parametrize("algo", [0, 1, 2])
@pytest.mark.parametrize("T", [1, 100, 5000])
def test_linear_workspace(algo, T):
    p = prob(algo=algo, T=T)
    st, need = query("gdr_linear_backward_workspace", p)
    assert st == 0 and need > 0 and need % 256 == 0
    assert bwd(p, ws=None, nws=0) == 1 and bwd(p, nws=need - 1) == 5
    st, need = query("gdr_linear_forward_workspace", p)
    assert st == 0 and need % 256 == 0
    if need:
        assert fwd(p, ws=None, nws=0) == 1 and fwd(p, nws=need - 1) == 5
    assert query("gdr_linear_backward_workspace", prob(algo=algo, T=0)) == (0, 0)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), 2), (dict(groups=0), 2), (dict(channels=0), 2), (dict(channels=12), 3), (dict(channels=520), 3),
    (dict(io_dtype=3), 3), (dict(out_dtype=2), 3), (dict(flags=8), 3), (dict(eps=-1.0), 2), (dict(eps=float("nan")), 2),
    (dict(groups=70000), 3), (dict(rows=1 << 41), 3), (dict(x_row=504), 2), (dict(z_row=516), 4),
])
def test_bad_norm_problems(kw, status):
    p = norm(**kw)
    lib = B.lib()
    assert query("gdr_group_norm_backward_workspace", p) == (status, 12345)
    assert lib.gdr_group_norm_forward(ctypes.byref(p), None, None, None, None, None, None) == status
    assert lib.gdr_group_norm_backward(ctypes.byref(p), *[None] * 9, None, 0, None) == status


def test_norm_arguments():
    lib, p = B.lib(), norm()
    f = lambda p, x=FAKE, w=FAKE, b=None, z=None, y=FAKE: lib.gdr_group_norm_forward(ctypes.byref(p), x, w, b, z, y,
                                                                                     None)
    assert f(p, x=None) == 1 and f(p, y=None) == 1 and f(p, x=FAKE + 8) == 4 and f(p, w=FAKE + 4) == 4
    assert f(norm(flags=2), z=FAKE) == 3
    need = query("gdr_group_norm_backward_workspace", p)[1]
    assert need > 0 and need % 256 == 0

    def g(p, ws=FAKE, nws=PAST, **over):
        a = dict(x=FAKE, w=FAKE, b=None, z=None, dy=FAKE, dx=FAKE, dz=None, dw=FAKE, db=None)
        a.update(over)
        return lib.gdr_group_norm_backward(ctypes.byref(p), *a.values(), ws, nws, None)

    assert g(p, dy=None) == 1 and g(p, dx=None) == 1 and g(p, z=FAKE) == 1 and g(p, dw=FAKE + 4) == 4
    assert g(norm(flags=2), z=FAKE, dz=FAKE) == 3
    assert g(p, ws=None, nws=0) == 1 and g(p, nws=need - 1) == 5 and g(p, ws=FAKE + 16) == 4


def test_binding_refuses_host_tensors():
    q = torch.zeros(1, 2, 2, 64)
    with pytest.raises(ValueError, match="device tensor"):
        gdr.gdr_linear_forward(q, q, q)
    with pytest.raises(ValueError, match="device tensor"):
        gdr.gdr_linear_backward(q, q, q, None, None, q)
    with pytest.raises(ValueError, match="device tensor"):
        gdr.gdr_group_norm_forward(q)
    with pytest.raises(ValueError, match="device tensor"):
        gdr.gdr_group_norm_backward(q, None, None, None, q)


def test_row_strides():
    row = torch.zeros(2, 5, 544, dtype=torch.bfloat16)
    assert L._row_stride(row[..., :128].unflatten(-1, (2, 64)), "q") == 544
    assert L._row_stride(row[:, 2:3, :128].unflatten(-1, (2, 64)), "q") == 544 * 5     # one token each
    assert L._row_stride(row[1:, 2:3, :128].unflatten(-1, (2, 64)), "q") == 0           # one row
    assert L._row_stride(torch.zeros(2, 5, 2, 64), "q") == 0
    for bad in (row[:, :3, :128].unflatten(-1, (2, 64)),                                 # uneven batches
                torch.zeros(2, 5, 64, 2).transpose(-1, -2), torch.zeros(2, 2, 5, 64).transpose(1, 2)):
        with pytest.raises(ValueError, match="strides"):
            L._row_stride(bad, "q")
