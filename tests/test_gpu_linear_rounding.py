"""bf16 results of linear attention are the 64-bit results rounded once: what
comes before the output's rounding does not show in it.

With A the same sums over absolute values (``forward_abs`` / ``backward_abs``),
a sum formed in fp32 through n roundings is off by at most n 2^-24 A.  The
chunked kernels' products take P and the state as two bf16 operands at least:
the second holds what the first leaves (at most 2^-8 of the value) to 2^-8 of
that, so a product is off by 2^-16 of its value, twice where its other factor
was formed from such operands.  So the value before the output's rounding lies
within d = (n 2^-24 + 2 2^-16) A of the exact one, and, rounding being
monotone, the bf16 result between the rounded ends of that interval.
"""

import numpy as np
import pytest
import torch

import gated_delta_rule_54_amd as gdr
from gated_delta_rule_54_amd.synth import round_bf16
from oracle import linear_oracle as lo
from tests.test_gpu_linear import BF, F, draw, host, to_dev

pytestmark = pytest.mark.gpu


def once(name, got, ref, A, n, chunked):
    d = (n * 2.0 ** -24 + (2 * 2.0 ** -16 if chunked else 0.0)) * A + 1e-30
    got = host(got)
    # the ends are stepped outward: round_bf16 goes through fp32, half of whose step is 2^-24 of the value
    lo_, hi = (round_bf16((e + s * 2.0 ** -24 * np.abs(e)).astype(np.float32)) for e, s in ((ref - d, -1), (ref + d, 1)))
    outside = (got < lo_) | (got > hi)
    two = np.linalg.norm(got - ref) / np.linalg.norm(ref)
    print(f"  {name}: {outside.sum()} of {ref.size} outside, 2-norm error {two:.2e}, "
          f"of rounding alone {np.linalg.norm(round_bf16(ref.astype(np.float32)) - ref) / np.linalg.norm(ref):.2e}")
    assert not outside.any(), (name, int(outside.sum()), ref.size)
    # a rounding's error is at most 2^-8 of the value, and its mean square over a binade a third of the most
    assert two <= 2.0 ** -8 / np.sqrt(3) + np.linalg.norm(d) / np.linalg.norm(ref), (name, two)


def compare(x, io, algo, want_dg, **kw):
    t = to_dev(x, io)
    chunked = algo == "chunked"
    args = x["q"], x["k"], x["v"], x["g"], x["h0"]
    T, Dk, Dv = x["q"].shape[1], x["q"].shape[3], x["v"].shape[3]
    n = max(Dk, Dv) + 4 * T + 64 + x["v"].shape[2] // x["q"].shape[2]
    o, _ = gdr.gdr_linear_forward(t["q"], t["k"], t["v"], t["g"], t["h0"], algo=algo, out_dtype=BF, **kw)
    once("o", o, lo.forward(*args)[0], lo.forward_abs(*args)[0], n, chunked)
    got = gdr.gdr_linear_backward(t["q"], t["k"], t["v"], t["g"], t["h0"], t["do"], t["dht"], algo=algo, out_dtype=BF,
                                  want_dg=want_dg, **kw)
    ref, A = lo.backward(*args, x["do"], x["dht"]), lo.backward_abs(*args, x["do"], x["dht"])
    for name, a, r, s in zip(("dq", "dk", "dv"), got, ref, A):
        once(name, a, r, s, n, chunked)


@pytest.mark.parametrize("algo", ["sequential", "chunked"])
@pytest.mark.parametrize("want_dg", [True, False])
@pytest.mark.parametrize("io", [BF, F])
@pytest.mark.parametrize("T,Dk,Dv", [(200, 128, 128), (130, 64, 64), (97, 256, 128), (70, 96, 208)])
def test_bf16_results_are_rounded_once(algo, want_dg, io, T, Dk, Dv):
    compare(draw(T + Dk, 2, T, 2, 4, Dk, Dv, io), io, algo, want_dg)


@pytest.mark.parametrize("gate", ["head", "none"])
def test_over_cut_sequences(gate):
    compare(draw(31, 1, 900, 1, 2, 64, 64, BF, gate, state=gate == "head"), BF, "chunked", gate == "head")


@pytest.mark.parametrize("want_dg", [True, False])
@pytest.mark.parametrize("D", [64, 128])
def test_summed_over_heads_launch_by_launch(want_dg, D):
    """Enough key heads that dq and dk are added to in fp32 rows; one sequence
    of the batch is compared."""
    B, T, Hk, Hv = 16, 70, 4, 8
    x = draw(32, B, T, Hk, Hv, D, D)
    t = to_dev(x, BF)
    gdr.gdr_profile_enable(True)
    got = gdr.gdr_linear_backward(t["q"], t["k"], t["v"], t["g"], t["h0"], t["do"], t["dht"], algo="chunked",
                                  out_dtype=BF, want_dg=want_dg)
    names = gdr.gdr_profile_read()
    gdr.gdr_profile_enable(False)
    assert "linear_group_sum" not in names, "the case no longer reaches the path it is for"
    one = {a: s if s is None else s[5:6] for a, s in x.items()}
    args = tuple(one[a] for a in ("q", "k", "v", "g", "h0", "do", "dht"))
    for name, a, r, s in zip(("dq", "dk", "dv"), got, lo.backward(*args), lo.backward_abs(*args)):
        once(name, a[5:6], r, s, D + 4 * T + 64 + Hv // Hk, True)


def test_a_ragged_batch():
    lens = [65, 0, 3, 190]
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int64)
    x = draw(33, 1, int(cu[-1]), 2, 4, 128, 64, state=False)
    t = to_dev(x, BF)
    kw = dict(algo="chunked", out_dtype=BF, cu_seqlens=torch.from_numpy(cu).cuda(), max_seqlen=190)
    o, _ = gdr.gdr_linear_forward(t["q"], t["k"], t["v"], t["g"], **kw)
    got = gdr.gdr_linear_backward(t["q"], t["k"], t["v"], t["g"], None, t["do"], **kw)
    for i, T in enumerate(lens):
        if T == 0:
            continue
        s = slice(cu[i], cu[i + 1])
        args = tuple(x[a][:, s] for a in ("q", "k", "v", "g")) + (None,)
        n = 128 + 4 * T + 64 + 2
        once("o", o[:, s], lo.forward(*args)[0], lo.forward_abs(*args)[0], n, True)
        ref, A = lo.backward(*args, x["do"][:, s]), lo.backward_abs(*args, x["do"][:, s])
        for name, a, r, b in zip(("dq", "dk", "dv"), got, ref, A):
            once(name, a[:, s], r, b, n, True)
