"""The 64-bit definitions of the attention layer's operators, against
differences, hand-worked values and torch's autograd (CPU)."""

import math

import numpy as np
import pytest
import torch

from oracle import attention_oracle as ao


def inputs(seed, T, Hq, Hk, D):
    r = np.random.default_rng(seed)
    return [r.standard_normal(s) for s in ((T, Hq, D), (T, Hk, D), (T, Hk, D), (T, Hq, D))]


@pytest.mark.parametrize("window,sinks", [(None, 0), (3, 0), (2, 2), (1, 0)])
def test_gradients_against_differences(window, sinks):
    q, k, v, do = inputs(1, 7, 4, 2, 3)
    grads = ao.attention_vjp(q, k, v, do, 0.6, window, sinks)
    r = np.random.default_rng(2)
    for x, dx in zip((q, k, v), grads):
        d = r.standard_normal(x.shape)
        eps = 1e-6
        x += eps * d
        up = np.sum(do * ao.attention(q, k, v, 0.6, window, sinks)[0])
        x -= 2 * eps * d
        down = np.sum(do * ao.attention(q, k, v, 0.6, window, sinks)[0])
        x += eps * d
        assert abs((up - down) / (2 * eps) - np.sum(dx * d)) < 1e-7 * (1 + abs(np.sum(dx * d)))


def test_attention_against_autograd():
    q, k, v, do = (torch.from_numpy(x) for x in inputs(3, 11, 6, 2, 8))
    for t in (q, k, v):
        t.requires_grad_()
    kk, vv = (t.repeat_interleave(3, 1) for t in (k, v))
    S = torch.einsum("ihd,jhd->hij", q, kk) * 0.3
    i = torch.arange(11)
    hidden = (i[:, None] < i) | ((i[:, None] - i >= 4) & (i >= 1))
    S = S.masked_fill(hidden, -math.inf)
    o = torch.einsum("hij,jhd->ihd", S.softmax(-1), vv)
    o.backward(do)
    x = [t.detach().numpy() for t in (q, k, v)]
    ro, lse = ao.attention(*x, 0.3, 4, 1)
    assert np.allclose(ro, o.detach().numpy(), atol=1e-12)
    assert np.allclose(lse, S.logsumexp(-1).T.detach().numpy(), atol=1e-12)
    for got, t in zip(ao.attention_vjp(*x, do.numpy(), 0.3, 4, 1), (q, k, v)):
        assert np.allclose(got, t.grad.numpy(), atol=1e-12)


def test_rotary_by_hand():
    x = np.arange(1.0, 7.0).reshape(1, 1, 6)
    freq = np.array([math.pi / 2, 0.0], np.float32)  # a quarter turn, no turn
    y = ao.rotary(x, [1], freq)
    assert np.allclose(y, [[[-3, 2, 1, 4, 5, 6]]], atol=1e-6)
    y = ao.rotary(x, [1], freq, adjacent=True)
    assert np.allclose(y, [[[-2, 1, 3, 4, 5, 6]]], atol=1e-6)
    assert np.allclose(ao.rotary(y, [1], freq, adjacent=True, back=True), x, atol=1e-12)


def test_axes_of_pairs():
    assert ao.pair_axis(6, (3, 1, 2)) == [0, 0, 0, 1, 2, 2]
    assert ao.pair_axis(8, (4, 2, 2), cycled=True) == [0, 1, 2, 0, 1, 2, 0, 0]
    assert ao.pair_axis(4) == [0] * 4


def test_scores_depend_on_the_distance_alone():
    r = np.random.default_rng(5)
    q, k = r.standard_normal((2, 1, 1, 16))
    freq = (10000.0 ** (-np.arange(8) / 8)).astype(np.float32)
    one = np.sum(ao.rotary(q, [40], freq) * ao.rotary(k, [33], freq))
    far = np.sum(ao.rotary(q, [1000007], freq) * ao.rotary(k, [1000000], freq))
    assert abs(one - far) < 1e-9


def test_tokens_over_a_cache_are_rows_of_the_sequence():
    q, k, v, _ = inputs(6, 13, 4, 2, 5)
    kc, vc = np.full((6, 4, 2, 5), np.nan), np.full((6, 4, 2, 5), np.nan)
    table = [[5, 2, 0, 3]]
    kc, vc = ao.append(kc, vc, table, [9], [(0, 9)], k, v)
    for n in range(10, 14):
        kc, vc = ao.append(kc, vc, table, [n], [(n - 1, 1)], k, v)
        for window, sinks in ((None, 0), (5, 2), (20, 0)):
            o, lse, _ = ao.cache_attention(q[n - 1:n], kc, vc, table, [n], 0.4, window, sinks)
            ro, rl = ao.attention(q[:n], k[:n], v[:n], 0.4, window, sinks)
            assert np.allclose(o[0], ro[-1]) and np.allclose(lse[0], rl[-1])
    o, lse, _ = ao.cache_attention(q[:1], kc, vc, [[-1, -1, -1, -1]], [13], 0.4)
    assert np.all(o == 0) and np.all(np.isneginf(lse))
