"""The 64-bit oracle of the rotary and cache operators against independent
statements of the same mathematics."""

import math

import numpy as np
import pytest
import torch

from oracle import attention as oa
from oracle import mx as omx


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rotation_is_a_complex_product(layout):
    g = np.random.default_rng(1)
    x = g.standard_normal((5, 3, 12))
    t = oa.rope_table(40, 8, 100.0)
    pos = np.array([0, 39, 7, 7, 1])
    y = oa.rotate(x, pos, t, layout)
    pair = (lambda a, i: (a[..., i], a[..., i + 4])) if layout == "half" else (lambda a, i: (a[..., 2 * i], a[..., 2 * i + 1]))
    for i in range(4):
        a, b = pair(x, i)
        z = (a + 1j * b) * np.exp(1j * pos * 100.0 ** (-2 * i / 8))[:, None]
        u, w = pair(y, i)
        assert np.allclose(u, z.real, atol=1e-14) and np.allclose(w, z.imag, atol=1e-14)
    assert np.array_equal(y[..., 8:], x[..., 8:])


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_inverse_is_the_gradient(layout):
    """d(w . rotate(x)) / dx = rotate(w, inverse), by differences."""
    g = np.random.default_rng(2)
    x, w = g.standard_normal((2, 3, 2, 6))
    t, pos = oa.rope_table(9, 6, 50.0, "yarn", 4.0, 8), np.array([3, 8, 0])
    grad = oa.rotate(w, pos, t, layout, inverse=True)
    for at in np.ndindex(x.shape):
        d = np.zeros_like(x)
        d[at] = 1e-6
        num = ((oa.rotate(x + d, pos, t, layout) - oa.rotate(x - d, pos, t, layout)) * w).sum() / 2e-6
        assert abs(num - grad[at]) < 1e-8


def test_scalings():
    f, m = oa.frequencies(64, 1e4)
    assert m == 1.0 and f[0] == 1.0 and math.isclose(f[31], 1e4 ** (-62 / 64))
    assert np.allclose(oa.frequencies(64, 1e4, "linear", 4.0)[0], f / 4)
    n = oa.frequencies(64, 1e4, "ntk", 4.0)[0]
    assert n[0] == 1.0 and math.isclose(n[31], f[31] / 4)       # the slowest pair stretched by the whole factor
    y, my = oa.frequencies(64, 1e4, "yarn", 4.0, 2048)
    assert my == 1 + 0.1 * math.log(4) and y[0] == f[0] and math.isclose(y[31], f[31] / 4)
    assert np.all(np.diff(y) < 0)
    b = oa.frequencies(64, 1e4, "bands", 4.0, 2048)[0]
    turns = 2048 * f / (2 * math.pi)
    assert np.allclose(b[turns > 4], f[turns > 4]) and np.allclose(b[turns < 1], f[turns < 1] / 4)


def test_attention_against_a_dense_softmax():
    g = np.random.default_rng(3)
    hk, page, dim = 2, 16, 64
    cache = [np.zeros((5, hk, page, n), np.uint8) for n in (dim, 2, dim, 2)]
    k, v = g.standard_normal((2, 40, hk, dim)).astype(np.float32)
    order = np.array([3, 0, 4])
    slots = order[np.arange(40) // page] * page + np.arange(40) % page
    oa.append(cache, k, v, slots)
    kd, vd = (omx.dequantize_exact(*omx.quantize_rowwise(x.reshape(-1, dim), "e4m3", "ceil"), "e4m3").reshape(40, hk, dim)
              for x in (k, v))
    q = g.standard_normal((6, 4, dim))
    out, lse, mag, big, seen = oa.attention(q, cache, order[None], [0, 6], [40], window=9)
    x = torch.from_numpy(q).permute(1, 0, 2)
    a = x @ torch.from_numpy(kd).permute(1, 2, 0).repeat_interleave(2, 0) / 8.0
    i, j = torch.arange(6)[:, None] + 34, torch.arange(40)[None]
    a = a.masked_fill((j > i) | (j <= i - 9), -math.inf)
    want = (a.softmax(-1) @ torch.from_numpy(vd).permute(1, 0, 2).repeat_interleave(2, 0)).permute(1, 0, 2)
    assert np.allclose(out, want.numpy(), atol=1e-13)
    assert np.allclose(lse, a.logsumexp(-1).T.numpy(), atol=1e-13)
    assert (seen == 9).all() and (mag >= np.abs(out) - 1e-15).all() and (big > 0).all()


def test_attention_without_keys_and_with_bad_pages():
    cache = [np.zeros((2, 1, 16, n), np.uint8) for n in (64, 2, 64, 2)]
    q = np.ones((3, 1, 64))
    out, lse, *_ = oa.attention(q, cache, np.array([[0]]), [0, 3], [1])
    assert (out[:2] == 0).all() and (lse[:2] == -np.inf).all() and lse[2] == 0
    out, lse, *_ = oa.attention(q, cache, np.array([[0, 7]]), [0, 3], [18])
    assert np.isfinite(out[0]).all() and np.isnan(out[1:]).all() and np.isnan(lse[1:]).all()
