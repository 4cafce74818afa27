"""Pins of the decode-step oracle: brute force on tiny inputs and closed forms."""
import math

import numpy as np
import pytest

from oracle import decode as od
from oracle.hadamard import sylvester


def _cache(rng, slots, heads):
    return (rng.integers(0, 16, (slots, heads * 128)),
            rng.uniform(0.1, 1.0, (slots, heads)).astype(np.float16),
            rng.integers(0, 16, (slots, heads)).astype(np.float16))


def test_visible_positions():
    assert od.visible(5, 0, 0).tolist() == [0, 1, 2, 3, 4]
    assert od.visible(5, 2, 0).tolist() == [3, 4]
    assert od.visible(5, 2, 1).tolist() == [0, 3, 4]
    assert od.visible(5, 2, 4).tolist() == [0, 1, 2, 3, 4]     # they overlap: each once
    assert od.visible(3, 9, 1).tolist() == [0, 1, 2]
    assert od.visible(0, 0, 0).size == 0 and od.visible(-4, 2, 2).size == 0


def test_cache_rows_follow_the_table():
    got = od.cache_rows([2, -1, 7, 0], 3, 9, np.arange(12))
    assert got.tolist() == [6, 7, 8, -1, -1, -1, -1, -1, -1, 0, 1, 2]


def test_attention_against_loops():
    rng = np.random.default_rng(0)
    k, v = _cache(rng, 12, 2), _cache(rng, 12, 2)
    q = rng.standard_normal((1, 4, 128))
    signs = rng.integers(0, 2, 256) * 2 - 1
    got = od.attn_decode(q, k, v, signs, None, np.array([[3, 1]]), 3, [5], 0.1, 2, 1)
    h = sylvester(128)
    rows = [9, 3, 4]                   # positions 0 (a sink), 3 and 4
    for i in range(4):
        head = i // 2
        a, vals = [], []
        for r in rows:
            key = [float(k[1][r, head]) * (int(k[0][r, head * 128 + d]) - float(k[2][r, head]))
                   for d in range(128)]
            qr = [sum(h[d][e] * signs[head * 128 + e] * q[0, i, e] for e in range(128)) /
                  math.sqrt(128) for d in range(128)]
            a.append(0.1 * sum(x * y for x, y in zip(qr, key)))     # rotated q . stored key
            vals.append([float(v[1][r, head]) * (int(v[0][r, head * 128 + d]) -
                                                 float(v[2][r, head])) for d in range(128)])
        p = [math.exp(x - max(a)) for x in a]
        o = [sum(p[t] * vals[t][d] for t in range(3)) / sum(p) for d in range(128)]
        back = [sum(h[e][d] * o[d] for d in range(128)) / math.sqrt(128) for e in range(128)]
        assert np.allclose(got[0, i], back, rtol=0, atol=1e-9)


def test_attention_without_a_visible_token_is_zero():
    rng = np.random.default_rng(1)
    k, v = _cache(rng, 4, 1), _cache(rng, 4, 1)
    q = rng.standard_normal((3, 1, 128))
    got = od.attn_decode(q, k, v, None, None, np.array([[0], [-1], [9]]), 2, [0, 2, 2], 1.0)
    assert not got.any()


def test_one_token_returns_its_value():
    rng = np.random.default_rng(2)
    k, v = _cache(rng, 4, 1), _cache(rng, 4, 1)
    got = od.attn_decode(rng.standard_normal((1, 1, 128)), k, v, None, None, np.array([[1]]), 2,
                         [1], 3.0)
    want = od.dequant_heads(v, np.array([2]), 0)[0] @ sylvester(128) / math.sqrt(128)
    assert np.allclose(got[0, 0], want, rtol=0, atol=1e-9)


@pytest.mark.parametrize("fmt", ["int4_sym", "int4_asym", "nvfp4", "mxfp4"])
def test_weights_agree_with_the_dequantizers(fmt):
    import oracle
    rng = np.random.default_rng(3)
    c = rng.integers(0, 16, (3, 256))
    if fmt == "int4_sym":
        s = rng.uniform(0.1, 1, 3).astype(np.float32)
        want = oracle.dequant_int4_sym(np.where(c >= 8, c - 16, c), s)
        got = od.weights(fmt, c, s)
    elif fmt == "int4_asym":
        s, z = (rng.uniform(0.1, 9, (3, 2)).astype(np.float16) for _ in range(2))
        want, got = oracle.dequant_int4_asym(c, s, z, 128), od.weights(fmt, c, s, z)
    elif fmt == "nvfp4":
        s = rng.integers(0, 0x7F, (3, 16)).astype(np.uint8)
        want, got = oracle.dequant_nvfp4(c, s, 0.37), od.weights(fmt, c, s, None, 0.37)
    else:
        s = rng.integers(100, 150, (3, 8)).astype(np.uint8)
        want, got = oracle.dequant_mxfp4(c, s), od.weights(fmt, c, s)
    assert np.array_equal(got.astype(np.float32), want)
    x = rng.standard_normal((2, 256))
    y = od.gemv(x, got)
    assert np.isclose(y[1, 2], sum(x[1, j] * got[2, j] for j in range(256)))


def test_copy_pages():
    a = np.arange(2 * 7 * 3).reshape(2, 7, 3)
    got = od.copy_pages(a, [(0, 2), (-1, 1), (1, 3)], 2)     # page 3 is not whole: skipped
    assert np.array_equal(got[:, 4:6], a[:, 0:2])
    assert np.array_equal(got[:, :4], a[:, :4]) and np.array_equal(got[:, 6:], a[:, 6:])
