"""Pins of the oracle's paged 8-bit key/value cache: hand-worked scales and codes, bit patterns, and the
attention against the textbook form in exact or brute-force arithmetic."""
import math

import numpy as np
import pytest

from oracle import e4m3_decode, kv as K


def empty(pages=4, heads=1, dim=64):
    return K.Cache(np.zeros((pages, heads, 64, dim)), np.zeros((pages, heads, dim, 64)), np.zeros((pages, heads)),
                   np.zeros((pages, heads)))


@pytest.mark.parametrize("top,e", [(448.0, 0), (448.0001, 1), (449.0, 1), (224.0, -1), (224.1, 0), (1.0, -8), (1.75, -8),
                                   (1.7501, -7), (0.0, -120), (1e-40, -120), (3e38, 119), (math.inf, -120)])
def test_exponent(top, e):
    assert K.exponent([0.0, -top]) == e


def test_exponent_ignores_what_is_not_finite():
    assert K.exponent([math.nan, math.inf, 3.0, -math.inf]) == K.exponent([3.0]) == -7


def test_write_one_token_by_hand():
    # 1.0 and 0.3 in a page of its own: e = -8, 1.0 = 256 2^-8 (0x78), 0.3 2^8 = 76.8 -> 80 (0x6A: 2^6 * 1.25)
    x = np.zeros((1, 1, 64))
    x[0, 0, :2] = [1.0, 0.3]
    c = K.write(empty(), np.array([[2]]), [0, 1], [1], x, -x)
    assert c.ks[2, 0] == 127 - 8 and c.k[2, 0, 0, 0] == 0x78 and c.k[2, 0, 0, 1] == 0x6A
    assert c.v[2, 0, 0, 0] == 0xF8 and c.v[2, 0, 1, 0] == 0xEA and c.vs[2, 0] == 127 - 8
    assert not c.k[[0, 1, 3]].any() and not c.k[2, 0, 1:].any()


def test_a_page_whose_scale_grows_is_scaled_over():
    table = np.array([[1]])
    x = np.full((1, 1, 64), 1.0)
    c = K.write(empty(), table, [0, 1], [1], x, x)
    c = K.write(c, table, [0, 1], [2], 16 * x, x / 4)
    # keys: 16 needs e = -4, so the first token's 256 becomes 16; values keep e = -8, 0.25 is 64
    assert c.ks[1, 0] == 127 - 4 and c.vs[1, 0] == 127 - 8
    assert e4m3_decode(c.k[1, 0, 0, 0]) == 16 and e4m3_decode(c.k[1, 0, 1, 0]) == 256
    assert e4m3_decode(c.v[1, 0, 0, 0]) == 256 and e4m3_decode(c.v[1, 0, 0, 1]) == 64
    k, v = K.read(c, table, [0, 2], [2], 2)
    assert (k[0] == 1).all() and (k[1] == 16).all() and (v[0] == 1).all() and (v[1] == 0.25).all()


def test_in_pieces_or_at_once():
    # without subnormal codes, writing token by token ends at the same cache as one call
    g = np.random.default_rng(0)
    x = np.exp(g.uniform(-1, 1, (150, 2, 64))) * g.choice([-1, 1], (150, 2, 64))
    table = np.array([[3, 0, 2]])
    once = K.write(empty(4, 2), table, [0, 150], [150], x, 2 * x)
    c = empty(4, 2)
    for a, b in ((0, 1), (1, 60), (60, 70), (70, 150)):
        c = K.write(c, table, [0, b - a], [b], x[a:b], 2 * x[a:b])
    got, want = (K.read(y, table, [0, 150], [150], 150) for y in (c, once))
    # a value may have been rounded under a finer scale first: never further than one coarser step
    assert (c.ks == once.ks).all() and (c.vs == once.vs).all()
    assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])


def test_what_is_not_cached():
    x = np.ones((3, 1, 64))
    c = K.write(empty(), np.array([[9], [-1]]), [0, 2, 3], [2, 1], x, x)
    assert not c.k.any() and not c.ks.any()
    c = K.write(empty(), np.array([[1]]), [0, 3], [2], x, x)    # the first row has no position
    assert (c.k[1, 0, :2] == 0x78).all() and not c.k[1, 0, 2:].any()


def test_attention_is_the_textbook_softmax():
    g = np.random.default_rng(1)
    n, D = 70, 64
    k, v, q = g.standard_normal((n, 2, D)), g.standard_normal((n, 2, D)), g.standard_normal((3, 4, D))
    table = np.array([[2, 0]])
    c = K.write(empty(4, 2), table, [0, n], [n], k, v)
    ck, cv = K.read(c, table, [0, n], [n], n)
    slopes = np.array([0.5, 0.25, 0.125, 0.0])
    for kw in (dict(), dict(causal=False), dict(window=5), dict(softcap=3.0), dict(slopes=slopes)):
        r = K.attention(q, c, table, [0, 3], [n], 0.3, **kw)
        for i in range(3):
            p = n - 3 + i
            for h in range(4):
                num, den = np.zeros(D), 0.0
                for j in range(n):
                    if (kw.get("causal", True) and j > p) or (kw.get("window") and j <= p - kw["window"]):
                        continue
                    s = 0.3 * math.fsum(q[i, h] * ck[j, h // 2])
                    if "softcap" in kw:
                        s = 3.0 * math.tanh(s / 3.0)
                    if "slopes" in kw:
                        s += slopes[h] * (j - p)
                    num += math.exp(s) * cv[j, h // 2]
                    den += math.exp(s)
                assert np.allclose(r["out"][i, h], num / den, rtol=1e-12, atol=1e-14)
                assert math.isclose(r["lse"][i, h], math.log(den), rel_tol=1e-12, abs_tol=1e-12)


def test_attention_that_sees_nothing():
    c = empty()
    q = np.ones((2, 1, 64))
    r = K.attention(q, c, np.array([[0], [0]]), [0, 1, 2], [0, 1], 1.0)
    assert not r["out"][0].any() and r["lse"][0, 0] == -math.inf
    assert r["lse"][1, 0] == 0.0 and r["seen"][1, 0] == 1
