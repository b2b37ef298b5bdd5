"""CPU pins of the oracle's gated feed-forward block and NVFP4 values
(oracle/ffn.py):

* the forward and the backward re-derived by pure Python loops on a small
  block (math.fsum, no matrix products);
* central finite differences of L = sum(dy * y) for dx, dW and dscales, both
  activations, with inputs on both sides of the clamps;
* NVFP4 values on a row worked by hand.
"""
import math

import numpy as np
import pytest

from oracle import ffn as F

LIM, ALPHA = 7.0, 1.702


def _loop_y(x, w, s, act):
    N, K = x.shape
    H = w.shape[0] // 2
    y = np.empty((N, H))
    for i in range(N):
        for j in range(H):
            a = math.fsum(x[i, k] * w[j, k] for k in range(K))
            b = math.fsum(x[i, k] * w[H + j, k] for k in range(K))
            if act == "swiglu":
                v = a / (1 + math.exp(-a)) * b
            else:
                a, b = min(a, LIM), max(-LIM, min(b, LIM))
                v = a / (1 + math.exp(-ALPHA * a)) * (b + 1)
            y[i, j] = s[i] * v
    return y


def _block(seed=3, N=3, K=5, H=4, std=4.0):
    r = np.random.default_rng(seed)
    return (r.normal(0, 1, (N, K)), r.normal(0, std / math.sqrt(K), (2 * H, K)), r.uniform(0.2, 1, N),
            r.normal(0, 1, (N, H)))


@pytest.mark.parametrize("act", ["swiglu", "clamped_swiglu"])
def test_forward_against_loops(act):
    x, w, s, _ = _block()
    got = F.gated_ffn_fwd(x, w, s, act)
    assert np.allclose(got["y"], _loop_y(x, w, s, act), rtol=1e-13, atol=1e-13)
    assert np.allclose(F.gated_ffn_fwd(x, w, None, act)["y"], _loop_y(x, w, np.ones(3), act), rtol=1e-13,
                       atol=1e-13)


@pytest.mark.parametrize("act", ["swiglu", "clamped_swiglu"])
def test_backward_against_differences(act):
    x, w, s, dy = _block()
    p = F.projections(x, w)
    assert act == "swiglu" or (np.abs(p) > LIM).any()  # some inputs lie beyond a clamp
    g = F.gated_ffn_bwd(dy, x, w, p, s, act)
    h = 1e-6

    def diff(f, v):
        d = np.empty_like(v)
        for i in np.ndindex(v.shape):
            up, down = v.copy(), v.copy()
            up[i] += h
            down[i] -= h
            d[i] = (np.sum(dy * f(up)) - np.sum(dy * f(down))) / (2 * h)
        return d

    assert np.allclose(g["dx"], diff(lambda v: _loop_y(v, w, s, act), x), rtol=1e-6, atol=1e-6)
    assert np.allclose(g["dw"], diff(lambda v: _loop_y(x, v, s, act), w), rtol=1e-6, atol=1e-6)
    assert np.allclose(g["dscales"], diff(lambda v: _loop_y(x, w, v, act), s), rtol=1e-6, atol=1e-6)


def test_nvfp4_values_by_hand():
    # codes 0x1 = 0.5, 0x9 = -0.5, 0x7 = 6, 0xF = -6, 0x2 = 1; low nibble first;
    # block scales 0x38 = 1.0 and 0x40 = 2.0; 1 / S = 0.25
    codes = np.zeros((1, 16), np.uint8)
    codes[0, 0], codes[0, 7], codes[0, 8], codes[0, 15] = 0x91, 0x7F, 0x20, 0x09
    v = F.nvfp4_values(codes, np.array([[0x38, 0x40]], np.uint8), np.float32(0.25))
    want = np.zeros((1, 32))
    want[0, 0], want[0, 1], want[0, 14], want[0, 15] = 0.125, -0.125, -1.5, 1.5
    want[0, 17], want[0, 30] = 0.5, -0.25
    assert np.array_equal(v, want)
