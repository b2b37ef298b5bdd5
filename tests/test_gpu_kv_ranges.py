"""GPU parity of the attention over the paged 8-bit cache where its numbers or its parts lie far apart."""
import numpy as np
import pytest
import torch

import mxfp8_quantization_gb300 as rn
from kv_check import check, make, randn, reference

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _no_device_error():
    yield
    assert rn.device_error() == 0


def f64(t):
    return t.double().cpu().numpy()


@pytest.mark.parametrize("group", [2, 8, 12])
@pytest.mark.parametrize("dim", [64, 128])
def test_row_tiles_of_one_page_behind_others(dim, group):
    # 20 to 120 rows a head; a CTA gets several of these in turn
    lens, news = [150, 30, 64, 200, 12, 40, 300, 63, 10] * 10, [10] * 90
    c, s, T = make(lens, news, 8, dim, seed=group)
    q = randn(T, 8 * group, dim, std=1.5)
    out, lse = rn.kv_attention(q, c, s, return_lse=True)
    check(out, lse, reference(q, c, s), dim)
    for _ in range(20):
        again, lse2 = rn.kv_attention(q, c, s, return_lse=True)
        assert torch.equal(again, out) and torch.equal(lse2, lse)


def bounds(want, dim, softcap=0.0):
    """kv_check.bounds, without what grows with the cap: its error is relative to the capped score (below 2^-21 of the
    cap where z / c is above 1/4, whose tanh is 0.245)."""
    seen = want["seen"].astype(np.float64)
    eps = want["big"] * ((dim + 8) * 2.0 ** -23) + 2.0 ** -20 + (seen / 64 + 2) * 2.0 ** -22
    if softcap:
        eps = eps + np.minimum(want["big"], softcap) * 2.0 ** -18
    part = 2.0 ** -11 + 2 * eps + (seen / 8 + 4) * 2.0 ** -23 + seen * 2.0 ** -24
    out = want["pv"] * part[..., None] + want["spread"] * 2.0 ** -25
    out = out + (np.abs(want["out"]) + out) * 2.0 ** -8
    lse = eps + seen * 2.0 ** -24 + (np.abs(want["lse"]) + 1) * 2.0 ** -22
    return out, lse


def close(out, lse, want, dim, softcap=0.0):
    tol, tol_lse = bounds(want, dim, softcap)
    err, err_lse = np.abs(f64(out) - want["out"]), np.abs(f64(lse) - want["lse"])
    assert np.all(err <= tol), (float((err / tol.clip(1e-300)).max()), int((err > tol).sum()))
    assert np.all(err_lse <= tol_lse), float((err_lse / tol_lse).max())


@pytest.mark.parametrize("cap", [1e-3, 1.0, 8.0, 50.0, 1e3, 1e4, 1e6, 1e12, 1e30])
@pytest.mark.parametrize("dim,new,group", [(64, 1, 4), (64, 4, 4), (64, 10, 8), (256, 1, 4), (256, 10, 8)])
def test_caps_of_any_size(dim, new, group, cap):
    c, s, T = make([700, 130], [new, new], 2, dim, seed=1)
    q = randn(T, 2 * group, dim, seed=2, std=2.0)
    out, lse = rn.kv_attention(q, c, s, softcap=cap, return_lse=True)
    close(out, lse, reference(q, c, s, softcap=cap), dim, cap)
