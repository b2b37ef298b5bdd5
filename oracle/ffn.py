"""Gated feed-forward block and NVFP4 products (oracle side, fp64, numpy).

Source: the page "Activation + GroupedLinear Fusion for MOE and other MOE
optimizations" (TransformerEngine pull request 3238), which fuses the scaled
activations with the products around them; it prints no formula.  Readings:

* W [2H, K] holds the H gate rows, then the H linear rows (the halves of the
  activation's input, see ``act``): p = x W^T [N, 2H], y = s_i act(p);
* backward at the stored projections ``pre``: dp = s_i dy act'(pre),
  dx = dp W, dW = dp^T x, dscales_i = sum_j dy[i, j] act(pre)[i, j];
* NVFP4 weights stand for E2M1 value * E4M3 block scale value * (1 / S), the
  block of element k of a row being k // 16.
"""
from __future__ import annotations

import numpy as np

from . import act as _act
from .formats import e2m1_decode, e2m1_unpack, e4m3_decode


def _f64(a) -> np.ndarray:
    return np.asarray(a, dtype=np.float64)


def projections(x, w) -> np.ndarray:
    return _f64(x) @ _f64(w).T


def gated_ffn_fwd(x, w, scales, act, mode="none", **kw) -> dict:
    """As ``act.scaled_act_fwd`` of the projections, which ``p`` holds (fp64)."""
    p = projections(x, w)
    return {"p": p, **_act.scaled_act_fwd(p, scales, act, mode, **kw)}


def gated_ffn_bwd(dy, x, w, pre, scales, act, limit=7.0, alpha=1.702) -> dict:
    """dp, dx, dw and dscales in fp64, without any rounding of dp."""
    r = _act.scaled_act_bwd(dy, pre, scales, act, "f32", limit, alpha)
    dp = r["dx64"]
    return {"dp": dp, "dx": dp @ _f64(w), "dw": dp.T @ _f64(x), "dscales": r["dscales64"]}


def nvfp4_values(codes, blocks, scale_inv) -> np.ndarray:
    """The fp64 values [R, K] of packed E2M1 codes [R, K/2] with E4M3 block scale codes [R, K/16]."""
    v = e2m1_decode(e2m1_unpack(codes))
    s = np.repeat(e4m3_decode(blocks), 16, axis=1)
    return v * s * float(scale_inv)
