"""Error bounds of the gated feed-forward block and the NVFP4 products,
against fp64 values of the same inputs.

u = 2**-8 is half a step of bf16 relative to a value (to nearest).

* A projection p = sum_k x_k w_k is a sum of K exact products (bf16 x bf16
  fits 24 bits; NVFP4 values without 1/S fit 6 bits) in fp32.  Every addition
  loses at most one step of fp32 (the tensor cores cut off instead of
  rounding), 2**-23 of the magnitudes summed so far, so |err| <= ep =
  K 2**-23 sum_k |x_k w_k|.
* y = s g(a) (b + c), g(a) = a sigmoid(alpha a): |g'| <= 1.1 for every alpha
  (max of sigmoid(z) + z sigmoid'(z) is 1.0998), clamps have slope <= 1, so
  |err| <= |s| (1.1 |b + c| ea + (|g| + 1.1 ea) eb), plus the evaluation in
  fp32 with the hardware exponential, 2**-18 |s g| (|b| + c)  (relative
  error <= 2 + 1.17 |z| ulp, |z| <= 25, and a few roundings).
* dp = s dy act' likewise within 2**-18 of its terms, then rounded to bf16
  (u |dp|); dx and dW are sums over it: |err| <= sum |e_dp| |w| plus the
  fp32 sum's own bound, plus u of the result.  That bound adds every
  rounding with one sign; the roundings are independent, so the 2-norm of the
  error is below sqrt(2 / 3) u = 3.2e-3 of the result's (two roundings of a
  uniform error each); 4e-3 is asked for results of 1000 values or more.
* A quantized output has to be a code that some y within the bound gives.
"""
import numpy as np

from oracle import act as A
from oracle.formats import e4m3_decode, e4m3_encode, e8m0_from_amax

U = 2.0 ** -8
LIM, ALPHA = 7.0, 1.702


def ep_bound(x, w):
    return x.shape[1] * 2.0 ** -23 * (np.abs(x) @ np.abs(w).T)


def y_bound(p, ep, s, act):
    H = p.shape[1] // 2
    a, b, ea, eb = p[:, :H], p[:, H:], ep[:, :H], ep[:, H:]
    if act == "swiglu":
        g, lin, mag = np.abs(a * A.sigmoid(a)), np.abs(b), np.abs(b)
    else:
        a, b = np.minimum(a, LIM), np.clip(b, -LIM, LIM)
        g, lin, mag = np.abs(a * A.sigmoid(ALPHA * a)), np.abs(b + 1), np.abs(b) + 1
    s = np.ones(len(p)) if s is None else np.abs(s.astype(np.float64))
    return s[:, None] * (1.1 * lin * ea + (g + 1.1 * ea) * eb + 2.0 ** -18 * g * mag)


def check_value(got, ref, err, bf16, what):
    tol = err + (U * (np.abs(ref) + err) if bf16 else 2.0 ** -24 * np.abs(ref)) + 1e-37
    d = np.abs(got - ref)
    assert np.all(d <= tol), f"{what}: {np.sum(~(d <= tol))} off, max err/tol {np.nanmax(d / tol):.3f}"


def check_codes(codes, ref, err, scale, what):
    """E4M3 codes of ref * scale, ref within err."""
    lo = e4m3_decode(e4m3_encode((ref - err) * scale * (1 - 2.0 ** -23 * np.sign(ref - err))))
    hi = e4m3_decode(e4m3_encode((ref + err) * scale * (1 + 2.0 ** -23 * np.sign(ref + err))))
    v = e4m3_decode(codes)
    bad = ~((v >= lo) & (v <= hi))
    assert not bad.any(), f"{what}: {bad.sum()} codes outside"


def check_mx(codes, scales, ref, err, what):
    N, H = ref.shape
    a, e = np.abs(ref).reshape(N, H // 32, 32), err.reshape(N, H // 32, 32)
    lo = e8m0_from_amax(np.max(np.maximum(a - e, 0), -1)).astype(int)
    hi = e8m0_from_amax(np.max(a + e, -1)).astype(int)
    s = scales.astype(int)
    assert np.all((s >= lo) & (s <= hi)), f"{what}: block scales"
    inv = np.repeat(np.ldexp(1.0, 127 - s), 32, axis=1)
    check_codes(codes, ref, err, inv, what)


def check_grad(got, ref, err, what):
    check_value(got, ref, err, True, what)
    if ref.size >= 1000 and np.linalg.norm(ref) > 0:
        rel = np.linalg.norm(got - ref) / np.linalg.norm(ref)
        assert rel <= 4e-3, f"{what}: relative error {rel:.2e}"


def dp_bound(pre, dy, s, act):
    """Magnitude of the terms that form dp, for the evaluation error 2**-18 of them."""
    H = dy.shape[1]
    a, b = pre[:, :H], pre[:, H:]
    sd = np.abs(dy) * (1.0 if s is None else np.abs(s.astype(np.float64))[:, None])
    if act == "swiglu":
        sg = A.sigmoid(a)
        return np.concatenate([sd * np.abs(b) * sg * (1 + np.abs(a) * (1 - sg)), sd * np.abs(a) * sg], 1)
    a, b = np.minimum(a, LIM), np.clip(b, -LIM, LIM)
    sg = A.sigmoid(ALPHA * a)
    return np.concatenate([sd * (np.abs(b) + 1) * sg * (1 + ALPHA * np.abs(a) * (1 - sg)),
                           sd * np.abs(a) * sg], 1)
