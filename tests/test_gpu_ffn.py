"""GPU parity of the gated feed-forward block (rn_gated_ffn_fwd / _bwd)
against the oracle (oracle/ffn.py); the bounds are derived in ffn_check.py."""
import ctypes

import numpy as np
import pytest
import torch

import matvec_plan
import mxfp8_quantization_gb300 as rn
import oracle
from ffn_check import (ALPHA, LIM, U, check_codes, check_grad, check_mx, check_value, dp_bound, ep_bound,
                       y_bound)
from oracle import ffn as F

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _no_device_error():
    yield
    assert rn.device_error() == 0


def f64(t):
    return t.detach().double().cpu().numpy()


def block(N, K, H, scaled, seed=0, std=2.0):
    """x, W (projections of spread `std`, so that some reach the clamps at 7), dy and scales."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(N, K, generator=g).bfloat16().cuda()
    w = (torch.randn(2 * H, K, generator=g) * (std / K ** 0.5)).bfloat16().cuda()
    dy = torch.randn(N, H, generator=g).bfloat16().cuda()
    s = torch.rand(N, generator=g).cuda() if scaled else None
    return x, w, dy, s


def np_scales(s):
    return None if s is None else s.cpu().numpy()


# one token to several tiles in each direction, odd sizes, K below and across a staged slice
SIZES = [(1, 8, 8), (1, 64, 64), (1, 2048, 264), (2, 72, 40), (5, 200, 1000), (8, 2048, 96), (9, 136, 104),
         (16, 520, 264), (17, 512, 136), (31, 1000, 72), (33, 96, 2056), (64, 4104, 128), (127, 64, 136),
         (128, 256, 128), (129, 264, 136), (255, 328, 248), (257, 72, 264), (300, 1000, 1032), (17, 136, 2056),
         (513, 128, 520), (2600, 64, 1104)]
MODES = ["bf16", "f32", "fp8_delayed", "mxfp8"]


def _check_fwd(N, K, H, act, scaled, mode, pre, std=2.0, seed=0):
    x, w, _, s = block(N, K, H, scaled, seed, std)
    quant = "none" if mode in ("bf16", "f32") else mode
    out, got_pre = rn.gated_ffn_fwd(x, w, act, s, quant=quant, limit=LIM, alpha=ALPHA,
                                    scale=torch.full((1,), 3.5, device="cuda") if mode == "fp8_delayed" else None,
                                    out_dtype=torch.float32 if mode == "f32" else None, save_pre=pre)
    x64, w64 = f64(x), f64(w)
    ref = F.gated_ffn_fwd(x64, w64, np_scales(s), act, limit=LIM, alpha=ALPHA)
    ep = ep_bound(x64, w64)
    err = y_bound(ref["p"], ep, np_scales(s), act)
    y = ref["y"]
    if mode in ("bf16", "f32"):
        assert out.dtype == (torch.bfloat16 if mode == "bf16" else torch.float32)
        check_value(f64(out), y, err, mode == "bf16", "y")
    elif mode == "fp8_delayed":
        check_codes(out.data.cpu().numpy(), y, err, 3.5, "y")
        amax = np.max(np.abs(y))
        assert abs(float(out.amax) - amax) <= np.max(err) + 2.0 ** -23 * amax
        assert float(out.scale_inv) == np.float32(1) / np.float32(3.5)
    else:
        check_mx(out.data.cpu().numpy(), out.row_scales.cpu().numpy(), y, err, "y")
    if pre:
        check_value(f64(got_pre), ref["p"], ep, True, "pre")
    else:
        assert got_pre is None


@pytest.mark.parametrize("i,size", list(enumerate(SIZES)), ids=lambda v: str(v))
def test_forward(i, size):
    N, K, H = size
    mode = MODES[i % 4]
    if mode == "mxfp8":
        H = (H + 31) // 32 * 32
    _check_fwd(N, K, H, ("swiglu", "clamped_swiglu")[(i // 4) % 2], i % 3 == 0, mode, i % 2 == 0)


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("act", ["swiglu", "clamped_swiglu"])
@pytest.mark.parametrize("N,K,H", [(3, 136, 160), (12, 1032, 32), (150, 200, 288)])
def test_forward_modes(mode, act, N, K, H):
    _check_fwd(N, K, H, act, True, mode, True, seed=1)


# few tiles and a long reduction: clusters of 4 and of 8 CTAs share a tile
@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("N,K,H", [(40, 2568, 1056), (300, 2056, 160), (200, 1288, 2080), (130, 4104, 288)])
def test_forward_shared_tiles(mode, N, K, H):
    _check_fwd(N, K, H, "clamped_swiglu" if N == 40 else "swiglu", N != 130, mode, True, seed=2)


@pytest.mark.parametrize("N,K,H,mode,split,slabs,rounds", [
    (8, 8192, 504, "bf16", 8, 1, 2), (9, 6144, 1504, "f32", 2, 1, 2), (32, 8192, 1024, "fp8_delayed", 4, 1, 2),
    (12, 8192, 2560, "mxfp8", 1, 2, 1), (8, 16384, 8192, "bf16", 1, 2, 4), (32, 12288, 504, "bf16", 8, 2, 2),
    (30, 20480, 512, "mxfp8", 8, 2, 2)])
def test_few_token_plans_of_every_kind(N, K, H, mode, split, slabs, rounds):
    """Clusters that run several steps, slabs of tokens, and both; some outputs of each against the oracle."""
    p = matvec_plan.plan(N, K, H, nvfp4=False, gated=True, mx=mode == "mxfp8")
    assert (p.split, p.slabs, p.rounds) == (split, slabs, rounds)
    g = torch.Generator(device="cuda").manual_seed(N)
    x = torch.randn(N, K, generator=g, device="cuda").bfloat16()
    w = (torch.randn(2 * H, K, generator=g, device="cuda") * (2 / K ** 0.5)).bfloat16()
    s = torch.rand(N, generator=g, device="cuda")
    quant = "none" if mode in ("bf16", "f32") else mode
    out, pre = rn.gated_ffn_fwd(x, w, "clamped_swiglu", s, quant=quant, scale=3.5 if mode == "fp8_delayed" else None,
                                out_dtype=torch.float32 if mode == "f32" else None, save_pre=True)
    cols = torch.tensor(sorted({c for a in (0, H // 64 * 32, H // 32 * 32 - 32) for c in range(a, a + 32)}
                               | set(range(H // 32 * 32, H))), device="cuda")
    x64, w64 = f64(x), f64(w[torch.cat([cols, cols + H])])
    ref = F.gated_ffn_fwd(x64, w64, np_scales(s), "clamped_swiglu", limit=LIM, alpha=ALPHA)
    ep = ep_bound(x64, w64)
    err = y_bound(ref["p"], ep, np_scales(s), "clamped_swiglu")
    check_value(f64(pre[:, torch.cat([cols, cols + H])]), ref["p"], ep, True, "pre")
    if mode in ("bf16", "f32"):
        check_value(f64(out[:, cols]), ref["y"], err, mode == "bf16", "y")
    elif mode == "fp8_delayed":
        check_codes(out.data[:, cols].cpu().numpy(), ref["y"], err, 3.5, "y")
    else:
        check_mx(out.data[:, cols].cpu().numpy(), out.row_scales[:, cols[::32] // 32].cpu().numpy(), ref["y"], err, "y")


@pytest.mark.parametrize("act", ["swiglu", "clamped_swiglu"])
@pytest.mark.parametrize("N", [8, 300])
def test_gates_far_from_zero(N, act):
    """Gates from -130 to 130, each projection one exact product, so that only the activation's own error is left:
    2 + 1.17 |z| units of 2**-23 for the exponential (CUDA's documented bound for __expf), 2 for the division and one
    for each of the sum, the product alpha a (whose half unit the exponential multiplies by |z|: another |z| / 2), the
    products with a, b and s, relative to y; and sigmoids below 2**-125, which may come out as 0."""
    H, K = 264, 8
    g = torch.Generator().manual_seed(6)
    x = torch.zeros(N, K)
    x[torch.arange(N), torch.arange(N) % K] = 2.0 ** (torch.arange(N) % 3 - 1)
    w = torch.cat([torch.linspace(-130, 130, H * K)[torch.randperm(H * K, generator=g)].view(H, K),
                   torch.randn(H, K, generator=g) * 3]).bfloat16()
    s = torch.rand(N, generator=g)
    out, pre = rn.gated_ffn_fwd(x.bfloat16().cuda(), w.cuda(), act, s.cuda(), limit=LIM, alpha=ALPHA,
                                out_dtype=torch.float32, save_pre=True)
    p = f64(x) @ f64(w).T
    assert np.array_equal(f64(pre), p)                           # exact in bf16 already
    a, b = p[:, :H], p[:, H:]
    if act == "swiglu":
        z, mag = a, np.abs(a * b)
    else:
        a, b = np.minimum(a, LIM), np.clip(b, -LIM, LIM) + 1
        z, mag = ALPHA * a, np.abs(a) * (np.abs(b - 1) + 1)      # the sum b + 1 rounds too
    mag = mag * f64(s)[:, None]
    y = F._act.scaled_act_fwd(p, np_scales(s), act, limit=LIM, alpha=ALPHA)["y"]
    tol = 2.0 ** -23 * (9 + 1.67 * np.abs(z)) * mag * F._act.sigmoid(z) + 2.0 ** -125 * mag
    assert np.all(np.abs(f64(out) - y) <= tol + 1e-37)


@pytest.mark.parametrize("i,size", list(enumerate(SIZES)), ids=lambda v: str(v))
def test_backward(i, size):
    N, K, H = size
    act = ("clamped_swiglu", "swiglu")[i % 2]
    x, w, dy, s = block(N, K, H, i % 3 != 1, seed=i)
    pre = (x.float() @ w.float().T).bfloat16()
    dx, dw, ds = rn.gated_ffn_bwd(dy, x, w, pre, act, s, limit=LIM, alpha=ALPHA)
    _check_bwd(x, w, dy, s, pre, act, dx, dw, ds)


# reductions split over the workspace: dx (many hidden rows), dW (many tokens), both
@pytest.mark.parametrize("N,K,H", [(40, 64, 3000), (3000, 72, 40), (2100, 264, 2104), (70, 520, 1544)])
def test_backward_split_reductions(N, K, H):
    x, w, dy, s = block(N, K, H, True, seed=N)
    pre = (x.float() @ w.float().T).bfloat16()
    need = rn.gated_ffn_bwd_workspace_bytes(N, K, H)
    assert need > 4 * N * H + 256                       # room for the parts' sums
    full = rn.gated_ffn_bwd(dy, x, w, pre, "swiglu", s)
    _check_bwd(x, w, dy, s, pre, "swiglu", *full)
    # a workspace on 16 bytes, and one product at a time
    ws = torch.empty(need + 16, dtype=torch.uint8, device="cuda")[16:]
    part = (*rn.gated_ffn_bwd(dy, x, w, pre, "swiglu", s, workspace=ws, need_dw=False)[:1],
            *rn.gated_ffn_bwd(dy, x, w, pre, "swiglu", s, workspace=ws, need_dx=False)[1:])
    for a, b in zip(full, part):
        assert torch.equal(a, b)


def _check_bwd(x, w, dy, s, pre, act, dx, dw, ds):
    x64, w64, dy64, pre64 = f64(x), f64(w), f64(dy), f64(pre)
    N, K = x64.shape
    ref = F.gated_ffn_bwd(dy64, x64, w64, pre64, np_scales(s), act, LIM, ALPHA)
    dp, e = ref["dp"], 2.0 ** -18 * dp_bound(pre64, dy64, np_scales(s), act)
    e = e + U * (np.abs(dp) + e)                                   # and the rounding to bf16
    if dx is not None:
        aw = np.abs(w64)
        check_grad(f64(dx), ref["dx"], e @ aw + dp.shape[1] * 2.0 ** -23 * ((np.abs(dp) + e) @ aw), "dx")
    if dw is not None:
        ax = np.abs(x64)
        check_grad(f64(dw), ref["dw"], e.T @ ax + N * 2.0 ** -23 * ((np.abs(dp) + e).T @ ax), "dw")
    if ds is not None:
        # the sum of H terms, each within 2**-18 of its magnitude, in fp32
        v = np.abs(dy64 * np.abs(F._act.act_value(pre64, act, LIM, ALPHA)))
        if act == "clamped_swiglu":                                # |b| + 1 in place of |b + 1|
            H = dy64.shape[1]
            a, b = np.minimum(pre64[:, :H], LIM), np.clip(pre64[:, H:], -LIM, LIM)
            v = np.abs(dy64 * a * F._act.sigmoid(ALPHA * a)) * (np.abs(b) + 1)
        tol = (2.0 ** -18 + dy64.shape[1] * 2.0 ** -23) * v.sum(1)
        assert np.all(np.abs(f64(ds) - ref["dscales"]) <= tol + 1e-37)


def shifted(t, by=16):
    """A contiguous copy that starts `by` bytes past an allocation's start."""
    buf = torch.empty(t.numel() * t.element_size() + by, dtype=torch.uint8, device="cuda")
    return buf[by:].view(t.dtype).view(t.shape).copy_(t)


@pytest.mark.parametrize("N,K,H", [(3, 256, 64), (3, 264, 72), (40, 128, 64), (300, 256, 320)])
def test_operands_on_16_bytes(N, K, H):
    """The documented alignment is 16 bytes: 32-byte loads and stores may only be taken where they fit."""
    lib = rn._load()
    x, w, dy, s = block(N, K, H, True)
    y, pre = rn.gated_ffn_fwd(x, w, "swiglu", s, save_pre=True)
    dx, dw, ds = rn.gated_ffn_bwd(dy, x, w, pre, "swiglu", s)
    x2, w2, dy2, y2, pre2, dx2, dw2 = (shifted(t) for t in (x, w, dy, y, pre, dx, dw))
    assert all(t.data_ptr() % 32 == 16 for t in (x2, w2, dy2, y2, pre2, dx2, dw2))
    for t in (y2, pre2, dx2, dw2):
        t.zero_()
    p = lambda t: ctypes.c_void_p(t.data_ptr())
    o = rn._Output()
    o.data, o.out_dtype = y2.data_ptr(), 0
    st = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    assert lib.rn_gated_ffn_fwd(1, p(x2), p(w2), 0, p(s), N, K, H, 7.0, 1.702, 0, ctypes.byref(o), p(pre2), st) == 0
    need = rn.gated_ffn_bwd_workspace_bytes(N, K, H)
    ws = torch.empty(need + 16, dtype=torch.uint8, device="cuda")[16:]
    n = ctypes.c_size_t(need)
    assert lib.rn_gated_ffn_bwd(1, p(dy2), p(x2), p(w2), p(pre2), 0, p(s), N, K, H, 7.0, 1.702, p(dx2), p(dw2),
                                p(ds), p(ws), ctypes.byref(n), st) == 0
    for a, b in ((y, y2), (pre, pre2), (dx, dx2), (dw, dw2)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("skip", ["dx", "dw", "ds", "both"])
def test_backward_parts(skip):
    x, w, dy, s = block(130, 136, 72, True, seed=4)
    pre = (x.float() @ w.float().T).bfloat16()
    full = rn.gated_ffn_bwd(dy, x, w, pre, "swiglu", s)
    part = rn.gated_ffn_bwd(dy, x, w, pre, "swiglu", s, dscales=skip != "ds", need_dx=skip not in ("dx", "both"),
                            need_dw=skip not in ("dw", "both"))
    for a, b in zip(full, part):
        assert b is None or torch.equal(a, b)
    assert [b is None for b in part] == [skip in ("dx", "both"), skip in ("dw", "both"), skip == "ds"]


def test_empty_batch():
    w = torch.randn(64, 32, device="cuda").bfloat16()
    x = torch.empty(0, 32, device="cuda", dtype=torch.bfloat16)
    y, pre = rn.gated_ffn_fwd(x, w, save_pre=True)
    assert y.shape == (0, 32) and pre.shape == (0, 64)
    o, _ = rn.gated_ffn_fwd(x, w, quant="fp8_delayed", scale=2.0)
    assert float(o.amax) == 0.0 and float(o.scale_inv) == 0.5
    o, _ = rn.gated_ffn_fwd(x, w, quant="mxfp8")
    assert o.data.shape == (0, 32)
    dx, dw, ds = rn.gated_ffn_bwd(y, x, w, pre)
    assert dx.shape == (0, 32) and ds.shape == (0,) and torch.equal(dw, torch.zeros_like(w))


@pytest.mark.parametrize("N,K,H", [(4, 264, 72), (130, 72, 200)])
def test_zero_scales_and_zero_rows(N, K, H):
    """Tokens of weight 0 and all-zero rows give zeros, not NaN, in every output."""
    x, w, dy, s = block(N, K, H, True)
    s[::2] = 0
    x[1] = 0
    y, pre = rn.gated_ffn_fwd(x, w, "swiglu", s, save_pre=True)
    assert torch.all(y[::2] == 0) and torch.all(y[1] == 0) and torch.all(pre[1] == 0)
    dx, dw, ds = rn.gated_ffn_bwd(dy, x, w, pre, "swiglu", s)
    assert torch.all(dx[::2] == 0) and torch.isfinite(dw.float()).all() and torch.isfinite(ds).all()
    _check_bwd(x, w, dy, s, pre, "swiglu", dx, dw, ds)
    H32 = (H + 31) // 32 * 32
    o, _ = rn.gated_ffn_fwd(x, torch.cat([w[:8].repeat(H32 // 8, 1)] * 2).contiguous(), "swiglu", s, quant="mxfp8")
    assert torch.all(o.data[::2] & 0x7F == 0) and torch.all(o.row_scales[::2] == 0)


@pytest.mark.parametrize("N,K,H", [(3, 264, 72), (12, 72, 64), (200, 136, 264)])
def test_non_finite_rows_stay_in_their_rows(N, K, H):
    x, w, dy, s = block(N, K, H, True)
    clean, pre = rn.gated_ffn_fwd(x, w, "swiglu", s, save_pre=True)
    bad = x.clone()
    bad[1, 5], bad[2, 0] = float("nan"), float("inf")
    y, p = rn.gated_ffn_fwd(bad, w, "swiglu", s, save_pre=True)
    keep = torch.ones(N, dtype=torch.bool, device="cuda")
    keep[1:3] = False
    assert torch.equal(y[keep], clean[keep]) and torch.equal(p[keep], pre[keep])
    assert torch.isnan(p[1]).all() and not torch.isfinite(p[2].float()).any()
    dy2 = dy.clone()
    dy2[1] = float("nan")
    a, b = (rn.gated_ffn_bwd(d, x, w, pre, "swiglu", s) for d in (dy, dy2))
    assert torch.equal(a[0][keep], b[0][keep]) and torch.isnan(b[0][1]).all()


@pytest.mark.parametrize("N,K,H", [(3, 264, 72), (12, 72, 64), (200, 136, 264)])
def test_nothing_is_written_behind_the_outputs(N, K, H):
    lib = rn._load()
    x, w, dy, s = block(N, K, H, True)
    fill = -2.0 ** 100                         # no result is that large

    def guarded(rows, cols, dtype=torch.bfloat16):
        return torch.full((rows + 3, cols), fill, dtype=dtype, device="cuda")

    p = lambda t: ctypes.c_void_p(t.data_ptr())
    y, pre, dx, dw = guarded(N, H), guarded(N, 2 * H), guarded(N, K), guarded(2 * H, K)
    ds = guarded(N, 1, torch.float32)
    need = rn.gated_ffn_bwd_workspace_bytes(N, K, H)
    ws = torch.full((need + 256,), 0x5A, dtype=torch.uint8, device="cuda")
    o = rn._Output()
    o.data, o.out_dtype = y.data_ptr(), 0
    st = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    assert lib.rn_gated_ffn_fwd(1, p(x), p(w), 0, p(s), N, K, H, 7.0, 1.702, 0, ctypes.byref(o), p(pre), st) == 0
    n = ctypes.c_size_t(need)
    assert lib.rn_gated_ffn_bwd(1, p(dy), p(x), p(w), p(pre), 0, p(s), N, K, H, 7.0, 1.702, p(dx), p(dw), p(ds),
                                p(ws), ctypes.byref(n), st) == 0
    for t, rows in ((y, N), (pre, N), (dx, N), (dw, 2 * H), (ds, N)):
        assert torch.all(t[rows:] == fill) and not torch.any(t[:rows] == fill).item()
    assert torch.all(ws[need:] == 0x5A)


def test_offsets_past_32_bits():
    """Projections of more than 2**31 elements: the last tokens' rows, checked against the same tokens alone,
    forward and backward (a token's row of y, pre and dx does not depend on how many there are)."""
    N, K, H = 133_000, 64, 8200
    assert N * 2 * H > 2 ** 31
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(N, K, generator=g, device="cuda").bfloat16()
    w = (torch.randn(2 * H, K, generator=g, device="cuda") / 8).bfloat16()
    dy = torch.randn(N, H, generator=g, device="cuda").bfloat16()
    y, pre = rn.gated_ffn_fwd(x, w, save_pre=True)
    dx, dw, ds = rn.gated_ffn_bwd(dy, x, w, pre)
    for lo in (0, N // 2, N - 300):
        t = slice(lo, lo + 300)
        y2, pre2 = rn.gated_ffn_fwd(x[t].contiguous(), w, save_pre=True)
        assert torch.equal(y[t], y2) and torch.equal(pre[t], pre2)
        p2 = f64(pre2)
        ref = F.gated_ffn_bwd(f64(dy[t]), f64(x[t]), f64(w), p2, None, "swiglu")
        e = 2.0 ** -18 * dp_bound(p2, f64(dy[t]), None, "swiglu")
        e = e + U * (np.abs(ref["dp"]) + e)
        aw = np.abs(f64(w))
        check_grad(f64(dx[t]), ref["dx"], e @ aw + 2 * H * 2.0 ** -23 * ((np.abs(ref["dp"]) + e) @ aw), "dx")
    # dW over all tokens: a sum of dp^T x over slices of tokens in fp64, on the device
    want = torch.zeros(2 * H, K, dtype=torch.float64, device="cuda")
    for lo in range(0, N, 8192):
        t = slice(lo, lo + 8192)
        a, b, d = pre[t, :H].double(), pre[t, H:].double(), dy[t].double()
        sg = torch.sigmoid(a)
        dp = torch.cat([d * b * sg * (1 + a * (1 - sg)), d * a * sg], 1)
        want += dp.T @ x[t].double()
    assert float((dw.double() - want).norm() / want.norm()) <= 4e-3


def _step(x, w, dy, s, ws=None):
    y, pre = rn.gated_ffn_fwd(x, w, "clamped_swiglu", s, save_pre=True)
    return (y, pre, *rn.gated_ffn_bwd(dy, x, w, pre, "clamped_swiglu", s, workspace=ws))


@pytest.mark.parametrize("N,K,H", [(1, 264, 72), (12, 520, 64), (300, 264, 520)])
def test_runs_repeat_bit_for_bit_on_any_stream(N, K, H):
    x, w, dy, s = block(N, K, H, True)
    want = _step(x, w, dy, s)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(3):
        for st in streams:                     # two calls at once, each with its own workspace
            with torch.cuda.stream(st):
                got.append(_step(x, w, dy, s))
    torch.cuda.synchronize()
    for g in got:
        for a, b in zip(want, g):
            assert torch.equal(a, b)


@pytest.mark.parametrize("N,K,H", [(1, 264, 72), (300, 264, 520)])
def test_capture_and_replay(N, K, H):
    x, w, dy, s = block(N, K, H, True)
    ws = torch.empty(rn.gated_ffn_bwd_workspace_bytes(N, K, H), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _step(x, w, dy, s, ws)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = _step(x, w, dy, s, ws)
        o8, _ = rn.gated_ffn_fwd(x, w, "swiglu", s, quant="fp8_delayed", scale=torch.ones(1, device="cuda"))
    for seed in (7, 8):
        x2, w2, dy2, s2 = block(N, K, H, True, seed=seed)
        for a, b in ((x, x2), (w, w2), (dy, dy2), (s, s2)):
            a.copy_(b)
        graph.replay()
        want = _step(x2, w2, dy2, s2)
        w8, _ = rn.gated_ffn_fwd(x2, w2, "swiglu", s2, quant="fp8_delayed", scale=1.0)
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert torch.equal(a, b)
        assert torch.equal(o8.data, w8.data) and torch.equal(o8.amax, w8.amax)


def _difference_inputs():
    """x, W of 4 significant bits and +-|v| / 16 steps of a tenth of their entries, along the oracle's
    gradient: v +- step is exact in bf16, and the slope is a sum of positive terms."""
    N, K, H = 40, 72, 64
    g = torch.Generator().manual_seed(5)

    def coarse(*shape, std):
        v = torch.randn(*shape, generator=g) * std
        m, e = torch.frexp(v)
        return torch.ldexp(torch.round(m * 8) / 8, e)

    x, w = coarse(N, K, std=1.0), coarse(2 * H, K, std=1.0 / K ** 0.5)
    dy = torch.randn(N, H, generator=g).bfloat16()
    o = F.gated_ffn_bwd(f64(dy), f64(x), f64(w), f64(x) @ f64(w).T, None, "swiglu")
    step = []
    for v, grad in ((x, o["dx"]), (w, o["dw"])):
        pick = torch.rand(v.shape, generator=g) < 0.1
        step.append(torch.where(pick, v.abs() / 16, 0.0) * torch.from_numpy(np.sign(grad)).float())
        for sg in (1, -1):
            assert torch.equal((v + sg * step[-1]).bfloat16().float(), v + sg * step[-1])
    return x, w, dy, step, o


@pytest.mark.parametrize("which", ["dx", "dw"])
def test_gradients_against_differences(which):
    """(L(v + t) - L(v - t)) / 2 of the kernel's own fp32 forward, L = sum dy * y, against <grad, t>.

    The forward's bound (ffn_check.py) carries through L; the third-order remainder is the oracle's own
    difference less its slope.  <grad, t> differs from the slope by the rounding of pre (u |p| in both
    arguments of act', whose derivatives there stay below 1.1 (1 + |b|): |act''| <= 1.1 (1 + |b|)), of dp (u |dp|)
    and of the result (u), all times |t|."""
    x, w, dy, step, o = _difference_inputs()
    t = step[0] if which == "dx" else step[1]
    val, ref, tol = [], [], 0.0
    for sg in (1, -1):
        xs, ws = (x + sg * t, w) if which == "dx" else (x, w + sg * t)
        y, _ = rn.gated_ffn_fwd(xs.bfloat16().cuda(), ws.bfloat16().cuda(), out_dtype=torch.float32)
        r = F.gated_ffn_fwd(f64(xs), f64(ws), None, "swiglu")
        err = y_bound(r["p"], ep_bound(f64(xs), f64(ws)), None, "swiglu") + 2.0 ** -24 * np.abs(r["y"])
        val.append(np.sum(f64(dy) * f64(y)))
        ref.append(np.sum(f64(dy) * r["y"]))
        tol += np.sum(np.abs(f64(dy)) * err) / 2
    diff = (val[0] - val[1]) / 2
    assert abs(diff - (ref[0] - ref[1]) / 2) <= tol
    xd, wd, dyd = x.bfloat16().cuda(), w.bfloat16().cuda(), dy.cuda()
    _, pre = rn.gated_ffn_fwd(xd, wd, save_pre=True)
    dx, dw, _ = rn.gated_ffn_bwd(dyd, xd, wd, pre)
    grad = f64(dx if which == "dx" else dw)
    slope, bound = _difference_slope(x, w, dy, t, o, which)
    third = abs((ref[0] - ref[1]) / 2 - slope)
    assert abs(diff - np.sum(grad * f64(t))) <= tol + third + bound


def _difference_slope(x, w, dy, t, o, which):
    H = dy.shape[1]
    p = np.abs(f64(x) @ f64(w).T)
    dev = np.tile(1.1 * (1 + p[:, H:]) * np.abs(f64(dy)) * U * (p[:, :H] + p[:, H:]), 2) + U * np.abs(o["dp"])
    lin = np.abs(f64(t)) @ np.abs(f64(w)).T if which == "dx" else np.abs(f64(x)) @ np.abs(f64(t)).T
    slope = np.sum(o[which] * f64(t))
    return slope, np.sum(dev * lin) + U * np.sum(np.abs(o[which] * f64(t)))


@pytest.mark.parametrize("quant", ["none", "mxfp8"])
def test_norm_block_and_backward_together(quant):
    """RMSNorm -> gated block -> a down projection, and back through all of them, as a training step runs
    them, against fp64 autograd of the same chain with the kernels' bf16 intermediates."""
    N, C, H = 150, 264, 320
    g = torch.Generator().manual_seed(2)
    x = torch.randn(N, C, generator=g).bfloat16().cuda()
    gamma = (1 + 0.1 * torch.randn(C, generator=g)).cuda()
    w = (torch.randn(2 * H, C, generator=g) / C ** 0.5).bfloat16().cuda()
    wd = (torch.randn(C, H, generator=g) / H ** 0.5).bfloat16().cuda()
    dz = torch.randn(N, C, generator=g).bfloat16().cuda()
    h, rs = rn.rmsnorm_fwd(x, gamma, 1e-5)
    y, pre = rn.gated_ffn_fwd(h, w, save_pre=True)
    dy = (dz.float() @ wd.float()).bfloat16()
    dh, dw, _ = rn.gated_ffn_bwd(dy, h, w, pre)
    dx, dg = rn.rmsnorm_bwd(dh, x, rs, gamma)
    xr, gr, wr = (t.double().requires_grad_() for t in (x, gamma, w))
    hr = xr * torch.rsqrt((xr * xr).mean(1, keepdim=True) + 1e-5) * gr
    pr = hr @ wr.T
    yr = pr[:, :H] * torch.sigmoid(pr[:, :H]) * pr[:, H:]
    (yr @ wd.double().T * dz.double()).sum().backward()
    # each bf16 intermediate (h, pre, dy, dp, dh and the result) adds an independent relative error of
    # u / sqrt(3) at most; seven of them in a row stay below sqrt(7 / 3) u = 6e-3
    for a, b in ((y, yr), (dw, wr.grad), (dx, xr.grad), (dg, gr.grad)):
        assert float((a.double() - b).detach().norm() / b.detach().norm()) <= 6e-3
    if quant == "mxfp8":
        o, _ = rn.gated_ffn_fwd(h, w, quant="mxfp8")
        p = F.projections(f64(h), f64(w))
        err = y_bound(p, ep_bound(f64(h), f64(w)), None, "swiglu")
        check_mx(o.data.cpu().numpy(), o.row_scales.cpu().numpy(), F._act.act_value(p, "swiglu"), err, "y")
