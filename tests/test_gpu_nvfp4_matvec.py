"""GPU parity of the products with NVFP4 weights (rn_nvfp4_matvec,
rn_nvfp4_gated_ffn) against the oracle; the bounds are derived in
ffn_check.py.  The sums run over E2M1 value * block scale (exact in bf16),
so 1/S multiplies their bound, and one more rounding of fp32 is added."""
import ctypes

import numpy as np
import pytest
import torch

import mxfp8_quantization_gb300 as rn
import matvec_plan
from ffn_check import ALPHA, LIM, check_codes, check_mx, check_value, ep_bound, y_bound
from oracle import ffn as F
from test_gpu_ffn import MODES, f64, np_scales

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _no_device_error():
    yield
    assert rn.device_error() == 0


def weights(R, K, seed=0, std=2.0):
    g = torch.Generator().manual_seed(seed)
    if K > 16384:   # wider than rn_quantize_only takes: any codes, block scales in [0.5, 2]
        si = torch.full((1,), 2.0 ** -9, device="cuda")
        return rn.NVFP4Output(torch.randint(0, 256, (R, K // 2), generator=g, dtype=torch.uint8).cuda(),
                              torch.randint(0x30, 0x41, (R, K // 16), generator=g, dtype=torch.uint8).cuda(),
                              1 / si, si, si)
    w = torch.randn(R, K, generator=g) * (std / K ** 0.5)
    return rn.quantize_only(w.cuda(), "nvfp4")


def tokens(N, K, seed=0):
    return torch.randn(N, K, generator=torch.Generator().manual_seed(seed + 100)).bfloat16().cuda()


def values(w):
    return F.nvfp4_values(w.data.cpu().numpy(), w.row_scales.cpu().numpy(), w.scale_inv.cpu().numpy()[0])


def proj(x, w):
    x64, v = f64(x), values(w)
    p = x64 @ v.T
    return p, ep_bound(x64, v) + 2.0 ** -23 * np.abs(p)


# (N, K, R): K of one block, of an odd number of blocks, across every split; R odd; tokens across groups of 8
SIZES = [(1, 16, 1), (1, 32, 7), (1, 48, 33), (1, 4096, 64), (1, 2064, 250), (2, 4112, 65), (3, 16384, 17),
         (4, 128, 513), (7, 1040, 64), (8, 2048, 100), (9, 512, 96), (13, 5136, 40), (16, 256, 31),
         (17, 1024, 64), (24, 144, 130), (32, 8192, 24), (33, 96, 48), (40, 2080, 66), (100, 1024, 72),
         (1, 1024, 20000), (5, 4160, 70), (3, 65536, 24), (12, 65536, 40), (20, 65520, 16)]


@pytest.mark.parametrize("i,size", list(enumerate(SIZES)), ids=lambda v: str(v))
def test_matvec(i, size):
    N, K, R = size
    x, w = tokens(N, K, i), weights(R, K, i)
    dt = (torch.bfloat16, torch.float32)[i % 2]
    y = rn.nvfp4_matvec(x, w, out_dtype=dt)
    p, ep = proj(x, w)
    assert y.dtype == dt
    check_value(f64(y), p, ep, dt == torch.bfloat16, "y")


@pytest.mark.parametrize("i,size", list(enumerate(SIZES)), ids=lambda v: str(v))
def test_gated(i, size):
    N, K, H = size
    mode = MODES[i % 4]
    if mode == "mxfp8":
        H = (H + 31) // 32 * 32
    _check_gated(N, K, H, ("swiglu", "clamped_swiglu")[(i // 4) % 2], i % 3 == 0, mode, i)


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("act", ["swiglu", "clamped_swiglu"])
@pytest.mark.parametrize("N,K,H", [(1, 144, 160), (12, 1040, 32)])
def test_gated_modes(mode, act, N, K, H):
    _check_gated(N, K, H, act, True, mode, 3)


def _check_gated(N, K, H, act, scaled, mode, seed):
    x, w = tokens(N, K, seed), weights(2 * H, K, seed)
    s = torch.rand(N, generator=torch.Generator().manual_seed(seed)).cuda() if scaled else None
    quant = "none" if mode in ("bf16", "f32") else mode
    out = rn.nvfp4_gated_ffn(x, w, act, s, quant=quant, limit=LIM, alpha=ALPHA,
                             scale=3.5 if mode == "fp8_delayed" else None,
                             out_dtype=torch.float32 if mode == "f32" else None)
    p, ep = proj(x, w)
    ref = F._act.scaled_act_fwd(p, np_scales(s), act, limit=LIM, alpha=ALPHA)["y"]
    err = y_bound(p, ep, np_scales(s), act)
    if mode in ("bf16", "f32"):
        check_value(f64(out), ref, err, mode == "bf16", "y")
    elif mode == "fp8_delayed":
        check_codes(out.data.cpu().numpy(), ref, err, 3.5, "y")
        assert abs(float(out.amax) - np.max(np.abs(ref))) <= np.max(err) + 2.0 ** -23 * np.max(np.abs(ref))
        assert float(out.scale_inv) == np.float32(1) / np.float32(3.5)
    else:
        check_mx(out.data.cpu().numpy(), out.row_scales.cpu().numpy(), ref, err, "y")


@pytest.mark.parametrize("N", [3, 9, 16, 30])
@pytest.mark.parametrize("K", [96, 1040, 2048])
def test_many_rows(N, K):
    # rows enough that a CTA's warps take several row tiles each, the reduction short or of middle length
    x, w = tokens(N, K, N), weights(20000, K, K)
    p, ep = proj(x, w)
    check_value(f64(rn.nvfp4_matvec(x, w, out_dtype=torch.float32)), p, ep, False, "y")
    _check_gated(N, K, 9984, "swiglu", True, "mxfp8", K)
    _check_gated(N, K, 9999, "clamped_swiglu", False, "bf16", K)


@pytest.mark.parametrize("N,K,H,gated,mode,kw", [(16, 2048, 20000, False, "f32", 2), (16, 2048, 32768, False, "f32", 3),
                                                 (12, 2208, 16068, True, "bf16", 3), (11, 784, 6000, True, "f32", 4),
                                                 (10, 512, 10240, True, "mxfp8", 2), (1, 624, 8797, True, "fp8_delayed", 4)])
def test_warps_along_the_reduction(N, K, H, gated, mode, kw):
    """Numbers of warps along the reduction that the halving alone does not come to."""
    assert matvec_plan.plan(N, K, H, True, gated, mode == "mxfp8").kw == kw
    if gated:
        _check_gated(N, K, H, "swiglu", True, mode, N)
    else:
        x, w = tokens(N, K, N), weights(H, K, K)
        p, ep = proj(x, w)
        check_value(f64(rn.nvfp4_matvec(x, w, out_dtype=torch.float32)), p, ep, False, "y")


def codes(R, K, seed):
    """Any codes, block scales in [0.5, 2], projections of spread about 2 for tokens of spread 1; made on the GPU."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    si = torch.full((1,), 0.6 / K ** 0.5, device="cuda")
    return rn.NVFP4Output(torch.randint(0, 256, (R, K // 2), generator=g, dtype=torch.uint8, device="cuda"),
                          torch.randint(0x30, 0x41, (R, K // 16), generator=g, dtype=torch.uint8, device="cuda"),
                          1 / si, si, si)


def some_outputs(H):
    """Blocks of 32 outputs at the start, in the middle and at the end, and the last ones."""
    at = {0, H // 64 * 32, max(0, H // 32 * 32 - 32)}
    cols = sorted({c for a in at for c in range(a, min(a + 32, H))} | set(range(H // 32 * 32, H)))
    return torch.tensor(cols, device="cuda")


def check_some(x, w, H, gated, mode):
    """Some outputs against the oracle."""
    cols = some_outputs(H)
    rows = torch.cat([cols, cols + H]) if gated else cols
    part = rn.NVFP4Output(w.data[rows], w.row_scales[rows], w.scale, w.scale_inv, w.amax)
    p, ep = proj(x, part)
    if not gated:
        y = rn.nvfp4_matvec(x, w, out_dtype=torch.float32)
        check_value(f64(y[:, cols]), p, ep, False, "y")
        return
    ref, err = F._act.scaled_act_fwd(p, None, "swiglu")["y"], y_bound(p, ep, None, "swiglu")
    y32 = rn.nvfp4_gated_ffn(x, w, out_dtype=torch.float32)
    check_value(f64(y32[:, cols]), ref, err, False, "y")
    if mode == "bf16":
        check_value(f64(rn.nvfp4_gated_ffn(x, w)[:, cols]), ref, err, True, "y")
    elif mode == "fp8_delayed":
        out = rn.nvfp4_gated_ffn(x, w, quant=mode, scale=3.5)
        check_codes(out.data[:, cols].cpu().numpy(), ref, err, 3.5, "y")
        assert float(out.amax) == float(y32.abs().max())        # the same sums
    elif mode == "mxfp8":
        out = rn.nvfp4_gated_ffn(x, w, quant=mode)
        blocks = cols[::32] // 32
        check_mx(out.data[:, cols].cpu().numpy(), out.row_scales[:, blocks].cpu().numpy(), ref, err, "y")


@pytest.mark.parametrize("N,K,H,gated,mode,rounds,batches", [
    (32, 16384, 64, False, "f32", 1, 1), (32, 16384, 1024, False, "f32", 1, 1), (32, 16384, 4096, False, "f32", 2, 1),
    (30, 16384, 1024, True, "mxfp8", 1, 1), (32, 12288, 500, True, "fp8_delayed", 1, 1), (12, 65536, 40, False, "f32", 1, 1),
    (16, 32768, 4096, False, "f32", 2, 1), (16, 49152, 500, True, "bf16", 2, 1), (24, 32768, 512, True, "mxfp8", 2, 1),
    (40, 16384, 200, True, "bf16", 1, 1)])
def test_clusters_with_slabs(N, K, H, gated, mode, rounds, batches):
    """The reduction over a cluster whose CTAs take their tokens slab after slab."""
    p = matvec_plan.plan(N, K, H, True, gated, mode == "mxfp8")
    assert p.split > 1 and p.slabs > 1 and (p.rounds, p.batches) == (rounds, batches)
    check_some(tokens(N, K, N), codes(H * (1 + gated), K, N), H, gated, mode)


@pytest.mark.parametrize("N,K,H,gated,mode,split,slabs,rounds,batches", [
    # clusters that run several steps, so that their leaders change and the sums' places are used again
    (8, 8192, 2500, False, "f32", 2, 1, 2, 1), (16, 20000, 500, False, "f32", 8, 1, 2, 1),
    (17, 16384, 1500, True, "bf16", 4, 1, 2, 1), (9, 24576, 1504, True, "mxfp8", 8, 1, 2, 1),
    (8, 40000, 2000, True, "fp8_delayed", 4, 1, 4, 1), (12, 49152, 2048, True, "bf16", 8, 1, 5, 1),
    # slabs whose steps' sums are kept, plain and gated; two batches of steps over the slabs
    (32, 4096, 32768, False, "f32", 1, 3, 2, 1), (32, 4096, 32768, True, "fp8_delayed", 1, 3, 2, 2),
    (24, 4096, 10016, True, "mxfp8", 1, 2, 2, 1), (9, 12288, 5024, True, "mxfp8", 1, 2, 2, 1),
    (8, 12288, 2500, True, "bf16", 1, 2, 2, 1), (32, 8192, 20000, False, "f32", 1, 5, 2, 1),
    (16, 16384, 30000, False, "f32", 1, 4, 2, 1)])
def test_plans_of_every_kind(N, K, H, gated, mode, split, slabs, rounds, batches):
    p = matvec_plan.plan(N, K, H, True, gated, mode == "mxfp8")
    assert (p.split, p.slabs, p.rounds, p.batches) == (split, slabs, rounds, batches)
    check_some(tokens(N, K, N), codes(H * (1 + gated), K, N), H, gated, mode)


@pytest.mark.parametrize("N,K,H,split", [(9, 12288, 5000, 1), (17, 8192, 5000, 1), (32, 16384, 512, 4), (12, 65536, 40, 8)])
@pytest.mark.parametrize("where", [0, 1])
def test_slabs_of_different_scale(N, K, H, split, where):
    """One slab's tokens span too much for f16 and stay bf16, another's are far smaller and scaled by their own
    power of two."""
    p = matvec_plan.plan(N, K, H)
    assert p.split == split and p.slabs > 1
    x, w = tokens(N, K, N), codes(H, K, N)
    slab = p.slab * 256
    if where == 0:
        w.data[:, :8] = 0                                     # the large elements' weights are 0
        x[:, :16] = 2.0 ** 60
        x[:, slab:] *= 2.0 ** -20
    else:
        x[:, :slab] *= 2.0 ** -30
        x[:, slab + 7] *= 2.0 ** -40                          # beside ordinary ones
    check_some(x, w, H, False, "f32")


def shifted(t, by=16):
    """A contiguous copy that starts `by` bytes past an allocation's start."""
    buf = torch.empty(t.numel() * t.element_size() + by, dtype=torch.uint8, device="cuda")
    out = buf[by:].view(t.dtype).view(t.shape)
    return out.copy_(t)


@pytest.mark.parametrize("N", [1, 13, 24])
@pytest.mark.parametrize("K", [512, 320, 288, 272])
def test_operands_on_16_bytes(N, K):
    """The documented alignment is 16 bytes: 32-byte loads may only be taken where they fit."""
    x, w = tokens(N, K), weights(96, K)
    v = rn.NVFP4Output(shifted(w.data), shifted(w.row_scales), w.scale, w.scale_inv, w.amax)
    assert v.data.data_ptr() % 32 == 16 and shifted(x).data_ptr() % 32 == 16
    for a, b in ((x, shifted(x)), (shifted(x), x)):
        assert torch.equal(rn.nvfp4_matvec(a, v), rn.nvfp4_matvec(b, w))
        assert torch.equal(rn.nvfp4_gated_ffn(a, v), rn.nvfp4_gated_ffn(b, w))


def test_every_code_and_scale():
    """Each E2M1 code under each finite E4M3 scale, subnormal and negative ones too, times powers of two
    of x that put a single term in the sum: exact."""
    R, K = 16, 256
    codes = np.zeros((R, K), np.uint8)
    codes[np.arange(R), :] = np.arange(R)[:, None]          # row r: code r everywhere
    blocks = np.array([c for c in range(256) if c & 0x7F != 0x7F], np.uint8)
    packed = torch.from_numpy(codes[:, 0::2] | codes[:, 1::2] << 4).cuda()
    si = torch.full((1,), 0.125, device="cuda")
    for b0 in range(0, len(blocks), 16):
        b = np.resize(blocks[b0:b0 + 16], 16)
        bs = np.tile(b, (R, 1))
        w = rn.NVFP4Output(packed, torch.from_numpy(bs).cuda(), si * 0 + 8, si, si)
        for k in (0, 1, 15):                                 # one element of each block
            x = torch.zeros(16, K)
            x[np.arange(16), np.arange(16) * 16 + k] = 2.0 ** torch.arange(-8, 8).float()
            x = x.bfloat16().cuda()
            y = rn.nvfp4_matvec(x, w, out_dtype=torch.float32)
            assert np.array_equal(f64(y), f64(x) @ F.nvfp4_values(packed.cpu().numpy(), bs, 0.125).T)


def test_offsets_past_32_bits():
    """Weights of more than 4 GiB: the last rows, against the same rows alone."""
    R, K = 133_000, 65536
    assert R * K // 2 > 2 ** 32
    g = torch.Generator(device="cuda").manual_seed(1)
    one = torch.ones(1, device="cuda")
    w = rn.NVFP4Output(torch.randint(0, 256, (R, K // 2), generator=g, dtype=torch.uint8, device="cuda"),
                       torch.randint(0x30, 0x41, (R, K // 16), generator=g, dtype=torch.uint8, device="cuda"),
                       one, one, one)
    for N in (1, 12):
        x = tokens(N, K, N)
        y = rn.nvfp4_matvec(x, w, out_dtype=torch.float32)
        for lo in (0, R - 40):
            part = rn.NVFP4Output(w.data[lo:lo + 40].clone(), w.row_scales[lo:lo + 40].clone(), one, one, one)
            p, ep = proj(x, part)
            check_value(f64(y[:, lo:lo + 40]), p, ep, False, "y")


def test_wide_range_of_inputs():
    """Activations near bf16's ends keep their products: 2**100 and 2**-100 beside ones whose weight is 0."""
    K, R = 512, 40
    w = weights(R, K, 9)
    w.data[:, :8] = 0                                        # the first block's weights are 0
    x = tokens(2, K, 9)
    x[0] *= 2.0 ** -100
    x[1] *= 2.0 ** 100
    x[:, :16] = 2.0 ** 110
    p, ep = proj(x, w)
    ep = ep_bound(np.where(np.arange(K) < 16, 0, f64(x)), values(w)) + 2.0 ** -23 * np.abs(p)
    y = rn.nvfp4_matvec(x, w, out_dtype=torch.float32)
    check_value(f64(y), p, ep, False, "y")


def test_non_finite_rows_stay_in_their_rows():
    x, w = tokens(11, 1040, 1), weights(96, 1040, 1)
    clean = rn.nvfp4_matvec(x, w)
    bad = x.clone()
    bad[3, 7], bad[9, 1] = float("nan"), float("inf")
    y = rn.nvfp4_matvec(bad, w)
    keep = [i for i in range(11) if i not in (3, 9)]
    assert torch.equal(y[keep], clean[keep]) and torch.isnan(y[3]).all()
    assert not torch.isfinite(y[9].float()).any()


@pytest.mark.parametrize("N", [1, 9, 16, 17])
@pytest.mark.parametrize("K", [16, 48, 96, 112, 128, 144, 240, 272, 304, 400, 528, 5136])
def test_scales_of_neighbouring_rows_stay_apart(N, K):
    # every second row's scales are NaN: the rows between end and begin beside them, on any byte
    R = 37
    x, w = tokens(N, K, K), weights(R, K, K)
    want = rn.nvfp4_matvec(x, w, out_dtype=torch.float32)
    p, ep = proj(x, w)
    check_value(f64(want), p, ep, False, "y")
    w.row_scales[1::2] = 0x7F
    y = rn.nvfp4_matvec(x, w, out_dtype=torch.float32)
    assert torch.equal(y[:, 0::2], want[:, 0::2])
    assert torch.isnan(y[:, 1::2]).all()


def test_empty_batch():
    w = weights(64, 32)
    x = torch.empty(0, 32, device="cuda", dtype=torch.bfloat16)
    assert rn.nvfp4_matvec(x, w).shape == (0, 64)
    o = rn.nvfp4_gated_ffn(x, w, quant="fp8_delayed", scale=4.0)
    assert float(o.amax) == 0.0 and float(o.scale_inv) == 0.25


@pytest.mark.parametrize("N,R", [(1, 33), (9, 250)])
def test_nothing_is_written_behind_the_output(N, R):
    lib = rn._load()
    x, w = tokens(N, 272, 2), weights(R, 272, 2)
    y = torch.full((N * R + 64,), -7.75, dtype=torch.float32, device="cuda")
    p = lambda t: ctypes.c_void_p(t.data_ptr())
    assert lib.rn_nvfp4_matvec(p(x), 0, p(w.data), p(w.row_scales), p(w.scale_inv), N, 272, R, 1, p(y),
                               ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)) == 0
    assert torch.all(y[N * R:] == -7.75)
    assert torch.equal(y[:N * R].view(N, R), rn.nvfp4_matvec(x, w, out_dtype=torch.float32))


@pytest.mark.parametrize("N,K,H", [(1, 1040, 96), (13, 528, 200)])
def test_repeats_and_replays(N, K, H):
    x, w = tokens(N, K), weights(2 * H, K)
    want = rn.nvfp4_matvec(x, w), rn.nvfp4_gated_ffn(x, w)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for st in streams * 3:
        with torch.cuda.stream(st):
            got.append((rn.nvfp4_matvec(x, w), rn.nvfp4_gated_ffn(x, w)))
    torch.cuda.synchronize()
    for g in got:
        assert torch.equal(g[0], want[0]) and torch.equal(g[1], want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = rn.nvfp4_matvec(x, w), rn.nvfp4_gated_ffn(x, w)
    x.copy_(tokens(N, K, 5))
    graph.replay()
    want = rn.nvfp4_matvec(x, w), rn.nvfp4_gated_ffn(x, w)
    torch.cuda.synchronize()
    assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])


@pytest.mark.parametrize("N,K,R", [(1, 4096, 64), (1, 4096, 4096), (3, 16384, 40), (12, 4096, 96), (20, 4096, 64)])
def test_clusters_that_start_apart(N, K, R):
    """Few rows and a long reduction go to clusters of CTAs; launches on two streams crowd each other, so that
    a cluster's CTAs find their places at different times."""
    x, w = tokens(N, K, N), weights(R, K, R)
    want = rn.nvfp4_matvec(x, w, out_dtype=torch.float32)
    p, ep = proj(x, w)
    check_value(f64(want), p, ep, False, "y")
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for _ in range(100):
        for st in streams:
            with torch.cuda.stream(st):
                got.append(rn.nvfp4_matvec(x, w, out_dtype=torch.float32))
    torch.cuda.synchronize()
    assert all(torch.equal(g, want) for g in got)


def test_generation_step_together():
    """RMSNorm -> gated block -> down projection on NVFP4 weights, as one token is generated; the block
    with bf16 weights of the same values gives the same result within both bounds."""
    C, H = 512, 1056
    x = tokens(1, C, 3)
    gamma = torch.ones(C, device="cuda")
    up, down = weights(2 * H, C, 4), weights(C, H, 5)
    h, _ = rn.rmsnorm_fwd(x, gamma, 1e-5)
    y = rn.nvfp4_gated_ffn(h, up)
    z = rn.nvfp4_matvec(y, down)
    p, ep = proj(h, up)
    err = y_bound(p, ep, None, "swiglu")
    check_value(f64(y), F._act.act_value(p, "swiglu"), err, True, "y")
    pz, ez = proj(y, down)
    check_value(f64(z), pz, ez, True, "z")
    # values of the codes times S are exact in bf16; S back in through the activations' own bound
    one = rn.NVFP4Output(up.data, up.row_scales, up.scale, torch.ones(1, device="cuda"), up.amax)
    wide = torch.from_numpy(values(one)).bfloat16().cuda()
    hs = (h.float() * 2.0 ** -12).bfloat16()                     # keeps the projections small; exact
    a = rn.nvfp4_gated_ffn(hs, one, out_dtype=torch.float32)
    b, _ = rn.gated_ffn_fwd(hs, wide, out_dtype=torch.float32)
    p, ep = proj(hs, one)
    err = y_bound(p, ep, None, "swiglu")
    ref = F._act.act_value(p, "swiglu")
    check_value(f64(a), ref, err, False, "nvfp4")
    check_value(f64(b), ref, err, False, "bf16")
