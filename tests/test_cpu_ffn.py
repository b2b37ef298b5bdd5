"""Host-side argument checks of the gated feed-forward block and the NVFP4
products: each answers before any device work (no GPU is touched)."""
import ctypes
import os
import subprocess
import sys

import pytest
import torch

import mxfp8_quantization_gb300 as rn
from mxfp8_quantization_gb300 import _build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3
f32 = ctypes.c_float


def P(a):
    return ctypes.c_void_p(a)


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return rn._load()


def _out(**kw):
    o = rn._Output()
    for k, v in kw.items():
        setattr(o, k, v)
    return o


FWD = dict(act=1, x=0x1000, w=0x2000, dtype=0, scales=None, N=4, K=64, H=32, limit=7.0, alpha=1.702,
           mode=0, out=dict(data=0x5000, out_dtype=0), pre=None)
FP8 = dict(data=0x5000, scale=0x6000, scale_inv=0x6010, amax=0x6020)
MX = dict(data=0x5000, row_scales=0x6000)
NV = dict(data=0x5000, row_scales=0x6000, scale_out=0x7000, scale_inv=0x7010, amax=0x7020)


def _fwd(lib, **kw):
    a = {**FWD, **kw}
    o = None if a["out"] is None else ctypes.byref(_out(**a["out"]))
    return lib.rn_gated_ffn_fwd(a["act"], P(a["x"]), P(a["w"]), a["dtype"], P(a["scales"]), a["N"], a["K"],
                                a["H"], f32(a["limit"]), f32(a["alpha"]), a["mode"], o, P(a["pre"]), None)


# refused by every entry point that takes the argument
SHARED = [
    (dict(act=7), INVALID), (dict(act=0), UNSUPPORTED), (dict(x=None), INVALID),
    (dict(dtype=7), INVALID), (dict(dtype=1), UNSUPPORTED), (dict(N=-1), INVALID),
    (dict(N=2 ** 31), INVALID), (dict(K=0), INVALID), (dict(K=-8), INVALID), (dict(K=2 ** 31), INVALID),
    (dict(H=0), INVALID), (dict(H=2 ** 30), INVALID), (dict(x=0x1008), UNSUPPORTED),
    (dict(scales=0x3002), UNSUPPORTED), (dict(act=2, limit=-1.0), INVALID),
    (dict(act=2, limit=float("nan")), INVALID), (dict(act=2, alpha=float("inf")), INVALID),
    (dict(out=None), INVALID), (dict(out=dict(data=None, out_dtype=0)), INVALID),
    (dict(out=dict(data=0x5000, out_dtype=5)), INVALID), (dict(out=dict(data=0x5004, out_dtype=0)), UNSUPPORTED),
    (dict(out=dict(data=0x5000, out_dtype=0, amax=0x6000)), INVALID), (dict(mode=9), INVALID),
    (dict(mode=1, out=dict(FP8, scale=None)), INVALID), (dict(mode=1, out=dict(FP8, amax=None)), INVALID),
    (dict(mode=2, out=dict(data=0x5000, scale_out=0x6000, scale_inv=0x6010, amax=0x6020)), UNSUPPORTED),
    (dict(mode=3, out=dict(MX, row_scales=None)), INVALID), (dict(mode=3, out=MX, H=40), UNSUPPORTED),
    (dict(mode=3, out=dict(MX, col_data=0x7000, col_scales=0x8000)), UNSUPPORTED),
    (dict(mode=3, out=dict(MX, data=0x5008)), UNSUPPORTED), (dict(mode=4, out=NV), UNSUPPORTED),
]


@pytest.mark.parametrize("kw,want", SHARED + [
    (dict(w=None), INVALID), (dict(w=0x2004), UNSUPPORTED), (dict(pre=0x7008), UNSUPPORTED),
    (dict(K=68), UNSUPPORTED), (dict(H=36), UNSUPPORTED), (dict(K=2 ** 26 + 8), UNSUPPORTED),
    (dict(N=64, K=2 ** 31 - 8, H=4096), UNSUPPORTED)], ids=str)
def test_forward_refusals(lib, kw, want):
    assert _fwd(lib, **kw) == want


BWD = dict(act=1, dy=0x1000, x=0x2000, w=0x3000, pre=0x4000, dtype=0, scales=None, N=4, K=64, H=32,
           limit=7.0, alpha=1.702, dx=0x5000, dw=0x6000, ds=0x7000, ws=0x8000, n=1 << 20)


def _bwd(lib, **kw):
    a = {**BWD, **kw}
    n = ctypes.c_size_t(a["n"] or 0)
    st = lib.rn_gated_ffn_bwd(a["act"], P(a["dy"]), P(a["x"]), P(a["w"]), P(a["pre"]), a["dtype"],
                              P(a["scales"]), a["N"], a["K"], a["H"], f32(a["limit"]), f32(a["alpha"]),
                              P(a["dx"]), P(a["dw"]), P(a["ds"]), P(a["ws"]),
                              None if a["n"] is None else ctypes.byref(n), None)
    return st, n.value


@pytest.mark.parametrize("kw,want", [s for s in SHARED if not set(s[0]) & {"out", "mode"}] + [
    (dict(dy=None), INVALID), (dict(pre=None), INVALID), (dict(w=None), INVALID),
    (dict(dy=0x1008), UNSUPPORTED), (dict(w=0x3004), UNSUPPORTED), (dict(pre=0x4002), UNSUPPORTED),
    (dict(dx=0x5008), UNSUPPORTED), (dict(dw=0x6008), UNSUPPORTED), (dict(ds=0x7002), UNSUPPORTED),
    (dict(ws=0x8008), UNSUPPORTED), (dict(K=60), UNSUPPORTED), (dict(H=36), UNSUPPORTED),
    (dict(ws=None), WORKSPACE), (dict(n=None), WORKSPACE), (dict(n=16), WORKSPACE)], ids=str)
def test_backward_refusals(lib, kw, want):
    assert _bwd(lib, **kw)[0] == want


def test_backward_workspace_query(lib):
    none = dict(ws=None, dx=None, dw=None, ds=None, dy=None, x=None, w=None, pre=None)
    st, need = _bwd(lib, **none)
    assert st == 0 and need >= 4 * 64 * 2            # the bf16 gradient of the projections
    assert need == rn.gated_ffn_bwd_workspace_bytes(4, 64, 32)
    assert _bwd(lib, **none, n=None)[0] == INVALID
    assert _bwd(lib, **none, K=60)[0] == UNSUPPORTED
    assert _bwd(lib, n=need - 1)[0] == WORKSPACE
    assert rn.gated_ffn_bwd_workspace_bytes(65536, 64, 65536) >= 2 ** 34  # past 32 bits


@pytest.mark.parametrize("N,K,H", [(733841920, 573239040, 229906560), (880610304, 573239040, 229906560),
                                   (2 ** 31 - 1, 2 ** 31 - 8, 2 ** 30 - 8)])
def test_backward_workspace_query_of_any_size(lib, N, K, H):
    # the product of the sizes passes 64 bits, for the first two to just below zero; asked in a process of its own
    code = f"import mxfp8_quantization_gb300 as rn; print(rn.gated_ffn_bwd_workspace_bytes({N}, {K}, {H}))"
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=ROOT)
    assert r.returncode == 0, r.returncode
    assert int(r.stdout) == (4 * N * H + 255) // 256 * 256      # the bf16 gradient; so many tiles are not split


GATED = dict(act=1, x=0x1000, dtype=0, codes=0x2000, blocks=0x3000, si=0x4000, scales=None, N=4, K=64,
             H=32, limit=7.0, alpha=1.702, mode=0, out=dict(data=0x5000, out_dtype=0))


def _gated(lib, **kw):
    a = {**GATED, **kw}
    o = None if a["out"] is None else ctypes.byref(_out(**a["out"]))
    return lib.rn_nvfp4_gated_ffn(a["act"], P(a["x"]), a["dtype"], P(a["codes"]), P(a["blocks"]), P(a["si"]),
                                  P(a["scales"]), a["N"], a["K"], a["H"], f32(a["limit"]), f32(a["alpha"]),
                                  a["mode"], o, None)


def _mv(lib, **kw):
    a = {**GATED, "y": 0x5000, "odt": 0, **kw}
    return lib.rn_nvfp4_matvec(P(a["x"]), a["dtype"], P(a["codes"]), P(a["blocks"]), P(a["si"]), a["N"],
                               a["K"], a["H"], a["odt"], P(a["y"]), None)


WEIGHTS = [(dict(codes=None), INVALID), (dict(blocks=None), INVALID), (dict(si=None), INVALID),
           (dict(codes=0x2008), UNSUPPORTED), (dict(blocks=0x3008), UNSUPPORTED),
           (dict(si=0x4002), UNSUPPORTED), (dict(K=72), UNSUPPORTED), (dict(K=2 ** 26 + 16), UNSUPPORTED),
           (dict(N=2 ** 20 + 1), UNSUPPORTED)]


@pytest.mark.parametrize("kw,want", SHARED + WEIGHTS, ids=str)
def test_nvfp4_gated_refusals(lib, kw, want):
    assert _gated(lib, **kw) == want


@pytest.mark.parametrize("kw,want", [s for s in SHARED if not set(s[0]) & {"out", "mode", "act", "scales"}]
                         + WEIGHTS + [(dict(y=None), INVALID), (dict(odt=4), INVALID),
                                      (dict(y=0x5008), UNSUPPORTED)], ids=str)
def test_nvfp4_matvec_refusals(lib, kw, want):
    assert _mv(lib, **kw) == want


class Fake:
    """A CUDA tensor's description, on a machine without a GPU."""
    is_cuda = True

    def __init__(self, shape, dtype=torch.bfloat16, contiguous=True, device=0):
        self.shape, self.dtype, self._c = torch.Size(shape), dtype, contiguous
        self.device = torch.device("cuda", device)

    def is_contiguous(self):
        return self._c

    def dim(self):
        return len(self.shape)


@pytest.fixture
def dev0(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)


@pytest.mark.parametrize("kw,match", [
    (dict(act="srelu"), "gated"), (dict(x=Fake((4, 64), torch.float32)), "bfloat16"),
    (dict(x=Fake((64,))), "2 dimensions"), (dict(x=Fake((4, 64), contiguous=False)), "contiguous"),
    (dict(x=Fake((4, 64), device=1)), "current device"), (dict(w=Fake((64, 72))), "shape"),
    (dict(w=Fake((63, 64))), "shape"), (dict(w=Fake((64, 64), torch.float16)), "bfloat16"),
    (dict(scales=Fake((5,), torch.float32)), "shape"), (dict(quant="nvfp4"), "gives"),
    (dict(quant="fp8_current"), "gives")], ids=lambda v: str(v)[:40])
def test_binding_forward_refusals(lib, dev0, kw, match):
    a = {"x": Fake((4, 64)), "w": Fake((64, 64)), **kw}
    with pytest.raises(rn.RNError, match=match):
        rn.gated_ffn_fwd(a.pop("x"), a.pop("w"), **a)


@pytest.mark.parametrize("kw,match", [
    (dict(dy=Fake((4, 33))), "dy"), (dict(pre=Fake((4, 32))), "pre"), (dict(act="relu"), "gated"),
    (dict(workspace=Fake((8,), torch.uint8, contiguous=False)), "workspace")], ids=lambda v: str(v)[:40])
def test_binding_backward_refusals(lib, dev0, kw, match):
    a = {"dy": Fake((4, 32)), "x": Fake((4, 64)), "w": Fake((64, 64)), "pre": Fake((4, 64)), **kw}
    with pytest.raises(rn.RNError, match=match):
        rn.gated_ffn_bwd(a.pop("dy"), a.pop("x"), a.pop("w"), a.pop("pre"), **a)


def _w(R=64, K=64, **kw):
    a = dict(data=Fake((R, K // 2), torch.uint8), row_scales=Fake((R, K // 16), torch.uint8),
             scale_inv=Fake((1,), torch.float32), scale=None, amax=None)
    return rn.NVFP4Output(**{**a, **kw})


@pytest.mark.parametrize("w,match", [
    (_w(K=128), "rows of 64"), (_w(row_scales=Fake((64, 5), torch.uint8)), "row_scales"),
    (_w(scale_inv=Fake((2,), torch.float32)), "scale_inv"), (_w(data=Fake((64, 32))), "uint8")])
def test_binding_nvfp4_refusals(lib, dev0, w, match):
    with pytest.raises(rn.RNError, match=match):
        rn.nvfp4_matvec(Fake((4, 64)), w)
    with pytest.raises(rn.RNError, match=match):
        rn.nvfp4_gated_ffn(Fake((4, 64)), w)


def test_binding_nvfp4_gated_needs_two_halves(lib, dev0):
    with pytest.raises(rn.RNError, match="even"):
        rn.nvfp4_gated_ffn(Fake((4, 64)), _w(R=63))


@pytest.mark.parametrize("name", ["x", "w", "dy", "pre"])
def test_binding_names_a_missing_tensor(lib, dev0, name):
    # pre is None after a forward without save_pre
    a = {"dy": Fake((4, 32)), "x": Fake((4, 64)), "w": Fake((64, 64)), "pre": Fake((4, 64)), name: None}
    with pytest.raises(rn.RNError, match=f"{name} is required"):
        rn.gated_ffn_bwd(a["dy"], a["x"], a["w"], a["pre"])
    if name in ("x", "w"):
        with pytest.raises(rn.RNError, match=f"{name} is required"):
            rn.gated_ffn_fwd(a["x"], a["w"])


@pytest.mark.parametrize("x,w,match", [
    (None, _w(), "x is required"), (Fake((4, 64)), None, "w is required"),
    (Fake((4, 64)), Fake((64, 64)), "NVFP4Output"), (Fake((4, 64)), _w(data=None), "w.data is required"),
    (Fake((4, 64)), _w(row_scales=None), "w.row_scales is required"),
    (Fake((4, 64)), _w(scale_inv=None), "w.scale_inv is required")], ids=lambda v: str(v)[:20])
def test_binding_names_what_is_missing_of_nvfp4_weights(lib, dev0, x, w, match):
    with pytest.raises(rn.RNError, match=match):
        rn.nvfp4_matvec(x, w)
    with pytest.raises(rn.RNError, match=match):
        rn.nvfp4_gated_ffn(x, w)
