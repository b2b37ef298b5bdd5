"""What the state of the host does to a call.  A call that fails on the host
fails alone: the next good one succeeds.  The failure is a launch into a stream whose capture was invalidated (by a
synchronize inside it), which the runtime refuses before anything reaches the
GPU."""
import ctypes
import os
import subprocess
import sys

import pytest
import torch

import mxfp8_quantization_gb300 as rn

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
THREAD_LOCAL, CUDA_ERROR = 1, 4


@pytest.fixture
def driver():
    d = ctypes.CDLL("libcuda.so.1")
    for f in ("cuStreamBeginCapture_v2", "cuStreamEndCapture", "cuStreamSynchronize"):
        getattr(d, f).restype = ctypes.c_int
    return d


def calls():
    """name -> function of a stream handle that makes the C call on tensors of its own."""
    lib = rn._load()
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(40, 64, generator=g, device="cuda").bfloat16()
    w = torch.randn(64, 64, generator=g, device="cuda").bfloat16()
    y, pre = torch.empty(40, 32, device="cuda", dtype=torch.bfloat16), torch.zeros(40, 64, device="cuda").bfloat16()
    dx, dw, ds = torch.empty_like(x), torch.empty_like(w), torch.empty(40, device="cuda")
    n = rn.gated_ffn_bwd_workspace_bytes(40, 64, 32)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    w4 = rn.quantize_only(w.float(), "nvfp4")
    y4 = torch.empty(40, 64, device="cuda", dtype=torch.bfloat16)
    hist, scale, si, am = (torch.ones(k, device="cuda") for k in (4, 1, 1, 1))
    gamma, rs = torch.ones(64, device="cuda"), torch.empty(40, device="cuda")
    o, on = rn._Output(), rn._Output()
    o.data, on.data = y.data_ptr(), dx.data_ptr()
    keep = (x, w, y, pre, dx, dw, ds, ws, w4, y4, hist, scale, si, am, gamma, rs, o, on)
    p = lambda t: ctypes.c_void_p(t.data_ptr())
    size = ctypes.c_size_t(n)
    return keep, {
        "gated_ffn_fwd": lambda s: lib.rn_gated_ffn_fwd(1, p(x), p(w), 0, None, 40, 64, 32, 7.0, 1.702, 0,
                                                        ctypes.byref(o), None, s),
        "gated_ffn_bwd": lambda s: lib.rn_gated_ffn_bwd(1, p(y), p(x), p(w), p(pre), 0, None, 40, 64, 32, 7.0, 1.702,
                                                        p(dx), p(dw), p(ds), p(ws), ctypes.byref(size), s),
        "nvfp4_matvec": lambda s: lib.rn_nvfp4_matvec(p(x), 0, p(w4.data), p(w4.row_scales), p(w4.scale_inv), 40, 64,
                                                      64, 0, p(y4), s),
        "scaled_act_bwd": lambda s: lib.rn_scaled_act_bwd(1, p(y), p(pre), 0, None, 40, 32, 7.0, 1.702, p(y4), p(ds), s),
        "rmsnorm_fwd": lambda s: lib.rn_rmsnorm_fwd(p(x), 0, p(gamma), 40, 64, 1e-5, 0, 0, 0, ctypes.byref(on), p(rs), s),
        "delayed_scaling_update": lambda s: lib.rn_delayed_scaling_update(p(hist), 4, p(am), p(scale), p(si), s),
    }


def test_a_failed_launch_does_not_fail_the_next_call(driver):
    keep, fs = calls()
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    h = ctypes.c_void_p(stream.cuda_stream)
    for name, f in fs.items():
        assert f(h) == 0, name                                   # first use outside the capture
    torch.cuda.synchronize()
    for name, f in fs.items():
        assert driver.cuStreamBeginCapture_v2(h, THREAD_LOCAL) == 0
        assert driver.cuStreamSynchronize(h) != 0                # not allowed in a capture: invalidates it
        assert f(h) == CUDA_ERROR, name
        graph = ctypes.c_void_p()
        assert driver.cuStreamEndCapture(h, ctypes.byref(graph)) != 0
        assert f(h) == 0, name
        torch.cuda.synchronize()
    assert rn.device_error() == 0


FIRST = """
import torch, mxfp8_quantization_gb300 as rn
g = torch.Generator(device="cuda").manual_seed(1)
r = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()
x, w, dy, t = r(300, 264), r(2 * 136, 264) / 16, r(300, 136), r(3, 4112)
w4 = rn.NVFP4Output(torch.randint(0, 256, (64, 2056), generator=g, dtype=torch.uint8, device="cuda"),
                    torch.randint(0x30, 0x41, (64, 257), generator=g, dtype=torch.uint8, device="cuda"),
                    None, torch.ones(1, device="cuda"), None)
def step():
    y, pre = rn.gated_ffn_fwd(x, w, save_pre=True)
    few, _ = rn.gated_ffn_fwd(x[:3], w, quant="fp8_delayed", scale=torch_one)
    return (y, pre, few.data, few.amax, *rn.gated_ffn_bwd(dy, x, w, pre), rn.nvfp4_matvec(t, w4),
            rn.nvfp4_gated_ffn(t, w4))
torch_one = torch.ones(1, device="cuda")
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    out = step()
graph.replay()
want = step()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(out, want))
assert rn.device_error() == 0
print("same")
"""


def test_first_use_inside_a_capture():
    """Nothing that a kernel's first launch sets up (its shared memory, the tensor maps' encoder, the clusters that fit)
    breaks a capture: a process whose first calls are captured."""
    r = subprocess.run([sys.executable, "-c", FIRST], capture_output=True, text=True, cwd=ROOT, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "same", r.stderr[-2000:]
