"""GB300 fused LayerNorm / RMSNorm with FP8, MXFP8 and NVFP4 output.

Thin Python binding over the C ABI in ``include/rn.h`` (``librn.so``, built
in-tree by ``_build.build()``).  This module only marshals arguments: it
allocates outputs with PyTorch, passes raw device pointers and the current
CUDA stream, and raises on a nonzero status.  Every step of the computation
runs in the library's CUDA kernels; there is no fallback.

Entry points mirror the page "Implementation:NVIDIA TransformerEngine
PyTorch Ext Normalization" (section "Signature"):

    layernorm_fwd(x, gamma, beta, eps, quant, sm_margin, zero_centered_gamma)
        -> (output, mu, rsigma)
    rmsnorm_fwd(x, gamma, eps, quant, sm_margin, zero_centered_gamma)
        -> (output, rsigma)
    layernorm_bwd(dz, x, mu, rsigma, gamma, sm_margin, zero_centered_gamma)
        -> (dx, dgamma, dbeta)
    rmsnorm_bwd(dz, x, rsigma, gamma, sm_margin, zero_centered_gamma)
        -> (dx, dgamma)

``quant`` is one of "none", "fp8_delayed" (needs ``scale``), "fp8_current",
"mxfp8", "nvfp4"; the page's quantizer object becomes this string plus the
scale.  ``scaled_act_fwd`` / ``scaled_act_bwd`` are the scaled SReLU, SwiGLU
and clamped SwiGLU of the page "Activation + GroupedLinear Fusion for MOE
and other MOE optimizations"; ``gated_ffn_fwd`` / ``gated_ffn_bwd`` are the
gated feed-forward block around them (both projections, the activation and
the product), ``nvfp4_matvec`` / ``nvfp4_gated_ffn`` the products of one or a
few tokens with the NVFP4 weights that ``quantize_only`` makes.
``kv_cache_write`` / ``kv_cache_read`` keep keys and values in a paged 8-bit
cache, and ``kv_attention`` is the attention that reads it.
"""
from __future__ import annotations

import ctypes
import functools
import os
from dataclasses import dataclass

import torch

__all__ = [
    "layernorm_fwd", "rmsnorm_fwd", "layernorm_bwd", "rmsnorm_bwd", "quantize_only",
    "layernorm_bwd_noalloc", "layernorm_add_fwd", "rmsnorm_add_fwd", "delayed_scaling_update",
    "bwd_workspace_bytes", "device_error", "Fp8Output", "MXFP8Output", "NVFP4Output", "lib_path",
    "RNError",
    "QUANT_MODES", "ACTS", "scaled_act_fwd", "scaled_act_bwd",
    "gated_ffn_fwd", "gated_ffn_bwd", "gated_ffn_bwd_workspace_bytes", "nvfp4_matvec",
    "nvfp4_gated_ffn",
    "KV_PAGE", "KVCache", "KVSequences", "kv_cache_alloc", "kv_cache_write", "kv_cache_read", "kv_attention",
    "kv_attention_workspace_bytes",
]

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "librn.so")
QUANT_MODES = {"none": 0, "fp8_delayed": 1, "fp8_current": 2, "mxfp8": 3, "nvfp4": 4}
_BF16, _F32 = 0, 1
ACTS = {"srelu": 0, "swiglu": 1, "clamped_swiglu": 2}


class RNError(RuntimeError):
    pass


class _Output(ctypes.Structure):
    _fields_ = [
        ("data", ctypes.c_void_p),
        ("row_scales", ctypes.c_void_p),
        ("col_data", ctypes.c_void_p),
        ("col_scales", ctypes.c_void_p),
        ("scale", ctypes.c_void_p),
        ("scale_out", ctypes.c_void_p),
        ("scale_inv", ctypes.c_void_p),
        ("amax", ctypes.c_void_p),
        ("out_dtype", ctypes.c_int),
    ]


class _KVCache(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("k", "v", "k_scales", "v_scales")] + \
               [(n, ctypes.c_int64) for n in ("pages", "heads", "dim")]


class _KVSeqs(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("table", "starts", "lens")] + \
               [(n, ctypes.c_int64) for n in ("sequences", "table_width", "tokens")]


_lib = None


def lib_path() -> str:
    return _LIB_PATH


def _load():
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_PATH):
        raise RNError(
            f"{_LIB_PATH} is missing: build it first (mxfp8_quantization_gb300._build.build())")
    lib = ctypes.CDLL(_LIB_PATH)
    vp, i64, i32, f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float
    outp = ctypes.POINTER(_Output)
    szp = ctypes.POINTER(ctypes.c_size_t)
    lib.rn_layernorm_fwd.argtypes = [vp, i32, vp, vp, i64, i64, f32, i32, i32, i32, outp, vp, vp, vp]
    lib.rn_rmsnorm_fwd.argtypes = [vp, i32, vp, i64, i64, f32, i32, i32, i32, outp, vp, vp]
    lib.rn_layernorm_bwd.argtypes = [vp, vp, i32, vp, vp, vp, i64, i64, i32, i32, vp, vp, vp, vp, szp, vp]
    lib.rn_rmsnorm_bwd.argtypes = [vp, vp, i32, vp, vp, i64, i64, i32, i32, vp, vp, vp, szp, vp]
    lib.rn_layernorm_add_fwd.argtypes = [vp, vp, i32, vp, vp, i64, i64, f32, i32, i32, i32, outp,
                                         vp, vp, vp, vp]
    lib.rn_rmsnorm_add_fwd.argtypes = [vp, vp, i32, vp, i64, i64, f32, i32, i32, i32, outp, vp, vp,
                                       vp]
    lib.rn_quantize_only.argtypes = [vp, i64, i64, i32, outp, vp]
    lib.rn_delayed_scaling_update.argtypes = [vp, i64, vp, vp, vp, vp]
    lib.rn_scaled_act_fwd.argtypes = [i32, vp, i32, vp, i64, i64, f32, f32, i32, outp, vp]
    lib.rn_scaled_act_bwd.argtypes = [i32, vp, vp, i32, vp, i64, i64, f32, f32, vp, vp, vp]
    lib.rn_layernorm_bwd_noalloc.argtypes = [vp, vp, i32, vp, vp, vp, i64, i64, i32, i32, vp, vp, vp, vp]
    lib.rn_gated_ffn_fwd.argtypes = [i32, vp, vp, i32, vp, i64, i64, i64, f32, f32, i32, outp, vp, vp]
    lib.rn_gated_ffn_bwd.argtypes = [i32, vp, vp, vp, vp, i32, vp, i64, i64, i64, f32, f32, vp, vp, vp,
                                     vp, szp, vp]
    lib.rn_nvfp4_matvec.argtypes = [vp, i32, vp, vp, vp, i64, i64, i64, i32, vp, vp]
    lib.rn_nvfp4_gated_ffn.argtypes = [i32, vp, i32, vp, vp, vp, vp, i64, i64, i64, f32, f32, i32,
                                       outp, vp]
    cachep, seqsp = ctypes.POINTER(_KVCache), ctypes.POINTER(_KVSeqs)
    lib.rn_kv_cache_write.argtypes = [vp, vp, i32, i64, i64, cachep, seqsp, vp]
    lib.rn_kv_cache_read.argtypes = [cachep, seqsp, vp, vp, i32, vp]
    lib.rn_kv_attention.argtypes = [vp, i32, i64, i64, cachep, seqsp, f32, i32, i64, f32, vp, vp, vp, vp, szp, vp]
    lib.rn_device_error.argtypes = [ctypes.POINTER(ctypes.c_uint)]
    lib.rn_status_str.argtypes = [i32]
    lib.rn_status_str.restype = ctypes.c_char_p
    for f in ("rn_layernorm_fwd", "rn_rmsnorm_fwd", "rn_layernorm_bwd", "rn_rmsnorm_bwd",
              "rn_quantize_only", "rn_device_error", "rn_abi_version", "rn_layernorm_bwd_noalloc",
              "rn_layernorm_add_fwd", "rn_rmsnorm_add_fwd", "rn_delayed_scaling_update",
              "rn_scaled_act_fwd", "rn_scaled_act_bwd", "rn_gated_ffn_fwd", "rn_gated_ffn_bwd",
              "rn_nvfp4_matvec", "rn_nvfp4_gated_ffn", "rn_kv_cache_write", "rn_kv_cache_read",
              "rn_kv_attention"):
        getattr(lib, f).restype = ctypes.c_int
    _lib = lib
    return lib


def _check(status: int, what: str):
    if status != 0:
        msg = _load().rn_status_str(status).decode()
        raise RNError(f"{what}: status {status} ({msg})")


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


# the current stream's handle without the Stream object around it (3 us of a
# small call)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda dev: torch.cuda.current_stream(dev).cuda_stream)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return _BF16
    if t.dtype == torch.float32:
        return _F32
    raise RNError(f"unsupported dtype {t.dtype}: x must be bfloat16 or float32")


def _need(t, name, dtype=None, shape=None):
    if t is None:
        raise RNError(f"{name} is required")
    if not t.is_cuda or not t.is_contiguous():
        raise RNError(f"{name} must be a contiguous CUDA tensor")
    # the library launches on the current device (and picks its per-device
    # state by it): a tensor on another device would be read through the
    # wrong device's pointers
    if t.device.index != torch.cuda.current_device():
        raise RNError(f"{name} is on {t.device}, but the current device is "
                      f"cuda:{torch.cuda.current_device()}")
    if dtype is not None and t.dtype != dtype:
        raise RNError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise RNError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    return t


@dataclass
class Fp8Output:
    """E4M3 codes with their per-tensor scale (FP8_DELAYED / FP8_CURRENT)."""
    data: torch.Tensor       # uint8 [N, H]
    scale_inv: torch.Tensor  # fp32 [1]
    amax: torch.Tensor       # fp32 [1]
    scale: torch.Tensor      # fp32 [1] (given for delayed, computed for current)


@dataclass
class MXFP8Output:
    """MXFP8: rowwise 1x32 and columnwise 32x1 blocks with E8M0 scales."""
    data: torch.Tensor | None        # uint8 [N, H]
    row_scales: torch.Tensor | None  # uint8 [N, H/32]
    col_data: torch.Tensor | None    # uint8 [H, N] (transposed)
    col_scales: torch.Tensor | None  # uint8 [H, N/32]


@dataclass
class NVFP4Output:
    """NVFP4: E2M1 codes with an E4M3 scale per 1x16 block and a tensor scale."""
    data: torch.Tensor        # uint8 [N, H/2], two codes per byte (even element low)
    row_scales: torch.Tensor  # uint8 [N, H/16] E4M3 block-scale codes
    scale: torch.Tensor       # fp32 [1] S = 448 * 6 / amax
    scale_inv: torch.Tensor   # fp32 [1] 1 / S
    amax: torch.Tensor        # fp32 [1]


def _make_output(x, quant, out_dtype, scale, rowwise=True, colwise=True):
    N, H = x.shape
    dev = x.device
    o = _Output()
    if quant == "none":
        odt = x.dtype if out_dtype is None else out_dtype
        data = torch.empty((N, H), dtype=odt, device=dev)
        o.data = data.data_ptr()
        o.out_dtype = _dtype_code(data)
        return o, data
    if quant in ("fp8_delayed", "fp8_current"):
        data = torch.empty((N, H), dtype=torch.uint8, device=dev)
        res = Fp8Output(data, torch.empty(1, dtype=torch.float32, device=dev),
                        torch.empty(1, dtype=torch.float32, device=dev), None)
        o.data = data.data_ptr()
        o.scale_inv = res.scale_inv.data_ptr()
        o.amax = res.amax.data_ptr()
        if quant == "fp8_delayed":
            if scale is None:
                raise RNError("fp8_delayed needs scale")
            s = scale if isinstance(scale, torch.Tensor) else torch.tensor([float(scale)], dtype=torch.float32)
            if not (s.dtype is torch.float32 and s.shape == (1,) and s.device == dev):
                s = s.to(device=dev, dtype=torch.float32).reshape(1).contiguous()
            res.scale = s
            o.scale = s.data_ptr()
        else:
            res.scale = torch.empty(1, dtype=torch.float32, device=dev)
            o.scale_out = res.scale.data_ptr()
        return o, res
    if quant == "mxfp8":
        res = MXFP8Output(None, None, None, None)
        if rowwise:
            res.data = torch.empty((N, H), dtype=torch.uint8, device=dev)
            res.row_scales = torch.empty((N, H // 32), dtype=torch.uint8, device=dev)
            o.data = res.data.data_ptr()
            o.row_scales = res.row_scales.data_ptr()
        if colwise:
            res.col_data = torch.empty((H, N), dtype=torch.uint8, device=dev)
            res.col_scales = torch.empty((H, N // 32), dtype=torch.uint8, device=dev)
            o.col_data = res.col_data.data_ptr()
            o.col_scales = res.col_scales.data_ptr()
        return o, res
    if quant == "nvfp4":
        f32 = dict(dtype=torch.float32, device=dev)
        res = NVFP4Output(torch.empty((N, H // 2), dtype=torch.uint8, device=dev),
                          torch.empty((N, H // 16), dtype=torch.uint8, device=dev),
                          torch.empty(1, **f32), torch.empty(1, **f32), torch.empty(1, **f32))
        o.data = res.data.data_ptr()
        o.row_scales = res.row_scales.data_ptr()
        o.scale_out = res.scale.data_ptr()
        o.scale_inv = res.scale_inv.data_ptr()
        o.amax = res.amax.data_ptr()
        return o, res
    raise RNError(f"unknown quant mode {quant!r}")


def layernorm_fwd(x, gamma, beta, eps, quant="none", sm_margin=0, zero_centered_gamma=False,
                  scale=None, out_dtype=None, rowwise=True, colwise=True):
    """LayerNorm forward -> (output, mu, rsigma); output per ``quant``."""
    lib = _load()
    _need(x, "x")
    N, H = x.shape
    _need(gamma, "gamma", torch.float32, (H,))
    if beta is not None:
        _need(beta, "beta", torch.float32, (H,))
    mu = torch.empty(N, dtype=torch.float32, device=x.device)
    rsigma = torch.empty(N, dtype=torch.float32, device=x.device)
    o, res = _make_output(x, quant, out_dtype, scale, rowwise, colwise)
    st = lib.rn_layernorm_fwd(_ptr(x), _dtype_code(x), _ptr(gamma), _ptr(beta), N, H, float(eps),
                              int(bool(zero_centered_gamma)), int(sm_margin), QUANT_MODES[quant],
                              ctypes.byref(o), _ptr(mu), _ptr(rsigma), _stream())
    _check(st, "rn_layernorm_fwd")
    return res, mu, rsigma


def rmsnorm_fwd(x, gamma, eps, quant="none", sm_margin=0, zero_centered_gamma=False, scale=None,
                out_dtype=None, rowwise=True, colwise=True):
    """RMSNorm forward -> (output, rsigma); output per ``quant``."""
    lib = _load()
    _need(x, "x")
    N, H = x.shape
    _need(gamma, "gamma", torch.float32, (H,))
    rsigma = torch.empty(N, dtype=torch.float32, device=x.device)
    o, res = _make_output(x, quant, out_dtype, scale, rowwise, colwise)
    st = lib.rn_rmsnorm_fwd(_ptr(x), _dtype_code(x), _ptr(gamma), N, H, float(eps),
                            int(bool(zero_centered_gamma)), int(sm_margin), QUANT_MODES[quant],
                            ctypes.byref(o), _ptr(rsigma), _stream())
    _check(st, "rn_rmsnorm_fwd")
    return res, rsigma


def layernorm_add_fwd(x, residual, gamma, beta, eps, quant="none", sm_margin=0,
                      zero_centered_gamma=False, scale=None, out_dtype=None, rowwise=True,
                      colwise=True):
    """h = x + residual (rounded to x's dtype), LayerNorm(h) -> (output, h, mu, rsigma);
    output per ``quant`` (MXFP8: the blocks ``rowwise`` / ``colwise`` select)."""
    lib = _load()
    _need(x, "x")
    N, H = x.shape
    _need(residual, "residual", x.dtype, (N, H))
    _need(gamma, "gamma", torch.float32, (H,))
    if beta is not None:
        _need(beta, "beta", torch.float32, (H,))
    h = torch.empty_like(x)
    mu = torch.empty(N, dtype=torch.float32, device=x.device)
    rsigma = torch.empty(N, dtype=torch.float32, device=x.device)
    o, res = _make_output(x, quant, out_dtype, scale, rowwise, colwise)
    st = lib.rn_layernorm_add_fwd(_ptr(x), _ptr(residual), _dtype_code(x), _ptr(gamma), _ptr(beta),
                                  N, H, float(eps), int(bool(zero_centered_gamma)), int(sm_margin),
                                  QUANT_MODES[quant], ctypes.byref(o), _ptr(h), _ptr(mu),
                                  _ptr(rsigma), _stream())
    _check(st, "rn_layernorm_add_fwd")
    return res, h, mu, rsigma


def rmsnorm_add_fwd(x, residual, gamma, eps, quant="none", sm_margin=0,
                    zero_centered_gamma=False, scale=None, out_dtype=None, rowwise=True,
                    colwise=True):
    """h = x + residual (rounded to x's dtype), RMSNorm(h) -> (output, h, rsigma); output per
    ``quant`` (MXFP8: the blocks ``rowwise`` / ``colwise`` select)."""
    lib = _load()
    _need(x, "x")
    N, H = x.shape
    _need(residual, "residual", x.dtype, (N, H))
    _need(gamma, "gamma", torch.float32, (H,))
    h = torch.empty_like(x)
    rsigma = torch.empty(N, dtype=torch.float32, device=x.device)
    o, res = _make_output(x, quant, out_dtype, scale, rowwise, colwise)
    st = lib.rn_rmsnorm_add_fwd(_ptr(x), _ptr(residual), _dtype_code(x), _ptr(gamma), N, H,
                                float(eps), int(bool(zero_centered_gamma)), int(sm_margin),
                                QUANT_MODES[quant], ctypes.byref(o), _ptr(h), _ptr(rsigma),
                                _stream())
    _check(st, "rn_rmsnorm_add_fwd")
    return res, h, rsigma


def delayed_scaling_update(amax_history, amax, scale):
    """One delayed-scaling step on device tensors: shifts `amax` (fp32 [1])
    into `amax_history` (fp32 [L], most recent first) and updates `scale`
    (fp32 [1]) in place; returns scale_inv (fp32 [1])."""
    lib = _load()
    _need(amax_history, "amax_history", torch.float32)
    _need(amax, "amax", torch.float32, (1,))
    _need(scale, "scale", torch.float32, (1,))
    scale_inv = torch.empty(1, dtype=torch.float32, device=scale.device)
    st = lib.rn_delayed_scaling_update(_ptr(amax_history), amax_history.numel(), _ptr(amax),
                                       _ptr(scale), _ptr(scale_inv), _stream())
    _check(st, "rn_delayed_scaling_update")
    return scale_inv


def _act_width(x, act):
    if act not in ACTS:
        raise RNError(f"unknown activation {act!r}")
    return x.shape[1] if act == "srelu" else x.shape[1] // 2


def scaled_act_fwd(x, act, scales=None, quant="none", limit=7.0, alpha=1.702, scale=None,
                   out_dtype=None):
    """y = scales[:, None] * act(x): x [N, H] (srelu) or [N, 2H] (swiglu,
    clamped_swiglu: gate half, then linear half); returns the output in the
    form of the forward norm calls (MXFP8: rowwise blocks only)."""
    lib = _load()
    _need(x, "x")
    N, H = x.shape[0], _act_width(x, act)
    if scales is not None:
        _need(scales, "scales", torch.float32, (N,))
    o, res = _make_output(x[:, :H], quant, out_dtype, scale, True, False)
    st = lib.rn_scaled_act_fwd(ACTS[act], _ptr(x), _dtype_code(x), _ptr(scales), N, H,
                               float(limit), float(alpha), QUANT_MODES[quant], ctypes.byref(o),
                               _stream())
    _check(st, "rn_scaled_act_fwd")
    return res


def scaled_act_bwd(dy, x, act, scales=None, limit=7.0, alpha=1.702, dscales=True):
    """-> (dx shaped like x, dscales fp32 [N] or None)."""
    lib = _load()
    _need(x, "x")
    N, H = x.shape[0], _act_width(x, act)
    _need(dy, "dy", x.dtype, (N, H))
    if scales is not None:
        _need(scales, "scales", torch.float32, (N,))
    dx = torch.empty_like(x)
    ds = torch.empty(N, dtype=torch.float32, device=x.device) if dscales else None
    st = lib.rn_scaled_act_bwd(ACTS[act], _ptr(dy), _ptr(x), _dtype_code(x), _ptr(scales), N, H,
                               float(limit), float(alpha), _ptr(dx), _ptr(ds), _stream())
    _check(st, "rn_scaled_act_bwd")
    return dx, ds


def _gated(act):
    if act not in ("swiglu", "clamped_swiglu"):
        raise RNError(f"a gated block takes 'swiglu' or 'clamped_swiglu', got {act!r}")
    return ACTS[act]


# Small calls spend more time in these checks than on the device, so each entry
# point asks for everything at once and goes through the refusals one by one
# only when something is amiss.
_BF, _U8, _FP32 = torch.bfloat16, torch.uint8, torch.float32


def _matrix(t, name, dtype):
    _need(t, name, dtype)
    if t.dim() != 2:
        raise RNError(f"{name} must have 2 dimensions, got {t.dim()}")
    return t.shape


def _refuse_block(x, w, **more):
    """The refusal of a block's tensors; ``more``: name=(tensor, dtype, shape from N and H)."""
    N, K = _matrix(x, "x", _BF)
    R = _matrix(w, "w", _BF)[0]
    if R % 2 or w.shape[1] != K:
        raise RNError(f"w must have shape (2 H, {K}), got {tuple(w.shape)}")
    for name, (t, dtype, shape) in more.items():
        if t is not None or name != "scales":
            _need(t, name, dtype, shape(N, R // 2))
    raise RNError("unsupported tensors")


def _refuse_nvfp4(x, w, scales, halves):
    N, K = _matrix(x, "x", _BF)
    if w is None:
        raise RNError("w is required")
    if not hasattr(w, "row_scales"):
        raise RNError(f"w must be an NVFP4Output, got {type(w).__name__}")
    R, half = _matrix(w.data, "w.data", _U8)
    if K % 16 or half * 2 != K:
        raise RNError(f"w must hold rows of {K} elements (a multiple of 16), got {2 * half}")
    _need(w.row_scales, "w.row_scales", _U8, (R, K // 16))
    _need(w.scale_inv, "w.scale_inv", _FP32, (1,))
    if halves and R % 2:
        raise RNError(f"w must have an even number of rows, got {R}")
    if scales is not None:
        _need(scales, "scales", _FP32, (N,))
    raise RNError("unsupported tensors")


def _addr(t):
    return None if t is None else t.data_ptr()


@dataclass
class _Like:
    """What ``_make_output`` reads of the tensor it makes an output for."""
    shape: tuple
    dtype: torch.dtype
    device: torch.device


def _make_rows_output(x, N, H, quant, out_dtype, scale):
    """The output of a block with rows of H: ``x`` gives the device and the default dtype."""
    if quant == "none":
        o = _Output()
        data = torch.empty((N, H), dtype=out_dtype or x.dtype, device=x.device)
        o.data = data.data_ptr()
        o.out_dtype = _dtype_code(data)
        return o, data
    if quant not in ("fp8_delayed", "mxfp8"):
        raise RNError(f"a gated block gives 'none', 'fp8_delayed' or 'mxfp8' output, got {quant!r}")
    return _make_output(_Like((N, H), x.dtype, x.device), quant, out_dtype, scale, True, False)


def _scales_ok(scales, N, dev):
    return scales is None or (scales.dtype is _FP32 and scales.shape == (N,) and scales.is_contiguous()
                              and scales.device.index == dev)


# a tensor that is missing (None) is refused by its name, like any other
def _block_ok(x, w, dev):
    try:
        return (x.dtype is _BF and w.dtype is _BF and x.dim() == 2 and w.dim() == 2 and w.shape[1] == x.shape[1]
                and w.shape[0] % 2 == 0 and x.is_contiguous() and w.is_contiguous() and x.device.index == dev
                and w.device.index == dev and x.is_cuda and w.is_cuda)
    except AttributeError:
        return False


def _grads_ok(dy, pre, x, w, dev):
    try:
        return (dy.dtype is _BF and pre.dtype is _BF and dy.shape == (x.shape[0], w.shape[0] // 2)
                and pre.shape == (x.shape[0], w.shape[0]) and dy.is_contiguous() and pre.is_contiguous()
                and dy.device.index == dev and pre.device.index == dev)
    except AttributeError:
        return False


def _nvfp4_ok(x, w, dev):
    try:
        d, b, si = w.data, w.row_scales, w.scale_inv
        if not (x.dtype is _BF and d.dtype is _U8 and b.dtype is _U8 and si.dtype is _FP32 and x.dim() == 2
                and d.dim() == 2):
            return False
        K, R = x.shape[1], d.shape[0]
        return (K % 16 == 0 and d.shape[1] * 2 == K and b.shape == (R, K // 16) and si.shape == (1,)
                and x.is_contiguous() and d.is_contiguous() and b.is_contiguous() and si.is_contiguous()
                and x.device.index == dev and d.device.index == dev and b.device.index == dev
                and si.device.index == dev and x.is_cuda)
    except AttributeError:
        return False


def gated_ffn_fwd(x, w, act="swiglu", scales=None, quant="none", limit=7.0, alpha=1.702, scale=None,
                  out_dtype=None, save_pre=False):
    """y = scales[:, None] * act(x @ w[:H].T, x @ w[H:].T): x bf16 [N, K], w bf16 [2H, K] (gate rows,
    then linear rows), act "swiglu" or "clamped_swiglu" -> (output, pre); output per ``quant``
    ("none", "fp8_delayed", "mxfp8" rowwise), pre the projections bf16 [N, 2H] for
    ``gated_ffn_bwd``, or None without ``save_pre``."""
    lib = _lib or _load()
    code = _gated(act)
    dev = torch.cuda.current_device()
    if not (_block_ok(x, w, dev) and _scales_ok(scales, x.shape[0], dev)):
        _refuse_block(x, w, scales=(scales, _FP32, lambda n, h: (n,)))
    N, K = x.shape
    R = w.shape[0]
    H = R // 2
    o, res = _make_rows_output(x, N, H, quant, out_dtype, scale)
    pre = torch.empty((N, R), dtype=x.dtype, device=x.device) if save_pre else None
    st = lib.rn_gated_ffn_fwd(code, x.data_ptr(), w.data_ptr(), _BF16, _addr(scales), N, K, H, float(limit),
                              float(alpha), QUANT_MODES[quant], ctypes.byref(o), _addr(pre), _raw_stream(dev))
    if st:
        _check(st, "rn_gated_ffn_fwd")
    return res, pre


@functools.lru_cache(maxsize=256)
def gated_ffn_bwd_workspace_bytes(N, K, H) -> int:
    """Workspace bytes ``gated_ffn_bwd`` needs (the query step of the protocol)."""
    n = ctypes.c_size_t(0)
    st = _load().rn_gated_ffn_bwd(ACTS["swiglu"], None, None, None, None, _BF16, None, N, K, H, 0.0, 0.0,
                                  None, None, None, None, ctypes.byref(n), None)
    _check(st, "workspace query")
    return int(n.value)


def gated_ffn_bwd(dy, x, w, pre, act="swiglu", scales=None, limit=7.0, alpha=1.702, dscales=True,
                  workspace=None, need_dx=True, need_dw=True):
    """Backward of ``gated_ffn_fwd`` at its ``pre``: dy bf16 [N, H] -> (dx bf16 [N, K] or None, dw
    bf16 [2H, K] or None, dscales fp32 [N] or None); ``need_dx`` / ``need_dw`` / ``dscales`` select."""
    lib = _lib or _load()
    code = _gated(act)
    dev = torch.cuda.current_device()
    if not (_block_ok(x, w, dev) and _scales_ok(scales, x.shape[0], dev) and _grads_ok(dy, pre, x, w, dev)):
        _refuse_block(x, w, dy=(dy, _BF, lambda n, h: (n, h)), pre=(pre, _BF, lambda n, h: (n, 2 * h)),
                      scales=(scales, _FP32, lambda n, h: (n,)))
    N, K = x.shape
    R = w.shape[0]
    H = R // 2
    if not (need_dx or need_dw or dscales):
        raise RNError("nothing to compute: dx, dw and dscales are all skipped")
    if workspace is None:
        workspace = torch.empty(max(gated_ffn_bwd_workspace_bytes(N, K, H), 16), dtype=torch.uint8,
                                device=x.device)
    else:
        _need(workspace, "workspace")
    n = ctypes.c_size_t(workspace.numel() * workspace.element_size())
    dx = torch.empty((N, K), dtype=x.dtype, device=x.device) if need_dx else None
    dw = torch.empty((R, K), dtype=x.dtype, device=x.device) if need_dw else None
    ds = torch.empty(N, dtype=torch.float32, device=x.device) if dscales else None
    st = lib.rn_gated_ffn_bwd(code, dy.data_ptr(), x.data_ptr(), w.data_ptr(), pre.data_ptr(), _BF16,
                              _addr(scales), N, K, H, float(limit), float(alpha), _addr(dx), _addr(dw), _addr(ds),
                              workspace.data_ptr(), ctypes.byref(n), _raw_stream(dev))
    if st:
        _check(st, "rn_gated_ffn_bwd")
    return dx, dw, ds


def nvfp4_matvec(x, w, out_dtype=None):
    """y = x @ W.T for one or a few tokens: x bf16 [N, K], w the ``NVFP4Output`` of a weight matrix
    [R, K] -> y [N, R] in ``out_dtype`` (x's by default, or float32)."""
    lib = _lib or _load()
    dev = torch.cuda.current_device()
    if not _nvfp4_ok(x, w, dev):
        _refuse_nvfp4(x, w, None, False)
    N, K = x.shape
    R = w.data.shape[0]
    y = torch.empty((N, R), dtype=x.dtype if out_dtype is None else out_dtype, device=x.device)
    st = lib.rn_nvfp4_matvec(x.data_ptr(), _BF16, w.data.data_ptr(), w.row_scales.data_ptr(),
                             w.scale_inv.data_ptr(), N, K, R, _dtype_code(y), y.data_ptr(),
                             _raw_stream(dev))
    if st:
        _check(st, "rn_nvfp4_matvec")
    return y


def nvfp4_gated_ffn(x, w, act="swiglu", scales=None, quant="none", limit=7.0, alpha=1.702, scale=None,
                    out_dtype=None):
    """``gated_ffn_fwd`` for one or a few tokens with NVFP4 weights: w the ``NVFP4Output`` of a
    weight matrix [2H, K] (gate rows, then linear rows) -> output per ``quant``."""
    lib = _lib or _load()
    code = _gated(act)
    dev = torch.cuda.current_device()
    if not (_nvfp4_ok(x, w, dev) and w.data.shape[0] % 2 == 0 and _scales_ok(scales, x.shape[0], dev)):
        _refuse_nvfp4(x, w, scales, True)
    N, K = x.shape
    R = w.data.shape[0]
    o, res = _make_rows_output(x, N, R // 2, quant, out_dtype, scale)
    st = lib.rn_nvfp4_gated_ffn(code, x.data_ptr(), _BF16, w.data.data_ptr(),
                                w.row_scales.data_ptr(), w.scale_inv.data_ptr(), _addr(scales), N, K,
                                R // 2, float(limit), float(alpha), QUANT_MODES[quant], ctypes.byref(o),
                                _raw_stream(dev))
    if st:
        _check(st, "rn_nvfp4_gated_ffn")
    return res


KV_PAGE = 64   # positions of a page of the key/value cache
_I32 = torch.int32


@dataclass
class KVCache:
    """A paged 8-bit key/value cache (``kv_cache_alloc``): an element stands for its code's value times
    2 ** (scale - 127) of its page and head (scales below 7 count as 7, above 246 as 246)."""
    k: torch.Tensor         # uint8 E4M3 [pages, heads, 64, dim]
    v: torch.Tensor         # uint8 E4M3 [pages, heads, dim, 64] (transposed)
    k_scales: torch.Tensor  # uint8 E8M0 [pages, heads]
    v_scales: torch.Tensor


@dataclass
class KVSequences:
    """The sequences of a call, on the device: rows starts[b] .. starts[b + 1] - 1 of the call's row
    tensors are the last of the lens[b] positions of sequence b, whose block of 64 positions i stands in
    page table[b, i] (none where that number is not a page)."""
    table: torch.Tensor   # int32 [sequences, width]
    starts: torch.Tensor  # int32 [sequences + 1]
    lens: torch.Tensor    # int32 [sequences]


def kv_cache_alloc(pages, heads, dim, device=None) -> KVCache:
    """A zeroed cache of ``pages`` pages of 64 positions."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else device
    zeros = functools.partial(torch.zeros, dtype=torch.uint8, device=dev)
    return KVCache(zeros((pages, heads, KV_PAGE, dim)), zeros((pages, heads, dim, KV_PAGE)), zeros((pages, heads)),
                   zeros((pages, heads)))


def _refuse_kv(cache, seqs):
    if not hasattr(cache, "k_scales"):
        raise RNError(f"cache must be a KVCache, got {type(cache).__name__}")
    if not hasattr(seqs, "starts"):
        raise RNError(f"seqs must be KVSequences, got {type(seqs).__name__}")
    _need(cache.k, "cache.k", _U8)
    if cache.k.dim() != 4 or cache.k.shape[2] != KV_PAGE:
        raise RNError(f"cache.k must have shape (pages, heads, {KV_PAGE}, dim), got {tuple(cache.k.shape)}")
    P, H, _, D = cache.k.shape
    _need(cache.v, "cache.v", _U8, (P, H, D, KV_PAGE))
    _need(cache.k_scales, "cache.k_scales", _U8, (P, H))
    _need(cache.v_scales, "cache.v_scales", _U8, (P, H))
    B = _matrix(seqs.table, "seqs.table", _I32)[0]
    _need(seqs.starts, "seqs.starts", _I32, (B + 1,))
    _need(seqs.lens, "seqs.lens", _I32, (B,))
    raise RNError("unsupported tensors")


def _kv_args(cache, seqs, tokens, dev):
    """The C structures of a cache and of a call's sequences."""
    try:
        k, v, ks, vs = cache.k, cache.v, cache.k_scales, cache.v_scales
        tb, st, ln = seqs.table, seqs.starts, seqs.lens
        P, H, n, D = k.shape
        B, width = tb.shape
        if (n == KV_PAGE and v.shape == (P, H, D, KV_PAGE) and ks.shape == (P, H) and vs.shape == (P, H)
                and st.shape == (B + 1,) and ln.shape == (B,) and k.dtype is _U8 and v.dtype is _U8
                and ks.dtype is _U8 and vs.dtype is _U8 and tb.dtype is _I32 and st.dtype is _I32
                and ln.dtype is _I32 and k.is_contiguous() and v.is_contiguous() and ks.is_contiguous()
                and vs.is_contiguous() and tb.is_contiguous() and st.is_contiguous() and ln.is_contiguous()
                and k.is_cuda and k.device.index == dev and v.device.index == dev and ks.device.index == dev
                and vs.device.index == dev and tb.device.index == dev and st.device.index == dev
                and ln.device.index == dev):
            return (_KVCache(k.data_ptr(), v.data_ptr(), ks.data_ptr(), vs.data_ptr(), P, H, D),
                    _KVSeqs(tb.data_ptr(), st.data_ptr(), ln.data_ptr(), B, width, tokens))
    except (AttributeError, ValueError):
        pass
    _refuse_kv(cache, seqs)


def _kv_rows(t, name, heads, dim, dev, dtypes):
    """The distance of the rows of t [tokens, heads, dim], whose heads and dims are contiguous, and their number."""
    try:
        T, h, d = t.shape
        row, hs, ds = t.stride()
        if (h == heads and d == dim and t.dtype in dtypes and t.is_cuda and t.device.index == dev
                and (ds == 1 and (h == 1 or hs == d) or T == 0)):
            return row if T > 1 else h * d, T
    except (AttributeError, ValueError, TypeError):
        pass
    if t is None:
        raise RNError(f"{name} is required")
    if not getattr(t, "is_cuda", False):
        raise RNError(f"{name} must be a CUDA tensor")
    if t.device.index != dev:
        raise RNError(f"{name} is on {t.device}, but the current device is cuda:{dev}")
    if t.dtype not in dtypes:
        raise RNError(f"{name} must be {' or '.join(map(str, dtypes))}, got {t.dtype}")
    if t.dim() != 3 or t.shape[1:] != (heads, dim):
        raise RNError(f"{name} must have shape (tokens, {heads}, {dim}), got {tuple(t.shape)}")
    raise RNError(f"the heads and dims of {name} must be contiguous (its rows may lie apart)")


def kv_cache_write(cache, seqs, k, v):
    """Quantizes the new rows k, v [tokens, heads, dim] (bf16 or fp32; their rows may lie apart, as in a
    slice of a joint projection) into the pages of their sequences, in place."""
    lib = _lib or _load()
    dev = torch.cuda.current_device()
    c, q = _kv_args(cache, seqs, 0, dev)
    heads, dim = c.heads, c.dim
    ks, T = _kv_rows(k, "k", heads, dim, dev, (_BF, _FP32))
    vs, vT = _kv_rows(v, "v", heads, dim, dev, (k.dtype,))
    q.tokens = T
    if vT != T:
        raise RNError(f"v must have shape {tuple(k.shape)}, got {tuple(v.shape)}")
    st = lib.rn_kv_cache_write(k.data_ptr(), v.data_ptr(), _BF16 if k.dtype is _BF else _F32, ks, vs, c, q,
                               _raw_stream(dev))
    if st:
        _check(st, "rn_kv_cache_write")


def kv_cache_read(cache, seqs, tokens, out_dtype=torch.bfloat16):
    """The last positions of each sequence (as many as it has rows) -> (k, v) [tokens, heads, dim] in
    bfloat16 or float32, both exact.  Rows outside every sequence are left uninitialized."""
    lib = _lib or _load()
    dev = torch.cuda.current_device()
    if tokens < 0:
        raise RNError(f"tokens must not be negative, got {tokens}")
    if tokens >= 1 << 30:
        raise RNError(f"tokens must be below 2**30, got {tokens}")
    c, q = _kv_args(cache, seqs, int(tokens), dev)
    shape = (q.tokens, c.heads, c.dim)
    k = torch.empty(shape, dtype=out_dtype, device=cache.k.device)
    v = torch.empty(shape, dtype=out_dtype, device=cache.k.device)
    st = lib.rn_kv_cache_read(c, q, k.data_ptr(), v.data_ptr(), _dtype_code(k), _raw_stream(dev))
    if st:
        _check(st, "rn_kv_cache_read")
    return k, v


@functools.lru_cache(maxsize=64)
def _kv_attention_bytes(tokens, q_heads, sequences, heads, dim):
    c = _KVCache(16, 16, 16, 16, 1, heads, dim)
    q = _KVSeqs(16, 16, 16, sequences, 1, tokens)
    n = ctypes.c_size_t(0)
    st = _load().rn_kv_attention(None, _BF16, 0, q_heads, c, q, 1.0, 1, 0, 0.0, None, None, None, None,
                                 ctypes.byref(n), None)
    _check(st, "workspace query")
    return int(n.value)


def kv_attention_workspace_bytes(tokens, q_heads, sequences, heads, dim) -> int:
    """Workspace bytes ``kv_attention`` needs (the query step of the protocol)."""
    return _kv_attention_bytes(int(tokens), int(q_heads), int(sequences), int(heads), int(dim))


def kv_attention(q, cache, seqs, scale=None, causal=True, window=0, softcap=0.0, slopes=None, return_lse=False,
                 workspace=None):
    """Attention of the queries q bf16 [tokens, q_heads, dim] (rows may lie apart) with the cached positions
    of their sequences -> out bf16 [tokens, q_heads, dim], or (out, lse fp32 [tokens, q_heads]) with
    ``return_lse``.  ``scale``: 1 / sqrt(dim) by default; ``causal``: positions up to the query's own;
    ``window`` > 0: the last ``window`` of those; ``softcap`` > 0: softcap * tanh(score / softcap);
    ``slopes`` fp32 [q_heads]: + slope * (position - the query's).  Rows outside every sequence are left
    uninitialized.  Prompts and single tokens are faster in two calls than in one."""
    lib = _lib or _load()
    dev = torch.cuda.current_device()
    c, s = _kv_args(cache, seqs, 0, dev)
    H, D = c.heads, c.dim
    heads = q.shape[1] if getattr(q, "is_cuda", False) and q.dim() == 3 else H
    qs, T = _kv_rows(q, "q", heads, D, dev, (_BF,))
    if heads == 0 or H == 0 or heads % H:
        raise RNError(f"q must have shape (tokens, a multiple of {H}, {D}), got {tuple(q.shape)}")
    s.tokens = T
    if slopes is not None:
        _need(slopes, "slopes", _FP32, (heads,))
    need = _kv_attention_bytes(0, H, 0, H, D)   # the dim decides
    if workspace is None:
        workspace = torch.empty(need, dtype=_U8, device=q.device)
    else:
        _need(workspace, "workspace")
    n = ctypes.c_size_t(workspace.numel() * workspace.element_size())
    out = torch.empty((T, heads, D), dtype=_BF, device=q.device)
    lse = torch.empty((T, heads), dtype=_FP32, device=q.device) if return_lse else None
    st = lib.rn_kv_attention(q.data_ptr(), _BF16, qs, heads, c, s, D ** -0.5 if scale is None else float(scale),
                             int(bool(causal)), min(max(int(window), -1), (1 << 63) - 1), float(softcap), _addr(slopes), out.data_ptr(),
                             _addr(lse), workspace.data_ptr(), ctypes.byref(n), _raw_stream(dev))
    if st:
        _check(st, "rn_kv_attention")
    return (out, lse) if return_lse else out


def bwd_workspace_bytes(N, H, dtype, layernorm=True) -> int:
    """Workspace bytes the backward needs (the query step of the protocol)."""
    lib = _load()
    n = ctypes.c_size_t(0)
    code = _BF16 if dtype == torch.bfloat16 else _F32
    if layernorm:
        st = lib.rn_layernorm_bwd(None, None, code, None, None, None, N, H, 0, 0, None, None, None,
                                  None, ctypes.byref(n), None)
    else:
        st = lib.rn_rmsnorm_bwd(None, None, code, None, None, N, H, 0, 0, None, None, None,
                                ctypes.byref(n), None)
    _check(st, "workspace query")
    return int(n.value)


def _workspace(N, H, dtype, layernorm, device, workspace):
    need = bwd_workspace_bytes(N, H, dtype, layernorm)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=device)
    return workspace, ctypes.c_size_t(workspace.numel() * workspace.element_size())


def layernorm_bwd(dz, x, mu, rsigma, gamma, sm_margin=0, zero_centered_gamma=False, workspace=None):
    """LayerNorm backward -> (dx, dgamma, dbeta)."""
    lib = _load()
    _need(x, "x")
    N, H = x.shape
    _need(dz, "dz", x.dtype, (N, H))
    _need(mu, "mu", torch.float32, (N,))
    _need(rsigma, "rsigma", torch.float32, (N,))
    _need(gamma, "gamma", torch.float32, (H,))
    dx = torch.empty_like(x)
    dgamma = torch.empty(H, dtype=torch.float32, device=x.device)
    dbeta = torch.empty(H, dtype=torch.float32, device=x.device)
    ws, n = _workspace(N, H, x.dtype, True, x.device, workspace)
    st = lib.rn_layernorm_bwd(_ptr(dz), _ptr(x), _dtype_code(x), _ptr(mu), _ptr(rsigma), _ptr(gamma),
                              N, H, int(bool(zero_centered_gamma)), int(sm_margin), _ptr(dx),
                              _ptr(dgamma), _ptr(dbeta), _ptr(ws), ctypes.byref(n), _stream())
    _check(st, "rn_layernorm_bwd")
    return dx, dgamma, dbeta


def rmsnorm_bwd(dz, x, rsigma, gamma, sm_margin=0, zero_centered_gamma=False, workspace=None):
    """RMSNorm backward -> (dx, dgamma)."""
    lib = _load()
    _need(x, "x")
    N, H = x.shape
    _need(dz, "dz", x.dtype, (N, H))
    _need(rsigma, "rsigma", torch.float32, (N,))
    _need(gamma, "gamma", torch.float32, (H,))
    dx = torch.empty_like(x)
    dgamma = torch.empty(H, dtype=torch.float32, device=x.device)
    ws, n = _workspace(N, H, x.dtype, False, x.device, workspace)
    st = lib.rn_rmsnorm_bwd(_ptr(dz), _ptr(x), _dtype_code(x), _ptr(rsigma), _ptr(gamma), N, H,
                            int(bool(zero_centered_gamma)), int(sm_margin), _ptr(dx), _ptr(dgamma),
                            _ptr(ws), ctypes.byref(n), _stream())
    _check(st, "rn_rmsnorm_bwd")
    return dx, dgamma


def layernorm_bwd_noalloc(dz, x, mu, rsigma, gamma, sm_margin=0, zero_centered_gamma=False):
    """LayerNorm backward -> (dx, dgamma, dbeta) without a workspace: the
    library's fixed per-device scratch array holds the partial sums (for
    callers that cannot allocate device memory; see include/rn.h for its size
    limit and the rule that overlapping calls race)."""
    lib = _load()
    _need(x, "x")
    N, H = x.shape
    _need(dz, "dz", x.dtype, (N, H))
    _need(mu, "mu", torch.float32, (N,))
    _need(rsigma, "rsigma", torch.float32, (N,))
    _need(gamma, "gamma", torch.float32, (H,))
    dx = torch.empty_like(x)
    dgamma = torch.empty(H, dtype=torch.float32, device=x.device)
    dbeta = torch.empty(H, dtype=torch.float32, device=x.device)
    st = lib.rn_layernorm_bwd_noalloc(_ptr(dz), _ptr(x), _dtype_code(x), _ptr(mu), _ptr(rsigma),
                                      _ptr(gamma), N, H, int(bool(zero_centered_gamma)),
                                      int(sm_margin), _ptr(dx), _ptr(dgamma), _ptr(dbeta), _stream())
    _check(st, "rn_layernorm_bwd_noalloc")
    return dx, dgamma, dbeta


def quantize_only(y, quant, scale=None, rowwise=True, colwise=True):
    """Quantize caller-given fp32 values [N, H] (the unfused quantize step)."""
    lib = _load()
    _need(y, "y", torch.float32)
    N, H = y.shape
    o, res = _make_output(y, quant, None, scale, rowwise, colwise)
    st = lib.rn_quantize_only(_ptr(y), N, H, QUANT_MODES[quant], ctypes.byref(o), _stream())
    _check(st, "rn_quantize_only")
    return res


def device_error() -> int:
    """Read and clear the kernels' device error word (synchronizes)."""
    code = ctypes.c_uint(0)
    _check(_load().rn_device_error(ctypes.byref(code)), "rn_device_error")
    return int(code.value)
