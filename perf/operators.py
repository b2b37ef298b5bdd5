"""Cases that measure the gated feed-forward block and the 4-bit matrix-vector products.

Four operators, named by a case's "op":

  ffn_fwd      y = s * act(x Wg^T, x Wl^T): both projections of a gated feed-forward block and the
               activation, unquantized (with the projections kept for the backward), FP8 with a given
               scale, or MXFP8 in 1x32 blocks
  ffn_bwd      dx, dW and ds from dy, x, W and the kept projections
  matvec       y = x W^T for one or a few tokens, W in NVFP4 (E2M1 codes, an E4M3 scale per 16, a tensor
               scale)
  gated_matvec y = s * act(x Wg^T, x Wl^T) for one or a few tokens, W in NVFP4

N tokens, K inputs, H outputs; W holds the H gate rows, then the H linear rows.  act is "swiglu"
(a sigmoid(a) b) or "clamped_swiglu" (min(a, L) sigmoid(alpha min(a, L)) (clamp(b, -L, L) + 1)).
"""
import math

import torch

own = False

LIMIT, ALPHA = 7.0, 1.702
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


def _case(name, op, N, K, H, act="", scaled=False, quant="none", out="bf16", pre=False):
    c = {"op": op, "N": N, "K": K, "H": H, "act": act, "scaled": scaled, "quant": quant, "out": out,
         "pre": pre}
    return {"name": name, **c} if name else c


def listed():
    return [
        # one token through the block while it is generated: a call that is all latency and weights
        _case("fwd 1x2048x2048", "ffn_fwd", 1, 2048, 2048, "swiglu"),
        # a short prompt, odd in every size, routed (a weight per token), FP8 for the next product
        _case("fwd 203x1000x2056 fp8", "ffn_fwd", 203, 1000, 2056, "clamped_swiglu", True, "fp8_delayed"),
        # a ragged batch of prompts, MXFP8 for the next product
        _case("fwd 3000x5120x5120 mxfp8", "ffn_fwd", 3000, 5120, 5120, "clamped_swiglu", True, "mxfp8"),
        # a training step's forward, which keeps the projections
        _case("fwd 8192x4096x8192", "ffn_fwd", 8192, 4096, 8192, "swiglu", pre=True),
        # the backward of a small, odd micro-batch of one expert
        _case("bwd 131x1000x1032", "ffn_bwd", 131, 1000, 1032, "clamped_swiglu", True),
        # the backward of a ragged batch, with the gradient of the routing weights
        _case("bwd 3000x5120x5120", "ffn_bwd", 3000, 5120, 5120, "clamped_swiglu", True),
        # a training step's backward
        _case("bwd 8192x4096x8192", "ffn_bwd", 8192, 4096, 8192, "swiglu"),
        # one token through one 4-bit projection
        _case("mv 1x4096x4096", "matvec", 1, 4096, 4096),
        # a few sequences at once, odd sizes, fp32 results
        _case("mv 13x5136x8200 f32", "matvec", 13, 5136, 8200, out="f32"),
        # one token through the last projection, onto the vocabulary
        _case("mv 1x8192x65536", "matvec", 1, 8192, 65536),
        # one token through a 4-bit gated block
        _case("gated mv 1x4096x8192", "gated_matvec", 1, 4096, 8192, "swiglu"),
        # a few routed tokens of one expert through a 4-bit gated block, odd sizes
        _case("gated mv 5x2080x5000", "gated_matvec", 5, 2080, 5000, "clamped_swiglu", True),
    ]


def _logs(rng, lo, hi, step):
    """A multiple of `step` in [lo, hi], spread over the logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return min(hi // step * step, max(step, int(v) // step * step))


def draw(rng):
    top = 8192 * 4096 * 8192
    most = work(_case("", "ffn_bwd", 8192, 4096, 8192, "swiglu"))["bytes"]
    op = rng.choice(["ffn_fwd", "ffn_bwd", "matvec", "gated_matvec"])
    while True:
        act = "" if op == "matvec" else rng.choice(["swiglu", "clamped_swiglu"])
        scaled = op != "matvec" and rng.random() < 0.5
        if op == "ffn_fwd":
            quant = rng.choice(["none", "none", "fp8_delayed", "mxfp8"])
            c = _case("", op, _logs(rng, 1, 16384, 1), _logs(rng, 64, 8192, 8),
                      _logs(rng, 64, 16384, 32 if quant == "mxfp8" else 8), act, scaled, quant,
                      pre=rng.random() < 0.5)
        elif op == "ffn_bwd":
            c = _case("", op, _logs(rng, 1, 16384, 1), _logs(rng, 64, 8192, 8),
                      _logs(rng, 64, 16384, 8), act, scaled)
        else:
            c = _case("", op, _logs(rng, 1, 32, 1), _logs(rng, 256, 16384, 16),
                      _logs(rng, 64, 65536 if op == "matvec" else 32768, 8), act, scaled,
                      out=rng.choice(["bf16", "bf16", "f32"]))
        if c["N"] * c["K"] * c["H"] > top or work(c)["bytes"] > most:
            continue
        if op in ("matvec", "gated_matvec") and c["K"] * _rows(c) > 8192 * 65536:
            continue
        return c


def _rows(case):
    return case["H"] if case["op"] == "matvec" else 2 * case["H"]


def _quantize_weights(w):
    """E2M1 codes (two a byte, the even element low), E4M3 scale codes per 16 and the tensor scale of
    w [R, K] (fp32), to nearest."""
    R, K = w.shape
    big = w.abs().max()
    S = 448.0 * 6.0 / big
    v = w.view(R, K // 16, 16)
    sc = (v.abs().amax(-1) * (S / 6.0)).clamp(max=448.0).to(torch.float8_e4m3fn)
    f = sc.float()
    t = v * torch.where(f > 0, S / f, torch.zeros_like(f))[..., None]
    m = t.abs()
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=w.device)
    code = torch.bucketize(m, edges).to(torch.uint8) | (t < 0).to(torch.uint8) << 3
    code = code.view(R, K // 2, 2)
    return code[..., 0] | code[..., 1] << 4, sc.view(torch.uint8), (1.0 / S).reshape(1), S.reshape(1), big.reshape(1)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    N, K, H, op = case["N"], case["K"], case["H"], case["op"]

    def randn(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device="cuda") * std

    s = {"case": case}
    s["x"] = randn(N, K).bfloat16()  # normalized activations
    w = randn(_rows(case), K, std=2.0 / math.sqrt(K))  # projections reach the clamps
    if case["scaled"]:
        s["scales"] = torch.rand(N, generator=g, device="cuda")
    if op in ("matvec", "gated_matvec"):
        s["codes"], s["blocks"], s["scale_inv"], s["scale"], s["amax"] = _quantize_weights(w)
        return s
    s["w"] = w.bfloat16()
    if case["quant"] == "fp8_delayed":
        s["scale"] = torch.full((1,), 448.0 / 128.0, device="cuda")
    if op == "ffn_bwd":
        s["pre"] = s["x"] @ s["w"].T
        s["dy"] = randn(N, H).bfloat16()
    return s


def _act(a, b, case):
    if case["act"] == "swiglu":
        return a * torch.sigmoid(a) * b
    a = a.clamp(max=LIMIT)
    return a * torch.sigmoid(ALPHA * a) * (b.clamp(-LIMIT, LIMIT) + 1.0)


def _scaled(y, state):
    return y * state["scales"][:, None] if "scales" in state else y


def _dtype(case):
    return torch.float32 if case["out"] == "f32" else torch.bfloat16


def _weights(state):
    """The fp32 values that NVFP4 codes stand for."""
    codes, blocks = state["codes"], state["blocks"]
    R, half = codes.shape
    lut = torch.tensor(E2M1, device=codes.device)
    v = lut[torch.stack([codes & 15, codes >> 4], -1).int()].view(R, half // 8, 16)
    sc = blocks.view(torch.float8_e4m3fn).float() * state["scale_inv"]
    return (v * sc[..., None]).view(R, 2 * half)


def _plain_fwd(state):
    case, H = state["case"], state["case"]["H"]
    p = state["x"].float() @ state["w"].float().T
    y = _scaled(_act(p[:, :H], p[:, H:], case), state)
    out = {}
    if case["quant"] == "fp8_delayed":
        out["y"] = (y * state["scale"]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
        out["amax"] = y.abs().max().reshape(1)
        out["scale_inv"] = 1.0 / state["scale"]
    elif case["quant"] == "mxfp8":
        v = y.view(y.shape[0], H // 32, 32)
        e = (torch.frexp(v.abs().amax(-1)).exponent - 9).clamp(-127, 127)
        out["y"] = (torch.ldexp(v, -e[..., None])).clamp(-448.0, 448.0).view_as(y).to(torch.float8_e4m3fn)
        out["scales"] = (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)
    else:
        out["y"] = y.to(_dtype(case))
    if case["pre"]:
        out["pre"] = p.bfloat16()
    return out


def _plain_bwd(state):
    case, H = state["case"], state["case"]["H"]
    p, dy = state["pre"].float(), state["dy"].float()
    a, b = p[:, :H], p[:, H:]
    if case["act"] == "swiglu":
        sg = torch.sigmoid(a)
        v, da, db = a * sg * b, b * sg * (1.0 + a * (1.0 - sg)), a * sg
    else:
        ac, bc = a.clamp(max=LIMIT), b.clamp(-LIMIT, LIMIT)
        sg = torch.sigmoid(ALPHA * ac)
        v = ac * sg * (bc + 1.0)
        da = torch.where(a <= LIMIT, (bc + 1.0) * sg * (1.0 + ALPHA * ac * (1.0 - sg)), 0.0)
        db = torch.where(b.abs() <= LIMIT, ac * sg, 0.0)
    out = {"dscales": (dy * v).sum(1)}
    sd = _scaled(dy, state)
    dp = torch.cat([sd * da, sd * db], 1)
    out["dx"] = (dp @ state["w"].float()).bfloat16()
    out["dw"] = (dp.T @ state["x"].float()).bfloat16()
    return out


def run(state):
    case, op = state["case"], state["case"]["op"]
    if not own:
        if op == "ffn_fwd":
            return _plain_fwd(state)
        if op == "ffn_bwd":
            return _plain_bwd(state)
        p = state["x"].float() @ _weights(state).T
        if op == "gated_matvec":
            p = _scaled(_act(p[:, :case["H"]], p[:, case["H"]:], case), state)
        return p.to(_dtype(case))

    import mxfp8_quantization_gb300 as rn
    scales = state.get("scales")
    if op == "ffn_fwd":
        y, pre = rn.gated_ffn_fwd(state["x"], state["w"], case["act"], scales, quant=case["quant"],
                                  limit=LIMIT, alpha=ALPHA, scale=state.get("scale"),
                                  save_pre=case["pre"])
        out = {}
        if case["quant"] == "fp8_delayed":
            out = {"y": y.data.view(torch.float8_e4m3fn), "amax": y.amax, "scale_inv": y.scale_inv}
        elif case["quant"] == "mxfp8":
            out = {"y": y.data.view(torch.float8_e4m3fn), "scales": y.row_scales.view(torch.float8_e8m0fnu)}
        else:
            out = {"y": y}
        if case["pre"]:
            out["pre"] = pre
        return out
    if op == "ffn_bwd":
        dx, dw, ds = rn.gated_ffn_bwd(state["dy"], state["x"], state["w"], state["pre"], case["act"],
                                      scales, limit=LIMIT, alpha=ALPHA)
        return {"dx": dx, "dw": dw, "dscales": ds}
    w = rn.NVFP4Output(state["codes"], state["blocks"], state["scale"], state["scale_inv"], state["amax"])
    if op == "matvec":
        return rn.nvfp4_matvec(state["x"], w, out_dtype=_dtype(case))
    return rn.nvfp4_gated_ffn(state["x"], w, case["act"], scales, limit=LIMIT, alpha=ALPHA,
                              out_dtype=_dtype(case))


def work(case):
    N, K, H, R, op = case["N"], case["K"], case["H"], _rows(case), case["op"]
    s = 4 * N if case["scaled"] else 0
    if op == "ffn_fwd":
        y = {"none": 2 * N * H, "fp8_delayed": N * H, "mxfp8": N * H + N * H // 32}[case["quant"]]
        pre = 2 * N * R if case["pre"] else 0
        return {"bytes": 2 * (N * K + R * K) + y + pre + s, "flops": 2 * N * K * R}
    if op == "ffn_bwd":
        return {"bytes": 2 * (N * H + N * K + R * K + N * R) + 2 * (N * K + R * K) + s + 4 * N,
                "flops": 4 * N * K * R}
    esz = 4 if case["out"] == "f32" else 2
    return {"bytes": R * K // 2 + R * K // 16 + 2 * N * K + esz * N * H + s, "flops": 2 * N * K * R}


def exact(case, seed):
    s = prepare(case, seed)
    op, N, H = case["op"], case["N"], case["H"]
    x = s["x"].double()
    if op in ("matvec", "gated_matvec"):
        values = torch.tensor(E2M1, dtype=torch.float64, device="cuda")
        low, high = values[(s["codes"] % 16).long()], values[(s["codes"] // 16).long()]
        group = s["blocks"].view(torch.float8_e4m3fn).double().repeat_interleave(8, 1)
        even, odd = low * group, high * group
        p = (x[:, 0::2] @ even.T + x[:, 1::2] @ odd.T) * s["scale_inv"].double()
        if op == "matvec":
            return p
    elif op == "ffn_fwd":
        p = torch.mm(x, s["w"].double().t())
    else:
        p = s["pre"].double()
    gate, lin = p.split(H, 1)
    if case["act"] == "swiglu":
        top, slope, inner, add, free_g, free_l = gate, 1.0, lin, 0.0, 1.0, 1.0
    else:
        top, slope, inner, add = torch.minimum(gate, gate.new_tensor(LIMIT)), ALPHA, lin.clamp(-LIMIT, LIMIT), 1.0
        free_g, free_l = (gate <= LIMIT).double(), ((lin >= -LIMIT) & (lin <= LIMIT)).double()
    q = 1.0 / (1.0 + torch.exp(-slope * top))
    value = top * q * (inner + add)
    weight = s["scales"].double() if case["scaled"] else torch.ones(N, dtype=torch.float64, device="cuda")
    if op == "ffn_bwd":
        dy = s["dy"].double()
        left = weight[:, None] * dy
        d_gate = left * (inner + add) * (q + slope * top * q * (1.0 - q)) * free_g
        d_lin = left * top * q * free_l
        w, out = s["w"].double(), {"dscales": torch.einsum("nh,nh->n", dy, value)}
        out["dx"] = d_gate @ w[:H] + d_lin @ w[H:]
        out["dw"] = torch.cat([d_gate.t() @ x, d_lin.t() @ x])
        return out
    y = weight[:, None] * value
    if op == "gated_matvec":
        return y
    if case["quant"] == "fp8_delayed":
        t = s["scale"].double()
        out = {"y": torch.clamp(y * t, -448.0, 448.0), "amax": y.abs().max().reshape(1), "scale_inv": 1.0 / t}
    elif case["quant"] == "mxfp8":
        blocks = y.reshape(N, H // 32, 32)
        power = torch.floor(torch.log2(blocks.abs().amax(-1))).clamp(min=-119.0) - 8.0
        out = {"y": (blocks * torch.exp2(-power)[..., None]).clamp(-448.0, 448.0).reshape(N, H),
               "scales": torch.exp2(power)}
    else:
        out = {"y": y}
    if case["pre"]:
        out["pre"] = p
    return out
