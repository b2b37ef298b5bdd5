"""Row counts that leave the last group of rows short, with the rows walked
from the last one (the second pass of current scaling and NVFP4): the short
group comes first there, and its slot of the ring is used again.

A ring holds Q slots of 2, 4 or 8 rows of less than 8 KB; the sizes give every
CTA more groups than that.  Rows of zeros appended up to whole groups change
neither the amax nor another row's codes, so the results have to be the same."""
import pytest
import torch

import mxfp8_quantization_gb300 as rn

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _no_device_error():
    yield
    assert rn.device_error() == 0


def padded(x):
    rows = -x.shape[0] % 8
    return torch.cat([x, torch.zeros(rows, x.shape[1], dtype=x.dtype, device="cuda")])


def same(a, b, N):
    assert torch.equal(a.amax, b.amax) and torch.equal(a.scale, b.scale)
    assert torch.equal(a.data, b.data[:N])
    if hasattr(a, "row_scales"):
        assert torch.equal(a.row_scales, b.row_scales[:N])


def rows(N, H, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(N, H, generator=g, device="cuda").to(dtype)


# rows a slot, slots: 4, 21; 8, 27; 4, 27; 2, 27 (fp32 624, bf16 512, 1024, 2048 columns)
@pytest.mark.parametrize("N", [17593, 17594, 17595])
@pytest.mark.parametrize("quant", ["nvfp4", "fp8_current"])
def test_quantizer(N, quant):
    x = rows(N, 624, torch.float32, N)
    same(rn.quantize_only(x, quant), rn.quantize_only(padded(x), quant), N)


@pytest.mark.parametrize("N,H", [(65537, 512), (65543, 512), (20001, 1024), (20003, 1024), (16385, 2048)])
@pytest.mark.parametrize("quant", ["nvfp4", "fp8_current"])
def test_norms(N, H, quant):
    x = rows(N, H, torch.bfloat16, N)
    gamma = 1 + 0.1 * torch.randn(H, generator=torch.Generator().manual_seed(H)).cuda()
    a, mu, rs = rn.layernorm_fwd(x, gamma, None, 1e-5, quant=quant)
    b, mu2, rs2 = rn.layernorm_fwd(padded(x), gamma, None, 1e-5, quant=quant)
    same(a, b, N)
    assert torch.equal(mu, mu2[:N]) and torch.equal(rs, rs2[:N])
    a, rs = rn.rmsnorm_fwd(x, gamma, 1e-5, quant=quant)
    b, rs2 = rn.rmsnorm_fwd(padded(x), gamma, 1e-5, quant=quant)
    same(a, b, N)
    if quant == "fp8_current":  # the same codes as one pass with that scale, which walks the rows forwards
        c, _ = rn.rmsnorm_fwd(x, gamma, 1e-5, quant="fp8_delayed", scale=a.scale)
        assert torch.equal(a.data, c.data)


@pytest.mark.parametrize("quant", ["nvfp4", "fp8_current"])
def test_residual_norm(quant):
    N, H = 20001, 1024
    x, r = rows(N, H, torch.bfloat16, 1), rows(N, H, torch.bfloat16, 2)
    gamma = torch.ones(H, device="cuda")
    a, h, rs = rn.rmsnorm_add_fwd(x, r, gamma, 1e-5, quant=quant)
    b, h2, rs2 = rn.rmsnorm_add_fwd(padded(x), padded(r), gamma, 1e-5, quant=quant)
    same(a, b, N)
    assert torch.equal(h, h2[:N]) and torch.equal(rs, rs2[:N])
