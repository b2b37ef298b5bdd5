"""GPU parity of the attention over the paged 8-bit cache where its numbers or its parts lie far apart."""
import numpy as np
import pytest
import torch

import mxfp8_quantization_gb300 as rn
from kv_check import arrays, check, make, oracle_cache, randn, reference
from oracle import kv as K

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
    """kv_check.bounds, without what grows with the cap and without what a weight far below the largest loses:

    cap      relative to the capped score: its error is below 2^-21 of the cap where z / c is above 1/4, whose tanh
             is 0.245
    weights  the largest stands at 2^9 or above in f16, so half a step of its subnormals, 2^-25, is 2^-34 of it
    """
    seen = want["seen"].astype(np.float64)
    eps = want["big"] * ((dim + 8) * 2.0 ** -23) + 2.0 ** -20 + (seen / 64 + 2) * 2.0 ** -22
    if softcap:
        eps = eps + np.minimum(want["big"], softcap) * 2.0 ** -18
    part = 2.0 ** -11 + 2 * eps + (seen / 8 + 4) * 2.0 ** -23 + seen * 2.0 ** -24
    out = want["pv"] * part[..., None] + want["spread"] * 2.0 ** -34
    out = out + (np.abs(want["out"]) + out) * 2.0 ** -8
    lse = eps + seen * 2.0 ** -24 + (np.abs(want["lse"]) + 1) * 2.0 ** -22
    return out, lse


def close(out, lse, want, dim, softcap=0.0):
    tol, tol_lse = bounds(want, dim, softcap)
    err, err_lse = np.abs(f64(out) - want["out"]), np.abs(f64(lse) - want["lse"])
    assert np.all(err <= tol), (float((err / tol.clip(1e-300)).max()), int((err > tol).sum()))
    assert np.all(err_lse <= tol_lse), float((err_lse / tol_lse).max())


def shared(k, v, sequences, new):
    """A cache of the rows k, v [n, heads, dim] (fp32) that all sequences read, with `new` rows each."""
    n, heads, dim = k.shape
    pages = -(-n // 64)
    c = rn.kv_cache_alloc(pages, heads, dim)
    i32 = lambda t: torch.tensor(t, dtype=torch.int32, device="cuda")
    table = i32([list(range(pages))])
    rn.kv_cache_write(c, rn.KVSequences(table, i32([0, n]), i32([n])), k, v)
    return c, rn.KVSequences(table.expand(sequences, pages).contiguous(), i32([new * b for b in range(sequences + 1)]),
                             i32([n] * sequences))


def shared_reference(q, c, s, new):
    """kv_check.reference of `shared`, whose sequences all see every position, in one piece."""
    n, H, D = int(s.lens[0]), c.k.shape[1], q.shape[2]
    G, B = q.shape[1] // H, len(s.lens)
    ids = s.table[0].long()
    unit = torch.exp2(c.v_scales[ids].double() - 127).T.repeat_interleave(64, 1)[:, None, :n]     # [H, 1, n]
    k = c.k[ids].view(torch.float8_e4m3fn).double() * torch.exp2(c.k_scales[ids].double() - 127)[..., None, None]
    k = k.transpose(0, 1).reshape(H, -1, D)[:, :n]
    codes = c.v[ids].view(torch.float8_e4m3fn).double().permute(1, 0, 3, 2).reshape(H, -1, D)[:, :n]
    v = codes * unit.transpose(1, 2)
    x = q.double().view(B * new, H, G, D).permute(1, 0, 2, 3).reshape(H, -1, D)
    t = D ** -0.5 * (x @ k.transpose(1, 2))
    lse = torch.logsumexp(t, 2)
    w = torch.exp(t - lse[..., None])
    r = {"out": w @ v, "pv": w @ v.abs(), "lse": lse, "big": D ** -0.5 * (x.abs() @ k.abs().transpose(1, 2)).amax(2),
         "spread": (w * unit).amax(2)[..., None] * codes.abs().sum(1, keepdim=True),
         "seen": torch.full_like(lse, n)}
    back = lambda y: y.view(H, B * new, G, *y.shape[2:]).transpose(0, 1).reshape(B * new, H * G, *y.shape[2:])
    return {name: back(y).cpu().numpy() for name, y in r.items()}


# few rows a head (8 at most, 16 at most) and many: (new rows, query heads a head)
FORMS = [(1, 4), (4, 4), (10, 8)]


@pytest.mark.parametrize("cap", [1e-3, 1.0, 8.0, 50.0, 1e3, 1e4, 1e6, 1e12, 1e30])
@pytest.mark.parametrize("dim,new,group", [(64, 1, 4), (64, 4, 4), (64, 10, 8), (256, 1, 4), (256, 10, 8)])
def test_caps_of_any_size(dim, new, group, cap):
    c, s, T = make([700, 130], [new, new], 2, dim, seed=1)
    q = randn(T, 2 * group, dim, seed=2, std=2.0)
    out, lse = rn.kv_attention(q, c, s, softcap=cap, return_lse=True)
    close(out, lse, reference(q, c, s, softcap=cap), dim, cap)


@pytest.mark.parametrize("at", [0, 1000])
@pytest.mark.parametrize("nats", [13.0, 16.0, 20.0])
@pytest.mark.parametrize("dim", [64, 256])
@pytest.mark.parametrize("new,group", FORMS)
def test_a_position_that_takes_most_of_the_weight(new, group, dim, nats, at):
    # with values of 0, so that the output is what the others leave; enough heads for ranges of whole sequences
    n, heads, B = 2000, 16, (76 if new == 1 else 40 if new == 4 else 12)
    g = torch.Generator(device="cuda").manual_seed(3)
    k, v = (torch.randn(n, heads, dim, device="cuda", generator=g) for _ in "kv")
    k[..., 0] = 0.0
    k[at] = 0.0
    k[at, :, 0] = nats * dim ** 0.5 / 8
    v[at] = 0.0
    c, s = shared(k, v, B, new)
    q = randn(B * new, heads * group, dim, seed=4, std=0.4)
    q[..., 0] = 8.0
    out, lse = rn.kv_attention(q, c, s, causal=False, return_lse=True)
    close(out, lse, shared_reference(q, c, s, new), dim)


@pytest.mark.parametrize("sequences", [2, 80])       # a page a worker, and several
@pytest.mark.parametrize("first", [0, 1])            # which page has the weight
@pytest.mark.parametrize("bits", [100, 161, 201])    # how far the other's scores lie below
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("new,group", FORMS)
def test_little_weight_on_very_large_values(new, group, dim, bits, first, sequences):
    # values of 2^-120 where the weight is, of 2^119 elsewhere: those decide the output
    heads = 16 if sequences > 2 else 2
    g = torch.Generator(device="cuda").manual_seed(5)
    k, v = (torch.randn(128, heads, dim, device="cuda", generator=g) for _ in "kv")
    there, far = slice(64 * first, 64 * first + 64), slice(64 - 64 * first, 128 - 64 * first)
    k[..., 0] = 0.0
    k[far, :, 0] = -bits * np.log(2) * dim ** 0.5 / 64
    v[there] *= 2.0 ** -116
    v[far] *= 2.0 ** 124
    c, s = shared(k, v, sequences, new)
    q = randn(sequences * new, heads * group, dim, seed=6, std=0.5)
    q[..., 0] = 64.0
    out, lse = rn.kv_attention(q, c, s, causal=False, return_lse=True)
    close(out, lse, shared_reference(q, c, s, new), dim)


@pytest.mark.parametrize("sequences", [1, 40])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("new,group", FORMS + [(10, 16)])
def test_values_at_the_least_scale(new, group, dim, sequences):
    # scores that rise from page to page by little, values of the smallest pages there are
    heads = 8 if sequences > 1 else 1
    g = torch.Generator(device="cuda").manual_seed(7)
    k, v = (torch.randn(320, heads, dim, device="cuda", generator=g) for _ in "kv")
    k[..., 0] = (torch.arange(5, device="cuda") * 1.9 * np.log(2) * dim ** 0.5 / 8).repeat_interleave(64)[:, None]
    v *= 2.0 ** -116
    c, s = shared(k, v, sequences, new)
    assert (c.v_scales == 7).all()
    q = randn(sequences * new, heads * group, dim, seed=8, std=0.1)
    q[..., 0] = 8.0
    out, lse = rn.kv_attention(q, c, s, causal=False, return_lse=True)
    close(out, lse, shared_reference(q, c, s, new), dim)


@pytest.mark.parametrize("new,group", FORMS)
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_scale_bytes_that_no_write_leaves(new, group, dim):
    c, s, T = make([64 * 7] * 3, [new] * 3, 2, dim, seed=9)
    for i, byte in enumerate((0, 6, 7, 246, 247, 255)):
        pages = s.table[:, i].long()
        c.v_scales[pages] = byte
        c.k_scales[pages] = min(byte, 7)     # (scores of 2^119 would be none)
    near = rn.KVCache(c.k, c.v, c.k_scales.clamp(7, 246), c.v_scales.clamp(7, 246))
    q = randn(T, 2 * group, dim, seed=9)
    for kw in (dict(), dict(causal=False, window=200)):
        got, want = (rn.kv_attention(q, x, s, return_lse=True, **kw) for x in (c, near))
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    c.k_scales[:] = c.v_scales
    every = rn.KVSequences(s.table, torch.arange(4, dtype=torch.int32, device="cuda") * 64 * 7, s.lens)
    for dtype in (torch.bfloat16, torch.float32):
        got = rn.kv_cache_read(c, every, 3 * 64 * 7, out_dtype=dtype)
        want = K.read(oracle_cache(c), *arrays(every), 3 * 64 * 7)
        assert all(np.array_equal(f64(x), y) for x, y in zip(got, want))


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("bits", [8, 13, 19])     # (8 * 2^19 is the largest score there may be)
@pytest.mark.parametrize("sequences", [1, 60])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("new,group", FORMS + [(10, 16)])
def test_scores_up_to_the_largest(new, group, dim, sequences, bits, sign):
    # exact multiples of 2^bits, so that all weight is at the two positions of the largest; pages of different size
    n, heads, at = 330, 2, [70, 75]
    g = torch.Generator(device="cuda").manual_seed(10)
    k, v = (torch.randn(n, heads, dim, device="cuda", generator=g) for _ in "kv")
    k[..., 0] = torch.randint(-7, 1, (n, heads), device="cuda", generator=g) - (1.0 if sign < 0 else 0.0)
    k[at, :, 0] = 8.0 if sign > 0 else -0.5
    v *= torch.exp2(torch.tensor([0.0, -15.0, 5.0, 1.0, -60.0, 3.0], device="cuda").repeat_interleave(64)[:n, None, None])
    c, s = shared(k, v, sequences, new)
    q = torch.zeros(sequences * new, heads * group, dim, dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 2.0 ** bits
    out, lse = rn.kv_attention(q, c, s, scale=1.0, causal=False, return_lse=True)
    every = rn.KVSequences(s.table[:1], torch.tensor([0, n], dtype=torch.int32, device="cuda"), s.lens[:1])
    kk, vv = rn.kv_cache_read(c, every, n, out_dtype=torch.float32)
    assert (kk[at, :, 0] == k[at, :, 0]).all()
    want = f64(vv[at].double().mean(0).repeat_interleave(group, 0))
    size = f64(vv[at].double().abs().mean(0).repeat_interleave(group, 0))
    # the others are e^-128 and less, and 2^20 larger at most.  Two equal weights, each rounded once to f16 (2^-11);
    # exponentials and divisions 2^-20; the output bf16
    tol = size * (2.0 ** -11 + 2.0 ** -20) + np.abs(want) * 2.0 ** -8 + 2.0 ** -60
    assert np.all(np.abs(f64(out) - want) <= tol), float((np.abs(f64(out) - want) / tol).max())
    top = 2.0 ** bits * float(k[at[0], 0, 0])
    # the maximum in base 2, its unit and back: four roundings of 2^-24 and the exponential's 2^-22
    assert np.all(np.abs(f64(lse) - top - np.log(2)) <= abs(top) * 2.0 ** -22 + 2.0 ** -20)
