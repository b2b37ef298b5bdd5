"""Caches, sequences and error bounds for the tests of the paged 8-bit key/value cache."""
import numpy as np
import torch

import mxfp8_quantization_gb300 as rn
from oracle import kv as K

PAGE = 64


def make(lens, news, heads, dim, seed=0, spare=3, spread=0.5, device="cuda"):
    """A cache of random pages and sequences with `news` rows each: (KVCache, KVSequences, tokens); the
    cache holds every position of every sequence.  `spread`: sigma of the pages' log2 sizes."""
    g = torch.Generator().manual_seed(seed)
    blocks = [(n + PAGE - 1) // PAGE for n in lens]
    pages, width = sum(blocks) + spare, max(max(blocks, default=0), 1)
    order = torch.randperm(pages, generator=g).int()
    table = torch.full((len(lens), width), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(blocks):
        table[b, :n] = order[at:at + n]
        at += n
    size = torch.exp2(torch.randn(pages, heads, 1, 1, generator=g) * spread)
    k = torch.randn(pages, heads, PAGE, dim, generator=g) * size
    v = torch.randn(pages, heads, dim, PAGE, generator=g) * size.flip(0)

    def codes(x):
        e = torch.ceil(torch.log2(x.abs().amax((2, 3)) / 448.0))
        c = (x * torch.exp2(-e)[..., None, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        return c.to(device), (e + 127).to(torch.uint8).to(device)

    kc, ks = codes(k)
    vc, vs = codes(v)
    starts = torch.tensor([0] + list(news)).cumsum(0).int()
    seqs = rn.KVSequences(table.to(device), starts.to(device), torch.tensor(lens, dtype=torch.int32).to(device))
    return rn.KVCache(kc, vc, ks, vs), seqs, int(starts[-1])


def oracle_cache(c):
    return K.Cache(*(t.cpu().numpy() for t in (c.k, c.v, c.k_scales, c.v_scales)))


def arrays(s):
    return tuple(t.cpu().numpy() for t in (s.table, s.starts, s.lens))


def randn(*shape, seed=0, std=1.0, dtype=torch.bfloat16):
    g = torch.Generator().manual_seed(seed + 7)
    return (torch.randn(*shape, generator=g) * std).to(dtype).cuda()


def bounds(want, dim, softcap=0.0):
    """How far out and lse may be from the oracle's, from the arithmetic:

    scores   sums of dim exact products that cut off: dim 2^-23 of the magnitudes ("big" bounds them and the
             bias' product), five fp32 roundings 2^-24 each, the row's elements in f16 2^-39 of the largest;
             the cap adds 2^-22 of itself (its exponential and its division); as a part of a weight, together
             with the exponential's own 2^-22 and the rescalings' 2^-23 a page: eps
    weights  rounded to f16: 2^-11, or 2^-25 of the largest weight times its page's scale ("spread")
    sums     n / 16 steps of 16 products that cut off, 2^-23 each of the magnitudes; the fp32 sum of the
             weights n 2^-24; joining the parts 2^-22
    output   bf16: 2^-8
    """
    seen = want["seen"].astype(np.float64)
    eps = want["big"] * ((dim + 8) * 2.0 ** -23) + softcap * 2.0 ** -21 + 2.0 ** -20 + (seen / 64 + 2) * 2.0 ** -22
    part = 2.0 ** -11 + 2 * eps + (seen / 8 + 4) * 2.0 ** -23 + seen * 2.0 ** -24
    out = want["pv"] * part[..., None] + want["spread"] * 2.0 ** -25
    out = out + (np.abs(want["out"]) + out) * 2.0 ** -8
    lse = eps + seen * 2.0 ** -24 + (np.abs(np.where(np.isfinite(want["lse"]), want["lse"], 0.0)) + 1) * 2.0 ** -22
    return out, lse


def check(out, lse, want, dim, softcap=0.0):
    tol, tol_lse = bounds(want, dim, softcap)
    got = out.double().cpu().numpy()
    rows = ~np.isnan(want["out"])
    err = np.abs(got - want["out"])[rows]
    assert np.all(np.isfinite(got[rows]))
    assert np.all(err <= tol[rows]), (float((err / tol[rows].clip(1e-30)).max()), int((err > tol[rows]).sum()))
    if lse is not None:
        g = lse.double().cpu().numpy()
        none = want["lse"] == -np.inf
        assert np.array_equal(g == -np.inf, none)
        some = ~none & ~np.isnan(want["lse"])
        assert np.all(np.abs(g - want["lse"])[some] <= tol_lse[some])
