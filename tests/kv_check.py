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
        assert np.all(np.abs(g[some] - want["lse"][some]) <= tol_lse[some])


def reference(q, c, s, scale=None, causal=True, window=0, softcap=0.0, slopes=None):
    """K.attention in fp64 torch operations on the GPU, for longer sequences (every position cached)."""
    T, heads, D = q.shape
    H = c.k.shape[1]
    G = heads // H
    scale = D ** -0.5 if scale is None else scale
    f = dict(dtype=torch.float64, device="cuda")
    r = {"out": torch.full(q.shape, float("nan"), **f), "lse": torch.full((T, heads), float("nan"), **f),
         "pv": torch.zeros(q.shape, **f), "big": torch.zeros(T, heads, **f), "spread": torch.zeros(q.shape, **f),
         "seen": torch.zeros(T, heads, **f)}
    table, starts, lens = (t.cpu() for t in (s.table, s.starts, s.lens))
    for b in range(len(lens)):
        n, a, z = int(lens[b]), int(starts[b]), int(starts[b + 1])
        if n == 0 or a == z:
            r["out"][a:z], r["lse"][a:z] = 0.0, -float("inf")
            continue
        ids = table[b, :(n + PAGE - 1) // PAGE].long().cuda()
        unit = torch.exp2(c.v_scales[ids].double() - 127).T.repeat_interleave(PAGE, 1)[:, :n]
        k = c.k[ids].view(torch.float8_e4m3fn).double() * torch.exp2(c.k_scales[ids].double() - 127)[..., None, None]
        v = c.v[ids].view(torch.float8_e4m3fn).double() * torch.exp2(c.v_scales[ids].double() - 127)[..., None, None]
        k = k.transpose(0, 1).reshape(H, -1, D)[:, :n]
        v = v.permute(1, 0, 3, 2).reshape(H, -1, D)[:, :n]
        p = (n - (z - a) + torch.arange(z - a, device="cuda"))[:, None]
        j = torch.arange(n, device="cuda")[None]
        sees = (j <= p if causal else j >= 0) & (j > p - window if window else j >= 0) & (j >= 0)
        sees = sees.expand(z - a, n)
        for h in range(heads):
            qq, kk, vv = q[a:z, h].double(), k[h // G], v[h // G]
            t = scale * (qq @ kk.T)
            big = (scale * (qq.abs() @ kk.abs().T)).masked_fill(~sees, 0).amax(1)
            if softcap:
                t = softcap * torch.tanh(t / softcap)
            if slopes is not None:
                t = t + slopes[h].double() * (j - p)
                big = torch.maximum(big, (slopes[h].double().abs() * (j - p).abs()).masked_fill(~sees, 0).amax(1))
            t = t.masked_fill(~sees, -float("inf"))
            lse = torch.logsumexp(t, 1)
            w = torch.exp(t - lse[:, None]).nan_to_num(0.0)
            r["lse"][a:z, h], r["out"][a:z, h], r["pv"][a:z, h], r["big"][a:z, h] = lse, w @ vv, w @ vv.abs(), big
            u = unit[h // G]
            r["spread"][a:z, h] = (w * u).amax(1)[:, None] * (vv.abs() / u[:, None]).sum(0)
            r["seen"][a:z, h] = sees.sum(1).double()
    return {n: t.cpu().numpy() for n, t in r.items()}
