"""The few-token kernel's plan on the host: that it covers the work, and fits."""
import math
import random

import pytest

from matvec_plan import plan

STATIC = 1024  # the kernel's own shared memory is below that, and the driver keeps 1 KB a CTA


def draws(n=4000, seed=1):
    r = random.Random(seed)

    def logs(lo, hi, step):
        return max(step, int(math.exp(r.uniform(math.log(lo), math.log(hi)))) // step * step)

    for _ in range(n):
        nvfp4 = r.random() < 0.75
        gated = not nvfp4 or r.random() < 0.5
        N = logs(1, 200, 1) if nvfp4 else logs(1, 32, 1)
        mx = gated and r.random() < 0.3
        yield dict(N=N, K=logs(8, 131072, 16 if nvfp4 else 8), H=logs(1, 200000, 32 if mx else 1), nvfp4=nvfp4,
                   gated=gated, mx=mx)


def test_every_plan_covers_the_work_and_fits():
    for c in draws():
        p = plan(**c)
        assert p is not None, c
        ck = 256 if c["nvfp4"] else 64
        assert p.chunks * ck >= c["K"] > (p.chunks - 1) * ck, c
        assert p.split in (1, 2, 4, 8) and p.split * p.part >= p.chunks, c
        assert p.W % p.kw == 0 and 1 <= p.kw <= p.W, c
        assert p.steps * p.rw >= p.tiles > (p.steps - 1) * p.rw, c
        assert 1 <= p.groups <= p.steps and p.ny * 8 * p.T >= c["N"], c
        assert 1 <= p.slab <= p.part and p.batch >= 1, c
        if c["mx"]:
            assert p.rw * 16 % 32 == 0, c          # a step's outputs are whole blocks
        # tokens, two steps' sums, a cluster's sums, and the sums that are kept while slabs change
        step = p.rw * p.n * 32 * 4
        need = p.slab * (ck // 32) * (p.n * 64 + 16) + 2 * p.W * p.n * 36 * 4
        need += p.split * step if p.split > 1 else 0
        need += p.batch * step if p.slabs > 1 else 0
        assert p.smem == need, c
        assert (p.smem + STATIC) * p.per_sm <= 227 * 1024, c
        assert p.batch >= p.rounds or p.slabs > 1, c


def busiest(p, kw):
    """Chunks of the warp with the most to do, tokens whole, with kw warps along the reduction."""
    steps = -(-p.tiles // (p.W // kw)) * p.ny * p.split
    return -(-steps // (152 * p.per_sm)) * -(-p.part // kw)


def test_no_plan_leaves_sms_idle_that_would_help():
    """Where a plan has fewer CTAs than SMs, no other number of warps along the reduction gives the busiest warp
    half as much to do or less (with at most twice the rounds of steps)."""
    for c in [dict(N=16, K=2048, H=20000), dict(N=16, K=2048, H=10240, gated=True), *draws()]:
        p = plan(**c)
        if p.ctas >= 152 or p.slabs > 1:
            continue
        now = busiest(p, p.kw)
        for kw in range(p.kw + 1, p.W + 1):
            steps = -(-p.tiles // (p.W // kw)) * p.ny * p.split
            if p.W % kw or (c.get("mx") and p.W // kw % 2) or steps > 2 * 152 * p.per_sm:
                continue
            assert 2 * busiest(p, kw) > now, (c, p.kw, kw)


def test_twelve_warps_take_the_divisors_in_between():
    # 3 warps along the reduction halve to 1, which leaves 53 and 86 CTAs
    assert plan(16, 2048, 20000).ctas == 105 and plan(16, 2048, 32768).ctas == 152
    assert plan(30, 1040, 20000).ctas == 79      # kept: no number of warps gives the busiest less


def test_clusters_whose_tokens_do_not_fit_go_on_in_slabs():
    """Few rows and a long reduction: the reduction stays split over clusters where a CTA's tokens do not fit."""
    assert plan(24, 16384, 512).ctas == 128
    for N, K, H, least in [(32, 16384, 64, 16), (32, 16384, 512, 64), (32, 16384, 1024, 128), (32, 16384, 2048, 128),
                           (32, 12288, 1024, 128), (32, 12288, 4096, 128), (12, 65536, 40, 16), (8, 88064, 64, 16)]:
        assert plan(N, K, H).ctas >= least, (N, K, H)
    for K in range(4096, 16385, 512):
        for N in range(17, 32):
            a, b = plan(N, K, 512), plan(N + 1, K, 512)
            assert 2 * b.ctas >= a.ctas, (N, K)  # a token more does not idle most of the machine


def test_slabs_of_a_cluster():
    for c in draws(seed=2):
        p = plan(**c)
        if p.split > 1 and p.slabs > 1:
            assert p.T > 1
            assert p.slab * p.slabs >= p.part and (p.slabs - 1) * p.slab < p.part, c
            assert p.groups * p.ny <= max(p.ny, 152 // p.split), c  # no second wave of clusters
