"""GPU parity of the paged 8-bit key/value cache (rn_kv_cache_write, rn_kv_cache_read) and of the attention
over it (rn_kv_attention) against the oracle."""
import numpy as np
import pytest
import torch

import mxfp8_quantization_gb300 as rn
from kv_check import arrays, check, make, oracle_cache, randn
from oracle import kv as K

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _no_device_error():
    yield
    assert rn.device_error() == 0


def same_cache(c, want):
    for got, ref in ((c.k, want.k), (c.v, want.v), (c.k_scales, want.ks), (c.v_scales, want.vs)):
        assert np.array_equal(got.cpu().numpy(), ref)


def f64(t):
    return t.double().cpu().numpy()


# (positions with the new ones, new ones) of each sequence
LENGTHS = [
    [(1, 1)],
    [(64, 64), (65, 1), (63, 63), (128, 1), (0, 0), (130, 70)],
    [(200, 136), (7, 3), (64, 1), (129, 129)],
    [(1, 1)] * 37,
    [(70, 0), (0, 0), (5, 5)],
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("heads,dim", [(1, 64), (3, 128), (2, 192), (1, 256)])
@pytest.mark.parametrize("i", range(len(LENGTHS)))
def test_write(i, heads, dim, dtype):
    lens, news = zip(*LENGTHS[i])
    c, s, T = make(lens, news, heads, dim, seed=i)
    # small, ordinary and large values: pages keep their scales, or grow
    k = randn(T, heads, dim, seed=i, std=3.0, dtype=dtype)
    v = randn(T, heads, dim, seed=i + 50, std=0.02, dtype=dtype)
    want = K.write(oracle_cache(c), *arrays(s), f64(k), f64(v))
    rn.kv_cache_write(c, s, k, v)
    same_cache(c, want)
    rn.kv_cache_write(c, s, k, v)   # again: the scales have grown already
    same_cache(c, K.write(want, *arrays(s), f64(k), f64(v)))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("heads,dim", [(1, 64), (3, 128), (2, 192), (1, 256)])
@pytest.mark.parametrize("i", range(len(LENGTHS)))
def test_read(i, heads, dim, dtype):
    lens, news = zip(*LENGTHS[i])
    c, s, T = make(lens, news, heads, dim, seed=i)
    k, v = rn.kv_cache_read(c, s, T, out_dtype=dtype)
    wk, wv = K.read(oracle_cache(c), *arrays(s), T)
    assert k.dtype == dtype and np.array_equal(f64(k), wk) and np.array_equal(f64(v), wv)


def attend(lens, news, heads, group, dim, seed=0, std=1.5, **kw):
    c, s, T = make(lens, news, heads, dim, seed=seed)
    q = randn(T, heads * group, dim, seed=seed, std=std)
    slopes = kw.get("slopes")
    out, lse = rn.kv_attention(q, c, s, return_lse=True, **kw)
    if slopes is not None:
        kw["slopes"] = slopes.cpu().numpy()
    want = K.attention(f64(q), oracle_cache(c), *arrays(s), dim ** -0.5, **kw)
    check(out, lse, want, dim, kw.get("softcap", 0.0))


@pytest.mark.parametrize("group", [1, 4, 5, 8, 16])
@pytest.mark.parametrize("dim", [64, 128, 192, 256])
def test_one_token(group, dim):
    attend([1, 64, 65, 300, 2, 1000], [1] * 6, 2, group, dim, seed=group)


@pytest.mark.parametrize("group", [1, 3, 8])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_several_tokens(group, dim):
    attend([5, 64, 130, 300, 66, 10], [5, 3, 2, 40, 0, 1], 2, group, dim, seed=group)


@pytest.mark.parametrize("kw", [dict(causal=False), dict(window=1), dict(window=70), dict(softcap=20.0),
                                dict(causal=False, window=33), dict(softcap=5.0, window=100)], ids=str)
@pytest.mark.parametrize("news", [[1, 1, 1], [9, 70, 2]], ids=str)
def test_options(news, kw):
    attend([150, 230, 66], news, 3, 2, 128, **kw)


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_slopes(dim):
    slopes = torch.exp2(-torch.arange(1, 7).float()).cuda()
    attend([150, 230, 66], [1, 5, 66], 3, 2, dim, slopes=slopes)
    attend([150, 230, 66], [1, 5, 66], 3, 2, dim, slopes=slopes, softcap=8.0, window=40)


def test_rows_that_see_nothing():
    # no positions at all; more rows than positions; pages that are none
    c, s, T = make([0, 3, 200], [2, 6, 3], 2, 64)
    s.table[2, :3] = torch.tensor([-1, c.k.shape[0], 1 << 30])
    q = randn(T, 4, 64)
    for causal in (True, False):
        out, lse = rn.kv_attention(q, c, s, causal=causal, return_lse=True)
        check(out, lse, K.attention(f64(q), oracle_cache(c), *arrays(s), 0.125, causal=causal), 64)
    k, v = rn.kv_cache_read(c, s, T)
    wk, wv = K.read(oracle_cache(c), *arrays(s), T)
    assert np.array_equal(f64(k), wk) and np.array_equal(f64(v), wv)
    want = K.write(oracle_cache(c), *arrays(s), f64(q)[:, :2], f64(q)[:, 2:])
    rn.kv_cache_write(c, s, q[:, :2], q[:, 2:])
    same_cache(c, want)
