"""GPU parity of the paged 8-bit key/value cache (rn_kv_cache_write, rn_kv_cache_read) and of the attention
over it (rn_kv_attention) against the oracle."""
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


# ------------------------------------------------------------------ many workers
# few rows (a warp a worker) and many (tiles): one head whose pages all workers share, more heads than workers, ragged
LONG = [([9000], [1], 1, 8, 128), ([20000, 70, 3000], [1, 1, 1], 2, 4, 64), ([5000], [2], 3, 8, 128),
        ([7000, 100], [1, 1], 1, 16, 256), ([2500] * 9, [1] * 9, 16, 1, 64), ([3000, 500], [1, 3], 2, 5, 192),
        ([130] * 70, [1] * 70, 3, 4, 128), ([9000], [30], 1, 8, 128), ([3000, 64], [300, 64], 2, 4, 128),
        ([6000], [20], 1, 8, 256), ([1500, 700], [100, 33], 3, 2, 192), ([2000], [257], 2, 1, 64),
        ([12000], [3], 1, 6, 64)]


@pytest.mark.parametrize("lens,news,heads,group,dim", LONG, ids=str)
def test_shared_by_workers(lens, news, heads, group, dim):
    c, s, T = make(lens, news, heads, dim, seed=dim)
    q = randn(T, heads * group, dim, seed=3, std=2.0)
    out, lse = rn.kv_attention(q, c, s, return_lse=True)
    check(out, lse, reference(q, c, s), dim)


@pytest.mark.parametrize("news", [[1] * 5, [40] * 5], ids=str)
def test_more_sequences_than_stand_in_shared_memory(news):
    lens = ([70, 1, 64, 130, 41] * 260)[:1300]
    c, s, T = make(lens, (news * 260)[:1300], 1, 64, seed=1)
    q = randn(T, 2, 64)
    out, lse = rn.kv_attention(q, c, s, return_lse=True)
    # rows of sequences with more rows than positions begin in front of them
    check(out, lse, reference(q, c, s), 64)


# ------------------------------------------------------------- what is not seen
@pytest.mark.parametrize("new,window", [(1, 0), (1, 50), (5, 0), (5, 50), (40, 0), (40, 50)])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_what_is_not_seen_has_no_part(new, window, dim):
    lens = [300, 65, 128]
    c, s, T = make(lens, [new] * 3, 2, dim, seed=2)
    q = randn(T, 8, dim)
    want, lse = rn.kv_attention(q, c, s, window=window, return_lse=True)
    table = s.table.cpu()
    for b, n in enumerate(lens):
        # NaN keys and values behind the end, in every page of nobody's, and in front of all windows
        page = int(table[b, (n - 1) // 64])
        if n % 64:
            c.k[page, :, n % 64:] = 0x7F
            c.v[page, :, :, n % 64:] = 0xFF
        first = max(0, n - new + 1 - window) if window else 0
        for j in range(first):
            c.k[int(table[b, j // 64]), :, j % 64] = 0x7F
            c.v[int(table[b, j // 64]), :, :, j % 64] = 0x7F
    used = set(table[table >= 0].tolist())
    for page in range(c.k.shape[0]):
        if page not in used:
            c.k[page], c.v[page], c.k_scales[page], c.v_scales[page] = 0x7F, 0x7F, 255, 255
    out, lse2 = rn.kv_attention(q, c, s, window=window, return_lse=True)
    assert torch.equal(out, want) and torch.equal(lse, lse2)


@pytest.mark.parametrize("new,group", [(6, 2), (6, 8), (40, 4)])
@pytest.mark.parametrize("dim", [64, 128, 192])
def test_a_nan_reaches_those_that_see_it(new, group, dim):
    n = 200
    c, s, T = make([n, n], [new, new], 2, dim, seed=4)
    q = randn(T, 2 * group, dim)
    want = rn.kv_attention(q, c, s)
    page = int(s.table[0, (n - 3) // 64])
    c.v[page, 1, 5, (n - 3) % 64] = 0x7F       # head 1, position n - 3 of sequence 0
    out = rn.kv_attention(q, c, s)
    assert torch.equal(out[:new - 3], want[:new - 3]) and torch.equal(out[new:], want[new:])
    assert torch.equal(out[new - 3:new, :group], want[new - 3:new, :group])
    assert torch.isnan(out[new - 3:new, group:, 5]).all()


@pytest.mark.parametrize("new", [1, 30])
def test_rows_of_non_finite_queries(new):
    c, s, T = make([150, 90], [new, new], 2, 128, seed=5)
    q = randn(T, 4, 128)
    want = rn.kv_attention(q, c, s)
    q2 = q.clone()
    q2[0, 1, 3], q2[new, 2, 0] = float("nan"), float("inf")
    out = rn.kv_attention(q2, c, s)
    keep = torch.ones(T, 4, dtype=torch.bool, device="cuda")
    keep[0, 1], keep[new, 2] = False, False
    assert torch.equal(out[keep], want[keep]) and torch.isnan(out[0, 1]).all()


# ------------------------------------------------------------------------ ranges
@pytest.mark.parametrize("new", [1, 33])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_pages_of_very_different_size(new, dim):
    c, s, T = make([640, 320], [new, new], 2, dim, seed=6)
    # values 2^40 apart from page to page, a page of zeros with the least scale; keys that hardly count
    c.v_scales[:] = (c.v_scales.int() + torch.randint(-20, 20, c.v_scales.shape, device="cuda") * 2).clamp(7, 246).byte()
    page = int(s.table[0, 2])
    c.v[page], c.v_scales[page] = 0, 7
    c.k_scales[int(s.table[0, 4])] -= 20
    q = randn(T, 4, dim, std=1.0)
    out, lse = rn.kv_attention(q, c, s, return_lse=True)
    check(out, lse, reference(q, c, s), dim)


@pytest.mark.parametrize("new", [1, 30])
@pytest.mark.parametrize("std", [2.0 ** -60, 2.0 ** -10, 30.0])
def test_small_and_large_queries(new, std):
    c, s, T = make([400, 64], [new, new], 2, 128, seed=7)
    q = randn(T, 8, 128, std=std)
    q[0, 0] = 0
    out, lse = rn.kv_attention(q, c, s, return_lse=True)
    check(out, lse, reference(q, c, s), 128)


def test_values_at_the_ends_of_the_scale():
    c = rn.kv_cache_alloc(3, 1, 64)
    s = rn.KVSequences(*(torch.tensor(t, dtype=torch.int32, device="cuda") for t in ([[2], [0]], [0, 3, 4], [3, 1])))
    k = torch.zeros(4, 1, 64, device="cuda")
    k[0, 0, 0], k[1, 0, 0], k[2, 0, :3] = 3e38, -1e30, torch.tensor([float("inf"), float("nan"), 1.0])
    k[3, 0, 0] = 1e-42
    want = K.write(oracle_cache(c), *arrays(s), f64(k), f64(k * 0))
    rn.kv_cache_write(c, s, k, k * 0)
    same_cache(c, want)
    got, _ = rn.kv_cache_read(c, s, 4, out_dtype=torch.float32)
    assert torch.isnan(got[2, 0, 1]) and got[2, 0, 0] == got[0, 0, 0] == 448 * 2.0 ** 119
    wk, _ = K.read(want, *arrays(s), 4)
    assert np.array_equal(f64(got), wk, equal_nan=True)


# --------------------------------------------------------------- calls in earnest
def test_strided_rows():
    H, G, D, T = 2, 4, 128, 45
    c, s, _ = make([100, 45], [20, 25], H, D, seed=8)
    joint = randn(T, (G * H + 2 * H) * D + 8)
    q = joint[:, :G * H * D].view(T, G * H, D)
    k = joint[:, G * H * D:(G + 1) * H * D].unflatten(1, (H, D))
    v = joint[:, (G + 1) * H * D:(G + 2) * H * D].unflatten(1, (H, D))
    assert not q.is_contiguous() and not k.is_contiguous()
    want = K.write(oracle_cache(c), *arrays(s), f64(k), f64(v))
    rn.kv_cache_write(c, s, k, v)
    same_cache(c, want)
    assert torch.equal(rn.kv_attention(q, c, s), rn.kv_attention(q.contiguous(), c, s))


@pytest.mark.parametrize("new", [1, 40])
def test_rows_of_no_sequence_stay(new):
    import ctypes
    lib = rn._load()
    c, s, T = make([100, 70], [new, new], 2, 64, seed=9)
    rows = T + 7
    s.starts += 3                                  # rows 0 .. 2 and the last four belong to nobody
    cs, qs = rn._kv_args(c, s, rows, 0)
    q = randn(rows, 4, 64)
    p = lambda t: ctypes.c_void_p(t.data_ptr())
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    out = torch.full((rows, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((rows, 4), 7.0, device="cuda")
    n = ctypes.c_size_t(rn.kv_attention_workspace_bytes(rows, 4, 2, 2, 64))
    ws = torch.full((n.value,), 0xFF, dtype=torch.uint8, device="cuda")
    assert lib.rn_kv_attention(p(q), 0, 256, 4, cs, qs, 0.125, 1, 0, 0.0, None, p(out), p(lse), p(ws), ctypes.byref(n),
                               stream) == 0
    inside = slice(3, 3 + T)
    assert (out[:3] == 7).all() and (out[3 + T:] == 7).all() and (lse[:3] == 7).all() and (lse[3 + T:] == 7).all()
    want = K.attention(f64(q), oracle_cache(c), *arrays(s), 0.125)
    assert np.isnan(want["out"][:3]).all()
    check(out, lse, want, 64)
    kk = torch.full((rows, 2, 64), 7.0, device="cuda")
    vv = kk.clone()
    assert lib.rn_kv_cache_read(cs, qs, p(kk), p(vv), 1, stream) == 0
    wk, wv = K.read(oracle_cache(c), *arrays(s), rows)
    for got, w in ((kk, wk), (vv, wv)):
        assert (got[:3] == 7).all() and (got[3 + T:] == 7).all() and np.array_equal(f64(got[inside]), w[inside])
    want = K.write(oracle_cache(c), *arrays(s), f64(q)[:, :2], f64(q)[:, 2:])
    rn.kv_cache_write(c, s, q[:, :2], q[:, 2:])
    same_cache(c, want)


def test_same_result_again_and_whatever_the_workspace_holds():
    for new in (1, 3, 50):
        c, s, T = make([3000, 500, 64], [new] * 3, 4, 128, seed=10)
        q = randn(T, 32, 128)
        ws = torch.full((rn.kv_attention_workspace_bytes(T, 32, 3, 4, 128),), 0xFF, dtype=torch.uint8, device="cuda")
        a = rn.kv_attention(q, c, s, workspace=ws)
        b = rn.kv_attention(q, c, s, workspace=ws)
        ws.zero_()
        assert torch.equal(a, b) and torch.equal(a, rn.kv_attention(q, c, s, workspace=ws))


def test_shared_pages_are_read_by_all():
    c, s, T = make([256, 256, 256], [1, 1, 1], 2, 128, seed=11)
    s.table[1:] = s.table[0]
    q = randn(1, 8, 128).expand(3, 8, 128).contiguous()
    out = rn.kv_attention(q, c, s)
    check(out, None, reference(q, c, s), 128)
    # three sequences are dealt to workers differently, so their sums round differently
    assert (out[0].float() - out[1].float()).abs().max() <= 2.0 ** -7 * out.float().abs().max()


def test_what_arrays_may_hold():
    # lengths below 0 and beyond the table, page numbers that are none, rows beyond the tensors
    c, s, T = make([300, 128, 64], [1, 2, 30], 2, 64, seed=12)
    clean = rn.KVCache(*(t.clone() for t in (c.k, c.v, c.k_scales, c.v_scales)))
    s.lens[:] = torch.tensor([2 ** 31 - 1, -5, 10 ** 6], dtype=torch.int32)
    s.table[0, 1:] = torch.tensor([-2 ** 31, 2 ** 31 - 1, c.k.shape[0], -1], dtype=torch.int32)[:s.table.shape[1] - 1]
    s.starts[3] = 2 ** 31 - 1
    q = randn(T, 4, 64)
    for causal in (True, False):
        out = rn.kv_attention(q, c, s, causal=causal)
        assert (out[1:3] == 0).all()
    rn.kv_cache_read(c, s, T)
    rn.kv_cache_write(c, s, q[:, :2], q[:, 2:])
    assert torch.equal(c.k, clean.k) and torch.equal(c.k_scales, clean.k_scales)   # no row has a cached position


@pytest.mark.parametrize("new", [1, 30])
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 40, 2 ** 30, 300, 299])
def test_windows_as_long_as_the_sequence(new, window):
    c, s, T = make([300, 40], [new, new], 2, 64, seed=14)
    q = randn(T, 4, 64)
    out = rn.kv_attention(q, c, s, window=window)
    check(out, None, reference(q, c, s, window=min(window, 10 ** 6)), 64)
    if window >= 300:
        assert torch.equal(out, rn.kv_attention(q, c, s))


@pytest.mark.parametrize("group", [37, 100, 300])
def test_large_groups(group):
    c, s, T = make([200, 64, 5], [1, 2, 1], 1, 64, seed=15)
    q = randn(T, group, 64)
    check(rn.kv_attention(q, c, s), None, reference(q, c, s), 64)


def test_no_rows():
    c, s, _ = make([100], [1], 2, 64)
    s.starts.zero_()
    q = torch.empty(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    assert rn.kv_attention(q, c, s).shape == (0, 4, 64)
    k, v = rn.kv_cache_read(c, s, 0)
    assert k.shape == v.shape == (0, 2, 64)
    rn.kv_cache_write(c, s, k, v)


def test_offsets_past_32_bits():
    pages, H, D = 40000, 8, 256                     # 5 GB of keys, 5 GB of values
    c = rn.kv_cache_alloc(pages, H, D)
    lens, news = [130, 70], [70, 1]
    table = torch.tensor([[pages - 1, 3, pages - 2], [pages - 7, pages - 3, -1]], dtype=torch.int32, device="cuda")
    ones = lambda t: torch.tensor(t, dtype=torch.int32, device="cuda")
    full = rn.KVSequences(table, ones([0, 130, 200]), ones(lens))
    k, v = randn(200, H, D, seed=1), randn(200, H, D, seed=2)
    rn.kv_cache_write(c, full, k, v)
    gk, gv = rn.kv_cache_read(c, full, 200, out_dtype=torch.float32)
    for got, x in ((gk, k), (gv, v)):
        # half a step of 3 mantissa bits, or of the subnormal codes under a page's scale
        assert ((got - x.float()).abs() <= x.float().abs() * 2.0 ** -4 + 2.0 ** -10 * x.float().abs().max() / 224).all()
    seqs = rn.KVSequences(table, ones([0, 70, 71]), ones(lens))
    q = randn(71, 2 * H, D, seed=3)
    check(rn.kv_attention(q, c, seqs), None, reference(q, c, seqs), D)


@pytest.mark.parametrize("H,G,D", [(2, 4, 128), (1, 8, 64), (2, 2, 256)])
def test_a_prompt_and_then_tokens(H, G, D):
    """As a server runs them: prompts of two sequences in parts, then tokens one by one from a captured step."""
    lens = [0, 0]
    pages = 10
    c = rn.kv_cache_alloc(pages, H, D)
    table = torch.tensor([[7, 2, 9, 0], [4, 1, 8, 3]], dtype=torch.int32, device="cuda")
    want_c = oracle_cache(c)

    def step(news, seed):
        for b in range(2):
            lens[b] += news[b]
        T = sum(news)
        s = rn.KVSequences(table, torch.tensor([0, news[0], T], dtype=torch.int32, device="cuda"),
                           torch.tensor(lens, dtype=torch.int32, device="cuda"))
        return s, randn(T, H * G, D, seed=seed), randn(T, H, D, seed=seed + 1), randn(T, H, D, seed=seed + 2, std=0.5)

    for i, news in enumerate(([50, 7], [20, 70], [3, 1])):
        s, q, k, v = step(news, 10 * i)
        rn.kv_cache_write(c, s, k, v)
        out, lse = rn.kv_attention(q, c, s, return_lse=True)
        want_c = K.write(want_c, *arrays(s), f64(k), f64(v))
        same_cache(c, want_c)
        check(out, lse, K.attention(f64(q), want_c, *arrays(s), D ** -0.5), D)

    # the step of a token each, captured: it follows the arrays
    s, q, k, v = step([1, 1], 100)
    ws = torch.empty(rn.kv_attention_workspace_bytes(2, H * G, 2, H, D), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        rn.kv_cache_write(c, s, k, v)
        rn.kv_attention(q, c, s, workspace=ws)
    torch.cuda.current_stream().wait_stream(side)
    graphs = []
    for _ in range(2):                              # two graphs on one workspace, replayed in turn
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            rn.kv_cache_write(c, s, k, v)
            out, lse = rn.kv_attention(q, c, s, return_lse=True, workspace=ws)
        graphs.append((g, out, lse))
    want_c = K.write(want_c, *arrays(s), f64(k), f64(v))
    for i in range(70):
        if i:
            s.lens += 1
            for t, seed, std in ((q, 0, 1.0), (k, 1, 1.0 + i / 20), (v, 2, 0.5)):
                t.copy_(randn(*t.shape, seed=200 + 10 * i + seed, std=std))
            want_c = K.write(want_c, *arrays(s), f64(k), f64(v))
        g, out, lse = graphs[i % 2]
        g.replay()
        if i % 9 == 0 or i > 66:
            torch.cuda.synchronize()
            same_cache(c, want_c)
            check(out, lse, K.attention(f64(q), want_c, *arrays(s), D ** -0.5), D)


def test_other_stream():
    c, s, T = make([700, 300], [1, 40], 2, 128, seed=13)
    q, k = randn(T, 8, 128), randn(T, 2, 128)
    twin = rn.KVCache(*(t.clone() for t in (c.k, c.v, c.k_scales, c.v_scales)))
    rn.kv_cache_write(twin, s, k, k)
    want = rn.kv_attention(q, twin, s)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        big = torch.empty(1 << 28, device="cuda").normal_()   # the side stream is behind
        rn.kv_cache_write(c, s, k, k)
        out = rn.kv_attention(q, c, s)
    side.synchronize()
    assert big is not None and torch.equal(out, want)


def test_calls_on_two_streams_at_once():
    """Reads and attentions of one cache, of few and of many rows a sequence, each call with a workspace of its own."""
    calls = []
    for i, new in enumerate(([1, 1, 1], [40, 2, 100])):
        c, s, T = make([3000, 150, 700], new, 2, 128, seed=20 + i)
        calls.append((c, s, T, randn(T, 8, 128, seed=i)))
    want = [(rn.kv_attention(q, c, s), *rn.kv_cache_read(c, s, T)) for c, s, T, q in calls]
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, (c, s, T, q) in enumerate(calls):
            with torch.cuda.stream(streams[i]):
                got[i].append((rn.kv_attention(q, c, s), *rn.kv_cache_read(c, s, T)))
    torch.cuda.synchronize()
    for i in range(2):
        for one in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(one, want[i]))
