"""Host-side refusals of the paged key/value cache's entry points (no GPU is touched), and of the binding."""
import ctypes

import pytest
import torch

import mxfp8_quantization_gb300 as rn
from mxfp8_quantization_gb300 import _build

P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return rn._load()


def cache(**kw):
    c = dict(k=0x1000, v=0x2000, k_scales=0x3001, v_scales=0x4003, pages=4, heads=2, dim=128)
    c.update(kw)
    return rn._KVCache(**c)


def seqs(**kw):
    s = dict(table=0x5000, starts=0x6000, lens=0x7000, sequences=3, table_width=5, tokens=7)
    s.update(kw)
    return rn._KVSeqs(**s)


BAD_CACHE = [(dict(k=None), 1), (dict(v=None), 1), (dict(k_scales=None), 1), (dict(v_scales=None), 1),
             (dict(pages=0), 1), (dict(heads=0), 1), (dict(dim=0), 1), (dict(dim=-64), 1), (dict(dim=96), 2),
             (dict(dim=512), 2), (dict(heads=65536), 2), (dict(pages=1 << 31), 2), (dict(k=0x1008), 2),
             (dict(v=0x2004), 2)]
BAD_SEQS = [(dict(sequences=-1), 1), (dict(tokens=-1), 1), (dict(table_width=-1), 1), (dict(table=None), 1),
            (dict(starts=None), 1), (dict(lens=None), 1), (dict(starts=0x6002), 2), (dict(lens=0x7001), 2),
            (dict(table=0x5002), 2), (dict(sequences=(1 << 24) + 1), 2), (dict(tokens=1 << 30), 2),
            (dict(table_width=1 << 25), 2)]


def write(lib, c, s, k=0x10000, v=0x20000, dt=0, ks=256, vs=256):
    return lib.rn_kv_cache_write(P(k), P(v), dt, ks, vs, c, s, None)


def read(lib, c, s, k=0x10000, v=0x20000, dt=0):
    return lib.rn_kv_cache_read(c, s, P(k), P(v), dt, None)


def attend(lib, c, s, q=0x10000, dt=0, stride=1024, heads=8, scale=1.0, window=0, cap=0.0, slopes=0, out=0x20000, lse=0,
           ws=0x30000, n=1 << 40):
    size = ctypes.c_size_t(n)
    return lib.rn_kv_attention(P(q), dt, stride, heads, c, s, scale, 1, window, cap, P(slopes), P(out), P(lse), P(ws),
                               ctypes.byref(size), None)


@pytest.mark.parametrize("call", [write, read, attend])
def test_bad_caches_and_sequences(lib, call):
    for kw, st in BAD_CACHE:
        assert call(lib, cache(**kw), seqs()) == st, kw
    for kw, st in BAD_SEQS:
        assert call(lib, cache(), seqs(**kw)) == st, kw
    assert call(lib, None, seqs()) == 1 and call(lib, cache(), None) == 1


@pytest.mark.parametrize("call", [write, read, attend])
def test_bad_dtype(lib, call):
    assert call(lib, cache(), seqs(), dt=5) == 1


def test_write_refusals(lib):
    c, s = cache(), seqs()
    assert write(lib, c, s, k=0) == 1 and write(lib, c, s, v=0) == 1
    assert write(lib, c, s, ks=248) == 1 and write(lib, c, s, vs=0) == 1     # rows overlap
    assert write(lib, c, s, ks=260) == 2                                     # 520 bytes
    assert write(lib, c, s, ks=260, vs=258, dt=1) == 2
    assert write(lib, c, s, k=0x10008) == 2 and write(lib, c, s, v=0x20002) == 2
    assert write(lib, c, s, ks=1 << 40) == 2


def test_read_refusals(lib):
    c, s = cache(), seqs()
    assert read(lib, c, s, k=0) == 1 and read(lib, c, s, v=0) == 1
    assert read(lib, c, s, k=0x10008) == 2 and read(lib, c, s, v=0x20004) == 2


def test_grids_past_31_bits(lib):
    for call in (write, read):
        wide = dict(ks=1 << 24, vs=1 << 24) if call is write else {}
        for heads, kw in ((65535, dict(sequences=8193)), (65535, dict(tokens=1 << 21)), (64, dict(tokens=(1 << 30) - 1))):
            assert call(lib, cache(heads=heads), seqs(**kw), **wide) == 2, kw


def test_attention_refusals(lib):
    c, s = cache(), seqs()
    nan, inf = float("nan"), float("inf")
    assert attend(lib, c, s, q=0) == 1 and attend(lib, c, s, out=0) == 1
    assert attend(lib, c, s, heads=7) == 1 and attend(lib, c, s, heads=0) == 1
    for scale in (0.0, -1.0, nan, inf):
        assert attend(lib, c, s, scale=scale) == 1
    for cap in (-1.0, nan, inf, 1e-38):
        assert attend(lib, c, s, cap=cap) == 1
    assert attend(lib, c, s, window=-1) == 1
    assert attend(lib, c, s, stride=1016) == 1
    assert attend(lib, c, s, dt=1) == 2                                      # fp32 queries
    assert attend(lib, c, s, stride=1028) == 2
    assert attend(lib, c, s, heads=2 * 8192, stride=2 * 8192 * 128) == 2     # group of 8192
    assert attend(lib, c, s, q=0x10004) == 2 and attend(lib, c, s, out=0x20008) == 2
    assert attend(lib, c, s, lse=0x40001) == 2 and attend(lib, c, s, slopes=0x40002) == 2
    assert attend(lib, c, s, ws=0x30008) == 2
    assert attend(lib, c, seqs(tokens=1 << 28)) == 2                         # 2^30 rows of a head
    for kw in (dict(scale=1.1e30), dict(cap=1.1e30)):
        assert attend(lib, c, s, **kw) == 1
    need = rn.kv_attention_workspace_bytes(7, 8, 3, 2, 128)
    assert need > 0
    assert attend(lib, c, s, ws=0) == 3 and attend(lib, c, s, n=need - 1) == 3
    size = ctypes.c_size_t(0)
    assert lib.rn_kv_attention(None, 0, 0, 8, c, s, 1.0, 1, 0, 0.0, None, None, None, None, None, None) == 1
    assert lib.rn_kv_attention(None, 0, 0, 8, c, s, 1.0, 1, 0, 0.0, None, None, None, None, ctypes.byref(size), None) == 0
    assert size.value == need


def test_workspace_query_of_any_size(lib):
    for dim in (64, 128, 192, 256):
        sizes = {rn.kv_attention_workspace_bytes(t, h, b, 2, dim)
                 for t, h, b in ((0, 2, 0), (1, 2, 1), (1000, 64, 3), (1 << 20, 8, 4096))}
        assert len(sizes) == 1 and 0 < sizes.pop() < 1 << 27


class Fake:
    """A tensor as the binding's checks see it."""
    is_cuda, device = True, torch.device("cuda", 0)

    def __init__(self, dtype, *shape, stride=None, contiguous=True):
        self.dtype, self.shape, self._c = dtype, torch.Size(shape), contiguous
        n, st = 1, []
        for d in reversed(shape):
            st.insert(0, n)
            n *= d
        self._s = stride or tuple(st)

    def dim(self):
        return len(self.shape)

    def stride(self, i=None):
        return self._s if i is None else self._s[i]

    def numel(self):
        return self.shape.numel()

    def is_contiguous(self):
        return self._c

    def data_ptr(self):
        return 0x1000


U8, I32, BF, F32 = torch.uint8, torch.int32, torch.bfloat16, torch.float32


def fakes():
    return (rn.KVCache(Fake(U8, 4, 2, 64, 128), Fake(U8, 4, 2, 128, 64), Fake(U8, 4, 2), Fake(U8, 4, 2)),
            rn.KVSequences(Fake(I32, 3, 5), Fake(I32, 4), Fake(I32, 3)))


@pytest.fixture
def device0(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(rn, "_raw_stream", lambda dev: 0)


BAD_TENSORS = [("cache", "k", Fake(U8, 4, 2, 32, 128), "cache.k"), ("cache", "k", Fake(F32, 4, 2, 64, 128), "cache.k"),
               ("cache", "v", Fake(U8, 4, 2, 64, 128), "cache.v"), ("cache", "v", None, "cache.v"),
               ("cache", "k_scales", Fake(U8, 4, 3), "cache.k_scales"),
               ("cache", "v_scales", Fake(U8, 4, 2, contiguous=False), "cache.v_scales"),
               ("seqs", "table", Fake(torch.int64, 3, 5), "seqs.table"), ("seqs", "table", Fake(I32, 3), "seqs.table"),
               ("seqs", "starts", Fake(I32, 3), "seqs.starts"), ("seqs", "lens", Fake(I32, 4), "seqs.lens"),
               ("seqs", "lens", None, "seqs.lens")]


@pytest.mark.parametrize("which,name,bad,text", BAD_TENSORS)
def test_binding_names_the_bad_tensor(lib, device0, which, name, bad, text):
    c, s = fakes()
    setattr(c if which == "cache" else s, name, bad)
    x = Fake(BF, 7, 2, 128)
    for call in (lambda: rn.kv_cache_write(c, s, x, x), lambda: rn.kv_cache_read(c, s, 7),
                 lambda: rn.kv_attention(x, c, s)):
        with pytest.raises(rn.RNError, match=text):
            call()


def test_binding_refuses_rows(lib, device0):
    c, s = fakes()
    good = Fake(BF, 7, 2, 128)
    for bad, text in ((None, "required"), (Fake(BF, 7, 3, 128), "shape"), (Fake(BF, 7, 2, 64), "shape"),
                      (Fake(torch.float16, 7, 2, 128), "float16"), (torch.zeros(7, 2, 128), "CUDA"),
                      (Fake(BF, 7, 2, 128, stride=(256, 128, 2)), "contiguous"),
                      (Fake(BF, 7, 2, 128, stride=(512, 256, 1)), "contiguous")):
        with pytest.raises(rn.RNError, match=text):
            rn.kv_cache_write(c, s, bad, good)
        with pytest.raises(rn.RNError, match=text):
            rn.kv_attention(bad, c, s)
    for bad in (Fake(BF, 7), Fake(BF, 7, 2, 128, 1), "q"):
        with pytest.raises(rn.RNError, match="shape|CUDA"):
            rn.kv_attention(bad, c, s)
        with pytest.raises(rn.RNError, match="shape|CUDA"):
            rn.kv_cache_write(c, s, bad, good)
    with pytest.raises(rn.RNError, match="multiple of 2"):
        rn.kv_attention(Fake(BF, 7, 3, 128), c, s)
    with pytest.raises(rn.RNError, match="negative"):
        rn.kv_cache_read(c, s, -1)
    with pytest.raises(rn.RNError, match="v must have shape"):
        rn.kv_cache_write(c, s, good, Fake(BF, 6, 2, 128))
    with pytest.raises(rn.RNError, match="v must be"):
        rn.kv_cache_write(c, s, good, Fake(F32, 7, 2, 128))
    with pytest.raises(rn.RNError, match="q must be"):
        rn.kv_attention(Fake(F32, 7, 2, 128), c, s)
    with pytest.raises(rn.RNError, match="slopes"):
        rn.kv_attention(good, c, s, slopes=Fake(F32, 3))
    with pytest.raises(rn.RNError, match="KVCache"):
        rn.kv_attention(good, s, s)
    with pytest.raises(rn.RNError, match="KVSequences"):
        rn.kv_attention(good, c, c)
