"""Numbers that the binding of the paged key/value cache hands to the library as 64-bit integers (no GPU is touched)."""
import types

import pytest
import torch

import mxfp8_quantization_gb300 as rn
from mxfp8_quantization_gb300 import _build
from test_cpu_kv import BF, Fake, fakes


@pytest.fixture
def calls(monkeypatch):
    """The arguments of the library's calls, which do nothing."""
    _build.build()
    rn._load()
    rn._kv_attention_bytes(0, 2, 0, 2, 128)
    seen = []
    call = lambda *a: seen.append(a) or 0
    monkeypatch.setattr(rn, "_lib", types.SimpleNamespace(rn_kv_attention=call, rn_kv_cache_read=call))
    monkeypatch.setattr(rn, "_raw_stream", lambda dev: 0)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch, "empty", lambda shape, dtype=None, device=None: Fake(
        dtype, *(shape if isinstance(shape, tuple) else (shape,))))
    monkeypatch.setattr(Fake, "element_size", lambda self: 1, raising=False)
    return seen


@pytest.mark.parametrize("window,passed", [(0, 0), (5, 5), (2 ** 63 - 1, 2 ** 63 - 1), (2 ** 63, 2 ** 63 - 1),
                                           (2 ** 64 + 5, 2 ** 63 - 1), (-1, -1), (-2 ** 64, -1)])
def test_windows_of_any_length(calls, window, passed):
    c, s = fakes()
    rn.kv_attention(Fake(BF, 7, 2, 128), c, s, window=window)
    assert calls[0][8] == passed


@pytest.mark.parametrize("tokens,text", [(-1, "negative"), (-2 ** 64, "negative"), (2 ** 30, "below"), (2 ** 64 + 3, "below")])
def test_numbers_of_tokens(calls, tokens, text):
    c, s = fakes()
    with pytest.raises(rn.RNError, match=text):
        rn.kv_cache_read(c, s, tokens)
    assert not calls
