"""GPU parity of the attention over the paged 8-bit cache where its numbers or its parts lie far apart."""
import pytest
import torch

import mxfp8_quantization_gb300 as rn
from kv_check import check, make, randn, reference

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _no_device_error():
    yield
    assert rn.device_error() == 0


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
