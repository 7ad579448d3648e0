"""Limits of shared_prefix_attention that no device is needed to see."""
import pytest

from paged_kv_cache_243_gb300 import _build, binding as B


@pytest.mark.parametrize("page_size,max_pages", [(16, (1 << 27) - 1), (16, (1 << 27) - 16)])
def test_tables_whose_last_tile_ends_past_32_bits(page_size, max_pages):
    # the tile of the last tokens would end beyond 2^31 - 1
    _build.build()
    assert 2 ** 31 - 257 < page_size * max_pages < 2 ** 31
    cache = B.PkvCache(8, page_size, 1, 64, B.F16, B.QUANT_NONE, 0x1000, 0x2000, 0, 0, 0, 0)
    with pytest.raises(B.PkvError) as e:
        B.shared_prefix_attention(cache, 1, 1, 0x4000, B.F16, 0.125, 0x5000, max_pages, 0x6000, 0x7000, 0x8000, 1,
                                  0x9000, B.F32, 0, 0x10000, 1 << 30, 0, 0)
    assert e.value.status == B.ERR_UNSUPPORTED
