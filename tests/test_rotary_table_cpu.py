"""Tables of cosines and sines: how many positions they may have."""
import numpy as np
import pytest

from paged_kv_cache_243_gb300 import _build, binding as B


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()


@pytest.mark.parametrize("positions", [2 ** 31 - 65535, 2 ** 31 - 1])
def test_positions_that_32_bits_do_not_count(positions):
    # (nothing is launched, so the address is never used)
    w = np.ones(8)
    with pytest.raises(B.PkvError) as e:
        B.rotary_table(0x10000, positions, 16, w.ctypes.data, 1.0, 0)
    assert e.value.status == B.ERR_UNSUPPORTED


@pytest.mark.parametrize("positions", [-1, 2 ** 31, 2 ** 32 + 10])
def test_the_wrapper_refuses_before_it_allocates(positions):
    from paged_kv_cache_243_gb300 import rotary_table
    with pytest.raises(ValueError):
        rotary_table(positions, 16)
