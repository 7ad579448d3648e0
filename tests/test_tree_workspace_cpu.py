"""The workspace of tree_attention: what the kernels write, and no more."""
import pytest

from paged_kv_cache_243_gb300 import _build, binding as B


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()


def desc(hkv, d, kv=B.BF16, quant=B.QUANT_NONE):
    return B.PkvCache(8, 16, hkv, d, kv, quant, 0x1000, 0x2000, 0x3000 if quant else 0, 0, 0, 0)


@pytest.mark.parametrize("batch,T,hq,hkv,d", [(128, 256, 64, 8, 128), (24, 64, 32, 8, 128), (1024, 40, 8, 2, 64), (3, 7, 64, 8, 128)])
def test_one_record_for_a_query_row(batch, T, hq, hkv, d):
    splits = 152
    rows = batch * hkv * -(-T * hq // hkv // 32) * 32 + (splits + 1) * 256
    size = B.tree_workspace_bytes(desc(hkv, d), batch, T, hq, splits)
    places = batch * hkv * -(-T * hq // hkv // 256) * 16
    assert rows * (d + 2) * 4 <= size <= rows * (d + 2) * 4 + places + 1024


def test_a_workspace_serves_fewer_drafts_too():
    for g in (1, 4, 7):
        sizes = [B.tree_workspace_bytes(desc(2, 128), 6, T, 2 * g, 9) for T in range(1, 257)]
        assert sizes == sorted(sizes)


def test_no_workspace_for_a_call_that_is_refused():
    # (a caller, the wrapper among them, would make it first: 8 GB and more)
    ask = lambda batch, T: B.tree_workspace_bytes(desc(8, 128), batch, T, 64, 152)  # noqa: E731
    assert ask(1000, 128) > 1 << 31
    for batch, T in ((1024, 256), (1024, 255), (1023, 256)):
        with pytest.raises(B.PkvError):
            ask(batch, T)
