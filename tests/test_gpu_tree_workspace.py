"""Nothing outside a workspace of just the bytes that are asked for is written, and calls whose records fit 32 bits run."""
import numpy as np
import pytest
import torch

from shared_batch import TORCH, int_dev
from tree_batch import TreeBatch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["f16", "i8t"])
@pytest.mark.parametrize("T,g", [(2, 3), (4, 4), (5, 2), (17, 1), (9, 7), (33, 4), (100, 4)])
@pytest.mark.parametrize("splits", [1, 3, 11, 152])
def test_a_workspace_of_just_its_size(kind, T, g, splits):
    from paged_kv_cache_243_gb300 import binding as B
    tb = TreeBatch(kind, 2, 64, 16, [1500, 90, T, 700, 2600], T, drafts=[T, T, T, 1, T], seed=T)
    q, qf = tb.tree_queries(g)
    n = B.tree_workspace_bytes(tb.cache._desc, tb.B, T, 2 * g, splits)
    room = torch.full((n + (2 << 20),), 0xA5, dtype=torch.uint8, device="cuda")
    at = (1 << 20) + -room.data_ptr() % 256
    for dt in (TORCH[tb.src], torch.float32):
        room[at:at + n] = 0xFF
        tb.tree_check(tb.tree_run(q, dt, num_splits=splits, workspace=room[at:at + n]), qf, g)
        assert bool((room[:at] == 0xA5).all()) and bool((room[at + n:] == 0xA5).all())
    assert int(tb.status.item()) == 0


def test_records_of_more_than_a_gigabyte():
    # 8 million query rows of 128 channels, nearly all of which have nothing to attend to
    B, T, hkv, g = 1000, 128, 8, 8
    tb = TreeBatch("bf16", hkv, 128, 16, [400, 129, 300], T, seed=3)
    small, qf = tb.tree_queries(g)
    rows = [0, 511, 999]
    table, lens = np.full((B, tb.width), -1, dtype=np.int32), np.zeros(B, dtype=np.int32)
    table[rows], lens[rows] = tb.table, tb.lens
    drafts = np.zeros(B, dtype=np.int32)
    drafts[rows] = T
    mask = torch.zeros((B, *tb.mask.shape[1:]), dtype=torch.int64, device="cuda")
    q = torch.zeros((B, *small.shape[1:]), dtype=torch.bfloat16, device="cuda")
    q[rows], mask[rows] = small, tb.mask
    out = tb.cache.tree_attention(q, int_dev(table), int_dev(lens), mask, int_dev(drafts), out_dtype=torch.bfloat16,
                                  dev_status=tb.status)
    torch.cuda.synchronize()
    assert int(tb.status.item()) == 0
    tb.tree_check(out[rows], qf, g)
    out[rows] = 0
    assert not bool(out.any())
    del q, out, mask
    torch.cuda.empty_cache()
