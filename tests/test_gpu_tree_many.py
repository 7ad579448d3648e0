"""Trees in batches of so many sequences that the plan leaves room for fewer tiles of K and V in flight, down to
one: from 288 sequences on 16-bit caches of 128 channels, from 128 on per-token INT8 ones. Parts of many visits, one
and two row tiles, drafts that span tiles, values that are no numbers, pages that are missing."""
import numpy as np
import pytest
import torch

from shared_batch import TORCH, int_dev
from test_gpu_tree import spoil
from tree_batch import TreeBatch

pytestmark = pytest.mark.gpu


def many(kind, B, T, seed, long=(128 * 37 + 20, 128 * 22 + 71, 128 * 9 + 128, 128 * 30 + 100), tree="tree"):
    """B short sequences with a few drafts, but for some long ones with T each."""
    rng = np.random.default_rng([95, seed])
    lens = rng.integers(0, 40, B)
    lens[:len(long)] = long
    tb = TreeBatch(kind, 1, 128, 64 if kind == "i8g" else 16, lens, T, seed=seed, tree=tree)
    tb.drafts = np.where(tb.lens > 1000, T, np.minimum(tb.lens, rng.integers(0, 4, B))).astype(np.int32)
    tb.drafts_dev = int_dev(tb.drafts)
    return tb


FEW_AND_MORE = [(3, 4), (30, 4), (200, 4)]     # transposed, one row tile, two of them and what is left of that


@pytest.mark.parametrize("kind,B,T,g", [(k, n, *x) for k, n in (("bf16", 287), ("bf16", 300), ("i8t", 127), ("i8t", 300), ("i8g", 300))
                                        for x in FEW_AND_MORE] +
                         [(k, n, *x) for k, n in (("f16", 1024), ("i8t", 1024), ("u4t", 800)) for x in FEW_AND_MORE[:2]])
@pytest.mark.parametrize("splits", [2, 0])
def test_many_sequences_some_of_them_long(kind, B, T, g, splits):
    tb = many(kind, B, T, T + B)
    q, qf = tb.tree_queries(g)
    for dt in (TORCH[tb.src], torch.float32):
        ref = tb.tree_run(q, dt, num_splits=splits)
        tb.tree_check(ref, qf, g)
        for _ in range(3):
            assert torch.equal(tb.tree_run(q, dt, num_splits=splits), ref)
    assert int(tb.status.item()) == 0


@pytest.mark.parametrize("kind,B", [("bf16", 300), ("f16", 400), ("i8t", 300)])
@pytest.mark.parametrize("T,g", FEW_AND_MORE)
@pytest.mark.parametrize("splits,value", [(2, float("nan")), (0, float("inf"))])
def test_no_number_among_many_sequences(kind, B, T, g, splits, value):
    tb = many(kind, B, T, T + B)
    q, qf = tb.tree_queries(g)
    for dt in (TORCH[tb.src], torch.float32):
        ref = tb.tree_run(q, dt, num_splits=splits)
        bound = torch.from_numpy(tb.tree_bound(qf, g, dt)[1]).cuda()
        kept = tb.cache.v_pages.clone(), None if tb.cache.kv_sz is None else tb.cache.kv_sz.clone()
        want = ref.clone()
        hit = [(int(b), j) for b in np.flatnonzero(tb.lens > 1000) for j in (T - 1, T // 2)]
        for b, j in hit:
            spoil(tb, b, int(tb.lens[b]) - T + j, 0, "v", value)
        out = tb.tree_run(q, dt, num_splits=splits)
        for b, j in hit:
            rows = torch.from_numpy(np.flatnonzero(tb.seen[b, :, j])).cuda()
            got = out[b, rows] if tb.cache.kv_sz is not None else out[b, rows][..., 5]
            assert not bool(torch.isfinite(got).any())
            if tb.cache.kv_sz is not None:
                want[b, rows] = out[b, rows]
            else:
                want[b, rows, :, 5] = out[b, rows, :, 5]
        same = torch.nan_to_num(out, nan=77.0) == torch.nan_to_num(want, nan=77.0)
        if tb.cache.kv_sz is not None:      # (other roundings: the sizes of the tile's values are others)
            same |= (out.double() - ref.double()).abs() <= 2 * bound
        assert bool(same.all())
        tb.cache.v_pages.copy_(kept[0])
        if kept[1] is not None:
            tb.cache.kv_sz.copy_(kept[1])
    assert int(tb.status.item()) == 0


@pytest.mark.parametrize("kind,B", [("f16", 300), ("i8t", 300)])
@pytest.mark.parametrize("T,g", FEW_AND_MORE)
def test_missing_pages_among_many_sequences(kind, B, T, g):
    # pages in the middle of long sequences, one in whole tiles and one beside the drafts; what is in V's
    # place of them from before does not count
    from paged_kv_cache_243_gb300 import binding
    tb = many(kind, B, T, T + B + 1, tree="chain")
    q, qf = tb.tree_queries(g)
    table = tb.table.copy()
    for b in np.flatnonzero(tb.lens > 1000):
        L = int(tb.lens[b])
        gone = np.array([3, 16, 17, 60, (L - T) // 16 - 2])
        table[b, gone] = -1
        keep = ~np.isin(np.arange(L) // 16, gone)
        tb.k[b], tb.v[b] = tb.k[b][keep], tb.v[b][keep]
        tb.lens[b] = keep.sum()
    for dt in (TORCH[tb.src], torch.float32):
        for splits in (2, 0):
            out = tb.cache.tree_attention(q, int_dev(table), tb.lens_dev, draft_lens=tb.drafts_dev, out_dtype=dt,
                                          num_splits=splits, dev_status=tb.status)
            torch.cuda.synchronize()
            assert int(tb.status.item()) == binding.DEV_BAD_PAGE
            tb.tree_check(out, qf, g)
