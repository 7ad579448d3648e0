"""NaN in queries, keys and scales that a row attends to reaches that row's output, whatever the
split of the work; NaN behind a row's length does not."""
import numpy as np
import pytest
import torch

from shared_batch import TORCH, SharedBatch

pytestmark = pytest.mark.gpu

KINDS4 = ["f16", "bf16", "i8t", "i8g", "u4t"]
SPLITS = [0, 1, 2, 7, 152]


def batch(kind, rows, seed):
    """A shared prefix of 300 tokens, rows with 1 to 150 tokens of their own, one without a group."""
    own = [1, 150, 17, 64] + [int(n) for n in np.random.default_rng(seed).integers(1, 90, rows - 4)]
    return SharedBatch(kind, 2, 64, 64, [(300, own)], alone=[1, 70], seed=seed)


def spoil(sb, b, t, h):
    """Token t of row b, kv head h: a key whose scores are NaN."""
    page, slot = int(sb.table[b, t // sb.ps]), t % sb.ps
    c = sb.cache
    if c.kv_sz is None:
        c.k_pages[page, h, slot, 5] = float("nan")
    else:
        c.kv_sz[page, h, slot * c.kv_sz.shape[2] // sb.ps, 0] = float("nan")


@pytest.mark.parametrize("kind", KINDS4)
@pytest.mark.parametrize("rows", [4, 12])      # few and many query rows of the prefix at G = 4 and 3
@pytest.mark.parametrize("splits", SPLITS)
def test_a_nan_query_gives_nan_and_touches_no_other_row(kind, rows, splits):
    sb = batch(kind, rows, 40 + rows)
    g = 1 if rows == 4 else 4
    q, _ = sb.queries(g)
    for dt in (torch.float32, TORCH[sb.src]):
        ref = sb.run(q, dt, num_splits=splits)
        bad = q.clone()
        b, h = int(np.flatnonzero(sb.group == 0)[1]), 2 * g - 1
        bad[b, h, 3] = float("nan")
        out = sb.run(bad, dt, num_splits=splits)
        assert bool(torch.isnan(out[b, h]).all())
        out[b, h] = ref[b, h]
        assert torch.equal(out, ref)


@pytest.mark.parametrize("kind", KINDS4)
@pytest.mark.parametrize("rows", [4, 12])
@pytest.mark.parametrize("splits", SPLITS)
def test_a_nan_key_gives_nan_to_the_rows_that_attend_to_it(kind, rows, splits):
    sb = batch(kind, rows, 50 + rows)
    g = 1 if rows == 4 else 4
    q, _ = sb.queries(g)
    ref = sb.run(q, num_splits=splits)
    # the only token of a row without a group, and the only own token of a row of the group
    alone = int(np.flatnonzero((sb.group < 0) & (sb.lens == 1))[0])
    one = int(np.flatnonzero((sb.group == 0) & (sb.lens == 301))[0])
    spoil(sb, alone, 0, 1)
    spoil(sb, one, 300, 0)
    out = sb.run(q, num_splits=splits)
    assert bool(torch.isnan(out[alone, g:]).all()) and bool(torch.isnan(out[one, :g]).all())
    out[alone, g:], out[one, :g] = ref[alone, g:], ref[one, :g]
    assert torch.equal(out, ref)


@pytest.mark.parametrize("kind", ["bf16", "i8t", "u4t"])
@pytest.mark.parametrize("splits", SPLITS)
def test_a_nan_key_of_the_prefix_reaches_every_row_of_its_group(kind, splits):
    sb = batch(kind, 12, 61)
    q, _ = sb.queries(4)
    ref = sb.run(q, num_splits=splits)
    spoil(sb, int(np.flatnonzero(sb.group == 0)[0]), 130, 1)
    out = sb.run(q, num_splits=splits)
    rows = torch.from_numpy(np.flatnonzero(sb.group == 0)).cuda()
    assert bool(torch.isnan(out[rows, 4:]).all())
    out[rows, 4:] = ref[rows, 4:]
    assert torch.equal(out, ref)
