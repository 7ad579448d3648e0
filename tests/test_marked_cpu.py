"""The marked batches' bound rejects what they are made to show: an oracle result with one tile left
out, taken twice, or with another tile's values or keys, whatever the output's type."""
import numpy as np
import pytest
import torch

from marked_batch import ALONE, PREFIX, MarkedRows, layout
from shared_batch import KINDS, TORCH


@pytest.mark.parametrize("kind", sorted(KINDS))
@pytest.mark.parametrize("rows,g", [(3, 2), (30, 4)])
def test_the_bound_rejects_a_tile_lost_doubled_or_mixed_up(kind, rows, g):
    src = KINDS[kind][2]
    some = [0, 1, 2] if rows == 3 else [0, 6, 29]
    group = [0] * len(some) + [-1] * len(ALONE)
    m = MarkedRows(kind, 64, group, [PREFIX], [PREFIX + layout(rows)[i] for i in some] + ALONE, g, src)
    half = torch.finfo(TORCH[src]).eps / 2
    for bound in (m.bound(half * half, 0), m.bound(half, torch.finfo(TORCH[src]).eps)):
        shown = 0
        for b in range(len(group)):
            # (a result that is off by its rounding, too, still has to be outside)
            limit = 2 * bound[b]
            if m.lens[b] <= 128:
                continue      # one tile: nothing to lose it among
            for t0, t1 in m.visits(b):
                for got in (m.with_weight(b, t0, t1, 0), m.with_weight(b, t0, t1, 2)):
                    assert (np.abs(got - m.out[b]) > limit).any(), (b, t0)
                other = (t0 + 128 if t1 + 128 <= m.lens[b] else t0 - 128) if t1 - t0 == 128 else 0
                assert (np.abs(m.with_values_of(b, t0, t1, other) - m.out[b]) > limit).any(), (b, t0)
                shown += (np.abs(m.with_keys_of(b, t0, t1, other) - m.out[b]) > limit).any()
        assert shown > 0      # keys: of the tiles that a head of the row looks for
