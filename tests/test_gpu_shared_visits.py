"""Every 128-token tile of every row counts once, with its own keys and values, however many of them a
block has: over the wraps of the visit descriptions, the rings and the parities."""
import numpy as np
import pytest
import torch

from marked_batch import ALONE, PREFIX, MarkedRows, layout
from shared_batch import KINDS, TORCH, SharedBatch, int_dev, to_dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", sorted(KINDS))
@pytest.mark.parametrize("rows,g", [(3, 2), (30, 4)])
def test_every_tile_counts_once(kind, rows, g):
    d, ps = 64, 64
    sb = SharedBatch(kind, 1, d, ps, [(PREFIX, layout(rows))], alone=ALONE, seed=rows)
    m = MarkedRows(kind, d, sb.group, sb.prefix, sb.lens, g, sb.src)
    # the first row of the group writes the prefix, the others what follows its whole pages
    first = int(np.flatnonzero(sb.group == 0)[0])
    start = np.where((sb.group == 0) & (np.arange(sb.B) != first), PREFIX // ps * ps, 0).astype(np.int32)
    count = (sb.lens - start).astype(np.int32)
    kv = np.zeros((2, sb.B, int(count.max()), 1, d), dtype=np.uint16)
    for b in range(sb.B):
        for i in range(2):
            kv[i, b, :count[b]] = m.bits[b][i][start[b]:]
    sb.cache.append(to_dev(kv[0], sb.src), to_dev(kv[1], sb.src), sb.table_dev, int_dev(start), int_dev(count),
                    dev_status=sb.status)
    q = to_dev(m.qbits, sb.src)
    half = torch.finfo(TORCH[sb.src]).eps / 2
    for dt in (torch.float32, TORCH[sb.src]):
        bound = m.bound(half * half, 0) if dt == torch.float32 else m.bound(half, torch.finfo(dt).eps)
        for splits in (1, 2, 5, 0):
            err = np.abs(sb.run(q, dt, num_splits=splits).double().cpu().numpy() - m.out)
            assert (err <= bound).all(), (dt, splits, float((err / bound).max()))
    assert int(sb.status.item()) == 0
