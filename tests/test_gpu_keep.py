"""Keeping accepted drafts: the tokens move bit for bit, and nothing else changes."""
import numpy as np
import pytest
import torch

import oracle
from oracle.quant import per_token_bbox_values
from oracle.quant4 import per_token_u4_bbox_values
from shared_batch import SharedBatch, int_dev

pytestmark = pytest.mark.gpu

FOUR = ["f16", "bf16", "i8t", "u4t"]


def parts(cache):
    return [x for x in (cache.k_pages, cache.v_pages, cache.kv_sz) if x is not None]


def raw(t):
    """Bits as numpy, [page][kv head][slot][...]."""
    return (t.view(torch.int16) if t.element_size() == 2 else t if t.element_size() == 1 else t.view(torch.int32)).cpu().numpy()


def check(sb, first, keep, lens, width=None, run=None):
    """keep: lists. Calls, and compares every part with the definition; returns the kept lengths."""
    K = width or max(1, max(len(k) for k in keep))
    arr = np.full((sb.B, K), -7, dtype=np.int32)
    for b, k in enumerate(keep):
        arr[b, :len(k)] = k
    want = [raw(x).copy() for x in parts(sb.cache)]
    for w in want:
        for b, k in enumerate(keep):
            at = lambda t: (sb.table[b, t // sb.ps], slice(None), t % sb.ps)  # noqa: E731
            moved = [w[at(first[b] + j)].copy() for j in k]
            for j, x in enumerate(moved):
                w[at(first[b] + j)] = x
    n = None if lens is None else int_dev(lens)
    (run or sb.cache.keep_tokens)(int_dev(arr), n, sb.table_dev, int_dev(first), dev_status=sb.status)
    torch.cuda.synchronize()
    assert int(sb.status.item()) == 0
    for x, w in zip(parts(sb.cache), want):
        assert np.array_equal(raw(x), w)


def random_keep(rng, T, n):
    return sorted(rng.choice(T, n, replace=False).tolist())


@pytest.mark.parametrize("kind", FOUR)
@pytest.mark.parametrize("d,hkv,ps", [(64, 1, 16), (128, 3, 48), (128, 8, 64)])
@pytest.mark.parametrize("T,n", [(1, 1), (7, 3), (64, 9), (64, 64), (200, 150), (256, 256), (256, 40)])
def test_tokens_move_bit_for_bit(kind, d, hkv, ps, T, n):
    rng = np.random.default_rng(T + n)
    ctx = [0, 1, 17, 100]
    sb = SharedBatch(kind, hkv, d, ps, [], alone=[c + T for c in ctx], seed=T)
    first = sb.lens - T
    counts = [n, max(0, n - 1), (n + 1) // 2, n]
    keep = [random_keep(rng, T, m) for m in counts]
    check(sb, first, keep, counts)


def test_nothing_kept_and_everything_in_place():
    sb = SharedBatch("f16", 2, 64, 16, [], alone=[40, 30], seed=1)
    first = sb.lens - 20
    check(sb, first, [[], []], [0, 0], width=5)
    check(sb, first, [list(range(20))] * 2, None)
    check(sb, first, [[0, 1, 2, 5, 6, 19]] * 2, None)


@pytest.mark.parametrize("kind", FOUR)
@pytest.mark.parametrize("d,ps", [(64, 16), (128, 48), (128, 256)])
def test_boxes_are_those_of_what_is_left(kind, d, ps):
    # bit-exact: boxes of the kept sequence as the oracle's quantiser restores it
    T = 40
    rng = np.random.default_rng(d + ps)
    sb = SharedBatch(kind, 3, d, ps, [], alone=[T, 70 + T, 16 + T, 300 + T, 48 + T], seed=ps, with_meta=True)
    first = sb.lens - T
    counts = [3, 0, 12, 33, 1]
    keep = [random_keep(rng, T, m) for m in counts]
    before = sb.cache.page_meta.clone()
    src = [sb.bits[b][0] for b in range(sb.B)]
    check(sb, first, keep, counts)
    touched = set()
    for b, k in enumerate(keep):
        f, end = int(first[b]), int(first[b]) + len(k)
        bits = np.concatenate([src[b][:f], src[b][f + np.array(k, dtype=int)]])
        x = np.float32(bits.view(np.float16)) if sb.src == "f16" else (bits.astype(np.uint32) << 16).view(np.float32)
        if kind == "i8t":
            x = per_token_bbox_values(*oracle.quantize_per_token(x))
        elif kind == "u4t":
            x = per_token_u4_bbox_values(*oracle.quantize_per_token_u4(x))
        if end == 0:
            continue
        mn, mx = oracle.page_bounding_boxes(x, ps)
        lo = max(0, f - 1) // ps
        pages = sb.table[b, lo:mn.shape[0]]
        touched |= set(pages.tolist())
        meta = sb.cache.page_meta.cpu().numpy()[pages]
        assert np.array_equal(meta[:, :, 0], mn[lo:]) and np.array_equal(meta[:, :, 1], mx[lo:])
    rest = [p for p in range(sb.cache.num_pages) if p not in touched]
    assert torch.equal(sb.cache.page_meta[rest].nan_to_num(5.0), before[rest].nan_to_num(5.0))


@pytest.mark.parametrize("kind", ["bf16", "u4t"])
def test_wrong_lists_leave_their_row_alone_and_are_reported(kind):
    from paged_kv_cache_243_gb300 import binding as B
    sb = SharedBatch(kind, 2, 64, 16, [], alone=[50, 60], seed=3, with_meta=True)
    cap = sb.width * 16
    good = [1, 4, 9]
    for first, keep, n in ((10, [1, 1, 5], 3), (10, [2, 1, 5], 3), (10, [-1, 0, 5], 3), (-1, [0, 1, 2], 3),
                           (10, [0, 1, cap - 10], 3), (cap, [0, 1, 2], 3), (10, [0, 1, 2], 4), (10, [0, 1, 2], -1),
                           (2 ** 31 - 2, [0, 1, 5], 3), (10, [0, 1, 2 ** 31 - 1], 3)):
        before = [x.clone() for x in parts(sb.cache)] + [sb.cache.page_meta.clone()]
        sb.status.zero_()
        sb.cache.keep_tokens(int_dev([keep, good]), int_dev([n, 0]), sb.table_dev, int_dev([first, 20]), dev_status=sb.status)
        torch.cuda.synchronize()
        assert int(sb.status.item()) == B.DEV_BAD_POSITION
        for x, y in zip(parts(sb.cache), before):
            assert np.array_equal(raw(x), raw(y))
        own = torch.from_numpy(sb.table[0].astype(np.int64)).cuda()
        assert torch.equal(sb.cache.page_meta[own].nan_to_num(3.0), before[-1][own].nan_to_num(3.0))
    # a bad page, that of token 3 + 14: it stays where it is, the others move
    sb.status.zero_()
    table = sb.table.copy()
    table[0, 1] = -1
    kept = [raw(x).copy() for x in parts(sb.cache)]
    sb.cache.keep_tokens(int_dev([[0, 1, 14, 31]]), None, int_dev(table[:1]), int_dev([3]), dev_status=sb.status)
    torch.cuda.synchronize()
    assert int(sb.status.item()) == B.DEV_BAD_PAGE
    for x, w in zip(parts(sb.cache), kept):
        w[table[0, 0], :, 6] = w[table[0, 2], :, 2]
        assert np.array_equal(raw(x), w)


def test_captured_and_on_another_stream():
    sb = SharedBatch("i8t", 2, 64, 16, [], alone=[50, 60], seed=4)
    s = torch.cuda.Stream()
    check(sb, sb.lens - 20, [[2, 5], [3, 4]], None, run=lambda *a, **k: sb.cache.keep_tokens(*a, stream=s, **k))

    def graphed(*a, **k):
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            sb.cache.keep_tokens(*a, **k)
        g.replay()

    check(sb, sb.lens - 20, [[2, 5], [3, 4]], None, run=graphed)
