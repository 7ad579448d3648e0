"""Attention for trees of drafted tokens against its definition, through the public wrapper."""
import numpy as np
import pytest
import torch

from shared_batch import KINDS, TORCH, int_dev
from tree_batch import TreeBatch, pack, random_parents, seen_from_parents

pytestmark = pytest.mark.gpu

ALL = sorted(KINDS)


@pytest.mark.parametrize("kind", ALL)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("ps", [16, 48, 64, 256])
def test_types_and_pages(kind, d, ps):
    if kind == "i8g" and ps % 64:
        ps = 128
    tb = TreeBatch(kind, 2, d, ps, [300, 5, 130, 12, 700], 11, drafts=[11, 5, 7, 1, 11], seed=d + ps)
    q, qf = tb.tree_queries(4)
    for dt in (torch.float32, TORCH[tb.src]):
        tb.tree_check(tb.tree_run(q, dt), qf, 4)
    assert int(tb.status.item()) == 0


@pytest.mark.parametrize("T,g", [(1, 1), (3, 2), (8, 1), (9, 1), (8, 2), (16, 1), (17, 1), (8, 16), (43, 3), (64, 4), (65, 4),
                                 (2, 128), (5, 64), (200, 4), (256, 5)])
@pytest.mark.parametrize("kind", ["bf16", "i8t"])
def test_query_rows(kind, T, g):
    # 8, 16, 128 and 256 query rows of a kv head are the kernel's borders: at, below and above them
    tb = TreeBatch(kind, 1 if g > 16 else 2, 64, 32, [400, T, 290], T, drafts=[T, T, max(1, T - 1)], seed=T)
    q, qf = tb.tree_queries(g)
    tb.tree_check(tb.tree_run(q, TORCH[tb.src]), qf, g)
    tb.tree_check(tb.tree_run(q), qf, g)


@pytest.mark.parametrize("kind", ["f16", "u4t"])
@pytest.mark.parametrize("T", [1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 200, 256])
@pytest.mark.parametrize("tree", ["tree", "chain", "any"])
def test_masks_of_every_length(kind, T, tree):
    # contexts of 0, 1, ... tokens: the drafts begin anywhere in a tile, and end there
    lens = [T, T + 1, T + 127, T + 128, T + 100, T + 500]
    tb = TreeBatch(kind, 1, 64, 16, lens, T, drafts=[T, T, T - T // 3, T, 1, T], seed=T, tree=tree)
    q, qf = tb.tree_queries(2)
    tb.tree_check(tb.tree_run(q), qf, 2)
    tb.tree_check(tb.tree_run(q, TORCH[tb.src]), qf, 2)
    assert int(tb.status.item()) == 0


@pytest.mark.parametrize("kind", ["bf16", "i8g", "u4t"])
@pytest.mark.parametrize("splits", [1, 2, 3, 7, 40, 152, 1000])
def test_split_counts(kind, splits):
    tb = TreeBatch(kind, 2, 64, 64, [1500, 90, 3, 700], 40, drafts=[40, 40, 3, 21], seed=5, tree="any")
    q, qf = tb.tree_queries(4)
    tb.tree_check(tb.tree_run(q, num_splits=splits), qf, 4)
    assert int(tb.status.item()) == 0


@pytest.mark.parametrize("kind", ["f16", "i8t"])
@pytest.mark.parametrize("T,g", [(4, 2), (40, 4), (100, 4)])
def test_many_visits_per_block(kind, T, g):
    tb = TreeBatch(kind, 1, 64, 32, [30000, 9000], T, seed=T)
    q, qf = tb.tree_queries(g)
    for splits in (1, 2):
        tb.tree_check(tb.tree_run(q, TORCH[tb.src], num_splits=splits), qf, g)
    assert int(tb.status.item()) == 0


@pytest.mark.parametrize("kind", ["bf16", "i8t"])
@pytest.mark.parametrize("T,g", [(3, 3), (13, 4), (30, 4), (64, 4), (100, 4)])
@pytest.mark.parametrize("last", [1, 64, 77, 113, 128])
def test_long_parts_end_in_drafts(kind, T, g, last):
    # blocks whose part of a segment is long and ends with the drafts' tile, part of a tile or all of it: transposed, one
    # and two row tiles, in either output type; and the same bits every time
    lens = [128 * 40 + last, 128 * 23 + last, 128 * 9 + last]
    tb = TreeBatch(kind, 1, 128, 16, lens, T, seed=T + last)
    q, qf = tb.tree_queries(g)
    for dt in (TORCH[tb.src], torch.float32):
        for splits in (0, 3, 7):
            ref = tb.tree_run(q, dt, num_splits=splits)
            tb.tree_check(ref, qf, g)
            for _ in range(5):
                assert torch.equal(tb.tree_run(q, dt, num_splits=splits), ref)


def test_every_call_of_a_large_batch_gives_the_same_bits():
    for kind, T, g, n in (("bf16", 16, 4, 8), ("f16", 40, 7, 6), ("i8t", 24, 4, 8), ("bf16", 3, 4, 16)):
        rng = np.random.default_rng(T)
        tb = TreeBatch(kind, 4, 128, 16, rng.integers(1500, 4000, n), T, seed=T)
        q, qf = tb.tree_queries(g)
        dt = TORCH[tb.src]
        tb.cache.k_pages.add_(0)      # (the pools are not in the cache of the first call)
        ref = tb.tree_run(q, dt)
        tb.tree_check(ref, qf, g)
        junk = torch.empty(64 << 20, dtype=torch.float32, device="cuda")
        for i in range(20):
            if i % 2:
                junk.zero_()          # K and V come from memory again
            assert torch.equal(tb.tree_run(q, dt), ref)


def test_forty_sequences():
    # more than a warp plans by itself, of one and of two row tiles
    rng = np.random.default_rng(5)
    for T, g in ((70, 4), (9, 2)):
        tb = TreeBatch("bf16", 2, 64, 32, rng.integers(0, 700, 40), T, drafts=rng.integers(0, T + 1, 40), seed=T)
        q, qf = tb.tree_queries(g)
        tb.tree_check(tb.tree_run(q, torch.bfloat16), qf, g)


def test_long_contexts():
    tb = TreeBatch("bf16", 2, 128, 16, [20000, 3001, 129], 24, seed=8)
    q, qf = tb.tree_queries(4)
    tb.tree_check(tb.tree_run(q, torch.bfloat16), qf, 4)
    tb.tree_check(tb.tree_run(q), qf, 4)


@pytest.mark.parametrize("kind,T,g", [("bf16", 5, 2), ("i8t", 5, 2), ("bf16", 40, 4), ("u4t", 40, 4)])
def test_more_tokens_than_a_float_counts(kind, T, g):
    # 2^24 tokens and more, 64 pages of context over and over; each of its tokens weighs as often as it comes
    times, ps, d, pages, tail = 16500, 16, 64, 64, 77
    tb = TreeBatch(kind, 1, d, ps, [pages * ps + tail], T, seed=T)
    L = pages * ps * times + tail
    assert L > 1 << 24
    table = int_dev(np.concatenate([np.tile(tb.table[0, :pages], times), tb.table[0, pages:]])[None])
    q, qf = tb.tree_queries(g)
    out = tb.cache.tree_attention(q, table, int_dev([L]), tb.mask, dev_status=tb.status)
    torch.cuda.synchronize()
    assert int(tb.status.item()) == 0
    n, k, v, on = pages * ps, tb.k[0][:, 0], tb.v[0][:, 0], tb.attends(0)
    often = np.where(np.arange(n + tail) < n, float(times), 1.0)
    got = out.cpu().numpy().astype(np.float64)[0]
    sm, half = 1.0 / np.sqrt(d), torch.finfo(TORCH[tb.src]).eps / 2
    for h in range(g):
        qq = qf[0, :, h].astype(np.float64)
        w = np.where(on, np.exp(sm * (qq @ k.T)), 0.0) * often
        w /= w.sum(1, keepdims=True)
        want, mass = w @ v, w @ np.abs(v) + tb.vmid[0]
        # the bound of TreeBatch.tree_expected, but for the sums: a block, of a hundred at least, adds up
        # its own tokens, 16 at a time
        most = (np.abs(qq) @ np.abs(k).T).max(1) + 2 * np.abs(qq).sum(1) * tb.kmid[0]
        rel = 2 * np.expm1(sm * (d + 8) * 2.0 ** -23 * most) + 2.0 ** -20 + (L / 1600 + 64) * 2.0 ** -23 + half * half
        if tb.src == "f16":
            rel = rel + 2.0 ** -24      # fp16's smallest step beside weights of 2^7 and more
        err = np.abs(got[:, h] - want)
        assert (err <= rel[:, None] * mass).all(), (err.max(), (rel[:, None] * mass).min())


def test_many_short_sequences():
    rng = np.random.default_rng(3)
    lens = rng.integers(0, 60, 1024)
    lens[:3] = 0
    tb = TreeBatch("f16", 1, 64, 16, lens, 7, drafts=rng.integers(0, 8, 1024), seed=9)
    q, qf = tb.tree_queries(2)
    tb.tree_check(tb.tree_run(q, torch.float16), qf, 2)


def test_one_mask_for_all_and_one_for_each():
    tb = TreeBatch("bf16", 2, 128, 32, [200, 77, 500], 70, seed=10)
    tb.seen = np.repeat(seen_from_parents(random_parents(np.random.default_rng(1), 70))[None], 3, 0)
    q, qf = tb.tree_queries(3)
    one = tb.tree_run(q, mask=pack(tb.seen[0]).cuda())
    tb.tree_check(one, qf, 3)
    assert torch.equal(one, tb.tree_run(q, mask=pack(tb.seen).cuda()))
    # bits of drafts that do not exist mean nothing
    more = tb.seen.copy()
    tb.drafts_dev = int_dev([60, 60, 60])
    tb.drafts = np.array([60, 60, 60], dtype=np.int32)
    ref = tb.tree_run(q, mask=pack(more).cuda())
    more[:, :, 60:] = True
    more[:, 60:] = True
    assert torch.equal(ref, tb.tree_run(q, mask=pack(more).cuda()))
    tb.tree_check(ref, qf, 3)


def test_a_single_draft_is_decode_attention():
    tb = TreeBatch("f16", 4, 128, 16, [333, 1, 1000], 1, seed=11)
    q, qf = tb.tree_queries(4)
    tree = tb.tree_run(q)[:, 0]
    one = tb.cache.attention(q[:, 0].contiguous(), tb.table_dev, tb.lens_dev)
    out, bound, mass = tb.tree_expected(qf, 4)
    tol = 2 * (bound + mass * 2.0 ** -20)[:, 0]      # each within its bound of the definition
    assert ((tree - one).abs().cpu().numpy() <= tol).all()


def test_no_draft_lens_means_all():
    tb = TreeBatch("u4t", 2, 64, 32, [100, 40, 300], 9, seed=12)
    q, qf = tb.tree_queries(5)
    ref = tb.tree_run(q)
    assert torch.equal(ref, tb.cache.tree_attention(q, tb.table_dev, tb.lens_dev, tb.mask))
    tb.tree_check(ref, qf, 5)


@pytest.mark.parametrize("kind", ["i8t", "i8g", "u4t"])
def test_bf16_queries_on_quantised_caches(kind):
    tb = TreeBatch(kind, 2, 64, 64, [400, 90, 65], 20, seed=13)
    q, qf = tb.tree_queries(4, "bf16")
    tb.tree_check(tb.tree_run(q), qf, 4, "bf16")
    tb.tree_check(tb.tree_run(q, torch.bfloat16), qf, 4, "bf16")


def test_large_scores_and_moving_maxima():
    for kind in ("bf16", "i8t", "u4t"):
        tb = TreeBatch(kind, 2, 128, 16, [900, 300], 30, seed=14, k_scale=6.0)
        q, qf = tb.tree_queries(4, scale=6.0)
        tb.tree_check(tb.tree_run(q), qf, 4)


def test_constant_keys_and_values_of_quantised_caches():
    # a scale of 0: a masked score must not become 0 times infinity
    for kind in ("i8t", "u4t"):
        tb = TreeBatch(kind, 2, 64, 16, [150, 20], 20, seed=15, k_scale=0.0, v_scale=0.0, tree="any")
        q, qf = tb.tree_queries(3)
        tb.tree_check(tb.tree_run(q), qf, 3)


# --------------------------------------------------------- what a row does not attend to
def spoil(tb, b, tok, h, what, value, channel=5):
    """Token tok of sequence b, kv head h: its key, or one channel of its values (all of them where a
    scale stands for them), becomes `value`."""
    page, slot = int(tb.table[b, tok // tb.ps]), tok % tb.ps
    c = tb.cache
    if c.kv_sz is None:
        (c.k_pages if what == "k" else c.v_pages)[page, h, slot, channel] = value
    else:
        gran = tb.ps // c.kv_sz.shape[2]
        assert gran == 1
        c.kv_sz[page, h, slot, 0 if what == "k" else 2] = value


@pytest.mark.parametrize("kind", ["f16", "bf16", "i8t", "u4t"])
@pytest.mark.parametrize("T,g", [(7, 1), (12, 1), (20, 2), (50, 4)])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("splits", [0, 1])
def test_no_number_reaches_rows_that_do_not_attend_to_it(kind, T, g, value, splits):
    tb = TreeBatch(kind, 2, 64, 16, [T + 121, T, T + 400], T, seed=T)
    q, qf = tb.tree_queries(g)
    for dt in (torch.float32, TORCH[tb.src]):
        ref = tb.tree_run(q, dt, num_splits=splits)
        bound = torch.from_numpy(tb.tree_bound(qf, g, dt)[1]).cuda()
        for what in ("k", "v"):
            keep = [x.clone() for x in (tb.cache.k_pages, tb.cache.v_pages)] + \
                [None if tb.cache.kv_sz is None else tb.cache.kv_sz.clone()]
            # two drafts of one sequence, and one of another
            hit = [(0, 2), (0, T - 1), (2, T // 2)]
            for b, j in hit:
                spoil(tb, b, int(tb.lens[b]) - T + j, 1, what, value)
            out = tb.tree_run(q, dt, num_splits=splits)
            want = ref.clone()
            for b, j in hit:
                rows = np.flatnonzero(tb.seen[b, :, j])
                assert len(rows) > 0
                for t in rows:
                    got = out[b, t, g:]        # the heads of kv head 1
                    if what == "k":
                        # (an infinite key may win every weight or none, with either sign: only NaN is certain)
                        if not (value == value):
                            assert bool(torch.isnan(got).all())
                    elif tb.cache.kv_sz is None:
                        assert not bool(torch.isfinite(got[:, 5]).any())
                        if value == value and not tb.seen[b, t, [i for c, i in hit if c == b and i != j]].any():
                            assert bool((got[:, 5] == value).all())
                        got = got.clone()
                        got[:, 5] = ref[b, t, g:, 5]
                        assert torch.equal(got, ref[b, t, g:])       # the other channels
                    else:
                        assert not bool(torch.isfinite(got).any())
                    want[b, t, g:] = out[b, t, g:]
            if tb.cache.kv_sz is None or what == "k":
                assert torch.equal(torch.nan_to_num(out, nan=77.0), torch.nan_to_num(want, nan=77.0))
            else:
                # The sizes of a tile's values choose what weights refer to, and a scale that is no number has
                # none: other roundings, each within the bound.
                same = torch.nan_to_num(out, nan=77.0) == torch.nan_to_num(want, nan=77.0)
                assert bool((same | ((out.double() - ref.double()).abs() <= 2 * bound)).all())
            tb.cache.k_pages.copy_(keep[0])
            tb.cache.v_pages.copy_(keep[1])
            if keep[2] is not None:
                tb.cache.kv_sz.copy_(keep[2])
    assert int(tb.status.item()) == 0


@pytest.mark.parametrize("kind", ["f16", "bf16", "i8t", "u4t"])
@pytest.mark.parametrize("T,g", [(3, 2), (20, 2), (50, 4)])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_no_numbers_before_the_drafts_reach_every_row(kind, T, g, value):
    # a value in the tile of the drafts, but not one of them; and one in a tile before it
    for back in (1, 9, 200):
        tb = TreeBatch(kind, 2, 64, 16, [T + 300, T + 64], T, seed=T)
        q, _ = tb.tree_queries(g)
        ref = tb.tree_run(q)
        b = int(np.argmax(tb.lens))
        spoil(tb, b, int(tb.lens[b]) - T - back, 1, "v", value)
        out = tb.tree_run(q)
        got = out[b, :, g:] if tb.cache.kv_sz is not None else out[b, :, g:, 5]
        assert not bool(torch.isfinite(got).any())
        assert torch.equal(out[b, :, :g], ref[b, :, :g]) and torch.equal(out[1 - b], ref[1 - b])


def test_huge_values_cost_rows_that_do_not_attend_to_them_nothing():
    tb = TreeBatch("f16", 2, 64, 16, [200, 60], 20, seed=21)
    q, qf = tb.tree_queries(2)
    ref = tb.tree_run(q)
    spoil(tb, 0, int(tb.lens[0]) - 1, 0, "v", 60000.0)
    spoil(tb, 0, int(tb.lens[0]) - 1, 0, "k", 60000.0)
    out = tb.tree_run(q)
    out[0, tb.seen[0, :, 19].nonzero()[0]] = ref[0, tb.seen[0, :, 19].nonzero()[0]]
    assert torch.equal(out, ref)


def test_tokens_behind_the_drafts_are_never_seen():
    tb = TreeBatch("bf16", 2, 64, 16, [100, 200], 9, seed=22, extra_pages=1)
    q, _ = tb.tree_queries(4)
    ref = tb.tree_run(q)
    for b in range(2):
        for tok in range(int(tb.lens[b]), int(tb.lens[b]) + 12):
            spoil(tb, b, tok, 0, "k", float("nan"))
            spoil(tb, b, tok, 1, "v", float("nan"))
    assert torch.equal(ref, tb.tree_run(q))


# ------------------------------------------------------------------ errors, order, streams
def test_lengths_and_counts_out_of_range_are_clamped_and_reported():
    from paged_kv_cache_243_gb300 import binding as B
    tb = TreeBatch("f16", 2, 64, 16, [100, 64, 30], 6, seed=23)
    q, _ = tb.tree_queries(2)
    ref = tb.tree_run(q)
    for lens, drafts, same in (([1 << 20, 64, 30], [6, 6, 6], [1, 2]), ([-3, 64, 30], [6, 6, 6], [1, 2]),
                               ([100, 64, 30], [7, 6, 6], [0, 1, 2]), ([100, 64, 30], [-1, 6, 6], [1, 2]),
                               ([100, 64, 4], [6, 6, 6], [0, 1])):
        rows = [list(tb.lens).index(n) for n in (100, 64, 30)]
        L, n = np.zeros(3, dtype=np.int32), np.zeros(3, dtype=np.int32)
        L[rows], n[rows] = lens, drafts
        tb.status.zero_()
        out = tb.cache.tree_attention(q, tb.table_dev, int_dev(L), tb.mask, int_dev(n), dev_status=tb.status)
        assert int(tb.status.item()) == B.DEV_BAD_POSITION
        for i in same:
            assert torch.equal(out[rows[i]], ref[rows[i]])
    tb.status.zero_()


def test_a_bad_page_is_skipped_and_reported():
    from paged_kv_cache_243_gb300 import binding as B
    for bad in (-1, 1 << 20):
        tb = TreeBatch("f16", 2, 64, 16, [100, 64], 6, seed=24)
        q, qf = tb.tree_queries(2)
        b = int(np.argmax(tb.lens))
        table = tb.table.copy()
        table[b, 2] = bad
        out = tb.cache.tree_attention(q, int_dev(table), tb.lens_dev, tb.mask, dev_status=tb.status)
        torch.cuda.synchronize()
        assert int(tb.status.item()) == B.DEV_BAD_PAGE
        # as if tokens 32 .. 47 were not there
        keep = np.r_[0:32, 48:int(tb.lens[b])]
        tb.k[b], tb.v[b] = tb.k[b][keep], tb.v[b][keep]
        tb.lens[b] -= 16
        tb.tree_check(out, qf, 2)


def test_the_same_call_gives_the_same_bits_captured_and_on_other_streams():
    tb = TreeBatch("bf16", 4, 128, 16, [700, 1300, 40], 33, seed=25)
    q, qf = tb.tree_queries(4)
    ref = tb.tree_run(q, torch.bfloat16)
    tb.tree_check(ref, qf, 4)
    for _ in range(5):
        assert torch.equal(ref, tb.tree_run(q, torch.bfloat16))
    s = torch.cuda.Stream()
    assert torch.equal(ref, tb.tree_run(q, torch.bfloat16, stream=s))
    outs = [torch.zeros_like(ref) for _ in range(2)]
    graphs = []
    for o in outs:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            for _ in range(4):
                tb.cache.tree_attention(q, tb.table_dev, tb.lens_dev, tb.mask, tb.drafts_dev, out=o)
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(10):
        for gr, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                gr.replay()
        again = tb.cache.tree_attention(q, tb.table_dev, tb.lens_dev, tb.mask, tb.drafts_dev, out_dtype=torch.bfloat16)
    torch.cuda.synchronize()
    assert torch.equal(again, ref) and all(torch.equal(o, ref) for o in outs)


def test_trees_and_shared_prefixes_take_turns_on_one_workspace():
    tb = TreeBatch("f16", 2, 64, 16, [500, 90], 10, seed=26)
    q, _ = tb.tree_queries(2)
    ref = tb.tree_run(q)
    one = q[:, 0].contiguous()
    shared = lambda: tb.cache.shared_attention(one, tb.table_dev, tb.lens_dev, int_dev([-1, -1]), int_dev([0]))  # noqa: E731
    ref1 = shared()
    for _ in range(10):
        a, b = shared(), tb.cache.tree_attention(q, tb.table_dev, tb.lens_dev, tb.mask, tb.drafts_dev)
    assert torch.equal(a, ref1) and torch.equal(b, ref)
    ws = tb.cache.tree_workspace(2, 10, 4)
    ws.fill_(255)
    assert torch.equal(ref, tb.tree_run(q, workspace=ws))
