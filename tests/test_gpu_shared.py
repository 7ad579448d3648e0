"""Decode attention over shared prefixes against the oracle, through the public wrapper."""
import numpy as np
import pytest
import torch

from shared_batch import KINDS, TORCH, SharedBatch, int_dev

pytestmark = pytest.mark.gpu

ALL = sorted(KINDS)


@pytest.mark.parametrize("kind", ALL)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("ps", [16, 48, 64, 256])
def test_groups_rows_and_types(kind, d, ps):
    if kind == "i8g" and ps % 64:
        ps = 128
    sb = SharedBatch(kind, 2, d, ps, [(200, [1, 17, 130, 0]), (64, [40, 5])], alone=[33, 1], seed=d + ps)
    q, qf = sb.queries(4)
    for dt in (torch.float32, TORCH[sb.src]):
        sb.check(sb.run(q, dt), qf, 4)
    assert int(sb.status.item()) == 0


@pytest.mark.parametrize("g", [1, 2, 3, 5, 7, 16, 64, 128])
@pytest.mark.parametrize("kind", ["bf16", "i8t"])
def test_head_groups(kind, g):
    sb = SharedBatch(kind, 1 if g > 16 else 3, 128, 32, [(300, [9, 40, 0])], alone=[70], seed=g)
    q, qf = sb.queries(g)
    sb.check(sb.run(q), qf, g)


@pytest.mark.parametrize("rows,g", [(1, 1), (32, 4), (33, 4), (64, 4), (65, 4), (100, 4), (13, 24)])
@pytest.mark.parametrize("kind", ["f16", "bf16", "u4t"])
def test_row_tiles(kind, rows, g):
    # 128 and 256 query rows of one kv head are the kernel's tiles: at, below and above them
    rng = np.random.default_rng(rows)
    sb = SharedBatch(kind, 1, 64, 16, [(333, list(rng.integers(0, 40, rows)))], seed=rows)
    q, qf = sb.queries(g)
    sb.check(sb.run(q, TORCH[sb.src]), qf, g)
    sb.check(sb.run(q), qf, g)


@pytest.mark.parametrize("prefix", [0, 1, 15, 16, 17, 63, 64, 127, 128, 129, 255, 256, 257, 1000])
@pytest.mark.parametrize("kind", ["bf16", "i8g"])
def test_prefix_lengths(kind, prefix):
    sb = SharedBatch(kind, 2, 128, 64, [(prefix, [1, 2, 100])], seed=prefix)
    q, qf = sb.queries(2)
    sb.check(sb.run(q, torch.bfloat16 if kind == "bf16" else torch.float16), qf, 2)


@pytest.mark.parametrize("kind", ["f16", "u4t"])
@pytest.mark.parametrize("splits", [1, 2, 3, 7, 40, 152, 1000])
def test_split_counts(kind, splits):
    sb = SharedBatch(kind, 2, 64, 16, [(1500, [3, 300, 77, 0]), (90, [1, 1])], alone=[400], seed=5)
    q, qf = sb.queries(3)
    sb.check(sb.run(q, num_splits=splits), qf, 3)
    assert int(sb.status.item()) == 0


@pytest.mark.parametrize("kind", ["bf16", "i8t"])
@pytest.mark.parametrize("rows,g", [(3, 2), (30, 4)])
def test_many_visits_per_block(kind, rows, g):
    # one and two blocks for everything: hundreds of tiles each
    rng = np.random.default_rng(rows)
    sb = SharedBatch(kind, 1, 64, 32, [(30000, list(rng.integers(0, 300, rows)))], alone=[9000, 50], seed=rows)
    q, qf = sb.queries(g)
    for splits in (1, 2):
        sb.check(sb.run(q, TORCH[sb.src], num_splits=splits), qf, g)
    assert int(sb.status.item()) == 0


def test_long_prefix_many_blocks():
    sb = SharedBatch("bf16", 2, 128, 16, [(20000, [5, 0, 700])], alone=[3000], seed=8)
    q, qf = sb.queries(4)
    sb.check(sb.run(q, torch.bfloat16), qf, 4)
    sb.check(sb.run(q), qf, 4)


def test_large_batch_of_short_rows():
    rng = np.random.default_rng(3)
    groups = [(int(p), list(rng.integers(0, 20, n))) for p, n in ((40, 300), (7, 90), (129, 2), (16, 50))]
    sb = SharedBatch("f16", 1, 64, 16, groups, alone=list(rng.integers(0, 60, 200)), seed=9)
    assert sb.B == 642
    q, qf = sb.queries(2)
    sb.check(sb.run(q, torch.float16), qf, 2)


def test_large_scores_and_moving_maxima():
    # scores of several hundred: the running maximum moves from tile to tile, most weights vanish
    for kind in ("bf16", "i8t", "u4t"):
        sb = SharedBatch(kind, 2, 128, 16, [(900, [10, 200, 0])], seed=11, k_scale=6.0)
        q, qf = sb.queries(4, scale=6.0)
        sb.check(sb.run(q), qf, 4)


@pytest.mark.parametrize("kind", ["i8t", "i8g", "u4t"])
@pytest.mark.parametrize("v_scale", [1e-5, 1.0, 200.0])
def test_value_ranges_of_quantised_caches(kind, v_scale):
    # weights times value scales must neither leave fp16's range nor vanish in it
    if v_scale == 1e-5:
        v_scale = 2.0 ** -10    # fp16 tokens: still normal numbers
    sb = SharedBatch(kind, 2, 128, 64, [(400, [10, 90])], seed=12, v_scale=v_scale)
    q, qf = sb.queries(4)
    sb.check(sb.run(q), qf, 4)
    sb.check(sb.run(q, torch.float16), qf, 4)


@pytest.mark.parametrize("kind", ["i8t", "i8g", "u4t"])
def test_bf16_queries_on_quantised_caches(kind):
    sb = SharedBatch(kind, 2, 64, 64, [(400, [10, 90, 1])], alone=[65], seed=13)
    q, qf = sb.queries(4, "bf16")
    sb.check(sb.run(q), qf, 4, "bf16")
    sb.check(sb.run(q, torch.bfloat16), qf, 4, "bf16")


@pytest.mark.parametrize("kind", ALL)
@pytest.mark.parametrize("d", [64, 128])
def test_the_most_groups(kind, d):
    # 1024 groups take so much shared memory that fp16/bf16 caches of 128 channels have one
    # tile of K and V at a time: partial tiles right behind whole ones
    rng = np.random.default_rng(d)
    sb = SharedBatch(kind, 2, d, 64, [(256, [300, 44, 172, 1]), (130, [260, 2])],
                     alone=[int(n) for n in rng.integers(129, 600, 12)], seed=21)
    sb.prefix_dev = int_dev(np.concatenate([sb.prefix, np.full(1024 - len(sb.prefix), 64, dtype=np.int32)]))
    q, qf = sb.queries(4)
    for splits in (0, 1, 5):
        sb.check(sb.run(q, num_splits=splits), qf, 4)
    assert int(sb.status.item()) == 0


def test_empty_rows_and_padding():
    # rows of length 0 (finished or padded), rows shorter than their group's prefix, a group with
    # no such rows at all, and no groups
    sb = SharedBatch("bf16", 2, 128, 16, [(150, [20, 30, 40, 3])], alone=[50], seed=14)
    q, qf = sb.queries(2)
    lens = sb.lens.copy()
    rows = np.flatnonzero(sb.group == 0)
    lens[rows[0]], lens[rows[1]] = 0, 77
    out = sb.cache.shared_attention(q, sb.table_dev, int_dev(lens), sb.group_dev, sb.prefix_dev)
    sb.check(out, qf, 2, lens=lens)
    assert torch.count_nonzero(out[rows[0]]) == 0
    empty = torch.zeros(0, dtype=torch.int32, device="cuda")
    none = torch.full_like(sb.group_dev, -1)
    out = sb.cache.shared_attention(q, sb.table_dev, sb.lens_dev, none, empty)
    sb.check(out, qf, 2)
    out = sb.cache.shared_attention(q, sb.table_dev, torch.zeros_like(sb.lens_dev), sb.group_dev, sb.prefix_dev)
    assert torch.count_nonzero(out) == 0


def test_rows_behind_the_batch_and_the_table_stay():
    sb = SharedBatch("f16", 2, 64, 16, [(50, [20, 30])], seed=15)
    q, qf = sb.queries(2)
    out = torch.full((sb.B + 2, 4, 64), 7.0, device="cuda")
    ref = sb.run(q)
    sb.cache.shared_attention(q, sb.table_dev, sb.lens_dev, sb.group_dev, sb.prefix_dev, out=out[:sb.B])
    torch.cuda.synchronize()
    assert torch.equal(out[:sb.B], ref) and bool((out[sb.B:] == 7.0).all())


def test_bad_pages_groups_and_lengths_are_reported():
    from paged_kv_cache_243_gb300 import binding as B
    sb = SharedBatch("bf16", 2, 128, 32, [(200, [40, 10, 70])], alone=[90], seed=16)
    q, qf = sb.queries(2)
    # a page outside the pool: its tokens are left out of the row's attention
    b = int(np.flatnonzero(sb.group < 0)[0])
    table = sb.table.copy()
    table[b, 1] = 10 ** 6
    out = sb.cache.shared_attention(q, int_dev(table), sb.lens_dev, sb.group_dev, sb.prefix_dev,
                                    dev_status=sb.status)
    torch.cuda.synchronize()
    assert int(sb.status.item()) == B.DEV_BAD_PAGE
    keep = np.r_[0:32, 64:90]
    k, v, lens = sb.k[b], sb.v[b], sb.lens.copy()
    sb.k[b], sb.v[b], lens[b] = k[keep], v[keep], len(keep)
    sb.check(out, qf, 2, lens=lens)
    sb.k[b], sb.v[b] = k, v
    # a whole row of bad pages gives zeros
    table[b] = -1
    sb.status.zero_()
    out = sb.cache.shared_attention(q, int_dev(table), sb.lens_dev, sb.group_dev, sb.prefix_dev,
                                    dev_status=sb.status)
    torch.cuda.synchronize()
    assert torch.count_nonzero(out[b]) == 0 and int(sb.status.item()) == B.DEV_BAD_PAGE
    # groups out of range attend on their own; a negative prefix shares nothing
    sb.status.zero_()
    group = sb.group.copy()
    group[b] = 5
    out = sb.cache.shared_attention(q, sb.table_dev, sb.lens_dev, int_dev(group), sb.prefix_dev,
                                    dev_status=sb.status)
    torch.cuda.synchronize()
    assert int(sb.status.item()) == B.DEV_BAD_GROUP
    sb.check(out, qf, 2)
    sb.status.zero_()
    out = sb.cache.shared_attention(q, sb.table_dev, sb.lens_dev, sb.group_dev, int_dev([-4]),
                                    dev_status=sb.status)
    torch.cuda.synchronize()
    assert int(sb.status.item()) == B.DEV_BAD_GROUP
    sb.check(out, qf, 2)
    # a prefix longer than its rows: each attends on its own
    out = sb.cache.shared_attention(q, sb.table_dev, sb.lens_dev, sb.group_dev, int_dev([10 ** 6]))
    sb.check(out, qf, 2)
    # a negative length gives zeros, one beyond the table is cut to it
    sb.status.zero_()
    lens = sb.lens.copy()
    lens[b] = -3
    out = sb.cache.shared_attention(q, sb.table_dev, int_dev(lens), sb.group_dev, sb.prefix_dev,
                                    dev_status=sb.status)
    torch.cuda.synchronize()
    assert int(sb.status.item()) == B.DEV_BAD_POSITION and torch.count_nonzero(out[b]) == 0


def test_streams_capture_and_devices():
    sb = SharedBatch("bf16", 2, 128, 16, [(500, [40, 10, 70, 8])], alone=[90], seed=17)
    q, qf = sb.queries(4)
    ref = sb.run(q)
    # another stream than the tensors' own, then a captured call replayed with new queries
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = torch.empty_like(ref)
    with torch.cuda.stream(s):
        sb.cache.shared_attention(q, sb.table_dev, sb.lens_dev, sb.group_dev, sb.prefix_dev, out=out)
    s.synchronize()
    assert torch.equal(out, ref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        sb.cache.shared_attention(q, sb.table_dev, sb.lens_dev, sb.group_dev, sb.prefix_dev, out=out)
    q2, qf2 = sb.queries(4, seed=3)
    q.copy_(q2)
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    sb.check(out, qf2, 4)
    # two captured calls with a workspace each, replayed at the same time
    outs, graphs = [torch.empty_like(ref) for _ in range(2)], []
    streams = [torch.cuda.Stream() for _ in range(2)]
    works = [torch.empty_like(sb.cache.shared_workspace(sb.B, 8)) for _ in range(2)]
    for o, w, st in zip(outs, works, streams):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            for _ in range(4):
                sb.cache.shared_attention(q, sb.table_dev, sb.lens_dev, sb.group_dev, sb.prefix_dev, out=o,
                                          workspace=w)
        graphs.append(g)
    torch.cuda.synchronize()
    for _ in range(10):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for o in outs:
        sb.check(o, qf2, 4)


def test_an_explicit_stream_owns_the_call_and_its_memory():
    sb = SharedBatch("f16", 2, 128, 16, [(300, [20, 5, 61])], alone=[33], seed=23)
    q, qf = sb.queries(4)
    ref = sb.run(q)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    outs = []
    for _ in range(20):
        # the current stream is busy with memory that it gives back at once
        torch.empty(1 << 20, device="cuda").fill_(float("nan"))
        outs.append(sb.cache.shared_attention(q, sb.table_dev, sb.lens_dev, sb.group_dev, sb.prefix_dev, stream=s))
    assert sb.cache.shared_workspace(sb.B, 8, stream=s) is not sb.cache.shared_workspace(sb.B, 8)
    s.synchronize()
    for o in outs:
        assert torch.equal(o, ref)


def test_same_call_twice_gives_the_same_bits():
    sb = SharedBatch("i8t", 4, 128, 16, [(3000, [400, 10, 70, 8])], alone=[900], seed=18)
    q, _ = sb.queries(4)
    a = sb.run(q, torch.float16)
    for _ in range(5):
        assert torch.equal(sb.run(q, torch.float16), a)


def test_unshared_attention_agrees():
    # the same rows through attention(): both are within their bounds of the oracle
    sb = SharedBatch("f16", 2, 128, 16, [(600, [40, 10]), (80, [7, 7, 7])], seed=19)
    q, qf = sb.queries(4)
    a = sb.run(q)
    b = sb.cache.attention(q, sb.table_dev, sb.lens_dev)
    sb.check(a, qf, 4)
    assert float((a - b).abs().max()) <= 2e-3
