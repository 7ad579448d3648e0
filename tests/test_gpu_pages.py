"""Copying pages and renaming them in block tables on the GPU, and forked sequences decoded
step by step: every byte and every output against the host's own bookkeeping."""
import numpy as np
import pytest
import torch

from shared_batch import KINDS, SharedBatch, int_dev, restore, to_dev

pytestmark = pytest.mark.gpu


def make_cache(kind, pages, hkv, d, ps, meta, rows=0):
    from paged_kv_cache_243_gb300.cache import PagedKVCache
    kv, quant, _ = KINDS[kind]
    c = PagedKVCache(pages, ps, hkv, d, kv_dtype=kv, quant=quant, with_meta=meta, tail_rows=rows)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(pages + d)
    for t in parts(c):
        t.view(torch.uint8).random_(0, 256, generator=gen)     # any bits, NaNs among them
    return c


def parts(c):
    return [t for t in (c.k_pages, c.v_pages, c.kv_sz, c.page_meta) if t is not None] + \
        ([c.tail] if c.tail is not None else [])


def bits(c):
    return [t.view(torch.uint8).cpu().numpy().reshape(t.shape[0], -1).copy() for t in parts(c)]


@pytest.mark.parametrize("kind", sorted(KINDS))
@pytest.mark.parametrize("hkv,d,ps,meta", [(1, 64, 64, False), (3, 128, 64, True), (8, 128, 256, True), (5, 64, 192, False)])
@pytest.mark.parametrize("n", [1, 2, 29])
def test_copies_are_exact_and_touch_nothing_else(kind, hkv, d, ps, meta, n):
    rows = 7 if kind == "i8g" else 0
    c = make_cache(kind, 64, hkv, d, ps, meta, rows)
    before = bits(c)
    order = np.random.default_rng(n).permutation(64)
    src, dst = order[:n], order[n:2 * n]
    if n == 29:
        src[5] = src[3]                         # one page copied to two places
    args = ([1, 0, 4], [2, 6, 3]) if rows else (None, None)
    c.copy_pages(src.tolist(), dst, *args)
    torch.cuda.synchronize()
    for i, (a, b) in enumerate(zip(before, bits(c))):
        if rows and i == len(before) - 1:
            a[args[1]] = a[args[0]]
        else:
            a[dst] = a[src]
        assert np.array_equal(a, b)


@pytest.mark.parametrize("pages", [20001, 70001])      # ids of 16 and of 32 bits
def test_long_lists_and_the_empty_one(pages):
    c = make_cache("u4t", pages, 1, 64, 16, False)
    before = bits(c)
    order = np.random.default_rng(0).permutation(pages)
    n = 9003                                    # more pairs than one launch holds
    c.copy_pages(order[:n], order[n:2 * n])
    c.copy_pages([], [])
    torch.cuda.synchronize()
    for a, b in zip(before, bits(c)):
        a[order[n:2 * n]] = a[order[:n]]
        assert np.array_equal(a, b)
    table = np.random.default_rng(1).integers(-1, pages, (37, 1001)).astype(np.int32)
    table[3, 5], table[4, 6] = 10 ** 9, -(10 ** 9)     # ids outside the pool stay
    dev = int_dev(table)
    c.remap_table(dev, order[:n], order[n:2 * n])
    to = np.arange(pages)
    to[order[:n]] = order[n:2 * n]
    ok = (table >= 0) & (table < pages)
    assert np.array_equal(dev.cpu().numpy(), np.where(ok, to[np.where(ok, table, 0)], table))


@pytest.mark.parametrize("n", [1, 63, 64, 65, 4000, 4001, 8000, 8001])
@pytest.mark.parametrize("pages", [16100, 66000])
@pytest.mark.parametrize("shape", [(1, 1), (3, 7), (64, 513)])
def test_remap(n, pages, shape):
    c = make_cache("u4t", pages, 1, 64, 16, False)
    rng = np.random.default_rng(n)
    order = rng.permutation(pages)
    src, dst = order[:n], rng.choice(order[n:], n)     # several pages may become one
    table = rng.integers(0, pages, shape).astype(np.int32)
    table.reshape(-1)[0] = src[0]
    dev = int_dev(table)
    c.remap_table(dev, src, dst)
    to = np.arange(pages)
    to[src] = dst
    assert np.array_equal(dev.cpu().numpy(), to[table])


def test_copy_on_another_stream_and_captured():
    c = make_cache("bf16", 40, 2, 64, 16, False)
    before = bits(c)
    table = int_dev([[1, 2, 3]])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        c.copy_pages([1, 2], [30, 31])
        c.remap_table(table, [1, 2], [30, 31])
        c.copy_pages([30], [32])
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    for a, b in zip(before, bits(c)):
        a[[30, 31]] = a[[1, 2]]
        a[32] = a[30]
        assert np.array_equal(a, b)
    assert table.tolist() == [[30, 31, 3]]
    with torch.cuda.stream(s):
        c.copy_pages([5], [33])
    s.synchronize()
    assert torch.equal(c.k_pages[33].view(torch.uint8), c.k_pages[5].view(torch.uint8))


@pytest.mark.parametrize("kind", sorted(KINDS))
def test_fork_append_attend_compact(kind):
    """A prompt, four sequences forked from it, twenty decode steps of shared_attention with
    the appends between them, one sequence ending and the pool drawn together in the middle."""
    from paged_kv_cache_243_gb300.cache import PageAllocator, PagedKVCache
    kv, quant, src_type = KINDS[kind]
    hkv, g, d, ps, prompt, steps, rows, width = 2, 2, 64, 64, 150, 20, 4, 8
    # the rows' final tokens: a batch whose layout is not used, only its values
    sb = SharedBatch(kind, hkv, d, ps, [(prompt, [steps] * rows)], seed=31)
    pool = PageAllocator(40)
    cache = PagedKVCache(40, ps, hkv, d, kv_dtype=kv, quant=quant, tail_rows=rows, poison=True)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    spare = pool.reserve(99, 5 * ps, ps, width)                       # keeps low pages busy at first
    table = np.full((rows, width), -1, dtype=np.int32)
    table[0] = pool.reserve(0, prompt, ps, width)
    kb, vb = sb.bits[0]
    cache.append(to_dev(kb[None, :prompt], src_type), to_dev(vb[None, :prompt], src_type), int_dev(table[:1]),
                 int_dev([0]), dev_status=status)
    for b in range(1, rows):
        table[b] = pool.fork(0, b, prompt, ps, width)
    assert pool.check() == 0 and pool.page_refs(int(table[0, 0])) == rows
    assert np.array_equal(table, np.repeat(table[:1], rows, 0))
    if quant == "per_group64":      # the open group's originals of the prompt, for each row's appends
        cache.copy_pages([], [], [0] * (rows - 1), list(range(1, rows)))
    group, prefix = int_dev([0] * rows), int_dev([prompt])
    copied = 0
    lens = np.full(rows, prompt, dtype=np.int32)
    for step in range(steps):
        for b in range(rows):
            src, dst, table[b] = pool.unshare(b, int(lens[b]), ps, width)
            cache.copy_pages(src, dst)
            copied += len(src)
            table[b] = pool.reserve(b, int(lens[b]) + 1, ps, width)
        if step == 9:
            pool.free(99)
            src, dst = pool.compact()
            assert len(src) > 0 and pool.check() == 0
            dev = int_dev(table)
            cache.copy_pages(src, dst)
            cache.remap_table(dev, src, dst)
            table = dev.cpu().numpy()
            assert table.max() < 40 - pool.num_free
            for b in range(rows):
                assert np.array_equal(table[b], pool.table(b, width))
            for p in src:           # what was left behind is no longer read
                for t in parts(cache):
                    if t is not cache.tail:
                        t[int(p)] = float("nan") if t.dtype.is_floating_point else 0
        at = prompt + step
        kb = np.stack([sb.bits[b][0][at] for b in range(rows)])[:, None]
        vb = np.stack([sb.bits[b][1][at] for b in range(rows)])[:, None]
        table_dev = int_dev(table)
        cache.append(to_dev(kb, src_type), to_dev(vb, src_type), table_dev, int_dev(lens), dev_status=status)
        lens += 1
        if step % 4 == 3 or step < 2:
            q, qf = sb.queries(g, seed=step)
            out = cache.shared_attention(q, table_dev, int_dev(lens), group, prefix, dev_status=status)
            torch.cuda.synchronize()
            if kind == "i8g" and lens[0] < prompt + steps:
                # the open group's codes depend on its members so far
                full = [(sb.k[b], sb.v[b]) for b in range(rows)]
                for b in range(rows):
                    sb.k[b] = restore(kind, sb.bits[b][0][:lens[b]].view(np.float16).astype(np.float32))[0]
                    sb.v[b] = restore(kind, sb.bits[b][1][:lens[b]].view(np.float16).astype(np.float32))[0]
                sb.check(out, qf, g, lens=lens)
                for b in range(rows):
                    sb.k[b], sb.v[b] = full[b]
            else:
                sb.check(out, qf, g, lens=lens)
    # the prompt's open page was split off by all rows but the last to write
    assert copied == rows - 1
    assert int(status.item()) == 0
    for b in range(rows):
        pool.free(b)
    assert pool.num_free == 40 and pool.check() == 0
    assert spare[0] == 0
