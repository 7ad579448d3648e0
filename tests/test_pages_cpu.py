"""Page sharing without a GPU: the allocator's fork, unshare and compact rules, and every
refusal of the calls that copy, rename and read shared pages."""
import numpy as np
import pytest


@pytest.fixture(scope="module")
def B():
    from paged_kv_cache_243_gb300 import _build, binding
    _build.build()
    binding.lib()
    return binding


@pytest.fixture
def pool(B):
    from paged_kv_cache_243_gb300.cache import PageAllocator
    a = PageAllocator(12)
    yield a
    a.close()


def refused(B, status, call, *args):
    with pytest.raises(B.PkvError) as e:
        call(*args)
    assert e.value.status == status


def test_fork_shares_pages_until_the_last_owner_frees_them(B, pool):
    assert pool.reserve(1, 40, 16, 6).tolist() == [0, 1, 2, -1, -1, -1]
    assert pool.fork(1, 2, 40, 16, 6).tolist() == [0, 1, 2, -1, -1, -1]
    assert pool.fork(1, 3, 16, 16, 6).tolist() == [0, -1, -1, -1, -1, -1]    # a shorter prefix
    assert pool.fork(2, 4, 0, 16, 6).tolist() == [-1] * 6                    # no tokens
    assert [pool.page_refs(p) for p in range(4)] == [3, 2, 2, 0] and pool.num_free == 9 and pool.check() == 0
    assert pool.page_refs(-1) == 0 and pool.page_refs(12) == 0
    pool.free(1)
    assert pool.num_free == 9 and pool.check() == 0
    pool.free(2)
    assert pool.num_free == 11 and [pool.page_refs(p) for p in range(3)] == [1, 0, 0]
    pool.free(3)
    pool.free(4)
    assert pool.num_free == 12 and pool.check() == 0


def test_fork_refusals_change_nothing(B, pool):
    pool.reserve(1, 40, 16, 6)
    refused(B, B.ERR_INVALID_ARG, pool.fork, 7, 2, 16, 16, 6)      # no such parent
    refused(B, B.ERR_INVALID_ARG, pool.fork, 1, 1, 16, 16, 6)      # the child exists
    refused(B, B.ERR_INVALID_ARG, pool.fork, 1, 2, 49, 16, 6)      # more than the parent has
    refused(B, B.ERR_INVALID_ARG, pool.fork, 1, 2, 40, 16, 2)      # a row too short
    refused(B, B.ERR_INVALID_ARG, pool.fork, 1, 2, -1, 16, 6)
    refused(B, B.ERR_INVALID_ARG, pool.fork, 1, 2, 16, 0, 6)
    assert pool.seq_pages(2) == 0 and pool.check() == 0 and pool.page_refs(0) == 1


def test_unshare_replaces_only_shared_pages(B, pool):
    pool.reserve(1, 40, 16, 6)
    pool.fork(1, 2, 40, 16, 6)
    src, dst, row = pool.unshare(2, 40, 16, 6)       # the page of token 40, the next to be written
    assert (src.tolist(), dst.tolist(), row.tolist()) == ([2], [3], [0, 1, 3, -1, -1, -1])
    src, dst, row = pool.unshare(1, 40, 16, 6)       # the other owner has the page to itself now
    assert src.size == 0 and row.tolist() == [0, 1, 2, -1, -1, -1]
    src, dst, row = pool.unshare(2, 0, 16, 6)
    assert (src.tolist(), dst.tolist(), row.tolist()) == ([0, 1], [4, 5], [4, 5, 3, -1, -1, -1])
    assert pool.check() == 0 and pool.num_free == 6
    src, dst, row = pool.unshare(2, 1000, 16, 6)     # past its pages: nothing to do
    assert src.size == 0 and pool.check() == 0


def test_unshare_refusals_change_nothing(B, pool):
    pool.reserve(1, 40, 16, 6)
    pool.fork(1, 2, 40, 16, 6)
    pool.reserve(3, 8 * 16, 16, 8)                   # one page left
    refused(B, B.ERR_OUT_OF_PAGES, pool.unshare, 2, 0, 16, 6)
    refused(B, B.ERR_INVALID_ARG, pool.unshare, 9, 0, 16, 6)
    refused(B, B.ERR_INVALID_ARG, pool.unshare, 2, -1, 16, 6)
    refused(B, B.ERR_INVALID_ARG, pool.unshare, 2, 0, 16, 2)       # a row too short
    src, dst, row = (np.zeros(6, dtype=np.int32) for _ in range(3))
    refused(B, B.ERR_INVALID_ARG, B.alloc_unshare, pool._h, 2, 0, 16, 2, src.ctypes.data, dst.ctypes.data,
            row.ctypes.data, 6)                      # room for two copies, three needed
    assert pool.table(2, 6).tolist() == [0, 1, 2, -1, -1, -1] and pool.check() == 0 and pool.num_free == 1
    src, dst, row = pool.unshare(2, 40, 16, 6)
    assert (src.tolist(), dst.tolist()) == ([2], [11])


def test_compact_moves_the_highest_pages_into_the_lowest_holes(B, pool):
    pool.reserve(1, 32, 16, 6)      # 0 1
    pool.reserve(2, 48, 16, 6)      # 2 3 4
    pool.reserve(3, 32, 16, 6)      # 5 6
    pool.fork(3, 4, 32, 16, 6)
    pool.free(2)
    src, dst = pool.compact()
    assert (src.tolist(), dst.tolist()) == ([6, 5], [2, 3])
    assert pool.table(1, 3).tolist() == [0, 1, -1]
    assert pool.table(3, 3).tolist() == [3, 2, -1] == pool.table(4, 3).tolist()
    assert pool.page_refs(2) == 2 and pool.page_refs(6) == 0 and pool.check() == 0 and pool.num_free == 8
    src, dst = pool.compact()
    assert src.size == 0
    refused(B, B.ERR_INVALID_ARG, pool.table, 2, 3)
    refused(B, B.ERR_INVALID_ARG, pool.table, 3, 1)


def test_compact_in_steps_and_free_list_order(B, pool):
    pool.reserve(1, 64, 16, 6)      # 0 1 2 3
    pool.reserve(2, 64, 16, 6)      # 4 5 6 7
    pool.free(1)
    src, dst = pool.compact(1)
    assert (src.tolist(), dst.tolist()) == ([7], [0]) and pool.check() == 0
    src, dst = pool.compact(0)
    assert src.size == 0
    src, dst = pool.compact(100)
    assert (src.tolist(), dst.tolist()) == ([6, 5, 4], [1, 2, 3]) and pool.check() == 0
    assert pool.table(2, 4).tolist() == [3, 2, 1, 0]
    # the rest of the list in its order, then the pages left, in the order they were left
    assert pool.reserve(3, 128, 16, 8).tolist() == [8, 9, 10, 11, 7, 6, 5, 4]
    refused(B, B.ERR_INVALID_ARG, pool.compact, -1)


def test_random_life_of_a_pool(B):
    from paged_kv_cache_243_gb300.cache import PageAllocator
    rng = np.random.default_rng(4)
    a, ps, width, live, content = PageAllocator(60), 16, 12, {}, {}
    for step in range(1500):
        op = rng.integers(0, 6)
        ids = sorted(live)
        try:
            if op == 0 or not ids:
                s, n = int(step) + 1000, int(rng.integers(0, 80))
                live[s] = [int(p) for p in a.reserve(s, n, ps, width) if p >= 0]
            elif op == 1:
                s, n = int(rng.choice(ids)), int(rng.integers(0, 150))
                live[s] = [int(p) for p in a.reserve(s, n, ps, width) if p >= 0]
            elif op == 2:
                s = int(rng.choice(ids))
                n = int(rng.integers(0, len(live[s]) * ps + 1))
                live[step] = [int(p) for p in a.fork(s, step, n, ps, width) if p >= 0]
            elif op == 3:
                s, t = int(rng.choice(ids)), int(rng.integers(0, 100))
                src, dst, row = a.unshare(s, t, ps, width)
                to = dict(zip(src.tolist(), dst.tolist()))
                live[s] = [to.get(p, p) if i >= t // ps else p for i, p in enumerate(live[s])]
                assert live[s] == [int(p) for p in row if p >= 0]
            elif op == 4:
                src, dst = a.compact(int(rng.integers(0, 20)))
                assert not set(src.tolist()) & set(dst.tolist()) and len(set(dst.tolist())) == dst.size
                to = dict(zip(src.tolist(), dst.tolist()))
                live = {s: [to.get(p, p) for p in pages] for s, pages in live.items()}
            else:
                s = int(rng.choice(ids))
                a.free(s)
                del live[s]
        except B.PkvError as e:
            assert e.status in (B.ERR_OUT_OF_PAGES, B.ERR_INVALID_ARG)
        assert a.check() == 0
        refs = np.zeros(60, dtype=int)
        for pages in live.values():
            refs[pages] += 1
        assert a.num_free == int((refs == 0).sum())
    for s, pages in live.items():
        assert a.table(s, width)[:len(pages)].tolist() == pages
    a.close()


# ------------------------------------------------------------ refusals, no CUDA call reached
def _desc(B, **kw):
    d = dict(num_pages=8, page_size=16, num_kv_heads=2, head_dim=64, kv_dtype=B.F16,
             quant=B.QUANT_NONE, k_pages=0x1000, v_pages=0x2000, kv_sz=0, tail=0, tail_rows=0, page_meta=0)
    d.update(kw)
    return B.PkvCache(**d)


def ids(*a):
    return np.array(a, dtype=np.int32)


@pytest.mark.parametrize("src,dst", [((8,), (1,)), ((-1,), (1,)), ((1,), (8,)), ((1,), (-1,)), ((1,), (1,)),
                                     ((1, 2), (3, 3)), ((1, 2), (2, 3)), ((1, 2), (3, 1))])
def test_copy_list_refusals(B, src, dst):
    s, d = ids(*src), ids(*dst)
    refused(B, B.ERR_INVALID_ARG, B.copy_pages, _desc(B), len(src), s.ctypes.data, d.ctypes.data, 0, 0, 0, 0)
    grouped = _desc(B, kv_dtype=B.I8, quant=B.QUANT_PER_GROUP64, kv_sz=0x3000, page_size=64, tail=0x4000,
                    tail_rows=8)
    refused(B, B.ERR_INVALID_ARG, B.copy_pages, grouped, 0, 0, 0, len(src), s.ctypes.data, d.ctypes.data, 0)
    if dst != (3, 3):       # two sources may become one page, everything else is refused alike
        t = np.zeros(4, dtype=np.int32)
        refused(B, B.ERR_INVALID_ARG, B.remap_block_table, t.ctypes.data, 1, 4, 8, len(src), s.ctypes.data,
                d.ctypes.data, 0)


def test_copy_and_remap_refusals(B):
    one, two = ids(1), ids(2)
    p = (one.ctypes.data, two.ctypes.data)
    refused(B, B.ERR_INVALID_ARG, B.copy_pages, _desc(B), -1, *p, 0, 0, 0, 0)
    refused(B, B.ERR_INVALID_ARG, B.copy_pages, _desc(B), 1, 0, p[1], 0, 0, 0, 0)
    refused(B, B.ERR_INVALID_ARG, B.copy_pages, _desc(B), 0, 0, 0, 1, *p, 0)          # rows without a tail
    refused(B, B.ERR_INVALID_ARG, B.copy_pages, _desc(B, k_pages=0x1001), 1, *p, 0, 0, 0, 0)
    refused(B, B.ERR_UNSUPPORTED, B.copy_pages, _desc(B, head_dim=96), 1, *p, 0, 0, 0, 0)
    refused(B, B.ERR_INVALID_ARG, B.remap_block_table, 0, 1, 4, 8, 1, *p, 0)
    refused(B, B.ERR_INVALID_ARG, B.remap_block_table, 0x1002, 1, 4, 8, 1, *p, 0)
    refused(B, B.ERR_INVALID_ARG, B.remap_block_table, 0x1000, -1, 4, 8, 1, *p, 0)
    refused(B, B.ERR_INVALID_ARG, B.remap_block_table, 0x1000, 1, 0, 8, 1, *p, 0)
    refused(B, B.ERR_INVALID_ARG, B.remap_block_table, 0x1000, 1, 4, 0, 1, *p, 0)
    twice, to = ids(1, 1), ids(2, 3)
    refused(B, B.ERR_INVALID_ARG, B.remap_block_table, 0x1000, 1, 4, 8, 2, twice.ctypes.data, to.ctypes.data, 0)
    # nothing to do is no error
    B.copy_pages(_desc(B), 0, 0, 0, 0, 0, 0, 0)
    B.remap_block_table(0x1000, 1, 4, 8, 0, 0, 0, 0)
    B.remap_block_table(0, 0, 4, 8, 1, *p, 0)


def test_shared_attention_refusals(B):
    def call(desc, status, batch=2, hq=4, q=0x4000, qd=None, scale=0.125, table=0x5000, mp=4, lens=0x6000,
             group=0x7000, prefix=0x8000, ng=1, out=0x9000, od=None, splits=0, ws=0x10000, n=1 << 30):
        refused(B, status, B.shared_prefix_attention, desc, batch, hq, q, B.F16 if qd is None else qd, scale, table,
                mp, lens, group, prefix, ng, out, B.F32 if od is None else od, splits, ws, n, 0, 0)

    good, bad, no = _desc(B), B.ERR_INVALID_ARG, B.ERR_UNSUPPORTED
    call(good, bad, q=0)
    call(good, bad, q=0x4008)
    call(good, bad, out=0x9004)
    call(good, bad, table=0)
    call(good, bad, lens=0)
    call(good, bad, group=0)
    call(good, bad, prefix=0)
    call(good, bad, ng=-1)
    call(good, bad, mp=0)
    call(good, bad, batch=-1)
    call(good, bad, hq=3)
    call(good, bad, hq=0)
    call(good, bad, splits=-1)
    call(good, bad, scale=0.0)
    call(good, bad, scale=float("nan"))
    call(good, bad, qd=B.I8)
    call(good, bad, od=B.U4)
    call(good, no, qd=B.BF16)                     # q of another type than an fp16 cache
    call(good, no, qd=B.F32)
    call(good, no, batch=1025)
    call(good, no, ng=1025)
    call(good, no, hq=2 * 129)
    call(good, no, mp=1 << 28)                    # positions past 32 bits
    call(_desc(B, num_pages=1 << 30), no)         # pool rows past 32 bits
    call(_desc(B, head_dim=96), no)
    call(_desc(B, page_size=24), no)
    call(_desc(B, v_pages=0), bad)
    assert B.shared_prefix_workspace_bytes(good, 0, 4, 1) > 0
    refused(B, bad, B.shared_prefix_workspace_bytes, good, 2, 3, 0)
    # an empty batch is no error
    B.shared_prefix_attention(good, 0, 4, 0x4000, B.F16, 0.125, 0x5000, 4, 0x6000, 0x7000, 0x8000, 1, 0x9000, B.F32,
                              0, 0x10000, 1 << 20, 0, 0)


def test_wrapper_refusals(B):
    import torch
    from paged_kv_cache_243_gb300.cache import PagedKVCache
    pages = torch.zeros(8, 2, 16, 64, dtype=torch.float16)
    c = PagedKVCache.from_pools(pages, pages.clone(), kv_dtype="f16")
    assert (c.num_pages, c.num_kv_heads, c.page_size, c.head_dim) == (8, 2, 16, 64)
    for args, err in ((([0, 1], [2]), ValueError), (([0.5], [1]), TypeError), (([1 << 40], [1]), ValueError),
                      (([[0]], [[1]]), TypeError)):
        with pytest.raises(err):
            c.copy_pages(*args)
    for kw in (dict(kv_dtype="bf16"), dict(kv_dtype="f16", kv_sz=torch.zeros(8, 2, 16, 4)),
               dict(kv_dtype="f16", page_meta=torch.zeros(8, 2, 2, 32)), dict(kv_dtype="int8", quant="per_token")):
        with pytest.raises((ValueError, TypeError)):
            PagedKVCache.from_pools(pages, pages.clone(), **kw)
    with pytest.raises(ValueError):
        PagedKVCache.from_pools(pages, pages.transpose(1, 2), kv_dtype="f16")
    u4 = torch.zeros(8, 2, 16, 32, dtype=torch.uint8)
    assert PagedKVCache.from_pools(u4, u4.clone(), kv_dtype="u4", quant="per_token",
                                   kv_sz=torch.zeros(8, 2, 16, 4)).head_dim == 64
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    q = torch.zeros(3, 4, 64, dtype=torch.float16)
    for bad in ((q[:, :, :32].contiguous(), i32(3, 2), i32(3), i32(3), i32(1)), (q, i32(2, 2), i32(3), i32(3), i32(1)),
                (q, i32(3, 2), i32(2), i32(3), i32(1)), (q, i32(3, 2), i32(3), i32(4), i32(1)),
                (q, i32(3, 2), i32(3), i32(3), i32(1, 1)), (q.transpose(0, 1), i32(4, 2), i32(4), i32(4), i32(1)),
                (q, i32(3, 2), i32(3).float(), i32(3), i32(1))):
        with pytest.raises((ValueError, TypeError)):
            c.shared_attention(*bad)
    with pytest.raises(ValueError):
        c.remap_table(i32(4), [1], [2])
