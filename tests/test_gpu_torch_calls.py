"""The calls that go from torch tensors to the library without Python in between: the same results, and the same
refusals, as the methods' own way."""
import threading

import numpy as np
import pytest
import torch

from shared_batch import int_dev
from test_gpu_rotary import Step, bits_of
from tree_batch import TreeBatch

pytestmark = pytest.mark.gpu


def both_ways(cache, call):
    """call() without and with the short way; whether the short one was taken."""
    native = cache._native
    assert native is not None, "the host code for torch tensors is not built"
    cache._native = None
    slow = call()
    cache._native = native
    taken = []
    real = cache._calls

    class Spy:
        def __getattr__(self, name):
            def f(*a):
                got = getattr(real, name)(*a)
                taken.append(got is not NotImplemented)
                return got
            return f
    cache._calls = Spy()
    fast = call()
    cache._calls = real
    torch.cuda.synchronize()
    return slow, fast, taken


@pytest.mark.parametrize("kind", ["bf16", "i8t", "i8g"])
def test_rotary_appends(kind):
    s = Step(kind, 2, 3, 64, 64, 3, 4, 32, True, 7, positions=[0, 64, 128], lens=[4, 2, 3], packed=True, turns=True)
    out = torch.zeros((3, 4, 6, 64), dtype=s.q.dtype, device="cuda")
    slow, fast, taken = both_ways(s.cache, lambda: s.run(q_out=out).clone())
    assert taken == [True]
    s.check(slow)
    s.check(fast)
    assert np.array_equal(bits_of(slow), bits_of(fast))
    s.cache.k_pages.zero_()
    _, fast, taken = both_ways(s.cache, s.run)
    assert taken == [True]
    s.check(fast)
    # given a stream, and without queries
    side = torch.cuda.Stream()
    _, fast, taken = both_ways(s.cache, lambda: s.run(stream=side))
    assert taken == [True]
    s.check(fast)
    args = (None, s.k, s.v, s.cs_dev, int_dev(s.table), int_dev(s.pos))
    slow, fast, taken = both_ways(s.cache, lambda: s.cache.rotary_append(*args))
    assert slow is None and fast is None and taken == [False]


def test_trees():
    tb = TreeBatch("f16", 2, 64, 16, [300, 40, 9], 9, seed=3)
    q, qf = tb.tree_queries(3)
    for kw in ({}, dict(mask=tb.mask[0].contiguous()), dict(mask=None), dict(sm_scale=0.3), dict(num_splits=5),
               dict(out_dtype=torch.float16), dict(out=torch.zeros_like(q)), dict(stream=torch.cuda.Stream())):
        tb.tree_run(q, **kw)        # its workspace is there
        slow, fast, taken = both_ways(tb.cache, lambda: tb.tree_run(q, **kw).clone())
        assert taken == [True] and slow.dtype == fast.dtype and torch.equal(slow, fast)
    # the first call of a shape makes its memory, and a captured one its own
    q2 = q[:, :8].contiguous()
    call = lambda: tb.cache.tree_attention(q2, tb.table_dev, tb.lens_dev)  # noqa: E731
    got = call()
    tb.cache._shared_fit.clear()
    slow, fast, taken = both_ways(tb.cache, call)
    assert taken == [True] and torch.equal(got, fast)
    graph = torch.cuda.CUDAGraph()
    out = torch.empty_like(got)
    with torch.cuda.graph(graph):
        tb.cache.tree_attention(q2, tb.table_dev, tb.lens_dev, out=out)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, got)


def test_kept_tokens():
    for given in (True, False):
        tb = TreeBatch("u4t", 2, 64, 16, [100, 60], 9, seed=4)
        before = tb.cache.k_pages.clone()
        keep, lens, first = int_dev([[1, 4, 7], [0, 3, 5]]), int_dev([3, 2]), int_dev(tb.lens - 9)
        states = []

        def call():
            tb.cache.k_pages.copy_(before)
            tb.cache.keep_tokens(keep, lens if given else None, tb.table_dev, first, dev_status=tb.status)
            states.append(tb.cache.k_pages.clone())
        _, _, taken = both_ways(tb.cache, call)
        assert taken == [True] and torch.equal(*states) and not torch.equal(states[0], before)


def test_refusals_are_the_methods_own():
    s = Step("bf16", 2, 3, 64, 16, 3, 4, 32, True, 7)
    from paged_kv_cache_243_gb300 import binding as B
    table, pos = int_dev(s.table), int_dev(s.pos)
    good = dict(q=s.q, k_new=s.k, v_new=s.v, cos_sin=s.cs_dev, block_table=table, positions=pos)
    for kw, error in ((dict(q=s.q.half()), TypeError), (dict(k_new=s.k[:, :2]), ValueError), (dict(positions=pos.long()), TypeError),
                      (dict(positions=pos.cpu()), (TypeError, ValueError)), (dict(cos_sin=s.cs_dev[:, :24].contiguous()), B.PkvError),
                      (dict(v_new=s.v.transpose(2, 3)), ValueError), (dict(q=s.q.float(), k_new=s.k.float(), v_new=s.v.float()), B.PkvError)):
        with pytest.raises(error):
            s.cache.rotary_append(**{**good, **kw})
    tb = TreeBatch("f16", 2, 64, 16, [300, 40, 9], 9, seed=3)
    q, _ = tb.tree_queries(3)
    good = dict(q=q, block_table=tb.table_dev, seq_lens=tb.lens_dev, mask=tb.mask)
    for kw, error in ((dict(q=q.bfloat16()), B.PkvError), (dict(mask=tb.mask[:2]), ValueError), (dict(sm_scale=-1.0), B.PkvError),
                      (dict(out_dtype=torch.int32), TypeError), (dict(num_splits=-1), B.PkvError), (dict(seq_lens=tb.lens_dev[:2]), ValueError),
                      (dict(q=q.transpose(1, 2)), ValueError)):
        with pytest.raises(error):
            tb.cache.tree_attention(**{**good, **kw})
    group = Step("i8g", 2, 3, 64, 64, 3, 4, 32, True, 7, positions=[0, 0, 64])
    for kw, error in ((dict(keep=int_dev([[0], [0]])), ValueError), (dict(keep=int_dev([[0]] * 3)), B.PkvError)):
        with pytest.raises(error):
            group.cache.keep_tokens(**{**dict(keep=None, keep_lens=None, block_table=int_dev(group.table), first=int_dev(group.pos)), **kw})


def test_threads_take_turns_on_a_workspace():
    # trees the short way, trees with a lock held elsewhere, and shared prefixes, all on one stream
    tb = TreeBatch("f16", 2, 64, 16, [500, 90], 10, seed=26)
    q, _ = tb.tree_queries(2)
    one, groups = q[:, 0].contiguous(), (int_dev([-1, -1]), int_dev([0]))
    calls = [lambda: tb.cache.tree_attention(q, tb.table_dev, tb.lens_dev, tb.mask, tb.drafts_dev),
             lambda: tb.cache.tree_attention(q[:, :4].contiguous(), tb.table_dev, tb.lens_dev),
             lambda: tb.cache.shared_attention(one, tb.table_dev, tb.lens_dev, *groups)]
    refs = [c() for c in calls]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        for _ in range(150):
            if not torch.equal(calls[i](), refs[i]):
                wrong.append(i)
    threads = [threading.Thread(target=work, args=(i,)) for i in (0, 1, 2, 0)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


def test_status_words_elsewhere_are_refused():
    # (the kernels would write to the host's memory)
    s = Step("bf16", 2, 3, 64, 16, 3, 4, 32, True, 7)
    table, pos = int_dev(s.table), int_dev(s.pos)
    for word, error in ((torch.zeros(1, dtype=torch.int32), ValueError), (torch.zeros(1, dtype=torch.int64, device="cuda"), TypeError)):
        for call in (lambda: s.cache.rotary_append(s.q, s.k, s.v, s.cs_dev, table, pos, dev_status=word),
                     lambda: s.cache.tree_attention(s.q.contiguous(), table, pos, dev_status=word),
                     lambda: s.cache.keep_tokens(int_dev([[0]] * 3), None, table, pos, dev_status=word)):
            with pytest.raises(error):
                call()


def test_a_failed_launch_is_an_error_of_the_library():
    # the entry points' place is taken by one that reports a failed launch
    import ctypes
    from paged_kv_cache_243_gb300 import binding as B
    s = Step("bf16", 2, 3, 64, 16, 3, 4, 32, True, 7)
    table, pos = int_dev(s.table), int_dev(s.pos)
    L, calls = B.lib(), s.cache._calls
    q = s.q.contiguous()
    s.cache.tree_attention(q, table, pos + 4)      # (makes the workspace)
    fails = ctypes.CFUNCTYPE(ctypes.c_int)(lambda: 4)
    at = [ctypes.cast(f, ctypes.c_void_p).value for f in (L.pkv_rotary_append, L.pkv_tree_attention, L.pkv_keep_tokens)]
    torch.cuda.synchronize()
    calls.bind(*[ctypes.cast(fails, ctypes.c_void_p).value] * 3, B.PkvError)
    try:
        for call, name in ((lambda: s.cache.rotary_append(s.q, s.k, s.v, s.cs_dev, table, pos), "rotary_append"),
                           (lambda: s.cache.tree_attention(q, table, pos + 4), "tree_attention"),
                           (lambda: s.cache.keep_tokens(int_dev([[0]] * 3), None, table, pos), "keep_tokens")):
            with pytest.raises(B.PkvError) as e:
                call()
            assert e.value.status == 4 and str(e.value).startswith(name)
    finally:
        calls.bind(*at, B.PkvError)
    s.cache.tree_attention(q, table, pos + 4)      # (no lock was kept)
    torch.cuda.synchronize()
