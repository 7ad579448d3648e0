"""Memory that shared_attention keeps and uses by default: how much of it, and who else uses it."""
import pytest
import torch

from shared_batch import SharedBatch

pytestmark = pytest.mark.gpu


def batch(rows, seed):
    sb = SharedBatch("bf16", 2, 64, 16, [(400, [20] * rows)], alone=[33], seed=seed)
    return sb, sb.queries(4, seed=seed)[0]


def first(sb, q, n, **kw):
    """The call for the first n rows."""
    return sb.cache.shared_attention(q[:n], sb.table_dev[:n], sb.lens_dev[:n], sb.group_dev[:n], sb.prefix_dev, **kw)


def forget(cache):
    for kept in (cache._shared_ws, cache._shared_fit, cache._shared_lent):
        kept.clear()


def test_every_batch_size_leaves_one_workspace():
    sb, q = batch(47, 1)
    ws = torch.empty_like(sb.cache.shared_workspace(48, 8))
    refs = {n: first(sb, q, n, workspace=ws) for n in range(1, 49)}
    most = ws.numel()
    forget(sb.cache)
    before = torch.cuda.memory_allocated()
    for n in list(range(1, 49)) + list(range(48, 0, -1)):
        assert torch.equal(first(sb, q, n), refs[n])
    assert torch.cuda.memory_allocated() - before <= 1.25 * most + (1 << 20)


def test_graphs_keep_their_workspace_when_larger_batches_come():
    sb, q = batch(47, 2)
    large = first(sb, q, 48)
    forget(sb.cache)
    ref = first(sb, q, 4)
    out = torch.empty_like(ref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        first(sb, q, 4, out=out)
    for n in (8, 20, 48):
        first(sb, q, n)
        junk = [torch.full((1 << 22,), float("nan"), device="cuda") for _ in range(8)]
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ref)
        del junk
    # memory of the graph's pool that a replay writes is nobody else's
    for _ in range(5):
        graph.replay()
        other = first(sb, q, 48)
    torch.cuda.synchronize()
    assert torch.equal(other, large) and torch.equal(out, ref)


def test_graphs_captured_on_one_stream_run_beside_each_other_and_beside_calls():
    sb, q = batch(23, 3)
    ref = first(sb, q, 24)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    outs, graphs = [torch.empty_like(ref) for _ in range(3)], []
    for o in outs[:2]:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            for _ in range(8):
                first(sb, q, 24, out=o)
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        with torch.cuda.stream(s):
            for _ in range(4):
                first(sb, q, 24, out=outs[2])
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o, ref)
