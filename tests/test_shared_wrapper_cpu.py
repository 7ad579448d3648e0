"""What the wrappers for shared pages hand to the library, without a GPU: the device they make
current, the stream they launch on, and the memory they keep."""
import contextlib
import threading
import time
import types

import pytest
import torch

BYTES = {}     # batch -> workspace bytes that the stand-in for the library asks for


class Calls(list):
    def named(self, name):
        return [c[1] for c in self if c[0] == name]


@pytest.fixture
def fake(monkeypatch):
    """cache.py over a recording binding; cache tensors are on the CPU and taken for device 1's."""
    from paged_kv_cache_243_gb300 import cache as C
    calls, state = Calls(), types.SimpleNamespace(current=0, streams={0: 100, 1: 111}, capturing=False)

    @contextlib.contextmanager
    def on_device(device):
        before, state.current = state.current, int(getattr(device, "index", device))
        yield
        state.current = before

    @contextlib.contextmanager
    def on_stream(s):
        before, dev = dict(state.streams), state.current
        state.streams[s.device_index], state.current = s.cuda_stream, s.device_index
        yield
        state.streams.update(before)
        state.current = dev

    def record(name):
        return lambda *a, **k: calls.append((name, dict(device=state.current, args=a)))

    monkeypatch.setattr(torch.cuda, "current_device", lambda: state.current)
    monkeypatch.setattr(torch.cuda, "device", on_device)
    monkeypatch.setattr(torch.cuda, "stream", on_stream)
    monkeypatch.setattr(C, "_capturing", lambda: state.capturing)
    monkeypatch.setattr(C, "_raw_stream", lambda index: state.streams[1])
    for name in ("copy_pages", "remap_block_table", "shared_prefix_attention"):
        monkeypatch.setattr(C.B, name, record(name))
    monkeypatch.setattr(C.B, "shared_prefix_workspace_bytes", lambda d, b, h, n: BYTES.get(b, 1000 * b) + n)
    pages = torch.zeros(8, 2, 16, 64, dtype=torch.float16)
    cache = C.PagedKVCache.from_pools(pages, pages.clone(), kv_dtype="f16")
    real = C.PagedKVCache._on_device
    there = types.SimpleNamespace(device=torch.device("cuda", 1))
    monkeypatch.setattr(C.PagedKVCache, "_on_device", lambda self: real(there))
    return cache, calls, state


def arguments(batch):
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    return (torch.zeros(batch, 4, 64, dtype=torch.float16), i32(batch, 2), i32(batch), i32(batch), i32(1))


def kept(cache):
    return sum({t.data_ptr(): t.nbytes for d in (cache._ws, cache._shared_ws, cache._shared_fit, cache._shared_lent)
                for t in d.values()}.values())


def test_calls_go_to_the_caches_device_and_its_current_stream(fake):
    cache, calls, state = fake
    cache.copy_pages([1], [2])
    cache.remap_table(torch.zeros(1, 2, dtype=torch.int32), [1], [2])
    cache.shared_attention(*arguments(3))
    assert len(calls) == 3 and all(c[1]["device"] == 1 for c in calls) and state.current == 0
    state.current = 1
    cache.copy_pages([1], [2])
    assert calls.pop()[1]["device"] == 1 and state.current == 1
    assert [c["args"][-1] for c in calls.named("copy_pages")] == [111]
    assert [c["args"][-1] for c in calls.named("remap_block_table")] == [111]
    assert [c["args"][-1] for c in calls.named("shared_prefix_attention")] == [111]


def test_a_stream_given_is_the_calls(fake):
    cache, calls, state = fake
    s = types.SimpleNamespace(cuda_stream=222, device_index=1)
    cache.copy_pages([1], [2], stream=s)
    cache.remap_table(torch.zeros(1, 2, dtype=torch.int32), [1], [2], stream=s)
    cache.shared_attention(*arguments(3), stream=s)
    assert [c[1]["args"][-1] for c in calls] == [222] * 3 and all(c[1]["device"] == 1 for c in calls)
    assert set(cache._shared_ws) == {222} and state.current == 0 and state.streams[1] == 111


def test_batches_of_every_size_keep_one_workspace_a_stream(fake):
    cache, calls, state = fake
    for order in (range(1, 257), range(256, 0, -1)):
        for b in order:
            cache.shared_attention(*arguments(b))
    assert 256000 <= kept(cache) <= 1.25 * 256000
    for (ws, n), b in zip(((c["args"][15], c["args"][16]) for c in calls.named("shared_prefix_attention")),
                          list(range(1, 257)) + list(range(256, 0, -1))):
        assert ws != 0 and n >= 1000 * b
    cache.shared_attention(*arguments(4), num_splits=7)
    assert kept(cache) <= 1.25 * 256000
    state.streams[1] = 112
    cache.shared_attention(*arguments(2))
    assert kept(cache) <= 1.25 * 256000 + 2000


def test_a_workspace_lent_out_stays_and_the_sizes_lent_stay_bounded(fake):
    cache, calls, state = fake
    lent = [cache.shared_workspace(b, 4) for b in range(1, 257)]
    held = {t.data_ptr() for t in lent}
    assert held <= set(cache._shared_lent) and kept(cache) <= 6 * 256000
    assert all(t.numel() >= 1000 * b for b, t in enumerate(lent, 1))
    assert cache.shared_workspace(256, 4) is cache.shared_workspace(1, 4)


def test_a_captured_call_has_a_workspace_of_its_own(fake):
    cache, calls, state = fake
    cache.shared_attention(*arguments(3))
    own = cache._shared_ws[111]
    state.capturing = True
    for _ in range(3):
        cache.shared_attention(*arguments(9))
    state.capturing = False
    ws = [c["args"][15] for c in calls.named("shared_prefix_attention")]
    assert own.data_ptr() == ws[0] not in ws[1:] and cache._shared_ws[111] is own and kept(cache) == 3000
    state.capturing = True
    cache.shared_workspace(9, 4)
    assert kept(cache) == 3000      # a graph's memory goes with the graph


def test_threads_take_turns_on_the_workspace(fake, monkeypatch):
    # a call is two launches with records in between: another thread's may not come between them
    from paged_kv_cache_243_gb300 import cache as C
    cache, calls, state = fake
    inside, most = [], []

    def call(*args):
        inside.append(args[1])
        most.append(len(inside))
        time.sleep(0.002)
        inside.remove(args[1])

    monkeypatch.setattr(C.B, "shared_prefix_attention", call)
    state.current = 1
    monkeypatch.setattr(C.PagedKVCache, "_on_device", lambda self: contextlib.nullcontext())
    threads = [threading.Thread(target=lambda b=b: [cache.shared_attention(*arguments(b)) for _ in range(10)])
               for b in (2, 3, 5)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert len(most) == 30 and max(most) == 1
