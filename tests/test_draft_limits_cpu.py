"""What the calls for drafted tokens refuse, and what they work out on the host, without a GPU."""
import math

import numpy as np
import pytest
import torch

from paged_kv_cache_243_gb300 import _build, binding as B


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()


def desc(**kw):
    d = dict(num_pages=8, page_size=16, num_kv_heads=2, head_dim=64, kv_dtype=B.F16, quant=B.QUANT_NONE, k_pages=0x1000,
             v_pages=0x2000, kv_sz=0, tail=0, tail_rows=0, page_meta=0)
    d.update(kw)
    return B.PkvCache(*d.values())


GROUP = dict(kv_dtype=B.I8, quant=B.QUANT_PER_GROUP64, kv_sz=0x3000, page_size=64)


def refused(call, status):
    with pytest.raises(B.PkvError) as e:
        call()
    assert e.value.status == status


def rotary(cache=None, **kw):
    a = dict(batch=1, t_new=1, num_q_heads=4, q=0x4000, k_new=0x5000, v_new=0x6000, src_dtype=B.F16, q_stride=256,
             k_stride=128, v_stride=128, cos_sin=0x7000, table_positions=100, rot_dim=64, interleaved=0,
             rotary_positions=0, block_table=0x8000, max_pages=4, positions=0x9000, new_lens=0, q_out=0xA000, dev_status=0,
             stream=0)
    a.update(kw)
    return lambda: B.rotary_append(cache or desc(), **a)


@pytest.mark.parametrize("kw", [
    dict(batch=-1), dict(t_new=-1), dict(max_pages=0), dict(num_q_heads=-1), dict(table_positions=0), dict(rot_dim=0),
    dict(rot_dim=80), dict(interleaved=2), dict(q_stride=255), dict(q_stride=248), dict(k_stride=127), dict(k_stride=132),
    dict(v_stride=120), dict(q=0), dict(q_out=0), dict(k_new=0), dict(v_new=0), dict(cos_sin=0), dict(block_table=0),
    dict(positions=0), dict(q=0x4008), dict(k_new=0x5002), dict(v_new=0x6004), dict(cos_sin=0x7004), dict(q_out=0xA008),
    dict(src_dtype=B.F32), dict(t_new=65)])
def test_rotary_append_refuses(kw):
    refused(rotary(**kw), B.ERR_INVALID_ARG)


def test_rotary_append_does_not_serve():
    refused(rotary(rot_dim=24), B.ERR_UNSUPPORTED)
    refused(rotary(batch=65536), B.ERR_UNSUPPORTED)
    refused(rotary(num_q_heads=65535, q_stride=65535 * 64), B.ERR_UNSUPPORTED)
    refused(rotary(batch=60000, t_new=30000, max_pages=4000), B.ERR_UNSUPPORTED)
    refused(rotary(desc(head_dim=96), q_stride=1 << 12, k_stride=1 << 12, v_stride=1 << 12), B.ERR_UNSUPPORTED)
    refused(rotary(desc(**GROUP)), B.ERR_INVALID_ARG)          # no originals
    refused(rotary(desc(**GROUP, tail=0xB000, tail_rows=1), batch=2), B.ERR_INVALID_ARG)
    # nothing to do
    rotary(batch=0)()
    rotary(t_new=0)()


def tree(cache=None, **kw):
    a = dict(batch=1, t_draft=4, num_q_heads=4, q=0x4000, q_dtype=B.F16, sm_scale=0.125, block_table=0x5000, max_pages=4,
             seq_lens=0x6000, draft_lens=0, tree_mask=0x7000, mask_shared=0, out=0x8000, out_dtype=B.F32, num_splits=1,
             workspace=0x10000, workspace_bytes=1 << 30, dev_status=0, stream=0)
    a.update(kw)
    return lambda: B.tree_attention(cache or desc(), **a)


@pytest.mark.parametrize("kw", [
    dict(batch=-1), dict(t_draft=-1), dict(num_q_heads=3), dict(num_q_heads=0), dict(num_splits=-1), dict(q_dtype=7),
    dict(out_dtype=B.I8), dict(max_pages=0), dict(sm_scale=0.0), dict(sm_scale=-1.0), dict(sm_scale=float("nan")),
    dict(sm_scale=1e31), dict(mask_shared=2), dict(q=0), dict(out=0), dict(block_table=0), dict(seq_lens=0), dict(q=0x4008),
    dict(out=0x8004), dict(tree_mask=0x7004)])
def test_tree_attention_refuses(kw):
    refused(tree(**kw), B.ERR_INVALID_ARG)


def test_tree_attention_does_not_serve():
    for kw in (dict(t_draft=257), dict(batch=1025), dict(num_splits=65536), dict(num_q_heads=258), dict(q_dtype=B.F32),
               dict(q_dtype=B.BF16), dict(max_pages=(1 << 27) - 16), dict(max_pages=1 << 28)):
        refused(tree(**kw), B.ERR_UNSUPPORTED)
    refused(tree(desc(num_pages=1 << 27)), B.ERR_UNSUPPORTED)
    tree(batch=0)()
    tree(t_draft=0)()
    for kw in (dict(t_draft=257), dict(batch=1025), dict(num_q_heads=3)):
        a = dict(batch=1, t_draft=4, num_q_heads=4, num_splits=1)
        a.update(kw)
        refused(lambda: B.tree_workspace_bytes(desc(), **a), B.ERR_INVALID_ARG)


def test_tree_workspace_grows_with_every_size():
    size = lambda **kw: B.tree_workspace_bytes(desc(), **{**dict(batch=2, t_draft=8, num_q_heads=4, num_splits=3), **kw})  # noqa: E731
    for kw in (dict(batch=64), dict(t_draft=256), dict(num_q_heads=256), dict(num_splits=500)):
        assert size(**kw) > size()


def keep(cache=None, **kw):
    a = dict(batch=1, max_keep=4, keep=0x4000, keep_lens=0, block_table=0x5000, max_pages=4, first=0x6000, dev_status=0,
             stream=0)
    a.update(kw)
    return lambda: B.keep_tokens(cache or desc(), **a)


def test_keep_tokens_refuses():
    for kw in (dict(batch=-1), dict(max_keep=-1), dict(max_pages=0), dict(keep=0), dict(block_table=0), dict(first=0)):
        refused(keep(**kw), B.ERR_INVALID_ARG)
    refused(keep(max_keep=257), B.ERR_UNSUPPORTED)
    refused(keep(batch=1 << 30), B.ERR_UNSUPPORTED)
    refused(keep(desc(**GROUP, tail=0xB000, tail_rows=1)), B.ERR_UNSUPPORTED)
    keep(batch=0)()


# ----------------------------------------------------------------- frequencies and masks
def frequencies(rot, base=10000.0, scaling=0, factor=1.0, low=1.0, high=4.0, original=8192.0):
    w, s = np.zeros(max(1, rot // 2)), np.zeros(1)
    B.rotary_frequencies(rot, base, scaling, factor, low, high, original, w.ctypes.data, s.ctypes.data)
    return w, float(s[0])


def test_frequencies_by_their_formulas():
    for rot in (16, 64, 128):
        i = np.arange(rot // 2)
        w = np.exp(-2 * i / rot * math.log(10000.0))
        near = lambda got, want: np.allclose(got, want, rtol=1e-13, atol=0)  # noqa: E731
        assert near(frequencies(rot)[0], w) and frequencies(rot)[1] == 1.0
        assert near(frequencies(rot, scaling=B.ROTARY_LINEAR, factor=4.0)[0], w / 4)
        scaled = frequencies(rot, scaling=B.ROTARY_BASE, factor=4.0)[0]
        assert near(scaled, np.exp(-2 * i / rot * math.log(10000.0 * 4.0 ** (rot / (rot - 2)))))
        assert near(scaled[0], 1.0) and near(scaled[-1], w[-1] / 4)        # the slowest turns `factor` times slower
        got, s = frequencies(rot, scaling=B.ROTARY_BANDS, factor=8.0, low=1.0, high=4.0, original=8192.0)
        turns = 8192 * w / (2 * math.pi)
        assert near(got[turns >= 4], w[turns >= 4]) and near(got[turns <= 1], w[turns <= 1] / 8) and s == 1.0
        mid = (turns > 1) & (turns < 4)
        part = (turns[mid] - 1) / 3
        assert near(got[mid], part * w[mid] + (1 - part) * w[mid] / 8)
        got, s = frequencies(rot, scaling=B.ROTARY_RAMP, factor=16.0, low=1.0, high=32.0, original=4096.0)
        assert s == pytest.approx(0.1 * math.log(16) + 1)
        at = lambda t: rot * math.log(4096 / (t * 2 * math.pi)) / (2 * math.log(10000.0))  # noqa: E731
        lo, hi = math.floor(at(32)), math.ceil(at(1))
        r = np.clip((i - lo) / (hi - lo), 0, 1)
        assert near(got, w / 16 * r + w * (1 - r))
        assert (np.diff(got) < 0).all()


def test_frequencies_refuse():
    for kw in (dict(base=1.0), dict(base=float("nan")), dict(scaling=5), dict(scaling=-1), dict(scaling=B.ROTARY_LINEAR, factor=0.5),
               dict(scaling=B.ROTARY_BANDS, factor=2.0, low=4.0, high=4.0), dict(scaling=B.ROTARY_RAMP, factor=2.0, low=0.0),
               dict(scaling=B.ROTARY_RAMP, factor=2.0, original=0.0), dict(scaling=B.ROTARY_BASE, factor=float("inf"))):
        refused(lambda: frequencies(64, **kw), B.ERR_INVALID_ARG)
    refused(lambda: frequencies(0), B.ERR_INVALID_ARG)
    for rot in (8, 24, 144):
        refused(lambda: frequencies(rot), B.ERR_UNSUPPORTED)
    from paged_kv_cache_243_gb300 import rotary_frequencies
    with pytest.raises(ValueError):
        rotary_frequencies(64, scaling="none such")
    refused(lambda: B.rotary_table(0, 5, 64, 0x1000, 1.0, 0), B.ERR_INVALID_ARG)
    refused(lambda: B.rotary_table(0x1000, 5, 24, 0x1000, 1.0, 0), B.ERR_UNSUPPORTED)
    refused(lambda: B.rotary_table(0x1000, -1, 64, 0x1000, 1.0, 0), B.ERR_INVALID_ARG)
    B.rotary_table(0, 0, 64, 0, 1.0, 0)


def test_tree_masks():
    from paged_kv_cache_243_gb300 import tree_mask
    rng = np.random.default_rng(0)
    for T in (1, 2, 63, 64, 65, 200):
        parents = np.stack([[-1] + [int(rng.integers(-1, t)) for t in range(1, T)] for _ in range(3)])
        mask = tree_mask(parents)
        assert mask.shape == (3, T, -(-T // 64)) and mask.dtype == torch.int64
        words = mask.numpy().view(np.uint64)
        for b in range(3):
            for t in range(T):
                path, at = set(), t
                while at >= 0:
                    path.add(at)
                    at = parents[b][at]
                assert {j for j in range(T) if int(words[b, t, j // 64]) >> j % 64 & 1} == path
            assert torch.equal(tree_mask(parents[b].tolist()), mask[b])
    for bad in ([0], [-1, 1], [-2], [-1, 0, 3]):
        with pytest.raises(ValueError):
            tree_mask(bad)
    with pytest.raises(TypeError):
        tree_mask([[[-1]]])
    with pytest.raises(TypeError):
        tree_mask([0.5])


# ------------------------------------------------------------------------ the wrappers
@pytest.fixture
def cache():
    from paged_kv_cache_243_gb300.cache import PagedKVCache
    pages = torch.zeros(8, 2, 16, 64, dtype=torch.float16)
    return PagedKVCache.from_pools(pages, pages.clone(), kv_dtype="f16")


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def f16(*shape):
    return torch.zeros(shape, dtype=torch.float16)


def test_wrappers_refuse(cache):
    table, pos, cs = i32(3, 4), i32(3), torch.zeros(50, 64)
    q, k = f16(3, 5, 4, 64), f16(3, 5, 2, 64)
    good = dict(q=q, k_new=k, v_new=k, cos_sin=cs, block_table=table, positions=pos)
    wrong = [dict(q=f16(3, 4, 4, 64)), dict(k_new=f16(3, 5, 3, 64)), dict(v_new=f16(3, 5, 2, 32)), dict(block_table=i32(2, 4)),
             dict(positions=i32(2)), dict(new_lens=i32(4)), dict(rotary_positions=i32(3, 4)), dict(q=q.transpose(0, 1)),
             dict(k_new=f16(3, 5, 2, 128)[..., ::2]), dict(q_out=f16(3, 5, 4, 32)), dict(q=q[:, :, 0]), dict(cos_sin=cs[0]),
             dict(q=f16(3, 9, 4, 64)[:, ::2][:, :5].expand(3, 5, 4, 64).as_strided((3, 5, 4, 64), (1000, 512, 64, 1)))]
    for kw in wrong:
        with pytest.raises(ValueError):
            cache.rotary_append(**{**good, **kw})
    for kw in (dict(q=q.bfloat16()), dict(v_new=k.bfloat16()), dict(cos_sin=cs.double()), dict(positions=pos.long()),
               dict(block_table=table.long())):
        with pytest.raises(TypeError):
            cache.rotary_append(**{**good, **kw})
    good = dict(q=q, block_table=table, seq_lens=pos)
    m = torch.zeros(3, 5, 1, dtype=torch.int64)
    for kw in (dict(q=q[..., :32].contiguous()), dict(q=q[:, 0]), dict(seq_lens=i32(2)), dict(draft_lens=i32(5)),
               dict(mask=m[..., 0]), dict(mask=m[:2].contiguous()), dict(mask=m[:, :4].contiguous()), dict(out=f16(3, 5, 4, 32)),
               dict(q=q.transpose(1, 2)), dict(mask=torch.zeros(3, 5, 2, dtype=torch.int64))):
        with pytest.raises(ValueError):
            cache.tree_attention(**{**good, **kw})
    for kw in (dict(mask=m.int()), dict(seq_lens=pos.long())):
        with pytest.raises(TypeError):
            cache.tree_attention(**{**good, **kw})
    good = dict(keep=i32(3, 5), keep_lens=pos, block_table=table, first=pos)
    for kw in (dict(keep=i32(5)), dict(keep=i32(2, 5)), dict(keep_lens=i32(2)), dict(first=i32(1)), dict(block_table=i32(2, 4))):
        with pytest.raises(ValueError):
            cache.keep_tokens(**{**good, **kw})
    for kw in (dict(keep=i32(3, 5).long()), dict(first=pos.long())):
        with pytest.raises(TypeError):
            cache.keep_tokens(**{**good, **kw})


def test_strided_tokens(cache):
    from paged_kv_cache_243_gb300.cache import _token_stride
    x = f16(3, 5, 8, 64)
    assert _token_stride(x, "x", (3, 5, 8, 64), -1) == 512
    assert _token_stride(x[:, :, 2:4], "x", (3, 5, 2, 64), -1) == 512
    assert _token_stride(x[:, :1, 2:4], "x", (3, 1, 2, 64), -1) == 2560
    assert _token_stride(x[:1, :1, 2:4], "x", (1, 1, 2, 64), -1) == 128
    assert _token_stride(x[1:2, 2:4], "x", (1, 2, 8, 64), -1) == 512
    with pytest.raises(ValueError):      # rows that do not go on where the one before ends
        _token_stride(x[:, :4], "x", (3, 4, 8, 64), -1)


def test_tables_of_2_31_tokens_are_refused():
    # (token positions are 32-bit on the device)
    for call in (rotary, keep):
        refused(call(max_pages=1 << 27), B.ERR_UNSUPPORTED)
        call(batch=0, max_pages=(1 << 27) - 1)()


def test_status_words_are_checked(cache):
    # what the kernels write to is a word on the cache's device
    table, pos, word = i32(3, 4), i32(3), torch.zeros(1, dtype=torch.int64)
    k = f16(3, 5, 2, 64)
    for call in (lambda w: cache.rotary_append(None, k, k, torch.zeros(50, 64), table, pos, dev_status=w),
                 lambda w: cache.tree_attention(f16(3, 5, 4, 64), table, pos, dev_status=w),
                 lambda w: cache.keep_tokens(i32(3, 5), None, table, pos, dev_status=w)):
        with pytest.raises(TypeError):
            call(word)
        with pytest.raises(ValueError):
            call(torch.zeros(1, dtype=torch.int32, device="meta"))
