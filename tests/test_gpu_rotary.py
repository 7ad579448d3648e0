"""Rotary appends: rotated queries and what the cache holds are bit-exact against the fp32 definition in
numpy, through the oracle's quantisers."""
import numpy as np
import pytest
import torch

import oracle
import synth
from oracle.quant import per_group_bbox_values, per_token_bbox_values
from oracle.quant4 import per_token_u4_bbox_values
from helpers import gather, int8_codes
from shared_batch import KINDS, TORCH, int_dev, to_dev

pytestmark = pytest.mark.gpu

ALL = sorted(KINDS)


def bits_of(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


def rotated(x, cs, interleaved):
    """x [..., H, d] fp32, cs [..., rot]: every step one fp32 rounding."""
    rot = cs.shape[-1]
    c, s = cs[..., None, :rot // 2], cs[..., None, rot // 2:]
    y = x.copy()
    first, second = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    u, v = x[..., first], x[..., second]
    y[..., first] = u * c - v * s
    y[..., second] = v * c + u * s
    assert y.dtype == np.float32
    return y


class Step:
    def __init__(self, kind, hkv, g, d, ps, B, T, rot, interleaved, seed, src=None, positions=None, lens=None,
                 packed=False, turns=False, meta=False):
        from paged_kv_cache_243_gb300 import rotary_table
        from paged_kv_cache_243_gb300.cache import PagedKVCache
        kv_dtype, quant, own = KINDS[kind]
        self.kind, self.src, self.inter, self.ps, self.d, self.hkv = kind, src or own, interleaved, ps, d, hkv
        rng = np.random.default_rng([83, seed])
        hq = hkv * g
        bits, val = synth.round_to_dtype(rng.standard_normal((B, T, hq + 2 * hkv, d)).astype(np.float32), self.src)
        x = to_dev(bits, self.src)
        self.val = np.split(val, [hq, hq + hkv], 2)
        self.v_bits = bits[:, :, hq + hkv:]
        parts = [x[:, :, :hq], x[:, :, hq:hq + hkv], x[:, :, hq + hkv:]]
        self.q, self.k, self.v = parts if packed else [p.contiguous() for p in parts]
        self.pos = np.array(positions if positions is not None else rng.integers(0, 200, B), dtype=np.int32)
        self.n = np.full(B, T, dtype=np.int32) if lens is None else np.array(lens, dtype=np.int32)
        self.width = int((self.pos.max() + T) // ps + 1)
        pages = B * self.width + 2
        self.table = rng.permutation(pages)[:B * self.width].reshape(B, self.width).astype(np.int32)
        self.cache = PagedKVCache(pages, ps, hkv, d, kv_dtype=kv_dtype, quant=quant, with_meta=meta, tail_rows=B, poison=True)
        most = int(self.pos.max()) + T
        self.turns = rng.integers(0, most, (B, T)).astype(np.int32) if turns else None
        self.cs_dev = rotary_table(most, rot)
        at = self.turns if turns else self.pos[:, None] + np.arange(T)
        self.cs = self.cs_dev.cpu().numpy()[at]
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def run(self, **kw):
        out = self.cache.rotary_append(self.q, self.k, self.v, self.cs_dev, int_dev(self.table), int_dev(self.pos),
                                       rotary_positions=None if self.turns is None else int_dev(self.turns),
                                       new_lens=int_dev(self.n), interleaved=self.inter, dev_status=self.status, **kw)
        torch.cuda.synchronize()
        return out

    def check(self, out, first=None):
        """Queries, and the tokens from first[b] on (by default those of the call) of every row."""
        q, k, v = self.val
        want_q = synth.round_to_dtype(rotated(q, self.cs, self.inter), self.src)[0]
        kr = rotated(k, self.cs, self.inter)
        kp, vp = self.cache.k_pages, self.cache.v_pages
        for b, n in enumerate(self.n):
            assert np.array_equal(bits_of(out[b, :n]), want_q[b, :n])
            t = self.pos[b] + np.arange(n)
            page, slot = self.table[b, t // self.ps], t % self.ps
            for x, pool, col in ((kr, kp, 0), (v, vp, 2)):
                x = x[b, :n]
                if self.kind in ("f16", "bf16"):
                    assert np.array_equal(bits_of(pool)[page, :, slot], synth.round_to_dtype(x, self.kind)[0])
                    continue
                got = pool.cpu().numpy()[page, :, slot]
                sz = self.cache.kv_sz.cpu().numpy()
                if self.kind == "i8g":
                    assert self.pos[b] % 64 == 0
                    c, s, z = oracle.quantize_per_group(x)
                    t0 = self.pos[b] + 64 * np.arange(s.shape[0])
                    gs = sz[self.table[b, t0 // self.ps], :, t0 % self.ps // 64]
                else:
                    c, s, z = oracle.quantize_per_token(x) if self.kind == "i8t" else oracle.quantize_per_token_u4(x)
                    gs = sz[page, :, slot]
                assert np.array_equal(int8_codes(got), c) if self.kind != "u4t" else np.array_equal(got, oracle.pack_u4(c))
                assert np.array_equal(gs[..., col], s) and np.array_equal(gs[..., col + 1], z)
        assert int(self.status.item()) == 0


@pytest.mark.parametrize("kind", ALL)
@pytest.mark.parametrize("d,rot", [(64, 64), (64, 16), (64, 48), (128, 128), (128, 32), (128, 112)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_queries_and_stored_tokens_are_exact(kind, d, rot, interleaved):
    ps = 64 if kind == "i8g" else 48
    pos = [0, 64, 320] if kind == "i8g" else [0, 61, 333]
    s = Step(kind, 3, 2, d, ps, 3, 5, rot, interleaved, rot, positions=pos, lens=[5, 1, 3])
    s.check(s.run())


@pytest.mark.parametrize("kind", ALL)
@pytest.mark.parametrize("B,T,hkv,g", [(1, 1, 1, 1), (1, 1, 8, 4), (5, 1, 2, 7), (64, 1, 8, 4), (2, 300, 8, 1), (3, 70, 1, 16)])
@pytest.mark.parametrize("src", ["f16", "bf16"])
def test_batches_lengths_and_source_types(kind, B, T, hkv, g, src):
    rng = np.random.default_rng(B + T)
    pos = rng.integers(0, 5, B) * 64 if kind == "i8g" else rng.integers(0, 300, B)
    s = Step(kind, hkv, g, 128 if T < 100 else 64, 64, B, T, 64, T % 2 == 0, B, src=src, positions=pos, packed=True,
             turns=B % 2 == 1)
    s.check(s.run())


def test_a_long_prompt():
    # sixteen heads a task, several blocks a head
    s = Step("bf16", 8, 4, 128, 16, 2, 2050, 128, False, 3, positions=[0, 7], packed=True)
    s.check(s.run())
    s = Step("i8t", 8, 4, 128, 16, 1, 2050, 128, True, 4, positions=[100], packed=True)
    s.check(s.run())


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("cuts", [[1] * 70, [60, 1, 3, 1, 65, 70], [200], [130, 70], [63, 65, 72]])
@pytest.mark.parametrize("interleaved", [False, True])
def test_open_groups_go_on_from_rotated_originals(d, cuts, interleaved):
    # the group's scale at every length is that of the rotated keys in 32 bits, however they came
    T, hkv, ps = sum(cuts), 2, 64
    s = Step("i8g", hkv, 1, d, ps, 1, T, 48, interleaved, d + len(cuts), positions=[0], packed=True)
    kr = rotated(s.val[1], s.cs, interleaved)[0]
    at = 0
    for n in cuts:
        out = s.cache.rotary_append(s.q[:, at:at + n], s.k[:, at:at + n], s.v[:, at:at + n], s.cs_dev, int_dev(s.table),
                                    int_dev([at]), interleaved=interleaved, dev_status=s.status)
        at += n
        for x, pool, col in ((kr[:at], s.cache.k_pages, 0), (s.val[2][0, :at], s.cache.v_pages, 2)):
            c, sc, z = oracle.quantize_per_group(x)
            assert np.array_equal(int8_codes(gather(pool.cpu().numpy(), s.table[0], at, ps)), c)
            sz = s.cache.kv_sz.cpu().numpy()[s.table[0, :sc.shape[0]], :, 0]
            assert np.array_equal(sz[..., col], sc) and np.array_equal(sz[..., col + 1], z)
    assert int(s.status.item()) == 0 and out.shape[1] == cuts[-1]


@pytest.mark.parametrize("kind", ALL)
def test_boxes_are_those_of_the_stored_keys(kind):
    ps = 64
    s = Step(kind, 5, 2, 128, ps, 2, 130, 64, True, 6, positions=[0, 0], lens=[130, 64], meta=True)
    s.check(s.run())
    kr = rotated(s.val[1], s.cs, True)
    for b, n in enumerate(s.n):
        x = kr[b, :n]
        x = {"f16": lambda: synth.round_to_dtype(x, "f16")[1], "bf16": lambda: synth.round_to_dtype(x, "bf16")[1],
             "i8t": lambda: per_token_bbox_values(*oracle.quantize_per_token(x)),
             "i8g": lambda: per_group_bbox_values(*oracle.quantize_per_group(x)),
             "u4t": lambda: per_token_u4_bbox_values(*oracle.quantize_per_token_u4(x))}[kind]()
        mn, mx = oracle.page_bounding_boxes(x, ps)
        meta = s.cache.page_meta.cpu().numpy()[s.table[b, :mn.shape[0]]]
        assert np.array_equal(meta[:, :, 0], mn) and np.array_equal(meta[:, :, 1], mx)


def test_strides_places_and_missing_queries():
    s = Step("bf16", 2, 3, 64, 16, 3, 4, 32, False, 7, lens=[4, 2, 3])
    ref = s.run()
    s.check(ref)
    # in place
    q = s.q.clone()
    assert s.cache.rotary_append(q, s.k, s.v, s.cs_dev, int_dev(s.table), int_dev(s.pos), new_lens=int_dev(s.n), q_out=q) is q
    for b, n in enumerate(s.n):
        assert torch.equal(q[b, :n], ref[b, :n]) and torch.equal(q[b, n:], s.q[b, n:])
    # tokens wide apart; rows beyond a row's tokens stay as they were
    wide = [torch.zeros(3, 4, 1000, dtype=torch.bfloat16, device="cuda") for _ in range(3)]
    part = []
    for w, x, off in zip(wide, (s.q, s.k, s.v), (8, 16, 40)):
        h = x.shape[2]
        w[:, :, off:off + h * 64] = x.reshape(3, 4, -1)
        part.append(w[:, :, off:off + h * 64].unflatten(-1, (h, 64)))
    out = torch.full_like(ref, 7.0)
    s.cache.k_pages.zero_()
    s.q, s.k, s.v = part
    s.run(q_out=out)
    s.check(out)
    for b, n in enumerate(s.n):
        assert bool((out[b, n:] == 7.0).all())
    # no queries
    s.cache.k_pages.zero_()
    assert s.cache.rotary_append(None, s.k, s.v, s.cs_dev, int_dev(s.table), int_dev(s.pos), new_lens=int_dev(s.n)) is None
    s.check(out)


def test_only_the_new_tokens_change():
    for kind in ALL:
        s = Step(kind, 2, 1, 64, 64, 2, 3, 64, False, 8, positions=[64, 128], lens=[3, 2])
        s.cache.k_pages.fill_(1)
        s.cache.v_pages.fill_(1)
        before = [x.clone() for x in (s.cache.k_pages, s.cache.v_pages)]
        s.check(s.run())
        for old, new in zip(before, (s.cache.k_pages, s.cache.v_pages)):
            mine = torch.zeros(new.shape[0], 64, dtype=torch.bool, device="cuda")
            for b, n in enumerate(s.n):
                for t in range(s.pos[b], s.pos[b] + n):
                    mine[int(s.table[b, t // 64]), t % 64] = True
            assert torch.equal(old.movedim(2, 1)[~mine], new.movedim(2, 1)[~mine])


def test_errors_on_the_device_are_reported_and_skipped():
    from paged_kv_cache_243_gb300 import binding as B
    for kind in ("bf16", "i8t", "i8g"):
        s = Step(kind, 2, 2, 64, 64, 3, 2, 64, False, 9, positions=[0, 64, 128])
        ref = s.run()
        s.check(ref)
        table, pos = s.table.copy(), s.pos.copy()
        for bad in ((1, -1), (1, 1 << 25)):
            table[1, 1] = bad[1]
            s.status.zero_()
            out = s.cache.rotary_append(s.q, s.k, s.v, s.cs_dev, int_dev(table), int_dev(pos), dev_status=s.status)
            assert int(s.status.item()) == B.DEV_BAD_PAGE and torch.equal(out, ref)   # queries have no page
        for p in (-1, 64 * s.width - 1, 2 ** 31 - 1):
            pos[1] = p
            s.status.zero_()
            out = s.cache.rotary_append(s.q, s.k, s.v, s.cs_dev, int_dev(s.table), int_dev(pos), q_out=torch.zeros_like(ref),
                                        dev_status=s.status)
            assert int(s.status.item()) == B.DEV_BAD_POSITION
            assert torch.equal(out[[0, 2]], ref[[0, 2]]) and not bool(out[1].any())
        # beyond the table: its nearest row
        turns = np.array([[-5, 0], [0, 1], [129, 1000]], dtype=np.int32)
        s.status.zero_()
        out = s.cache.rotary_append(s.q, s.k, s.v, s.cs_dev, int_dev(s.table), int_dev(s.pos), int_dev(turns),
                                    dev_status=s.status)
        assert int(s.status.item()) == B.DEV_BAD_POSITION
        s.turns = turns.clip(0, s.cs_dev.shape[0] - 1)
        s.cs = s.cs_dev.cpu().numpy()[s.turns]
        s.status.zero_()
        s.check(out)


def test_captured_and_on_another_stream():
    s = Step("i8t", 4, 4, 128, 16, 5, 3, 128, False, 10)
    ref = s.run()
    st = torch.cuda.Stream()
    assert torch.equal(s.run(stream=st), ref)
    args = (s.q, s.k, s.v, s.cs_dev, int_dev(s.table), int_dev(s.pos))
    out = torch.zeros_like(ref)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.cache.rotary_append(*args, q_out=out)
    s.cache.k_pages.zero_()
    graph.replay()
    torch.cuda.synchronize()
    s.check(out)


@pytest.mark.parametrize("rot", [16, 48, 128])
def test_tables(rot):
    from paged_kv_cache_243_gb300 import rotary_frequencies, rotary_table
    for kw in ({}, dict(scaling="linear", factor=4.0), dict(scaling="ramp", factor=16.0, low=1.0, high=32.0, original=4096)):
        w, scale = rotary_frequencies(rot, 500000.0, **kw)
        t = rotary_table(70001, rot, base=500000.0, **kw).cpu().numpy().astype(np.float64)
        angle = np.arange(70001)[:, None] * w
        want = np.concatenate([np.cos(angle), np.sin(angle)], 1) * scale
        # half a step of fp32, and 64-bit angles of up to 70000 that are each half a step off
        assert (np.abs(t - want) <= np.abs(want) * 2.0 ** -24 + scale * 70001 * 2.0 ** -51).all()
