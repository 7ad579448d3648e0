"""Steps with drafted tokens as a program runs them: keep what was accepted, rotate and store the new
drafts, attend; against the whole sequence in one piece."""
import numpy as np
import pytest
import torch

import synth
from shared_batch import KINDS, SharedBatch, int_dev, restore, to_dev
from test_gpu_rotary import rotated
from tree_batch import TreeBatch, pack, random_parents, seen_from_parents

pytestmark = pytest.mark.gpu


class Tokens:
    """The stored sequences of a program, token by token, as the oracle restores them."""

    def __init__(self, kind, hkv, g, d, ps, B, T, rot, interleaved, seed):
        from paged_kv_cache_243_gb300 import PageAllocator, rotary_table
        from paged_kv_cache_243_gb300.cache import PagedKVCache
        kv_dtype, quant, self.src = KINDS[kind]
        self.kind, self.hkv, self.hq, self.d, self.ps, self.B, self.T = kind, hkv, hkv * g, d, ps, B, T
        self.rng = np.random.default_rng([85, seed])
        self.rot, self.inter, self.width = rot, interleaved, 40
        self.alloc = PageAllocator(B * self.width)
        self.cache = PagedKVCache(B * self.width, ps, hkv, d, kv_dtype=kv_dtype, quant=quant, with_meta=True,
                                  tail_rows=B, poison=True)
        self.table = np.stack([self.alloc.reserve(b, ps * self.width, ps, self.width) for b in range(B)])
        self.cs_dev = rotary_table(ps * self.width, rot)
        self.cs = self.cs_dev.cpu().numpy()
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.k = [np.zeros((0, hkv, d), np.float32) for _ in range(B)]      # rotated, before the cache's rounding
        self.v = [np.zeros((0, hkv, d), np.float32) for _ in range(B)]

    def draw(self, n):
        bits, val = synth.round_to_dtype(
            self.rng.standard_normal((self.B, n, self.hq + 2 * self.hkv, self.d)).astype(np.float32), self.src)
        x = to_dev(bits, self.src)
        cut = [self.hq, self.hq + self.hkv]
        return torch.tensor_split(x, cut, 2), np.split(val, cut, 2)

    def append(self, base, turns, n=None):
        """Draws and stores drafts at base; returns device q, and (q, k) rotated and v on the host."""
        (q, k, v), (qf, kf, vf) = self.draw(turns.shape[1])
        out = self.cache.rotary_append(q, k, v, self.cs_dev, int_dev(self.table), int_dev(base), int_dev(turns),
                                       interleaved=self.inter, dev_status=self.status,
                                       new_lens=None if n is None else int_dev(n))
        cs = self.cs[turns]
        qr = synth.round_to_dtype(rotated(qf, cs, self.inter), self.src)[1]
        return out, qr, rotated(kf, cs, self.inter), vf


@pytest.mark.parametrize("kind,hkv,g,d,ps,rot,inter", [
    ("bf16", 2, 4, 128, 16, 128, False), ("f16", 3, 1, 64, 48, 32, True), ("i8t", 2, 4, 64, 16, 64, False),
    ("u4t", 2, 3, 128, 32, 112, True)])
def test_steps_equal_the_sequence_in_one_piece(kind, hkv, g, d, ps, rot, inter):
    B, T = 3, 21
    s = Tokens(kind, hkv, g, d, ps, B, T, rot, inter, hkv + g)
    prompt = np.array([70, 1, 33])
    at = np.broadcast_to(np.arange(70), (B, 70))
    _, _, kr, vf = s.append(np.zeros(B), at, prompt)
    for b in range(B):
        s.k[b], s.v[b] = kr[b, :prompt[b]], vf[b, :prompt[b]]
    base, keep, n_keep = prompt.copy(), None, None
    tb = TreeBatch.__new__(TreeBatch)
    for step in range(6):
        if keep is not None:
            s.cache.keep_tokens(int_dev(keep), int_dev(n_keep), int_dev(s.table), int_dev(base), dev_status=s.status)
            for b in range(B):
                s.k[b] = np.concatenate([s.k[b], kr[b, keep[b, :n_keep[b]]]])
                s.v[b] = np.concatenate([s.v[b], vf[b, keep[b, :n_keep[b]]]])
            base = base + n_keep
        parents = np.stack([random_parents(s.rng, T) for _ in range(B)])
        seen = np.stack([seen_from_parents(p) for p in parents])
        q, qr, kr, vf = s.append(base, base[:, None] + seen.sum(-1) - 1)
        out = s.cache.tree_attention(q, int_dev(s.table), int_dev(base + T), pack(seen).cuda(), dev_status=s.status,
                                     out_dtype=torch.float32 if step % 2 else q.dtype)
        torch.cuda.synchronize()
        assert int(s.status.item()) == 0
        # the definition over what each sequence holds
        tb.B, tb.T, tb.d, tb.src, tb.seen = B, T, d, s.src, seen
        tb.lens, tb.drafts = (base + T).astype(np.int32), np.full(B, T)
        tb.k, tb.v, tb.kmid, tb.vmid = [], [], [], []
        for b in range(B):
            for mine, mid, x in ((tb.k, tb.kmid, np.concatenate([s.k[b], kr[b]])), (tb.v, tb.vmid, np.concatenate([s.v[b], vf[b]]))):
                if kind in ("f16", "bf16"):
                    x = synth.round_to_dtype(x, kind)[1]
                val, m = restore(kind, x)
                mine.append(val)
                mid.append(m)
        tb.tree_check(out, qr, g)
        # accept a path: from a random draft up to its root
        keep, n_keep = np.full((B, T), -1), np.zeros(B, dtype=np.int64)
        for b in range(B):
            path = np.flatnonzero(seen[b, s.rng.integers(0, T)])
            keep[b, :len(path)], n_keep[b] = path, len(path)
        if step == 3:
            n_keep[1] = 0


def test_steps_on_a_per_group_cache():
    # accepted drafts are appended anew: the open group goes on from its originals, whatever the drafts
    # did to it
    B, T, ps, hkv, d = 2, 20, 64, 2, 64
    s = Tokens("i8g", hkv, 2, d, ps, B, T, 64, False, 9)
    base = np.array([50, 61])
    at = np.broadcast_to(np.arange(61), (B, 61))
    _, _, kr, vf = s.append(np.zeros(B), at, base)
    for b in range(B):
        s.k[b], s.v[b] = kr[b, :base[b]], vf[b, :base[b]]
    import oracle
    from helpers import int8_codes
    for step in range(5):
        chain = base[:, None] + np.arange(T)
        (q, k, v), (qf, kf, vf) = s.draw(T)
        s.cache.rotary_append(q, k, v, s.cs_dev, int_dev(s.table), int_dev(base), dev_status=s.status)
        s.cache.tree_attention(q.contiguous(), int_dev(s.table), int_dev(base + T), dev_status=s.status)
        n = np.array([3 + step, 7])
        s.cache.rotary_append(None, k, v, s.cs_dev, int_dev(s.table), int_dev(base), new_lens=int_dev(n), dev_status=s.status)
        kr = rotated(kf, s.cs[chain], False)
        for b in range(B):
            s.k[b] = np.concatenate([s.k[b], kr[b, :n[b]]])
            s.v[b] = np.concatenate([s.v[b], vf[b, :n[b]]])
        base = base + n
        torch.cuda.synchronize()
        assert int(s.status.item()) == 0
        for b in range(B):
            t = np.arange(base[b])
            c, sc, z = oracle.quantize_per_group(s.k[b])
            got = s.cache.k_pages.cpu().numpy()[s.table[b, t // ps], :, t % ps]
            assert np.array_equal(int8_codes(got), c)
            sz = s.cache.kv_sz.cpu().numpy()[s.table[b, :sc.shape[0]], :, 0]
            assert np.array_equal(sz[..., 0], sc) and np.array_equal(sz[..., 1], z)


@pytest.mark.parametrize("kind", ["bf16", "i8t"])
def test_pools_beyond_32_bits(kind):
    # the last pages of pools of more than 4 GiB (and 2^31 values) hold the same as a small pool's
    from paged_kv_cache_243_gb300 import rotary_table
    from paged_kv_cache_243_gb300.cache import PagedKVCache
    kv_dtype, quant, src = KINDS[kind]
    B, T, hkv, g, d, ps, width = 2, 12, 8, 4, 128, 16, 20
    pages = (4 << 30) // (hkv * ps * d * (1 if quant != "none" else 2)) + 500
    rng = np.random.default_rng(86)
    draw = lambda n, h: to_dev(synth.round_to_dtype(rng.standard_normal((B, n, h, d)).astype(np.float32), src)[0], src)
    prompt, drafts = [draw(200, h) for h in (hkv * g, hkv, hkv)], [draw(T, h) for h in (hkv * g, hkv, hkv)]
    table = rng.permutation(B * width).reshape(B, width)
    cs, base, keep = rotary_table(ps * width, d), int_dev([200, 200]), int_dev([[1, 2, 6, 11]] * B)
    got = []
    for n in (B * width, pages):
        cache = PagedKVCache(n, ps, hkv, d, kv_dtype=kv_dtype, quant=quant, with_meta=True)
        rows = int_dev(table + n - B * width)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        cache.rotary_append(*prompt, cs, rows, base - 200, dev_status=status)
        q = cache.rotary_append(*drafts, cs, rows, base, dev_status=status)
        out = cache.tree_attention(q, rows, base + T, dev_status=status)
        cache.keep_tokens(keep, None, rows, base, dev_status=status)
        after = cache.tree_attention(q[:, :4].contiguous(), rows, base + 4, dev_status=status)
        torch.cuda.synchronize()
        assert int(status.item()) == 0
        got.append((q, out, after, cache.page_meta[rows.long()][:, :204 // ps].clone()))
        del cache
    for a, b in zip(*got):
        assert torch.equal(a, b)
    torch.cuda.empty_cache()
