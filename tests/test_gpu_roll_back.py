"""Per-group INT8 caches: drafts stored by one append, however many, and the accepted ones appended anew
where they began. What the sequence had before its drafts is quantised from its originals again: the
rejected drafts leave nothing behind, codes and scales are those of the sequence written at once."""
import numpy as np
import pytest
import torch

import oracle
import synth
from helpers import int8_codes
from shared_batch import int_dev, restore, to_dev
from test_gpu_draft_steps import Tokens
from test_gpu_rotary import rotated
from tree_batch import TreeBatch, pack, random_parents, seen_from_parents

pytestmark = pytest.mark.gpu

H, PS, WIDTH = 2, 64, 20


class Sequences:
    def __init__(self, d, rows, seed, rot=0):
        from paged_kv_cache_243_gb300.cache import PagedKVCache, rotary_table
        self.d, self.B, self.rot, self.rng = d, rows, rot, np.random.default_rng([94, seed])
        self.cache = PagedKVCache(rows * WIDTH, PS, H, d, kv_dtype="int8", quant="per_group64", tail_rows=rows, poison=True)
        self.table = self.rng.permutation(rows * WIDTH).reshape(rows, WIDTH).astype(np.int32)
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        if rot:
            self.cs_dev = rotary_table(PS * WIDTH, rot)
            self.cs = self.cs_dev.cpu().numpy()
        self.held = [[np.zeros((0, H, d), np.float32)] * 2 for _ in range(rows)]   # K (rotated) and V

    def tokens(self, n, scale=1.0):
        """Bits and values [2][B][n][H][d]."""
        return synth.round_to_dtype((scale * self.rng.standard_normal((2, self.B, n, H, self.d))).astype(np.float32), "f16")

    def append(self, bits, val, pos, lens, keep=True):
        """The first lens[b] of the tokens to row b at pos[b]; with keep they are what the row holds from there."""
        k, v = (to_dev(x, "f16") for x in bits)
        if self.rot:
            self.cache.rotary_append(None, k, v, self.cs_dev, int_dev(self.table), int_dev(pos), new_lens=int_dev(lens),
                                     dev_status=self.status)
        else:
            self.cache.append(k, v, int_dev(self.table), int_dev(pos), int_dev(lens), dev_status=self.status)
        if keep:
            kv = (rotated(val[0], self.cs[pos[:, None] + np.arange(val.shape[2])], False) if self.rot else val[0], val[1])
            for b in range(self.B):
                self.held[b] = [np.concatenate([h[:pos[b]], x[b, :lens[b]]]) for h, x in zip(self.held[b], kv)]

    def check(self):
        torch.cuda.synchronize()
        assert int(self.status.item()) == 0
        sz = self.cache.kv_sz.cpu().numpy()
        for i, pool in enumerate((self.cache.k_pages.cpu().numpy(), self.cache.v_pages.cpu().numpy())):
            for b in range(self.B):
                x = self.held[b][i]
                t = np.arange(len(x))
                codes, scale, zero = oracle.quantize_per_group(x)
                pages = self.table[b, :scale.shape[0]]
                assert np.array_equal(sz[pages, :, 0, 2 * i], scale) and np.array_equal(sz[pages, :, 0, 2 * i + 1], zero), (i, b)
                assert np.array_equal(int8_codes(pool[self.table[b, t // PS], :, t % PS]), codes), (i, b)


@pytest.mark.parametrize("rot", [0, 64])
@pytest.mark.parametrize("d,T", [(64, 66), (64, 100), (128, 129), (64, 200), (128, 256)])
def test_rejected_drafts_leave_nothing(d, T, rot):
    # rows that begin at every kind of place of a group, 255 drafts and more reaching the fifth group
    s = Sequences(d, 6, T + rot, rot)
    base = np.array([37, 63, 65, 64, 1, 127])
    prompt = s.tokens(127)
    s.append(*prompt, np.zeros(6, np.int64), base)
    s.check()
    for step, n in enumerate(([3, 1, 0, 20, 2, 5], [64, 30, 7, 66, 0, 1], [1] * 6)):
        bits, val = s.tokens(T)
        n = np.array(n)
        loud = np.arange(T)[None] >= n[:, None]            # the drafts that will be rejected
        bits, val = synth.round_to_dtype(val * np.where(loud, 60.0, 1.0).astype(np.float32)[None, :, :, None, None], "f16")
        s.append(bits, val, base, np.full(6, T), keep=False)
        s.append(bits, val, base, n)
        base = base + n
        if n.all():
            s.check()
    s.check()


def test_drafts_again_and_again_before_anything_is_kept():
    # the same place several times, with drafts of other lengths; and then from a place before it
    s = Sequences(64, 3, 7)
    base = np.array([50, 127, 70])
    s.append(*s.tokens(127), np.zeros(3, np.int64), base)
    for T in (150, 256, 3, 90, 129):
        s.append(*s.tokens(T, 30.0), base, np.full(3, T), keep=False)
    s.append(*s.tokens(10), base, np.full(3, 10))
    s.check()
    base = base + 10
    s.append(*s.tokens(140, 30.0), base, np.full(3, 140), keep=False)
    s.append(*s.tokens(9), base - 5, np.full(3, 9))
    s.check()


def test_random_appends_and_returns():
    # appends of every length that go on at the end, where the last one began, or inside the first or last group
    # that it touched: the originals of all of these are there
    s = Sequences(64, 4, 8)
    pos, end = np.zeros(4, np.int64), np.zeros(4, np.int64)
    for step in range(60):
        at = end.copy()
        for b in range(4):
            how = s.rng.integers(4)
            if how == 1:
                at[b] = pos[b]
            elif how == 2:
                at[b] = s.rng.integers(pos[b] // 64 * 64, pos[b] + 1)
            elif how == 3:
                at[b] = s.rng.integers(max(pos[b], end[b] // 64 * 64), end[b] + 1)
            if at[b] > 900:
                at[b] = 0                                    # another sequence
        n = s.rng.integers(1, [2, 40, 70, 300][step % 4], 4)
        s.append(*s.tokens(int(n.max()) + 5 * (step % 3)), at, n)
        pos, end = at, at + n
        if step % 6 == 5:
            s.check()
    s.check()


def test_a_chunked_prompt_on_every_grid():
    # nothing is cut back: a prompt in pieces has the codes of one in one piece, as ever
    s = Sequences(128, 2, 9, 64)
    at = np.zeros(2, np.int64)
    for n in (30, 100, 64, 130, 1, 200, 65, 190, 77):
        s.append(*s.tokens(n), at, np.full(2, n))
        at = at + n
        s.check()


@pytest.mark.parametrize("cut", [137, 130, 37, 20])
@pytest.mark.parametrize("more", [1, 40, 200])
def test_a_fork_behind_a_long_append(cut, more):
    # the child's row says where the originals are as its parent's does: of the group that is open, and of the one
    # in which the last append began
    s = Sequences(64, 2, cut + more)
    s.append(*s.tokens(37), np.zeros(2, np.int64), np.array([37, 0]))
    s.append(*s.tokens(100), np.array([37, 0]), np.array([100, 0]))
    s.cache.copy_pages(s.table[0], s.table[1], [0], [1])
    s.held[1] = [x[:cut] for x in s.held[0]]
    for _ in range(3):
        at = np.array([len(s.held[b][0]) for b in range(2)])
        s.append(*s.tokens(more), at, np.full(2, more))
        s.check()


@pytest.mark.parametrize("d,g,T", [(64, 2, 100), (128, 4, 70), (64, 3, 256)])
def test_steps_with_trees_that_reach_the_third_group(d, g, T):
    # attention for the drafts, by the definition over the sequence quantised at once; then the accepted path is
    # appended anew, turned by its depth as before
    B = 3
    s = Tokens("i8g", 2, g, d, 64, B, T, d, False, T)
    prompt = np.array([70, 1, 33])
    _, _, kr, vf = s.append(np.zeros(B), np.broadcast_to(np.arange(70), (B, 70)), prompt)
    for b in range(B):
        s.k[b], s.v[b] = kr[b, :prompt[b]], vf[b, :prompt[b]]
    base, tb = prompt.copy(), TreeBatch.__new__(TreeBatch)
    for step in range(4):
        seen = np.stack([seen_from_parents(random_parents(s.rng, T)) for _ in range(B)])
        turns = base[:, None] + seen.sum(-1) - 1
        (q, k, v), (qf, kf, vf) = s.draw(T)
        q = s.cache.rotary_append(q, k, v, s.cs_dev, int_dev(s.table), int_dev(base), int_dev(turns), dev_status=s.status)
        out = s.cache.tree_attention(q, int_dev(s.table), int_dev(base + T), pack(seen).cuda(), dev_status=s.status,
                                     out_dtype=torch.float32 if step % 2 else q.dtype)
        qr, kr = synth.round_to_dtype(rotated(qf, s.cs[turns], False), s.src)[1], rotated(kf, s.cs[turns], False)
        tb.B, tb.T, tb.d, tb.src, tb.seen = B, T, d, s.src, seen
        tb.lens, tb.drafts = (base + T).astype(np.int32), np.full(B, T)
        tb.k, tb.v, tb.kmid, tb.vmid = [], [], [], []
        for b in range(B):
            for mine, mid, x in ((tb.k, tb.kmid, np.concatenate([s.k[b], kr[b]])), (tb.v, tb.vmid, np.concatenate([s.v[b], vf[b]]))):
                val, m = restore("i8g", x)
                mine.append(val)
                mid.append(m)
        tb.tree_check(out, qr, g)
        paths = [np.flatnonzero(seen[b, s.rng.integers(0, T)]) for b in range(B)]
        n = np.array([len(p) for p in paths])
        at = np.stack([np.resize(p, n.max()) for p in paths])
        rows = torch.arange(B, device="cuda")[:, None], torch.from_numpy(at).cuda()
        s.cache.rotary_append(None, k[rows], v[rows], s.cs_dev, int_dev(s.table), int_dev(base),
                              int_dev(np.take_along_axis(turns, at, 1)), new_lens=int_dev(n), dev_status=s.status)
        for b, p in enumerate(paths):
            s.k[b], s.v[b] = np.concatenate([s.k[b], kr[b, p]]), np.concatenate([s.v[b], vf[b, p]])
        base = base + n
        torch.cuda.synchronize()
        assert int(s.status.item()) == 0
