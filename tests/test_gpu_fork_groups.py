"""Sequences of a per-group INT8 cache that go on from inside a 64-token group: the group is
quantised anew at every append, from values that the batch row may or may not hold."""
import numpy as np
import pytest
import torch

from shared_batch import int_dev, to_dev
import synth

pytestmark = pytest.mark.gpu

H, PS, WIDTH = 2, 64, 24


class Rows:
    def __init__(self, d, rows, seed):
        from paged_kv_cache_243_gb300.cache import PageAllocator, PagedKVCache
        self.d, self.rng = d, np.random.default_rng([91, seed])
        self.pool = PageAllocator(80)
        self.cache = PagedKVCache(80, PS, H, d, kv_dtype="int8", quant="per_group64", tail_rows=rows, poison=True)
        self.table = np.full((rows, WIDTH), -1, dtype=np.int32)
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def tokens(self, n):
        """Bits and values of n tokens of K and of V: [2][n][H][d]."""
        return synth.round_to_dtype(self.rng.standard_normal((2, n, H, self.d)).astype(np.float32), "f16")

    def append(self, row, pos, bits, t_new=None):
        """The tokens at pos of one row; the call covers every row and has room for t_new tokens."""
        rows, n = len(self.table), bits.shape[1]
        kv = np.zeros((2, rows, t_new or n, H, self.d), dtype=np.uint16)
        kv[:, row, :n] = bits
        lens = np.zeros(rows, dtype=np.int32)
        lens[row] = n
        self.cache.append(to_dev(kv[0], "f16"), to_dev(kv[1], "f16"), int_dev(self.table),
                          int_dev([pos] * rows), int_dev(lens), dev_status=self.status)
        torch.cuda.synchronize()
        assert int(self.status.item()) == 0

    def read(self, row, first, end):
        """(values, scales) of tokens [first, end) of a row as they are stored: [2][n][H][d], [2][n][H]."""
        t = np.arange(first, end)
        pages = self.table[row, t // PS].astype(np.int64)
        sz = self.cache.kv_sz[:, :, 0].double().cpu().numpy()[pages]       # [n][H][4]
        out, scales = [], []
        for i, pool in enumerate((self.cache.k_pages, self.cache.v_pages)):
            u = pool.cpu().numpy()[pages, :, t % PS].astype(np.float64)
            out.append(u * sz[..., 2 * i:2 * i + 1] + sz[..., 2 * i + 1:2 * i + 2])
            scales.append(sz[..., 2 * i])
        return np.stack(out), np.stack(scales)


def close(got, scale, want):
    """Within half a step of the codes, and of fp32 steps of values up to 255 scales and the zero."""
    tol = 0.5 * scale[..., None] * (1 + 2.0 ** -20) + 2.0 ** -21 * (np.abs(want) + 255 * scale[..., None])
    assert (np.abs(got - want) <= tol).all(), float((np.abs(got - want) / tol).max())


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("tokens", [150, 129, 191, 64, 1, 65])
@pytest.mark.parametrize("copy_row", [True, False])
@pytest.mark.parametrize("t_new", [None, 100])       # the append's kernels for short and for long calls
def test_a_fork_inside_a_closed_group_keeps_what_it_shares(d, tokens, copy_row, t_new):
    # a prompt written in one call and forked long before its end, as a system prompt is: the
    # originals of the group where the child goes on are not kept anywhere
    r = Rows(d, 3, tokens)
    r.table[2] = r.pool.reserve(7, 200, PS, WIDTH)   # an earlier sequence leaves its originals in every row
    r.table[0] = r.table[1] = r.table[2]
    for row in range(3):
        for pos in range(128, 200, 9):
            r.append(row, pos, r.tokens(9)[0])
    r.table[:] = -1
    r.pool.free(7)
    r.table[0] = r.pool.reserve(0, 1000, PS, WIDTH)
    r.append(0, 0, r.tokens(1000)[0])
    r.table[1] = r.pool.fork(0, 1, tokens, PS, WIDTH)
    if copy_row:
        r.cache.copy_pages([], [], [0], [1])
    else:
        r.cache.tail[1].zero_()                      # a row that no sequence has had
    src, dst, r.table[1] = r.pool.unshare(1, tokens, PS, WIDTH)
    r.cache.copy_pages(src, dst)
    r.table[1] = r.pool.reserve(1, tokens + 90, PS, WIDTH)
    before, _ = r.read(1, 0, tokens)
    parent, _ = r.read(0, 0, 1000)
    first = tokens // 64 * 64
    want = before
    n = 0
    for step in (1, 1, 3, 40, 1, 30):
        bits, new = r.tokens(step)
        r.append(1, tokens + n, bits, t_new)
        want = np.concatenate([want, new.astype(np.float64)], 1)
        n += step
        got, scale = r.read(1, 0, tokens + n)
        assert np.array_equal(got[:, :first], before[:, :first])        # groups before the fork stay
        close(got[:, first:], scale[:, first:], want[:, first:])
    assert np.array_equal(r.read(0, 0, 1000)[0], parent)


@pytest.mark.parametrize("tokens", [963, 990, 999, 1000])
def test_a_fork_inside_the_open_group_goes_on_from_the_originals(tokens):
    # the child's codes are those of a sequence that was appended from the start
    r = Rows(64, 3, tokens)
    bits, val = r.tokens(1000)
    more, more_val = r.tokens(30)
    r.table[0] = r.pool.reserve(0, 1000, PS, WIDTH)
    r.append(0, 0, bits)
    r.table[1] = r.pool.fork(0, 1, tokens, PS, WIDTH)
    r.cache.copy_pages([], [], [0], [1])
    src, dst, r.table[1] = r.pool.unshare(1, tokens, PS, WIDTH)
    r.cache.copy_pages(src, dst)
    r.table[1] = r.pool.reserve(1, tokens + 30, PS, WIDTH)
    r.table[2] = r.pool.reserve(2, tokens + 30, PS, WIDTH)
    r.append(2, 0, np.concatenate([bits[:, :tokens], more], 1))
    for i in range(0, 30, 5):
        r.append(1, tokens + i, more[:, i:i + 5])
    assert np.array_equal(r.read(1, 0, tokens + 30)[0], r.read(2, 0, tokens + 30)[0])


def test_a_sequence_cut_back_and_written_again():
    # positions that go back: originals of tokens that were replaced are not taken for those there now
    r = Rows(64, 1, 5)
    r.table[0] = r.pool.reserve(0, 400, PS, WIDTH)
    r.append(0, 0, r.tokens(10)[0])
    for pos in range(10, 63):
        r.append(0, pos, r.tokens(1)[0])
    r.append(0, 20, r.tokens(200)[0])                # tokens 20 to 219, through the groups of both parities
    for pos in (30, 60, 100, 150, 215):
        first = pos // 64 * 64
        # the open group's originals are there; of a closed one's there is what its codes say
        old = whole if pos > 192 else r.read(0, 0, pos)[0]
        bits, new = r.tokens(3)
        r.append(0, pos, bits)
        got, scale = r.read(0, first, pos + 3)
        close(got, scale, np.concatenate([old[:, first:pos], new.astype(np.float64)], 1))
        bits, new = r.tokens(220 - pos)
        r.append(0, pos, bits)
        whole = np.concatenate([old[:, :pos], new.astype(np.float64)], 1)


def test_originals_that_are_still_there_are_used():
    # the same long append twice, from inside a group: between the two runs nothing wrote over the
    # first group's originals, and the second run gives the first one's codes
    r = Rows(128, 1, 6)
    r.table[0] = r.pool.reserve(0, 1200, PS, WIDTH)
    r.append(0, 0, r.tokens(20)[0])
    bits, _ = r.tokens(1000)
    r.append(0, 20, bits)
    once = r.read(0, 0, 1020)[0]
    r.append(0, 20, bits)
    assert np.array_equal(r.read(0, 0, 1020)[0], once)
