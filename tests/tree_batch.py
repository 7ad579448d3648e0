"""Batches whose last tokens are drafts, for the tests of tree_attention: sequences of SharedBatch
without shared prefixes, masks drawn here, and the outputs by the definition in 64 bits."""
from __future__ import annotations

import numpy as np
import torch

import synth
from shared_batch import TORCH, SharedBatch, int_dev, to_dev


def random_parents(rng, T, spread=3):
    """A tree of T drafts: each hangs on one of the `spread` before it, or so."""
    return np.array([-1] + [max(0, t - int(rng.integers(1, spread + 1))) for t in range(1, T)], dtype=np.int64)


def seen_from_parents(parents):
    T = len(parents)
    seen = np.zeros((T, T), dtype=bool)
    for t, p in enumerate(parents):
        if p >= 0:
            seen[t] = seen[p]
        seen[t, t] = True
    return seen


def pack(seen) -> torch.Tensor:
    """[..., T, T] truth values -> int64 [..., T, ceil(T / 64)]."""
    T = seen.shape[-1]
    out = np.zeros((*seen.shape[:-1], -(-T // 64)), dtype=np.uint64)
    for j in range(T):
        out[..., j // 64] |= np.where(seen[..., j], np.uint64(1 << j % 64), np.uint64(0))
    return torch.from_numpy(out.view(np.int64))


class TreeBatch(SharedBatch):
    """drafts: of each sequence, by the rows' order; T of the call."""

    def __init__(self, kind, hkv, d, ps, lens, T, drafts=None, seed=0, tree="tree", **kw):
        super().__init__(kind, hkv, d, ps, [], alone=list(lens), seed=seed, **kw)
        rng = np.random.default_rng([79, seed])
        self.T = T
        n = np.full(self.B, T) if drafts is None else np.asarray(drafts)
        self.drafts = np.minimum(n, self.lens).astype(np.int32)
        if tree == "chain":
            self.seen, self.mask = np.tril(np.ones((T, T), dtype=bool))[None].repeat(self.B, 0), None
        elif tree == "any":       # any set of drafts, some rows with none
            self.seen = rng.random((self.B, T, T)) < rng.choice([0.0, 0.2, 0.9], (self.B, T, 1))
            self.mask = pack(self.seen).cuda()
        else:
            self.seen = np.stack([seen_from_parents(random_parents(rng, T)) for _ in range(self.B)])
            self.mask = pack(self.seen).cuda()
        self.drafts_dev = int_dev(self.drafts)

    def tree_queries(self, g, q_name=None, seed=1, scale=1.0):
        rng = np.random.default_rng([80, seed])
        x = rng.standard_normal((self.B, self.T, self.hkv * g, self.d)).astype(np.float32) * scale
        name = q_name or self.src
        bits, val = synth.round_to_dtype(x, name)
        return to_dev(bits, name), val

    def attends(self, b):
        """[n][L] truth values of sequence b."""
        L, n = int(self.lens[b]), int(self.drafts[b])
        on = np.ones((n, L), dtype=bool)
        on[:, L - n:] = self.seen[b, :n, :n]
        return on

    def tree_expected(self, q, g, sm_scale=None):
        """(outputs, bound on their error before the weights' and their own rounding, what the weights'
        roundings meet): see SharedBatch.expected, whose terms these are."""
        sm = 1.0 / np.sqrt(self.d) if sm_scale is None else sm_scale
        out, bound, mass = np.zeros(q.shape), np.zeros(q.shape), np.zeros(q.shape)
        for b in range(self.B):
            L, n = int(self.lens[b]), int(self.drafts[b])
            on = self.attends(b)
            rows = on.any(1)
            if not rows.any():
                continue
            for h in range(q.shape[2]):
                k, v = self.k[b][:L, h // g], self.v[b][:L, h // g]
                qq = q[b, :n, h].astype(np.float64)[rows]
                s = np.where(on[rows], sm * (qq @ k.T), -np.inf)
                p = np.exp(s - s.max(1, keepdims=True))
                p /= p.sum(1, keepdims=True)
                at = np.flatnonzero(rows)
                out[b, at, h] = p @ v
                mass[b, at, h] = p @ np.abs(v) + self.vmid[b]
                a = (np.abs(qq) @ np.abs(k).T).max(1) + 2 * np.abs(qq).sum(1) * self.kmid[b]
                ds = sm * (self.d + 8) * 2.0 ** -23 * a
                rel = 2 * np.expm1(ds) + 2.0 ** -20 + (L / 16 + 64) * 2.0 ** -23
                bound[b, at, h] = rel[:, None] * mass[b, at, h] + 1e-30
        return out, bound, mass

    def tree_bound(self, q, g, dtype, q_name=None, sm_scale=None):
        """(outputs, bound on their error) of a call that returns dtype."""
        name = q_name or self.src
        out, bound, mass = self.tree_expected(q, g, sm_scale)
        half = torch.finfo(TORCH[name]).eps / 2
        if dtype == torch.float32:
            bound = bound + mass * half * half     # weights as two values of q's type
        else:
            bound = bound + mass * half            # weights rounded once, and the output itself
            bound = bound + (np.abs(out) + bound) * torch.finfo(dtype).eps / 2
        if name == "f16":
            # fp16's smallest step for each weight (see SharedBatch.check)
            vmax = np.array([np.abs(v).max() if v.size else 0.0 for v in self.v])[:, None, None, None]
            bound = bound + np.asarray(self.lens)[:, None, None, None] * 2.0 ** -24 * vmax
        return out, bound

    def tree_check(self, got, q, g, q_name=None, sm_scale=None):
        out, bound = self.tree_bound(q, g, got.dtype, q_name, sm_scale)
        x = got.float().cpu().numpy().astype(np.float64)
        assert np.isfinite(x).all(), "a non-finite output"
        err = np.abs(x - out)
        assert (err <= bound).all(), (float((err - bound).max()), float(err.max()), float(bound.max()))
        # what attends to nothing, and rows beyond a sequence's drafts
        for b in range(self.B):
            n = int(self.drafts[b])
            none = np.concatenate([np.flatnonzero(~self.attends(b).any(1)), np.arange(n, self.T)]).astype(int)
            assert not x[b, none].any()
        return float(err.max()) if err.size else 0.0

    def tree_run(self, q, out_dtype=torch.float32, **kw):
        kw.setdefault("mask", self.mask)
        out = self.cache.tree_attention(q, self.table_dev, self.lens_dev, draft_lens=self.drafts_dev,
                                        out_dtype=out_dtype, dev_status=self.status, **kw)
        torch.cuda.synchronize()
        return out
