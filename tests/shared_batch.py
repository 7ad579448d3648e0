"""Batches whose rows share prefixes, for the tests of page sharing: tokens drawn here,
written with kv_append through block tables that share the prefix's whole pages, and the
values attention must see, restored by the oracle's quantisers."""
from __future__ import annotations

import numpy as np
import torch

import oracle
import synth
from oracle.quant import per_group_dequant, per_token_dequant
from oracle.quant4 import per_token_u4_dequant

KINDS = {  # kv_dtype, quant of PagedKVCache, type of the tokens
    "f16": ("f16", "none", "f16"), "bf16": ("bf16", "none", "bf16"),
    "i8t": ("int8", "per_token", "f16"), "i8g": ("int8", "per_group64", "f16"),
    "u4t": ("u4", "per_token", "f16"),
}
TORCH = {"f16": torch.float16, "bf16": torch.bfloat16}


def to_dev(bits: np.ndarray, name: str) -> torch.Tensor:
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).view(TORCH[name]).cuda()


def int_dev(a) -> torch.Tensor:
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


def restore(kind: str, x: np.ndarray):
    """(values as attention sees them in fp64, largest |scale midpoint|) of tokens [T][H][d]."""
    if kind in ("f16", "bf16"):
        return x.astype(np.float64), 0.0
    if x.shape[0] == 0:
        return x.astype(np.float64), 0.0
    if kind == "i8t":
        c, s, z = oracle.quantize_per_token(x)
        return per_token_dequant(c, s, z), float(np.abs(z + 128 * s.astype(np.float64)).max())
    if kind == "u4t":
        c, s, z = oracle.quantize_per_token_u4(x)
        return per_token_u4_dequant(c, s, z), float(np.abs(z + 8 * s.astype(np.float64)).max())
    c, s, z = oracle.quantize_per_group(x)
    return per_group_dequant(c, s, z), float(np.abs(z + 128 * s.astype(np.float64)).max())


class SharedBatch:
    """groups: a list of (prefix tokens, [tokens after it of each row]); alone: lengths of rows
    without a group. Rows are put in a drawn order."""

    def __init__(self, kind, hkv, d, ps, groups, alone=(), seed=0, k_scale=1.0, v_scale=1.0, with_meta=False,
                 extra_pages=0):
        from paged_kv_cache_243_gb300.cache import PagedKVCache
        self.kind, self.hkv, self.d, self.ps = kind, hkv, d, ps
        kv_dtype, quant, self.src = KINDS[kind]
        rng = np.random.default_rng([77, seed])
        rows = [(g, n) for g, (_, ns) in enumerate(groups) for n in ns] + [(-1, n) for n in alone]
        rows = [rows[i] for i in rng.permutation(len(rows))]
        self.group = np.array([g for g, _ in rows], dtype=np.int32)
        self.prefix = np.array([p for p, _ in groups], dtype=np.int32)
        B = self.B = len(rows)

        def tokens(n, scale):
            bits, val = synth.round_to_dtype(rng.standard_normal((n, hkv, d)).astype(np.float32) * scale, self.src)
            return bits, val

        pre = [(tokens(p, k_scale), tokens(p, v_scale)) for p, _ in groups]
        self.bits, self.k, self.v, self.kmid, self.vmid = [], [], [], [], []
        for g, n in rows:
            own = (tokens(n, k_scale), tokens(n, v_scale))
            parts = [pre[g], own] if g >= 0 else [own]
            kb, vb = (np.concatenate([p[i][0] for p in parts]) for i in (0, 1))
            kf, vf = (np.concatenate([p[i][1] for p in parts]) for i in (0, 1))
            self.bits.append((kb, vb))
            k, mid = restore(kind, kf)
            self.k.append(k)
            v, vmid = restore(kind, vf)
            self.v.append(v)
            self.kmid.append(mid)
            self.vmid.append(vmid)
        self.lens = np.array([k.shape[0] for k in self.k], dtype=np.int32)
        # tables: the prefix's whole pages are the same pages, everything else a row's own
        whole = [p // ps for p, _ in groups]
        self.width = max(1, max(-(-int(n) // ps) for n in self.lens)) + extra_pages
        need = [-(-int(n) // ps) + extra_pages - (whole[g] if g >= 0 else 0) for (g, _), n in zip(rows, self.lens)]
        total = sum(whole) + sum(need) + 3
        ids = rng.permutation(total).astype(np.int32)
        shared, at = [], 0
        for w in whole:
            shared.append(ids[at:at + w])
            at += w
        self.table = np.full((B, self.width), -1, dtype=np.int32)
        for b, (g, _) in enumerate(rows):
            w = whole[g] if g >= 0 else 0
            if w:
                self.table[b, :w] = shared[g]
            self.table[b, w:w + need[b]] = ids[at:at + need[b]]
            at += need[b]
        self.cache = PagedKVCache(total, ps, hkv, d, kv_dtype=kv_dtype, quant=quant, with_meta=with_meta,
                                  tail_rows=max(1, B), poison=True)
        self.table_dev, self.lens_dev = int_dev(self.table), int_dev(self.lens)
        self.group_dev, self.prefix_dev = int_dev(self.group), int_dev(self.prefix)
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        # the first row of a group writes the whole prefix, the others what follows its whole pages
        first = {}
        for b, (g, _) in enumerate(rows):
            first.setdefault(g, b)
        start = np.array([0 if g < 0 or first[g] == b else whole[g] * ps for b, (g, _) in enumerate(rows)],
                         dtype=np.int32)
        count = self.lens - start
        T = int(count.max()) if B else 0
        if T > 0:
            kb = np.zeros((B, T, hkv, d), dtype=np.uint16)
            vb = np.zeros_like(kb)
            for b in range(B):
                kb[b, :count[b]] = self.bits[b][0][start[b]:]
                vb[b, :count[b]] = self.bits[b][1][start[b]:]
            self.cache.append(to_dev(kb, self.src), to_dev(vb, self.src), self.table_dev, int_dev(start),
                              int_dev(count), dev_status=self.status)
        torch.cuda.synchronize()
        assert int(self.status.item()) == 0

    def queries(self, g, q_name=None, seed=1, scale=1.0):
        """(device q [B][Hkv g][d], its values)."""
        rng = np.random.default_rng([78, seed])
        x = rng.standard_normal((self.B, self.hkv * g, self.d)).astype(np.float32) * scale
        name = q_name or self.src
        bits, val = synth.round_to_dtype(x, name)
        return to_dev(bits, name), val

    def expected(self, q, g, sm_scale=None, lens=None):
        """Oracle outputs [B][Hq][d] and the bound on each output's error before its own rounding,
        without the rounding of the weights: (out, bound without weights, what their roundings meet)."""
        sm = 1.0 / np.sqrt(self.d) if sm_scale is None else sm_scale
        out = np.zeros(q.shape)
        bound = np.zeros(q.shape)
        mass = np.zeros(q.shape)
        for b in range(self.B):
            n = int(self.lens[b] if lens is None else lens[b])
            if n == 0:
                continue
            for h in range(q.shape[1]):
                k, v = self.k[b][:n, h // g], self.v[b][:n, h // g]
                qq = q[b, h].astype(np.float64)
                s = sm * (k @ qq)
                p = np.exp(s - s.max())
                p /= p.sum()
                out[b, h] = p @ v
                # a weight meets a quantised value in two parts, sum p vs (u - c) and sum p mid with
                # mid = vz + c vs: |vs (u - c)| = |v - mid| <= |v| + |mid|, so that is what the
                # weights' roundings are multiplied with
                mass[b, h] = p @ np.abs(v) + self.vmid[b]
                # scores: fp32 sums of d products (each |q_i k_i|; quantised keys as code and
                # midpoint parts, |code part| <= |k| + |mid|), each step at most 2^-23 off
                a = (np.abs(k) @ np.abs(qq)).max() + 2 * np.abs(qq).sum() * self.kmid[b]
                ds = sm * (self.d + 8) * 2.0 ** -23 * a
                # weights: e^ds - 1 on either side of the quotient, ex2 at 2^-21, sums of n terms
                # in fp32 in up to n / 16 steps
                rel = 2 * np.expm1(ds) + 2.0 ** -20 + (n / 16 + 64) * 2.0 ** -23
                bound[b, h] = rel * mass[b, h] + 1e-30
        return out, bound, mass

    def check(self, got: torch.Tensor, q, g, q_name=None, sm_scale=None, lens=None):
        """Every output within the derived bound of the oracle's."""
        name = q_name or self.src
        out, bound, mass = self.expected(q, g, sm_scale, lens)
        half = torch.finfo(TORCH[name]).eps / 2
        if got.dtype == torch.float32:
            # weights as two values of q's type: each rounding is at most half a step of what is left
            bound = bound + mass * half * half
        else:
            # weights rounded once, and the output itself
            bound = bound + mass * half
            bound = bound + (np.abs(out) + bound) * torch.finfo(got.dtype).eps / 2
        n = self.lens if lens is None else lens
        vmax = np.array([np.abs(v[:m]).max() if m else 0.0 for v, m in zip(self.v, n)])[:, None, None]
        if name == "f16":
            # fp16 keeps an absolute step of 2^-24 below 2^-14: half of it for each weight (of at
            # most 1 where the largest is 1), times |v|; for codes the weight carries the scale,
            # relative to at most twice the largest one, and |code| <= 128 of 255 (8 of 15) steps
            # of at most 2 |v|: under twice as much
            bound = bound + np.asarray(n)[:, None, None] * 2.0 ** -24 * vmax
        err = np.abs(got.float().cpu().numpy().astype(np.float64) - out)
        worst = float((err - bound).max()) if err.size else 0.0
        assert np.isfinite(err).all(), "a non-finite output"
        assert worst <= 0.0, (worst, float(err.max()), float(bound.max()))
        return float(err.max()) if err.size else 0.0

    def run(self, q, out_dtype=torch.float32, **kw):
        out = self.cache.shared_attention(q, self.table_dev, self.lens_dev, self.group_dev, self.prefix_dev,
                                          out_dtype=out_dtype, dev_status=self.status, **kw)
        torch.cuda.synchronize()
        return out
