"""Rows whose tokens are marked by 128-token tile, so that an attention that leaves out a tile, takes
one twice or takes another's keys or values shows in the outputs, well above their rounding.

The token at position t of a row lies in tile i = t // 128. Its values are +m in channel i mod d and
-m half of the channels further, m = 1 + i // d, times 1 to 1.75 by row after the prefix; its key is
1 in channel 7 i + 3 mod d. A query is a single channel, worth a factor of 4 in weight to the
tiles whose keys have it, all other weights being equal.
"""
import numpy as np

import synth
from shared_batch import restore


class MarkedRows:
    def __init__(self, kind, d, group, prefix, lens, g, src):
        self.kind, self.d, self.g, self.src = kind, d, g, src
        self.group, self.lens = [int(x) for x in group], [int(x) for x in lens]
        self.prefix = [int(prefix[x]) if x >= 0 else 0 for x in self.group]
        self.bits, self.k, self.v = [], [], []
        for b, n in enumerate(self.lens):
            t = np.arange(n)
            i = t // 128
            m = (1.0 + i // d) * np.where(t < self.prefix[b], 1.0, 1 + (b % 7) / 8)
            k, v = np.zeros((2, n, 1, d), dtype=np.float32)
            k[t, 0, (7 * i + 3) % d] = 1
            v[t, 0, i % d] = m
            v[t, 0, (i + d // 2) % d] = -m
            kb, kf = synth.round_to_dtype(k, src)
            vb, vf = synth.round_to_dtype(v, src)
            self.bits.append((kb, vb))
            self.k.append(restore(kind, kf)[0][:, 0])
            self.v.append(restore(kind, vf)[0][:, 0])
        B = len(self.lens)
        q = np.zeros((B, g, d), dtype=np.float32)
        for b in range(B):
            for h in range(g):
                q[b, h, 5 * (b * g + h) % d] = np.log(4) * np.sqrt(d)
        self.qbits, self.q = synth.round_to_dtype(q, src)
        self.p = []
        for b in range(B):
            s = self.q[b].astype(np.float64) @ self.k[b].T / np.sqrt(d)
            w = np.exp(s)
            self.p.append(w / w.sum(-1, keepdims=True))
        self.out = np.stack([p @ v for p, v in zip(self.p, self.v)])

    def bound(self, half, out_eps):
        """Each output's error at most: `half` is what a weight's roundings are off, out_eps the output
        type's step (0: fp32)."""
        e = np.zeros(self.out.shape)
        for b, n in enumerate(self.lens):
            # scores are sums of d products, the largest |q| <= 1.5 sqrt(d) times a key of 1, in two parts
            # (code and middle) for codes: each step 2^-23 off; sums of n weights in n / 16 steps;
            # ex2 and the quotient 2^-20
            ds = (self.d + 8) * 2.0 ** -23 * 1.5 * 2
            rel = 2 * ds + (n / 16 + 64) * 2.0 ** -23 + 2.0 ** -20 + half
            mid = 0.0 if self.kind in ("f16", "bf16") else 0.02   # of m: (max + min) / 2 of the codes' range
            e[b] = rel * (self.p[b] @ (np.abs(self.v[b]) + mid * np.abs(self.v[b]).max(1, keepdims=True)))
        return e + (np.abs(self.out) + e) * out_eps / 2

    def visits(self, b):
        """The token ranges that are one tile of work each: those of the prefix, then the row's own."""
        skip = self.prefix[b] // 16 * 16 if self.group[b] >= 0 else 0
        for a, z in ((0, skip), (skip, self.lens[b])):
            for t in range(a, z, 128):
                yield t, min(t + 128, z)

    def with_weight(self, b, t0, t1, times):
        """Row b's outputs if tokens [t0, t1) counted `times` times."""
        p, v = self.p[b][:, t0:t1], self.v[b][t0:t1]
        return (self.out[b] + (times - 1) * (p @ v)) / (1 + (times - 1) * p.sum(-1, keepdims=True))

    def with_values_of(self, b, t0, t1, o0):
        """Row b's outputs if tokens [t0, t1) had the values of those from o0 on."""
        return self.out[b] + self.p[b][:, t0:t1] @ (self.v[b][o0:o0 + t1 - t0] - self.v[b][t0:t1])

    def with_keys_of(self, b, t0, t1, o0):
        """Row b's outputs if tokens [t0, t1) had the weights of those from o0 on."""
        p, v = self.p[b], self.v[b][t0:t1]
        change = p[:, o0:o0 + t1 - t0] - p[:, t0:t1]
        return (self.out[b] + change @ v) / (1 + change.sum(-1, keepdims=True))


# (rows, heads, own tokens of each row) of the batches that both the CPU and the GPU tests use
OWN = [64, 100, 128, 200, 256, 90, 180]
PREFIX, ALONE = 30000, [9000, 80]


def layout(rows):
    return [OWN[i % len(OWN)] for i in range(rows)]
