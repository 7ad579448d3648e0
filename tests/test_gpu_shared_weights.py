"""The softmax weights of shared_attention in 16 bits: what their rounding may cost, where a few
values are far larger than those that carry the output, and where many small weights add up."""
import numpy as np
import pytest
import torch

import oracle
import synth
from shared_batch import TORCH, SharedBatch, int_dev, to_dev

pytestmark = pytest.mark.gpu


def parts(kind, x):
    """Tokens [T][H][d] as attention sees them (fp64), and per token and head the middle of its
    codes' range and their scale (0 for 16-bit caches)."""
    T, H, _ = x.shape
    if kind in ("f16", "bf16"):
        return x.astype(np.float64), np.zeros((T, H)), np.zeros((T, H))
    from oracle.quant import per_group_dequant, per_token_dequant
    from oracle.quant4 import per_token_u4_dequant
    if kind == "u4t":
        c, s, z = oracle.quantize_per_token_u4(x)
        val, centre = per_token_u4_dequant(c, s, z), 8.0
    elif kind == "i8t":
        c, s, z = oracle.quantize_per_token(x)
        val, centre = per_token_dequant(c, s, z), 128.0
    else:
        c, s, z = oracle.quantize_per_group(x)
        val, centre = per_group_dequant(c, s, z), 128.0
        s, z = (np.repeat(np.asarray(a), 64, 0)[:T] for a in (s, z))
    s, z = (np.asarray(a, dtype=np.float64).reshape(T, H) for a in (s, z))
    return val, z + centre * s, s


def rewrite(sb, k, v):
    """Give every row of a batch with one group the tokens k, v [T][H][d] (its first len of them)."""
    bits = [synth.round_to_dtype(x.astype(np.float32), sb.src) for x in (k, v)]
    n = int(sb.lens.max())
    dev = [to_dev(np.repeat(b[0][None, :n], sb.B, 0), sb.src) for b in bits]
    sb.cache.append(*dev, sb.table_dev, int_dev([0] * sb.B), sb.lens_dev, dev_status=sb.status)
    torch.cuda.synchronize()
    assert int(sb.status.item()) == 0
    return [b[1] for b in bits]


def outcome(sb, kf, vf, q, g, out_dtype):
    """Oracle outputs and the bound on each one's error, relative to the tokens that carry it."""
    half = torch.finfo(TORCH[sb.src]).eps / 2
    sm = 1.0 / np.sqrt(sb.d)
    k, kmid, _ = parts(sb.kind, kf)
    v, vmid, vs = parts(sb.kind, vf)
    out, bound = np.zeros(q.shape), np.zeros(q.shape)
    for b in range(sb.B):
        n = int(sb.lens[b])
        for h in range(q.shape[1]):
            j = h // g
            kk, vv, qq = k[:n, j], v[:n, j], q[b, h].astype(np.float64)
            s = sm * (kk @ qq)
            p = np.exp(s - s.max())
            p /= p.sum()
            out[b, h] = p @ vv
            # fp32 sums of d products, each step at most 2^-23 off; quantised keys as code and
            # midpoint parts
            ds = sm * (sb.d + 8) * 2.0 ** -23 * (np.abs(kk) @ np.abs(qq) + 2 * np.abs(qq).sum() * np.abs(kmid[:n, j]))
            rel = np.expm1(ds) + 2.0 ** -20 + (n / 16 + 64) * 2.0 ** -23
            size = np.abs(vv) + np.abs(vmid[:n, j])[:, None]
            e = (p * rel) @ size + (p @ rel) * np.abs(out[b, h])
            # weights (times the value scale, for codes): fp16 and bf16 round each to half a step,
            # twice with fp32 outputs, where the second term holds what the first left
            e += (p @ size) * (half * half if out_dtype == torch.float32 else half)
            if sb.src == "f16":
                # fp16's smallest step is 2^-24. The largest weight is stored as at least 2^7; with
                # codes, the largest product of a weight and its value's size as at least 2^3 (sizes
                # are powers of two, and may differ by 2^4 within a tile). So a weight is off by half a
                # step, 2^-32 of the largest (2^-28), or by all of itself where that is less
                w, most, step = (p, p.max(), 2.0 ** -32) if sb.kind == "f16" else \
                    (p * vs[:n, j], 2 * (p * np.maximum(vs[:n, j], np.abs(vmid[:n, j]) / 128)).max(), 2.0 ** -28)
                values = np.abs(vv) if sb.kind == "f16" else np.full_like(vv, 8 if sb.kind == "u4t" else 128)
                e += np.minimum(w, step * most) @ values
            if out_dtype != torch.float32:
                # the output's own rounding: half a step of its type, whose smallest is 2^-24 in fp16
                least = 2.0 ** -25 if out_dtype == torch.float16 else 0.0
                e += np.maximum((np.abs(out[b, h]) + e) * torch.finfo(out_dtype).eps / 2, least)
            bound[b, h] = e + 1e-30
    return out, bound


def check(sb, kf, vf, g, scale0, seed, splits=(0,)):
    """Queries with `scale0` in channel 0, which the keys use to set the weights."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((sb.B, sb.hkv * g, sb.d)).astype(np.float32)
    x[..., 0] = scale0
    bits, qf = synth.round_to_dtype(x, sb.src)
    q = to_dev(bits, sb.src)
    for dt in (torch.float32, TORCH[sb.src]):
        out, bound = outcome(sb, kf, vf, qf, g, dt)
        for n in splits:
            got = sb.run(q, dt, num_splits=n).double().cpu().numpy()
            assert np.isfinite(got).all()
            worst = np.abs(got - out) / bound
            assert worst.max() <= 1.0, (dt, n, float(worst.max()), float(np.abs(got - out).max()))


@pytest.mark.parametrize("kind", ["f16", "i8t", "i8g", "u4t"])
@pytest.mark.parametrize("rows,g", [(1, 4), (2, 8), (12, 4), (70, 4)])
def test_loud_values_of_negligible_weight(kind, rows, g):
    # one token in each of two tiles with values 12000 times the others' and a weight of 2^-60:
    # it may cost the others no bits
    n, d = 300, 128
    sb = SharedBatch(kind, 1, d, 64, [(256, [n - 256] * rows)], seed=rows)
    rng = np.random.default_rng(rows)
    k, v = rng.standard_normal((2, n, 1, d)).astype(np.float32)
    k[..., 0] = 0
    for t in (70, 290):
        k[t] = 0
        k[t, 0, 0] = -60 * np.log(2) * np.sqrt(d) / 8
        v[t] *= 12000
    kf, vf = rewrite(sb, k, v)
    check(sb, kf, vf, g, 8.0, rows, (0, 1))


@pytest.mark.parametrize("kind", ["f16", "i8t", "u4t"])
@pytest.mark.parametrize("rows,g", [(1, 4), (2, 8), (12, 4)])
def test_many_small_weights_beside_a_large_one(kind, rows, g):
    # the first token's weight is 2^25.5 times each of 30000 others', which together make the
    # whole output (its own values are 0); with one block all of them share its reference
    n, d = 30000, 64
    sb = SharedBatch(kind, 1, d, 64, [(n - 40, [40] * rows)], seed=rows)
    k, v = np.zeros((2, n, 1, d), dtype=np.float32)
    k[0, 0, 0] = 25.5 * np.log(2) * np.sqrt(d) / 8
    v[:] = np.where(np.arange(d) % 3 == 0, -1.0, 1.0)
    v[0] = 0
    kf, vf = rewrite(sb, k, v)
    check(sb, kf, vf, g, 8.0, rows, (0, 1, 2))


@pytest.mark.parametrize("kind", ["i8t", "i8g", "u4t"])
@pytest.mark.parametrize("rows,g", [(1, 4), (12, 4)])
def test_value_scales_far_from_one(kind, rows, g):
    # a power of two in the values' scales and zero points is that power in the outputs. Exponents
    # s - r are then up to 128 in magnitude, so that each is rounded by up to 2^-18 (half a step of
    # fp32 from 64 on): weights 2^-18 ln 2 off, above and below the quotient, here and in `ref`
    # (which has less): 4 * 2^-18 ln 2 < 2^-16 of the largest value
    sb = SharedBatch(kind, 1, 64, 64, [(300, [40] * rows)], seed=rows)
    q, _ = sb.queries(g)
    ref = sb.run(q)
    tol = 2.0 ** -16 * max(np.abs(v).max() for v in sb.v)
    sz = sb.cache.kv_sz.clone()
    for power in (2.0 ** -65, 2.0 ** 90):
        sb.cache.kv_sz[..., 2:] = sz[..., 2:] * power
        assert float((sb.run(q) / power - ref).abs().max()) <= tol
    sb.cache.kv_sz[..., 2:] = 0       # values that are all 0
    assert torch.count_nonzero(sb.run(q)) == 0
