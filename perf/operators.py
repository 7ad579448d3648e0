"""Cases that measure the operators for sequences that share pages: page copies,
pool compaction, and decode attention over a shared prefix.

Plain forms are elementary torch operations; with `own` set, the same work goes
through paged_kv_cache_243_gb300.cache.
"""
import math
import random

import numpy as np
import torch

own = False

# kind of cache -> (kv_dtype and quant of PagedKVCache, bits of a stored value,
# tokens that share one scale, type of q and of the output)
KINDS = {
    "bf16": ("bf16", "none", 16, 0, torch.bfloat16),
    "f16": ("f16", "none", 16, 0, torch.float16),
    "int8 token": ("int8", "per_token", 8, 1, torch.float16),
    "int8 group": ("int8", "per_group64", 8, 64, torch.bfloat16),
    "u4 token": ("u4", "per_token", 4, 1, torch.float16),
}


def listed():
    return [
        # one sequence forked at a token inside a page: the one page that both would write
        {"name": "copy, one forked page", "op": "copy", "kind": "bf16", "hkv": 8, "d": 128, "ps": 16,
         "pages": 1, "rows": 0, "boxes": False},
        # 32 beams that each split off their open page, with its boxes and the open groups' originals
        {"name": "copy, 32 beams per-group int8", "op": "copy", "kind": "int8 group", "hkv": 8, "d": 128,
         "ps": 64, "pages": 32, "rows": 32, "boxes": True},
        # a whole long context duplicated (32 heads of 128 channels, pages of 16)
        {"name": "copy, 16K tokens bf16", "op": "copy", "kind": "bf16", "hkv": 32, "d": 128, "ps": 16,
         "pages": 1024, "rows": 0, "boxes": False},
        # the pool after a third of its sequences has ended, drawn together
        {"name": "compact, small u4 pool", "op": "compact", "kind": "u4 token", "hkv": 4, "d": 64, "ps": 48,
         "pages": 701, "batch": 13, "boxes": True},
        {"name": "compact, large int8 pool", "op": "compact", "kind": "int8 token", "hkv": 8, "d": 128,
         "ps": 16, "pages": 16384, "batch": 48, "boxes": False},
        # a short prompt answered twice: the smallest call, all latency
        {"name": "attend, 2 rows short", "op": "attend", "kind": "f16", "hkv": 4, "g": 1, "d": 64, "ps": 16,
         "batch": 2, "groups": 1, "alone": 0, "prefix": 100, "suffix": 17, "mix": 1},
        # parallel samples of one system prompt, ordinary sizes
        {"name": "attend, 32 rows 2K bf16", "op": "attend", "kind": "bf16", "hkv": 8, "g": 4, "d": 128,
         "ps": 16, "batch": 32, "groups": 1, "alone": 0, "prefix": 2048, "suffix": 512, "mix": 2},
        # requests of several applications with prompts of their own, some requests with none
        {"name": "attend, 5 groups f16", "op": "attend", "kind": "f16", "hkv": 8, "g": 8, "d": 128, "ps": 64,
         "batch": 61, "groups": 5, "alone": 7, "prefix": 5000, "suffix": 777, "mix": 3},
        # a long document asked about 16 times, one kv head per query head: its reading is the whole time
        {"name": "attend, 16 rows 32K heads 32", "op": "attend", "kind": "bf16", "hkv": 32, "g": 1, "d": 128,
         "ps": 16, "batch": 16, "groups": 1, "alone": 0, "prefix": 32768, "suffix": 64, "mix": 4},
        # a large batch behind one prompt: the products outweigh the reading
        {"name": "attend, 256 rows 8K bf16", "op": "attend", "kind": "bf16", "hkv": 8, "g": 4, "d": 128,
         "ps": 32, "batch": 256, "groups": 1, "alone": 0, "prefix": 8192, "suffix": 256, "mix": 5},
        # quantised caches
        {"name": "attend, 64 rows 8K int8", "op": "attend", "kind": "int8 token", "hkv": 8, "g": 4, "d": 128,
         "ps": 16, "batch": 64, "groups": 2, "alone": 0, "prefix": 8192, "suffix": 300, "mix": 6},
        {"name": "attend, 24 rows 16K u4", "op": "attend", "kind": "u4 token", "hkv": 8, "g": 4, "d": 128,
         "ps": 16, "batch": 24, "groups": 1, "alone": 2, "prefix": 16384, "suffix": 200, "mix": 7},
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], even over its logarithm."""
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    kind = rng.choice(sorted(KINDS))
    d = rng.choice([64, 128])
    ps = rng.choice([64, 128, 256] if kind == "int8 group" else [16, 32, 48, 64, 128, 256])
    op = rng.choice(["copy", "compact", "attend", "attend", "attend"])
    if op != "attend":
        case = {"op": op, "kind": kind, "hkv": _log(rng, 1, 32), "d": d, "ps": ps, "boxes": rng.random() < 0.4}
        page = case["hkv"] * ps * d * KINDS[kind][2] // 4          # bytes of K and V
        if op == "copy":
            case["pages"] = _log(rng, 1, max(1, min(1100, (250 << 20) // page)))
            case["rows"] = rng.randint(0, 40) if kind == "int8 group" else 0
        else:
            case["pages"] = _log(rng, 16, max(16, min(16384, (500 << 20) // page)))
            case["batch"] = rng.randint(1, 64)
        return case
    hkv, g = rng.choice([(1, 8), (1, 16), (2, 7), (4, 1), (4, 3), (5, 2), (8, 1), (8, 4), (8, 8), (16, 2), (32, 1)])
    prefix, suffix = _log(rng, 1, 32768), rng.choice([0, 1, _log(rng, 2, 1024)])
    # the largest listed case gathers 2.2e9 values of K
    most = max(1, min(256, int(1.6e9 / ((prefix + suffix + 1) * hkv * d))))
    batch = _log(rng, 1, most)
    groups = rng.randint(1, max(1, min(8, batch // 2)))
    alone = rng.randint(0, batch - groups) if rng.random() < 0.3 else 0
    return {"op": op, "kind": kind, "hkv": hkv, "g": g, "d": d, "ps": ps, "batch": batch, "groups": groups,
            "alone": alone, "prefix": prefix, "suffix": suffix, "mix": rng.randint(0, 1 << 20)}


def _layout(case):
    """Group of every row (-1: none), the groups' prefix lengths and the rows' lengths."""
    r = random.Random(case["mix"])
    B, ng = case["batch"], case["groups"]
    group = list(range(ng)) + [r.randrange(ng) for _ in range(B - ng - case["alone"])] + [-1] * case["alone"]
    r.shuffle(group)
    prefix = [case["prefix"]] + [r.randint((case["prefix"] + 1) // 2, case["prefix"]) for _ in range(ng - 1)]
    lens = [(prefix[g] if g >= 0 else 0) + r.randint(1 if case["suffix"] else 0, case["suffix"]) for g in group]
    return group, prefix, lens


def _plan_compact(case):
    """The pages in use (by row) and the moves that bring them to the pool's start."""
    r = random.Random(case["pages"] * 64 + case["batch"])
    live = max(1, case["pages"] * 2 // 3)
    ids = sorted(r.sample(range(case["pages"]), live))
    used = set(ids)
    src = [p for p in ids if p >= live]
    dst = [p for p in range(live) if p not in used]
    r.shuffle(ids)
    return ids, src, dst[: len(src)]


# ------------------------------------------------------------------- inputs
def _pools(case, pages, gen):
    """Pools of normally distributed tokens, stored as the cache stores them: K and V,
    the scales, and (where kept) the pages' boxes."""
    kv_dtype, quant, bits, gran, q_dtype = KINDS[case["kind"]]
    hkv, ps, d = case["hkv"], case["ps"], case["d"]
    if bits == 16:
        k, v = (torch.empty((pages, hkv, ps, d), dtype=q_dtype, device="cuda").normal_(generator=gen) for _ in range(2))
        return {"k": k, "v": v, "sz": None}
    row = d * bits // 8
    st = {"k": torch.empty((pages, hkv, ps, row), dtype=torch.uint8, device="cuda"),
          "v": torch.empty((pages, hkv, ps, row), dtype=torch.uint8, device="cuda"),
          "sz": torch.empty((pages, hkv, ps // gran, 4), device="cuda")}
    # a few loud channels in K, as the workloads of this repository have them
    loud = torch.ones(hkv, 1, d, device="cuda")
    loud[..., torch.randperm(d, generator=gen, device="cuda")[:4]] = 15.0
    step = max(1, (64 << 20) // (hkv * ps * d))
    for p in range(0, pages, step):
        n = min(step, pages - p)
        for c, name in enumerate(("k", "v")):
            x = torch.empty((n, hkv, ps, d), device="cuda").normal_(generator=gen)
            x = (x * loud if c == 0 else x).view(n, hkv, ps // gran, gran * d)
            lo, hi = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
            s = (hi - lo) / (2 ** bits - 1)
            u = ((x - lo) / s).round().clamp(0, 2 ** bits - 1).to(torch.uint8).view(n, hkv, ps, d)
            st[name][p:p + n] = u if bits == 8 else u[..., 0::2] | (u[..., 1::2] << 4)
            st["sz"][p:p + n, ..., 2 * c] = s[..., 0]
            st["sz"][p:p + n, ..., 2 * c + 1] = lo[..., 0]
    return st


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    kv_dtype, quant, bits, gran, q_dtype = KINDS[case["kind"]]
    dev = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    if case["op"] != "attend":
        n = case["pages"]
        st = _pools(case, 2 * n + 3 if case["op"] == "copy" else n, gen)
        st["boxes"] = (torch.empty((st["k"].shape[0], case["hkv"], 2, case["d"]), device="cuda").normal_(generator=gen)
                       if case["boxes"] else None)
        st["tail"] = None
        st["src_rows"] = st["dst_rows"] = None
        if case["op"] == "copy":
            order = np.random.default_rng(seed).permutation(2 * n + 3).astype(np.int32)
            st["src"], st["dst"] = order[:n].copy(), order[n:2 * n].copy()
            if case["rows"]:
                m = case["rows"]
                st["tail"] = torch.empty((2 * m, case["hkv"], 2, 2, 64, case["d"]), device="cuda").normal_(generator=gen)
                order = np.random.default_rng(seed + 1).permutation(2 * m).astype(np.int32)
                st["src_rows"], st["dst_rows"] = order[:m].copy(), order[m:].copy()
        else:
            ids, src, dst = _plan_compact(case)
            st["src"], st["dst"] = np.array(src, dtype=np.int32), np.array(dst, dtype=np.int32)
            width = -(-len(ids) // case["batch"])
            table = np.full(case["batch"] * width, -1, dtype=np.int32)
            table[: len(ids)] = ids
            st["table"] = dev(table.reshape(case["batch"], width))
        st["at"] = {k: torch.from_numpy(st[k]).long().cuda() for k in ("src", "dst", "src_rows", "dst_rows")
                    if st[k] is not None}
    else:
        group, prefix, lens = _layout(case)
        ps = case["ps"]
        whole = [p // ps for p in prefix]                       # pages that a group's rows have in common
        shared = [0] * len(prefix)
        need = 0
        for g, w in enumerate(whole):
            shared[g], need = need, need + w
        width = max(1, max(-(-n // ps) for n in lens) + 1)
        table = np.full((len(lens), width), -1, dtype=np.int64)
        for b, (g, n) in enumerate(zip(group, lens)):
            w = whole[g] if g >= 0 else 0
            mine = -(-n // ps) - w
            table[b, :w] = np.arange(w) + (shared[g] if g >= 0 else 0)
            table[b, w:w + mine] = np.arange(need, need + mine)
            need += mine
        pages = need + 2
        table = np.where(table < 0, -1, np.random.default_rng(seed).permutation(pages)[table])
        st = _pools(case, pages, gen)
        # a prefix that ends inside a page: each row has its own copy of that page,
        # with the prefix's tokens in it (per-group scales: its whole groups)
        first = {g: b for b, g in reversed(list(enumerate(group))) if g >= 0}
        for b, g in enumerate(group):
            rest = prefix[g] % ps if g >= 0 else 0
            rest = rest if gran != 64 else rest // 64 * 64
            if rest and b != first[g]:
                mine, other = int(table[b, whole[g]]), int(table[first[g], whole[g]])
                for name, per in (("k", 1), ("v", 1), ("sz", gran)):
                    if st[name] is not None:
                        st[name][mine, :, :rest // per] = st[name][other, :, :rest // per]
        st["table"], st["lens"] = dev(table), dev(lens)
        st["group"], st["prefix"] = dev(group), dev(prefix)
        st["q"] = torch.empty((len(lens), case["hkv"] * case["g"], case["d"]), dtype=q_dtype,
                              device="cuda").normal_(generator=gen)
        st["longest"] = max(lens)
    st["case"] = dict(case)
    return st


# ---------------------------------------------------------------- the passes
def _handle(st):
    """The cache object that a program makes once for its pools."""
    if "cache" not in st:
        from paged_kv_cache_243_gb300.cache import PagedKVCache
        kv_dtype, quant, bits, gran, q_dtype = KINDS[st["case"]["kind"]]
        st["cache"] = PagedKVCache.from_pools(st["k"], st["v"], kv_dtype=kv_dtype, quant=quant, kv_sz=st["sz"],
                                              tail=st.get("tail"), page_meta=st.get("boxes"))
    return st["cache"]


def _buffers(st):
    """The pools' bits (whole numbers: a copy is exact), and the rewritten table."""
    got = {n: st[n].view(torch.int16 if st[n].element_size() == 2 else torch.uint8 if st[n].element_size() == 1
                         else torch.int32) for n in ("k", "v", "sz", "boxes", "tail") if st[n] is not None}
    if st["case"]["op"] == "compact":
        got["table"] = st["table"]
    return got


def _restored(st, name, pages, slots):
    """Tokens [B][T][Hkv][d] in 32 bits through page and slot indexes [B][T]."""
    kv_dtype, quant, bits, gran, q_dtype = KINDS[st["case"]["kind"]]
    x = st[name][pages, :, slots]
    if bits == 16:
        return x.float()
    if bits == 4:
        x = torch.stack((x & 15, x >> 4), -1).flatten(-2)
    sz = st["sz"][pages, :, slots // gran]
    c = 0 if name == "k" else 2
    return x.float() * sz[..., c:c + 1] + sz[..., c + 1:c + 2]


def run(st):
    case = st["case"]
    if case["op"] != "attend":
        if own:
            cache = _handle(st)
            cache.copy_pages(st["src"], st["dst"], st["src_rows"], st["dst_rows"])
            if case["op"] == "compact":
                cache.remap_table(st["table"], st["src"], st["dst"])
            return _buffers(st)
        at = st["at"]
        for name in [n for n in ("k", "v", "sz", "boxes") if st[n] is not None]:
            st[name][at["dst"]] = st[name][at["src"]]
        if st["tail"] is not None:
            st["tail"][at["dst_rows"]] = st["tail"][at["src_rows"]]
        if case["op"] == "compact":
            to = torch.arange(st["k"].shape[0], device="cuda", dtype=torch.int32)
            to[at["src"]] = at["dst"].int()
            t = st["table"]
            t.copy_(torch.where(t >= 0, to[t.clamp(min=0).long()], t))
        return _buffers(st)
    if own:
        return _handle(st).shared_attention(st["q"], st["table"], st["lens"], st["group"], st["prefix"],
                                            out_dtype=st["q"].dtype)
    q, ps, hkv, g = st["q"].float(), case["ps"], case["hkv"], case["g"]
    t = torch.arange(max(1, st["longest"]), device="cuda")
    pages = st["table"][:, t // ps].long().clamp(min=0)
    slots = (t % ps).expand_as(pages)
    seen = t < st["lens"][:, None]                                        # [B][T]
    k = _restored(st, "k", pages, slots)
    s = torch.einsum("bhgd,bthd->bhgt", q.view(q.shape[0], hkv, g, -1), k) / math.sqrt(case["d"])
    del k
    s = s.masked_fill(~seen[:, None, None], float("-inf"))
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(torch.isinf(top), torch.zeros_like(top), top))
    del s
    v = _restored(st, "v", pages, slots) * seen[..., None, None]
    o = torch.einsum("bhgt,bthd->bhgd", p, v) / p.sum(-1, keepdim=True).clamp(min=1e-30)
    return o.reshape(q.shape).to(st["q"].dtype)


def work(case):
    kv_dtype, quant, bits, gran, q_dtype = KINDS[case["kind"]]
    hkv, d, ps = case["hkv"], case["d"], case["ps"]
    token = hkv * (d * bits // 4 + (16 / gran if gran else 0))             # bytes of K, V and scales
    if case["op"] != "attend":
        n = case["pages"]
        if case["op"] == "compact":
            ids, src, dst = _plan_compact(case)
            n = len(src)
        page = ps * token + (hkv * 2 * d * 4 if case["boxes"] else 0)
        b = 2 * n * page
        if case["op"] == "copy":
            b += 2 * case["rows"] * hkv * 2 * 2 * 64 * d * 4
        else:
            b += 4 * 2 * len(ids)
        return {"bytes": b, "flops": 0}
    group, prefix, lens = _layout(case)
    once = sum(p for g, p in enumerate(prefix) if g in group)
    each = sum(n - (prefix[g] if g >= 0 else 0) for g, n in zip(group, lens))
    rows = len(lens) * hkv * case["g"] * d
    return {"bytes": (once + each) * token + 2 * 2 * rows + 4 * sum(-(-n // ps) for n in lens),
            "flops": 4 * sum(lens) * hkv * case["g"] * d}


def exact(case, seed):
    """Attention row by row in 64 bits; copies have no computed numbers."""
    if case["op"] != "attend":
        return None
    st = prepare(case, seed)
    kv_dtype, quant, bits, gran, q_dtype = KINDS[case["kind"]]
    ps, hkv, g, d = case["ps"], case["hkv"], case["g"], case["d"]
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    lens, table = st["lens"].tolist(), st["table"].long()

    def whole(name, ids):
        x = st[name][ids].transpose(0, 1)                                  # [Hkv][pages][ps][...]
        if bits == 4:
            y = torch.empty(*x.shape[:-1], d, dtype=torch.float64, device="cuda")
            y[..., 0::2], y[..., 1::2] = (x % 16).double(), (x // 16).double()
        else:
            y = x.double()
        if gran:
            sz = st["sz"][ids].transpose(0, 1).double().repeat_interleave(gran, 2)
            y = y * sz[..., :1] + sz[..., 1:2] if name == "k" else y * sz[..., 2:3] + sz[..., 3:]
        return y.reshape(hkv, -1, d)

    for b, n in enumerate(lens):
        if n == 0:
            continue
        ids = table[b, : -(-n // ps)]
        w = torch.softmax(st["q"][b].double().view(hkv, g, d) @ whole("k", ids)[:, :n].transpose(1, 2) / d ** 0.5, -1)
        out[b] = (w @ whole("v", ids)[:, :n]).reshape(hkv * g, d)
    return out
