"""Cases that measure the operators of a decode step with drafted tokens: rotary positions on the
way into the cache, attention for a tree of drafted tokens, and keeping the tokens of the path
that was accepted.

Plain forms are elementary torch operations; with `own` set, the same work goes
through paged_kv_cache_243_gb300.cache.
"""
import math
import random

import numpy as np
import torch

own = False

# kind of cache -> (kv_dtype and quant of PagedKVCache, bits of a stored value,
# tokens that share one scale, type of q, k, v and of the output)
KINDS = {
    "bf16": ("bf16", "none", 16, 0, torch.bfloat16),
    "f16": ("f16", "none", 16, 0, torch.float16),
    "int8 token": ("int8", "per_token", 8, 1, torch.float16),
    "int8 group": ("int8", "per_group64", 8, 64, torch.bfloat16),
    "u4 token": ("u4", "per_token", 4, 1, torch.float16),
}


def listed():
    return [
        # one decode step of a small batch: one token a sequence, all latency
        {"name": "rotary, 4 tokens bf16", "op": "rotary", "kind": "bf16", "hkv": 8, "g": 4, "d": 128, "ps": 16,
         "batch": 4, "tokens": 1, "start": 2048, "rot": 128, "pairs": "halves", "packed": True, "mix": 1},
        # drafts of a large batch, neighbouring channels paired, half of each head rotated, far positions
        {"name": "rotary, 61 x 11 f16 part", "op": "rotary", "kind": "f16", "hkv": 4, "g": 7, "d": 64, "ps": 48,
         "batch": 61, "tokens": 11, "start": 120000, "rot": 32, "pairs": "neighbours", "packed": False, "mix": 2},
        # prompts of ordinary length on their way into the cache
        {"name": "rotary, 4 x 8K prompt bf16", "op": "rotary", "kind": "bf16", "hkv": 8, "g": 4, "d": 128, "ps": 16,
         "batch": 4, "tokens": 8192, "start": 0, "rot": 128, "pairs": "halves", "packed": True, "mix": 3},
        # what a step leaves: a few tokens of one sequence
        {"name": "keep, 1 row", "op": "keep", "kind": "f16", "hkv": 4, "g": 1, "d": 64, "ps": 16, "batch": 1,
         "tokens": 13, "len": 100, "path": 4, "boxes": False, "mix": 4},
        # a large batch with page boxes, trees of 64 tokens
        {"name": "keep, 128 rows boxes", "op": "keep", "kind": "bf16", "hkv": 8, "g": 4, "d": 128, "ps": 16,
         "batch": 128, "tokens": 64, "len": 500, "path": 9, "boxes": True, "mix": 5},
        # the smallest tree: five tokens of one short sequence
        {"name": "tree, 1 row short", "op": "tree", "kind": "f16", "hkv": 4, "g": 1, "d": 64, "ps": 16, "batch": 1,
         "tokens": 5, "len": 107, "tree": "tree", "ragged": False, "mix": 6},
        # an ordinary serving batch, 64 query rows for each kv head
        {"name": "tree, 8 x 4K bf16", "op": "tree", "kind": "bf16", "hkv": 8, "g": 4, "d": 128, "ps": 16, "batch": 8,
         "tokens": 16, "len": 4096, "tree": "tree", "ragged": True, "mix": 7},
        # long contexts with a kv head for every query head: reading them is the whole time
        {"name": "tree, 4 x 32K heads 32", "op": "tree", "kind": "f16", "hkv": 32, "g": 1, "d": 128, "ps": 16,
         "batch": 4, "tokens": 13, "len": 32768, "tree": "tree", "ragged": False, "mix": 8},
        # a large batch with large trees: the products outweigh the reading
        {"name": "tree, 24 x 8K of 64", "op": "tree", "kind": "bf16", "hkv": 8, "g": 4, "d": 128, "ps": 32,
         "batch": 24, "tokens": 64, "len": 8192, "tree": "tree", "ragged": False, "mix": 9},
        # the last 200 tokens of two long prompts, each after the one before (no mask)
        {"name": "chain, 2 x 16K of 200", "op": "tree", "kind": "f16", "hkv": 4, "g": 8, "d": 128, "ps": 64,
         "batch": 2, "tokens": 200, "len": 16000, "tree": "chain", "ragged": True, "mix": 10},
        # whole steps on quantised caches: keep the last step's path, rotate and store the
        # new drafts, attend
        {"name": "step, 16 x 8K int8", "op": "step", "kind": "int8 token", "hkv": 8, "g": 4, "d": 128, "ps": 16,
         "batch": 16, "tokens": 24, "len": 8192, "path": 5, "rot": 128, "pairs": "halves", "tree": "tree",
         "ragged": True, "mix": 11},
        {"name": "step, 5 x 1K u4", "op": "step", "kind": "u4 token", "hkv": 4, "g": 2, "d": 64, "ps": 32,
         "batch": 5, "tokens": 7, "len": 1000, "path": 3, "rot": 48, "pairs": "neighbours", "tree": "tree",
         "ragged": False, "mix": 12},
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], even over its logarithm."""
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


HEADS = [(1, 8), (1, 16), (2, 7), (4, 1), (4, 3), (5, 2), (8, 1), (8, 4), (8, 8), (16, 2), (32, 1)]   # (hkv, g)


def draw(rng):
    op = rng.choice(["rotary", "rotary", "keep", "tree", "tree", "tree", "step"])
    kind = rng.choice({"tree": sorted(KINDS), "step": ["int8 token", "u4 token"]}.get(op, ["bf16", "f16"]))
    (hkv, g), d = rng.choice(HEADS), rng.choice([64, 128])
    ps = rng.choice([64, 128, 256] if kind == "int8 group" else [16, 32, 48, 64, 128, 256])
    case = {"op": op, "kind": kind, "hkv": hkv, "g": g, "d": d, "ps": ps, "mix": rng.randint(0, 1 << 20)}
    turn = {"rot": 16 * rng.randint(1, d // 16), "pairs": rng.choice(["halves", "neighbours"])}
    if op == "rotary":
        most = max(1, 200_000_000 // ((g + 2) * hkv * d))              # tokens of the largest listed case
        case["tokens"] = 1 if rng.random() < 0.4 else _log(rng, 2, min(8192, most))
        case["batch"] = _log(rng, 1, max(1, min(512, most // case["tokens"])))
        return dict(case, start=_log(rng, 1, 120000), packed=rng.random() < 0.5, **turn)
    if op == "keep":
        T = _log(rng, 1, 256)
        return dict(case, tokens=T, path=rng.randint(1, min(T, 24)), batch=_log(rng, 1, 128), len=_log(rng, 1, 1000),
                    boxes=rng.random() < 0.5)
    T, L = (1 if rng.random() < 0.15 else _log(rng, 2, 256)), _log(rng, 1, 32768)
    # no more values of K, and no more scores, than the largest listed cases have
    most = min(800_000_000 // ((L + T) * hkv * d), 400_000_000 // ((L + T) * hkv * g * T))
    if most < 1:
        L = max(1, L // 16)
        most = max(1, min(800_000_000 // ((L + T) * hkv * d), 400_000_000 // ((L + T) * hkv * g * T)))
    case.update(tokens=T, len=L + T, batch=_log(rng, 1, min(128, most)), tree=rng.choice(["tree", "tree", "chain"]),
                ragged=rng.random() < 0.5)
    return case if op == "tree" else dict(case, path=rng.randint(1, min(T, 12)), **turn)


def _layout(case):
    """For each row: tokens in the cache before the drafts, its drafts, and the tokens kept of the step before."""
    r = random.Random(case["mix"])
    T, B = case["tokens"], case["batch"]
    drafts = [T] + [r.randint(max(1, T // 2), T) for _ in range(B - 1)] if case.get("ragged") else [T] * B
    keep = [0] * B
    if "path" in case:
        keep = [case["path"]] + [r.randint(1, case["path"]) for _ in range(B - 1)]
    if case["op"] == "rotary":
        base = [r.randint(case["start"] // 2, case["start"]) for _ in range(B)]
    else:
        top = max(0, case["len"] - T)
        base = [top] + [r.randint(top // 2, top) for _ in range(B - 1)]
    return base, drafts, keep


def _parents(case):
    """A tree for each row: the parent of every draft, -1 for the first."""
    r = random.Random(case["mix"] + 1)
    T = case["tokens"]
    return [[-1] + [max(0, i - 1 - int(r.expovariate(0.4))) for i in range(1, T)] for _ in range(case["batch"])]


def _masks(parents):
    """[B][T][T]: whether draft t attends to draft j, i.e. j lies on the path to t."""
    B, T = len(parents), len(parents[0])
    seen = np.zeros((B, T, T), dtype=bool)
    for b in range(B):
        for t, p in enumerate(parents[b]):
            if p >= 0:
                seen[b, t] = seen[b, p]
            seen[b, t, t] = True
    return seen


def _path(r, parents, n):
    """n drafts of one path, from the tree's first on: strictly ascending."""
    T = len(parents)
    children = [[] for _ in range(T)]
    for t, p in enumerate(parents):
        if p >= 0:
            children[p].append(t)
    at, path = 0, [0]
    while len(path) < n and children[at]:
        at = r.choice(children[at])
        path.append(at)
    return path


def _paths(case, kept):
    """The drafts that each row keeps: a path of its tree, or as much of one as there is."""
    r = random.Random(case["mix"] + 2)
    paths = [_path(r, p, n) if n else [] for p, n in zip(_parents(case), kept)]
    if case["op"] == "keep":
        return paths
    # a step goes on behind the number of tokens that it has counted: other drafts make it up
    return [sorted(p + r.sample([t for t in range(case["tokens"]) if t not in p], n - len(p))) for p, n in zip(paths, kept)]


# ------------------------------------------------------------------- inputs
def _pools(case, pages, gen):
    """Pools of normally distributed tokens, stored as the cache stores them: K and V, and the scales."""
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


def _frequencies(rot):
    return 10000.0 ** (-np.arange(0, rot, 2, dtype=np.float64) / rot)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    kv_dtype, quant, bits, gran, dtype = KINDS[case["kind"]]
    hkv, hq, d, ps, B, T = (case[n] for n in ("hkv", "g", "d", "ps", "batch", "tokens"))
    hq *= hkv
    dev = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    base, drafts, kept = _layout(case)
    first = [max(0, b - k) for b, k in zip(base, kept)] if case["op"] == "step" else base
    kept = [b - f for b, f in zip(base, first)] if case["op"] == "step" else kept
    # pages: every one that the call reads or writes is a row's own; the others stand for pages that it does not touch
    ends = [b + n for b, n in zip(base, drafts)] if case["op"] != "keep" else [b + T for b in base]
    lo = [0 if case["op"] in ("tree", "step") else max(0, f - 1) // ps for f in first]
    if case["op"] == "step":                       # the drafts of the step before may reach further
        ends = [max(e, f + T) for e, f in zip(ends, first)]
    hi = [-(-e // ps) for e in ends]
    width = max(hi) + 1
    pages = sum(h - l for h, l in zip(hi, lo)) + 2
    ids = np.random.default_rng(seed).permutation(pages)
    spare = int(ids[-1])
    table = np.full((B, width), spare, dtype=np.int64)
    at = 0
    for b in range(B):
        table[b, lo[b]:hi[b]] = ids[at:at + hi[b] - lo[b]]
        at += hi[b] - lo[b]
    st = _pools(case, pages, gen)
    st["table"], st["first"], st["spare"] = dev(table), dev(first), spare
    if case["op"] in ("rotary", "step"):
        st["base"], st["drafts"] = dev(base), dev(drafts)
        # angles in 64 bits, for the positions that the sequences may reach
        rot = case["rot"]
        angle = torch.arange(max(base) + T, device="cuda", dtype=torch.float64)[:, None] * \
            torch.from_numpy(_frequencies(rot)).cuda()
        st["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float()
        if case.get("packed"):       # slices of one projection's output
            x = torch.empty((B, T, hq + 2 * hkv, d), dtype=dtype, device="cuda").normal_(generator=gen)
            st["q"], st["kn"], st["vn"] = x[:, :, :hq], x[:, :, hq:hq + hkv], x[:, :, hq + hkv:]
        else:
            st["q"], st["kn"], st["vn"] = (torch.empty((B, T, h, d), dtype=dtype, device="cuda").normal_(generator=gen)
                                           for h in (hq, hkv, hkv))
    if case["op"] in ("keep", "step"):
        path = _paths(case, kept)
        keep = np.full((B, case["path"]), -1, dtype=np.int64)
        for b, p in enumerate(path):
            keep[b, :len(p)] = p
        st["keep"], st["keep_lens"] = dev(keep), dev([len(p) for p in path])
        st["boxes"] = (torch.empty((pages, hkv, 2, d), device="cuda").normal_(generator=gen) if case.get("boxes") else None)
    if case["op"] in ("tree", "step"):
        st["lens"], st["drafts"] = dev([b + n for b, n in zip(base, drafts)]), dev(drafts)
        st["longest"] = max(b + n for b, n in zip(base, drafts))
        st["mask"] = depth = None
        if case["tree"] == "tree":
            seen = _masks(_parents(case))
            words = -(-T // 64)
            bit = np.left_shift(np.uint64(1), np.arange(T, dtype=np.uint64) % np.uint64(64))
            mask = np.zeros((B, T, words), dtype=np.uint64)
            for w in range(words):
                mask[..., w] = np.where(seen[..., 64 * w:64 * w + 64], bit[64 * w:64 * w + 64], np.uint64(0)).sum(-1, dtype=np.uint64)
            st["mask"] = torch.from_numpy(mask.view(np.int64)).cuda()
            depth = seen.sum(-1) - 1
        if case["op"] == "tree":
            st["q"] = torch.empty((B, T, hq, d), dtype=dtype, device="cuda").normal_(generator=gen)
        else:                        # a draft's position goes by its depth in the tree
            depth = np.broadcast_to(np.arange(T), (B, T)) if depth is None else depth
            st["turns"] = dev((np.array(base)[:, None] + depth).tolist())
    st["case"] = dict(case)
    return st


# ---------------------------------------------------------------- the passes
def _handle(st):
    """The cache object that a program makes once for its pools."""
    if "cache" not in st:
        from paged_kv_cache_243_gb300.cache import PagedKVCache
        kv_dtype, quant, bits, gran, q_dtype = KINDS[st["case"]["kind"]]
        st["cache"] = PagedKVCache.from_pools(st["k"], st["v"], kv_dtype=kv_dtype, quant=quant, kv_sz=st["sz"],
                                              page_meta=st.get("boxes"))
    return st["cache"]


def _places(st, at, on):
    """Pages and slots of positions at [B][N]; the spare page's where they are not `on`."""
    ps = st["case"]["ps"]
    at = at.clamp(min=0).long()
    page = st["table"].long().gather(1, (at // ps).clamp(max=st["table"].shape[1] - 1))
    return torch.where(on, page, st["spare"]), torch.where(on, at % ps, 0)


def _rotate(st, x, at):
    """x [B][T][H][d] rotated by the angles of positions at [B][T], in 32 bits."""
    rot = st["case"]["rot"]
    cs = st["cos_sin"][at.long()]
    c, s = cs[:, :, None, :rot // 2], cs[:, :, None, rot // 2:]
    y = x.float()
    if st["case"]["pairs"] == "halves":
        a, b = y[..., :rot // 2], y[..., rot // 2:rot]
        turned = torch.cat([a * c - b * s, b * c + a * s], -1)
    else:
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
        turned = torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
    return torch.cat([turned, y[..., rot:]], -1)


def _store(st, k, v):
    """New tokens k, v [B][T][Hkv][d] in 32 bits into the pools from base on; drafts beyond a row's go nowhere."""
    kv_dtype, quant, bits, gran, dtype = KINDS[st["case"]["kind"]]
    t = torch.arange(k.shape[1], device="cuda")
    on = t < st["drafts"][:, None]
    page, slot = _places(st, st["base"][:, None] + t, on)
    own_row = lambda pool, new: torch.where(on.view(*on.shape, *[1] * (new.dim() - 2)), new, pool[page, :, slot])  # noqa: E731
    if bits == 16:
        st["k"][page, :, slot] = own_row(st["k"], k.to(dtype))
        st["v"][page, :, slot] = own_row(st["v"], v.to(dtype))
        return

    def codes(x):
        lo, hi = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
        s = (hi - lo) / torch.full_like(hi, 2 ** bits - 1)
        u = ((x - lo) / s).round().clamp(0, 2 ** bits - 1)
        u = torch.where(s > 0, u, torch.zeros_like(u)).to(torch.uint8)
        return (u if bits == 8 else u[..., 0::2] | (u[..., 1::2] << 4)), s, lo

    (uk, sk, zk), (uv, sv, zv) = codes(k), codes(v)
    st["k"][page, :, slot] = own_row(st["k"], uk)
    st["v"][page, :, slot] = own_row(st["v"], uv)
    st["sz"][page, :, slot] = own_row(st["sz"], torch.cat([sk, zk, sv, zv], -1))


def _restored(st, name, pages, slots):
    """Tokens [B][N][Hkv][d] in 32 bits through page and slot indexes [B][N]."""
    kv_dtype, quant, bits, gran, q_dtype = KINDS[st["case"]["kind"]]
    x = st[name][pages, :, slots]
    if bits == 16:
        return x.float()
    if bits == 4:
        x = torch.stack((x & 15, x >> 4), -1).flatten(-2)
    sz = st["sz"][pages, :, slots // gran]
    c = 0 if name == "k" else 2
    return x.float() * sz[..., c:c + 1] + sz[..., c + 1:c + 2]


def _plain_keep(st):
    case = st["case"]
    ps, keep, n, first = case["ps"], st["keep"], st["keep_lens"], st["first"]
    j = torch.arange(keep.shape[1], device="cuda")
    on = j < n[:, None]
    sp, ss = _places(st, first[:, None] + keep, on)
    dp, ds = _places(st, first[:, None] + j, on)
    moved = {name: st[name][sp, :, ss] for name in ("k", "v", "sz") if st[name] is not None}
    if st["k"] is not None:
        st["k"][dp, :, ds], st["v"][dp, :, ds] = moved["k"], moved["v"]
    if st["sz"] is not None:
        st["sz"][dp, :, ds] = moved["sz"]
    if st["boxes"] is None:
        return
    # boxes of the pages from the last old token's on
    begin = (first - 1).clamp(min=0)[:, None]
    p = torch.arange((keep.shape[1] + ps) // ps + 1, device="cuda") + begin // ps
    end = (first + n)[:, None]
    page, _ = _places(st, p * ps, p * ps < end)
    tok = st["k"][page].float()                                                  # [B][P][Hkv][ps][d]
    seen = (p[..., None] * ps + torch.arange(ps, device="cuda") < end[..., None])[:, :, None, :, None]
    box = torch.stack([tok.masked_fill(~seen, float("inf")).amin(3), tok.masked_fill(~seen, float("-inf")).amax(3)], 3)
    st["boxes"][page] = torch.where((p * ps < end)[:, :, None, None, None], box, st["boxes"][page])


def _plain_attention(st, q):
    """q [B][T][Hq][d] in 32 bits."""
    case = st["case"]
    ps, hkv, g, d, T = (case[n] for n in ("ps", "hkv", "g", "d", "tokens"))
    B = q.shape[0]
    i = torch.arange(max(1, st["longest"]), device="cuda")
    pages = st["table"].long()[:, i // ps]
    slots = (i % ps).expand_as(pages)
    t = torch.arange(T, device="cuda")
    if st["mask"] is None:
        tree = (t <= t[:, None]).expand(B, T, T)
    else:
        tree = (st["mask"][:, :, t // 64] >> (t % 64) & 1) != 0
    tree = tree & (t < st["drafts"][:, None])[:, None] & (t < st["drafts"][:, None])[:, :, None]
    base = (st["lens"] - st["drafts"])[:, None]
    draft = i - base                                                              # [B][N]
    seen = tree.gather(2, draft.clamp(0, T - 1)[:, None].expand(B, T, -1)) & (draft < T)[:, None]
    seen = torch.where((draft < 0)[:, None], (t < st["drafts"][:, None])[:, :, None], seen)   # [B][T][N]
    k = _restored(st, "k", pages, slots)
    x = q.view(B, T, hkv, g, d).permute(0, 2, 1, 3, 4).reshape(B, hkv, T * g, d)
    s = torch.matmul(x, k.permute(0, 2, 3, 1)) / math.sqrt(d)
    del k
    s = s.view(B, hkv, T, g, -1).masked_fill_(~seen[:, None, :, None], float("-inf"))
    top = s.amax(-1, keepdim=True)
    s = s.sub_(torch.where(torch.isinf(top), torch.zeros_like(top), top)).exp_()
    v = _restored(st, "v", pages, slots) * (i < st["lens"][:, None])[..., None, None]
    o = torch.matmul(s.view(B, hkv, T * g, -1), v.permute(0, 2, 1, 3)).view(B, hkv, T, g, d)
    o = o / s.sum(-1, keepdim=True).clamp(min=1e-30)
    return o.permute(0, 2, 1, 3, 4).reshape(B, T, hkv * g, d)


def run(st):
    case = st["case"]
    op, dtype = case["op"], KINDS[case["kind"]][4]
    if own:
        cache = _handle(st)
        got = {}
        if op in ("keep", "step"):
            cache.keep_tokens(st["keep"], st["keep_lens"], st["table"], st["first"])
        if op in ("rotary", "step"):
            q = cache.rotary_append(st["q"], st["kn"], st["vn"], st["cos_sin"], st["table"], st["base"],
                                    rotary_positions=st.get("turns"), new_lens=st["drafts"],
                                    interleaved=case["pairs"] == "neighbours")
            got["q"] = q
        if op in ("tree", "step"):
            got["out"] = cache.tree_attention(st["q"] if op == "tree" else got.pop("q"), st["table"], st["lens"],
                                              st["mask"], st["drafts"], out_dtype=dtype)
    else:
        got = {}
        if op in ("keep", "step"):
            _plain_keep(st)
        if op in ("rotary", "step"):
            at = st["turns"] if op == "step" else st["base"][:, None] + torch.arange(case["tokens"], device="cuda")
            got["q"] = _rotate(st, st["q"], at).to(dtype)
            _store(st, _rotate(st, st["kn"], at), st["vn"].float())
        if op in ("tree", "step"):
            got["out"] = _plain_attention(st, (st["q"] if op == "tree" else got.pop("q")).float()).to(dtype)
    if op in ("rotary", "keep"):
        got["k"], got["v"] = st["k"], st["v"]
    if op == "keep" and st["boxes"] is not None:
        got["boxes"] = st["boxes"]
    return got


def work(case):
    kv_dtype, quant, bits, gran, q_dtype = KINDS[case["kind"]]
    hkv, hq, d, ps, B, T = case["hkv"], case["hkv"] * case["g"], case["d"], case["ps"], case["batch"], case["tokens"]
    token = hkv * (d * bits // 4 + (16 / gran if gran else 0))             # bytes of K, V and scales
    base, drafts, kept = _layout(case)
    if case["op"] == "step":
        kept = [min(x, n) for x, n in zip(base, kept)]
    elif case["op"] == "keep":
        kept = [len(p) for p in _paths(case, kept)]
    b = f = 0
    if case["op"] in ("rotary", "step"):
        n = sum(drafts)
        b += n * (2 * 2 * hq * d + 2 * 2 * hkv * d + token + 4 * case["rot"])
        f += n * 3 * case["rot"] * (hq + hkv)
    if case["op"] in ("keep", "step"):
        b += 2 * sum(kept) * token
        if case.get("boxes"):
            b += sum(-(-(f0 % ps + n) // ps) for f0, n in zip(base, kept)) * hkv * (2 * ps * d + 8 * d)
    if case["op"] in ("tree", "step"):
        lens = [x + n for x, n in zip(base, drafts)]
        b += sum(lens) * token + 2 * 2 * sum(drafts) * hq * d + 4 * sum(-(-n // ps) for n in lens)
        if case["tree"] == "tree":
            b += 8 * -(-T // 64) * sum(drafts)
            seen = _masks(_parents(case))
            pairs = sum(n * x + int(seen[i, :n, :n].sum()) for i, (x, n) in enumerate(zip(base, drafts)))
        else:
            pairs = sum(n * x + n * (n + 1) // 2 for x, n in zip(base, drafts))
        f += 4 * pairs * hq * d
    return {"bytes": b, "flops": f}


# ------------------------------------------------------------------ in 64 bits
def _exact_rotation(x, at, case):
    """x [N][H][d], at [N]: as complex numbers."""
    rot = case["rot"]
    y = x.double().clone()
    z = y[..., :rot]
    z = z.view(*z.shape[:-1], 2, rot // 2).transpose(-1, -2) if case["pairs"] == "halves" else z.view(*z.shape[:-1], rot // 2, 2)
    z = torch.view_as_complex(z.contiguous())
    angle = at.double()[:, None] * torch.from_numpy(_frequencies(rot)).cuda()
    z = torch.view_as_real(z * torch.polar(torch.ones_like(angle), angle)[:, None])
    y[..., :rot] = (z.transpose(-1, -2) if case["pairs"] == "halves" else z).reshape(*y.shape[:-1], rot)
    return y


def exact(case, seed):
    """Row by row in 64 bits."""
    st = prepare(case, seed)
    kv_dtype, quant, bits, gran, dtype = KINDS[case["kind"]]
    ps, hkv, g, d, T, op = (case[n] for n in ("ps", "hkv", "g", "d", "tokens", "op"))
    table = st["table"].tolist()
    first = st["first"].tolist()
    pools = {n: st[n].double() if bits == 16 and op != "tree" else st[n] for n in ("k", "v", "sz") if st[n] is not None}
    boxes = st.get("boxes")
    got = {}
    if op in ("keep", "step"):
        keep, n_keep = st["keep"].tolist(), st["keep_lens"].tolist()
        for b, n in enumerate(n_keep):
            for j in range(n):
                s, t = first[b] + keep[b][j], first[b] + j
                for x in pools.values():
                    x[table[b][t // ps], :, t % ps] = x[table[b][s // ps], :, s % ps].clone()
            for p in range(max(0, first[b] - 1) // ps, -(-(first[b] + n) // ps)) if boxes is not None else ():
                tok = pools["k"][table[b][p], :, :min(ps, first[b] + n - p * ps)]
                boxes[table[b][p], :, 0], boxes[table[b][p], :, 1] = tok.amin(1), tok.amax(1)
    if op in ("rotary", "step"):
        base, drafts = st["base"].tolist(), st["drafts"].tolist()
        at = st["turns"] if op == "step" else st["base"][:, None] + torch.arange(T, device="cuda")
        turned = [_exact_rotation(x.flatten(0, 1), at.flatten(), case).view(x.shape) for x in (st["q"], st["kn"])]
        got["q"] = turned[0]
        for b, n in enumerate(drafts):
            w = base[b] + torch.arange(n, device="cuda")
            page, slot = st["table"][b, w // ps].long(), w % ps
            for c, (name, x) in enumerate((("k", turned[1][b, :n]), ("v", st["vn"][b, :n].double()))):
                if bits == 16:
                    pools[name][page, :, slot] = x
                    continue
                lo, hi = x.min(-1)[0], x.max(-1)[0]
                s = (hi - lo) / (2 ** bits - 1)
                u = torch.round((x - lo[..., None]) / torch.where(s > 0, s, torch.ones_like(s))[..., None]).to(torch.uint8)
                pools[name][page, :, slot] = u if bits == 8 else u[..., 0::2] + 16 * u[..., 1::2]
                pools["sz"][page, :, slot, 2 * c] = s.float()
                pools["sz"][page, :, slot, 2 * c + 1] = lo.float()
    if op in ("rotary", "keep"):
        got["k"], got["v"] = pools["k"], pools["v"]
        if boxes is not None:
            got["boxes"] = boxes.double()
        return got

    def whole(name, ids):
        x = pools[name][ids].transpose(0, 1)                                  # [Hkv][pages][ps][...]
        if bits == 4:
            y = torch.empty(*x.shape[:-1], d, dtype=torch.float64, device="cuda")
            y[..., 0::2], y[..., 1::2] = (x % 16).double(), (x // 16).double()
        else:
            y = x.double()
        if gran:
            sz = pools["sz"][ids].transpose(0, 1).double().repeat_interleave(gran, 2)
            y = y * sz[..., :1] + sz[..., 1:2] if name == "k" else y * sz[..., 2:3] + sz[..., 3:]
        return y.reshape(hkv, -1, d)

    seen = _masks(_parents(case)) if case["tree"] == "tree" else np.tril(np.ones((T, T), dtype=bool))[None].repeat(case["batch"], 0)
    seen = torch.from_numpy(seen).cuda()
    q = got["q"] if op == "step" else st["q"].double()
    out = torch.zeros((case["batch"], T, hkv * g, d), dtype=torch.float64, device="cuda")
    for b, (L, n) in enumerate(zip(st["lens"].tolist(), st["drafts"].tolist())):
        ids = st["table"][b, : -(-L // ps)].long()
        k, v = whole("k", ids)[:, :L], whole("v", ids)[:, :L]
        on = torch.ones((n, L), dtype=torch.bool, device="cuda")
        on[:, L - n:] = seen[b, :n, :n]
        for h in range(hkv * g):
            s = (q[b, :n, h] @ k[h // g].T / d ** 0.5).masked_fill(~on, -math.inf)
            out[b, :n, h] = torch.softmax(s, -1) @ v[h // g]
    return {"out": out}
