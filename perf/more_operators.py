"""The operators of a step with drafted tokens, and of attention over a window, measured: their plain forms beside the library's calls.

Kinds of case
  rope     per-head norms and the position rotation of a step's heads, the keys and values put into the cache in the same pass
           (kv_append_rope), and the written tokens read back (kv_gather)
  tree     attention of every request's tree of drafted tokens over its cached tokens and its own ancestors (paged_tree_attn)
  window   decode attention over the last tokens and a few first ones (paged_window_attn)
  commit   the accepted drafted tokens' rows moved to where the next step expects them, the pages that are left over
           given back (kv_tree_commit), and the kept tokens read back (kv_gather)

Caches: FP8 (e4m3 codes times the KV head's scale), BF16, or FP4 (rows of 72 bytes per token and KV head: 64 bytes of e2m1
codes, byte j holding dims 2j and 2j + 1, low nibble first, and 8 e4m3 scales, one per 16 dims; a value is code * scale *
the KV head's scale).
"""
import math

import numpy as np
import torch

own = False

D = 128
ROW = 72
DEV = "cuda"
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
BYTES = {"fp8": D, "bf16": 2 * D, "fp4": ROW}            # of a token row in the cache


# ---------------------------------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------------------------------
def listed():
    return [
        # one decode step of 64 requests, 64 query / 8 KV heads, FP8 cache
        dict(name="rope_decode_64", kind="rope", cache="fp8", tokens=64, hq=64, hkv=8, page=64, rot=128, axes=1, pairs="half", norm=True),
        # eight drafted tokens for each of 33 requests, 4-bit cache
        dict(name="rope_drafts_fp4", kind="rope", cache="fp4", tokens=264, hq=32, hkv=4, page=16, rot=64, axes=1, pairs="half", norm=False),
        # a prompt of images and text, three position axes, interleaved pairs
        dict(name="rope_prompt_bf16", kind="rope", cache="bf16", tokens=16411, hq=32, hkv=4, page=64, rot=128, axes=3, pairs="next", norm=True),
        # a handful of short requests with up to six drafted tokens, 16-token pages
        dict(name="tree_tiny", kind="tree", cache="fp8", batch=4, hq=8, hkv=2, page=16, ctx="uniform", mid=150, drafts=6, ragged=True, window=0, sinks=0, stale=0.0),
        # the headline mix, 64 requests around 16k tokens, eight drafted tokens each
        dict(name="tree_mixed_64", kind="tree", cache="fp8", batch=64, hq=64, hkv=8, page=64, ctx="lognormal", mid=16384, drafts=8, ragged=False, window=0, sinks=0, stale=0.0),
        # wide trees: most of the time goes into the products
        dict(name="tree_wide_bf16", kind="tree", cache="bf16", batch=16, hq=64, hkv=8, page=64, ctx="fixed", mid=8192, drafts=61, ragged=False, window=0, sinks=0, stale=0.0),
        # small trees over a 4-bit cache, layers with a sliding window, some requests aborted by the integrity check
        dict(name="tree_window_fp4", kind="tree", cache="fp4", batch=33, hq=32, hkv=4, page=32, ctx="lognormal", mid=16384, drafts=7, ragged=True, window=4096, sinks=4, stale=0.1),
        # the headline mix in a layer with a window of 4096 tokens
        dict(name="window_mixed_64", kind="window", cache="fp8", batch=64, hq=64, hkv=8, page=64, ctx="lognormal", mid=16384, window=4096, sinks=4, stale=0.0),
        # 256 requests over 16-token pages, a short window, 4-bit cache
        dict(name="window_page16_256", kind="window", cache="fp4", batch=256, hq=32, hkv=8, page=16, ctx="fixed", mid=4097, window=1024, sinks=16, stale=0.1),
        # a few very long requests with a wide window
        dict(name="window_long_bf16", kind="window", cache="bf16", batch=8, hq=32, hkv=4, page=64, ctx="fixed", mid=131072, window=32768, sinks=128, stale=0.0),
        # what 64 requests accept of eight drafted tokens
        dict(name="commit_64", kind="commit", cache="fp8", batch=64, hkv=8, page=64, ctx="uniform", mid=1024, drafts=8, ragged=False, stale=0.0),
        # what 256 requests accept of wide trees, 16-token pages
        dict(name="commit_wide_256", kind="commit", cache="bf16", batch=256, hkv=8, page=16, ctx="uniform", mid=256, drafts=61, ragged=True, stale=0.05),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    kind = rng.choice(("rope", "tree", "tree", "window", "window", "commit"))
    cache = rng.choice(("fp8", "fp8", "bf16", "fp4"))
    page = rng.choice((16, 32, 64, 128))
    hq, hkv = rng.choice(((8, 2), (4, 4), (32, 4), (32, 8), (64, 8), (24, 8), (32, 2), (40, 8), (24, 2)))
    if kind == "rope":
        return dict(kind=kind, cache=cache, tokens=_log(rng, 1, 2048 if cache == "fp4" else 8192), hq=hq, hkv=hkv, page=page, rot=rng.choice((32, 64, 96, 128, 128)), axes=rng.choice((1, 1, 3)),
                    pairs=rng.choice(("half", "next")), norm=rng.random() < 0.7)
    batch = _log(rng, 1, 256)
    c = dict(kind=kind, cache=cache, batch=batch)
    if kind != "commit":
        c["hq"] = hq
    c |= dict(hkv=hkv, page=page, ctx=rng.choice(("uniform", "lognormal", "fixed")), mid=_log(rng, 2, min(32768, 131072 // batch)))
    if kind != "window":
        c |= dict(drafts=_log(rng, 1, min(100, 2048 // batch)), ragged=rng.random() < 0.5)
    if kind != "commit":
        windowed = kind == "window" or rng.random() < 0.3
        c |= dict(window=_log(rng, 1, 8192) if windowed else 0, sinks=rng.choice((0, 1, 4, 4, 130)) if windowed else 0)
    c["stale"] = rng.choice((0.0, 0.0, 0.05))
    return c


# ---------------------------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------------------------
def _lengths(case, rng):
    b, mid = case["batch"], case["mid"]
    if case["ctx"] == "fixed":
        return np.full(b, mid, np.int64)
    if case["ctx"] == "uniform":
        return rng.integers(0, 2 * mid, b).astype(np.int64)
    return np.clip(np.rint(rng.lognormal(math.log(mid), 0.8, b)), max(1, mid // 32), 4 * mid).astype(np.int64)


def _drafts(case):
    """Drafted tokens per request: one number of them for the step, spread over the requests the same way for every seed."""
    b, most = case["batch"], case["drafts"]
    return np.random.default_rng(b * 1000 + most).integers(1, most + 1, b) if case["ragged"] else np.full(b, most, np.int64)


def _longest(case):
    return {"fixed": 1, "uniform": 2, "lognormal": 4}[case["ctx"]] * case["mid"]


def _t(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def _normal(gen, *shape):
    return torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32).to(torch.bfloat16)


def _pool(case, gen, pages, scale):
    """A pool of N(0, 1) values in the case's format."""
    hkv, page, kind = case["hkv"], case["page"], case["cache"]
    dtype, row = {"fp8": (torch.uint8, D), "bf16": (torch.bfloat16, D), "fp4": (torch.uint8, ROW)}[kind]
    out = torch.empty(pages, hkv, page, row, dtype=dtype, device=DEV)
    step = max(1, (1 << 27) // (hkv * page * D))
    for a in range(0, pages, step):
        x = _normal(gen, min(step, pages - a), hkv, page, D)
        out[a:a + step] = _encode(kind, x, scale.view(1, hkv, 1, 1))
    return out


def _tree(rng, n):
    """A random tree of n drafted tokens, parents first: the parent of each (-1: the last cached token)."""
    return np.array([rng.integers(max(-1, i // 2 - 2), i) if i else -1 for i in range(n)], np.int64)


def _tree_words(parents, words):
    """Each node's ancestors and itself, as bits of 64-bit words."""
    seen = []
    for i, p in enumerate(parents):
        seen.append((seen[p] if p >= 0 else 0) | (1 << i))
    return np.array([[(m >> (64 * w)) & 0xFFFFFFFFFFFFFFFF for w in range(words)] for m in seen], np.uint64)


def _accepted(rng, parents):
    """A path from the root, as long as chance has it."""
    path, at = [], -1
    while True:
        nexts = np.nonzero(parents == at)[0]
        if not len(nexts) or rng.random() < 0.15:
            return path
        at = int(rng.choice(nexts))
        path.append(at)


def prepare(case, seed):
    rng = np.random.default_rng(seed)
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    kind, hkv, page = case["kind"], case["hkv"], case["page"]
    s = dict(case)
    s["ks"], s["vs"] = (torch.rand(hkv, generator=gen, device=DEV) * 0.004 + 0.008 for _ in range(2))
    if kind == "rope":
        n, hq, half = case["tokens"], case["hq"], case["rot"] // 2
        pages = n * 5 // 4 // page + 8
        s["kc"], s["vc"] = (_pool(case, gen, pages, s[x]) for x in ("ks", "vs"))
        qkv = _normal(gen, n, (hq + 2 * hkv) * D)                     # one projection's output
        s["q"], s["k"], s["v"] = (x.unflatten(1, (-1, D)) for x in qkv.split((hq * D, hkv * D, hkv * D), 1))
        s["pos"] = _t(rng.integers(0, 131072, (case["axes"], n)).astype(np.int32))
        s["inv_freq"] = _t((500000.0 ** (-np.arange(half) / half)).astype(np.float32))
        s["axis"] = _t((np.arange(half) % case["axes"]).astype(np.uint8)) if case["axes"] > 1 else None
        s["qw"], s["kw"] = ((1 + 0.1 * _normal(gen, D).float()).to(torch.bfloat16) if case["norm"] else None for _ in range(2))
        s["slots"] = _t(rng.permutation(pages * page)[:n].astype(np.int64))
        return s
    ctx = _lengths(case, rng)
    b = case["batch"]
    n = _drafts(case) if kind != "window" else np.ones(b, np.int64)
    if kind == "window":
        ctx = np.maximum(ctx, 1) - 1
    lens = ctx + n
    pages = -(-lens // page)
    used = int(pages.sum())
    pool = used + 7 if kind != "commit" else b * -(-(_longest(case) + case["drafts"]) // page) + 7
    table = rng.permutation(pool).astype(np.int32)
    s["kc"], s["vc"] = (_pool(case, gen, pool, s[x]) for x in ("ks", "vs"))
    s["indptr"], s["indices"] = _t(np.concatenate([[0], np.cumsum(pages)]).astype(np.int32)), _t(table[:used])
    s["lens"] = _t(lens.astype(np.int32))
    s["abort"] = _t((rng.random(b) < case["stale"]).astype(np.uint8))
    s["most"] = int(n.max())                                          # rows of the widest request
    if kind != "window":
        trees = [_tree(rng, int(k)) for k in n]
        s["qptr"] = _t(np.concatenate([[0], np.cumsum(n)]).astype(np.int32))
    if kind != "commit":
        s["q"] = _normal(gen, int(n.sum()), case["hq"], D)
        lo = np.maximum(ctx - case["window"] + 1, 0) if case["window"] else np.zeros(b, np.int64)
        s["tiles"] = int((-(-(np.minimum(case["sinks"], lo) + lens - lo) // 64)).sum())
    if kind == "tree":
        words = -(-int(case["drafts"]) // 64)
        s["mask"] = _t(np.concatenate([_tree_words(t, words) for t in trees]).view(np.int64))
    if kind == "commit":
        paths = [_accepted(rng, t) for t in trees]
        acc = np.full((b, s["most"]), -1, np.int32)
        for r, p in enumerate(paths):
            acc[r, :len(p)] = p
        count = np.array([len(p) for p in paths], np.int64)
        s["accepted"], s["count"] = _t(acc), _t(count.astype(np.int32))
        s["kept"] = _t(lens.astype(np.int32))                        # the lengths kept for the next step, as the step's tables left them
        s["free"] = _t(np.concatenate([table[used:], np.full(used, -1, np.int32)]))
        s["free_count"] = _t(np.array([pool - used], np.int32))
        s["tags"] = _t(rng.integers(0, 2 ** 31, pool).astype(np.int32))
        first = np.concatenate([[0], np.cumsum(pages)])
        at = np.full((b, s["most"]), -1, np.int64)                    # the kept tokens' slots; -1: none
        for r, (c, k) in enumerate(zip(ctx, count)):
            t = c + np.arange(k)
            at[r, :k] = table[first[r] + t // page].astype(np.int64) * page + t % page
        s["at"] = _t(at.flatten())
    return s


# ---------------------------------------------------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------------------------------------------------
def _encode(kind, x, g):
    """Values [..., 128] as rows of the cache; g: the KV head's scale, broadcast against [..., 1]."""
    if kind == "bf16":
        return x.to(torch.bfloat16)
    x = x.float()
    if kind == "fp8":
        return (x / g).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
    x, g = x.unflatten(-1, (8, 16)), g.unsqueeze(-1)
    s = (x.abs().amax(-1, keepdim=True) / (6.0 * g)).clamp(max=448.0).to(torch.float8_e4m3fn)
    d = s.float() * g
    a = (x / d).abs()
    code = (a > 0.25).byte() + (a >= 0.75).byte() + (a > 1.25).byte() + (a >= 1.75).byte() + (a > 2.5).byte() + (a >= 3.5).byte() + (a > 5.0).byte()
    code = torch.where((d == 0) | d.isnan(), 0, code + 8 * torch.signbit(x).byte()).flatten(-2)
    return torch.cat([code[..., 0::2] + 16 * code[..., 1::2], s.view(torch.uint8).squeeze(-1)], -1)


def _decode(kind, rows, g):
    """Rows of the cache as fp32 values [..., 128]."""
    if kind == "bf16":
        return rows.float()
    if kind == "fp8":
        return rows.view(torch.float8_e4m3fn).float() * g
    code = torch.stack([rows[..., :64] & 15, rows[..., :64] >> 4], -1).flatten(-2)
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=rows.device)
    s = rows[..., 64:].contiguous().view(torch.float8_e4m3fn).float()
    return (table[code.int()].unflatten(-1, (8, 16)) * s.unsqueeze(-1)).flatten(-2) * g


def _plain_heads(x, w, cos, sin, nxt):
    """fp32 head rows [N][H][128], normed and turned; cos, sin [N][1][rot / 2]."""
    y = x.float()
    if w is not None:
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + 1e-6) * w.float()
    half = cos.shape[-1]
    a, b = (y[..., 0:2 * half:2], y[..., 1:2 * half:2]) if nxt else (y[..., :half], y[..., half:2 * half])
    p, q = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([p, q], -1).flatten(-2) if nxt else torch.cat([p, q], -1)
    return torch.cat([turned, y[..., 2 * half:]], -1)


def _plain_read(s, slots):
    live, at = (slots >= 0).view(-1, 1, 1), slots.clamp(min=0)
    page, off = at // s["page"], at % s["page"]
    return [torch.where(live, _decode(s["cache"], c[page, :, off], g.view(1, -1, 1)), 0.0).to(torch.bfloat16) for c, g in ((s["kc"], s["ks"]), (s["vc"], s["vs"]))]


def _plain_rope(s):
    pos = s["pos"].double().t() if s["axis"] is None else s["pos"].double().t()[:, s["axis"].long()]
    angle = (pos * s["inv_freq"].double()).unsqueeze(1)               # far positions' low bits
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    nxt = s["pairs"] == "next"
    q, k = _plain_heads(s["q"], s["qw"], cos, sin, nxt).to(torch.bfloat16), _plain_heads(s["k"], s["kw"], cos, sin, nxt)
    page, off = s["slots"] // s["page"], s["slots"] % s["page"]
    s["kc"][page, :, off] = _encode(s["cache"], k, s["ks"].view(1, -1, 1))
    s["vc"][page, :, off] = _encode(s["cache"], s["v"], s["vs"].view(1, -1, 1))
    return [q, *_plain_read(s, s["slots"])]


def _plain_attn(s):
    """Tiles of 64 seen tokens (the first ones and the window's, side by side), each against its request's rows; the tiles' sums
    joined per request in 64 bits."""
    q, page, nt, most, hkv = s["q"], s["page"], s["tiles"], s["most"], s["hkv"]
    lens, b = s["lens"].long(), s["lens"].numel()
    n_rows, hq = q.shape[:2]
    group = hq // hkv
    zero = torch.zeros(1, dtype=torch.int64, device=DEV)
    qptr = s["qptr"].long() if "qptr" in s else torch.arange(b + 1, device=DEV)
    n = qptr[1:] - qptr[:-1]
    ctx = lens - n
    node = torch.arange(most, device=DEV)
    row = (qptr[:-1].unsqueeze(1) + node).clamp(max=n_rows - 1)                                                   # [b][most]
    there = node < n.unsqueeze(1)
    bit = torch.arange(64, device=DEV)
    bits = ((s["mask"].unsqueeze(2) >> bit) & 1).flatten(1).bool() if "mask" in s else torch.ones(n_rows, 1, dtype=torch.bool, device=DEV)
    depth = (bits.sum(1) - 1).clamp(min=0)
    lo = (ctx - s["window"] + 1).clamp(min=0) if s["window"] else torch.zeros_like(ctx)
    head = lo.clamp(max=s["sinks"])
    first = torch.cat([zero, ((head + lens - lo + 63) // 64).cumsum(0)])
    tile = torch.arange(nt, device=DEV)
    r = (torch.searchsorted(first, tile, right=True) - 1).clamp(max=b - 1)
    at = (tile - first[r]).unsqueeze(1) * 64 + bit
    pos = torch.where(at < head[r].unsqueeze(1), at, at - (head - lo)[r].unsqueeze(1))                            # [nt][64]
    entry = (s["indptr"].long()[r].unsqueeze(1) + pos // page).clamp(max=s["indices"].numel() - 1)
    pg, off = s["indices"].long()[entry], pos % page
    qp = q.float()[row].unflatten(2, (hkv, group)).transpose(1, 2).flatten(2, 3)                                  # [b][hkv][most * group][128]
    z = torch.empty(nt, hkv, most * group, 64, device=DEV)
    top = torch.full((b, hkv, most * group), -math.inf, device=DEV)
    num = torch.zeros(b, hkv, most * group, D, dtype=torch.float64, device=DEV)
    den = torch.zeros(b, hkv, most * group, dtype=torch.float64, device=DEV)
    step = max(1, (1 << 29) // (hkv * D * max(64, most * group)))
    parts = [slice(a, min(nt, a + step)) for a in range(0, nt, step)]
    for p in parts:
        i, t = r[p], pos[p]
        k = _decode(s["cache"], s["kc"][pg[p], :, off[p]], s["ks"].view(1, 1, -1, 1)).transpose(1, 2)             # [tiles][hkv][64][128]
        j = t - ctx[i].unsqueeze(1)                                                                               # which drafted token
        drawn = bits[row[i].unsqueeze(2), j.clamp(0, bits.shape[1] - 1).unsqueeze(1)]                             # [tiles][most][64]
        far = (ctx[i].unsqueeze(1) + depth[row[i]]).unsqueeze(2) - t.unsqueeze(1)                                 # how far back
        near = (far < s["window"]) | (t < s["sinks"]).unsqueeze(1) if s["window"] else torch.ones_like(drawn)
        see = torch.where((j >= 0).unsqueeze(1), drawn, near) & (t < lens[i].unsqueeze(1)).unsqueeze(1) & there[i].unsqueeze(2)
        see = see.unsqueeze(2).expand(-1, -1, group, -1).flatten(1, 2).unsqueeze(1)                               # [tiles][1][most * group][64]
        z[p] = ((qp[i] @ k.transpose(2, 3)) / math.sqrt(D)).masked_fill(~see, -math.inf)
        top.index_reduce_(0, i, z[p].amax(-1), "amax")
    top = torch.where(top == -math.inf, 0.0, top)
    for p in parts:
        w = torch.exp(z[p] - top[r[p]].unsqueeze(-1))
        v = _decode(s["cache"], s["vc"][pg[p], :, off[p]], s["vs"].view(1, 1, -1, 1)).transpose(1, 2)
        num.index_add_(0, r[p], (w @ v).double())
        den.index_add_(0, r[p], w.sum(-1).double())
    out = torch.where(den.unsqueeze(-1) > 0, num / den.unsqueeze(-1), 0.0).unflatten(2, (most, group)).transpose(1, 2).flatten(2, 3)
    out = torch.where((s["abort"] == 0).view(-1, 1, 1, 1), out, 0.0)
    return out[there].to(torch.bfloat16)


def _plain_commit(s):
    page, lens, b, most = s["page"], s["lens"].long(), s["lens"].numel(), s["accepted"].shape[1]
    qptr, ptr, idx = s["qptr"].long(), s["indptr"].long(), s["indices"].long()
    ctx = lens - (qptr[1:] - qptr[:-1])
    live = s["abort"] == 0
    count = torch.where(live, s["count"].long(), 0)
    i = torch.arange(most, device=DEV)
    moved = i < count.unsqueeze(1)
    slot = lambda t: idx[(ptr[:-1].unsqueeze(1) + t // page).clamp(max=idx.numel() - 1)] * page + t % page  # noqa: E731
    src, dst = (slot(t)[moved] for t in (ctx.unsqueeze(1) + s["accepted"].long().clamp(min=0), ctx.unsqueeze(1) + i))
    for c in (s["kc"], s["vc"]):
        c[dst // page, :, dst % page] = c[src // page, :, src % page]
    kept = torch.where(live, ctx + count, s["kept"].long())
    # the pages past the kept length, given back so that the next step takes them in the order in which this one did
    pages, keep = (lens + page - 1) // page, (kept + page - 1) // page
    back = torch.where(live, pages - keep, 0)
    last = torch.cat([torch.zeros(1, dtype=torch.int64, device=DEV), back.cumsum(0)])
    k = torch.arange(s["indices"].numel(), device=DEV)
    r = (torch.searchsorted(ptr, k, right=True) - 1).clamp(max=b - 1)
    nth = k - ptr[r] - keep[r]
    goes = (nth >= 0) & (nth < back[r])
    have = s["free_count"].long()
    s["kept"].copy_(kept)
    s["free"][(have + last[-1] - 1 - last[r] - nth)[goes]] = idx[goes].int()
    s["tags"][idx[goes]] += 1
    k, v = _plain_read(s, s["at"])
    return dict(kept=s["kept"], free=s["free"], free_left=(have + last[-1]).int(), tags=s["tags"], k=k, v=v)


# ---------------------------------------------------------------------------------------------------------------------
# the library's calls
# ---------------------------------------------------------------------------------------------------------------------
def _own_read(fkv, s, slots):
    if "kb" not in s:
        s["kb"], s["vb"] = (torch.empty(slots.numel(), s["hkv"], D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    fkv.kv_gather(s["kc"], s["vc"], slots, s["kb"], s["vb"], k_scale=s["ks"], v_scale=s["vs"])
    return [s["kb"], s["vb"]]


def _own_rope(fkv, s):
    if "qo" not in s:
        s["qo"] = torch.empty(s["q"].shape, dtype=torch.bfloat16, device=DEV)
    fkv.kv_append_rope(s["q"], s["k"], s["v"], s["pos"], s["inv_freq"], s["slots"], s["qo"], s["kc"], s["vc"], k_scale=s["ks"], v_scale=s["vs"],
                       q_weight=s["qw"], k_weight=s["kw"], eps=1e-6, axis_map=s["axis"], interleaved=s["pairs"] == "next")
    return [s["qo"], *_own_read(fkv, s, s["slots"])]


def _own_attn(fkv, s):
    q = s["q"]
    if "ws" not in s:
        kv = {"fp8": fkv.KV_FP8_E4M3, "bf16": fkv.KV_BF16, "fp4": fkv.KV_FP4}[s["cache"]]
        s["ws"] = fkv.alloc_tree_workspace(q.shape[0], s["batch"], s["hq"], s["hkv"], kv)
        s["out"] = torch.empty_like(q)
    args = dict(k_scale=s["ks"], v_scale=s["vs"], abort_mask=s["abort"], window=s["window"], sinks=s["sinks"])
    if s["kind"] == "tree":
        return fkv.paged_tree_attn(q, s["kc"], s["vc"], s["indptr"], s["indices"], s["lens"], s["qptr"], s["mask"], 1.0 / math.sqrt(D), s["out"], s["ws"], **args)
    return fkv.paged_window_attn(q, s["kc"], s["vc"], s["indptr"], s["indices"], s["lens"], 1.0 / math.sqrt(D), s["out"], s["ws"], **args)


def _own_commit(fkv, s):
    if "left" not in s:
        s["left"] = torch.empty(1, dtype=torch.int32, device=DEV)
    fkv.kv_tree_commit(s["kc"], s["vc"], s["indptr"], s["indices"], s["lens"], s["qptr"], s["accepted"], s["count"], s["kept"], abort_mask=s["abort"],
                       free_pages=s["free"], free_count=s["free_count"], free_left=s["left"], page_tags=s["tags"])
    k, v = _own_read(fkv, s, s["at"])
    return dict(kept=s["kept"], free=s["free"], free_left=s["left"], tags=s["tags"], k=k, v=v)


def run(s):
    if own:
        import fp8_paged_kv_decode_gb300 as fkv
        return {"rope": _own_rope, "commit": _own_commit}.get(s["kind"], _own_attn)(fkv, s)
    return {"rope": _plain_rope, "commit": _plain_commit}.get(s["kind"], _plain_attn)(s)


# ---------------------------------------------------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------------------------------------------------
def work(case):
    kind, hkv = case["kind"], case["hkv"]
    token = hkv * 2 * BYTES[case["cache"]]                            # a token's K and V in the cache
    if kind == "rope":
        n = case["tokens"]
        written = n * ((case["hq"] + 2 * hkv) * 2 * D + case["hq"] * 2 * D + token + 8 + 4 * case["axes"])
        return {"bytes": written + n * (token + hkv * 4 * D + 8), "flops": n * (case["hq"] + 2 * hkv) * 10 * D}
    rng = np.random.default_rng(0)                                    # lengths as the case has them on the average
    ctx = _lengths(case, rng).astype(np.float64)
    live = 1 - case["stale"]
    if kind == "commit":
        moved = live * sum(len(_accepted(rng, _tree(rng, int(n)))) for n in _drafts(case))
        return {"bytes": moved * (3 * token + hkv * 4 * D + 12) + case["batch"] * 40, "flops": 0}
    n = np.ones(case["batch"]) if kind == "window" else _drafts(case).astype(np.float64)
    seen = np.minimum(ctx, case["window"] + case["sinks"]) if case["window"] else ctx
    seen = seen + n * (kind == "tree")
    return {"bytes": live * float(seen.sum()) * token + float(n.sum()) * case["hq"] * D * 4, "flops": live * float((seen * n).sum()) * case["hq"] * D * 4}


# ---------------------------------------------------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------------------------------------------------
def _grid8():
    """The magnitudes of e4m3 in order: three mantissa bits, four exponent bits, bias 7, the last pattern left out."""
    c = torch.arange(127, device=DEV)
    e, m = c // 8, (c % 8).double()
    return torch.where(e == 0, m * 2.0 ** -9, torch.exp2((e - 7).double()) * (1 + m / 8))


def _nearest(x, grid):
    """The grid's nearest magnitude to |x|, with x's sign; ties to the even place, the largest where x is beyond it."""
    a = x.abs().clamp(max=float(grid[-1]))
    hi = torch.searchsorted(grid, a).clamp(1, grid.numel() - 1)
    down, up = a - grid[hi - 1], grid[hi] - a
    pick = torch.where(up < down, hi, torch.where(up > down, hi - 1, hi - hi % 2))
    return torch.where(x < 0, -grid[pick], grid[pick])


def _exact_held(kind, x, g):
    """What the cache holds of 64-bit values [n][hkv][128]."""
    if kind == "bf16":
        return x
    g = g.double().view(1, -1, 1)
    if kind == "fp8":
        return _nearest(x / g, _grid8()) * g
    x, g = x.unflatten(2, (8, 16)), g.unsqueeze(-1)
    s = _nearest(x.abs().amax(-1, keepdim=True) / (6 * g), _grid8())
    held = _nearest(torch.where(s > 0, x / (s * g), 0.0), torch.tensor(E2M1, dtype=torch.float64, device=DEV)) * s * g
    return held.flatten(2)


def _exact_rows(kind, rows, g):
    """64-bit values of rows of the cache (n rows of one KV head)."""
    if kind == "bf16":
        return rows.double()
    grid = torch.cat([_grid8(), torch.full((1,), math.nan, dtype=torch.float64, device=DEV)])
    sign = lambda c: 1.0 - 2.0 * (c >= 128)  # noqa: E731
    if kind == "fp8":
        c = rows.long()
        return grid[c % 128] * sign(c) * g.double()
    c = rows[:, :64].long()
    e2m1 = torch.tensor(E2M1, dtype=torch.float64, device=DEV)
    out = torch.empty(rows.shape[0], D, dtype=torch.float64, device=DEV)
    for k, nibble in enumerate((c % 16, c // 16)):
        out[:, k::2] = e2m1[nibble % 8] * torch.where(nibble >= 8, -1.0, 1.0)
    c = rows[:, 64:].long()
    return out * (grid[c % 128] * sign(c)).repeat_interleave(16, 1) * g.double()


def _exact_rope(s):
    turned = []
    for x, w in ((s["q"], s["qw"]), (s["k"], s["kw"])):
        y = x.double()
        if w is not None:
            y = y / torch.sqrt((y ** 2).mean(-1, keepdim=True) + 1e-6) * w.double()
        half, out = s["rot"] // 2, y.clone()
        for j in range(half):
            t = s["pos"][0 if s["axis"] is None else int(s["axis"][j])].double() * s["inv_freq"][j].double()
            c, n = torch.cos(t).unsqueeze(1), torch.sin(t).unsqueeze(1)
            a, b = (2 * j, 2 * j + 1) if s["pairs"] == "next" else (j, half + j)
            out[..., a], out[..., b] = y[..., a] * c - y[..., b] * n, y[..., a] * n + y[..., b] * c
        turned.append(out)
    return [turned[0], _exact_held(s["cache"], turned[1], s["ks"]), _exact_held(s["cache"], s["v"].double(), s["vs"])]


def _exact_attn(s):
    q, page, hkv = s["q"], s["page"], s["hkv"]
    group = q.shape[1] // hkv
    out = torch.zeros(q.shape, dtype=torch.float64, device=DEV)
    lens, ptr = s["lens"].tolist(), s["indptr"].tolist()
    qptr = s["qptr"].tolist() if "qptr" in s else list(range(len(lens) + 1))
    masks = s["mask"].cpu().numpy().view(np.uint64) if "mask" in s else np.ones((q.shape[0], 1), np.uint64)
    for r, length in enumerate(lens):
        if s["abort"][r]:
            continue
        n = qptr[r + 1] - qptr[r]
        c = length - n
        see = torch.ones(n, length, dtype=torch.bool)
        for i in range(n):
            word = sum(int(w) << (64 * k) for k, w in enumerate(masks[qptr[r] + i]))
            see[i, c:] = torch.tensor([bool((word >> j) & 1) for j in range(n)])
            if s["window"]:
                at = c + max(bin(word).count("1") - 1, 0)
                see[i, min(s["sinks"], c):min(c, max(at - s["window"] + 1, min(s["sinks"], c)))] = False
        some = see.any(0).nonzero().squeeze(1).to(DEV)
        see = see.to(DEV)[:, some]
        pages = s["indices"][ptr[r]:ptr[r + 1]].long()[some // page]
        for h in range(hkv):
            k, v = (_exact_rows(s["cache"], x[pages, h, some % page], g[h]) for x, g in ((s["kc"], s["ks"]), (s["vc"], s["vs"])))
            for i in range(group):
                z = (q[qptr[r]:qptr[r + 1], h * group + i].double() @ k.t()) / math.sqrt(D)
                w = torch.softmax(z.masked_fill(~see, -math.inf), -1)
                out[qptr[r]:qptr[r + 1], h * group + i] = torch.where(see.any(1, keepdim=True), w @ v, 0.0)
    return out


def _exact_commit(s):
    """The kept tokens' values, read where the drafted ones lie."""
    page, ptr, idx = s["page"], s["indptr"].tolist(), s["indices"].tolist()
    lens, qptr, count, acc = (s[x].tolist() for x in ("lens", "qptr", "count", "accepted"))
    dead = s["abort"].tolist()
    at, to = [], []
    for r, length in enumerate(lens):
        c = length - (qptr[r + 1] - qptr[r])
        for i in range(count[r]):
            t = c + (i if dead[r] else acc[r][i])
            at.append(idx[ptr[r] + t // page] * page + t % page)
            to.append(r * s["most"] + i)
    at, to = (torch.tensor(x, dtype=torch.int64, device=DEV) for x in (at, to))
    values = [torch.zeros(s["at"].numel(), s["hkv"], D, dtype=torch.float64, device=DEV) for _ in range(2)]
    for v, x, g in zip(values, (s["kc"], s["vc"]), (s["ks"], s["vs"])):
        v[to] = torch.stack([_exact_rows(s["cache"], x[at // page, h, at % page], g[h]) for h in range(s["hkv"])], 1)
    return dict(kept=None, free=None, free_left=None, tags=None, k=values[0], v=values[1])


def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _exact_rope, "commit": _exact_commit}.get(case["kind"], _exact_attn)(s)
