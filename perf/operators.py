"""The operators of a decode step over a 4-bit cache, measured: their plain forms beside the library's calls.

Kinds of case
  tables   page tables, slots and positions of a step made on the GPU from request lengths (kv_step_tables)
  rope     per-head norms of q and k with the position rotation in the same pass (qk_norm_rope)
  write    new tokens written into the 4-bit cache, then cached tokens read back as bf16 (kv_append_fp4, kv_gather)
  read     cached tokens of an FP8, BF16 or 4-bit cache read back as bf16 (kv_gather)
  attn     decode attention over the 4-bit cache (paged_decode_attn)
  step     all of them in a row, as one decode step of a layer calls them

The 4-bit cache: a row of 72 bytes per (token, KV head), 64 bytes of e2m1 codes (byte j holds dims 2j and 2j + 1, low
nibble first) and 8 e4m3 scales, one per 16 dims; a value is code * scale * (the KV head's fp32 scale).
"""
import math

import numpy as np
import torch

own = False

D = 128
ROW = 72
DEV = "cuda"
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---------------------------------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------------------------------
def listed():
    return [
        # the headline batch's tables: 64 requests around 16k tokens, one new token each
        dict(name="tables_decode_64", kind="tables", batch=64, page=64, ctx="lognormal", mid=16384, new=1),
        # a mixed step of many requests with prompt chunks, 16-token pages
        dict(name="tables_chunks_256", kind="tables", batch=256, page=16, ctx="uniform", mid=4096, new=2048),
        # one decode step of 64 requests, 64 query / 8 KV heads, one position axis
        dict(name="rope_decode_64", kind="rope", tokens=64, hq=64, hkv=8, rot=128, axes=1, pairs="half", norm=True, fused=True),
        # a prompt of images and text, three position axes, interleaved pairs
        dict(name="rope_prompt_3axes", kind="rope", tokens=16411, hq=32, hkv=4, rot=128, axes=3, pairs="next", norm=True, fused=False),
        # a decode step's tokens of 256 requests into the 4-bit cache
        dict(name="write_decode_256", kind="write", tokens=256, hkv=8, page=16, pool=4096, back=256),
        # a whole prompt batch (32 x 8192) into the 4-bit cache and back out of it
        dict(name="write_prompt_262k", kind="write", tokens=262144, hkv=8, page=64, pool=5120, back=262144),
        # a cached prefix of one 131072-token request read out of an FP8 cache for a prompt's next chunk
        dict(name="read_prefix_fp8", kind="read", cache="fp8", tokens=131072, hkv=4, page=64, pool=2560),
        # a handful of short requests, 16-token pages
        dict(name="attn_tiny", kind="attn", batch=4, hq=8, hkv=2, page=16, ctx="uniform", mid=150, stale=0.0),
        # 32 requests of 8192 tokens, 64 query / 8 KV heads
        dict(name="attn_uniform_8k", kind="attn", batch=32, hq=64, hkv=8, page=64, ctx="fixed", mid=8193, stale=0.0),
        # 64 requests of mixed lengths around 16k tokens, the headline mix
        dict(name="attn_mixed_64", kind="attn", batch=64, hq=64, hkv=8, page=64, ctx="lognormal", mid=16384, stale=0.0),
        # 256 requests over 16-token pages, some of them aborted by the integrity check
        dict(name="attn_page16_256", kind="attn", batch=256, hq=32, hkv=8, page=16, ctx="fixed", mid=4097, stale=0.1),
        # a whole step of 33 requests, from lengths to attention
        dict(name="step_33", kind="step", batch=33, hq=32, hkv=4, page=32, ctx="lognormal", mid=4096),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(("tables", "rope", "write", "read", "attn", "attn", "step"))
    page = rng.choice((16, 32, 64, 128))
    hq, hkv = rng.choice(((8, 2), (4, 4), (32, 4), (32, 8), (64, 8), (24, 8), (32, 2)))
    if kind == "tables":
        batch = _log(rng, 1, 512)
        new = rng.choice((1, _log(rng, 2, 2048)))
        return dict(kind=kind, batch=batch, page=page, ctx=rng.choice(("uniform", "lognormal", "fixed")), mid=_log(rng, 16, max(17, 1000000 // batch // 2)), new=min(new, max(1, 400000 // batch)))
    if kind == "rope":
        return dict(kind=kind, tokens=_log(rng, 1, 8192), hq=hq, hkv=hkv, rot=rng.choice((32, 64, 96, 128, 128)), axes=rng.choice((1, 3)), pairs=rng.choice(("half", "next")), norm=rng.random() < 0.8, fused=rng.random() < 0.5)
    if kind == "write":
        tokens = _log(rng, 1, 131072)
        pool = tokens * 5 // 4 // page + 8
        return dict(kind=kind, tokens=tokens, hkv=hkv, page=page, pool=pool, back=_log(rng, 1, pool * page))
    if kind == "read":
        tokens = _log(rng, 1, 65536)
        return dict(kind=kind, cache=rng.choice(("fp8", "bf16", "fp4")), tokens=tokens, hkv=hkv, page=page, pool=tokens // page + _log(rng, 1, 512))
    batch = _log(rng, 1, 256)
    c = dict(kind=kind, batch=batch, hq=hq, hkv=hkv, page=page, ctx=rng.choice(("uniform", "lognormal", "fixed")), mid=_log(rng, 2, min(65536, 262144 // batch)))
    if kind == "attn":
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
        return rng.integers(1, 2 * mid, b).astype(np.int64)
    return np.clip(np.rint(rng.lognormal(math.log(mid), 0.8, b)), max(1, mid // 32), 4 * mid).astype(np.int64)


def _longest(case):
    return {"fixed": 1, "uniform": 2, "lognormal": 4}[case["ctx"]] * case["mid"]


def _t(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def _normal(gen, *shape):
    return torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32).to(torch.bfloat16)


def _fill_fp4(gen, pool, hkv, page, scale):
    """A pool of rows drawn from N(0, 1), as the 4-bit write leaves them."""
    out = torch.empty(pool, hkv, page, ROW, dtype=torch.uint8, device=DEV)
    step = max(1, (1 << 26) // (hkv * page * D))
    for a in range(0, pool, step):
        x = _normal(gen, min(step, pool - a), hkv, page, D)
        out[a:a + step] = _encode_fp4(x, scale.view(1, hkv, 1, 1))
    return out


def _tables_case(case, rng):
    b, s = case["batch"], case["page"]
    cached = np.maximum(_lengths(case, rng) - 1, 0)
    new = np.ones(b, np.int64) if case["new"] == 1 else rng.integers(0, case["new"] + 1, b)
    have = -(-cached // s)
    pages = -(-(cached + new) // s)
    blocks = -(-(_longest(case) + case["new"]) // s)           # what a step of these requests may need at most
    pool = int(pages.sum()) + 64
    perm = rng.permutation(pool).astype(np.int32)
    used = int(have.sum())
    table = np.full((b, blocks), -1, np.int32)
    tags_of = np.zeros((b, blocks), np.int64)
    tags = rng.integers(0, 2 ** 31, pool)
    at = 0
    for r in range(b):
        n = int(have[r])
        table[r, :n] = perm[at:at + n]
        tags_of[r, :n] = tags[perm[at:at + n]]
        at += n
    free = perm[used:]
    return dict(cached=_t(cached.astype(np.int32)), new=_t(new.astype(np.int32)), table=_t(table), table_tags=_t(tags_of.astype(np.int32)),
                free=_t(free), free_count=_t(np.array([free.size], np.int32)), tags=_t(tags.astype(np.int32)), page=s, pool=pool,
                nnz=b * blocks, tokens=b * case["new"] + 3)


def _rope_case(case, rng, gen):
    n, hq, hkv = case["tokens"], case["hq"], case["hkv"]
    half = case["rot"] // 2
    if case["fused"]:                          # q and k as parts of one projection's output
        qkv = _normal(gen, n, (hq + 2 * hkv) * D)
        q, k = qkv[:, :hq * D].unflatten(1, (hq, D)), qkv[:, hq * D:(hq + hkv) * D].unflatten(1, (hkv, D))
    else:
        q, k = _normal(gen, n, hq, D), _normal(gen, n, hkv, D)
    pos = rng.integers(0, 131072, (case["axes"], n)).astype(np.int32)
    return dict(q=q, k=k, pos=_t(pos), inv_freq=_t((500000.0 ** (-np.arange(half) / half)).astype(np.float32)),
                axis=_t((np.arange(half) % case["axes"]).astype(np.uint8)) if case["axes"] > 1 else None,
                qw=(1 + 0.1 * _normal(gen, D).float()).to(torch.bfloat16) if case["norm"] else None,
                kw=(1 + 0.1 * _normal(gen, D).float()).to(torch.bfloat16) if case["norm"] else None,
                eps=1e-6, next=case["pairs"] == "next", rot_scale=1.0)


def prepare(case, seed):
    rng = np.random.default_rng(seed)
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    kind = case["kind"]
    s = dict(case)
    if kind == "tables":
        s |= _tables_case(case, rng)
    elif kind == "rope":
        s |= _rope_case(case, rng, gen)
    elif kind in ("write", "read"):
        hkv, page, pool, n = case["hkv"], case["page"], case["pool"], case["tokens"]
        s["ks"], s["vs"] = (torch.rand(hkv, generator=gen, device=DEV) * 0.004 + 0.008 for _ in range(2))
        cache = case.get("cache", "fp4")
        if cache == "fp4":
            s["kc"], s["vc"] = (_fill_fp4(gen, pool, hkv, page, s[x]) for x in ("ks", "vs"))
        elif cache == "fp8":
            s["kc"], s["vc"] = ((_normal(gen, pool, hkv, page, D).float() / 0.01).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8) for _ in range(2))
        else:
            s["kc"], s["vc"] = (_normal(gen, pool, hkv, page, D) for _ in range(2))
        if kind == "write":
            s["k"], s["v"] = _normal(gen, n, hkv, D), _normal(gen, n, hkv, D)
            s["slots"] = _t(rng.permutation(pool * page)[:n].astype(np.int64))
            s["from"] = _t(rng.permutation(pool * page)[:case["back"]].astype(np.int64))
        else:
            pages = rng.permutation(pool)[:-(-n // page)].astype(np.int64)
            at = np.arange(n)
            s["from"] = _t(pages[at // page] * page + at % page)
    elif kind == "attn":
        b, hkv, page = case["batch"], case["hkv"], case["page"]
        lens = _lengths(case, rng)
        pages = -(-lens // page)
        used = int(pages.sum())
        s["ks"], s["vs"] = (torch.rand(hkv, generator=gen, device=DEV) * 0.004 + 0.008 for _ in range(2))
        s["kc"], s["vc"] = (_fill_fp4(gen, used + 7, hkv, page, s[x]) for x in ("ks", "vs"))
        s["q"] = _normal(gen, b, case["hq"], D)
        s["indptr"] = _t(np.concatenate([[0], np.cumsum(pages)]).astype(np.int32))
        s["indices"] = _t(rng.permutation(used + 7)[:used].astype(np.int32))
        s["lens"] = _t(lens.astype(np.int32))
        s["abort"] = _t((rng.random(b) < case["stale"]).astype(np.uint8))
        s["tiles"] = int((-(-lens // 64)).sum())
    else:
        s |= _tables_case(dict(case, new=1), rng)
        s |= _rope_case(dict(tokens=s["tokens"], hq=case["hq"], hkv=case["hkv"], rot=128, axes=1, pairs="half", norm=True, fused=False), rng, gen)
        hkv = case["hkv"]
        s["v"] = _normal(gen, s["tokens"], hkv, D)
        s["ks"], s["vs"] = (torch.rand(hkv, generator=gen, device=DEV) * 0.004 + 0.008 for _ in range(2))
        s["kc"], s["vc"] = (_fill_fp4(gen, s["pool"], hkv, case["page"], s[x]) for x in ("ks", "vs"))
        lens = s["cached"].cpu().numpy().astype(np.int64) + 1
        s["tiles"] = int((-(-lens // 64)).sum())
    return s


# ---------------------------------------------------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------------------------------------------------
def _encode_fp4(x, g):
    """bf16 [..., 128] to rows of 72 bytes; g: the KV head's scale, broadcast against [..., 1]."""
    x = x.float().unflatten(-1, (8, 16))
    g = g.unsqueeze(-1)
    six = torch.full_like(g, 6.0)
    s = (x.abs().amax(-1, keepdim=True) / (six * g)).clamp(max=448.0).to(torch.float8_e4m3fn)
    d = s.float() * g
    a = (x / d).abs()
    code = (a > 0.25).byte() + (a >= 0.75).byte() + (a > 1.25).byte() + (a >= 1.75).byte() + (a > 2.5).byte() + (a >= 3.5).byte() + (a > 5.0).byte()
    code = torch.where((d == 0) | d.isnan(), 0, code + 8 * torch.signbit(x).byte()).flatten(-2)
    return torch.cat([code[..., 0::2] + 16 * code[..., 1::2], s.view(torch.uint8).squeeze(-1)], -1)


def _decode_fp4(rows, g):
    """Rows of 72 bytes as fp32 values [..., 128]."""
    code = torch.stack([rows[..., :64] & 15, rows[..., :64] >> 4], -1).flatten(-2)
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=rows.device)
    s = rows[..., 64:].contiguous().view(torch.float8_e4m3fn).float()
    return (table[code.int()].unflatten(-1, (8, 16)) * s.unsqueeze(-1)).flatten(-2) * g


def _plain_tables(s):
    page, nnz, n_tok, pool = s["page"], s["nnz"], s["tokens"], s["pool"]
    c, n = s["cached"].long(), s["new"].long()
    blocks = s["table"].shape[1]
    have, pages = (c + page - 1) // page, (c + n + page - 1) // page
    ok = (c >= 0) & (n >= 0) & (pages <= blocks)
    zero = torch.zeros(1, dtype=torch.int64, device=DEV)
    rows = torch.cat([zero, torch.where(ok, pages, 0).cumsum(0)])
    toks = torch.cat([zero, n.clamp(min=0).cumsum(0)])
    ok = ok & (toks[1:] <= n_tok) & (rows[1:] <= nnz)
    need = torch.where(ok, pages - have, 0)
    taken = torch.cat([zero, need.cumsum(0)])
    free = s["free_count"].long()
    ok = ok & ((need == 0) | (taken[1:] <= free))
    # page table entries
    j = torch.arange(nnz, device=DEV)
    r = (torch.searchsorted(rows, j, right=True) - 1).clamp(max=c.numel() - 1)
    col = j - rows[r]
    inside = j < rows[-1]
    top = free - 1 - taken[:-1]
    fresh = s["free"][(top[r] - (col - have[r])).clamp(0, s["free"].numel() - 1)].long()
    old = s["table"][r, col.clamp(0, blocks - 1)].long()
    is_new = col >= have[r]
    idx = torch.where(is_new, torch.where(ok[r], fresh, -1), old)
    tag = torch.where(is_new, torch.where(ok[r], s["tags"][idx.clamp(0, pool - 1)], 0), s["table_tags"][r, col.clamp(0, blocks - 1)])
    put = inside & is_new & ok[r]
    cell = torch.where(put, r * blocks + col, c.numel() * blocks)                               # one cell more, for the entries that stay
    table, table_tags = (torch.cat([x.flatten(), x.new_zeros(1)]).index_put_((cell,), y)[:-1].view(-1, blocks) for x, y in ((s["table"], idx.int()), (s["table_tags"], tag)))
    idx, tag = torch.where(inside, idx, 0), torch.where(inside, tag, 0)
    # tokens
    i = torch.arange(n_tok, device=DEV)
    q = (torch.searchsorted(toks, i, right=True) - 1).clamp(max=c.numel() - 1)
    pos = c[q] + i - toks[q]
    live = i < toks[-1]
    pg = torch.where(live, table[q, (pos // page).clamp(0, blocks - 1)].long(), -1)
    slot = torch.where(live & ok[q], pg * page + pos % page, -1)
    used = torch.where(ok, need, 0).sum()
    return dict(step_lens=torch.where(ok, c + n, 0).int(), cached_out=torch.where(ok, c + n, c).int(), refused=(~ok).byte(), indptr=rows.clamp(max=nnz).int(),
                indices=idx.int(), expected=tag, token_indptr=toks.clamp(max=n_tok).int(), slots=slot, positions=torch.where(live, pos, 0).int(),
                free_left=(free - used).int(), table=table, table_tags=table_tags)


def _plain_rope_one(x, w, cos, sin, eps, nxt):
    """fp32 rows [N][H][128]; cos, sin [N][1][rot / 2]."""
    y = x.float()
    if w is not None:
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + eps) * w.float()
    half = cos.shape[-1]
    a, b = (y[..., 0:2 * half:2], y[..., 1:2 * half:2]) if nxt else (y[..., :half], y[..., half:2 * half])
    p, q = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([p, q], -1).flatten(-2) if nxt else torch.cat([p, q], -1)
    return torch.cat([turned, y[..., 2 * half:]], -1).to(torch.bfloat16)


def _plain_rope(s, pos):
    pos = pos.double().t() if s["axis"] is None else pos.double().t()[:, s["axis"].long()]
    angle = (pos * s["inv_freq"].double()).unsqueeze(1)
    cos, sin = ((f(angle) * s["rot_scale"]).float() for f in (torch.cos, torch.sin))
    return _plain_rope_one(s["q"], s["qw"], cos, sin, s["eps"], s["next"]), _plain_rope_one(s["k"], s["kw"], cos, sin, s["eps"], s["next"])


def _plain_write(s, k, v, slots):
    """The new tokens' rows put into the caches; a negative slot writes nothing."""
    g = (slots >= 0).nonzero().squeeze(1) if s["kind"] == "step" else slice(None)
    at = slots[g]
    page, off = at // s["page"], at % s["page"]
    s["kc"][page, :, off] = _encode_fp4(k[g], s["ks"].view(1, -1, 1))
    s["vc"][page, :, off] = _encode_fp4(v[g], s["vs"].view(1, -1, 1))


def _plain_read(s, cache, slots):
    live = (slots >= 0).view(-1, 1, 1)
    at = slots.clamp(min=0)
    got = []
    for c, g in ((s["kc"], s["ks"]), (s["vc"], s["vs"])):
        rows = c[at // s["page"], :, at % s["page"]]
        g = g.view(1, -1, 1)
        x = _decode_fp4(rows, g) if cache == "fp4" else rows.view(torch.float8_e4m3fn).float() * g if cache == "fp8" else rows
        got.append(torch.where(live, x, 0).to(torch.bfloat16))
    return got


def _plain_attn(s, q, indptr, indices, lens, abort):
    """Tiles of 64 tokens, each against its request's queries; the tiles' sums joined per request in 64 bits."""
    page, nt = s["page"], s["tiles"]
    b, hq = q.shape[:2]
    hkv = s["kc"].shape[1]
    lens = lens.long()
    first = torch.cat([torch.zeros(1, dtype=torch.int64, device=DEV), ((lens + 63) // 64).cumsum(0)])
    tile = torch.arange(nt, device=DEV)
    r = (torch.searchsorted(first, tile, right=True) - 1).clamp(max=b - 1)
    pos = (tile - first[r]).unsqueeze(1) * 64 + torch.arange(64, device=DEV)
    live = pos < lens[r].unsqueeze(1)
    entry = (indptr.long()[r].unsqueeze(1) + pos // page).clamp(max=indices.numel() - 1)
    pg = indices.long()[entry].clamp(min=0)
    off = pos % page
    k = _decode_fp4(s["kc"][pg, :, off], s["ks"].view(1, 1, -1, 1)).transpose(1, 2)                 # [nt][hkv][64][128]
    qt = q.float().unflatten(1, (hkv, hq // hkv))[r]                                             # [nt][hkv][G][128]
    z = (qt @ k.transpose(2, 3)) / math.sqrt(D)
    del k
    z = z.masked_fill(~live[:, None, None, :], -math.inf)
    top = torch.full((b, hkv, hq // hkv), -math.inf, device=DEV).index_reduce_(0, r, z.amax(-1), "amax")
    p = torch.exp(z - top[r].unsqueeze(-1))
    v = _decode_fp4(s["vc"][pg, :, off], s["vs"].view(1, 1, -1, 1)).transpose(1, 2)
    num = torch.zeros(b, hkv, hq // hkv, D, dtype=torch.float64, device=DEV).index_add_(0, r, (p @ v).double())
    den = torch.zeros(b, hkv, hq // hkv, dtype=torch.float64, device=DEV).index_add_(0, r, p.sum(-1).double())
    out = (num / den.unsqueeze(-1)).flatten(1, 2)
    keep = (lens > 0) if abort is None else (lens > 0) & (abort == 0)
    return torch.where(keep.view(-1, 1, 1), out, 0.0).to(torch.bfloat16)


# ---------------------------------------------------------------------------------------------------------------------
# the library's calls
# ---------------------------------------------------------------------------------------------------------------------
def _own_tables(fkv, s):
    b, n_tok, nnz = s["cached"].numel(), s["tokens"], s["nnz"]
    if "t" not in s:
        i32 = dict(dtype=torch.int32, device=DEV)
        s["t"] = dict(step_lens=torch.empty(b, **i32), cached_out=torch.empty(b, **i32), refused=torch.empty(b, dtype=torch.uint8, device=DEV),
                      indptr=torch.empty(b + 1, **i32), indices=torch.zeros(nnz, **i32), expected=torch.zeros(nnz, **i32), token_indptr=torch.empty(b + 1, **i32),
                      slots=torch.empty(n_tok, dtype=torch.int64, device=DEV), positions=torch.empty(n_tok, **i32), free_left=torch.empty(1, **i32))
        s["tables_ws"] = fkv.alloc_step_tables_workspace(b)
    t = s["t"]
    fkv.kv_step_tables(s["cached"], s["new"], s["table"], s["table_tags"], s["free"], s["free_count"], s["tags"], s["page"],
                       t["step_lens"], t["cached_out"], t["refused"], t["indptr"], t["indices"], t["expected"], t["token_indptr"], t["slots"], t["positions"],
                       t["free_left"], s["tables_ws"])
    return t


def _own_rope(fkv, s, pos):
    q, k = s["q"], s["k"]
    if "qo" not in s:
        s["qo"], s["ko"] = (torch.empty(x.shape, dtype=x.dtype, device=DEV) for x in (q, k))
    fkv.qk_norm_rope(q, k, pos, s["inv_freq"], s["qo"], s["ko"], q_weight=s["qw"], k_weight=s["kw"], eps=s["eps"], axis_map=s["axis"],
                     interleaved=s["next"], rot_scale=s["rot_scale"])
    return s["qo"], s["ko"]


def _own_read(fkv, s, slots):
    if "kb" not in s:
        s["kb"], s["vb"] = (torch.empty(slots.numel(), s["kc"].shape[1], D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    fkv.kv_gather(s["kc"], s["vc"], slots, s["kb"], s["vb"], k_scale=s["ks"], v_scale=s["vs"])
    return [s["kb"], s["vb"]]


def _own_attn(fkv, s, q, indptr, indices, lens, abort):
    if "ws" not in s:
        s["ws"] = fkv.alloc_workspace(q.shape[0], q.shape[1], s["kc"].shape[1], fkv.KV_FP4)
        s["out"] = torch.empty_like(q)
    return fkv.paged_decode_attn(q, s["kc"], s["vc"], indptr, indices, lens, 1.0 / math.sqrt(D), s["out"], s["ws"], k_scale=s["ks"], v_scale=s["vs"], abort_mask=abort)


def run(s):
    kind = s["kind"]
    if own:
        import fp8_paged_kv_decode_gb300 as fkv
    if kind == "tables":
        if own:
            return dict(_own_tables(fkv, s), table=s["table"], table_tags=s["table_tags"])
        return _plain_tables(s)
    if kind == "rope":
        return list(_own_rope(fkv, s, s["pos"])) if own else list(_plain_rope(s, s["pos"]))
    if kind == "write":
        if own:
            fkv.kv_append_fp4(s["k"], s["v"], s["slots"], s["ks"], s["vs"], s["kc"], s["vc"])
            return _own_read(fkv, s, s["from"])
        _plain_write(s, s["k"], s["v"], s["slots"])
        return _plain_read(s, "fp4", s["from"])
    if kind == "read":
        return _own_read(fkv, s, s["from"]) if own else _plain_read(s, s["cache"], s["from"])
    if kind == "attn":
        f = (lambda *a: _own_attn(fkv, *a)) if own else _plain_attn
        return f(s, s["q"], s["indptr"], s["indices"], s["lens"], s["abort"])
    if own:
        t = _own_tables(fkv, s)
        q, k = _own_rope(fkv, s, t["positions"])
        fkv.kv_append_fp4(k, s["v"], t["slots"], s["ks"], s["vs"], s["kc"], s["vc"])
        b = t["step_lens"].numel()
        out = _own_attn(fkv, s, q[:b], t["indptr"], t["indices"], t["step_lens"], None)
        return [out, *_own_read(fkv, s, t["slots"])]
    t = _plain_tables(s)
    q, k = _plain_rope(s, t["positions"].unsqueeze(0))
    _plain_write(s, k, s["v"], t["slots"])
    out = _plain_attn(s, q[:t["step_lens"].numel()], t["indptr"], t["indices"], t["step_lens"], None)
    return [out, *_plain_read(s, "fp4", t["slots"])]


# ---------------------------------------------------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------------------------------------------------
def _mean(case):
    """The expected tokens per request."""
    return case["mid"] if case["ctx"] != "lognormal" else case["mid"] * min(1.377, 4.0)


def _work_tables(case):
    b, page = case["batch"], case["page"]
    new = 1 if case["new"] == 1 else case["new"] / 2
    nnz = b * math.ceil((_mean(case) + new) / page)
    return b * 32 + nnz * 16 + b * case["new"] * 12 + b * new / page * 20


def _work_rope(tokens, hq, hkv):
    return tokens * (hq + hkv) * D * 4, tokens * (hq + hkv) * D * 10


def _work_attn(case):
    t = case["batch"] * _mean(case) * (1 - case.get("stale", 0.0))
    return t * case["hkv"] * 2 * ROW + case["batch"] * case["hq"] * D * 4, t * case["hq"] * D * 4


def work(case):
    kind = case["kind"]
    if kind == "tables":
        return {"bytes": _work_tables(case), "flops": 0}
    if kind == "rope":
        b, f = _work_rope(case["tokens"], case["hq"], case["hkv"])
        return {"bytes": b, "flops": f}
    per = {"fp4": 2 * ROW, "fp8": 2 * D, "bf16": 4 * D}
    if kind == "write":
        return {"bytes": case["tokens"] * (case["hkv"] * (4 * D + 2 * ROW) + 8) + case["back"] * (case["hkv"] * (4 * D + 2 * ROW) + 8), "flops": (case["tokens"] + case["back"]) * case["hkv"] * 4 * D}
    if kind == "read":
        return {"bytes": case["tokens"] * (case["hkv"] * (4 * D + per[case["cache"]]) + 8), "flops": case["tokens"] * case["hkv"] * 2 * D}
    a, f = _work_attn(case)
    if kind == "attn":
        return {"bytes": a, "flops": f}
    b, g = _work_rope(case["batch"], case["hq"], case["hkv"])
    return {"bytes": a + b + _work_tables(dict(case, new=1)) + case["batch"] * case["hkv"] * 2 * (4 * D + 2 * ROW), "flops": f + g}


# ---------------------------------------------------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------------------------------------------------
def _exact_values(rows, g):
    """64-bit values of 72-byte rows, nibble by nibble: sign, two exponent bits, one mantissa bit."""
    lo, hi = rows[..., :64].long() % 16, rows[..., :64].long() // 16
    out = torch.empty(*rows.shape[:-1], D, dtype=torch.float64, device=rows.device)
    for parity, c in ((0, lo), (1, hi)):
        e, m = (c // 2) % 4, c % 2
        mag = torch.where(e == 0, 0.5 * m, torch.exp2((e - 1).double()) * (1 + 0.5 * m))
        out[..., parity::2] = torch.where(c >= 8, -mag, mag)
    b = rows[..., 64:].long()
    e, m = (b // 8) % 16, (b % 8).double()
    s = torch.where(e == 0, m * 2.0 ** -9, torch.exp2((e - 7).double()) * (1 + m / 8))
    s = torch.where(b % 128 == 127, math.nan, s) * torch.where(b >= 128, -1.0, 1.0)
    return out * s.repeat_interleave(16, -1) * g


def _exact_rounded(x, g):
    """What the 4-bit cache holds of bf16 x [n][H][128] (nearest e2m1 value by search; ties to the even code), in 64 bits."""
    n, h = x.shape[:2]
    x = x.float().view(n, h, 8, 16)
    g32 = g.view(1, h, 1, 1)
    ratio = x.abs().amax(-1, keepdim=True) / (g32 * torch.full_like(g32, 6.0))
    grid = torch.arange(127, dtype=torch.int64, device=DEV)
    e, m = grid // 8, (grid % 8).double()
    grid = torch.where(e == 0, m * 2.0 ** -9, torch.exp2((e - 7).double()) * (1 + m / 8))
    hi = torch.searchsorted(grid, ratio.double().clamp(max=448.0)).clamp(1, 126)
    down, up = ratio.double() - grid[hi - 1], grid[hi] - ratio.double()
    pick = torch.where(up < down, hi, torch.where(up > down, hi - 1, torch.where(hi % 2 == 0, hi, hi - 1)))
    s = grid[pick]
    d = s.float() * g32
    q = (x / d).double().abs()
    mags = torch.tensor(E2M1, dtype=torch.float64, device=DEV)
    hi = torch.searchsorted(mags, q.clamp(max=6.0)).clamp(1, 7)
    down, up = q - mags[hi - 1], mags[hi] - q
    pick = torch.where(up < down, hi, torch.where(up > down, hi - 1, torch.where(hi % 2 == 0, hi, hi - 1)))
    v = mags[pick] * torch.sign(x.double())
    return (torch.where(d == 0, 0.0, v) * s * g32.double()).view(n, h, D)


def _exact_rope(x, w, pos, s):
    y = x.double()
    if w is not None:
        y = y / torch.sqrt((y ** 2).mean(-1, keepdim=True) + s["eps"]) * w.double()
    half = s["inv_freq"].numel()
    out = y.clone()
    for j in range(half):
        axis = 0 if s["axis"] is None else int(s["axis"][j])
        t = pos[axis].double() * s["inv_freq"][j].double()
        c, n = (torch.cos(t) * s["rot_scale"]).unsqueeze(1), (torch.sin(t) * s["rot_scale"]).unsqueeze(1)
        a, b = (2 * j, 2 * j + 1) if s["next"] else (j, half + j)
        out[..., a], out[..., b] = y[..., a] * c - y[..., b] * n, y[..., a] * n + y[..., b] * c
    return out


def _exact_attn(s, q, pages_of, lens, dead, last=None):
    """`last`: the K and V values of each request's last token, where the cache does not hold it yet."""
    b, hq = q.shape[:2]
    hkv, page = s["kc"].shape[1], s["page"]
    out = torch.zeros(b, hq, D, dtype=torch.float64, device=DEV)
    for r in range(b):
        n = int(lens[r])
        if dead[r] or n <= 0:
            continue
        pg = pages_of(r)[:-(-n // page)].long()
        for h in range(hkv):
            k = _exact_values(s["kc"][pg, h].reshape(-1, ROW)[:n], s["ks"][h].double())
            v = _exact_values(s["vc"][pg, h].reshape(-1, ROW)[:n], s["vs"][h].double())
            if last is not None:
                k[-1], v[-1] = last[0][r, h], last[1][r, h]
            grp = slice(h * (hq // hkv), (h + 1) * (hq // hkv))
            w = torch.softmax(q[r, grp].double() @ k.t() / math.sqrt(D), -1)
            out[r, grp] = w @ v
    return out


def exact(case, seed):
    kind = case["kind"]
    if kind == "tables":
        return None                            # whole numbers
    if kind in ("attn", "step") and case["batch"] * _mean(case) * case["hkv"] > 3.0e6:
        return None                            # too long in 64 bits
    s = prepare(case, seed)
    if kind == "rope":
        return [_exact_rope(s["q"], s["qw"], s["pos"], s), _exact_rope(s["k"], s["kw"], s["pos"], s)]
    if kind in ("write", "read"):
        got, page = [], s["page"]
        for c, g, new in (("kc", "ks", "k"), ("vc", "vs", "v")):
            g = s[g]
            rows = s[c][s["from"] // page, :, s["from"] % page]
            if s.get("cache") == "bf16":
                got.append(rows.double())
                continue
            if s.get("cache") == "fp8":
                b = rows.long()
                e, m = (b // 8) % 16, (b % 8).double()
                got.append(torch.where(e == 0, m * 2.0 ** -9, torch.exp2((e - 7).double()) * (1 + m / 8)) * torch.where(b >= 128, -1.0, 1.0) * g.double().view(1, -1, 1))
                continue
            x = _exact_values(rows, g.double().view(1, -1, 1))
            if kind == "write":                # the tokens that the pass wrote
                where = torch.full((s["pool"] * page,), -1, dtype=torch.int64, device=DEV)
                where[s["slots"]] = torch.arange(s["tokens"], device=DEV)
                w = where[s["from"]]
                x = torch.where((w >= 0).view(-1, 1, 1), _exact_rounded(s[new], g)[w.clamp(min=0)], x)
            got.append(x)
        return got
    if kind == "attn":
        ptr = s["indptr"].tolist()
        return _exact_attn(s, s["q"], lambda r: s["indices"][ptr[r]:ptr[r + 1]], s["lens"].tolist(), s["abort"].tolist())
    # a step: every request gets one token at its length; a new page is the next one from the top of the free list
    b, page = case["batch"], s["page"]
    cached = s["cached"].tolist()
    top, rows = s["free"].numel(), s["table"].clone()
    for r in range(b):
        if cached[r] % page == 0:
            top -= 1
            rows[r, cached[r] // page] = s["free"][top]
    pos = torch.zeros(1, s["tokens"], device=DEV)
    pos[0, :b] = s["cached"].float()
    q = _exact_rope(s["q"], s["qw"], pos, s).to(torch.bfloat16)
    k = _exact_rope(s["k"], s["kw"], pos, s).to(torch.bfloat16)
    back = [torch.zeros(s["tokens"], case["hkv"], D, dtype=torch.float64, device=DEV) for _ in range(2)]
    for x, g, held in ((k, "ks", back[0]), (s["v"], "vs", back[1])):
        held[:b] = _exact_rounded(x[:b], s[g])
    return [_exact_attn(s, q[:b], lambda r: rows[r], [c + 1 for c in cached], [0] * b, back), *back]
