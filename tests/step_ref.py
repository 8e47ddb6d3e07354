"""Plain references of the 4-bit cache, the read-back, the head norms with
rotation and the step tables (numpy, 64-bit floats, loops where they are clearer)."""
from __future__ import annotations

import numpy as np

from fp8_paged_kv_decode_gb300 import workloads as W

D = 128
ROW = 72
MAGS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def e4m3_values() -> np.ndarray:
    """The 256 e4m3 codes' values from the format's definition."""
    out = np.zeros(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        v = np.nan if (e, m) == (15, 7) else (m / 8.0) * 2.0 ** -6 if e == 0 else (1 + m / 8.0) * 2.0 ** (e - 7)
        out[c] = -v if c & 128 else v
    return out


E4M3 = e4m3_values()


def nearest(x, grid):
    """Index of the nearest grid value (ascending, ties to the even index)."""
    i = np.clip(np.searchsorted(grid, x), 1, len(grid) - 1)
    lo, hi = x - grid[i - 1], grid[i] - x
    return np.where(lo < hi, i - 1, np.where(hi < lo, i, np.where(i % 2 == 0, i, i - 1)))


def fp4_encode(bits: np.ndarray, g: np.ndarray) -> np.ndarray:
    """bf16 bit patterns [n][H][128] with fp32 scales [H] to rows [n][H][72].
    Quotients are numpy's IEEE binary32 divisions."""
    n, h = bits.shape[:2]
    with np.errstate(all="ignore"):
        x = W.bits_to_f32(bits).reshape(n, h, 8, 16)
        g = g.astype(np.float32).reshape(1, h, 1, 1)
        amax = np.abs(x).max(-1, keepdims=True)                    # NaN if the block has one
        ratio = (amax / (np.float32(6) * g)).astype(np.float32)
        sc = nearest(np.minimum(np.nan_to_num(ratio.astype(np.float64), nan=0.0, posinf=448.0), 448.0), E4M3[:127])
        sc = np.where(np.isnan(ratio), 0x7F, sc)
        d = (E4M3[sc].astype(np.float32) * g).astype(np.float32)
        q = (x / d).astype(np.float32)
        code = nearest(np.minimum(np.nan_to_num(np.abs(q).astype(np.float64), nan=0.0, posinf=6.0), 6.0), MAGS)
        code = code + 8 * np.signbit(x)
        code = np.where(np.isnan(d) | (d == 0), 0, code).reshape(n, h, D).astype(np.uint8)
    return np.concatenate([code[..., 0::2] | (code[..., 1::2] << 4), sc[..., 0].astype(np.uint8)], -1)


def fp4_values(rows: np.ndarray) -> np.ndarray:
    """code * block scale of rows [..., 72], before the head's scale."""
    code = np.stack([rows[..., :64] & 15, rows[..., :64] >> 4], -1).reshape(rows.shape[:-1] + (D,))
    v = np.where(code >= 8, -1.0, 1.0) * MAGS[code & 7]
    return v * np.repeat(E4M3[rows[..., 64:]], 16, -1)


def bf16_of(x: np.ndarray) -> np.ndarray:
    """64-bit values rounded to fp32 and then to bf16, as values."""
    with np.errstate(all="ignore"):
        f = x.astype(np.float32)
        return np.where(np.isfinite(f), W.bits_to_f32(W.bf16_bits(f)), f).astype(np.float64)


def gather(cache, slots, page, scale, kind):
    """[n][H][128] values of a pool [P][H][S][...]; `cache` holds bytes (fp4,
    fp8) or bf16 bits."""
    P, H = cache.shape[:2]
    out = np.zeros((len(slots), H, D))
    for i, s in enumerate(slots):
        if s < 0 or s // page >= P:
            continue
        rows = cache[s // page, :, s % page]
        if kind == "bf16":
            out[i] = W.bits_to_f32(rows)
        else:
            v = fp4_values(rows) if kind == "fp4" else E4M3[rows]
            with np.errstate(all="ignore"):
                out[i] = bf16_of(v.astype(np.float32) * scale.astype(np.float32)[:, None])
    return out


def attention(q_bits, kc, vc, ks, vs, indptr, indices, lens, sm, dead=None):
    """Dense softmax in 64 bits over an FP4 pool; also max |v| per (request, KV head)."""
    B, Hq = q_bits.shape[:2]
    H, S = kc.shape[1], kc.shape[2]
    G = Hq // H
    out = np.zeros((B, Hq, D))
    vmax = np.zeros((B, Hq, 1))
    q = W.bits_to_f32(q_bits).astype(np.float64)
    for r in range(B):
        n = int(lens[r])
        if n <= 0 or (dead is not None and dead[r]):
            continue
        pages = indices[indptr[r]:indptr[r + 1]][:-(-n // S)]
        for h in range(H):
            k = fp4_values(kc[pages, h].reshape(-1, ROW)[:n]) * np.float64(ks[h])
            v = fp4_values(vc[pages, h].reshape(-1, ROW)[:n]) * np.float64(vs[h])
            z = q[r, h * G:(h + 1) * G] @ k.T * sm
            p = np.exp(z - z.max(-1, keepdims=True))
            out[r, h * G:(h + 1) * G] = (p / p.sum(-1, keepdims=True)) @ v
            vmax[r, h * G:(h + 1) * G] = np.abs(v).max()
    return out, vmax


def norm_rope(bits, weight_bits, pos, inv_freq, axis_map, eps, interleaved, rot_scale):
    """Rows [N][H][128] in 64 bits, and the size of what each output adds up."""
    y = W.bits_to_f32(bits).astype(np.float64)
    if weight_bits is not None:
        y = y / np.sqrt((y ** 2).mean(-1, keepdims=True) + eps) * W.bits_to_f32(weight_bits).astype(np.float64)
    out, size = y.copy(), np.abs(y)
    half = len(inv_freq)
    for j in range(half):
        axis = 0 if axis_map is None else int(axis_map[j])
        if axis >= len(pos):
            continue
        t = pos[axis].astype(np.float64) * np.float64(inv_freq[j])
        c, s = (np.cos(t) * rot_scale)[:, None], (np.sin(t) * rot_scale)[:, None]
        a, b = (2 * j, 2 * j + 1) if interleaved else (j, j + half)
        out[..., a], out[..., b] = y[..., a] * c - y[..., b] * s, y[..., b] * c + y[..., a] * s
        size[..., a] = size[..., b] = (np.abs(y[..., a]) + np.abs(y[..., b])) * abs(rot_scale)
    return out, size


def step_tables(cached, new, table, table_tags, free_pages, free_count, page_tags, page, nnz, n_tokens, indices,
                expected):
    """One request after the other.  Returns a dict of the outputs; `indices`
    and `expected` are what those arrays held before."""
    B, M = table.shape
    P = len(page_tags)
    table, table_tags = table.copy(), table_tags.copy()
    indices, expected = indices.copy(), expected.copy()
    free = min(max(int(free_count), 0), len(free_pages))
    o = dict(step_lens=np.zeros(B, np.int32), cached_out=np.array(cached, np.int32), refused=np.zeros(B, np.uint8),
             indptr=np.zeros(B + 1, np.int32), token_indptr=np.zeros(B + 1, np.int32),
             slots=np.full(n_tokens, -1, np.int64), positions=np.zeros(n_tokens, np.int32))
    row = tok = asked = used = 0
    bad = False
    for r in range(B):
        c, n = int(cached[r]), int(new[r])
        pages = -(-(c + n) // page) if c >= 0 and n >= 0 else 0
        valid = c >= 0 and n >= 0 and c + n <= 2 ** 31 - 1 and pages <= M
        pages = pages if valid else 0
        have = -(-c // page) if valid else 0
        row0, tok0 = row, tok
        row, tok = row + pages, tok + max(n, 0)
        fits = valid and row <= nnz and tok <= n_tokens
        need = pages - have if fits else 0
        asked += need
        ok = fits and (need == 0 or asked <= free)
        o["indptr"][r + 1], o["token_indptr"][r + 1] = min(row, nnz), min(tok, n_tokens)
        o["refused"][r] = not ok
        bad |= not ok
        if ok:
            o["step_lens"][r] = o["cached_out"][r] = c + n
            used += need
        for j in range(pages):
            if j < have:
                i, t = int(table[r, j]), table_tags[r, j]
                if row0 + j < nnz and not 0 <= i < P:
                    i, bad = -1, True
            elif ok:
                i = int(free_pages[free - 1 - (asked - need + j - have)])
                t = 0
                if not 0 <= i < P:
                    i, bad = -1, True
                else:
                    t = page_tags[i]
                    table_tags[r, j] = t
                table[r, j] = i
            else:
                i, t = -1, 0
            if row0 + j < nnz:
                indices[row0 + j], expected[row0 + j] = i, t
        for i in range(max(n, 0)):
            if tok0 + i >= n_tokens or not valid:
                continue
            o["positions"][tok0 + i] = c + i
            pg = int(table[r, (c + i) // page]) if ok else -1
            if 0 <= pg < P:
                o["slots"][tok0 + i] = pg * page + (c + i) % page
    o |= dict(indices=indices, expected=expected, table=table, table_tags=table_tags,
              free_left=np.array([free - used], np.int32), bad=bad)
    return o
