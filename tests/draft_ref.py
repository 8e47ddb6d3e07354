"""Plain references of a drafted step: attention of trees of drafted tokens and over
a window, the move of the accepted ones, and the append with the rotation on the way
(numpy, 64-bit floats)."""
from __future__ import annotations

import numpy as np

import step_ref as R
from fp8_paged_kv_decode_gb300 import workloads as W

D = 128
ROWS = {"fp8": 128, "bf16": 128, "fp4": 72}


def pool(rng, kind, P, H, S, garbage=True):
    """A pool of N(0, 1) values in the format (bytes, or bf16 bits), and its scales."""
    scale = rng.uniform(0.008, 0.012, H).astype(np.float32)
    x = rng.standard_normal((P * S, H, D)).astype(np.float32)
    if kind == "bf16":
        rows = W.bf16_bits(x)
    elif kind == "fp4":
        rows = R.fp4_encode(W.bf16_bits(x), scale)
    else:
        c = R.nearest(np.minimum(np.abs(x / scale[None, :, None]), 448.0).astype(np.float64), R.E4M3[:127])
        rows = (c + 128 * (x < 0)).astype(np.uint8)
    return np.ascontiguousarray(rows.reshape(P, S, H, ROWS[kind]).transpose(0, 2, 1, 3)), scale


def values(rows, kind, scale):
    """64-bit values of cache rows of one KV head."""
    if kind == "bf16":
        return W.bits_to_f32(rows).astype(np.float64)
    return (R.fp4_values(rows) if kind == "fp4" else R.E4M3[rows]) * np.float64(scale)


def random_tree(rng, n):
    """Ancestor-or-self sets of a random tree, as Python integers."""
    seen = []
    for i in range(n):
        p = int(rng.integers(-1, i)) if i else -1
        seen.append((seen[p] if p >= 0 else 0) | (1 << i))
    return seen


def words_of(sets, words):
    return np.array([[(m >> (64 * w)) & (2 ** 64 - 1) for w in range(words)] for m in sets], np.uint64).reshape(len(sets), words)


def visible(bits, n, c, window, sinks):
    """Which of c + n tokens each of the rows with these masks sees."""
    see = np.zeros((len(bits), c + n), bool)
    for i, m in enumerate(bits):
        p = c + max(bin(m).count("1") - 1, 0)
        t = np.arange(c)
        see[i, :c] = (t < sinks) | (t > p - window) if window else True
        see[i, c:] = [(m >> j) & 1 for j in range(n)]
    return see


def tree_attention(q_bits, kc, vc, kind, ks, vs, indptr, indices, lens, tptr, masks, sm, window=0, sinks=0, dead=None,
                   max_drafts=None):
    """(out, the largest |v| each row sees, which rows are written)."""
    N, Hq = q_bits.shape[:2]
    P, H, S = kc.shape[:3]
    G = Hq // H
    q = W.bits_to_f32(q_bits).astype(np.float64)
    out, vmax, written = np.zeros((N, Hq, D)), np.zeros((N, Hq, 1)), np.zeros(N, bool)
    for r in range(len(lens)):
        t0, t1, L = int(tptr[r]), int(tptr[r + 1]), int(lens[r])
        if t0 < 0 or t1 < t0 or t1 > N:
            continue
        n = t1 - t0
        written[t0:t1] = True
        b, e = int(indptr[r]), int(indptr[r + 1])
        if n == 0 or L < n or (dead is not None and dead[r]) or (max_drafts and n > max_drafts):
            continue
        if b < 0 or e < b or e > len(indices) or (e - b) * S < L:
            continue
        see = visible(masks[t0:t1], n, L - n, window, sinks)
        t = np.nonzero(see.any(0))[0]
        pg = indices[b + t // S].astype(np.int64)
        if ((pg < 0) | (pg >= P)).any():
            continue
        see = see[:, t]
        for h in range(H):
            k, v = values(kc[pg, h, t % S], kind, 1 if ks is None else ks[h]), values(vc[pg, h, t % S], kind, 1 if vs is None else vs[h])
            for i in range(n):
                s = see[i]
                if not s.any():
                    continue
                rows = slice(h * G, (h + 1) * G)
                with np.errstate(all="ignore"):
                    z = q[t0 + i, rows] @ k[s].T * sm
                    w = np.exp(z - z.max(-1, keepdims=True))
                    out[t0 + i, rows] = (w / w.sum(-1, keepdims=True)) @ v[s]
                    vmax[t0 + i, rows] = np.abs(v[s]).max()
    return out, vmax, written


def commit(kc, vc, S, indptr, indices, lens, tptr, accepted, counts, lens_out, dead, free, count, tags, n_tokens=2 ** 31 - 1):
    """One request after the other, one row after the other.  Returns what the call leaves, and whether it
    reports an invalid request."""
    P = kc.shape[0]
    kc, vc, lens_out, free = kc.copy(), vc.copy(), lens_out.copy(), None if free is None else free.copy()
    tags = None if tags is None else tags.copy()
    bad, back = False, []
    for r in range(len(lens)):
        t0, t1, L = int(tptr[r]), int(tptr[r + 1]), int(lens[r])
        b, e = int(indptr[r]), int(indptr[r + 1])
        n = t1 - t0
        if (dead is not None and dead[r]) or t0 < 0 or n < 0 or t1 > n_tokens or L < n or b < 0 or e < b or e > len(indices) or (e - b) * S < L:
            continue
        c, k = L - n, int(counts[r])
        ok = 0 <= k <= min(n, accepted.shape[1])
        path = accepted[r, :k].tolist() if ok else []
        ok = ok and all(0 <= a < n for a in path) and all(x < y for x, y in zip(path, path[1:]))
        if ok and n:
            drafted = indices[b + c // S:b + (L - 1) // S + 1]
            ok = bool(((drafted >= 0) & (drafted < P)).all())
        if not ok:
            bad = True
            continue
        for i, a in enumerate(path):
            src, dst = c + a, c + i
            for x in (kc, vc):
                x[indices[b + dst // S], :, dst % S] = x[indices[b + src // S], :, src % S]
        lens_out[r] = c + k
        back += indices[b + -(-(c + k) // S):b + -(-L // S)].tolist()
    left = None
    if free is not None:
        have = min(max(int(count), 0), len(free))
        if have + len(back) <= len(free):
            for i, p in enumerate(back):                        # the first one on top
                free[have + len(back) - 1 - i] = p
                if tags is not None:
                    tags[p] += 1
            left = have + len(back)
        else:
            bad, left = True, have
    return kc, vc, lens_out, free, left, tags, bad
