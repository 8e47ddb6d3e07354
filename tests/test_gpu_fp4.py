"""The 4-bit cache on the GPU: append and read-back bit for bit, attention
against 64-bit softmax on the same bytes."""
import numpy as np
import pytest

import step_ref as R
from fp8_paged_kv_decode_gb300 import workloads as W
from gpu_util import bf16_out, dev

pytestmark = pytest.mark.gpu
D, ROW = 128, 72


def same_rows(got, want):
    """Equal bytes; a NaN scale and a zero code may carry either sign."""
    g, w = got.copy(), want.copy()
    for x in (g, w):
        s = x[..., 64:]
        s[(s & 0x7F) == 0x7F] = 0x7F
        c = x[..., :64]
        c[(c & 0x0F) == 0x08] &= 0xF0
        c[(c & 0xF0) == 0x80] &= 0x0F
    return np.array_equal(g, w)


def append(k, v, slots, ks, vs, kc, vc):
    import torch
    import fp8_paged_kv_decode_gb300 as fkv
    kt, vt = dev(kc), dev(vc)
    fkv.kv_append_fp4(dev(k, dtype=torch.bfloat16), dev(v, dtype=torch.bfloat16), dev(slots), dev(ks), dev(vs), kt, vt)
    return kt.cpu().numpy(), vt.cpu().numpy()


@pytest.mark.parametrize("n,H,S,P", [(1, 1, 16, 1), (5, 2, 16, 3), (33, 3, 32, 4), (257, 8, 64, 9), (1000, 4, 24, 60)])
def test_append_bytes(n, H, S, P):
    rng = np.random.default_rng(n)
    k, v = (W.bf16_bits((rng.standard_normal((n, H, D)) * 10.0 ** rng.integers(-3, 3, (n, H, 1))).astype(np.float32)) for _ in range(2))
    ks, vs = (np.exp(rng.uniform(-6, 0, H)).astype(np.float32) for _ in range(2))
    slots = np.full(n, -1, np.int64)
    m = min(n, P * S) - (n > 4)
    slots[rng.permutation(n)[:m]] = rng.permutation(P * S)[:m]
    kc, vc = (rng.integers(0, 256, (P, H, S, ROW)).astype(np.uint8) for _ in range(2))
    got = append(k, v, slots, ks, vs, kc, vc)
    for g, x, sc, c in zip(got, (k, v), (ks, vs), (kc, vc)):
        want = c.copy()
        rows = R.fp4_encode(x, sc)
        for i, s in enumerate(slots):
            if s >= 0:
                want[s // S, :, s % S] = rows[i]
        assert same_rows(g, want)


@pytest.mark.parametrize("scale", [1.0, 0.0078125, 0.3, 2.0 ** -40, 2.0 ** 40, 1e-44, 1e38])
def test_append_every_bf16_pattern(scale):
    """All 65536 patterns, each block one pattern's neighbourhood plus specials
    in some: NaN, infinities, subnormals, zeros, and scales past the fast path."""
    bits = np.arange(65536, dtype=np.uint16).reshape(512, 1, D)
    rng = np.random.default_rng(3)
    mixed = rng.permutation(65536).astype(np.uint16).reshape(512, 1, D)
    for x in (bits, mixed):
        g = np.array([scale], np.float32)
        kc, vc = (np.zeros((8, 1, 64, ROW), np.uint8) for _ in range(2))
        got = append(x, x, np.arange(512, dtype=np.int64), g, g, kc, vc)
        want = R.fp4_encode(x, g).reshape(8, 64, 1, ROW).transpose(0, 2, 1, 3)
        assert same_rows(got[0], want) and same_rows(got[1], want)


def test_append_next_to_code_borders():
    """Quotients within a few ulps of the midpoints between codes."""
    rng = np.random.default_rng(4)
    n = 4096
    g = np.float32(0.0123)
    mids = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    x = np.zeros((n, 1, 8, 16), np.float32)
    top = rng.uniform(0.5, 4, (n, 1, 8)).astype(np.float32)
    x[..., 0] = W.bits_to_f32(W.bf16_bits(top))
    s = R.nearest((x[..., 0] / (np.float32(6) * g)).astype(np.float64), R.E4M3[:127])
    d = R.E4M3[s].astype(np.float32) * g
    x[..., 1:] = (mids[rng.integers(0, 7, (n, 1, 8, 15))] * d[..., None]) * np.where(rng.random((n, 1, 8, 15)) < 0.5, -1, 1)
    bits = W.bf16_bits(x.reshape(n, 1, D))
    kc = np.zeros((n // 64, 1, 64, ROW), np.uint8)
    got = append(bits, bits, np.arange(n, dtype=np.int64), np.array([g]), np.array([g]), kc, kc.copy())
    want = R.fp4_encode(bits, np.array([g], np.float32)).reshape(n // 64, 64, 1, ROW).transpose(0, 2, 1, 3)
    assert same_rows(got[0], want) and same_rows(got[1], want)


def test_append_slots_past_the_pool_and_tag_check():
    import torch
    import fp8_paged_kv_decode_gb300 as fkv
    rng = np.random.default_rng(5)
    n, H, S, P = 9, 2, 16, 4
    k, v = (W.bf16_bits(rng.standard_normal((n, H, D)).astype(np.float32)) for _ in range(2))
    sc = np.array([0.01, 0.02], np.float32)
    slots = np.array([0, 63, 64, -1, 17, 1 << 40, 5, -(1 << 40), 40], np.int64)
    fkv.device_error()
    kc = np.full((P, H, S, ROW), 0x5A, np.uint8)
    got = append(k, v, slots, sc, sc, kc, kc.copy())
    assert fkv.device_error() == fkv.DEVERR_APPEND_SLOT
    for g, x in zip(got, (k, v)):
        want = kc.copy()
        rows = R.fp4_encode(x, sc)
        for i, s in enumerate(slots):
            if 0 <= s < P * S:
                want[s // S, :, s % S] = rows[i]
        assert same_rows(g, want)
    # the append and the check in one launch: the same bytes, the check's own mask
    live = rng.integers(0, 2 ** 32, P, dtype=np.uint64).astype(np.uint32)
    indptr, indices = np.array([0, 2, 2, 4], np.int32), np.array([0, 3, 1, 2], np.int32)
    exp = live[indices].copy()
    exp[2] += 1
    kt, vt = dev(kc), dev(kc)
    mask = torch.full((3,), 7, dtype=torch.uint8, device="cuda")
    fkv.kv_append_fp4_tag_check(dev(k, dtype=torch.bfloat16), dev(v, dtype=torch.bfloat16), dev(slots), dev(sc), dev(sc), kt, vt,
                                dev(live.view(np.int32)), dev(indptr), dev(indices), dev(exp.view(np.int32)), mask)
    assert mask.tolist() == [0, 0, 1]
    assert np.array_equal(kt.cpu().numpy(), got[0]) and np.array_equal(vt.cpu().numpy(), got[1])
    assert fkv.device_error() == fkv.DEVERR_APPEND_SLOT


@pytest.mark.parametrize("kind", ["fp4", "fp8", "bf16"])
@pytest.mark.parametrize("n,H,S,P", [(1, 1, 16, 1), (37, 3, 64, 5), (700, 8, 24, 40)])
def test_gather(kind, n, H, S, P):
    import torch
    import fp8_paged_kv_decode_gb300 as fkv
    rng = np.random.default_rng(n + len(kind))
    shape = (P, H, S, ROW if kind == "fp4" else D)
    ks, vs = (np.exp(rng.uniform(-6, 1, H)).astype(np.float32) for _ in range(2))
    if kind == "bf16":
        kc, vc = (W.bf16_bits(rng.standard_normal(shape).astype(np.float32)) for _ in range(2))
        kt, vt = dev(kc, dtype=torch.bfloat16), dev(vc, dtype=torch.bfloat16)
    else:
        kc, vc = (rng.integers(0, 256, shape).astype(np.uint8) for _ in range(2))      # every code, NaN among them
        kt, vt = dev(kc), dev(vc)
    slots = rng.integers(0, P * S, n).astype(np.int64)                                 # repeats
    if n > 2:
        slots[1], slots[2] = -1, P * S
    ko, vo = (torch.full((n, H, D), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    fkv.device_error()
    fkv.kv_gather(kt, vt, dev(slots), ko, vo, k_scale=dev(ks), v_scale=dev(vs))
    assert fkv.device_error() == (fkv.DEVERR_GATHER_SLOT if n > 2 else 0)
    for o, c, sc in ((ko, kc, ks), (vo, vc, vs)):
        want = R.gather(c, slots, S, sc, kind)
        got = bf16_out(o)
        assert np.array_equal(np.isnan(got), np.isnan(want))
        assert np.array_equal(np.nan_to_num(got), np.nan_to_num(want))


class Fp4Case:
    """A paged batch whose unwritten rows hold every byte at once (0xFF: NaN scales)."""

    def __init__(self, B, Hq, H, S, seq, seed=0, q_std=1.0, spare=5, extra_pages=0):
        rng = np.random.default_rng(seed)
        self.B, self.Hq, self.H, self.S = B, Hq, H, S
        self.seq = np.asarray(seq, np.int32)
        npages = -(-np.maximum(self.seq.astype(np.int64), 0) // S) + extra_pages
        used = int(npages.sum())
        self.P = used + spare
        self.indptr = np.concatenate([[0], np.cumsum(npages)]).astype(np.int32)
        self.indices = rng.permutation(self.P).astype(np.int32)[:used]
        self.ks, self.vs = (rng.uniform(0.006, 0.02, H).astype(np.float32) for _ in range(2))
        self.kc, self.vc = (np.full((self.P, H, S, ROW), 0xFF, np.uint8) for _ in range(2))
        for r in range(B):
            n = int(self.seq[r])
            if n <= 0:
                continue
            pages = self.indices[self.indptr[r]:self.indptr[r + 1]][:-(-n // S)]
            for c, g in ((self.kc, self.ks), (self.vc, self.vs)):
                rows = R.fp4_encode(W.bf16_bits(rng.standard_normal((n, H, D)).astype(np.float32)), g)
                full = np.full((len(pages) * S, H, ROW), 0xFF, np.uint8)
                full[:n] = rows
                c[pages] = full.reshape(len(pages), S, H, ROW).transpose(0, 2, 1, 3)
        self.q = W.bf16_bits((q_std * rng.standard_normal((B, Hq, D))).astype(np.float32))
        self.sm = 1.0 / np.sqrt(D)

    def gpu(self, seq=None, indices=None, mask=None, noalloc=False, indptr=None, large=False):
        """large: a page table with room for so many pages that the call takes
        the kernel's large-call instance (60000 tiles of 64 tokens and more)."""
        import torch
        import fp8_paged_kv_decode_gb300 as fkv
        out = torch.full((self.B, self.Hq, D), float("nan"), dtype=torch.bfloat16, device="cuda")
        indices = self.indices if indices is None else indices
        if large:
            R = next(r for r in (1, 2, 4, 8) if (self.Hq // self.H) % r == 0 and self.Hq // self.H // r <= 8)
            room = 60000 * 64 // (self.S * self.H * R) + 2
            indices = np.concatenate([indices, np.zeros(max(0, room - len(indices)), np.int32)])
        args = [dev(self.q, dtype=torch.bfloat16), dev(self.kc), dev(self.vc), dev(self.indptr if indptr is None else indptr),
                dev(indices), dev(self.seq if seq is None else np.asarray(seq, np.int32)), self.sm, out]
        kw = dict(k_scale=dev(self.ks), v_scale=dev(self.vs), abort_mask=None if mask is None else dev(np.asarray(mask, np.uint8)))
        if noalloc:
            fkv.paged_decode_attn_noalloc(*args, **kw)
        else:
            fkv.paged_decode_attn(*args, fkv.alloc_workspace(self.B, self.Hq, self.H, fkv.KV_FP4), **kw)
        torch.cuda.synchronize()
        return out

    def check(self, out, seq=None, dead=None, rows=None):
        want, vmax = R.attention(self.q, self.kc, self.vc, self.ks, self.vs, self.indptr, self.indices,
                                 self.seq if seq is None else seq, self.sm, dead)
        got = bf16_out(out)
        # bf16 rounding 2^-8 of the value; P in f16: 2^-11 of each weight, so 2^-11 max|v| in the sum; the logits'
        # and exponentials' fp32 errors stay under another 2^-12 max|v| for |logit| < 2^8
        tol = 2.0 ** -8 * np.abs(want) + (2.0 ** -11 + 2.0 ** -12) * vmax
        sel = slice(None) if rows is None else rows
        assert np.isfinite(got[sel]).all()
        err = np.abs(got - want)
        assert (err[sel] <= tol[sel]).all(), (float((err - tol)[sel].max()), np.argwhere(err > tol)[:4])


@pytest.mark.parametrize("large", [False, True])
@pytest.mark.parametrize("B,Hq,H,S,seq", [
    (1, 1, 1, 16, [1]), (1, 8, 1, 64, [2]), (3, 6, 2, 16, [1, 15, 16]), (4, 16, 4, 32, [31, 32, 33, 64]),
    (5, 40, 8, 64, [63, 64, 65, 127, 129]), (2, 14, 2, 128, [1, 300]), (3, 8, 8, 128, [64, 65, 1000]),
    (2, 20, 2, 16, [700, 45]), (2, 64, 2, 64, [500, 90]), (1, 12, 4, 32, [9000]), (1, 4, 1, 16, [20000]),
    (64, 8, 2, 16, list(range(1, 65))), (65, 8, 2, 64, list(range(1, 650, 10))), (130, 4, 1, 32, list(range(1, 1301, 10))),
    (300, 2, 1, 16, [7 * (i % 40) + 1 for i in range(300)])])
def test_attention(B, Hq, H, S, seq, large):
    c = Fp4Case(B, Hq, H, S, seq, seed=B * 100 + Hq + S)
    c.check(c.gpu(large=large))


@pytest.mark.parametrize("large", [False, True])
@pytest.mark.parametrize("S", [16, 64, 128])
def test_attention_peaky_softmax(S, large):
    c = Fp4Case(3, 8, 2, S, [200, 1, 777], seed=9, q_std=8.0)
    c.check(c.gpu(large=large))


@pytest.mark.parametrize("large", [False, True])
@pytest.mark.parametrize("S", [16, 64])
def test_attention_fail_closed(S, large):
    import fp8_paged_kv_decode_gb300 as fkv
    c = Fp4Case(6, 8, 2, S, [100, 200, 50, 300, 80, 130], seed=11)
    seq = c.seq.copy()
    seq[2] = 0
    seq[4] = 10 ** 6                                            # more tokens than its pages hold
    dead = [0, 1, 1, 0, 1, 0]
    fkv.device_error()
    out = c.gpu(seq=seq, mask=[0, 1, 0, 0, 0, 0], large=large)
    c.check(out, seq=np.where(np.array(dead) > 0, 0, c.seq), dead=dead)
    assert (out.float().cpu().numpy()[np.array(dead) > 0] == 0).all() and fkv.device_error() == 0
    idx = c.indices.copy()
    idx[c.indptr[3] + 1] = c.P
    idx[c.indptr[5]] = -1
    out = c.gpu(indices=idx, large=large)
    assert fkv.device_error() == fkv.DEVERR_ATTN_PAGE
    got = out.float().cpu().numpy()
    assert (got[[3, 5]] == 0).all()
    c.check(out, rows=[0, 1, 2, 4])


def test_attention_nan_block_reaches_its_dims_only():
    """A NaN in V's block 3 of one token: dims 48..63 of the heads that read it, nothing else."""
    c = Fp4Case(2, 4, 2, 16, [40, 50], seed=12)
    page = c.indices[c.indptr[1] + 1]
    c.vc[page, 1, 5, 64 + 3] = 0x7F
    got = c.gpu().float().cpu().numpy()
    bad = np.isnan(got)
    want = np.zeros_like(bad)
    want[1, 2:4, 48:64] = True
    assert np.array_equal(bad, want)


@pytest.mark.parametrize("large", [False, True])
@pytest.mark.parametrize("B,S,seq", [(3, 16, [900, 5000, 64]), (40, 64, [64 * i + 3 for i in range(40)]), (140, 32, [300] * 140)])
def test_attention_repeats_byte_for_byte(B, S, seq, large):
    import torch
    c = Fp4Case(B, 16, 2, S, seq, seed=13)
    first = c.gpu(large=large)
    for _ in range(4):
        assert torch.equal(first.view(torch.int16), c.gpu(large=large).view(torch.int16))


def test_attention_noalloc_is_the_same_call():
    import torch
    c = Fp4Case(5, 16, 4, 32, [10, 2000, 333, 64, 65], seed=14)
    for large in (False, True):
        assert torch.equal(c.gpu(large=large).view(torch.int16), c.gpu(noalloc=True, large=large).view(torch.int16))


@pytest.mark.parametrize("B,Hq,H,S,seq", [(9, 32, 4, 64, [20000, 50000, 1, 33, 5000, 21000, 64, 9000, 12345]),
                                          (66, 16, 4, 16, [2049] * 66), (3, 16, 2, 128, [90000, 129, 40001])])
def test_attention_long(B, Hq, H, S, seq):
    """Units over hundreds of warps, and warps over many units, in both instances."""
    c = Fp4Case(B, Hq, H, S, seq, seed=B)
    for large in (False, True):
        c.check(c.gpu(large=large))


def test_attention_shared_pages():
    c = Fp4Case(3, 8, 2, 16, [64, 64, 64], seed=15)
    idx = c.indices.copy()
    idx[4:8] = idx[0:4]
    idx[8:10] = idx[0:2]
    c.indices = idx
    c.check(c.gpu())


def test_large_pool():
    """Byte offsets past 2^32: the batch's pages at the top of a 4.9 GB pool."""
    import torch
    import fp8_paged_kv_decode_gb300 as fkv
    c = Fp4Case(2, 16, 8, 64, [150, 70], seed=16, spare=0)
    P = 2 ** 32 // (8 * 64 * ROW) + 16000
    kt, vt = (torch.zeros(P, 8, 64, ROW, dtype=torch.uint8, device="cuda") for _ in range(2))
    kt[P - c.P:], vt[P - c.P:] = dev(c.kc), dev(c.vc)
    idx = c.indices + (P - c.P)
    out = torch.empty(2, 16, D, dtype=torch.bfloat16, device="cuda")
    fkv.device_error()
    fkv.paged_decode_attn(dev(c.q, dtype=torch.bfloat16), kt, vt, dev(c.indptr), dev(idx), dev(c.seq), c.sm, out,
                          fkv.alloc_workspace(2, 16, 8, fkv.KV_FP4), k_scale=dev(c.ks), v_scale=dev(c.vs))
    c.check(out)
    k = W.bf16_bits(np.random.default_rng(17).standard_normal((3, 8, D)).astype(np.float32))
    slots = np.array([P * 64 - 1, (P - 2) * 64 + 5, 0], np.int64)
    fkv.kv_append_fp4(dev(k, dtype=torch.bfloat16), dev(k, dtype=torch.bfloat16), dev(slots), dev(c.ks), dev(c.vs), kt, vt)
    for t, g in ((kt, c.ks), (vt, c.vs)):
        rows = torch.stack([t[s // 64, :, s % 64] for s in slots.tolist()]).cpu().numpy()
        assert same_rows(rows, R.fp4_encode(k, g))
    ko, vo = (torch.empty(3, 8, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    fkv.kv_gather(kt, vt, dev(slots), ko, vo, k_scale=dev(c.ks), v_scale=dev(c.vs))
    want = R.bf16_of(R.fp4_values(R.fp4_encode(k, c.ks)) .astype(np.float32) * c.ks[None, :, None])
    assert np.array_equal(bf16_out(ko), want) and fkv.device_error() == 0


def test_realloc_scrubs_whole_pages():
    import torch
    import fp8_paged_kv_decode_gb300 as fkv
    kt, vt = (torch.full((5, 3, 16, ROW), 9, dtype=torch.uint8, device="cuda") for _ in range(2))
    tags = torch.arange(5, dtype=torch.int32, device="cuda")
    new = torch.empty(2, dtype=torch.int32, device="cuda")
    fkv.kv_page_realloc(tags, torch.tensor([3, 0], dtype=torch.int32, device="cuda"), new, kt, vt)
    assert new.tolist() == [4, 1] and tags.tolist() == [1, 1, 2, 4, 4]
    for t in (kt, vt):
        assert t.view(5, -1).float().mean(1).tolist() == [0, 9, 9, 0, 9]


def test_python_refusals():
    import torch
    import fp8_paged_kv_decode_gb300 as fkv
    kt = torch.zeros(4, 2, 16, ROW, dtype=torch.uint8, device="cuda")
    x = torch.zeros(3, 2, D, dtype=torch.bfloat16, device="cuda")
    s = torch.ones(2, device="cuda")
    slots = torch.zeros(3, dtype=torch.int64, device="cuda")
    for bad in (dict(k_new=x.float()), dict(k_new=x[:2]), dict(slot_mapping=slots.int()), dict(k_scale=s[:1]), dict(k_cache=kt[:, :, :, :64].contiguous()),
                dict(v_cache=kt[:2].contiguous()), dict(k_new=x.cpu())):
        a = dict(k_new=x, v_new=x, slot_mapping=slots, k_scale=s, v_scale=s, k_cache=kt, v_cache=kt.clone())
        a.update(bad)
        with pytest.raises(fkv.FkvError):
            fkv.kv_append_fp4(**a)
    o = torch.zeros(3, 2, D, dtype=torch.bfloat16, device="cuda")
    for bad in (dict(k_scale=None), dict(k_out=o[:2]), dict(slots=slots.int()), dict(v_cache=kt[:2].contiguous()), dict(k_out=o.float())):
        a = dict(k_cache=kt, v_cache=kt.clone(), slots=slots, k_out=o, v_out=o.clone(), k_scale=s, v_scale=s)
        a.update(bad)
        with pytest.raises(fkv.FkvError):
            fkv.kv_gather(**a)
