"""paged_tree_attn and paged_window_attn on the GPU against a dense softmax in 64 bits."""
import numpy as np
import pytest

import draft_ref as T
from fp8_paged_kv_decode_gb300 import workloads as W
from gpu_util import bf16_out, dev

pytestmark = pytest.mark.gpu
D = 128
KINDS = ["fp8", "bf16", "fp4"]


class Case:
    """Requests of c committed and n drafted tokens over scattered pages."""

    def __init__(self, kind, Hq, H, S, ctx, n, seed, words=None, q_std=1.0, sets=None, spare=5):
        rng = np.random.default_rng(seed)
        self.kind, self.Hq, self.H, self.S, self.rng = kind, Hq, H, S, rng
        self.ctx, self.n = np.asarray(ctx), np.asarray(n)
        self.lens = (self.ctx + self.n).astype(np.int32)
        self.tptr = np.concatenate([[0], np.cumsum(self.n)]).astype(np.int32)
        pages = -(-self.lens.astype(np.int64) // S)
        self.P = int(pages.sum()) + spare
        self.ptr = np.concatenate([[0], np.cumsum(pages)]).astype(np.int32)
        self.idx = rng.permutation(self.P)[:int(pages.sum())].astype(np.int32)
        (self.kc, self.ks), (self.vc, self.vs) = T.pool(rng, kind, self.P, H, S), T.pool(rng, kind, self.P, H, S)
        if kind == "bf16":
            self.ks = self.vs = None
        self.N = int(self.n.sum())
        self.q = W.bf16_bits((q_std * rng.standard_normal((self.N, Hq, D))).astype(np.float32))
        self.sets = sets if sets is not None else [m for k in self.n for m in T.random_tree(rng, int(k))]
        self.words = words or max(1, -(-int(max(self.n, default=1)) // 64))
        self.sm = 1.0 / np.sqrt(D)
        self.dead = None

    def ref(self, window=0, sinks=0):
        return T.tree_attention(self.q, self.kc, self.vc, self.kind, self.ks, self.vs, self.ptr, self.idx, self.lens, self.tptr, self.sets, self.sm,
                                window, sinks, self.dead, 64 * self.words)

    def tensors(self):
        import torch
        b16 = dict(dtype=torch.bfloat16)
        pool = (lambda a: dev(a, **b16)) if self.kind == "bf16" else dev
        return dict(q=dev(self.q, **b16), k_cache=pool(self.kc), v_cache=pool(self.vc), page_indptr=dev(self.ptr), page_indices=dev(self.idx),
                    seq_lens=dev(self.lens), sm_scale=self.sm, out=torch.full((self.N, self.Hq, D), float("nan"), device="cuda", **b16),
                    workspace=self.workspace(), k_scale=None if self.ks is None else dev(self.ks), v_scale=None if self.vs is None else dev(self.vs),
                    abort_mask=None if self.dead is None else dev(self.dead.astype(np.uint8)))

    def workspace(self):
        import fp8_paged_kv_decode_gb300 as fkv
        ws = fkv.alloc_tree_workspace(self.N, len(self.lens), self.Hq, self.H, dict(fp8=fkv.KV_FP8_E4M3, bf16=fkv.KV_BF16, fp4=fkv.KV_FP4)[self.kind])
        return ws.fill_(0xA5)                                       # no initialisation is needed

    def tree(self, t=None, **k):
        import fp8_paged_kv_decode_gb300 as fkv
        t = t or self.tensors()
        fkv.paged_tree_attn(**t, token_indptr=dev(self.tptr), tree_mask=dev(T.words_of(self.sets, self.words).view(np.int64)), **k)
        return t["out"]

    def window(self, t=None, **k):
        import fp8_paged_kv_decode_gb300 as fkv
        t = t or self.tensors()
        fkv.paged_window_attn(**t, **k)
        return t["out"]

    def check(self, out, window=0, sinks=0):
        want, vmax, written = self.ref(window, sinks)
        got = bf16_out(out)
        assert np.isnan(got[~written]).all()                        # rows of no request are not written
        got, want, vmax = got[written], want[written], vmax[written]
        assert np.array_equal(np.isnan(got), np.isnan(want)), np.argwhere(np.isnan(got) != np.isnan(want))[:4]
        fine = np.isfinite(want) & np.isfinite(vmax)
        # bf16's half step, 2^-8 of the value; a weight in 11 bits (f16), or two words of 8 (bf16), and the logit in
        # fp32 (|z| < 40 over 128 products: 2^-24 * 40 * 12 < 2^-15) move the mean by at most 2^-11 + 2^-12 of max|v|,
        # the normaliser included
        err = np.abs(got - want)
        tol = 2.0 ** -8 * np.abs(want) + (2.0 ** -11 + 2.0 ** -12) * vmax
        with np.errstate(all="ignore"):
            bad = (err > tol) & fine
        assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist(), float(err[fine].max()))
        odd = ~np.isfinite(want)
        assert np.array_equal(got[odd & ~np.isnan(want)], want[odd & ~np.isnan(want)])


SHAPES = [  # q heads, KV heads, page, committed, drafted
    (8, 2, 16, [0], [1]), (8, 2, 16, [1, 0, 15, 16, 17], [1, 3, 1, 16, 2]), (4, 4, 32, [5, 300, 127, 128, 129], [2, 7, 1, 4, 5]),
    (64, 8, 64, [1000, 63, 64, 65], [8, 8, 8, 8]), (16, 2, 128, [511, 512, 513, 0], [16, 1, 17, 5]), (6, 2, 16, [40, 0, 333], [11, 1, 64]),
    (24, 2, 32, [200, 77], [13, 3]), (40, 8, 64, [150, 700], [6, 9]), (16, 1, 64, [90], [61]), (5, 1, 128, [1300], [33]),
    (128, 1, 16, [70, 20], [2, 1]), (64, 1, 32, [129], [5]), (8, 8, 64, [2000] * 3, [4, 0, 1])]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("Hq,H,S,ctx,n", SHAPES)
def test_trees(kind, Hq, H, S, ctx, n):
    import fp8_paged_kv_decode_gb300 as fkv
    fkv.device_error()
    c = Case(kind, Hq, H, S, ctx, n, seed=Hq + S + len(ctx))
    c.check(c.tree())
    assert fkv.device_error() == 0


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 3), (2, 0), (7, 1), (64, 4), (100, 130), (129, 16), (500, 0), (10 ** 9, 4), (2 ** 31 - 1, 2 ** 31 - 1)])
def test_trees_with_a_window(kind, window, sinks):
    c = Case(kind, 16, 2, 16, [0, 1, 40, 200, 333, 640, 1000], [3, 5, 12, 1, 20, 7, 9], seed=window % 1000 + sinks % 1000)
    c.check(c.tree(window=window, sinks=sinks), window, sinks)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("Hq,H,S", [(8, 2, 16), (4, 4, 32), (64, 8, 64), (16, 1, 128), (24, 2, 64)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (64, 4), (130, 0), (300, 200), (1024, 16), (2 ** 31 - 1, 0)])
def test_windows(kind, Hq, H, S, window, sinks):
    import fp8_paged_kv_decode_gb300 as fkv
    fkv.device_error()
    lens = np.array([1, 2, 63, 64, 65, 127, 128, 129, 130, 131, 256, 300, 1025, 1500])
    c = Case(kind, Hq, H, S, lens - 1, np.ones(len(lens), int), seed=Hq + S, sets=[1] * len(lens))
    c.check(c.window(window=window, sinks=sinks), window, sinks)
    assert fkv.device_error() == 0


@pytest.mark.parametrize("kind", KINDS)
def test_many_drafted_tokens(kind):
    """Up to 256, several words, query rows of several tiles."""
    c = Case(kind, 8, 2, 32, [300, 10, 0, 129], [130, 64, 256, 65], seed=3)
    assert c.words == 4
    c.check(c.tree())
    c.check(c.tree(window=90, sinks=5), 90, 5)


@pytest.mark.parametrize("kind", KINDS)
def test_long_contexts(kind):
    """Units split over many blocks."""
    c = Case(kind, 16, 2, 64, [9000, 30, 20001], [4, 2, 7], seed=5)
    c.check(c.tree())
    c.check(c.tree(window=6000, sinks=100), 6000, 100)


@pytest.mark.parametrize("batch", [130, 700, 3000])
def test_many_requests(batch):
    rng = np.random.default_rng(batch)
    c = Case("fp8", 4, 1, 16, rng.integers(0, 200, batch), rng.integers(0, 4, batch), seed=batch)
    c.check(c.tree())
    c = Case("fp4", 2, 2, 16, rng.integers(0, 90, batch), np.ones(batch, int), seed=batch, sets=[1] * batch)
    c.check(c.window(window=33, sinks=2), 33, 2)


@pytest.mark.parametrize("kind", KINDS)
def test_masks_that_are_no_trees(kind):
    """Rows that see nothing, not themselves, later tokens, or bits of tokens that are not there."""
    ctx, n = [0, 0, 50, 130], [3, 70, 5, 4]
    rng = np.random.default_rng(8)
    sets = [0, 0b100, 0] + [int(rng.integers(0, 2 ** 62)) << 7 for _ in range(70)] + [0, 0b10, 0b11111, 2 ** 63, (2 ** 128 - 1)] + [2 ** 100, 0b1000, 0, 1]
    c = Case(kind, 8, 2, 16, ctx, n, seed=9, sets=sets)
    out = c.tree()
    c.check(out)
    assert (bf16_out(out)[[0, 2]] == 0).all()
    c.check(c.tree(window=2, sinks=0), 2, 0)


@pytest.mark.parametrize("kind", KINDS)
def test_nan_and_infinity_where_rows_do_not_look(kind):
    """A NaN or infinity in K or V reaches the rows that see its token, and no other."""
    ctx, n, S = [37, 300, 5], [6, 9, 4], 16
    c = Case(kind, 8, 2, S, ctx, n, seed=11)
    nan = {"fp8": 0x7F, "bf16": 0x7FC0, "fp4": 0x7F}[kind]

    def put(cache, r, t, d, value):
        pg, off = c.idx[c.ptr[r] + t // S], t % S
        cache[pg, :, off, 64 + d // 16 if kind == "fp4" else d] = value
    put(c.vc, 0, 37 + 2, 5, nan)                                   # a drafted token's V
    put(c.kc, 1, 300 + 4, 100, nan)                                # and K
    put(c.vc, 1, 300 + 8, 77, nan)                                 # one that only itself sees
    put(c.vc, 2, 5 + 1, 127, nan)
    put(c.vc, 2, 5 + 3, 0, nan)
    if kind == "bf16":
        put(c.vc, 0, 37 + 4, 6, 0x7F80)
        put(c.vc, 2, 5 + 2, 9, 0xFF80)
    # slots past the last token, pages' ends
    for r in range(3):
        for t in range(ctx[r] + n[r], -(-(ctx[r] + n[r]) // S) * S):
            put(c.kc, r, t, 3, nan)
            put(c.vc, r, t, 50, nan)
    c.check(c.tree())
    # committed tokens that a window leaves out, for the deeper rows or for all
    c = Case(kind, 8, 2, S, ctx, n, seed=12)
    for t in range(280, 299):
        put(c.vc, 1, t, t % 128, nan)
    put(c.kc, 1, 100, 1, nan)
    put(c.vc, 1, 100, 1, nan)
    c.check(c.tree(window=12, sinks=3), 12, 3)
    w = Case(kind, 8, 2, S, [300, 200], [1, 1], seed=13, sets=[1, 1])
    for t in (0, 1, 3, 250, 289):
        pg, off = w.idx[w.ptr[0] + t // S], t % S
        w.kc[pg, :, off, -1] = w.vc[pg, :, off, -1] = nan
    w.check(w.window(window=11, sinks=0), 11, 0)
    w.check(w.window(window=12, sinks=1), 12, 1)                   # sees 289 and 0


@pytest.mark.parametrize("kind", KINDS)
def test_failing_closed(kind):
    import fp8_paged_kv_decode_gb300 as fkv
    fkv.device_error()
    ctx, n = [100, 40, 70, 200, 30, 60, 90, 10], [5, 3, 8, 2, 4, 6, 7, 1]
    c = Case(kind, 8, 2, 16, ctx, n, seed=14)
    c.dead = np.array([0, 1, 0, 0, 0, 0, 0, 0])
    c.lens[2] = 7                                                  # fewer tokens than drafted ones
    c.lens[3] = 300                                                # more than its pages hold
    c.lens[5] = 0
    c.check(c.tree())
    assert fkv.device_error() == 0
    c.idx[c.ptr[4] + 1], c.idx[c.ptr[6] + 2] = c.P, -1              # pages outside the pool
    out = c.tree()
    c.check(out)
    assert fkv.device_error() == fkv.DEVERR_ATTN_PAGE
    got = bf16_out(out)
    for r in (1, 2, 3, 4, 5, 6):
        assert (got[c.tptr[r]:c.tptr[r + 1]] == 0).all()
    assert (np.abs(got[:5]).max(-1) > 0).all()
    c.ptr[1] = -4                                                  # requests 0 and 1
    c.check(c.tree())
    fkv.device_error()


def test_page_outside_the_window_is_not_read():
    import fp8_paged_kv_decode_gb300 as fkv
    fkv.device_error()
    c = Case("fp8", 8, 2, 16, [400, 500], [1, 1], seed=15, sets=[1, 1])
    want = bf16_out(c.window(window=60, sinks=5))
    c.idx[c.ptr[0] + 3:c.ptr[0] + 20] = -1
    got = bf16_out(c.window(window=60, sinks=5))
    assert np.array_equal(got, want) and fkv.device_error() == 0


def test_rows_of_no_request():
    """token_indptr that begins late, ends early or is out of order."""
    c = Case("fp8", 8, 2, 16, [100, 40, 70, 20], [5, 3, 8, 4], seed=16)
    c.tptr[0], c.tptr[4] = 2, 18                                   # rows 0, 1 and 18, 19 are nobody's
    c.sets[2:5] = [1, 3, 7]
    c.check(c.tree())
    c = Case("fp8", 8, 2, 16, [100, 40, 70, 20], [5, 3, 8, 4], seed=16)
    c.tptr[4] = 30                                                 # past the rows
    c.check(c.tree())
    c.tptr[:] = [0, 5, 3, 8, 12]                                   # decreasing; request 2's rows are 3 ..
    c.n = np.array([5, 0, 5, 4])
    t = c.tensors()
    out = bf16_out(c.tree(t))
    assert np.isfinite(out[:12]).all() and np.isnan(out[12:]).all()
    c = Case("fp4", 8, 2, 16, [100, 40], [80, 3], seed=17, words=1)  # more drafted tokens than mask bits
    c.check(c.tree())


@pytest.mark.parametrize("kind", KINDS)
def test_peaky_and_flat(kind):
    """Logits of standard deviation 30: one token takes all; and queries of zeros: the mean."""
    c = Case(kind, 8, 2, 64, [700, 1300], [5, 9], seed=18, q_std=30.0)
    want, vmax, _ = c.ref()
    got = bf16_out(c.tree())
    # |z| up to 200: fp32 products and their sum leave 2^-24 * 200 * 12 < 2^-12 in an exponent of e, on both sides
    assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -10 * vmax).all()
    c.q[:] = 0
    c.check(c.tree())


def test_sink_tokens_hide_nothing():
    """A token of large weight and zero V, the others 18 nats lower: they still make the output."""
    for kind in ("fp8", "bf16"):
        c = Case(kind, 8, 2, 64, [1500], [3], seed=19)
        one = np.uint16(0x3F80) if kind == "bf16" else np.uint8(0x38)
        c.q[:] = 0
        c.q[..., 0] = W.bf16_bits(np.full((1,), 8.0, np.float32))[0]
        c.kc[..., 0] = 0
        if c.ks is not None:
            c.ks[:], c.vs[:] = 1.0, 0.01
        c.sm = 18.0 / 8.0
        for t in (0, 700):
            pg = c.idx[t // 64]
            c.kc[pg, :, t % 64, 0], c.vc[pg, :, t % 64] = one, 0
        want, vmax, _ = c.ref()
        got = bf16_out(c.tree())
        # every other weight is 2^-26 of the largest: f16 keeps it to 2^-29, so within 2^-3 of itself, and the average
        # of some 1500 of one sign's rounding at worst the same
        assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -3 * np.abs(want) + 2.0 ** -12 * 2.0 ** -26 * 1500 * vmax + 1e-12).all()
        assert (np.abs(want).max(-1) > 0).all()


def test_same_bytes_every_time_and_padding():
    """Repeated calls, and the same requests beside an aborted one."""
    import torch
    c = Case("fp8", 64, 8, 64, [5000, 40, 900, 3000], [8, 3, 1, 12], seed=20)
    t = c.tensors()
    first = c.tree(t).clone()
    flush = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    for i in range(10):
        flush.fill_(i)
        t["out"].fill_(float("nan"))
        assert torch.equal(c.tree(t).view(torch.int16), first.view(torch.int16))


def test_streams_graphs_and_workspaces():
    """Two calls at once on streams and workspaces of their own; captured and replayed with changed inputs."""
    import torch
    a, b = Case("fp8", 32, 4, 64, [3000, 700], [8, 5], seed=21), Case("bf16", 16, 2, 32, [900, 2100, 5], [3, 9, 2], seed=22)
    ta, tb = a.tensors(), b.tensors()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    ga, gb = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    ma, mb = (dev(T.words_of(x.sets, x.words).view(np.int64)) for x in (a, b))
    pa, pb = dev(a.tptr), dev(b.tptr)
    import fp8_paged_kv_decode_gb300 as fkv
    with torch.cuda.graph(ga):
        fkv.paged_tree_attn(**ta, token_indptr=pa, tree_mask=ma)
    with torch.cuda.graph(gb):
        fkv.paged_tree_attn(**tb, token_indptr=pb, tree_mask=mb, window=500, sinks=4)
    for k in range(3):
        for x, t in ((a, ta), (b, tb)):
            x.q = W.bf16_bits(x.rng.standard_normal(x.q.shape).astype(np.float32))
            t["q"].copy_(dev(x.q, dtype=torch.bfloat16))
            t["out"].fill_(float("nan"))
        a.lens[0] = 3008 - 60 * k                                  # committed tokens change between replays
        ta["seq_lens"].copy_(dev(a.lens))
        torch.cuda.synchronize()
        with torch.cuda.stream(s1):
            ga.replay()
        with torch.cuda.stream(s2):
            gb.replay()
        torch.cuda.synchronize()
        a.check(ta["out"])
        b.check(tb["out"], 500, 4)


def test_float8_cache_and_uint64_mask():
    import torch
    import fp8_paged_kv_decode_gb300 as fkv
    c = Case("fp8", 8, 2, 16, [100, 40], [5, 3], seed=23)
    t = c.tensors()
    t["k_cache"], t["v_cache"] = (t[x].view(torch.float8_e4m3fn) for x in ("k_cache", "v_cache"))
    mask = dev(T.words_of(c.sets, 1)[:, 0].view(np.int64)).view(torch.uint64)
    fkv.paged_tree_attn(**t, token_indptr=dev(c.tptr), tree_mask=mask)
    c.check(t["out"])


def test_python_refusals():
    import torch
    import fp8_paged_kv_decode_gb300 as fkv
    c = Case("fp8", 8, 2, 16, [100, 40], [1, 1], seed=24, sets=[1, 1])
    z = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt, device="cuda")   # noqa: E731
    t = c.tensors()
    tree = dict(t, token_indptr=dev(c.tptr), tree_mask=z(2, dt=torch.int64))
    win = dict(t, window=4)
    common = (dict(q=t["q"].float()), dict(out=z(2, 8, 64)), dict(out=z(3, 8, D)), dict(k_scale=None), dict(k_scale=z(1, dt=torch.float32)),
              dict(seq_lens=z(2, dt=torch.int64)), dict(seq_lens=z(3, dt=torch.int32)), dict(abort_mask=z(2, dt=torch.int32)), dict(abort_mask=z(1, dt=torch.uint8)),
              dict(page_indptr=z(2, dt=torch.int32)), dict(page_indices=z(9, dt=torch.int64)), dict(workspace=z(16, dt=torch.uint8)), dict(sm_scale=0.0),
              dict(k_cache=t["k_cache"][:3]), dict(q=t["q"].cpu()), dict(q=z(2, D, 8).transpose(1, 2)), dict(sinks=-1), dict(window=-1), dict(window=2 ** 31),
              dict(window=1.5))
    for bad in common + (dict(token_indptr=z(2, dt=torch.int32)), dict(token_indptr=z(3, dt=torch.int64)), dict(tree_mask=z(2, dt=torch.int32)),
                         dict(tree_mask=z(3, dt=torch.int64)), dict(tree_mask=z(2, 5, dt=torch.int64)), dict(tree_mask=z(2, 0, dt=torch.int64))):
        with pytest.raises(fkv.FkvError):
            fkv.paged_tree_attn(**dict(tree, **bad))
    for bad in common + (dict(window=0), dict(q=z(3, 8, D), out=z(3, 8, D))):
        with pytest.raises(fkv.FkvError):
            fkv.paged_window_attn(**dict(win, **bad))
    with pytest.raises(fkv.FkvError):
        fkv.alloc_tree_workspace(2, 2, 7, 2)


WIDE = [  # 72 to 1300 rows of a KV head, in units of 128 and 256
    (16, 1, 16, [90, 0, 1000], [9, 30, 17]), (32, 1, 32, [130, 255, 256], [5, 8, 64]), (48, 2, 64, [700, 3], [11, 6]),
    (128, 1, 128, [400, 127], [2, 3]), (20, 4, 16, [4000, 60], [33, 61]), (8, 8, 64, [500, 30], [256, 200]), (127, 1, 32, [77], [10]),
    (16, 1, 64, [900, 50, 3], [6, 7, 5]), (72, 1, 16, [300], [1]), (96, 1, 32, [2000, 127, 0], [1, 1, 1]), (7, 1, 64, [5000], [18])]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("Hq,H,S,ctx,n", WIDE)
def test_wide_units(kind, Hq, H, S, ctx, n):
    import fp8_paged_kv_decode_gb300 as fkv
    fkv.device_error()
    c = Case(kind, Hq, H, S, ctx, n, seed=Hq + S)
    out = c.tree()
    c.check(out)
    first = out.clone()
    assert fkv.device_error() == 0
    for window, sinks in ((1, 0), (70, 3), (200, 130), (3000, 1)):
        c.check(c.tree(window=window, sinks=sinks), window, sinks)
    assert (c.tree().view(-1).view(dtype=first.dtype) == first.view(-1)).all()


@pytest.mark.parametrize("kind", KINDS)
def test_wide_units_of_odd_values_and_bad_requests(kind):
    """NaN and infinities where some rows do not look, bad pages, requests without work, rows that see nothing."""
    import fp8_paged_kv_decode_gb300 as fkv
    fkv.device_error()
    ctx, n, S = [37, 300, 5, 600], [16, 29, 24, 20], 16
    c = Case(kind, 32, 2, S, ctx, n, seed=31)
    nan = {"fp8": 0x7F, "bf16": 0x7FC0, "fp4": 0x7F}[kind]

    def put(cache, r, t, d, value):
        pg, off = c.idx[c.ptr[r] + t // S], t % S
        cache[pg, :, off, 64 + d // 16 if kind == "fp4" else d] = value
    put(c.vc, 0, 37 + 2, 5, nan)
    put(c.kc, 1, 300 + 4, 100, nan)
    put(c.vc, 1, 300 + 8, 77, nan)
    put(c.vc, 2, 5 + 23, 127, nan)
    if kind == "bf16":
        put(c.vc, 0, 37 + 4, 6, 0x7F80)
        put(c.vc, 0, 37 + 7, 6, 0xFF80)
        put(c.vc, 3, 600 + 9, 9, 0xFF80)
    for r in range(4):
        for t in range(ctx[r] + n[r], -(-(ctx[r] + n[r]) // S) * S):
            put(c.kc, r, t, 3, nan)
            put(c.vc, r, t, 50, nan)
    c.check(c.tree())
    c.sets[3], c.sets[20], c.sets[50] = 0, 0, 1 << 23
    c.check(c.tree())
    c.check(c.tree(window=13, sinks=2), 13, 2)
    c = Case(kind, 32, 2, S, ctx, n, seed=32)
    c.idx[c.ptr[1] + 7] = c.P
    c.dead = np.array([0, 0, 1, 0])
    out = c.tree()
    c.check(out)
    assert fkv.device_error() == fkv.DEVERR_ATTN_PAGE
    got = bf16_out(out)
    assert (got[c.tptr[1]:c.tptr[3]] == 0).all() and (np.abs(got[:c.tptr[1]]).max(-1) > 0).all()


@pytest.mark.parametrize("kind", KINDS)
def test_few_requests_in_many_parts(kind):
    """A hundred parts of a unit, joined by all warps of a block; rows past the unit's in the last eight."""
    c = Case(kind, 6, 1, 64, [30000, 9], [3, 1], seed=33)
    c.check(c.tree())
    c.check(c.tree(window=20000, sinks=70), 20000, 70)
    c = Case(kind, 5, 1, 16, [40000], [1], seed=34, sets=[1])
    c.check(c.window(window=39000, sinks=3), 39000, 3)


@pytest.mark.parametrize("kind", ["fp8", "bf16"])
@pytest.mark.parametrize("n", [[12, 17], [5, 7]])
def test_wide_units_of_rising_logits(kind, n):
    """Logits that grow along the tokens, by 150 nats in all and again: references move in either half of a tile."""
    c = Case(kind, 16, 1, 64, [900, 333], n, seed=35)
    one = np.uint16(0x3F80) if kind == "bf16" else np.uint8(0x38)
    c.kc[..., 0], c.sm = 0, 0.3
    if c.ks is not None:
        c.ks[:] = 1.0
    for r in range(2):
        for t in range(49, int(c.lens[r]), 50):                        # 1, 2, 4, ... 128 times the query's first dim
            c.kc[c.idx[c.ptr[r] + t // 64], :, t % 64, 0] = one + (t // 50 % 8 << (7 if kind == "bf16" else 3))
    c.q[..., 0] = W.bf16_bits(np.full((1,), 4.0, np.float32))[0]
    want, vmax, _ = c.ref()
    got = bf16_out(c.tree())
    # |z| up to 200: fp32 products and their sum leave 2^-24 * 200 * 12 < 2^-12 in an exponent of e, on both sides
    assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -10 * vmax).all()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("window,sinks", [(300, 40), (1000, 0), (1, 200)])
def test_lengths_near_the_largest(kind, tree, window, sinks):
    """Requests of up to 2^31 - 1 tokens whose window and first tokens are those of short ones: the same outputs."""
    import torch
    S, long = 128, 2 ** 31 - 1
    n = 3 if tree else 1
    tail = [long % S + 9 * S, 77 + 9 * S]                             # the short requests
    c = Case(kind, 4, 1, S, [x - n for x in tail], [n, n], seed=36, sets=None if tree else [1, 1])
    call = c.tree if tree else c.window
    c.check(call(window=window, sinks=sinks), window, sinks)
    lens = np.array([long, 2 ** 30 + 77], np.int64)
    pages = -(-lens // S)
    ptr = np.concatenate([[0], np.cumsum(pages)]).astype(np.int32)
    idx = torch.zeros(int(ptr[-1]), dtype=torch.int32, device="cuda")
    for r in range(2):
        row = c.idx[c.ptr[r]:c.ptr[r + 1]]
        idx[int(ptr[r]):int(ptr[r]) + 2] = dev(row[:2])                # the first tokens' pages, and at the end all of them
        idx[int(ptr[r + 1]) - len(row):int(ptr[r + 1])] = dev(row)
    t = c.tensors()
    t.update(page_indptr=dev(ptr), page_indices=idx, seq_lens=dev(lens.astype(np.int32)))
    c.check(call(t, window=window, sinks=sinks), window, sinks)
    if window == 1:                                                    # first tokens without end: all of the short request's
        t = c.tensors()
        c.check(call(t, window=1, sinks=2 ** 31 - 1), 1, 2 ** 31 - 1)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("Hq,H", [(8, 2), (64, 8), (24, 1), (100, 1)])
def test_a_workspace_of_more_tokens_fits_fewer(kind, Hq, H):
    import fp8_paged_kv_decode_gb300 as fkv
    kv = dict(fp8=fkv.KV_FP8_E4M3, bf16=fkv.KV_BF16, fp4=fkv.KV_FP4)[kind]
    sizes = [fkv.paged_tree_attn_workspace_size(n, b, Hq, H, kv_dtype=kv) for n in (1, 2, 7, 30, 64, 300, 5000) for b in (1, 3, 64)]
    assert sizes == sorted(sizes)
    ws = fkv.alloc_tree_workspace(500, 64, Hq, H, kv)
    for ctx, n in (([40], [1]), ([30, 5], [1, 3]), ([200], [33]), ([100], [60]), ([9] * 30, [1] * 30)):
        c = Case(kind, Hq, H, 16, ctx, n, seed=37)
        t = c.tensors()
        t["workspace"] = ws
        c.check(c.tree(t))


def test_two_graphs_of_other_kernels_at_once():
    """A window over a 4-bit cache and wide trees over BF16, replayed on two streams with lengths that change, and eagerly
    on a third; the first replay's state does not reach the next."""
    import torch
    import fp8_paged_kv_decode_gb300 as fkv
    a = Case("fp4", 32, 8, 16, [3000] * 40, [1] * 40, seed=41, sets=[1] * 40)
    b = Case("bf16", 32, 2, 64, [2500, 300, 5], [20, 31, 11], seed=42)
    e = Case("fp8", 16, 2, 32, [900, 2100, 5], [3, 4, 2], seed=43)
    ta, tb, te = a.tensors(), b.tensors(), e.tensors()
    pb, mb = dev(b.tptr), dev(T.words_of(b.sets, b.words).view(np.int64))
    pe, me = dev(e.tptr), dev(T.words_of(e.sets, e.words).view(np.int64))
    s1, s2, s3 = (torch.cuda.Stream() for _ in range(3))
    torch.cuda.synchronize()
    ga, gb = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(ga):
        fkv.paged_window_attn(**ta, window=777, sinks=5)
    with torch.cuda.graph(gb):
        fkv.paged_tree_attn(**tb, token_indptr=pb, tree_mask=mb)
    for k in range(4):
        for x, t in ((a, ta), (b, tb), (e, te)):
            x.q = W.bf16_bits(x.rng.standard_normal(x.q.shape).astype(np.float32))
            t["q"].copy_(dev(x.q, dtype=torch.bfloat16))
            t["out"].fill_(float("nan"))
        a.lens[:] = [3001 - (37 * k * i) % 3000 for i in range(40)]
        b.lens[0] = 2520 - 800 * k
        ta["seq_lens"].copy_(dev(a.lens))
        tb["seq_lens"].copy_(dev(b.lens))
        torch.cuda.synchronize()
        with torch.cuda.stream(s1):
            ga.replay()
        with torch.cuda.stream(s2):
            gb.replay()
        fkv.paged_tree_attn(**te, token_indptr=pe, tree_mask=me, window=50, sinks=1, stream=s3.cuda_stream)
        torch.cuda.synchronize()
        a.check(ta["out"], 777, 5)
        b.check(tb["out"])
        e.check(te["out"], 50, 1)


@pytest.mark.parametrize("kind", ["fp8", "fp4"])
@pytest.mark.parametrize("Hq,n", [(2, [3, 1]), (16, [3, 3]), (16, [7, 6]), (16, [40, 30])])
def test_head_scales_of_zero_and_below(kind, Hq, n):
    """16, 32 to 64, 128 and 256 rows a unit: a K scale of zero makes all logits equal, one below zero turns them around."""
    for ks in (0.0, -1.0):
        c = Case(kind, Hq, 2, 16, [70, 300], n, seed=44)
        c.ks[0] *= ks
        c.vs[1] = -c.vs[1]
        c.check(c.tree())
        c.check(c.tree(window=60, sinks=2), 60, 2)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n", [40, 47])
def test_wide_units_of_one_and_two_blocks_in_turn(kind, n):
    """Each KV head's drafted tokens are a unit of 256 rows and one of 64 (or 120), whose sums lie where the next Q goes."""
    import torch
    c = Case(kind, 64, 8, 16, [5, 150, 2, 90, 260, 31, 0, 120] * 8, [n] * 64, seed=n)
    t = c.tensors()
    first = c.tree(t).clone()
    c.check(first)
    for _ in range(10):
        t["out"].fill_(float("nan"))
        assert torch.equal(c.tree(t).view(torch.int16), first.view(torch.int16))


ROWS = [(4, 3), (4, 7), (8, 8), (16, 7), (16, 13)]                    # query heads a KV head, drafted tokens: 16, 32, 64, 128 and 256 rows a unit


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("G,n", ROWS)
@pytest.mark.parametrize("words", [1, 4])
def test_bits_of_tokens_that_are_not_there(kind, G, n, words):
    """They change nothing, the depth by which a window is placed included (the reference counts every bit that it is given:
    it gets the masks without them)."""
    import torch
    c = Case(kind, 2 * G, 2, 64, [1000, 3000, 700], [n, n - 1, n], seed=45, words=words)
    own = c.sets
    most = [k for k in (n, n - 1, n) for _ in range(k)]
    every = [m | (((1 << 64 * words) - 1) >> k << k) for m, k in zip(own, most)]
    for window, sinks in ((0, 0), (300, 0), (1000, 5), (129, 70), (650, 0)):
        c.sets = every
        out = c.tree(window=window, sinks=sinks)
        c.sets = own
        c.check(out, window, sinks)
        assert torch.equal(out.view(torch.int16), c.tree(window=window, sinks=sinks).view(torch.int16))


def one_dim_keys(c, value, rows):
    """Keys of dim 0 alone: `value` (1, 0.5, -1 or -2; the K scales become 1) at these cache rows [page, offset]."""
    code = {"fp8": {1: 0x38, 0.5: 0x30, -1: 0xB8, -2: 0xC0}, "bf16": {1: 0x3F80, 0.5: 0x3F00, -1: 0xBF80, -2: 0xC000}, "fp4": {1: 2, 0.5: 1, -1: 10, -2: 12}}
    if c.ks is not None:
        c.ks[:] = 1.0
    for pg, off in rows:
        c.kc[pg, :, off] = 0
        c.kc[pg, :, off, 0] = code[c.kind][value]
        if c.kind == "fp4":
            c.kc[pg, :, off, 64] = 0x38


def few_on_top(kind, G, n, sign):
    """A few tokens share each row's largest logit, of either sign, and the others are far below it: the output is the mean of
    those few.  Rows' logits are 1, 1.125 ... 1.5 times 1024 c.sm."""
    c = Case(kind, 2 * G, 2, 64, [300, 500], [n, n], seed=46)
    top, low = (1, 0.5) if sign > 0 else (-1, -2)
    for r in range(2):
        at = [(c.idx[c.ptr[r] + t // 64], t % 64) for t in range(int(c.lens[r]))]
        one_dim_keys(c, low, at)
        one_dim_keys(c, top, [at[t] for t in (3, 70, 71, 200, 290)])
    q = np.zeros(c.q.shape, np.float32)
    q[..., 0] = 1024 * (1 + np.arange(c.q.shape[0] * 2 * G).reshape(c.q.shape[:2]) % 5 / 8)
    c.q = W.bf16_bits(q)
    return c


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("G,n", ROWS)
@pytest.mark.parametrize("sign", [1, -1])
def test_logits_whose_references_round(kind, G, n, sign):
    """Logits (in log2 units) up to 4e8, where fp32 neighbours are 8, 16 and 32 apart."""
    c = few_on_top(kind, G, n, sign)
    for z in (3e4, 3e6, 6e7, 1.4e8, 2e8, 2.6e8):
        c.sm = z * np.log(2.0) / 1024
        c.check(c.tree())
        c.check(c.tree(window=260, sinks=4), 260, 4)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("G,n", ROWS)
@pytest.mark.parametrize("sign", [1, -1])
def test_huge_logits(kind, G, n, sign):
    """Logits (in log2 units) of 1e9 and more, where a product that is not rounded as the reference was leaves tens to
    thousands of log2 units in the exponent."""
    c = few_on_top(kind, G, n, sign)
    for z in (1e9, 1e10, 3e12, 1e30):
        c.sm = z * np.log(2.0) / 1024
        c.check(c.tree())
        c.check(c.tree(window=260, sinks=4), 260, 4)


@pytest.mark.parametrize("kind", ["fp8", "fp4"])
@pytest.mark.parametrize("G,n", ROWS)
@pytest.mark.parametrize("size", [1e-12, 1e-30, 1e-37])
def test_a_head_scale_of_zero_and_tiny_queries(kind, G, n, size):
    c = Case(kind, 2 * G, 2, 16, [70, 300], [n, n - 1], seed=47, q_std=size)
    c.ks[0] = 0.0
    c.check(c.tree())
    c.check(c.tree(window=60, sinks=2), 60, 2)


@pytest.mark.parametrize("kind", ["fp8", "fp4"])
@pytest.mark.parametrize("G,n", ROWS)
def test_a_head_scale_that_is_no_number(kind, G, n):
    c = Case(kind, 2 * G, 2, 16, [70, 300], [n, n - 1], seed=53)
    c.ks[0] = np.nan
    got = bf16_out(c.tree())
    assert np.isnan(got[:, :G]).all() and np.isfinite(got[:, G:]).all()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("G,n", ROWS)
def test_query_elements_far_below_the_largest(kind, G, n):
    """2^-32 of the largest of a KV head's rows counts, to its last bit: a logit of 8 + 1/16 against 3000 of zero."""
    c = Case(kind, 2 * G, 2, 64, [3000], [n], seed=48)
    q = np.zeros(c.q.shape, np.float32)
    q[::2, :, 0] = 1.0                                                # the other rows have only the small element
    q[..., 1] = 2.0 ** -32 * (1 + 2.0 ** -7)
    c.q, c.sm = W.bf16_bits(q), 2.0 ** 32
    c.kc[...] = 0
    if c.ks is not None:
        c.ks[:] = 1.0
    pg, off = c.idx[1234 // 64], 1234 % 64
    if kind == "fp4":
        c.kc[pg, :, off, 0], c.kc[pg, :, off, 64] = 0x60, 0x40        # 4 times 2
    else:
        c.kc[pg, :, off, 1] = 0x50 if kind == "fp8" else 0x4100
    c.check(c.tree())


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("S", [16, 32, 64])
@pytest.mark.parametrize("window,sinks", [(60, 5), (60, 0), (33, 17), (100, 40), (100, 130)])
@pytest.mark.parametrize("tree", [False, True])
def test_pages_between_the_first_tokens_and_the_window(kind, S, window, sinks, tree):
    """They are not read and may hold any id, however near the two are."""
    import fp8_paged_kv_decode_gb300 as fkv
    fkv.device_error()
    lens = np.arange(30, 420, 11)
    k = 3 if tree else 1
    c = Case(kind, 8, 2, S, lens - k, np.full(len(lens), k), seed=49, sets=None if tree else [1] * len(lens))
    gone = 0
    for r, length in enumerate(lens):
        first = max(0, length - k - window + 1)                       # of the committed tokens of a row at depth 0
        for j in range(c.ptr[r], c.ptr[r + 1]):
            a = (j - c.ptr[r]) * S
            if a >= min(sinks, first) and a + S <= first:
                c.idx[j] = (-1, c.P, 2 ** 31 - 1)[j % 3]
                gone += 1
    assert gone or sinks == 130
    c.check((c.tree if tree else c.window)(window=window, sinks=sinks), window, sinks)
    assert fkv.device_error() == 0


@pytest.mark.parametrize("Hq,H", [(8, 2), (64, 2), (128, 1)])
def test_no_tokens(Hq, H):
    """A workspace for no tokens, and the calls that it is for."""
    import torch
    import fp8_paged_kv_decode_gb300 as fkv
    c = Case("fp8", Hq, H, 16, [40, 5], [1, 1], seed=50, sets=[1, 1])
    t = c.tensors()
    ws = fkv.alloc_tree_workspace(0, 0, Hq, H)
    assert ws.numel() <= fkv.alloc_tree_workspace(1, 1, Hq, H).numel()
    none = dict(t, q=t["q"][:0], out=t["out"][:0], workspace=ws)
    fkv.paged_tree_attn(**none, token_indptr=torch.zeros(3, dtype=torch.int32, device="cuda"), tree_mask=torch.zeros(0, dtype=torch.int64, device="cuda"))
    none.update(page_indptr=t["page_indptr"][:1], seq_lens=t["seq_lens"][:0])
    fkv.paged_window_attn(**none, window=5)
    assert fkv.device_error() == 0


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("window,sinks", [(5, 0), (5, 3), (40, 8)])
def test_a_chain_deeper_than_the_window(kind, window, sinks):
    """With the bits of the ancestors unset that the window leaves out, each row is paged_window_attn's of the same token."""
    ctx, n = np.array([90, 3, 400]), np.array([12, 50, 9])
    sets = [sum(1 << j for j in range(i + 1) if i - j < window or c + j < sinks) for c, k in zip(ctx, n) for i in range(k)]
    c = Case(kind, 8, 2, 16, ctx, n, seed=52, sets=sets)
    c.check(c.tree(window=window, sinks=sinks), window, sinks)
    w = Case(kind, 8, 2, 16, ctx, n, seed=52, sets=sets)                # the same pools, one token of each request at a time
    w.sets, w.N = [1] * 3, 3
    rows = c.tptr[:-1]
    for i in range(int(n.max())):
        at = np.minimum(i, n - 1)
        w.lens, w.q, w.tptr = (ctx + at + 1).astype(np.int32), c.q[rows + at], np.arange(4, dtype=np.int32)
        w.check(w.window(window=window, sinks=sinks), window, sinks)
        want, got = w.ref(window, sinks)[0], c.ref(window, sinks)[0][rows + at]
        assert np.allclose(got, want)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("Hq,H", [(8, 2), (16, 2), (16, 1)])
def test_requests_beside_an_aborted_one(kind, Hq, H):
    """Aborted requests take nothing from the others, whose bytes stay the same, and leave zeros."""
    import torch
    c = Case(kind, Hq, H, 64, [2000, 40, 900, 600], [8, 8, 8, 8], seed=51)
    alone = c.tree().clone()
    c.dead = np.array([0, 1, 0, 1])
    for r in (1, 3):
        c.idx[c.ptr[r]:c.ptr[r + 1]] = -1                              # not read either
    out = c.tree()
    c.check(out)
    assert (out[8:16] == 0).all() and (out[24:] == 0).all()
    c = Case(kind, Hq, H, 64, [2000, 40, 900, 600], [8, 8, 8, 8], seed=51)
    c.dead = np.zeros(4)
    assert torch.equal(c.tree().view(torch.int16), alone.view(torch.int16))


@pytest.mark.parametrize("G,n", ROWS)
@pytest.mark.parametrize("power", [110, 119])
def test_bf16_values_near_the_largest(G, n, power):
    """Values of 2^110 and 2^119: their sum over 400 tokens is below 2^128, and so is every sum on the way."""
    c = Case("bf16", 2 * G, 2, 64, [300, 390], [n, n - 1], seed=54, q_std=3.0)
    c.vc = ((c.vc & 0x8000) | ((c.vc & 0x7F) + ((power + 127) << 7))).astype(np.uint16)      # [2^power, 2^(power + 1)), either sign
    c.check(c.tree())
    c.check(c.tree(window=100, sinks=2), 100, 2)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("G,n", ROWS)
@pytest.mark.parametrize("levels", [(-2, -1, 0), (0, 0.5, 1), (-2, 0, 0.5), (0.5, 1, -2)])
def test_references_that_get_huge_and_small_again(kind, G, n, levels):
    """Logits that rise along the tokens, from huge negative ones to zero or from there to huge ones: the output is the mean of the
    last level's (or, falling, the second's)."""
    c = Case(kind, 2 * G, 2, 64, [290, 600], [n, n], seed=55)
    for r in range(2):
        at = [(c.idx[c.ptr[r] + t // 64], t % 64) for t in range(int(c.lens[r]))]
        one_dim_keys(c, -2, at)
        for k, value in enumerate(levels):
            rows = at[45 + 75 * k:45 + 75 * (k + 1)]
            if value:
                one_dim_keys(c, value, rows)
            else:
                for pg, off in rows:
                    c.kc[pg, :, off] = 0
    q = np.zeros(c.q.shape, np.float32)
    q[..., 0] = 1024 * (1 + np.arange(c.q.shape[0] * 2 * G).reshape(c.q.shape[:2]) % 5 / 8)
    c.q = W.bf16_bits(q)
    for z in (4e5, 2e6, 1e9, 1e12):
        c.sm = z * np.log(2.0) / 1024
        c.check(c.tree())
