"""Steps with drafted tokens as a serving loop makes them: tables from lengths, rotation
and append in one pass, the integrity check, tree attention, the accepted tokens moved and
the left-over pages given back; eager and replayed."""
import contextlib
import ctypes

import numpy as np
import pytest

import draft_ref as T
from fp8_paged_kv_decode_gb300 import workloads as W
from gpu_util import bf16_out, dev

pytestmark = pytest.mark.gpu
D = 128


class Loop:
    def __init__(self, kind, B, Hq, H, S, drafts, pool, blocks, seed, window=0, sinks=0):
        import torch
        import fp8_paged_kv_decode_gb300 as fkv
        rng = np.random.default_rng(seed)
        self.kind, self.B, self.Hq, self.H, self.S, self.drafts, self.rng = kind, B, Hq, H, S, drafts, rng
        self.window, self.sinks, self.P = window, sinks, pool
        i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")        # noqa: E731
        self.cached, self.new, self.table, self.btags = i32(B), i32(B), i32(B, blocks) - 1, i32(B, blocks)
        self.free0 = rng.permutation(pool).astype(np.int32)
        self.free, self.count = dev(self.free0), dev(np.array([pool], np.int32))
        self.tags0 = rng.integers(0, 2 ** 31, pool).astype(np.int32)
        self.live = dev(self.tags0)
        nnz = B * blocks
        self.step, self.refused, self.ptr, self.idx, self.exp, self.tptr = i32(B), torch.zeros(B, dtype=torch.uint8, device="cuda"), i32(B + 1), i32(nnz), i32(nnz), i32(B + 1)
        self.kc, self.vc = (dev(T.pool(rng, kind, pool, H, S)[0]) for _ in range(2))
        if kind == "bf16":
            self.kc, self.vc = (x.view(torch.bfloat16) for x in (self.kc, self.vc))
        self.ks, self.vs = (rng.uniform(0.01, 0.03, H).astype(np.float32) for _ in range(2))
        self.kst, self.vst = dev(self.ks), dev(self.vs)
        self.freq = dev((10000.0 ** (-np.arange(64) / 64)).astype(np.float32))
        self.w = dev(W.bf16_bits(np.ones(D, np.float32)), dtype=torch.bfloat16)
        self.mask = torch.zeros(B, dtype=torch.uint8, device="cuda")
        self.tws = fkv.alloc_step_tables_workspace(B)
        self.kv = dict(fp8=fkv.KV_FP8_E4M3, bf16=fkv.KV_BF16, fp4=fkv.KV_FP4)[kind]
        self.acc, self.kept = i32(B, max(drafts, 1)), i32(B)
        self.depth = i32(0)

    def buffers(self, n):
        import torch
        import fp8_paged_kv_decode_gb300 as fkv
        self.N = n
        self.slots, self.pos = torch.zeros(n, dtype=torch.int64, device="cuda"), torch.zeros(n, dtype=torch.int32, device="cuda")
        self.qkv = torch.zeros(n, (self.Hq + 2 * self.H) * D, dtype=torch.bfloat16, device="cuda")
        self.qo, self.out = (torch.zeros(n, self.Hq, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        self.tree = torch.zeros(n, dtype=torch.int64, device="cuda")
        self.back = torch.zeros(n, dtype=torch.int32, device="cuda")      # how far a token's depth is behind its place
        self.ws = fkv.alloc_tree_workspace(n, self.B, self.Hq, self.H, self.kv)

    def calls(self, attend=True):
        import fp8_paged_kv_decode_gb300 as fkv
        Hq, H = self.Hq, self.H
        fkv.kv_step_tables(self.cached, self.new, self.table, self.btags, self.free, self.count, self.live, self.S, self.step, self.cached, self.refused,
                           self.ptr, self.idx, self.exp, self.tptr, self.slots, self.pos, self.count, self.tws)
        self.pos.sub_(self.back)
        q, k, v = (x.unflatten(1, (-1, D)) for x in self.qkv.split((Hq * D, H * D, H * D), 1))
        fkv.kv_append_rope(q, k, v, self.pos, self.freq, self.slots, self.qo, self.kc, self.vc, k_scale=self.kst, v_scale=self.vst, q_weight=self.w, k_weight=self.w)
        fkv.kv_page_tag_check(self.live, self.ptr, self.idx, self.exp, self.mask)
        if attend:
            fkv.paged_tree_attn(self.qo, self.kc, self.vc, self.ptr, self.idx, self.step, self.tptr, self.tree, D ** -0.5, self.out, self.ws,
                                k_scale=self.kst, v_scale=self.vst, abort_mask=self.mask, window=self.window, sinks=self.sinks)

    def commit(self):
        import fp8_paged_kv_decode_gb300 as fkv
        fkv.kv_tree_commit(self.kc, self.vc, self.ptr, self.idx, self.step, self.tptr, self.acc, self.kept, self.cached, abort_mask=self.mask,
                           free_pages=self.free, free_count=self.count, free_left=self.count, page_tags=self.live)

    def fill(self, n):
        """Inputs of a step of n[r] drafted tokens: trees, and paths that are kept."""
        import torch
        self.n = np.asarray(n)
        trees = [T.random_tree(self.rng, int(k)) for k in n]
        self.sets = [m for t in trees for m in t] + [0] * (self.N - int(self.n.sum()))
        depth = np.array([bin(m).count("1") - 1 for m in self.sets])
        place = np.concatenate([np.arange(k) for k in n] + [np.full(self.N - int(self.n.sum()), -1)])
        self.back.copy_(dev((place - depth).astype(np.int32)))
        self.tree.copy_(dev(T.words_of(self.sets, 1)[:, 0].view(np.int64)))
        self.qkv.copy_(dev(W.bf16_bits(self.rng.standard_normal(self.qkv.shape).astype(np.float32)), dtype=torch.bfloat16))
        self.new.copy_(dev(self.n.astype(np.int32)))
        acc, kept = np.full(self.acc.shape, -1, np.int32), np.zeros(self.B, np.int32)
        for r, t in enumerate(trees):
            if t:
                leaf = t[int(self.rng.integers(len(t)))]            # a node's ancestors, some of them
                path = [j for j in range(len(t)) if (leaf >> j) & 1][:int(self.rng.integers(0, len(t) + 1))]
                acc[r, :len(path)], kept[r] = path, len(path)
        self.acc.copy_(dev(acc))
        self.kept.copy_(dev(kept))
        self.keeps = kept

    def host(self, t):
        import torch
        if t.dtype == torch.bfloat16:
            return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)
        return t.cpu().numpy()

    def check_attention(self):
        scales = (None, None) if self.kind == "bf16" else (self.ks, self.vs)
        want, vmax, written = T.tree_attention(self.host(self.qo), self.host(self.kc), self.host(self.vc), self.kind, *scales, self.host(self.ptr),
                                               self.host(self.idx), self.host(self.step), self.host(self.tptr), self.sets, D ** -0.5, self.window, self.sinks,
                                               self.host(self.mask))
        err = np.abs(bf16_out(self.out) - want)[written]
        # as in the attention's own tests
        assert (err <= (2.0 ** -8 * np.abs(want) + (2.0 ** -11 + 2.0 ** -12) * vmax)[written]).all()

    def values(self, r, t):
        """K and V of request r's tokens t, as the cache holds them."""
        pg = self.host(self.table)[r][t // self.S]
        return [self.host(c)[pg, :, t % self.S] for c in (self.kc, self.vc)]


@pytest.mark.parametrize("kind,B,Hq,H,S,drafts,window,sinks", [("fp8", 5, 16, 2, 16, 9, 0, 0), ("bf16", 3, 8, 1, 32, 20, 25, 3), ("fp4", 33, 8, 2, 16, 5, 0, 0)])
def test_serving_loop(kind, B, Hq, H, S, drafts, window, sinks):
    import torch
    import fp8_paged_kv_decode_gb300 as fkv
    fkv.device_error()
    s = Loop(kind, B, Hq, H, S, drafts, pool=B * 14, blocks=14, seed=B, window=window, sinks=sinks)
    lens = s.rng.integers(0, 4 * S, B)
    s.buffers(int(lens.sum()) + 2)                                # the prompts
    s.sets, s.back[:] = None, 0
    s.new.copy_(dev(lens.astype(np.int32)))
    s.qkv.copy_(dev(W.bf16_bits(s.rng.standard_normal(s.qkv.shape).astype(np.float32)), dtype=torch.bfloat16))
    s.calls(attend=False)
    assert s.cached.tolist() == lens.tolist()
    s.buffers(B * drafts + 3)
    graph = None
    for step in range(6):
        n = s.rng.integers(0, drafts + 1, B)
        s.fill(n)
        s.out.fill_(float("nan"))
        if step < 3:
            s.calls()
        else:
            if graph is None:
                torch.cuda.synchronize()
                graph = torch.cuda.CUDAGraph()
                kept = [x.clone() for x in (s.cached, s.table, s.btags, s.free, s.count, s.live, s.kc, s.vc)]
                with torch.cuda.graph(graph):
                    s.calls()
                for x, y in zip((s.cached, s.table, s.btags, s.free, s.count, s.live, s.kc, s.vc), kept):
                    assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))      # a capture runs nothing
            graph.replay()
        assert s.refused.sum() == 0 and s.mask.sum() == 0 and s.cached.tolist() == (lens + n).tolist()
        s.check_attention()
        acc = s.host(s.acc)
        want = [s.values(r, lens[r] + acc[r, :k]) for r, k in enumerate(s.keeps)]
        s.commit()
        lens = lens + s.keeps
        assert s.cached.tolist() == lens.tolist()
        for r, k in enumerate(s.keeps):
            for g, w in zip(s.values(r, lens[r] - k + np.arange(k)), want[r]):
                assert np.array_equal(g, w)
        # every page is on the list or held by one request
        left = int(s.count.item())
        held = [p for r in range(B) for p in s.host(s.table)[r][:-(-int(lens[r]) // S)]]
        assert sorted(held + s.host(s.free)[:left].tolist()) == list(range(s.P))
    assert fkv.device_error() == 0


def test_a_page_given_back_fails_its_old_holder():
    """The tag of a page that a commit gave back is another one: who still lists it is aborted, and its rows are zeros."""
    import torch
    import fp8_paged_kv_decode_gb300 as fkv
    s = Loop("fp8", 2, 8, 2, 16, 20, pool=12, blocks=6, seed=7)
    s.buffers(40)
    s.fill([20, 20])
    s.calls()
    ptr, idx, exp, step = (x.clone() for x in (s.ptr, s.idx, s.exp, s.step))
    s.acc[0, :2], s.kept[0] = torch.tensor([0, 1], dtype=torch.int32), 2
    s.acc[1, :20], s.kept[1] = torch.arange(20, dtype=torch.int32), 20
    s.commit()
    assert s.cached.tolist() == [2, 20]
    fkv.kv_page_tag_check(s.live, ptr, idx, exp, s.mask)
    assert s.mask.tolist() == [1, 0]                              # request 0's second page is no longer its own
    fkv.paged_tree_attn(s.qo, s.kc, s.vc, ptr, idx, step, s.tptr, s.tree, D ** -0.5, s.out, s.ws, k_scale=s.kst, v_scale=s.vst, abort_mask=s.mask)
    got = bf16_out(s.out)
    assert (got[:20] == 0).all() and (np.abs(got[20:40]).max(-1) > 0).all()


def test_rotation_of_siblings_matches_their_commit():
    """A kept token's key is rotated for the position it moves to: appended there directly it has the same bytes."""
    import torch
    import fp8_paged_kv_decode_gb300 as fkv
    s = Loop("fp8", 1, 8, 2, 16, 6, pool=4, blocks=4, seed=8)
    s.buffers(6)
    s.fill([6])
    s.sets = [0b1, 0b11, 0b101, 0b1001, 0b10101, 0b110101]        # 0 - 2 - 4 - 5, with 1 and 3 beside 2
    depth = np.array([0, 1, 1, 1, 2, 3])
    s.back.copy_(dev((np.arange(6) - depth).astype(np.int32)))
    s.acc[0, :4], s.kept[0] = torch.tensor([0, 2, 4, 5], dtype=torch.int32), 4
    s.calls(attend=False)
    s.commit()
    got = s.values(0, np.arange(4))
    x = s.qkv[[0, 2, 4, 5]]
    q, k, v = (y.unflatten(1, (-1, D)) for y in x.split((8 * D, 2 * D, 2 * D), 1))
    kc, vc = torch.zeros_like(s.kc), torch.zeros_like(s.vc)
    fkv.kv_append_rope(None, k, v, torch.arange(4, dtype=torch.int32, device="cuda"), s.freq, torch.arange(4, device="cuda"), None, kc, vc, k_scale=s.kst,
                       v_scale=s.vst, k_weight=s.w)
    for g, c in zip(got, (kc, vc)):
        assert np.array_equal(g, s.host(c)[0, :, :4].transpose(1, 0, 2))


# ---- what the marshalling does besides its checks ----
@contextlib.contextmanager
def entry_points(address):
    import fp8_paged_kv_decode_gb300 as fkv
    mod, lib = fkv._load_bind(), fkv.load_library()
    own = [ctypes.cast(getattr(lib, f), ctypes.c_void_p).value for f in fkv._BIND_CALLS]
    mod.setup(fkv.FkvError, own[0], *[address] * (len(own) - 1))
    try:
        yield
    finally:
        mod.setup(fkv.FkvError, *own)


def calls(stream):
    import torch
    import fp8_paged_kv_decode_gb300 as fkv
    z = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt, device="cuda")   # noqa: E731
    i32 = lambda *s: z(*s, dt=torch.int32)                                       # noqa: E731
    kc, sc, q, k = z(4, 2, 16, 72, dt=torch.uint8), z(2, dt=torch.float32) + 1, z(3, 8, D), z(3, 2, D)
    a = (q, kc, kc.clone(), i32(4), i32(3), i32(3))
    more = dict(k_scale=sc, v_scale=sc, stream=stream)
    return dict(
        kv_append_rope=lambda: fkv.kv_append_rope(q, k, k, i32(3), z(64, dt=torch.float32), z(3, dt=torch.int64), q, kc, kc.clone(), **more),
        paged_tree_attn=lambda: fkv.paged_tree_attn(*a, i32(4), z(3, dt=torch.int64), 0.1, q.clone(), z(256, dt=torch.uint8), **more),
        paged_window_attn=lambda: fkv.paged_window_attn(*a, 0.1, q.clone(), z(256, dt=torch.uint8), 4, 1, **more),
        kv_tree_commit=lambda: fkv.kv_tree_commit(kc, kc.clone(), i32(4), i32(3), i32(3), i32(4), i32(3, 2), i32(3), i32(3), stream=stream))


class OddStream:
    cuda_stream = "not a handle"


def test_lock_and_streams():
    """The calls run with the interpreter lock released (CPython's own check of it stands in for them: 0, not held, is
    success), and a stream that is none is refused."""
    import fp8_paged_kv_decode_gb300 as fkv
    check = ctypes.cast(ctypes.pythonapi.PyGILState_Check, ctypes.c_void_p).value
    with entry_points(check):
        for f in calls(None).values():
            f()
        for stream in (2 ** 70, OddStream(), "a stream", object()):
            for f in calls(stream).values():
                with pytest.raises(fkv.FkvError, match="stream"):
                    f()
