"""kv_step_tables on the GPU against the one-request-at-a-time reference."""
import numpy as np
import pytest

import step_ref as R
from gpu_util import dev

pytestmark = pytest.mark.gpu


class Tables:
    def __init__(self, cached, new, page, blocks, pool, free, nnz, n_tokens, seed=0, free_count=None):
        rng = np.random.default_rng(seed)
        self.cached, self.new = np.asarray(cached, np.int32), np.asarray(new, np.int32)
        self.page, self.nnz, self.n_tokens = page, nnz, n_tokens
        B = len(self.cached)
        self.table = rng.integers(0, pool, (B, blocks)).astype(np.int32)
        self.tags = rng.integers(0, 2 ** 32, (B, blocks), dtype=np.uint64).astype(np.uint32)
        self.free = rng.permutation(pool).astype(np.int32)[:free] if free <= pool else rng.integers(0, pool, free).astype(np.int32)
        self.free_count = np.array([len(self.free) if free_count is None else free_count], np.int32)
        self.live = rng.integers(0, 2 ** 32, pool, dtype=np.uint64).astype(np.uint32)

    def run(self, alias=False, into=None, stream=None):
        import torch
        import fp8_paged_kv_decode_gb300 as fkv
        B = len(self.cached)
        t = into if into is not None else self.tensors()
        if alias:
            t["cached_out"], t["free_left"] = t["cached"], t["free_count"]
        fkv.kv_step_tables(t["cached"], t["new"], t["table"], t["table_tags"], t["free"], t["free_count"], t["live"], self.page,
                           t["step_lens"], t["cached_out"], t["refused"], t["indptr"], t["indices"], t["expected"], t["token_indptr"],
                           t["slots"], t["positions"], t["free_left"], t["ws"], stream=stream)
        torch.cuda.synchronize()
        assert t["step_lens"].numel() == B
        return t

    def tensors(self):
        import torch
        import fp8_paged_kv_decode_gb300 as fkv
        B = len(self.cached)
        full = lambda n, v, dt=torch.int32: torch.full((n,), v, dtype=dt, device="cuda")     # noqa: E731
        return dict(cached=dev(self.cached), new=dev(self.new), table=dev(self.table), table_tags=dev(self.tags.view(np.int32)), free=dev(self.free),
                    free_count=dev(self.free_count), live=dev(self.live.view(np.int32)), step_lens=full(B, -9), cached_out=full(B, -9),
                    refused=full(B, 9, torch.uint8), indptr=full(B + 1, -9), indices=full(self.nnz, -7), expected=full(self.nnz, -7),
                    token_indptr=full(B + 1, -9), slots=full(self.n_tokens, -9, torch.int64), positions=full(self.n_tokens, -9), free_left=full(1, -9),
                    ws=fkv.alloc_step_tables_workspace(B))

    def want(self):
        return R.step_tables(self.cached, self.new, self.table, self.tags, self.free, self.free_count[0], self.live, self.page, self.nnz, self.n_tokens,
                             np.full(self.nnz, -7, np.int32), np.full(self.nnz, -7, np.int32).view(np.uint32))

    def check(self, **kw):
        import fp8_paged_kv_decode_gb300 as fkv
        fkv.device_error()
        t, w = self.run(**kw), self.want()
        for name, v in w.items():
            if name == "bad":
                continue
            got = t[name].cpu().numpy()
            got = got.view(v.dtype) if got.dtype != v.dtype else got
            assert np.array_equal(got, v), (name, np.argwhere(got != v)[:5].tolist(), got[got != v][:5], v[got != v][:5])
        assert fkv.device_error() == (fkv.DEVERR_TABLES if w["bad"] else 0)
        return w


@pytest.mark.parametrize("B,page,new,far", [(1, 16, 1, 1), (3, 64, 1, 300), (64, 64, 1, 20000), (31, 16, 40, 500), (129, 128, 300, 2000),
                                            (1025, 32, 3, 100), (2500, 16, 1, 70), (7, 24, 100, 90), (5, 1, 3, 9)])
def test_against_the_reference(B, page, new, far):
    rng = np.random.default_rng(B + page)
    cached, fresh = rng.integers(0, far, B), rng.integers(0, new + 1, B) if new > 1 else np.ones(B, int)
    blocks = -(-(far + new) // page) + 1
    need = int((-(-(cached + fresh) // page) - -(-cached // page)).sum())
    nnz = int((-(-(cached + fresh) // page)).sum())
    w = Tables(cached, fresh, page, blocks, max(need, 1) + 20, need + 9, nnz + 11, int(fresh.sum()) + 7, seed=B).check()
    assert not w["bad"] and int(w["free_left"][0]) == 9


def test_cached_lengths_and_free_count_in_place():
    rng = np.random.default_rng(1)
    t = Tables(rng.integers(0, 99, 50), rng.integers(0, 9, 50), 16, 8, 400, 300, 500, 500)
    w = t.want()
    got = t.run(alias=True)
    assert np.array_equal(got["cached"].cpu().numpy(), w["cached_out"]) and got["free_count"].tolist() == w["free_left"].tolist()
    assert np.array_equal(got["slots"].cpu().numpy(), w["slots"]) and np.array_equal(got["indices"].cpu().numpy(), w["indices"])


@pytest.mark.parametrize("free_count", [0, 1, 5, 17, -3, 1000])
def test_too_few_pages(free_count):
    rng = np.random.default_rng(2)
    Tables(rng.integers(0, 50, 40), rng.integers(0, 30, 40), 16, 6, 90, 60, 400, 900, seed=3, free_count=free_count).check()


@pytest.mark.parametrize("nnz,n_tokens", [(0, 0), (10, 900), (400, 100), (57, 211), (1, 1)])
def test_too_little_room(nnz, n_tokens):
    rng = np.random.default_rng(4)
    Tables(rng.integers(0, 50, 40), rng.integers(0, 30, 40), 16, 6, 90, 90, nnz, n_tokens, seed=5).check()


def test_bad_lengths_and_rows_too_wide():
    cached = [5, -1, 3, 2 ** 31 - 1, 2 ** 31 - 2, 100, 0, 7]
    new = [1, 4, -2, 1, 1, 30, 0, 1]
    Tables(cached, new, 16, 8, 40, 30, 60, 60, seed=6).check()


def test_ids_outside_the_pool():
    rng = np.random.default_rng(7)
    t = Tables(rng.integers(0, 60, 30), rng.integers(0, 40, 30), 16, 8, 200, 150, 400, 900, seed=8)
    t.free[[3, 148, 120]] = [-1, 200, 2 ** 31 - 1]
    t.table[4, 0], t.table[9, :] = 200, -5
    assert t.check()["bad"]


def test_no_requests():
    t = Tables([], [], 16, 4, 10, 5, 3, 4)
    w = t.check()
    assert w["indptr"].tolist() == [0] and w["slots"].tolist() == [-1] * 4


def test_a_long_prompt():
    w = Tables([0, 131071, 17], [131072, 1, 2000], 16, 8200, 9000, 8900, 17000, 140000, seed=9).check()
    assert w["step_lens"].tolist() == [131072, 131072, 2017]


def test_repeated_and_replayed():
    """The same call twice, and captured once and replayed on changed lengths."""
    import torch
    rng = np.random.default_rng(10)
    t = Tables(rng.integers(0, 99, 70), rng.integers(0, 9, 70), 16, 8, 700, 600, 800, 800, seed=11)
    x = t.tensors()
    a = {k: v.clone() for k, v in t.run(into=x).items()}
    b = t.run(into=x)
    for k, v in a.items():
        assert k == "ws" or torch.equal(v, b[k]), k
    g = torch.cuda.CUDAGraph()
    y = t.tensors()
    with torch.cuda.graph(g):
        s = torch.cuda.current_stream()
        import fp8_paged_kv_decode_gb300 as fkv
        fkv.kv_step_tables(y["cached"], y["new"], y["table"], y["table_tags"], y["free"], y["free_count"], y["live"], t.page, y["step_lens"], y["cached_out"],
                           y["refused"], y["indptr"], y["indices"], y["expected"], y["token_indptr"], y["slots"], y["positions"], y["free_left"], y["ws"], stream=s)
    t.cached = rng.integers(0, 99, 70).astype(np.int32)
    y["cached"].copy_(dev(t.cached))
    g.replay()
    torch.cuda.synchronize()
    w = t.want()
    for k in ("slots", "positions", "indices", "indptr", "step_lens", "table", "free_left"):
        assert np.array_equal(y[k].cpu().numpy(), w[k]), k


def test_python_refusals():
    import fp8_paged_kv_decode_gb300 as fkv
    t = Tables([3, 4], [1, 1], 16, 4, 10, 5, 8, 8)
    for name, bad in (("cached", lambda x: x.long()), ("new", lambda x: x[:1]), ("table", lambda x: x[:1]), ("table_tags", lambda x: x[:, :2].contiguous()),
                      ("indptr", lambda x: x[:2]), ("slots", lambda x: x.int()), ("positions", lambda x: x[:3]), ("expected", lambda x: x[:3]),
                      ("refused", lambda x: x.int()), ("free_left", lambda x: x.cpu()), ("live", lambda x: x.float()), ("ws", lambda x: x[:16])):
        x = t.tensors()
        x[name] = bad(x[name])
        with pytest.raises(fkv.FkvError):
            t.run(into=x)
