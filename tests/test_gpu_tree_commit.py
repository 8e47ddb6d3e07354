"""kv_tree_commit on the GPU: the whole pools, lengths, free list and tags against the reference."""
import numpy as np
import pytest

import draft_ref as T
from gpu_util import dev

pytestmark = pytest.mark.gpu
KINDS = ["fp8", "bf16", "fp4"]


class Case:
    def __init__(self, kind, H, S, ctx, n, counts, seed, most=None, spare=9, free=None):
        rng = np.random.default_rng(seed)
        self.kind, self.S, self.rng = kind, S, rng
        self.lens = (np.asarray(ctx) + np.asarray(n)).astype(np.int32)
        self.tptr = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
        pages = -(-self.lens.astype(np.int64) // S)
        used = int(pages.sum())
        self.P = used + spare
        self.ptr = np.concatenate([[0], np.cumsum(pages)]).astype(np.int32)
        perm = rng.permutation(self.P).astype(np.int32)
        self.idx = perm[:used].copy()
        dt = np.uint16 if kind == "bf16" else np.uint8
        self.kc, self.vc = (rng.integers(0, np.iinfo(dt).max + 1, (self.P, H, S, T.ROWS[kind])).astype(dt) for _ in range(2))
        self.most = max(1, max(n, default=0)) if most is None else most
        self.counts = np.asarray(counts, np.int32)
        self.acc = rng.integers(-9, 99, (len(n), self.most)).astype(np.int32)
        for r, k in enumerate(self.counts):
            self.acc[r, :k] = np.sort(rng.permutation(int(n[r]))[:k])
        self.kept = rng.integers(0, 99, len(n)).astype(np.int32)
        self.dead = None
        self.free = np.full(self.P + 3, -7, np.int32) if free is None else np.full(free, -7, np.int32)
        self.free[:min(spare, len(self.free))] = perm[used:][:len(self.free)]
        self.count = min(spare, len(self.free))
        self.tags = rng.integers(0, 2 ** 32, self.P).astype(np.uint32)

    def ref(self, release=True):
        return T.commit(self.kc, self.vc, self.S, self.ptr, self.idx, self.lens, self.tptr, self.acc, self.counts, self.kept, self.dead,
                        self.free if release else None, self.count, self.tags if release else None)

    def run(self, release=True, tags=True, stream=None, in_place=False):
        import torch
        import fp8_paged_kv_decode_gb300 as fkv
        pool = (lambda a: dev(a, dtype=torch.bfloat16)) if self.kind == "bf16" else dev
        kc, vc, kept = pool(self.kc), pool(self.vc), dev(self.kept)
        free, count, live = dev(self.free), dev(np.array([self.count], np.int32)), dev(self.tags.view(np.int32))
        left = count if in_place else torch.full((1,), -5, dtype=torch.int32, device="cuda")
        more = dict(free_pages=free, free_count=count, free_left=left, page_tags=live if tags else None) if release else {}
        fkv.kv_tree_commit(kc, vc, dev(self.ptr), dev(self.idx), dev(self.lens), dev(self.tptr), dev(self.acc), dev(self.counts), kept,
                           abort_mask=None if self.dead is None else dev(self.dead.astype(np.uint8)), stream=stream, **more)
        torch.cuda.synchronize()
        bits = lambda t: t.view(torch.uint8).cpu().numpy()              # noqa: E731
        return bits(kc), bits(vc), kept.cpu().numpy(), free.cpu().numpy(), int(left.item()), live.cpu().numpy().view(np.uint32)

    def check(self, got, release=True, tags=True):
        want = self.ref(release)
        for g, w in zip(got[:2], want[:2]):
            assert np.array_equal(g, np.ascontiguousarray(w).view(np.uint8).reshape(g.shape))
        assert got[2].tolist() == want[2].tolist()
        if release:
            assert got[3].tolist() == want[3].tolist() and got[4] == want[4]
        assert np.array_equal(got[5], want[5] if release and tags else self.tags)
        return want[6]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("H,S,ctx,n,counts", [
    (1, 16, [0], [1], [0]), (2, 16, [0, 5, 16, 31], [1, 8, 8, 8], [1, 3, 8, 0]), (8, 64, [100, 63, 64, 65], [8] * 4, [2, 5, 1, 7]),
    (3, 32, [10, 20, 30], [61, 0, 64], [20, 0, 40]), (2, 128, [500, 127], [130, 256], [64, 256]), (1, 24, [7, 100], [33, 50], [33, 31])])
def test_moves(kind, H, S, ctx, n, counts):
    import fp8_paged_kv_decode_gb300 as fkv
    fkv.device_error()
    c = Case(kind, H, S, ctx, n, counts, seed=S + len(n))
    assert not c.check(c.run())
    assert not c.check(c.run(release=False), release=False)
    assert not c.check(c.run(tags=False), tags=False)
    assert not c.check(c.run(in_place=True))
    assert fkv.device_error() == 0


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("batch", [300, 1000])
def test_many_requests(kind, batch):
    rng = np.random.default_rng(batch)
    n = rng.integers(0, 20, batch)
    c = Case(kind, 2, 16, rng.integers(0, 60, batch), n, [int(rng.integers(0, k + 1)) for k in n], seed=batch)
    c.dead = (rng.random(batch) < 0.1).astype(np.uint8)
    assert not c.check(c.run())


def test_chains_move_nothing():
    c = Case("fp8", 2, 16, [5, 40], [6, 9], [6, 4], seed=1)
    c.acc[0, :6], c.acc[1, :4] = range(6), range(4)
    got = c.run()
    c.check(got)
    assert np.array_equal(got[0], c.kc) and np.array_equal(got[1], c.vc)


@pytest.mark.parametrize("kind", ["fp8", "fp4"])
def test_requests_left_as_they_are(kind):
    import fp8_paged_kv_decode_gb300 as fkv
    fkv.device_error()
    c = Case(kind, 2, 16, [20] * 9, [8] * 9, [3] * 9, seed=2)
    c.dead = np.zeros(9, np.uint8)
    c.dead[1] = 1
    c.lens[2] = 5                                                  # fewer tokens than drafted ones
    c.lens[3] = 60                                                 # more than its pages hold
    assert not c.check(c.run())
    assert fkv.device_error() == 0
    for change in (lambda: c.acc.__setitem__((4, slice(0, 3)), [2, 2, 5]), lambda: c.acc.__setitem__((5, slice(0, 3)), [3, 1, 5]),
                   lambda: c.acc.__setitem__((6, 2), 8), lambda: c.acc.__setitem__((7, 0), -1), lambda: c.counts.__setitem__(8, 9),
                   lambda: c.counts.__setitem__(0, -1), lambda: c.idx.__setitem__(c.ptr[0] + 1, c.P)):
        change()
        assert c.check(c.run())
        assert fkv.device_error() == fkv.DEVERR_TREE
    c = Case(kind, 2, 16, [20] * 3, [8] * 3, [3] * 3, seed=3)
    c.ptr[1] = -1
    assert not c.check(c.run())
    c = Case(kind, 2, 16, [20] * 3, [8] * 3, [3] * 3, seed=3)
    c.tptr[:] = [0, 8, 4, 12]
    c.check(c.run())
    fkv.device_error()


def test_a_list_without_room():
    import fp8_paged_kv_decode_gb300 as fkv
    fkv.device_error()
    c = Case("fp8", 1, 16, [20] * 6, [40] * 6, [3] * 6, seed=4, free=14)
    assert c.check(c.run())
    assert fkv.device_error() == fkv.DEVERR_TREE
    c = Case("fp8", 1, 16, [20] * 6, [40] * 6, [3] * 6, seed=4, free=21)      # just enough: 9 and 12
    assert not c.check(c.run())
    c.count = -4                                                   # counts outside the list are cut to it
    assert not c.check(c.run())
    c.count = 99
    assert c.check(c.run())
    fkv.device_error()


def test_no_requests():
    import torch
    import fp8_paged_kv_decode_gb300 as fkv
    z = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")              # noqa: E731
    pool, left = torch.zeros(4, 2, 16, 128, dtype=torch.uint8, device="cuda"), z(1) - 1
    fkv.kv_tree_commit(pool, pool.clone(), z(1), z(0), z(0), z(1), z(0, 3), z(0), z(0), free_pages=z(5), free_count=z(1) + 3, free_left=left)
    assert left.item() == 3
    fkv.kv_tree_commit(pool, pool.clone(), z(1), z(0), z(0), z(1), z(0, 3), z(0), z(0))


def test_python_refusals():
    import torch
    import fp8_paged_kv_decode_gb300 as fkv
    z = lambda *s, dt=torch.int32: torch.zeros(*s, dtype=dt, device="cuda")       # noqa: E731
    pool = z(4, 2, 16, 128, dt=torch.uint8)
    a = dict(k_cache=pool, v_cache=pool.clone(), page_indptr=z(3), page_indices=z(4), seq_lens=z(2), token_indptr=z(3), accepted=z(2, 3), accepted_counts=z(2),
             lens_out=z(2), abort_mask=None, free_pages=z(5), free_count=z(1), free_left=z(1), page_tags=z(4))
    for bad in (dict(v_cache=pool[:2]), dict(v_cache=pool.float()), dict(seq_lens=z(3)), dict(seq_lens=z(2, dt=torch.int64)), dict(token_indptr=z(2)),
                dict(accepted=z(6)), dict(accepted=z(3, 3)), dict(accepted=z(2, 6)[:, ::2]), dict(accepted_counts=z(1)), dict(lens_out=z(1)),
                dict(abort_mask=z(2)), dict(free_left=None), dict(free_pages=None), dict(free_count=z(2)), dict(page_tags=z(3)),
                dict(page_tags=z(4, dt=torch.int64)), dict(lens_out=a["seq_lens"]), dict(k_cache=pool.cpu())):
        with pytest.raises(fkv.FkvError):
            fkv.kv_tree_commit(**dict(a, **bad))
