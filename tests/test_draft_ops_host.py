"""The drafted step's operators on the CPU: what their references say about themselves,
and the calls' refusals."""
import numpy as np
import pytest

import draft_ref as T
import fp8_paged_kv_decode_gb300 as fkv
import step_ref as R
from fp8_paged_kv_decode_gb300 import _build
from fp8_paged_kv_decode_gb300 import workloads as W

D = 128


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return fkv.load_library()


# ---- the references ----
def test_visible_by_hand():
    # six committed tokens, a root (0), its children 1 and 2, 3 below 1
    sets = [0b1, 0b11, 0b101, 0b1011]
    see = T.visible(sets, 4, 6, 0, 0)
    assert see[:, :6].all() and see[:, 6:].astype(int).tolist() == [[1, 0, 0, 0], [1, 1, 0, 0], [1, 0, 1, 0], [1, 1, 0, 1]]
    see = T.visible(sets, 4, 6, 3, 1)          # the root stands at 6 and sees 4, 5 of the committed ones, and the first
    assert see[:, :6].astype(int).tolist() == [[1, 0, 0, 0, 1, 1], [1, 0, 0, 0, 0, 1], [1, 0, 0, 0, 0, 1], [1, 0, 0, 0, 0, 0]]


def test_a_chain_is_decode_attention():
    """The last row of a chain of drafted tokens is the decode step's row over all of them."""
    rng = np.random.default_rng(0)
    kc, ks = T.pool(rng, "fp4", 4, 2, 16)
    vc, vs = T.pool(rng, "fp4", 4, 2, 16)
    q = W.bf16_bits(rng.standard_normal((3, 8, D)).astype(np.float32))
    ptr, idx = np.array([0, 3], np.int32), np.array([2, 0, 3], np.int32)
    out, _, _ = T.tree_attention(q, kc, vc, "fp4", ks, vs, ptr, idx, [40], [0, 3], [1, 3, 7], 0.1)
    for i in range(3):
        want, _ = R.attention(q[i:i + 1], kc, vc, ks, vs, ptr, idx, [38 + i], 0.1)
        assert np.allclose(out[i], want[0])


def test_commit_by_hand():
    kc = np.arange(3 * 1 * 4 * 2).reshape(3, 1, 4, 2)
    vc = kc + 100
    # pages 2, 0, 1 of 4 tokens; 3 committed, 7 drafted; kept: 1, 4, 5
    got = T.commit(kc, vc, 4, [0, 3], np.array([2, 0, 1]), [10], [0, 7], np.array([[1, 4, 5]]), [3], np.array([10]), None,
                   np.array([-1, -1, -1]), 0, np.array([5, 6, 7]))
    flat = lambda c: c[[2, 0, 1], 0].reshape(12, 2)                   # noqa: E731
    want = flat(kc).copy()
    want[[3, 4, 5]] = flat(kc)[[4, 7, 8]]
    assert np.array_equal(flat(got[0]), want) and np.array_equal(flat(got[1]), want + 100)
    assert got[2].tolist() == [6] and got[3].tolist() == [1, -1, -1] and got[4] == 1 and got[5].tolist() == [5, 7, 7] and not got[6]


# ---- refusals (nothing is launched) ----
A = 4096                                          # an address that is never followed


def rope(lib, **k):
    a = dict(q=A, qs=1024, hq=8, k=A, ks=256, v=A, vs=256, hkv=2, qo=A, qos=1024, n=0, qw=None, kw=None, eps=1e-6, pos=A, axes=1, freq=A,
             amap=None, rot=128, inter=0, rs=1.0, slots=A, kv=0, sk=A, sv=A, kc=A, vc=A, pages=4, page=16, d=128)
    a.update(k)
    return lib.kv_append_rope(*a.values(), None)


def test_rope_append_refusals(lib):
    assert rope(lib) == 0
    for bad in (dict(n=-1), dict(hq=-1), dict(hkv=0), dict(axes=0), dict(pages=0), dict(page=0), dict(kv=3), dict(eps=-1.0), dict(eps=float("nan")),
                dict(rs=float("inf")), dict(qs=1016), dict(qs=1028), dict(ks=248), dict(vs=248), dict(qos=1000)):
        assert rope(lib, **bad) == 1, bad
    for bad in (dict(d=64), dict(axes=9), dict(rot=8), dict(rot=144), dict(rot=40), dict(hkv=40000, ks=40000 * 128, vs=40000 * 128)):
        assert rope(lib, **bad) == 2, bad
    for bad in (dict(q=None), dict(qo=None), dict(k=None), dict(v=None), dict(pos=None), dict(freq=None), dict(slots=None), dict(sk=None), dict(sv=None),
                dict(kc=None), dict(vc=None), dict(q=A + 8), dict(k=A + 2), dict(v=A + 8), dict(kc=A + 8), dict(qw=A + 8)):
        assert rope(lib, n=3, **bad) == 1, bad


def tree(lib, **k):
    a = dict(q=A, n=4, hq=8, kc=A, vc=A, kv=0, sk=A, sv=A, pages=4, hkv=2, page=16, d=128, ptr=A, idx=A, nnz=4, lens=A, batch=0, tptr=A, mask=A, words=1,
             window=0, sinks=0, abort=None, sm=0.1, out=A, ws=A, size=1 << 40)
    a.update(k)
    return lib.paged_tree_attn(*a.values(), None)


def window(lib, **k):
    a = dict(q=A, batch=0, hq=8, kc=A, vc=A, kv=0, sk=A, sv=A, pages=4, hkv=2, page=16, d=128, ptr=A, idx=A, nnz=4, lens=A, window=5, sinks=0, abort=None,
             sm=0.1, out=A, ws=A, size=1 << 40)
    a.update(k)
    return lib.paged_window_attn(*a.values(), None)


def test_attention_refusals(lib):
    for call in (tree, window):
        assert call(lib) == 0
        for bad in (dict(batch=-1), dict(hq=0), dict(hq=7), dict(hkv=0), dict(pages=0), dict(nnz=-1), dict(kv=3), dict(sm=0.0), dict(sm=-1.0),
                    dict(sm=float("nan")), dict(window=-1), dict(sinks=-1)):
            assert call(lib, **bad) == 1, bad
        for bad in (dict(d=64), dict(page=24), dict(page=256), dict(hq=258)):
            assert call(lib, **bad) == 2, bad
        for bad in (dict(q=None), dict(kc=None), dict(vc=None), dict(ptr=None), dict(idx=None), dict(lens=None), dict(out=None), dict(ws=None),
                    dict(sk=None), dict(sv=None), dict(q=A + 8), dict(out=A + 8), dict(kc=A + 8), dict(ws=A + 128)):
            assert call(lib, batch=2, **bad) == 1, bad
    assert tree(lib, n=-1) == 1 and tree(lib, words=0) == 1 and tree(lib, words=-1) == 1 and tree(lib, words=5) == 2
    assert tree(lib, batch=2, tptr=None) == 1 and tree(lib, batch=2, mask=None) == 1 and tree(lib, batch=2, n=0) == 0
    assert window(lib, window=0) == 1
    size = lib.paged_tree_attn_workspace_size
    assert size(4, 2, 7, 2, 128, 0) == 0 and size(4, 2, 8, 2, 64, 0) == 0 and size(4, 2, 8, 2, 128, 3) == 0 and size(-1, 2, 8, 2, 128, 0) == 0
    assert size(4, 2, 258, 2, 128, 0) == 0


def commit(lib, **k):
    a = dict(kc=A, vc=A, kv=0, pages=4, hkv=2, page=16, d=128, ptr=A, idx=A, nnz=4, lens=A, batch=0, tptr=A, n=4, acc=A, most=3, counts=A, abort=None,
             out=2 * A, free=None, num=0, count=None, left=None, tags=None)
    a.update(k)
    return lib.kv_tree_commit(*a.values(), None)


def test_commit_refusals(lib):
    assert commit(lib) == 0
    for bad in (dict(batch=-1), dict(n=-1), dict(pages=0), dict(hkv=0), dict(page=0), dict(nnz=-1), dict(most=-1), dict(num=-1), dict(kv=3),
                dict(free=A), dict(free=A, num=3, count=A), dict(free=A, num=3, left=A), dict(num=3, count=A, left=A), dict(tags=A)):
        assert commit(lib, **bad) == 1, bad
    assert commit(lib, d=64) == 2 and commit(lib, hkv=40000) == 2
    for bad in (dict(kc=None), dict(vc=None), dict(ptr=None), dict(idx=None), dict(lens=None), dict(tptr=None), dict(acc=None), dict(counts=None),
                dict(out=None), dict(out=A), dict(kc=A + 8)):
        assert commit(lib, batch=2, **bad) == 1, bad


def test_launch_counts(lib):
    assert fkv.kernels_per_call("kv_append_rope") == 1 and fkv.kernels_per_call("kv_tree_commit") == 1
    assert fkv.kernels_per_call("paged_tree_attn") == fkv.kernels_per_call("paged_window_attn") > 0


def test_commit_refuses_lengths_over_what_it_reads(lib):
    """Other warps still read a request's count, list and length when one of them writes its kept length."""
    for name in ("lens", "counts", "acc"):
        assert commit(lib, batch=2, **{name: 7 * A, "out": 7 * A}) == 1, name


@pytest.mark.parametrize("ctx,window,sinks", [(6, 4, 1), (0, 3, 0), (1, 3, 3), (20, 1, 2), (3, 9, 0), (5, 30, 0)])
def test_a_chain_deeper_than_the_window(ctx, window, sinks):
    """Drafted tokens are seen by their bits alone: with those of the ancestors unset that a sliding window leaves out, each row is
    the windowed decode step's of its token."""
    rng = np.random.default_rng(1)
    n = 9
    kc, ks = T.pool(rng, "fp8", 4, 2, 16)
    vc, vs = T.pool(rng, "fp8", 4, 2, 16)
    q = W.bf16_bits(rng.standard_normal((n, 8, D)).astype(np.float32))
    ptr, idx = np.array([0, 3], np.int32), np.array([2, 0, 3], np.int32)
    sets = [sum(1 << j for j in range(i + 1) if i - j < window or ctx + j < sinks) for i in range(n)]
    out, _, _ = T.tree_attention(q, kc, vc, "fp8", ks, vs, ptr, idx, [ctx + n], [0, n], sets, 0.1, window, sinks)
    for i in range(n):
        see = T.visible([1], 1, ctx + i, window, sinks)[0]
        assert see.nonzero()[0].tolist() == [t for t in range(ctx + i + 1) if t < sinks or t > ctx + i - window]
        want, _, _ = T.tree_attention(q[i:i + 1], kc, vc, "fp8", ks, vs, ptr, idx, [ctx + i + 1], [0, 1], [1], 0.1, window, sinks)
        assert np.allclose(out[i], want[0])
