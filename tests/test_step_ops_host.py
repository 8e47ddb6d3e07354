"""The 4-bit cache, read-back, head norms with rotation and step tables on the
CPU: what the references say about themselves, and the calls' refusals."""
import ctypes

import numpy as np
import pytest

import fp8_paged_kv_decode_gb300 as fkv
import step_ref as R
from fp8_paged_kv_decode_gb300 import _build
from fp8_paged_kv_decode_gb300 import workloads as W


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return fkv.load_library()


# ---- the references ----
def test_e4m3_table():
    assert R.E4M3[0x7E] == 448 and R.E4M3[1] == 2.0 ** -9 and R.E4M3[0x38] == 1.0 and np.isnan(R.E4M3[0x7F])
    assert (np.diff(R.E4M3[:127]) > 0).all()


def test_fp4_ties_and_saturation():
    # scale 1 / 6 and a block maximum of 6 make s = 1 (6 / 1) and D = 1 / 6 exactly representable apart:
    # take g = 1 and amax 6, so s = 1, D = 1 and codes are the values themselves
    vals = [6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.25, -0.75, -5.0, 0.0, -0.0, 0.2578125, 4.96875, -6]
    x = np.tile(np.array(vals, np.float32), 8).reshape(1, 1, 128)
    rows = R.fp4_encode(W.bf16_bits(x), np.ones(1, np.float32))
    assert (rows[0, 0, 64:] == 0x38).all()
    got = R.fp4_values(rows)[0, 0, :16]
    want = [6, 0, 1, 1, 2, 2, 4, 4, -0.0, -1, -4, 0, -0.0, 0.5, 4, -6]
    assert np.array_equal(got, want) and np.array_equal(np.signbit(got), np.signbit(want))


def test_fp4_round_trip_error():
    rng = np.random.default_rng(0)
    x = W.bf16_bits(rng.standard_normal((64, 2, 128)).astype(np.float32))
    g = np.array([0.01, 0.013], np.float32)
    v = R.fp4_values(R.fp4_encode(x, g)) * g[None, :, None].astype(np.float64)
    f = W.bits_to_f32(x).astype(np.float64)
    a = np.abs(f).reshape(64, 2, 8, 16).max(-1).repeat(16, -1)
    # the widest code step is 2 of 6; the e4m3 block scale is off by at most 2^-4 of itself
    # (half a step of 2^-3), so the largest element may also saturate by that much
    assert (np.abs(v - f) <= a * (1 / 6 + 2.0 ** -4) * (1 + 2.0 ** -4)).all()


def test_fp4_nan_inf_and_zero_blocks():
    x = np.zeros((1, 1, 128), np.float32)
    x[0, 0, 3] = np.nan
    x[0, 0, 16] = np.inf
    x[0, 0, 17] = 1.0
    rows = R.fp4_encode(W.bf16_bits(x), np.ones(1, np.float32))
    v = R.fp4_values(rows)[0, 0]
    assert np.isnan(v[:16]).all() and v[16] == 6 * 448 and v[17] == 0 and (v[18:] == 0).all()


def test_norm_rope_reference_is_a_rotation():
    rng = np.random.default_rng(1)
    x = W.bf16_bits(rng.standard_normal((5, 3, 128)).astype(np.float32))
    f = W.bits_to_f32(x).astype(np.float64)
    for inter in (False, True):
        out, _ = R.norm_rope(x, None, rng.integers(0, 1000, (1, 5)), 10000.0 ** (-np.arange(32) / 32), None, 0.0, inter, 1.0)
        assert np.allclose((out ** 2).sum(-1), (f ** 2).sum(-1)) and np.array_equal(out[..., 64:], f[..., 64:])
    out, _ = R.norm_rope(x, None, np.full((1, 5), 0), np.ones(64), None, 0.0, False, 1.0)
    assert np.array_equal(out, f)


def test_step_tables_reference_by_hand():
    # page 4; request 0 holds 4 tokens (1 page), gets 1; request 1 holds 3, gets 1 (fits); request 2 is new with 5
    table = np.full((3, 3), -1, np.int32)
    table[0, 0], table[1, 0] = 7, 2
    tags = np.zeros((3, 3), np.uint32)
    tags[0, 0], tags[1, 0] = 70, 20
    live = np.arange(10).astype(np.uint32) * 11
    o = R.step_tables([4, 3, 0], [1, 1, 5], table, tags, np.array([5, 9, 1], np.int32), 3, live, 4, 8, 8,
                      np.full(8, -7, np.int32), np.full(8, 9, np.uint32))
    assert o["indptr"].tolist() == [0, 2, 3, 5] and o["indices"].tolist() == [7, 1, 2, 9, 5, -7, -7, -7]
    assert o["expected"].tolist() == [70, 11, 20, 99, 55, 9, 9, 9]
    assert o["slots"].tolist() == [4, 11, 36, 37, 38, 39, 20, -1] and o["positions"].tolist() == [4, 3, 0, 1, 2, 3, 4, 0]
    assert o["step_lens"].tolist() == [5, 4, 5] and int(o["free_left"][0]) == 0 and not o["bad"]
    o = R.step_tables([4, 3, 0], [1, 1, 5], table, tags, np.array([5, 9, 1], np.int32), 2, live, 4, 8, 8,
                      np.full(8, -7, np.int32), np.full(8, 9, np.uint32))
    assert o["refused"].tolist() == [0, 0, 1] and o["indices"].tolist()[:5] == [7, 9, 2, -1, -1]
    assert int(o["free_left"][0]) == 1 and o["step_lens"].tolist() == [5, 4, 0] and o["cached_out"].tolist() == [5, 4, 0]


# ---- refusals: checked before anything touches the device ----
X = 1 << 20          # an aligned address that no refused call follows


def test_append_fp4_refusals(lib):
    f = lib.kv_append_fp4
    assert f(None, None, None, 0, None, None, None, None, 4, 2, 16, 64, None) == 2
    assert f(None, None, None, -1, None, None, None, None, 4, 2, 16, 128, None) == 1
    assert f(None, None, None, 0, None, None, None, None, 4, 2, 16, 128, None) == 0
    assert f(X, X, X, 1, None, X, X, X, 4, 2, 16, 128, None) == 1           # no scale
    assert f(X + 8, X, X, 1, X, X, X, X, 4, 2, 16, 128, None) == 1          # alignment
    assert f(X, X, None, 1, X, X, X, X, 4, 2, 16, 128, None) == 1
    t = lib.kv_append_fp4_tag_check
    assert t(None, None, None, 0, None, None, None, None, 4, 2, 16, 128, None, None, None, None, -1, 0, None, None) == 1
    assert t(None, None, None, 0, None, None, None, None, 4, 2, 16, 128, None, None, None, None, 3, 0, None, None) == 1
    assert t(None, None, None, 0, None, None, None, None, 4, 2, 16, 128, None, None, None, None, 0, 0, None, None) == 0


def test_gather_refusals(lib):
    f = lib.kv_gather
    assert f(X, X, 3, X, X, X, 1, X, X, 4, 2, 16, 128, None) == 1           # no such format
    assert f(X, X, 2, X, X, X, 1, X, X, 4, 2, 16, 64, None) == 2
    assert f(X, X, 2, X, X, X, -1, X, X, 4, 2, 16, 128, None) == 1
    assert f(X, X, 2, None, X, X, 1, X, X, 4, 2, 16, 128, None) == 1
    assert f(X, X, 1, None, None, X, 1, X, X + 8, 4, 2, 16, 128, None) == 1
    assert f(X, X, 1, None, None, X, 1, X, X, 4, 0, 16, 128, None) == 1
    assert f(None, None, 2, None, None, None, 0, None, None, 4, 2, 16, 128, None) == 0


def rope_args(**over):
    a = dict(q=X, qs=1024, hq=8, k=X, ks=256, hkv=2, qo=X, qos=1024, ko=X, kos=256, n=1, qw=X, kw=X, eps=1e-6, pos=X,
             axes=1, freq=X, map=None, rot=128, inter=0, scale=1.0, dim=128, stream=None)
    a.update(over)
    return list(a.values())


@pytest.mark.parametrize("want,over", [
    (2, dict(dim=64)), (1, dict(n=-1)), (1, dict(hq=0)), (2, dict(rot=24)), (2, dict(rot=144)), (2, dict(rot=0)),
    (1, dict(axes=0)), (2, dict(axes=9)), (1, dict(eps=-1.0)), (1, dict(eps=float("nan"))),
    (1, dict(scale=float("inf"))), (1, dict(qs=1016)), (1, dict(qs=1028)), (1, dict(kos=128)), (1, dict(q=X + 8)),
    (1, dict(ko=None)), (1, dict(pos=None)), (1, dict(freq=None)), (1, dict(qw=X + 2)), (0, dict(n=0)),
    (0, dict(n=0, q=None, k=None))])
def test_rope_refusals(lib, want, over):
    assert lib.qk_norm_rope(*rope_args(**over)) == want


def tables_args(lib, **over):
    n = lib.kv_step_tables_workspace_size(2)
    a = dict(c=X, n=X, b=2, table=X, tags=X, m=4, free=X, nfree=3, count=X, live=X, pages=8, page=16, step=X, out=X,
             refused=X, ptr=X, idx=X, exp=X, nnz=8, tptr=X, slots=X, pos=X, ntok=4, left=X, ws=X, wsn=n, stream=None)
    a.update(over)
    return list(a.values())


@pytest.mark.parametrize("over", [dict(b=-1), dict(m=0), dict(page=0), dict(pages=0), dict(nnz=-1), dict(ntok=-1),
                                  dict(nfree=-1), dict(c=None), dict(table=None), dict(free=None), dict(count=None),
                                  dict(idx=None), dict(slots=None), dict(ws=None), dict(ws=X + 16), dict(wsn=16),
                                  dict(left=None), dict(ptr=None), dict(refused=None)])
def test_tables_refusals(lib, over):
    assert lib.kv_step_tables(*tables_args(lib, **over)) == 1


def test_attention_knows_the_format(lib):
    P = ctypes.c_void_p
    args = [None, 2, 8, None, None, 2, None, None, 4, 2, 16, 128, None, None, 0, None, None, 0.1, None, None, 0, P(0)]
    assert lib.paged_decode_attn(*args) == 1                   # FP4: null pointers
    args[8:11] = [4, 300000, 128]
    args[2] = 300000
    assert lib.paged_decode_attn(*args) == 2                   # a page of 300000 heads' rows
    args[5] = 3
    assert lib.paged_decode_attn(*args) == 1                   # no such format
    assert lib.paged_decode_attn_workspace_size(2, 8, 2, 128, 3) == 0
    assert lib.kv_page_realloc(X, 4, X, 1, X, X, X, 3, 2, 16, 128, None) == 1
    assert lib.kv_page_realloc(X, 4, X, 1, X, X, X, 2, 1, 1, 128, None) == 2     # a 72-byte page


def test_launch_counts(lib):
    for name, n in (("kv_append_fp4", 1), ("kv_append_fp4_tag_check", 1), ("kv_gather", 1), ("qk_norm_rope", 1)):
        assert fkv.kernels_per_call(name) == n
    assert fkv.kernels_per_call("kv_step_tables") in (1, 2)
