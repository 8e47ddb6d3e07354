"""The kernels that large calls take: several tokens a thread in the 4-bit append
and the read-back, several batches of rows a warp in the head norms.  Sizes
are past the switch on any GPU of up to 160 SMs, with ragged ends."""
import numpy as np
import pytest

import step_ref as R
from fp8_paged_kv_decode_gb300 import workloads as W
from gpu_util import bf16_out, dev
from test_gpu_fp4 import ROW, same_rows
from test_gpu_rope import bits, check

pytestmark = pytest.mark.gpu
D = 128


def scattered(rng, n, P, S):
    """n different slots in random order, with padding and slots past the pool between them."""
    slots = rng.permutation(P * S)[:n].astype(np.int64)
    slots[rng.permutation(n)[:n // 20]] = -1
    past = rng.permutation(n)[:n // 50]
    slots[past] = P * S + rng.integers(0, 2 ** 40, len(past))
    slots[-1] = P * S
    return slots


@pytest.mark.parametrize("n,H,S", [(4099, 8, 64), (4099, 8, 24), (10307, 3, 16), (64 * 165 + 33, 3, 128), (33000, 1, 1)])
def test_append_fp4(n, H, S):
    """64 tokens to a block: two per thread, the last group partly or wholly empty."""
    import torch
    import fp8_paged_kv_decode_gb300 as fkv
    rng = np.random.default_rng(n + S)
    assert -(-n // 64) * 2 * H >= 6 * 160
    P = -(-n // S) + 3
    k, v = (W.bf16_bits((rng.standard_normal((n, H, D)) * 10.0 ** rng.integers(-2, 2, (n, H, 1))).astype(np.float32)) for _ in range(2))
    ks, vs = (np.exp(rng.uniform(-6, 0, H)).astype(np.float32) for _ in range(2))
    slots = scattered(rng, n, P, S)
    fill = rng.integers(0, 256, (P, H, S, ROW)).astype(np.uint8)
    a = [dev(k, dtype=torch.bfloat16), dev(v, dtype=torch.bfloat16), dev(slots), dev(ks), dev(vs)]
    pools = [dev(fill) for _ in range(4)]
    fkv.device_error()
    fkv.kv_append_fp4(*a, *pools[:2])
    assert fkv.device_error() == fkv.DEVERR_APPEND_SLOT
    ok = np.flatnonzero((slots >= 0) & (slots < P * S))
    for t, x, sc in zip(pools, (k, v), (ks, vs)):
        want = fill.copy()
        want[slots[ok] // S, :, slots[ok] % S] = R.fp4_encode(x, sc)[ok]
        assert same_rows(t.cpu().numpy(), want)
    # the append and the check in one launch: the same bytes
    z = lambda m: torch.zeros(m, dtype=torch.int32, device="cuda")               # noqa: E731
    mask = torch.full((1,), 7, dtype=torch.uint8, device="cuda")
    fkv.kv_append_fp4_tag_check(*a, *pools[2:], z(P), z(2), z(0), z(0), mask)
    assert mask.tolist() == [0] and fkv.device_error() == fkv.DEVERR_APPEND_SLOT
    assert torch.equal(pools[0], pools[2]) and torch.equal(pools[1], pools[3])


@pytest.mark.parametrize("kind", ["fp4", "fp8", "bf16"])
@pytest.mark.parametrize("n,H,S", [(10300, 8, 64), (27400, 3, 24), (128 * 645 + 97, 1, 16)])
def test_gather(kind, n, H, S):
    """128 tokens to a block, four per thread."""
    import torch
    import fp8_paged_kv_decode_gb300 as fkv
    rng = np.random.default_rng(n + len(kind))
    assert 2 * n * H >= 160 * 8 * 32 * 4
    P = 200
    shape = (P, H, S, ROW if kind == "fp4" else D)
    ks, vs = (np.exp(rng.uniform(-6, 1, H)).astype(np.float32) for _ in range(2))
    if kind == "bf16":
        kc, vc = (W.bf16_bits(rng.standard_normal(shape).astype(np.float32)) for _ in range(2))
    else:
        kc, vc = (rng.integers(0, 256, shape).astype(np.uint8) for _ in range(2))      # every code, NaN among them
    slots = rng.integers(0, P * S, n).astype(np.int64)                                 # repeats
    slots[rng.permutation(n)[:n // 20]] = -1
    slots[rng.permutation(n)[:n // 50]] = P * S + 5
    slots[-1] = 2 ** 62
    dt = torch.bfloat16 if kind == "bf16" else None
    ko, vo = (torch.full((n + 1, H, D), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    fkv.device_error()
    fkv.kv_gather(dev(kc, dtype=dt), dev(vc, dtype=dt), dev(slots), ko[:n], vo[:n], k_scale=dev(ks), v_scale=dev(vs))
    assert fkv.device_error() == fkv.DEVERR_GATHER_SLOT
    ok = np.flatnonzero((slots >= 0) & (slots < P * S))
    for o, c, sc in ((ko, kc, ks), (vo, vc, vs)):
        every = R.gather(c, np.arange(P * S), S, sc, kind)                             # each slot's rows, once
        want = np.zeros((n, H, D))
        want[ok] = every[slots[ok]]
        got = bf16_out(o)
        assert (got[n] == 7).all() and np.array_equal(np.isnan(got[:n]), np.isnan(want))
        assert np.array_equal(np.nan_to_num(got[:n]), np.nan_to_num(want))


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("n,hq,hk,rot", [(4100, 24, 4, 128), (3901, 17, 3, 96), (1999, 29, 11, 128), (4003, 1, 20, 32), (4001, 33, 0, 64)])
def test_norm_rope(n, hq, hk, rot, inter, in_place):
    """Warps with two to five batches of rows: all of a token's heads from about 3700
    tokens on, and (1999) two warps a token, the second's rows of q and of k."""
    import torch
    import fp8_paged_kv_decode_gb300 as fkv
    rng = np.random.default_rng(n + rot)
    x = bits(rng, n, (hq + 2 * hk) * D, std=2.0)                                       # a projection's rows: q, k, v
    qw, kw = (W.bf16_bits((1 + 0.3 * rng.standard_normal(D)).astype(np.float32)) for _ in range(2))
    pos = rng.integers(0, 100000, n).astype(np.int32)
    freq = (10000.0 ** (-np.arange(rot // 2) / (rot // 2))).astype(np.float32)
    t = dev(x, dtype=torch.bfloat16)
    q, k = t[:, :hq * D].unflatten(1, (hq, D)), t[:, hq * D:(hq + hk) * D].unflatten(1, (hk, D)) if hk else None
    qo = q if in_place else torch.full((n, hq, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    ko = None if k is None else k if in_place else torch.full((n, hk, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    fkv.device_error()
    fkv.qk_norm_rope(q, k, dev(pos), dev(freq), qo, ko, q_weight=dev(qw, dtype=torch.bfloat16), k_weight=dev(kw, dtype=torch.bfloat16), eps=1e-5, interleaved=inter)
    assert fkv.device_error() == 0
    got = t.view(torch.int16).cpu().numpy().view(np.uint16)
    kept = slice((hq + hk) * D if in_place else 0, None)
    assert np.array_equal(got[:, kept], x[:, kept])
    check(qo, *R.norm_rope(x[:, :hq * D].reshape(n, hq, D), qw, pos[None], freq, None, 1e-5, inter, 1.0))
    if hk:
        check(ko, *R.norm_rope(x[:, hq * D:(hq + hk) * D].reshape(n, hk, D), kw, pos[None], freq, None, 1e-5, inter, 1.0))


def test_pages_past_4_gib():
    """One page of 2^26 tokens, 4.8 GB: its rows' offsets need more than 32 bits."""
    import torch
    import fp8_paged_kv_decode_gb300 as fkv
    rng = np.random.default_rng(5)
    S = 2 ** 26
    kt, vt = (torch.zeros(1, 1, S, ROW, dtype=torch.uint8, device="cuda") for _ in range(2))
    k, sc = bits(rng, 4, 1, D), np.array([0.01], np.float32)
    slots = np.array([S - 1, 2 ** 32 // ROW + 7, 0, S], np.int64)
    a = dev(k, dtype=torch.bfloat16)
    fkv.device_error()
    fkv.kv_append_fp4(a, a, dev(slots), dev(sc), dev(sc), kt, vt)
    rows = R.fp4_encode(k, sc)
    for t in (kt, vt):
        assert same_rows(torch.stack([t[0, :, s] for s in slots[:3].tolist()]).cpu().numpy(), rows[:3])
        assert int((t[0, 0, 1:2 ** 32 // ROW] != 0).any()) == 0
    ko, vo = (torch.empty(4, 1, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    fkv.kv_gather(kt, vt, dev(slots), ko, vo, k_scale=dev(sc), v_scale=dev(sc))
    want = R.bf16_of(R.fp4_values(rows).astype(np.float32) * sc[0])
    want[3] = 0
    assert np.array_equal(bf16_out(ko), want) and np.array_equal(bf16_out(vo), want)
    assert fkv.device_error() == fkv.DEVERR_APPEND_SLOT | fkv.DEVERR_GATHER_SLOT


@pytest.mark.parametrize("new", [1, 40])
def test_tables_in_arrays_off_16_bytes(new):
    """Entry and token arrays that start 4 or 8 bytes past a 16-byte border."""
    import torch
    from test_gpu_step_tables import Tables
    rng = np.random.default_rng(new)
    B = 130
    cached, fresh = rng.integers(0, 300, B), rng.integers(0, new + 1, B) if new > 1 else np.ones(B, int)
    t = Tables(cached, fresh, 16, 24, 4000, 3500, 3001, int(fresh.sum()) + 5, seed=new)
    x = t.tensors()
    whole = {k: torch.full((x[k].numel() + 2,), -5, dtype=x[k].dtype, device="cuda") for k in ("indices", "expected", "slots", "positions")}
    for k, v in whole.items():
        v[1:-1] = x[k]
        x[k] = v[1:-1]
    assert all(x[k].data_ptr() % 16 for k in whole)
    t.run(into=x)
    w = t.want()
    for k in ("indices", "slots", "positions", "indptr", "step_lens", "table", "free_left"):
        assert np.array_equal(x[k].cpu().numpy(), w[k]), k
    assert np.array_equal(x["expected"].cpu().numpy().view(np.uint32), w["expected"])
    assert all(v[0] == -5 and v[-1] == -5 for v in whole.values())
