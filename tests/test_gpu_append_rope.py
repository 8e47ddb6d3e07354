"""kv_append_rope on the GPU: the heads against 64-bit arithmetic, the values' bytes
against the append's, and nothing else touched."""
import numpy as np
import pytest

import step_ref as R
from fp8_paged_kv_decode_gb300 import workloads as W
from gpu_util import bf16_out, dev

pytestmark = pytest.mark.gpu
D = 128
ROW = {"fp8": 128, "bf16": 256, "fp4": 72}


def bits(rng, *shape, std=1.0):
    return W.bf16_bits((std * rng.standard_normal(shape)).astype(np.float32))


def raw(t):
    """A pool's bytes [P][H][S][row]."""
    import torch
    return t.view(torch.uint8).cpu().numpy()


def near_grid(x, v, slack, grid):
    """v is a grid value next to x: no further off than the nearest one, but for the slack in x."""
    a = np.minimum(np.abs(x), grid[-1])
    hi = np.clip(np.searchsorted(grid, a), 1, len(grid) - 1)
    best = np.minimum(a - grid[hi - 1], grid[hi] - a)
    return (np.abs(v - np.sign(x) * a) <= best + 2 * slack + 1e-30) | (np.abs(np.abs(v) - a) <= best + 2 * slack + 1e-30) & (a <= slack)


def check_bf16(got, want, size):
    # as in the rotation's own test: bf16's half step 2^-8, fp32's steps and the angle under 2^-18 of the terms
    err = np.abs(got - want)
    tol = 2.0 ** -8 * np.abs(want) + 2.0 ** -18 * size + 1e-38
    assert (err <= tol).all(), (float((err - tol).max()), np.argwhere(err > tol)[:4])


def check_keys(kind, rows, want, size, scale):
    """Cached key rows [n][H][row bytes] against 64-bit values; the slack is what fp32 and the angle are off
    (2^-18 of the terms, as above) and the quotient's ulps (2^-22)."""
    if kind == "bf16":
        return check_bf16(W.bits_to_f32(rows.view(np.uint16)).astype(np.float64), want, size)
    g = scale.astype(np.float64)[None, :, None]
    x, slack = want / g, 2.0 ** -18 * size / g + 2.0 ** -22 * np.abs(want / g)
    if kind == "fp8":
        assert near_grid(x, R.E4M3[rows], slack, R.E4M3[:127]).all()
        return
    n, h = rows.shape[:2]
    blocks = lambda a: a.reshape(n, h, 8, 16)                       # noqa: E731
    s = R.E4M3[rows[..., 64:]]
    amax, far = blocks(np.abs(x)).max(-1) / 6, blocks(slack).max(-1) / 6 + 2.0 ** -22 * blocks(np.abs(x)).max(-1)
    assert near_grid(amax, s, far, R.E4M3[:127]).all()
    code = blocks(np.stack([rows[..., :64] & 15, rows[..., :64] >> 4], -1).reshape(n, h, D))
    v = np.where(code >= 8, -1.0, 1.0) * R.MAGS[code & 7]
    with np.errstate(all="ignore"):
        t = blocks(x) / s[..., None]
        ok = near_grid(t, v, blocks(slack) / s[..., None] + 2.0 ** -22 * np.abs(t), R.MAGS) | (s[..., None] == 0)
    assert ok.all()


class Case:
    def __init__(self, kind, n, hq, hk, rot, axes, inter, norm, far, S, seed, fused=True, spare=5):
        import torch
        rng = np.random.default_rng(seed)
        self.kind, self.n, self.hq, self.hk, self.S, self.inter, self.norm = kind, n, hq, hk, S, inter, norm
        x = np.concatenate([bits(rng, n, hq * D, std=3.0), bits(rng, n, hk * D, std=0.7), bits(rng, n, hk * D)], 1)
        self.q, self.k, self.v = (a.reshape(n, -1, D) for a in np.split(x, [hq * D, (hq + hk) * D], 1))
        if fused:
            t = dev(x, dtype=torch.bfloat16)
            self.qt, self.kt, self.vt = (a.unflatten(1, (-1, D)) for a in t.split((hq * D, hk * D, hk * D), 1))
        else:
            self.qt, self.kt, self.vt = (dev(a, dtype=torch.bfloat16) for a in (self.q, self.k, self.v))
        self.qw, self.kw = (W.bf16_bits((1 + 0.3 * rng.standard_normal(D)).astype(np.float32)) if norm else None for _ in range(2))
        self.pos = rng.integers(-far // 8, far, (axes, n)).astype(np.int32)
        self.freq = (10000.0 ** (-np.arange(rot // 2) / (rot // 2))).astype(np.float32)
        self.amap = (rng.permutation(rot // 2) % axes).astype(np.uint8) if axes > 1 else None
        self.P = n // S + spare
        self.slots = rng.permutation(self.P * S)[:n].astype(np.int64)
        self.ks, self.vs = (rng.uniform(0.004, 0.03, hk).astype(np.float32) for _ in range(2))
        self.kc, self.vc = (self.pool(rng) for _ in range(2))
        self.before = raw(self.kc).copy(), raw(self.vc).copy()
        self.qo = torch.full((n, hq, D), float("nan"), dtype=torch.bfloat16, device="cuda")

    def pool(self, rng):
        import torch
        t = dev(rng.integers(0, 256, (self.P, self.hk, self.S, ROW[self.kind])).astype(np.uint8))
        return t.view(torch.bfloat16) if self.kind == "bf16" else t

    def args(self, **k):
        import torch
        a = dict(q=self.qt, k=self.kt, v=self.vt, positions=dev(self.pos), inv_freq=dev(self.freq), slot_mapping=dev(self.slots), q_out=self.qo,
                 k_cache=self.kc, v_cache=self.vc, k_scale=dev(self.ks), v_scale=dev(self.vs),
                 q_weight=None if self.qw is None else dev(self.qw, dtype=torch.bfloat16), k_weight=None if self.kw is None else dev(self.kw, dtype=torch.bfloat16),
                 eps=1e-5, axis_map=None if self.amap is None else dev(self.amap), interleaved=self.inter, rot_scale=1.25)
        a.update(k)
        return a

    def rows(self, cache, slots):
        return raw(cache)[slots // self.S, :, slots % self.S]

    def value_rows(self, orc):
        if self.kind == "bf16":
            return self.v.view(np.uint8).reshape(self.n, self.hk, 256)
        if self.kind == "fp4":
            return R.fp4_encode(self.v, self.vs)
        out = np.zeros((1, self.hk, self.n, D), np.uint8)
        orc.kv_append_fp8(self.v, self.v, np.arange(self.n), self.vs, self.vs, out, out.copy())
        return out[0].transpose(1, 0, 2)

    def check(self, orc, live=None):
        live = np.ones(self.n, bool) if live is None else live
        if self.hq:
            check_bf16(bf16_out(self.qo), *R.norm_rope(self.q, self.qw, self.pos, self.freq, self.amap, 1e-5, self.inter, 1.25))
        want, size = R.norm_rope(self.k, self.kw, self.pos, self.freq, self.amap, 1e-5, self.inter, 1.25)
        check_keys(self.kind, self.rows(self.kc, self.slots[live]), want[live], size[live], self.ks)
        got, ref = self.rows(self.vc, self.slots[live]), self.value_rows(orc)[live]
        if self.kind == "fp4":                                     # a zero code's sign is not specified
            clean = lambda r: np.where(r[..., :64] & 7, r[..., :64], r[..., :64] & 0xF7) & np.where(r[..., :64] & 0x70, 0xFF, 0x7F)   # noqa: E731
            assert np.array_equal(clean(got), clean(ref)) and np.array_equal(got[..., 64:], ref[..., 64:])
        else:
            assert np.array_equal(got, ref)
        for now, was in ((self.kc, self.before[0]), (self.vc, self.before[1])):
            rest = np.ones((self.P, self.S), bool)
            rest[self.slots[live] // self.S, self.slots[live] % self.S] = False
            assert np.array_equal(raw(now).transpose(0, 2, 1, 3)[rest], was.transpose(0, 2, 1, 3)[rest])


CASES = [  # tokens, q heads, k heads, rotary dim, axes, interleaved, norm, largest position, page
    (1, 1, 1, 128, 1, False, True, 10, 16), (1, 64, 8, 128, 1, False, True, 131072, 64), (3, 8, 2, 64, 1, False, True, 1000, 16),
    (5, 6, 3, 128, 3, True, True, 5000, 32), (64, 32, 8, 128, 1, True, False, 131072, 128), (7, 4, 4, 16, 2, False, True, 100, 16),
    (2, 40, 1, 96, 4, False, True, 2 ** 20, 48), (130, 24, 8, 32, 1, True, True, 70000, 16), (700, 16, 2, 128, 3, False, True, 131072, 64),
    (33, 0, 5, 48, 1, False, False, 3000, 24), (9, 12, 7, 80, 1, True, False, 3000, 16)]


@pytest.mark.parametrize("kind", ["fp8", "bf16", "fp4"])
@pytest.mark.parametrize("n,hq,hk,rot,axes,inter,norm,far,S", CASES)
def test_against_64_bits(orc, kind, n, hq, hk, rot, axes, inter, norm, far, S):
    import fp8_paged_kv_decode_gb300 as fkv
    c = Case(kind, n, hq, hk, rot, axes, inter, norm, far, S, seed=n * 7 + rot, fused=n % 2 == 1)
    fkv.device_error()
    a = c.args()
    if hq == 0:
        a.update(q=None, q_out=None)
    fkv.kv_append_rope(**a)
    assert fkv.device_error() == 0
    c.check(orc)


@pytest.mark.parametrize("kind", ["fp8", "bf16", "fp4"])
def test_many_tokens(orc, kind):
    """As many as make every warp take whole tokens."""
    import fp8_paged_kv_decode_gb300 as fkv
    c = Case(kind, 4500, 10, 3, 128, 1, False, True, 131072, 64, seed=5)
    fkv.kv_append_rope(**c.args())
    c.check(orc)


def test_as_the_two_calls():
    """BF16 without norm: the bytes of qk_norm_rope and kv_append_bf16."""
    import torch
    import fp8_paged_kv_decode_gb300 as fkv
    for inter, rot in ((False, 128), (True, 128), (False, 48)):
        c = Case("bf16", 77, 8, 4, rot, 1, inter, False, 131072, 16, seed=rot, fused=False)
        qo, ko = torch.empty_like(c.qt), torch.empty_like(c.kt)
        kc, vc = c.kc.clone(), c.vc.clone()
        fkv.qk_norm_rope(c.qt, c.kt, dev(c.pos), dev(c.freq), qo, ko, interleaved=inter, rot_scale=1.25)
        fkv.kv_append_bf16(ko, c.vt, dev(c.slots), kc, vc)
        fkv.kv_append_rope(**c.args())
        assert torch.equal(qo.view(torch.int16), c.qo.view(torch.int16))
        assert np.array_equal(raw(kc), raw(c.kc)) and np.array_equal(raw(vc), raw(c.vc))


@pytest.mark.parametrize("kind", ["fp8", "fp4"])
def test_values_are_the_appends_bytes(kind):
    """Zeros of both signs, infinities, NaN, huge and tiny elements, scales beyond the quotient's fast range."""
    import torch
    import fp8_paged_kv_decode_gb300 as fkv
    c = Case(kind, 48, 2, 4, 128, 1, False, False, 100, 16, seed=3, fused=False)
    rng = np.random.default_rng(9)
    v = rng.integers(0, 1 << 16, (48, 4, D)).astype(np.uint16)
    v[0] = 0
    v[1] = 0x8000
    v[2, :, ::16], v[3, :, 3], v[4, :, 5] = 0x7F80, 0x7FC0, 0xFF80
    v[5:20] = bits(rng, 15, 4, D, std=1e-3)
    vt = dev(v, dtype=torch.bfloat16)
    scales = dev(np.array([0.01, 2.0 ** -40, 2.0 ** 35, 1.0], np.float32))
    kc, vc = c.kc.clone(), c.vc.clone()
    (fkv.kv_append_fp8 if kind == "fp8" else fkv.kv_append_fp4)(c.kt, vt, dev(c.slots), scales, scales, kc, vc)
    fkv.kv_append_rope(**c.args(v=vt, v_scale=scales, k_scale=scales))
    a, b = c.rows(vc, c.slots), c.rows(c.vc, c.slots)
    if kind == "fp8":
        nan = (a & 0x7F) == 0x7F
        assert np.array_equal(nan, (b & 0x7F) == 0x7F) and np.array_equal(a[~nan], b[~nan])
    else:
        nan = (a[..., 64:] & 0x7F) == 0x7F
        assert np.array_equal(nan, (b[..., 64:] & 0x7F) == 0x7F) and np.array_equal(a[..., 64:][~nan], b[..., 64:][~nan])
        x, y = R.fp4_values(a), R.fp4_values(b)
        assert np.array_equal(x[~np.isnan(x)], y[~np.isnan(x)]) and np.isnan(y[np.isnan(x)]).all()


@pytest.mark.parametrize("kind", ["fp8", "bf16", "fp4"])
def test_nan_and_infinite_keys(kind):
    import fp8_paged_kv_decode_gb300 as fkv
    import torch
    c = Case(kind, 3, 2, 2, 64, 1, False, False, 100, 16, seed=4, fused=False)
    k = c.k.copy()
    k[0, 1, 70] = 0x7FC0                                         # past rotary_dim: stays alone
    k[1, 0, 100] = 0xFF80
    k[2, 1, 3] = 0x7FC0                                          # turns with element 35
    fkv.kv_append_rope(**c.args(k=dev(k, dtype=torch.bfloat16)))
    rows = c.rows(c.kc, c.slots)
    if kind == "bf16":
        got = W.bits_to_f32(rows.view(np.uint16))
    else:
        got = R.fp4_values(rows) if kind == "fp4" else R.E4M3[rows]
    bad = np.zeros((3, 2, D), bool)
    if kind == "fp4":                                            # the blocks of 16
        bad[0, 1, 64:80] = bad[2, 1, 0:16] = bad[2, 1, 32:48] = True
    else:
        bad[0, 1, 70] = bad[2, 1, 3] = bad[2, 1, 35] = True
    assert np.array_equal(np.isnan(got), bad)
    assert got[1, 0, 100] == {"bf16": -np.inf, "fp8": -448, "fp4": -6 * 448}[kind]


@pytest.mark.parametrize("kind", ["fp8", "fp4"])
def test_padding_and_slots_outside(orc, kind):
    """Tokens without a place still have their query heads turned."""
    import fp8_paged_kv_decode_gb300 as fkv
    c = Case(kind, 20, 5, 2, 128, 1, False, True, 1000, 16, seed=6)
    live = np.ones(20, bool)
    c.slots[[3, 7, 19]], live[[3, 7, 19]] = -1, False
    fkv.device_error()
    fkv.kv_append_rope(**c.args())
    assert fkv.device_error() == 0
    c.check(orc, live)
    c = Case(kind, 20, 5, 2, 128, 1, False, True, 1000, 16, seed=6)
    c.slots[4], live[:] = c.P * 16, True
    live[4] = False
    fkv.kv_append_rope(**c.args())
    assert fkv.device_error() == fkv.DEVERR_APPEND_SLOT
    c.check(orc, live)


def test_in_place_and_axis_outside(orc):
    import fp8_paged_kv_decode_gb300 as fkv
    c = Case("fp8", 41, 8, 2, 128, 1, False, True, 5000, 16, seed=8)
    c.qo = c.qt
    fkv.kv_append_rope(**c.args())
    c.check(orc)
    c = Case("bf16", 2, 2, 2, 128, 2, False, False, 50, 16, seed=9)
    c.amap[10] = 2
    fkv.device_error()
    fkv.kv_append_rope(**c.args())
    assert fkv.device_error() == fkv.DEVERR_ROPE_AXIS
    c.check(orc)


def test_graph_and_side_stream(orc):
    import torch
    import fp8_paged_kv_decode_gb300 as fkv
    c = Case("fp4", 64, 16, 4, 128, 1, False, True, 5000, 16, seed=10)
    a = c.args()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    fkv.kv_append_rope(**a, stream=side)
    side.synchronize()
    c.check(orc)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fkv.kv_append_rope(**a)
    c.qo.fill_(0)
    for t, was in ((c.kc, c.before[0]), (c.vc, c.before[1])):
        t.copy_(dev(was))
    g.replay()
    torch.cuda.synchronize()
    c.check(orc)


def test_python_refusals():
    import torch
    import fp8_paged_kv_decode_gb300 as fkv
    c = Case("fp8", 3, 4, 2, 128, 1, False, True, 100, 16, seed=1, fused=False)
    z = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt, device="cuda")   # noqa: E731
    for bad in (dict(q=c.qt.float()), dict(q_out=z(3, 4, 64)), dict(q_out=None), dict(k=c.kt[:2]), dict(v=z(3, 3, D)), dict(positions=z(2, dt=torch.int32)),
                dict(positions=z(3, dt=torch.int64)), dict(inv_freq=z(12, dt=torch.float32)), dict(slot_mapping=z(3, dt=torch.int32)),
                dict(slot_mapping=z(4, dt=torch.int64)), dict(k_scale=None), dict(v_scale=z(1, dt=torch.float32)), dict(k_cache=c.kc[:2]),
                dict(k_cache=c.kc.view(torch.int8)), dict(k_cache=c.kc.cpu()), dict(q_weight=z(64)), dict(axis_map=z(32, dt=torch.uint8)), dict(eps=-1.0),
                dict(v=z(3, D, 2).transpose(1, 2)), dict(k=z(3, 4, D)[:, ::2]), dict(v_cache=z(*c.vc.shape))):
        with pytest.raises(fkv.FkvError):
            fkv.kv_append_rope(**c.args(**bad))
    e = lambda *s: z(0, *s)                                                      # noqa: E731
    fkv.kv_append_rope(**c.args(q=e(4, D), k=e(2, D), v=e(2, D), q_out=e(4, D), positions=z(0, dt=torch.int32), slot_mapping=z(0, dt=torch.int64)))


def test_bf16_values_are_copied_bit_by_bit():
    """Every BF16 value, NaN with their payloads and signs among them, as kv_append_bf16 puts it."""
    import torch
    import fp8_paged_kv_decode_gb300 as fkv
    c = Case("bf16", 128, 2, 4, 128, 1, False, False, 100, 16, seed=11, fused=False)
    v = np.random.default_rng(12).permutation(1 << 16).astype(np.uint16).reshape(128, 4, D)
    vt = dev(v, dtype=torch.bfloat16)
    kc, vc = c.kc.clone(), c.vc.clone()
    fkv.kv_append_bf16(c.kt, vt, dev(c.slots), kc, vc)
    fkv.kv_append_rope(**c.args(v=vt))
    assert np.array_equal(c.rows(c.vc, c.slots), v.view(np.uint8).reshape(128, 4, 256)) and np.array_equal(raw(c.vc), raw(vc))
