"""qk_norm_rope on the GPU against 64-bit arithmetic."""
import numpy as np
import pytest

import step_ref as R
from fp8_paged_kv_decode_gb300 import workloads as W
from gpu_util import bf16_out, dev

pytestmark = pytest.mark.gpu
D = 128


def bits(rng, *shape, std=1.0):
    return W.bf16_bits((std * rng.standard_normal(shape)).astype(np.float32))


def check(out, want, size):
    # bf16 rounding: 2^-8 of the value.  fp32: the mean's 12 roundings, rsqrt (2 ulp) and two products under 2^-20 of each
    # term, the angle under 2^-22 of a turn (2 pi 2^-22 < 2^-19 of each term), sin, cos and the last product-sum under 2^-21.
    tol = 2.0 ** -8 * np.abs(want) + 2.0 ** -18 * size + 1e-38
    err = np.abs(bf16_out(out) - want)
    assert (err <= tol).all(), (float((err - tol).max()), np.argwhere(err > tol)[:4])


CASES = [  # tokens, q heads, k heads, rotary dim, axes, interleaved, norm, largest position
    (1, 1, 1, 128, 1, False, True, 10), (1, 64, 8, 128, 1, False, True, 131072), (3, 8, 2, 64, 1, False, True, 1000),
    (5, 6, 3, 128, 3, True, True, 5000), (64, 32, 8, 128, 1, True, False, 131072), (7, 4, 4, 16, 2, False, True, 100),
    (2, 40, 1, 96, 4, False, True, 2 ** 20), (130, 24, 8, 32, 1, True, True, 70000), (700, 16, 2, 128, 3, False, True, 131072)]


@pytest.mark.parametrize("n,hq,hk,rot,axes,inter,norm,far", CASES)
def test_against_64_bits(n, hq, hk, rot, axes, inter, norm, far):
    import torch
    import fp8_paged_kv_decode_gb300 as fkv
    rng = np.random.default_rng(n * 7 + rot)
    q, k = bits(rng, n, hq, D, std=3.0), bits(rng, n, hk, D, std=0.1)
    qw, kw = (W.bf16_bits((1 + 0.3 * rng.standard_normal(D)).astype(np.float32)) if norm else None for _ in range(2))
    pos = rng.integers(-far // 8, far, (axes, n)).astype(np.int32)
    freq = (10000.0 ** (-np.arange(rot // 2) / (rot // 2))).astype(np.float32)
    amap = (rng.permutation(rot // 2) % axes).astype(np.uint8) if axes > 1 else None
    qo, ko = (torch.full((n, h, D), float("nan"), dtype=torch.bfloat16, device="cuda") for h in (hq, hk))
    fkv.device_error()
    fkv.qk_norm_rope(dev(q, dtype=torch.bfloat16), dev(k, dtype=torch.bfloat16), dev(pos), dev(freq), qo, ko,
                     q_weight=None if qw is None else dev(qw, dtype=torch.bfloat16), k_weight=None if kw is None else dev(kw, dtype=torch.bfloat16),
                     eps=1e-5, axis_map=None if amap is None else dev(amap), interleaved=inter, rot_scale=1.25)
    assert fkv.device_error() == 0
    for o, x, w in ((qo, q, qw), (ko, k, kw)):
        check(o, *R.norm_rope(x, w, pos, freq, amap, 1e-5, inter, 1.25))


def test_parts_of_one_projection_in_place():
    """q and k as parts of one tensor's rows, written back in place; V beside them stays."""
    import torch
    import fp8_paged_kv_decode_gb300 as fkv
    rng = np.random.default_rng(1)
    n, hq, hk = 37, 8, 2
    x = bits(rng, n, (hq + 2 * hk) * D)
    w = W.bf16_bits(np.ones(D, np.float32))
    pos = rng.integers(0, 9000, n).astype(np.int32)
    freq = (10000.0 ** (-np.arange(64) / 64)).astype(np.float32)
    t = dev(x, dtype=torch.bfloat16)
    q, k = t[:, :hq * D].unflatten(1, (hq, D)), t[:, hq * D:(hq + hk) * D].unflatten(1, (hk, D))
    fkv.qk_norm_rope(q, k, dev(pos), dev(freq), q, k, q_weight=dev(w, dtype=torch.bfloat16), k_weight=dev(w, dtype=torch.bfloat16))
    got = t.view(torch.int16).cpu().numpy().view(np.uint16)
    assert np.array_equal(got[:, (hq + hk) * D:], x[:, (hq + hk) * D:])
    check(q, *R.norm_rope(x[:, :hq * D].reshape(n, hq, D), w, pos[None], freq, None, 1e-6, False, 1.0))
    check(k, *R.norm_rope(x[:, hq * D:(hq + hk) * D].reshape(n, hk, D), w, pos[None], freq, None, 1e-6, False, 1.0))


def test_special_rows():
    """A row of zeros stays zeros (eps keeps the norm finite), a NaN stays in its row, no k at all."""
    import torch
    import fp8_paged_kv_decode_gb300 as fkv
    rng = np.random.default_rng(2)
    x = bits(rng, 3, 4, D)
    x[0, 1] = 0
    x[1, 2, 9] = 0x7FC0
    w = W.bf16_bits(np.ones(D, np.float32))
    pos, freq = np.array([5, 6, 7], np.int32), (10000.0 ** (-np.arange(64) / 64)).astype(np.float32)
    q = dev(x, dtype=torch.bfloat16)
    out = torch.empty_like(q)
    fkv.qk_norm_rope(q, None, dev(pos), dev(freq), out, None, q_weight=dev(w, dtype=torch.bfloat16))
    got = bf16_out(out)
    assert (got[0, 1] == 0).all() and np.isnan(got[1, 2]).all()
    want, size = R.norm_rope(x, w, pos[None], freq, None, 1e-6, False, 1.0)
    keep = np.ones((3, 4), bool)
    keep[1, 2] = False
    assert (np.abs(got - want)[keep] <= (2.0 ** -8 * np.abs(want) + 2.0 ** -18 * size + 1e-38)[keep]).all()


def test_axis_outside_is_recorded_and_left_unturned():
    import torch
    import fp8_paged_kv_decode_gb300 as fkv
    rng = np.random.default_rng(3)
    x = bits(rng, 2, 2, D)
    amap = np.zeros(64, np.uint8)
    amap[10] = 2
    pos, freq = rng.integers(0, 50, (2, 2)).astype(np.int32), np.ones(64, np.float32)
    q = dev(x, dtype=torch.bfloat16)
    out = torch.empty_like(q)
    fkv.device_error()
    fkv.qk_norm_rope(q, None, dev(pos), dev(freq), out, None, axis_map=dev(amap))
    assert fkv.device_error() == fkv.DEVERR_ROPE_AXIS
    check(out, *R.norm_rope(x, None, pos, freq, amap, 0.0, False, 1.0))
    assert np.array_equal(bf16_out(out)[..., [10, 74]], W.bits_to_f32(x)[..., [10, 74]])


def test_far_positions():
    """At 2^30 the angle is still known to 2^-18 of a turn."""
    import torch
    import fp8_paged_kv_decode_gb300 as fkv
    rng = np.random.default_rng(4)
    x = bits(rng, 64, 1, D)
    pos = rng.integers(2 ** 29, 2 ** 30, (1, 64)).astype(np.int32)
    freq = np.concatenate([[1.0], rng.uniform(0, 1, 63)]).astype(np.float32)
    q = dev(x, dtype=torch.bfloat16)
    out = torch.empty_like(q)
    fkv.qk_norm_rope(q, None, dev(pos), dev(freq), out, None)
    want, size = R.norm_rope(x, None, pos, freq, None, 0.0, False, 1.0)
    tol = 2.0 ** -8 * np.abs(want) + (2 * np.pi * 2.0 ** -18 + 2.0 ** -20) * size
    assert (np.abs(bf16_out(out) - want) <= tol).all()


def test_python_refusals():
    import torch
    import fp8_paged_kv_decode_gb300 as fkv
    z = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt, device="cuda")   # noqa: E731
    q, k, pos, freq = z(3, 4, D), z(3, 2, D), z(3, dt=torch.int32), z(64, dt=torch.float32)
    for bad in (dict(q=q.float()), dict(q_out=z(3, 4, 64)), dict(k_out=None), dict(positions=pos.long()), dict(positions=z(2, dt=torch.int32)),
                dict(inv_freq=z(12, dt=torch.float32)), dict(inv_freq=freq.double()), dict(q_weight=z(64)), dict(axis_map=z(32, dt=torch.uint8)),
                dict(q=z(3, D, 4).transpose(1, 2)), dict(q=z(3, 8, D)[:, ::2]), dict(q=q.cpu()), dict(eps=-1.0)):
        a = dict(q=q, k=k, positions=pos, inv_freq=freq, q_out=z(3, 4, D), k_out=z(3, 2, D))
        a.update(bad)
        with pytest.raises(fkv.FkvError):
            fkv.qk_norm_rope(**a)
    fkv.qk_norm_rope(z(0, 4, D), z(0, 2, D), z(0, dt=torch.int32), freq, z(0, 4, D), z(0, 2, D))
