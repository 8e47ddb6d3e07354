"""Attention rows in which tokens of large weight and zero V (attention sinks)
stand in every tile, so that all of the output comes from small weights."""
import numpy as np
import pytest

import step_ref as R
from fp8_paged_kv_decode_gb300 import workloads as W
from gpu_util import bf16_out, dev

pytestmark = pytest.mark.gpu
D = 128


def encode(x, g, kind):
    """[P][1][S][row] cache rows of values x, and the values that they stand for."""
    if kind == "bf16":
        bits = W.bf16_bits(x.astype(np.float32))
        return bits, W.bits_to_f32(bits).astype(np.float64)
    if kind == "fp4":
        rows = R.fp4_encode(W.bf16_bits(x.astype(np.float32)).reshape(-1, 1, D), np.array([g], np.float32)).reshape(*x.shape[:-1], 72)
        return rows, R.fp4_values(rows) * np.float64(g)
    code = R.nearest(np.minimum(np.abs(x) / g, 448.0), R.E4M3[:127]).astype(np.uint8) | (np.signbit(x) * np.uint8(128))
    return code, R.E4M3[code] * np.float64(g)


@pytest.mark.parametrize("nats", [8, 14, 18, 22])
@pytest.mark.parametrize("kind,S,large", [("fp4", 64, False), ("fp4", 16, True), ("fp8", 64, False), ("fp8", 16, False), ("bf16", 64, False)])
def test_weights_far_below_the_largest(kind, S, large, nats):
    import torch
    import fp8_paged_kv_decode_gb300 as fkv
    rng = np.random.default_rng(nats)
    G, n, sm = 8, 4096, D ** -0.5
    u = rng.choice([-1.0, 1.0], D)
    q = W.bf16_bits((2 * u + 0.1 * rng.standard_normal((G, D))).astype(np.float32))
    k = 0.05 * rng.standard_normal((n, D)) - u * nats / (2 * D * sm)      # q . k sm is near -nats, 0 for a sink
    v = rng.standard_normal((n, D)) + 0.5
    k[::64] = v[::64] = 0
    ks, vs = np.float32(np.abs(k).max() / 448), np.float32(np.abs(v).max() / 448)
    P = n // S
    kc, kv = encode(k.reshape(P, 1, S, D), ks, kind)
    vc, vv = encode(v.reshape(P, 1, S, D), vs, kind)
    kv, vv = kv.reshape(n, D), vv.reshape(n, D)
    z = W.bits_to_f32(q).astype(np.float64) @ kv.T * sm
    p = np.exp(z - z.max(-1, keepdims=True))
    L = p.sum(-1, keepdims=True)
    want, size = p @ vv / L, p @ np.abs(vv) / L
    dt = torch.bfloat16 if kind == "bf16" else None
    idx = np.zeros(60000 * 64 // S + 2 if large else P, np.int32)         # (a long page table takes the large-call instance)
    idx[:P] = np.arange(P)
    out = torch.full((1, G, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    fmt = dict(fp4=fkv.KV_FP4, fp8=fkv.KV_FP8_E4M3, bf16=fkv.KV_BF16)[kind]
    fkv.paged_decode_attn(dev(q[None], dtype=torch.bfloat16), dev(kc, dtype=dt), dev(vc, dtype=dt), dev(np.array([0, P], np.int32)), dev(idx),
                          dev(np.array([n], np.int32)), float(sm), out, fkv.alloc_workspace(1, G, 1, fmt), k_scale=dev(np.array([ks])), v_scale=dev(np.array([vs])))
    # the output's rounding: 2^-8 of the value.  P: 2^-11 of each weight, or half of f16's smallest step, 2^-25, where the
    # largest weight is 2^15: 2^-40 of that.  Logits below 32 in fp32 (128 products, 2^-17 of a weight at most) and ex2: 2^-14.
    tol = 2.0 ** -8 * np.abs(want) + (2.0 ** -11 + 2.0 ** -14) * size + n * 2.0 ** -40 * np.abs(vv).max() / L
    err = np.abs(bf16_out(out)[0] - want)
    assert (err <= tol).all(), (float((err / tol).max()), float((err / size).max()))
