"""The longest request that a length can say, 2^31 - 1 tokens, over a page table
that lists a few pages again and again."""
import numpy as np
import pytest

import step_ref as R
from fp8_paged_kv_decode_gb300 import workloads as W
from gpu_util import bf16_out, dev
from test_gpu_attention_weights import encode

pytestmark = pytest.mark.gpu
D = 128


@pytest.mark.parametrize("kind,S", [("fp4", 128), ("fp4", 16), ("fp8", 128), ("fp8", 16), ("bf16", 64)])
def test_every_token_of_the_longest_request(kind, S):
    import torch
    import fp8_paged_kv_decode_gb300 as fkv
    rng = np.random.default_rng(S)
    G, P, n, short, sm = 4, 64, 2 ** 31 - 1, 37, D ** -0.5
    q = W.bf16_bits(rng.standard_normal((2, G, D)).astype(np.float32))
    g = np.float32(0.01)
    kc, kv = encode(rng.standard_normal((P, 1, S, D)), g, kind)
    vc, vv = encode(rng.standard_normal((P, 1, S, D)) + 0.5, g, kind)
    pages = -(-n // S)
    idx = torch.arange(pages + 1 + short // S + 1, dtype=torch.int32, device="cuda") % P
    indptr = np.array([0, pages, len(idx)], np.int32)
    dt = torch.bfloat16 if kind == "bf16" else None
    fmt = dict(fp4=fkv.KV_FP4, fp8=fkv.KV_FP8_E4M3, bf16=fkv.KV_BF16)[kind]
    out = torch.full((2, G, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    sc = dev(np.array([g]))
    fkv.device_error()
    fkv.paged_decode_attn(dev(q, dtype=torch.bfloat16), dev(kc, dtype=dt), dev(vc, dtype=dt), dev(indptr), idx, dev(np.array([n, short], np.int32)), float(sm),
                          out, fkv.alloc_workspace(2, G, 1, fmt), k_scale=sc, v_scale=sc)
    got = bf16_out(out)
    assert fkv.device_error() == 0
    count = np.zeros((2, P, S))                                  # how often each cached token stands in the request
    count[0] = (pages - np.arange(P) + P - 1)[:, None] // P
    count[0, (pages - 1) % P, S - 1 - (pages * S - 1 - n):] -= 1
    for t in range(short):
        count[1, (pages + t // S) % P, t % S] += 1
    assert count.sum((1, 2)).tolist() == [n, short]
    count = count.reshape(2, 1, P * S)
    z = W.bits_to_f32(q).astype(np.float64) @ kv.reshape(P * S, D).T * sm
    p = count * np.exp(z - z.max(-1, keepdims=True))
    L = p.sum(-1, keepdims=True)
    want, size = p @ vv.reshape(P * S, D) / L, p @ np.abs(vv.reshape(P * S, D)) / L
    # rounding of the output and of P, logits and exponentials as for any request; then the running fp32 sums of a warp:
    # 2^25 tiles of four additions over 600 warps or more, each off by at most 2^-23 (the tensor core may truncate) of a
    # sum that grows evenly, so half of that count, for o and again for l
    adds = 4 * 2 ** 25 / 600
    tol = 2.0 ** -8 * np.abs(want) + (2.0 ** -11 + 2.0 ** -14 + adds * 2.0 ** -23) * size
    err = np.abs(got - want)
    assert (err[1] <= (2.0 ** -8 * np.abs(want) + (2.0 ** -11 + 2.0 ** -14) * size)[1]).all()
    assert (err <= tol).all(), (float((err / tol).max()), float((err / size).max()))
