"""Two layers' attention in flight at once, each with a workspace of its own."""
import numpy as np
import pytest

from gpu_util import dev
from test_gpu_fp4 import D, Fp4Case

pytestmark = pytest.mark.gpu


class Layer:
    def __init__(self, seed, seq, Hq, H, S):
        import torch
        import fp8_paged_kv_decode_gb300 as fkv
        self.c = c = Fp4Case(len(seq), Hq, H, S, seq, seed=seed)
        self.a = [dev(c.q, dtype=torch.bfloat16), dev(c.kc), dev(c.vc), dev(c.indptr), dev(c.indices), dev(c.seq), c.sm]
        self.kw = dict(k_scale=dev(c.ks), v_scale=dev(c.vs))
        self.ws = fkv.alloc_workspace(c.B, Hq, H, fkv.KV_FP4)
        self.stream = torch.cuda.Stream()

    def outs(self, n):
        import torch
        return [torch.full((self.c.B, self.c.Hq, D), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(n)]

    def attend(self, out):
        import fp8_paged_kv_decode_gb300 as fkv
        fkv.paged_decode_attn(*self.a, out, self.ws, **self.kw, stream=self.stream)


def test_two_layers_at_once_give_each_its_own_rows():
    """Layers of other queries, caches and lengths, with units split over many warps
    and merged through the workspaces: while both run, each call gives the bytes
    that the layer gives alone."""
    import torch
    import fp8_paged_kv_decode_gb300 as fkv
    rng = np.random.default_rng(3)
    layers = [Layer(1, [9000, 1, 300, 5000, 64, 700, 2000], 16, 2, 64), Layer(2, rng.integers(1, 700, 90), 8, 2, 16), Layer(3, [20000], 8, 1, 32)]
    fkv.device_error()
    alone = []
    for x in layers:
        out, = x.outs(1)
        torch.cuda.synchronize()
        x.attend(out)
        torch.cuda.synchronize()
        x.c.check(out)
        alone.append(out.view(torch.int16))
    n = 40
    got = [x.outs(n) for x in layers]
    torch.cuda.synchronize()
    for i in range(n):
        for x, o in zip(layers, got):
            x.attend(o[i])
    torch.cuda.synchronize()
    for outs, one in zip(got, alone):
        assert all(torch.equal(o.view(torch.int16), one) for o in outs)
    assert fkv.device_error() == 0
