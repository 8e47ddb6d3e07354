"""A whole decode step over the 4-bit cache: tables from lengths, head norms with
rotation, append and integrity check, attention, read-back; eager and replayed."""
import numpy as np
import pytest

import step_ref as R
from fp8_paged_kv_decode_gb300 import workloads as W
from gpu_util import bf16_out, dev

pytestmark = pytest.mark.gpu
D, ROW = 128, 72


class Step:
    """B requests that grow token by token in a pool of pages, every table made on the GPU."""

    def __init__(self, B, Hq, H, S, blocks, pool, nnz, seed):
        import torch
        import fp8_paged_kv_decode_gb300 as fkv
        rng = np.random.default_rng(seed)
        self.B, self.Hq, self.H, self.S, self.rng = B, Hq, H, S, rng
        i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")        # noqa: E731
        self.cached, self.new, self.table, self.tags = i32(B), i32(B), i32(B, blocks) - 1, i32(B, blocks)
        self.free, self.count = dev(rng.permutation(pool).astype(np.int32)), dev(np.array([pool], np.int32))
        self.live = dev(rng.integers(0, 2 ** 31, pool).astype(np.int32))
        self.step, self.refused, self.ptr, self.idx, self.exp, self.tptr = i32(B), torch.zeros(B, dtype=torch.uint8, device="cuda"), i32(B + 1), i32(nnz), i32(nnz), i32(B + 1)
        self.nnz = nnz
        self.ks, self.vs = (rng.uniform(0.01, 0.03, H).astype(np.float32) for _ in range(2))
        self.kst, self.vst = dev(self.ks), dev(self.vs)
        self.kc, self.vc = (torch.full((pool, H, S, ROW), 0xFF, dtype=torch.uint8, device="cuda") for _ in range(2))
        self.freq = (10000.0 ** (-np.arange(64) / 64)).astype(np.float32)
        self.freqt = dev(self.freq)
        self.qw, self.kw = (W.bf16_bits((1 + 0.1 * rng.standard_normal(D)).astype(np.float32)) for _ in range(2))
        self.qwt, self.kwt = dev(self.qw, dtype=torch.bfloat16), dev(self.kw, dtype=torch.bfloat16)
        self.mask = torch.zeros(B, dtype=torch.uint8, device="cuda")
        self.tws, self.aws = fkv.alloc_step_tables_workspace(B), fkv.alloc_workspace(B, Hq, H, fkv.KV_FP4)
        self.out = torch.empty(B, Hq, D, dtype=torch.bfloat16, device="cuda")

    def buffers(self, n):
        import torch
        self.n = n
        self.slots, self.pos = torch.zeros(n, dtype=torch.int64, device="cuda"), torch.zeros(n, dtype=torch.int32, device="cuda")
        self.qkv = torch.zeros(n, (self.Hq + 2 * self.H) * D, dtype=torch.bfloat16, device="cuda")
        self.v = torch.zeros(n, self.H, D, dtype=torch.bfloat16, device="cuda")
        self.qo, self.ko = (torch.zeros(n, h, D, dtype=torch.bfloat16, device="cuda") for h in (self.Hq, self.H))

    def calls(self, attend):
        import fp8_paged_kv_decode_gb300 as fkv
        Hq, H = self.Hq, self.H
        fkv.kv_step_tables(self.cached, self.new, self.table, self.tags, self.free, self.count, self.live, self.S, self.step, self.cached, self.refused,
                           self.ptr, self.idx, self.exp, self.tptr, self.slots, self.pos, self.count, self.tws)
        q, k = self.qkv[:, :Hq * D].unflatten(1, (Hq, D)), self.qkv[:, Hq * D:(Hq + H) * D].unflatten(1, (H, D))
        fkv.qk_norm_rope(q, k, self.pos, self.freqt, self.qo, self.ko, q_weight=self.qwt, k_weight=self.kwt)
        fkv.kv_append_fp4_tag_check(self.ko, self.v, self.slots, self.kst, self.vst, self.kc, self.vc, self.live, self.ptr, self.idx, self.exp, self.mask)
        if attend:
            fkv.paged_decode_attn(self.qo[:self.B], self.kc, self.vc, self.ptr, self.idx, self.step, 1 / np.sqrt(D), self.out, self.aws,
                                  k_scale=self.kst, v_scale=self.vst, abort_mask=self.mask)

    def fill(self):
        import torch
        x = W.bf16_bits(self.rng.standard_normal((self.n, (self.Hq + 2 * self.H) * D)).astype(np.float32))
        v = W.bf16_bits(self.rng.standard_normal((self.n, self.H, D)).astype(np.float32))
        self.qkv.copy_(dev(x, dtype=torch.bfloat16))
        self.v.copy_(dev(v, dtype=torch.bfloat16))
        return v

    def check(self):
        """Attention against 64-bit softmax on the cache's own bytes, through the tables' own pages."""
        lens = self.step.cpu().numpy()
        q = self.qo[:self.B].contiguous().view(__import__("torch").int16).cpu().numpy().view(np.uint16)
        want, vmax = R.attention(q, self.kc.cpu().numpy(), self.vc.cpu().numpy(), self.ks, self.vs, self.ptr.cpu().numpy(), self.idx.cpu().numpy(), lens,
                                 1 / np.sqrt(D), self.mask.cpu().numpy())
        err = np.abs(bf16_out(self.out) - want)
        assert (err <= 2.0 ** -8 * np.abs(want) + (2.0 ** -11 + 2.0 ** -12) * vmax).all()


@pytest.mark.parametrize("B,Hq,H,S", [(3, 8, 2, 16), (9, 16, 4, 64), (70, 8, 1, 32)])
def test_prompt_then_decode_steps(B, Hq, H, S):
    import torch
    import fp8_paged_kv_decode_gb300 as fkv
    fkv.device_error()
    s = Step(B, Hq, H, S, blocks=12, pool=B * 12, nnz=B * 12, seed=B)
    lens = s.rng.integers(1, 4 * S, B)
    s.new.copy_(dev(lens.astype(np.int32)))
    s.buffers(int(lens.sum()) + 3)
    s.fill()
    s.calls(attend=False)                                        # the prompts
    assert s.cached.tolist() == lens.tolist() and s.mask.sum() == 0
    # what the cache holds of the prompts' V, read back, is the encoding of what went in
    vo, ko = (torch.empty(s.n, H, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    fkv.kv_gather(s.kc, s.vc, s.slots, ko, vo, k_scale=s.kst, v_scale=s.vst)
    v = s.v.view(torch.int16).cpu().numpy().view(np.uint16)
    want = R.bf16_of(R.fp4_values(R.fp4_encode(v, s.vs)).astype(np.float32) * s.vs[None, :, None])
    want[int(lens.sum()):] = 0
    assert np.array_equal(bf16_out(vo), want)
    s.new.fill_(1)
    s.buffers(B)
    for _ in range(3):                                           # eager
        s.fill()
        s.calls(attend=True)
        s.check()
    assert s.cached.tolist() == (lens + 3).tolist()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        s.calls(attend=True)
    for _ in range(S + 2):                                       # replayed past a page border
        s.fill()
        g.replay()
    torch.cuda.synchronize()
    s.check()
    assert s.cached.tolist() == (lens + 5 + S).tolist() and fkv.device_error() == 0
    used = int((-(-(lens + 5 + S) // S)).sum())
    assert s.count.tolist() == [B * 12 - used]


def test_a_refused_and_a_stale_request_get_zeros():
    import fp8_paged_kv_decode_gb300 as fkv
    B, S = 4, 16
    s = Step(B, 8, 2, S, blocks=4, pool=7, nnz=16, seed=1)
    s.new.copy_(dev(np.array([16, 20, 32, 5], np.int32)))        # 1 + 2 + 2 + 1 pages, one left
    s.buffers(73)
    s.fill()
    s.calls(attend=False)
    assert s.count.tolist() == [1]
    s.new.fill_(1)
    s.buffers(B)
    s.fill()
    s.live[int(s.table[3, 0])] += 1                              # request 3's page changed hands
    fkv.device_error()
    s.calls(attend=True)                                         # requests 0 and 2 need a page, one is there
    assert s.refused.tolist() == [0, 0, 1, 0] and fkv.device_error() == fkv.DEVERR_TABLES
    assert s.mask.tolist() == [0, 0, 1, 1] and s.cached.tolist() == [17, 21, 32, 6]
    s.check()
    out = s.out.float().cpu().numpy()
    assert (out[2:] == 0).all() and (out[:2] != 0).any(-1).all()


def test_on_a_side_stream():
    """Every call of the step on a stream that is not the current one."""
    import torch
    import fp8_paged_kv_decode_gb300 as fkv
    s = Step(3, 8, 2, 16, blocks=4, pool=12, nnz=12, seed=2)
    s.new.copy_(dev(np.array([5, 6, 7], np.int32)))
    s.buffers(18)
    s.fill()
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        s.calls(attend=False)
    st.synchronize()
    assert s.cached.tolist() == [5, 6, 7]
    ko, vo = (torch.empty(18, 2, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    fkv.kv_gather(s.kc, s.vc, s.slots, ko, vo, k_scale=s.kst, v_scale=s.vst, stream=st)
    st.synchronize()
    assert torch.isfinite(vo).all() and vo.abs().amax() > 1


def test_empty_calls():
    """No tokens, no requests: nothing is launched that could touch anything."""
    import torch
    import fp8_paged_kv_decode_gb300 as fkv
    z = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt, device="cuda")   # noqa: E731
    kc, sc, none = z(2, 2, 16, ROW, dt=torch.uint8), z(2, dt=torch.float32) + 1, z(0, dt=torch.int64)
    fkv.kv_append_fp4(z(0, 2, D), z(0, 2, D), none, sc, sc, kc, kc.clone())
    fkv.kv_gather(kc, kc.clone(), none, z(0, 2, D), z(0, 2, D), k_scale=sc, v_scale=sc)
    ptr = z(1, dt=torch.int32)
    fkv.kv_append_fp4_tag_check(z(0, 2, D), z(0, 2, D), none, sc, sc, kc, kc.clone(), z(2, dt=torch.int32), ptr, z(0, dt=torch.int32), z(0, dt=torch.int32),
                                z(0, dt=torch.uint8))
    fkv.paged_decode_attn(z(0, 8, D), kc, kc.clone(), ptr, z(0, dt=torch.int32), z(0, dt=torch.int32), 0.1, z(0, 8, D), fkv.alloc_workspace(0, 8, 2, fkv.KV_FP4),
                          k_scale=sc, v_scale=sc)
    torch.cuda.synchronize()
    assert (kc == 0).all()


def test_two_layers_on_two_streams():
    """Two layers' norms, appends and attention at once, a workspace each: the same bytes as one after the other."""
    import torch
    import fp8_paged_kv_decode_gb300 as fkv
    a, b = (Step(9, 16, 4, 64, blocks=6, pool=54, nnz=54, seed=7) for _ in range(2))
    for s in (a, b):
        s.new.copy_(dev(np.arange(9, dtype=np.int32) * 30 + 1))
        s.buffers(int((np.arange(9) * 30 + 1).sum()))
        s.fill()
        s.calls(attend=False)
        s.new.fill_(1)
        s.buffers(9)
        s.fill()
    torch.cuda.synchronize()
    x, y = torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.stream(x):
        a.calls(attend=True)
    with torch.cuda.stream(y):
        b.calls(attend=True)
    torch.cuda.synchronize()
    assert torch.equal(a.out.view(torch.int16), b.out.view(torch.int16)) and torch.equal(a.kc, b.kc)
    a.check()
    assert fkv.device_error() == 0
