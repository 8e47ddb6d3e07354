"""What the compiled marshalling does besides its checks: the interpreter lock,
stream arguments and cache formats.  The calls here launch nothing wrong: the
entry points are replaced, or the call is refused."""
import contextlib
import ctypes

import pytest

pytestmark = pytest.mark.gpu
D = 128


@contextlib.contextmanager
def entry_points(address):
    """Every call of the marshalling goes to the C function at `address`."""
    import fp8_paged_kv_decode_gb300 as fkv
    mod, lib = fkv._load_bind(), fkv.load_library()
    own = [ctypes.cast(getattr(lib, f), ctypes.c_void_p).value for f in fkv._BIND_CALLS]
    mod.setup(fkv.FkvError, own[0], *[address] * (len(own) - 1))
    try:
        yield
    finally:
        mod.setup(fkv.FkvError, *own)


def calls(stream=None):
    """One valid call of each marshalled entry point, by name."""
    import torch
    import fp8_paged_kv_decode_gb300 as fkv
    z = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt, device="cuda")   # noqa: E731
    i32 = lambda *s: z(*s, dt=torch.int32)                                       # noqa: E731
    kc, sc, x, slots = z(4, 2, 16, 72, dt=torch.uint8), z(2, dt=torch.float32) + 1, z(3, 2, D), z(3, dt=torch.int64)
    ptr, idx, tags, mask = i32(4), i32(3), i32(4), z(3, dt=torch.uint8)
    q, k = z(3, 8, D), z(3, 2, D)
    return dict(
        kv_append_fp4=lambda: fkv.kv_append_fp4(x, x, slots, sc, sc, kc, kc.clone(), stream=stream),
        kv_append_fp4_tag_check=lambda: fkv.kv_append_fp4_tag_check(x, x, slots, sc, sc, kc, kc.clone(), tags, ptr, idx, idx.clone(), mask, stream=stream),
        kv_gather=lambda: fkv.kv_gather(kc, kc, slots, x, k, sc, sc, stream=stream),
        qk_norm_rope=lambda: fkv.qk_norm_rope(q, k, i32(3), z(64, dt=torch.float32), q, k, stream=stream),
        kv_step_tables=lambda: fkv.kv_step_tables(i32(3), i32(3), i32(3, 2), i32(3, 2), i32(4), i32(1), tags, 16, i32(3), i32(3), mask, ptr, idx, idx.clone(),
                                                  i32(4), slots, i32(3), i32(1), fkv.alloc_step_tables_workspace(3), stream=stream),
        paged_decode_attn=lambda: fkv.paged_decode_attn(q, kc, kc, ptr, idx, i32(3), 0.1, q.clone(), z(256, dt=torch.uint8), k_scale=sc, v_scale=sc,
                                                        stream=stream))


def test_the_interpreter_lock_is_released():
    """CPython's own check of the lock stands in for the entry points: its 0 (not
    held) is their success, its 1 their first error."""
    check = ctypes.pythonapi.PyGILState_Check
    check.restype = ctypes.c_int
    assert check() == 1                                          # a PyDLL call keeps the lock
    with entry_points(ctypes.cast(check, ctypes.c_void_p).value):
        for f in calls().values():
            f()
    assert check() == 1


class OddStream:
    cuda_stream = "not a handle"


@pytest.mark.parametrize("stream", [2 ** 70, -2 ** 70, OddStream(), "a stream", object()], ids=["past64", "below64", "attribute", "text", "object"])
def test_a_stream_that_is_none_is_refused(stream):
    import fp8_paged_kv_decode_gb300 as fkv
    check = ctypes.cast(ctypes.pythonapi.PyGILState_Check, ctypes.c_void_p).value      # (so that nothing is launched)
    with entry_points(check):
        for f in calls(stream=None).values():
            f()
        for f in calls(stream=stream).values():
            with pytest.raises(fkv.FkvError, match="stream"):
                f()


def test_only_uint8_rows_of_72_are_fp4():
    """An e4m3 tensor's last dimension is its head_dim: 72 is not supported."""
    import torch
    import fp8_paged_kv_decode_gb300 as fkv
    z = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt, device="cuda")   # noqa: E731
    sc, k8 = z(2, dt=torch.float32) + 1, z(4, 2, 16, 72, dt=torch.uint8)
    ke = k8.view(torch.float8_e4m3fn)
    slots, ptr, idx, lens = z(3, dt=torch.int64), z(2, dt=torch.int32), z(1, dt=torch.int32), z(1, dt=torch.int32)
    ws = fkv.alloc_workspace(1, 4, 2, fkv.KV_FP4)
    for kc, vc in ((ke, ke), (ke, k8), (k8, ke)):
        with pytest.raises(fkv.FkvError):
            fkv.kv_gather(kc, vc, slots, z(3, 2, D), z(3, 2, D), sc, sc)
        with pytest.raises(fkv.FkvError):
            fkv.kv_gather(kc, vc, slots, z(3, 2, 72), z(3, 2, 72), sc, sc)
        for d in (D, 72):
            q = z(1, 4, d)
            with pytest.raises(fkv.FkvError):
                fkv.paged_decode_attn(q, kc, vc, ptr, idx, lens, 0.1, q.clone(), ws, k_scale=sc, v_scale=sc)
            with pytest.raises(fkv.FkvError):
                fkv.paged_decode_attn_noalloc(q, kc, vc, ptr, idx, lens, 0.1, q.clone(), k_scale=sc, v_scale=sc)
    with pytest.raises(fkv.FkvError):
        fkv.kv_page_realloc(z(4, dt=torch.int32), idx, idx.clone(), ke, ke)
