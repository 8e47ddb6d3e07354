"""The checks that the Python binding makes itself, on the CPU: tensors that say
they are on a GPU, and a library that only records its calls."""
import pytest

import fp8_paged_kv_decode_gb300 as fkv


class OnGpu:
    """A CPU tensor that says it is a CUDA tensor."""

    def __init__(self, t):
        self.t = t

    def __getattr__(self, name):
        return True if name == "is_cuda" else getattr(self.t, name)


class Recorder:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        return lambda *a: (self.calls.append((name, a)), 0)[1]


@pytest.fixture
def lib(monkeypatch):
    r = Recorder()
    monkeypatch.setattr(fkv, "load_library", lambda: r)
    return r


def z(*shape, dt="bfloat16"):
    import torch
    return OnGpu(torch.zeros(*shape, dtype=getattr(torch, dt)))


def attn(kind="fp4", **over):
    pool = {"fp4": dict(k_cache=z(5, 4, 16, 72, dt="uint8"), v_cache=z(5, 4, 16, 72, dt="uint8")),
            "fp8": dict(k_cache=z(5, 4, 16, 128, dt="uint8"), v_cache=z(5, 4, 16, 128, dt="float8_e4m3fn")),
            "bf16": dict(k_cache=z(5, 4, 16, 128), v_cache=z(5, 4, 16, 128))}[kind]
    a = dict(q=z(3, 8, 128), **pool, page_indptr=z(4, dt="int32"), page_indices=z(7, dt="int32"), seq_lens=z(3, dt="int32"), sm_scale=0.1, out=z(3, 8, 128),
             k_scale=z(4, dt="float32"), v_scale=z(4, dt="float32"), abort_mask=z(3, dt="uint8"), stream=0)
    a.update(over)
    return a


@pytest.mark.parametrize("kind,fmt", [("fp4", 2), ("fp8", 0), ("bf16", 1)])
def test_noalloc_passes_its_arguments(lib, kind, fmt):
    a = attn(kind, abort_mask=None)
    fkv.paged_decode_attn_noalloc(**a)
    (name, c), = lib.calls
    p = lambda k: a[k].data_ptr()                                                # noqa: E731
    assert name == "paged_decode_attn_noalloc" and c == (
        p("q"), 3, 8, p("k_cache"), p("v_cache"), fmt, None if fmt == 1 else p("k_scale"), None if fmt == 1 else p("v_scale"), 5, 4, 16, 128,
        p("page_indptr"), p("page_indices"), 7, p("seq_lens"), None, 0.1, p("out"), 0)


SCALES = [dict(k_scale=z(3, dt="float32")), dict(v_scale=z(1, dt="float32")), dict(k_scale=z(4, dt="float64")), dict(v_scale=z(4)), dict(k_scale=None)]
SIZES = [dict(seq_lens=z(2, dt="int32")), dict(seq_lens=z(3, dt="int64")), dict(abort_mask=z(2, dt="uint8")), dict(abort_mask=z(3, dt="bool")),
         dict(page_indptr=z(4, dt="int64")), dict(page_indptr=z(3, dt="int32")), dict(page_indices=z(7, dt="int64")), dict(out=z(3, 8, 64)),
         dict(out=z(3, 8, 128, dt="float32")), dict(q=z(3, 8, 128, dt="float16")), dict(v_cache=z(4, 4, 16, 128, dt="uint8")), dict(v_cache=z(5, 4, 16, 72)),
         dict(v_cache=z(5, 4, 16, 128, dt="float32"))]


@pytest.mark.parametrize("kind", ["fp4", "fp8", "bf16"])
@pytest.mark.parametrize("i", range(len(SCALES) + len(SIZES)))
def test_noalloc_refusals(lib, kind, i):
    """Nothing shorter than what the kernels read, and no other type, reaches them."""
    over = (SCALES + SIZES)[i]
    if kind == "bf16" and i < len(SCALES):                       # ignored there
        fkv.paged_decode_attn_noalloc(**attn(kind, **over))
        assert len(lib.calls) == 1
        return
    with pytest.raises(fkv.FkvError):
        fkv.paged_decode_attn_noalloc(**attn(kind, **over))
    assert not lib.calls


@pytest.mark.parametrize("row,dt,fmt", [(72, "uint8", 2), (128, "uint8", 0), (128, "float8_e4m3fn", 0), (128, "bfloat16", 1)])
def test_realloc_pools(lib, row, dt, fmt):
    """A scrub writes whole pages of both pools, so both have to hold every tagged page in one format."""
    tags, pages, new, pool = z(5, dt="int32"), z(2, dt="int32"), z(2, dt="int32"), z(5, 4, 16, row, dt=dt)
    fkv.kv_page_realloc(tags, pages, new, pool, z(5, 4, 16, row, dt=dt), stream=0)
    assert [c[1][7] for c in lib.calls] == [fmt]
    for kc, vc in ((z(4, 4, 16, row, dt=dt), z(4, 4, 16, row, dt=dt)), (pool, z(4, 4, 16, row, dt=dt)), (pool, z(5, 4, 16, row, dt="float32")), (pool, None),
                   (None, pool), (z(5, 4, 16, row, dt="float32"), z(5, 4, 16, row, dt="float32")),
                   (pool, z(5, 4, 16, row, dt="uint8" if fmt == 1 else "bfloat16"))):
        with pytest.raises(fkv.FkvError):
            fkv.kv_page_realloc(tags, pages, new, kc, vc, stream=0)
    assert len(lib.calls) == 1


@pytest.fixture
def no_module(monkeypatch, tmp_path):
    """As after a change of torch: the marshalling module has not been built for it."""
    from fp8_paged_kv_decode_gb300 import _build
    monkeypatch.setattr(fkv, "_bind", None)
    monkeypatch.setattr(_build, "bind_path", lambda: str(tmp_path / "_fkv_bind.none.so"))


@pytest.mark.parametrize("kind", ["fp4", "fp8", "bf16"])
def test_attention_needs_the_library_alone(lib, no_module, kind):
    a, ws = attn(kind), z(1024, dt="uint8")
    assert fkv.paged_decode_attn(**a, workspace=ws) is a["out"]
    fkv.paged_decode_attn_noalloc(**a)
    (n0, c0), (n1, c1) = lib.calls
    assert n0 == "paged_decode_attn" and c0 == c1[:-1] + (ws.data_ptr(), 1024, 0)
    with pytest.raises(fkv.FkvError, match="not built"):
        fkv.kv_gather(a["k_cache"], a["v_cache"], a["seq_lens"], a["out"], a["out"])


def test_the_module_belongs_to_one_torch(monkeypatch):
    """Another torch version is another file, so that one built before is neither loaded nor taken as built."""
    import torch
    from fp8_paged_kv_decode_gb300 import _build
    here = _build.bind_path()
    assert here.endswith(".so") and str(torch.__version__) in here
    monkeypatch.setattr(torch, "__version__", "99.0")
    assert _build.bind_path() != here and _build._stale(_build.bind_path(), [])


def test_a_variant_build_brings_the_module(monkeypatch, tmp_path):
    """A library built elsewhere is called through the module too."""
    from fp8_paged_kv_decode_gb300 import _build
    ran = []

    def run(cmd, **kw):
        ran.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()
        return type("R", (), dict(returncode=0, stdout="", stderr=""))
    monkeypatch.setattr(_build, "bind_path", lambda: str(tmp_path / "_fkv_bind.new.so"))
    monkeypatch.setattr(_build.subprocess, "run", run)
    out = str(tmp_path / "libvariant.so")
    assert _build.build(out_lib=out, build_dir=str(tmp_path / "b")) == out
    assert (tmp_path / "_fkv_bind.new.so").exists() and len(ran) == len(_build.SOURCES) + 2
    n = len(ran)
    _build.build(out_lib=out, build_dir=str(tmp_path / "b"), force=True)
    assert len(ran) == n + len(_build.SOURCES) + 1               # and is not built again for it
