// bind.cpp -- argument marshalling of the calls a decode step makes.
//
// The checks of a call (type, device, shape and layout of each tensor) and the
// conversion of its arguments cost 4-9 us a call in Python, as long as the
// kernels of a decode step run, so the step's calls do both here.  Nothing is
// computed: each function checks tensor metadata and calls the C entry point of
// the same name, whose address the package passes in after loading the library.
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAStream.h>

#include "../../include/fkv.h"

namespace {

PyObject *g_error = nullptr;                 // the package's FkvError
decltype(&fkv_status_string) g_status_string = nullptr;
decltype(&kv_append_fp4) g_append = nullptr;
decltype(&kv_append_fp4_tag_check) g_append_check = nullptr;
decltype(&kv_gather) g_gather = nullptr;
decltype(&qk_norm_rope) g_rope = nullptr;
decltype(&kv_step_tables) g_tables = nullptr;
decltype(&paged_decode_attn) g_attn = nullptr;
decltype(&kv_append_rope) g_append_rope = nullptr;
decltype(&paged_tree_attn) g_tree = nullptr;
decltype(&paged_window_attn) g_window = nullptr;
decltype(&kv_tree_commit) g_commit = nullptr;

struct Refused {
    const char *why;
};
void need(bool ok, const char *why) {
    if (!ok) throw Refused{why};
}

using at::ScalarType;
constexpr ScalarType kI32 = ScalarType::Int, kU32 = ScalarType::UInt32, kI64 = ScalarType::Long, kU8 = ScalarType::Byte,
                     kF32 = ScalarType::Float, kB16 = ScalarType::BFloat16, kE4M3 = ScalarType::Float8_e4m3fn;

// A positional argument as a tensor, or null for None where that is allowed.
const at::Tensor *tensor(PyObject *o, bool optional = false) {
    if (optional && o == Py_None) return nullptr;
    need(THPVariable_Check(o), "a tensor was expected");
    return &THPVariable_Unpack(o);
}

// The device a call launches on: its first tensor's, which has to be current.
int device_of(const at::Tensor &t) {
    need(t.is_cuda() && t.get_device() == c10::cuda::current_device(),
         "tensors must be contiguous CUDA tensors of the current device");
    return static_cast<int>(t.get_device());
}
void here(int dev, std::initializer_list<const at::Tensor *> ts) {
    for (const at::Tensor *t : ts)
        need(!t || (t->is_cuda() && t->get_device() == dev && t->is_contiguous()),
             "tensors must be contiguous CUDA tensors of the current device");
}
void *ptr(const at::Tensor *t) { return t ? t->data_ptr() : nullptr; }
bool is(const at::Tensor &t, ScalarType s) { return t.scalar_type() == s; }
bool tag32(const at::Tensor &t) { return is(t, kI32) || is(t, kU32); }
bool shape3(const at::Tensor &t, int64_t a, int64_t b, int64_t c) {
    return t.dim() == 3 && t.size(0) == a && t.size(1) == b && t.size(2) == c;
}
int32_t i32(int64_t v) {
    need(v >= 0 && v <= 0x7FFFFFFF, "a size does not fit 32 bits");
    return static_cast<int32_t>(v);
}

// The stream argument: None (the current stream), a torch stream or a handle.
void *stream_of(PyObject *o, int dev) {
    if (o == Py_None) return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream();
    PyObject *h = PyObject_HasAttrString(o, "cuda_stream") ? PyObject_GetAttrString(o, "cuda_stream") : PyNumber_Long(o);
    need(h != nullptr, "stream must be a torch.cuda.Stream or a handle");
    void *s = PyLong_AsVoidPtr(h);
    Py_DECREF(h);
    need(s || !PyErr_Occurred(), "stream must be a torch.cuda.Stream or a handle");
    return s;
}
double number(PyObject *o) {
    const double v = PyFloat_AsDouble(o);
    need(!(v == -1.0 && PyErr_Occurred()), "a number was expected");
    return v;
}
int64_t integer(PyObject *o) {
    PyObject *n = PyNumber_Index(o);
    need(n != nullptr, "a whole number was expected");
    const long long v = PyLong_AsLongLong(n);
    Py_DECREF(n);
    need(!(v == -1 && PyErr_Occurred()), "a whole number was expected");
    return v;
}

// Runs a C entry point with the interpreter lock released, as ctypes does: a
// launch may wait (for room in the launch queue, for a module's first load), and
// what it waits for may be a stream's host callback in Python.  Its arguments
// are plain values by then.
struct Unlocked {
    PyThreadState *state = PyEval_SaveThread();
    ~Unlocked() { PyEval_RestoreThread(state); }
};
template <typename F, typename... A>
fkv_status call(F f, A... a) {
    const Unlocked u;
    return f(a...);
}

template <typename F>
PyObject *guarded(const char *name, Py_ssize_t n, Py_ssize_t want, F f) {
    fkv_status st;
    try {
        need(n == want, "wrong number of arguments");
        st = f();
    } catch (const Refused &r) {
        PyErr_Clear();
        PyErr_SetString(g_error, r.why);
        return nullptr;
    } catch (const std::exception &e) {
        PyErr_SetString(g_error, e.what());
        return nullptr;
    }
    if (st != FKV_OK) {
        PyErr_Format(g_error, "%s failed: %s (status %d)", name, g_status_string(st), static_cast<int>(st));
        return nullptr;
    }
    Py_RETURN_NONE;
}

// ---------------------------------------------------------------------------
// the 4-bit append
// ---------------------------------------------------------------------------
struct Append {
    const at::Tensor *k, *v, *slots, *ks, *vs, *kc, *vc;
    int dev;
    int32_t pages, heads, page, n;
};
Append append_args(PyObject *const *a) {
    Append p{tensor(a[0]), tensor(a[1]), tensor(a[2]), tensor(a[3]), tensor(a[4]), tensor(a[5]), tensor(a[6]), 0, 0, 0, 0, 0};
    p.dev = device_of(*p.kc);
    here(p.dev, {p.k, p.v, p.slots, p.ks, p.vs, p.kc, p.vc});
    need(is(*p.k, kB16) && is(*p.v, kB16), "k_new/v_new must be bf16");
    need(is(*p.slots, kI64), "slot_mapping must be int64");
    need(is(*p.kc, kU8) && is(*p.vc, kU8) && p.kc->dim() == 4 && p.kc->size(3) == FKV_FP4_ROW_BYTES &&
             p.vc->sizes() == p.kc->sizes(),
         "FP4 caches must both be uint8 [P][Hkv][S][72]");
    p.pages = i32(p.kc->size(0));
    p.heads = i32(p.kc->size(1));
    p.page = i32(p.kc->size(2));
    need(is(*p.ks, kF32) && is(*p.vs, kF32) && p.ks->numel() == p.heads && p.vs->numel() == p.heads,
         "scales must be float32 [Hkv]");
    p.n = i32(p.slots->numel());
    need(shape3(*p.k, p.n, p.heads, 128) && shape3(*p.v, p.n, p.heads, 128), "k_new/v_new must be [N][Hkv][128]");
    return p;
}

PyObject *py_append(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded("kv_append_fp4", n, 8, [&] {
        const Append p = append_args(a);
        return call(g_append, ptr(p.k), ptr(p.v), static_cast<const int64_t *>(ptr(p.slots)), p.n,
                    static_cast<const float *>(ptr(p.ks)), static_cast<const float *>(ptr(p.vs)),
                    static_cast<uint8_t *>(ptr(p.kc)), static_cast<uint8_t *>(ptr(p.vc)), p.pages, p.heads, p.page,
                    128, stream_of(a[7], p.dev));
    });
}

PyObject *py_append_check(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded("kv_append_fp4_tag_check", n, 13, [&] {
        const Append p = append_args(a);
        const at::Tensor *tags = tensor(a[7]), *indptr = tensor(a[8]), *indices = tensor(a[9]), *expected = tensor(a[10]),
                         *mask = tensor(a[11]);
        here(p.dev, {tags, indptr, indices, expected, mask});
        need(tag32(*tags) && expected->scalar_type() == tags->scalar_type(), "tags must be 32-bit, both of one dtype");
        need(tags->numel() == p.pages, "page_tags must have one entry per page of the pool");
        need(is(*indptr, kI32) && is(*indices, kI32), "CSR must be int32");
        const int64_t batch = indptr->numel() - 1, nnz = indices->numel();
        need(batch >= 0 && is(*mask, kU8) && mask->numel() == batch && expected->numel() == nnz,
             "abort_mask must be uint8 [B], expected_tags parallel to page_indices");
        return call(g_append_check, ptr(p.k), ptr(p.v), static_cast<const int64_t *>(ptr(p.slots)), p.n,
                    static_cast<const float *>(ptr(p.ks)), static_cast<const float *>(ptr(p.vs)),
                    static_cast<uint8_t *>(ptr(p.kc)), static_cast<uint8_t *>(ptr(p.vc)), p.pages, p.heads,
                    p.page, 128, static_cast<const uint32_t *>(ptr(tags)),
                    static_cast<const int32_t *>(ptr(indptr)), static_cast<const int32_t *>(ptr(indices)),
                    static_cast<const uint32_t *>(ptr(expected)), i32(batch), nnz,
                    static_cast<uint8_t *>(ptr(mask)), stream_of(a[12], p.dev));
    });
}

// The format of a pair of caches, with its scales checked.
bool bytes8(const at::Tensor &t) { return is(t, kU8) || is(t, kE4M3); }
int32_t cache_format(const at::Tensor &kc, const at::Tensor &vc, const at::Tensor *ks, const at::Tensor *vs) {
    need(kc.dim() == 4 && vc.sizes() == kc.sizes(), "k_cache and v_cache shapes differ");
    if (is(kc, kB16)) {
        need(is(vc, kB16), "k_cache and v_cache types differ");
        return FKV_KV_BF16;
    }
    need(bytes8(kc) && bytes8(vc), "cache must be uint8 (e4m3, or FP4 rows of 72) or bf16");
    need(ks && vs && is(*ks, kF32) && is(*vs, kF32) && ks->numel() >= kc.size(1) && vs->numel() >= kc.size(1),
         "scales must be float32 [Hkv]");
    return is(kc, kU8) && is(vc, kU8) && kc.size(3) == FKV_FP4_ROW_BYTES ? FKV_KV_FP4 : FKV_KV_FP8_E4M3;
}

PyObject *py_gather(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded("kv_gather", n, 8, [&] {
        const at::Tensor *kc = tensor(a[0]), *vc = tensor(a[1]), *slots = tensor(a[2]), *ko = tensor(a[3]), *vo = tensor(a[4]),
                         *ks = tensor(a[5], true), *vs = tensor(a[6], true);
        const int dev = device_of(*kc);
        here(dev, {kc, vc, slots, ko, vo, ks, vs});
        const int32_t kv = cache_format(*kc, *vc, ks, vs);
        need(is(*slots, kI64), "slots must be int64");
        const int64_t rows = slots->numel(), heads = kc->size(1), dim = kv == FKV_KV_FP4 ? 128 : kc->size(3);
        need(is(*ko, kB16) && is(*vo, kB16) && shape3(*ko, rows, heads, dim) && shape3(*vo, rows, heads, dim),
             "k_out/v_out must be bf16 [N][Hkv][128]");
        return call(g_gather, ptr(kc), ptr(vc), kv, static_cast<const float *>(ptr(ks)), static_cast<const float *>(ptr(vs)),
                    static_cast<const int64_t *>(ptr(slots)), i32(rows), ptr(ko), ptr(vo), i32(kc->size(0)),
                    i32(heads), i32(kc->size(2)), i32(dim), stream_of(a[7], dev));
    });
}

// The token stride of bf16 [N][H][dim] whose head rows lie together.
int64_t head_rows(const at::Tensor &t, int dev, int64_t n, int64_t h, int64_t dim) {
    need(is(t, kB16) && t.is_cuda() && t.get_device() == dev && shape3(t, n, h, dim),
         "q/k and outputs must be bf16 [N][H][128] on the current device");
    if (n == 0) return h * dim;
    need(t.stride(2) == 1 && (h == 1 || t.stride(1) == dim), "head rows must be contiguous");
    return n == 1 ? h * dim : t.stride(0);
}

// q, k, positions, inv_freq, q_out, k_out, q_weight, k_weight, eps, axis_map, interleaved, rot_scale, stream
PyObject *py_rope(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded("qk_norm_rope", n, 13, [&] {
        const at::Tensor *q = tensor(a[0]), *k = tensor(a[1], true), *pos = tensor(a[2]), *freq = tensor(a[3]),
                         *qo = tensor(a[4]), *ko = tensor(a[5], true), *qw = tensor(a[6], true), *kw = tensor(a[7], true),
                         *map = tensor(a[9], true);
        const int dev = device_of(*pos);
        here(dev, {pos, freq, qw, kw, map});
        need(q->dim() == 3, "q must be bf16 [N][H][128]");
        need((k == nullptr) == (ko == nullptr) && (!k || k->dim() == 3), "k and k_out go together, both [N][Hkv][128]");
        const int64_t rows = q->size(0), hq = q->size(1), dim = q->size(2), hk = k ? k->size(1) : 0;
        const int64_t qs = head_rows(*q, dev, rows, hq, dim), qos = head_rows(*qo, dev, rows, hq, dim);
        const int64_t ks = k ? head_rows(*k, dev, rows, hk, dim) : 0, kos = k ? head_rows(*ko, dev, rows, hk, dim) : 0;
        for (const at::Tensor *w : {qw, kw}) need(!w || (is(*w, kB16) && w->numel() == dim), "weights must be bf16 [128]");
        need(is(*pos, kI32) && (pos->dim() == 1 || pos->dim() == 2) && pos->size(-1) == rows,
             "positions must be int32 [N] or [axes][N]");
        need(is(*freq, kF32) && freq->dim() == 1, "inv_freq must be float32 [R/2]");
        need(!map || (is(*map, kU8) && map->numel() == freq->numel()), "axis_map must be uint8 [R/2]");
        const int inter = PyObject_IsTrue(a[10]);
        need(inter >= 0, "interleaved must be true or false");
        return call(g_rope, ptr(q), qs, i32(hq), ptr(k), ks, i32(hk), ptr(qo), qos, ptr(ko), kos, i32(rows), ptr(qw), ptr(kw),
                    static_cast<float>(number(a[8])), static_cast<const int32_t *>(ptr(pos)),
                    pos->dim() == 1 ? 1 : i32(pos->size(0)), static_cast<const float *>(ptr(freq)),
                    static_cast<const uint8_t *>(ptr(map)), i32(2 * freq->numel()), inter,
                    static_cast<float>(number(a[11])), i32(dim), stream_of(a[12], dev));
    });
}

// cached, new, table, table tags, free pages, free count, page tags, page size, step lens, cached out, refused,
// page indptr, page indices, expected, token indptr, slots, positions, free left, workspace, stream
PyObject *py_tables(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded("kv_step_tables", n, 20, [&] {
        const at::Tensor *t[19];
        for (int i = 0; i < 19; ++i) t[i] = i == 7 ? nullptr : tensor(a[i]);
        const int dev = device_of(*t[0]);
        for (int i = 0; i < 19; ++i) here(dev, {t[i]});
        for (int i : {0, 1, 2, 4, 5, 8, 9, 11, 12, 14, 16, 17})
            need(is(*t[i], kI32), "lengths, tables, free list, indptr, indices and positions must be int32");
        need(tag32(*t[6]) && t[3]->scalar_type() == t[6]->scalar_type() && t[13]->scalar_type() == t[6]->scalar_type(),
             "tags must be 32-bit, of one dtype");
        need(is(*t[15], kI64) && is(*t[10], kU8), "slot_mapping must be int64, refused uint8");
        const int64_t batch = t[0]->numel();
        need(t[2]->dim() == 2 && t[2]->size(0) == batch && t[3]->sizes() == t[2]->sizes(),
             "block_table and block_tags must be [B][max_blocks]");
        need(t[1]->numel() == batch && t[8]->numel() == batch && t[9]->numel() == batch && t[10]->numel() == batch &&
                 t[11]->numel() == batch + 1 && t[14]->numel() == batch + 1,
             "one length per request, indptr arrays of B + 1");
        need(t[13]->numel() == t[12]->numel() && t[16]->numel() == t[15]->numel() && t[5]->numel() == 1 &&
                 t[17]->numel() == 1,
             "expected_tags parallel to page_indices, positions to slot_mapping; free counts of one value");
        auto i = [&](int k) { return static_cast<int32_t *>(ptr(t[k])); };
        auto u = [&](int k) { return static_cast<uint32_t *>(ptr(t[k])); };
        const int64_t page = integer(a[7]);
        need(page > 0 && page <= 0x7FFFFFFF, "page_size must be positive");
        return call(g_tables, i(0), i(1), i32(batch), i(2), u(3), i32(t[2]->size(1)), i(4), i32(t[4]->numel()), i(5), u(6),
                    i32(t[6]->numel()), static_cast<int32_t>(page), i(8), i(9), static_cast<uint8_t *>(ptr(t[10])),
                    i(11), i(12), u(13), i32(t[12]->numel()), i(14), static_cast<int64_t *>(ptr(t[15])), i(16),
                    i32(t[15]->numel()), i(17), ptr(t[18]), t[18]->nbytes(), stream_of(a[19], dev));
    });
}

// q, k_cache, v_cache, indptr, indices, seq_lens, sm_scale, out, workspace, k_scale, v_scale, abort_mask, stream
PyObject *py_attn(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded("paged_decode_attn", n, 13, [&] {
        const at::Tensor *q = tensor(a[0]), *kc = tensor(a[1]), *vc = tensor(a[2]), *indptr = tensor(a[3]),
                         *indices = tensor(a[4]), *lens = tensor(a[5]), *out = tensor(a[7]), *ws = tensor(a[8]),
                         *ks = tensor(a[9], true), *vs = tensor(a[10], true), *mask = tensor(a[11], true);
        const int dev = device_of(*q);
        here(dev, {q, kc, vc, indptr, indices, lens, out, ws, ks, vs, mask});
        const int32_t kv = cache_format(*kc, *vc, ks, vs);
        need(is(*q, kB16) && is(*out, kB16), "q/out must be bf16");
        need(is(*lens, kI32), "seq_lens must be int32");
        need(!mask || is(*mask, kU8), "abort_mask must be uint8");
        need(tag32(*indptr) && tag32(*indices), "CSR must be int32");
        need(q->dim() == 3 && out->sizes() == q->sizes(), "shape mismatch");
        const int64_t batch = q->size(0), dim = q->size(2);
        need((kv == FKV_KV_FP4 ? 128 : kc->size(3)) == dim && indptr->numel() == batch + 1 && lens->numel() >= batch &&
                 (!mask || mask->numel() >= batch),
             "shape mismatch");
        const bool scaled = kv != FKV_KV_BF16;
        return call(g_attn, ptr(q), i32(batch), i32(q->size(1)), ptr(kc), ptr(vc), kv,
                    scaled ? static_cast<const float *>(ptr(ks)) : nullptr,
                    scaled ? static_cast<const float *>(ptr(vs)) : nullptr, i32(kc->size(0)), i32(kc->size(1)),
                    i32(kc->size(2)), i32(dim), static_cast<const int32_t *>(ptr(indptr)),
                    static_cast<const int32_t *>(ptr(indices)), indices->numel(),
                    static_cast<const int32_t *>(ptr(lens)), static_cast<const uint8_t *>(ptr(mask)),
                    static_cast<float>(number(a[6])), ptr(out), ptr(ws), ws->nbytes(), stream_of(a[12], dev));
    });
}

// q, k, v, positions, inv_freq, slots, q_out, k_cache, v_cache, k_scale, v_scale, q_weight, k_weight, eps, axis_map,
// interleaved, rot_scale, stream
PyObject *py_append_rope(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded("kv_append_rope", n, 18, [&] {
        const at::Tensor *q = tensor(a[0], true), *k = tensor(a[1]), *v = tensor(a[2]), *pos = tensor(a[3]), *freq = tensor(a[4]),
                         *slots = tensor(a[5]), *qo = tensor(a[6], true), *kc = tensor(a[7]), *vc = tensor(a[8]),
                         *ks = tensor(a[9], true), *vs = tensor(a[10], true), *qw = tensor(a[11], true),
                         *kw = tensor(a[12], true), *map = tensor(a[14], true);
        const int dev = device_of(*kc);
        here(dev, {pos, freq, slots, kc, vc, ks, vs, qw, kw, map});
        const int32_t kv = cache_format(*kc, *vc, ks, vs);
        need((q == nullptr) == (qo == nullptr) && (!q || q->dim() == 3), "q and q_out go together, both [N][Hq][128]");
        need(is(*slots, kI64), "slot_mapping must be int64");
        const int64_t rows = slots->numel(), hk = kc->size(1), dim = kv == FKV_KV_FP4 ? 128 : kc->size(3), hq = q ? q->size(1) : 0;
        const int64_t qst = q ? head_rows(*q, dev, rows, hq, dim) : 0, qos = q ? head_rows(*qo, dev, rows, hq, dim) : 0;
        const int64_t kst = head_rows(*k, dev, rows, hk, dim), vst = head_rows(*v, dev, rows, hk, dim);
        for (const at::Tensor *w : {qw, kw}) need(!w || (is(*w, kB16) && w->numel() == dim), "weights must be bf16 [128]");
        need(is(*pos, kI32) && (pos->dim() == 1 || pos->dim() == 2) && pos->size(-1) == rows,
             "positions must be int32 [N] or [axes][N]");
        need(is(*freq, kF32) && freq->dim() == 1, "inv_freq must be float32 [R/2]");
        need(!map || (is(*map, kU8) && map->numel() == freq->numel()), "axis_map must be uint8 [R/2]");
        const int inter = PyObject_IsTrue(a[15]);
        need(inter >= 0, "interleaved must be true or false");
        const bool scaled = kv != FKV_KV_BF16;
        return call(g_append_rope, ptr(q), qst, i32(hq), ptr(k), kst, ptr(v), vst, i32(hk), ptr(qo), qos, i32(rows), ptr(qw), ptr(kw),
                    static_cast<float>(number(a[13])), static_cast<const int32_t *>(ptr(pos)),
                    pos->dim() == 1 ? 1 : i32(pos->size(0)), static_cast<const float *>(ptr(freq)),
                    static_cast<const uint8_t *>(ptr(map)), i32(2 * freq->numel()), inter, static_cast<float>(number(a[16])),
                    static_cast<const int64_t *>(ptr(slots)), kv, scaled ? static_cast<const float *>(ptr(ks)) : nullptr,
                    scaled ? static_cast<const float *>(ptr(vs)) : nullptr, ptr(kc), ptr(vc), i32(kc->size(0)), i32(kc->size(2)),
                    i32(dim), stream_of(a[17], dev));
    });
}

// The arguments that tree and window attention share.
struct Paged {
    const at::Tensor *q, *kc, *vc, *indptr, *indices, *lens, *out, *ws, *ks, *vs, *mask;
    int dev;
    int32_t kv, batch, dim;
};
Paged paged_args(PyObject *q, PyObject *kc, PyObject *vc, PyObject *indptr, PyObject *indices, PyObject *lens, PyObject *out,
                 PyObject *ws, PyObject *ks, PyObject *vs, PyObject *mask) {
    Paged p{tensor(q), tensor(kc), tensor(vc), tensor(indptr), tensor(indices), tensor(lens), tensor(out), tensor(ws),
            tensor(ks, true), tensor(vs, true), tensor(mask, true), 0, 0, 0, 0};
    p.dev = device_of(*p.q);
    here(p.dev, {p.q, p.kc, p.vc, p.indptr, p.indices, p.lens, p.out, p.ws, p.ks, p.vs, p.mask});
    p.kv = cache_format(*p.kc, *p.vc, p.ks, p.vs);
    need(is(*p.q, kB16) && is(*p.out, kB16), "q/out must be bf16");
    need(is(*p.lens, kI32), "seq_lens must be int32");
    need(!p.mask || is(*p.mask, kU8), "abort_mask must be uint8");
    need(tag32(*p.indptr) && tag32(*p.indices), "CSR must be int32");
    need(p.q->dim() == 3 && p.out->sizes() == p.q->sizes(), "shape mismatch");
    need(p.indptr->numel() >= 1, "page_indptr has batch + 1 entries");
    p.batch = i32(p.indptr->numel() - 1);
    p.dim = i32(p.q->size(2));
    need((p.kv == FKV_KV_FP4 ? 128 : p.kc->size(3)) == p.dim && p.lens->numel() == p.batch &&
             (!p.mask || p.mask->numel() == p.batch),
         "shape mismatch");
    if (p.kv == FKV_KV_BF16) p.ks = p.vs = nullptr;
    return p;
}
int32_t small(PyObject *o, const char *why) {
    const int64_t v = integer(o);
    need(v >= 0 && v <= 0x7FFFFFFF, why);
    return static_cast<int32_t>(v);
}

// q, k_cache, v_cache, indptr, indices, seq_lens, token_indptr, tree_mask, sm_scale, out, workspace, k_scale, v_scale,
// abort_mask, window, sinks, stream
PyObject *py_tree(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded("paged_tree_attn", n, 17, [&] {
        const Paged p = paged_args(a[0], a[1], a[2], a[3], a[4], a[5], a[9], a[10], a[11], a[12], a[13]);
        const at::Tensor *rows = tensor(a[6]), *mask = tensor(a[7]);
        here(p.dev, {rows, mask});
        need(is(*rows, kI32) && rows->numel() == p.batch + 1, "token_indptr must be int32 [B + 1]");
        need((is(*mask, kI64) || is(*mask, ScalarType::UInt64)) && (mask->dim() == 1 || mask->dim() == 2) &&
                 mask->size(0) == p.q->size(0) && (mask->dim() == 1 || mask->size(1) >= 1),
             "tree_mask must be int64 or uint64 [N] or [N][words]");
        return call(g_tree, ptr(p.q), i32(p.q->size(0)), i32(p.q->size(1)), ptr(p.kc), ptr(p.vc), p.kv,
                    static_cast<const float *>(ptr(p.ks)), static_cast<const float *>(ptr(p.vs)), i32(p.kc->size(0)),
                    i32(p.kc->size(1)), i32(p.kc->size(2)), p.dim, static_cast<const int32_t *>(ptr(p.indptr)),
                    static_cast<const int32_t *>(ptr(p.indices)), p.indices->numel(), static_cast<const int32_t *>(ptr(p.lens)),
                    p.batch, static_cast<const int32_t *>(ptr(rows)), static_cast<const uint64_t *>(ptr(mask)),
                    mask->dim() == 1 ? 1 : i32(mask->size(1)), small(a[14], "window must not be negative"),
                    small(a[15], "sinks must not be negative"), static_cast<const uint8_t *>(ptr(p.mask)),
                    static_cast<float>(number(a[8])), ptr(p.out), ptr(p.ws), p.ws->nbytes(), stream_of(a[16], p.dev));
    });
}

// q, k_cache, v_cache, indptr, indices, seq_lens, sm_scale, out, workspace, k_scale, v_scale, abort_mask, window, sinks,
// stream
PyObject *py_window(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded("paged_window_attn", n, 15, [&] {
        const Paged p = paged_args(a[0], a[1], a[2], a[3], a[4], a[5], a[7], a[8], a[9], a[10], a[11]);
        need(p.q->size(0) == p.batch, "shape mismatch");
        return call(g_window, ptr(p.q), p.batch, i32(p.q->size(1)), ptr(p.kc), ptr(p.vc), p.kv,
                    static_cast<const float *>(ptr(p.ks)), static_cast<const float *>(ptr(p.vs)), i32(p.kc->size(0)),
                    i32(p.kc->size(1)), i32(p.kc->size(2)), p.dim, static_cast<const int32_t *>(ptr(p.indptr)),
                    static_cast<const int32_t *>(ptr(p.indices)), p.indices->numel(), static_cast<const int32_t *>(ptr(p.lens)),
                    small(a[12], "window must be positive"), small(a[13], "sinks must not be negative"),
                    static_cast<const uint8_t *>(ptr(p.mask)), static_cast<float>(number(a[6])), ptr(p.out), ptr(p.ws),
                    p.ws->nbytes(), stream_of(a[14], p.dev));
    });
}

// k_cache, v_cache, indptr, indices, seq_lens, token_indptr, accepted, counts, lens_out, abort_mask, free_pages, free_count,
// free_left, page_tags, stream
PyObject *py_commit(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded("kv_tree_commit", n, 15, [&] {
        const at::Tensor *kc = tensor(a[0]), *vc = tensor(a[1]), *indptr = tensor(a[2]), *indices = tensor(a[3]), *lens = tensor(a[4]),
                         *rows = tensor(a[5]), *acc = tensor(a[6]), *counts = tensor(a[7]), *kept = tensor(a[8]),
                         *mask = tensor(a[9], true), *pages = tensor(a[10], true), *have = tensor(a[11], true),
                         *left = tensor(a[12], true), *tags = tensor(a[13], true);
        const int dev = device_of(*kc);
        here(dev, {kc, vc, indptr, indices, lens, rows, acc, counts, kept, mask, pages, have, left, tags});
        need(kc->dim() == 4 && vc->sizes() == kc->sizes(), "k_cache and v_cache shapes differ");
        const bool b16 = is(*kc, kB16);
        need(b16 ? is(*vc, kB16) : bytes8(*kc) && bytes8(*vc), "caches must both be uint8 (e4m3, or FP4 rows of 72) or bf16");
        const bool fp4 = is(*kc, kU8) && is(*vc, kU8) && kc->size(3) == FKV_FP4_ROW_BYTES;
        for (const at::Tensor *t : {indptr, indices, lens, rows, acc, counts, kept})
            need(is(*t, kI32), "CSR, lengths, token_indptr and accepted lists must be int32");
        const int64_t batch = indptr->numel() - 1;
        need(batch >= 0 && lens->numel() == batch && rows->numel() == batch + 1 && counts->numel() == batch &&
                 kept->numel() == batch && acc->dim() == 2 && acc->size(0) == batch,
             "one length, count and list per request, indptr arrays of B + 1");
        need(!mask || (is(*mask, kU8) && mask->numel() == batch), "abort_mask must be uint8 [B]");
        need((pages != nullptr) == (have != nullptr) && (pages != nullptr) == (left != nullptr) && (pages || !tags),
             "free_pages, free_count and free_left go together");
        for (const at::Tensor *t : {pages, have, left}) need(!t || is(*t, kI32), "the free list must be int32");
        need(!pages || (have->numel() == 1 && left->numel() == 1), "free counts of one value");
        need(!tags || (tag32(*tags) && tags->numel() == kc->size(0)), "page_tags must be 32-bit, one per page of the pool");
        return call(g_commit, ptr(kc), ptr(vc), b16 ? FKV_KV_BF16 : fp4 ? FKV_KV_FP4 : FKV_KV_FP8_E4M3, i32(kc->size(0)),
                    i32(kc->size(1)), i32(kc->size(2)), fp4 ? 128 : i32(kc->size(3)), static_cast<const int32_t *>(ptr(indptr)),
                    static_cast<const int32_t *>(ptr(indices)), indices->numel(), static_cast<const int32_t *>(ptr(lens)), i32(batch),
                    static_cast<const int32_t *>(ptr(rows)), 0x7FFFFFFF, static_cast<const int32_t *>(ptr(acc)), i32(acc->size(1)),
                    static_cast<const int32_t *>(ptr(counts)), static_cast<const uint8_t *>(ptr(mask)),
                    static_cast<int32_t *>(ptr(kept)), static_cast<int32_t *>(ptr(pages)), pages ? i32(pages->numel()) : 0,
                    static_cast<const int32_t *>(ptr(have)), static_cast<int32_t *>(ptr(left)), static_cast<uint32_t *>(ptr(tags)),
                    stream_of(a[14], dev));
    });
}

// setup(FkvError, status_string, append, append_check, gather, rope, tables, attn, append_rope, tree, window, commit): the
// exception and the C entry points' addresses.
PyObject *py_setup(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != 12) {
        PyErr_SetString(PyExc_TypeError, "setup takes 12 arguments");
        return nullptr;
    }
    void *f[12] = {};
    for (int i = 1; i < 12; ++i) {
        f[i] = PyLong_AsVoidPtr(a[i]);
        if (!f[i]) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "an entry point is missing");
            return nullptr;
        }
    }
    Py_INCREF(a[0]);
    Py_XDECREF(g_error);
    g_error = a[0];
    g_status_string = reinterpret_cast<decltype(g_status_string)>(f[1]);
    g_append = reinterpret_cast<decltype(g_append)>(f[2]);
    g_append_check = reinterpret_cast<decltype(g_append_check)>(f[3]);
    g_gather = reinterpret_cast<decltype(g_gather)>(f[4]);
    g_rope = reinterpret_cast<decltype(g_rope)>(f[5]);
    g_tables = reinterpret_cast<decltype(g_tables)>(f[6]);
    g_attn = reinterpret_cast<decltype(g_attn)>(f[7]);
    g_append_rope = reinterpret_cast<decltype(g_append_rope)>(f[8]);
    g_tree = reinterpret_cast<decltype(g_tree)>(f[9]);
    g_window = reinterpret_cast<decltype(g_window)>(f[10]);
    g_commit = reinterpret_cast<decltype(g_commit)>(f[11]);
    Py_RETURN_NONE;
}

#define FKV_METHOD(name, f) {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FKV_METHOD("setup", py_setup),
                         FKV_METHOD("kv_append_fp4", py_append),
                         FKV_METHOD("kv_append_fp4_tag_check", py_append_check),
                         FKV_METHOD("kv_gather", py_gather),
                         FKV_METHOD("qk_norm_rope", py_rope),
                         FKV_METHOD("kv_step_tables", py_tables),
                         FKV_METHOD("paged_decode_attn", py_attn),
                         FKV_METHOD("kv_append_rope", py_append_rope),
                         FKV_METHOD("paged_tree_attn", py_tree),
                         FKV_METHOD("paged_window_attn", py_window),
                         FKV_METHOD("kv_tree_commit", py_commit),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fkv_bind", "Argument marshalling of a decode step's calls.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fkv_bind() { return PyModule_Create(&module); }
