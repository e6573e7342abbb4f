// paged_torch.cpp -- the torch side of runtime.PagedKV: checks of the tensors,
// allocation of what the caller did not pass, and the call of the C entry point
// (include/ember.h, "paged key/value cache").  Marshalling only, as in ember.py;
// it is compiled because a small call's time is its marshalling: 16 us for a
// decode step of one token through ctypes, of which the kernel takes 4.5.
//
// The entry points come as addresses from the loaded library, so that this module
// serves whichever build of it ember.py loads.
#include "torch_args.h"

namespace {

decltype(&ember_paged_append) f_append = nullptr;
decltype(&ember_paged_decode) f_decode = nullptr;
decltype(&ember_paged_decode_workspace) f_workspace = nullptr;
decltype(&ember_paged_prefill) f_prefill = nullptr;
decltype(&ember_paged_decode_shared) f_shared = nullptr;
decltype(&ember_paged_decode_shared_workspace) f_shared_workspace = nullptr;

// One PagedKV: the C view of the cache and where its status word lives.
struct Cache {
    ember_paged_kv kv;
    int32_t* status;
    c10::DeviceIndex device;
    at::ScalarType dtype;
    Tensor k_pages, v_pages, table, status_word;
    ember_stream_t home = nullptr;   // the stream that status_word was allocated on
    // decode's workspace of the last (B, heads): the query is a function of these
    int64_t ws_rows = -1, ws_heads = -1;
    size_t ws_bytes = 0;
    int64_t shared_rows = -1, shared_heads = -1, shared_groups = -1;   // decode_shared's likewise
    size_t shared_bytes = 0;
};

// [n, heads, head_dim] whose rows hold the heads side by side.
struct Rows {
    void* p;
    int64_t ld;
};
Rows rows(const Cache& c, const Tensor& t, const char* what, at::ScalarType dtype, int64_t n, int64_t heads) {
    on_device(c, t, what);
    const int64_t D = c.kv.head_dim;
    if (t.dim() != 3 || t.size(0) != n || t.size(1) != heads || t.size(2) != D || t.scalar_type() != dtype)
        bad(std::string(what) + " must be " + c10::toString(dtype) + " [" + std::to_string(n) + ", " +
            std::to_string(heads) + ", " + std::to_string(D) + "], not " + describe(t));
    if (t.stride(2) != 1 || (heads > 1 && t.stride(1) != D)) bad(std::string(what) + ": a row's heads must lie side by side");
    return {t.data_ptr(), n > 1 ? t.stride(0) : heads * D};
}

void* pages(const Cache& c, const Tensor& t, const char* what) {
    on_device(c, t, what);
    const int64_t shape[4] = {c.kv.n_pages, c.kv.n_kv_heads, c.kv.page_size, c.kv.head_dim};
    const int64_t strides[4] = {c.kv.page_stride, c.kv.head_stride, c.kv.row_stride, 1};
    bool same = t.scalar_type() == c.dtype && t.sizes() == at::IntArrayRef(shape, 4);
    for (int i = 0; same && i < 4; ++i) same = shape[i] == 1 || t.stride(i) == strides[i];
    if (!same)
        bad(std::string(what) + " must keep the type, shape and strides that the cache was made with, not become " + describe(t));
    return t.data_ptr();
}

Cache& cache_of(PyObject* o) {
    auto* c = static_cast<Cache*>(PyCapsule_GetPointer(o, "ember.paged"));
    if (!c) throw python_error();
    // Where the tensors lie and whether they are what they were: at every call, since a tensor may
    // get other storage (t.data = ..) or be asked for its gradient at any time.
    if (c->k_pages.defined()) {
        no_gradient(c->k_pages, "k_pages");
        no_gradient(c->v_pages, "v_pages");
    }
    if (c->table.defined()) {
        c->kv.k = pages(*c, c->k_pages, "k_pages");
        c->kv.v = pages(*c, c->v_pages, "v_pages");
        c->kv.table = static_cast<const int32_t*>(flat(*c, c->table, "table", at::kInt, {c->kv.n_seqs, c->kv.table_width}));
    }
    return *c;
}

// out and lse, given or made
struct Outputs {
    Tensor out, lse;
    Rows r;
    float* lse_p = nullptr;
    bool out_given = false, lse_given = false;
    void done() const {
        if (out_given) written(out);
        if (lse_given) written(lse);
    }
};
Outputs outputs(const Cache& c, int64_t n, int64_t heads, PyObject* out, PyObject* lse, bool want_lse) {
    Outputs o;
    const int64_t D = c.kv.head_dim;
    if ((o.out_given = given(out))) {
        o.out = tensor(out, "out");
        o.r = rows(c, o.out, "out", c.dtype, n, heads);
    } else {
        o.out = make(c, {n, heads, D}, c.dtype);
        o.r = {o.out.data_ptr(), heads * D};
    }
    if ((o.lse_given = given(lse))) {
        o.lse = tensor(lse, "lse");
        o.lse_p = static_cast<float*>(flat(c, o.lse, "lse", at::kFloat, {n, heads}));
    } else if (want_lse) {
        o.lse = make(c, {n, heads}, at::kFloat);
        o.lse_p = static_cast<float*>(o.lse.data_ptr());
    }
    return o;
}
PyObject* answer(Outputs& o) {
    if (!o.lse.defined()) return THPVariable_Wrap(o.out);
    PyObject* t = PyTuple_New(2);
    if (!t) return nullptr;
    PyTuple_SET_ITEM(t, 0, THPVariable_Wrap(o.out));
    PyTuple_SET_ITEM(t, 1, THPVariable_Wrap(o.lse));
    return t;
}

// The call's stream.  A kernel on another one than status_word's may still raise an
// error when the cache is gone: the allocator keeps the word until then.
ember_stream_t stream_of(const Cache& c) {
    const c10::cuda::CUDAStream s = c10::cuda::getCurrentCUDAStream(c.device);
    auto* p = reinterpret_cast<ember_stream_t>(s.stream());
    if (c.status_word.defined() && p != c.home)
        c10::cuda::CUDACachingAllocator::recordStream(c.status_word.storage().data_ptr(), s);
    return p;
}

// append(cache, k, v, seqs, positions, cos, sin, q, q_norm, k_norm, eps, q_out)
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
    return guarded(nargs, 12, [&]() -> PyObject* {
        const Cache& c = cache_of(a[0]);
        const Tensor &k = tensor(a[1], "k"), &v = tensor(a[2], "v");
        const at::ScalarType dt = k.scalar_type();
        const int src = dt == at::kFloat ? EMBER_F32 : dt == at::kBFloat16 ? EMBER_BF16 : dt == at::kHalf ? EMBER_F16 : -1;
        if (src < 0) throw Bad{PyExc_TypeError, "q, k and v must be float32, bfloat16 or float16"};
        const int64_t n = k.dim() ? k.size(0) : 0, D = c.kv.head_dim, NKV = c.kv.n_kv_heads;
        const Rows kr = rows(c, k, "k", dt, n, NKV), vr = rows(c, v, "v", dt, n, NKV);
        const int32_t *seqs = ints(c, a[3], "seqs", n), *pos = ints(c, a[4], "positions", n);
        const Tensor &cos = tensor(a[5], "cos"), &sin = tensor(a[6], "sin");
        const int64_t n_pos = cos.dim() ? cos.size(0) : 0;
        const auto* cp = static_cast<const float*>(flat(c, cos, "cos", at::kFloat, {n_pos, D / 2}));
        const auto* sp = static_cast<const float*>(flat(c, sin, "sin", at::kFloat, {n_pos, D / 2}));
        auto norm = [&](PyObject* o, const char* what) {
            return given(o) ? static_cast<const uint16_t*>(flat(c, tensor(o, what), what, at::kBFloat16, {D})) : nullptr;
        };
        const uint16_t *qn = norm(a[8], "q_norm"), *kn = norm(a[9], "k_norm");
        const double eps = real(a[10]);
        const c10::cuda::OptionalCUDAGuard on(c10::Device(at::kCUDA, c.device));
        Rows qr{nullptr, 0}, orow{nullptr, 0};
        Tensor q_out;
        int64_t heads = 0;
        if (given(a[7])) {
            const Tensor& q = tensor(a[7], "q");
            heads = q.dim() == 3 ? q.size(1) : 0;
            qr = rows(c, q, "q", dt, n, heads);
            if (given(a[11])) {
                q_out = tensor(a[11], "q_out");
                orow = rows(c, q_out, "q_out", c.dtype, n, heads);
            } else {
                q_out = make(c, {n, heads, D}, c.dtype);
                orow = {q_out.data_ptr(), heads * D};
            }
        } else if (given(a[11])) {
            bad("q_out without q");
        }
        if (n > 0) {
            check(f_append(&c.kv, qr.p, kr.p, vr.p, src, qr.ld, kr.ld, vr.ld, count(n, "k"), count(heads, "q"), seqs, pos,
                           qn, kn, (float)eps, cp, sp, count(n_pos, "cos"), orow.p, orow.ld, c.status, stream_of(c)),
                  "ember_paged_append");
            written(c.k_pages);
            written(c.v_pages);
            if (given(a[11])) written(q_out);
        }
        if (!q_out.defined()) Py_RETURN_NONE;
        return THPVariable_Wrap(q_out);
    });
}

size_t workspace_of(Cache& c, int64_t B, int64_t heads) {
    if (c.ws_rows != B || c.ws_heads != heads) {
        c.ws_bytes = f_workspace(&c.kv, count(B, "q"), count(heads, "q"));
        c.ws_rows = B;
        c.ws_heads = heads;
    }
    return c.ws_bytes;
}

size_t shared_workspace_of(Cache& c, int64_t B, int64_t heads, int64_t groups) {
    if (c.shared_rows != B || c.shared_heads != heads || c.shared_groups != groups) {
        c.shared_bytes = f_shared_workspace(&c.kv, count(B, "q"), count(heads, "q"), count(groups, "shared"));
        c.shared_rows = B;
        c.shared_heads = heads;
        c.shared_groups = groups;
    }
    return c.shared_bytes;
}

// A workspace, given or made.
struct Workspace {
    Tensor t;
    void* p = nullptr;
    size_t bytes;
};
Workspace workspace(const Cache& c, PyObject* o, size_t need) {
    Workspace w;
    w.bytes = need;
    if (given(o)) {
        w.t = tensor(o, "workspace");
        on_device(c, w.t, "workspace");
        if (w.t.scalar_type() != at::kByte || !w.t.is_contiguous()) bad("workspace must be contiguous uint8");
        w.bytes = (size_t)w.t.numel();
    } else if (need) {
        w.t = make(c, {(int64_t)need}, at::kByte);
    }
    if (w.bytes) w.p = w.t.data_ptr();
    return w;
}

// decode(cache, q, lens, seqs, window, sinks, scale, out, lse, return_lse, workspace)
PyObject* decode(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
    return guarded(nargs, 11, [&]() -> PyObject* {
        Cache& c = cache_of(a[0]);
        const Tensor& q = tensor(a[1], "q");
        const int64_t B = q.dim() == 3 ? q.size(0) : 0, heads = q.dim() == 3 ? q.size(1) : 0;
        const Rows qr = rows(c, q, "q", c.dtype, B, heads);
        const int32_t *lens = ints(c, a[2], "lens", B), *seqs = given(a[3]) ? ints(c, a[3], "seqs", B) : nullptr;
        const int32_t window = number(a[4], "window"), sinks = number(a[5], "sinks");
        const double scale = given(a[6]) ? real(a[6]) : 1.0 / std::sqrt((double)c.kv.head_dim);
        const c10::cuda::OptionalCUDAGuard on(c10::Device(at::kCUDA, c.device));
        Outputs o = outputs(c, B, heads, a[7], a[8], truth(a[9]));
        if (B > 0) {
            const Workspace ws = workspace(c, a[10], workspace_of(c, B, heads));
            check(f_decode(&c.kv, qr.p, qr.ld, count(B, "q"), count(heads, "q"), seqs, lens, window, sinks, (float)scale, o.r.p,
                           o.r.ld, o.lse_p, ws.p, ws.bytes, c.status, stream_of(c)),
                  "ember_paged_decode");
            o.done();
        }
        return answer(o);
    });
}

// decode_shared(cache, q, lens, groups, shared, prefixes, seqs, scale, out, lse, return_lse, workspace)
PyObject* decode_shared(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
    return guarded(nargs, 12, [&]() -> PyObject* {
        Cache& c = cache_of(a[0]);
        const Tensor &q = tensor(a[1], "q"), &st = any_tensor(a[4], "shared");
        const int64_t B = q.dim() == 3 ? q.size(0) : 0, heads = q.dim() == 3 ? q.size(1) : 0;
        const int64_t groups = st.dim() == 1 ? st.size(0) : 0;
        const Rows qr = rows(c, q, "q", c.dtype, B, heads);
        const int32_t *lens = ints(c, a[2], "lens", B), *cu = ints(c, a[3], "groups", groups + 1);
        const int32_t *shared = ints(c, a[4], "shared", groups), *prefixes = ints(c, a[5], "prefixes", groups);
        const int32_t* seqs = given(a[6]) ? ints(c, a[6], "seqs", B) : nullptr;
        const double scale = given(a[7]) ? real(a[7]) : 1.0 / std::sqrt((double)c.kv.head_dim);
        const c10::cuda::OptionalCUDAGuard on(c10::Device(at::kCUDA, c.device));
        Outputs o = outputs(c, B, heads, a[8], a[9], truth(a[10]));
        if (B > 0) {
            const Workspace ws = workspace(c, a[11], shared_workspace_of(c, B, heads, groups));
            check(f_shared(&c.kv, qr.p, qr.ld, count(B, "q"), count(heads, "q"), seqs, lens, cu, shared, prefixes,
                           count(groups, "shared"), (float)scale, o.r.p, o.r.ld, o.lse_p, ws.p, ws.bytes, c.status, stream_of(c)),
                  "ember_paged_decode_shared");
            o.done();
        }
        return answer(o);
    });
}

// prefill(cache, q, cu, lens, seqs, window, sinks, scale, out, lse, return_lse)
PyObject* prefill(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
    return guarded(nargs, 11, [&]() -> PyObject* {
        const Cache& c = cache_of(a[0]);
        const Tensor &q = tensor(a[1], "q"), &lt = tensor(a[3], "lens");
        const int64_t n = q.dim() == 3 ? q.size(0) : 0, heads = q.dim() == 3 ? q.size(1) : 0;
        const int64_t B = lt.dim() == 1 ? lt.size(0) : 0;
        const Rows qr = rows(c, q, "q", c.dtype, n, heads);
        const int32_t *cu = ints(c, a[2], "cu", B + 1), *lens = ints(c, a[3], "lens", B);
        const int32_t* seqs = given(a[4]) ? ints(c, a[4], "seqs", B) : nullptr;
        const int32_t window = number(a[5], "window"), sinks = number(a[6], "sinks");
        const double scale = given(a[7]) ? real(a[7]) : 1.0 / std::sqrt((double)c.kv.head_dim);
        const c10::cuda::OptionalCUDAGuard on(c10::Device(at::kCUDA, c.device));
        Outputs o = outputs(c, n, heads, a[8], a[9], truth(a[10]));
        if (n > 0 && B > 0) {
            check(f_prefill(&c.kv, qr.p, qr.ld, count(n, "q"), count(B, "lens"), count(heads, "q"), seqs, cu, lens, window, sinks,
                            (float)scale, o.r.p, o.r.ld, o.lse_p, c.status, stream_of(c)),
                  "ember_paged_prefill");
            o.done();
        }
        return answer(o);
    });
}

// workspace_bytes(cache, B, heads)
PyObject* workspace_bytes(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
    return guarded(nargs, 3, [&]() -> PyObject* {
        Cache& c = cache_of(a[0]);
        const c10::cuda::OptionalCUDAGuard on(c10::Device(at::kCUDA, c.device));
        return PyLong_FromSize_t(workspace_of(c, number(a[1], "B"), number(a[2], "n_heads")));
    });
}

// shared_workspace_bytes(cache, B, heads, groups)
PyObject* shared_workspace_bytes(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
    return guarded(nargs, 4, [&]() -> PyObject* {
        Cache& c = cache_of(a[0]);
        const c10::cuda::OptionalCUDAGuard on(c10::Device(at::kCUDA, c.device));
        return PyLong_FromSize_t(shared_workspace_of(c, number(a[1], "B"), number(a[2], "n_heads"), number(a[3], "n_groups")));
    });
}

// cache(address of an ember_paged_kv, address of the status word, device index[, k_pages, v_pages[, status word, table]])
PyObject* cache(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
    return guarded(nargs, nargs == 5 || nargs == 7 ? nargs : 3, [&]() -> PyObject* {
        Tensor k_pages, v_pages, table, status_word;
        if (nargs >= 5) k_pages = tensor(a[3], "k_pages"), v_pages = tensor(a[4], "v_pages");
        if (nargs == 7) status_word = tensor(a[5], "status"), table = any_tensor(a[6], "table");
        auto* c = new Cache;
        c->k_pages = k_pages;
        c->v_pages = v_pages;
        c->status_word = status_word;
        c->table = table;
        c->kv = *static_cast<const ember_paged_kv*>(PyLong_AsVoidPtr(a[0]));
        c->status = static_cast<int32_t*>(PyLong_AsVoidPtr(a[1]));
        c->device = (c10::DeviceIndex)PyLong_AsLong(a[2]);
        c->dtype = c->kv.dtype == EMBER_BF16 ? at::kBFloat16 : at::kHalf;
        if (status_word.defined()) c->home = reinterpret_cast<ember_stream_t>(c10::cuda::getCurrentCUDAStream(c->device).stream());
        return PyCapsule_New(c, "ember.paged", [](PyObject* o) { delete static_cast<Cache*>(PyCapsule_GetPointer(o, "ember.paged")); });
    });
}

// entries(append, decode, decode_workspace, prefill, decode_shared, decode_shared_workspace, last_error, EmberError)
PyObject* entries(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
    return guarded(nargs, 8, [&]() -> PyObject* {
        f_append = reinterpret_cast<decltype(f_append)>(PyLong_AsVoidPtr(a[0]));
        f_decode = reinterpret_cast<decltype(f_decode)>(PyLong_AsVoidPtr(a[1]));
        f_workspace = reinterpret_cast<decltype(f_workspace)>(PyLong_AsVoidPtr(a[2]));
        f_prefill = reinterpret_cast<decltype(f_prefill)>(PyLong_AsVoidPtr(a[3]));
        f_shared = reinterpret_cast<decltype(f_shared)>(PyLong_AsVoidPtr(a[4]));
        f_shared_workspace = reinterpret_cast<decltype(f_shared_workspace)>(PyLong_AsVoidPtr(a[5]));
        f_error = reinterpret_cast<decltype(f_error)>(PyLong_AsVoidPtr(a[6]));
        Py_INCREF(a[7]);
        ember_error = a[7];
        Py_RETURN_NONE;
    });
}

PyMethodDef methods[] = {FAST("append", append), FAST("decode", decode), FAST("decode_shared", decode_shared), FAST("prefill", prefill),
                         FAST("workspace_bytes", workspace_bytes),
                         FAST("shared_workspace_bytes", shared_workspace_bytes), FAST("cache", cache), FAST("entries", entries),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "paged_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_paged_torch() { return PyModule_Create(&module); }
