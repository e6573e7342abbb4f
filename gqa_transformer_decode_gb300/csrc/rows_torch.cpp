// rows_torch.cpp -- the torch side of runtime.logprobs and runtime.Adapters: checks of the
// tensors, allocation of what the caller did not pass, and the calls of the C entry points
// (include/ember.h).  Marshalling only, compiled for the reason that paged_torch.cpp gives.
#include "torch_args.h"

#include <torch/csrc/Dtype.h>

#include <memory>

namespace {

decltype(&ember_logprobs) f_logprobs = nullptr;
decltype(&ember_adapter_project) f_project = nullptr;
decltype(&ember_adapter_workspace) f_workspace = nullptr;

struct Place {   // where a call runs
    c10::DeviceIndex device;
};

int type_of(at::ScalarType t) {
    return t == at::kFloat ? EMBER_F32 : t == at::kBFloat16 ? EMBER_BF16 : t == at::kHalf ? EMBER_F16 : -1;
}
ember_stream_t stream_of(const Place& p) {
    return reinterpret_cast<ember_stream_t>(c10::cuda::getCurrentCUDAStream(p.device).stream());
}
// [n, cols], a row's elements side by side; the rows' distance
int64_t matrix(const Tensor& t, const char* what) {
    if (t.dim() != 2) bad(std::string(what) + " must have two dimensions, not " + describe(t));
    if (t.size(1) > 1 && t.stride(1) != 1) bad(std::string(what) + ": a row's elements must lie side by side");
    return t.size(0) > 1 ? t.stride(0) : t.size(1);
}

// logprobs(logits, ids, top, temperature) -> (logprob, rank, entropy, top_ids, top_logprobs)
PyObject* logprobs(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
    return guarded(nargs, 4, [&]() -> PyObject* {
        const Tensor& l = tensor(a[0], "logits");
        if (!l.is_cuda()) bad("logits must be on a CUDA device, not " + l.device().str());
        const Place p{l.device().index()};
        const int type = type_of(l.scalar_type());
        if (type < 0) throw Bad{PyExc_TypeError, "logits must be float32, bfloat16 or float16"};
        const int64_t ld = matrix(l, "logits"), n = l.size(0), V = l.size(1);
        const bool ids = given(a[1]);
        const int32_t* id = ids ? ints(p, a[1], "ids", n) : nullptr;
        const int32_t top = number(a[2], "top");
        const double t = real(a[3]);
        if (top < 0) bad("top must not be negative");
        const c10::cuda::OptionalCUDAGuard on(c10::Device(at::kCUDA, p.device));
        Tensor lp, rank, entropy = make(p, {n}, at::kFloat), best = make(p, {n, top}, at::kInt), best_lp = make(p, {n, top}, at::kFloat);
        if (ids) lp = make(p, {n}, at::kFloat), rank = make(p, {n}, at::kInt);
        auto at_of = [](const Tensor& x) { return x.defined() ? x.data_ptr() : nullptr; };
        check(f_logprobs(l.data_ptr(), type, count(n, "logits"), count(V, "logits"), ld, (float)t, id, top,
                         static_cast<float*>(at_of(lp)), static_cast<int32_t*>(at_of(rank)), static_cast<float*>(at_of(entropy)),
                         static_cast<int32_t*>(at_of(best)), static_cast<float*>(at_of(best_lp)), stream_of(p)),
              "ember_logprobs");
        PyObject* r = PyTuple_New(5);
        if (!r) return nullptr;
        int i = 0;
        for (const Tensor& x : {lp, rank, entropy, best, best_lp}) {
            if (!x.defined()) Py_INCREF(Py_None);
            PyTuple_SET_ITEM(r, i++, x.defined() ? THPVariable_Wrap(x) : Py_None);
        }
        return r;
    });
}

// One runtime.Adapters: the C view of them and where their status word lives.
struct Adapters {
    ember_adapters c;
    c10::DeviceIndex device;
    at::ScalarType dtype;
    int64_t K, N;
    Tensor a, b, scale, status;
    ember_stream_t home;             // the stream that status was allocated on
};
// Where the tensors lie and whether they are what they were: at every call, since a tensor may get
// other storage (t.data = ..) or be asked for its gradient at any time.
Adapters& adapters_of(PyObject* o) {
    auto* p = static_cast<Adapters*>(PyCapsule_GetPointer(o, "ember.adapters"));
    if (!p) throw python_error();
    const int64_t n = p->c.n_adapters, R = p->c.rank;
    no_gradient(p->a, "a");
    no_gradient(p->b, "b");
    p->c.a = flat(*p, p->a, "a", p->dtype, {n, R, p->K});
    p->c.b = flat(*p, p->b, "b", p->dtype, {n, p->N, R});
    if (p->scale.defined()) {
        no_gradient(p->scale, "scale");
        p->c.scale = static_cast<const float*>(flat(*p, p->scale, "scale", at::kFloat, {n}));
    }
    return *p;
}

// adapters(a, b, scale, status)
PyObject* adapters(PyObject*, PyObject* const* x, Py_ssize_t nargs) {
    return guarded(nargs, 4, [&]() -> PyObject* {
        const Tensor &a = tensor(x[0], "a"), &b = tensor(x[1], "b");
        if (!a.is_cuda()) bad("a must be on a CUDA device, not " + a.device().str());
        if (type_of(a.scalar_type()) < EMBER_BF16) throw Bad{PyExc_TypeError, "a and b must be bfloat16 or float16"};
        if (a.dim() != 3 || b.dim() != 3) bad("a must be [n_adapters, rank, K], b [n_adapters, N, rank], not " + describe(a) + " and " + describe(b));
        auto made = std::make_unique<Adapters>();
        Adapters& p = *made;
        p.device = a.device().index();
        p.dtype = a.scalar_type();
        p.K = a.size(2);
        p.N = b.size(1);
        p.c.a = flat(p, a, "a", p.dtype, a.sizes());
        p.c.b = flat(p, b, "b", p.dtype, {a.size(0), p.N, a.size(1)});
        p.c.scale = given(x[2]) ? static_cast<const float*>(flat(p, tensor(x[2], "scale"), "scale", at::kFloat, {a.size(0)})) : nullptr;
        p.c.n_adapters = count(a.size(0), "a");
        p.c.rank = count(a.size(1), "a");
        p.a = a;
        p.b = b;
        if (given(x[2])) p.scale = tensor(x[2], "scale");
        p.status = tensor(x[3], "status");
        (void)flat(p, p.status, "status", at::kInt, {1});
        p.home = stream_of({p.device});
        return PyCapsule_New(made.release(), "ember.adapters",
                             [](PyObject* o) { delete static_cast<Adapters*>(PyCapsule_GetPointer(o, "ember.adapters")); });
    });
}

// project(adapters, x, w, ids, bias, out, out_dtype (a torch.dtype or None), workspace)
PyObject* project(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
    return guarded(nargs, 8, [&]() -> PyObject* {
        const Adapters& p = adapters_of(a[0]);
        const Tensor &x = tensor(a[1], "x"), &w = tensor(a[2], "w");
        on_device(p, x, "x");
        const int64_t ld_x = matrix(x, "x"), n = x.size(0);
        if (x.scalar_type() != p.dtype || x.size(1) != p.K)
            bad(std::string("x must be ") + c10::toString(p.dtype) + " [n, " + std::to_string(p.K) + "], not " + describe(x));
        const void* wp = flat(p, w, "w", p.dtype, {p.N, p.K});
        const int32_t* ids = ints(p, a[3], "ids", n);
        const void* bias = given(a[4]) ? flat(p, tensor(a[4], "bias"), "bias", p.dtype, {p.N}) : nullptr;
        at::ScalarType ot = p.dtype;
        if (given(a[6])) {
            if (!THPDtype_Check(a[6])) throw Bad{PyExc_TypeError, "out_dtype must be a torch.dtype"};
            ot = reinterpret_cast<THPDtype*>(a[6])->scalar_type;
            if (ot != p.dtype && ot != at::kFloat) bad("out_dtype must be the adapters' type or float32");
        }
        const c10::cuda::OptionalCUDAGuard on(c10::Device(at::kCUDA, p.device));
        Tensor out, ws;
        int64_t ld_out = p.N;
        if (given(a[5])) {
            out = tensor(a[5], "out");
            on_device(p, out, "out");
            if (!given(a[6])) ot = out.scalar_type();
            ld_out = matrix(out, "out");
            if (out.scalar_type() != ot || (ot != p.dtype && ot != at::kFloat) || out.size(0) != n || out.size(1) != p.N)
                bad(std::string("out must be ") + c10::toString(p.dtype) + " or Float [" + std::to_string(n) + ", " + std::to_string(p.N) +
                    "], not " + describe(out));
        } else {
            out = make(p, {n, p.N}, ot);
        }
        if (n > 0) {
            const size_t need = f_workspace(count(n, "x"), p.c.rank);
            if (given(a[7])) {
                ws = tensor(a[7], "workspace");
                on_device(p, ws, "workspace");
                if (ws.scalar_type() != at::kByte || !ws.is_contiguous()) bad("workspace must be contiguous uint8");
            } else {
                ws = make(p, {(int64_t)need}, at::kByte);
            }
            const ember_stream_t s = stream_of({p.device});
            if (s != p.home)   // a kernel may raise an error when the object is gone: the word stays until then
                c10::cuda::CUDACachingAllocator::recordStream(p.status.storage().data_ptr(), c10::cuda::getCurrentCUDAStream(p.device));
            check(f_project(&p.c, x.data_ptr(), ld_x, wp, bias, type_of(p.dtype), count(n, "x"), count(p.N, "w"), count(p.K, "w"), ids,
                            out.data_ptr(), type_of(ot), ld_out, ws.numel() ? ws.data_ptr() : nullptr, (size_t)ws.numel(),
                            static_cast<int32_t*>(p.status.data_ptr()), s),
                  "ember_adapter_project");
            if (given(a[5])) written(out);
        }
        return THPVariable_Wrap(out);
    });
}

// entries(logprobs, project, adapter_workspace, last_error, EmberError)
PyObject* entries(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
    return guarded(nargs, 5, [&]() -> PyObject* {
        f_logprobs = reinterpret_cast<decltype(f_logprobs)>(PyLong_AsVoidPtr(a[0]));
        f_project = reinterpret_cast<decltype(f_project)>(PyLong_AsVoidPtr(a[1]));
        f_workspace = reinterpret_cast<decltype(f_workspace)>(PyLong_AsVoidPtr(a[2]));
        f_error = reinterpret_cast<decltype(f_error)>(PyLong_AsVoidPtr(a[3]));
        Py_INCREF(a[4]);
        ember_error = a[4];
        Py_RETURN_NONE;
    });
}

PyMethodDef methods[] = {FAST("logprobs", logprobs), FAST("adapters", adapters), FAST("project", project), FAST("entries", entries), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "rows_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_rows_torch() { return PyModule_Create(&module); }
