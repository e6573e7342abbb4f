// rows_torch.cpp -- the torch side of runtime.logprobs: checks of the tensors, allocation
// of the outputs, and the call of the C entry point (include/ember.h).  Marshalling only,
// compiled for the reason that paged_torch.cpp gives.
#include "torch_args.h"

namespace {

decltype(&ember_logprobs) f_logprobs = nullptr;

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

// A contiguous tensor on a part of another's memory: five outputs cost one allocation.
Tensor piece(const Tensor& buffer, int64_t& at, at::IntArrayRef shape, at::ScalarType dtype) {
    Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(buffer.storage()), buffer.key_set(),
                                                        c10::scalarTypeToTypeMeta(dtype));
    t.unsafeGetTensorImpl()->set_storage_offset(at / 4);
    t.unsafeGetTensorImpl()->set_sizes_contiguous(shape);
    at += (t.numel() * 4 + 15) & ~(int64_t)15;
    return t;
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
        const Tensor buffer = make(p, {n * (3 + 2 * (int64_t)top) + 20}, at::kFloat);   // + what rounding up to 16 bytes takes
        int64_t used = 0;
        Tensor lp, rank, entropy = piece(buffer, used, {n}, at::kFloat), best = piece(buffer, used, {n, top}, at::kInt),
                         best_lp = piece(buffer, used, {n, top}, at::kFloat);
        if (ids) lp = piece(buffer, used, {n}, at::kFloat), rank = piece(buffer, used, {n}, at::kInt);
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

// entries(logprobs, last_error, EmberError)
PyObject* entries(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
    return guarded(nargs, 3, [&]() -> PyObject* {
        f_logprobs = reinterpret_cast<decltype(f_logprobs)>(PyLong_AsVoidPtr(a[0]));
        f_error = reinterpret_cast<decltype(f_error)>(PyLong_AsVoidPtr(a[1]));
        Py_INCREF(a[2]);
        ember_error = a[2];
        Py_RETURN_NONE;
    });
}

PyMethodDef methods[] = {FAST("logprobs", logprobs), FAST("entries", entries), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "rows_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_rows_torch() { return PyModule_Create(&module); }
