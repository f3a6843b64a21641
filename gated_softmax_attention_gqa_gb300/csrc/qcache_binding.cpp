// qcache_binding.cpp -- the 4-bit KV cache's entry points as a CPython module.
//
// The wrappers in __init__.py hand their tensors here: the layout checks, the outputs'
// allocation and the call into libgattn.  A decode step is ten microseconds on the GPU; the
// same checks written in Python over ctypes took 16 us (read) to 21 us (decode) of host time
// a call, which set a serving loop's pace.  Here they take 4.5 and 7 us, half of it the launches.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>

#include "gattn.h"

namespace {

// Raised as ValueError; thrown, so that helpers can refuse.
struct Refused : std::exception {
    std::string text;
    explicit Refused(std::string t) : text(std::move(t)) {}
    const char* what() const noexcept override { return text.c_str(); }
};
void need(bool ok, const char* text) {
    if (!ok) throw Refused(text);
}
std::string shape(at::IntArrayRef s) {
    std::string t = "[";
    for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
    return t + "]";
}

const at::Tensor& tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) throw Refused(std::string(name) + " must be a tensor");
    return THPVariable_Unpack(o);
}
const at::Tensor* optional(PyObject* o, const char* name) { return o == Py_None ? nullptr : &tensor(o, name); }

long integer(PyObject* o) {
    const long v = PyLong_AsLong(o);
    if (v == -1 && PyErr_Occurred()) throw python_error();
    return v;
}
double real(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw python_error();
    return v;
}
int to_int(int64_t v) {
    need(v >= INT_MIN && v <= INT_MAX, "a size or option is beyond 32 bits");
    return (int)v;
}

// A contiguous tensor of the given shape and type on the cache's device.
void* dense(const char* name, const at::Tensor& t, at::IntArrayRef size, at::ScalarType dtype, int dev) {
    if (t.sizes() != size || t.scalar_type() != dtype || !t.is_contiguous() || t.get_device() != dev)
        throw Refused(std::string(name) + " must be a contiguous " + toString(dtype) + " " + shape(size) +
                      " tensor on the cache's device");
    return t.data_ptr();
}
const int32_t* index(const char* name, const at::Tensor& t, int64_t n, int dev) {
    return static_cast<const int32_t*>(dense(name, t, {n}, at::kInt, dev));
}
// A dimension's stride for the C call, where 0 selects the contiguous default: a dimension
// of one has no stride to speak of, and a broadcast one cannot be passed.
int64_t stride(const at::Tensor& t, int i, const char* name) {
    if (t.size(i) <= 1) return 0;
    if (t.stride(i) == 0)
        throw Refused(std::string(name) + ": broadcast (stride 0) views are not supported; pass a contiguous copy");
    return t.stride(i);
}
int code_of(at::ScalarType t) {
    need(t == at::kBFloat16 || t == at::kFloat, "the dtype must be bfloat16 or float32");
    return t == at::kFloat ? GATTN_FP32 : GATTN_BF16;
}

// A cache and its table, checked.
struct Cache {
    int num_pages, G, page_size, d, B, max_pages, dev;
    void* pages;
    const int32_t* table;
    Cache(PyObject* qcache, PyObject* block_table) {
        const at::Tensor &q = tensor(qcache, "qcache"), &t = tensor(block_table, "block_table");
        need(q.dim() == 5 && q.size(0) == 2 && q.size(4) % 10 == 0 && q.scalar_type() == at::kByte && q.is_contiguous(),
             "qcache must be a contiguous uint8 [2,num_pages,G,page_size/16,10 d] tensor");
        dev = q.get_device();
        need(t.dim() == 2 && t.scalar_type() == at::kInt && t.is_contiguous() && t.get_device() == dev,
             "block_table must be a contiguous int32 [B,max_pages] tensor on the cache's device");
        num_pages = to_int(q.size(1));
        G = to_int(q.size(2));
        page_size = to_int(16 * q.size(3));
        d = to_int(q.size(4) / 10);
        B = to_int(t.size(0));
        max_pages = to_int(t.size(1));
        pages = q.data_ptr();
        table = t.data_ptr<int32_t>();
    }
    // A new tensor on the cache's device (torch.empty without its dispatcher: 1.2 us each).
    at::Tensor fresh(at::IntArrayRef size, at::ScalarType dtype) const {
        return at::detail::empty_cuda(size, dtype, c10::Device(c10::kCUDA, (c10::DeviceIndex)dev), std::nullopt);
    }
};

// The scope of a call: the cache's device is current, what it allocates belongs to its
// stream (a handle from the caller, or None for the device's current one), and other Python
// threads may run.  The GIL is taken back last.
class Scope {
    struct Released {
        PyThreadState* state = PyEval_SaveThread();
        ~Released() { PyEval_RestoreThread(state); }
    };
    static c10::cuda::CUDAStream pick(PyObject* o, int dev) {
        need(dev >= 0, "the tensors must be on a CUDA device");
        if (o == Py_None) return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev);
        void* s = PyLong_AsVoidPtr(o);
        if (!s && PyErr_Occurred()) throw python_error();
        return c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(s), (c10::DeviceIndex)dev);
    }
    c10::cuda::CUDAStream chosen;
    Released gil;
    c10::cuda::OptionalCUDAStreamGuard guard;

public:
    Scope(PyObject* o, int dev) : chosen(pick(o, dev)) {
        if (o != Py_None || c10::cuda::current_device() != dev) guard.reset_stream(chosen);
    }
    void* stream() const { return chosen.stream(); }
};

void arguments(Py_ssize_t n, Py_ssize_t want) {
    if (n != want) throw Refused("expected " + std::to_string(want) + " arguments");
}

// write(k, v, qcache, block_table, seqlens, knorm_w, cu_seqlens, rotary_dim, rope_base, eps, stream)
PyObject* write(PyObject* const* a, Py_ssize_t n) {
    arguments(n, 11);
    const Cache c(a[2], a[3]);
    const at::Tensor &k = tensor(a[0], "k"), &v = tensor(a[1], "v");
    if (k.dim() != 3 || k.size(1) != c.G || k.size(2) != c.d || v.sizes() != k.sizes())
        throw Refused("k and v must both be [T," + std::to_string(c.G) + "," + std::to_string(c.d) + "], as the cache's heads");
    need(k.stride(2) == 1 && v.stride(2) == 1, "k and v: the last dimension must be contiguous");
    const at::ScalarType dtype = k.scalar_type();
    const int code = code_of(dtype);
    need(v.scalar_type() == dtype && k.get_device() == c.dev && v.get_device() == c.dev,
         "k and v must have one dtype and be on the cache's device");
    const int T = to_int(k.size(0));
    const int32_t* lens = index("seqlens", tensor(a[4], "seqlens"), c.B, c.dev);
    const void* w = dense("knorm_w", tensor(a[5], "knorm_w"), {c.d}, dtype, c.dev);
    const at::Tensor* cu = optional(a[6], "cu_seqlens");
    need(cu || T == c.B, "without cu_seqlens every sequence gets one token: T must be B");
    const int32_t* cup = cu ? index("cu_seqlens", *cu, c.B + 1, c.dev) : nullptr;
    const int64_t ks = stride(k, 0, "k"), kh = stride(k, 1, "k"), vs = stride(v, 0, "v"), vh = stride(v, 1, "v");
    const int rotary = to_int(integer(a[7]));
    const double base = real(a[8]), eps = real(a[9]);
    int st;
    {
        const Scope scope(a[10], c.dev);
        st = gattn_qcache_write(k.data_ptr(), v.data_ptr(), c.pages, c.table, c.num_pages, c.page_size, c.max_pages, lens,
                                cup, w, T, c.B, c.G, c.d, rotary, base, (float)eps, ks, kh, vs, vh, code, scope.stream());
    }
    return PyLong_FromLong(st);
}

// read(qcache, block_table, starts, cu_seqlens, total, fp32, k_out, v_out, stream) -> status, k, v
PyObject* read(PyObject* const* a, Py_ssize_t n) {
    arguments(n, 9);
    const Cache c(a[0], a[1]);
    const at::Tensor *starts = optional(a[2], "starts"), *cu = optional(a[3], "cu_seqlens");
    const at::Tensor *ko = optional(a[6], "k_out"), *vo = optional(a[7], "v_out");
    need(!ko == !vo, "k_out and v_out go together");
    int64_t total = c.B;
    if (a[4] != Py_None) total = integer(a[4]);
    else if (cu && ko && ko->dim() > 0) total = ko->size(0);
    else need(!cu, "total (the number of rows) is needed with cu_seqlens");
    need(cu || total == c.B, "without cu_seqlens one token of each sequence is read");
    need(total >= 0, "total must not be negative");
    const int rows = to_int(total);
    const int32_t* sp = starts ? index("starts", *starts, c.B, c.dev) : nullptr;
    const int32_t* cup = cu ? index("cu_seqlens", *cu, c.B + 1, c.dev) : nullptr;
    at::ScalarType dtype = integer(a[5]) ? at::kFloat : at::kBFloat16;
    at::Tensor k, v;
    if (ko) {
        dtype = ko->scalar_type();
        code_of(dtype);
        dense("k_out", *ko, {total, c.G, c.d}, dtype, c.dev);
        dense("v_out", *vo, {total, c.G, c.d}, dtype, c.dev);
        k = *ko;
        v = *vo;
    }
    int st;
    {
        const Scope scope(a[8], c.dev);
        if (!ko) {
            // one allocation, [2, total, G, d]: a second one would take as long as the checks
            k = c.fresh({2, total, c.G, c.d}, dtype);
            v = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(k.storage()), k.key_set(), k.dtype());
            k.unsafeGetTensorImpl()->set_sizes_contiguous({total, c.G, c.d});
            v.unsafeGetTensorImpl()->set_sizes_contiguous({total, c.G, c.d});
            v.unsafeGetTensorImpl()->set_storage_offset(k.numel());
        }
        st = gattn_qcache_read(c.pages, c.table, c.num_pages, c.page_size, c.max_pages, sp, cup, rows, c.B, c.G,
                               c.d, code_of(dtype), k.data_ptr(), v.data_ptr(), scope.stream());
    }
    return Py_BuildValue("iNN", st, THPVariable_Wrap(k), THPVariable_Wrap(v));
}

// decode(q_new, k_new, v_new, qcache, block_table, seqlens, gate, qnorm_w, knorm_w, rotary_dim, rope_base, eps,
//        gate_mode, workspace, out, stream) -> status, out
PyObject* decode(PyObject* const* a, Py_ssize_t n) {
    arguments(n, 16);
    const Cache c(a[3], a[4]);
    const at::Tensor& q = tensor(a[0], "q_new");
    need(q.dim() == 3 && q.scalar_type() == at::kBFloat16 && q.get_device() == c.dev && q.size(0) == c.B &&
             q.size(2) == c.d && q.stride(2) == 1,
         "q_new must be a bfloat16 [B,H,d] tensor on the cache's device, B and d as the table's and the cache's, its last "
         "dimension contiguous");
    const int H = to_int(q.size(1));
    const int32_t* lens = index("seqlens", tensor(a[5], "seqlens"), c.B, c.dev);
    const void* qw = dense("qnorm_w", tensor(a[7], "qnorm_w"), {c.d}, at::kBFloat16, c.dev);
    const int mode = to_int(integer(a[12])), layout = mode & GATTN_GATE_LAYOUT_MASK;
    const void* gate = nullptr;
    int64_t gs = 0, gh = 0;
    if (layout != GATTN_GATE_NONE) {
        need(a[6] != Py_None, "this gate_mode needs gate logits");
        const at::Tensor& g = tensor(a[6], "gate");
        const int dims = layout == GATTN_GATE_ELEMENTWISE ? 3 : 2;
        need(g.dim() == dims && g.size(0) == c.B && g.scalar_type() == at::kBFloat16 && g.get_device() == c.dev &&
                 g.size(1) == (layout == GATTN_GATE_HEAD_SHARED ? c.d : H) && (dims == 2 || g.size(2) == c.d),
             "gate must be a bfloat16 [B,H,d], [B,H] or (head_shared) [B,d] tensor on the cache's device");
        need(layout == GATTN_GATE_HEADWISE || g.stride(dims - 1) == 1, "gate: the last dimension must be contiguous");
        gate = g.data_ptr();
        gs = stride(g, 0, "gate");
        if (layout != GATTN_GATE_HEAD_SHARED) gh = stride(g, 1, "gate");
    }
    const void *kn = nullptr, *vn = nullptr, *kw = nullptr;
    if (a[1] != Py_None || a[2] != Py_None || a[8] != Py_None) {
        need(a[1] != Py_None && a[2] != Py_None && a[8] != Py_None, "an append needs k_new, v_new and knorm_w");
        kn = dense("k_new", tensor(a[1], "k_new"), {c.B, c.G, c.d}, at::kBFloat16, c.dev);
        vn = dense("v_new", tensor(a[2], "v_new"), {c.B, c.G, c.d}, at::kBFloat16, c.dev);
        kw = dense("knorm_w", tensor(a[8], "knorm_w"), {c.d}, at::kBFloat16, c.dev);
    }
    const int64_t qs = stride(q, 0, "q_new"), qh = stride(q, 1, "q_new");
    const at::Tensor *ws = optional(a[13], "workspace"), *given = optional(a[14], "out");
    if (given) dense("out", *given, {c.B, (int64_t)H * c.d}, at::kBFloat16, c.dev);
    need(!ws || (ws->is_contiguous() && ws->get_device() == c.dev), "workspace must be a contiguous tensor on the cache's device");
    const int rotary = to_int(integer(a[9]));
    const double base = real(a[10]), eps = real(a[11]);
    at::Tensor out, own;
    int st;
    {
        const Scope scope(a[15], c.dev);
        out = given ? *given : c.fresh({c.B, (int64_t)H * c.d}, at::kBFloat16);
        if (!ws) {
            const size_t bytes = gattn_decode_qcache_workspace_size(c.B, H, c.G, c.d, to_int((int64_t)c.max_pages * c.page_size));
            own = c.fresh({(int64_t)(bytes ? bytes : 1)}, at::kByte);
            ws = &own;
        }
        st = gattn_decode_qcache(q.data_ptr(), kn, vn, c.pages, c.table, c.num_pages, c.page_size, c.max_pages, lens, gate,
                                 qw, kw, c.B, H, c.G, c.d, rotary, base, (float)eps, mode, qs, qh, gs, gh, ws->data_ptr(),
                                 ws->nbytes(), out.data_ptr(), scope.stream());
    }
    return Py_BuildValue("iN", st, THPVariable_Wrap(out));
}

// No C++ exception leaves the module: refusals become ValueError, torch's errors their own types.
template <PyObject* (*F)(PyObject* const*, Py_ssize_t)>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    try {
        return F(args, n);
    } catch (const Refused& e) {
        PyErr_SetString(PyExc_ValueError, e.what());
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

template <PyObject* (*F)(PyObject* const*, Py_ssize_t)>
constexpr PyCFunction method() {
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<F>));
}

PyMethodDef methods[] = {{"write", method<write>(), METH_FASTCALL, "gattn_qcache_write; returns its status"},
                         {"read", method<read>(), METH_FASTCALL, "gattn_qcache_read; returns (status, k, v)"},
                         {"decode", method<decode>(), METH_FASTCALL, "gattn_decode_qcache; returns (status, out)"},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_qcache", "4-bit KV cache entry points of libgattn", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__qcache() { return PyModule_Create(&module); }
