// The tensor level of the operators around a convolution: checks of tensors,
// allocation of outputs and workspaces, and the call of the C ABI, for
// block.py.  It is native because a small call costs its host time: a token
// through a norm takes 3 us on the device, and its checks, two allocations and
// the call took 9 us in Python (a list of 600 gradients, a third of a
// millisecond).
//
// Functions take the arguments of block.py's in order (activation and norm as
// codes, the raw stream last) and return the result, or the status of a call
// that failed as an int.  What a tensor does not fit raises ValueError.
#include <Python.h>

#include <ATen/ops/empty.h>
#include <torch/csrc/autograd/python_variable.h>

#include <array>
#include <initializer_list>
#include <stdexcept>
#include <string>
#include <vector>

#include "convmi.h"

namespace {

typedef std::vector<int64_t> Shape;

struct Refused : std::runtime_error {
    using std::runtime_error::runtime_error;
};

std::string text(at::IntArrayRef s)
{
    std::string t = "[";
    for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
    return t + "]";
}

// The C ABI, bound by address (the loaded library is block.py's choice).
struct Api {
    decltype(&conv_gated_fwd_ex) gated_fwd;
    decltype(&conv_gated_fwd_workspace_size) gated_fwd_workspace;
    decltype(&conv_gated_bwd) gated_bwd;
    decltype(&conv_gated_bwd_workspace_size) gated_bwd_workspace;
    decltype(&conv_block_norm_fwd) norm_fwd;
    decltype(&conv_block_norm_bwd) norm_bwd;
    decltype(&conv_block_norm_bwd_workspace_size) norm_bwd_workspace;
    decltype(&conv_grad_norm) grad_norm;
    decltype(&conv_grad_clip) grad_clip;
    decltype(&conv_grad_workspace_size) grad_workspace;
} api;

// An optional tensor.
const at::Tensor* tensor(PyObject* o, const char* name)
{
    if (o == Py_None) return nullptr;
    if (!THPVariable_Check(o)) throw Refused(std::string(name) + " must be a tensor");
    return &THPVariable_Unpack(o);
}
const at::Tensor& needed(PyObject* o, const char* name)
{
    const at::Tensor* t = tensor(o, name);
    if (!t) throw Refused(std::string(name) + " must be a tensor");
    return *t;
}

// What a call's tensors have in common, taken from its input.
struct Call {
    at::ScalarType type;
    at::Device device;
    int dtype;

    explicit Call(const at::Tensor& x) : type(x.scalar_type()), device(x.device()), dtype(code(x)) {}

    static int code(const at::Tensor& t)
    {
        if (t.scalar_type() == at::kFloat) return CONV_F32;
        if (t.scalar_type() == at::kBFloat16) return CONV_BF16;
        throw Refused(std::string("unsupported dtype ") + c10::toString(t.scalar_type()) + "; convmi takes float32 or bfloat16");
    }
    void fits(const at::Tensor* t, const char* name, at::IntArrayRef shape) const
    {
        if (!t) return;
        if (t->sizes() != shape)
            throw Refused(std::string(name) + " must have shape " + text(shape) + "; found " + text(t->sizes()));
        if (t->scalar_type() != type || t->device() != device)
            throw Refused(std::string(name) + " must have the dtype and device of the input (" + c10::toString(type) + ", " + device.str() +
                          "); found " + c10::toString(t->scalar_type()) + ", " + t->device().str());
        if (!t->is_contiguous()) throw Refused(std::string(name) + " must be contiguous");
    }
    // Last of the checks.
    void on_gpu() const
    {
        if (!device.is_cuda()) throw Refused("tensors passed to convmi must be on a GPU device");
    }
};

void* at_of(const at::Tensor* t) { return t ? t->data_ptr() : nullptr; }
// A caller's tensor that a call has written: automatic differentiation counts
// its versions (an inference tensor has none).
void wrote(const at::Tensor* t)
{
    if (t && !t->is_inference()) t->unsafeGetTensorImpl()->bump_version();
}
at::Tensor like(const at::Tensor& t) { return at::empty(t.sizes(), t.options().memory_format(at::MemoryFormat::Contiguous)); }
at::Tensor bytes_like(const at::Tensor& t, size_t n) { return at::empty({static_cast<int64_t>(n < 16 ? 16 : n)}, t.options().dtype(at::kByte)); }

struct Workspace {
    at::Tensor own;
    void* at;
    size_t bytes;
    Workspace(const at::Tensor* given, const at::Tensor& x, size_t need)
    {
        if (given) {
            if (given->device() != x.device() || !given->is_contiguous())
                throw Refused("the workspace must be a contiguous tensor on the input's device");
            at = given->data_ptr();
            bytes = given->nbytes();
        } else {
            own = bytes_like(x, need);
            at = own.data_ptr();
            bytes = own.nbytes();
        }
    }
};

int64_t rows_of(const at::Tensor& x)
{
    if (x.dim() < 1 || x.size(-1) < 1) throw Refused("an input has at least one dimension and one channel");
    return x.numel() / x.size(-1);
}
int narrow(int64_t n, const char* name)
{
    if (n > INT32_MAX) throw Refused(std::string(name) + " is 2^31 or more");
    return static_cast<int>(n);
}
PyObject* wrap(const at::Tensor* t)
{
    if (!t || !t->defined()) Py_RETURN_NONE;
    return THPVariable_Wrap(*t);
}
PyObject* status(int rc) { return PyLong_FromLong(rc); }

template <typename F>
int call(F f)
{
    int rc;
    Py_BEGIN_ALLOW_THREADS;
    rc = f();
    Py_END_ALLOW_THREADS;
    return rc;
}

// Runs a function's body: `n` arguments, C++ exceptions as Python's.
template <typename F>
PyObject* guarded(Py_ssize_t have, Py_ssize_t n, F body)
{
    if (have != n) {
        PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", n, have);
        return nullptr;
    }
    try {
        PyObject* r = body();
        return PyErr_Occurred() ? (Py_XDECREF(r), nullptr) : r;
    } catch (const Refused& e) {
        PyErr_SetString(PyExc_ValueError, e.what());
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}
int integer(PyObject* o) { return static_cast<int>(PyLong_AsLong(o)); }
void* address(PyObject* o) { return PyLong_AsVoidPtr(o); }

// --------------------------------------------------------- gated layer --

struct Gated {
    const at::Tensor &x, &wg, &wu;
    const at::Tensor *bg, *bu, *saved;
    Call c;
    int64_t rows;
    int C, F, act;
    Shape hidden;  // of h

    Gated(PyObject* const* a, int act_code, PyObject* kept)
        : x(needed(a[0], "x")), wg(needed(a[1], "w_gate")), wu(needed(a[2], "w_up")), bg(tensor(a[3], "b_gate")),
          bu(tensor(a[4], "b_up")), saved(tensor(kept, "saved")), c(x), rows(rows_of(x)), C(narrow(x.size(-1), "C")), F(0), act(act_code)
    {
        if (wg.dim() < 2 || wg.size(0) < 1 || wg.size(-1) != C || wg.numel() != wg.size(0) * C)
            throw Refused("w_gate must be a 1x1 weight [F, " + std::to_string(C) + "] (or [F, 1, 1, " + std::to_string(C) + "]); found " + text(wg.sizes()));
        F = narrow(wg.size(0), "F");
        if (!bg != !bu) throw Refused("b_gate and b_up come together");
        c.fits(&x, "x", x.sizes());
        c.fits(&wg, "w_gate", wg.sizes());
        c.fits(&wu, "w_up", wg.sizes());
        c.fits(bg, "b_gate", {F});
        c.fits(bu, "b_up", {F});
        hidden = x.sizes().vec();
        hidden.back() = F;
        if (saved && (saved->scalar_type() != at::kFloat || saved->dim() < 1 || saved->size(-1) != 2 * static_cast<int64_t>(F) ||
                      saved->numel() != rows * 2 * F || saved->device() != x.device() || !saved->is_contiguous()))
            throw Refused("saved must be contiguous float32 on the input's device, with " + std::to_string(rows) + " rows of " +
                          std::to_string(2 * static_cast<int64_t>(F)) + " values; found " + c10::toString(saved->scalar_type()) + " " + text(saved->sizes()));
    }
};

// x w_gate w_up b_gate b_up act out saved stream
PyObject* gated(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded(n, 9, [&]() -> PyObject* {
        Gated g(a, integer(a[5]), a[7]);
        const at::Tensor* out = tensor(a[6], "out");
        g.c.fits(out, "out", g.hidden);
        g.c.on_gpu();
        size_t need = 0;
        if (int rc = api.gated_fwd_workspace(g.rows, g.C, g.F, g.c.dtype, &need)) return status(rc);
        at::Tensor h = out ? *out : at::empty(g.hidden, g.x.options()), ws;
        if (need) ws = bytes_like(g.x, need);
        void* stream = address(a[8]);
        const int rc = call([&] {
            return api.gated_fwd(g.x.data_ptr(), g.wg.data_ptr(), g.wu.data_ptr(), at_of(g.bg), at_of(g.bu), h.data_ptr(),
                                 static_cast<float*>(at_of(g.saved)), need ? ws.data_ptr() : nullptr, need, g.rows, g.C, g.F, g.act,
                                 g.c.dtype, stream);
        });
        if (rc) return status(rc);
        wrote(out);
        wrote(g.saved);
        return THPVariable_Wrap(h);
    });
}

// x w_gate w_up b_gate b_up act dh saved workspace stream
PyObject* gated_grad(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded(n, 10, [&]() -> PyObject* {
        Gated g(a, integer(a[5]), a[7]);
        const at::Tensor& dh = needed(a[6], "dh");
        g.c.fits(&dh, "dh", g.hidden);
        g.c.on_gpu();
        size_t need = 0;
        if (int rc = api.gated_bwd_workspace(g.rows, g.C, g.F, g.c.dtype, &need)) return status(rc);
        Workspace ws(tensor(a[8], "workspace"), g.x, need);
        std::array<at::Tensor, 5> d = {like(g.x), like(g.wg), like(g.wu)};
        if (g.bg) d[3] = like(*g.bg), d[4] = like(*g.bu);
        void* stream = address(a[9]);
        const int rc = call([&] {
            return api.gated_bwd(dh.data_ptr(), g.x.data_ptr(), g.wg.data_ptr(), g.wu.data_ptr(), at_of(g.bg), at_of(g.bu),
                                 static_cast<const float*>(at_of(g.saved)), d[0].data_ptr(), d[1].data_ptr(), d[2].data_ptr(),
                                 g.bg ? d[3].data_ptr() : nullptr, g.bg ? d[4].data_ptr() : nullptr, ws.at, ws.bytes, g.rows, g.C, g.F,
                                 g.act, g.c.dtype, stream);
        });
        if (rc) return status(rc);
        PyObject* r = PyTuple_New(5);
        for (int i = 0; r && i < 5; ++i) PyTuple_SET_ITEM(r, i, wrap(&d[i]));
        return r;
    });
}

// --------------------------------------------------------------- norms --

// x branch gate scale post_weight post_bias pre_weight pre_bias, post pre act eps
struct Norm {
    static constexpr int kInputs = 8;
    std::array<const at::Tensor*, kInputs> in;
    const at::Tensor& x;
    Call c;
    int64_t rows, gate_rows = 1;
    int C, post, pre, act;
    float eps;

    explicit Norm(PyObject* const* a) : x(needed(a[0], "x")), c(x), rows(rows_of(x)), C(narrow(x.size(-1), "C"))
    {
        static const char* names[kInputs] = {"x", "branch", "gate", "scale", "post_weight", "post_bias", "pre_weight", "pre_bias"};
        for (int i = 0; i < kInputs; ++i) in[i] = tensor(a[i], names[i]);
        post = integer(a[8]);
        pre = integer(a[9]);
        act = integer(a[10]);
        eps = static_cast<float>(PyFloat_AsDouble(a[11]));
        const at::Tensor* gate = in[2];
        if (gate && gate->sizes() != x.sizes()) {
            if (x.dim() > 1 && gate->dim() == 2 && gate->size(0) == x.size(0) && gate->size(1) == C)
                gate_rows = std::max<int64_t>(rows / std::max<int64_t>(x.size(0), 1), 1);
            else if (gate->dim() == 1 && gate->size(0) == C)
                gate_rows = std::max<int64_t>(rows, 1);
            else
                throw Refused("gate must have shape " + text(x.sizes()) + ", [" + std::to_string(x.size(0)) + ", " + std::to_string(C) +
                              "] or [" + std::to_string(C) + "]; found " + text(gate->sizes()));
        }
        const std::array<int64_t, 1> row = {C};
        for (int i = 0; i < kInputs; ++i)
            c.fits(in[i], names[i], i == 2 && gate ? gate->sizes() : i < 2 ? x.sizes() : at::IntArrayRef(row));
    }
    void* operator[](int i) const { return at_of(in[i]); }
};

// the twelve of Norm, stream
PyObject* norm(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded(n, 13, [&]() -> PyObject* {
        Norm k(a);
        if (PyErr_Occurred()) return nullptr;
        if (!k.in[1] && k.pre == CONV_NORM_NONE) throw Refused("without a branch and a pre norm there is nothing to compute");
        k.c.on_gpu();
        at::Tensor y, out;
        if (k.in[1]) y = like(k.x);
        if (k.pre != CONV_NORM_NONE) out = like(k.x);
        void* stream = address(a[12]);
        const int rc = call([&] {
            return api.norm_fwd(k[0], k[1], k[2], k[3], k[4], k[5], k[6], k[7], y.defined() ? y.data_ptr() : nullptr,
                                out.defined() ? out.data_ptr() : nullptr, k.rows, k.C, k.gate_rows, k.post, k.pre, k.act, k.eps, k.c.dtype, stream);
        });
        if (rc) return status(rc);
        PyObject* r = PyTuple_New(2);
        if (!r) return nullptr;
        PyTuple_SET_ITEM(r, 0, k.in[1] ? wrap(&y) : (Py_INCREF(a[0]), a[0]));
        PyTuple_SET_ITEM(r, 1, wrap(&out));
        return r;
    });
}

// the twelve of Norm, dy da workspace stream
PyObject* norm_grad(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded(n, 16, [&]() -> PyObject* {
        Norm k(a);
        if (PyErr_Occurred()) return nullptr;
        const at::Tensor *dy = tensor(a[12], "dy"), *da = tensor(a[13], "da");
        k.c.fits(dy, "dy", k.x.sizes());
        k.c.fits(da, "da", k.x.sizes());
        k.c.on_gpu();
        size_t need = 0;
        if (int rc = api.norm_bwd_workspace(k.rows, k.C, k.in[2] ? k.gate_rows : 0, &need)) return status(rc);
        Workspace ws(tensor(a[14], "workspace"), k.x, need);
        std::array<at::Tensor, Norm::kInputs> d;
        std::array<void*, Norm::kInputs> to{};
        for (int i = 0; i < Norm::kInputs; ++i)
            if (k.in[i]) {
                d[i] = like(*k.in[i]);
                // To the C call a gate has rows / gate_rows rows: none, while
                // an image's or a batch's gate may still be there.
                if (i == 2 && k.rows == 0) d[i].zero_();
                to[i] = d[i].data_ptr();
            }
        void* stream = address(a[15]);
        const int rc = call([&] {
            return api.norm_bwd(at_of(dy), at_of(da), k[0], k[1], k[2], k[3], k[4], k[5], k[6], k[7], to[0], to[1], to[2], to[3], to[4], to[5],
                                to[6], to[7], ws.at, ws.bytes, k.rows, k.C, k.gate_rows, k.post, k.pre, k.act, k.eps, k.c.dtype, stream);
        });
        if (rc) return status(rc);
        PyObject* r = PyTuple_New(Norm::kInputs);
        for (int i = 0; r && i < Norm::kInputs; ++i) PyTuple_SET_ITEM(r, i, wrap(&d[i]));
        return r;
    });
}

// --------------------------------------------------------------- lists --

struct List {
    std::vector<const at::Tensor*> tensors;
    std::vector<void*> at;
    std::vector<size_t> counts;
    std::vector<int> dtypes;
    const at::Tensor* first = nullptr;

    explicit List(PyObject* o)
    {
        if (!PyList_Check(o)) throw Refused("the gradients must be a list of tensors");
        const Py_ssize_t n = PyList_GET_SIZE(o);
        if (n == 0) throw Refused("the list of gradients is empty");
        narrow(n, "the number of tensors");
        tensors.reserve(n);
        at.reserve(n);
        counts.reserve(n);
        dtypes.reserve(n);
        for (Py_ssize_t i = 0; i < n; ++i) {
            const at::Tensor& t = needed(PyList_GET_ITEM(o, i), "a gradient");
            if (!first) first = &t;
            dtypes.push_back(Call::code(t));
            if (!t.is_cuda() || t.device() != first->device()) throw Refused("tensors passed to convmi must be on one GPU device");
            // Any order of dimensions: each element counts for itself.
            if (!t.is_non_overlapping_and_dense()) throw Refused("the tensors of a list must be dense");
            tensors.push_back(&t);
            at.push_back(t.data_ptr());
            counts.push_back(static_cast<size_t>(t.numel()));
        }
    }
    int n() const { return static_cast<int>(at.size()); }
};

// grads out (None: the norm alone) max_norm eps stream
PyObject* clip(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded(n, 5, [&]() -> PyObject* {
        const bool only_norm = a[1] == Py_None;
        List g(a[0]);
        const float max_norm = static_cast<float>(PyFloat_AsDouble(a[2])), eps = static_cast<float>(PyFloat_AsDouble(a[3]));
        if (PyErr_Occurred()) return nullptr;
        std::vector<void*> out;
        std::vector<const at::Tensor*> written = g.tensors;
        if (!only_norm && a[1] != a[0]) {
            if (PyList_Check(a[1]) && PyList_GET_SIZE(a[1]) != PyList_GET_SIZE(a[0]))
                throw Refused("out has " + std::to_string(PyList_GET_SIZE(a[1])) + " tensors for " + std::to_string(g.n()) + " gradients");
            List o(a[1]);
            if (o.counts != g.counts || o.dtypes != g.dtypes || o.first->device() != g.first->device())
                throw Refused("the tensors of out must have the sizes, dtypes and device of the gradients");
            for (int i = 0; i < g.n(); ++i) {
                const at::Tensor &from = *g.tensors[i], &to = *o.tensors[i];
                if (!(from.is_contiguous() && to.is_contiguous()) && (from.sizes() != to.sizes() || from.strides() != to.strides()))
                    throw Refused("the tensors of out must lie in memory as the gradients do");
            }
            out = std::move(o.at);
            written = std::move(o.tensors);
        }
        size_t need = 0;
        if (int rc = api.grad_workspace(g.n(), &need)) return status(rc);
        at::Tensor v = at::empty({}, g.first->options().dtype(at::kFloat)), ws = bytes_like(*g.first, need);
        void* stream = address(a[4]);
        float* to = static_cast<float*>(v.data_ptr());
        const int rc = call([&] {
            return only_norm ? api.grad_norm(g.at.data(), g.counts.data(), g.dtypes.data(), g.n(), to, ws.data_ptr(), ws.nbytes(), stream)
                             : api.grad_clip(g.at.data(), out.empty() ? g.at.data() : out.data(), g.counts.data(), g.dtypes.data(), g.n(),
                                             max_norm, eps, to, ws.data_ptr(), ws.nbytes(), stream);
        });
        if (rc) return status(rc);
        if (!only_norm)
            for (const at::Tensor* t : written) wrote(t);
        return THPVariable_Wrap(v);
    });
}

// The addresses of the C functions, in the order of Api.
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    static_assert(sizeof(Api) == 10 * sizeof(void*), "");
    return guarded(n, 10, [&]() -> PyObject* {
        for (int i = 0; i < 10; ++i) reinterpret_cast<void**>(&api)[i] = address(a[i]);
        Py_RETURN_NONE;
    });
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f))
PyMethodDef methods[] = {{"bind", FAST(bind), METH_FASTCALL, nullptr},
                         {"gated", FAST(gated), METH_FASTCALL, nullptr},
                         {"gated_grad", FAST(gated_grad), METH_FASTCALL, nullptr},
                         {"norm", FAST(norm), METH_FASTCALL, nullptr},
                         {"norm_grad", FAST(norm_grad), METH_FASTCALL, nullptr},
                         {"clip", FAST(clip), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_native", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__native() { return PyModule_Create(&module); }
