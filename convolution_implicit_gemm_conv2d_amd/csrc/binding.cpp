// The tensor level of the operators around a convolution, of those along a
// sequence and of the optimizer step: checks of tensors, allocation of outputs
// and workspaces, and the call of the C ABI, for block.py, sequence.py and
// optimizer.py.  It is native because a small call costs its host time: a token
// through a norm takes 3 us on the device, and its checks, two allocations and
// the call took 9 us in Python (a list of 600 gradients, a third of a
// millisecond).
//
// Functions take those modules' arguments in order (activation and norm as
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
    decltype(&conv_causal_fwd) causal_fwd;
    decltype(&conv_causal_bwd) causal_bwd;
    decltype(&conv_causal_bwd_workspace_size) causal_bwd_workspace;
    decltype(&conv_causal_step) causal_step;
    decltype(&conv_scan_fwd) scan_fwd;
    decltype(&conv_scan_bwd) scan_bwd;
    decltype(&conv_scan_step) scan_step;
    decltype(&conv_scan_saved_size) scan_saved;
    decltype(&conv_scan_fwd_workspace_size) scan_fwd_workspace;
    decltype(&conv_scan_bwd_workspace_size) scan_bwd_workspace;
    decltype(&conv_adamw) adamw;
    decltype(&conv_adamw_moments) moments;
} api;
constexpr int kApi = sizeof(Api) / sizeof(void*);

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

// Two dense tensors whose elements lie in memory in the same order.  A dimension
// of one entry has no say, whatever its stride is.
bool lie_alike(const at::Tensor& a, const at::Tensor& b)
{
    if (a.is_contiguous() && b.is_contiguous()) return true;
    if (a.sizes() != b.sizes()) return false;
    for (int64_t i = 0; i < a.dim(); ++i)
        if (a.size(i) != 1 && a.stride(i) != b.stride(i)) return false;
    return true;
}

struct List {
    std::vector<const at::Tensor*> tensors;
    std::vector<void*> at;
    std::vector<size_t> counts;
    std::vector<int> dtypes;
    const at::Tensor* first = nullptr;

    // `one`: what an entry is.
    List(PyObject* o, const char* one)
    {
        if (!PyList_Check(o)) throw Refused(std::string("the ") + one + "s must be a list of tensors");
        const Py_ssize_t n = PyList_GET_SIZE(o);
        if (n == 0) throw Refused(std::string("the list of ") + one + "s is empty");
        narrow(n, "the number of tensors");
        const std::string entry = std::string("an entry of the ") + one + "s";
        tensors.reserve(n);
        at.reserve(n);
        counts.reserve(n);
        dtypes.reserve(n);
        for (Py_ssize_t i = 0; i < n; ++i) {
            const at::Tensor& t = needed(PyList_GET_ITEM(o, i), entry.c_str());
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
        List g(a[0], "gradient");
        const float max_norm = static_cast<float>(PyFloat_AsDouble(a[2])), eps = static_cast<float>(PyFloat_AsDouble(a[3]));
        if (PyErr_Occurred()) return nullptr;
        std::vector<void*> out;
        std::vector<const at::Tensor*> written = g.tensors;
        if (!only_norm && a[1] != a[0]) {
            if (PyList_Check(a[1]) && PyList_GET_SIZE(a[1]) != PyList_GET_SIZE(a[0]))
                throw Refused("out has " + std::to_string(PyList_GET_SIZE(a[1])) + " tensors for " + std::to_string(g.n()) + " gradients");
            List o(a[1], "output");
            if (o.counts != g.counts || o.dtypes != g.dtypes || o.first->device() != g.first->device())
                throw Refused("the tensors of out must have the sizes, dtypes and device of the gradients");
            for (int i = 0; i < g.n(); ++i) {
                if (!lie_alike(*g.tensors[i], *o.tensors[i]))
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

// ---------------------------------------------------- along a sequence --

// A tensor of `rows` rows whose last `tail` dimensions are dense; the rows may
// lie apart, evenly.  Returns the elements from one row to the next.
int64_t spread(const at::Tensor& t, int tail, const char* name)
{
    const int lead = static_cast<int>(t.dim()) - tail;
    int64_t width = 1;
    bool ok = true;
    for (int i = static_cast<int>(t.dim()) - 1; i >= lead; --i) {
        ok = ok && (t.size(i) == 1 || t.stride(i) == width);
        width *= t.size(i);
    }
    int64_t stride = width, next = 0;  // of a row, and of the dimension before
    for (int i = lead - 1; i >= 0; --i) {
        if (t.size(i) == 1) continue;
        if (!next) stride = t.stride(i);
        ok = ok && stride >= width && (!next || t.stride(i) == next);
        next = t.stride(i) * t.size(i);
    }
    if (t.numel() == 0) return width;
    if (!ok)
        throw Refused(std::string(name) + " must have dense channels and evenly spaced rows; found shape " + text(t.sizes()) + " with strides " + text(t.strides()));
    return stride;
}

// Tensors of a given type, dense, on the input's device.
void plain(const at::Tensor* t, const char* name, at::IntArrayRef shape, at::ScalarType type, const at::Device& device)
{
    if (!t) return;
    if (t->sizes() != shape) throw Refused(std::string(name) + " must have shape " + text(shape) + "; found " + text(t->sizes()));
    if (t->scalar_type() != type || t->device() != device || !t->is_contiguous())
        throw Refused(std::string(name) + " must be contiguous " + c10::toString(type) + " on the input's device; found " + c10::toString(t->scalar_type()) + " on " +
                      t->device().str());
}

// The rows of a call's input x and its sequences.
struct Rows {
    const at::Tensor &x, *starts;
    Call c;
    int64_t rows;
    int C, seqs;

    Rows(const at::Tensor& input, const at::Tensor* st, bool tokens)
        : x(input), starts(st), c(input), rows(rows_of(input)), C(narrow(input.size(-1), "the number of channels")), seqs(0)
    {
        if (tokens) return;
        if (starts) {
            if (x.dim() != 2) throw Refused("with starts, x has rows and channels; found " + text(x.sizes()));
            if (starts->dim() != 1 || starts->size(0) < 1 || (starts->size(0) < 2 && rows > 0))
                throw Refused("starts must hold the first row of each sequence and the end of the last; found shape " + text(starts->sizes()));
            plain(starts, "starts", starts->sizes(), at::kInt, x.device());
            seqs = narrow(starts->size(0) - 1, "the number of sequences");
        } else {
            if (x.dim() != 2 && x.dim() != 3) throw Refused("x must have shape [sequences, rows, channels] or [rows, channels]; found " + text(x.sizes()));
            seqs = x.dim() == 3 ? narrow(x.size(0), "the number of sequences") : 1;
        }
    }
    // A tensor of the input's rows; its last dimensions may be others.
    int64_t like(const at::Tensor* t, const char* name, at::IntArrayRef shape, int tail) const
    {
        if (!t) return 0;
        if (t->sizes() != shape) throw Refused(std::string(name) + " must have shape " + text(shape) + "; found " + text(t->sizes()));
        if (t->scalar_type() != c.type || t->device() != c.device)
            throw Refused(std::string(name) + " must have the dtype and device of the input (" + c10::toString(c.type) + ", " + c.device.str() + "); found " +
                          c10::toString(t->scalar_type()) + ", " + t->device().str());
        return spread(*t, tail, name);
    }
    const int* at_starts() const { return static_cast<const int*>(at_of(starts)); }
};

// The pool of a token call and the slots of its rows.
struct Pool {
    const at::Tensor& state;
    const at::Tensor* slots;
    int count;
    Pool(const at::Tensor& t, const at::Tensor* s, int64_t rows, const at::Device& device) : state(t), slots(s), count(0)
    {
        if (state.dim() != 3) throw Refused("state must have three dimensions; found " + text(state.sizes()));
        count = narrow(state.size(0), "the number of states");
        const std::array<int64_t, 1> one = {rows};
        plain(slots, "slots", one, at::kInt, device);
        if (!slots && rows > count) throw Refused("without slots, state must have a row for each of x's");
    }
};

struct Causal : Rows {
    const at::Tensor &w, *bias;
    int K, act;
    int64_t xs;
    Causal(const at::Tensor& input, PyObject* weight, PyObject* b, int act_code, const at::Tensor* st, bool tokens)
        : Rows(input, st, tokens), w(needed(weight, "weight")), bias(tensor(b, "bias")), K(0), act(act_code), xs(0)
    {
        if (w.dim() < 2 || w.dim() > 4 || w.size(0) != C || w.numel() % C != 0 || w.numel() / C > INT32_MAX)
            throw Refused("weight must be a depthwise weight [" + std::to_string(C) + ", K]; found " + text(w.sizes()));
        K = static_cast<int>(w.numel() / C);
        int64_t most = 1;
        for (int i = 1; i < w.dim(); ++i) most = std::max(most, w.size(i));
        if (most != K || K < 2 || K > 8) throw Refused("weight must have 2 to 8 taps for each channel, each of one input channel; found " + text(w.sizes()));
        c.fits(&w, "weight", w.sizes());
        c.fits(bias, "bias", {C});
        xs = like(&x, "x", x.sizes(), 1);
    }
    std::array<int64_t, 3> states() const { return {seqs, K - 1, C}; }
};

// x weight bias act starts initial last out stream
PyObject* causal(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded(n, 9, [&]() -> PyObject* {
        Causal k(needed(a[0], "x"), a[1], a[2], integer(a[3]), tensor(a[4], "starts"), false);
        const at::Tensor *initial = tensor(a[5], "initial"), *last = tensor(a[6], "last"), *out = tensor(a[7], "out");
        k.c.fits(initial, "initial", k.states());
        k.c.fits(last, "last", k.states());
        k.c.fits(out, "out", k.x.sizes());
        k.c.on_gpu();
        at::Tensor y = out ? *out : like(k.x);
        void* stream = address(a[8]);
        const int rc = call([&] {
            return api.causal_fwd(k.x.data_ptr(), k.w.data_ptr(), at_of(k.bias), k.at_starts(), at_of(initial), y.data_ptr(), at_of(last), k.rows, k.seqs,
                                  k.C, k.K, k.xs, k.act, !out, k.c.dtype, stream);
        });
        if (rc) return status(rc);
        wrote(out);
        wrote(last);
        return THPVariable_Wrap(y);
    });
}

// dy x weight bias act starts initial dlast workspace stream
PyObject* causal_grad(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded(n, 10, [&]() -> PyObject* {
        Causal k(needed(a[1], "x"), a[2], a[3], integer(a[4]), tensor(a[5], "starts"), false);
        const at::Tensor &dy = needed(a[0], "dy"), *initial = tensor(a[6], "initial"), *dlast = tensor(a[7], "dlast");
        k.c.fits(&dy, "dy", k.x.sizes());
        k.c.fits(initial, "initial", k.states());
        k.c.fits(dlast, "dlast", k.states());
        k.c.on_gpu();
        size_t need = 0;
        if (int rc = api.causal_bwd_workspace(k.rows, k.C, k.K, k.c.dtype, &need)) return status(rc);
        Workspace ws(tensor(a[8], "workspace"), k.x, need);
        std::array<at::Tensor, 4> d = {like(k.x), like(k.w)};
        if (k.bias) d[2] = like(*k.bias);
        if (initial) d[3] = like(*initial);
        void* stream = address(a[9]);
        const int rc = call([&] {
            return api.causal_bwd(dy.data_ptr(), at_of(dlast), k.x.data_ptr(), k.w.data_ptr(), at_of(k.bias), k.at_starts(), at_of(initial), d[0].data_ptr(),
                                  d[1].data_ptr(), k.bias ? d[2].data_ptr() : nullptr, initial ? d[3].data_ptr() : nullptr, ws.at, ws.bytes, k.rows, k.seqs,
                                  k.C, k.K, k.xs, k.act, 1, k.c.dtype, stream);
        });
        if (rc) return status(rc);
        PyObject* r = PyTuple_New(4);
        for (int i = 0; r && i < 4; ++i) PyTuple_SET_ITEM(r, i, wrap(&d[i]));
        return r;
    });
}

// x weight state bias act slots out stream
PyObject* causal_step(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded(n, 8, [&]() -> PyObject* {
        Causal k(needed(a[0], "x"), a[1], a[3], integer(a[4]), nullptr, true);
        const at::Tensor* out = tensor(a[6], "out");
        Pool p(needed(a[2], "state"), tensor(a[5], "slots"), k.rows, k.c.device);
        k.c.fits(&p.state, "state", {p.count, k.K - 1, k.C});
        k.c.fits(out, "out", k.x.sizes());
        k.c.on_gpu();
        at::Tensor y = out ? *out : like(k.x);
        void* stream = address(a[7]);
        const int rc = call([&] {
            return api.causal_step(k.x.data_ptr(), k.w.data_ptr(), at_of(k.bias), p.state.data_ptr(), static_cast<const int*>(at_of(p.slots)), y.data_ptr(),
                                   k.rows, p.count, k.C, k.K, k.xs, k.act, !out, k.c.dtype, stream);
        });
        if (rc) return status(rc);
        wrote(out);
        wrote(&p.state);
        return THPVariable_Wrap(y);
    });
}

// x delta A B C D z delta_bias softplus act
struct Scan : Rows {
    const at::Tensor &delta, &A, &B, &C_, *D, *z, *bias;
    int N, groups, softplus, act;
    int64_t xs, ds, zs, bs, cs;
    Shape shared;  // of B and C

    Scan(PyObject* const* a, const at::Tensor* st, bool tokens)
        : Rows(needed(a[0], "x"), st, tokens), delta(needed(a[1], "delta")), A(needed(a[2], "A")), B(needed(a[3], "B")), C_(needed(a[4], "C")),
          D(tensor(a[5], "D")), z(tensor(a[6], "z")), bias(tensor(a[7], "delta_bias")), N(0), groups(1), softplus(integer(a[8])), act(integer(a[9]))
    {
        if (A.dim() != 2 || A.size(0) != C || A.size(1) < 1 || A.size(1) > 64)
            throw Refused("A must have shape [" + std::to_string(C) + ", N] with 1 to 64 states; found " + text(A.sizes()));
        N = static_cast<int>(A.size(1));
        shared = x.sizes().vec();
        if (B.dim() == x.dim() + 1) {
            shared.back() = B.size(-2);
            shared.push_back(N);
            groups = narrow(B.size(-2), "the number of groups");
            if (groups < 1 || C % groups != 0 || groups > 65535) throw Refused("the groups of B and C must divide the channels of x; found " + std::to_string(groups));
        } else {
            shared.back() = N;
        }
        const at::IntArrayRef full = x.sizes();
        xs = like(&x, "x", full, 1);
        ds = like(&delta, "delta", full, 1);
        zs = like(z, "z", full, 1);
        const int tail = B.dim() == x.dim() + 1 ? 2 : 1;
        bs = like(&B, "B", shared, tail);
        cs = like(&C_, "C", shared, tail);
        const std::array<int64_t, 2> an = {C, N};
        const std::array<int64_t, 1> one = {C};
        plain(&A, "A", an, at::kFloat, x.device());
        plain(D, "D", one, at::kFloat, x.device());
        plain(bias, "delta_bias", one, at::kFloat, x.device());
    }
    void state(const at::Tensor* t, const char* name, int64_t count) const
    {
        const std::array<int64_t, 3> shape = {count, C, N};
        plain(t, name, shape, at::kFloat, x.device());
    }
    void kept(const at::Tensor* t) const
    {
        size_t need = 0;
        if (t && api.scan_saved(rows, C, N, &need) == CONV_OK && (t->scalar_type() != at::kFloat || t->device() != x.device() || !t->is_contiguous() || t->nbytes() != need))
            throw Refused("saved must be contiguous float32 on the input's device with " + std::to_string(need / 4) + " values; found " + c10::toString(t->scalar_type()) +
                          " " + text(t->sizes()));
    }
    const float* f(const at::Tensor* t) const { return static_cast<const float*>(at_of(t)); }
};
float* floats(const at::Tensor* t) { return static_cast<float*>(at_of(t)); }

// the ten of Scan, starts initial last saved out stream
PyObject* scan(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded(n, 16, [&]() -> PyObject* {
        Scan k(a, tensor(a[10], "starts"), false);
        const at::Tensor *initial = tensor(a[11], "initial"), *last = tensor(a[12], "last"), *saved = tensor(a[13], "saved"), *out = tensor(a[14], "out");
        k.state(initial, "initial", k.seqs);
        k.state(last, "last", k.seqs);
        k.kept(saved);
        k.c.fits(out, "out", k.x.sizes());
        k.c.on_gpu();
        size_t need = 0;
        if (int rc = api.scan_fwd_workspace(k.rows, k.seqs, k.C, k.N, k.groups, k.starts != nullptr, &need)) return status(rc);
        at::Tensor y = out ? *out : like(k.x), ws;
        if (need) ws = bytes_like(k.x, need);
        void* stream = address(a[15]);
        const int rc = call([&] {
            return api.scan_fwd(k.x.data_ptr(), k.delta.data_ptr(), k.f(&k.A), k.B.data_ptr(), k.C_.data_ptr(), k.f(k.D), at_of(k.z), k.f(k.bias), k.at_starts(),
                                k.f(initial), y.data_ptr(), floats(last), floats(saved), need ? ws.data_ptr() : nullptr, need, k.rows, k.seqs, k.C, k.N,
                                k.groups, k.xs, k.ds, k.zs, k.bs, k.cs, k.softplus, k.act, !out, k.c.dtype, stream);
        });
        if (rc) return status(rc);
        wrote(out);
        wrote(last);
        wrote(saved);
        return THPVariable_Wrap(y);
    });
}

// the ten of Scan, starts initial dy dlast saved workspace stream
PyObject* scan_grad(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded(n, 17, [&]() -> PyObject* {
        Scan k(a, tensor(a[10], "starts"), false);
        const at::Tensor *initial = tensor(a[11], "initial"), &dy = needed(a[12], "dy"), *dlast = tensor(a[13], "dlast"), *saved = tensor(a[14], "saved");
        k.state(initial, "initial", k.seqs);
        k.state(dlast, "dlast", k.seqs);
        k.kept(saved);
        k.c.fits(&dy, "dy", k.x.sizes());
        k.c.on_gpu();
        size_t need = 0;
        if (int rc = api.scan_bwd_workspace(k.rows, k.seqs, k.C, k.N, k.groups, k.starts != nullptr, saved != nullptr, &need)) return status(rc);
        Workspace ws(tensor(a[15], "workspace"), k.x, need);
        // x delta A B C D z delta_bias initial
        const std::array<const at::Tensor*, 9> in = {&k.x, &k.delta, &k.A, &k.B, &k.C_, k.D, k.z, k.bias, initial};
        std::array<at::Tensor, 9> d;
        std::array<void*, 9> to{};
        for (int i = 0; i < 9; ++i)
            if (in[i]) {
                d[i] = like(*in[i]);
                to[i] = d[i].data_ptr();
            }
        void* stream = address(a[16]);
        const int rc = call([&] {
            return api.scan_bwd(dy.data_ptr(), k.f(dlast), k.x.data_ptr(), k.delta.data_ptr(), k.f(&k.A), k.B.data_ptr(), k.C_.data_ptr(), k.f(k.D), at_of(k.z),
                                k.f(k.bias), k.at_starts(), k.f(initial), k.f(saved), to[0], to[1], static_cast<float*>(to[2]), to[3], to[4],
                                static_cast<float*>(to[5]), to[6], static_cast<float*>(to[7]), static_cast<float*>(to[8]), ws.at, ws.bytes, k.rows, k.seqs,
                                k.C, k.N, k.groups, k.xs, k.ds, k.zs, k.bs, k.cs, k.softplus, k.act, 1, k.c.dtype, stream);
        });
        if (rc) return status(rc);
        PyObject* r = PyTuple_New(9);
        for (int i = 0; r && i < 9; ++i) PyTuple_SET_ITEM(r, i, wrap(&d[i]));
        return r;
    });
}

// the ten of Scan, state slots out stream
PyObject* scan_step(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded(n, 14, [&]() -> PyObject* {
        Scan k(a, nullptr, true);
        const at::Tensor* out = tensor(a[12], "out");
        Pool p(needed(a[10], "state"), tensor(a[11], "slots"), k.rows, k.c.device);
        k.state(&p.state, "state", p.count);
        k.c.fits(out, "out", k.x.sizes());
        k.c.on_gpu();
        at::Tensor y = out ? *out : like(k.x);
        void* stream = address(a[13]);
        const int rc = call([&] {
            return api.scan_step(k.x.data_ptr(), k.delta.data_ptr(), k.f(&k.A), k.B.data_ptr(), k.C_.data_ptr(), k.f(k.D), at_of(k.z), k.f(k.bias),
                                 floats(&p.state), static_cast<const int*>(at_of(p.slots)), y.data_ptr(), k.rows, p.count, k.C, k.N, k.groups, k.xs, k.ds,
                                 k.zs, k.bs, k.cs, k.softplus, k.act, !out, k.c.dtype, stream);
        });
        if (rc) return status(rc);
        wrote(out);
        wrote(&p.state);
        return THPVariable_Wrap(y);
    });
}

// ------------------------------------------------------------ optimizer --

// A list of tensors beside the list of parameters; None entries where allowed.
struct Beside {
    std::vector<const at::Tensor*> tensors;
    std::vector<void*> at;
    std::vector<int> dtypes;
    bool given;

    Beside(PyObject* o, const char* name, int n, bool none_entries) : given(o != Py_None)
    {
        if (!given) return;
        if (!PyList_Check(o) || PyList_GET_SIZE(o) != n)
            throw Refused(std::string(name) + " must be a list of " + std::to_string(n) + " tensors, one for each parameter");
        for (int i = 0; i < n; ++i) {
            PyObject* e = PyList_GET_ITEM(o, i);
            const at::Tensor* t = none_entries ? tensor(e, name) : &needed(e, name);
            tensors.push_back(t);
            at.push_back(at_of(t));
            dtypes.push_back(0);
        }
    }
    void typed(const at::Tensor& p, int i, const char* name, at::ScalarType type) const
    {
        if (tensors[i]->scalar_type() != type || tensors[i]->device() != p.device())
            throw Refused(std::string(name) + " must be " + c10::toString(type) + " on the parameters' device; found " + c10::toString(tensors[i]->scalar_type()) + " on " +
                          tensors[i]->device().str());
    }
    // Elements of the i-th tensor lie as the parameter's do.
    void lies_as(const at::Tensor& p, int i, const char* name) const
    {
        const at::Tensor& t = *tensors[i];
        if (t.device() != p.device() || t.numel() != p.numel() || !lie_alike(t, p))
            throw Refused(std::string(name) + " must have the size, device and order in memory of their parameters; found " + text(t.sizes()) + " with strides " +
                          text(t.strides()) + " for " + text(p.sizes()) + " with strides " + text(p.strides()));
    }
    void bytes(const at::Tensor& p, int i, const char* name, int64_t count, at::ScalarType type) const
    {
        typed(p, i, name, type);
        if (tensors[i]->numel() != count || !tensors[i]->is_contiguous())
            throw Refused(std::string(name) + " must be contiguous with " + std::to_string(count) + " values; found " + text(tensors[i]->sizes()));
    }
    template <typename T>
    T* const* to() const
    {
        return given ? reinterpret_cast<T* const*>(at.data()) : nullptr;
    }
};
int64_t blocks_of(const at::Tensor& p) { return (p.numel() + 127) / 128; }

// params grads m v m_scales v_scales copies lr lr_tensor beta1 beta2 eps weight_decay step step_tensor norm max_norm norm_eps stream
PyObject* adamw(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded(n, 19, [&]() -> PyObject* {
        List p(a[0], "parameter");
        const int count = p.n();
        Beside g(a[1], "grads", count, false), m(a[2], "the states' m", count, false), v(a[3], "the states' v", count, false);
        Beside ms(a[4], "the states' m_scale", count, false), vs(a[5], "the states' v_scale", count, false), copies(a[6], "copies", count, true);
        if (!g.given || !m.given || !v.given || ms.given != vs.given) throw Refused("an AdamW step needs gradients, m and v, and with 8-bit states both scales");
        const int bits = ms.given ? 8 : 32;
        for (int i = 0; i < count; ++i) {
            const at::Tensor& t = *p.tensors[i];
            g.dtypes[i] = Call::code(*g.tensors[i]);
            g.lies_as(t, i, "grads");
            if (bits == 8) {
                m.bytes(t, i, "the states' m", t.numel(), at::kChar);
                v.bytes(t, i, "the states' v", t.numel(), at::kByte);
                ms.bytes(t, i, "the states' m_scale", blocks_of(t), at::kFloat);
                vs.bytes(t, i, "the states' v_scale", blocks_of(t), at::kFloat);
            } else {
                m.typed(t, i, "the states' m", at::kFloat);
                v.typed(t, i, "the states' v", at::kFloat);
                m.lies_as(t, i, "the states' m");
                v.lies_as(t, i, "the states' v");
            }
            if (copies.given && copies.tensors[i]) {
                copies.dtypes[i] = Call::code(*copies.tensors[i]);
                copies.lies_as(t, i, "copies");
            }
        }
        auto scalar = [&](PyObject* o, const char* name, at::ScalarType type) {
            const at::Tensor* t = tensor(o, name);
            if (t && (t->numel() != 1 || t->scalar_type() != type || t->device() != p.first->device()))
                throw Refused(std::string(name) + " as a tensor is one " + c10::toString(type) + " value on the parameters' device");
            return t;
        };
        const at::Tensor *lr = scalar(a[8], "lr", at::kFloat), *step = scalar(a[14], "step", at::kLong), *norm = scalar(a[15], "norm", at::kFloat);
        double f[7];
        const int from[7] = {7, 9, 10, 11, 12, 16, 17};  // lr beta1 beta2 eps weight_decay max_norm norm_eps
        for (int i = 0; i < 7; ++i) f[i] = PyFloat_AsDouble(a[from[i]]);
        const long long number = PyLong_AsLongLong(a[13]);
        if (PyErr_Occurred()) return nullptr;
        void* stream = address(a[18]);
        const int rc = call([&] {
            return api.adamw(p.at.data(), g.to<const void>(), m.to<void>(), v.to<void>(), ms.to<float>(), vs.to<float>(), copies.to<void>(), p.counts.data(),
                             p.dtypes.data(), g.dtypes.data(), copies.dtypes.data(), count, bits, f[0], f[1], f[2], f[3], f[4], number,
                             static_cast<const float*>(at_of(lr)), static_cast<const long long*>(at_of(step)), static_cast<const float*>(at_of(norm)), f[5], f[6],
                             stream);
        });
        if (rc) return status(rc);
        for (const at::Tensor* t : p.tensors) wrote(t);
        for (const Beside* b : {&m, &v, &ms, &vs, &copies})
            for (const at::Tensor* t : b->tensors) wrote(t);
        Py_RETURN_NONE;
    });
}

// m v m_scales v_scales m_out v_out stream
PyObject* moments(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded(n, 7, [&]() -> PyObject* {
        if (!PyList_Check(a[0])) throw Refused("the states' m must be a list of tensors");
        if (PyList_GET_SIZE(a[0]) == 0) throw Refused("the list of states is empty");
        const int count = narrow(PyList_GET_SIZE(a[0]), "the number of tensors");
        Beside m(a[0], "m", count, false), v(a[1], "v", count, false), ms(a[2], "m_scale", count, false), vs(a[3], "v_scale", count, false);
        Beside mo(a[4], "out's m", count, false), vo(a[5], "out's v", count, false);
        std::vector<size_t> counts;
        for (int i = 0; i < count; ++i) {
            const at::Tensor& t = *m.tensors[i];
            if (!t.is_cuda() || t.device() != m.tensors[0]->device()) throw Refused("tensors passed to convmi must be on one GPU device");
            m.bytes(t, i, "m", t.numel(), at::kChar);
            v.bytes(t, i, "v", t.numel(), at::kByte);
            ms.bytes(t, i, "m_scale", blocks_of(t), at::kFloat);
            vs.bytes(t, i, "v_scale", blocks_of(t), at::kFloat);
            mo.bytes(t, i, "out's m", t.numel(), at::kFloat);
            vo.bytes(t, i, "out's v", t.numel(), at::kFloat);
            counts.push_back(static_cast<size_t>(t.numel()));
        }
        void* stream = address(a[6]);
        const int rc = call([&] {
            return api.moments(m.to<const void>(), v.to<const void>(), ms.to<const float>(), vs.to<const float>(), mo.to<float>(), vo.to<float>(), counts.data(),
                               count, stream);
        });
        if (rc) return status(rc);
        for (const Beside* b : {&mo, &vo})
            for (const at::Tensor* t : b->tensors) wrote(t);
        Py_RETURN_NONE;
    });
}

// The addresses of the C functions, in the order of Api.
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded(n, kApi, [&]() -> PyObject* {
        for (int i = 0; i < kApi; ++i) reinterpret_cast<void**>(&api)[i] = address(a[i]);
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
                         {"causal", FAST(causal), METH_FASTCALL, nullptr},
                         {"causal_grad", FAST(causal_grad), METH_FASTCALL, nullptr},
                         {"causal_step", FAST(causal_step), METH_FASTCALL, nullptr},
                         {"scan", FAST(scan), METH_FASTCALL, nullptr},
                         {"scan_grad", FAST(scan_grad), METH_FASTCALL, nullptr},
                         {"scan_step", FAST(scan_step), METH_FASTCALL, nullptr},
                         {"adamw", FAST(adamw), METH_FASTCALL, nullptr},
                         {"moments", FAST(moments), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_native", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__native() { return PyModule_Create(&module); }
