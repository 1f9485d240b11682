// block_binding.cpp -- the Python binding of include/gma_block.h (module _block): checks torch CUDA tensors,
// allocates outputs and workspaces through torch, fills the header's structs and calls libgma.so on the
// current stream.  A call for one token takes a few microseconds on the GPU; with the marshalling in
// Python the host took 17 us a call, here 5.  ssm.py and norm.py hold the documented functions; each passes its
// arguments on in order.  Tensors are checked for type, device, dtype, shape and contiguous channels; what the C
// entry points refuse comes back as gma.GmaError.
#include <string>
#include <vector>

#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <ATen/ops/empty.h>
#include <ATen/ops/zeros.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>

#include "gma_block.h"

namespace {

struct Fail {
    PyObject *type;
    std::string words;
};
[[noreturn]] void type_error(const std::string &w) { throw Fail{PyExc_TypeError, w}; }
[[noreturn]] void value_error(const std::string &w) { throw Fail{PyExc_ValueError, w}; }
struct Raised {};        // a Python exception is set already

std::string list_of(at::IntArrayRef s)
{
    std::string r = "[";
    for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
    return r + "]";
}

bool given(PyObject *o) { return o != Py_None; }

const at::Tensor &tensor(PyObject *o, const char *name)
{
    if (!THPVariable_Check(o)) type_error(std::string(name) + " must be a CUDA tensor");
    const at::Tensor &t = THPVariable_Unpack(o);
    if (!t.is_cuda()) type_error(std::string(name) + " must be a CUDA tensor");
    return t;
}

// What the first activation fixes for the whole call.
struct Call {
    at::ScalarType T;
    int dev;
    c10::TensorOptions options, f32;
    int32_t dtype() const { return T == at::kBFloat16 ? GMA_BF16 : GMA_F32; }
    gma_stream_t stream() const { return (gma_stream_t)c10::cuda::getCurrentCUDAStream(dev).stream(); }
    at::Tensor empty(at::IntArrayRef shape) const { return at::empty(shape, options); }
    at::Tensor empty32(at::IntArrayRef shape) const { return at::empty(shape, f32); }
    at::Tensor rows(at::IntArrayRef shape, bool zero) const { return zero ? at::zeros(shape, options) : at::empty(shape, options); }
};

Call begin(const at::Tensor &t, const char *name)
{
    const at::ScalarType T = t.scalar_type();
    if (T != at::kBFloat16 && T != at::kFloat)
        type_error(std::string(name) + " must be bf16 or fp32, got " + c10::toString(T));
    const int dev = t.get_device();
    if (dev != c10::cuda::current_device()) value_error(std::string(name) + " must be on the current CUDA device");
    const c10::TensorOptions o = c10::TensorOptions().device(t.device()).dtype(T);
    return Call{T, dev, o, o.dtype(at::kFloat)};
}

void check(const at::Tensor &t, const char *name, at::IntArrayRef shape, at::ScalarType T, const Call &c)
{
    if (t.scalar_type() != T)
        type_error(std::string(name) + " must be " + c10::toString(T) + ", got " + c10::toString(t.scalar_type()));
    if (t.get_device() != c.dev) value_error(std::string(name) + " must be on the same device as the other tensors");
    if (t.sizes() != shape) value_error(std::string(name) + " must be " + list_of(shape) + ", got " + list_of(t.sizes()));
}

// Rows [B, N, channels...] whose channels are contiguous; `at` is the token dimension (0: there is none, one token).
gma_rows_t rows(const at::Tensor &t, const char *name, at::IntArrayRef shape, size_t at, at::ScalarType T, const Call &c)
{
    check(t, name, shape, T, c);
    const at::IntArrayRef s = t.strides();
    int64_t width = 1;
    for (size_t k = shape.size(); k-- > at + 1;) {
        if (s[k] != width && shape[k] != 1) value_error(std::string(name) + "'s channels must be contiguous");
        width *= shape[k];
    }
    return gma_rows_t{t.data_ptr(), s[0], at ? s[at] : 0};
}
gma_rows_t rows(PyObject *o, const char *name, at::IntArrayRef shape, size_t at, at::ScalarType T, const Call &c)
{
    return rows(tensor(o, name), name, shape, at, T, c);
}
gma_rows_t maybe_rows(PyObject *o, const char *name, at::IntArrayRef shape, size_t at, at::ScalarType T, const Call &c)
{
    return given(o) ? rows(o, name, shape, at, T, c) : gma_rows_t{nullptr, 0, 0};
}

// Heads [B, H, N, d] (or rows [B, N, D]) and the stride between them.
gma_rows_t heads(const at::Tensor &t, const char *name, at::IntArrayRef shape, const Call &c, int64_t *head)
{
    check(t, name, shape, c.T, c);
    const at::IntArrayRef s = t.strides();
    if (s.back() != 1 && shape.back() != 1) value_error(std::string(name) + "'s channels must be contiguous");
    *head = shape.size() == 4 ? s[1] : 0;
    return gma_rows_t{t.data_ptr(), s[0], shape.size() == 4 ? s[2] : s[1]};
}

// An output must not start where another tensor of the call does (the header forbids any overlap; rows of one
// buffer may lie beside one another, so that is as much as the addresses tell).
void apart(const gma_rows_t &out, const char *name, std::initializer_list<const gma_rows_t *> others)
{
    for (const gma_rows_t *o : others)
        if (out.ptr && out.ptr == o->ptr) value_error(std::string(name) + " must not be another tensor of the call");
}

template <typename P = float> P *dense(PyObject *o, const char *name, at::IntArrayRef shape, at::ScalarType T, const Call &c)
{
    if (!given(o)) return nullptr;
    const at::Tensor &t = tensor(o, name);
    check(t, name, shape, T, c);
    if (!t.is_contiguous()) value_error(std::string(name) + " must be contiguous");
    return (P *)t.data_ptr();
}
template <typename P = float> P *need(PyObject *o, const char *name, at::IntArrayRef shape, at::ScalarType T, const Call &c)
{
    if (!given(o)) type_error(std::string(name) + " is required");
    return dense<P>(o, name, shape, T, c);
}

int64_t param_size(PyObject *o, const char *name, const char *what)
{
    if (!THPVariable_Check(o) || THPVariable_Unpack(o).dim() != 2) value_error(std::string(name) + " must be " + what);
    return THPVariable_Unpack(o).size(1);
}

// GmaError(status, what), or the other kinds of error.
PyObject *raise_status(gma_status_t r, const char *what)
{
    PyObject *mod = PyImport_ImportModule("linear_latent_routing_gb300.gma");
    PyObject *cls = mod ? PyObject_GetAttrString(mod, "GmaError") : nullptr;
    PyObject *err = cls ? PyObject_CallFunction(cls, "is", (int)r, what) : nullptr;
    if (err) PyErr_SetObject(cls, err);
    Py_XDECREF(err);
    Py_XDECREF(cls);
    Py_XDECREF(mod);
    return nullptr;
}

template <typename F> PyObject *guarded(Py_ssize_t have, Py_ssize_t want, F f)
{
    if (have != want) {
        PyErr_Format(PyExc_TypeError, "%zd arguments, got %zd", want, have);
        return nullptr;
    }
    try {
        return f();
    } catch (const Fail &e) {
        PyErr_SetString(e.type, e.words.c_str());
    } catch (const Raised &) {
    } catch (const c10::OutOfMemoryError &) {
        torch::translate_exception_to_python(std::current_exception());      // torch.OutOfMemoryError
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

PyObject *wrap(const at::Tensor &t) { return THPVariable_Wrap(t); }
PyObject *none() { Py_RETURN_NONE; }

// The caller's tensor for an output, or a new one.
template <typename F> at::Tensor out_or(PyObject *o, const char *name, F make) { return given(o) ? tensor(o, name) : make(); }

struct Workspace {
    at::Tensor t;
    size_t bytes;
    Workspace(size_t n, const Call &c) : bytes(n)
    {
        if (n) t = at::empty({(int64_t)n}, c.options.dtype(at::kByte));
    }
    void *ptr() const { return bytes ? t.data_ptr() : nullptr; }
};

void set(PyObject *dict, const char *key, const at::Tensor &t)
{
    PyObject *v = t.defined() ? wrap(t) : none();
    if (!v || PyDict_SetItemString(dict, key, v) < 0) {
        Py_XDECREF(v);
        throw Fail{PyExc_RuntimeError, "cannot fill the result"};
    }
    Py_DECREF(v);
}

// ------------------------------------------------------------------ selective scan

// u, dt, a_log, b, c, d_skip, dt_bias, z: arguments 0 .. 7 of every scan call; one token: no token dimension.
gma_scan_t scan_of(PyObject *const *a, bool step, Call *call, std::vector<int64_t> *full, std::vector<int64_t> *bc)
{
    const at::Tensor &u = tensor(a[0], "u");
    *call = begin(u, "u");
    if (u.dim() != (step ? 2 : 3)) value_error(step ? "u must be [B, D]" : "u must be [B, N, D]");
    gma_scan_t s = {};
    const int64_t B = u.size(0), N = step ? 1 : u.size(1), D = u.size(-1), S = param_size(a[2], "a_log", "[D, S]");
    const at::Tensor &b = tensor(a[3], "b");
    const bool groups = b.dim() == (step ? 3 : 4);
    const int64_t G = groups ? b.size(step ? 1 : 2) : 1;
    *full = step ? std::vector<int64_t>{B, D} : std::vector<int64_t>{B, N, D};
    *bc = step ? std::vector<int64_t>{B} : std::vector<int64_t>{B, N};
    if (groups) bc->push_back(G);
    bc->push_back(S);
    const size_t at = step ? 0 : 1;
    const at::ScalarType T = call->T;
    if (B > INT32_MAX || N > INT32_MAX || D > INT32_MAX || G > INT32_MAX || S > INT32_MAX) value_error("a size is too large");
    s.B = (int32_t)B; s.N = (int32_t)N; s.D = (int32_t)D; s.S = (int32_t)S; s.G = (int32_t)G;
    s.dtype = call->dtype();
    s.u = rows(u, "u", *full, at, T, *call);
    s.dt = rows(a[1], "dt", *full, at, T, *call);
    s.z = maybe_rows(a[7], "z", *full, at, T, *call);
    s.b = rows(b, "b", *bc, at, T, *call);
    s.c = rows(a[4], "c", *bc, at, T, *call);
    s.a_log = dense(a[2], "a_log", {D, S}, at::kFloat, *call);
    s.d_skip = dense(a[5], "d_skip", {D}, at::kFloat, *call);
    s.dt_bias = dense(a[6], "dt_bias", {D}, at::kFloat, *call);
    return s;
}

int64_t checkpoints_of(const gma_scan_t &s)
{
    const int n = gma_scan_checkpoint_tokens(&s);
    return n ? (s.N + n - 1) / n : 0;
}

// u, S: a buffer for the checkpoints
PyObject *scan_checkpoints(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 2, [&]() -> PyObject * {
        const at::Tensor &u = tensor(a[0], "u");
        const Call c = begin(u, "u");
        const long S = PyLong_AsLong(a[1]);
        if (PyErr_Occurred()) {
            PyErr_Clear();
            type_error("S must be a whole number");
        }
        if (u.dim() != 3) value_error("u must be [B, N, D]");
        if (u.size(0) > INT32_MAX || u.size(1) > INT32_MAX || u.size(2) > INT32_MAX || S > 64 || S < 1) value_error("sizes do not fit");
        gma_scan_t s = {};
        s.B = (int32_t)u.size(0); s.N = (int32_t)u.size(1); s.D = (int32_t)u.size(2); s.S = (int32_t)S;
        const int64_t kept = checkpoints_of(s);
        if (!kept && s.B && s.N && s.D) value_error("sizes do not fit");
        return wrap(c.empty32({s.B, kept, s.D, s.S}));
    });
}

// ..., state, state_out, lengths, checkpoints, out
PyObject *scan(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 13, [&]() -> PyObject * {
        Call c;
        std::vector<int64_t> full, bc;
        gma_scan_t s = scan_of(a, false, &c, &full, &bc);
        const int64_t B = s.B, N = s.N, D = s.D, S = s.S;
        s.state_in = dense(a[8], "state", {B, D, S}, at::kFloat, c);
        s.state_out = dense(a[9], "state_out", {B, D, S}, at::kFloat, c);
        s.lengths = dense<int32_t>(a[10], "lengths", {B}, at::kInt, c);
        s.checkpoints = dense(a[11], "checkpoints", {B, checkpoints_of(s), D, S}, at::kFloat, c);
        if (s.lengths && !given(a[12])) s.flags |= GMA_ROWS_ZERO_TAIL;      // in a buffer allocated here
        const at::Tensor y = out_or(a[12], "out", [&] { return c.empty(full); });
        s.y = rows(y, "out", full, 1, c.T, c);
        if (given(a[12])) apart(s.y, "out", {&s.u, &s.dt, &s.z, &s.b, &s.c});
        const Workspace ws(gma_scan_workspace_size(&s), c);
        const gma_status_t r = gma_scan_forward(&s, ws.ptr(), ws.bytes, c.stream());
        return r == GMA_OK ? wrap(y) : raise_status(r, "gma_scan_forward");
    });
}

// ..., state, out
PyObject *scan_step(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 10, [&]() -> PyObject * {
        Call c;
        std::vector<int64_t> full, bc;
        gma_scan_t s = scan_of(a, true, &c, &full, &bc);
        s.state_out = need(a[8], "state", {s.B, s.D, s.S}, at::kFloat, c);
        s.state_in = s.state_out;
        const at::Tensor y = out_or(a[9], "out", [&] { return c.empty(full); });
        s.y = rows(y, "out", full, 0, c.T, c);
        if (given(a[9])) apart(s.y, "out", {&s.u, &s.dt, &s.z, &s.b, &s.c});
        const gma_status_t r = gma_scan_step(&s, c.stream());
        return r == GMA_OK ? wrap(y) : raise_status(r, "gma_scan_step");
    });
}

// ..., dy, checkpoints, dstate_out, lengths, out of u, dt, z, b, c
PyObject *scan_backward(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 17, [&]() -> PyObject * {
        Call c;
        std::vector<int64_t> full, bc;
        gma_scan_grad_t g = {};
        g.fwd = scan_of(a, false, &c, &full, &bc);
        gma_scan_t &s = g.fwd;
        const int64_t B = s.B, N = s.N, D = s.D, S = s.S;
        g.dy = rows(a[8], "dy", full, 1, c.T, c);
        s.checkpoints = need(a[9], "checkpoints", {B, checkpoints_of(s), D, S}, at::kFloat, c);
        g.dstate_out = dense(a[10], "dstate_out", {B, D, S}, at::kFloat, c);
        s.lengths = dense<int32_t>(a[11], "lengths", {B}, at::kInt, c);
        // the rows behind a sequence's end: zero in buffers allocated here, left alone in the caller's
        const bool z = s.z.ptr != nullptr, some = given(a[12]) || given(a[13]) || given(a[14]) || given(a[15]) || given(a[16]);
        const bool zero = s.lengths && some;
        if (s.lengths && !some) s.flags |= GMA_ROWS_ZERO_TAIL;
        const at::Tensor du = out_or(a[12], "out['u']", [&] { return c.rows(full, zero); });
        const at::Tensor ddt = out_or(a[13], "out['dt']", [&] { return c.rows(full, zero); });
        const at::Tensor dz = z ? out_or(a[14], "out['z']", [&] { return c.rows(full, zero); }) : at::Tensor();
        const at::Tensor db = out_or(a[15], "out['b']", [&] { return c.rows(bc, zero); });
        const at::Tensor dc = out_or(a[16], "out['c']", [&] { return c.rows(bc, zero); });
        g.du = rows(du, "out['u']", full, 1, c.T, c);
        g.ddt = rows(ddt, "out['dt']", full, 1, c.T, c);
        if (z) g.dz = rows(dz, "out['z']", full, 1, c.T, c);
        g.db = rows(db, "out['b']", bc, 1, c.T, c);
        g.dc = rows(dc, "out['c']", bc, 1, c.T, c);
        if (some) {
            const gma_rows_t *outs[5] = {&g.du, &g.ddt, &g.dz, &g.db, &g.dc};
            for (int i = 0; i < 5; ++i) {
                apart(*outs[i], "an output", {&s.u, &s.dt, &s.z, &s.b, &s.c, &g.dy});
                for (int j = 0; j < i; ++j) apart(*outs[i], "an output", {outs[j]});
            }
        }
        const at::Tensor da = c.empty32({D, S}), dstate = c.empty32({B, D, S});
        const at::Tensor dskip = s.d_skip ? c.empty32({D}) : at::Tensor(), dbias = s.dt_bias ? c.empty32({D}) : at::Tensor();
        g.da_log = (float *)da.data_ptr();
        g.dstate_in = (float *)dstate.data_ptr();
        if (s.d_skip) g.dd_skip = (float *)dskip.data_ptr();
        if (s.dt_bias) g.ddt_bias = (float *)dbias.data_ptr();
        const Workspace ws(gma_scan_backward_workspace_size(&g), c);
        const gma_status_t r = gma_scan_backward(&g, ws.ptr(), ws.bytes, c.stream());
        if (r != GMA_OK) return raise_status(r, "gma_scan_backward");
        PyObject *d = PyDict_New();
        if (!d) return nullptr;
        set(d, "u", du); set(d, "dt", ddt); set(d, "z", dz); set(d, "b", db); set(d, "c", dc);
        set(d, "a_log", da); set(d, "d_skip", dskip); set(d, "dt_bias", dbias); set(d, "state", dstate);
        return d;
    });
}

// ------------------------------------------------------------------ convolution

// x, weight, bias, state, silu: arguments 0 .. 4 of every convolution call
gma_conv_t conv_of(PyObject *const *a, bool step, Call *call, std::vector<int64_t> *full)
{
    const at::Tensor &x = tensor(a[0], "x");
    *call = begin(x, "x");
    if (x.dim() != (step ? 2 : 3)) value_error(step ? "x must be [B, D]" : "x must be [B, N, D]");
    const int64_t B = x.size(0), N = step ? 1 : x.size(1), D = x.size(-1), W = param_size(a[1], "weight", "[D, W]");
    if (B > INT32_MAX || N > INT32_MAX || D > INT32_MAX || W > INT32_MAX) value_error("a size is too large");
    *full = x.sizes().vec();
    const int silu = PyObject_IsTrue(a[4]);
    if (silu < 0) throw Fail{PyExc_TypeError, "silu must be a truth value"};
    gma_conv_t s = {};
    s.B = (int32_t)B; s.N = (int32_t)N; s.D = (int32_t)D; s.W = (int32_t)W;
    s.dtype = call->dtype();
    s.flags = silu ? 0 : GMA_CONV_LINEAR;
    s.x = rows(x, "x", *full, step ? 0 : 1, call->T, *call);
    s.weight = dense(a[1], "weight", {D, W}, at::kFloat, *call);
    s.bias = dense(a[2], "bias", {D}, at::kFloat, *call);
    s.state_in = dense<void>(a[3], "state", {B, W - 1, D}, call->T, *call);
    return s;
}

// ..., state_out, lengths, out
PyObject *conv(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 8, [&]() -> PyObject * {
        Call c;
        std::vector<int64_t> full;
        gma_conv_t s = conv_of(a, false, &c, &full);
        s.state_out = dense<void>(a[5], "state_out", {s.B, s.W - 1, s.D}, c.T, c);
        s.lengths = dense<int32_t>(a[6], "lengths", {s.B}, at::kInt, c);
        if (s.lengths && !given(a[7])) s.flags |= GMA_ROWS_ZERO_TAIL;
        const at::Tensor y = out_or(a[7], "out", [&] { return c.empty(full); });
        s.y = rows(y, "out", full, 1, c.T, c);
        if (given(a[7])) apart(s.y, "out", {&s.x});
        const gma_status_t r = gma_conv_forward(&s, c.stream());
        return r == GMA_OK ? wrap(y) : raise_status(r, "gma_conv_forward");
    });
}

// ..., out
PyObject *conv_step(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 6, [&]() -> PyObject * {
        Call c;
        std::vector<int64_t> full;
        gma_conv_t s = conv_of(a, true, &c, &full);
        if (!s.state_in) type_error("state is required");
        s.state_out = const_cast<void *>(s.state_in);
        const at::Tensor y = out_or(a[5], "out", [&] { return c.empty(full); });
        s.y = rows(y, "out", full, 0, c.T, c);
        if (given(a[5])) apart(s.y, "out", {&s.x});
        const gma_status_t r = gma_conv_step(&s, c.stream());
        return r == GMA_OK ? wrap(y) : raise_status(r, "gma_conv_step");
    });
}

// ..., dy, lengths, out
PyObject *conv_backward(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 8, [&]() -> PyObject * {
        Call c;
        std::vector<int64_t> full;
        gma_conv_grad_t g = {};
        g.fwd = conv_of(a, false, &c, &full);
        gma_conv_t &s = g.fwd;
        g.dy = rows(a[5], "dy", full, 1, c.T, c);
        s.lengths = dense<int32_t>(a[6], "lengths", {s.B}, at::kInt, c);
        if (s.lengths && !given(a[7])) s.flags |= GMA_ROWS_ZERO_TAIL;
        const at::Tensor dx = out_or(a[7], "out", [&] { return c.empty(full); });
        g.dx = rows(dx, "out", full, 1, c.T, c);
        if (given(a[7])) apart(g.dx, "out", {&s.x, &g.dy});
        const at::Tensor dw = c.empty32({s.D, s.W}), db = s.bias ? c.empty32({s.D}) : at::Tensor();
        g.dweight = (float *)dw.data_ptr();
        if (s.bias) g.dbias = (float *)db.data_ptr();
        const Workspace ws(gma_conv_backward_workspace_size(&g), c);
        const gma_status_t r = gma_conv_backward(&g, ws.ptr(), ws.bytes, c.stream());
        if (r != GMA_OK) return raise_status(r, "gma_conv_backward");
        PyObject *d = PyDict_New();
        if (!d) return nullptr;
        set(d, "x", dx); set(d, "weight", dw); set(d, "bias", db);
        return d;
    });
}

// ------------------------------------------------------------------ norms

// o, w_post, gate, scale, w_pre, eps, group: arguments 0 .. 6; R: the residual stream's type
gma_norm_t norm_of(PyObject *const *a, Call *call, std::vector<int64_t> *full)
{
    const at::Tensor &o = tensor(a[0], "o");
    *call = begin(o, "o");
    if (o.dim() != 3 && o.dim() != 4) value_error("o must be [B, H, N, d] or [B, N, D]");
    const bool h4 = o.dim() == 4;
    const int64_t B = o.size(0), H = h4 ? o.size(1) : 1, N = o.size(h4 ? 2 : 1), d = o.size(-1), D = H * d;
    if (B > INT32_MAX || N > INT32_MAX || D > INT32_MAX) value_error("a size is too large");
    *full = {B, N, D};
    gma_norm_t s = {};
    s.B = (int32_t)B; s.N = (int32_t)N; s.H = (int32_t)H; s.d = (int32_t)d;
    const long group = PyLong_AsLong(a[6]);
    const double eps = PyFloat_AsDouble(a[5]);
    if (PyErr_Occurred()) {
        PyErr_Clear();
        type_error("eps must be a number and group a whole one");
    }
    s.group = group ? (group > INT32_MAX || group < INT32_MIN ? -1 : (int32_t)group) : (int32_t)D;
    s.dtype = s.residual_dtype = call->dtype();
    s.eps = (float)eps;
    s.o = heads(o, "o", o.sizes(), *call, &s.o_head);
    s.gate = maybe_rows(a[2], "gate", *full, 1, call->T, *call);
    s.w_post = dense(a[1], "w_post", {D}, at::kFloat, *call);
    s.scale = dense(a[3], "scale", {D}, at::kFloat, *call);
    s.w_pre = dense(a[4], "w_pre", {D}, at::kFloat, *call);
    return s;
}

at::ScalarType stream_type(const at::Tensor &t, const char *name, const Call &c)
{
    if (t.scalar_type() != c.T && t.scalar_type() != at::kFloat)
        type_error(std::string(name) + " must be " + c10::toString(c.T) + " or Float");
    return t.scalar_type();
}
int32_t code(at::ScalarType T) { return T == at::kBFloat16 ? GMA_BF16 : GMA_F32; }

// ..., residual, out, out_h
PyObject *block_norm(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 10, [&]() -> PyObject * {
        Call c;
        std::vector<int64_t> full;
        gma_norm_t s = norm_of(a, &c, &full);
        at::ScalarType R = c.T;
        if (given(a[7])) {
            R = stream_type(tensor(a[7], "residual"), "residual", c);
            s.residual = rows(a[7], "residual", full, 1, R, c);
            s.residual_dtype = code(R);
        }
        const at::Tensor r = out_or(a[8], "out", [&] { return at::empty(full, c.options.dtype(R)); });
        s.r = rows(r, "out", full, 1, R, c);
        if (given(a[8])) apart(s.r, "out", {&s.o, &s.gate});
        at::Tensor h;
        if (s.w_pre) {
            h = out_or(a[9], "out_h", [&] { return c.empty(full); });
            s.h = rows(h, "out_h", full, 1, c.T, c);
            if (given(a[9])) apart(s.h, "out_h", {&s.o, &s.gate, &s.residual, &s.r});
        }
        const gma_status_t q = gma_norm_forward(&s, c.stream());
        if (q != GMA_OK) return raise_status(q, "gma_norm_forward");
        PyObject *rp = wrap(r), *hp = h.defined() ? wrap(h) : none();
        PyObject *both = rp && hp ? PyTuple_Pack(2, rp, hp) : nullptr;
        Py_XDECREF(rp);
        Py_XDECREF(hp);
        return both;
    });
}

// ..., dr, r, dh, residual (the forward call's tensor, a truth value or None), out
PyObject *block_norm_backward(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 12, [&]() -> PyObject * {
        Call c;
        std::vector<int64_t> full;
        gma_norm_grad_t g = {};
        g.fwd = norm_of(a, &c, &full);
        gma_norm_t &s = g.fwd;
        const at::Tensor &kept = tensor(a[8], "r");
        const at::ScalarType R = stream_type(kept, "r", c);
        s.r = rows(kept, "r", full, 1, R, c);
        bool residual = s.scale || R != c.T;
        if (given(a[10]) && THPVariable_Check(a[10])) {
            rows(a[10], "residual", full, 1, R, c);       // checked alone: its values are not used
            residual = true;
        } else if (given(a[10])) {
            const int truth = PyObject_IsTrue(a[10]);
            if (truth < 0) throw Raised{};
            residual = truth != 0;
        }
        if (!residual && R != c.T) type_error("without a residual r has o's dtype");
        if (residual) {
            s.residual = s.r;
            s.residual_dtype = code(R);
        }
        g.dr = maybe_rows(a[7], "dr", full, 1, R, c);
        g.dh = maybe_rows(a[9], "dh", full, 1, c.T, c);
        const at::IntArrayRef shape = tensor(a[0], "o").sizes();
        const at::Tensor d_o = out_or(a[11], "out", [&] { return c.empty(shape); });
        g.d_o = heads(d_o, "out", shape, c, &g.d_o_head);
        if (given(a[11])) apart(g.d_o, "out", {&s.o, &s.gate, &s.r, &g.dr, &g.dh});
        at::Tensor dgate, dres, dw[3];
        if (s.gate.ptr) {
            dgate = c.empty(full);
            g.dgate = rows(dgate, "gate", full, 1, c.T, c);
        }
        if (residual) {
            dres = at::empty(full, c.options.dtype(R));
            g.dresidual = rows(dres, "residual", full, 1, R, c);
        }
        const float *params[3] = {s.w_post, s.scale, s.w_pre};
        float **grads[3] = {&g.dw_post, &g.dscale, &g.dw_pre};
        for (int k = 0; k < 3; ++k)
            if (params[k]) {
                dw[k] = c.empty32({full[2]});
                *grads[k] = (float *)dw[k].data_ptr();
            }
        const Workspace ws(gma_norm_backward_workspace_size(&g), c);
        const gma_status_t q = gma_norm_backward(&g, ws.ptr(), ws.bytes, c.stream());
        if (q != GMA_OK) return raise_status(q, "gma_norm_backward");
        PyObject *d = PyDict_New();
        if (!d) return nullptr;
        set(d, "o", d_o); set(d, "gate", dgate); set(d, "residual", dres);
        set(d, "w_post", dw[0]); set(d, "scale", dw[1]); set(d, "w_pre", dw[2]);
        return d;
    });
}

#define METHOD(f) {#f, (PyCFunction)(void *)f, METH_FASTCALL, ""}
PyMethodDef methods[] = {METHOD(scan_checkpoints), METHOD(scan), METHOD(scan_step), METHOD(scan_backward), METHOD(conv), METHOD(conv_step),
                         METHOD(conv_backward), METHOD(block_norm), METHOD(block_norm_backward), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_block", "Binding of gma_block.h; see ssm and norm.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__block() { return PyModule_Create(&module); }
