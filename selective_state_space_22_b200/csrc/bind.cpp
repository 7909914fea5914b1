// bind.cpp -- the Python binding of the mixer-block operators (mixer.py): checks of the
// tensors, outputs and scratch, and the call of the C entry point, in one native step.
// A call on one token of a 1024-channel scan takes 4.8 us this way, launch included, 14.8 us
// from Python.
//
// The C entry points' addresses come from the library that the package has loaded
// (bind()), so this module neither links nor finds libssd itself.  A function returns
// its outputs, or the C status (an int) when that is not SSD_OK, which the package
// turns into its SSDError.  A refused tensor raises ValueError.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <stdexcept>
#include <string>

#include "../../include/ssd.h"

namespace {

using at::Tensor;
using Shape = c10::SmallVector<int64_t, 3>;

struct Refused : std::runtime_error {
    using std::runtime_error::runtime_error;
};
struct PythonError {};  // already set

// ---------------------------------------------------------------- C entry points
#define ENTRY_POINTS(X)                                                                                                \
    X(ssd_conv1d_varlen) X(ssd_conv1d_update) X(ssd_conv1d_bwd_workspace_size) X(ssd_conv1d_bwd)                       \
    X(ssd_selective_scan_chunk_states) X(ssd_selective_scan_workspace_size) X(ssd_selective_scan_varlen)               \
    X(ssd_selective_state_update) X(ssd_selective_scan_bwd_workspace_size) X(ssd_selective_scan_bwd)                   \
    X(ssd_residual_rmsnorm) X(ssd_rmsnorm_bwd_workspace_size) X(ssd_residual_rmsnorm_bwd) X(ssd_gated_rmsnorm)         \
    X(ssd_gated_rmsnorm_bwd)
struct {
#define MEMBER(name) decltype(&::name) name;
    ENTRY_POINTS(MEMBER)
#undef MEMBER
} entry;

// -------------------------------------------------------------------- arguments
bool none(PyObject *o) { return o == nullptr || o == Py_None; }

const Tensor &tensor(PyObject *o, const char *name) {
    if (none(o)) throw Refused(std::string(name) + " is required");
    if (!THPVariable_Check(o)) throw Refused(std::string(name) + " must be a tensor");
    return THPVariable_Unpack(o);
}
int integer(PyObject *o) {
    const long v = PyLong_AsLong(o);
    if (v == -1 && PyErr_Occurred()) throw PythonError();
    if (v < INT_MIN || v > INT_MAX) throw Refused("an integer argument does not fit 32 bits");
    return (int)v;
}
int truth(PyObject *o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw PythonError();
    return v;
}
float real(PyObject *o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw PythonError();
    return (float)v;
}
int size32(int64_t n, const char *name) {
    if (n > INT_MAX) throw Refused(std::string(name) + " is too large");
    return (int)n;
}

std::string text(c10::IntArrayRef s) {
    std::string t = "(";
    for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
    return t + ")";
}
const char *type_name(at::ScalarType t) {
    return t == at::kFloat ? "torch.float32" : t == at::kBFloat16 ? "torch.bfloat16" : t == at::kInt ? "torch.int32" : t == at::kBool ? "torch.bool" : "another dtype";
}

// The device a call runs on, and what its tensors must be.
struct Call {
    c10::Device dev;
    c10::cuda::CUDAGuard guard;
    explicit Call(const Tensor &t, const char *name) : dev(on_gpu(t, name)), guard(dev) {}
    static c10::Device on_gpu(const Tensor &t, const char *name) {
        if (!t.is_cuda()) throw Refused(std::string(name) + " must be a CUDA tensor");
        return t.device();
    }
    void *stream() const { return c10::cuda::getCurrentCUDAStream(dev.index()).stream(); }

    void check(const Tensor &t, const char *name, at::ScalarType type, c10::IntArrayRef shape) const {
        if (!t.is_cuda()) throw Refused(std::string(name) + " must be a CUDA tensor");
        if (t.device() != dev) throw Refused(std::string(name) + " is on " + t.device().str() + ", expected " + dev.str());
        if (t.scalar_type() != type) throw Refused(std::string(name) + " must be " + type_name(type) + ", got " + type_name(t.scalar_type()));
        if (t.sizes() != shape) throw Refused(std::string(name) + " has shape " + text(t.sizes()) + ", expected " + text(shape));
    }
    // Data pointer of a contiguous tensor.
    void *whole(const Tensor &t, const char *name, at::ScalarType type, c10::IntArrayRef shape) const {
        check(t, name, type, shape);
        if (!t.is_contiguous()) throw Refused(std::string(name) + " must be contiguous");
        return t.data_ptr();
    }
    void *whole(PyObject *o, const char *name, at::ScalarType type, c10::IntArrayRef shape) const { return whole(tensor(o, name), name, type, shape); }
    void *maybe(PyObject *o, const char *name, at::ScalarType type, c10::IntArrayRef shape) const { return none(o) ? nullptr : whole(o, name, type, shape); }
    // Data pointer and row stride of rows whose inner dimensions are contiguous.
    void *rows(PyObject *o, const char *name, at::ScalarType type, c10::IntArrayRef shape, long long &ld) const {
        const Tensor &t = tensor(o, name);
        check(t, name, type, shape);
        int64_t width = 1;
        bool inner = true;
        for (size_t i = shape.size() - 1; i > 0; --i) {
            inner &= shape[i] == 1 || t.stride(i) == width;
            width *= shape[i];
        }
        ld = std::max<int64_t>(t.stride(0), width);
        if (!inner || (shape[0] > 1 && t.stride(0) < width))
            throw Refused(std::string(name) + ": the dimensions after the first must be contiguous and rows must not overlap");
        return t.data_ptr();
    }
    Tensor fresh(at::ScalarType type, c10::IntArrayRef shape) const { return at::empty(shape, at::TensorOptions().dtype(type).device(dev)); }
    Tensor scratch(size_t bytes) const { return bytes ? fresh(at::kByte, {(int64_t)bytes}) : Tensor(); }
    // An output: the given tensor checked, or a new one.
    Tensor given_or_new(PyObject *o, const char *name, at::ScalarType type, c10::IntArrayRef shape) const {
        if (none(o)) return fresh(type, shape);
        const Tensor &t = tensor(o, name);
        whole(t, name, type, shape);
        return t;
    }
};
void *ptr(const Tensor &t) { return t.defined() && t.numel() ? t.data_ptr() : nullptr; }
// Whether two contiguous tensors have memory in common.
bool overlap(const Tensor &a, const Tensor &b) {
    const char *p = static_cast<const char *>(ptr(a)), *q = static_cast<const char *>(ptr(b));
    return p && q && p < q + b.nbytes() && q < p + a.nbytes();
}

int io_of(const Tensor &t, const char *name) {
    if (t.scalar_type() == at::kFloat) return SSD_F32;
    if (t.scalar_type() == at::kBFloat16) return SSD_BF16;
    throw Refused(std::string(name) + " must be bfloat16 or float32");
}
void need_dim(const Tensor &t, const char *name, int n) {
    if (t.dim() != n) throw Refused(std::string(name) + " must have " + std::to_string(n) + " dimensions, got " + std::to_string(t.dim()));
}
size_t sized(size_t n, const char *what) {
    if (n == SSD_WORKSPACE_INVALID) throw Refused(std::string("invalid sizes for ") + what);
    return n;
}

// A cache of no slots is a cache, in which no sequence has a state: it goes in as this
// address, which nothing follows (a slot below zero is none, any other out of range).
alignas(16) char no_slots[16];
void *cache(void *p, int nslots) { return nslots ? p : no_slots; }

PyObject *status(int s) { return PyLong_FromLong(s); }
PyObject *wrap(Tensor t) { return THPVariable_Wrap(std::move(t)); }

// A dict of outputs, the caller's or a new one.
struct Outputs {
    PyObject *d;
    explicit Outputs(PyObject *given) {
        if (none(given)) {
            d = PyDict_New();
        } else {
            if (!PyDict_Check(given)) throw Refused("out must be a dict");
            Py_INCREF(d = given);
        }
    }
    ~Outputs() { Py_XDECREF(d); }
    PyObject *release() {
        PyObject *r = d;
        d = nullptr;
        return r;
    }
    void set(const char *name, PyObject *o) {  // takes o
        const int r = o ? PyDict_SetItemString(d, name, o) : -1;
        Py_XDECREF(o);
        if (r) throw PythonError();
    }
    Tensor fresh(const Call &c, const char *name, at::ScalarType type, c10::IntArrayRef shape) {
        Tensor t = c.fresh(type, shape);
        set(name, wrap(t));
        return t;
    }
    Tensor tensor_of(const Call &c, const char *name, at::ScalarType type, c10::IntArrayRef shape) {
        PyObject *o = PyDict_GetItemString(d, name);
        return none(o) ? fresh(c, name, type, shape) : c.given_or_new(o, name, type, shape);
    }
    void absent(const char *name) {  // also over what an earlier call left there
        Py_INCREF(Py_None);
        set(name, Py_None);
    }
};

struct Sequences {
    const int *cu;
    int n;
    Sequences(const Call &c, PyObject *o) {
        if (none(o) || tensor(o, "cu_seqlens").dim() != 1 || tensor(o, "cu_seqlens").size(0) < 1)
            throw Refused("cu_seqlens must be a vector of the sequences' bounds");
        n = size32(tensor(o, "cu_seqlens").size(0) - 1, "cu_seqlens");
        cu = static_cast<const int *>(c.whole(o, "cu_seqlens", at::kInt, {n + 1}));
    }
};

// ------------------------------------------------------------------ convolution
struct ConvIn {
    const Tensor &xbc, &weight;
    Call c;
    int io, n, ct, cx, cb, width;
    long long ld;
    void *x;
    const float *w, *b;
    // a: xbc, weight, bias; x_channels may be None
    ConvIn(PyObject *const *a, PyObject *x_channels, int bc_channels)
        : xbc(tensor(a[0], "xbc")), weight(tensor(a[1], "weight")), c(xbc, "xbc") {
        Call::on_gpu(weight, "weight");
        need_dim(xbc, "xbc", 2);
        need_dim(weight, "weight", 2);
        io = io_of(xbc, "xbc");
        n = size32(xbc.size(0), "xbc"), ct = size32(xbc.size(1), "xbc"), cb = bc_channels, width = size32(weight.size(1), "weight");
        cx = none(x_channels) ? ct - 2 * cb : integer(x_channels);
        if ((int64_t)cx + 2LL * cb != ct) throw Refused("xbc width must be x_channels + 2 bc_channels");
        x = c.rows(a[0], "xbc", xbc.scalar_type(), {n, ct}, ld);
        w = static_cast<const float *>(c.whole(weight, "weight", at::kFloat, {ct, width}));
        b = static_cast<const float *>(c.maybe(a[2], "bias", at::kFloat, {ct}));
    }
    void *state(const Tensor &t, int nslots) const {  // one tap has none
        void *p = c.whole(t, "conv_state", xbc.scalar_type(), {nslots, ct, width - 1});
        return width > 1 ? cache(p, nslots) : nullptr;
    }
    void outputs(PyObject *given, Tensor (&t)[3]) const {
        const int widths[3] = {cx, cb, cb};
        const char *const names[3] = {"x", "B", "C"};
        if (none(given)) {
            for (int i = 0; i < 3; ++i) t[i] = c.fresh(xbc.scalar_type(), {n, widths[i]});
            return;
        }
        if (!PySequence_Check(given) || PySequence_Size(given) != 3) throw Refused("out must hold the three outputs x, B and C");
        for (int i = 0; i < 3; ++i) {
            PyObject *o = PySequence_GetItem(given, i);
            if (!o) throw PythonError();
            const Tensor held = THPVariable_Check(o) ? THPVariable_Unpack(o) : Tensor();
            Py_DECREF(o);
            if (!held.defined()) throw Refused("out must hold three tensors");
            c.whole(held, names[i], xbc.scalar_type(), {n, widths[i]});
            t[i] = held;
        }
    }
    static PyObject *result(PyObject *given, Tensor (&t)[3]) {
        if (!none(given)) {
            Py_INCREF(given);
            return given;
        }
        PyObject *r = PyTuple_New(3);
        for (int i = 0; r && i < 3; ++i) PyTuple_SET_ITEM(r, i, wrap(std::move(t[i])));
        return r;
    }
};

// xbc, weight, bias, cu_seqlens, x_channels, bc_channels, silu, conv_state, slots, has_init, out
PyObject *conv1d_varlen(PyObject *const *a) {
    const ConvIn in(a, a[4], integer(a[5]));
    const Sequences seq(in.c, a[3]);
    void *state = nullptr;
    int nslots = 0;
    if (!none(a[7])) {
        need_dim(tensor(a[7], "conv_state"), "conv_state", 3);
        nslots = size32(tensor(a[7], "conv_state").size(0), "conv_state");
        state = in.state(tensor(a[7], "conv_state"), nslots);
    }
    const int *slots = static_cast<const int *>(in.c.maybe(a[8], "slots", at::kInt, {seq.n}));
    const auto *has = static_cast<const unsigned char *>(in.c.maybe(a[9], "has_init", at::kBool, {seq.n}));
    Tensor t[3];
    in.outputs(a[10], t);
    const int s = entry.ssd_conv1d_varlen(in.x, in.ld, in.w, in.b, seq.cu, state, slots, has, ptr(t[0]), ptr(t[1]), ptr(t[2]),
                                          (ssd_dtype)in.io, in.n, seq.n, nslots, in.cx, in.cb, in.width, truth(a[6]), in.c.stream());
    return s ? status(s) : ConvIn::result(a[10], t);
}

// xbc, weight, bias, conv_state, x_channels, bc_channels, silu, slots, out
PyObject *conv1d_update(PyObject *const *a) {
    const ConvIn in(a, a[4], integer(a[5]));
    const Tensor &st = tensor(a[3], "conv_state");
    need_dim(st, "conv_state", 3);
    const int nslots = size32(st.size(0), "conv_state");
    void *state = in.state(st, nslots);
    const int *slots = static_cast<const int *>(in.c.maybe(a[7], "slots", at::kInt, {in.n}));
    Tensor t[3];
    in.outputs(a[8], t);
    const int s = entry.ssd_conv1d_update(state, slots, in.x, in.ld, in.w, in.b, ptr(t[0]), ptr(t[1]), ptr(t[2]), (ssd_dtype)in.io,
                                          in.n, nslots, in.cx, in.cb, in.width, truth(a[6]), in.c.stream());
    return s ? status(s) : ConvIn::result(a[8], t);
}

// xbc, weight, bias, cu_seqlens, dx, dB, dC, silu, out
PyObject *conv1d_bwd(PyObject *const *a) {
    const Tensor &dx = tensor(a[4], "dx");
    Call::on_gpu(tensor(a[0], "xbc"), "xbc");
    Call::on_gpu(dx, "dx");
    need_dim(dx, "dx", 2);
    int cb = 0;
    if (!none(a[5])) {
        need_dim(tensor(a[5], "dB"), "dB", 2);
        cb = size32(tensor(a[5], "dB").size(1), "dB");
    }
    PyObject *cx = PyLong_FromLongLong(dx.size(1));
    if (!cx) throw PythonError();
    struct Drop {
        PyObject *o;
        ~Drop() { Py_DECREF(o); }
    } drop{cx};
    const ConvIn in(a, cx, cb);
    const Sequences seq(in.c, a[3]);
    const auto type = in.xbc.scalar_type();
    const void *gx = in.c.whole(dx, "dx", type, {in.n, in.cx}), *gb = nullptr, *gc = nullptr;
    if (cb) gb = in.c.whole(a[5], "dB", type, {in.n, cb}), gc = in.c.whole(a[6], "dC", type, {in.n, cb});
    Outputs out(a[8]);
    const Tensor dxbc = out.tensor_of(in.c, "dxbc", type, {in.n, in.ct}), dw = out.tensor_of(in.c, "dweight", at::kFloat, {in.ct, in.width});
    const Tensor db = none(a[2]) ? Tensor() : out.tensor_of(in.c, "dbias", at::kFloat, {in.ct});
    if (none(a[2])) out.absent("dbias");
    const size_t bytes = sized(entry.ssd_conv1d_bwd_workspace_size(in.n, in.ct, in.width), "the conv's gradient");
    const Tensor ws = in.c.scratch(bytes);
    const int s = entry.ssd_conv1d_bwd(in.x, in.ld, in.w, in.b, seq.cu, gx, gb, gc, ptr(dxbc), static_cast<float *>(ptr(dw)),
                                       static_cast<float *>(ptr(db)), (ssd_dtype)in.io, in.n, seq.n, in.cx, in.cb, in.width, truth(a[7]),
                                       ptr(ws), bytes, in.c.stream());
    return s ? status(s) : out.release();
}

// --------------------------------------------------------------- selective scan
struct SelIn {
    const Tensor &x, &B;
    Call c;
    at::ScalarType type;
    int n, d, G, N;
    ssd_sel_args args{};
    // a: x, dt, A, B, C, D, z, dt_bias, softplus
    explicit SelIn(PyObject *const *a) : x(tensor(a[0], "x")), B(tensor(a[3], "B")), c(x, "x"), type(x.scalar_type()) {
        Call::on_gpu(B, "B");
        need_dim(x, "x", 2);
        need_dim(B, "B", 3);
        n = size32(x.size(0), "x"), d = size32(x.size(1), "x"), G = size32(B.size(1), "B"), N = size32(B.size(2), "B");
        args.io_dtype = (ssd_dtype)io_of(x, "x");
        const Shape rows{n, d}, states{n, G, N};
        args.x = c.rows(a[0], "x", type, rows, args.x_stride);
        args.dt = c.rows(a[1], "dt", type, rows, args.dt_stride);
        args.A = static_cast<const float *>(c.whole(a[2], "A", at::kFloat, {d, N}));
        args.B = c.rows(a[3], "B", type, states, args.b_stride);
        args.C = c.rows(a[4], "C", type, states, args.c_stride);
        args.D = static_cast<const float *>(c.maybe(a[5], "D", at::kFloat, {d}));
        if (!none(a[6])) args.z = c.rows(a[6], "z", type, rows, args.z_stride);
        args.dt_bias = static_cast<const float *>(c.maybe(a[7], "dt_bias", at::kFloat, {d}));
        args.softplus = truth(a[8]), args.channels = d, args.ngroups = G, args.dstate = N;
    }
    float *states(PyObject *o, int &nslots) const {
        const Tensor &t = tensor(o, "state");
        need_dim(t, "state", 3);
        nslots = size32(t.size(0), "state");
        return static_cast<float *>(cache(c.whole(t, "state", at::kFloat, {nslots, d, N}), nslots));
    }
};

// the nine of SelIn, then cu_seqlens, state, slots, has_init, y, return_chunk_states
PyObject *selective_scan_varlen(PyObject *const *a) {
    const SelIn in(a);
    const Sequences seq(in.c, a[9]);
    int nslots = 0;
    float *state = none(a[10]) ? nullptr : in.states(a[10], nslots);
    const int *slots = none(a[10]) ? nullptr : static_cast<const int *>(in.c.maybe(a[11], "slots", at::kInt, {seq.n}));
    const auto *has = static_cast<const unsigned char *>(in.c.maybe(a[12], "has_init", at::kBool, {seq.n}));
    Tensor y = in.c.given_or_new(a[13], "y", in.type, {in.n, in.d}), kept;
    if (truth(a[14]))
        kept = in.c.fresh(at::kFloat, {(int64_t)sized(entry.ssd_selective_scan_chunk_states(in.n, seq.n), "the scan"), in.N, in.d});
    const size_t bytes = sized(entry.ssd_selective_scan_workspace_size(in.n, seq.n, in.d, in.N), "the scan");
    const Tensor ws = in.c.scratch(bytes);
    const int s = entry.ssd_selective_scan_varlen(&in.args, seq.cu, state, slots, has, static_cast<float *>(ptr(kept)), ptr(y), in.n, seq.n,
                                                  nslots, ptr(ws), bytes, in.c.stream());
    if (s) return status(s);
    PyObject *r = PyTuple_New(2);
    if (!r) throw PythonError();
    PyTuple_SET_ITEM(r, 0, wrap(std::move(y)));
    if (!kept.defined()) Py_INCREF(Py_None);
    PyTuple_SET_ITEM(r, 1, kept.defined() ? wrap(std::move(kept)) : Py_None);
    return r;
}

// the nine of SelIn, then state, slots, y
PyObject *selective_state_update(PyObject *const *a) {
    const SelIn in(a);
    int nslots = 0;
    float *state = in.states(a[9], nslots);
    const int *slots = static_cast<const int *>(in.c.maybe(a[10], "slots", at::kInt, {in.n}));
    Tensor y = in.c.given_or_new(a[11], "y", in.type, {in.n, in.d});
    const int s = entry.ssd_selective_state_update(&in.args, state, slots, ptr(y), in.n, nslots, in.c.stream());
    return s ? status(s) : wrap(std::move(y));
}

// the nine of SelIn, then cu_seqlens, dy, chunk_states, out
PyObject *selective_scan_bwd(PyObject *const *a) {
    const SelIn in(a);
    const Sequences seq(in.c, a[9]);
    const void *dy = in.c.whole(a[10], "dy", in.type, {in.n, in.d});
    const int64_t chunks = sized(entry.ssd_selective_scan_chunk_states(in.n, seq.n), "the scan");
    const auto *kept = static_cast<const float *>(in.c.whole(a[11], "chunk_states", at::kFloat, {chunks, in.N, in.d}));
    Outputs out(a[12]);
    const Shape rows{in.n, in.d}, states{in.n, in.G, in.N};
    const Tensor dx = out.tensor_of(in.c, "dx", in.type, rows), ddt = out.tensor_of(in.c, "ddt", in.type, rows);
    const Tensor dz = none(a[6]) ? Tensor() : out.tensor_of(in.c, "dz", in.type, rows);
    const Tensor dB = out.tensor_of(in.c, "dB", in.type, states), dC = out.tensor_of(in.c, "dC", in.type, states);
    const Tensor dA = out.tensor_of(in.c, "dA", at::kFloat, {in.d, in.N});
    const Tensor dD = none(a[5]) ? Tensor() : out.tensor_of(in.c, "dD", at::kFloat, {in.d});
    const Tensor db = none(a[7]) ? Tensor() : out.tensor_of(in.c, "ddt_bias", at::kFloat, {in.d});
    if (none(a[6])) out.absent("dz");
    if (none(a[5])) out.absent("dD");
    if (none(a[7])) out.absent("ddt_bias");
    const size_t bytes = sized(entry.ssd_selective_scan_bwd_workspace_size(in.n, seq.n, in.d, in.G, in.N), "the scan's gradient");
    const Tensor ws = in.c.scratch(bytes);
    const int s = entry.ssd_selective_scan_bwd(&in.args, seq.cu, dy, kept, ptr(dx), ptr(ddt), ptr(dz), ptr(dB), ptr(dC),
                                               static_cast<float *>(ptr(dA)), static_cast<float *>(ptr(dD)), static_cast<float *>(ptr(db)),
                                               in.n, seq.n, ptr(ws), bytes, in.c.stream());
    return s ? status(s) : out.release();
}

// ------------------------------------------------------------------------ norms
// x, weight, residual, scale, eps, out, residual_out
PyObject *residual_rmsnorm(PyObject *const *a) {
    const Tensor &x = tensor(a[0], "x");
    const Call c(x, "x");
    need_dim(x, "x", 2);
    const Shape shape{x.size(0), x.size(1)};
    const int n = size32(shape[0], "x"), d = size32(shape[1], "x"), io = io_of(x, "x");
    const auto type = x.scalar_type(), rtype = none(a[2]) ? type : tensor(a[2], "residual").scalar_type();
    if (rtype != type && rtype != at::kFloat) throw Refused("residual must have x's dtype or float32");
    long long ldx, ldr = 0;
    const void *xp = c.rows(a[0], "x", type, shape, ldx), *rp = none(a[2]) ? nullptr : c.rows(a[2], "residual", rtype, shape, ldr);
    const auto *w = static_cast<const float *>(c.whole(a[1], "weight", at::kFloat, {d})), *sc = static_cast<const float *>(c.maybe(a[3], "scale", at::kFloat, {d}));
    Tensor out = c.given_or_new(a[5], "out", type, shape), res = c.given_or_new(a[6], "residual_out", rtype, shape);
    const int s = entry.ssd_residual_rmsnorm(xp, ldx, rp, ldr, sc, w, ptr(out), ptr(res), (ssd_dtype)io, rtype == at::kFloat ? SSD_F32 : SSD_BF16,
                                             n, d, real(a[4]), c.stream());
    if (s) return status(s);
    PyObject *r = PyTuple_New(2);
    if (!r) throw PythonError();
    PyTuple_SET_ITEM(r, 0, wrap(std::move(out)));
    PyTuple_SET_ITEM(r, 1, wrap(std::move(res)));
    return r;
}

// residual, weight, dout, dresidual, x, scale, eps, out
PyObject *residual_rmsnorm_bwd(PyObject *const *a) {
    const Tensor &r = tensor(a[0], "residual"), &dout = tensor(a[2], "dout");
    const Call c(r, "residual");
    Call::on_gpu(dout, "dout");
    need_dim(r, "residual", 2);
    const Shape shape{r.size(0), r.size(1)};
    const int n = size32(shape[0], "residual"), d = size32(shape[1], "residual"), io = io_of(dout, "dout");
    const auto type = dout.scalar_type(), rtype = r.scalar_type();
    if (rtype != type && rtype != at::kFloat) throw Refused("residual must have dout's dtype or float32");
    const bool scaled = !none(a[5]), apart = scaled || rtype != type;
    if (scaled && none(a[4])) throw Refused("x is required with scale");
    long long ldr, ldx = 0;
    const void *rp = c.rows(a[0], "residual", rtype, shape, ldr), *xp = scaled ? c.rows(a[4], "x", type, shape, ldx) : nullptr;
    const auto *w = static_cast<const float *>(c.whole(a[1], "weight", at::kFloat, {d})), *sc = static_cast<const float *>(c.maybe(a[5], "scale", at::kFloat, {d}));
    const void *up = c.whole(dout, "dout", type, shape), *ur = c.maybe(a[3], "dresidual", rtype, shape);
    Outputs out(a[7]);
    const Tensor gr = out.tensor_of(c, "dresidual", rtype, shape);
    PyObject *given = PyDict_GetItemString(out.d, "dx");  // a tensor of the caller's is filled in any case
    if (apart && !none(given) && given == PyDict_GetItemString(out.d, "dresidual")) {
        out.fresh(c, "dx", type, shape);  // one tensor for both, as a call that does not set them apart leaves it
        given = PyDict_GetItemString(out.d, "dx");
    }
    const Tensor gx = apart || !none(given) ? out.tensor_of(c, "dx", type, shape) : Tensor();
    if (gx.defined() && overlap(gx, gr) && (apart || ptr(gx) != ptr(gr)))
        throw Refused("out: dx and dresidual share memory and are not the same values at the same place");
    if (!gx.defined()) out.set("dx", wrap(gr));
    const Tensor gw = out.tensor_of(c, "dweight", at::kFloat, {d}), gs = scaled ? out.tensor_of(c, "dscale", at::kFloat, {d}) : Tensor();
    if (!scaled) out.absent("dscale");
    const size_t bytes = sized(entry.ssd_rmsnorm_bwd_workspace_size(n, d), "the norm's gradient");
    const Tensor ws = c.scratch(bytes);
    const int s = entry.ssd_residual_rmsnorm_bwd(rp, ldr, w, up, ur, xp, ldx, sc, ptr(gx), ptr(gr), static_cast<float *>(ptr(gw)),
                                                 static_cast<float *>(ptr(gs)), (ssd_dtype)io, rtype == at::kFloat ? SSD_F32 : SSD_BF16, n, d,
                                                 real(a[6]), ptr(ws), bytes, c.stream());
    return s ? status(s) : out.release();
}

struct GatedIn {
    const Tensor &y;
    Call c;
    Shape shape;
    at::ScalarType type;
    int n, d, io;
    long long ldy, ldz = 0;
    const void *yp, *zp = nullptr;
    const float *w, *sc;
    GatedIn(PyObject *py, PyObject *pz, PyObject *weight, PyObject *scale) : y(tensor(py, "y")), c(y, "y"), type(y.scalar_type()) {
        need_dim(y, "y", 2);
        shape = {y.size(0), y.size(1)};
        n = size32(shape[0], "y"), d = size32(shape[1], "y"), io = io_of(y, "y");
        yp = c.rows(py, "y", type, shape, ldy);
        if (!none(pz)) zp = c.rows(pz, "z", type, shape, ldz);
        w = static_cast<const float *>(c.whole(weight, "weight", at::kFloat, {d}));
        sc = static_cast<const float *>(c.maybe(scale, "scale", at::kFloat, {d}));
    }
};

// y, z, weight, residual, scale, ngroups, norm_before_gate, eps, out
PyObject *gated_rmsnorm(PyObject *const *a) {
    const GatedIn in(a[0], a[1], a[2], a[4]);
    long long ldr = 0;
    const void *rp = none(a[3]) ? nullptr : in.c.rows(a[3], "residual", in.type, in.shape, ldr);
    Tensor out = in.c.given_or_new(a[8], "out", in.type, in.shape);
    const int s = entry.ssd_gated_rmsnorm(in.yp, in.ldy, in.zp, in.ldz, rp, ldr, in.sc, in.w, ptr(out), (ssd_dtype)in.io, in.n, in.d,
                                          integer(a[5]), truth(a[6]), real(a[7]), in.c.stream());
    return s ? status(s) : wrap(std::move(out));
}

// y, z, weight, dout, scale, ngroups, norm_before_gate, eps, out
PyObject *gated_rmsnorm_bwd(PyObject *const *a) {
    const GatedIn in(a[0], a[1], a[2], a[4]);
    const void *up = in.c.whole(a[3], "dout", in.type, in.shape);
    Outputs out(a[8]);
    const Tensor gy = out.tensor_of(in.c, "dy", in.type, in.shape), gz = in.zp || !none(a[1]) ? out.tensor_of(in.c, "dz", in.type, in.shape) : Tensor();
    const Tensor gw = out.tensor_of(in.c, "dweight", at::kFloat, {in.d}), gs = none(a[4]) ? Tensor() : out.tensor_of(in.c, "dscale", at::kFloat, {in.d});
    if (none(a[1])) out.absent("dz");
    if (none(a[4])) out.absent("dscale");
    const size_t bytes = sized(entry.ssd_rmsnorm_bwd_workspace_size(in.n, in.d), "the norm's gradient");
    const Tensor ws = in.c.scratch(bytes);
    const int s = entry.ssd_gated_rmsnorm_bwd(in.yp, in.ldy, in.zp, in.ldz, in.w, up, in.sc, ptr(gy), ptr(gz), static_cast<float *>(ptr(gw)),
                                              static_cast<float *>(ptr(gs)), (ssd_dtype)in.io, in.n, in.d, integer(a[5]), truth(a[6]), real(a[7]),
                                              ptr(ws), bytes, in.c.stream());
    return s ? status(s) : out.release();
}

// ----------------------------------------------------------------------- module
void set_error(const char *module, const char *type, const char *what) {
    PyObject *m = PyImport_ImportModule(module), *t = m ? PyObject_GetAttrString(m, type) : nullptr;
    if (t) PyErr_SetString(t, what);
    Py_XDECREF(t);
    Py_XDECREF(m);
}
template <PyObject *(*F)(PyObject *const *), int N> PyObject *guarded(PyObject *, PyObject *const *args, Py_ssize_t n) {
    if (n != N) {
        PyErr_Format(PyExc_TypeError, "%d arguments expected, got %zd", N, n);
        return nullptr;
    }
    try {
        return F(args);
    } catch (const Refused &e) {
        PyErr_SetString(PyExc_ValueError, e.what());
    } catch (const PythonError &) {
    } catch (const c10::OutOfMemoryError &e) {
        set_error("torch", "OutOfMemoryError", e.what_without_backtrace());
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

// bind({name: address}): the loaded library's entry points.
PyObject *bind(PyObject *, PyObject *addresses) {
#define TAKE(name)                                                                              \
    {                                                                                           \
        PyObject *o = PyDict_GetItemString(addresses, #name);                                   \
        void *p = o ? PyLong_AsVoidPtr(o) : nullptr;                                            \
        if (!p) {                                                                               \
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, "no address for " #name); \
            return nullptr;                                                                     \
        }                                                                                       \
        entry.name = reinterpret_cast<decltype(entry.name)>(p);                                 \
    }
    ENTRY_POINTS(TAKE)
#undef TAKE
    Py_RETURN_NONE;
}
PyObject *names(PyObject *, PyObject *) {
    PyObject *l = PyList_New(0);
#define NAME(name)                                     \
    if (l) {                                           \
        PyObject *s = PyUnicode_FromString(#name);     \
        if (!s || PyList_Append(l, s)) Py_CLEAR(l);    \
        Py_XDECREF(s);                                 \
    }
    ENTRY_POINTS(NAME)
#undef NAME
    return l;
}

#define CALL(f, n) \
    { #f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&guarded<f, n>)), METH_FASTCALL, nullptr }
PyMethodDef methods[] = {CALL(conv1d_varlen, 11),
                         CALL(conv1d_update, 9),
                         CALL(conv1d_bwd, 9),
                         CALL(selective_scan_varlen, 15),
                         CALL(selective_state_update, 12),
                         CALL(selective_scan_bwd, 13),
                         CALL(residual_rmsnorm, 7),
                         CALL(residual_rmsnorm_bwd, 8),
                         CALL(gated_rmsnorm, 9),
                         CALL(gated_rmsnorm_bwd, 9),
                         {"bind", bind, METH_O, nullptr},
                         {"names", names, METH_NOARGS, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_bind", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__bind() { return PyModule_Create(&module); }
