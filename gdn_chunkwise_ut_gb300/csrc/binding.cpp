// binding.cpp -- the Python binding of the serving operators (include/gdn_layer.h): argument checks,
// output allocation, and the calls into libkkt.so on torch's current stream.  A decode step makes
// these calls for every layer and token with kernels of a few microseconds, so the marshalling is
// native: a call takes 3.5 to 8 us of the host's time, and took 16 to 68 through ctypes.
//
// A function returns its outputs, or as an int the kkt_status of a refused call, or, negated, what a
// checked call found in the device's status word; what the arguments themselves show to be wrong raises
// ValueError.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <cstdlib>
#include <cstring>
#include <string>
#include <vector>

#include "gdn_layer.h"

namespace {

using at::ScalarType;
using at::Tensor;

struct Refusal {
    std::string what;
};

[[noreturn]] void refuse(const std::string &what) { throw Refusal{what}; }

std::string text(at::IntArrayRef s) {
    std::string out = "(";
    for (size_t i = 0; i < s.size(); ++i) out += (i ? ", " : "") + std::to_string(s[i]);
    return out + (s.size() == 1 ? ",)" : ")");
}

const Tensor &tensor(PyObject *o, const char *name) {
    if (!THPVariable_Check(o)) refuse(std::string(name) + " must be a CUDA tensor");
    return THPVariable_Unpack(o);
}

// A tensor or an undefined one for None.
Tensor optional(PyObject *o, const char *name) { return o == Py_None ? Tensor() : tensor(o, name); }

void check(const Tensor &t, const char *name, ScalarType dtype, at::IntArrayRef shape, c10::Device dev) {
    if (t.is_cuda() && t.device() == dev && t.scalar_type() == dtype && t.sizes() == shape && t.is_contiguous()) return;
    const std::string n(name);
    if (!t.is_cuda()) refuse(n + " must be a CUDA tensor");
    if (t.device() != dev) refuse(n + " is on another device");
    if (t.scalar_type() != dtype)
        refuse(n + " must be of type " + c10::toString(dtype) + ", got " + c10::toString(t.scalar_type()));
    if (t.sizes() != shape) refuse(n + " must have shape " + text(shape) + ", got " + text(t.sizes()));
    refuse(n + " must be contiguous");
}

// Checks a tensor that may also be a slice of a larger one: its last dimensions, `packed` values together,
// lie behind one another, and those before them are one axis of equal steps.  Returns the step.
int64_t check_sliced(const Tensor &t, const char *name, ScalarType dtype, at::IntArrayRef shape, int64_t packed,
                     c10::Device dev) {
    if (t.is_cuda() && t.device() == dev && t.scalar_type() == dtype && t.sizes() == shape && !t.is_contiguous()) {
        int64_t inner = 1, step = 0, next = 0;  // next: the stride of the outer axis's next dimension
        bool ok = true;
        for (int64_t d = t.dim() - 1; d >= 0 && ok; --d) {
            const int64_t size = t.size(d), stride = t.stride(d);
            if (inner < packed) {
                ok = size == 1 || stride == inner;
                inner *= size;
            } else if (size > 1) {
                if (step == 0) step = next = stride;
                ok = stride == next && step >= packed;
                next *= size;
            }
        }
        if (ok && inner == packed && step > 0) return step;
        refuse(std::string(name) + " must be contiguous, or a slice whose tokens are equal steps apart");
    }
    check(t, name, dtype, shape, dev);
    return packed;
}

int io_type(const Tensor &t, const char *name) {
    if (t.scalar_type() == at::kBFloat16) return KKT_IO_BF16;
    if (t.scalar_type() == at::kFloat) return KKT_IO_F32;
    refuse(std::string(name) + " must be torch.bfloat16 or torch.float32, got " + c10::toString(t.scalar_type()));
}

void need_dim(const Tensor &t, const char *what, int64_t dim) {
    if (t.dim() != dim) refuse(std::string("expected ") + what);
}

c10::Device device_of(const Tensor &t, const char *name) {
    if (!t.is_cuda()) refuse(std::string(name) + " must be a CUDA tensor");
    return t.device();
}

template <typename T>
T *ptr(const Tensor &t) { return t.defined() ? static_cast<T *>(t.data_ptr()) : nullptr; }
void *raw(const Tensor &t) { return t.defined() ? t.data_ptr() : nullptr; }

CUstream_st *stream_on(c10::Device dev) { return c10::cuda::getCurrentCUDAStream(dev.index()).stream(); }

Tensor empty(at::IntArrayRef shape, ScalarType dtype, c10::Device dev) {
    return at::detail::empty_cuda(shape, dtype, dev, std::nullopt);
}

int small(int64_t v, const char *name) {
    if (v < INT32_MIN || v > INT32_MAX) refuse(std::string(name) + " is too large");
    return static_cast<int>(v);
}

int integer(PyObject *o, const char *name) {
    const long v = PyLong_AsLong(o);
    if (v == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        refuse(std::string(name) + " must be an integer");
    }
    return small(v, name);
}

double number(PyObject *o, const char *name) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) {
        PyErr_Clear();
        refuse(std::string(name) + " must be a number");
    }
    return v;
}

// Number of sequences, from cu_seqlens where it is given (then the batch dimension is 1).
int sequences(const Tensor &cu, int64_t batch, c10::Device dev) {
    if (!cu.defined()) return small(batch, "the batch dimension");
    if (batch != 1) refuse("with cu_seqlens the batch dimension must be 1");
    if (cu.scalar_type() != at::kInt || !cu.is_cuda() || cu.device() != dev || cu.dim() != 1 || !cu.is_contiguous())
        refuse("cu_seqlens must be a contiguous 1-D int32 CUDA tensor");
    if (cu.size(0) < 2) refuse("cu_seqlens must hold at least two offsets");
    return small(cu.size(0) - 1, "cu_seqlens");
}

// Runs f, with C++ exceptions turned into Python's.
template <typename F>
PyObject *guarded(F f) {
    HANDLE_TH_ERRORS
    try {
        return f();
    } catch (python_error &e) {  // Python's own error, set where it was met
        e.persist();
        throw;
    } catch (const Refusal &r) {
        PyErr_SetString(PyExc_ValueError, r.what.c_str());
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

// The end of a call: its status as an int where there is something to say, else nullptr.  In the checked
// mode (`check` true, or None and KKT_CHECK=1 in the environment) the stream is waited for and the
// device's status word read and cleared.
PyObject *trouble(int rc, PyObject *check, CUstream_st *stream) {
    if (rc != KKT_OK) return PyLong_FromLong(rc);
    bool checked = check == Py_True;
    if (check == Py_None) {
        const char *env = std::getenv("KKT_CHECK");
        checked = env && std::strcmp(env, "1") == 0;
    } else if (!checked) {
        const int truth = PyObject_IsTrue(check);
        if (truth < 0) throw python_error();
        checked = truth != 0;
    }
    if (checked && (rc = kkt_device_status(stream)) != KKT_OK) return PyLong_FromLong(-rc);
    return nullptr;
}

bool arity(Py_ssize_t n, Py_ssize_t want) {
    if (n == want) return true;
    PyErr_Format(PyExc_TypeError, "%zd arguments expected, %zd given", want, n);
    return false;
}

PyObject *wrap(const Tensor &t) {
    if (!t.defined()) Py_RETURN_NONE;
    return THPVariable_Wrap(t);
}

template <typename... T>
PyObject *wrap_all(const T &...t) {
    PyObject *items[] = {wrap(t)...};
    PyObject *tuple = PyTuple_New(sizeof...(T));
    for (size_t i = 0; i < sizeof...(T); ++i) PyTuple_SET_ITEM(tuple, i, items[i]);
    return tuple;
}

// q, k, v, beta, state, g, slots, slots_out, cu_seqlens, scale, o, check
PyObject *recurrent(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (!arity(n, 12)) return nullptr;
    return guarded([&]() -> PyObject * {
        const Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k"), &v = tensor(a[2], "v"), &beta = tensor(a[3], "beta"),
                     &state = tensor(a[4], "state");
        const Tensor g = optional(a[5], "g"), slots = optional(a[6], "slots"), slots_out = optional(a[7], "slots_out"),
                     cu = optional(a[8], "cu_seqlens");
        Tensor o = optional(a[10], "o");
        const char *shapes = "q, k [B,T,Hk,dk], v [B,T,Hv,dv], state [P,Hv,dk,dv]";
        need_dim(q, shapes, 4); need_dim(k, shapes, 4); need_dim(v, shapes, 4); need_dim(state, shapes, 4);
        const int64_t B = k.size(0), T = k.size(1), Hk = k.size(2), dk = k.size(3), Hv = v.size(2), dv = v.size(3),
                      P = state.size(0);
        const c10::Device dev = device_of(q, "q");
        const ScalarType dt = q.scalar_type();
        const int io = io_type(q, "q"), st = io_type(state, "state");
        check(q, "q", dt, {B, T, Hk, dk}, dev);
        check(k, "k", dt, {B, T, Hk, dk}, dev);
        check(v, "v", dt, {B, T, Hv, dv}, dev);
        check(beta, "beta", at::kFloat, {B, T, Hv}, dev);
        if (g.defined()) check(g, "g", at::kFloat, {B, T, Hv}, dev);
        check(state, "state", state.scalar_type(), {P, Hv, dk, dv}, dev);
        const int N = sequences(cu, B, dev);
        if (slots.defined()) check(slots, "slots", at::kInt, {N}, dev);
        if (slots_out.defined()) check(slots_out, "slots_out", at::kInt, {N}, dev);
        const double scale = a[9] == Py_None ? 1.0 / std::sqrt((double)dk) : number(a[9], "scale");
        const c10::cuda::CUDAGuard guard(dev);
        CUstream_st *stream = stream_on(dev);
        if (o.defined()) check(o, "o", dt, v.sizes(), dev);
        else o = empty(v.sizes(), dt, dev);
        const int rc = gdn_recurrent_fwd(raw(q), raw(k), raw(v), ptr<float>(beta), ptr<float>(g), ptr<int32_t>(cu), N,
                                         small(T, "T"), small(Hk, "Hk"), small(Hv, "Hv"), small(dk, "dk"),
                                         small(dv, "dv"), (float)scale, io, raw(state), st, small(P, "P"),
                                         ptr<int32_t>(slots), ptr<int32_t>(slots_out), raw(o), stream);
        if (PyObject *said = trouble(rc, a[11], stream)) return said;
        if (a[10] != Py_None) return Py_NewRef(a[10]);
        return wrap(o);
    });
}

// x, weight, a, b, A_log, dt_bias, conv_state, Hk, Hv, dk, dv, bias, slots, cu_seqlens, expand, eps, check
PyObject *prep(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (!arity(n, 17)) return nullptr;
    return guarded([&]() -> PyObject * {
        const Tensor &x = tensor(a[0], "x"), &weight = tensor(a[1], "weight"), &ga = tensor(a[2], "a"),
                     &gb = tensor(a[3], "b"), &A_log = tensor(a[4], "A_log"), &dt_bias = tensor(a[5], "dt_bias"),
                     &conv = tensor(a[6], "conv_state");
        const int Hk = integer(a[7], "Hk"), Hv = integer(a[8], "Hv"), dk = integer(a[9], "dk"), dv = integer(a[10], "dv");
        const Tensor bias = optional(a[11], "bias"), slots = optional(a[12], "slots"), cu = optional(a[13], "cu_seqlens");
        const int expand = PyObject_IsTrue(a[14]);
        if (expand < 0) throw python_error();
        const double eps = number(a[15], "eps");
        const char *shapes = "x [B,T,D], weight [D,taps], conv_state [P,taps-1,D]";
        need_dim(x, shapes, 3); need_dim(weight, shapes, 2); need_dim(conv, shapes, 3);
        const int64_t B = x.size(0), T = x.size(1), D = x.size(2), taps = weight.size(1), P = conv.size(0);
        const int64_t want = (int64_t)2 * Hk * dk + (int64_t)Hv * dv;
        if (Hk < 1 || Hv < 1 || dk < 1 || dv < 1 || D != want)
            refuse("x must have 2 Hk dk + Hv dv = " + std::to_string(want) + " channels, got " + std::to_string(D));
        const c10::Device dev = device_of(x, "x");
        const ScalarType dt = x.scalar_type();
        const int io = io_type(x, "x");
        const int64_t x_stride = check_sliced(x, "x", dt, {B, T, D}, D, dev);
        check(weight, "weight", dt, {D, taps}, dev);
        if (bias.defined()) check(bias, "bias", dt, {D}, dev);
        const int64_t a_stride = check_sliced(ga, "a", dt, {B, T, Hv}, Hv, dev),
                      b_stride = check_sliced(gb, "b", dt, {B, T, Hv}, Hv, dev);
        check(A_log, "A_log", at::kFloat, {Hv}, dev);
        check(dt_bias, "dt_bias", at::kFloat, {Hv}, dev);
        check(conv, "conv_state", dt, {P, taps - 1, D}, dev);
        const int N = sequences(cu, B, dev);
        if (slots.defined()) check(slots, "slots", at::kInt, {N}, dev);
        const c10::cuda::CUDAGuard guard(dev);
        CUstream_st *stream = stream_on(dev);
        const int64_t Hq = expand ? Hv : Hk;
        const Tensor q = empty({B, T, Hq, dk}, dt, dev), k = empty({B, T, Hq, dk}, dt, dev),
                     v = empty({B, T, Hv, dv}, dt, dev), g = empty({B, T, Hv}, at::kFloat, dev),
                     beta = empty({B, T, Hv}, at::kFloat, dev);
        const int rc = gdn_prep_fwd(raw(x), x_stride, raw(weight), raw(bias), raw(ga), a_stride, raw(gb), b_stride,
                                    ptr<float>(A_log), ptr<float>(dt_bias), ptr<int32_t>(cu), N, small(T, "T"), Hk,
                                    Hv, dk, dv, small(taps, "taps"), (float)eps, expand, io, raw(conv),
                                    small(P, "P"), ptr<int32_t>(slots), raw(q), raw(k), raw(v), ptr<float>(g),
                                    ptr<float>(beta), stream);
        if (PyObject *said = trouble(rc, a[16], stream)) return said;
        return wrap_all(q, k, v, g, beta);
    });
}

// The output's type: a torch.dtype, or None for x's.
ScalarType out_type(PyObject *o, const Tensor &x, int &code) {
    ScalarType t = x.scalar_type();
    if (o != Py_None) {
        if (!THPDtype_Check(o)) refuse("out_dtype must be a torch.dtype");
        t = reinterpret_cast<THPDtype *>(o)->scalar_type;
    }
    if (t == at::kBFloat16) code = GDN_OUT_BF16;
    else if (t == at::kFloat) code = GDN_OUT_F32;
    else if (t == at::kFloat8_e4m3fn) code = GDN_OUT_E4M3;
    else refuse(std::string("out_dtype must be torch.bfloat16, torch.float32 or torch.float8_e4m3fn, got ") + c10::toString(t));
    return t;
}

// x, weight, residual, eps, out_dtype, group, residual_out, check
PyObject *add_norm(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (!arity(n, 8)) return nullptr;
    return guarded([&]() -> PyObject * {
        const Tensor &x = tensor(a[0], "x"), &w = tensor(a[1], "weight");
        const Tensor r = optional(a[2], "residual");
        Tensor r_out = optional(a[6], "residual_out");
        if (x.dim() < 1) refuse("expected x [..., dim]");
        const c10::Device dev = device_of(x, "x");
        const ScalarType dt = x.scalar_type();
        const int io = io_type(x, "x");
        const int64_t dim = x.size(-1);
        check(x, "x", dt, x.sizes(), dev);
        check(w, "weight", dt, {dim}, dev);
        if (r.defined()) check(r, "residual", dt, x.sizes(), dev);
        else if (r_out.defined()) refuse("residual_out given without a residual");
        if (r_out.defined()) check(r_out, "residual_out", dt, x.sizes(), dev);
        int code;
        const ScalarType out = out_type(a[4], x, code);
        const int group = a[5] == Py_None ? 0 : integer(a[5], "group");
        if (a[5] != Py_None && group != 128) refuse("group must be 128 or None, got " + std::to_string(group));
        const double eps = number(a[3], "eps");
        const c10::cuda::CUDAGuard guard(dev);
        CUstream_st *stream = stream_on(dev);
        if (r.defined() && !r_out.defined()) r_out = empty(x.sizes(), dt, dev);
        const Tensor y = empty(x.sizes(), out, dev);
        Tensor scales;
        if (code == GDN_OUT_E4M3) {
            std::vector<int64_t> shape(x.sizes().begin(), x.sizes().end());
            if (group) shape.back() = (dim + group - 1) / group;
            else shape.pop_back();
            scales = empty(shape, at::kFloat, dev);
        }
        const int rc = add_rms_norm_fwd(raw(x), raw(r), raw(w), dim ? x.numel() / dim : 0, small(dim, "dim"), (float)eps,
                                        io, code, group, raw(y), ptr<float>(scales), raw(r_out), stream);
        if (PyObject *said = trouble(rc, a[7], stream)) return said;
        if (a[6] != Py_None) {
            PyObject *tuple = wrap_all(y, scales, Tensor());
            PyTuple_SetItem(tuple, 2, Py_NewRef(a[6]));
            return tuple;
        }
        return wrap_all(y, scales, r_out);
    });
}

// x, z, weight, eps, out_dtype, check
PyObject *gated_norm(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (!arity(n, 6)) return nullptr;
    return guarded([&]() -> PyObject * {
        const Tensor &x = tensor(a[0], "x"), &z = tensor(a[1], "z"), &w = tensor(a[2], "weight");
        if (x.dim() < 1) refuse("expected x [..., d]");
        const c10::Device dev = device_of(x, "x");
        const ScalarType dt = x.scalar_type();
        const int io = io_type(x, "x");
        const int64_t dim = x.size(-1);
        check(x, "x", dt, x.sizes(), dev);
        // z may be a slice: the dimensions before d that lie behind one another are a token's rows
        int64_t packed = 1;
        for (int64_t d = z.dim() - 1; d >= 0 && (z.size(d) == 1 || z.stride(d) == packed); --d) packed *= z.size(d);
        const int64_t z_stride = check_sliced(z, "z", dt, x.sizes(), packed, dev);
        int64_t z_rows = 0;
        if (!z.is_contiguous()) {
            if (packed % dim != 0) refuse("z's rows must be contiguous");
            z_rows = packed / dim;
        }
        check(w, "weight", dt, {dim}, dev);
        int code;
        const ScalarType out = out_type(a[4], x, code);
        const double eps = number(a[3], "eps");
        const c10::cuda::CUDAGuard guard(dev);
        CUstream_st *stream = stream_on(dev);
        const Tensor y = empty(x.sizes(), out, dev);
        Tensor scales;
        if (code == GDN_OUT_E4M3) scales = empty(x.sizes().slice(0, x.dim() - 1), at::kFloat, dev);
        const int rc = gated_rms_norm_fwd(raw(x), raw(z), small(z_rows, "z's rows"), z_stride, raw(w), dim ? x.numel() / dim : 0, small(dim, "dim"),
                                          (float)eps, io, code, raw(y), ptr<float>(scales), stream);
        if (PyObject *said = trouble(rc, a[5], stream)) return said;
        return wrap_all(y, scales);
    });
}

// One side of a copy: a tensor, or a sequence of them, [P, ...] of one P, whose slots are contiguous.
struct Side {
    std::vector<Tensor> t;
    std::vector<void *> ptrs;
    std::vector<size_t> bytes, stride;
    int64_t slots = 0;
};

Side side(PyObject *o, const char *name) {
    const std::string n(name);
    Side s;
    if (THPVariable_Check(o)) {
        s.t.push_back(THPVariable_Unpack(o));
    } else {
        PyObject *seq = PySequence_Fast(o, "");
        if (!seq) {
            PyErr_Clear();
            refuse(n + " must be a tensor or a list of tensors");
        }
        const Py_ssize_t len = PySequence_Fast_GET_SIZE(seq);
        bool ok = true;
        for (Py_ssize_t i = 0; i < len && ok; ++i) {
            PyObject *item = PySequence_Fast_GET_ITEM(seq, i);
            if ((ok = THPVariable_Check(item))) s.t.push_back(THPVariable_Unpack(item));
        }
        Py_DECREF(seq);
        if (!ok) refuse(n + " must hold tensors");
    }
    if (s.t.empty() || s.t.size() > GDN_COPY_MAX_TENSORS)
        refuse("1 to " + std::to_string(GDN_COPY_MAX_TENSORS) + " tensors, got " + std::to_string(s.t.size()));
    for (const Tensor &t : s.t) {
        if (!t.is_cuda() || t.dim() < 2 || t.size(0) != s.t[0].size(0) || t.device() != s.t[0].device())
            refuse(n + " must be CUDA tensors [P, ...] of one device and one slot count P");
        int64_t count = 1;  // values of a slot; contiguous where the strides behind the first are the packed ones
        bool packed = true;
        for (int64_t d = t.dim() - 1; d >= 1; --d) {
            packed = packed && (t.size(d) == 1 || t.stride(d) == count);
            count *= t.size(d);
        }
        if (t.size(0) > 0 && (count == 0 || !packed || (t.size(0) > 1 && t.stride(0) < count)))
            refuse(n + " must have contiguous, non-empty slots that do not overlap");
        const size_t e = t.element_size();
        s.ptrs.push_back(t.data_ptr());
        s.bytes.push_back((size_t)count * e);
        s.stride.push_back((size_t)(t.size(0) > 1 ? t.stride(0) : count) * e);
    }
    s.slots = s.t[0].size(0);
    return s;
}

// dst, dst_slots, src, src_slots, check
PyObject *state_copy(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (!arity(n, 5)) return nullptr;
    return guarded([&]() -> PyObject * {
        const Side dst = side(a[0], "dst");
        const c10::Device dev = dst.t[0].device();
        const Tensor &dst_slots = tensor(a[1], "dst_slots");
        check(dst_slots, "dst_slots", at::kInt, {dst_slots.numel()}, dev);
        const Tensor src_slots = optional(a[3], "src_slots");
        const bool copies = a[2] != Py_None;
        if (copies != src_slots.defined())
            refuse(copies ? "src given without src_slots" : "src_slots given without src");
        Side other;
        if (copies && a[2] != a[0]) {
            other = side(a[2], "src");
            if (other.t.size() != dst.t.size())
                refuse(std::to_string(dst.t.size()) + " destination tensors and " + std::to_string(other.t.size()) + " sources");
            for (size_t i = 0; i < dst.t.size(); ++i)
                if (dst.t[i].scalar_type() != other.t[i].scalar_type() || dst.t[i].sizes().slice(1) != other.t[i].sizes().slice(1))
                    refuse("a source's slots must have the shape and type of its destination's");
            if (other.t[0].device() != dev) refuse("src is on another device");
        }
        const Side &src = copies && a[2] != a[0] ? other : dst;
        if (copies) check(src_slots, "src_slots", at::kInt, dst_slots.sizes(), dev);
        if (dst.slots == 0 || dst_slots.numel() == 0) Py_RETURN_NONE;
        const c10::cuda::CUDAGuard guard(dev);
        CUstream_st *stream = stream_on(dev);
        const int rc = gdn_state_copy(
            dst.ptrs.data(), copies ? const_cast<const void *const *>(src.ptrs.data()) : nullptr, dst.bytes.data(),
            dst.stride.data(), copies ? src.stride.data() : nullptr, (int)dst.t.size(), ptr<int32_t>(dst_slots),
            ptr<int32_t>(src_slots), small(dst_slots.numel(), "dst_slots"), small(dst.slots, "P"),
            copies ? small(src.slots, "P") : 0, stream);
        if (PyObject *said = trouble(rc, a[4], stream)) return said;
        Py_RETURN_NONE;
    });
}

PyMethodDef kMethods[] = {
    {"recurrent", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(recurrent)), METH_FASTCALL, nullptr},
    {"prep", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(prep)), METH_FASTCALL, nullptr},
    {"add_norm", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(add_norm)), METH_FASTCALL, nullptr},
    {"gated_norm", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(gated_norm)), METH_FASTCALL, nullptr},
    {"state_copy", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(state_copy)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_gdn_binding", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__gdn_binding() { return PyModule_Create(&kModule); }
