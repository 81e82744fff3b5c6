// The Python calls of the gated linear recurrence and of the norms: checks of
// the tensors, the outputs, and the C entry point, compiled because a decode
// step's kernel is shorter than the same checks in Python (a step takes 11 us
// through ctypes).  Like the ctypes binding it only marshals arguments.
//
// Each function takes positional arguments in the order of its Python wrapper
// (mamba_ssd_sequence_b200/__init__.py), which holds the documentation.
#include <Python.h>

#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <optional>
#include <string>
#include <vector>

#include "ssd.h"

namespace {

using at::IntArrayRef;
using at::ScalarType;
using at::Tensor;

PyObject *g_error = nullptr;  // SSDError(code, where)

// A Python exception on its way out of the checks.
struct Refused {};

[[noreturn]] void refuse(PyObject *type, const std::string &what) {
    PyErr_SetString(type, what.c_str());
    throw Refused{};
}

std::string shape_text(IntArrayRef s) {
    std::string r = "(";
    for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
    return r + (s.size() == 1 ? ",)" : ")");
}

const char *type_text(ScalarType t) {
    switch (t) {
    case at::kFloat: return "torch.float32";
    case at::kBFloat16: return "torch.bfloat16";
    case at::kInt: return "torch.int32";
    case at::kByte: return "torch.uint8";
    default: return c10::toString(t);
    }
}

// A tensor argument; null for None.
const Tensor *tensor(PyObject *o, const char *name) {
    if (o == Py_None) return nullptr;
    if (!THPVariable_Check(o)) refuse(PyExc_TypeError, std::string(name) + " must be a tensor");
    return &THPVariable_Unpack(o);
}
const Tensor &needed(PyObject *o, const char *name, const char *why = "") {
    const Tensor *t = tensor(o, name);
    if (!t) refuse(PyExc_ValueError, *why ? why : std::string(name) + " must be a tensor, got None");
    return *t;
}
bool truth(PyObject *o) {
    const int r = PyObject_IsTrue(o);
    if (r < 0) throw Refused{};
    return r != 0;
}
int integer(PyObject *o, const char *name) {
    const long v = PyLong_AsLong(o);
    if (v == -1 && PyErr_Occurred()) throw Refused{};
    if (v != (int)v) refuse(PyExc_ValueError, std::string(name) + " is out of range");
    return (int)v;
}
int size_of(int64_t v) {  // the entry points refuse what does not fit
    return v > 0x7fffffff ? 0x7fffffff : (int)v;
}

int code_of(const Tensor &t, const char *name) {
    if (t.scalar_type() == at::kFloat) return SSD_F32;
    if (t.scalar_type() == at::kBFloat16) return SSD_BF16;
    refuse(PyExc_TypeError, std::string(name) + " must be float32 or bfloat16, got " + type_text(t.scalar_type()));
}

// The device and stream of one call.
struct Call {
    int index = -1;
    void *handle = nullptr;
    std::optional<c10::cuda::CUDAStream> side;  // a stream other than the current one
    std::vector<Tensor> used;                   // what was given to a call on it

    Call(const Tensor &first, PyObject *stream) {
        if (!first.is_cuda()) refuse(PyExc_ValueError, "tensors must be on a CUDA device");
        index = first.get_device();
        if (c10::cuda::current_device() != index)
            refuse(PyExc_ValueError, "tensors are on cuda:" + std::to_string(index) + ", which is not the current CUDA device");
        const cudaStream_t current = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)index).stream();
        handle = current;
        if (stream == Py_None) return;
        PyObject *on = PyObject_GetAttrString(stream, "device_index"), *raw = PyObject_GetAttrString(stream, "cuda_stream");
        if (!on || !raw) {
            Py_XDECREF(on);
            Py_XDECREF(raw);
            throw Refused{};
        }
        const long at = PyLong_AsLong(on);
        handle = PyLong_AsVoidPtr(raw);
        Py_DECREF(on);
        Py_DECREF(raw);
        if (PyErr_Occurred()) throw Refused{};
        if (at != index)
            refuse(PyExc_ValueError, "the stream is on cuda:" + std::to_string(at) + ", the tensors on cuda:" + std::to_string(index));
        if (handle != current)
            side = c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(handle), (c10::DeviceIndex)index);
    }

    void *use(const Tensor &t, const char *name, IntArrayRef shape, ScalarType type) {
        if (t.scalar_type() != type)
            refuse(PyExc_TypeError, std::string(name) + " must be " + type_text(type) + ", got " + type_text(t.scalar_type()));
        if (t.sizes() != shape)
            refuse(PyExc_ValueError, std::string(name) + " must have shape " + shape_text(shape) + ", got " + shape_text(t.sizes()));
        if (!t.is_cuda() || t.get_device() != index)
            refuse(PyExc_ValueError, std::string(name) + " must be on CUDA device " + std::to_string(index) + ", got " + t.device().str());
        if (side) used.push_back(t);
        return t.data_ptr();
    }
    void *flat(const Tensor *t, const char *name, IntArrayRef shape, ScalarType type) {
        if (!t) return nullptr;
        if (!t->is_contiguous()) refuse(PyExc_ValueError, std::string(name) + " must be contiguous");
        return use(*t, name, shape, type);
    }
    float *floats(const Tensor *t, const char *name, IntArrayRef shape) {
        return static_cast<float *>(flat(t, name, shape, at::kFloat));
    }
    // a new tensor that belongs to the call's stream
    Tensor make(IntArrayRef shape, ScalarType type) {
        const c10::Device device(c10::kCUDA, (c10::DeviceIndex)index);
        if (!side) return at::detail::empty_cuda(shape, type, device, std::nullopt);
        c10::cuda::CUDAStreamGuard on(*side);
        return at::detail::empty_cuda(shape, type, device, std::nullopt);
    }
    Tensor given_or(const Tensor *t, IntArrayRef shape, ScalarType type) { return t ? *t : make(shape, type); }

    ssd_view heads(const Tensor &t, const char *name, IntArrayRef shape, ScalarType type) {
        void *p = use(t, name, shape, type);
        const IntArrayRef s = t.strides();
        contiguous_end(s, shape, name);
        return {p, s[0], s[1], shape.size() == 4 ? s[2] : 0};
    }
    ssd_view tokens(const Tensor &t, const char *name, IntArrayRef shape, ScalarType type, int64_t d) {
        void *p = use(t, name, shape, type);
        const IntArrayRef s = t.strides();
        contiguous_end(s, shape, name);
        return {p, s[0], d, s[1]};
    }
    // [..., C] whose leading dimensions have one stride
    ssd_rows rows(const Tensor &t, const char *name, IntArrayRef shape, ScalarType type) {
        void *p = use(t, name, shape, type);
        const IntArrayRef s = t.strides();
        contiguous_end(s, shape, name);
        int64_t step = -1, n = 1;
        for (int64_t i = (int64_t)shape.size() - 2; i >= 0; --i) {
            if (shape[i] == 1) continue;
            if (step < 0)
                step = s[i];
            else if (s[i] != step * n)
                refuse(PyExc_ValueError,
                       std::string(name) + ": the leading dimensions must be evenly spaced (one stride between rows)");
            n *= shape[i];
        }
        return {p, step < 0 ? shape.back() : step};
    }
    static void contiguous_end(IntArrayRef strides, IntArrayRef shape, const char *name) {
        if (strides.back() != 1 && shape.back() != 1)
            refuse(PyExc_ValueError, std::string(name) + ": the last dimension must be contiguous");
    }
    void *workspace(const Tensor *given, size_t bytes, Tensor &keep, size_t &size) {
        if (given) {
            size = (size_t)given->numel();
            return flat(given, "workspace", given->sizes(), at::kByte);
        }
        keep = make({(int64_t)(bytes ? bytes : 1)}, at::kByte);
        size = bytes;
        return keep.data_ptr();
    }

    void done(int rc, const char *where) {
        if (side)
            for (const Tensor &t : used)
                c10::cuda::CUDACachingAllocator::recordStream(t.storage().data_ptr(), *side);
        if (rc == SSD_OK) return;
        PyObject *e = PyObject_CallFunction(g_error, "is", rc, where);
        if (e) {
            PyErr_SetObject(g_error, e);
            Py_DECREF(e);
        }
        throw Refused{};
    }
};

PyObject *wrap(const Tensor &t) { return THPVariable_Wrap(t); }
PyObject *wrap_or_none(const Tensor *t) {
    if (t) return wrap(*t);
    Py_RETURN_NONE;
}
// The same Python object when the caller gave it.
PyObject *same_or(PyObject *given, const Tensor &t) {
    if (given == Py_None) return wrap(t);
    Py_INCREF(given);
    return given;
}
PyObject *tuple_of(std::initializer_list<PyObject *> items) {
    PyObject *r = PyTuple_New((Py_ssize_t)items.size());
    Py_ssize_t i = 0;
    for (PyObject *o : items) PyTuple_SET_ITEM(r, i++, o);
    return r;
}

void dims(const Tensor &t, size_t n, const char *name, const char *what) {
    if (t.sizes().size() != n) refuse(PyExc_ValueError, std::string(name) + " must be " + what + ", got shape " + shape_text(t.sizes()));
}

// The gate of a recurrence: dt_p or log_decay, and the flags.
const Tensor &gate_of(PyObject *dt_p, PyObject *log_decay, PyObject *value_dt, PyObject *complement, int &flags) {
    const bool vd = truth(value_dt), vc = truth(complement);
    if ((dt_p == Py_None) == (log_decay == Py_None)) refuse(PyExc_ValueError, "give either dt_p or log_decay");
    if (vd && (vc || dt_p == Py_None)) refuse(PyExc_ValueError, "value_dt needs dt_p, and excludes value_complement");
    flags = (vd ? SSD_VALUE_DT : 0) | (vc ? SSD_GLR_COMPLEMENT : 0) | (dt_p == Py_None ? SSD_GLR_LOG_DECAY : 0);
    return dt_p == Py_None ? needed(log_decay, "log_decay") : needed(dt_p, "dt_p");
}

PyObject *glr_fwd(PyObject *const *a) {
    int flags;
    const Tensor &gate = gate_of(a[1], a[4], a[5], a[6], flags), &x = needed(a[0], "x");
    dims(x, 4, "x", "[B, H, N, d_h]");
    const IntArrayRef shape = x.sizes();
    const int64_t B = shape[0], H = shape[1], N = shape[2], d = shape[3];
    Call call(x, a[12]);
    const int code = code_of(x, "x");
    const ScalarType type = x.scalar_type();
    const Tensor *given = tensor(a[11], "out");
    const int64_t C[] = {H * d}, state[] = {B, H, d}, saved[] = {B, H, (N + SSD_GLR_CHUNK - 1) / SSD_GLR_CHUNK, d}, batch[] = {B};
    const ssd_view xv = call.heads(x, "x", shape, type), gv = call.heads(gate, "the gate", shape, type);
    float *A = call.floats(tensor(a[2], "A_log"), "A_log", C), *b = call.floats(tensor(a[3], "dt_bias"), "dt_bias", C);
    float *h0 = call.floats(tensor(a[7], "h0"), "h0", state), *h_out = call.floats(tensor(a[8], "h_out"), "h_out", state);
    float *states = call.floats(tensor(a[9], "states"), "states", saved);
    const int *lengths = static_cast<int *>(call.flat(tensor(a[10], "lengths"), "lengths", batch, at::kInt));
    const Tensor out = call.given_or(given, shape, type);
    const ssd_view ov = call.heads(out, "out", shape, type);
    call.done(ssd_glr_fwd(&xv, &gv, A, b, h0, lengths, size_of(B), size_of(H), size_of(N), size_of(d), code, flags, &ov, h_out,
                          states, call.handle),
              "ssd_glr_fwd");
    return same_or(a[11], out);
}

PyObject *glr_bwd(PyObject *const *a) {
    int flags;
    const Tensor &gate = gate_of(a[2], a[6], a[7], a[8], flags), &dy = needed(a[0], "dy"), &x = needed(a[1], "x");
    const Tensor &saved = needed(a[5], "states", "ssd_glr_bwd needs the states that ssd_glr_fwd saved");
    dims(x, 4, "x", "[B, H, N, d_h]");
    const IntArrayRef shape = x.sizes();
    const int64_t B = shape[0], H = shape[1], N = shape[2], d = shape[3];
    Call call(x, a[14]);
    const int code = code_of(x, "x");
    const ScalarType type = x.scalar_type();
    const int64_t C[] = {H * d}, state[] = {B, H, d}, kept[] = {B, H, (N + SSD_GLR_CHUNK - 1) / SSD_GLR_CHUNK, d}, batch[] = {B};
    const Tensor *A_log = tensor(a[3], "A_log"), *bias = tensor(a[4], "dt_bias"), *dh_out = tensor(a[10], "dh_out");
    float *A = call.floats(A_log, "A_log", C), *b = call.floats(bias, "dt_bias", C);
    const ssd_view yv = call.heads(dy, "dy", shape, type), xv = call.heads(x, "x", shape, type),
                   gv = call.heads(gate, "the gate", shape, type);
    float *st = call.floats(&saved, "states", kept), *dh = call.floats(dh_out, "dh_out", state);
    const int *lengths = static_cast<int *>(call.flat(tensor(a[9], "lengths"), "lengths", batch, at::kInt));
    const bool log = flags & SSD_GLR_LOG_DECAY;
    const Tensor dx = call.given_or(tensor(a[11], "dx"), shape, type), dg = call.given_or(tensor(a[12], "dgate"), shape, type);
    const ssd_view dxv = call.heads(dx, "dx", shape, type), dgv = call.heads(dg, "dgate", shape, type);
    const Tensor dh0 = call.make(state, at::kFloat);
    Tensor dA, db, ws;
    if (A_log && !log) dA = call.make(C, at::kFloat);
    if (bias && !log) db = call.make(C, at::kFloat);
    size_t bytes;
    const int nB = size_of(B), nH = size_of(H), nN = size_of(N), nd = size_of(d);
    void *w = call.workspace(tensor(a[13], "workspace"), ssd_glr_bwd_workspace_bytes(nB, nH, nN, nd, code, flags), ws, bytes);
    call.done(ssd_glr_bwd(&yv, &xv, &gv, A, b, st, lengths, dh, nB, nH, nN, nd, code, flags, &dxv, &dgv,
                          dA.defined() ? dA.data_ptr<float>() : nullptr, db.defined() ? db.data_ptr<float>() : nullptr,
                          dh0.data_ptr<float>(), w, bytes, call.handle),
              "ssd_glr_bwd");
    return tuple_of({same_or(a[11], dx), same_or(a[12], dg), wrap_or_none(dA.defined() ? &dA : nullptr),
                     wrap_or_none(db.defined() ? &db : nullptr), wrap(dh0)});
}

PyObject *glr_step(PyObject *const *a) {
    int flags;
    const Tensor &gate = gate_of(a[1], a[5], a[6], a[7], flags), &x = needed(a[0], "x");
    const Tensor &h = needed(a[4], "h", "ssd_glr_step needs the state h");
    dims(x, 3, "x", "[B, H, d_h]");
    const IntArrayRef shape = x.sizes();
    Call call(x, a[9]);
    const int code = code_of(x, "x");
    const ScalarType type = x.scalar_type();
    const int64_t C[] = {shape[1] * shape[2]};
    const ssd_view xv = call.heads(x, "x", shape, type), gv = call.heads(gate, "the gate", shape, type);
    float *A = call.floats(tensor(a[2], "A_log"), "A_log", C), *b = call.floats(tensor(a[3], "dt_bias"), "dt_bias", C);
    float *hp = call.floats(&h, "h", shape);
    const Tensor out = call.given_or(tensor(a[8], "out"), shape, type);
    const ssd_view ov = call.heads(out, "out", shape, type);
    call.done(ssd_glr_step(&xv, &gv, A, b, size_of(shape[0]), size_of(shape[1]), size_of(shape[2]), code, flags, hp, &ov,
                           call.handle),
              "ssd_glr_step");
    return same_or(a[8], out);
}

ssd_norm_params norm_params(PyObject *eps, int groups, int flags) {
    ssd_norm_params p{1.0f, groups, flags};
    if (eps) {
        p.eps = (float)PyFloat_AsDouble(eps);
        if (PyErr_Occurred()) throw Refused{};
    }
    return p;
}

// [..., C] as M rows
void matrix(const Tensor &t, const char *name, int64_t &M, int64_t &C) {
    if (t.dim() < 1) refuse(PyExc_ValueError, std::string(name) + " must have at least one dimension");
    C = t.sizes().back();
    M = C ? t.numel() / C : 0;
}

PyObject *add_norm(PyObject *const *a) {
    const Tensor &x = needed(a[0], "x");
    const Tensor *res = tensor(a[1], "residual"), *scale = tensor(a[2], "scale"), *w = tensor(a[3], "w");
    int64_t M, C;
    matrix(x, "x", M, C);
    const IntArrayRef shape = x.sizes(), lead = shape.slice(0, shape.size() - 1);
    Call call(x, a[8]);
    const int code = code_of(x, "x"), rcode = res ? code_of(*res, "residual") : code;
    const ScalarType type = x.scalar_type(), kept = res ? res->scalar_type() : type;
    const ssd_norm_params p = norm_params(a[4], 1, 0);
    const bool plain = !res && !scale;
    if (plain && a[5] != Py_None) refuse(PyExc_ValueError, "without residual and scale r is x: none is written");
    const int64_t Cs[] = {C};
    const ssd_rows xv = call.rows(x, "x", shape, type);
    ssd_rows rv{}, sv{};
    if (res) sv = call.rows(*res, "residual", shape, kept);
    float *sp = call.floats(scale, "scale", Cs), *wp = call.floats(w, "w", Cs);
    Tensor r;
    if (!plain) {
        r = call.given_or(tensor(a[5], "r"), shape, kept);
        rv = call.rows(r, "r", shape, kept);
    }
    const Tensor out = call.given_or(tensor(a[6], "out"), shape, type);
    const ssd_rows ov = call.rows(out, "out", shape, type);
    const Tensor rstd = call.given_or(tensor(a[7], "rstd"), lead, at::kFloat);
    float *rs = call.floats(&rstd, "rstd", lead);
    call.done(ssd_add_norm(&xv, res ? &sv : nullptr, sp, wp, size_of(M), size_of(C), code, rcode, &p, plain ? nullptr : &rv, &ov,
                           rs, call.handle),
              "ssd_add_norm");
    return tuple_of({same_or(a[6], out), plain ? same_or(a[0], x) : same_or(a[5], r), same_or(a[7], rstd)});
}

PyObject *add_norm_bwd(PyObject *const *a) {
    const Tensor &dy = needed(a[0], "dy"), &r = needed(a[1], "r"), &rstd = needed(a[2], "rstd");
    const Tensor *w = tensor(a[3], "w"), *x = tensor(a[4], "x"), *scale = tensor(a[5], "scale"), *dres = tensor(a[6], "dres");
    if (scale && !x) refuse(PyExc_ValueError, "the gradient of scale needs x");
    int64_t M, C;
    matrix(dy, "dy", M, C);
    const IntArrayRef shape = dy.sizes(), lead = shape.slice(0, shape.size() - 1);
    Call call(dy, a[10]);
    const int code = code_of(dy, "dy"), rcode = code_of(r, "r");
    const ScalarType type = dy.scalar_type(), kept = r.scalar_type();
    const int64_t Cs[] = {C};
    const ssd_rows yv = call.rows(dy, "dy", shape, type), rv = call.rows(r, "r", shape, kept);
    ssd_rows xv{}, sv{}, dxv{};
    if (scale) xv = call.rows(*x, "x", shape, type);
    if (dres) sv = call.rows(*dres, "dres", shape, kept);
    float *rs = call.floats(&rstd, "rstd", lead), *wp = call.floats(w, "w", Cs), *sp = call.floats(scale, "scale", Cs);
    const Tensor dr = call.given_or(tensor(a[7], "dr"), shape, kept);
    const ssd_rows drv = call.rows(dr, "dr", shape, kept);
    Tensor dx, dw, ds, ws;
    const bool has_dx = a[8] != Py_None || scale || kept != type;  // else it equals dr
    if (has_dx) {
        dx = call.given_or(tensor(a[8], "dx"), shape, type);
        dxv = call.rows(dx, "dx", shape, type);
    }
    if (w) dw = call.make(Cs, at::kFloat);
    if (scale) ds = call.make(Cs, at::kFloat);
    size_t bytes;
    const int nM = size_of(M), nC = size_of(C);
    void *wk = call.workspace(tensor(a[9], "workspace"), ssd_add_norm_bwd_workspace_bytes(nM, nC), ws, bytes);
    call.done(ssd_add_norm_bwd(&yv, &rv, rs, wp, scale ? &xv : nullptr, sp, dres ? &sv : nullptr, nM, nC, code, rcode, &drv,
                               has_dx ? &dxv : nullptr, w ? dw.data_ptr<float>() : nullptr,
                               scale ? ds.data_ptr<float>() : nullptr, wk, bytes, call.handle),
              "ssd_add_norm_bwd");
    PyObject *pr = same_or(a[7], dr), *px;
    if (has_dx) {
        px = same_or(a[8], dx);
    } else {
        Py_INCREF(pr);
        px = pr;
    }
    return tuple_of({pr, px, wrap_or_none(w ? &dw : nullptr), wrap_or_none(scale ? &ds : nullptr)});
}

PyObject *gated_norm(PyObject *const *a) {
    const Tensor &x = needed(a[0], "x");
    const Tensor *z = tensor(a[1], "z");
    dims(x, 4, "x", "[B, H, N, d_h]");
    const IntArrayRef shape = x.sizes();
    const int64_t B = shape[0], H = shape[1], N = shape[2], d = shape[3];
    const int groups = integer(a[3], "groups");
    Call call(x, a[8]);
    const int code = code_of(x, "x");
    const ScalarType type = x.scalar_type();
    const ssd_norm_params p = norm_params(a[4], groups, truth(a[5]) ? SSD_NORM_GATE_AFTER : 0);
    const int64_t tok[] = {B, N, H * d}, rows[] = {B, N, groups < 0 ? 0 : groups}, C[] = {H * d};
    const ssd_view xv = call.heads(x, "x", shape, type);
    ssd_view zv{};
    if (z) zv = call.tokens(*z, "z", tok, type, d);
    float *w = call.floats(tensor(a[2], "w"), "w", C);
    const Tensor out = call.given_or(tensor(a[6], "out"), tok, type);
    const ssd_view ov = call.tokens(out, "out", tok, type, d);
    const Tensor rstd = call.given_or(tensor(a[7], "rstd"), rows, at::kFloat);
    float *rs = call.floats(&rstd, "rstd", rows);
    call.done(ssd_gated_norm(&xv, z ? &zv : nullptr, w, size_of(B), size_of(H), size_of(N), size_of(d), code, &p, &ov, rs,
                             call.handle),
              "ssd_gated_norm");
    return tuple_of({same_or(a[6], out), same_or(a[7], rstd)});
}

PyObject *gated_norm_bwd(PyObject *const *a) {
    const Tensor &dy = needed(a[0], "dy"), &x = needed(a[1], "x"), &rstd = needed(a[2], "rstd");
    const Tensor *z = tensor(a[3], "z"), *w = tensor(a[4], "w");
    dims(x, 4, "x", "[B, H, N, d_h]");
    if (!z && a[8] != Py_None) refuse(PyExc_ValueError, "without z there is no dz");
    const IntArrayRef shape = x.sizes();
    const int64_t B = shape[0], H = shape[1], N = shape[2], d = shape[3];
    const int groups = integer(a[5], "groups");
    Call call(x, a[10]);
    const int code = code_of(x, "x");
    const ScalarType type = x.scalar_type();
    const ssd_norm_params p = norm_params(nullptr, groups, truth(a[6]) ? SSD_NORM_GATE_AFTER : 0);
    const int64_t tok[] = {B, N, H * d}, rows[] = {B, N, groups < 0 ? 0 : groups}, C[] = {H * d};
    const ssd_view yv = call.tokens(dy, "dy", tok, type, d), xv = call.heads(x, "x", shape, type);
    ssd_view zv{}, dzv{};
    if (z) zv = call.tokens(*z, "z", tok, type, d);
    float *wp = call.floats(w, "w", C), *rs = call.floats(&rstd, "rstd", rows);
    const Tensor dx = call.given_or(tensor(a[7], "dx"), shape, type);
    const ssd_view dxv = call.heads(dx, "dx", shape, type);
    Tensor dz, dw, ws;
    if (z) {
        dz = call.given_or(tensor(a[8], "dz"), tok, type);
        dzv = call.tokens(dz, "dz", tok, type, d);
    }
    if (w) dw = call.make(C, at::kFloat);
    size_t bytes;
    const int nB = size_of(B), nH = size_of(H), nN = size_of(N), nd = size_of(d);
    void *wk = call.workspace(tensor(a[9], "workspace"), ssd_gated_norm_bwd_workspace_bytes(nB, nH, nN, nd, groups), ws, bytes);
    call.done(ssd_gated_norm_bwd(&yv, &xv, z ? &zv : nullptr, wp, rs, nB, nH, nN, nd, code, &p, &dxv, z ? &dzv : nullptr,
                                 w ? dw.data_ptr<float>() : nullptr, wk, bytes, call.handle),
              "ssd_gated_norm_bwd");
    return tuple_of({same_or(a[7], dx), z ? same_or(a[8], dz) : wrap_or_none(nullptr), wrap_or_none(w ? &dw : nullptr)});
}

template <PyObject *(*call)(PyObject *const *), int n>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t given) {
    HANDLE_TH_ERRORS
    if (given != n) {
        PyErr_Format(PyExc_TypeError, "%d arguments expected, got %zd", n, given);
        return nullptr;
    }
    try {
        return call(args);
    } catch (const Refused &) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

PyObject *set_error(PyObject *, PyObject *type) {
    Py_INCREF(type);
    Py_XSETREF(g_error, type);
    Py_RETURN_NONE;
}

template <PyObject *(*call)(PyObject *const *), int n>
PyMethodDef method(const char *name) {
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(entry<call, n>)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {
    method<glr_fwd, 13>("glr_fwd"),
    method<glr_bwd, 15>("glr_bwd"),
    method<glr_step, 10>("glr_step"),
    method<add_norm, 9>("add_norm"),
    method<add_norm_bwd, 11>("add_norm_bwd"),
    method<gated_norm, 9>("gated_norm"),
    method<gated_norm_bwd, 11>("gated_norm_bwd"),
    {"set_error", set_error, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() {
    PyObject *m = PyModule_Create(&module);
    if (m && PyModule_AddStringConstant(m, "torch_version", SSD_TORCH_VERSION) < 0) Py_CLEAR(m);
    return m;
}
