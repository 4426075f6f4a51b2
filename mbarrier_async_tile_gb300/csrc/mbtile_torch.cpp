// The layer operators' Python calls: argument checks, allocation of results and the
// C entry point in one compiled step, because at one token the checks and
// allocations in Python cost several times the kernel (RMS norm of one row with a
// residual and an e4m3 output: 17.6 us a call, 3.4 of them on the GPU).  Nothing
// is computed here.  The functions' signatures and documentation are in layer.py.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <stdexcept>
#include <string>

#include "mbtile.h"

namespace {

PyObject *g_mbt_error = nullptr;   // the package's MbtError(code, what)

struct BadArgument : std::runtime_error {
    using std::runtime_error::runtime_error;
};

int code_of(at::ScalarType t) {
    switch (t) {
        case at::kHalf: return MBT_F16;
        case at::kBFloat16: return MBT_BF16;
        case at::kFloat: return MBT_F32;
        case at::kFloat8_e4m3fn: return MBT_E4M3;
        default: return -1;
    }
}

bool is_wide(at::ScalarType t) { return t == at::kHalf || t == at::kBFloat16 || t == at::kFloat; }

[[noreturn]] void bad(const char *name, const std::string &what) {
    throw BadArgument(std::string(name) + " " + what);
}

std::string shape_text(at::IntArrayRef s) {
    std::string r = "(";
    for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
    return r + ")";
}

const at::Tensor &tensor(PyObject *o, const char *name) {
    if (!THPVariable_Check(o)) bad(name, "must be a tensor");
    return THPVariable_Unpack(o);
}

// A matrix that fixes the call's shape, type and device.
const at::Tensor &input(PyObject *o, const char *name) {
    const at::Tensor &t = tensor(o, name);
    if (t.dim() != 2 || !t.is_cuda()) bad(name, "must be a 2-D CUDA tensor");
    return t;
}

// Row pitch of a matrix that must have this shape, type and device.
int64_t rows(const at::Tensor &t, const char *name, int64_t M, int64_t N, at::ScalarType type, at::Device device) {
    if (t.dim() != 2 || t.size(0) != M || t.size(1) != N)
        bad(name, "must be a tensor of shape " + shape_text({M, N}));
    if (t.scalar_type() != type || t.device() != device) bad(name, "has another type or device than the call's matrices");
    if (M == 0 || N == 0) return N;
    if (t.stride(1) != 1 && N > 1) bad(name, "must be row-major (unit column stride)");
    if (M == 1) return N;
    if (t.stride(0) < N) bad(name, "has rows that overlap");
    return t.stride(0);
}

void *dense(const at::Tensor &t, const char *name, at::IntArrayRef shape, at::Device device) {
    if (t.sizes() != shape) bad(name, "must be a tensor of shape " + shape_text(shape));
    if (t.device() != device || !t.is_contiguous()) bad(name, "must be contiguous and on the call's device");
    return t.data_ptr();
}

void *dense_f32(const at::Tensor &t, const char *name, at::IntArrayRef shape, at::Device device) {
    if (t.scalar_type() != at::kFloat) bad(name, "must be float32");
    return dense(t, name, shape, device);
}

void *stream_of(at::Device device) {
    const auto current = c10::cuda::current_device();
    if (device.index() != current)
        throw BadArgument("tensors are on " + device.str() + ", the current device is cuda:" + std::to_string(current));
    return c10::cuda::getCurrentCUDAStream(device.index()).stream();
}

at::Tensor empty(at::IntArrayRef shape, at::ScalarType type, at::Device device) {
    return at::detail::empty_cuda(shape, type, device, c10::nullopt);
}

// Autograd is told that a tensor of the caller's was written.
void written(const at::Tensor &t) {
    if (t.defined() && !t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

// None or a tensor.
bool given(PyObject *o) { return o != Py_None; }

bool check(int rc, const char *what) {
    if (rc == MBT_OK) return true;
    PyObject *e = PyObject_CallFunction(g_mbt_error, "is", rc, what);
    if (e) {
        PyErr_SetObject(g_mbt_error, e);
        Py_DECREF(e);
    }
    return false;
}

PyObject *wrap(const at::Tensor &t) { return t.defined() ? THPVariable_Wrap(t) : Py_NewRef(Py_None); }

// Runs f, turning C++ exceptions into Python's.
template <class F>
PyObject *guarded(F f) {
    try {
        return f();
    } catch (const BadArgument &e) {
        PyErr_SetString(PyExc_ValueError, e.what());
    } catch (const c10::OutOfMemoryError &e) {
        PyErr_SetString(PyExc_MemoryError, e.what_without_backtrace());
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

bool arity(Py_ssize_t n, Py_ssize_t want) {
    if (n == want) return true;
    PyErr_Format(PyExc_TypeError, "%zd arguments, not %zd", want, n);
    return false;
}

bool number(PyObject *o, double *v) {
    *v = PyFloat_AsDouble(o);
    return !(*v == -1.0 && PyErr_Occurred());
}

// (x, weight, residual, eps, weight_offset, quant, out, scales, residual_out, rstd)
// -> (out, scales, residual_out, rstd); quant as in mbtile.h
PyObject *rmsnorm(PyObject *, PyObject *const *a, Py_ssize_t n) {
    double eps, offset;
    if (!arity(n, 10) || !number(a[3], &eps) || !number(a[4], &offset)) return nullptr;
    const long quant = PyLong_AsLong(a[5]);
    if (quant == -1 && PyErr_Occurred()) return nullptr;
    return guarded([&]() -> PyObject * {
        const at::Tensor &x = input(a[0], "x");
        const at::ScalarType type = x.scalar_type();
        if (!is_wide(type)) bad("x", "has an unsupported dtype");
        const at::Device device = x.device();
        const int64_t M = x.size(0), N = x.size(1);
        void *stream = stream_of(device);
        const int64_t ld_x = rows(x, "x", M, N, type, device);
        int64_t ld_res = 0, ld_ro = 0, ld_out = 0;
        void *w = nullptr, *res = nullptr, *ro = nullptr, *sc = nullptr;
        int wcode = 0;
        at::Tensor out, scales, residual_out, rstd;
        if (given(a[1])) {
            const at::Tensor &t = tensor(a[1], "weight");
            if (!is_wide(t.scalar_type())) bad("weight", "has an unsupported dtype");
            w = dense(t, "weight", {N}, device);
            wcode = code_of(t.scalar_type());
        }
        if (given(a[2])) {
            const at::Tensor &t = tensor(a[2], "residual");
            ld_res = rows(t, "residual", M, N, type, device);
            res = t.data_ptr();
            if (given(a[8])) {
                residual_out = tensor(a[8], "residual_out");
                ld_ro = rows(residual_out, "residual_out", M, N, type, device);
            } else {
                residual_out = empty({M, N}, type, device);
            }
            ro = residual_out.data_ptr();
        } else if (given(a[8])) {
            bad("residual_out", "needs a residual");
        }
        const bool quantised = quant != MBT_QUANT_NONE;
        const at::ScalarType out_type = quantised ? at::kFloat8_e4m3fn : type;
        if (given(a[6])) {
            out = tensor(a[6], "out");
            ld_out = rows(out, "out", M, N, out_type, device);
        } else {
            out = empty({M, N}, out_type, device);
        }
        if (quantised) {
            const int64_t groups = quant ? (N + quant - 1) / quant : 1;
            if (given(a[7])) {
                scales = tensor(a[7], "scales");
                sc = dense_f32(scales, "scales", {M, groups}, device);
            } else {
                scales = empty({M, groups}, at::kFloat, device);
                sc = scales.data_ptr();
            }
        } else if (given(a[7])) {
            bad("scales", "need quant");
        }
        if (given(a[9])) {
            rstd = tensor(a[9], "rstd");
            dense_f32(rstd, "rstd", {M}, device);
        } else {
            rstd = empty({M}, at::kFloat, device);
        }
        if (!check(tile_rmsnorm(x.data_ptr(), res, w, out.data_ptr(), ro, static_cast<float *>(sc),
                                static_cast<float *>(rstd.data_ptr()), M, N, ld_x, ld_res, ld_out, ld_ro, code_of(type),
                                wcode, static_cast<int>(quant), static_cast<float>(eps), static_cast<float>(offset),
                                stream),
                   "tile_rmsnorm"))
            return nullptr;
        for (const at::Tensor *t : {&out, &scales, &residual_out, &rstd}) written(*t);
        return Py_BuildValue("(NNNN)", wrap(out), wrap(scales), wrap(residual_out), wrap(rstd));
    });
}

// (dy, h, rstd, weight, dresidual, weight_offset, dx, dweight) -> (dx, dweight)
PyObject *rmsnorm_backward(PyObject *, PyObject *const *a, Py_ssize_t n) {
    double offset;
    if (!arity(n, 8) || !number(a[5], &offset)) return nullptr;
    return guarded([&]() -> PyObject * {
        const at::Tensor &h = input(a[1], "h");
        const at::ScalarType type = h.scalar_type();
        if (!is_wide(type)) bad("h", "has an unsupported dtype");
        const at::Device device = h.device();
        const int64_t M = h.size(0), N = h.size(1);
        void *stream = stream_of(device);
        const int64_t ld_h = rows(h, "h", M, N, type, device);
        const at::Tensor &dy = tensor(a[0], "dy");
        const int64_t ld_dy = rows(dy, "dy", M, N, type, device);
        const void *rstd = dense_f32(tensor(a[2], "rstd"), "rstd", {M}, device);
        void *w = nullptr, *res = nullptr;
        int64_t ld_res = 0, ld_dx = 0;
        int wcode = 0;
        at::Tensor dx, dw;
        if (given(a[3])) {
            const at::Tensor &t = tensor(a[3], "weight");
            if (!is_wide(t.scalar_type())) bad("weight", "has an unsupported dtype");
            w = dense(t, "weight", {N}, device);
            wcode = code_of(t.scalar_type());
        }
        if (given(a[7])) {
            dw = tensor(a[7], "dweight");
            dense_f32(dw, "dweight", {N}, device);
        } else if (w || given(a[3])) {
            dw = empty({N}, at::kFloat, device);
        }
        if (given(a[4])) {
            const at::Tensor &t = tensor(a[4], "dresidual");
            ld_res = rows(t, "dresidual", M, N, type, device);
            res = t.data_ptr();
        }
        if (given(a[6])) {
            dx = tensor(a[6], "dx");
            ld_dx = rows(dx, "dx", M, N, type, device);
        } else {
            dx = empty({M, N}, type, device);
        }
        if (!check(tile_rmsnorm_backward(dy.data_ptr(), h.data_ptr(), static_cast<const float *>(rstd), w, res,
                                         dx.data_ptr(), dw.defined() ? static_cast<float *>(dw.data_ptr()) : nullptr, M,
                                         N, ld_dy, ld_h, ld_res, ld_dx, code_of(type), wcode,
                                         static_cast<float>(offset), stream),
                   "tile_rmsnorm_backward"))
            return nullptr;
        written(dx);
        written(dw);
        return Py_BuildValue("(NN)", wrap(dx), wrap(dw));
    });
}

// (x, q, scales, zeros, group, x_scales, out, out_code) -> out; out_code: of a new
// out's type, -1 for x's (bf16 for e4m3)
PyObject *w4_matvec(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (!arity(n, 8)) return nullptr;
    const long group = PyLong_AsLong(a[4]), out_code = PyLong_AsLong(a[7]);
    if (PyErr_Occurred()) return nullptr;
    return guarded([&]() -> PyObject * {
        const at::Tensor &x = input(a[0], "x"), &q = input(a[1], "q");
        const at::ScalarType type = x.scalar_type();
        if (type != at::kHalf && type != at::kBFloat16 && type != at::kFloat8_e4m3fn)
            bad("x", "has an unsupported dtype");
        const at::Device device = x.device();
        const int64_t T = x.size(0), K = x.size(1), N = q.size(0);
        if (q.scalar_type() != at::kByte || q.size(1) * 2 != K || (group != 32 && group != 64 && group != 128))
            throw BadArgument("q must be uint8 with K / 2 columns and group be 32, 64 or 128");
        void *stream = stream_of(device);
        const int64_t ld_x = rows(x, "x", T, K, type, device);
        const int64_t ld_q = rows(q, "q", N, K / 2, at::kByte, device), groups = (K + group - 1) / group;
        const at::Tensor &s = tensor(a[2], "scales");
        if (!is_wide(s.scalar_type())) bad("scales", "has an unsupported dtype");
        const void *sp = dense(s, "scales", {N, groups}, device);
        const void *zp = nullptr;
        if (given(a[3])) {
            const at::Tensor &z = tensor(a[3], "zeros");
            if (z.scalar_type() != at::kByte) bad("zeros", "must be uint8");
            zp = dense(z, "zeros", {N, groups}, device);
        }
        const void *xs = nullptr;
        int x_group = 0;
        if (type == at::kFloat8_e4m3fn) {
            if (!given(a[5])) throw BadArgument("e4m3 x needs x_scales, T x 1 or T x ceil(K / 128)");
            const at::Tensor &t = tensor(a[5], "x_scales");
            x_group = t.dim() == 2 && t.size(1) != 1 ? 128 : 0;
            xs = dense_f32(t, "x_scales", {T, x_group ? (K + 127) / 128 : 1}, device);
        } else if (given(a[5])) {
            bad("x_scales", "need e4m3 x");
        }
        at::Tensor out;
        int64_t ld_out = 0;
        if (given(a[6])) {
            out = tensor(a[6], "out");
            if (!is_wide(out.scalar_type()) || (out_code >= 0 && code_of(out.scalar_type()) != out_code))
                bad("out", "has another type than out_dtype, or an unsupported one");
            ld_out = rows(out, "out", T, N, out.scalar_type(), device);
        } else {
            const at::ScalarType o = out_code == MBT_F16    ? at::kHalf
                                     : out_code == MBT_BF16 ? at::kBFloat16
                                     : out_code == MBT_F32  ? at::kFloat
                                     : type == at::kHalf    ? at::kHalf
                                                            : at::kBFloat16;
            out = empty({T, N}, o, device);
        }
        if (!check(tile_w4_matvec(x.data_ptr(), static_cast<const float *>(xs), static_cast<const uint8_t *>(q.data_ptr()),
                                  sp, static_cast<const uint8_t *>(zp), out.data_ptr(), T, N, K, ld_x, ld_q, ld_out,
                                  static_cast<int>(group), x_group, code_of(type), code_of(s.scalar_type()),
                                  code_of(out.scalar_type()), stream),
                   "tile_w4_matvec"))
            return nullptr;
        written(out);
        return THPVariable_Wrap(out);
    });
}

// (address of the descriptors, their sizes as a tuple, device index, parameter code,
// state code, grads, step, lr, beta1, beta2, eps, weight_decay, grad_scale, seed, the
// tensors that are written as a tuple, address of their addresses)
PyObject *adamw(PyObject *, PyObject *const *a, Py_ssize_t n) {
    double v[5];
    if (!arity(n, 16)) return nullptr;
    for (int i = 0; i < 5; ++i)
        if (!number(a[7 + i], &v[i])) return nullptr;
    auto *t = static_cast<mbt_adamw_tensor *>(PyLong_AsVoidPtr(a[0]));
    const void *const *addresses = static_cast<const void *const *>(PyLong_AsVoidPtr(a[15]));
    const long index = PyLong_AsLong(a[2]), pcode = PyLong_AsLong(a[3]), scode = PyLong_AsLong(a[4]);
    const long long step = PyLong_AsLongLong(a[6]);
    const unsigned long seed = PyLong_AsUnsignedLongMask(a[13]);
    if (PyErr_Occurred()) return nullptr;
    PyObject *grads = PySequence_Fast(a[5], "grads must be a sequence of tensors");
    if (!grads) return nullptr;
    PyObject *r = guarded([&]() -> PyObject * {
        // a tensor whose data were replaced meanwhile would be updated where it lay
        const Py_ssize_t all = PyTuple_GET_SIZE(a[14]);
        for (Py_ssize_t k = 0; k < all; ++k)
            if (tensor(PyTuple_GET_ITEM(a[14], k), "params").const_data_ptr() != addresses[k])
                throw BadArgument("tensor " + std::to_string(k) + " (params, exp_avg, exp_avg_sq, ... in turn) has "
                                  "other data than when the AdamwTensors was made");
        const Py_ssize_t count = PySequence_Fast_GET_SIZE(grads);
        if (count != PyTuple_GET_SIZE(a[1])) throw BadArgument("grads must have one tensor per parameter");
        const at::Device device(at::kCUDA, static_cast<c10::DeviceIndex>(index));
        void *stream = count ? stream_of(device) : nullptr;
        at::ScalarType type = at::kFloat;
        for (Py_ssize_t k = 0; k < count; ++k) {
            const at::Tensor &g = tensor(PySequence_Fast_GET_ITEM(grads, k), "grads");
            if (k == 0) type = g.scalar_type();
            if (!is_wide(type)) bad("grads", "have an unsupported dtype");
            if (g.scalar_type() != type || g.numel() != PyLong_AsLongLong(PyTuple_GET_ITEM(a[1], k)) ||
                g.device() != device || !g.is_contiguous())
                throw BadArgument("grads[" + std::to_string(k) + "] must be contiguous, of the first one's type and of " +
                                  "its parameter's size and device");
            t[k].grad = g.data_ptr();
        }
        const float *scale = nullptr;
        if (given(a[12])) {
            const at::Tensor &s = tensor(a[12], "grad_scale");
            if (s.numel() != 1) bad("grad_scale", "must hold one element");
            scale = static_cast<const float *>(dense_f32(s, "grad_scale", s.sizes(), device));
        }
        if (!check(tile_adamw(t, count, static_cast<int>(pcode), code_of(type), static_cast<int>(scode), step, v[0], v[1],
                              v[2], v[3], v[4], scale, static_cast<uint32_t>(seed), stream),
                   "tile_adamw"))
            return nullptr;
        for (Py_ssize_t k = 0; k < all; ++k) written(tensor(PyTuple_GET_ITEM(a[14], k), "params"));
        return Py_NewRef(Py_None);
    });
    Py_DECREF(grads);
    return r;
}

PyObject *set_error(PyObject *, PyObject *type) {
    Py_XSETREF(g_mbt_error, Py_NewRef(type));
    return Py_NewRef(Py_None);
}

PyMethodDef methods[] = {
    {"rmsnorm", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(rmsnorm)), METH_FASTCALL, nullptr},
    {"rmsnorm_backward", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(rmsnorm_backward)), METH_FASTCALL, nullptr},
    {"w4_matvec", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(w4_matvec)), METH_FASTCALL, nullptr},
    {"adamw", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(adamw)), METH_FASTCALL, nullptr},
    {"set_error", set_error, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_mbtile_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__mbtile_torch() { return PyModule_Create(&module); }
