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
#include <vector>

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

// The new results of a call, of which the small ones share an allocation (each costs as much
// as the rest of a call of one token): want() for all of them, then give() for each.  A
// result over kMost bytes has its own, so that large memory is not held by others.
class Together {
public:
    explicit Together(at::Device device) : device_(device) {}
    void want(int64_t elements, at::ScalarType type) {
        if (elements * size(type) <= kMost) total_ += padded(elements * size(type));
    }
    at::Tensor give(at::IntArrayRef shape, at::ScalarType type) {
        int64_t bytes = size(type);
        for (const int64_t n : shape) bytes *= n;
        if (bytes > kMost) return empty(shape, type, device_);
        if (!flat_.defined()) flat_ = empty({total_}, at::kByte, device_);
        at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(flat_.storage()), flat_.key_set(),
                                                                c10::scalarTypeToTypeMeta(type));
        t.unsafeGetTensorImpl()->set_storage_offset(used_ / size(type));
        t.unsafeGetTensorImpl()->set_sizes_contiguous(shape);
        used_ += padded(bytes);
        return t;
    }

private:
    static constexpr int64_t kMost = 64 << 10;
    static int64_t size(at::ScalarType type) { return static_cast<int64_t>(c10::elementSize(type)); }
    static int64_t padded(int64_t bytes) { return (bytes + 127) / 128 * 128; }
    at::Device device_;
    at::Tensor flat_;
    int64_t total_ = 0, used_ = 0;
};

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

// (x, weight, bias, residual, eps, weight_offset, quant, out, scales, residual_out, mean, rstd)
// -> (out, scales, residual_out, mean, rstd); quant as in mbtile.h
PyObject *layernorm(PyObject *, PyObject *const *a, Py_ssize_t n) {
    double eps, offset;
    if (!arity(n, 12) || !number(a[4], &eps) || !number(a[5], &offset)) return nullptr;
    const long quant = PyLong_AsLong(a[6]);
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
        void *w = nullptr, *b = nullptr, *res = nullptr, *ro = nullptr, *sc = nullptr;
        int wcode = 0;
        at::Tensor out, scales, residual_out;
        if (given(a[1])) {
            const at::Tensor &t = tensor(a[1], "weight");
            if (!is_wide(t.scalar_type())) bad("weight", "has an unsupported dtype");
            w = dense(t, "weight", {N}, device);
            wcode = code_of(t.scalar_type());
        }
        if (given(a[2])) {
            const at::Tensor &t = tensor(a[2], "bias");
            if (!given(a[1])) bad("bias", "needs a weight");
            if (code_of(t.scalar_type()) != wcode) bad("bias", "must have weight's type");
            b = dense(t, "bias", {N}, device);
        }
        const bool quantised = quant != MBT_QUANT_NONE;
        const at::ScalarType out_type = quantised ? at::kFloat8_e4m3fn : type;
        const int64_t groups = quant > 0 ? (N + quant - 1) / quant : 1;
        Together fresh(device);
        if (given(a[3]) && !given(a[9])) fresh.want(M * N, type);
        if (!given(a[7])) fresh.want(M * N, out_type);
        if (quantised && !given(a[8])) fresh.want(M * groups, at::kFloat);
        for (int k = 10; k < 12; ++k)
            if (!given(a[k])) fresh.want(M, at::kFloat);
        if (given(a[3])) {
            const at::Tensor &t = tensor(a[3], "residual");
            ld_res = rows(t, "residual", M, N, type, device);
            res = t.data_ptr();
            if (given(a[9])) {
                residual_out = tensor(a[9], "residual_out");
                ld_ro = rows(residual_out, "residual_out", M, N, type, device);
            } else {
                residual_out = fresh.give({M, N}, type);
            }
            ro = residual_out.data_ptr();
        } else if (given(a[9])) {
            bad("residual_out", "needs a residual");
        }
        if (given(a[7])) {
            out = tensor(a[7], "out");
            ld_out = rows(out, "out", M, N, out_type, device);
        } else {
            out = fresh.give({M, N}, out_type);
        }
        if (quantised) {
            if (given(a[8])) {
                scales = tensor(a[8], "scales");
                sc = dense_f32(scales, "scales", {M, groups}, device);
            } else {
                scales = fresh.give({M, groups}, at::kFloat);
                sc = scales.data_ptr();
            }
        } else if (given(a[8])) {
            bad("scales", "need quant");
        }
        at::Tensor stats[2];
        for (int k = 0; k < 2; ++k) {
            const char *name = k ? "rstd" : "mean";
            if (given(a[10 + k])) {
                stats[k] = tensor(a[10 + k], name);
                dense_f32(stats[k], name, {M}, device);
            } else {
                stats[k] = fresh.give({M}, at::kFloat);
            }
        }
        if (!check(tile_layernorm(x.data_ptr(), res, w, b, out.data_ptr(), ro, static_cast<float *>(sc),
                                  static_cast<float *>(stats[0].data_ptr()), static_cast<float *>(stats[1].data_ptr()),
                                  M, N, ld_x, ld_res, ld_out, ld_ro, code_of(type), wcode, static_cast<int>(quant),
                                  static_cast<float>(eps), static_cast<float>(offset), stream),
                   "tile_layernorm"))
            return nullptr;
        for (const at::Tensor *t : {&out, &scales, &residual_out, &stats[0], &stats[1]}) written(*t);
        return Py_BuildValue("(NNNNN)", wrap(out), wrap(scales), wrap(residual_out), wrap(stats[0]), wrap(stats[1]));
    });
}

// (dy, h, mean, rstd, weight, dresidual, weight_offset, bias, dx, dweight, dbias) -> (dx, dweight, dbias)
PyObject *layernorm_backward(PyObject *, PyObject *const *a, Py_ssize_t n) {
    double offset;
    if (!arity(n, 11) || !number(a[6], &offset)) return nullptr;
    const int bias = PyObject_IsTrue(a[7]);
    if (bias < 0) return nullptr;
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
        const void *mean = dense_f32(tensor(a[2], "mean"), "mean", {M}, device);
        const void *rstd = dense_f32(tensor(a[3], "rstd"), "rstd", {M}, device);
        void *w = nullptr, *res = nullptr;
        int64_t ld_res = 0, ld_dx = 0;
        int wcode = 0;
        at::Tensor dx, dw, db;
        const bool new_dw = !given(a[9]) && given(a[4]), new_db = !given(a[10]) && given(a[4]) && bias;
        Together fresh(device);
        if (!given(a[8])) fresh.want(M * N, type);
        if (new_dw) fresh.want(N, at::kFloat);
        if (new_db) fresh.want(N, at::kFloat);
        if (given(a[4])) {
            const at::Tensor &t = tensor(a[4], "weight");
            if (!is_wide(t.scalar_type())) bad("weight", "has an unsupported dtype");
            w = dense(t, "weight", {N}, device);
            wcode = code_of(t.scalar_type());
        }
        if (given(a[9])) {
            dw = tensor(a[9], "dweight");
            dense_f32(dw, "dweight", {N}, device);
        } else if (new_dw) {
            dw = fresh.give({N}, at::kFloat);
        }
        if (given(a[10])) {
            db = tensor(a[10], "dbias");
            dense_f32(db, "dbias", {N}, device);
        } else if (new_db) {
            db = fresh.give({N}, at::kFloat);
        }
        if (given(a[5])) {
            const at::Tensor &t = tensor(a[5], "dresidual");
            ld_res = rows(t, "dresidual", M, N, type, device);
            res = t.data_ptr();
        }
        if (given(a[8])) {
            dx = tensor(a[8], "dx");
            ld_dx = rows(dx, "dx", M, N, type, device);
        } else {
            dx = fresh.give({M, N}, type);
        }
        if (!check(tile_layernorm_backward(dy.data_ptr(), h.data_ptr(), static_cast<const float *>(mean),
                                           static_cast<const float *>(rstd), w, res, dx.data_ptr(),
                                           dw.defined() ? static_cast<float *>(dw.data_ptr()) : nullptr,
                                           db.defined() ? static_cast<float *>(db.data_ptr()) : nullptr, M, N, ld_dy,
                                           ld_h, ld_res, ld_dx, code_of(type), wcode, static_cast<float>(offset), stream),
                   "tile_layernorm_backward"))
            return nullptr;
        for (const at::Tensor *t : {&dx, &dw, &db}) written(*t);
        return Py_BuildValue("(NNN)", wrap(dx), wrap(dw), wrap(db));
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

// Scales of an M x K matrix in 4-bit floats, tiled.
std::vector<int64_t> mx4_scales_shape(int64_t M, int64_t K, long block) {
    return {(M + 127) / 128, (K / block + 3) / 4, 512};
}

const float *tensor_scale(PyObject *o, at::Device device) {
    if (!given(o)) return nullptr;
    const at::Tensor &t = tensor(o, "tensor_scale");
    if (t.numel() != 1) bad("tensor_scale", "must hold one element");
    return static_cast<const float *>(dense_f32(t, "tensor_scale", t.sizes(), device));
}

// An Mx4 from its parts: q, scales, tensor scale.
struct Mx4Parts {
    at::Device device;
    int64_t rows, K, ld;
    const uint8_t *q, *scales;
    const float *ts;
    Mx4Parts(PyObject *const *a, long block, const char *name) : device(at::kCPU) {
        const at::Tensor &t = input(a[0], name);
        if (t.scalar_type() != at::kByte) bad(name, "must hold uint8 codes");
        device = t.device();
        rows = t.size(0);
        K = 2 * t.size(1);
        if (K % 32 != 0 || (block != 16 && block != 32)) bad(name, "must have a multiple of 32 columns and blocks of 16 or 32");
        ld = ::rows(t, name, rows, K / 2, at::kByte, device);
        q = static_cast<const uint8_t *>(t.data_ptr());
        const at::Tensor &s = tensor(a[1], "scales");
        if (s.scalar_type() != at::kByte) bad("scales", "must be uint8");
        scales = static_cast<const uint8_t *>(dense(s, "scales", mx4_scales_shape(rows, K, block), device));
        ts = tensor_scale(a[2], device);
        if (ts && block != 16) bad("tensor_scale", "goes with blocks of 16");
    }
};

at::ScalarType type_of(long code) {
    return code == MBT_F16 ? at::kHalf : code == MBT_F32 ? at::kFloat : at::kBFloat16;
}

// (x, tensor_scale, block, q, scales) -> (q, scales)
PyObject *mx4_quantize(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (!arity(n, 5)) return nullptr;
    const long block = PyLong_AsLong(a[2]);
    if (PyErr_Occurred()) return nullptr;
    return guarded([&]() -> PyObject * {
        const at::Tensor &x = input(a[0], "x");
        const at::ScalarType type = x.scalar_type();
        if (!is_wide(type)) bad("x", "has an unsupported dtype");
        const at::Device device = x.device();
        const int64_t M = x.size(0), K = x.size(1);
        if (K % 32 != 0) bad("x", "must have a multiple of 32 columns");
        void *stream = stream_of(device);
        const int64_t ld_x = rows(x, "x", M, K, type, device);
        const float *ts = tensor_scale(a[1], device);
        if (ts && block != 16) bad("tensor_scale", "goes with blocks of 16");
        const auto shape = mx4_scales_shape(M, K, block);
        Together fresh(device);
        if (!given(a[3])) fresh.want(M * (K / 2), at::kByte);
        if (!given(a[4])) fresh.want(shape[0] * shape[1] * shape[2], at::kByte);
        at::Tensor q, s;
        int64_t ld_q = 0;
        if (given(a[3])) {
            q = tensor(a[3], "q");
            ld_q = rows(q, "q", M, K / 2, at::kByte, device);
        } else {
            q = fresh.give({M, K / 2}, at::kByte);
        }
        if (given(a[4])) {
            s = tensor(a[4], "scales");
            if (s.scalar_type() != at::kByte) bad("scales", "must be uint8");
            dense(s, "scales", shape, device);
        } else {
            s = fresh.give(shape, at::kByte);
        }
        if (!check(tile_mx4_quantize(x.data_ptr(), ts, static_cast<uint8_t *>(q.data_ptr()),
                                     static_cast<uint8_t *>(s.data_ptr()), M, K, ld_x, ld_q, static_cast<int>(block),
                                     code_of(type), stream),
                   "tile_mx4_quantize"))
            return nullptr;
        written(q);
        written(s);
        return Py_BuildValue("(NN)", wrap(q), wrap(s));
    });
}

// (q, scales, tensor_scale, block, out, out_code) -> out
PyObject *mx4_dequantize(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (!arity(n, 6)) return nullptr;
    const long block = PyLong_AsLong(a[3]), code = PyLong_AsLong(a[5]);
    if (PyErr_Occurred()) return nullptr;
    return guarded([&]() -> PyObject * {
        const Mx4Parts m(a, block, "q");
        void *stream = stream_of(m.device);
        at::Tensor out;
        int64_t ld_out = 0;
        if (given(a[4])) {
            out = tensor(a[4], "out");
            ld_out = rows(out, "out", m.rows, m.K, type_of(code), m.device);
        } else {
            out = empty({m.rows, m.K}, type_of(code), m.device);
        }
        if (!check(tile_mx4_dequantize(m.q, m.scales, m.ts, out.data_ptr(), m.rows, m.K, m.ld, ld_out,
                                       static_cast<int>(block), static_cast<int>(code), stream),
                   "tile_mx4_dequantize"))
            return nullptr;
        written(out);
        return THPVariable_Wrap(out);
    });
}

// (a's q, scales, tensor_scale, b's q, scales, tensor_scale, block, out, out_code) -> out
PyObject *mx4_matmul(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (!arity(n, 9)) return nullptr;
    const long block = PyLong_AsLong(a[6]), code = PyLong_AsLong(a[8]);
    if (PyErr_Occurred()) return nullptr;
    return guarded([&]() -> PyObject * {
        const Mx4Parts l(a, block, "a"), r(a + 3, block, "b");
        if (l.K != r.K || l.device != r.device) throw BadArgument("a and b must have the same number of columns and device");
        void *stream = stream_of(l.device);
        at::Tensor out;
        int64_t ld_out = 0;
        if (given(a[7])) {
            out = tensor(a[7], "out");
            ld_out = rows(out, "out", l.rows, r.rows, type_of(code), l.device);
        } else {
            out = empty({l.rows, r.rows}, type_of(code), l.device);
        }
        if (!check(tile_mx4_matmul(l.q, l.scales, l.ts, r.q, r.scales, r.ts, out.data_ptr(), l.rows, r.rows, l.K, l.ld,
                                   r.ld, ld_out, static_cast<int>(block), static_cast<int>(code), stream),
                   "tile_mx4_matmul"))
            return nullptr;
        written(out);
        return THPVariable_Wrap(out);
    });
}

// A tensor of one fp32 element.
at::Tensor scalar(PyObject *o, const char *name, at::Device device) {
    const at::Tensor &t = tensor(o, name);
    if (t.numel() != 1) bad(name, "must hold one element");
    dense_f32(t, name, t.sizes(), device);
    return t;
}

// (grads, grad_scale, max_norm, eps, norm, scale, in_place) -> (norm, scale)
PyObject *grad_norm(PyObject *, PyObject *const *a, Py_ssize_t n) {
    double most, eps;
    if (!arity(n, 7) || !number(a[2], &most) || !number(a[3], &eps)) return nullptr;
    const int in_place = PyObject_IsTrue(a[6]);
    if (in_place < 0) return nullptr;
    PyObject *grads = PySequence_Fast(a[0], "grads must be a sequence of tensors");
    if (!grads) return nullptr;
    PyObject *r = guarded([&]() -> PyObject * {
        const Py_ssize_t count = PySequence_Fast_GET_SIZE(grads);
        at::Device device(at::kCUDA, 0);
        if (count) {
            device = tensor(PySequence_Fast_GET_ITEM(grads, 0), "grads").device();
            if (!device.is_cuda()) bad("grads", "must be CUDA tensors");
        } else {
            device.set_index(c10::cuda::current_device());
        }
        std::vector<mbt_grad> list(static_cast<size_t>(count));
        for (Py_ssize_t k = 0; k < count; ++k) {
            const at::Tensor &g = tensor(PySequence_Fast_GET_ITEM(grads, k), "grads");
            if (!is_wide(g.scalar_type()) || g.device() != device || g.layout() != at::kStrided ||
                !(g.is_contiguous() || g.is_non_overlapping_and_dense()))
                throw BadArgument("grads[" + std::to_string(k) + "] must be a dense fp16, bf16 or fp32 tensor on the first one's device");
            list[static_cast<size_t>(k)] = {g.data_ptr(), g.numel(), code_of(g.scalar_type()), 0};
        }
        void *stream = stream_of(device);
        const float *gs = nullptr;
        at::Tensor factor;
        if (given(a[1])) {
            factor = scalar(a[1], "grad_scale", device);
            gs = static_cast<const float *>(factor.data_ptr());
        }
        Together fresh(device);
        for (int k = 4; k < 6; ++k)
            if (!given(a[k])) fresh.want(1, at::kFloat);
        const at::Tensor norm = given(a[4]) ? scalar(a[4], "norm", device) : fresh.give({}, at::kFloat);
        const at::Tensor scale = given(a[5]) ? scalar(a[5], "scale", device) : fresh.give({}, at::kFloat);
        float *to = static_cast<float *>(scale.data_ptr());
        const int rc = (in_place ? tile_grad_clip : tile_grad_norm)(list.data(), count, gs, static_cast<float>(most),
                                                                    static_cast<float>(eps),
                                                                    static_cast<float *>(norm.data_ptr()), to, stream);
        if (!check(rc, in_place ? "tile_grad_clip" : "tile_grad_norm")) return nullptr;
        written(norm);
        written(scale);
        if (in_place)
            for (Py_ssize_t k = 0; k < count; ++k) written(tensor(PySequence_Fast_GET_ITEM(grads, k), "grads"));
        return Py_BuildValue("(NN)", wrap(norm), wrap(scale));
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
    {"mx4_quantize", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(mx4_quantize)), METH_FASTCALL, nullptr},
    {"mx4_dequantize", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(mx4_dequantize)), METH_FASTCALL, nullptr},
    {"mx4_matmul", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(mx4_matmul)), METH_FASTCALL, nullptr},
    {"grad_norm", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(grad_norm)), METH_FASTCALL, nullptr},
    {"layernorm", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(layernorm)), METH_FASTCALL, nullptr},
    {"layernorm_backward", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(layernorm_backward)), METH_FASTCALL, nullptr},
    {"set_error", set_error, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_mbtile_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__mbtile_torch() { return PyModule_Create(&module); }
