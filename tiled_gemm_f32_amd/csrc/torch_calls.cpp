// The torch wrappers' common calls (experts.py, routing.py), checked, allocated and
// forwarded here: in Python that costs the host 9 to 12 us a call, as long as
// a small kernel runs; here 5 to 7.
//
// A function takes its wrapper's tensors and options and returns the wrapper's
// result, or an int (the C entry point's status, if it is an error), or None
// for any call outside the common case (outputs or a stream passed in, another
// current device, an argument that is not as it should be): the wrapper then
// takes it itself, and makes the message if there is something to refuse.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/hip/EmptyTensor.h>
#include <ATen/record_function.h>
#include <c10/core/impl/LocalDispatchKeySet.h>
#include <c10/core/impl/TorchDispatchModeTLS.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "gemm.h"

namespace {

using at::Tensor;

// Groups that the C entry points' 32-bit numbers hold.
constexpr int64_t kMostGroups = 0x7fffffff;

// A matrix (or, of three dimensions, a stack of them) with unit stride along its rows.
struct Matrix {
    const Tensor *t = nullptr;
    void *data = nullptr;
    int64_t groups = 1, rows = 0, cols = 0, ld = 0, stride = 0;
};

// Device that a call runs on and the stream it goes to, from the wrapper.
struct Where {
    int64_t device;
    gemm_stream_t stream;
};

const Tensor *tensor(PyObject *o) { return THPVariable_CheckExact(o) ? &THPVariable_Unpack(o) : nullptr; }

bool on(const Tensor &t, const Where &w) { return t.is_cuda() && t.get_device() == w.device; }

// False for anything but a plain non-empty matrix of `type` on the call's device.
bool matrix(PyObject *o, const Where &w, at::ScalarType type, Matrix &m, int dim = 2) {
    m.t = tensor(o);
    if (m.t == nullptr || m.t->dim() != dim || m.t->scalar_type() != type || !on(*m.t, w)) return false;
    const auto sizes = m.t->sizes(), strides = m.t->strides();
    m.rows = sizes[dim - 2];
    m.cols = sizes[dim - 1];
    if (dim == 3) {
        m.groups = sizes[0];
        m.stride = m.groups > 1 ? strides[0] : 0;
    }
    if (m.groups <= 0 || m.rows <= 0 || m.cols <= 0 || (m.cols > 1 && strides[dim - 1] != 1)) return false;
    if (m.groups > kMostGroups) return false;
    m.ld = m.rows > 1 ? strides[dim - 2] : m.cols;
    if (m.ld < m.cols) return false;
    m.data = m.t->data_ptr();
    return true;
}

bool vector(PyObject *o, const Where &w, at::ScalarType type, int64_t n, void *&data) {
    const Tensor *t = tensor(o);
    if (t == nullptr || t->dim() != 1 || t->size(0) != n || t->scalar_type() != type || !on(*t, w) ||
        (n > 1 && t->stride(0) != 1))
        return false;
    data = t->data_ptr();
    return true;
}

// fp32 or bf16, and the gemm_dtype that it is.
bool float_type(PyObject *o, at::ScalarType &type, int32_t &dtype) {
    const Tensor *t = tensor(o);
    if (t == nullptr) return false;
    type = t->scalar_type();
    dtype = type == at::kFloat ? GEMM_DTYPE_F32 : GEMM_DTYPE_BF16F32;
    return type == at::kFloat || type == at::kBFloat16;
}

// An output's type: `o` a torch.dtype, or None for `otherwise`.
bool out_type(PyObject *o, at::ScalarType otherwise, at::ScalarType &type, int32_t &kind) {
    if (o == Py_None) type = otherwise;
    else if (THPDtype_Check(o)) type = reinterpret_cast<THPDtype *>(o)->scalar_type;
    else return false;
    kind = type == at::kFloat ? GEMM_OUT_F32 : type == at::kBFloat16 ? GEMM_OUT_BF16 : GEMM_OUT_FP8;
    return type == at::kFloat || type == at::kBFloat16 || type == at::kFloat8_e4m3fn;
}

// Whether anything but the allocation would see or change an allocation that goes through torch's dispatcher:
// a dispatch mode or another key that this thread's state adds (functional transforms, tracing), a profiler's
// callbacks, or the filling of uninitialised memory in deterministic mode.
bool watched() {
    const auto &global = at::globalContext();
    return c10::impl::TorchDispatchModeTLS::any_modes_set() ||
           !(c10::impl::tls_local_dispatch_key_set().included_ - c10::default_included_set).empty() ||
           at::hasCallbacks() ||
           (global.deterministicAlgorithms() && global.deterministicFillUninitializedMemory());
}

// The dispatcher takes as long as the allocation itself (0.3 us a result), so it is passed by where nobody watches.
Tensor allocate(const Tensor &like, at::IntArrayRef sizes, at::IntArrayRef strides, at::ScalarType type) {
    if (watched()) return at::empty_strided(sizes, strides, like.options().dtype(type));
    return at::detail::empty_strided_cuda(sizes, strides, type, like.device());
}
Tensor make(const Tensor &like, int64_t rows, int64_t cols, int64_t ld, at::ScalarType type) {
    return allocate(like, {rows, cols}, {ld, 1}, type);
}
Tensor row_of(const Tensor &like, int64_t n, at::ScalarType type) { return allocate(like, {n}, {1}, type); }
int64_t blocks(int64_t n) { return (n + GEMM_SCALE_BLOCK - 1) / GEMM_SCALE_BLOCK; }
int64_t on16(int64_t n) { return (n + 15) / 16 * 16; }

PyObject *none() { Py_RETURN_NONE; }
PyObject *give(gemm_status st, const Tensor &a) { return st == GEMM_OK ? THPVariable_Wrap(a) : PyLong_FromLong(st); }
PyObject *give(gemm_status st, const Tensor &a, const Tensor &b, const Tensor &c) {
    return st == GEMM_OK ? Py_BuildValue("NNN", THPVariable_Wrap(a), THPVariable_Wrap(b), THPVariable_Wrap(c))
                         : PyLong_FromLong(st);
}
PyObject *give(gemm_status st, const Tensor &a, const Tensor &b) {
    return st == GEMM_OK ? Py_BuildValue("NN", THPVariable_Wrap(a), THPVariable_Wrap(b)) : PyLong_FromLong(st);
}

// The last two arguments of every function.
bool where(PyObject *const *args, Py_ssize_t n, Py_ssize_t want, Where &w) {
    if (n != want) return false;
    w.device = PyLong_AsLongLong(args[n - 2]);
    w.stream = PyLong_AsVoidPtr(args[n - 1]);
    if (PyErr_Occurred() == nullptr) return true;
    PyErr_Clear();
    return false;
}

// quantize(x, block_rows, device, stream)
PyObject *quantize(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    Where w;
    Matrix x;
    at::ScalarType type;
    int32_t dtype;
    if (!where(args, n, 4, w) || !float_type(args[0], type, dtype) || !matrix(args[0], w, type, x)) return none();
    const int64_t block_rows = PyLong_AsLongLong(args[1]);
    if (block_rows != 1 && block_rows != GEMM_SCALE_BLOCK) {
        PyErr_Clear();
        return none();
    }
    const int64_t scale_rows = (x.rows + block_rows - 1) / block_rows;
    const Tensor codes = make(*x.t, x.rows, x.cols, on16(x.cols), at::kFloat8_e4m3fn);
    const Tensor scales = make(*x.t, scale_rows, blocks(x.cols), blocks(x.cols), at::kFloat);
    return give(gemm_quantize(dtype, (int32_t)block_rows, x.rows, x.cols, x.data, x.ld,
                              static_cast<uint8_t *>(codes.data_ptr()), on16(x.cols),
                              static_cast<float *>(scales.data_ptr()), blocks(x.cols), w.stream),
                codes, scales);
    END_HANDLE_TH_ERRORS
}

// rms_norm(x, weight, residual, eps, out_dtype, device, stream)
PyObject *rms_norm(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    Where w;
    Matrix x, r;
    void *weight;
    at::ScalarType type, out;
    int32_t dtype, kind;
    if (!where(args, n, 7, w) || !float_type(args[0], type, dtype) || !matrix(args[0], w, type, x) ||
        !vector(args[1], w, type, x.cols, weight) || !PyFloat_Check(args[3]) || !out_type(args[4], type, out, kind))
        return none();
    const bool with = args[2] != Py_None;
    if (with && (!matrix(args[2], w, type, r) || r.rows != x.rows || r.cols != x.cols)) return none();
    const bool fp8 = kind == GEMM_OUT_FP8;
    Tensor sum, scales;
    if (with) sum = make(*x.t, x.rows, x.cols, x.cols, type);
    const int64_t ldo = fp8 ? on16(x.cols) : x.cols;
    const Tensor y = make(*x.t, x.rows, x.cols, ldo, out);
    if (fp8) scales = make(*x.t, x.rows, blocks(x.cols), blocks(x.cols), at::kFloat);
    const gemm_status st = gemm_rms_norm(
        dtype, x.rows, x.cols, x.data, x.ld, with ? r.data : nullptr, r.ld, weight, (float)PyFloat_AS_DOUBLE(args[3]),
        with ? sum.data_ptr() : nullptr, with ? x.cols : 0, kind, y.data_ptr(), ldo,
        fp8 ? static_cast<float *>(scales.data_ptr()) : nullptr, fp8 ? blocks(x.cols) : 0, w.stream);
    if (st != GEMM_OK) return PyLong_FromLong(st);
    PyObject *total = with ? THPVariable_Wrap(sum) : Py_NewRef(args[0]);
    return Py_BuildValue("NNN", THPVariable_Wrap(y), total, fp8 ? THPVariable_Wrap(scales) : none());
    END_HANDLE_TH_ERRORS
}

// rms_norm_backward(dy, summed, weight, dsum, eps, device, stream)
PyObject *rms_norm_backward(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    Where w;
    Matrix dy, s, ds;
    void *weight;
    at::ScalarType type;
    int32_t dtype;
    if (!where(args, n, 7, w) || !float_type(args[0], type, dtype) || !matrix(args[0], w, type, dy) ||
        !matrix(args[1], w, type, s) || s.rows != dy.rows || s.cols != dy.cols ||
        !vector(args[2], w, type, dy.cols, weight) || !PyFloat_Check(args[4]))
        return none();
    const bool with = args[3] != Py_None;
    if (with && (!matrix(args[3], w, type, ds) || ds.rows != dy.rows || ds.cols != dy.cols)) return none();
    const Tensor dx = make(*dy.t, dy.rows, dy.cols, dy.cols, type);
    const Tensor dweight = row_of(*dy.t, dy.cols, at::kFloat);
    const int64_t need = gemm_rms_norm_workspace_size(dy.rows, dy.cols);
    const Tensor space = row_of(*dy.t, need, at::kByte);
    return give(gemm_rms_norm_backward(dtype, dy.rows, dy.cols, dy.data, dy.ld, s.data, s.ld, weight,
                                       (float)PyFloat_AS_DOUBLE(args[4]), with ? ds.data : nullptr, ds.ld,
                                       dx.data_ptr(), dy.cols, static_cast<float *>(dweight.data_ptr()),
                                       space.data_ptr(), need, w.stream),
                dx, dweight);
    END_HANDLE_TH_ERRORS
}

// Scales of fp8 operands: a's one for each row and block, b's one for each tile of B as it is stored.
bool block_scales(PyObject *a, PyObject *b, const Where &w, const Matrix &A, const Matrix &B, bool transposed, int dim,
                  gemm_block_scales &sc) {
    const Tensor *ta = tensor(a), *tb = tensor(b);
    if (ta == nullptr || tb == nullptr || ta->scalar_type() != at::kFloat || tb->scalar_type() != at::kFloat ||
        !on(*ta, w) || !on(*tb, w) || ta->dim() != 2 || tb->dim() != dim || ta->size(0) != A.rows ||
        ta->size(1) != blocks(A.cols) || tb->size(dim - 2) != blocks(B.rows) || tb->size(dim - 1) != blocks(B.cols) ||
        (dim == 3 && tb->size(0) != B.groups))
        return false;
    const int64_t rows = tb->stride(dim - 2), cols = tb->stride(dim - 1);
    sc = {static_cast<const float *>(ta->data_ptr()), ta->stride(0), ta->stride(1),
          static_cast<const float *>(tb->data_ptr()), transposed ? rows : cols, transposed ? cols : rows,
          dim == 3 ? tb->stride(0) : 0};
    return true;
}

// op_b "T" or "N".
bool transposes(PyObject *o, bool &t) {
    if (!PyUnicode_Check(o) || PyUnicode_GET_LENGTH(o) != 1) return false;
    const Py_UCS4 c = PyUnicode_READ_CHAR(o, 0);
    t = c == 'T';
    return c == 'T' || c == 'N';
}

// block_gemm(A, B, a_scales, b_scales, op_b, alpha, out_dtype, device, stream)
PyObject *block_gemm(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    Where w;
    Matrix A, B;
    bool t;
    at::ScalarType out;
    int32_t kind;
    gemm_block_scales sc;
    if (!where(args, n, 9, w) || !matrix(args[0], w, at::kFloat8_e4m3fn, A) ||
        !matrix(args[1], w, at::kFloat8_e4m3fn, B) || !transposes(args[4], t) || !PyFloat_Check(args[5]) ||
        !out_type(args[6], at::kBFloat16, out, kind) || kind == GEMM_OUT_FP8 || (t ? B.cols : B.rows) != A.cols ||
        !block_scales(args[2], args[3], w, A, B, t, 2, sc))
        return none();
    const int64_t N = t ? B.rows : B.cols;
    const Tensor y = make(*A.t, A.rows, N, N, out);
    return give(gemm_block_scaled(t ? GEMM_OP_T : GEMM_OP_N, A.rows, N, A.cols, (float)PyFloat_AS_DOUBLE(args[5]),
                                  static_cast<const uint8_t *>(A.data), A.ld, static_cast<const uint8_t *>(B.data), B.ld,
                                  &sc, kind, y.data_ptr(), N, w.stream),
                y);
    END_HANDLE_TH_ERRORS
}

// grouped_gemm(A, B, ends, a_scales, b_scales, op_b, alpha, out_dtype, device, stream)
PyObject *grouped_gemm(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    Where w;
    Matrix A, B;
    bool t;
    void *ends;
    at::ScalarType type, out;
    int32_t dtype, kind;
    gemm_block_scales sc;
    if (!where(args, n, 10, w) || tensor(args[0]) == nullptr) return none();
    const bool fp8 = tensor(args[0])->scalar_type() == at::kFloat8_e4m3fn;
    if (fp8) {
        type = at::kFloat8_e4m3fn;
        dtype = GEMM_DTYPE_FP8F32;
    } else if (!float_type(args[0], type, dtype)) {
        return none();
    }
    if (!matrix(args[0], w, type, A) || !matrix(args[1], w, type, B, 3) ||
        !vector(args[2], w, at::kInt, B.groups, ends) || !transposes(args[5], t) || !PyFloat_Check(args[6]) ||
        !out_type(args[7], fp8 ? at::kBFloat16 : type, out, kind) || kind == GEMM_OUT_FP8 ||
        (t ? B.cols : B.rows) != A.cols)
        return none();
    if (fp8 ? !block_scales(args[3], args[4], w, A, B, t, 3, sc) : args[3] != Py_None || args[4] != Py_None)
        return none();
    const int64_t N = t ? B.rows : B.cols;
    const Tensor y = make(*A.t, A.rows, N, N, out);
    return give(gemm_grouped(dtype, t ? GEMM_OP_T : GEMM_OP_N, (int32_t)B.groups, static_cast<const int32_t *>(ends),
                             A.rows, N, A.cols, (float)PyFloat_AS_DOUBLE(args[6]), A.data, A.ld, B.data, B.ld, B.stride,
                             fp8 ? &sc : nullptr, kind, y.data_ptr(), N, w.stream),
                y);
    END_HANDLE_TH_ERRORS
}

// grouped_wgrad(dy, x, ends, alpha, device, stream)
PyObject *grouped_wgrad(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    Where w;
    Matrix dy, x;
    void *ends;
    at::ScalarType type;
    int32_t dtype;
    if (!where(args, n, 6, w) || !float_type(args[0], type, dtype) || !matrix(args[0], w, type, dy) ||
        !matrix(args[1], w, type, x) || x.rows != dy.rows || tensor(args[2]) == nullptr ||
        tensor(args[2])->dim() != 1 || !PyFloat_Check(args[3]))
        return none();
    const int64_t groups = tensor(args[2])->size(0), N = dy.cols, K = x.cols;
    if (groups <= 0 || groups > kMostGroups || !vector(args[2], w, at::kInt, groups, ends)) return none();
    const Tensor out = allocate(*dy.t, {groups, N, K}, {N * K, K, 1}, at::kFloat);
    return give(gemm_grouped_wgrad(dtype, (int32_t)groups, static_cast<const int32_t *>(ends), dy.rows, N, K,
                                   (float)PyFloat_AS_DOUBLE(args[3]), dy.data, dy.ld, x.data, x.ld, 0.0f,
                                   static_cast<float *>(out.data_ptr()), K, groups > 1 ? N * K : 0, w.stream),
                out);
    END_HANDLE_TH_ERRORS
}

// layer_norm(x, weight, bias, residual, eps, out_dtype, device, stream)
PyObject *layer_norm(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    Where w;
    Matrix x, r;
    void *weight, *bias = nullptr;
    at::ScalarType type, out;
    int32_t dtype, kind;
    if (!where(args, n, 8, w) || !float_type(args[0], type, dtype) || !matrix(args[0], w, type, x) ||
        !vector(args[1], w, type, x.cols, weight) || (args[2] != Py_None && !vector(args[2], w, type, x.cols, bias)) ||
        !PyFloat_Check(args[4]))
        return none();
    if (THPDtype_Check(args[5]) && reinterpret_cast<THPDtype *>(args[5])->scalar_type == at::kChar) {
        out = at::kChar;
        kind = GEMM_OUT_INT8;
    } else if (!out_type(args[5], type, out, kind)) {
        return none();
    }
    const bool with = args[3] != Py_None;
    if (with && (!matrix(args[3], w, type, r) || r.rows != x.rows || r.cols != x.cols)) return none();
    const bool fp8 = kind == GEMM_OUT_FP8, int8 = kind == GEMM_OUT_INT8;
    Tensor sum, scales;
    if (with) sum = make(*x.t, x.rows, x.cols, x.cols, type);
    const int64_t ldo = fp8 || int8 ? on16(x.cols) : x.cols, lds = fp8 ? blocks(x.cols) : 1;
    const Tensor y = make(*x.t, x.rows, x.cols, ldo, out);
    if (fp8) scales = make(*x.t, x.rows, lds, lds, at::kFloat);
    if (int8) scales = row_of(*x.t, x.rows, at::kFloat);
    const gemm_status st = gemm_layer_norm(
        dtype, x.rows, x.cols, x.data, x.ld, with ? r.data : nullptr, r.ld, weight, bias,
        (float)PyFloat_AS_DOUBLE(args[4]), with ? sum.data_ptr() : nullptr, with ? x.cols : 0, kind, y.data_ptr(), ldo,
        fp8 || int8 ? static_cast<float *>(scales.data_ptr()) : nullptr, lds, w.stream);
    if (st != GEMM_OK) return PyLong_FromLong(st);
    PyObject *total = with ? THPVariable_Wrap(sum) : Py_NewRef(args[0]);
    return Py_BuildValue("NNN", THPVariable_Wrap(y), total, fp8 || int8 ? THPVariable_Wrap(scales) : none());
    END_HANDLE_TH_ERRORS
}

// layer_norm_backward(dy, summed, weight, dsum, eps, device, stream)
PyObject *layer_norm_backward(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    Where w;
    Matrix dy, s, ds;
    void *weight;
    at::ScalarType type;
    int32_t dtype;
    if (!where(args, n, 7, w) || !float_type(args[0], type, dtype) || !matrix(args[0], w, type, dy) ||
        !matrix(args[1], w, type, s) || s.rows != dy.rows || s.cols != dy.cols ||
        !vector(args[2], w, type, dy.cols, weight) || !PyFloat_Check(args[4]))
        return none();
    const bool with = args[3] != Py_None;
    if (with && (!matrix(args[3], w, type, ds) || ds.rows != dy.rows || ds.cols != dy.cols)) return none();
    const Tensor dx = make(*dy.t, dy.rows, dy.cols, dy.cols, type);
    const Tensor dweight = row_of(*dy.t, dy.cols, at::kFloat), dbias = row_of(*dy.t, dy.cols, at::kFloat);
    const int64_t need = gemm_layer_norm_workspace_size(dy.rows, dy.cols);
    const Tensor space = row_of(*dy.t, need, at::kByte);
    return give(gemm_layer_norm_backward(dtype, dy.rows, dy.cols, dy.data, dy.ld, s.data, s.ld, weight,
                                         (float)PyFloat_AS_DOUBLE(args[4]), with ? ds.data : nullptr, ds.ld,
                                         dx.data_ptr(), dy.cols, static_cast<float *>(dweight.data_ptr()),
                                         static_cast<float *>(dbias.data_ptr()), space.data_ptr(), need, w.stream),
                dx, dweight, dbias);
    END_HANDLE_TH_ERRORS
}

// quantize_int8(x, device, stream)
PyObject *quantize_int8(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    Where w;
    Matrix x;
    at::ScalarType type;
    int32_t dtype;
    if (!where(args, n, 3, w) || !float_type(args[0], type, dtype) || !matrix(args[0], w, type, x)) return none();
    const Tensor codes = make(*x.t, x.rows, x.cols, on16(x.cols), at::kChar);
    const Tensor scales = row_of(*x.t, x.rows, at::kFloat);
    return give(gemm_quantize_int8(dtype, x.rows, x.cols, x.data, x.ld, static_cast<int8_t *>(codes.data_ptr()),
                                   on16(x.cols), static_cast<float *>(scales.data_ptr()), w.stream),
                codes, scales);
    END_HANDLE_TH_ERRORS
}

// A value a column of the product, for each group: [groups,] n floats.
bool columns(PyObject *o, const Where &w, int dim, int64_t groups, int64_t n, const float *&data, int64_t &col,
             int64_t &group) {
    const Tensor *t = tensor(o);
    if (t == nullptr || t->scalar_type() != at::kFloat || t->dim() != dim || !on(*t, w) || t->size(dim - 1) != n ||
        (dim == 2 && t->size(0) != groups))
        return false;
    data = static_cast<const float *>(t->data_ptr());
    col = t->stride(dim - 1);
    group = dim == 2 && groups > 1 ? t->stride(0) : 0;
    return true;
}

// int8_gemm(A, B, a_scales, b_scales, ends, bias, op_b, out_dtype, device, stream)
PyObject *int8_gemm(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    Where w;
    Matrix A, B;
    bool t;
    void *ends = nullptr;
    at::ScalarType out;
    int32_t kind;
    gemm_int8_scales sc = {};
    int64_t group;
    if (!where(args, n, 10, w)) return none();
    const bool grouped = args[4] != Py_None;
    if (!matrix(args[0], w, at::kChar, A) || !matrix(args[1], w, at::kChar, B, grouped ? 3 : 2) ||
        (grouped && !vector(args[4], w, at::kInt, B.groups, ends)) || !transposes(args[6], t) ||
        !out_type(args[7], at::kBFloat16, out, kind) || kind == GEMM_OUT_FP8 || (t ? B.cols : B.rows) != A.cols)
        return none();
    const int64_t N = t ? B.rows : B.cols;
    const int dim = grouped ? 2 : 1;
    if (!columns(args[2], w, 1, 1, A.rows, sc.a, sc.a_row, group) ||
        !columns(args[3], w, dim, B.groups, N, sc.b, sc.b_col, sc.b_group))
        return none();
    if (args[5] != Py_None) {
        int64_t col;
        if (!columns(args[5], w, dim, B.groups, N, sc.bias, col, sc.bias_group) || (N > 1 && col != 1)) return none();
    }
    const Tensor y = make(*A.t, A.rows, N, N, out);
    return give(gemm_int8(t ? GEMM_OP_T : GEMM_OP_N, (int32_t)B.groups, static_cast<const int32_t *>(ends), A.rows, N,
                          A.cols, static_cast<const int8_t *>(A.data), A.ld, static_cast<const int8_t *>(B.data), B.ld,
                          B.stride, &sc, kind, y.data_ptr(), N, w.stream),
                y);
    END_HANDLE_TH_ERRORS
}

// expert_plan(experts, groups, device, stream)
PyObject *expert_plan(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    Where w;
    Matrix e;
    if (!where(args, n, 4, w) || tensor(args[0]) == nullptr || !PyLong_CheckExact(args[1])) return none();
    const at::ScalarType type = tensor(args[0])->scalar_type();
    const int64_t groups = PyLong_AsLongLong(args[1]);
    if (PyErr_Occurred() != nullptr) {
        PyErr_Clear();
        return none();
    }
    if ((type != at::kInt && type != at::kLong) || !matrix(args[0], w, type, e) || groups < 1 || groups > 1 << 30 ||
        e.cols > 1 << 30 || e.rows > 1 << 30)
        return none();
    const Tensor order = row_of(*e.t, e.rows * e.cols, at::kInt), ends = row_of(*e.t, groups, at::kInt);
    const Tensor place = make(*e.t, e.rows, e.cols, e.cols, at::kInt);
    const int64_t need = gemm_expert_plan_workspace_size(e.rows, (int32_t)e.cols, (int32_t)groups);
    Tensor space;
    if (need > 0) space = row_of(*e.t, need, at::kByte);
    return give(gemm_expert_plan(type == at::kLong ? 8 : 4, e.rows, (int32_t)e.cols, (int32_t)groups, e.data, e.ld,
                                 static_cast<int32_t *>(order.data_ptr()), static_cast<int32_t *>(place.data_ptr()),
                                 static_cast<int32_t *>(ends.data_ptr()), need > 0 ? space.data_ptr() : nullptr, need,
                                 w.stream),
                order, place, ends);
    END_HANDLE_TH_ERRORS
}

// A plan's places, tokens x top without padding, and (o not null) its last end.
bool places(PyObject *o, const Where &w, int64_t tokens, Matrix &place) {
    return matrix(o, w, at::kInt, place) && place.rows == tokens && place.ld == place.cols && place.cols <= 1 << 30;
}
bool last_end(PyObject *o, const Where &w, const int32_t *&last) {
    const Tensor *t = tensor(o);
    void *ends;
    if (t == nullptr || t->dim() != 1 || t->size(0) < 1 || !vector(o, w, at::kInt, t->size(0), ends)) return false;
    last = static_cast<const int32_t *>(ends) + t->size(0) - 1;
    return true;
}
bool weights_of(PyObject *o, const Where &w, const Matrix &place, Matrix &m) {
    return matrix(o, w, at::kFloat, m) && m.rows == place.rows && m.cols == place.cols;
}

// dispatch(x, place, ends, scales, device, stream)
PyObject *dispatch(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    Where w;
    Matrix x, place, sc;
    const int32_t *last;
    if (!where(args, n, 6, w) || tensor(args[0]) == nullptr) return none();
    const at::ScalarType type = tensor(args[0])->scalar_type();
    if ((type != at::kFloat && type != at::kBFloat16 && type != at::kFloat8_e4m3fn && type != at::kChar) ||
        !matrix(args[0], w, type, x) || !places(args[1], w, x.rows, place) || !last_end(args[2], w, last))
        return none();
    const int64_t rows = place.rows * place.cols;
    const bool with = args[3] != Py_None;
    Tensor out_scales;
    if (with) {
        const Tensor *t = tensor(args[3]);
        if (t == nullptr) return none();
        if (t->dim() == 1) {
            void *data;
            if (!vector(args[3], w, at::kFloat, x.rows, data)) return none();
            sc.data = data;
            sc.cols = sc.ld = 1;
            out_scales = row_of(*x.t, rows, at::kFloat);
        } else {
            if (!matrix(args[3], w, at::kFloat, sc) || sc.rows != x.rows) return none();
            out_scales = make(*x.t, rows, sc.cols, sc.cols, at::kFloat);
        }
    }
    const int64_t bytes = (int64_t)x.t->element_size(), ldo = bytes == 1 ? on16(x.cols) : x.cols;
    const Tensor out = make(*x.t, rows, x.cols, ldo, type);
    const gemm_status st = gemm_dispatch(
        (int32_t)bytes, x.rows, (int32_t)place.cols, x.cols, x.data, x.ld, static_cast<const int32_t *>(place.data), last,
        rows, out.data_ptr(), ldo, sc.cols, static_cast<const float *>(sc.data), sc.ld,
        with ? static_cast<float *>(out_scales.data_ptr()) : nullptr, sc.cols, w.stream);
    return with ? give(st, out, out_scales) : give(st, out);
    END_HANDLE_TH_ERRORS
}

// combine(rows, place, weights, residual, device, stream)
PyObject *combine(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    Where w;
    Matrix rows, place, share, r;
    at::ScalarType type;
    int32_t dtype;
    if (!where(args, n, 6, w) || !float_type(args[0], type, dtype) || !matrix(args[0], w, type, rows) ||
        tensor(args[1]) == nullptr || tensor(args[1])->dim() != 2 ||
        !places(args[1], w, tensor(args[1])->size(0), place))
        return none();
    if (args[2] != Py_None && !weights_of(args[2], w, place, share)) return none();
    if (args[3] != Py_None && (!matrix(args[3], w, type, r) || r.rows != place.rows || r.cols != rows.cols))
        return none();
    const Tensor out = make(*rows.t, place.rows, rows.cols, rows.cols, type);
    return give(gemm_combine(dtype, place.rows, (int32_t)place.cols, rows.cols, rows.data, rows.ld, rows.rows,
                             static_cast<const int32_t *>(place.data), static_cast<const float *>(share.data), share.ld,
                             r.data, r.ld, out.data_ptr(), rows.cols, w.stream),
                out);
    END_HANDLE_TH_ERRORS
}

// combine_backward(dout, rows, place, weights, ends, device, stream)
PyObject *combine_backward(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    Where w;
    Matrix d, rows, place, share;
    const int32_t *last;
    at::ScalarType type;
    int32_t dtype;
    if (!where(args, n, 7, w) || !float_type(args[0], type, dtype) || !matrix(args[0], w, type, d) ||
        !matrix(args[1], w, type, rows) || rows.cols != d.cols || !places(args[2], w, d.rows, place) ||
        !weights_of(args[3], w, place, share) || !last_end(args[4], w, last))
        return none();
    const Tensor drows = make(*d.t, rows.rows, rows.cols, rows.cols, type);
    const Tensor dweights = make(*d.t, place.rows, place.cols, place.cols, at::kFloat);
    return give(gemm_combine_backward(dtype, d.rows, (int32_t)place.cols, d.cols, d.data, d.ld, rows.data, rows.ld,
                                      rows.rows, static_cast<const int32_t *>(place.data), last,
                                      static_cast<const float *>(share.data), share.ld, drows.data_ptr(), rows.cols,
                                      static_cast<float *>(dweights.data_ptr()), place.cols, w.stream),
                drows, dweights);
    END_HANDLE_TH_ERRORS
}

#define CALL(name) {#name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {CALL(quantize), CALL(rms_norm), CALL(rms_norm_backward), CALL(block_gemm),
                         CALL(grouped_gemm), CALL(grouped_wgrad), CALL(layer_norm), CALL(layer_norm_backward),
                         CALL(quantize_int8), CALL(int8_gemm), CALL(expert_plan), CALL(dispatch), CALL(combine),
                         CALL(combine_backward), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_torch_calls", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__torch_calls() { return PyModule_Create(&module); }
