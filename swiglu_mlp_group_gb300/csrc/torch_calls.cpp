// torch_calls.cpp -- the Python binding's calls of the 4-bit operators and of the
// block norm, for arguments that are all in order: the checks, the outputs and the
// call without the interpreter, which takes some 9 us of a small call (a norm of 16
// tokens 13.8 us in Python, the launch itself 1.8).  Where anything is not as it should
// be (a type, a shape, a device, a status) a function returns None, and the Python
// function of the same name says what.  Nothing is computed or kept here.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "ck.h"

namespace {

using at::Tensor;
constexpr auto kBf16 = at::kBFloat16;
constexpr auto kU8 = at::kByte;

// A call's arguments, read one by one; `ok` turns false at the first that is not in order.
struct Reader {
    PyObject *const *args;
    bool ok = true;
    int dev = -1;

    PyObject *object(int i) const { return args[i]; }
    // a tensor, or null for None
    const Tensor *tensor(int i) {
        if (args[i] == Py_None) return nullptr;
        if (!THPVariable_CheckExact(args[i])) {
            ok = false;
            return nullptr;
        }
        const Tensor *t = &THPVariable_Unpack(args[i]);
        if (!t->defined() || !t->is_cuda() || t->layout() != at::kStrided || (dev >= 0 && t->get_device() != dev)) {
            ok = false;
            return nullptr;
        }
        return t;
    }
    // the tensor that says where the call runs: the current device
    const Tensor *first(int i) {
        const Tensor *t = tensor(i);
        if (!t || !ok) {
            ok = false;
            return nullptr;
        }
        dev = t->get_device();
        if (dev != c10::cuda::current_device()) ok = false;
        return t;
    }
    double number(int i) {
        if (PyFloat_CheckExact(args[i])) return PyFloat_AS_DOUBLE(args[i]);
        if (PyLong_CheckExact(args[i])) {
            const double v = PyLong_AsDouble(args[i]);
            if (!PyErr_Occurred()) return v;
            PyErr_Clear();
        }
        ok = false;
        return 0.;
    }
    int64_t integer(int i) {
        if (PyLong_CheckExact(args[i])) {
            const int64_t v = PyLong_AsLongLong(args[i]);
            if (!PyErr_Occurred()) return v;
            PyErr_Clear();
        }
        ok = false;
        return 0;
    }
    // which of two words: 0 or 1
    int choice(int i, const char *zero, const char *one) {
        if (PyUnicode_CheckExact(args[i])) {
            if (PyUnicode_CompareWithASCIIString(args[i], zero) == 0) return 0;
            if (PyUnicode_CompareWithASCIIString(args[i], one) == 0) return 1;
        }
        ok = false;
        return 0;
    }
    void want(bool c) { ok = ok && c; }

    // Data of contiguous tensors of a type and shape, or null.
    const void *flat(const Tensor *t, at::ScalarType type) {
        if (!t) return nullptr;
        want(t->scalar_type() == type && t->is_contiguous());
        return t->const_data_ptr();
    }
    // The same of a tensor that is written: memory that it still shares with the tensor it
    // was lazily cloned from becomes its own.  (What may be the same tensor, x or a
    // residual, is asked for its address after it.)
    void *written(const Tensor *t, at::ScalarType type) {
        if (!t) return nullptr;
        want(t->scalar_type() == type && t->is_contiguous());
        return ok ? t->mutable_data_ptr() : nullptr;
    }
    const void *vector(int i, at::ScalarType type, int64_t n) {
        const Tensor *t = tensor(i);
        if (t) want(t->dim() == 1 && t->size(0) == n);
        return flat(t, type);
    }
    const void *matrix(int i, at::ScalarType type, int64_t rows, int64_t cols) {
        const Tensor *t = tensor(i);
        if (t) want(t->dim() == 2 && t->size(0) == rows && t->size(1) == cols);
        return flat(t, type);
    }
    // Elements between rows that may lie apart.
    int64_t rows(const Tensor &t, at::ScalarType type) {
        if (t.dim() != 2 || t.scalar_type() != type || (t.stride(1) != 1 && t.size(1) > 1)) {
            ok = false;
            return 0;
        }
        return t.size(0) > 1 ? t.stride(0) : t.size(1);
    }
    int64_t rows(const Tensor &t, at::ScalarType type, int64_t n, int64_t cols) {
        const int64_t ld = rows(t, type);
        want(ok && t.size(0) == n && t.size(1) == cols);
        return ld;
    }
};

ck_stream_t stream_of(int dev) { return reinterpret_cast<ck_stream_t>(c10::cuda::getCurrentCUDAStream(dev).stream()); }

// A new tensor, from the allocator without the dispatcher (0.3 us of 1.2).
Tensor fresh(const Tensor &like, at::ScalarType type, at::IntArrayRef shape) {
    return Tensor(at::detail::empty_cuda(shape, type, like.device(), std::nullopt));
}

int64_t tiled_bytes(int format, int64_t rows, int64_t K) {
    return (rows + 127) / 128 * (format == CK_FP4_NV ? (K + 63) / 64 : (K + 127) / 128) * 512;
}

// An output: the tensor given (checked), or a new one.  `keep` owns the new one.
struct Out {
    Tensor keep;
    PyObject *given = nullptr;
    void *data = nullptr;
    PyObject *result() { return given ? Py_NewRef(given) : THPVariable_Wrap(std::move(keep)); }
};
Out out_matrix(Reader &r, int i, const Tensor &like, at::ScalarType type, int64_t rows, int64_t cols) {
    Out o;
    if (r.object(i) != Py_None) {
        o.given = r.object(i);
        const Tensor *t = r.tensor(i);
        if (t) r.want(t->dim() == 2 && t->size(0) == rows && t->size(1) == cols);
        o.data = r.written(t, type);
    } else if (r.ok) {
        o.keep = fresh(like, type, {rows, cols});
        o.data = o.keep.mutable_data_ptr();
    }
    return o;
}
Out out_scales(Reader &r, int i, const Tensor &like, int64_t bytes) {
    Out o;
    if (r.object(i) != Py_None) {
        o.given = r.object(i);
        const Tensor *t = r.tensor(i);
        if (t) r.want(t->numel() >= bytes);
        o.data = r.written(t, kU8);
    } else if (r.ok) {
        o.keep = fresh(like, kU8, {bytes});
        o.data = o.keep.mutable_data_ptr();
    }
    return o;
}
// Rows that may lie apart, of x's shape.
Out out_rows(Reader &r, int i, const Tensor &like, int64_t rows, int64_t cols, int64_t &ld) {
    Out o;
    if (r.object(i) != Py_None) {
        o.given = r.object(i);
        const Tensor *t = r.tensor(i);
        if (t) {
            ld = r.rows(*t, kBf16, rows, cols);
            if (r.ok) o.data = t->mutable_data_ptr();
        }
    } else if (r.ok) {
        ld = cols;
        o.keep = fresh(like, kBf16, {rows, cols});
        o.data = o.keep.mutable_data_ptr();
    }
    return o;
}

// Codes [rows, K / 2] and tiled scales of an operand.
struct Operand {
    const void *codes = nullptr, *scales = nullptr;
    int64_t rows = 0, K = 0;
};
Operand operand(Reader &r, int codes, int scales, int format) {
    Operand o;
    const Tensor *c = r.tensor(codes), *s = r.tensor(scales);
    if (!c || !s || c->dim() != 2) {
        r.ok = false;
        return o;
    }
    o.rows = c->size(0), o.K = 2 * c->size(1);
    o.codes = r.flat(c, kU8), o.scales = r.flat(s, kU8);
    r.want(s->numel() >= tiled_bytes(format, o.rows, o.K));
    return o;
}

struct Workspace {
    Tensor keep;
    void *data = nullptr;
    size_t bytes = 0;
};
Workspace workspace(Reader &r, int i, const Tensor &like, size_t need) {
    Workspace w;
    const Tensor *t = r.tensor(i);
    if (!r.ok) return w;
    if (t) {
        r.want(t->is_contiguous());
        if (!r.ok) return w;
    } else {
        w.keep = fresh(like, kU8, {static_cast<int64_t>(need > 16 ? need : 16)});
        t = &w.keep;
    }
    w.data = t->mutable_data_ptr(), w.bytes = t->nbytes();
    return w;
}

// Both forms of the norm: arguments at the same places up to h_out's.
struct NormArgs {
    const Tensor *x = nullptr, *branch = nullptr;
    int64_t T = 0, H = 0, ldx = 0, ldb = 0, ldm = 0, ldh = 0, per_group = 0;
    const void *mod[3] = {}, *weights[3] = {};  // gate, scale, shift; weight, bias, post_weight
    double x_factor = 1., branch_factor = 1., eps = 0.;
    int norm = 0;
    ck_dtype wdt = CK_BF16;
    Out h;
    bool h_is_x = false;

    void read(Reader &r, int branch_i, int post, int gate, int xf, int bf, int norm_i, int weight, int bias, int scale, int shift,
              int group, int eps_i, int h_out) {
        x = r.first(0), branch = r.tensor(branch_i);
        if (!r.ok) return;
        ldx = r.rows(*x, kBf16);
        if (!r.ok) return;
        T = x->size(0), H = x->size(1);
        if (branch) ldb = r.rows(*branch, kBf16, T, H);
        x_factor = r.number(xf), branch_factor = r.number(bf), eps = r.number(eps_i);
        norm = r.choice(norm_i, "rms", "layer") ? CK_NORM_LAYER : CK_NORM_RMS;
        per_group = r.integer(group);
        if (!r.ok) return;
        const int64_t groups = per_group > 0 && per_group < T ? (T + per_group - 1) / per_group : 1;
        // several groups: rows of gate, scale and shift at one stride, each row's own memory (an
        // expanded one's stride is 0); else only the first row is read
        ldm = H;
        bool first_mod = true;
        const int mods[3] = {gate, scale, shift};
        for (int i = 0; i < 3; ++i)
            if (const Tensor *t = r.tensor(mods[i])) {
                const int64_t ld = r.rows(*t, kBf16);
                r.want(r.ok && t->size(0) >= groups && t->size(1) == H);
                if (groups > 1) {
                    r.want(ld >= H && (first_mod || ld == ldm));
                    ldm = ld, first_mod = false;
                }
                mod[i] = t->const_data_ptr();
            }
        const int ws[3] = {weight, bias, post};
        at::ScalarType type = kBf16;
        bool seen = false;
        for (int i = 0; i < 3; ++i)
            if (const Tensor *t = r.tensor(ws[i])) {
                if (!seen && t->scalar_type() == at::kFloat) type = at::kFloat, wdt = CK_F32;
                seen = true;
                weights[i] = r.vector(ws[i], type, H);
            }
        if (!r.ok) return;
        if (r.object(h_out) == Py_None && !branch && x_factor == 1.)
            h_is_x = true;  // without a branch and a factor the stream itself is h
        else
            h = out_rows(r, h_out, *x, T, H, ldh);
    }
    PyObject *h_result(Reader &r) { return h_is_x ? Py_NewRef(r.object(0)) : h.result(); }
};

#define CK_TRY(N)             \
    if (n != N) Py_RETURN_NONE; \
    Reader r{args};           \
    try
#define CK_CATCH                         \
    catch (const std::exception &) { \
        Py_RETURN_NONE;                  \
    }
#define CK_CALL(...)                         \
    ck_status st;                            \
    Py_BEGIN_ALLOW_THREADS st = __VA_ARGS__; \
    Py_END_ALLOW_THREADS if (st != CK_OK) Py_RETURN_NONE

// (x, branch, post_weight, gate, x_factor, branch_factor, norm, weight, bias, scale, shift, tokens_per_group, eps, h_out, n_out)
PyObject *block_norm(PyObject *, PyObject *const *args, Py_ssize_t n) {
    CK_TRY(15) {
        NormArgs a;
        a.read(r, 1, 2, 3, 4, 5, 6, 7, 8, 9, 10, 11, 12, 13);
        if (!r.ok) Py_RETURN_NONE;
        int64_t ldn = 0;
        Out o = out_rows(r, 14, *a.x, a.T, a.H, ldn);
        if (!r.ok) Py_RETURN_NONE;
        const ck_stream_t s = stream_of(r.dev);
        const void *x = a.x->const_data_ptr(), *b = a.branch ? a.branch->const_data_ptr() : nullptr;
        CK_CALL(ck_block_norm(x, a.ldx, b, a.ldb, a.T, a.H, a.weights[2], a.mod[0], a.mod[1], a.mod[2], a.ldm, a.per_group,
                              static_cast<float>(a.x_factor), static_cast<float>(a.branch_factor), static_cast<ck_norm>(a.norm),
                              a.weights[0], a.weights[1], a.wdt, static_cast<float>(a.eps), a.h.data, a.ldh, o.data, ldn, s));
        return Py_BuildValue("(NN)", a.h_result(r), o.result());
    }
    CK_CATCH
}

// (x, branch, fmt, n_scale, post_weight, gate, x_factor, branch_factor, norm, weight, bias, scale, shift, tokens_per_group,
//  eps, h_out, codes, scales)
PyObject *block_norm_fp4(PyObject *, PyObject *const *args, Py_ssize_t n) {
    CK_TRY(18) {
        NormArgs a;
        const int f = r.choice(2, "mx", "nv") ? CK_FP4_NV : CK_FP4_MX;
        const double t = r.number(3);
        a.read(r, 1, 4, 5, 6, 7, 8, 9, 10, 11, 12, 13, 14, 15);
        if (!r.ok || a.H % 32 != 0) Py_RETURN_NONE;
        Out codes = out_matrix(r, 16, *a.x, kU8, a.T, a.H / 2);
        Out scales = out_scales(r, 17, *a.x, tiled_bytes(f, a.T, a.H));
        if (!r.ok) Py_RETURN_NONE;
        const ck_stream_t s = stream_of(r.dev);
        const void *x = a.x->const_data_ptr(), *b = a.branch ? a.branch->const_data_ptr() : nullptr;
        CK_CALL(ck_block_norm_fp4(x, a.ldx, b, a.ldb, a.T, a.H, a.weights[2], a.mod[0], a.mod[1], a.mod[2], a.ldm, a.per_group,
                                  static_cast<float>(a.x_factor), static_cast<float>(a.branch_factor),
                                  static_cast<ck_norm>(a.norm), a.weights[0], a.weights[1], a.wdt, static_cast<float>(a.eps),
                                  a.h.data, a.ldh, static_cast<ck_fp4_format>(f), static_cast<float>(t), codes.data, scales.data, s));
        return Py_BuildValue("(NNN)", a.h_result(r), codes.result(), scales.result());
    }
    CK_CATCH
}

// (codes, scales, W, w_scales, fmt, alpha, bias, residual, out)
PyObject *fp4_gemm(PyObject *, PyObject *const *args, Py_ssize_t n) {
    CK_TRY(9) {
        const Tensor *x = r.first(0);
        if (!r.ok) Py_RETURN_NONE;
        const int f = r.choice(4, "mx", "nv") ? CK_FP4_NV : CK_FP4_MX;
        const Operand a = operand(r, 0, 1, f), w = operand(r, 2, 3, f);
        const double alpha = r.number(5);
        if (!r.ok || a.K != w.K) Py_RETURN_NONE;
        const void *bias = r.vector(6, kBf16, w.rows);
        Out y = out_matrix(r, 8, *x, kBf16, a.rows, w.rows);
        const void *residual = r.matrix(7, kBf16, a.rows, w.rows);
        if (!r.ok) Py_RETURN_NONE;
        const ck_stream_t s = stream_of(r.dev);
        CK_CALL(ck_fp4_gemm(a.codes, a.scales, a.rows, a.K, static_cast<ck_fp4_format>(f), w.codes, w.scales, w.rows,
                            static_cast<float>(alpha), bias, residual, y.data, s));
        return y.result();
    }
    CK_CATCH
}

// (x, W, w_scales, fmt, x_scale, w_scale, bias, act, out, workspace, residual)
PyObject *fp4_linear(PyObject *, PyObject *const *args, Py_ssize_t n) {
    CK_TRY(11) {
        const Tensor *x = r.first(0);
        if (!r.ok) Py_RETURN_NONE;
        const int f = r.choice(3, "mx", "nv") ? CK_FP4_NV : CK_FP4_MX;
        const int act = r.choice(7, "none", "swiglu") ? CK_ACT_SWIGLU : CK_ACT_NONE;
        const double tx = r.number(4), tw = r.number(5);
        const int64_t ldx = r.rows(*x, kBf16);
        const Operand w = operand(r, 1, 2, f);
        if (!r.ok) Py_RETURN_NONE;
        if (act == CK_ACT_SWIGLU && x->size(1) % 2 != 0) Py_RETURN_NONE;
        const int64_t M = x->size(0), K = act == CK_ACT_SWIGLU ? x->size(1) / 2 : x->size(1);
        r.want(K == w.K);
        const void *bias = r.vector(6, kBf16, w.rows);
        Out y = out_matrix(r, 8, *x, kBf16, M, w.rows);
        const void *residual = r.matrix(10, kBf16, M, w.rows);
        const Workspace ws = workspace(r, 9, *x, ck_fp4_linear_workspace_bytes(M, K, static_cast<ck_fp4_format>(f)));
        if (!r.ok) Py_RETURN_NONE;
        const ck_stream_t s = stream_of(r.dev);
        const void *px = x->const_data_ptr();
        CK_CALL(ck_fp4_linear(px, M, K, ldx, static_cast<ck_input_act>(act), static_cast<ck_fp4_format>(f), static_cast<float>(tx),
                              w.codes, w.scales, static_cast<float>(tw), w.rows, bias, residual, y.data, ws.data, ws.bytes, s));
        return y.result();
    }
    CK_CATCH
}

// (x, Wgu, gu_scales, Wd, d_scales, fmt, x_scale, gate_up_scale, act_scale, down_scale, bgu, bd, residual, out, workspace)
PyObject *fp4_swiglu_mlp(PyObject *, PyObject *const *args, Py_ssize_t n) {
    CK_TRY(15) {
        const Tensor *x = r.first(0);
        if (!r.ok) Py_RETURN_NONE;
        const int f = r.choice(5, "mx", "nv") ? CK_FP4_NV : CK_FP4_MX;
        double t[4];
        for (int i = 0; i < 4; ++i) t[i] = r.number(6 + i);
        const Operand gu = operand(r, 1, 2, f), d = operand(r, 3, 4, f);
        if (!r.ok || x->dim() != 2) Py_RETURN_NONE;
        const int64_t M = x->size(0), H = x->size(1), I = d.K;
        r.want(gu.K == H && d.rows == H && gu.rows == 2 * I);
        const void *bgu = r.vector(10, kBf16, 2 * I), *bd = r.vector(11, kBf16, H);
        Out y = out_matrix(r, 13, *x, kBf16, M, H);
        const void *px = r.flat(x, kBf16), *residual = r.matrix(12, kBf16, M, H);
        const Workspace ws = workspace(r, 14, *x, ck_fp4_swiglu_mlp_workspace_bytes(M, H, I, static_cast<ck_fp4_format>(f)));
        if (!r.ok) Py_RETURN_NONE;
        const ck_stream_t s = stream_of(r.dev);
        CK_CALL(ck_fp4_swiglu_mlp(px, M, H, I, static_cast<ck_fp4_format>(f), static_cast<float>(t[0]), gu.codes, gu.scales,
                                  static_cast<float>(t[1]), bgu, static_cast<float>(t[2]), d.codes, d.scales,
                                  static_cast<float>(t[3]), bd, residual, y.data, ws.data, ws.bytes, s));
        return y.result();
    }
    CK_CATCH
}

// (x, fmt, scale, act, codes, scales)
PyObject *fp4_quantize(PyObject *, PyObject *const *args, Py_ssize_t n) {
    CK_TRY(6) {
        const Tensor *x = r.first(0);
        if (!r.ok) Py_RETURN_NONE;
        const int f = r.choice(1, "mx", "nv") ? CK_FP4_NV : CK_FP4_MX;
        const double t = r.number(2);
        const int act = r.choice(3, "none", "swiglu") ? CK_ACT_SWIGLU : CK_ACT_NONE;
        const bool f32 = x->scalar_type() == at::kFloat;
        const int64_t ldx = r.rows(*x, f32 ? at::kFloat : kBf16);
        if (!r.ok) Py_RETURN_NONE;
        if (act == CK_ACT_SWIGLU && x->size(1) % 2 != 0) Py_RETURN_NONE;
        const int64_t M = x->size(0), K = act == CK_ACT_SWIGLU ? x->size(1) / 2 : x->size(1);
        const int64_t bytes = static_cast<int64_t>(ck_fp4_scale_bytes(static_cast<ck_fp4_format>(f), M, K));
        if (bytes == 0) Py_RETURN_NONE;
        Out codes = out_matrix(r, 4, *x, kU8, M, K / 2), scales = out_scales(r, 5, *x, bytes);
        if (!r.ok) Py_RETURN_NONE;
        const ck_stream_t s = stream_of(r.dev);
        const void *px = x->const_data_ptr();
        CK_CALL(ck_fp4_quantize(px, f32 ? CK_F32 : CK_BF16, M, K, ldx, static_cast<ck_input_act>(act),
                                static_cast<ck_fp4_format>(f), static_cast<float>(t), codes.data, scales.data, s));
        return Py_BuildValue("(NN)", codes.result(), scales.result());
    }
    CK_CATCH
}

PyMethodDef kMethods[] = {
#define CK_METHOD(NAME) {#NAME, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(NAME)), METH_FASTCALL, nullptr}
    CK_METHOD(block_norm), CK_METHOD(block_norm_fp4), CK_METHOD(fp4_gemm),
    CK_METHOD(fp4_linear), CK_METHOD(fp4_swiglu_mlp), CK_METHOD(fp4_quantize),
#undef CK_METHOD
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "ck_torch_calls", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_ck_torch_calls() { return PyModule_Create(&kModule); }
