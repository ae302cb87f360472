// binding.cpp -- native argument marshalling for the entry points whose calls
// carry many tensors: checks dtype, device, shape and strides, allocates what
// the caller did not give, and calls the C ABI on the device's current stream.
// No arithmetic.  api.py holds the public functions and their documentation.
//
// A call's checks and allocations take 1-2 us here; the same steps in Python
// took 15-40 us, several times what the kernels of a decode step run.
//
// The C entry points come as addresses from the loaded library (bind), so this
// module links against torch alone.
#include <Python.h>

#include <ATen/EmptyTensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <optional>
#include <string>

#include "rmsnorm.h"

namespace {

using at::Tensor;

// ---- errors ----------------------------------------------------------------
struct PyError {};  // a Python exception is set

[[noreturn]] void fail(PyObject *type, const char *fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    std::vsnprintf(buf, sizeof(buf), fmt, ap);
    va_end(ap);
    PyErr_SetString(type, buf);
    throw PyError{};
}

std::string shape_str(c10::IntArrayRef s) {
    std::string r = "(";
    for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
    return r + (s.size() == 1 ? ",)" : ")");
}

const char *dtype_str(at::ScalarType t) {
    return t == at::kHalf      ? "torch.float16"
           : t == at::kBFloat16 ? "torch.bfloat16"
           : t == at::kFloat    ? "torch.float32"
           : t == at::kDouble   ? "torch.float64"
           : t == at::kInt      ? "torch.int32"
           : t == at::kLong     ? "torch.int64"
           : t == at::kBool     ? "torch.bool"
           : t == at::kChar     ? "torch.int8"
           : t == at::kFloat8_e4m3fn ? "torch.float8_e4m3fn"
                                : c10::toString(t);
}

// ---- the library -----------------------------------------------------------
PyObject *g_check = nullptr;  // check(name, status): raises for a status other than 0

// The entry points as rmsnorm.h declares them.
#define ENTRY(name) decltype(&rmsnorm_##name) c_##name
ENTRY(block_fwd);
ENTRY(block_vjp_ws);
ENTRY(block_vjp_workspace_size);
ENTRY(rope);
ENTRY(rope_kv_append_ex);
ENTRY(rope_axes);
ENTRY(kv_append);
ENTRY(kv_read);
ENTRY(fwd_q8);
ENTRY(kv_release);
ENTRY(kv_plan);
#undef ENTRY

void check_status(const char *name, int st) {
    if (st == 0) return;
    PyObject *r = PyObject_CallFunction(g_check, "si", name, st);
    Py_XDECREF(r);
    if (r) PyErr_SetString(PyExc_RuntimeError, "library call failed");
    throw PyError{};
}

// ---- arguments -------------------------------------------------------------
struct Args {
    PyObject *const *a;
    Py_ssize_t n;

    const Tensor &tensor(int i, const char *name) const {
        if (!THPVariable_Check(a[i])) fail(PyExc_TypeError, "%s must be a tensor", name);
        return THPVariable_Unpack(a[i]);
    }
    const Tensor *optional(int i, const char *name) const {
        return a[i] == Py_None ? nullptr : &tensor(i, name);
    }
    double number(int i) const {
        const double v = PyFloat_AsDouble(a[i]);
        if (v == -1.0 && PyErr_Occurred()) throw PyError{};
        return v;
    }
    int64_t integer(int i) const {
        const long long v = PyLong_AsLongLong(a[i]);
        if (v == -1 && PyErr_Occurred()) throw PyError{};
        return v;
    }
    bool truth(int i) const {
        const int v = PyObject_IsTrue(a[i]);
        if (v < 0) throw PyError{};
        return v != 0;
    }
};

void *ptr(const Tensor *t) { return t && t->numel() ? t->data_ptr() : nullptr; }

// A tensor of the caller's that the call wrote: an in-place change to autograd, which
// then refuses a backward pass through what was there.
void wrote(const Tensor *t) {
    if (t && !t->is_inference()) t->unsafeGetTensorImpl()->bump_version();
}
template <typename... P> void wrote(const Tensor *t, const P *...more) {
    wrote(t);
    wrote(more...);
}

void need_cuda(const Tensor &t) {
    if (!t.is_cuda()) fail(PyExc_ValueError, "tensors must be CUDA tensors (there is no CPU path)");
}

int dtype_code(const Tensor &t) {
    switch (t.scalar_type()) {
        case at::kHalf: return 0;
        case at::kBFloat16: return 1;
        case at::kFloat: return 2;
        default: fail(PyExc_TypeError, "unsupported dtype %s (fp16 or bf16 or fp32)", dtype_str(t.scalar_type()));
    }
}

void same_kind(const char *name, const Tensor &t, const Tensor &ref) {
    if (t.scalar_type() != ref.scalar_type() || t.device() != ref.device())
        fail(PyExc_ValueError, "%s must be %s on %s", name, dtype_str(ref.scalar_type()),
             ref.device().str().c_str());
}

// A [..., D] tensor whose rows are contiguous and a common stride apart.
struct Rows {
    int64_t rows, D, ld;
};

Rows rows_ld(const char *name, const Tensor &t) {
    const int64_t dim = t.dim();
    if (dim < 1) fail(PyExc_ValueError, "%s must have at least one dimension", name);
    need_cuda(t);
    const auto sizes = t.sizes(), strides = t.strides();
    const int64_t D = sizes[dim - 1], rows = D ? t.numel() / D : 0;
    if (rows && D > 1 && strides[dim - 1] != 1)
        fail(PyExc_ValueError, "%s: the elements of a row must be contiguous", name);
    if (rows <= 1) return {rows, D, D};
    int64_t ld = 0, span = 0;  // stride of the innermost long dimension; what the next one must step
    for (int64_t i = dim - 2; i >= 0; --i) {
        if (sizes[i] == 1) continue;
        if (!ld) ld = strides[i];
        else if (strides[i] != span)
            fail(PyExc_ValueError, "%s: leading dimensions do not flatten to one row stride", name);
        span = strides[i] * sizes[i];
    }
    if (ld < D)
        fail(PyExc_ValueError, "%s: rows overlap (row stride %lld < D = %lld)", name, (long long)ld, (long long)D);
    return {rows, D, ld};
}

int64_t rows_like(const char *name, const Tensor &t, const Tensor &ref) {
    same_kind(name, t, ref);
    if (t.sizes() != ref.sizes())
        fail(PyExc_ValueError, "%s must have shape %s, got %s", name, shape_str(ref.sizes()).c_str(),
             shape_str(t.sizes()).c_str());
    return rows_ld(name, t).ld;
}

void weight(const char *name, const Tensor &w, const Tensor &x, int64_t D) {
    if (w.scalar_type() != x.scalar_type() || w.device() != x.device() || w.dim() != 1 || w.size(0) != D ||
        !w.is_contiguous())
        fail(PyExc_ValueError, "%s must be a contiguous [%lld] %s tensor on %s", name, (long long)D,
             dtype_str(x.scalar_type()), x.device().str().c_str());
}

void exactly(const char *name, const Tensor &t, at::ScalarType type, c10::IntArrayRef shape, const c10::Device &dev) {
    if (t.scalar_type() != type || t.sizes() != shape || t.device() != dev || !t.is_contiguous())
        fail(PyExc_ValueError, "%s must be a contiguous %s %s tensor on %s", name, shape_str(shape).c_str(),
             dtype_str(type), dev.str().c_str());
}

// A new tensor on the current device (OnDevice), from torch's allocator for the
// current stream, without the operator dispatch of at::empty.
Tensor empty(c10::IntArrayRef shape, at::ScalarType type) {
    return at::detail::empty_generic(shape, c10::cuda::CUDACachingAllocator::get(),
                                     c10::DispatchKeySet(c10::DispatchKey::CUDA), type, std::nullopt);
}

Tensor given_or_empty(const char *name, const Tensor *t, at::ScalarType type, c10::IntArrayRef shape,
                      const c10::Device &dev) {
    if (!t) return empty(shape, type);
    exactly(name, *t, type, shape, dev);
    return *t;
}

// Makes the tensors' device current for the call; its current stream.
struct OnDevice {
    c10::cuda::OptionalCUDAGuard guard;
    void *stream;
    explicit OnDevice(const c10::Device &d) : guard(d), stream(c10::cuda::getCurrentCUDAStream(d.index()).stream()) {}
};

PyObject *wrap(const Tensor &t) { return THPVariable_Wrap(t); }
PyObject *none() {
    Py_INCREF(Py_None);
    return Py_None;
}
PyObject *wrap_or_none(const std::optional<Tensor> &t) { return t ? wrap(*t) : none(); }

template <typename... P> PyObject *tuple_of(P *...items) {
    PyObject *all[] = {items...};
    PyObject *t = PyTuple_New(sizeof...(items));
    bool bad = !t;
    for (size_t i = 0; i < sizeof...(items); ++i) {
        bad = bad || !all[i];
        if (t) PyTuple_SET_ITEM(t, i, all[i]);
        else Py_XDECREF(all[i]);
    }
    if (bad) {
        Py_XDECREF(t);
        return nullptr;
    }
    return t;
}

// Runs f with C++ exceptions turned into Python ones (torch's own into theirs).
template <typename F> PyObject *guarded(Py_ssize_t n, Py_ssize_t want, F f) {
    if (n != want) {
        PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, n);
        return nullptr;
    }
    HANDLE_TH_ERRORS
    try {
        return f();
    } catch (const PyError &) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

// ---- the norm pair around a block ------------------------------------------
struct Gate {
    int64_t G = 0, ld = 0;
};

Gate check_gate(const Tensor *gate, const Tensor &x, int64_t rows, int64_t D) {
    if (!gate) return {};
    same_kind("gate", *gate, x);
    if (gate->dim() < 1 || gate->size(-1) != D)
        fail(PyExc_ValueError, "gate must be [..., %lld], got %s", (long long)D, shape_str(gate->sizes()).c_str());
    const Rows r = rows_ld("gate", *gate);
    if (r.rows < 1 ? rows != 0 : rows % r.rows != 0)
        fail(PyExc_ValueError, "the gate's %lld rows must divide the %lld rows", (long long)r.rows, (long long)rows);
    return {r.rows, r.ld};
}

void check_rstd(const Tensor &rstd, int64_t rows, const c10::Device &dev) {
    if (rstd.scalar_type() != at::kFloat || rstd.dim() < 1 || rstd.size(0) != 2 || rstd.numel() != 2 * rows ||
        rstd.device() != dev || !rstd.is_contiguous())
        fail(PyExc_ValueError, "rstd must be a contiguous float32 tensor [2, rows] of %lld rows on %s",
             (long long)rows, dev.str().c_str());
}

// A row output: the given tensor, or a dense new one like ref.
std::pair<Tensor, int64_t> row_output(const char *name, const Tensor *t, const Tensor &ref, int64_t D) {
    if (!t) return {empty(ref.sizes(), ref.scalar_type()), D};
    return {*t, rows_like(name, *t, ref)};
}

PyObject *block_fwd(PyObject *, PyObject *const *argv, Py_ssize_t n) {
    return guarded(n, 11, [&]() -> PyObject * {
        const Args a{argv, n};
        const Tensor &y = a.tensor(0, "y"), &res = a.tensor(1, "residual"), &w_pre = a.tensor(3, "w_pre");
        const Tensor *w_post = a.optional(2, "w_post"), *gate = a.optional(6, "gate");
        const Rows r = rows_ld("y", y);
        const int code = dtype_code(y);
        const int64_t ld_r = rows_like("residual", res, y);
        weight("w_pre", w_pre, y, r.D);
        if (w_post) weight("w_post", *w_post, y, r.D);
        const Gate g = check_gate(gate, y, r.rows, r.D);
        const OnDevice on(y.device());
        const auto out = row_output("out", a.optional(8, "out"), y, r.D);
        const auto nr = row_output("new_residual", a.optional(9, "new_residual"), y, r.D);
        std::optional<Tensor> rstd;
        if (argv[10] == Py_True) {
            c10::SmallVector<int64_t, 6> shape{2};
            shape.append(y.sizes().begin(), y.sizes().end() - 1);
            rstd = empty(shape, at::kFloat);
        } else if (argv[10] != Py_None) {
            rstd = a.tensor(10, "rstd");
            check_rstd(*rstd, r.rows, y.device());
        }
        check_status("rmsnorm_block_fwd",
                     c_block_fwd(ptr(&y), r.ld, ptr(&res), ld_r, ptr(w_post), ptr(&w_pre), ptr(gate), g.ld, g.G,
                                 (float)a.number(7), (float)a.number(4), (float)a.number(5), ptr(&out.first),
                                 out.second, ptr(&nr.first), nr.second,
                                 rstd ? static_cast<float *>(ptr(&*rstd)) : nullptr, r.rows, r.D, code, on.stream));
        wrote(a.optional(8, "out"), a.optional(9, "new_residual"), argv[10] == Py_True ? nullptr : a.optional(10, "rstd"));
        return tuple_of(wrap(out.first), wrap(nr.first), wrap_or_none(rstd));
    });
}

PyObject *block_vjp(PyObject *, PyObject *const *argv, Py_ssize_t n) {
    return guarded(n, 16, [&]() -> PyObject * {
        const Args a{argv, n};
        const Tensor &y = a.tensor(0, "y"), &h = a.tensor(1, "h"), &w_pre = a.tensor(3, "w_pre");
        const Tensor &g_out = a.tensor(4, "g_out");
        const Tensor *w_post = a.optional(2, "w_post"), *gate = a.optional(7, "gate");
        const Tensor *g_res = a.optional(9, "g_residual"), *rstd = a.optional(10, "rstd");
        const Rows r = rows_ld("y", y);
        const int code = dtype_code(y);
        const int64_t ld_h = rows_like("h", h, y), ld_g = rows_like("g_out", g_out, y);
        const int64_t ld_gr = g_res ? rows_like("g_residual", *g_res, y) : r.D;
        weight("w_pre", w_pre, y, r.D);
        if (w_post) weight("w_post", *w_post, y, r.D);
        const Gate g = check_gate(gate, y, r.rows, r.D);
        if (rstd) check_rstd(*rstd, r.rows, y.device());
        if (!w_post && argv[13] != Py_None) fail(PyExc_ValueError, "gw_post given without w_post");
        if (!gate && argv[15] != Py_None) fail(PyExc_ValueError, "g_gate given without a gate");
        const OnDevice on(y.device());
        const auto g_y = row_output("g_y", a.optional(11, "g_y"), y, r.D);
        const auto g_h = row_output("g_h", a.optional(12, "g_h"), y, r.D);
        const Tensor gw_pre = given_or_empty("gw_pre", a.optional(14, "gw_pre"), at::kFloat, {r.D}, y.device());
        std::optional<Tensor> gw_post, g_gate;
        if (w_post) gw_post = given_or_empty("gw_post", a.optional(13, "gw_post"), at::kFloat, {r.D}, y.device());
        if (gate)
            g_gate = given_or_empty("g_gate", a.optional(15, "g_gate"), at::kFloat, gate->sizes(), y.device());
        auto f32 = [](const std::optional<Tensor> &t) { return t ? static_cast<float *>(ptr(&*t)) : nullptr; };
        const int64_t bytes = (int64_t)c_block_vjp_workspace_size(r.rows, r.D, code);
        const Tensor ws = empty({bytes}, at::kByte);
        check_status("rmsnorm_block_vjp",
                     c_block_vjp_ws(ptr(&y), r.ld, ptr(&h), ld_h, ptr(w_post), ptr(&w_pre), ptr(gate), g.ld, g.G,
                                 (float)a.number(8), ptr(&g_out), ld_g, ptr(g_res), ld_gr,
                                 static_cast<const float *>(ptr(rstd)), (float)a.number(5), (float)a.number(6),
                                 ptr(&g_y.first), g_y.second, ptr(&g_h.first), g_h.second, f32(gw_post),
                                 static_cast<float *>(ptr(&gw_pre)), f32(g_gate), r.rows, r.D, code, ptr(&ws), (size_t)bytes,
                                 on.stream));
        wrote(a.optional(11, "g_y"), a.optional(12, "g_h"), a.optional(13, "gw_post"), a.optional(14, "gw_pre"),
              a.optional(15, "g_gate"));
        return tuple_of(wrap(g_y.first), wrap(g_h.first), wrap_or_none(gw_post), wrap(gw_pre), wrap_or_none(g_gate));
    });
}

// ---- the norm with an 8-bit output -------------------------------------------
PyObject *fwd_q8(PyObject *, PyObject *const *argv, Py_ssize_t n) {
    return guarded(n, 9, [&]() -> PyObject * {
        const Args a{argv, n};
        const Tensor &x = a.tensor(0, "x"), &w = a.tensor(1, "w");
        const Tensor *res = a.optional(4, "residual");
        const Rows r = rows_ld("x", x);
        const int code = dtype_code(x);
        const int64_t ld_r = res ? rows_like("residual", *res, x) : r.D;
        weight("w", w, x, r.D);
        const int64_t group = a.integer(5);
        if (group != 0 && group != 32 && group != 64 && group != 128)
            fail(PyExc_ValueError, "group must be 0 (the row), 32, 64 or 128");
        if (!res && argv[8] != Py_None) fail(PyExc_ValueError, "new_residual given without residual");
        c10::SmallVector<int64_t, 6> shape(x.sizes().begin(), x.sizes().end() - 1);
        if (group) shape.push_back((r.D + group - 1) / group);
        const OnDevice on(x.device());
        const Tensor *given = a.optional(6, "out");
        int64_t ld_o = r.D;
        if (given) {
            if (given->scalar_type() != at::kFloat8_e4m3fn || given->sizes() != x.sizes() || given->device() != x.device())
                fail(PyExc_ValueError, "out must be a %s torch.float8_e4m3fn tensor on %s", shape_str(x.sizes()).c_str(),
                     x.device().str().c_str());
            ld_o = rows_ld("out", *given).ld;
        }
        const Tensor out = given ? *given : empty(x.sizes(), at::kFloat8_e4m3fn);
        const Tensor scale = given_or_empty("scale", a.optional(7, "scale"), at::kFloat, shape, x.device());
        std::optional<Tensor> nr;
        int64_t ld_n = r.D;
        if (res) {
            const auto made = row_output("new_residual", a.optional(8, "new_residual"), x, r.D);
            nr = made.first;
            ld_n = made.second;
        }
        check_status("rmsnorm_fwd_q8",
                     c_fwd_q8(ptr(&x), r.ld, ptr(res), ld_r, ptr(&w), (float)a.number(2), (float)a.number(3), ptr(&out),
                              ld_o, static_cast<float *>(ptr(&scale)), group, nr ? ptr(&*nr) : nullptr, ld_n, r.rows,
                              r.D, code, on.stream));
        wrote(given, a.optional(7, "scale"), a.optional(8, "new_residual"));
        return tuple_of(wrap(out), wrap(scale), wrap_or_none(nr));
    });
}

// ---- rotary positions --------------------------------------------------------
int64_t rot_dim(const Tensor &inv, int64_t Dh) {
    if (inv.scalar_type() != at::kDouble || inv.dim() != 1 || !inv.device().is_cpu() || !inv.is_contiguous())
        fail(PyExc_ValueError, "inv_freq must be a contiguous [rot_dim / 2] float64 CPU tensor");
    const int64_t rot = 2 * inv.size(0);
    if (rot < 2 || rot > Dh)
        fail(PyExc_ValueError, "inv_freq has %lld pairs, a head of %lld elements at most %lld",
             (long long)(rot / 2), (long long)Dh, (long long)(Dh / 2));
    return rot;
}

// Batch, token and head strides of a [(B,) S, H, Dh] tensor.
struct Strides {
    int64_t s[3];
};

Strides head_strides(const char *name, const Tensor &t) {
    if (t.numel() && t.size(-1) > 1 && t.stride(-1) != 1)
        fail(PyExc_ValueError, "%s: the elements of a head must be contiguous", name);
    return {{t.dim() == 4 ? t.stride(0) : 0, t.stride(-3), t.stride(-2)}};
}

// t has ref's shape but for H heads.
void heads_like(const char *name, const Tensor &t, const Tensor &ref, int64_t H) {
    same_kind(name, t, ref);
    bool ok = t.dim() == ref.dim() && t.size(-2) == H && t.size(-1) == ref.size(-1);
    for (int64_t i = 0; ok && i < ref.dim() - 2; ++i) ok = t.size(i) == ref.size(i);
    if (!ok) {
        c10::SmallVector<int64_t, 4> want(ref.sizes().begin(), ref.sizes().end());
        want[want.size() - 2] = H;
        fail(PyExc_ValueError, "%s must have shape %s, got %s", name, shape_str(want).c_str(),
             shape_str(t.sizes()).c_str());
    }
}

Tensor heads_output(const char *name, const Tensor *t, const Tensor &ref) {
    if (!t) return empty(ref.sizes(), ref.scalar_type());
    heads_like(name, *t, ref, ref.size(-2));
    return *t;
}

PyObject *rope(PyObject *, PyObject *const *argv, Py_ssize_t n) {
    return guarded(n, 9, [&]() -> PyObject * {
        const Args a{argv, n};
        const Tensor &q = a.tensor(0, "q"), &pos = a.tensor(2, "positions"), &inv = a.tensor(3, "inv_freq");
        const Tensor *k = a.optional(1, "k");
        const int64_t dim = q.dim();
        if (dim != 3 && dim != 4) fail(PyExc_ValueError, "q must be [S, Hq, Dh] or [B, S, Hq, Dh]");
        need_cuda(q);
        const int code = dtype_code(q);
        const int64_t Hq = q.size(-2), Dh = q.size(-1), rot = rot_dim(inv, Dh);
        exactly("positions", pos, at::kLong, q.sizes().slice(0, dim - 2), q.device());
        int64_t Hkv = 0;
        if (k) {
            if (k->dim() != dim) fail(PyExc_ValueError, "k must have q's leading dimensions");
            Hkv = k->size(-2);
            heads_like("k", *k, q, Hkv);
        } else if (argv[8] != Py_None) {
            fail(PyExc_ValueError, "k_out given without k");
        }
        const OnDevice on(q.device());
        const Tensor qo = heads_output("q_out", a.optional(7, "q_out"), q);
        std::optional<Tensor> ko;
        Strides sk{}, sko{};
        if (k) {
            ko = heads_output("k_out", a.optional(8, "k_out"), *k);
            sk = head_strides("k", *k);
            sko = head_strides("k_out", *ko);
        }
        const Strides sq = head_strides("q", q), sqo = head_strides("q_out", qo);
        check_status("rmsnorm_rope",
                     c_rope(ptr(&q), sq.s, ptr(k), sk.s, static_cast<const int64_t *>(ptr(&pos)), ptr(&qo), sqo.s,
                            ko ? ptr(&*ko) : nullptr, sko.s, static_cast<const double *>(inv.data_ptr()),
                            (float)a.number(4), a.truth(5) ? 1 : 0, a.truth(6) ? 1 : 0, dim == 4 ? q.size(0) : 1,
                            q.size(dim - 3), Hq, Hkv, Dh, rot, code, on.stream));
        wrote(a.optional(7, "q_out"), a.optional(8, "k_out"));
        return tuple_of(wrap(qo), wrap_or_none(ko));
    });
}

// Positions [axes, ...] of `tokens` leading dimensions, or those dimensions alone (one
// axis), and the axis of each pair.
struct Axes {
    int n;
    const int32_t *of;
};

Axes check_axes(const Tensor &pos, const Tensor *pair_axis, c10::IntArrayRef tokens, int64_t rot, const c10::Device &dev) {
    if (!pair_axis) {
        exactly("positions", pos, at::kLong, tokens, dev);
        return {1, nullptr};
    }
    if (pair_axis->scalar_type() != at::kInt || pair_axis->dim() != 1 || pair_axis->size(0) != rot / 2 ||
        !pair_axis->device().is_cpu() || !pair_axis->is_contiguous())
        fail(PyExc_ValueError, "pair_axis must be a contiguous [%lld] int32 CPU tensor, an axis for each pair",
             (long long)(rot / 2));
    const int64_t n = pos.dim() ? pos.size(0) : 0;
    if (n < 1 || n > RMSNORM_ROPE_MAX_AXES)
        fail(PyExc_ValueError, "positions must have one to %d axes in their first dimension", RMSNORM_ROPE_MAX_AXES);
    c10::SmallVector<int64_t, 4> want{n};
    want.append(tokens.begin(), tokens.end());
    exactly("positions", pos, at::kLong, want, dev);
    const int32_t *of = pair_axis->const_data_ptr<int32_t>();
    for (int64_t i = 0; i < rot / 2; ++i)
        if (of[i] < 0 || of[i] >= n)
            fail(PyExc_ValueError, "pair_axis[%lld] is %d, the positions have %lld axes", (long long)i, (int)of[i],
                 (long long)n);
    return {(int)n, of};
}

PyObject *rope_axes(PyObject *, PyObject *const *argv, Py_ssize_t n) {
    return guarded(n, 10, [&]() -> PyObject * {
        const Args a{argv, n};
        const Tensor &q = a.tensor(0, "q"), &pos = a.tensor(2, "positions"), &inv = a.tensor(3, "inv_freq");
        const Tensor *k = a.optional(1, "k");
        const int64_t dim = q.dim();
        if (dim != 3 && dim != 4) fail(PyExc_ValueError, "q must be [S, Hq, Dh] or [B, S, Hq, Dh]");
        need_cuda(q);
        const int code = dtype_code(q);
        const int64_t Hq = q.size(-2), Dh = q.size(-1), rot = rot_dim(inv, Dh);
        const Axes axes = check_axes(pos, &a.tensor(4, "pair_axis"), q.sizes().slice(0, dim - 2), rot, q.device());
        int64_t Hkv = 0;
        if (k) {
            if (k->dim() != dim) fail(PyExc_ValueError, "k must have q's leading dimensions");
            Hkv = k->size(-2);
            heads_like("k", *k, q, Hkv);
        } else if (argv[9] != Py_None) {
            fail(PyExc_ValueError, "k_out given without k");
        }
        const OnDevice on(q.device());
        const Tensor qo = heads_output("q_out", a.optional(8, "q_out"), q);
        std::optional<Tensor> ko;
        Strides sk{}, sko{};
        if (k) {
            ko = heads_output("k_out", a.optional(9, "k_out"), *k);
            sk = head_strides("k", *k);
            sko = head_strides("k_out", *ko);
        }
        const Strides sq = head_strides("q", q), sqo = head_strides("q_out", qo);
        check_status("rmsnorm_rope_axes",
                     c_rope_axes(ptr(&q), sq.s, ptr(k), sk.s, static_cast<const int64_t *>(ptr(&pos)), axes.n, axes.of,
                                 ptr(&qo), sqo.s, ko ? ptr(&*ko) : nullptr, sko.s,
                                 static_cast<const double *>(inv.data_ptr()), (float)a.number(5), a.truth(6) ? 1 : 0,
                                 a.truth(7) ? 1 : 0, dim == 4 ? q.size(0) : 1, q.size(dim - 3), Hq, Hkv, Dh, rot, code,
                                 on.stream));
        wrote(a.optional(8, "q_out"), a.optional(9, "k_out"));
        return tuple_of(wrap(qo), wrap_or_none(ko));
    });
}

// What a cache of this type holds: RMSNORM_CACHE_*.
int cache_format(const Tensor &c) {
    return c.scalar_type() == at::kFloat8_e4m3fn ? RMSNORM_CACHE_E4M3
           : c.scalar_type() == at::kChar        ? RMSNORM_CACHE_I8
                                                 : RMSNORM_CACHE_SAME;
}

void check_scales(const char *name, const Tensor &t, int64_t slots, int64_t Hkv, const c10::Device &dev) {
    if (t.scalar_type() != at::kFloat || t.dim() != 2 || t.size(0) != slots || t.size(1) != Hkv || t.device() != dev)
        fail(PyExc_ValueError, "%s must be a (%lld, %lld) torch.float32 tensor on %s", name, (long long)slots,
             (long long)Hkv, dev.str().c_str());
}

// Both caches [num_slots, Hkv, Dh] of one type.
void check_caches(const Tensor &kc, const Tensor &vc, int64_t Hkv, int64_t Dh, const c10::Device &dev) {
    for (const Tensor *c : {&kc, &vc})
        if (c->scalar_type() != kc.scalar_type() || c->device() != dev || c->dim() != 3 || c->size(1) != Hkv ||
            c->size(2) != Dh || c->size(0) != kc.size(0))
            fail(PyExc_ValueError, "the caches must be [num_slots, %lld, %lld] of one type on %s", (long long)Hkv,
                 (long long)Dh, dev.str().c_str());
}

// Token (or slot) and head strides of scales [num_slots, Hkv].
Strides scale_strides(const Tensor *t) {
    return t ? Strides{{0, t->stride(0), t->stride(1)}} : Strides{};
}

PyObject *kv_append(PyObject *, PyObject *const *argv, Py_ssize_t n) {
    return guarded(n, 14, [&]() -> PyObject * {
        const Args a{argv, n};
        const Tensor &q = a.tensor(0, "q"), &k = a.tensor(1, "k"), &v = a.tensor(2, "v");
        const Tensor &pos = a.tensor(3, "positions"), &slots = a.tensor(4, "slots");
        const Tensor &kc = a.tensor(5, "k_cache"), &vc = a.tensor(6, "v_cache"), &inv = a.tensor(7, "inv_freq");
        const Tensor *ks = a.optional(8, "k_scale"), *vs = a.optional(9, "v_scale");
        if (q.dim() != 3 || k.dim() != 3 || v.sizes() != k.sizes())
            fail(PyExc_ValueError, "q must be [T, Hq, Dh] and k, v [T, Hkv, Dh]");
        need_cuda(q);
        const int code = dtype_code(q), format = cache_format(kc);
        const int64_t T = q.size(0), Hq = q.size(1), Dh = q.size(2), Hkv = k.size(1), rot = rot_dim(inv, Dh);
        heads_like("k", k, q, Hkv);
        heads_like("v", v, q, Hkv);
        check_caches(kc, vc, Hkv, Dh, q.device());
        if (format == RMSNORM_CACHE_SAME) {
            if (kc.scalar_type() != q.scalar_type())
                fail(PyExc_ValueError, "the caches must be torch.float8_e4m3fn, torch.int8 or %s", dtype_str(q.scalar_type()));
            if (ks || vs) fail(PyExc_ValueError, "k_scale and v_scale go with 8-bit caches");
        } else {
            if (!ks || !vs) fail(PyExc_ValueError, "8-bit caches need k_scale and v_scale");
            check_scales("k_scale", *ks, kc.size(0), Hkv, q.device());
            check_scales("v_scale", *vs, kc.size(0), Hkv, q.device());
        }
        const Axes axes = check_axes(pos, a.optional(10, "pair_axis"), {T}, rot, q.device());
        exactly("slots", slots, at::kLong, {T}, q.device());
        const OnDevice on(q.device());
        const Tensor qo = heads_output("q_out", a.optional(13, "q_out"), q);
        const Strides sq = head_strides("q", q), sk = head_strides("k", k), sv = head_strides("v", v);
        const Strides sqo = head_strides("q_out", qo), skc = head_strides("k_cache", kc), svc = head_strides("v_cache", vc);
        const Strides sks = scale_strides(ks), svs = scale_strides(vs);
        check_status("rmsnorm_kv_append",
                     c_kv_append(ptr(&q), sq.s + 1, ptr(&k), sk.s + 1, ptr(&v), sv.s + 1,
                                 static_cast<const int64_t *>(ptr(&pos)), axes.n, axes.of,
                                 static_cast<const int64_t *>(ptr(&slots)), ptr(&qo), sqo.s + 1, ptr(&kc), skc.s + 1,
                                 ptr(&vc), svc.s + 1, static_cast<float *>(ptr(ks)), sks.s + 1,
                                 static_cast<float *>(ptr(vs)), svs.s + 1, static_cast<const double *>(inv.data_ptr()),
                                 (float)a.number(11), a.truth(12) ? 1 : 0, T, Hq, Hkv, Dh, rot, kc.size(0), format, code,
                                 on.stream));
        wrote(&kc, &vc, ks, vs, a.optional(13, "q_out"));
        return wrap(qo);
    });
}

PyObject *kv_read(PyObject *, PyObject *const *argv, Py_ssize_t n) {
    return guarded(n, 8, [&]() -> PyObject * {
        const Args a{argv, n};
        const Tensor &kc = a.tensor(0, "k_cache"), &vc = a.tensor(1, "v_cache");
        const Tensor &ks = a.tensor(2, "k_scale"), &vs = a.tensor(3, "v_scale"), &slots = a.tensor(4, "slots");
        need_cuda(kc);
        const c10::Device dev = kc.device();
        const int format = cache_format(kc);
        if (kc.dim() != 3 || format == RMSNORM_CACHE_SAME)
            fail(PyExc_ValueError, "the caches must be [num_slots, Hkv, Dh], torch.float8_e4m3fn or torch.int8");
        const int64_t Hkv = kc.size(1), Dh = kc.size(2);
        check_caches(kc, vc, Hkv, Dh, dev);
        check_scales("k_scale", ks, kc.size(0), Hkv, dev);
        check_scales("v_scale", vs, kc.size(0), Hkv, dev);
        if (slots.dim() != 1) fail(PyExc_ValueError, "slots must be [T]");
        const int64_t T = slots.size(0);
        exactly("slots", slots, at::kLong, {T}, dev);
        if (!THPDtype_Check(argv[5])) fail(PyExc_TypeError, "dtype must be a torch.dtype");
        const at::ScalarType type = reinterpret_cast<THPDtype *>(argv[5])->scalar_type;
        const int code = type == at::kHalf ? 0 : type == at::kBFloat16 ? 1 : type == at::kFloat ? 2 : -1;
        if (code < 0) fail(PyExc_TypeError, "unsupported dtype %s (fp16 or bf16 or fp32)", dtype_str(type));
        const OnDevice on(dev);
        auto output = [&](const char *name, const Tensor *t) {
            if (!t) return empty({T, Hkv, Dh}, type);
            if (t->scalar_type() != type || t->device() != dev || t->sizes() != c10::IntArrayRef({T, Hkv, Dh}))
                fail(PyExc_ValueError, "%s must be a (%lld, %lld, %lld) %s tensor on %s", name, (long long)T,
                     (long long)Hkv, (long long)Dh, dtype_str(type), dev.str().c_str());
            return *t;
        };
        const Tensor ko = output("k_out", a.optional(6, "k_out")), vo = output("v_out", a.optional(7, "v_out"));
        const Strides skc = head_strides("k_cache", kc), svc = head_strides("v_cache", vc);
        const Strides sks = scale_strides(&ks), svs = scale_strides(&vs);
        const Strides sko = head_strides("k_out", ko), svo = head_strides("v_out", vo);
        check_status("rmsnorm_kv_read",
                     c_kv_read(ptr(&kc), skc.s + 1, ptr(&vc), svc.s + 1, static_cast<const float *>(ptr(&ks)), sks.s + 1,
                               static_cast<const float *>(ptr(&vs)), svs.s + 1, static_cast<const int64_t *>(ptr(&slots)),
                               ptr(&ko), sko.s + 1, ptr(&vo), svo.s + 1, T, Hkv, Dh, kc.size(0), format, code, on.stream));
        wrote(a.optional(6, "k_out"), a.optional(7, "v_out"));
        return tuple_of(wrap(ko), wrap(vo));
    });
}

PyObject *rope_append(PyObject *, PyObject *const *argv, Py_ssize_t n) {
    return guarded(n, 11, [&]() -> PyObject * {
        const Args a{argv, n};
        const Tensor &q = a.tensor(0, "q"), &k = a.tensor(1, "k"), &v = a.tensor(2, "v");
        const Tensor &pos = a.tensor(3, "positions"), &slots = a.tensor(4, "slots");
        const Tensor &kc = a.tensor(5, "k_cache"), &vc = a.tensor(6, "v_cache"), &inv = a.tensor(7, "inv_freq");
        if (q.dim() != 3 || k.dim() != 3 || v.sizes() != k.sizes())
            fail(PyExc_ValueError, "q must be [T, Hq, Dh] and k, v [T, Hkv, Dh]");
        need_cuda(q);
        const int code = dtype_code(q);
        const int64_t T = q.size(0), Hq = q.size(1), Dh = q.size(2), Hkv = k.size(1), rot = rot_dim(inv, Dh);
        heads_like("k", k, q, Hkv);
        heads_like("v", v, q, Hkv);
        for (const Tensor *c : {&kc, &vc})
            if (c->scalar_type() != q.scalar_type() || c->device() != q.device() || c->dim() != 3 ||
                c->size(1) != Hkv || c->size(2) != Dh || c->size(0) != kc.size(0))
                fail(PyExc_ValueError, "the caches must be [num_slots, %lld, %lld] %s on %s", (long long)Hkv,
                     (long long)Dh, dtype_str(q.scalar_type()), q.device().str().c_str());
        exactly("positions", pos, at::kLong, {T}, q.device());
        exactly("slots", slots, at::kLong, {T}, q.device());
        const OnDevice on(q.device());
        const Tensor qo = heads_output("q_out", a.optional(10, "q_out"), q);
        const Strides sq = head_strides("q", q), sk = head_strides("k", k), sv = head_strides("v", v);
        const Strides sqo = head_strides("q_out", qo), skc = head_strides("k_cache", kc), svc = head_strides("v_cache", vc);
        check_status("rmsnorm_rope_kv_append_ex",
                     c_rope_kv_append_ex(ptr(&q), sq.s + 1, ptr(&k), sk.s + 1, ptr(&v), sv.s + 1,
                                         static_cast<const int64_t *>(ptr(&pos)), static_cast<const int64_t *>(ptr(&slots)),
                                         ptr(&qo), sqo.s + 1, ptr(&kc), skc.s + 1, ptr(&vc), svc.s + 1,
                                         static_cast<const double *>(inv.data_ptr()), (float)a.number(8),
                                         a.truth(9) ? 1 : 0, T, Hq, Hkv, Dh, rot, kc.size(0), code, on.stream));
        wrote(&kc, &vc, a.optional(10, "q_out"));
        return wrap(qo);
    });
}

// ---- block tables and slot maps ------------------------------------------------
struct Pool {
    int64_t B, W, ld, N = 0;
};

Pool check_pool(const Tensor &lens, const Tensor &table, const Tensor *free_blocks, const Tensor *free_count) {
    need_cuda(lens);
    const c10::Device dev = lens.device();
    const int64_t B = lens.dim() == 1 ? lens.size(0) : -1;
    exactly("lens", lens, at::kInt, {B}, dev);
    if (table.scalar_type() != at::kInt || table.dim() != 2 || table.size(0) != B || table.device() != dev ||
        (table.size(1) > 1 && table.stride(1) != 1))
        fail(PyExc_ValueError, "block_table must be a [%lld, width] int32 tensor on %s with contiguous rows",
             (long long)B, dev.str().c_str());
    Pool p{B, table.size(1), B > 1 ? table.stride(0) : table.size(1)};
    if (p.ld < p.W) fail(PyExc_ValueError, "block_table: rows overlap");
    if ((free_blocks != nullptr) != (free_count != nullptr))
        fail(PyExc_ValueError, "free_blocks and free_count go together");
    if (free_blocks) {
        if (free_blocks->dim() != 1) fail(PyExc_ValueError, "free_blocks must be [num_blocks]");
        p.N = free_blocks->size(0);
        exactly("free_blocks", *free_blocks, at::kInt, {p.N}, dev);
        exactly("free_count", *free_count, at::kInt, {1}, dev);
    }
    return p;
}

int32_t *i32(const Tensor *t) { return static_cast<int32_t *>(ptr(t)); }

PyObject *kv_release(PyObject *, PyObject *const *argv, Py_ssize_t n) {
    return guarded(n, 8, [&]() -> PyObject * {
        const Args a{argv, n};
        const Tensor &lens = a.tensor(0, "lens"), &fin = a.tensor(1, "finished"), &table = a.tensor(2, "block_table");
        const Tensor &free_blocks = a.tensor(4, "free_blocks"), &count = a.tensor(5, "free_count");
        const Pool p = check_pool(lens, table, &free_blocks, &count);
        const c10::Device dev = lens.device();
        exactly("finished", fin, at::kBool, {p.B}, dev);
        const Tensor *lo = a.optional(6, "lens_out"), *co = a.optional(7, "free_count_out");
        if (lo) exactly("lens_out", *lo, at::kInt, {p.B}, dev);
        else lo = &lens;
        if (co) exactly("free_count_out", *co, at::kInt, {1}, dev);
        else co = &count;
        const OnDevice on(dev);
        check_status("rmsnorm_kv_release",
                     c_kv_release(i32(&lens), static_cast<const uint8_t *>(ptr(&fin)), i32(&table), p.ld, p.W,
                                  a.integer(3), i32(&free_blocks), i32(&count), p.N, i32(lo), i32(co), p.B,
                                  on.stream));
        wrote(lo, co, &free_blocks);
        return tuple_of(wrap(*lo), wrap(*co));
    });
}

PyObject *kv_plan(PyObject *, PyObject *const *argv, Py_ssize_t n) {
    return guarded(n, 14, [&]() -> PyObject * {
        const Args a{argv, n};
        const Tensor &lens = a.tensor(0, "lens"), &fresh = a.tensor(1, "new_lens"), &table = a.tensor(2, "block_table");
        const Tensor *free_blocks = a.optional(5, "free_blocks"), *count = a.optional(6, "free_count");
        const Pool p = check_pool(lens, table, free_blocks, count);
        const c10::Device dev = lens.device();
        exactly("new_lens", fresh, at::kInt, {p.B}, dev);
        const int64_t T = a.integer(4);
        if (T < 0) fail(PyExc_ValueError, "num_tokens must not be negative");
        const Tensor *lo = a.optional(7, "lens_out"), *co = a.optional(8, "free_count_out");
        if (lo) exactly("lens_out", *lo, at::kInt, {p.B}, dev);
        else lo = &lens;
        if (co && !count) fail(PyExc_ValueError, "free_count_out given without a pool");
        if (co) exactly("free_count_out", *co, at::kInt, {1}, dev);
        else co = count;
        const OnDevice on(dev);
        const Tensor positions = given_or_empty("positions", a.optional(9, "positions"), at::kLong, {T}, dev);
        const Tensor slots = given_or_empty("slots", a.optional(10, "slots"), at::kLong, {T}, dev);
        const Tensor requests = given_or_empty("requests", a.optional(11, "requests"), at::kInt, {T}, dev);
        const Tensor starts = given_or_empty("starts", a.optional(12, "starts"), at::kLong, {p.B + 1}, dev);
        const Tensor granted = given_or_empty("granted", a.optional(13, "granted"), at::kBool, {p.B}, dev);
        check_status("rmsnorm_kv_plan",
                     c_kv_plan(i32(&lens), i32(&fresh), i32(&table), p.ld, p.W, a.integer(3), i32(free_blocks),
                               i32(count), p.N, i32(lo), i32(co), static_cast<int64_t *>(ptr(&starts)),
                               static_cast<int64_t *>(ptr(&positions)), static_cast<int64_t *>(ptr(&slots)),
                               i32(&requests), static_cast<uint8_t *>(ptr(&granted)), p.B, T, on.stream));
        wrote(lo, co, count ? &table : nullptr, a.optional(9, "positions"), a.optional(10, "slots"),
              a.optional(11, "requests"), a.optional(12, "starts"), a.optional(13, "granted"));
        return tuple_of(wrap(positions), wrap(slots), wrap(requests), wrap(starts), wrap(granted), wrap(*lo),
                        co ? wrap(*co) : none());
    });
}

// bind(check, {name: address}): the library's entry points.
PyObject *bind(PyObject *, PyObject *const *argv, Py_ssize_t n) {
    return guarded(n, 2, [&]() -> PyObject * {
#define SLOT(name) {"rmsnorm_" #name, &c_##name}
        const struct { const char *name; void *slot; } table[] = {
            SLOT(block_fwd), SLOT(block_vjp_ws), SLOT(block_vjp_workspace_size), SLOT(rope), SLOT(rope_kv_append_ex),
            SLOT(rope_axes), SLOT(kv_append), SLOT(kv_read), SLOT(fwd_q8), SLOT(kv_release), SLOT(kv_plan)};
#undef SLOT
        for (const auto &e : table) {
            PyObject *v = PyDict_GetItemString(argv[1], e.name);  // borrowed
            if (!v) fail(PyExc_KeyError, "%s", e.name);
            void *p = PyLong_AsVoidPtr(v);
            if (!p) fail(PyExc_ValueError, "%s: no address", e.name);
            std::memcpy(e.slot, &p, sizeof(p));
        }
        Py_INCREF(argv[0]);
        Py_XDECREF(g_check);
        g_check = argv[0];
        return none();
    });
}

#define METHOD(name) {#name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {METHOD(bind),        METHOD(block_fwd),  METHOD(block_vjp), METHOD(rope),
                         METHOD(rope_append), METHOD(kv_release), METHOD(kv_plan),   METHOD(rope_axes),
                         METHOD(kv_append),   METHOD(kv_read),    METHOD(fwd_q8),    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
