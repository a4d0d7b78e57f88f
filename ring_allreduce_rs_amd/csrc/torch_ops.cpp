// torch_ops.cpp -- the training operators on torch tensors: a CPython module
// that checks the tensors, allocates outputs and scratch from torch's
// allocator on torch's current stream, and calls the C entry points of
// libar.so.  operators.py holds the documentation.
//
// A module instead of ctypes calls because the small operators are bound by
// the host: on MI355X a layer norm of one row took 14.7 us through ctypes and
// torch.empty from Python.
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/core/GradMode.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cfloat>
#include <climits>
#include <cmath>
#include <stdexcept>
#include <string>

#include "ar.h"

namespace {

constexpr int kMaxDevices = 64;

// This thread's contexts, one per device: a context is used by one host
// thread only.  Its arrays come from tensors that were looked at here, so the
// library does not ask the runtime about them again.
struct Contexts {
    ar_ctx* c[kMaxDevices] = {};
    hipStream_t stream[kMaxDevices] = {};
    ~Contexts() {
        for (ar_ctx* p : c) ar_destroy(p);
    }
};
thread_local Contexts t_contexts;

// A refused argument (ValueError), and a status from the library (ArError).
struct Refused : std::invalid_argument {
    using std::invalid_argument::invalid_argument;
};
struct Failed {
    ar_status status;
    const char* func;
    std::string detail;
};

ar_ctx* context(int device) {
    if (device < 0 || device >= kMaxDevices) throw Refused("device out of range");
    const hipStream_t s = c10::hip::getCurrentHIPStream((c10::DeviceIndex)device).stream();
    ar_ctx*& c = t_contexts.c[device];
    if (!c) {
        const ar_status st = ar_create(&c, device, s);
        if (st != AR_OK) throw Failed{st, "ar_create", ar_last_error(nullptr)};
        ar_set_operator_checks(c, 0);
        t_contexts.stream[device] = s;
    } else if (t_contexts.stream[device] != s) {
        ar_set_stream(c, s);
        t_contexts.stream[device] = s;
    }
    return c;
}

void must(ar_ctx* c, ar_status st, const char* func) {
    if (st != AR_OK) throw Failed{st, func, c ? ar_last_error(c) : "sizes"};
}

std::string shape_of(const at::Tensor& t) {
    std::string s = "(";
    for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + std::to_string(t.size(i));
    return s + ")";
}

// A tensor argument.  The outputs have no history, so one whose gradient (or
// forward-mode tangent) would be lost is refused.
const at::Tensor& tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) throw Refused(std::string(name) + " is not a tensor");
    const at::Tensor& t = THPVariable_Unpack(o);
    if (t.requires_grad() && c10::GradMode::is_enabled())
        throw Refused(std::string(name) + " requires grad, which this call does not record: "
                      "detach it or call under torch.no_grad()");
    if (t._fw_grad(0).defined())
        throw Refused(std::string(name) + " has a forward-mode tangent, which this call does not "
                      "carry on");
    return t;
}

ar_dtype dtype_of(const at::Tensor& t, const char* name) {
    const at::ScalarType s = t.scalar_type();
    if (s == at::kFloat) return AR_FLOAT32;
    if (s == at::kBFloat16) return AR_BFLOAT16;
    throw Refused(std::string(name) + ": unsupported dtype " + c10::toString(s) +
                  "; use float32 or bfloat16");
}

// A float32 or bfloat16 tensor on a GPU.
const at::Tensor& floats(PyObject* o, const char* name, ar_dtype* dt) {
    const at::Tensor& t = tensor(o, name);
    *dt = dtype_of(t, name);
    if (!t.is_cuda()) throw Refused(std::string(name) + " is not on a GPU");
    return t;
}

int index_bytes(const at::Tensor& t, const char* name) {
    if (t.scalar_type() == at::kLong) return 8;
    if (t.scalar_type() == at::kInt) return 4;
    throw Refused(std::string(name) + ": unsupported dtype " + c10::toString(t.scalar_type()) +
                  "; use int32 or int64");
}

void same_device(const at::Tensor& t, const char* name, const at::Tensor& like) {
    if (t.device() != like.device())
        throw Refused(std::string(name) + " is on " + t.device().str() + ", needs " +
                      like.device().str());
}

// t is dense, of this type and shape, on like's device; its address.
void* dense(const at::Tensor& t, const char* name, at::ScalarType type, at::IntArrayRef shape,
            const at::Tensor& like) {
    if (t.scalar_type() != type)
        throw Refused(std::string(name) + " has dtype " + c10::toString(t.scalar_type()) +
                      ", needs " + c10::toString(type));
    if (t.sizes() != shape)
        throw Refused(std::string(name) + " has shape " + shape_of(t) + ", needs another");
    same_device(t, name, like);
    if (!t.is_contiguous()) throw Refused(std::string(name) + " is not contiguous");
    return t.data_ptr();
}

// Elements from one row (the last dimension) to the next.  Rows are dense and
// evenly spaced, and do not overlap.
int64_t row_stride(const at::Tensor& t, const char* name) {
    const int64_t d = t.dim();
    if (d == 0) throw Refused(std::string(name) + " has no dimensions");
    const int64_t cols = t.size(d - 1);
    if (t.is_contiguous()) return cols;
    const auto uneven = [&] {
        throw Refused(std::string(name) + ": the rows of " + shape_of(t) +
                      " are not dense and evenly spaced");
    };
    if (cols > 1 && t.stride(d - 1) != 1) uneven();
    // leading dimensions from the inside: each has to continue the one below
    int64_t stride = -1, reach = 0;
    for (int64_t i = d - 2; i >= 0; --i) {
        if (t.size(i) == 1) continue;
        if (stride < 0) {
            stride = t.stride(i);
            reach = stride * t.size(i);
        } else {
            if (t.stride(i) != reach) uneven();
            reach *= t.size(i);
        }
    }
    if (stride < 0) return cols;
    if (stride < cols)
        throw Refused(std::string(name) + ": rows " + std::to_string(stride) +
                      " elements apart overlap");
    return stride;
}

at::Tensor make(at::IntArrayRef shape, at::ScalarType type, const at::Tensor& like) {
    return at::empty(shape, at::TensorOptions(type).device(like.device()));
}

struct Scratch {
    at::Tensor t;
    void* p = nullptr;
    size_t bytes = 0;
    Scratch(size_t n, const at::Tensor& like) : bytes(n) {
        if (!n) return;
        t = make({(int64_t)n}, at::kByte, like);
        p = t.data_ptr();
    }
};

int64_t whole(PyObject* o, const char* name) {
    const int64_t v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        throw Refused(std::string(name) + " is not a whole number");
    }
    return v;
}

double number(PyObject* o, const char* name) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) {
        PyErr_Clear();
        throw Refused(std::string(name) + " is not a number");
    }
    return v;
}

// A tuple of new references to the tensors.
template <class... T>
PyObject* tuple_of(const T&... t) {
    PyObject* out = PyTuple_New(sizeof...(T));
    if (!out) return nullptr;
    Py_ssize_t i = 0;
    bool ok = true;
    ((ok = ok && [&] {
        PyObject* o = THPVariable_Wrap(t);
        if (o) PyTuple_SET_ITEM(out, i++, o);
        return o != nullptr;
    }()), ...);
    if (!ok) {
        Py_DECREF(out);
        return nullptr;
    }
    return out;
}

void raise_ar_error(const Failed& f) {
    PyObject* mod = PyImport_ImportModule("ring_allreduce_rs_amd._lib");
    PyObject* cls = mod ? PyObject_GetAttrString(mod, "ArError") : nullptr;
    PyObject* err =
        cls ? PyObject_CallFunction(cls, "iss", (int)f.status, f.func, f.detail.c_str()) : nullptr;
    if (err) PyErr_SetObject(cls, err);
    Py_XDECREF(err);
    Py_XDECREF(cls);
    Py_XDECREF(mod);
}

// Runs body(); no C++ exception reaches Python.
template <class F>
PyObject* guarded(Py_ssize_t got, Py_ssize_t want, F body) {
    if (got != want) {
        PyErr_Format(PyExc_TypeError, "%zd arguments, needs %zd", got, want);
        return nullptr;
    }
    try {
        return body();
    } catch (const Refused& e) {
        PyErr_SetString(PyExc_ValueError, e.what());
    } catch (const Failed& f) {
        raise_ar_error(f);
    } catch (const c10::OutOfMemoryError& e) {
        PyObject* cls = nullptr;
        PyObject* mod = PyImport_ImportModule("torch");
        if (mod) cls = PyObject_GetAttrString(mod, "OutOfMemoryError");
        if (cls) PyErr_SetString(cls, e.what_without_backtrace());
        Py_XDECREF(cls);
        Py_XDECREF(mod);
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    } catch (...) {
        PyErr_SetString(PyExc_RuntimeError, "unexpected exception");
    }
    return nullptr;
}

// ------------------------------------------------------------------------ layer norm

// A norm's weight or bias (None: no array); its address and dtype.
const void* param(PyObject* o, const char* name, int64_t cols, const at::Tensor& like,
                  ar_dtype* dt) {
    if (o == Py_None) return nullptr;
    const at::Tensor& t = floats(o, name, dt);
    return dense(t, name, t.scalar_type(), {cols}, like);
}

PyObject* layer_norm(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded(n, 4, [&]() -> PyObject* {
        ar_dtype dt, wdt, bdt;
        const at::Tensor& x = floats(args[0], "x", &dt);
        const int64_t stride = row_stride(x, "x"), cols = x.size(-1);
        if (cols == 0) throw Refused("x has rows of no elements");
        wdt = bdt = dt;
        const void* w = param(args[1], "weight", cols, x, &wdt);
        const void* b = param(args[2], "bias", cols, x, &bdt);
        if (w && b && wdt != bdt) throw Refused("weight and bias need one dtype");
        const double eps = number(args[3], "eps");
        if (!(eps >= 0.0) || std::isinf((float)eps))
            throw Refused("eps is negative or not finite");
        const at::IntArrayRef lead = x.sizes().slice(0, x.dim() - 1);
        at::Tensor y = make(x.sizes(), x.scalar_type(), x);
        at::Tensor mean = make(lead, at::kFloat, x), rstd = make(lead, at::kFloat, x);
        ar_ctx* c = context(x.get_device());
        must(c, ar_layer_norm(c, x.data_ptr(), (size_t)stride, w, b, w ? wdt : bdt, y.data_ptr(),
                              static_cast<float*>(mean.data_ptr()),
                              static_cast<float*>(rstd.data_ptr()), (size_t)mean.numel(),
                              (size_t)cols, dt, (float)eps), "ar_layer_norm");
        return tuple_of(y, mean, rstd);
    });
}

PyObject* layer_norm_backward(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded(n, 5, [&]() -> PyObject* {
        ar_dtype dt, gdt, pdt;
        const at::Tensor& dy = floats(args[0], "dy", &gdt);
        const at::Tensor& x = floats(args[1], "x", &dt);
        if (gdt != dt || dy.sizes() != x.sizes() || dy.device() != x.device())
            throw Refused("dy " + shape_of(dy) + " does not match x " + shape_of(x) +
                          " in dtype, shape or device");
        const int64_t xs = row_stride(x, "x"), gs = row_stride(dy, "dy"), cols = x.size(-1);
        if (cols == 0) throw Refused("x has rows of no elements");
        const at::IntArrayRef lead = x.sizes().slice(0, x.dim() - 1);
        const at::Tensor& mean = tensor(args[2], "mean");
        const void* m = dense(mean, "mean", at::kFloat, lead, x);
        const void* r = dense(tensor(args[3], "rstd"), "rstd", at::kFloat, lead, x);
        pdt = dt;
        const void* w = param(args[4], "weight", cols, x, &pdt);
        const at::ScalarType p = pdt == AR_FLOAT32 ? at::kFloat : at::kBFloat16;
        const size_t rows = (size_t)mean.numel();
        size_t bytes = 0;
        must(nullptr, ar_layer_norm_backward_workspace(rows, (size_t)cols, dt, &bytes),
             "ar_layer_norm_backward_workspace");
        at::Tensor dx = make(x.sizes(), x.scalar_type(), x);
        at::Tensor dw = make({cols}, p, x), db = make({cols}, p, x);
        const Scratch ws(bytes, x);
        ar_ctx* c = context(x.get_device());
        must(c, ar_layer_norm_backward(c, dy.data_ptr(), (size_t)gs, x.data_ptr(), (size_t)xs,
                                       static_cast<const float*>(m), static_cast<const float*>(r),
                                       w, pdt, dx.data_ptr(), dw.data_ptr(), db.data_ptr(), rows,
                                       (size_t)cols, dt, ws.p, ws.bytes),
             "ar_layer_norm_backward");
        return tuple_of(dx, dw, db);
    });
}

// -------------------------------------------------------- tokens by expert and back

void check_experts(int64_t experts) {
    if (experts < 1 || experts > AR_MAX_EXPERTS)
        throw Refused("experts " + std::to_string(experts) + " outside [1, " +
                      std::to_string(AR_MAX_EXPERTS) + "]");
}

PyObject* expert_dispatch(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded(n, 3, [&]() -> PyObject* {
        ar_dtype dt;
        const at::Tensor& x = floats(args[0], "x", &dt);
        const at::Tensor& ids = tensor(args[1], "ids");
        const int64_t experts = whole(args[2], "experts");
        if (x.dim() != 2) throw Refused("x has shape " + shape_of(x) + ", needs (tokens, hidden)");
        if (ids.dim() != 2 || ids.size(0) != x.size(0))
            throw Refused("ids has shape " + shape_of(ids) + ", needs (tokens, topk) with x's tokens");
        const int ib = index_bytes(ids, "ids");
        const int64_t tokens = x.size(0), hidden = x.size(1), topk = ids.size(1);
        const void* i = dense(ids, "ids", ids.scalar_type(), ids.sizes(), x);
        if (topk == 0 || hidden == 0) throw Refused("topk and hidden have to be positive");
        if (topk > INT_MAX) throw Refused("topk above 2^31 - 1");
        check_experts(experts);
        const int64_t stride = row_stride(x, "x");
        size_t bytes = 0;
        must(nullptr, ar_expert_dispatch_workspace((size_t)tokens, (int)topk, (int)experts, &bytes),
             "ar_expert_dispatch_workspace");
        at::Tensor rows = make({tokens * topk, hidden}, x.scalar_type(), x);
        at::Tensor dest = make({tokens, topk}, at::kInt, x);
        at::Tensor slot = make({tokens * topk}, at::kInt, x);
        at::Tensor offsets = make({experts + 1}, at::kInt, x);
        const Scratch ws(bytes, x);
        ar_ctx* c = context(x.get_device());
        must(c, ar_expert_dispatch(c, x.data_ptr(), (size_t)stride, i, ib, (size_t)tokens, (int)topk,
                                   (int)experts, (size_t)hidden, dt, rows.data_ptr(),
                                   static_cast<int*>(dest.data_ptr()),
                                   static_cast<int*>(slot.data_ptr()),
                                   static_cast<int*>(offsets.data_ptr()), ws.p, ws.bytes),
             "ar_expert_dispatch");
        return tuple_of(rows, dest, slot, offsets);
    });
}

// The sizes and addresses that the calls after a dispatch take.
struct Plan {
    const int *dest, *offsets;
    int64_t tokens, topk, experts, hidden;
    Plan(PyObject* d, PyObject* o, const at::Tensor& rows, const char* name) {
        const at::Tensor &td = tensor(d, "plan.dest"), &to = tensor(o, "plan.offsets");
        if (td.dim() != 2 || td.size(1) == 0 || td.size(1) > INT_MAX)
            throw Refused("plan.dest has shape " + shape_of(td) + ", needs (tokens, topk)");
        if (to.dim() != 1 || to.size(0) < 2)
            throw Refused("plan.offsets has shape " + shape_of(to) + ", needs (experts + 1,)");
        tokens = td.size(0);
        topk = td.size(1);
        experts = to.size(0) - 1;
        check_experts(experts);
        dest = static_cast<const int*>(dense(td, "plan.dest", at::kInt, td.sizes(), rows));
        offsets = static_cast<const int*>(dense(to, "plan.offsets", at::kInt, to.sizes(), rows));
        if (rows.dim() != 2 || rows.size(0) != tokens * topk || rows.size(1) == 0)
            throw Refused(std::string(name) + " has shape " + shape_of(rows) + ", needs (" +
                          std::to_string(tokens * topk) + ", hidden)");
        if (!rows.is_contiguous()) throw Refused(std::string(name) + " is not contiguous");
        hidden = rows.size(1);
    }
};

PyObject* expert_dispatch_backward(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded(n, 3, [&]() -> PyObject* {
        ar_dtype dt;
        const at::Tensor& drows = floats(args[0], "drows", &dt);
        const Plan p(args[1], args[2], drows, "drows");
        at::Tensor dx = make({p.tokens, p.hidden}, drows.scalar_type(), drows);
        ar_ctx* c = context(drows.get_device());
        must(c, ar_expert_dispatch_backward(c, drows.data_ptr(), p.dest, p.offsets,
                                            (size_t)p.tokens, (int)p.topk, (int)p.experts,
                                            (size_t)p.hidden, dt, dx.data_ptr()),
             "ar_expert_dispatch_backward");
        return THPVariable_Wrap(dx);
    });
}

PyObject* expert_combine(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded(n, 4, [&]() -> PyObject* {
        ar_dtype dt;
        const at::Tensor& rows = floats(args[0], "rows", &dt);
        const Plan p(args[2], args[3], rows, "rows");
        const void* w = dense(tensor(args[1], "weights"), "weights", at::kFloat, {p.tokens, p.topk},
                              rows);
        at::Tensor y = make({p.tokens, p.hidden}, rows.scalar_type(), rows);
        ar_ctx* c = context(rows.get_device());
        must(c, ar_expert_combine(c, rows.data_ptr(), static_cast<const float*>(w), p.dest,
                                  p.offsets, (size_t)p.tokens, (int)p.topk, (int)p.experts,
                                  (size_t)p.hidden, dt, y.data_ptr()), "ar_expert_combine");
        return THPVariable_Wrap(y);
    });
}

PyObject* expert_combine_backward(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded(n, 5, [&]() -> PyObject* {
        ar_dtype dt, gdt;
        const at::Tensor& dy = floats(args[0], "dy", &gdt);
        const at::Tensor& rows = floats(args[1], "rows", &dt);
        const Plan p(args[3], args[4], rows, "rows");
        const void* w = dense(tensor(args[2], "weights"), "weights", at::kFloat, {p.tokens, p.topk},
                              rows);
        if (gdt != dt || dy.sizes() != at::IntArrayRef({p.tokens, p.hidden}) ||
            dy.device() != rows.device())
            throw Refused("dy " + shape_of(dy) + " does not match rows " + shape_of(rows) +
                          " in dtype, shape or device");
        const int64_t stride = row_stride(dy, "dy");
        at::Tensor drows = make(rows.sizes(), rows.scalar_type(), rows);
        at::Tensor dw = make({p.tokens, p.topk}, at::kFloat, rows);
        ar_ctx* c = context(rows.get_device());
        must(c, ar_expert_combine_backward(c, dy.data_ptr(), (size_t)stride, rows.data_ptr(),
                                           static_cast<const float*>(w), p.dest, p.offsets,
                                           (size_t)p.tokens, (int)p.topk, (int)p.experts,
                                           (size_t)p.hidden, dt, drows.data_ptr(),
                                           static_cast<float*>(dw.data_ptr())),
             "ar_expert_combine_backward");
        return tuple_of(drows, dw);
    });
}

// ---------------------------------------------------------------------- distillation

// What the three calls share.
struct Distill {
    const at::Tensor& logits;
    ar_dtype dt;
    int64_t rows, vocab, top, stride;
    int ib;
    const void *indices, *teacher;
    float temperature;
    Distill(PyObject* l, PyObject* i, PyObject* t, PyObject* T) : logits(floats(l, "logits", &dt)) {
        if (logits.dim() != 2)
            throw Refused("logits has shape " + shape_of(logits) + ", needs (rows, vocab)");
        rows = logits.size(0);
        vocab = logits.size(1);
        const at::Tensor& at_ = tensor(i, "indices");
        if (at_.dim() != 2 || at_.size(0) != rows)
            throw Refused("indices has shape " + shape_of(at_) +
                          ", needs (rows, top) with the logits' rows");
        ib = index_bytes(at_, "indices");
        top = at_.size(1);
        indices = dense(at_, "indices", at_.scalar_type(), at_.sizes(), logits);
        teacher = dense(tensor(t, "teacher"), "teacher", logits.scalar_type(), at_.sizes(), logits);
        if (vocab == 0 || top < 1 || top > AR_DISTILL_MAX_TOP)
            throw Refused("vocab " + std::to_string(vocab) + " is 0 or top " + std::to_string(top) +
                          " outside [1, " + std::to_string(AR_DISTILL_MAX_TOP) + "]");
        temperature = (float)number(T, "temperature");
        if (!(temperature >= FLT_MIN) || std::isinf(temperature))
            throw Refused("temperature is not positive, normal and finite");
        stride = row_stride(logits, "logits");
    }
    const float* per_row(PyObject* o, const char* name) const {
        return static_cast<const float*>(dense(tensor(o, name), name, at::kFloat, {rows}, logits));
    }
    size_t workspace(int gradient) const {
        size_t bytes = 0;
        must(nullptr, ar_distill_workspace((size_t)rows, (size_t)vocab, (size_t)top, dt, gradient,
                                           &bytes), "ar_distill_workspace");
        return bytes;
    }
};

PyObject* distill_loss(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded(n, 4, [&]() -> PyObject* {
        const Distill d(args[0], args[1], args[2], args[3]);
        at::Tensor loss = make({d.rows}, at::kFloat, d.logits);
        at::Tensor lse = make({d.rows}, at::kFloat, d.logits);
        const Scratch ws(d.workspace(0), d.logits);
        ar_ctx* c = context(d.logits.get_device());
        must(c, ar_distill_loss(c, d.logits.data_ptr(), (size_t)d.stride, d.indices, d.ib, d.teacher,
                                (size_t)d.rows, (size_t)d.vocab, (size_t)d.top, d.dt, d.temperature,
                                static_cast<float*>(loss.data_ptr()),
                                static_cast<float*>(lse.data_ptr()), ws.p, ws.bytes),
             "ar_distill_loss");
        return tuple_of(loss, lse);
    });
}

PyObject* distill_backward(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded(n, 6, [&]() -> PyObject* {
        const Distill d(args[1], args[2], args[3], args[5]);
        const float *g = d.per_row(args[0], "dloss"), *lse = d.per_row(args[4], "lse");
        at::Tensor out = make({d.rows, d.vocab}, d.logits.scalar_type(), d.logits);
        ar_ctx* c = context(d.logits.get_device());
        must(c, ar_distill_backward(c, g, d.logits.data_ptr(), (size_t)d.stride, d.indices, d.ib,
                                    d.teacher, lse, (size_t)d.rows, (size_t)d.vocab, (size_t)d.top,
                                    d.dt, d.temperature, out.data_ptr()), "ar_distill_backward");
        return THPVariable_Wrap(out);
    });
}

PyObject* distill_step(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded(n, 5, [&]() -> PyObject* {
        const Distill d(args[1], args[2], args[3], args[4]);
        const float* g = d.per_row(args[0], "dloss");
        at::Tensor loss = make({d.rows}, at::kFloat, d.logits);
        at::Tensor out = make({d.rows, d.vocab}, d.logits.scalar_type(), d.logits);
        const Scratch ws(d.workspace(1), d.logits);
        ar_ctx* c = context(d.logits.get_device());
        must(c, ar_distill_step(c, g, d.logits.data_ptr(), (size_t)d.stride, d.indices, d.ib,
                                d.teacher, (size_t)d.rows, (size_t)d.vocab, (size_t)d.top, d.dt,
                                d.temperature, static_cast<float*>(loss.data_ptr()), out.data_ptr(),
                                ws.p, ws.bytes), "ar_distill_step");
        return tuple_of(loss, out);
    });
}

// ------------------------------------------------------------------------- embedding

// ids: any shape, dense, on like's device.
const void* token_ids(const at::Tensor& ids, const at::Tensor& like, int* ib) {
    *ib = index_bytes(ids, "ids");
    return dense(ids, "ids", ids.scalar_type(), ids.sizes(), like);
}

float finite(PyObject* o, const char* name) {
    const float v = (float)number(o, name);
    if (!std::isfinite(v)) throw Refused(std::string(name) + " is not finite");
    return v;
}

PyObject* embedding(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded(n, 3, [&]() -> PyObject* {
        ar_dtype dt;
        int ib;
        const at::Tensor& table = floats(args[0], "table", &dt);
        if (table.dim() != 2 || table.size(0) == 0 || table.size(1) == 0)
            throw Refused("table has shape " + shape_of(table) + ", needs (vocab, hidden)");
        if (!table.is_contiguous()) throw Refused("table is not contiguous");
        const at::Tensor& ids = tensor(args[1], "ids");
        const void* i = token_ids(ids, table, &ib);
        const float scale = finite(args[2], "scale");
        c10::SmallVector<int64_t, 6> shape(ids.sizes().begin(), ids.sizes().end());
        shape.push_back(table.size(1));
        at::Tensor y = make(shape, table.scalar_type(), table);
        ar_ctx* c = context(table.get_device());
        must(c, ar_embedding(c, table.data_ptr(), i, ib, (size_t)ids.numel(), (size_t)table.size(0),
                             (size_t)table.size(1), dt, scale, y.data_ptr()), "ar_embedding");
        return THPVariable_Wrap(y);
    });
}

PyObject* embedding_backward(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded(n, 4, [&]() -> PyObject* {
        ar_dtype dt;
        int ib;
        const at::Tensor& dy = floats(args[0], "dy", &dt);
        const at::Tensor& ids = tensor(args[1], "ids");
        const void* i = token_ids(ids, dy, &ib);
        if (dy.dim() != ids.dim() + 1 || dy.sizes().slice(0, ids.dim()) != ids.sizes() ||
            dy.size(-1) == 0)
            throw Refused("dy " + shape_of(dy) + " does not match ids " + shape_of(ids));
        const int64_t vocab = whole(args[2], "vocab"), hidden = dy.size(-1);
        if (vocab < 1) throw Refused("vocab " + std::to_string(vocab) + " below 1");
        const float scale = finite(args[3], "scale");
        const int64_t stride = row_stride(dy, "dy");
        const size_t tokens = (size_t)ids.numel();
        size_t bytes = 0;
        must(nullptr, ar_embedding_backward_workspace(tokens, (size_t)vocab, (size_t)hidden, dt,
                                                      &bytes), "ar_embedding_backward_workspace");
        at::Tensor dtable = make({vocab, hidden}, dy.scalar_type(), dy);
        const Scratch ws(bytes, dy);
        ar_ctx* c = context(dy.get_device());
        must(c, ar_embedding_backward(c, dy.data_ptr(), (size_t)stride, i, ib, tokens, (size_t)vocab,
                                      (size_t)hidden, dt, scale, dtable.data_ptr(), ws.p, ws.bytes),
             "ar_embedding_backward");
        return THPVariable_Wrap(dtable);
    });
}

// ------------------------------------------------------------------ the experts' products

// The rows of a product: a matrix with rows at any stride.
struct Rows {
    const at::Tensor& t;
    ar_dtype dt;
    int64_t stride;
    Rows(PyObject* o, const char* name) : t(floats(o, name, &dt)) {
        if (t.dim() != 2 || t.size(1) == 0)
            throw Refused(std::string(name) + " has shape " + shape_of(t) + ", needs (rows, width)");
        stride = row_stride(t, name);
    }
};

const int* plan_offsets(PyObject* o, const at::Tensor& like, int64_t* experts) {
    const at::Tensor& t = tensor(o, "plan.offsets");
    if (t.dim() != 1 || t.size(0) < 2)
        throw Refused("plan.offsets has shape " + shape_of(t) + ", needs (experts + 1,)");
    *experts = t.size(0) - 1;
    check_experts(*experts);
    return static_cast<const int*>(dense(t, "plan.offsets", at::kInt, t.sizes(), like));
}

// The rows of a product are those of the plan's dispatch, as many as it has slots.
void plan_rows(PyObject* o, const at::Tensor& rows, const char* name) {
    const at::Tensor& t = tensor(o, "plan.dest");
    if (t.dim() != 2 || t.size(1) == 0)
        throw Refused("plan.dest has shape " + shape_of(t) + ", needs (tokens, topk)");
    dense(t, "plan.dest", at::kInt, t.sizes(), rows);
    if (rows.size(0) != t.numel())
        throw Refused(std::string(name) + " has shape " + shape_of(rows) + ", needs the plan's " +
                      std::to_string(t.numel()) + " rows");
}

size_t product_workspace(ar_expert_product p, int64_t rows, int64_t experts, int64_t hidden,
                         int64_t out, ar_dtype dt) {
    size_t bytes = 0;
    must(nullptr, ar_expert_matmul_workspace(p, (size_t)rows, (int)experts, (size_t)hidden,
                                             (size_t)out, dt, &bytes), "ar_expert_matmul_workspace");
    return bytes;
}

// ar_expert_matmul (KIND AR_EXPERT_FORWARD) or ar_expert_matmul_drows
template <ar_expert_product KIND>
PyObject* product_of_rows(PyObject* const* args, Py_ssize_t n, const char* name) {
    return guarded(n, 4, [&]() -> PyObject* {
        constexpr bool kForward = KIND == AR_EXPERT_FORWARD;
        const Rows r(args[0], name);
        const at::Tensor& w = tensor(args[1], "weights");
        if (w.dim() != 3 || w.size(1) == 0 || w.size(2) == 0)
            throw Refused("weights has shape " + shape_of(w) + ", needs (experts, out, hidden)");
        const int64_t out = w.size(1), hidden = w.size(2), rows = r.t.size(0);
        const void* wp = dense(w, "weights", r.t.scalar_type(), w.sizes(), r.t);
        if (r.t.size(1) != (kForward ? hidden : out))
            throw Refused(std::string(name) + " " + shape_of(r.t) + " does not match weights " +
                          shape_of(w));
        int64_t experts;
        const int* offsets = plan_offsets(args[3], r.t, &experts);
        if (experts != w.size(0))
            throw Refused("weights " + shape_of(w) + " are not of the plan's " +
                          std::to_string(experts) + " experts");
        plan_rows(args[2], r.t, name);
        at::Tensor y = make({rows, kForward ? out : hidden}, r.t.scalar_type(), r.t);
        const Scratch ws(product_workspace(KIND, rows, experts, hidden, out, r.dt), r.t);
        ar_ctx* c = context(r.t.get_device());
        must(c, (kForward ? ar_expert_matmul : ar_expert_matmul_drows)(
                    c, r.t.data_ptr(), (size_t)r.stride, wp, offsets, (size_t)rows, (int)experts,
                    (size_t)hidden, (size_t)out, r.dt, y.data_ptr(), ws.p, ws.bytes),
             kForward ? "ar_expert_matmul" : "ar_expert_matmul_drows");
        return THPVariable_Wrap(y);
    });
}

PyObject* expert_matmul(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return product_of_rows<AR_EXPERT_FORWARD>(args, n, "rows");
}

PyObject* expert_matmul_drows(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return product_of_rows<AR_EXPERT_DROWS>(args, n, "dout");
}

PyObject* expert_matmul_dweights(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded(n, 4, [&]() -> PyObject* {
        const Rows d(args[0], "dout"), r(args[1], "rows");
        if (d.dt != r.dt || d.t.size(0) != r.t.size(0) || d.t.device() != r.t.device())
            throw Refused("dout " + shape_of(d.t) + " does not match rows " + shape_of(r.t) +
                          " in dtype, rows or device");
        int64_t experts;
        const int* offsets = plan_offsets(args[3], r.t, &experts);
        plan_rows(args[2], r.t, "rows");
        const int64_t rows = r.t.size(0), hidden = r.t.size(1), out = d.t.size(1);
        const size_t bytes = product_workspace(AR_EXPERT_DWEIGHTS, rows, experts, hidden, out, r.dt);
        at::Tensor dw = make({experts, out, hidden}, r.t.scalar_type(), r.t);
        const Scratch ws(bytes, r.t);
        ar_ctx* c = context(r.t.get_device());
        must(c, ar_expert_matmul_dweights(c, d.t.data_ptr(), (size_t)d.stride, r.t.data_ptr(),
                                          (size_t)r.stride, offsets, (size_t)rows, (int)experts,
                                          (size_t)hidden, (size_t)out, r.dt, dw.data_ptr(), ws.p,
                                          ws.bytes), "ar_expert_matmul_dweights");
        return THPVariable_Wrap(dw);
    });
}

// ------------------------------------------------------ checkpoints in 8 bits and the gate

int64_t groups_of(int64_t cols) { return (cols + AR_SAVE_GROUP - 1) / AR_SAVE_GROUP; }

// The shape `lead` + the given dimensions.
template <class... N>
c10::SmallVector<int64_t, 6> shape_with(at::IntArrayRef lead, N... n) {
    c10::SmallVector<int64_t, 6> s(lead.begin(), lead.end());
    (s.push_back(n), ...);
    return s;
}

// A checkpoint's tensors; its rows have to be dense.
struct Saved {
    const at::Tensor& codes;
    signed char* c;
    unsigned char* s;
    Saved(PyObject* co, PyObject* so) : codes(tensor(co, "saved.codes")) {
        if (!codes.is_cuda()) throw Refused("saved.codes is not on a GPU");
        if (codes.dim() == 0 || codes.size(-1) == 0)
            throw Refused("saved.codes has shape " + shape_of(codes) + ", needs (..., values)");
        c = static_cast<signed char*>(dense(codes, "saved.codes", at::kChar, codes.sizes(), codes));
        s = static_cast<unsigned char*>(
            dense(tensor(so, "saved.scales"), "saved.scales", at::kByte,
                  shape_with(codes.sizes().slice(0, codes.dim() - 1), groups_of(codes.size(-1))),
                  codes));
    }
};

PyObject* save_8bit(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded(n, 1, [&]() -> PyObject* {
        ar_dtype dt;
        const at::Tensor& x = floats(args[0], "x", &dt);
        const int64_t stride = row_stride(x, "x"), cols = x.size(-1);
        if (cols == 0) throw Refused("x has rows of no elements");
        at::Tensor codes = make(x.sizes(), at::kChar, x);
        at::Tensor scales =
            make(shape_with(x.sizes().slice(0, x.dim() - 1), groups_of(cols)), at::kByte, x);
        ar_ctx* c = context(x.get_device());
        must(c, ar_save_8bit(c, x.data_ptr(), (size_t)stride, (size_t)(x.numel() / cols),
                             (size_t)cols, dt, static_cast<signed char*>(codes.data_ptr()),
                             static_cast<unsigned char*>(scales.data_ptr())), "ar_save_8bit");
        return tuple_of(codes, scales);
    });
}

PyObject* restore_8bit(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded(n, 3, [&]() -> PyObject* {
        const Saved v(args[0], args[1]);
        const int64_t eb = whole(args[2], "dtype"), cols = v.codes.size(-1);
        if (eb != 2 && eb != 4) throw Refused("dtype is neither bfloat16 nor float32");
        at::Tensor x = make(v.codes.sizes(), eb == 2 ? at::kBFloat16 : at::kFloat, v.codes);
        ar_ctx* c = context(x.get_device());
        must(c, ar_restore_8bit(c, v.c, v.s, (size_t)(x.numel() / cols), (size_t)cols,
                                eb == 2 ? AR_BFLOAT16 : AR_FLOAT32, x.data_ptr()),
             "ar_restore_8bit");
        return THPVariable_Wrap(x);
    });
}

PyObject* silu_gate(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded(n, 1, [&]() -> PyObject* {
        ar_dtype dt;
        const at::Tensor& h = floats(args[0], "h", &dt);
        const int64_t stride = row_stride(h, "h");
        if (h.size(-1) == 0 || h.size(-1) % 2)
            throw Refused("h has shape " + shape_of(h) + ", needs (..., 2 n)");
        const int64_t cols = h.size(-1) / 2, rows = h.numel() / (2 * cols);
        const at::IntArrayRef lead = h.sizes().slice(0, h.dim() - 1);
        at::Tensor acts = make(shape_with(lead, cols), h.scalar_type(), h);
        at::Tensor codes = make(shape_with(lead, 2, cols), at::kChar, h);
        at::Tensor scales = make(shape_with(lead, 2, groups_of(cols)), at::kByte, h);
        ar_ctx* c = context(h.get_device());
        must(c, ar_silu_gate(c, h.data_ptr(), (size_t)stride, (size_t)rows, (size_t)cols, dt,
                             acts.data_ptr(), static_cast<signed char*>(codes.data_ptr()),
                             static_cast<unsigned char*>(scales.data_ptr())), "ar_silu_gate");
        return tuple_of(acts, codes, scales);
    });
}

PyObject* silu_gate_backward(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded(n, 3, [&]() -> PyObject* {
        ar_dtype dt;
        const at::Tensor& d = floats(args[0], "dacts", &dt);
        const int64_t stride = row_stride(d, "dacts"), cols = d.size(-1);
        const Saved v(args[1], args[2]);
        const at::IntArrayRef lead = d.sizes().slice(0, d.dim() - 1);
        if (v.codes.sizes() != at::IntArrayRef(shape_with(lead, 2, cols)))
            throw Refused("saved.codes " + shape_of(v.codes) + " does not match dacts " +
                          shape_of(d));
        same_device(v.codes, "saved.codes", d);
        at::Tensor dh = make(shape_with(lead, 2 * cols), d.scalar_type(), d);
        at::Tensor acts = make(d.sizes(), d.scalar_type(), d);
        ar_ctx* c = context(d.get_device());
        must(c, ar_silu_gate_backward(c, d.data_ptr(), (size_t)stride, v.c, v.s,
                                      (size_t)(d.numel() / cols), (size_t)cols, dt, dh.data_ptr(),
                                      acts.data_ptr()), "ar_silu_gate_backward");
        return tuple_of(dh, acts);
    });
}

#define ENTRY(name) \
    {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(name)), METH_FASTCALL, nullptr}
PyMethodDef kMethods[] = {
    ENTRY(layer_norm),      ENTRY(layer_norm_backward),     ENTRY(expert_dispatch),
    ENTRY(expert_combine),  ENTRY(expert_dispatch_backward), ENTRY(expert_combine_backward),
    ENTRY(distill_loss),    ENTRY(distill_backward),        ENTRY(distill_step),
    ENTRY(embedding),       ENTRY(embedding_backward),      ENTRY(expert_matmul),
    ENTRY(expert_matmul_drows), ENTRY(expert_matmul_dweights), ENTRY(save_8bit),
    ENTRY(restore_8bit),    ENTRY(silu_gate),               ENTRY(silu_gate_backward),
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_torch_ops", nullptr, -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__torch_ops(void) { return PyModule_Create(&kModule); }
