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

#define ENTRY(name) \
    {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(name)), METH_FASTCALL, nullptr}
PyMethodDef kMethods[] = {
    ENTRY(layer_norm),      ENTRY(layer_norm_backward),     ENTRY(expert_dispatch),
    ENTRY(expert_combine),  ENTRY(expert_dispatch_backward), ENTRY(expert_combine_backward),
    ENTRY(distill_loss),    ENTRY(distill_backward),        ENTRY(distill_step),
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_torch_ops", nullptr, -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__torch_ops(void) { return PyModule_Create(&kModule); }
