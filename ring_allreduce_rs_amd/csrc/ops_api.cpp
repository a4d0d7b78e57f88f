// ops_api.cpp -- the C entry points of the training operators declared in
// include/ar.h: argument validation and error reporting.  The kernels live in
// norm.hip, route.hip and distill.hip.
#include <hip/hip_runtime_api.h>

#include <cfloat>
#include <climits>
#include <cmath>
#include <cstdint>

#include "ar.h"
#include "ctx.h"
#include "ops.h"
#include "ops_args.h"

using arlib::fail;
using arlib::Arrays;
using arlib::bad_size;
using arlib::check_index_bytes;
using arlib::float_bytes;
using arlib::guarded;
using arlib::kMostCols;
using arlib::launched;
using arlib::strided_bytes;
using arlib::times;
using arlib::workspace;

namespace {

size_t norm_workspace(size_t rows, size_t cols, size_t eb) {
    return arlib::norm_grad_parts(rows, cols, (int)eb) * 2 * cols * sizeof(float);
}

// What the calls over tokens and experts share.
ar_status check_route(ar_ctx* ctx, size_t tokens, int topk, int experts, size_t hidden, int dtype,
                      size_t* eb, size_t* slots, size_t* row_bytes) {
    *eb = float_bytes(dtype);
    if (!*eb) return fail(ctx, AR_ERR_INVALID_ARG, "unknown or unsupported dtype %d", dtype);
    if (topk < 1) return fail(ctx, AR_ERR_INVALID_ARG, "topk %d below 1", topk);
    if (experts < 1) return fail(ctx, AR_ERR_INVALID_ARG, "experts %d below 1", experts);
    if (hidden < 1) return fail(ctx, AR_ERR_INVALID_ARG, "hidden is 0");
    if (experts > AR_MAX_EXPERTS)
        return fail(ctx, AR_ERR_UNSUPPORTED, "experts %d above %d", experts, AR_MAX_EXPERTS);
    if (hidden > kMostCols)
        return fail(ctx, AR_ERR_UNSUPPORTED, "hidden %zu above 2^28", hidden);
    size_t bytes;
    if (!times(tokens, (size_t)topk, slots) || !times(hidden, *eb, row_bytes) ||
        !times(*slots, *row_bytes, &bytes))
        return bad_size(ctx);
    if (*slots > (size_t)INT_MAX)
        return fail(ctx, AR_ERR_UNSUPPORTED, "tokens * topk = %zu above 2^31 - 1", *slots);
    return AR_OK;
}

// The arguments that the distillation calls share; fills d and the arrays.
ar_status check_distill(ar_ctx* ctx, Arrays& arrays, arlib::DistillArgs& d, const void* logits,
                        size_t stride, const void* indices, int index_bytes, const void* teacher,
                        size_t rows, size_t vocab, size_t top, int dtype, float temperature) {
    const size_t eb = float_bytes(dtype);
    if (!eb) return fail(ctx, AR_ERR_INVALID_ARG, "unknown or unsupported dtype %d", dtype);
    const ar_status s = check_index_bytes(ctx, index_bytes);
    if (s != AR_OK) return s;
    if (vocab < 1 || top < 1) return fail(ctx, AR_ERR_INVALID_ARG, "vocab or top is 0");
    if (vocab > kMostCols)
        return fail(ctx, AR_ERR_UNSUPPORTED, "vocab %zu above 2^28", vocab);
    if (top > AR_DISTILL_MAX_TOP)
        return fail(ctx, AR_ERR_UNSUPPORTED, "top %zu above %d", top, AR_DISTILL_MAX_TOP);
    // (the kernels multiply by log2(e) / T, which overflows below the normal numbers)
    if (!(temperature >= FLT_MIN) || std::isinf(temperature))
        return fail(ctx, AR_ERR_INVALID_ARG, "temperature %g is not positive, normal and finite",
                    (double)temperature);
    if (rows > 1 && stride < vocab)
        return fail(ctx, AR_ERR_INVALID_ARG, "logits_stride %zu below vocab %zu", stride, vocab);
    size_t lbytes, places, ibytes, tbytes;
    if (!strided_bytes(rows, vocab, stride, eb, &lbytes) || !times(rows, top, &places) ||
        !times(places, (size_t)index_bytes, &ibytes) || !times(places, eb, &tbytes))
        return bad_size(ctx);
    arrays.in(logits, lbytes, eb, "logits");
    arrays.in(indices, ibytes, (size_t)index_bytes, "indices");
    arrays.in(teacher, tbytes, eb, "teacher");
    d = {};
    d.logits = logits;
    d.indices = indices;
    d.teacher = teacher;
    d.lstride = stride;
    d.rows = rows;
    d.vocab = vocab;
    d.top = top;
    d.temperature = temperature;
    d.eb = (int)eb;
    d.ib = index_bytes;
    return AR_OK;
}

}  // namespace

#pragma GCC visibility push(default)
extern "C" {

ar_status ar_set_operator_checks(ar_ctx* ctx, int enable) {
    if (!ctx) return fail(nullptr, AR_ERR_INVALID_ARG, "ctx is NULL");
    ctx->operator_checks = enable != 0;
    return AR_OK;
}

ar_status ar_layer_norm(ar_ctx* ctx, const void* x, size_t x_stride, const void* weight,
                        const void* bias, ar_dtype param_dtype, void* y, float* mean, float* rstd,
                        size_t rows, size_t cols, ar_dtype dtype, float eps) {
    return guarded(ctx, [&]() -> ar_status {
        const size_t eb = float_bytes((int)dtype), pb = float_bytes((int)param_dtype);
        if (!eb || !pb)
            return fail(ctx, AR_ERR_INVALID_ARG, "unknown or unsupported dtype %d / %d", (int)dtype,
                        (int)param_dtype);
        if (cols < 1) return fail(ctx, AR_ERR_INVALID_ARG, "cols is 0");
        if (!(eps >= 0.0f) || std::isinf(eps))
            return fail(ctx, AR_ERR_INVALID_ARG, "eps %g is negative or not finite", (double)eps);
        if (cols > kMostCols)
            return fail(ctx, AR_ERR_UNSUPPORTED, "cols %zu above 2^28", cols);
        if (rows > 1 && x_stride < cols)
            return fail(ctx, AR_ERR_INVALID_ARG, "x_stride %zu below cols %zu", x_stride, cols);
        size_t xbytes, ybytes, pbytes, sbytes;
        if (!strided_bytes(rows, cols, x_stride, eb, &xbytes) ||
            !strided_bytes(rows, cols, cols, eb, &ybytes) || !times(cols, pb, &pbytes) ||
            !times(rows, sizeof(float), &sbytes))
            return bad_size(ctx);
        Arrays arrays(ctx);
        arrays.in(x, xbytes, eb, "x");
        if (weight) arrays.in(weight, pbytes, pb, "weight");
        if (bias) arrays.in(bias, pbytes, pb, "bias");
        arrays.out(y, ybytes, eb, "y");
        arrays.out(mean, sbytes, 4, "mean");
        arrays.out(rstd, sbytes, 4, "rstd");
        const ar_status s = arrays.check();
        if (s != AR_OK) return s;
        arlib::NormArgs a{x, weight, bias, y, mean, rstd, x_stride, rows, cols, eps, (int)eb,
                          (int)pb};
        return launched(ctx, arlib::launch_norm(a, ctx->stream), "layer norm");
    });
}

ar_status ar_layer_norm_backward(ar_ctx* ctx, const void* dy, size_t dy_stride, const void* x,
                                 size_t x_stride, const float* mean, const float* rstd,
                                 const void* weight, ar_dtype param_dtype, void* dx, void* dweight,
                                 void* dbias, size_t rows, size_t cols, ar_dtype dtype,
                                 void* workspace_, size_t workspace_bytes) {
    return guarded(ctx, [&]() -> ar_status {
        const size_t eb = float_bytes((int)dtype), pb = float_bytes((int)param_dtype);
        if (!eb || !pb)
            return fail(ctx, AR_ERR_INVALID_ARG, "unknown or unsupported dtype %d / %d", (int)dtype,
                        (int)param_dtype);
        if (cols < 1) return fail(ctx, AR_ERR_INVALID_ARG, "cols is 0");
        if (cols > kMostCols)
            return fail(ctx, AR_ERR_UNSUPPORTED, "cols %zu above 2^28", cols);
        if (rows > 1 && x_stride < cols)
            return fail(ctx, AR_ERR_INVALID_ARG, "x_stride %zu below cols %zu", x_stride, cols);
        if (rows > 1 && dy_stride < cols)
            return fail(ctx, AR_ERR_INVALID_ARG, "dy_stride %zu below cols %zu", dy_stride, cols);
        size_t xbytes, gbytes, ybytes, pbytes, sbytes;
        if (!strided_bytes(rows, cols, x_stride, eb, &xbytes) ||
            !strided_bytes(rows, cols, dy_stride, eb, &gbytes) ||
            !strided_bytes(rows, cols, cols, eb, &ybytes) || !times(cols, pb, &pbytes) ||
            !times(rows, sizeof(float), &sbytes))
            return bad_size(ctx);
        Arrays arrays(ctx);
        arrays.in(dy, gbytes, eb, "dy");
        arrays.in(x, xbytes, eb, "x");
        arrays.in(mean, sbytes, 4, "mean");
        arrays.in(rstd, sbytes, 4, "rstd");
        if (weight) arrays.in(weight, pbytes, pb, "weight");
        arrays.out(dx, ybytes, eb, "dx");
        if (dweight) arrays.out(dweight, pbytes, pb, "dweight");
        if (dbias) arrays.out(dbias, pbytes, pb, "dbias");
        const size_t need = dweight || dbias ? norm_workspace(rows, cols, eb) : 0;
        ar_status s = workspace(ctx, arrays, workspace_, workspace_bytes, need);
        if (s == AR_OK) s = arrays.check();
        if (s != AR_OK) return s;
        arlib::NormGradArgs a{dy,        x,        mean, rstd, weight, dx,      dweight, dbias,
                              static_cast<float*>(workspace_), dy_stride, x_stride, rows, cols,
                              (int)eb,   (int)pb};
        return launched(ctx, arlib::launch_norm_grad(a, ctx->stream), "layer norm gradient");
    });
}

ar_status ar_layer_norm_backward_workspace(size_t rows, size_t cols, ar_dtype dtype,
                                           size_t* bytes) {
    const size_t eb = float_bytes((int)dtype);
    if (!bytes || !eb || cols < 1) return AR_ERR_INVALID_ARG;
    if (cols > kMostCols) return AR_ERR_UNSUPPORTED;
    *bytes = norm_workspace(rows, cols, eb);
    return AR_OK;
}

ar_status ar_expert_dispatch(ar_ctx* ctx, const void* x, size_t x_stride, const void* ids,
                             int index_bytes, size_t tokens, int topk, int experts, size_t hidden,
                             ar_dtype dtype, void* rows, int* dest, int* slot, int* offsets,
                             void* workspace_, size_t workspace_bytes) {
    return guarded(ctx, [&]() -> ar_status {
        size_t eb, slots, row_bytes, xbytes;
        ar_status s = check_route(ctx, tokens, topk, experts, hidden, (int)dtype, &eb, &slots,
                                  &row_bytes);
        if (s == AR_OK) s = check_index_bytes(ctx, index_bytes);
        if (s != AR_OK) return s;
        if (tokens > 1 && x_stride < hidden)
            return fail(ctx, AR_ERR_INVALID_ARG, "x_stride %zu below hidden %zu", x_stride, hidden);
        if (!strided_bytes(tokens, hidden, x_stride, eb, &xbytes)) return bad_size(ctx);
        Arrays arrays(ctx);
        arrays.in(x, xbytes, eb, "x");
        arrays.in(ids, slots * (size_t)index_bytes, (size_t)index_bytes, "ids");
        arrays.out(rows, slots * row_bytes, eb, "rows");
        arrays.out(dest, slots * sizeof(int), 4, "dest");
        arrays.out(slot, slots * sizeof(int), 4, "slot");
        arrays.out(offsets, ((size_t)experts + 1) * sizeof(int), 4, "offsets");
        s = workspace(ctx, arrays, workspace_, workspace_bytes,
                      arlib::dispatch_work_ints(tokens, topk, experts) * sizeof(int));
        if (s == AR_OK) s = arrays.check();
        if (s != AR_OK) return s;
        arlib::DispatchArgs a{x,       ids,    rows,        dest, slot,    offsets,
                              static_cast<int*>(workspace_), x_stride, hidden, (int)tokens, topk,
                              experts, (int)eb, index_bytes};
        return launched(ctx, arlib::launch_dispatch(a, ctx->stream), "expert dispatch");
    });
}

ar_status ar_expert_dispatch_workspace(size_t tokens, int topk, int experts, size_t* bytes) {
    size_t slots;
    if (!bytes || topk < 1 || experts < 1 || !times(tokens, (size_t)topk, &slots))
        return AR_ERR_INVALID_ARG;
    if (experts > AR_MAX_EXPERTS || slots > (size_t)INT_MAX) return AR_ERR_UNSUPPORTED;
    *bytes = arlib::dispatch_work_ints(tokens, topk, experts) * sizeof(int);
    return AR_OK;
}

// ar_expert_combine, and ar_expert_dispatch_backward as the same sum with
// every weight 1.
static ar_status combine(ar_ctx* ctx, const void* rows, const char* rows_name, bool weighted,
                         const float* weights, const int* dest, const int* offsets, size_t tokens,
                         int topk, int experts, size_t hidden, ar_dtype dtype, void* y,
                         const char* y_name) {
    return guarded(ctx, [&]() -> ar_status {
        size_t eb, slots, row_bytes;
        ar_status s = check_route(ctx, tokens, topk, experts, hidden, (int)dtype, &eb, &slots,
                                  &row_bytes);
        if (s != AR_OK) return s;
        Arrays arrays(ctx);
        arrays.in(rows, slots * row_bytes, eb, rows_name);
        if (weighted) arrays.in(weights, slots * sizeof(float), 4, "weights");
        arrays.in(dest, slots * sizeof(int), 4, "dest");
        arrays.in(offsets, ((size_t)experts + 1) * sizeof(int), 4, "offsets");
        arrays.out(y, tokens * row_bytes, eb, y_name);
        s = arrays.check();
        if (s != AR_OK) return s;
        arlib::CombineArgs a{};
        a.rows = rows;
        a.weights = weighted ? weights : nullptr;
        a.dest = dest;
        a.offsets = offsets;
        a.y = y;
        a.hidden = hidden;
        a.tokens = (int)tokens;
        a.topk = topk;
        a.experts = experts;
        a.eb = (int)eb;
        return launched(ctx, arlib::launch_combine(a, ctx->stream), "expert combine");
    });
}

ar_status ar_expert_dispatch_backward(ar_ctx* ctx, const void* drows, const int* dest,
                                      const int* offsets, size_t tokens, int topk, int experts,
                                      size_t hidden, ar_dtype dtype, void* dx) {
    return combine(ctx, drows, "drows", false, nullptr, dest, offsets, tokens, topk, experts,
                   hidden, dtype, dx, "dx");
}

ar_status ar_expert_combine(ar_ctx* ctx, const void* rows, const float* weights, const int* dest,
                            const int* offsets, size_t tokens, int topk, int experts,
                            size_t hidden, ar_dtype dtype, void* y) {
    return combine(ctx, rows, "rows", true, weights, dest, offsets, tokens, topk, experts, hidden,
                   dtype, y, "y");
}

ar_status ar_expert_combine_backward(ar_ctx* ctx, const void* dy, size_t dy_stride,
                                     const void* rows, const float* weights, const int* dest,
                                     const int* offsets, size_t tokens, int topk, int experts,
                                     size_t hidden, ar_dtype dtype, void* drows, float* dweights) {
    return guarded(ctx, [&]() -> ar_status {
        size_t eb, slots, row_bytes, gbytes;
        ar_status s = check_route(ctx, tokens, topk, experts, hidden, (int)dtype, &eb, &slots,
                                  &row_bytes);
        if (s != AR_OK) return s;
        if (tokens > 1 && dy_stride < hidden)
            return fail(ctx, AR_ERR_INVALID_ARG, "dy_stride %zu below hidden %zu", dy_stride,
                        hidden);
        if (!strided_bytes(tokens, hidden, dy_stride, eb, &gbytes)) return bad_size(ctx);
        Arrays arrays(ctx);
        arrays.in(dy, gbytes, eb, "dy");
        arrays.in(rows, slots * row_bytes, eb, "rows");
        arrays.in(weights, slots * sizeof(float), 4, "weights");
        arrays.in(dest, slots * sizeof(int), 4, "dest");
        arrays.in(offsets, ((size_t)experts + 1) * sizeof(int), 4, "offsets");
        arrays.out(drows, slots * row_bytes, eb, "drows");
        arrays.out(dweights, slots * sizeof(float), 4, "dweights");
        s = arrays.check();
        if (s != AR_OK) return s;
        arlib::CombineArgs a{};
        a.rows = rows;
        a.weights = weights;
        a.dest = dest;
        a.offsets = offsets;
        a.dy = dy;
        a.drows = drows;
        a.dweights = dweights;
        a.dystride = dy_stride;
        a.hidden = hidden;
        a.tokens = (int)tokens;
        a.topk = topk;
        a.experts = experts;
        a.eb = (int)eb;
        return launched(ctx, arlib::launch_combine_grad(a, ctx->stream), "expert combine gradient");
    });
}

ar_status ar_distill_loss(ar_ctx* ctx, const void* logits, size_t logits_stride,
                          const void* indices, int index_bytes, const void* teacher, size_t rows,
                          size_t vocab, size_t top, ar_dtype dtype, float temperature, float* loss,
                          float* lse, void* workspace_, size_t workspace_bytes) {
    return guarded(ctx, [&]() -> ar_status {
        Arrays arrays(ctx);
        arlib::DistillArgs d;
        ar_status s = check_distill(ctx, arrays, d, logits, logits_stride, indices, index_bytes,
                                    teacher, rows, vocab, top, (int)dtype, temperature);
        if (s != AR_OK) return s;
        arrays.out(loss, rows * sizeof(float), 4, "loss");
        arrays.out(lse, rows * sizeof(float), 4, "lse");
        s = workspace(ctx, arrays, workspace_, workspace_bytes,
                      arlib::distill_work_floats(rows, vocab, top, d.eb, false) * sizeof(float));
        if (s == AR_OK) s = arrays.check();
        if (s != AR_OK) return s;
        d.loss = loss;
        d.lse = lse;
        d.part = static_cast<float*>(workspace_);
        return launched(ctx, arlib::launch_distill_loss(d, ctx->stream), "distillation");
    });
}

ar_status ar_distill_backward(ar_ctx* ctx, const float* dloss, const void* logits,
                              size_t logits_stride, const void* indices, int index_bytes,
                              const void* teacher, const float* lse, size_t rows, size_t vocab,
                              size_t top, ar_dtype dtype, float temperature, void* dlogits) {
    return guarded(ctx, [&]() -> ar_status {
        Arrays arrays(ctx);
        arlib::DistillArgs d;
        ar_status s = check_distill(ctx, arrays, d, logits, logits_stride, indices, index_bytes,
                                    teacher, rows, vocab, top, (int)dtype, temperature);
        if (s != AR_OK) return s;
        size_t bytes;
        if (!strided_bytes(rows, vocab, vocab, (size_t)d.eb, &bytes)) return bad_size(ctx);
        arrays.in(dloss, rows * sizeof(float), 4, "dloss");
        arrays.in(lse, rows * sizeof(float), 4, "lse");
        arrays.out(dlogits, bytes, (size_t)d.eb, "dlogits");
        s = arrays.check();
        if (s != AR_OK) return s;
        d.dloss = dloss;
        d.lse_in = lse;
        d.dlogits = dlogits;
        return launched(ctx, arlib::launch_distill_backward(d, ctx->stream),
                        "distillation gradient");
    });
}

ar_status ar_distill_step(ar_ctx* ctx, const float* dloss, const void* logits,
                          size_t logits_stride, const void* indices, int index_bytes,
                          const void* teacher, size_t rows, size_t vocab, size_t top,
                          ar_dtype dtype, float temperature, float* loss, void* dlogits,
                          void* workspace_, size_t workspace_bytes) {
    return guarded(ctx, [&]() -> ar_status {
        Arrays arrays(ctx);
        arlib::DistillArgs d;
        ar_status s = check_distill(ctx, arrays, d, logits, logits_stride, indices, index_bytes,
                                    teacher, rows, vocab, top, (int)dtype, temperature);
        if (s != AR_OK) return s;
        size_t bytes;
        if (!strided_bytes(rows, vocab, vocab, (size_t)d.eb, &bytes)) return bad_size(ctx);
        arrays.in(dloss, rows * sizeof(float), 4, "dloss");
        arrays.out(loss, rows * sizeof(float), 4, "loss");
        arrays.out(dlogits, bytes, (size_t)d.eb, "dlogits");
        s = workspace(ctx, arrays, workspace_, workspace_bytes,
                      arlib::distill_work_floats(rows, vocab, top, d.eb, true) * sizeof(float));
        if (s == AR_OK) s = arrays.check();
        if (s != AR_OK) return s;
        d.dloss = dloss;
        d.loss = loss;
        d.dlogits = dlogits;
        d.part = static_cast<float*>(workspace_);
        return launched(ctx, arlib::launch_distill_step(d, ctx->stream), "distillation step");
    });
}

ar_status ar_distill_workspace(size_t rows, size_t vocab, size_t top, ar_dtype dtype, int gradient,
                               size_t* bytes) {
    const size_t eb = float_bytes((int)dtype);
    size_t all;
    if (!bytes || !eb || vocab < 1 || top < 1 || !times(vocab, eb, &all) ||
        !times(all, rows, &all))
        return AR_ERR_INVALID_ARG;
    if (vocab > kMostCols || top > AR_DISTILL_MAX_TOP) return AR_ERR_UNSUPPORTED;
    *bytes = arlib::distill_work_floats(rows, vocab, top, (int)eb, gradient != 0) * sizeof(float);
    return AR_OK;
}

}  // extern "C"
#pragma GCC visibility pop
