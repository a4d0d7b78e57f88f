// model_api.cpp -- the C entry points of the embedding, the experts' products
// and the gated activation with its 8-bit checkpoint (include/ar.h): argument
// validation and error reporting.  The kernels live in embed.hip, product.hip
// and gate.hip.
#include <hip/hip_runtime_api.h>

#include <climits>
#include <cmath>
#include <cstdint>

#include "ar.h"
#include "ctx.h"
#include "model_ops.h"
#include "ops_args.h"

using arlib::Arrays;
using arlib::bad_size;
using arlib::check_index_bytes;
using arlib::fail;
using arlib::float_bytes;
using arlib::guarded;
using arlib::kMostCols;
using arlib::launched;
using arlib::ProductKind;
using arlib::strided_bytes;
using arlib::times;
using arlib::workspace;

namespace {

// The sizes of an embedding and of its gradient.
struct EmbedSizes {
    size_t eb, ids, table, dense;   // bytes: an element, ids, the table, tokens x hidden
};
ar_status check_embed(ar_ctx* ctx, int index_bytes, size_t tokens, size_t vocab, size_t hidden,
                      int dtype, float scale, EmbedSizes* z) {
    z->eb = float_bytes(dtype);
    if (!z->eb) return fail(ctx, AR_ERR_INVALID_ARG, "unknown or unsupported dtype %d", dtype);
    const ar_status s = check_index_bytes(ctx, index_bytes);
    if (s != AR_OK) return s;
    if (vocab < 1 || hidden < 1) return fail(ctx, AR_ERR_INVALID_ARG, "vocab or hidden is 0");
    if (!std::isfinite(scale))
        return fail(ctx, AR_ERR_INVALID_ARG, "scale %g is not finite", (double)scale);
    if (vocab > kMostCols) return fail(ctx, AR_ERR_UNSUPPORTED, "vocab %zu above 2^28", vocab);
    if (hidden > kMostCols) return fail(ctx, AR_ERR_UNSUPPORTED, "hidden %zu above 2^28", hidden);
    if (tokens > (size_t)INT_MAX)
        return fail(ctx, AR_ERR_UNSUPPORTED, "tokens %zu above 2^31 - 1", tokens);
    if (!times(tokens, (size_t)index_bytes, &z->ids) ||
        !strided_bytes(vocab, hidden, hidden, z->eb, &z->table) ||
        !strided_bytes(tokens, hidden, hidden, z->eb, &z->dense))
        return bad_size(ctx);
    return AR_OK;
}

// Widest rows of a product, and furthest apart: the rows of a tile span less than
// 2^31 bytes.
constexpr size_t kMostWide = size_t(1) << 20;

// Whether the sizes of a product are in range; the weights' bytes.
ar_status check_product(ar_ctx* ctx, size_t nrows, int experts, size_t hidden, size_t out, int dtype,
                        size_t* eb, size_t* wbytes) {
    *eb = float_bytes(dtype);
    if (!*eb) return fail(ctx, AR_ERR_INVALID_ARG, "unknown or unsupported dtype %d", dtype);
    if (experts < 1) return fail(ctx, AR_ERR_INVALID_ARG, "experts %d below 1", experts);
    if (hidden < 1 || out < 1) return fail(ctx, AR_ERR_INVALID_ARG, "hidden or out is 0");
    if (experts > AR_MAX_EXPERTS)
        return fail(ctx, AR_ERR_UNSUPPORTED, "experts %d above %d", experts, AR_MAX_EXPERTS);
    if (hidden > kMostWide || out > kMostWide)
        return fail(ctx, AR_ERR_UNSUPPORTED, "hidden %zu or out %zu above 2^20", hidden, out);
    if (nrows > (size_t)INT_MAX)
        return fail(ctx, AR_ERR_UNSUPPORTED, "nrows %zu above 2^31 - 1", nrows);
    size_t w;
    if (!times(hidden, out, &w) || !times(w, (size_t)experts, &w) || !times(w, *eb, wbytes))
        return bad_size(ctx);
    return AR_OK;
}

ar_status check_stride(ar_ctx* ctx, const char* name, size_t rows, size_t stride, size_t cols) {
    if (rows > 1 && stride < cols)
        return fail(ctx, AR_ERR_INVALID_ARG, "%s %zu below the row's %zu elements", name, stride,
                    cols);
    return AR_OK;
}

// A product's stride between `rows` rows of `cols`; that of a single row is of no
// meaning and becomes its width.
ar_status check_product_stride(ar_ctx* ctx, const char* name, size_t rows, size_t* stride,
                               size_t cols) {
    if (rows <= 1) *stride = cols;
    if (*stride > kMostWide)
        return fail(ctx, AR_ERR_UNSUPPORTED, "%s %zu above 2^20", name, *stride);
    return check_stride(ctx, name, rows, *stride, cols);
}

// ar_expert_matmul and ar_expert_matmul_drows: c[j] = a[j] W^T or a[j] W.
ar_status product_rows(ar_ctx* ctx, ProductKind kind, const char* what, const void* in,
                       const char* in_name, size_t stride, const char* stride_name,
                       const void* weights, const int* offsets, size_t nrows, int experts,
                       size_t hidden, size_t out, ar_dtype dtype, void* y, const char* y_name,
                       void* workspace_, size_t workspace_bytes) {
    return guarded(ctx, [&]() -> ar_status {
        size_t eb, wbytes, ibytes, ybytes;
        ar_status s = check_product(ctx, nrows, experts, hidden, out, (int)dtype, &eb, &wbytes);
        const size_t icols = kind == arlib::PRODUCT_FORWARD ? hidden : out;
        const size_t ycols = kind == arlib::PRODUCT_FORWARD ? out : hidden;
        if (s == AR_OK) s = check_product_stride(ctx, stride_name, nrows, &stride, icols);
        if (s != AR_OK) return s;
        if (!strided_bytes(nrows, icols, stride, eb, &ibytes) ||
            !strided_bytes(nrows, ycols, ycols, eb, &ybytes))
            return bad_size(ctx);
        Arrays arrays(ctx);
        arrays.in(in, ibytes, eb, in_name);
        arrays.in(weights, wbytes, eb, "weights");
        arrays.in(offsets, ((size_t)experts + 1) * sizeof(int), 4, "offsets");
        arrays.out(y, ybytes, eb, y_name);
        s = workspace(ctx, arrays, workspace_, workspace_bytes,
                      arlib::product_work_bytes(kind, nrows, experts, hidden, out, (int)eb));
        if (s == AR_OK) s = arrays.check();
        if (s != AR_OK) return s;
        arlib::ProductArgs a{in,      weights, y,      offsets, static_cast<float*>(workspace_),
                             stride,  0,       nrows,  hidden,  out,
                             experts, (int)eb};
        return launched(ctx, arlib::launch_product(kind, a, ctx->stream), what);
    });
}

// The arguments that the checkpoint's calls share: `halves` x cols values a row.
struct SaveSizes {
    size_t eb, codes, scales;   // bytes
};
ar_status check_save(ar_ctx* ctx, size_t rows, size_t cols, size_t halves, int dtype, SaveSizes* z) {
    z->eb = float_bytes(dtype);
    if (!z->eb) return fail(ctx, AR_ERR_INVALID_ARG, "unknown or unsupported dtype %d", dtype);
    if (cols < 1) return fail(ctx, AR_ERR_INVALID_ARG, "cols is 0");
    if (cols > kMostCols) return fail(ctx, AR_ERR_UNSUPPORTED, "cols %zu above 2^28", cols);
    size_t line;
    if (!times(rows, halves, &line) || !times(line, cols, &z->codes) ||
        !times(line, arlib::save_groups(cols), &z->scales))
        return bad_size(ctx);
    return AR_OK;
}

}  // namespace

#pragma GCC visibility push(default)
extern "C" {

ar_status ar_embedding(ar_ctx* ctx, const void* table, const void* ids, int index_bytes,
                       size_t tokens, size_t vocab, size_t hidden, ar_dtype dtype, float scale,
                       void* y) {
    return guarded(ctx, [&]() -> ar_status {
        EmbedSizes z;
        ar_status s = check_embed(ctx, index_bytes, tokens, vocab, hidden, (int)dtype, scale, &z);
        if (s != AR_OK) return s;
        Arrays arrays(ctx);
        arrays.in(table, z.table, z.eb, "table");
        arrays.in(ids, z.ids, (size_t)index_bytes, "ids");
        arrays.out(y, z.dense, z.eb, "y");
        s = arrays.check();
        if (s != AR_OK) return s;
        arlib::EmbedArgs a{table, ids, y, tokens, vocab, hidden, scale, (int)z.eb, index_bytes};
        return launched(ctx, arlib::launch_embed(a, ctx->stream), "embedding");
    });
}

ar_status ar_embedding_backward(ar_ctx* ctx, const void* dy, size_t dy_stride, const void* ids,
                                int index_bytes, size_t tokens, size_t vocab, size_t hidden,
                                ar_dtype dtype, float scale, void* dtable, void* workspace_,
                                size_t workspace_bytes) {
    return guarded(ctx, [&]() -> ar_status {
        EmbedSizes z;
        size_t gbytes;
        ar_status s = check_embed(ctx, index_bytes, tokens, vocab, hidden, (int)dtype, scale, &z);
        if (s == AR_OK) s = check_stride(ctx, "dy_stride", tokens, dy_stride, hidden);
        if (s != AR_OK) return s;
        if (!strided_bytes(tokens, hidden, dy_stride, z.eb, &gbytes)) return bad_size(ctx);
        Arrays arrays(ctx);
        arrays.in(dy, gbytes, z.eb, "dy");
        arrays.in(ids, z.ids, (size_t)index_bytes, "ids");
        arrays.out(dtable, z.table, z.eb, "dtable");
        s = workspace(ctx, arrays, workspace_, workspace_bytes,
                      arlib::embed_grad_work_bytes(tokens, vocab, hidden, (int)z.eb));
        if (s == AR_OK) s = arrays.check();
        if (s != AR_OK) return s;
        arlib::EmbedGradArgs a{dy,     ids,   dtable, static_cast<int*>(workspace_), dy_stride, tokens,
                               vocab,  hidden, scale,  (int)z.eb, index_bytes};
        return launched(ctx, arlib::launch_embed_grad(a, ctx->stream), "embedding gradient");
    });
}

ar_status ar_embedding_backward_workspace(size_t tokens, size_t vocab, size_t hidden, ar_dtype dtype,
                                          size_t* bytes) {
    const size_t eb = float_bytes((int)dtype);
    size_t n;
    if (!bytes || !eb || vocab < 1 || hidden < 1) return AR_ERR_INVALID_ARG;
    if (vocab > kMostCols || hidden > kMostCols || tokens > (size_t)INT_MAX)
        return AR_ERR_UNSUPPORTED;
    if (!times(tokens, hidden, &n)) return AR_ERR_INVALID_ARG;
    *bytes = arlib::embed_grad_work_bytes(tokens, vocab, hidden, (int)eb);
    return AR_OK;
}

ar_status ar_expert_matmul(ar_ctx* ctx, const void* rows, size_t rows_stride, const void* weights,
                           const int* offsets, size_t nrows, int experts, size_t hidden, size_t out,
                           ar_dtype dtype, void* y, void* workspace_, size_t workspace_bytes) {
    return product_rows(ctx, arlib::PRODUCT_FORWARD, "expert product", rows, "rows", rows_stride,
                        "rows_stride", weights, offsets, nrows, experts, hidden, out, dtype, y, "y",
                        workspace_, workspace_bytes);
}

ar_status ar_expert_matmul_drows(ar_ctx* ctx, const void* dy, size_t dy_stride, const void* weights,
                                 const int* offsets, size_t nrows, int experts, size_t hidden,
                                 size_t out, ar_dtype dtype, void* drows, void* workspace_,
                                 size_t workspace_bytes) {
    return product_rows(ctx, arlib::PRODUCT_DROWS, "expert product's gradient of rows", dy, "dy",
                        dy_stride, "dy_stride", weights, offsets, nrows, experts, hidden, out, dtype,
                        drows, "drows", workspace_, workspace_bytes);
}

ar_status ar_expert_matmul_dweights(ar_ctx* ctx, const void* dy, size_t dy_stride, const void* rows,
                                    size_t rows_stride, const int* offsets, size_t nrows,
                                    int experts, size_t hidden, size_t out, ar_dtype dtype,
                                    void* dweights, void* workspace_, size_t workspace_bytes) {
    return guarded(ctx, [&]() -> ar_status {
        size_t eb, wbytes, gbytes, rbytes;
        ar_status s = check_product(ctx, nrows, experts, hidden, out, (int)dtype, &eb, &wbytes);
        if (s == AR_OK) s = check_product_stride(ctx, "dy_stride", nrows, &dy_stride, out);
        if (s == AR_OK) s = check_product_stride(ctx, "rows_stride", nrows, &rows_stride, hidden);
        if (s != AR_OK) return s;
        if (!strided_bytes(nrows, out, dy_stride, eb, &gbytes) ||
            !strided_bytes(nrows, hidden, rows_stride, eb, &rbytes))
            return bad_size(ctx);
        Arrays arrays(ctx);
        arrays.in(dy, gbytes, eb, "dy");
        arrays.in(rows, rbytes, eb, "rows");
        arrays.in(offsets, ((size_t)experts + 1) * sizeof(int), 4, "offsets");
        arrays.out(dweights, wbytes, eb, "dweights");
        s = workspace(ctx, arrays, workspace_, workspace_bytes,
                      arlib::product_work_bytes(arlib::PRODUCT_DWEIGHTS, nrows, experts, hidden, out,
                                                (int)eb));
        if (s == AR_OK) s = arrays.check();
        if (s != AR_OK) return s;
        arlib::ProductArgs a{dy,        rows,        dweights, offsets, static_cast<float*>(workspace_),
                             dy_stride, rows_stride, nrows,    hidden,  out,
                             experts,   (int)eb};
        return launched(ctx, arlib::launch_product(arlib::PRODUCT_DWEIGHTS, a, ctx->stream),
                        "expert product's gradient of weights");
    });
}

ar_status ar_expert_matmul_workspace(ar_expert_product product, size_t nrows, int experts,
                                     size_t hidden, size_t out, ar_dtype dtype, size_t* bytes) {
    const size_t eb = float_bytes((int)dtype);
    size_t w;
    if (!bytes || !eb || experts < 1 || hidden < 1 || out < 1 || (int)product < 0 ||
        (int)product > (int)AR_EXPERT_DWEIGHTS)
        return AR_ERR_INVALID_ARG;
    if (experts > AR_MAX_EXPERTS || hidden > kMostWide || out > kMostWide ||
        nrows > (size_t)INT_MAX)
        return AR_ERR_UNSUPPORTED;
    if (!times(hidden, out, &w) || !times(w, (size_t)experts, &w) || !times(w, eb, &w))
        return AR_ERR_INVALID_ARG;
    *bytes = arlib::product_work_bytes((ProductKind)(int)product, nrows, experts, hidden, out,
                                       (int)eb);
    return AR_OK;
}

ar_status ar_save_8bit(ar_ctx* ctx, const void* x, size_t x_stride, size_t rows, size_t cols,
                       ar_dtype dtype, signed char* codes, unsigned char* scales) {
    return guarded(ctx, [&]() -> ar_status {
        SaveSizes z;
        size_t xbytes;
        ar_status s = check_save(ctx, rows, cols, 1, (int)dtype, &z);
        if (s == AR_OK) s = check_stride(ctx, "x_stride", rows, x_stride, cols);
        if (s != AR_OK) return s;
        if (!strided_bytes(rows, cols, x_stride, z.eb, &xbytes)) return bad_size(ctx);
        Arrays arrays(ctx);
        arrays.in(x, xbytes, z.eb, "x");
        arrays.out(codes, z.codes, 1, "codes");
        arrays.out(scales, z.scales, 1, "scales");
        s = arrays.check();
        if (s != AR_OK) return s;
        arlib::GateArgs a{};
        a.x = x;
        a.codes = codes;
        a.scales = scales;
        a.stride = x_stride;
        a.rows = rows;
        a.cols = cols;
        a.eb = (int)z.eb;
        return launched(ctx, arlib::launch_save(a, ctx->stream), "8-bit checkpoint");
    });
}

ar_status ar_restore_8bit(ar_ctx* ctx, const signed char* codes, const unsigned char* scales,
                          size_t rows, size_t cols, ar_dtype dtype, void* x) {
    return guarded(ctx, [&]() -> ar_status {
        SaveSizes z;
        size_t xbytes;
        ar_status s = check_save(ctx, rows, cols, 1, (int)dtype, &z);
        if (s != AR_OK) return s;
        if (!strided_bytes(rows, cols, cols, z.eb, &xbytes)) return bad_size(ctx);
        Arrays arrays(ctx);
        arrays.in(codes, z.codes, 1, "codes");
        arrays.in(scales, z.scales, 1, "scales");
        arrays.out(x, xbytes, z.eb, "x");
        s = arrays.check();
        if (s != AR_OK) return s;
        arlib::GateArgs a{};
        a.codes = const_cast<signed char*>(codes);
        a.scales = const_cast<unsigned char*>(scales);
        a.y = x;
        a.rows = rows;
        a.cols = cols;
        a.eb = (int)z.eb;
        return launched(ctx, arlib::launch_restore(a, ctx->stream), "8-bit checkpoint's values");
    });
}

ar_status ar_silu_gate(ar_ctx* ctx, const void* h, size_t h_stride, size_t rows, size_t cols,
                       ar_dtype dtype, void* acts, signed char* codes, unsigned char* scales) {
    return guarded(ctx, [&]() -> ar_status {
        SaveSizes z;
        size_t hbytes, abytes;
        ar_status s = check_save(ctx, rows, cols, 2, (int)dtype, &z);
        if (s == AR_OK) s = check_stride(ctx, "h_stride", rows, h_stride, 2 * cols);
        if (s != AR_OK) return s;
        if (!strided_bytes(rows, 2 * cols, h_stride, z.eb, &hbytes) ||
            !strided_bytes(rows, cols, cols, z.eb, &abytes))
            return bad_size(ctx);
        Arrays arrays(ctx);
        arrays.in(h, hbytes, z.eb, "h");
        arrays.out(acts, abytes, z.eb, "acts");
        arrays.out(codes, z.codes, 1, "codes");
        arrays.out(scales, z.scales, 1, "scales");
        s = arrays.check();
        if (s != AR_OK) return s;
        arlib::GateArgs a{};
        a.x = h;
        a.codes = codes;
        a.scales = scales;
        a.y = acts;
        a.stride = h_stride;
        a.rows = rows;
        a.cols = cols;
        a.eb = (int)z.eb;
        return launched(ctx, arlib::launch_gate(a, ctx->stream), "gate");
    });
}

ar_status ar_silu_gate_backward(ar_ctx* ctx, const void* dacts, size_t dacts_stride,
                                const signed char* codes, const unsigned char* scales, size_t rows,
                                size_t cols, ar_dtype dtype, void* dh, void* acts) {
    return guarded(ctx, [&]() -> ar_status {
        SaveSizes z;
        size_t dbytes, hbytes, abytes;
        ar_status s = check_save(ctx, rows, cols, 2, (int)dtype, &z);
        if (s == AR_OK) s = check_stride(ctx, "dacts_stride", rows, dacts_stride, cols);
        if (s != AR_OK) return s;
        if (!strided_bytes(rows, cols, dacts_stride, z.eb, &dbytes) ||
            !strided_bytes(rows, 2 * cols, 2 * cols, z.eb, &hbytes) ||
            !strided_bytes(rows, cols, cols, z.eb, &abytes))
            return bad_size(ctx);
        Arrays arrays(ctx);
        arrays.in(dacts, dbytes, z.eb, "dacts");
        arrays.in(codes, z.codes, 1, "codes");
        arrays.in(scales, z.scales, 1, "scales");
        arrays.out(dh, hbytes, z.eb, "dh");
        arrays.out(acts, abytes, z.eb, "acts");
        s = arrays.check();
        if (s != AR_OK) return s;
        arlib::GateArgs a{};
        a.dacts = dacts;
        a.codes = const_cast<signed char*>(codes);
        a.scales = const_cast<unsigned char*>(scales);
        a.y = dh;
        a.acts = acts;
        a.stride = dacts_stride;
        a.rows = rows;
        a.cols = cols;
        a.eb = (int)z.eb;
        return launched(ctx, arlib::launch_gate_grad(a, ctx->stream), "gate gradient");
    });
}

}  // extern "C"
#pragma GCC visibility pop
