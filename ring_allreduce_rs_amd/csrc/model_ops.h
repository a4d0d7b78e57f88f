// model_ops.h -- internal interface between the C entry points of the
// embedding, the experts' products and the gated activation with its 8-bit
// checkpoint (model_api.cpp) and their kernels (embed.hip, product.hip,
// gate.hip).  Not part of the public ABI.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stddef.h>
#include <stdint.h>

namespace arlib {

// ------------------------------------------------------------------- embedding
struct EmbedArgs {
    const void* table;    // vocab x hidden
    const void* ids;      // tokens, `ib` bytes each
    void* y;              // tokens x hidden
    size_t tokens, vocab, hidden;
    float scale;
    int eb, ib;
};

struct EmbedGradArgs {
    const void* dy;
    const void* ids;
    void* dtable;         // vocab x hidden
    int* work;            // embed_grad_work_bytes() bytes
    size_t dystride;
    size_t tokens, vocab, hidden;
    float scale;
    int eb, ib;
};

size_t embed_grad_work_bytes(size_t tokens, size_t vocab, size_t hidden, int eb);
hipError_t launch_embed(const EmbedArgs& a, hipStream_t s);
hipError_t launch_embed_grad(const EmbedGradArgs& a, hipStream_t s);

// ------------------------------------------------------- products by expert
// PRODUCT_FORWARD:  c[j] = a[j] W_e^T     a: nrows x hidden, c: nrows x out
// PRODUCT_DROWS:    c[j] = a[j] W_e       a: nrows x out,    c: nrows x hidden
// PRODUCT_DWEIGHTS: c_e = sum a[j]^T b[j] a: nrows x out,    b: nrows x hidden
// over the rows j of expert e, [offsets[e], offsets[e + 1]).
enum ProductKind { PRODUCT_FORWARD, PRODUCT_DROWS, PRODUCT_DWEIGHTS };

struct ProductArgs {
    const void* a;
    const void* b;          // the weights, or the rows of PRODUCT_DWEIGHTS
    void* c;
    const int* offsets;     // experts + 1
    float* work;            // product_work_bytes() bytes
    size_t astride, bstride;    // elements between rows (bstride: PRODUCT_DWEIGHTS only)
    size_t nrows, hidden, out;
    int experts;
    int eb;
};

size_t product_work_bytes(ProductKind kind, size_t nrows, int experts, size_t hidden, size_t out,
                          int eb);
hipError_t launch_product(ProductKind kind, const ProductArgs& a, hipStream_t s);

// ------------------------------------------------- gate and 8-bit checkpoint
// A checkpoint holds `halves` x cols values a row: codes (rows x halves x cols
// bytes) and, for each group of kSaveGroup along cols, the biased exponent of
// their scale (rows x halves x save_groups(cols) bytes).
constexpr int kSaveGroup = 32;
inline size_t save_groups(size_t cols) { return (cols + kSaveGroup - 1) / kSaveGroup; }

struct GateArgs {
    const void* x;        // save: rows x cols; gate: rows x 2 cols
    const void* dacts;    // gate's backward pass
    int8_t* codes;
    uint8_t* scales;
    void* y;              // restore: the values; gate: acts; its backward pass: dh
    void* acts;           // gate's backward pass
    size_t stride;        // of x or dacts
    size_t rows, cols;
    int eb;
};

hipError_t launch_save(const GateArgs& a, hipStream_t s);
hipError_t launch_restore(const GateArgs& a, hipStream_t s);
hipError_t launch_gate(const GateArgs& a, hipStream_t s);
hipError_t launch_gate_grad(const GateArgs& a, hipStream_t s);

}  // namespace arlib
