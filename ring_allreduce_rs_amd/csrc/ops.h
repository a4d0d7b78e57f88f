// ops.h -- internal interface between the C entry points of the training
// operators (ops_api.cpp) and their kernels (norm.hip, route.hip,
// distill.hip).  Not part of the public ABI.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stddef.h>
#include <stdint.h>

namespace arlib {

// ------------------------------------------------------------------ layer norm
// Row strides are in elements.  `eb` is the element size of x, dy, y and dx
// (2: bf16, 4: fp32), `pb` that of weight, bias and their gradients.
struct NormArgs {
    const void* x;
    const void* weight;   // NULL: 1
    const void* bias;     // NULL: 0
    void* y;
    float* mean;
    float* rstd;
    size_t xstride;
    size_t rows, cols;
    float eps;
    int eb, pb;
};

struct NormGradArgs {
    const void* dy;
    const void* x;
    const float* mean;
    const float* rstd;
    const void* weight;   // NULL: 1
    void* dx;
    void* dweight;        // NULL: not wanted
    void* dbias;          // NULL: not wanted
    float* part;          // norm_grad_parts() x 2 x cols partial sums
    size_t dystride, xstride;
    size_t rows, cols;
    int eb, pb;
};

// Rows of partial sums that the backward pass leaves for its last step.
size_t norm_grad_parts(size_t rows, size_t cols, int eb);
hipError_t launch_norm(const NormArgs& a, hipStream_t s);
hipError_t launch_norm_grad(const NormGradArgs& a, hipStream_t s);

// ------------------------------------------------ tokens by expert and back
struct DispatchArgs {
    const void* x;
    const void* ids;      // tokens x topk, `ib` bytes each
    void* rows;           // tokens*topk x hidden
    int* dest;            // tokens x topk
    int* slot;            // tokens*topk
    int* offsets;         // experts + 1
    int* work;            // dispatch_work_ints() ints
    size_t xstride;
    size_t hidden;
    int tokens, topk, experts;
    int eb, ib;
};

// One step of the way back: y[t] = sum_k w[t,k] rows[dest[t,k]] (weights NULL:
// 1), or its gradient when dy is given: drows[dest[t,k]] = w[t,k] dy[t],
// dweights[t,k] = rows[dest[t,k]] . dy[t].
struct CombineArgs {
    const void* rows;
    const float* weights;
    const int* dest;
    const int* offsets;
    void* y;
    const void* dy;
    void* drows;
    float* dweights;
    size_t dystride;
    size_t hidden;
    int tokens, topk, experts;
    int eb;
};

size_t dispatch_work_ints(size_t tokens, int topk, int experts);
hipError_t launch_dispatch(const DispatchArgs& a, hipStream_t s);
hipError_t launch_combine(const CombineArgs& a, hipStream_t s);
hipError_t launch_combine_grad(const CombineArgs& a, hipStream_t s);

// ---------------------------------------------------------------- distillation
struct DistillArgs {
    const void* logits;
    const void* indices;  // rows x top, `ib` bytes each
    const void* teacher;  // rows x top, element size eb
    const float* dloss;   // gradient passes
    const float* lse_in;  // backward: the forward pass's lse
    float* loss;
    float* lse;
    void* dlogits;
    float* part;          // distill_work_floats() floats
    size_t lstride;
    size_t rows, vocab, top;
    float temperature;
    int eb, ib;
};

size_t distill_work_floats(size_t rows, size_t vocab, size_t top, int eb, bool step);
hipError_t launch_distill_loss(const DistillArgs& a, hipStream_t s);
hipError_t launch_distill_backward(const DistillArgs& a, hipStream_t s);
hipError_t launch_distill_step(const DistillArgs& a, hipStream_t s);

}  // namespace arlib
