// Internal launch interface of the output head's kernels (not part of the C
// ABI).  The caller has validated every argument; each function launches on
// stream s and returns the launch status.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace dlk {

struct NormArgs {
    const void* x;
    int64_t ldx;
    const void* residual;        // or nullptr
    int64_t ldres;
    const float* weight;
    float eps;
    int64_t rows;
    int cols;
    void* sum;                   // or nullptr
    int64_t ldsum;
    void* y;
    int64_t ldy;
    void* scales;
    float* inv_rms;              // or nullptr
};
// dtype, y_dtype and scale_kind as in dlhead.h
hipError_t rmsnorm(const NormArgs& a, int dtype, int y_dtype, int scale_kind, hipStream_t s);

struct NormBackwardArgs {
    const void* dy;
    int64_t lddy;
    const void* dsum;            // or nullptr
    int64_t lddsum;
    const void* sum;
    int64_t ldsum;
    const float* weight;
    const float* inv_rms;
    int64_t rows;
    int cols;
    void* dx;
    int64_t lddx;
    float* dweight;              // or nullptr
    float* partial;              // rmsnorm_workspace_bytes, with dweight
};
int64_t rmsnorm_workspace_bytes(int64_t rows, int64_t cols);
hipError_t rmsnorm_backward(const NormBackwardArgs& a, int dtype, hipStream_t s);

hipError_t w4_quantize(const void* w, int64_t ldw, int dtype, int64_t rows, int64_t cols,
                       uint8_t* packed, uint8_t* scales, void* values, int64_t ldvalues,
                       hipStream_t s);

struct MatvecArgs {
    const uint8_t* packed;
    const uint8_t* scales;
    int64_t rows;
    int64_t cols;
    const void* x;
    int64_t ldx;
    const void* x_scales;
    int count;
    void* y;
    int64_t ldy;
};
// x in bfloat16 with DL_SCALE_NONE, in e4m3 with the other kinds
hipError_t w4_matvec(const MatvecArgs& a, int x_scale_kind, int y_dtype, hipStream_t s);

struct LogprobsArgs {
    const void* logits;
    int64_t ld;
    int64_t rows;
    int64_t vocab;
    const int64_t* targets;      // or nullptr
    float* logprobs;             // or nullptr
    float* entropy;              // or nullptr
    float* stats;                // or nullptr
    int top_k;
    int64_t* top_ids;
    float* top_logprobs;
    void* workspace;             // logprobs_workspace_bytes
};
int64_t logprobs_workspace_bytes(int64_t rows, int64_t vocab, int top_k);
hipError_t logprobs(const LogprobsArgs& a, int dtype, hipStream_t s);

struct LogprobsBackwardArgs {
    const void* logits;
    int64_t ld;
    int64_t rows;
    int64_t vocab;
    const int64_t* targets;
    const float* stats;
    const float* entropy;        // or nullptr
    const float* dlogprobs;
    const float* dentropy;       // or nullptr
    void* dlogits;
    int64_t ldd;
};
hipError_t logprobs_backward(const LogprobsBackwardArgs& a, int dtype, hipStream_t s);

struct HeadArgs {
    const void* x;
    int64_t ldx;
    const void* embed;
    int64_t lde;
    int64_t rows;
    int64_t vocab;
    int64_t width;
    const int64_t* targets;      // or nullptr
    float* logprobs;             // or nullptr
    float* entropy;              // or nullptr
    float* stats;                // or nullptr
    void* workspace;             // head_workspace_bytes
};
int64_t head_workspace_bytes(int64_t rows, int64_t vocab, int64_t width, int dtype,
                             bool with_backward);
hipError_t head_logprobs(const HeadArgs& a, int dtype, hipStream_t s);

struct HeadBackwardArgs {
    const void* x;
    int64_t ldx;
    const void* embed;
    int64_t lde;
    int64_t rows;
    int64_t vocab;
    int64_t width;
    const int64_t* targets;
    const float* stats;
    const float* entropy;        // or nullptr
    const float* dlogprobs;
    const float* dentropy;       // or nullptr
    void* dx;                    // or nullptr
    int64_t lddx;
    void* dembed;                // or nullptr
    int64_t ldde;
    void* workspace;             // head_workspace_bytes, with the backward pass
};
hipError_t head_logprobs_backward(const HeadBackwardArgs& a, int dtype, hipStream_t s);

hipError_t e4m3_quantize(const void* x, int64_t ldx, int dtype, int64_t rows, int64_t cols,
                         uint8_t* codes, int64_t ldc, uint8_t* scales, int scale_kind,
                         void* values, int64_t ldvalues, hipStream_t s);

struct E4m3ProductArgs {
    const uint8_t* w;
    int64_t ldw;
    const uint8_t* w_scales;
    int64_t rows;
    int64_t cols;
    const uint8_t* x;
    int64_t ldx;
    const uint8_t* x_scales;
    int64_t count;
    void* y;
    int64_t ldy;
};
hipError_t e4m3_matmul(const E4m3ProductArgs& a, int y_dtype, hipStream_t s);

}  // namespace dlk
