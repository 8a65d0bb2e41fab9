// Host-side declarations of the launchers behind spl_local.h (internal header).
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

namespace spl {

// Token ids of a call: 32- or 64-bit signed integers, or none.
struct TokenIds {
    const void* data;
    bool wide;
};

// The current device's SM count, asked for once per device.
cudaError_t sm_count(int* sms);

// Launches a kernel of a call behind the call's previous one: its CTAs may become resident while
// that one ends, and wait for its results where they call after_previous().  Every thread of such
// a kernel calls that before it returns, so that the kernel ends after all of the call before it.
// Saves 1 to 2 us a launch (2,000 tokens' embedding gradient 30.9 us against 34.7 one call after the
// other, accumulating 21 against 26; orthogonalize 300 x 1000 117 against 120).
template <typename... Params, typename... Args>
cudaError_t launch_behind(void (*kernel)(Params...), dim3 grid, unsigned threads, cudaStream_t stream,
                          Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

constexpr int kMaxTop = 32;   // alternatives per row: one list entry per lane of a warp

struct LogprobsArgs {
    const void* logits;
    int64_t rows, vocab, stride;
    TokenIds targets;
    float scale;
    int top;
    float* logp;
    float* lse;
    float* entropy;
    int64_t* top_ids;
    float* top_logp;
    uint32_t* flags;
};

struct LogprobsGradArgs {
    const void* logits;
    int64_t rows, vocab, stride;
    TokenIds targets;
    float scale;
    const float* lse;
    const float* d_logp;      // or NULL
    const float* entropy;     // with d_entropy only
    const float* d_entropy;   // or NULL
    void* out;
    int64_t out_stride;
    uint32_t* flags;
};

cudaError_t launch_logprobs(const LogprobsArgs& a, bool bf16, cudaStream_t stream);
cudaError_t launch_logprobs_grad(const LogprobsGradArgs& a, bool bf16, cudaStream_t stream);

struct EmbeddingArgs {
    TokenIds ids;
    int64_t count;
    const void* table;
    int64_t vocab, width, stride;
    float scale;
    void* out;
    int64_t out_stride;
    uint32_t* flags;
};

struct EmbeddingGradArgs {
    TokenIds ids;
    int64_t count;
    const void* d_out;
    int64_t d_out_stride;
    int64_t vocab, width;
    float scale;
    int64_t padding_id;
    bool accumulate;
    float* d_table;
    int64_t stride;
    void* workspace;
    uint32_t* flags;
};

cudaError_t launch_embedding(const EmbeddingArgs& a, bool bf16, cudaStream_t stream);
size_t embedding_grad_workspace(int64_t count, int64_t vocab, int64_t width);
cudaError_t launch_embedding_grad(const EmbeddingGradArgs& a, bool bf16, cudaStream_t stream);

struct OrthogonalizeArgs {
    const void* update;
    int64_t batch, rows, cols, row_stride, batch_stride;
    float* momentum;   // or NULL
    float mu;
    bool nesterov;
    int steps;
    float coef[3];
    float eps;
    uint16_t* out;
    void* workspace;
    uint32_t* flags;
};

size_t orthogonalize_workspace(int64_t batch, int64_t rows, int64_t cols);
cudaError_t launch_orthogonalize(const OrthogonalizeArgs& a, bool bf16, cudaStream_t stream);

#if SPL_CHECKED
cudaError_t debug_read_logprobs(uint32_t* out, bool reset);
cudaError_t debug_read_embedding(uint32_t* out, bool reset);
cudaError_t debug_read_orthogonalize(uint32_t* out, bool reset);
#endif

}  // namespace spl
