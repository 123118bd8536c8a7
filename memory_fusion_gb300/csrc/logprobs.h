// logprobs.h -- launchers of the log probabilities of given tokens (logprobs.cu), shared with the C-ABI layer.  Not part
// of the public ABI.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace cf {

constexpr int kLogprobsMaxTop = 32;
constexpr int64_t kLogprobsMaxVocab = int64_t(1) << 24;

struct LogprobsArgs {
    const void *logits;
    const int64_t *targets;  // [rows] or null
    float *logprob, *lse, *entropy, *top_logprobs;  // each or null
    int64_t *top_ids;        // or null
    uint32_t *err;
    int64_t rows, stride;    // stride: elements from a row to the next
    int vocab, top, dtype;
    float scale;
    int cluster;             // CTAs of a row (the launcher's)
};
cudaError_t launch_logprobs(LogprobsArgs a, int sms, bool pdl, cudaStream_t stream);

struct LogprobsGradArgs {
    const void *logits;
    const int64_t *targets;  // or null
    const float *lse, *entropy, *dlogprob, *dlse, *dentropy;  // lse: always; entropy where dentropy is
    void *dlogits;
    uint32_t *err;
    int64_t rows, stride, dstride;
    int vocab, dtype;
    float scale;
    int chunks, turns;       // CTAs of a row, and turns of a CTA's loop (the launcher's)
};
cudaError_t launch_logprobs_grad(LogprobsGradArgs a, bool pdl, cudaStream_t stream);
// CTAs that a gradient takes
int64_t logprobs_grad_ctas(int64_t rows, int64_t vocab, int dtype);

}  // namespace cf
