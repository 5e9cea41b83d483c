// sv_score.cuh -- parameters of the operators that score rows of logits
// (include/spec_score.h), and what their kernels share.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "spec_score.h"
#include "sv_internal.cuh"

namespace sv {

// n / d for 0 <= n < 2^28, by a product (Granlund and Montgomery's division by an invariant)
struct FastDiv {
    uint32_t mul = 0, shift = 0;
    FastDiv() = default;
    explicit FastDiv(uint32_t d)
    {
        while (((uint64_t)1 << shift) < d) ++shift;
        mul = (uint32_t)((((uint64_t)1 << 32) * (((uint64_t)1 << shift) - d)) / d + 1);
    }
    __device__ __forceinline__ int of(int n) const { return (int)((__umulhi((uint32_t)n, mul) + (uint32_t)n) >> shift); }
};

struct ScoreParams {
    const char* x;           // logits
    int64_t x_seq, x_tok;    // strides, elements
    char* grad;              // gradient rows or NULL
    int64_t g_seq, g_tok;
    int32_t rows, T, V;
    float inv_temp, c;       // 1 / temperature, log2(e) / it
    // what the launch fills in
    FastDiv by_tokens;       // of a row: its sequence
    int32_t cluster;         // CTAs of a row
    int32_t per;             // vectors of 16 bytes of a CTA
    int32_t* row_status;
    const int32_t* ids;      // logprobs: [rows] or NULL; distill: [rows, k]
    // logprobs
    const float* g_logprob;  // [rows] or NULL
    const float* g_entropy;
    int32_t top_n;
    float* logprob;
    int32_t* rank;
    float* entropy;
    float* lse;
    int32_t* top_ids;        // [rows, top_n]
    float* top_lp;
    // distill
    const void* teacher;     // [rows, k]
    int32_t teacher_dtype;
    int32_t k, tail;
    float inv_tt, inv_tt_lo; // 1 / the teacher's temperature, and what is left of it
    const float* teacher_lse;
    const float* g_loss;
    float* loss;
    float* accept;
};

cudaError_t launch_score_logprobs(const ScoreParams& p, int dtype, int num_sms, cudaStream_t s);
cudaError_t launch_score_distill(const ScoreParams& p, int dtype, int num_sms, cudaStream_t s);

constexpr int SCORE_MAX_CTAS = 8;                                    // of a row
constexpr double SCORE_L2_ROWS = 100e6;                             // bytes of rows under way between two passes
constexpr size_t SCORE_MAX_ROW_BYTES = SCORE_MAX_CTAS * 208 * 1024;  // of one row of logits

}  // namespace sv
