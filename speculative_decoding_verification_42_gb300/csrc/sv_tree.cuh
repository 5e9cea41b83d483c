// sv_tree.cuh -- parameters and small device helpers of the operators around a
// verify step (include/spec_tree.h): plan, append, attend, keep.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "sv_internal.cuh"
#include "spec_tree.h"

namespace sv {

// what every operator knows of the batch and of the cache
struct TreeShape {
    int32_t B, T;            // sequences, padded nodes per sequence
    int32_t Hq, Hkv, D;
    int32_t page_log2;       // tokens per page = 1 << page_log2
    int32_t width;           // pages per row of a block table
    int32_t num_pages;
    const int32_t* ctx_len;  // [B]
    const int32_t* n_tokens; // [B] or NULL
};

struct SeqLen {
    int ctx, n;  // n = 0 for a sequence whose lengths are outside their ranges
    bool ok;
};

__device__ __forceinline__ int tree_nodes(const TreeShape& s, int b)
{
    return s.n_tokens ? __ldg(s.n_tokens + b) : s.T;
}

__device__ __forceinline__ SeqLen tree_len(const TreeShape& s, int b)
{
    SeqLen l;
    l.ctx = __ldg(s.ctx_len + b);
    l.n = tree_nodes(s, b);
    // width << page_log2 is below 2^31 (checked at create), n <= T
    l.ok = l.ctx >= 0 && l.n >= 0 && l.n <= s.T && (int64_t)l.ctx + l.n <= ((int64_t)s.width << s.page_log2);
    if (!l.ok) l.ctx = l.n = 0;
    return l;
}

struct TreePlanParams {
    TreeShape s;
    const int32_t* parents;
    const int32_t* held;
    const int64_t* ring;
    int32_t* free_pages;
    int32_t* table;
    int32_t* held_out;
    int64_t* ring_out;
    int32_t* slot_map;
    int32_t* positions;
    uint32_t* mask;
    int32_t* row_status;
    int32_t rows_per_cta;
    int32_t words;           // ceil(T / 32)
};

struct TreeRows {
    const void* ptr;
    int64_t seq, token, head;  // strides in elements
};

struct TreeCachePtrs {
    void *k, *v;
    int64_t page, token, head, layer;  // strides in elements
    int32_t layers;
};

struct TreeAppendParams {
    TreeShape s;
    TreeRows q, k, v;
    TreeCachePtrs c;
    const int32_t* slot_map;
    const int32_t* positions;
    const void* qw;
    const void* kw;
    const float* cos_sin;
    int32_t table_len, rot, interleaved;
    float eps;
    void* q_out;
};

struct TreeAttendParams {
    TreeShape s;
    TreeRows q;
    TreeCachePtrs c;
    const int32_t* table;
    const uint32_t* mask;
    int32_t words;
    float scale;
    void* out;
    float* lse;
};

struct TreeKeepParams {
    TreeShape s;
    TreeCachePtrs c;
    const int32_t* table;
    const int32_t* path;
    const int32_t* path_len;
    const int32_t* plan_status;
    int32_t* ctx_out;
    int32_t* row_status;
};

cudaError_t launch_tree_plan(TreePlanParams p, int num_sms, cudaStream_t s);
cudaError_t launch_tree_append(const TreeAppendParams& p, int dtype, int num_sms, cudaStream_t s);
// bytes of workspace (zeroed before the first call) for `ctas` CTAs, and where
// in it the (m, l) and the joins begin
size_t tree_attend_bytes(int D, int ctas, size_t* ml_at, size_t* join_at);
// key tiles of a call are counted in 32 bits
bool tree_attend_fits(const TreeShape& s);
// err: bit 0 set when a bounded wait ran out; stall: issue no copy
cudaError_t launch_tree_attend(const TreeAttendParams& p, int dtype, int num_sms, void* ws, unsigned* err, bool stall,
                               cudaStream_t s);
cudaError_t launch_tree_keep(const TreeKeepParams& p, cudaStream_t s);

// 16-bit element types: unpacking two of a word, packing, converting
template <bool F16> struct Half2;
template <> struct Half2<false> {
    static __device__ __forceinline__ float2 unpack(uint32_t w) { return make_float2(bf16_lo(w), bf16_hi(w)); }
    static __device__ __forceinline__ uint32_t pack(float a, float b)
    {
        uint32_t r;
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
        return r;
    }
    static __device__ __forceinline__ float one(uint16_t h) { return __uint_as_float((uint32_t)h << 16); }
};
template <> struct Half2<true> {
    static __device__ __forceinline__ float2 unpack(uint32_t w)
    {
        const __half2 h = *reinterpret_cast<const __half2*>(&w);
        return __half22float2(h);
    }
    static __device__ __forceinline__ uint32_t pack(float a, float b)
    {
        uint32_t r;
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
        return r;
    }
    static __device__ __forceinline__ float one(uint16_t h) { return __half2float(__ushort_as_half(h)); }
};

}  // namespace sv
