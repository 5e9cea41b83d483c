// sv_tree_attend.cu -- attention of a tree of drafted tokens over the paged
// cache (spec_tree_attend).
#include "sv_tree.cuh"

namespace sv {

// One warp per (sequence, node, query head); lanes hold the head's elements;
// one pass over the keys with the running maximum and sum of the softmax.
constexpr int ATT_WARPS = 8;

template <bool F16>
__global__ void __launch_bounds__(ATT_WARPS * 32) k_tree_attend(const TreeAttendParams p)
{
    using H = Half2<F16>;
    const int64_t r = (int64_t)blockIdx.x * ATT_WARPS + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31, D = p.s.D, Hq = p.s.Hq;
    if (r >= (int64_t)p.s.B * p.s.T * Hq) return;
    const int h = (int)(r % Hq), j = (int)(r / Hq % p.s.T), b = (int)(r / Hq / p.s.T);
    const SeqLen l = tree_len(p.s, b);
    const int hk = h / (Hq / p.s.Hkv);
    const uint16_t* q = (const uint16_t*)p.q.ptr + b * p.q.seq + (int64_t)j * p.q.token + h * p.q.head;
    const uint32_t* mask = p.mask ? p.mask + ((int64_t)b * p.s.T + j) * p.words : nullptr;
    float qv[8], o[8] = {};
    for (int i = 0; i < 8; ++i) qv[i] = lane + 32 * i < D && j < l.n ? H::one(q[lane + 32 * i]) : 0.f;
    float m = -INFINITY, sum = 0.f;
    const int keys = j < l.n ? l.ctx + l.n : 0;
    for (int k = 0; k < keys; ++k) {
        const int node = k - l.ctx;
        if (node >= 0 && !(mask ? (mask[node >> 5] >> (node & 31)) & 1u : node <= j)) continue;
        const int page = p.table[(int64_t)b * p.s.width + (k >> p.s.page_log2)];
        const bool in = page >= 0 && page < p.s.num_pages;
        const int64_t off = (int64_t)page * p.c.page + (k & ((1 << p.s.page_log2) - 1)) * p.c.token + hk * p.c.head;
        const uint16_t *kr = (const uint16_t*)p.c.k + off, *vr = (const uint16_t*)p.c.v + off;
        float s = 0.f;
        for (int i = 0; i < 8; ++i)
            if (in && lane + 32 * i < D) s += qv[i] * H::one(kr[lane + 32 * i]);
        for (int w = 16; w > 0; w >>= 1) s += __shfl_xor_sync(0xffffffffu, s, w);
        s *= p.scale;
        const float nm = fmaxf(m, s), ref = nm == -INFINITY ? 0.f : nm;
        const float c = expf(m - ref), e = expf(s - ref);
        m = nm;
        sum = sum * c + e;
        for (int i = 0; i < 8; ++i)
            o[i] = o[i] * c + (in && lane + 32 * i < D ? e * H::one(vr[lane + 32 * i]) : 0.f);
    }
    const bool none = !(sum > 0.f) && sum == sum;
    uint16_t* out = (uint16_t*)p.out + r * D;
    for (int i = 0; i < 8; ++i)
        if (lane + 32 * i < D) out[lane + 32 * i] = (uint16_t)H::pack(none ? 0.f : o[i] / sum, 0.f);
    if (p.lse && lane == 0) p.lse[r] = none ? -INFINITY : m + logf(sum);
}

cudaError_t launch_tree_attend(const TreeAttendParams& p, int dtype, int num_sms, cudaStream_t s)
{
    const int64_t rows = (int64_t)p.s.B * p.s.T * p.s.Hq;
    const unsigned grid = (unsigned)((rows + ATT_WARPS - 1) / ATT_WARPS);
    if (dtype == SPEC_F16) k_tree_attend<true><<<grid, ATT_WARPS * 32, 0, s>>>(p);
    else k_tree_attend<false><<<grid, ATT_WARPS * 32, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace sv
