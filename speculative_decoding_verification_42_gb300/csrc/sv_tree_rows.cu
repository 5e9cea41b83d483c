// sv_tree_rows.cu -- plan, append and keep (include/spec_tree.h): the operators
// that move integers and rows; every one of them is one launch.
#include <algorithm>

#include "sv_tree.cuh"

namespace sv {

// ------------------------------------------------------------------------- //
// k_tree_plan                                                               //
// ------------------------------------------------------------------------- //
// The pages of sequence b start at ring place head + sum of the wants of the
// sequences before it: a prefix sum over the batch.  Every CTA forms its own
// prefix from the lengths (a few integers per sequence, L2 resident), so no CTA
// waits for another and one launch suffices; the prefix costs B / 256 loads a
// thread, which at B = 1000 is less than a second launch would be.
constexpr int PLAN_THREADS = 256;
constexpr int PLAN_TOKENS = 1024;  // tokens of a sequence per CTA (grid y)
constexpr int PLAN_WORDS = SPEC_TREE_MAX_NODES / 32;
static_assert(SPEC_TREE_MAX_NODES <= PLAN_THREADS, "one thread per node of a tree");

// pages sequence b wants (> 0) or returns (< 0); 0 for lengths out of range
__device__ __forceinline__ int plan_delta(const TreePlanParams& p, int b, bool* ok)
{
    const SeqLen l = tree_len(p.s, b);
    const int held = __ldg(p.held + b);
    *ok = l.ok && held >= 0 && held <= p.s.width;
    if (!*ok) return 0;
    // ctx + n + page - 1 may pass 2^31
    const int need = (int)(((int64_t)l.ctx + l.n + (1 << p.s.page_log2) - 1) >> p.s.page_log2);
    return need - held;
}

__device__ __forceinline__ long long plan_block_sum(long long v, long long* red)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0;
    for (int i = 0; i < PLAN_THREADS / 32; ++i) v += red[i];
    __syncthreads();
    return v;
}

__global__ void __launch_bounds__(PLAN_THREADS) k_tree_plan(const TreePlanParams p)
{
    __shared__ long long red[PLAN_THREADS / 32];
    __shared__ int par[SPEC_TREE_MAX_NODES];
    const int tid = threadIdx.x, T = p.s.T;
    const int b0 = blockIdx.x * p.rows_per_cta, b1 = min(p.s.B, b0 + p.rows_per_cta);
    long long want = 0, back = 0;  // over the sequences before the current one
    for (int b = tid; b < b0; b += PLAN_THREADS) {
        bool ok;
        const int d = plan_delta(p, b, &ok);
        want += max(d, 0);
        back += max(-d, 0);
    }
    want = plan_block_sum(want, red);
    back = plan_block_sum(back, red);
    const long long N = p.s.num_pages, head = p.ring[0], tail = p.ring[1];
    // a ring outside its range holds nothing
    const long long avail = head >= 0 && tail - head >= 0 && tail - head <= N ? tail - head : 0;
    const long long head_at = ((head % N) + N) % N, tail_at = ((tail % N) + N) % N;
    const bool first_chunk = blockIdx.y == 0;
    for (int b = b0; b < b1; ++b) {
        bool ok;
        const int d = plan_delta(p, b, &ok);
        const SeqLen l = tree_len(p.s, b);
        const int held = __ldg(p.held + b), w = max(d, 0), r = max(-d, 0);
        const bool shortage = w > 0 && want + w > avail;
        const int need = shortage ? held : held + d;
        int32_t* row = p.table + (int64_t)b * p.s.width;
        // page i of the sequence: held, or the ring's (want + w <= N here)
        auto ring_page = [&](int i) {
            long long at = head_at + want + (i - held);
            if (at >= N) at -= N;
            return __ldg(p.free_pages + at);
        };
        bool bad = false;
        if (p.parents) {
            if (tid < l.n) {
                par[tid] = __ldg(p.parents + (int64_t)b * T + tid);
                bad = par[tid] < -1 || par[tid] >= tid;
            }
            bad = __syncthreads_or(bad);
        }
        const int status = !ok ? SPEC_ROW_BAD_LEN : shortage ? SPEC_ROW_NO_PAGES : bad ? SPEC_ROW_BAD_TREE : 0;
        if (first_chunk) {
            if (!shortage)
                for (int i = held + tid; i < need; i += PLAN_THREADS) row[i] = ring_page(i);
            for (int i = tid; i < r; i += PLAN_THREADS)
                p.free_pages[(tail_at + back + i) % N] = row[need + i];
            if (tid == 0) {
                p.held_out[b] = need;
                p.row_status[b] = status;
                if (shortage && want <= avail) p.ring_out[0] = head + want;  // the first that is short
            }
        }
        for (int j = blockIdx.y * PLAN_TOKENS + tid; j < min(T, (int)(blockIdx.y + 1) * PLAN_TOKENS);
             j += PLAN_THREADS) {
            const int64_t at = (int64_t)b * T + j;
            int slot = -1, pos = -1;
            uint32_t m[PLAN_WORDS] = {};
            if (status == 0 && j < l.n) {
                const int place = l.ctx + j, pg = place >> p.s.page_log2;
                const int page = pg < held ? row[pg] : ring_page(pg);
                if (page >= 0 && page < p.s.num_pages)
                    slot = (page << p.s.page_log2) + (place & ((1 << p.s.page_log2) - 1));
                pos = l.ctx + j;
                if (p.parents) {
                    int depth = -1;
                    for (int a = j; a >= 0; a = par[a], ++depth)
#pragma unroll
                        for (int x = 0; x < PLAN_WORDS; ++x)
                            if ((a >> 5) == x) m[x] |= 1u << (a & 31);
                    pos = l.ctx + depth;
                }
            }
            p.slot_map[at] = slot;
            p.positions[at] = pos;
            if (p.parents)
#pragma unroll
                for (int x = 0; x < PLAN_WORDS; ++x)
                    if (x < p.words) p.mask[at * p.words + x] = m[x];
        }
        want += w;
        back += r;
        __syncthreads();  // par is reused
    }
    if (first_chunk && b1 == p.s.B && tid == 0) {
        if (want <= avail) p.ring_out[0] = head + want;
        p.ring_out[1] = tail + back;
    }
}

cudaError_t launch_tree_plan(TreePlanParams p, int num_sms, cudaStream_t s)
{
    const int want = 4 * num_sms;
    p.rows_per_cta = std::max(1, (p.s.B + want - 1) / want);
    const dim3 grid(std::max(1, (p.s.B + p.rows_per_cta - 1) / p.rows_per_cta),
                    (p.s.T + PLAN_TOKENS - 1) / PLAN_TOKENS);
    k_tree_plan<<<grid, PLAN_THREADS, 0, s>>>(p);
    return cudaGetLastError();
}

// ------------------------------------------------------------------------- //
// k_tree_append                                                             //
// ------------------------------------------------------------------------- //
// One CTA per token; LANES threads hold one head, 8 elements (16 bytes) each.
constexpr int APP_THREADS = 256;

template <bool F16, int LANES>
__global__ void __launch_bounds__(APP_THREADS) k_tree_append(const TreeAppendParams p)
{
    using H = Half2<F16>;
    const int tok = blockIdx.x, b = tok / p.s.T, j = tok - b * p.s.T;
    const int li = threadIdx.x % LANES, gid = threadIdx.x / LANES;
    constexpr int GROUPS = APP_THREADS / LANES;
    const int Hq = p.s.Hq, Hkv = p.s.Hkv, D = p.s.D;
    const bool lane_on = li * 8 < D;
    const int slot = __ldg(p.slot_map + tok);
    const bool live = j < tree_nodes(p.s, b) && slot >= 0 && (slot >> p.s.page_log2) < p.s.num_pages;
    char* qo = (char*)p.q_out + ((int64_t)tok * Hq * D + li * 8) * 2;
    if (!live) {
        if (lane_on)
            for (int h = gid; h < Hq; h += GROUPS) *(uint4*)(qo + (int64_t)h * D * 2) = make_uint4(0, 0, 0, 0);
        return;
    }
    // the pair of element e sits rot / 2 away (halves) or beside it (interleaved)
    const int half = p.rot / 2, e0 = li * 8;
    const bool turn = p.cos_sin && e0 < p.rot;
    const bool lower = e0 < half;
    const int partner = (lower ? e0 + half : e0 - half) / 8;
    float cs[8], sn[8];  // angles of this thread's elements (interleaved: 4 pairs)
#pragma unroll
    for (int i = 0; i < 8; ++i) cs[i] = 1.f, sn[i] = 0.f;
    if (turn) {
        const int pos = __ldg(p.positions + tok);
        if (pos < 0 || pos >= p.table_len) {
#pragma unroll
            for (int i = 0; i < 8; ++i) cs[i] = sn[i] = __int_as_float(0x7fc00000);
        } else {
            const float* t = p.cos_sin + (int64_t)pos * p.rot;
            const int i0 = p.interleaved ? e0 / 2 : lower ? e0 : e0 - half;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < (p.interleaved ? 4 : 8)) cs[i] = __ldg(t + i0 + i), sn[i] = __ldg(t + half + i0 + i);
        }
    }
    const int64_t row = (int64_t)(slot >> p.s.page_log2) * p.c.page +
                        (int64_t)(slot & ((1 << p.s.page_log2) - 1)) * p.c.token;
    const int total = Hq + 2 * Hkv;
    for (int h0 = 0; h0 < total; h0 += GROUPS) {
        const int h = h0 + gid;
        const bool on = h < total && lane_on;
        const int kind = h < Hq ? 0 : h < Hq + Hkv ? 1 : 2;
        const int hh = kind == 0 ? h : kind == 1 ? h - Hq : h - Hq - Hkv;
        const TreeRows& src = kind == 0 ? p.q : kind == 1 ? p.k : p.v;
        uint4 x = make_uint4(0, 0, 0, 0);
        if (on)
            x = ld_stream16((const char*)src.ptr +
                            (b * src.seq + (int64_t)j * src.token + hh * src.head + e0) * 2);
        float y[8];
        const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = H::unpack(xs[i]);
            y[2 * i] = f.x, y[2 * i + 1] = f.y;
        }
        const void* w = kind == 0 ? p.qw : p.kw;
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss += y[i] * y[i];
#pragma unroll
        for (int o = LANES / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        if (kind < 2 && w && on) {
            const float r = 1.f / sqrtf(ss / (float)D + p.eps);
            const uint4 wv = __ldg((const uint4*)((const char*)w + e0 * 2));
            const uint32_t ws[4] = {wv.x, wv.y, wv.z, wv.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 f = H::unpack(ws[i]);
                y[2 * i] *= r * f.x, y[2 * i + 1] *= r * f.y;
            }
        }
        float z[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) z[i] = __shfl_sync(0xffffffffu, y[i], partner, LANES);
        if (kind < 2 && turn) {
            if (p.interleaved) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float a = y[2 * i], c = y[2 * i + 1];
                    y[2 * i] = a * cs[i] - c * sn[i];
                    y[2 * i + 1] = c * cs[i] + a * sn[i];
                }
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) y[i] = y[i] * cs[i] + (lower ? -z[i] : z[i]) * sn[i];
            }
        }
        if (!on) continue;
        if (kind < 2)
            x = make_uint4(H::pack(y[0], y[1]), H::pack(y[2], y[3]), H::pack(y[4], y[5]), H::pack(y[6], y[7]));
        char* dst = kind == 0 ? qo + (int64_t)hh * D * 2
                              : (char*)(kind == 1 ? p.c.k : p.c.v) + (row + hh * p.c.head + e0) * 2;
        *(uint4*)dst = x;
    }
}

cudaError_t launch_tree_append(const TreeAppendParams& p, int dtype, cudaStream_t s)
{
    const int tokens = p.s.B * p.s.T;
    auto go = [&](auto kernel) { kernel<<<tokens, APP_THREADS, 0, s>>>(p); };
    const bool f16 = dtype == SPEC_F16;
    if (p.s.D <= 64) f16 ? go(k_tree_append<true, 8>) : go(k_tree_append<false, 8>);
    else if (p.s.D <= 128) f16 ? go(k_tree_append<true, 16>) : go(k_tree_append<false, 16>);
    else f16 ? go(k_tree_append<true, 32>) : go(k_tree_append<false, 32>);
    return cudaGetLastError();
}

// ------------------------------------------------------------------------- //
// k_tree_keep                                                               //
// ------------------------------------------------------------------------- //
// Thread = one 16-byte column of a head row; it takes the path's rows in
// ascending order, four at a time (loads before stores).  path is strictly
// ascending, so path[i] >= i and a row stored at place i < path[k] for every
// k > i: no store reaches a row that is still to be read.
constexpr int KEEP_THREADS = 256;

__global__ void __launch_bounds__(KEEP_THREADS) k_tree_keep(const TreeKeepParams p)
{
    const int b = blockIdx.x, layer = blockIdx.y;
    const SeqLen l = tree_len(p.s, b);
    const int len = __ldg(p.path_len + b);
    const bool len_ok = l.ok && len >= 0 && len <= l.n;
    const int32_t* path = p.path + (int64_t)b * p.s.T;
    bool bad = false;
    if (len_ok)
        for (int i = threadIdx.x; i < len; i += KEEP_THREADS)
            bad = bad || path[i] <= (i ? path[i - 1] : -1) || path[i] >= l.n;
    bad = __syncthreads_or(bad);
    if (layer == 0 && blockIdx.z == 0 && threadIdx.x == 0) {
        const bool moves = len_ok && !bad;
        p.ctx_out[b] = __ldg(p.s.ctx_len + b) + (moves ? len : 0);
        if (p.row_status) p.row_status[b] = !len_ok ? SPEC_ROW_BAD_LEN : bad ? SPEC_ROW_BAD_TREE : 0;
    }
    if (!len_ok || bad) return;
    const int32_t* row = p.table + (int64_t)b * p.s.width;
    // element offset of token `at` of the sequence; -1 for a page outside the cache
    auto offset = [&](int at) -> int64_t {
        const int page = __ldg(row + (at >> p.s.page_log2));
        if (page < 0 || page >= p.s.num_pages) return -1;
        return (int64_t)page * p.c.page + (int64_t)(at & ((1 << p.s.page_log2) - 1)) * p.c.token;
    };
    const int per_head = p.s.D / 8, cols = p.s.Hkv * per_head;
    char* base = (char*)(blockIdx.z ? p.c.v : p.c.k) + (int64_t)layer * p.c.layer * 2;
    for (int col = threadIdx.x; col < cols; col += KEEP_THREADS) {
        const int head = col / per_head;
        char* at = base + (head * p.c.head + (col - head * per_head) * 8) * 2;
        for (int i0 = 0; i0 < len; i0 += 4) {
            uint4 x[4];
            int64_t to[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int i = i0 + k;
                to[k] = -1;
                if (i < len && path[i] != i) {
                    const int64_t from = offset(l.ctx + path[i]);
                    if (from >= 0) {
                        to[k] = offset(l.ctx + i);
                        x[k] = *(const uint4*)(at + from * 2);
                    }
                }
            }
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (to[k] >= 0) *(uint4*)(at + to[k] * 2) = x[k];
        }
    }
}

cudaError_t launch_tree_keep(const TreeKeepParams& p, cudaStream_t s)
{
    k_tree_keep<<<dim3(p.s.B, p.c.layers, 2), KEEP_THREADS, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace sv
