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
// thread, which at B = 1000 is less than a second launch would be.  Bound by
// latency: the dependent loads (lengths, ring, then pages), the barriers and the
// walks up the trees.  A warm call takes 6.4 us for 64 trees of 9 nodes and 10.4
// us for 1000 of up to 64, a launch alone some 2.5.
constexpr int PLAN_THREADS = 256;
constexpr int PLAN_TOKENS = 1024;  // tokens of a sequence per CTA (grid y), more where the grid ends
constexpr int PLAN_MAX_Y = 65535;  // most CTAs of a grid's y
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
            // a sequence that gets no pages loses what these entries held before: pages it gave
            // back, which may be another sequence's by now
            for (int i = held + tid; i < held + w; i += PLAN_THREADS) row[i] = shortage ? -1 : ring_page(i);
            for (int i = tid; i < r; i += PLAN_THREADS)
                p.free_pages[(tail_at + back + i) % N] = row[need + i];
            if (tid == 0) {
                p.held_out[b] = need;
                p.row_status[b] = status;
                if (shortage && want <= avail) p.ring_out[0] = head + want;  // the first that is short
            }
        }
        for (int64_t i = (int64_t)blockIdx.y * PLAN_THREADS + tid; i < T; i += (int64_t)gridDim.y * PLAN_THREADS) {
            const int j = (int)i;
            const int64_t at = (int64_t)b * T + j;
            int slot = -1, pos = -1;
            uint32_t m[PLAN_WORDS] = {};
            if (status == 0 && j < l.n) {
                const int place = l.ctx + j, pg = place >> p.s.page_log2;
                const int page = pg < held ? row[pg] : ring_page(pg);
                if (page >= 0 && page < p.s.num_pages) {
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
                    std::min((p.s.T - 1) / PLAN_TOKENS + 1, PLAN_MAX_Y));
    k_tree_plan<<<grid, PLAN_THREADS, 0, s>>>(p);
    return cudaGetLastError();
}

// ------------------------------------------------------------------------- //
// k_tree_append                                                             //
// ------------------------------------------------------------------------- //
// LANES threads hold one head, 8 elements (16 bytes) each.  With x the head, z
// each element's mate in its pair, w the weights and r = 1 / sqrt(mean(x^2) +
// eps), the norm and the rotation are y = r (x A + z B) with A = w cos and B =
// -+ w(mate) sin, which a thread forms once per token for all query heads and
// once for all key heads.  Its bytes (each element read and written once) would
// be HBM's to bound, but it is bound by latency and registers: A, B and the loads
// take 80 of them and spill, which leaves 24 warps to an SM, and the schedulers
// issue in half of their cycles.  So few instructions per element, and a token's
// heads on as few warps as still fill the machine (1, 2, 4 or 8; the angles and
// weights are per thread).  Loads of APP_UNROLL heads are in flight together (with
// eight, registers leave too few warps: 57 us for 6000 tokens).
// Everything is fp32 up to the one rounding of the output; rsqrtf is within two
// ulps.  Warm: one token of 80 heads of 128 elements 8.3 us, 64 sequences of up to
// 9 of them 12.5 us (1.6 TB/s), 100 of up to 60 f16 tokens of 36 heads of 80
// elements 31 us (1.8 TB/s), where a head of 80 leaves 6 of its 16 lanes idle.
constexpr int APP_THREADS = 256, APP_UNROLL = 4;

template <bool F16, int LANES>
__global__ void __launch_bounds__(APP_THREADS, 3) k_tree_append(const TreeAppendParams p, int warps_log2)
{
    using H = Half2<F16>;
    const int gwarp = blockIdx.x * (APP_THREADS / 32) + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    const int tok = gwarp >> warps_log2;
    if (tok >= p.s.B * p.s.T) return;  // whole warps
    const int b = tok / p.s.T, j = tok - b * p.s.T;
    const int li = lane % LANES, e0 = li * 8, D = p.s.D;
    const float inv_d = 1.f / (float)D;
    const int groups = (32 / LANES) << warps_log2;  // heads of the token at a time
    const int gid = (gwarp & ((1 << warps_log2) - 1)) * (32 / LANES) + lane / LANES;
    const bool lane_on = e0 < D;
    const int slot = __ldg(p.slot_map + tok), pos = p.cos_sin ? __ldg(p.positions + tok) : 0;
    const bool live = j < tree_nodes(p.s, b) && slot >= 0 && (slot >> p.s.page_log2) < p.s.num_pages;
    const int64_t row = (int64_t)(slot >> p.s.page_log2) * p.c.page +
                        (int64_t)(slot & ((1 << p.s.page_log2) - 1)) * p.c.token + e0;
    // the mate of element e is rot / 2 away (halves) or beside it (interleaved)
    const int half = p.rot / 2;
    const bool turn = lane_on && e0 < p.rot, lower = e0 < half, far = p.cos_sin && !p.interleaved;
    const int mate = turn && far ? (lower ? e0 + half : e0 - half) : e0;  // first element of the mates' lane
    float c[8], sn[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i] = 1.f, sn[i] = 0.f;
    if (turn) {
        if (pos < 0 || pos >= p.table_len) {
#pragma unroll
            for (int i = 0; i < 8; ++i) c[i] = sn[i] = __int_as_float(0x7fc00000);
        } else if (p.interleaved) {
            const float* t = p.cos_sin + (int64_t)pos * p.rot + e0 / 2;
            const float4 x = __ldg((const float4*)t), y = __ldg((const float4*)(t + half));
            c[0] = c[1] = x.x, c[2] = c[3] = x.y, c[4] = c[5] = x.z, c[6] = c[7] = x.w;
            sn[1] = y.x, sn[3] = y.y, sn[5] = y.z, sn[7] = y.w;
            sn[0] = -y.x, sn[2] = -y.y, sn[4] = -y.z, sn[6] = -y.w;
        } else {
            const float* t = p.cos_sin + (int64_t)pos * p.rot + (lower ? e0 : e0 - half);
#pragma unroll
            for (int i = 0; i < 8; i += 4) {
                const float4 x = __ldg((const float4*)(t + i)), y = __ldg((const float4*)(t + half + i));
                c[i] = x.x, c[i + 1] = x.y, c[i + 2] = x.z, c[i + 3] = x.w;
                sn[i] = lower ? -y.x : y.x, sn[i + 1] = lower ? -y.y : y.y;
                sn[i + 2] = lower ? -y.z : y.z, sn[i + 3] = lower ? -y.w : y.w;
            }
        }
    }

#pragma unroll 1
    for (int kind = 0; kind < 3; ++kind) {
        const TreeRows& src = kind == 0 ? p.q : kind == 1 ? p.k : p.v;
        const void* w = kind == 0 ? p.qw : kind == 1 ? p.kw : nullptr;
        const int heads = kind == 0 ? p.s.Hq : p.s.Hkv;
        const char* from = (const char*)src.ptr + (b * src.seq + (int64_t)j * src.token + e0) * 2;
        char* to = kind == 0 ? (char*)p.q_out + ((int64_t)tok * p.s.Hq * D + e0) * 2
                             : (char*)(kind == 1 ? p.c.k : p.c.v) + row * 2;
        const int64_t from_head = src.head * 2, to_head = kind == 0 ? (int64_t)D * 2 : p.c.head * 2;
        float A[8], Bm[8];
        if (kind < 2) {
            uint4 wa = make_uint4(0, 0, 0, 0), wb = wa;
            if (w && lane_on) wa = __ldg((const uint4*)((const char*)w + e0 * 2)), wb = __ldg((const uint4*)((const char*)w + mate * 2));
            const uint32_t was[4] = {wa.x, wa.y, wa.z, wa.w}, wbs[4] = {wb.x, wb.y, wb.z, wb.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 own = w ? H::unpack(was[i]) : make_float2(1.f, 1.f);
                float2 other = w ? H::unpack(wbs[i]) : make_float2(1.f, 1.f);
                if (!far) other = make_float2(other.y, other.x);
                A[2 * i] = own.x * c[2 * i], A[2 * i + 1] = own.y * c[2 * i + 1];
                Bm[2 * i] = other.x * sn[2 * i], Bm[2 * i + 1] = other.y * sn[2 * i + 1];
            }
        }
#pragma unroll 1
        for (int h0 = 0; h0 < heads; h0 += groups * APP_UNROLL) {
            uint4 x[APP_UNROLL];
#pragma unroll
            for (int u = 0; u < APP_UNROLL; ++u) {
                const int h = h0 + u * groups + gid;
                x[u] = make_uint4(0, 0, 0, 0);
                if (h < heads && lane_on && live) x[u] = ld_stream16(from + h * from_head);
            }
#pragma unroll
            for (int u = 0; u < APP_UNROLL; ++u) {
                if (h0 + u * groups >= heads) break;  // the same for the whole warp
                const int h = h0 + u * groups + gid;
                uint4 v = x[u];
                if (kind < 2) {
                    const uint32_t xs[4] = {v.x, v.y, v.z, v.w};
                    float y[8];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 f = H::unpack(xs[i]);
                        y[2 * i] = f.x, y[2 * i + 1] = f.y;
                    }
                    float r = 1.f;
                    if (w) {
                        float ss = 0.f;
#pragma unroll
                        for (int i = 0; i < 8; ++i) ss += y[i] * y[i];
#pragma unroll
                        for (int o = LANES / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
                        r = rsqrtf(ss * inv_d + p.eps);
                    }
                    uint32_t out[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float2 z = make_float2(y[2 * i + 1], y[2 * i]);
                        if (far) z = H::unpack(__shfl_sync(0xffffffffu, xs[i], mate / 8, LANES));
                        float a0 = y[2 * i] * A[2 * i], a1 = y[2 * i + 1] * A[2 * i + 1];
                        // not past rot_dim, where Bm is 0: 0 times an infinite or NaN mate is NaN
                        if (turn) a0 += z.x * Bm[2 * i], a1 += z.y * Bm[2 * i + 1];
                        out[i] = H::pack(a0 * r, a1 * r);
                    }
                    v = make_uint4(out[0], out[1], out[2], out[3]);
                }
                if (!live) v = make_uint4(0, 0, 0, 0);
                if (h < heads && lane_on && (live || kind == 0)) *(uint4*)(to + h * to_head) = v;
            }
        }
        if (!live) break;  // only q_out is written, with zeros
    }
}

cudaError_t launch_tree_append(const TreeAppendParams& p, int dtype, int num_sms, cudaStream_t s)
{
    const int64_t tokens = (int64_t)p.s.B * p.s.T;
    // as many warps per token, up to 8, as leave no more than 24 to an SM (what its registers hold): one
    // token of 80 heads takes 8.4 us with eight warps and 20.6 with one, 576 such tokens 12.5 us with
    // four, 16.5 with eight and 24.7 with one, 6000 tokens of 36 heads 31 us with one and 68 with eight
    int log2 = 0;
    while (log2 < 3 && (tokens << (log2 + 1)) <= 24 * (int64_t)num_sms) ++log2;
    const unsigned grid = (unsigned)(((tokens << log2) + APP_THREADS / 32 - 1) / (APP_THREADS / 32));
    auto go = [&](auto kernel) { kernel<<<grid, APP_THREADS, 0, s>>>(p, log2); };
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
// k > i: no store reaches a row that is still to be read.  The path and its pages
// are looked over first, so that a sequence that cannot move keeps all its rows.
// Bound by the latency of its dependent loads (path, table, row): warm 6.2 us for
// 64 sequences and 4 layers, 10.5 us for 200 and 8 (10.1 without the pages).
constexpr int KEEP_THREADS = 256;

__global__ void __launch_bounds__(KEEP_THREADS) k_tree_keep(const TreeKeepParams p)
{
    const int b = blockIdx.x, layer = blockIdx.y;
    const SeqLen l = tree_len(p.s, b);
    const int len = __ldg(p.path_len + b), planned = p.plan_status ? __ldg(p.plan_status + b) : 0;
    const bool len_ok = l.ok && len >= 0 && len <= l.n;
    const int32_t* path = p.path + (int64_t)b * p.s.T;
    const int32_t* row = p.table + (int64_t)b * p.s.width;
    auto in_cache = [&](int at) { return (unsigned)__ldg(row + (at >> p.s.page_log2)) < (unsigned)p.s.num_pages; };
    bool bad = false, lost = false;
    if (len_ok && planned == 0)
        for (int i = threadIdx.x; i < len; i += KEEP_THREADS) {
            // two loads at a time: the path's, then the tables'
            const int node = path[i], before = i ? path[i - 1] : -1;
            const bool inside = node >= 0 && node < l.n, from = in_cache(l.ctx + (inside ? node : 0)),
                       to = in_cache(l.ctx + i);
            bad = bad || !inside || node <= before;
            lost = lost || !from || !to;
        }
    if (__syncthreads_or(bad || lost)) {  // rare
        bad = __syncthreads_or(bad);
        lost = !bad;
    }
    const int status = planned ? planned : !len_ok ? SPEC_ROW_BAD_LEN : bad ? SPEC_ROW_BAD_TREE
                                                                            : lost ? SPEC_ROW_NO_PAGES : 0;
    if (layer == 0 && blockIdx.z == 0 && threadIdx.x == 0) {
        p.ctx_out[b] = __ldg(p.s.ctx_len + b) + (status == 0 ? len : 0);
        if (p.row_status) p.row_status[b] = status;
    }
    if (status != 0) return;
    // element offset of token `at` of the sequence, whose page is in the cache
    auto offset = [&](int at) {
        const int page = __ldg(row + (at >> p.s.page_log2));
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
                    to[k] = offset(l.ctx + i);
                    x[k] = *(const uint4*)(at + offset(l.ctx + path[i]) * 2);
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
