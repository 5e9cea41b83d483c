// sv_score_distill.cu -- the divergence of a row's distribution from a
// teacher's top logits, and its gradient.
//
// The mass of the tokens without an entry (the rest) is summed apart, relative
// to their own maximum: what is left of a confident row when its entries are
// taken out may be far below what fp32 holds beside them, and as a difference it
// would be noise.  The loss is a sum of h(q, p) = q ln(q / p) - q + p >= 0, one
// for each entry and one for the rest (the q and the p sum to 1, so the added
// terms cancel): near its minimum, where sum q ln(q / p) is a small difference
// of terms of the size of ln Z, every h is small by itself and fp32 is enough.
#include "sv_score_row.cuh"

namespace sv {

namespace {

constexpr int SC_EPT = SPEC_SCORE_MAX_ENTRIES / SC_NT;  // entries of a thread: tid, tid + SC_NT

__device__ __forceinline__ float teacher_value(const ScoreParams& p, int64_t at)
{
    return p.teacher_dtype == SPEC_F32 ? ((const float*)p.teacher)[at]
           : p.teacher_dtype == SPEC_BF16 ? __bfloat162float(((const __nv_bfloat16*)p.teacher)[at])
                                          : __half2float(((const __half*)p.teacher)[at]);
}

struct KdPart {      // a warp's sum of the rest
    float m, s;
};
struct KdRow {
    float mr, m;      // maximum of the rest and of the row
    float sr, z;      // their sums, each relative to its own
    float scale;      // of the rest's in the row's
    float inv_z, inv_sr;
};
__device__ __forceinline__ bool finite_row(float m) { return m > -INFINITY && m < INFINITY; }

template <typename E> __device__ void no_distill(const ScoreParams& p, int r, int status, int rank, int C)
{
    if (rank == 0 && threadIdx.x == 0) {
        const float none = status == SPEC_ROW_OK ? 0.f : __int_as_float(0x7FFFFFFF);
        p.row_status[r] = status;
        if (p.loss) p.loss[r] = none;
        if (p.accept) p.accept[r] = none;
    }
    if (p.grad) zero_grad<E>(p, r, rank, C);
}

// a row's entries, this thread's: token, teacher's value, the student's logit
struct Entries {
    int id[SC_EPT];
    float tv[SC_EPT], l[SC_EPT];
    __device__ __forceinline__ void fetch(const ScoreParams& p, int r)
    {
#pragma unroll
        for (int u = 0; u < SC_EPT; ++u) {
            const int i = threadIdx.x + u * SC_NT;
            const bool in = r < p.rows && i < p.k;
            id[u] = in ? p.ids[(int64_t)r * p.k + i] : -1;
            tv[u] = in ? teacher_value(p, (int64_t)r * p.k + i) : -INFINITY;
        }
    }
    template <typename E> __device__ __forceinline__ void fetch_logits(const E* x, int V)
    {
#pragma unroll
        for (int u = 0; u < SC_EPT; ++u) l[u] = id[u] >= 0 && id[u] < V ? widen(x[id[u]]) : -INFINITY;
    }
    __device__ __forceinline__ bool some() const
    {
        bool s = false;
#pragma unroll
        for (int u = 0; u < SC_EPT; ++u) s |= id[u] != -1;
        return s;
    }
};

// the teacher's distribution over a row's entries, this thread's
struct Teacher {
    float q[SC_EPT], lq[SC_EPT];  // lq: ln q
    float in, left;               // sum of q, what it leaves of 1
};

// what the threads of a CTA tell one another of a row's entries; the next row has another, as some are still at the
// last row's end when others begin it
struct EntryShared {
    int32_t ids[SPEC_SCORE_MAX_ENTRIES];
    int32_t slots[SPEC_SCORE_MAX_ENTRIES];
    float w_max[SC_WARPS], w_sum[SC_WARPS];
    float w_me[SC_WARPS], w_se[SC_WARPS];  // the student's largest logit at a warp's entries, and the sum of their 2^d
};

// Checks a row's entries (a barrier, then the checks; the caller passes bad to the next one) and starts the teacher's
// sums.  slots: see below; mark(u): called between the barriers.
template <typename Mark>
__device__ __forceinline__ bool check_entries(const ScoreParams& p, EntryShared& es, Entries& en, const int (&slot)[SC_EPT],
                                              bool (&first)[SC_EPT], float& tmax, Mark mark)
{
    const int tid = threadIdx.x, lane = tid % 32;
    tmax = -INFINITY;
#pragma unroll
    for (int u = 0; u < SC_EPT; ++u) {
        es.ids[tid + u * SC_NT] = en.id[u];
        es.slots[tid + u * SC_NT] = slot[u];
        if (en.id[u] == -1) en.tv[u] = -INFINITY;
        tmax = fmax_nan(tmax, en.tv[u]);
    }
    tmax = warp_max(tmax);
    if (lane == 0) es.w_max[tid / 32] = tmax;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < SC_WARPS; ++i) tmax = fmax_nan(tmax, es.w_max[i]);
    bool bad = false;
#pragma unroll
    for (int u = 0; u < SC_EPT; ++u) {
        const int i = tid + u * SC_NT, id = en.id[u];
        first[u] = slot[u] >= 0;
        if (id == -1) continue;
        bad |= id < -1 || id >= p.V;
        for (int j = 0; j < i; j += 4) {
            const int4 o = *(const int4*)(es.ids + j);
            bad |= o.x == id || (o.y == id && j + 1 < i) || (o.z == id && j + 2 < i) || (o.w == id && j + 3 < i);
        }
        if (first[u])
            for (int j = 0; j < i; j += 4) {
                const int4 o = *(const int4*)(es.slots + j);
                if (o.x == slot[u] || (o.y == slot[u] && j + 1 < i) || (o.z == slot[u] && j + 2 < i) ||
                    (o.w == slot[u] && j + 3 < i))
                    first[u] = false;
            }
        mark(u);
    }
    return bad;
}
__device__ __forceinline__ bool dull(const ScoreParams& p, float tmax, float lse)
{
    return !(tmax < INFINITY) || (!p.tail && tmax == -INFINITY) || !(fabsf(lse) < INFINITY);
}
// q up to the row's sum: differences first, and 1 / t in two parts, as the values may be large
__device__ __forceinline__ void begin_teacher(const ScoreParams& p, EntryShared& es, const Entries& en, float tmax, float lse,
                                              Teacher& te)
{
    float sum = 0.f;
#pragma unroll
    for (int u = 0; u < SC_EPT; ++u) {
        te.q[u] = 0.f;
        te.lq[u] = -INFINITY;
        if (en.tv[u] > -INFINITY) {
            te.lq[u] = p.tail ? fmaf(en.tv[u], p.inv_tt_lo, fmaf(en.tv[u], p.inv_tt, -lse))
                              : fmaf(en.tv[u] - tmax, p.inv_tt_lo, (en.tv[u] - tmax) * p.inv_tt);
            te.q[u] = expf(te.lq[u]);
        }
        sum += te.q[u];
    }
    sum = warp_sum(sum);
    if (threadIdx.x % 32 == 0) es.w_sum[threadIdx.x / 32] = sum;
}
__device__ __forceinline__ void end_teacher(const ScoreParams& p, const EntryShared& es, Teacher& te)
{
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < SC_WARPS; ++i) sum += es.w_sum[i];
    te.in = p.tail ? sum : 1.f;
    te.left = p.tail ? fmaxf(0.f, 1.f - sum) : 0.f;
    if (!p.tail) {
        const float ln = logf(sum), inv = 1.f / sum;
#pragma unroll
        for (int u = 0; u < SC_EPT; ++u) {
            te.q[u] *= inv;
            te.lq[u] -= ln;
        }
    }
}
// the entries' sums of a warp
__device__ __forceinline__ void sum_entries(const ScoreParams& p, EntryShared& es, const Entries& en)
{
    float me = -INFINITY, se = 0.f;
#pragma unroll
    for (int u = 0; u < SC_EPT; ++u) me = fmax_nan(me, en.l[u]);
    me = warp_max(me);
#pragma unroll
    for (int u = 0; u < SC_EPT; ++u) se += ex2_fast(dist(en.l[u], me, p.c));
    se = warp_sum(se);
    if (threadIdx.x % 32 == 0) {
        es.w_me[threadIdx.x / 32] = me;
        es.w_se[threadIdx.x / 32] = se;
    }
}
// one warp: the row of its warps' parts
__device__ __forceinline__ KdRow join(const KdPart* parts, const EntryShared& es, float c, int C)
{
    const int lane = threadIdx.x % 32;
    KdPart u = {-INFINITY, 0.f};
    if (lane < C * SC_WARPS) u = parts[lane];
    KdRow row;
    row.mr = warp_max(u.m);
    row.m = row.mr;
#pragma unroll
    for (int i = 0; i < SC_WARPS; ++i) row.m = fmax_nan(row.m, es.w_me[i]);
    row.sr = warp_sum(u.m == -INFINITY ? 0.f : u.s * ex2_fast(between(u.m, row.mr, c)));
    row.scale = row.mr == -INFINITY ? 0.f : ex2_fast(between(row.mr, row.m, c));
    row.z = row.sr * row.scale;
#pragma unroll
    for (int i = 0; i < SC_WARPS; ++i)
        if (es.w_me[i] > -INFINITY) row.z += es.w_se[i] * ex2_fast(between(es.w_me[i], row.m, c));
    row.inv_z = 1.f / row.z;
    row.inv_sr = row.sr > 0.f ? 1.f / row.sr : 0.f;
    return row;
}

// h(q, p); lr: ln(q / p), for a p too small for a quotient
__device__ __forceinline__ float divergence(float q, float p, float lr)
{
    if (q == 0.f) return p;
    if (!(p > 1e-30f)) return q * lr - q + p;
    const float d = (q - p) / p;
    return fabsf(d) < 0.5f ? p * ((1.f + d) * log1pf(d) - d) : q * logf(q / p) - q + p;
}

// CTA 0: a row's loss and acceptance
__device__ __forceinline__ void finish(const ScoreParams& p, int r, const KdRow& row, const Teacher& te,
                                       const float (&l)[SC_EPT])
{
    __shared__ float w_h[SC_WARPS], w_acc[SC_WARPS];
    const int tid = threadIdx.x, lane = tid % 32;
    const float ln_z = logf(row.z) - dist(row.m, row.m, p.c) * LN2;  // relative to m
    float h = 0.f, acc = 0.f;
#pragma unroll
    for (int u = 0; u < SC_EPT; ++u) {
        const float pi = ex2_fast(dist(l[u], row.m, p.c)) * row.inv_z;
        h += divergence(te.q[u], pi, te.lq[u] - ((l[u] - row.m) * p.inv_temp - ln_z));
        acc += fminf(te.q[u], pi);
    }
    h = warp_sum(h);
    acc = warp_sum(acc);
    if (lane == 0) {
        w_h[tid / 32] = h;
        w_acc[tid / 32] = acc;
    }
    __syncthreads();
    if (tid == 0) {
        h = acc = 0.f;
        for (int i = 0; i < SC_WARPS; ++i) {
            h += w_h[i];
            acc += w_acc[i];
        }
        const float pr = row.sr * row.scale * row.inv_z;
        if (p.tail) {
            // ln of the rest's share, from the logarithms of both sums and the distance of their references
            const float ln_pr = row.sr > 0.f ? (row.mr - row.m) * p.inv_temp + logf(row.sr) -
                                                   dist(row.mr, row.mr, p.c) * LN2 - ln_z
                                             : -INFINITY;
            h += divergence(te.left, pr, logf(te.left) - ln_pr) + fmaxf(0.f, te.in - 1.f);
        } else {
            h += pr;
        }
        const bool ok = finite_row(row.m);
        const float nan = __int_as_float(0x7FFFFFFF);
        p.row_status[r] = ok ? SPEC_ROW_OK : SPEC_ROW_NONFINITE;
        if (p.loss) p.loss[r] = ok ? h : nan;
        if (p.accept) p.accept[r] = ok ? acc : nan;
    }
}

// ---- forward -------------------------------------------------------------------- //
// A thread leaves out the copy groups of its vectors in which an entry lies (flags: a bit for each group and thread, the
// row's ends being group full + 1).  Those are read once more, each by the thread of the first entry in it (slots: group
// and thread), which takes the entries out.
template <typename E> __global__ void __launch_bounds__(SC_NT, 5) k_score_distill(const ScoreParams p)
{
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ __align__(16) EntryShared es;
    __shared__ KdPart parts[SC_PARTS];
    __shared__ KdRow s_row;
    const int C = p.cluster, rank = (int)cluster_rank(), r = cluster_id(), tid = threadIdx.x, lane = tid % 32;
    const int warp = tid / 32;
    Entries en;
    en.fetch(p, r);
    if (!__syncthreads_or(en.some())) {
        no_distill<E>(p, r, SPEC_ROW_OK, rank, C);
        return;
    }
    const E* x = row_of<E>(p, r);
    const Slice<E> sl(p, x, rank);
    Ring<E> ring(p, sl, rank, smem);
    en.fetch_logits(x, p.V);
    const uint4 edge = ring.edge();
    const float lse = p.teacher_lse ? p.teacher_lse[r] : 0.f;
    uint32_t* const flags = (uint32_t*)(smem + SC_RING_BYTES);
    for (int i = tid; i < (ring.full + 2) * SC_WARPS; i += SC_NT) flags[i] = 0;
    int slot[SC_EPT];
#pragma unroll
    for (int u = 0; u < SC_EPT; ++u) {
        slot[u] = -1;
        if (en.id[u] < sl.first || en.id[u] >= p.V || en.id[u] < 0) continue;
        const int i = (en.id[u] - sl.first) / EPV<E>;
        if (i >= sl.n) continue;
        slot[u] = i >= sl.lo && i < sl.hi ? i / Ring<E>::GROUP * SC_NT + i % SC_NT
                                          : (ring.full + 1) * SC_NT + (i < sl.lo ? 0 : 32);
    }
    float tmax;
    bool first[SC_EPT];
    bool bad = check_entries(p, es, en, slot, first, tmax, [&](int u) {
        if (slot[u] >= 0) atomicOr(flags + slot[u] / 32, 1u << (slot[u] % 32));
    });
    Teacher te;
    begin_teacher(p, es, en, tmax, lse, te);
    bad = __syncthreads_or(bad);
    if (bad || dull(p, tmax, lse)) {
        no_distill<E>(p, r, bad ? SPEC_ROW_BAD_TOKEN : SPEC_ROW_NONFINITE, rank, C);
        copy_arrived(0);
        return;
    }
    // every CTA of the cluster runs before another stores into its shared memory
    if (C > 1) cluster_arrive();
    Summer<E, false, false> rest;
    rest.c = p.c;
    rest.stream(ring, edge, [&](int b) { return flags[b * SC_WARPS + warp] >> lane & 1; }, [](int, float) {});
#pragma unroll
    for (int u = 0; u < SC_EPT; ++u) {
        if (!first[u]) continue;
        const int g = slot[u] / SC_NT, owner = slot[u] % SC_NT;
        const bool end = g > ring.full;
        uint4 w[SC_GROUP];
        int at[SC_GROUP];
#pragma unroll
        for (int j = 0; j < SC_GROUP; ++j) {
            at[j] = end ? (owner == 0 ? 0 : sl.n - 1) : (g * SC_GROUP + j) * SC_NT + owner;
            w[j] = end ? (j ? no_vector<E>() : load_vector(sl, p.V, at[j]))
                       : at[j] >= sl.lo && at[j] < sl.hi ? load_vector(sl, p.V, at[j]) : no_vector<E>();
        }
        uint32_t out = 0;  // the entries' elements
        for (int j = 0; j < p.k; j += 4) {
            const int4 o = *(const int4*)(es.slots + j);
            auto one = [&](int s, int j) {
                if (s != slot[u]) return;
                const int e = es.ids[j] - sl.first;
                out |= 1u << ((end ? 0 : (e / EPV<E> - at[0]) / SC_NT) * EPV<E> + e % EPV<E>);
            };
            one(o.x, j);
            one(o.y, j + 1);
            one(o.z, j + 2);
            one(o.w, j + 3);
        }
#pragma unroll
        for (int j = 0; j < SC_GROUP; ++j) {
            Bits<E> v[EPV<E>];
#pragma unroll
            for (int q = 0; q < EPV<E>; ++q)
                v[q] = out >> (j * EPV<E> + q) & 1 ? (Bits<E>)Vec<E>::NEG : bits_at<E>(w[j], q);
            w[j] = vector_of<E>(v);
        }
        rest.take(w, 0, 0);
    }
    Run run = rest.result();
    KdPart w;
    w.m = warp_max(run.m);
    to_max(run, w.m, p.c);
    w.s = warp_sum(run.s);
    if (C > 1) cluster_wait();
    if (lane == 0) {
        const uint32_t to = remote(parts + rank * SC_WARPS + warp, 0);
        remote_st(to, __float_as_uint(w.m));
        remote_st(to + 4, __float_as_uint(w.s));
    }
    if (rank == 0) sum_entries(p, es, en);
    row_arrive(C);
    if (rank != 0) return;
    if (C > 1) {
        row_wait(C);
        __syncthreads();
    }
    if (tid < 32) {
        const KdRow row = join(parts, es, p.c, C);
        if (lane == 0) s_row = row;
    }
    end_teacher(p, es, te);
    __syncthreads();
    finish(p, r, s_row, te, en.l);
}

// ---- with the gradient ------------------------------------------------------------ //
template <typename E> __global__ void __launch_bounds__(SC_NT) k_score_distill_grad(const ScoreParams p)
{
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ __align__(16) EntryShared shared[2];
    __shared__ KdPart parts[2][SC_PARTS];
    __shared__ KdRow s_row;
    const int C = p.cluster, rank = (int)cluster_rank(), tid = threadIdx.x, lane = tid % 32;
    const int step = gridDim.x / C;
    const Buffer<E> bf(p, rank, smem);
    auto settle = [&](int& r, Entries& en) {
        while (r < p.rows && !__syncthreads_or(en.some())) {
            no_distill<E>(p, r, SPEC_ROW_OK, rank, C);
            r += step;
            en.fetch(p, r);
        }
    };
    int r = cluster_id();
    Entries en, en2, en3;
    en.fetch(p, r);
    settle(r, en);
    if (r >= p.rows) return;
    if (C > 1) cluster_arrive();  // every CTA of the cluster runs before another stores into its shared memory
    bool started = false;
    const E* x = row_of<E>(p, r);
    Slice<E> sl(p, x, rank);
    bf.copy(sl);
    en.fetch_logits(x, p.V);
    int r2 = r + step, par = 0, sp = 0;
    en2.fetch(p, r2);
    while (true) {
        settle(r2, en2);
        const bool more = r2 < p.rows;
        Slice<E> next;
        if (more) {
            x = row_of<E>(p, r2);
            next = Slice<E>(p, x, rank);
            en2.fetch_logits(x, p.V);
        }
        const int r3 = r2 + step;
        en3.fetch(p, r3);
        const float lse = p.teacher_lse ? p.teacher_lse[r] : 0.f;
        EntryShared& es = shared[sp];
        sp ^= 1;
        int slot[SC_EPT];
        bool first[SC_EPT], mine[SC_EPT];
#pragma unroll
        for (int u = 0; u < SC_EPT; ++u) slot[u] = -1;
        float tmax;
        bool bad = check_entries(p, es, en, slot, first, tmax, [](int) {});
        Teacher te;
        begin_teacher(p, es, en, tmax, lse, te);
        sum_entries(p, es, en);
        copy_arrived(0);
        bad = __syncthreads_or(bad);
        if (bad || dull(p, tmax, lse)) {
            no_distill<E>(p, r, bad ? SPEC_ROW_BAD_TOKEN : SPEC_ROW_NONFINITE, rank, C);
            bf.copy(next);
        } else {
            end_teacher(p, es, te);
            // the entries leave the slice, whose sum and gradient are those of the rest
#pragma unroll
            for (int u = 0; u < SC_EPT; ++u) {
                mine[u] = en.id[u] >= 0 && bf.has(sl, en.id[u]);
                if (mine[u]) *bf.at(sl, en.id[u]) = (Bits<E>)Vec<E>::NEG;
            }
            __syncthreads();
            Summer<E, false, false> rest;
            rest.c = p.c;
            Run run = rest.template run<false>(bf, sl);
            KdPart w;
            w.m = warp_max(run.m);
            to_max(run, w.m, p.c);
            w.s = warp_sum(run.s);
            if (!started) row_wait(C);
            started = true;
            if (lane < C) {
                const uint32_t to = remote(&parts[par][rank * SC_WARPS + tid / 32], lane);
                remote_st(to, __float_as_uint(w.m));
                remote_st(to + 4, __float_as_uint(w.s));
            }
            row_arrive(C);
            row_wait(C);
            if (tid < 32) {
                const KdRow row = join(parts[par], es, p.c, C);
                if (lane == 0) s_row = row;
            }
            __syncthreads();
            const KdRow row = s_row;
            if (finite_row(row.m)) {
                const float gl = (p.g_loss ? p.g_loss[r] : 1.f) * p.inv_temp, ps = (te.in + te.left) * row.inv_z;
                const float pr = gl * (ps * row.scale - te.left * row.inv_sr);
                const uint64_t pr2 = pair(pr, pr);
                E* g = grad_of<E>(p, r);
                grad_slice(bf, sl, next, g, row.mr, p.c, 0, [&](uint64_t, uint64_t e2) { return mul2(e2, pr2); });
                __syncthreads();
#pragma unroll
                for (int u = 0; u < SC_EPT; ++u)
                    if (mine[u])
                        g[en.id[u]] = narrow<E>(gl * (ps * ex2_fast(dist(en.l[u], row.m, p.c)) - te.q[u]));
            } else {
                zero_grad<E>(p, r, rank, C);
                bf.copy(next);
            }
            if (rank == 0) finish(p, r, row, te, en.l);
            par ^= 1;
        }
        if (!more) break;
        sl = next;
        r = r2;
        en = en2;
        r2 = r3;
        en2 = en3;
    }
}

template <typename E> cudaError_t go(ScoreParams p, int num_sms, cudaStream_t s)
{
    static ScoreKernel sk[2];
    if (!p.grad) {
        const auto kernel = k_score_distill<E>;
        auto smem = [](size_t per) { return SC_RING_BYTES + (per / Ring<E>::GROUP + 2) * SC_WARPS * 4; };
        cudaError_t e = score_ready(kernel, sk[0], smem(SCORE_MAX_ROW_BYTES / 16 + 2));
        if (e == cudaSuccess) e = score_split_forward(kernel, sk[0], p, sizeof(E), 40, smem);
        return e == cudaSuccess ? score_launch(kernel, sk[0], p, smem(p.per), false, s) : e;
    }
    const cudaError_t e = score_ready(k_score_distill_grad<E>, sk[1], SC_MOST_SLICE);
    if (e != cudaSuccess) return e;
    score_split_gradient(p, sizeof(E), num_sms);
    return score_launch(k_score_distill_grad<E>, sk[1], p, (size_t)p.per * 16, true, s);
}

}  // namespace

cudaError_t launch_score_distill(const ScoreParams& p, int dtype, int num_sms, cudaStream_t s)
{
    return dtype == SPEC_F32 ? go<float>(p, num_sms, s)
           : dtype == SPEC_BF16 ? go<__nv_bfloat16>(p, num_sms, s)
                                : go<__half>(p, num_sms, s);
}

}  // namespace sv
