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

template <int NT> constexpr int EPT = SPEC_SCORE_MAX_ENTRIES / NT;  // entries of a thread: tid, tid + NT

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

template <typename E, int NT> __device__ void no_distill(const ScoreParams& p, int r, int status, int rank, int C)
{
    if (rank == 0 && threadIdx.x == 0) {
        const float none = status == SPEC_ROW_OK ? 0.f : __int_as_float(0x7FFFFFFF);
        p.row_status[r] = status;
        if (p.loss) p.loss[r] = none;
        if (p.accept) p.accept[r] = none;
    }
    if (p.grad) zero_grad<E, NT>(p, r, rank, C);
}

// a row's entries, this thread's: token, teacher's value, the student's logit
template <int NT> struct Entries {
    int id[EPT<NT>];
    float tv[EPT<NT>], l[EPT<NT>];
    __device__ __forceinline__ void fetch(const ScoreParams& p, int r)
    {
#pragma unroll
        for (int u = 0; u < EPT<NT>; ++u) {
            const int i = threadIdx.x + u * NT;
            const bool in = r < p.rows && i < p.k;
            id[u] = in ? p.ids[(int64_t)r * p.k + i] : -1;
            tv[u] = in ? teacher_value(p, (int64_t)r * p.k + i) : -INFINITY;
        }
    }
    template <typename E> __device__ __forceinline__ void fetch_logits(const E* x, int V)
    {
#pragma unroll
        for (int u = 0; u < EPT<NT>; ++u) l[u] = id[u] >= 0 && id[u] < V ? widen(x[id[u]]) : -INFINITY;
    }
    __device__ __forceinline__ bool some() const
    {
        bool s = false;
#pragma unroll
        for (int u = 0; u < EPT<NT>; ++u) s |= id[u] != -1;
        return s;
    }
};

// the teacher's distribution over a row's entries, this thread's
template <int NT> struct Teacher {
    float q[EPT<NT>], lq[EPT<NT>];  // lq: ln q
    float in, left;               // sum of q, what it leaves of 1
};

// what the threads of a CTA tell one another of a row's entries; the next row has another, as some are still at the
// last row's end when others begin it
template <int NT> struct EntryShared {
    int32_t ids[SPEC_SCORE_MAX_ENTRIES];
    int32_t slots[SPEC_SCORE_MAX_ENTRIES];
    float w_max[NT / 32], w_sum[NT / 32];
    float w_me[NT / 32], w_se[NT / 32];  // the student's largest logit at a warp's entries, and the sum of their 2^d
};

// Checks a row's entries (a barrier, then the checks; the caller passes bad to the next one) and starts the teacher's
// sums.  slots: see below; mark(u): called between the barriers.
template <int NT, typename Mark>
__device__ __forceinline__ bool check_entries(const ScoreParams& p, EntryShared<NT>& es, Entries<NT>& en, const int (&slot)[EPT<NT>],
                                              bool (&first)[EPT<NT>], float& tmax, Mark mark)
{
    const int tid = threadIdx.x, lane = tid % 32;
    tmax = -INFINITY;
#pragma unroll
    for (int u = 0; u < EPT<NT>; ++u) {
        es.ids[tid + u * NT] = en.id[u];
        es.slots[tid + u * NT] = slot[u];
        if (en.id[u] == -1) en.tv[u] = -INFINITY;
        tmax = fmax_nan(tmax, en.tv[u]);
    }
    tmax = warp_max(tmax);
    if (lane == 0) es.w_max[tid / 32] = tmax;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NT / 32; ++i) tmax = fmax_nan(tmax, es.w_max[i]);
    bool bad = false;
#pragma unroll
    for (int u = 0; u < EPT<NT>; ++u) {
        const int i = tid + u * NT, id = en.id[u];
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
template <int NT>
__device__ __forceinline__ void begin_teacher(const ScoreParams& p, EntryShared<NT>& es, const Entries<NT>& en, float tmax,
                                              float lse, Teacher<NT>& te)
{
    float sum = 0.f;
#pragma unroll
    for (int u = 0; u < EPT<NT>; ++u) {
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
template <int NT>
__device__ __forceinline__ void end_teacher(const ScoreParams& p, const EntryShared<NT>& es, Teacher<NT>& te)
{
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < NT / 32; ++i) sum += es.w_sum[i];
    te.in = p.tail ? sum : 1.f;
    te.left = p.tail ? fmaxf(0.f, 1.f - sum) : 0.f;
    if (!p.tail) {
        const float ln = logf(sum), inv = 1.f / sum;
#pragma unroll
        for (int u = 0; u < EPT<NT>; ++u) {
            te.q[u] *= inv;
            te.lq[u] -= ln;
        }
    }
}
// the entries' sums of a warp
template <int NT>
__device__ __forceinline__ void sum_entries(const ScoreParams& p, EntryShared<NT>& es, const Entries<NT>& en)
{
    float me = -INFINITY, se = 0.f;
#pragma unroll
    for (int u = 0; u < EPT<NT>; ++u) me = fmax_nan(me, en.l[u]);
    me = warp_max(me);
#pragma unroll
    for (int u = 0; u < EPT<NT>; ++u) se += ex2_fast(dist(en.l[u], me, p.c));
    se = warp_sum(se);
    if (threadIdx.x % 32 == 0) {
        es.w_me[threadIdx.x / 32] = me;
        es.w_se[threadIdx.x / 32] = se;
    }
}
// one warp: the row of the parts of n warps and of its entries
template <int NT>
__device__ __forceinline__ KdRow join(const KdPart* parts, const EntryShared<NT>& es, float c, int n)
{
    KdRow row = {-INFINITY, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int i = threadIdx.x % 32; i < n; i += 32) row.mr = fmax_nan(row.mr, parts[i].m);
    row.mr = warp_max(row.mr);
    row.m = row.mr;
#pragma unroll
    for (int i = 0; i < NT / 32; ++i) row.m = fmax_nan(row.m, es.w_me[i]);
    for (int i = threadIdx.x % 32; i < n; i += 32)
        if (parts[i].m > -INFINITY) row.sr += parts[i].s * ex2_fast(between(parts[i].m, row.mr, c));
    row.sr = warp_sum(row.sr);
    row.scale = row.mr == -INFINITY ? 0.f : ex2_fast(between(row.mr, row.m, c));
    row.z = row.sr * row.scale;
#pragma unroll
    for (int i = 0; i < NT / 32; ++i)
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
template <int NT>
__device__ __forceinline__ void finish(const ScoreParams& p, int r, const KdRow& row, const Teacher<NT>& te,
                                       const float (&l)[EPT<NT>])
{
    __shared__ float w_h[NT / 32], w_acc[NT / 32];
    const int tid = threadIdx.x, lane = tid % 32;
    const float ln_z = logf(row.z) - dist(row.m, row.m, p.c) * LN2;  // relative to m
    float h = 0.f, acc = 0.f;
#pragma unroll
    for (int u = 0; u < EPT<NT>; ++u) {
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
        for (int i = 0; i < NT / 32; ++i) {
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

// ---- both passes' first part -------------------------------------------------------- //
// A thread leaves out the copy groups of its vectors in which an entry lies (flags: a bit for each group and thread, the
// row's ends being group full + 1).  Those are read once more, each by the thread of the first entry in it (slots: group
// and thread), which takes the entries out.
template <typename E, int NT>
__device__ __forceinline__ void slots_of(const Slice<E>& sl, int V, int full, const Entries<NT>& en, int (&slot)[EPT<NT>])
{
#pragma unroll
    for (int u = 0; u < EPT<NT>; ++u) {
        slot[u] = -1;
        if (en.id[u] < sl.first || en.id[u] >= V || en.id[u] < 0) continue;
        const int i = (en.id[u] - sl.first) / EPV<E>;
        if (i >= sl.n) continue;
        slot[u] = i >= sl.lo && i < sl.hi ? i / (NT * SC_GROUP) * NT + i % NT : (full + 1) * NT + (i < sl.lo ? 0 : 32);
    }
}
template <typename E, int NT, typename S>
__device__ __forceinline__ void take_left_out(const ScoreParams& p, const Slice<E>& sl, int full, const EntryShared<NT>& es,
                                              const int (&slot)[EPT<NT>], const bool (&first)[EPT<NT>], S& rest)
{
#pragma unroll
    for (int u = 0; u < EPT<NT>; ++u) {
        if (!first[u]) continue;
        const int g = slot[u] / NT, owner = slot[u] % NT;
        const bool end = g > full;
        uint4 w[SC_GROUP];
        int at[SC_GROUP];
#pragma unroll
        for (int j = 0; j < SC_GROUP; ++j) {
            at[j] = end ? (owner == 0 ? 0 : sl.n - 1) : (g * SC_GROUP + j) * NT + owner;
            w[j] = end ? (j ? no_vector<E>() : load_vector(sl, p.V, at[j]))
                       : at[j] >= sl.lo && at[j] < sl.hi ? load_vector(sl, p.V, at[j]) : no_vector<E>();
        }
        uint32_t out = 0;  // the entries' elements
        for (int j = 0; j < p.k; j += 4) {
            const int4 o = *(const int4*)(es.slots + j);
            auto one = [&](int s, int j) {
                if (s != slot[u]) return;
                const int e = es.ids[j] - sl.first;
                out |= 1u << ((end ? 0 : (e / EPV<E> - at[0]) / NT) * EPV<E> + e % EPV<E>);
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
        rest.template take<NT>(w, 0, 0);
    }
}

template <typename E, int NT, bool GRAD> __device__ __forceinline__ void distill_row(const ScoreParams& p)
{
    constexpr int W = NT / 32;
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ __align__(16) EntryShared<NT> es;
    __shared__ KdPart parts[SC_MAXC * W];
    __shared__ KdRow s_row;
    const int C = p.cluster, rank = (int)cluster_rank(), r = cluster_id(), tid = threadIdx.x, lane = tid % 32;
    const int warp = tid / 32;
    Entries<NT> en;
    en.fetch(p, r);
    if (!__syncthreads_or(en.some())) {
        no_distill<E, NT>(p, r, SPEC_ROW_OK, rank, C);
        return;
    }
    const E* x = row_of<E>(p, r);
    const Slice<E> sl(p, x, rank);
    Ring<E, NT, GRAD> ring(p, sl, rank, smem);
    en.fetch_logits(x, p.V);
    const uint4 edge = ring.edge();
    const float lse = p.teacher_lse ? p.teacher_lse[r] : 0.f;
    uint32_t* const flags = (uint32_t*)(smem + RING_BYTES<NT>);
    for (int i = tid; i < (ring.full + 2) * W; i += NT) flags[i] = 0;
    int slot[EPT<NT>];
    slots_of(sl, p.V, ring.full, en, slot);
    float tmax;
    bool first[EPT<NT>];
    bool bad = check_entries(p, es, en, slot, first, tmax, [&](int u) {
        if (slot[u] >= 0) atomicOr(flags + slot[u] / 32, 1u << (slot[u] % 32));
    });
    Teacher<NT> te;
    begin_teacher(p, es, en, tmax, lse, te);
    bad = __syncthreads_or(bad);
    if (bad || dull(p, tmax, lse)) {
        copy_done();
        no_distill<E, NT>(p, r, bad ? SPEC_ROW_BAD_TOKEN : SPEC_ROW_NONFINITE, rank, C);
        return;
    }
    // every CTA of the cluster runs before another stores into its shared memory
    if (C > 1) cluster_arrive();
    Summer<E, false, false> rest;
    rest.c = p.c;
    rest.stream(ring, edge, [&](int b) { return flags[b * W + warp] >> lane & 1; }, [](int, float) {});
    take_left_out(p, sl, ring.full, es, slot, first, rest);
    Run run = rest.result();
    KdPart w;
    w.m = warp_max(run.m);
    to_max(run, w.m, p.c);
    w.s = warp_sum(run.s);
    if (GRAD || rank == 0) sum_entries(p, es, en);
    if (C > 1) cluster_wait();
    if (lane < (GRAD ? C : 1)) {
        const uint32_t to = remote(parts + rank * W + warp, lane);
        remote_st(to, __float_as_uint(w.m));
        remote_st(to + 4, __float_as_uint(w.s));
    }
    row_arrive(C);
    if (!GRAD && rank != 0) return;
    if (C > 1) {
        row_wait(C);
        __syncthreads();
    }
    if (tid < 32) {
        const KdRow row = join(parts, es, p.c, C * W);
        if (lane == 0) s_row = row;
    }
    end_teacher(p, es, te);
    __syncthreads();
    const KdRow row = s_row;
    if (GRAD) {
        if (finite_row(row.m)) {
            const float gl = (p.g_loss ? p.g_loss[r] : 1.f) * p.inv_temp, ps = (te.in + te.left) * row.inv_z;
            const float pr = gl * (ps * row.scale - te.left * row.inv_sr);
            const uint64_t pr2 = pair(pr, pr);
            E* g = grad_of<E>(p, r);
            grad_slice(ring, edge, g, row.mr, p.c, 0, [&](uint64_t, uint64_t e2) { return mul2(e2, pr2); });
            __syncthreads();  // the entries' elements are written last
#pragma unroll
            for (int u = 0; u < EPT<NT>; ++u)
                if (en.id[u] >= 0 && ring.has(en.id[u]))
                    g[en.id[u]] = narrow<E>(gl * (ps * ex2_fast(dist(en.l[u], row.m, p.c)) - te.q[u]));
        } else {
            copy_done();
            zero_grad<E, NT>(p, r, rank, C);
        }
        if (rank != 0) return;
    }
    finish(p, r, row, te, en.l);
}

template <typename E> __global__ void __launch_bounds__(SC_NT, 5) k_score_distill(const ScoreParams p)
{
    distill_row<E, SC_NT, false>(p);
}
template <typename E> __global__ void __launch_bounds__(SC_NT_GRAD, 2) k_score_distill_grad(const ScoreParams p)
{
    distill_row<E, SC_NT_GRAD, true>(p);
}

template <typename E> cudaError_t go(ScoreParams p, int num_sms, cudaStream_t s)
{
    static ScoreKernel sk[2];
    if (!p.grad) {
        const auto kernel = k_score_distill<E>;
        auto smem = [](size_t per) { return RING_BYTES<SC_NT> + (per / (SC_NT * SC_GROUP) + 2) * (SC_NT / 32) * 4; };
        cudaError_t e = score_ready(kernel, sk[0], smem(SCORE_MAX_ROW_BYTES / 16 + 2));
        if (e == cudaSuccess) e = score_split_forward(kernel, sk[0], p, sizeof(E), 40, smem);
        return e == cudaSuccess ? score_launch(kernel, p, SC_NT, smem(p.per), s) : e;
    }
    static_assert(RING_BYTES<SC_NT_GRAD> + (SCORE_MAX_ROW_BYTES / 16 / (SC_NT_GRAD * SC_GROUP) + 3) * (SC_NT_GRAD / 32) * 4 <=
                  SC_GRAD_BYTES, "flags of the largest row");
    const cudaError_t e = score_ready(k_score_distill_grad<E>, sk[1], SC_GRAD_BYTES);
    if (e != cudaSuccess) return e;
    score_split_gradient(p, sizeof(E), num_sms);
    return score_launch(k_score_distill_grad<E>, p, SC_NT_GRAD, SC_GRAD_BYTES, s);
}

}  // namespace

cudaError_t launch_score_distill(const ScoreParams& p, int dtype, int num_sms, cudaStream_t s)
{
    return dtype == SPEC_F32 ? go<float>(p, num_sms, s)
           : dtype == SPEC_BF16 ? go<__nv_bfloat16>(p, num_sms, s)
                                : go<__half>(p, num_sms, s);
}

}  // namespace sv
