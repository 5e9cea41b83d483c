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
//
// Entries leave the ring before their thread reads it (a chain per thread), so the
// pass is the plain one.  Measured with L2 flushed: 2048 x 152064 bf16 with 64
// entries 105 us (six CTAs an SM, 0.71 of a copy; five took 112), gradients of
// 777 x 128256 fp32 with 128 entries 167 us and of 1500 x 100003 fp16 122 us (0.7).
#include "sv_score_row.cuh"

namespace sv {

namespace {

constexpr int EPT = (SPEC_SCORE_MAX_ENTRIES + SC_NT - 1) / SC_NT;  // entries of a thread: tid, tid + SC_NT

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
    int id[EPT];
    float tv[EPT], l[EPT];
    __device__ __forceinline__ void fetch(const ScoreParams& p, int r)
    {
#pragma unroll
        for (int u = 0; u < EPT; ++u) {
            const int i = threadIdx.x + u * SC_NT;
            const bool in = r < p.rows && i < p.k;
            id[u] = in ? p.ids[(int64_t)r * p.k + i] : -1;
            tv[u] = in ? teacher_value(p, (int64_t)r * p.k + i) : -INFINITY;
        }
    }
    template <typename E> __device__ __forceinline__ void fetch_logits(const E* x, int V)
    {
#pragma unroll
        for (int u = 0; u < EPT; ++u) l[u] = id[u] >= 0 && id[u] < V ? widen(x[id[u]]) : -INFINITY;
    }
    __device__ __forceinline__ bool some() const
    {
        bool s = false;
#pragma unroll
        for (int u = 0; u < EPT; ++u) s |= id[u] != -1;
        return s;
    }
};

// the teacher's distribution over a row's entries, this thread's
struct Teacher {
    float q[EPT], lq[EPT];  // lq: ln q
    float in, left;               // sum of q, what it leaves of 1
};

// What the threads of a CTA tell one another of a row's entries.  The entries of a slice are chained by the thread whose
// vectors they lie in (head, next), with their place there: copy group (the row's ends being group full + 1) and element
// of the group.
constexpr int SC_SEEN = 16384;  // places of ids
struct EntryShared {
    int32_t ids[EPT * SC_NT];
    int16_t next[EPT * SC_NT];
    uint16_t place[EPT * SC_NT];  // a slice has fewer than 256 groups
    int32_t head[SC_NT];
    uint32_t seen[SC_SEEN / 32];
    uint32_t state;                          // 1: a bad id; 2: two ids with one place in `seen`
    float w_max[SC_NT / 32], w_sum[SC_NT / 32];
    float w_me[SC_NT / 32], w_se[SC_NT / 32];  // the student's largest logit at a warp's entries, and the sum of their 2^d
};
__device__ __forceinline__ void clear(EntryShared& es)
{
    es.head[threadIdx.x] = -1;
    for (int i = threadIdx.x; i < SC_SEEN / 32; i += SC_NT) es.seen[i] = 0;
    if (threadIdx.x == 0) es.state = 0;
}

// Enters a row's entries (es is clear, and a barrier has passed): ids out of range and, maybe, ids that are there twice
// go to `state`; the warps' largest teacher values to w_max.
template <typename E>
__device__ __forceinline__ void enter(const ScoreParams& p, EntryShared& es, Entries& en, const Slice<E>& sl, int full)
{
    const int tid = threadIdx.x;
    float tmax = -INFINITY;
#pragma unroll
    for (int u = 0; u < EPT; ++u) {
        const int e = tid + u * SC_NT, id = en.id[u];
        es.ids[e] = id;
        if (id == -1) {
            en.tv[u] = -INFINITY;
            continue;
        }
        tmax = fmax_nan(tmax, en.tv[u]);
        if (id < 0 || id >= p.V) {
            atomicOr(&es.state, 1u);
            continue;
        }
        const uint32_t at = (uint32_t)(id ^ id >> 14) % SC_SEEN, bit = 1u << (at % 32);
        if (atomicOr(es.seen + at / 32, bit) & bit) atomicOr(&es.state, 2u);
        if (id < sl.first) continue;
        const int i = (id - sl.first) / EPV<E>, q = (id - sl.first) % EPV<E>;
        if (i >= sl.n) continue;
        const bool inner = i >= sl.lo && i < sl.hi;
        const int owner = inner ? i % SC_NT : i < sl.lo ? 0 : 32;
        static_assert(SCORE_MAX_ROW_BYTES / SC_GROUP_BYTES + 3 < 256, "a place's group");
        es.place[e] = inner ? i / (SC_NT * SC_GROUP) << 8 | i / SC_NT % SC_GROUP * EPV<E> + q : (full + 1) << 8 | q;
        es.next[e] = (int16_t)atomicExch(es.head + owner, e);
    }
    tmax = warp_max(tmax);
    if (tid % 32 == 0) es.w_max[tid / 32] = tmax;
}
// after a barrier: whether the row is bad, for all CTAs of a cluster alike
__device__ __forceinline__ bool bad_entries(const EntryShared& es, const Entries& en)
{
    if (es.state & 1) return true;
    if (!(es.state & 2)) return false;
    bool twice = false;
#pragma unroll
    for (int u = 0; u < EPT; ++u) {
        const int e = threadIdx.x + u * SC_NT, id = en.id[u];
        if (id == -1) continue;
        for (int j = 0; j < e; j += 4) {
            const int4 o = *(const int4*)(es.ids + j);
            twice |= o.x == id || (o.y == id && j + 1 < e) || (o.z == id && j + 2 < e) || (o.w == id && j + 3 < e);
        }
    }
    return __syncthreads_or(twice);
}
// The entries of a thread's vectors leave them, group by group.  (Which of two comes first in the chain is a matter of
// chance, but both leave.)
template <typename E> struct Leaving {
    const EntryShared& es;
    int group;  // the next with an entry
    __device__ __forceinline__ explicit Leaving(const EntryShared& s) : es(s) { after(-1); }
    __device__ __forceinline__ void after(int b)
    {
        group = INT32_MAX;
        for (int e = es.head[threadIdx.x]; e >= 0; e = es.next[e])
            if (es.place[e] >> 8 > b) group = min(group, es.place[e] >> 8);
    }
    template <int STEP> __device__ __forceinline__ void from(int b, uint4* v)
    {
        if (b != group) return;
        for (int e = es.head[threadIdx.x]; e >= 0; e = es.next[e]) {
            const int at = es.place[e];
            if (at >> 8 != b) continue;
            // element q of vector j, by words, as the vector is read
            const int j = (at & 255) / EPV<E>, q = (at & 255) % EPV<E>;
            uint32_t* const w = (uint32_t*)(v + j * STEP) + q * (int)sizeof(E) / 4;
            *w = sizeof(E) == 4 ? Vec<E>::NEG : q % 2 ? (*w & 0xFFFFu) | (Vec<E>::NEG & 0xFFFF0000u)
                                                       : (*w & 0xFFFF0000u) | (Vec<E>::NEG & 0xFFFFu);
        }
        after(b);
    }
};
__device__ __forceinline__ bool dull(const ScoreParams& p, float tmax, float lse)
{
    return !(tmax < INFINITY) || (!p.tail && tmax == -INFINITY) || !(fabsf(lse) < INFINITY);
}
// q up to the row's sum: differences first, and 1 / t in two parts, as the values may be large
__device__ __forceinline__ void begin_teacher(const ScoreParams& p, EntryShared& es, const Entries& en, float tmax,
                                              float lse, Teacher& te)
{
    float sum = 0.f;
#pragma unroll
    for (int u = 0; u < EPT; ++u) {
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
    for (int i = 0; i < SC_NT / 32; ++i) sum += es.w_sum[i];
    te.in = p.tail ? sum : 1.f;
    te.left = p.tail ? fmaxf(0.f, 1.f - sum) : 0.f;
    if (!p.tail) {
        const float ln = logf(sum), inv = 1.f / sum;
#pragma unroll
        for (int u = 0; u < EPT; ++u) {
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
    for (int u = 0; u < EPT; ++u) me = fmax_nan(me, en.l[u]);
    me = warp_max(me);
#pragma unroll
    for (int u = 0; u < EPT; ++u) se += ex2_fast(dist(en.l[u], me, p.c));
    se = warp_sum(se);
    if (threadIdx.x % 32 == 0) {
        es.w_me[threadIdx.x / 32] = me;
        es.w_se[threadIdx.x / 32] = se;
    }
}
// one warp: the row of the parts of n warps and of its entries
__device__ __forceinline__ KdRow join(const KdPart* parts, const EntryShared& es, float c, int n)
{
    KdRow row = {-INFINITY, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int i = threadIdx.x % 32; i < n; i += 32) row.mr = fmax_nan(row.mr, parts[i].m);
    row.mr = warp_max(row.mr);
    row.m = row.mr;
#pragma unroll
    for (int i = 0; i < SC_NT / 32; ++i) row.m = fmax_nan(row.m, es.w_me[i]);
    for (int i = threadIdx.x % 32; i < n; i += 32)
        if (parts[i].m > -INFINITY) row.sr += parts[i].s * ex2_fast(between(parts[i].m, row.mr, c));
    row.sr = warp_sum(row.sr);
    row.scale = row.mr == -INFINITY ? 0.f : ex2_fast(between(row.mr, row.m, c));
    row.z = row.sr * row.scale;
#pragma unroll
    for (int i = 0; i < SC_NT / 32; ++i)
        if (es.w_me[i] > -INFINITY) row.z += es.w_se[i] * ex2_fast(between(es.w_me[i], row.m, c));
    row.inv_z = 1.f / row.z;
    row.inv_sr = row.sr > 0.f ? 1.f / row.sr : 0.f;
    return row;
}

// h(q, p); for a p too small for a quotient, ln(q / p) = a - b inv_temp, b the distance of a logit, which its product
// with 1 / t may take out of range where that with q too is in it
__device__ __forceinline__ float divergence(float q, float p, float a, float b, float inv_temp)
{
    if (q == 0.f) return p;
    if (!(p > 1e-30f)) return q * a - q * b * inv_temp - q + p;
    const float d = (q - p) / p;
    return fabsf(d) < 0.5f ? p * ((1.f + d) * log1pf(d) - d) : q * logf(q / p) - q + p;
}

// CTA 0: a row's loss and acceptance
__device__ __forceinline__ void finish(const ScoreParams& p, int r, const KdRow& row, const Teacher& te,
                                       const float (&l)[EPT])
{
    __shared__ float w_h[SC_NT / 32], w_acc[SC_NT / 32];
    const int tid = threadIdx.x, lane = tid % 32;
    const float ln_z = logf(row.z) - dist(row.m, row.m, p.c) * LN2;  // relative to m
    float h = 0.f, acc = 0.f;
#pragma unroll
    for (int u = 0; u < EPT; ++u) {
        const float pi = ex2_fast(dist(l[u], row.m, p.c)) * row.inv_z;
        h += divergence(te.q[u], pi, te.lq[u] + ln_z, l[u] - row.m, p.inv_temp);
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
        for (int i = 0; i < SC_NT / 32; ++i) {
            h += w_h[i];
            acc += w_acc[i];
        }
        const float pr = row.sr * row.scale * row.inv_z;
        if (p.tail) {
            // ln of the rest's share, from the logarithms of both sums and the distance of their references
            const float ln_r = row.sr > 0.f ? logf(row.sr) - dist(row.mr, row.mr, p.c) * LN2 : 0.f;
            h += divergence(te.left, pr, logf(te.left) - ln_r + ln_z, row.sr > 0.f ? row.mr - row.m : -INFINITY,
                            p.inv_temp) + fmaxf(0.f, te.in - 1.f);
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

template <typename E, bool GRAD> __device__ __forceinline__ void distill_row(const ScoreParams& p)
{
    constexpr int W = SC_NT / 32;
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ __align__(16) EntryShared es;
    __shared__ KdPart parts[SC_MAXC * W];
    __shared__ KdRow s_row;
    const int C = p.cluster, rank = (int)cluster_rank(), r = cluster_id(), tid = threadIdx.x, lane = tid % 32;
    Entries en;
    en.fetch(p, r);
    const float lse = p.teacher_lse ? p.teacher_lse[r] : 0.f, g_loss = GRAD && p.g_loss ? p.g_loss[r] : 1.f;
    clear(es);
    if (!__syncthreads_or(en.some())) {
        no_distill<E>(p, r, SPEC_ROW_OK, rank, C);
        return;
    }
    const E* x = row_of<E>(p, r);
    const Slice<E> sl(p, x, rank);
    Ring<E, GRAD ? SC_RING_GRAD : SC_RING> ring(p, sl, rank, smem);
    en.fetch_logits(x, p.V);
    const uint4 edge = ring.edge();
    enter(p, es, en, sl, ring.full);
    __syncthreads();
    const bool bad = bad_entries(es, en);
    float tmax = -INFINITY;
#pragma unroll
    for (int i = 0; i < W; ++i) tmax = fmax_nan(tmax, es.w_max[i]);
    if (bad || dull(p, tmax, lse)) {
        copy_done();
        no_distill<E>(p, r, bad ? SPEC_ROW_BAD_TOKEN : SPEC_ROW_NONFINITE, rank, C);
        return;
    }
    // every CTA of the cluster runs before another stores into its shared memory
    if (C > 1) cluster_begin();
    Teacher te;
    begin_teacher(p, es, en, tmax, lse, te);
    Leaving<E> leaving(es);
    Summer<E, false, false> rest;
    rest.c = p.c;
    rest.stream(
        ring, edge,
        [&](int b, uint4* v) {
            if (b <= ring.full) leaving.template from<SC_NT>(b, v);
            else leaving.template from<1>(b, v);
        },
        [](int, float) {});
    Run run = rest.result();
    if (GRAD || rank == 0) sum_entries(p, es, en);  // (their logits have come by now)
    KdPart w;
    w.m = warp_max(run.m);
    to_max(run, w.m, p.c);
    w.s = warp_sum(run.s);
    if (C > 1) cluster_wait();
    if (lane < (GRAD ? C : 1)) {
        const uint32_t to = remote(parts + rank * W + tid / 32, lane);
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
            const float gl = g_loss * p.inv_temp, ps = (te.in + te.left) * row.inv_z;
            const float pr = gl * (ps * row.scale - te.left * row.inv_sr);
            const uint64_t pr2 = pair(pr, pr);
            E* g = grad_of<E>(p, r);
            grad_slice(ring, edge, g, row.mr, p.c, 0, [&](uint64_t, uint64_t e2) { return mul2(e2, pr2); });
            __syncthreads();  // the entries' elements are written last
#pragma unroll
            for (int u = 0; u < EPT; ++u)
                if (en.id[u] >= 0 && ring.has(en.id[u]))
                    g[en.id[u]] = narrow<E>(gl * (ps * ex2_fast(dist(en.l[u], row.m, p.c)) - te.q[u]));
        } else {
            copy_done();
            zero_grad<E>(p, r, rank, C);
        }
        if (rank != 0) return;
    }
    finish(p, r, row, te, en.l);
}

template <typename E> __global__ void __launch_bounds__(SC_NT, 6) k_score_distill(const ScoreParams p)
{
    distill_row<E, false>(p);
}
template <typename E> __global__ void __launch_bounds__(SC_NT, 4) k_score_distill_grad(const ScoreParams p)
{
    distill_row<E, true>(p);
}

template <typename E> cudaError_t go(ScoreParams p, int num_sms, cudaStream_t s)
{
    static ScoreKernel sk[2];
    if (!p.grad) {
        const auto kernel = k_score_distill<E>;
        constexpr size_t smem = SC_RING * SC_GROUP_BYTES;
        cudaError_t e = score_ready(kernel, sk[0], smem, smem);
        if (e == cudaSuccess) e = score_split_forward(sk[0], p, sizeof(E), num_sms, 32, [](size_t) { return smem; });
        return e == cudaSuccess ? score_launch(kernel, p, smem, s) : e;
    }
    const cudaError_t e = score_ready(k_score_distill_grad<E>, sk[1], SC_GRAD_BYTES, SC_GRAD_BYTES);
    if (e != cudaSuccess) return e;
    score_split_gradient(p, sizeof(E), num_sms);
    return score_launch(k_score_distill_grad<E>, p, SC_GRAD_BYTES, s);
}

}  // namespace

cudaError_t launch_score_distill(const ScoreParams& p, int dtype, int num_sms, cudaStream_t s)
{
    return dtype == SPEC_F32 ? go<float>(p, num_sms, s)
           : dtype == SPEC_BF16 ? go<__nv_bfloat16>(p, num_sms, s)
                                : go<__half>(p, num_sms, s);
}

}  // namespace sv
