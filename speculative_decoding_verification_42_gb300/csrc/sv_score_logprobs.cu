// sv_score_logprobs.cu -- log probabilities of given tokens with rank, entropy
// and top alternatives, and the gradient of log probability and entropy.
//
// ln p_x = (x - m) / t - ln s and H = ln s - ln 2 (sum d 2^d) / s, relative to 2^B,
// from one pass; the gradient p_v (A + B d_v) needs both and takes a second.
// Measured with L2 flushed: 608 x 131072 bf16 30 us (5.3 TB/s; a pass is 5.9
// instructions an element, issue 59 % where rows are short), fp32 53 us (6 TB/s);
// top 64 of 2000 x 152064 bf16 147 us; both gradients of 2000 x 128256 bf16
// 198 us (HBM, which moves a fifth more than it must as L2 loses some of the
// rows under way).
#include "sv_score_row.cuh"

namespace sv {

namespace {

constexpr int SC_LIST = 1024;   // candidates for the top tokens, all CTAs of a row together
constexpr uint32_t KEY_NEG_INF = 0x007FFFFFu;  // key_of(-inf)

struct LpPart {      // what a warp knows of the row
    float m, s, t;
    int32_t ahead;
};
struct LpRow {
    float m, s, t;
    int32_t ahead;
    uint32_t bound;  // a key that the top tokens reach, and not many others
};

// The search for the top tokens.  A bound first: the row's CTAs exchange 512 largest keys, of groups of a thread's
// vectors, and take one that at least n of them reach and not many more, by halving the range of keys.  With n of g
// groups above it, a bound has g ln(g / (g - n)) tokens above it when they lie at random (n = 128: 147).  Then the copy
// groups whose largest element reaches the bound are read once more, and what reaches it in them are the candidates,
// which CTA 0 puts in order.  All of it takes some 7 us behind the row's last element (bound 1.4, candidates 1 to 3, order
// and barriers the rest); other rows' CTAs stream meanwhile, five on an SM (top 20 of 152 x 128256 fp32: 33 us, with
// four 41).
constexpr int SC_GROUPS = 512;
constexpr int SC_AGAIN = 512;       // copy groups of a CTA that are read again
// It is where the ring was: used when every CTA of the row is through with its slice.  Behind the ring are the keys that
// the CTAs exchange, which may come earlier, and Bits<E> [full + 1][SC_NT]: the largest element of each thread's copy
// groups.
struct TopScratch {
    unsigned long long list[SC_LIST];  // CTA 0: candidates, key and inverted id, SC_LIST / C to a CTA
    uint32_t again[SC_AGAIN];          // copy group * SC_NT + thread
    int32_t counts[SC_MAXC];           // CTA 0: candidates of each CTA
    int32_t mine, agains;              // candidates of this CTA, entries of `again`
    int32_t tally[2][(SC_NT / 32)];
};
static_assert(sizeof(TopScratch) <= SC_RING * SC_GROUP_BYTES, "where the ring was");

__device__ __forceinline__ int tally_of(TopScratch& ts, int round, int x)
{
    // one barrier a round: the other buffer is free again when it is passed
    x = __reduce_add_sync(~0u, x);
    if (threadIdx.x % 32 == 0) ts.tally[round & 1][threadIdx.x / 32] = x;
    __syncthreads();
    int n = 0;
#pragma unroll
    for (int i = 0; i < (SC_NT / 32); ++i) n += ts.tally[round & 1][i];
    return n;
}

template <typename E, typename F> __device__ __forceinline__ void each_of(const uint4& w, int e, F f)
{
#pragma unroll
    for (int q = 0; q < EPV<E>; ++q) f(key_of(value_of<E>(bits_at<E>(w, q))), e + q);
}

// The candidates of a CTA, whose keys reach `bound`, into the list of CTA 0.  When they are too many for its share of
// the list (equal logits), its first n in the order (key desc, id asc), found by halving the range of keys and of ids
// and counting.
template <typename E>
__device__ void give_candidates(const Slice<E>& sl, int V, int full, TopScratch& ts, const Bits<E>* most, uint32_t bound,
                                int n, int rank, int C)
{
    const int share = SC_LIST / C, tid = threadIdx.x;
    const uint32_t list = remote(ts.list + rank * share, 0);
    auto give = [&](uint32_t key, int id) {
        const int at = atomicAdd(&ts.mine, 1);
        if (at < share) {
            remote_st(list + at * 8, ~(uint32_t)id);
            remote_st(list + at * 8 + 4, key);
        }
    };
    const float least = val_of(bound);
    for (int b = 0; b <= full; ++b)
        if (value_of<E>(most[b * SC_NT + tid]) >= least) {
            const int at = atomicAdd(&ts.agains, 1);
            if (at < SC_AGAIN) ts.again[at] = b * SC_NT + tid;
        }
    __syncthreads();
    const int agains = ts.agains;
    if (agains <= SC_AGAIN) {
        for (int a = tid; a < agains; a += SC_NT) {
            const int g = ts.again[a] / SC_NT, owner = ts.again[a] % SC_NT;
            uint4 w[SC_GROUP + 1];
            int at[SC_GROUP + 1];
#pragma unroll
            for (int j = 0; j < SC_GROUP; ++j) {
                at[j] = (g * SC_GROUP + j) * SC_NT + owner;
                w[j] = at[j] >= sl.lo && at[j] < sl.hi ? load_vector(sl, V, at[j]) : no_vector<E>();
            }
            // the row's ends count to the last group of threads 0 and 32
            const bool first = owner == 0 && sl.lo && sl.n, last = owner == 32 && sl.hi < sl.n;
            at[SC_GROUP] = first ? 0 : sl.n - 1;
            w[SC_GROUP] = g == full && (first || last) ? load_vector(sl, V, at[SC_GROUP]) : no_vector<E>();
            // first which elements they are, then one of each lane's at a time: lanes have them at different places
            unsigned long long hits = 0;
#pragma unroll
            for (int j = 0; j <= SC_GROUP; ++j)
#pragma unroll
                for (int q = 0; q < EPV<E>; ++q)
                    if (value_of<E>(bits_at<E>(w[j], q)) >= least) hits |= 1ull << (j * EPV<E> + q);
            while (hits) {
                const int h = __ffsll(hits) - 1, j = h / EPV<E>;
                hits &= hits - 1;
                const int e = (j == SC_GROUP ? at[SC_GROUP] : (g * SC_GROUP + j) * SC_NT + owner) * EPV<E> + h % EPV<E>;
                const uint32_t key = key_of(widen(((const E*)sl.src)[e]));
                if (key >= bound) give(key, sl.first + e);
            }
        }
    }
    __syncthreads();
    int found = ts.mine;
    if (found > share || agains > SC_AGAIN) {
        __syncthreads();
        if (tid == 0) ts.mine = 0;
        auto number = [&](int round, auto pred) {
            int k = 0;
            for (int i = tid; i < sl.n; i += SC_NT)
                each_of<E>(load_vector(sl, V, i), sl.first + i * EPV<E>, [&](uint32_t key, int id) { k += pred(key, id); });
            return tally_of(ts, round, k);
        };
        int round = 0;
        const int all = number(round++, [&](uint32_t key, int) { return key >= bound; });
        found = min(n, all);
        uint32_t lo = bound, hi = 0xFF800000u;
        while (lo < hi) {  // the last of them
            const uint32_t mid = lo + (hi - lo + 1) / 2;
            if (number(round++, [&](uint32_t key, int) { return key >= mid; }) >= found) lo = mid;
            else hi = mid - 1;
        }
        const int ties = found - number(round++, [&](uint32_t key, int) { return key > lo; });
        int first = sl.first, last = sl.first + sl.n * EPV<E> - 1;  // the last id among its equals
        while (first < last) {
            const int mid = first + (last - first) / 2;
            if (number(round++, [&](uint32_t key, int id) { return key == lo && id <= mid; }) >= ties) last = mid;
            else first = mid + 1;
        }
        if (found > 0)
            for (int i = tid; i < sl.n; i += SC_NT)
                each_of<E>(load_vector(sl, V, i), sl.first + i * EPV<E>, [&](uint32_t key, int id) {
                    if (key > lo || (key == lo && id <= last)) give(key, id);
                });
    }
    if (tid == 0) remote_st(remote(ts.counts + rank, 0), (uint32_t)found);
}

// the keys of this thread's copy groups, 512 / C from a CTA, to all CTAs
template <typename E>
__device__ __forceinline__ void give_keys(const uint32_t* keys, const Bits<E>* most, int full, int rank, int C)
{
    const int tid = threadIdx.x, parts = C == 1 ? 4 : C == 2 ? 2 : 1, per = (full + parts) / parts;
    int b = 0;
    for (int q = 0; q < parts; ++q) {
        float m = -INFINITY;
        for (const int end = min(full + 1, b + per); b < end; ++b) m = fmaxf(m, value_of<E>(most[b * SC_NT + tid]));
        uint32_t k = key_of(m);
        if (C == 8) {
            k = max(k, __shfl_xor_sync(~0u, k, 1));
            for (int i = tid % 2; i < C; i += 2) remote_st(remote(keys + (rank * SC_NT + tid) / 2, i), k);
        } else {
            for (int i = 0; i < C; ++i) remote_st(remote(keys + (rank * parts + q) * SC_NT + tid, i), k);
        }
    }
}
__device__ __forceinline__ uint32_t bound_of(const uint32_t* keys, int n)
{
    uint32_t mine[SC_GROUPS / 32], lo = ~0u, hi = 0;
    int k = 0;
#pragma unroll
    for (int i = 0; i < SC_GROUPS / 32; ++i) {
        mine[i] = keys[i * 32 + threadIdx.x % 32];
        hi = max(hi, mine[i]);
        if (mine[i] > KEY_NEG_INF) {
            lo = min(lo, mine[i]);
            ++k;
        }
    }
    lo = __reduce_min_sync(~0u, lo);
    // fewer than n groups have an unmasked token at all: every unmasked token is a candidate
    if (__reduce_add_sync(~0u, k) < n) return KEY_NEG_INF + 1;
    hi = __reduce_max_sync(~0u, hi);
    while (lo < hi) {
        const uint32_t mid = lo + (hi - lo + 1) / 2;
        k = 0;
#pragma unroll
        for (int i = 0; i < SC_GROUPS / 32; ++i) k += mine[i] >= mid;
        k = __reduce_add_sync(~0u, k);
        if (k < n) {
            hi = mid - 1;
        } else {
            lo = mid;
            if (k <= n + n / 4 + 4) break;
        }
    }
    return lo;
}

// CTA 0: the candidates in order
__device__ void write_top(const ScoreParams& p, int r, TopScratch& ts, const LpRow& row, float logz, int C)
{
    const int share = SC_LIST / C;
    int before[SC_MAXC + 1];
    before[0] = 0;
#pragma unroll
    for (int i = 0; i < SC_MAXC; ++i) before[i + 1] = before[i] + (i < C ? ts.counts[i] : 0);
    const int all = before[SC_MAXC], n = min(all, p.top_n);
    int32_t* ids = p.top_ids + (int64_t)r * p.top_n;
    float* lps = p.top_lp + (int64_t)r * p.top_n;
    for (int i = threadIdx.x; i < all; i += SC_NT) {
        int part = 0, base = 0;
#pragma unroll
        for (int j = 1; j < SC_MAXC; ++j)
            if (j < C && i >= before[j]) part = j, base = before[j];
        const unsigned long long mine = ts.list[part * share + i - base];
        int at = 0;
        for (int j = 0; j < C; ++j) {
            const unsigned long long* l = ts.list + j * share;
            const int k = ts.counts[j];
            for (int q = 0; q < k; ++q) at += l[q] > mine;
        }
        if (at < n) {
            ids[at] = (int32_t)~(uint32_t)mine;
            lps[at] = (val_of((uint32_t)(mine >> 32)) - row.m) * p.inv_temp - logz;
        }
    }
    for (int i = n + threadIdx.x; i < p.top_n; i += SC_NT) {
        ids[i] = -1;
        lps[i] = -INFINITY;
    }
}

__device__ __forceinline__ void no_top(const ScoreParams& p, int r, int status)
{
    for (int i = threadIdx.x; i < p.top_n; i += SC_NT) {
        p.top_ids[(int64_t)r * p.top_n + i] = -1;
        p.top_lp[(int64_t)r * p.top_n + i] = status == SPEC_ROW_OK ? -INFINITY : __int_as_float(0x7FFFFFFF);
    }
}

// a row that is not scored, or has a bad token
template <typename E> __device__ void no_logprobs(const ScoreParams& p, int r, int status, int rank, int C)
{
    if (rank == 0) {
        const float none = status == SPEC_ROW_OK ? 0.f : __int_as_float(0x7FFFFFFF);
        if (threadIdx.x == 0) {
            p.row_status[r] = status;
            if (p.logprob) p.logprob[r] = none;
            if (p.rank) p.rank[r] = -1;
            if (p.entropy) p.entropy[r] = none;
            if (p.lse) p.lse[r] = none;
        }
        no_top(p, r, status);
    }
    if (p.grad) zero_grad<E>(p, r, rank, C);
}

// one warp: the row of the parts of n warps
__device__ __forceinline__ LpRow join(const LpPart* parts, float c, int n)
{
    LpRow row = {-INFINITY, 0.f, 0.f, 0, 0};
    for (int i = threadIdx.x % 32; i < n; i += 32) row.m = fmax_nan(row.m, parts[i].m);
    row.m = warp_max(row.m);
    for (int i = threadIdx.x % 32; i < n; i += 32) {
        Run u = {parts[i].m, parts[i].s, parts[i].t};
        to_max(u, row.m, c);
        row.s += u.s;
        row.t += u.t;
        row.ahead += parts[i].ahead;
    }
    row.s = warp_sum(row.s);
    row.t = warp_sum(row.t);
    row.ahead = __reduce_add_sync(~0u, row.ahead);
    return row;
}

// ln Z relative to the largest logit m, whose term in the sum is e = 2^d.  Of a row that m dominates ln Z is what the other
// terms are to e: so e is taken off as the instruction gave it, and its error is no part of the result.
__device__ __forceinline__ float log_z(const LpRow& row, float c)
{
    const float e = ex2_fast(dist(row.m, row.m, c));
    return log1pf((row.s - e) / e);
}

// one thread: the results of a row (top tokens apart)
__device__ __forceinline__ void write_row(const ScoreParams& p, int r, const LpRow& row, float xt)
{
    const bool ok = finite_row(row.m);
    const float nan = __int_as_float(0x7FFFFFFF), logz = log_z(row, p.c);
    p.row_status[r] = ok ? SPEC_ROW_OK : SPEC_ROW_NONFINITE;
    if (p.logprob) p.logprob[r] = ok ? (xt - row.m) * p.inv_temp - logz : nan;
    if (p.rank) p.rank[r] = ok ? row.ahead : -1;
    // ln Z - sum p ln(p Z), the sum relative to m's term
    if (p.entropy)
        p.entropy[r] = ok ? fmaxf(0.f, logz + LN2 * (fmaf(dist(row.m, row.m, p.c), row.s, -row.t) / row.s)) : nan;
    if (p.lse) p.lse[r] = ok ? row.m * p.inv_temp + logz : nan;
}

template <typename E, bool TOP> __global__ void __launch_bounds__(SC_NT, TOP ? 5 : 6) k_score_logprobs(const ScoreParams p)
{
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ LpPart parts[SC_MAXC * (SC_NT / 32)];
    __shared__ LpRow s_row;
    const int C = p.cluster, rank = (int)cluster_rank(), r = cluster_id(), tid = threadIdx.x, lane = tid % 32;
    const int id = p.ids ? p.ids[r] : 0;
    if (id < 0 || id >= p.V) {
        no_logprobs<E>(p, r, id == -1 ? SPEC_ROW_OK : SPEC_ROW_BAD_TOKEN, rank, C);
        return;
    }
    // every CTA of the cluster runs before another stores into its shared memory
    if (C > 1) cluster_begin();
    const E* x = row_of<E>(p, r);
    const Slice<E> sl(p, x, rank);
    Ring<E, SC_RING> ring(p, sl, rank, smem);
    const E raw = x[id];
    const uint4 edge = ring.edge();
    const float xt = widen(raw);
    TopScratch& ts = *(TopScratch*)smem;
    uint32_t* const keys = (uint32_t*)(smem + SC_RING * SC_GROUP_BYTES);
    Bits<E>* const most = (Bits<E>*)(keys + SC_GROUPS);
    int ahead = 0;
    Run run;
    auto none = [](int, uint4*) {};
    auto seen = [&](int b, float m) {
        if (TOP) {
            const E e = narrow<E>(m);  // exact: m is a value of E
            most[b * SC_NT + tid] = *reinterpret_cast<const Bits<E>*>(&e);
        }
    };
    if (p.rank) {
        // the equal ones among the elements before x in its vector
        if (rank == 0 && tid >= 64 && tid - 64 < (int)((uintptr_t)(x + id) & 15) / (int)sizeof(E) && tid - 64 < id)
            ahead = widen(x[id - 1 - (tid - 64)]) == xt && xt > -INFINITY;
        Summer<E, true, true> sum;
        sum.c = p.c;
        sum.x = xt;
        sum.tvec = (id - sl.first) >> (sizeof(E) == 4 ? 2 : 3);
        // a masked token: those in front are the unmasked ones
        sum.at = Vec<E>::thr_of(xt);
        sum.under = Vec<E>::thr_of(xt == -INFINITY ? xt : below<E>(raw));
        sum.stream(ring, edge, none, seen);
        run = sum.result();
        ahead += sum.ahead;
    } else {
        Summer<E, true, false> sum;
        sum.c = p.c;
        sum.stream(ring, edge, none, seen);
        run = sum.result();
    }
    // threads to warp
    LpPart w;
    w.m = warp_max(run.m);
    to_max(run, w.m, p.c);
    w.s = warp_sum(run.s);
    w.t = warp_sum(run.t);
    w.ahead = __reduce_add_sync(~0u, ahead);
    // warps to cluster: to CTA 0, or to all
    if (C > 1) cluster_wait();
    if (lane < (TOP ? C : 1)) {
        const uint32_t to = remote(parts + rank * (SC_NT / 32) + tid / 32, lane);
        remote_st(to, __float_as_uint(w.m));
        remote_st(to + 4, __float_as_uint(w.s));
        remote_st(to + 8, __float_as_uint(w.t));
        remote_st(to + 12, (uint32_t)w.ahead);
    }
    if (TOP) give_keys<E>(keys, most, ring.full, rank, C);
    row_arrive(C);
    if (!TOP && rank != 0) return;
    row_wait(C);
    if (tid < 32) {
        LpRow row = join(parts, p.c, C * (SC_NT / 32));
        if (TOP) row.bound = bound_of(keys, p.top_n);
        if (lane == 0) {
            if (rank == 0) write_row(p, r, row, xt);
            if (TOP) ts.mine = ts.agains = 0;
            s_row = row;
        }
    }
    if (!TOP) return;
    __syncthreads();
    const LpRow row = s_row;
    if (!finite_row(row.m)) {
        if (rank == 0) no_top(p, r, SPEC_ROW_NONFINITE);
        return;
    }
    give_candidates(sl, p.V, ring.full, ts, most, row.bound, p.top_n, rank, C);
    row_arrive(C);
    if (rank != 0) return;
    row_wait(C);
    write_top(p, r, ts, row, log_z(row, p.c), C);
}

template <typename E> __global__ void __launch_bounds__(SC_NT, 4) k_score_logprobs_grad(const ScoreParams p)
{
    constexpr int W = SC_NT / 32;
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ LpPart parts[SC_MAXC * W];
    __shared__ LpRow s_row;
    const int C = p.cluster, rank = (int)cluster_rank(), r = cluster_id(), tid = threadIdx.x, lane = tid % 32;
    const int id = p.ids ? p.ids[r] : 0;
    if (id < 0 || id >= p.V) {
        no_logprobs<E>(p, r, id == -1 ? SPEC_ROW_OK : SPEC_ROW_BAD_TOKEN, rank, C);
        return;
    }
    // every CTA of the cluster runs before another stores into its shared memory
    if (C > 1) cluster_begin();
    const E* x = row_of<E>(p, r);
    const Slice<E> sl(p, x, rank);
    Ring<E, SC_RING_GRAD> ring(p, sl, rank, smem);
    // (waited for where they are used)
    const E xt = x[id];
    const float gl = p.g_logprob ? p.g_logprob[r] : 0.f, gh = p.g_entropy ? p.g_entropy[r] : 0.f;
    const uint4 edge = ring.edge();
    Summer<E, true, false> sum;
    sum.c = p.c;
    sum.stream(ring, edge, [](int, uint4*) {}, [](int, float) {});
    Run run = sum.result();
    LpPart w;
    w.m = warp_max(run.m);
    to_max(run, w.m, p.c);
    w.s = warp_sum(run.s);
    w.t = warp_sum(run.t);
    if (C > 1) cluster_wait();
    if (lane < C) {
        const uint32_t to = remote(parts + rank * W + tid / 32, lane);
        remote_st(to, __float_as_uint(w.m));
        remote_st(to + 4, __float_as_uint(w.s));
        remote_st(to + 8, __float_as_uint(w.t));
        remote_st(to + 12, 0u);
    }
    row_arrive(C);
    row_wait(C);
    if (tid < 32) {
        const LpRow row = join(parts, p.c, C * W);
        if (lane == 0) {
            s_row = row;
            if (rank == 0) write_row(p, r, row, widen(xt));
        }
    }
    __syncthreads();
    const LpRow row = s_row;
    if (!finite_row(row.m)) {
        copy_done();
        zero_grad<E>(p, r, rank, C);
        return;
    }
    // e (A + B d), e = 2^d: p = e / s, ln p = d ln 2 - ln s.  The product e d comes first, which is 0 where e is; B d may
    // be out of range there.
    const float f = p.inv_temp / row.s, A = -(gl - gh * LN2 * (row.t / row.s)) * f, B = -gh * LN2 * f;
    const uint64_t A2 = pair(A, A), B2 = pair(B, B);
    E* g = grad_of<E>(p, r);
    if (p.g_entropy)
        grad_slice(ring, edge, g, row.m, p.c, sum.masked,
                   [&](uint64_t d2, uint64_t e2) { return fma2(mul2(e2, d2), B2, mul2(e2, A2)); });
    else
        grad_slice(ring, edge, g, row.m, p.c, 0, [&](uint64_t, uint64_t e2) { return mul2(e2, A2); });
    if (p.g_logprob && ring.has(id)) {
        __syncthreads();
        if (tid == 0) {
            const float d = dist(widen(xt), row.m, p.c), e = ex2_fast(d);
            g[id] = narrow<E>(gl * p.inv_temp + e * (A + B * fmaxf(d, NONE)));
        }
    }
}

template <typename E, bool TOP> cudaError_t go_forward(ScoreParams p, int num_sms, cudaStream_t s)
{
    static ScoreKernel sk;
    const auto kernel = k_score_logprobs<E, TOP>;
    auto smem = [](size_t per) {
        return SC_RING * SC_GROUP_BYTES + (TOP ? SC_GROUPS * 4 + (per / (SC_NT * SC_GROUP) + 2) * SC_NT * sizeof(E) : 0);
    };
    cudaError_t e = score_ready(kernel, sk, smem(0), smem(SCORE_MAX_ROW_BYTES / 16 + 2));
    if (e == cudaSuccess) e = score_split_forward(sk, p, sizeof(E), num_sms, TOP ? 48 : 16, smem);
    return e == cudaSuccess ? score_launch(kernel, p, smem(p.per), s) : e;
}
template <typename E> cudaError_t go(ScoreParams p, int num_sms, cudaStream_t s)
{
    if (!p.grad || p.top_n || p.rank) {
        ScoreParams q = p;
        q.grad = nullptr;
        const cudaError_t e = p.top_n ? go_forward<E, true>(q, num_sms, s) : go_forward<E, false>(q, num_sms, s);
        if (e != cudaSuccess || !p.grad) return e;
        // the gradient's kernel writes none of that again
        p.top_n = 0;
        p.rank = nullptr;
    }
    static ScoreKernel sk;
    const cudaError_t e = score_ready(k_score_logprobs_grad<E>, sk, SC_GRAD_BYTES, SC_GRAD_BYTES);
    if (e != cudaSuccess) return e;
    score_split_gradient(p, sizeof(E), num_sms);
    return score_launch(k_score_logprobs_grad<E>, p, SC_GRAD_BYTES, s);
}

}  // namespace

cudaError_t launch_score_logprobs(const ScoreParams& p, int dtype, int num_sms, cudaStream_t s)
{
    return dtype == SPEC_F32 ? go<float>(p, num_sms, s)
           : dtype == SPEC_BF16 ? go<__nv_bfloat16>(p, num_sms, s)
                                : go<__half>(p, num_sms, s);
}

}  // namespace sv
