// sv_score.cu -- the operators that score rows of logits: log probabilities of
// given tokens with entropy and top alternatives, the divergence from a
// teacher's top logits, and their gradients.
//
// A row is taken by a cluster of 1 to 8 CTAs, each of which holds its slice of
// the row in shared memory: one trip to HBM whatever follows (the sums, the
// search for the top tokens, the gradient, which needs the row's sum before its
// first element).  Slices are whole 16-byte vectors of the row's addresses, so
// rows of any alignment are copied and read alike; what a row's first and last
// vector have outside the row is -inf, which counts nowhere.
//
//   copy     each thread copies the vectors that it will read itself
//            (cp.async; no barrier between the copy and the sums)
//   sums     per thread, a running maximum m, s = sum 2^d and (entropy) sum d
//            2^d with d = (l - m) log2(e) / t; the difference comes first, as
//            a product with l may overflow where it does not (rows of the
//            type's lowest values)
//   join     threads, then CTAs by stores into each other's shared memory and
//            one cluster barrier, in a fixed order
//   the rest each CTA for its slice (gradient), CTA 0 for the row
#include <type_traits>

#include "sv_score.cuh"

namespace sv {

namespace {

constexpr int SC_NT = 128;      // threads of a CTA
constexpr int SC_WARPS = SC_NT / 32;
constexpr int SC_BATCH = 4;     // vectors of a thread per copy group
constexpr int SC_MAXC = SCORE_MAX_CTAS;  // CTAs of a cluster (portable)
constexpr int SC_PARTS = SC_MAXC * SC_WARPS;  // warps of a cluster: one lane each where they are joined
constexpr int SC_LIST = 1024;   // candidates for the top tokens, all CTAs of a row together
constexpr uint32_t KEY_NEG_INF = 0x007FFFFFu;  // key_of(-inf)
constexpr float LN2 = 0.693147180559945f;
constexpr float NONE = -200.f;  // a power of 2 that is 0 in fp32; products with it are, too, and with -inf are not

// ---- elements and vectors of 16 bytes ------------------------------------- //
template <typename E> __device__ __forceinline__ float widen(E x);
template <> __device__ __forceinline__ float widen(float x) { return x; }
template <> __device__ __forceinline__ float widen(__nv_bfloat16 x) { return __bfloat162float(x); }
template <> __device__ __forceinline__ float widen(__half x) { return __half2float(x); }
template <typename E> __device__ __forceinline__ E narrow(float x);
template <> __device__ __forceinline__ float narrow(float x) { return x; }
template <> __device__ __forceinline__ __nv_bfloat16 narrow(float x) { return __float2bfloat16_rn(x); }
template <> __device__ __forceinline__ __half narrow(float x) { return __float2half_rn(x); }

template <typename E> constexpr int EPV = 16 / (int)sizeof(E);  // elements of a vector
template <typename E> using Bits = std::conditional_t<sizeof(E) == 4, uint32_t, uint16_t>;

// elements of a vector in registers (q known when the loop around it is unrolled)
__device__ __forceinline__ uint32_t word_of(const uint4& w, int q) { return q == 0 ? w.x : q == 1 ? w.y : q == 2 ? w.z : w.w; }
template <typename E> __device__ __forceinline__ Bits<E> bits_at(const uint4& w, int q)
{
    if constexpr (sizeof(E) == 4) return word_of(w, q);
    else return (uint16_t)(word_of(w, q / 2) >> (q % 2 * 16));
}
template <typename E> __device__ __forceinline__ uint4 vector_of(const Bits<E> (&b)[EPV<E>])
{
    if constexpr (sizeof(E) == 4) return make_uint4(b[0], b[1], b[2], b[3]);
    else return make_uint4(b[0] | (uint32_t)b[1] << 16, b[2] | (uint32_t)b[3] << 16, b[4] | (uint32_t)b[5] << 16,
                           b[6] | (uint32_t)b[7] << 16);
}
template <typename E> __device__ __forceinline__ float value_of(Bits<E> b)
{
    if constexpr (sizeof(E) == 4) return __uint_as_float(b);
    else return widen(*reinterpret_cast<const E*>(&b));
}

// pairs of fp32 in one 64-bit register
__device__ __forceinline__ uint64_t pair(float a, float b)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpair(uint64_t x, float& a, float& b)
{
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x));
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

template <typename E> struct Vec;
template <> struct Vec<float> {
    static constexpr uint32_t NEG = 0xFF800000u;  // -inf
    static __device__ __forceinline__ uint64_t two(uint32_t a, uint32_t b)
    {
        return pair(__uint_as_float(a), __uint_as_float(b));
    }
    static __device__ __forceinline__ void pairs(const uint4& w, uint64_t (&x)[2])
    {
        x[0] = two(w.x, w.y);
        x[1] = two(w.z, w.w);
    }
    static __device__ __forceinline__ float top(const uint4& w)
    {
        return fmax_nan(fmax_nan(__uint_as_float(w.x), __uint_as_float(w.y)),
                        fmax_nan(__uint_as_float(w.z), __uint_as_float(w.w)));
    }
    static __device__ __forceinline__ uint4 pack(const uint64_t (&y)[2])
    {
        float a, b, c, d;
        unpair(y[0], a, b);
        unpair(y[1], c, d);
        return make_uint4(__float_as_uint(a), __float_as_uint(b), __float_as_uint(c), __float_as_uint(d));
    }
    using Thr = float;
    static __device__ __forceinline__ Thr thr_of(float x) { return x; }
    static __device__ __forceinline__ int above(const uint4& w, Thr thr)
    {
        return (__uint_as_float(w.x) > thr) + (__uint_as_float(w.y) > thr) + (__uint_as_float(w.z) > thr) +
               (__uint_as_float(w.w) > thr);
    }
};
// 16-bit types: what differs is how a word of two becomes fp32 and back
template <typename E> struct Vec16 {
    static __device__ __forceinline__ void pairs(const uint4& w, uint64_t (&x)[4])
    {
        x[0] = Vec<E>::wide(w.x);
        x[1] = Vec<E>::wide(w.y);
        x[2] = Vec<E>::wide(w.z);
        x[3] = Vec<E>::wide(w.w);
    }
    static __device__ __forceinline__ float top(const uint4& w)
    {
        const uint32_t m = Vec<E>::max2(Vec<E>::max2(w.x, w.y), Vec<E>::max2(w.z, w.w));
        float a, b;
        unpair(Vec<E>::wide(m), a, b);
        return fmax_nan(a, b);
    }
    static __device__ __forceinline__ uint4 pack(const uint64_t (&y)[4])
    {
        return make_uint4(Vec<E>::thin(y[0]), Vec<E>::thin(y[1]), Vec<E>::thin(y[2]), Vec<E>::thin(y[3]));
    }
    using Thr = uint32_t;
    static __device__ __forceinline__ Thr thr_of(float x) { return Vec<E>::thin(pair(x, x)); }  // x is a value of E
    // counts of up to 8 elements in two halves, exact in either type
    static __device__ __forceinline__ int above(const uint4& w, Thr t)
    {
        const uint32_t n = Vec<E>::plus(Vec<E>::plus(Vec<E>::gt(w.x, t), Vec<E>::gt(w.y, t)),
                                        Vec<E>::plus(Vec<E>::gt(w.z, t), Vec<E>::gt(w.w, t)));
        float a, b;
        unpair(Vec<E>::wide(n), a, b);
        return (int)(a + b);
    }
};
template <> struct Vec<__nv_bfloat16> : Vec16<__nv_bfloat16> {
    static constexpr uint32_t NEG = 0xFF80FF80u;
    static __device__ __forceinline__ uint64_t wide(uint32_t w) { return pair(bf16_lo(w), bf16_hi(w)); }
    static __device__ __forceinline__ uint32_t thin(uint64_t y)
    {
        float a, b;
        unpair(y, a, b);
        uint32_t r;
        asm("cvt.rn.bf16x2.f32 %0, %2, %1;" : "=r"(r) : "f"(a), "f"(b));
        return r;
    }
    static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b)
    {
        uint32_t r;
        asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        return r;
    }
    static __device__ __forceinline__ uint32_t gt(uint32_t a, uint32_t b)
    {
        uint32_t r;
        asm("set.gt.bf16x2.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        return r;
    }
    static __device__ __forceinline__ uint32_t plus(uint32_t a, uint32_t b)
    {
        uint32_t r;
        asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        return r;
    }
};
template <> struct Vec<__half> : Vec16<__half> {
    static constexpr uint32_t NEG = 0xFC00FC00u;
    static __device__ __forceinline__ uint64_t wide(uint32_t w)
    {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
        return pair(f.x, f.y);
    }
    static __device__ __forceinline__ uint32_t thin(uint64_t y)
    {
        float a, b;
        unpair(y, a, b);
        uint32_t r;
        asm("cvt.rn.f16x2.f32 %0, %2, %1;" : "=r"(r) : "f"(a), "f"(b));
        return r;
    }
    static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b)
    {
        uint32_t r;
        asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        return r;
    }
    static __device__ __forceinline__ uint32_t gt(uint32_t a, uint32_t b)
    {
        uint32_t r;
        asm("set.gt.f16x2.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        return r;
    }
    static __device__ __forceinline__ uint32_t plus(uint32_t a, uint32_t b)
    {
        uint32_t r;
        asm("add.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        return r;
    }
};

// the next value of the type below a finite x (-0 and +0 are one value)
template <typename E> __device__ __forceinline__ float below(E x)
{
    if constexpr (sizeof(E) == 4) {
        const uint32_t b = __float_as_uint(x);
        return __uint_as_float((b << 1) == 0 ? 0x80000001u : (b >> 31) ? b + 1 : b - 1);
    } else {
        unsigned short b = *reinterpret_cast<unsigned short*>(&x);
        b = (b & 0x7FFF) == 0 ? 0x8001 : (b >> 15) ? b + 1 : b - 1;
        return widen(*reinterpret_cast<E*>(&b));
    }
}

// ---- the cluster ----------------------------------------------------------- //
__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ int cluster_id()
{
    int r;
    asm volatile("mov.u32 %0, %%clusterid.x;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }
// the address of a shared variable in CTA `rank` of the cluster
__device__ __forceinline__ uint32_t remote(const void* p, int rank)
{
    uint32_t a = (uint32_t)__cvta_generic_to_shared(p), r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
    return r;
}
__device__ __forceinline__ void remote_st(uint32_t a, uint32_t v)
{
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}

// ---- a CTA's slice of a row ------------------------------------------------ //
template <typename E> struct Slice {
    uint4* buf;       // its vectors, in shared memory
    const char* src;  // global address of the first
    int n;            // vectors
    int first;        // element of the row at the first vector's start (negative: outside the row)
    int lo, hi;       // vectors lo .. hi - 1 lie in the row as a whole; one before and one behind may not
    int V;

    __device__ __forceinline__ Slice(const ScoreParams& p, const E* x, int rank, void* smem)
    {
        const int mis = (int)((uintptr_t)x & 15), all = (mis + p.V * (int)sizeof(E) + 15) / 16, v0 = rank * p.per;
        n = max(0, min(p.per, all - v0));
        first = v0 * EPV<E> - mis / (int)sizeof(E);
        src = (const char*)x - mis + (int64_t)v0 * 16;
        buf = (uint4*)smem;
        V = p.V;
        lo = first < 0 ? 1 : 0;
        hi = max(lo, first + n * EPV<E> > V ? n - 1 : n);
    }
    __device__ __forceinline__ int full() const { return n / (SC_NT * SC_BATCH); }  // batches of all threads
    __device__ __forceinline__ bool has(int id) const { return id >= first && id < first + n * EPV<E> && id < V; }
    __device__ __forceinline__ Bits<E>* at(int id) const { return (Bits<E>*)buf + (id - first); }

    // vector i by its elements, -inf outside the row
    __device__ __forceinline__ void copy_part(int i) const
    {
        const int e = first + i * EPV<E>;
        const Bits<E>* from = (const Bits<E>*)(src + (int64_t)i * 16);
        Bits<E> v[EPV<E>];
#pragma unroll
        for (int q = 0; q < EPV<E>; ++q) v[q] = e + q >= 0 && e + q < V ? from[q] : (Bits<E>)Vec<E>::NEG;
        buf[i] = vector_of<E>(v);
    }
    // every thread copies what it reads: vectors tid, tid + SC_NT, ...; a group for each full batch, one for the rest
    __device__ __forceinline__ void copy() const
    {
        const uint32_t to = (uint32_t)__cvta_generic_to_shared(buf);
        auto one = [&](int i) {
            if (i >= lo && i < hi)
                asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16;" ::"r"(to + i * 16),
                             "l"(src + (int64_t)i * 16)
                             : "memory");
        };
        int i = threadIdx.x;
        for (int b = full(); b > 0; --b) {
#pragma unroll
            for (int j = 0; j < SC_BATCH; ++j, i += SC_NT) one(i);
            asm volatile("cp.async.commit_group;" ::: "memory");
        }
        for (; i < n; i += SC_NT) one(i);
        asm volatile("cp.async.commit_group;" ::: "memory");
        if (lo && n && threadIdx.x == 0) copy_part(0);
        if (hi < n && n - 1 >= lo && (n - 1) % SC_NT == threadIdx.x) copy_part(n - 1);
    }
    // this thread's copies but those of the last `left` groups have arrived (of these, some may have, too)
    static __device__ __forceinline__ void arrived(int left)
    {
        switch (left) {
        case 0: asm volatile("cp.async.wait_group 0;" ::: "memory"); break;
        case 1: asm volatile("cp.async.wait_group 1;" ::: "memory"); break;
        case 2: asm volatile("cp.async.wait_group 2;" ::: "memory"); break;
        case 3: asm volatile("cp.async.wait_group 3;" ::: "memory"); break;
        case 4: asm volatile("cp.async.wait_group 4;" ::: "memory"); break;
        case 5: asm volatile("cp.async.wait_group 5;" ::: "memory"); break;
        default: asm volatile("cp.async.wait_group 6;" ::: "memory"); break;
        }
    }
};

// a running softmax: maximum, sum of 2^d, sum of d 2^d, d relative to the maximum
struct Run {
    float m, s, t;
};
__device__ __forceinline__ float ref_of(float m) { return m == -INFINITY ? 0.f : m; }

// sums of a thread's vectors, by ENTROPY those of d 2^d too; without it c is taken in two parts (c + c_lo, c_lo > 0),
// since a loss near its minimum shows the constant's rounding; with RANK also the number of elements above x (in
// vectors before tvec: or equal to it, written as above the next value below x)
template <typename E, bool ENTROPY, bool RANK> struct Summer {
    float m = -INFINITY;
    uint64_t s2 = 0, t2 = 0, c2, l2;
    typename Vec<E>::Thr at, under;
    int tvec, ahead = 0;

    template <int N> __device__ __forceinline__ void take(const uint4 (&w)[N], int i)
    {
        float mx = Vec<E>::top(w[0]);
#pragma unroll
        for (int j = 1; j < N; ++j) mx = fmax_nan(mx, Vec<E>::top(w[j]));
        if (!(mx <= m)) {  // a new maximum (or NaN, which stays): rescale
            mx = fmax_nan(m, mx);
            if (m > -INFINITY) {
                float c, c_;
                unpair(c2, c, c_);
                const float d = fmaxf((m - mx) * c, NONE), f = ex2_fast(d);
                const uint64_t f2 = pair(f, f);
                if (ENTROPY) t2 = mul2(f2, fma2(pair(d, d), s2, t2));
                s2 = mul2(f2, s2);
            }
            m = mx;
        }
        const float ref = -ref_of(m);
        const uint64_t r2 = pair(ref, ref);
#pragma unroll
        for (int j = 0; j < N; ++j) {
            uint64_t v[EPV<E> / 2];
            Vec<E>::pairs(w[j], v);
#pragma unroll
            for (int q = 0; q < EPV<E> / 2; ++q) {
                const uint64_t x2 = add2(v[q], r2), d2 = ENTROPY ? mul2(x2, c2) : fma2(x2, c2, mul2(x2, l2));
                float a, z;
                unpair(d2, a, z);
                const uint64_t e2 = pair(ex2_fast(a), ex2_fast(z));
                s2 = add2(s2, e2);
                if (ENTROPY) t2 = fma2(e2, pair(fmaxf(a, NONE), fmaxf(z, NONE)), t2);
            }
            if (RANK) ahead += Vec<E>::above(w[j], i + j * SC_NT < tvec ? under : at);
        }
    }
    __device__ __forceinline__ Run run(const Slice<E>& sl, bool waits)
    {
        int i = threadIdx.x;
        for (int b = sl.full(); b > 0; --b, i += SC_NT * SC_BATCH) {
            if (waits) sl.arrived(b);
            uint4 w[SC_BATCH];
#pragma unroll
            for (int j = 0; j < SC_BATCH; ++j) w[j] = sl.buf[i + j * SC_NT];
            take(w, i);
        }
        if (waits) sl.arrived(0);
        for (; i < sl.n; i += SC_NT) {
            const uint4 w[1] = {sl.buf[i]};
            take(w, i);
        }
        float a, z;
        Run r;
        r.m = m;
        unpair(s2, a, z);
        r.s = a + z;
        unpair(t2, a, z);
        r.t = a + z;
        return r;
    }
};

// rescales a run to a maximum that is no smaller
__device__ __forceinline__ void to_max(Run& r, float m, float c)
{
    const float d = fmaxf((r.m - m) * c, NONE), f = ex2_fast(d);
    r.t = r.m == -INFINITY ? 0.f : f * (r.t + d * r.s);
    r.s = r.m == -INFINITY ? 0.f : f * r.s;
    r.m = m;
}

template <typename X, typename F> __device__ __forceinline__ X warp_reduce(X x, F op)
{
#pragma unroll
    for (int d = 16; d; d >>= 1) x = op(x, __shfl_xor_sync(~0u, x, d));
    return x;
}
__device__ __forceinline__ float warp_max(float x)
{
    return warp_reduce(x, [](float a, float b) { return fmax_nan(a, b); });
}
template <typename X> __device__ __forceinline__ X warp_sum(X x)
{
    return warp_reduce(x, [](X a, X b) { return a + b; });
}

template <typename E> __device__ __forceinline__ const E* row_of(const ScoreParams& p, int r)
{
    const int b = p.by_tokens.of(r);
    return (const E*)p.x + (int64_t)b * p.x_seq + (int64_t)(r - b * p.T) * p.x_tok;
}
template <typename E> __device__ __forceinline__ E* grad_of(const ScoreParams& p, int r)
{
    const int b = p.by_tokens.of(r);
    return (E*)p.grad + (int64_t)b * p.g_seq + (int64_t)(r - b * p.T) * p.g_tok;
}

// a row without a gradient, by the cluster's CTAs
template <typename E> __device__ void zero_grad(const ScoreParams& p, int r, int rank, int C)
{
    E* g = grad_of<E>(p, r);
    const int head = (int)min((int64_t)p.V, (int64_t)(-(intptr_t)((uintptr_t)g / sizeof(E))) & (EPV<E> - 1));
    const int nv = (p.V - head) / EPV<E>, i0 = rank * SC_NT + threadIdx.x;
    uint4* to = (uint4*)(g + head);
    for (int i = i0; i < nv; i += C * SC_NT) to[i] = make_uint4(0, 0, 0, 0);
    if (i0 < head) g[i0] = narrow<E>(0.f);
    const int rest = head + nv * EPV<E> + i0;
    if (rest < p.V) g[rest] = narrow<E>(0.f);
}

// the gradient of a slice: f(distances d of a pair of logits from m, times c; 2^d) -> pair
template <typename E, typename F>
__device__ __forceinline__ void grad_slice(const Slice<E>& sl, E* g, float m, float c, F f)
{
    const float ref = -ref_of(m);
    const uint64_t r2 = pair(ref, ref), c2 = pair(c, c);
    auto grad = [&](int i) {
        uint64_t v[EPV<E> / 2], y[EPV<E> / 2];
        Vec<E>::pairs(sl.buf[i], v);
#pragma unroll
        for (int q = 0; q < EPV<E> / 2; ++q) {
            const uint64_t d2 = mul2(add2(v[q], r2), c2);
            float a, z;
            unpair(d2, a, z);
            y[q] = f(a, z, pair(ex2_fast(a), ex2_fast(z)));
        }
        return Vec<E>::pack(y);
    };
    E* out = g + sl.first;  // its element at the slice's start
    if (((uintptr_t)out & 15) == 0) {
        uint4* to = (uint4*)out;
        int i = threadIdx.x;
        for (int b = sl.full(); b > 0; --b)
#pragma unroll
            for (int j = 0; j < SC_BATCH; ++j, i += SC_NT) {
                const uint4 w = grad(i);
                if (i >= sl.lo && i < sl.hi) to[i] = w;
            }
        for (; i < sl.n; i += SC_NT) {
            const uint4 w = grad(i);
            if (i >= sl.lo && i < sl.hi) to[i] = w;
        }
        // the vectors that are not the row's as a whole
        const int part = threadIdx.x == 0 ? 0 : sl.n - 1;
        if (threadIdx.x < 2 && sl.n > 0 && (part < sl.lo || part >= sl.hi)) {
            const uint4 w = grad(part);
            const int e = sl.first + part * EPV<E>;
#pragma unroll
            for (int q = 0; q < EPV<E>; ++q)
                if (e + q >= 0 && e + q < sl.V) ((Bits<E>*)g)[e + q] = bits_at<E>(w, q);
        }
        return;
    }
    // the gradient's rows start elsewhere in a vector than the logits': elements change vectors on the way out
    for (int i = threadIdx.x; i < sl.n; i += SC_NT) sl.buf[i] = grad(i);
    __syncthreads();
    const int e0 = max(sl.first, 0), e1 = min(sl.first + sl.n * EPV<E>, sl.V);
    if (e0 >= e1) return;
    const int head = min(e1 - e0, (int)((-(intptr_t)((uintptr_t)(g + e0) / sizeof(E))) & (EPV<E> - 1)));
    const int nv = (e1 - e0 - head) / EPV<E>;
    const Bits<E>* from = sl.at(e0);
    Bits<E>* to = (Bits<E>*)g + e0;
    for (int i = threadIdx.x; i < nv; i += SC_NT) {
        Bits<E> v[EPV<E>];
#pragma unroll
        for (int q = 0; q < EPV<E>; ++q) v[q] = from[head + i * EPV<E> + q];
        *(uint4*)(to + head + i * EPV<E>) = vector_of<E>(v);
    }
    if (threadIdx.x < head) to[threadIdx.x] = from[threadIdx.x];
    const int rest = head + nv * EPV<E> + threadIdx.x;
    if (rest < e1 - e0) to[rest] = from[rest];
}

// ---- log probabilities ------------------------------------------------------ //
struct LpPart {      // what a warp knows of the row
    float m, s, t;
    int32_t ahead;
};
struct LpRow {
    float m, s, t;
    int32_t ahead;
    uint32_t bound;  // a key that the top tokens reach, and not many others
};

// scratch of the search for the top tokens, behind the slice
struct TopScratch {
    uint32_t keys[SC_MAXC][32];         // the largest key of every four threads of the cluster
    unsigned long long list[SC_LIST];   // CTA 0: candidates, key and inverted id, SC_LIST / C to a CTA
    int32_t counts[SC_MAXC];            // CTA 0: candidates of each CTA
    int32_t mine;                       // candidates of this CTA
    int32_t tally[2][SC_WARPS];
};

__device__ __forceinline__ int tally_of(TopScratch& ts, int round, int x)
{
    // one barrier a round: the other buffer is free again when it is passed
    x = __reduce_add_sync(~0u, x);
    if (threadIdx.x % 32 == 0) ts.tally[round & 1][threadIdx.x / 32] = x;
    __syncthreads();
    int n = 0;
#pragma unroll
    for (int i = 0; i < SC_WARPS; ++i) n += ts.tally[round & 1][i];
    return n;
}

template <typename E, typename F> __device__ __forceinline__ void each_mine(const Slice<E>& sl, F f)
{
    for (int i = threadIdx.x; i < sl.n; i += SC_NT) {
        const uint4 w = sl.buf[i];
#pragma unroll
        for (int q = 0; q < EPV<E>; ++q) f(key_of(value_of<E>(bits_at<E>(w, q))), sl.first + i * EPV<E> + q);
    }
}

// The candidates of a CTA whose keys reach `bound`, into the list of CTA 0.  When they are too many for its share of
// the list (equal logits, masks), its first n in the order (key desc, id asc), found by halving the range of keys and
// of ids and counting.
template <typename E>
__device__ void give_candidates(const Slice<E>& sl, TopScratch& ts, uint32_t bound, uint32_t my_key, int n, int rank, int C)
{
    const int share = SC_LIST / C;
    const uint32_t list = remote(ts.list + rank * share, 0);
    auto give = [&](uint32_t key, int id) {
        const int at = atomicAdd(&ts.mine, 1);
        if (at < share) {
            remote_st(list + at * 8, ~(uint32_t)id);
            remote_st(list + at * 8 + 4, key);
        }
    };
    if (my_key >= bound) {
        const float least = val_of(bound);
        for (int i = threadIdx.x; i < sl.n; i += SC_NT) {
            const uint4 w = sl.buf[i];
            if (Vec<E>::top(w) < least) continue;
#pragma unroll
            for (int q = 0; q < EPV<E>; ++q) {
                const uint32_t key = key_of(value_of<E>(bits_at<E>(w, q)));
                if (key >= bound) give(key, sl.first + i * EPV<E> + q);
            }
        }
    }
    __syncthreads();
    int found = ts.mine;
    if (found > share) {
        __syncthreads();
        if (threadIdx.x == 0) ts.mine = 0;
        int round = 0;
        uint32_t lo = bound, hi = 0xFF800000u;
        while (lo < hi) {  // the n-th largest key
            const uint32_t mid = lo + (hi - lo + 1) / 2;
            int k = 0;
            if (my_key >= mid) each_mine(sl, [&](uint32_t key, int) { k += key >= mid; });
            if (tally_of(ts, round++, k) >= n) lo = mid;
            else hi = mid - 1;
        }
        int k = 0;
        each_mine(sl, [&](uint32_t key, int) { k += key > lo; });
        const int ties = n - tally_of(ts, round++, k);
        int first = sl.first, last = sl.first + sl.n * EPV<E> - 1;  // the last id among its equals
        while (first < last) {
            const int mid = first + (last - first) / 2;
            k = 0;
            if (my_key >= lo) each_mine(sl, [&](uint32_t key, int id) { k += key == lo && id <= mid; });
            if (tally_of(ts, round++, k) >= ties) last = mid;
            else first = mid + 1;
        }
        if (my_key >= lo)
            each_mine(sl, [&](uint32_t key, int id) {
                if (key > lo || (key == lo && id <= last)) give(key, id);
            });
        found = n;
    }
    if (threadIdx.x == 0) remote_st(remote(ts.counts + rank, 0), (uint32_t)found);
}

// One warp: a key that at least n (all, if fewer) of the row's unmasked tokens reach, and not many more: at least n
// groups' largest do, by halving the range of keys until their number is near n.  Up to 256 groups, n at most half of
// them: with n of g groups above it, a bound has g ln(g / (g - n)) tokens above it when they lie at random (n = 128,
// g = 256: 177).
__device__ __forceinline__ uint32_t bound_of(const TopScratch& ts, float m, int n, int C)
{
    uint32_t mine[SC_MAXC], lo = ~0u;
    int k = 0;
#pragma unroll
    for (int i = 0; i < SC_MAXC; ++i) {
        mine[i] = i < C ? ts.keys[i][threadIdx.x % 32] : 0;
        if (mine[i] > KEY_NEG_INF) {
            lo = min(lo, mine[i]);
            ++k;
        }
    }
    lo = __reduce_min_sync(~0u, lo);
    // fewer than n groups have an unmasked token at all: every unmasked token is a candidate
    if (__reduce_add_sync(~0u, k) < n) return KEY_NEG_INF + 1;
    uint32_t hi = key_of(m);
    while (lo < hi) {
        const uint32_t mid = lo + (hi - lo + 1) / 2;
        k = 0;
#pragma unroll
        for (int i = 0; i < SC_MAXC; ++i) k += mine[i] >= mid;
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

// a row that is not scored, or has a status
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
        for (int i = threadIdx.x; i < p.top_n; i += SC_NT) {
            p.top_ids[(int64_t)r * p.top_n + i] = -1;
            p.top_lp[(int64_t)r * p.top_n + i] = status == SPEC_ROW_OK ? -INFINITY : none;
        }
    }
    if (p.grad) zero_grad<E>(p, r, rank, C);
}

template <typename E, bool GRAD> __global__ void __launch_bounds__(SC_NT) k_score_logprobs(const ScoreParams p)
{
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ LpPart parts[SC_PARTS];
    __shared__ LpRow s_row;
    const int C = p.cluster, rank = (int)cluster_rank(), r = cluster_id(), tid = threadIdx.x, lane = tid % 32;
    const int id = p.ids ? p.ids[r] : 0;
    if (id < 0 || id >= p.V) {
        no_logprobs<E>(p, r, id == -1 ? SPEC_ROW_OK : SPEC_ROW_BAD_TOKEN, rank, C);
        return;
    }
    const E* x = row_of<E>(p, r);
    const Slice<E> sl(p, x, rank, smem);
    TopScratch& ts = *(TopScratch*)(smem + p.top_at);
    sl.copy();
    const E raw = x[id];
    const float xt = widen(raw);
    // every CTA of the cluster runs before another stores into its shared memory
    if (C > 1) cluster_arrive();
    if (tid == 0 && p.top_n) ts.mine = 0;
    int ahead = 0;
    Run run;
    if (p.rank && !GRAD) {
        Summer<E, true, true> sum;
        sum.c2 = pair(p.c, p.c);
        sum.tvec = (id - sl.first) >> (sizeof(E) == 4 ? 2 : 3);
        // a masked token: those in front are the unmasked ones
        sum.at = Vec<E>::thr_of(xt);
        sum.under = Vec<E>::thr_of(xt == -INFINITY ? xt : below<E>(raw));
        run = sum.run(sl, true);
        ahead = sum.ahead;
        if (sum.tvec >= 0 && sum.tvec < sl.n && sum.tvec % SC_NT == tid && xt > -INFINITY)
            for (int q = 0; q < id - sl.first - sum.tvec * EPV<E>; ++q)
                ahead += value_of<E>(bits_at<E>(sl.buf[sum.tvec], q)) == xt;
    } else {
        Summer<E, true, false> sum;
        sum.c2 = pair(p.c, p.c);
        run = sum.run(sl, true);
        if (p.rank) {  // with a gradient, where the loop above has no room for it
            each_mine(sl, [&](uint32_t key, int v) {
                const uint32_t k = key_of(xt);
                ahead += key > k || (key == k && v < id && key > KEY_NEG_INF);
            });
        }
    }
    const uint32_t my_key = key_of(run.m);
    // threads to warp
    LpPart w;
    w.m = warp_max(run.m);
    to_max(run, w.m, p.c);
    w.s = warp_sum(run.s);
    w.t = warp_sum(run.t);
    w.ahead = __reduce_add_sync(~0u, ahead);
    // warps to cluster: to CTA 0, or (what comes next needs the row's sum, or a bound) to all
    const bool all = GRAD || p.top_n;
    if (C > 1) cluster_wait();
    if (lane < (all ? C : 1)) {
        const uint32_t to = remote(parts + rank * SC_WARPS + tid / 32, lane);
        remote_st(to, __float_as_uint(w.m));
        remote_st(to + 4, __float_as_uint(w.s));
        remote_st(to + 8, __float_as_uint(w.t));
        remote_st(to + 12, (uint32_t)w.ahead);
    }
    if (p.top_n) {
        uint32_t k = max(my_key, __shfl_xor_sync(~0u, my_key, 1));
        k = max(k, __shfl_xor_sync(~0u, k, 2));
        for (int i = lane % 4; i < C; i += 4) remote_st(remote(&ts.keys[rank][tid / 4], i), k);
    }
    if (C > 1) {
        cluster_arrive();
        if (!all && rank != 0) return;
        cluster_wait();
    } else {
        __syncthreads();
    }
    if (tid < 32) {
        LpPart q = {-INFINITY, 0.f, 0.f, 0};
        if (lane < C * SC_WARPS) q = parts[lane];
        Run u = {q.m, q.s, q.t};
        LpRow row;
        row.m = warp_max(u.m);
        to_max(u, row.m, p.c);
        row.s = warp_sum(u.s);
        row.t = warp_sum(u.t);
        row.ahead = __reduce_add_sync(~0u, q.ahead);
        row.bound = p.top_n ? bound_of(ts, row.m, p.top_n, C) : 0;
        if (lane == 0) s_row = row;
    }
    __syncthreads();
    const LpRow row = s_row;
    if (!(row.m > -INFINITY && row.m < INFINITY)) {
        no_logprobs<E>(p, r, SPEC_ROW_NONFINITE, rank, C);
        return;
    }
    const float logz = logf(row.s), ent = logz - LN2 * (row.t / row.s);
    if (rank == 0 && tid == 0) {
        p.row_status[r] = SPEC_ROW_OK;
        if (p.logprob) p.logprob[r] = (xt - row.m) * p.inv_temp - logz;
        if (p.rank) p.rank[r] = row.ahead;
        if (p.entropy) p.entropy[r] = ent;
        if (p.lse) p.lse[r] = row.m * p.inv_temp + logz;
    }
    if (p.top_n) {
        give_candidates(sl, ts, row.bound, my_key, p.top_n, rank, C);
        if (C > 1) cluster_arrive();
        else __syncthreads();
    }
    if (GRAD) {
        // e (A + B d), e = 2^d: p = e / s, ln p = d ln 2 - ln s
        const float gl = p.g_logprob ? p.g_logprob[r] : 0.f, gh = p.g_entropy ? p.g_entropy[r] : 0.f;
        const float f = p.inv_temp / row.s, A = -(gl + gh * (ent - logz)) * f, B = -gh * LN2 * f;
        const uint64_t A2 = pair(A, A), B2 = pair(B, B);
        E* g = grad_of<E>(p, r);
        if (p.g_entropy)
            grad_slice(sl, g, row.m, p.c, [&](float a, float z, uint64_t e2) {
                return mul2(e2, fma2(B2, pair(fmaxf(a, NONE), fmaxf(z, NONE)), A2));
            });
        else
            grad_slice(sl, g, row.m, p.c, [&](float, float, uint64_t e2) { return mul2(e2, A2); });
        if (p.g_logprob && sl.has(id)) {
            __syncthreads();
            if (tid == 0) {
                const float d = (xt - row.m) * p.c, e = ex2_fast(d);
                g[id] = narrow<E>(gl * p.inv_temp + e * (A + B * fmaxf(d, NONE)));
            }
        }
    }
    if (p.top_n && rank == 0) {
        if (C > 1) cluster_wait();
        write_top(p, r, ts, row, logz, C);
    }
}

// ---- distillation ------------------------------------------------------------ //
__device__ __forceinline__ float teacher_value(const ScoreParams& p, int64_t at)
{
    return p.teacher_dtype == SPEC_F32 ? ((const float*)p.teacher)[at]
           : p.teacher_dtype == SPEC_BF16 ? __bfloat162float(((const __nv_bfloat16*)p.teacher)[at])
                                          : __half2float(((const __half*)p.teacher)[at]);
}

// the sums of a warp: tokens without an entry (the rest) and entries, each with its own maximum, as the rest of a
// confident row may be far below what fp32 holds beside the entries
struct KdPart {
    float mr, me, sr, se;
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

constexpr int SC_EPT = SPEC_SCORE_MAX_ENTRIES / SC_NT;  // entries of a thread: tid, tid + SC_NT

template <typename E, bool GRAD> __global__ void __launch_bounds__(SC_NT) k_score_distill(const ScoreParams p)
{
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ __align__(16) int32_t ids[SPEC_SCORE_MAX_ENTRIES];
    __shared__ float vals[SPEC_SCORE_MAX_ENTRIES];  // CTA 0: the student's logits at the entries
    __shared__ KdPart parts[SC_PARTS];
    __shared__ KdRow s_row;
    __shared__ float w_max[SC_WARPS], w_sum[SC_WARPS], w_acc[SC_WARPS];
    __shared__ double w_part[SC_WARPS][3];
    const int C = p.cluster, rank = (int)cluster_rank(), r = cluster_id(), tid = threadIdx.x, lane = tid % 32;
    const int k = p.k;
    int id[SC_EPT];
    bool some = false;
#pragma unroll
    for (int u = 0; u < SC_EPT; ++u) {
        const int i = tid + u * SC_NT;
        ids[i] = id[u] = i < k ? p.ids[(int64_t)r * k + i] : -1;
        some |= id[u] != -1;
    }
    if (!__syncthreads_or(some)) {
        no_distill<E>(p, r, SPEC_ROW_OK, rank, C);
        return;
    }
    const Slice<E> sl(p, row_of<E>(p, r), rank, smem);
    sl.copy();
    // the teacher, while the row is on its way: ln q_i = y_i - nq
    const float lse = p.teacher_lse ? p.teacher_lse[r] : 0.f;
    float tv[SC_EPT], tmax = -INFINITY;
    bool bad = false;
#pragma unroll
    for (int u = 0; u < SC_EPT; ++u) {
        const int i = tid + u * SC_NT;
        tv[u] = -INFINITY;
        if (id[u] == -1) continue;
        bad |= id[u] < -1 || id[u] >= p.V;
        tv[u] = teacher_value(p, (int64_t)r * k + i);
        tmax = fmax_nan(tmax, tv[u]);
        for (int j = 0; j < i; j += 4) {
            const int4 o = *(const int4*)(ids + j);
            bad |= o.x == id[u] || (o.y == id[u] && j + 1 < i) || (o.z == id[u] && j + 2 < i) ||
                   (o.w == id[u] && j + 3 < i);
        }
    }
    tmax = warp_max(tmax);
    if (lane == 0) w_max[tid / 32] = tmax;
    bad = __syncthreads_or(bad);
#pragma unroll
    for (int i = 0; i < SC_WARPS; ++i) tmax = fmax_nan(tmax, w_max[i]);
    if (bad || !(tmax < INFINITY) || (!p.tail && tmax == -INFINITY) || !(fabsf(lse) < INFINITY)) {
        sl.arrived(0);
        no_distill<E>(p, r, bad ? SPEC_ROW_BAD_TOKEN : SPEC_ROW_NONFINITE, rank, C);
        return;
    }
    if (C > 1) cluster_arrive();  // every CTA of the cluster runs before another stores into its shared memory
    // q up to the row's sum: differences first, and 1 / t in two parts, as the values may be large
    float q[SC_EPT], sum = 0.f;
#pragma unroll
    for (int u = 0; u < SC_EPT; ++u) {
        q[u] = 0.f;
        if (tv[u] > -INFINITY)
            q[u] = expf(p.tail ? fmaf(tv[u], p.inv_tt_lo, fmaf(tv[u], p.inv_tt, -lse))
                               : fmaf(tv[u] - tmax, p.inv_tt_lo, (tv[u] - tmax) * p.inv_tt));
        sum += q[u];
    }
    sum = warp_sum(sum);
    if (lane == 0) w_sum[tid / 32] = sum;
    // the entries' logits leave the row
    sl.arrived(0);
    __syncthreads();
    sum = 0.f;
#pragma unroll
    for (int i = 0; i < SC_WARPS; ++i) sum += w_sum[i];
    float l[SC_EPT], me = -INFINITY;
    bool mine[SC_EPT];
#pragma unroll
    for (int u = 0; u < SC_EPT; ++u) {
        mine[u] = id[u] >= 0 && sl.has(id[u]);
        l[u] = -INFINITY;
        if (mine[u]) {
            l[u] = value_of<E>(*sl.at(id[u]));
            *sl.at(id[u]) = (Bits<E>)Vec<E>::NEG;
        }
        me = fmax_nan(me, l[u]);
        if (!p.tail) q[u] /= sum;
    }
    __syncthreads();
    Summer<E, false, false> rest;
    rest.c2 = pair(p.c, p.c);
    rest.l2 = pair(p.c_lo, p.c_lo);
    Run run = rest.run(sl, false);
    KdPart w;
    w.mr = warp_max(run.m);
    to_max(run, w.mr, p.c);
    w.sr = warp_sum(run.s);
    w.me = warp_max(me);
    w.se = 0.f;
#pragma unroll
    for (int u = 0; u < SC_EPT; ++u) w.se += ex2_fast((l[u] - ref_of(w.me)) * p.c);
    w.se = warp_sum(w.se);
    if (C > 1) cluster_wait();
    if (lane < (GRAD ? C : 1)) {
        const uint32_t to = remote(parts + rank * SC_WARPS + tid / 32, lane);
        remote_st(to, __float_as_uint(w.mr));
        remote_st(to + 4, __float_as_uint(w.me));
        remote_st(to + 8, __float_as_uint(w.sr));
        remote_st(to + 12, __float_as_uint(w.se));
    }
#pragma unroll
    for (int u = 0; u < SC_EPT; ++u)
        if (mine[u]) remote_st(remote(vals + tid + u * SC_NT, 0), __float_as_uint(l[u]));
    if (C > 1) {
        cluster_arrive();
        if (!GRAD && rank != 0) return;
        cluster_wait();
    } else {
        __syncthreads();
    }
    if (tid < 32) {
        KdPart u = {-INFINITY, -INFINITY, 0.f, 0.f};
        if (lane < C * SC_WARPS) u = parts[lane];
        KdRow row;
        row.mr = warp_max(u.mr);
        row.m = fmax_nan(row.mr, warp_max(u.me));
        row.sr = warp_sum(u.mr == -INFINITY ? 0.f : u.sr * exp2f((u.mr - row.mr) * p.c));
        const float in_e = warp_sum(u.me == -INFINITY ? 0.f : u.se * exp2f((u.me - row.m) * p.c));
        row.scale = row.mr == -INFINITY ? 0.f : exp2f((row.mr - row.m) * p.c);
        row.z = row.sr * row.scale + in_e;
        row.inv_z = 1.f / row.z;
        row.inv_sr = row.sr > 0.f ? 1.f / row.sr : 0.f;
        if (lane == 0) s_row = row;
    }
    __syncthreads();
    const KdRow row = s_row;
    if (!(row.m > -INFINITY && row.m < INFINITY)) {
        no_distill<E>(p, r, SPEC_ROW_NONFINITE, rank, C);
        return;
    }
    if (GRAD) {
        const float in_q = p.tail ? sum : 1.f, qr = p.tail ? fmaxf(0.f, 1.f - sum) : 0.f;
        const float gl = (p.g_loss ? p.g_loss[r] : 1.f) * p.inv_temp, ps = (in_q + qr) * row.inv_z;
        const float pr = gl * (ps * row.scale - qr * row.inv_sr);
        const uint64_t pr2 = pair(pr, pr);
        E* g = grad_of<E>(p, r);
        grad_slice(sl, g, row.mr, p.c, [&](float, float, uint64_t e2) { return mul2(e2, pr2); });
        __syncthreads();
#pragma unroll
        for (int u = 0; u < SC_EPT; ++u)
            if (mine[u]) g[id[u]] = narrow<E>(gl * (ps * ex2_fast((l[u] - row.m) * p.c) - q[u]));
    }
    if (rank != 0) return;
    // The row's loss: near its minimum a small difference of terms of the size of ln Z, which are taken in 64 bits.
    // That pipe takes 16 cycles for a warp's instruction: the entries' warps alone use it, and exponentials and
    // logarithms are one each, of different values in a warp's lanes.
    float acc = 0.f;
    double part = 0.0, in_q = 0.0, in_e = 0.0;
#pragma unroll
    for (int u = 0; u < SC_EPT; ++u) {
        if (tid / 32 * 32 + u * SC_NT >= k) continue;
        const float li = id[u] >= 0 ? vals[tid + u * SC_NT] : -INFINITY;
        const float e = exp2f(fmaf(li - row.m, p.c, (li - row.m) * p.c_lo));
        const double lq = p.tail ? (double)tv[u] * p.inv_tt_d - (double)lse : ((double)tv[u] - (double)tmax) * p.inv_tt_d;
        if (q[u] > 0.f) part += q[u] * (lq - ((double)li - (double)row.m) * p.inv_temp_d);
        in_q += q[u];
        in_e += e;
        acc += fminf(q[u], e * row.inv_z);
    }
    acc = warp_sum(acc);
    if (tid / 32 * 32 < k) {
        part = warp_sum(part);
        in_q = warp_sum(in_q);
        in_e = warp_sum(in_e);
    }
    if (lane == 0) {
        w_acc[tid / 32] = acc;
        w_part[tid / 32][0] = part;
        w_part[tid / 32][1] = in_q;
        w_part[tid / 32][2] = in_e;
    }
    __syncthreads();
    if (tid >= 32) return;
    // lane i: the share that warp i's sum of the rest has
    const KdPart u = lane < C * SC_WARPS ? parts[lane] : KdPart{-INFINITY, -INFINITY, 0.f, 0.f};
    double in_r = 0.0;
    if (u.mr > -INFINITY) in_r = u.sr * exp(((double)u.mr - (double)row.mr) * p.inv_temp_d);
    in_r = warp_sum(in_r);
    const double shift = in_r > 0.0 ? ((double)row.mr - (double)row.m) * p.inv_temp_d : 0.0;
    double loss = 0.0, in = 0.0, z = in_r > 0.0 ? in_r * exp(shift) : 0.0;
    for (int i = 0; i < SC_WARPS; ++i) {
        loss += w_part[i][0];
        in += w_part[i][1];
        z += w_part[i][2];
    }
    const double left = p.tail ? fmax(0.0, 1.0 - in) : 0.0;
    const double ln = log(lane == 0 ? z : lane == 1 ? in_r : lane == 2 ? left : (double)sum);
    const double ln_r = __shfl_sync(~0u, ln, 1), ln_left = __shfl_sync(~0u, ln, 2), ln_sum = __shfl_sync(~0u, ln, 3);
    if (lane == 0) {
        loss += in * (p.tail ? ln : ln - ln_sum);
        if (left > 0.0) loss += in_r > 0.0 ? left * (ln_left + ln - ln_r - shift) : (double)INFINITY;
        p.row_status[r] = SPEC_ROW_OK;
        if (p.loss) p.loss[r] = (float)loss;
        if (p.accept) p.accept[r] = w_acc[0] + w_acc[1] + w_acc[2] + w_acc[3];
    }
}

// ---- launches ------------------------------------------------------------------ //
// CTAs of a row.  A slice of at most SLICE bytes leaves room for four CTAs on an SM, so that some copy while others
// compute; rows beyond eight of them have larger slices.  Few rows are spread over up to eight CTAs, for the SMs
// that would idle, while every thread still has a vector or two; and the search for the top tokens wants twice as
// many groups of threads (32 a CTA) as tokens.
constexpr int SLICE = 52 * 1024, SLICE_TOP = 46 * 1024;

template <typename K>
cudaError_t go(K kernel, DeviceOnce& once, ScoreParams p, size_t size, size_t scratch, int num_sms, cudaStream_t s)
{
    const size_t limit = SCORE_MAX_ROW_BYTES / SC_MAXC + 64 + scratch;
    const int row = (int)(((size_t)p.V * size + 30) / 16);  // vectors, at any alignment
    const int most = (p.top_n ? SLICE_TOP : SLICE) / 16;
    int C = (row + most - 1) / most;
    C = C > SC_MAXC ? SC_MAXC : C;
    while (C < SC_MAXC && (C * 16 < p.top_n || ((int64_t)p.rows * C < num_sms && row / (C + 1) >= SC_NT))) ++C;
    p.cluster = C;
    p.per = (row + C - 1) / C;
    p.top_at = p.per * 16;
    p.by_tokens = FastDiv(p.T);
    const cudaError_t e = cuda_once(once, nullptr, [&](int, int*) {
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)limit);
    });
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)p.rows * C);
    cfg.blockDim = dim3(SC_NT);
    cfg.dynamicSmemBytes = (size_t)p.per * 16 + (p.top_n ? scratch : 0);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = C;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <typename E> cudaError_t go_logprobs(const ScoreParams& p, int num_sms, cudaStream_t s)
{
    static DeviceOnce once[2];
    return p.grad ? go(k_score_logprobs<E, true>, once[1], p, sizeof(E), sizeof(TopScratch), num_sms, s)
                  : go(k_score_logprobs<E, false>, once[0], p, sizeof(E), sizeof(TopScratch), num_sms, s);
}
template <typename E> cudaError_t go_distill(const ScoreParams& p, int num_sms, cudaStream_t s)
{
    static DeviceOnce once[2];
    return p.grad ? go(k_score_distill<E, true>, once[1], p, sizeof(E), 0, num_sms, s)
                  : go(k_score_distill<E, false>, once[0], p, sizeof(E), 0, num_sms, s);
}

}  // namespace

cudaError_t launch_score_logprobs(const ScoreParams& p, int dtype, int num_sms, cudaStream_t s)
{
    return dtype == SPEC_F32 ? go_logprobs<float>(p, num_sms, s)
           : dtype == SPEC_BF16 ? go_logprobs<__nv_bfloat16>(p, num_sms, s)
                                : go_logprobs<__half>(p, num_sms, s);
}

cudaError_t launch_score_distill(const ScoreParams& p, int dtype, int num_sms, cudaStream_t s)
{
    return dtype == SPEC_F32 ? go_distill<float>(p, num_sms, s)
           : dtype == SPEC_BF16 ? go_distill<__nv_bfloat16>(p, num_sms, s)
                                : go_distill<__half>(p, num_sms, s);
}

}  // namespace sv
