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

constexpr int SC_NT = 256;      // threads of a CTA
constexpr int SC_WARPS = SC_NT / 32;
constexpr int SC_BATCH = 4;     // vectors of a thread per copy group
constexpr int SC_MAXC = 8;      // CTAs of a cluster (portable)
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
    int nb;           // copy groups of a thread
    int V;

    __device__ __forceinline__ Slice(const ScoreParams& p, const E* x, int rank, int C, void* smem)
    {
        const int mis = (int)((uintptr_t)x & 15);
        const int all = (int)((mis + (int64_t)p.V * (int)sizeof(E) + 15) / 16), per = (all + C - 1) / C;
        const int v0 = min(rank * per, all);
        n = min(per, all - v0);
        first = v0 * EPV<E> - mis / (int)sizeof(E);
        src = (const char*)x - mis + (int64_t)v0 * 16;
        nb = (n + SC_NT * SC_BATCH - 1) / (SC_NT * SC_BATCH);
        buf = (uint4*)smem;
        V = p.V;
    }
    // a vector that lies in the row as a whole
    __device__ __forceinline__ bool whole(int i) const
    {
        const int e = first + i * EPV<E>;
        return e >= 0 && e <= V - EPV<E>;
    }
    __device__ __forceinline__ bool has(int id) const { return id >= first && id < first + n * EPV<E> && id < V; }
    __device__ __forceinline__ Bits<E>* at(int id) const { return (Bits<E>*)buf + (id - first); }

    __device__ __forceinline__ void copy() const
    {
        const uint32_t to = (uint32_t)__cvta_generic_to_shared(buf);
        for (int b = 0; b < nb; ++b) {
#pragma unroll
            for (int j = 0; j < SC_BATCH; ++j) {
                const int i = (b * SC_BATCH + j) * SC_NT + threadIdx.x;
                if (i >= n) continue;
                if (whole(i)) {
                    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16;" ::"r"(to + i * 16),
                                 "l"(src + (int64_t)i * 16)
                                 : "memory");
                } else {
                    const int e = first + i * EPV<E>;
                    const Bits<E>* from = (const Bits<E>*)(src + (int64_t)i * 16);
                    Bits<E> v[EPV<E>];
#pragma unroll
                    for (int q = 0; q < EPV<E>; ++q) v[q] = e + q >= 0 && e + q < V ? from[q] : (Bits<E>)Vec<E>::NEG;
                    buf[i] = vector_of<E>(v);
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        }
    }
    // this thread's copies of groups 0 .. b have arrived (later ones may have, too)
    __device__ __forceinline__ void arrived(int b) const
    {
        switch (nb - 1 - b) {
        case 0: asm volatile("cp.async.wait_group 0;" ::: "memory"); break;
        case 1: asm volatile("cp.async.wait_group 1;" ::: "memory"); break;
        case 2: asm volatile("cp.async.wait_group 2;" ::: "memory"); break;
        case 3: asm volatile("cp.async.wait_group 3;" ::: "memory"); break;
        default: asm volatile("cp.async.wait_group 4;" ::: "memory"); break;
        }
    }
    __device__ __forceinline__ void arrived_all() const { asm volatile("cp.async.wait_group 0;" ::: "memory"); }
};

// a running softmax: maximum, sum of 2^d, sum of d 2^d, d relative to the maximum
struct Run {
    float m, s, t;
};
__device__ __forceinline__ float ref_of(float m) { return m == -INFINITY ? 0.f : m; }

// sums of a thread's vectors, by ENTROPY those of d 2^d too; without it c is taken in two parts (c + c_lo, c_lo > 0),
// since a loss near its minimum shows the constant's rounding; with RANK also the number of elements above x (in
// vectors before tvec: or equal to it, written as above the next value below x)
template <typename E, bool ENTROPY, bool RANK>
__device__ __forceinline__ Run sum_slice(const Slice<E>& sl, float c, float c_lo, bool waits, int tvec, float x, float x_below,
                                         int& ahead)
{
    float m = -INFINITY;
    uint64_t s2 = pair(0.f, 0.f), t2 = s2;
    const uint64_t c2 = pair(c, c), l2 = pair(c_lo, c_lo);
    const typename Vec<E>::Thr at = Vec<E>::thr_of(x), under = Vec<E>::thr_of(x_below);
    for (int b = 0; b < sl.nb; ++b) {
        if (waits) sl.arrived(b);
        uint4 w[SC_BATCH];
        float mx = -INFINITY;
#pragma unroll
        for (int j = 0; j < SC_BATCH; ++j) {
            const int i = (b * SC_BATCH + j) * SC_NT + threadIdx.x;
            w[j] = i < sl.n ? sl.buf[i] : make_uint4(Vec<E>::NEG, Vec<E>::NEG, Vec<E>::NEG, Vec<E>::NEG);
            mx = fmax_nan(mx, Vec<E>::top(w[j]));
        }
        if (!(mx <= m)) {  // a new maximum (or NaN, which stays): rescale
            mx = fmax_nan(m, mx);
            if (m > -INFINITY) {
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
        for (int j = 0; j < SC_BATCH; ++j) {
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
            if (RANK) {
                const int i = (b * SC_BATCH + j) * SC_NT + threadIdx.x;
                ahead += Vec<E>::above(w[j], i < tvec ? under : at);
            }
        }
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
// reductions over the CTA in a fixed order; every thread gets the result
template <typename X, typename F> __device__ __forceinline__ X block_reduce(X x, F op)
{
    __shared__ X part[SC_WARPS];
    x = warp_reduce(x, op);
    __syncthreads();
    if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = x;
    __syncthreads();
    x = part[0];
#pragma unroll
    for (int i = 1; i < SC_WARPS; ++i) x = op(x, part[i]);
    return x;
}
template <typename X> __device__ __forceinline__ X block_sum(X x)
{
    return block_reduce(x, [](X a, X b) { return a + b; });
}
__device__ __forceinline__ float block_max(float x)
{
    return block_reduce(x, [](float a, float b) { return fmax_nan(a, b); });
}

template <typename E> __device__ const E* row_of(const ScoreParams& p, int r)
{
    return (const E*)p.x + (int64_t)(r / p.T) * p.x_seq + (int64_t)(r % p.T) * p.x_tok;
}
template <typename E> __device__ E* grad_of(const ScoreParams& p, int r)
{
    return (E*)p.grad + (int64_t)(r / p.T) * p.g_seq + (int64_t)(r % p.T) * p.g_tok;
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

// the gradient of a slice: f(logits of a pair, as distances d from -ref times c, and 2^d) -> pair
template <typename E, typename F>
__device__ __forceinline__ void grad_slice(const Slice<E>& sl, E* g, float m, float c, F f)
{
    const float ref = -ref_of(m);
    const uint64_t r2 = pair(ref, ref), c2 = pair(c, c);
    E* out = g + sl.first;  // its element at the slice's start
    const bool straight = ((uintptr_t)out & 15) == 0;
    for (int i = threadIdx.x; i < sl.n; i += SC_NT) {
        uint64_t v[EPV<E> / 2], y[EPV<E> / 2];
        Vec<E>::pairs(sl.buf[i], v);
#pragma unroll
        for (int q = 0; q < EPV<E> / 2; ++q) {
            const uint64_t d2 = mul2(add2(v[q], r2), c2);
            float a, z;
            unpair(d2, a, z);
            y[q] = f(a, z, pair(ex2_fast(a), ex2_fast(z)));
        }
        const uint4 w = Vec<E>::pack(y);
        if (straight && sl.whole(i)) ((uint4*)out)[i] = w;
        else sl.buf[i] = w;
        if (straight && !sl.whole(i)) {
            const int e = sl.first + i * EPV<E>;
#pragma unroll
            for (int q = 0; q < EPV<E>; ++q)
                if (e + q >= 0 && e + q < sl.V) ((Bits<E>*)g)[e + q] = bits_at<E>(w, q);
        }
    }
    if (straight) return;
    // the gradient's rows start elsewhere in a vector than the logits': elements change vectors on the way out
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
struct LpPart {      // what a CTA knows of the row
    float m, s, t;
    int32_t ahead;
    uint32_t kmin;   // the smallest of its threads' largest keys, of those with an unmasked token
};
struct LpRow {
    float m, s, t;
    int32_t ahead;
    uint32_t kmin;
};

// scratch of the search for the top tokens, behind the slice
struct TopScratch {
    uint32_t keys[SC_MAXC][SC_NT];      // the largest key of every thread of the cluster
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
    if (my_key >= bound)
        each_mine(sl, [&](uint32_t key, int id) {
            if (key >= bound) give(key, id);
        });
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

// a key that at least n (all, if fewer) of the row's unmasked tokens reach, and not many more: at least n threads'
// largest do, by halving the range of keys until their number is near n
__device__ uint32_t bound_of(TopScratch& ts, const LpRow& row, int n, int C)
{
    uint32_t lo = row.kmin, hi = key_of(row.m), mid = lo;
    uint32_t mine[SC_MAXC];
#pragma unroll
    for (int i = 0; i < SC_MAXC; ++i) mine[i] = i < C ? ts.keys[i][threadIdx.x] : 0;
    for (int round = 0;; ++round) {
        int k = 0;
#pragma unroll
        for (int i = 0; i < SC_MAXC; ++i) k += mine[i] >= mid;
        k = tally_of(ts, round, k);
        // fewer than n threads have an unmasked token at all: every unmasked token is a candidate
        if (round == 0 && k < n) return KEY_NEG_INF + 1;
        if (k < n) hi = mid - 1;
        else lo = mid;
        if (lo >= hi || (k >= n && k <= n + n / 4 + 8)) return lo;
        mid = lo + (hi - lo + 1) / 2;
    }
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

template <typename E, bool GRAD> __global__ void __launch_bounds__(SC_NT, 4) k_score_logprobs(const ScoreParams p)
{
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ LpPart parts[SC_MAXC];
    __shared__ float w_m[SC_WARPS], w_s[SC_WARPS], w_t[SC_WARPS];
    __shared__ int w_a[SC_WARPS];
    __shared__ uint32_t w_k[SC_WARPS];
    __shared__ LpRow s_row;
    const int C = p.cluster, rank = (int)cluster_rank(), r = blockIdx.x / C, tid = threadIdx.x, lane = tid % 32;
    const int id = p.ids ? p.ids[r] : 0;
    if (id < 0 || id >= p.V) {
        no_logprobs<E>(p, r, id == -1 ? SPEC_ROW_OK : SPEC_ROW_BAD_TOKEN, rank, C);
        return;
    }
    const E* x = row_of<E>(p, r);
    const Slice<E> sl(p, x, rank, C, smem);
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
        const int tvec = (id - sl.first) >> (sizeof(E) == 4 ? 2 : 3);
        // a masked token: those in front are the unmasked ones
        run = sum_slice<E, true, true>(sl, p.c, 0.f, true, tvec, xt, xt == -INFINITY ? xt : below<E>(raw), ahead);
        if (tvec >= 0 && tvec < sl.n && tvec % SC_NT == tid && xt > -INFINITY)
            for (int q = 0; q < id - sl.first - tvec * EPV<E>; ++q)
                ahead += value_of<E>(bits_at<E>(sl.buf[tvec], q)) == xt;
    } else {
        run = sum_slice<E, true, false>(sl, p.c, 0.f, true, 0, 0.f, 0.f, ahead);
        if (p.rank) {  // with a gradient, where the loop above has no room for it
            each_mine(sl, [&](uint32_t key, int v) {
                const uint32_t k = key_of(xt);
                ahead += key > k || (key == k && v < id && key > KEY_NEG_INF);
            });
        }
    }
    const float my_max = run.m;
    const uint32_t my_key = key_of(my_max);
    // threads to CTA
    float m = warp_reduce(run.m, [](float a, float b) { return fmax_nan(a, b); });
    if (lane == 0) w_m[tid / 32] = m;
    __syncthreads();
    m = w_m[0];
#pragma unroll
    for (int i = 1; i < SC_WARPS; ++i) m = fmax_nan(m, w_m[i]);
    to_max(run, m, p.c);
    run.s = warp_reduce(run.s, [](float a, float b) { return a + b; });
    run.t = warp_reduce(run.t, [](float a, float b) { return a + b; });
    ahead = __reduce_add_sync(~0u, ahead);
    const uint32_t kmin = p.top_n ? __reduce_min_sync(~0u, my_key > KEY_NEG_INF ? my_key : ~0u) : 0;
    if (lane == 0) {
        w_s[tid / 32] = run.s;
        w_t[tid / 32] = run.t;
        w_a[tid / 32] = ahead;
        w_k[tid / 32] = kmin;
    }
    __syncthreads();
    // CTA to cluster: to CTA 0, or (what comes next needs the row's sum, or a bound) to all
    const bool all = GRAD || p.top_n;
    if (C > 1) cluster_wait();
    if (tid < (all ? C : 1)) {
        LpPart q = {m, 0.f, 0.f, 0, ~0u};
#pragma unroll
        for (int i = 0; i < SC_WARPS; ++i) {
            q.s += w_s[i];
            q.t += w_t[i];
            q.ahead += w_a[i];
            q.kmin = min(q.kmin, w_k[i]);
        }
        const uint32_t to = remote(parts + rank, tid);
        remote_st(to, __float_as_uint(q.m));
        remote_st(to + 4, __float_as_uint(q.s));
        remote_st(to + 8, __float_as_uint(q.t));
        remote_st(to + 12, (uint32_t)q.ahead);
        remote_st(to + 16, q.kmin);
    }
    if (p.top_n)
        for (int i = 0; i < C; ++i) remote_st(remote(&ts.keys[rank][tid], i), my_key);
    if (C > 1) {
        cluster_arrive();
        if (!all && rank != 0) return;
        cluster_wait();
    } else {
        __syncthreads();
    }
    if (tid < 32) {
        LpPart q = {-INFINITY, 0.f, 0.f, 0, ~0u};
        if (lane < C) q = parts[lane];
        Run u = {q.m, q.s, q.t};
        LpRow row;
        row.m = warp_reduce(u.m, [](float a, float b) { return fmax_nan(a, b); });
        to_max(u, row.m, p.c);
        row.s = warp_reduce(u.s, [](float a, float b) { return a + b; });
        row.t = warp_reduce(u.t, [](float a, float b) { return a + b; });
        row.ahead = __reduce_add_sync(~0u, q.ahead);
        row.kmin = __reduce_min_sync(~0u, q.kmin);
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
        give_candidates(sl, ts, bound_of(ts, row, p.top_n, C), my_key, p.top_n, rank, C);
        if (C > 1) cluster_arrive();
        else __syncthreads();
    }
    if (GRAD) {
        // e (A + B d), e = 2^d: p = e / s, ln p = d ln 2 - ln s
        const float gl = p.g_logprob ? p.g_logprob[r] : 0.f, gh = p.g_entropy ? p.g_entropy[r] : 0.f;
        const float f = p.inv_temp / row.s, A = -(gl + gh * (ent - logz)) * f, B = -gh * LN2 * f;
        const uint64_t A2 = pair(A, A), B2 = pair(B, B);
        E* g = grad_of<E>(p, r);
        grad_slice(sl, g, row.m, p.c, [&](float a, float z, uint64_t e2) {
            return mul2(e2, fma2(B2, pair(fmaxf(a, NONE), fmaxf(z, NONE)), A2));
        });
        if (p.g_logprob && sl.has(id)) {
            __syncthreads();
            if (tid == 0) {
                const float d = (xt - row.m) * p.c, e = ex2_fast(d);
                g[id] = narrow<E>(gl * p.inv_temp + e * (A + B * fmaxf(d, NONE)));
            }
        }
    }
    if (p.top_n && C > 1 && rank == 0) cluster_wait();
    if (p.top_n && rank == 0) write_top(p, r, ts, row, logz, C);
}

// ---- distillation ------------------------------------------------------------ //
__device__ __forceinline__ float teacher_value(const ScoreParams& p, int64_t at)
{
    return p.teacher_dtype == SPEC_F32 ? ((const float*)p.teacher)[at]
           : p.teacher_dtype == SPEC_BF16 ? __bfloat162float(((const __nv_bfloat16*)p.teacher)[at])
                                          : __half2float(((const __half*)p.teacher)[at]);
}

// the sums of a CTA's slice: tokens without an entry (the rest) and entries, each with its own maximum, as the rest
// of a confident row may be far below what fp32 holds beside the entries
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

template <typename E, bool GRAD> __global__ void __launch_bounds__(SC_NT, 4) k_score_distill(const ScoreParams p)
{
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ __align__(16) int32_t ids[SPEC_SCORE_MAX_ENTRIES];
    __shared__ float vals[SPEC_SCORE_MAX_ENTRIES];  // CTA 0: the student's logits at the entries
    __shared__ float sums[SC_MAXC][SC_WARPS];       // CTA 0: the sums of the slices' warps
    __shared__ KdPart parts[SC_MAXC];
    __shared__ KdRow s_row;
    const int C = p.cluster, rank = (int)cluster_rank(), r = blockIdx.x / C, tid = threadIdx.x, lane = tid % 32;
    const int k = p.k;
    const int64_t at = (int64_t)r * k + tid;
    const int id = tid < k ? p.ids[at] : -1;
    if (!__syncthreads_or(id != -1)) {
        no_distill<E>(p, r, SPEC_ROW_OK, rank, C);
        return;
    }
    const Slice<E> sl(p, row_of<E>(p, r), rank, C, smem);
    sl.copy();
    // the teacher, while the row is on its way: ln q_i = y_i - nq
    ids[tid] = id;
    const float tv = id >= 0 ? teacher_value(p, at) : -INFINITY, lse = p.teacher_lse ? p.teacher_lse[r] : 0.f;
    const float tmax = block_max(tv);
    bool bad = id < -1 || id >= p.V;
    if (id >= 0)
        for (int j = 0; j < tid; j += 4) {
            const int4 o = *(const int4*)(ids + j);
            bad |= o.x == id || (o.y == id && j + 1 < tid) || (o.z == id && j + 2 < tid) || (o.w == id && j + 3 < tid);
        }
    bad = __syncthreads_or(bad);
    const bool dull = !(tmax < INFINITY) || (!p.tail && tmax == -INFINITY) || !(fabsf(lse) < INFINITY);
    if (bad || dull) {
        sl.arrived_all();
        no_distill<E>(p, r, bad ? SPEC_ROW_BAD_TOKEN : SPEC_ROW_NONFINITE, rank, C);
        return;
    }
    if (C > 1) cluster_arrive();  // every CTA of the cluster runs before another stores into its shared memory
    // ln q up to the row's sum: differences first, and 1 / t in two parts, as the values may be large
    float w = 0.f;
    if (tv > -INFINITY)
        w = expf(p.tail ? fmaf(tv, p.inv_tt_lo, fmaf(tv, p.inv_tt, -lse))
                        : fmaf(tv - tmax, p.inv_tt_lo, (tv - tmax) * p.inv_tt));
    const float sum = block_sum(w);
    const float q = p.tail ? w : w / sum, in_q = p.tail ? sum : 1.f, qr = p.tail ? fmaxf(0.f, 1.f - sum) : 0.f;
    // the entries' logits leave the row
    sl.arrived_all();
    __syncthreads();
    const bool mine = id >= 0 && sl.has(id);
    float l = -INFINITY;
    if (mine) {
        l = value_of<E>(*sl.at(id));
        *sl.at(id) = (Bits<E>)Vec<E>::NEG;
    }
    __syncthreads();
    int none = 0;
    Run run = sum_slice<E, false, false>(sl, p.c, p.c_lo, false, 0, 0.f, 0.f, none);
    const float mr = block_max(run.m), me = block_max(l);
    to_max(run, mr, p.c);
    // (a warp's sum goes to CTA 0 as it is: there the loss takes them in 64 bits)
    const float sw = warp_reduce(run.s, [](float a, float b) { return a + b; });
    const float sr = block_sum(lane == 0 ? sw : 0.f);
    const float se = block_sum(ex2_fast((l - ref_of(me)) * p.c));
    if (C > 1) cluster_wait();
    if (tid < (GRAD ? C : 1)) {
        const uint32_t to = remote(parts + rank, tid);
        remote_st(to, __float_as_uint(mr));
        remote_st(to + 4, __float_as_uint(me));
        remote_st(to + 8, __float_as_uint(sr));
        remote_st(to + 12, __float_as_uint(se));
    }
    if (mine) remote_st(remote(vals + tid, 0), __float_as_uint(l));
    if (lane == 0) remote_st(remote(&sums[rank][tid / 32], 0), __float_as_uint(sw));
    if (C > 1) {
        cluster_arrive();
        if (!GRAD && rank != 0) return;
        cluster_wait();
    } else {
        __syncthreads();
    }
    if (tid < 32) {
        KdPart u = {-INFINITY, -INFINITY, 0.f, 0.f};
        if (lane < C) u = parts[lane];
        auto max_of = [](float a, float b) { return fmax_nan(a, b); };
        auto sum_of = [](float a, float b) { return a + b; };
        KdRow row;
        row.mr = warp_reduce(u.mr, max_of);
        const float e = warp_reduce(u.me, max_of);
        row.m = fmax_nan(row.mr, e);
        row.sr = warp_reduce(u.mr == -INFINITY ? 0.f : u.sr * exp2f((u.mr - row.mr) * p.c), sum_of);
        const float in_e = warp_reduce(u.me == -INFINITY ? 0.f : u.se * exp2f((u.me - row.m) * p.c), sum_of);
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
        const float gl = (p.g_loss ? p.g_loss[r] : 1.f) * p.inv_temp, ps = (in_q + qr) * row.inv_z;
        const float pr = gl * (ps * row.scale - qr * row.inv_sr);
        const uint64_t pr2 = pair(pr, pr);
        E* g = grad_of<E>(p, r);
        grad_slice(sl, g, row.mr, p.c, [&](float, float, uint64_t e2) { return mul2(e2, pr2); });
        __syncthreads();
        if (mine) g[id] = narrow<E>(gl * (ps * ex2_fast((l - row.m) * p.c) - q));
    }
    if (rank != 0) return;
    // The row's loss: near its minimum a small difference of terms of the size of ln Z, which are taken in 64 bits.
    // That pipe takes 16 cycles for a warp's instruction: the entries' warps alone use it, and exponentials and
    // logarithms are one each, of different values in a warp's lanes.
    __shared__ double w_part[SC_WARPS][3];
    auto sum_of = [](double a, double b) { return a + b; };
    const float li = id >= 0 ? vals[tid] : -INFINITY;
    const float e = exp2f(fmaf(li - row.m, p.c, (li - row.m) * p.c_lo));
    if (tid < (k + 31) / 32 * 32) {
        const double lq = p.tail ? (double)tv * p.inv_tt_d - (double)lse : ((double)tv - (double)tmax) * p.inv_tt_d;
        const double part =
            warp_reduce(q > 0.f ? q * (lq - ((double)li - (double)row.m) * p.inv_temp_d) : 0.0, sum_of);
        const double in_q = warp_reduce((double)q, sum_of), in_e = warp_reduce((double)e, sum_of);
        if (lane == 0) {
            w_part[tid / 32][0] = part;
            w_part[tid / 32][1] = in_q;
            w_part[tid / 32][2] = in_e;
        }
    }
    const float acc = block_sum(fminf(q, e * row.inv_z));  // (its barriers are w_part's)
    if (tid >= 32) return;
    // lane i: CTA i's share of the rest; lane SC_MAXC: the rest's of the row
    const float from = lane < C ? parts[lane].mr : row.mr;
    const double scale = exp(((double)from - (double)(lane < SC_MAXC ? row.mr : row.m)) * p.inv_temp_d);
    double rest = 0.0;
    if (lane < C && from > -INFINITY) {
        for (int i = 0; i < SC_WARPS; ++i) rest += sums[lane][i];
        rest *= scale;
    }
    for (int i = 1; i < SC_MAXC; i *= 2) rest += __shfl_xor_sync(~0u, rest, i);
    rest = __shfl_sync(~0u, rest, 0);
    double loss = 0.0, in = 0.0, z = rest > 0.0 ? rest * __shfl_sync(~0u, scale, SC_MAXC) : 0.0;
    for (int i = 0; i < (k + 31) / 32; ++i) {
        loss += w_part[i][0];
        in += w_part[i][1];
        z += w_part[i][2];
    }
    const double left = p.tail ? fmax(0.0, 1.0 - in) : 0.0;
    const double ln = log(lane == 0 ? z : lane == 1 ? rest : lane == 2 ? left : (double)sum);
    const double ln_rest = __shfl_sync(~0u, ln, 1), ln_left = __shfl_sync(~0u, ln, 2), ln_sum = __shfl_sync(~0u, ln, 3);
    if (lane == 0) {
        loss += in * (p.tail ? ln : ln - ln_sum);
        if (left > 0.0)
            loss += rest > 0.0 ? left * (ln_left + ln - ln_rest - ((double)row.mr - (double)row.m) * p.inv_temp_d)
                               : (double)INFINITY;
        p.row_status[r] = SPEC_ROW_OK;
        if (p.loss) p.loss[r] = (float)loss;
        if (p.accept) p.accept[r] = acc;
    }
}

// ---- launches ------------------------------------------------------------------ //
// CTAs of a row.  A slice of at most SLICE bytes leaves room for four CTAs on an SM, so that some copy while others
// compute; rows beyond eight of them have larger slices.  Few rows are spread over up to eight CTAs, for the SMs
// that would idle, while a thread still has a vector to itself.
constexpr int SLICE = 52 * 1024, SLICE_TOP = 39 * 1024;

template <typename K>
cudaError_t go(K kernel, DeviceOnce& once, ScoreParams p, size_t size, size_t scratch, int num_sms, cudaStream_t s)
{
    const size_t limit = SCORE_MAX_ROW_BYTES / SC_MAXC + 64 + scratch;
    const size_t row = (size_t)p.V * size + 16;
    const int most = p.top_n ? SLICE_TOP : SLICE;
    int C = (int)((row + most - 1) / most);
    C = C > SC_MAXC ? SC_MAXC : C;
    while (C < SC_MAXC && (int64_t)p.rows * C < num_sms && row / (C + 1) >= SC_NT * 16) ++C;
    const size_t per = ((row + 15) / 16 + C - 1) / C;
    p.cluster = C;
    p.top_at = (int)(per * 16);
    const cudaError_t e = cuda_once(once, nullptr, [&](int, int*) {
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)limit);
    });
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)p.rows * C);
    cfg.blockDim = dim3(SC_NT);
    cfg.dynamicSmemBytes = per * 16 + (p.top_n ? scratch : 0);
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
