// sv_score_row.cuh -- device-side building blocks of the operators that score
// rows of logits: vectors of elements, slices of rows and their copies, running
// softmax sums, gradients, and the join of a cluster's warps.
//
// A row is taken by a cluster of 1 to 8 CTAs, a slice each.  A thread copies the
// vectors that it will read itself (cp.async), so that no barrier lies between a
// copy and its use: a ring of copy groups, where what it has used makes room for
// what comes.
//
//   forward    one cluster per row: five or six CTAs share an SM, and those that
//              stream keep HBM busy while others begin or end
//   gradient   the row's sum comes before the gradient's first element, so the
//              row is streamed twice, the second time in reverse: first what the
//              rings still hold, then the rest from L2, where as many rows are
//              under way as it has room for
//
// Slices are whole 16-byte vectors of the row's addresses, so rows of any
// alignment are copied and read alike; what a row's first and last vector have
// outside the row is -inf, which counts nowhere.
#pragma once

#include <type_traits>

#include "sv_score.cuh"

namespace sv {

namespace {

constexpr int SC_NT = 128;               // threads of a CTA
constexpr int SC_GROUP = 4;              // vectors of a thread in a copy group
constexpr int SC_RING = 4;               // groups of a ring in the forward passes,
constexpr int SC_RING_GRAD = 6;          // and with a gradient
constexpr int SC_MAXC = SCORE_MAX_CTAS;  // CTAs of a cluster (portable)
constexpr int SC_GROUP_BYTES = SC_GROUP * SC_NT * 16;
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
    // the largest element of a vector, as something to be compared further (most), and as a number
    using Most = float;
    static __device__ __forceinline__ Most top_of(const uint4& w)
    {
        return fmax_nan(fmax_nan(__uint_as_float(w.x), __uint_as_float(w.y)),
                        fmax_nan(__uint_as_float(w.z), __uint_as_float(w.w)));
    }
    static __device__ __forceinline__ Most most(Most a, Most b) { return fmax_nan(a, b); }
    static __device__ __forceinline__ float value(Most a) { return a; }
    static __device__ __forceinline__ float top(const uint4& w) { return top_of(w); }
    static __device__ __forceinline__ uint4 pack(const uint64_t (&y)[2])
    {
        float a, b, c, d;
        unpair(y[0], a, b);
        unpair(y[1], c, d);
        return make_uint4(__float_as_uint(a), __float_as_uint(b), __float_as_uint(c), __float_as_uint(d));
    }
    using Thr = float;
    static __device__ __forceinline__ Thr thr_of(float x) { return x; }
    using Count = int;
    static __device__ __forceinline__ Count more(Count a, Count b) { return a + b; }
    static __device__ __forceinline__ int number(Count n) { return n; }
    static __device__ __forceinline__ Count above(const uint4& w, Thr thr)
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
    using Most = uint32_t;
    static __device__ __forceinline__ Most top_of(const uint4& w)
    {
        return Vec<E>::max2(Vec<E>::max2(w.x, w.y), Vec<E>::max2(w.z, w.w));
    }
    static __device__ __forceinline__ Most most(Most a, Most b) { return Vec<E>::max2(a, b); }
    static __device__ __forceinline__ float value(Most m)
    {
        float a, b;
        unpair(Vec<E>::wide(m), a, b);
        return fmax_nan(a, b);
    }
    static __device__ __forceinline__ float top(const uint4& w) { return value(top_of(w)); }
    static __device__ __forceinline__ uint4 pack(const uint64_t (&y)[4])
    {
        return make_uint4(Vec<E>::thin(y[0]), Vec<E>::thin(y[1]), Vec<E>::thin(y[2]), Vec<E>::thin(y[3]));
    }
    using Thr = uint32_t;
    static __device__ __forceinline__ Thr thr_of(float x) { return Vec<E>::thin(pair(x, x)); }  // x is a value of E
    // counts in two halves of a word, exact in either type up to 256 (bf16) words
    using Count = uint32_t;
    static __device__ __forceinline__ Count above(const uint4& w, Thr t)
    {
        return Vec<E>::plus(Vec<E>::plus(Vec<E>::gt(w.x, t), Vec<E>::gt(w.y, t)),
                            Vec<E>::plus(Vec<E>::gt(w.z, t), Vec<E>::gt(w.w, t)));
    }
    static __device__ __forceinline__ Count more(Count a, Count b) { return Vec<E>::plus(a, b); }
    static __device__ __forceinline__ int number(Count n)
    {
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
// (nothing is written before it that the others read)
__device__ __forceinline__ void cluster_begin() { asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory"); }
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

// the barrier of a row's CTAs, in two halves
__device__ __forceinline__ void row_arrive(int C)
{
    if (C > 1) cluster_arrive();
    else __syncthreads();
}
__device__ __forceinline__ void row_wait(int C)
{
    if (C > 1) cluster_wait();
}

// ---- a CTA's slice of a row ------------------------------------------------ //
template <typename E> struct Slice {
    const char* src;  // global address of its first vector
    int n;            // vectors
    int first;        // element of the row at the first vector's start (negative: outside the row)
    int lo, hi;       // vectors lo .. hi - 1 lie in the row as a whole; one before may not, and one behind is its last

    __device__ __forceinline__ Slice() : src(nullptr), n(0), first(0), lo(0), hi(0) {}
    __device__ __forceinline__ Slice(const ScoreParams& p, const E* x, int rank)
    {
        const int mis = (int)((uintptr_t)x & 15), all = (mis + p.V * (int)sizeof(E) + 15) / 16, v0 = rank * p.per;
        n = max(0, min(p.per, all - v0));
        first = v0 * EPV<E> - mis / (int)sizeof(E);
        src = (const char*)x - mis + (int64_t)v0 * 16;
        lo = first < 0 ? 1 : 0;
        hi = max(lo, n > 0 && first + n * EPV<E> >= p.V ? n - 1 : n);
    }
};

// vector i of a slice by its elements, -inf outside the row
template <typename E> __device__ __forceinline__ uint4 part_vector(const Slice<E>& s, int V, int i)
{
    const int e = s.first + i * EPV<E>;
    const Bits<E>* from = (const Bits<E>*)(s.src + (int64_t)i * 16);
    Bits<E> v[EPV<E>];
#pragma unroll
    for (int q = 0; q < EPV<E>; ++q) v[q] = e + q >= 0 && e + q < V ? from[q] : (Bits<E>)Vec<E>::NEG;
    return vector_of<E>(v);
}
template <typename E> __device__ __forceinline__ uint4 no_vector()
{
    return make_uint4(Vec<E>::NEG, Vec<E>::NEG, Vec<E>::NEG, Vec<E>::NEG);
}
// vector i from global memory, nothing beyond the slice
template <typename E> __device__ __forceinline__ uint4 load_vector(const Slice<E>& s, int V, int i)
{
    if (i >= s.lo && i < s.hi) return *(const uint4*)(s.src + (int64_t)i * 16);
    return i >= 0 && i < s.n ? part_vector(s, V, i) : no_vector<E>();
}
template <int OFF> __device__ __forceinline__ void copy16(uint32_t to, const char* from)
{
    asm volatile("cp.async.cg.shared.global.L2::128B [%0+%2], [%1+%2], 16;" ::"r"(to), "l"(from), "n"(OFF) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void copy_done() { asm volatile("cp.async.wait_group 0;" ::: "memory"); }
// ---- a ring of copy groups ----------------------------------------------------- //
// A group is SC_GROUP vectors of every thread; a slice has `full` groups and one of what is left (up to SC_GROUP
// vectors a thread).  The row's last vector and its first, if that is not the row's as a whole, are no part of the ring:
// thread 32 has the last, thread 0 the first, in registers (edge).  After turn() the slice comes a second time, its last
// group first: the ring has the last ones still, and of the others what was read last is the likeliest to be in L2.
template <typename E, int RING> struct Ring {
    static constexpr int GROUP = SC_NT * SC_GROUP;  // vectors
    const Slice<E>& s;
    uint4* buf;
    int V, full;
    const char* src;   // this thread's first vector of the next group to be copied,
    int cb, to, from;  // that group and its place; the place of the next to be used

    __device__ __forceinline__ Ring(const ScoreParams& p, const Slice<E>& sl, int rank, void* smem)
        : s(sl), buf((uint4*)smem + threadIdx.x), V(p.V), src(sl.src + threadIdx.x * 16), cb(0), to(0), from(0)
    {
        const int least = (p.V * (int)sizeof(E) + 15) / 16 - rank * p.per;
        full = max(0, min(p.per, least) - 1) / GROUP;
#pragma unroll
        for (int i = 0; i < RING; ++i) copy_next();
    }
    __device__ __forceinline__ void copy_group()
    {
        static_assert(SC_GROUP == 4, "the calls below");
        uint4* place = buf + to;
        const uint32_t dst = (uint32_t)__cvta_generic_to_shared(place);
        if (cb >= 0 && cb < full) {
            // whole vectors, but the first of the row
            if (cb > 0 || threadIdx.x >= s.lo) copy16<0 * SC_NT * 16>(dst, src);
            else *place = no_vector<E>();
            copy16<1 * SC_NT * 16>(dst, src);
            copy16<2 * SC_NT * 16>(dst, src);
            copy16<3 * SC_NT * 16>(dst, src);
        } else if (cb == full) {
            const int i = cb * GROUP + threadIdx.x;
            if (i < s.lo) *place = no_vector<E>();
            else if (i < s.hi) copy16<0 * SC_NT * 16>(dst, src);
            if (i + SC_NT < s.hi) copy16<1 * SC_NT * 16>(dst, src);
            if (i + 2 * SC_NT < s.hi) copy16<2 * SC_NT * 16>(dst, src);
            if (i + 3 * SC_NT < s.hi) copy16<3 * SC_NT * 16>(dst, src);
        }
        copy_commit();  // (behind the last group, groups of nothing: the waits below count them)
    }
    // the oldest group has arrived; this thread's first vector of it
    __device__ __forceinline__ uint4* first() const
    {
        asm volatile("cp.async.wait_group %0;" ::"n"(RING - 1) : "memory");
        return buf + from;
    }
    __device__ __forceinline__ void copy_next()
    {
        copy_group();
        to = to + GROUP == RING * GROUP ? 0 : to + GROUP;
        src += GROUP * 16;
        ++cb;
    }
    __device__ __forceinline__ void used()
    {
        from = from + GROUP == RING * GROUP ? 0 : from + GROUP;
        copy_next();
    }
    // the second time: groups in reverse, the last of them from where they are
    __device__ __forceinline__ void turn()
    {
        cb = full - RING;
        src = s.src + ((int64_t)cb * GROUP + threadIdx.x) * 16;
        from = full % RING * GROUP;
    }
    __device__ __forceinline__ void used_again()
    {
        to = from;
        copy_group();
        from = from == 0 ? (RING - 1) * GROUP : from - GROUP;
        src -= GROUP * 16;
        --cb;
    }
    __device__ __forceinline__ bool has_edge() const
    {
        return (threadIdx.x == 0 && s.lo && s.n) || (threadIdx.x == 32 && s.hi < s.n);
    }
    __device__ __forceinline__ int edge_at() const { return threadIdx.x == 0 ? 0 : s.n - 1; }
    __device__ __forceinline__ uint4 edge() const
    {
        return has_edge() ? part_vector(s, V, edge_at()) : no_vector<E>();
    }
    __device__ __forceinline__ bool has(int id) const
    {
        return id >= s.first && id < s.first + s.n * EPV<E> && id < V;
    }
};

// ---- softmax sums ------------------------------------------------------------ //
// Terms are 2^d with d = l c - B, c = log2(e) / t and B = m c rounded to an integer, m the reference: one exact product
// and one rounding per logit, and sums of different m differ by powers of 2, exactly.  Where m c is so large that its
// integer is no help (a row of the type's lowest values, say, where products with c overflow), d = (l - m) c instead.
// A thread's reference is the first largest logit that it met, and moves only when one is 2^AWAY times above it: fp32
// has room for terms of that size, and moving at every new maximum is a long chain of dependent instructions that some
// lane of a warp would ask for at most vectors (608 x 131072 bf16: 38.8 -> 30.3 us).  The sum of d 2^d is as inexact as
// the largest d in it times an ulp of the sum of 2^d, and the entropy is what is left of ln of the one minus the other:
// with entropies AWAY is 4, which costs up to 1.5 us of a verify batch's 38 and leaves them 2e-7 off, where 32 leaves
// 3e-6.
__device__ __forceinline__ bool plain_ref(float m, float c) { return fabsf(m * c) < 4194304.f; }
__device__ __forceinline__ float dist(float l, float m, float c)
{
    return plain_ref(m, c) ? fmaf(l, c, -rintf(m * c)) : (l - (m == -INFINITY ? 0.f : m)) * c;
}
// the exponent by which terms relative to m1 become terms relative to m2 >= m1; m1 above -inf
__device__ __forceinline__ float between(float m1, float m2, float c)
{
    const bool a = plain_ref(m1, c), b = plain_ref(m2, c);
    if (a && b) return fmaxf(rintf(m1 * c) - rintf(m2 * c), NONE);
    return fmaxf((m1 - m2) * c - (a ? dist(m1, m1, c) : 0.f) + (b ? dist(m2, m2, c) : 0.f), NONE);
}
// reference, sum of 2^d, sum of d 2^d
struct Run {
    float m, s, t;
};
__device__ __forceinline__ void to_max(Run& r, float m, float c)
{
    const bool some = r.m > -INFINITY;
    const float d = some ? between(r.m, m, c) : 0.f, f = ex2_fast(d);
    r.t = some ? f * (r.t + d * r.s) : 0.f;
    r.s = some ? f * r.s : 0.f;
    r.m = m;
}

// sums of a thread's vectors, by ENTROPY those of d 2^d too; with RANK also the number of elements above x (in vectors
// before tvec: or equal to it, written as above the next value below x)
template <typename E, bool ENTROPY, bool RANK> struct Summer {
    static constexpr float AWAY = ENTROPY ? 4.f : 32.f;
    float m = -INFINITY, limit = -INFINITY, c;
    uint64_t s2 = 0, t2 = 0;
    uint32_t masked = 0;  // ENTROPY: batches where d is -inf or may be relative to the row's m; the last bit has all behind 30
    float x;
    typename Vec<E>::Thr at, under;
    int tvec, ahead = 0;

    // the terms of some vectors; CLAMP: those of d 2^d alone, where d may be -inf
    template <bool FAST, bool CLAMP, int N> __device__ __forceinline__ void terms(const uint4 (&w)[N])
    {
        const float ref = FAST ? -rintf(m * c) : m == -INFINITY ? 0.f : -m;
        const uint64_t r2 = pair(ref, ref), c2 = pair(c, c);
#pragma unroll
        for (int j = 0; j < N; ++j) {
            uint64_t v[EPV<E> / 2];
            Vec<E>::pairs(w[j], v);
#pragma unroll
            for (int q = 0; q < EPV<E> / 2; ++q) {
                const uint64_t d2 = FAST ? fma2(v[q], c2, r2) : mul2(add2(v[q], r2), c2);
                float a, z;
                unpair(d2, a, z);
                const uint64_t e2 = pair(ex2_fast(a), ex2_fast(z));
                if (!CLAMP) s2 = add2(s2, e2);
                if (ENTROPY) t2 = fma2(e2, CLAMP ? pair(fmaxf(a, NONE), fmaxf(z, NONE)) : d2, t2);
            }
        }
    }
    // vectors i, i + SC_NT, ...; returns their largest element
    template <int N> __device__ __forceinline__ float take(const uint4 (&w)[N], int i, int batch)
    {
        typename Vec<E>::Most most = Vec<E>::top_of(w[0]);
#pragma unroll
        for (int j = 1; j < N; ++j) most = Vec<E>::most(most, Vec<E>::top_of(w[j]));
        const float mx = Vec<E>::value(most);
        if (!(mx <= limit)) {  // a new reference (or NaN, which stays)
            const float mn = fmax_nan(m, mx);
            if (m > -INFINITY) {
                const float d = between(m, mn, c), f = ex2_fast(d);
                const uint64_t f2 = pair(f, f);
                if (ENTROPY) t2 = mul2(f2, fma2(pair(d, d), s2, t2));
                s2 = mul2(f2, s2);
            }
            m = mn;
            limit = mn + AWAY / c;
        }
        const uint64_t t0 = t2;
        const bool fast = plain_ref(m, c);
        if (fast) terms<true, false>(w);
        else terms<false, false>(w);
        if (ENTROPY) {
            float a, z;
            unpair(t2, a, z);
            a += z;
            if (a != a) {  // 0 times -inf
                t2 = t0;
                if (fast) terms<true, true>(w);
                else terms<false, true>(w);
            }
            if (a != a || !fast) masked |= 1u << min(batch, 31);
        }
        if (RANK && mx >= x) {
            typename Vec<E>::Count n = Vec<E>::above(w[0], i < tvec ? under : at);
#pragma unroll
            for (int j = 1; j < N; ++j) n = Vec<E>::more(n, Vec<E>::above(w[j], i + j * SC_NT < tvec ? under : at));
            ahead += Vec<E>::number(n);
        }
        return mx;
    }
    __device__ __forceinline__ Run result() const
    {
        float a, z;
        Run r;
        r.m = m;
        unpair(s2, a, z);
        r.s = a + z;
        unpair(t2, a, z);
        r.t = a + z;
        return r;
    }
    // A slice in the ring, and its edge.  change(b, v): before this thread's vectors v, v + SC_NT, ... of group b are read
    // (full + 1: the edge); seen(b, x): their largest element.
    template <typename R, typename Change, typename Seen>
    __device__ __forceinline__ void stream(R& ring, uint4 edge, Change change, Seen seen)
    {
        int i = threadIdx.x;
#pragma unroll 1
        for (int b = 0; b < ring.full; ++b, i += R::GROUP) {
            uint4* v = ring.first();
            change(b, v);
            uint4 w[SC_GROUP];
#pragma unroll
            for (int j = 0; j < SC_GROUP; ++j) w[j] = v[j * SC_NT];
            seen(b, take(w, i, b));
            ring.used();
        }
        uint4* v = ring.first();
        change(ring.full, v);
        float mx = -INFINITY;
#pragma unroll 1
        for (; i < ring.s.hi; i += SC_NT, v += SC_NT) {
            const uint4 w[1] = {*v};
            mx = fmax_nan(mx, take(w, i, ring.full));
        }
        ring.used();
        if (ring.has_edge()) {
            change(ring.full + 1, &edge);
            const uint4 w[1] = {edge};
            mx = fmax_nan(mx, take(w, ring.edge_at(), ring.full));
        }
        seen(ring.full, mx);
    }
};

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

// a row's largest logit, NaN where one is
__device__ __forceinline__ bool finite_row(float m) { return m > -INFINITY && m < INFINITY; }

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

// ---- gradients ----------------------------------------------------------------- //
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

// 16 bytes of a row that begin at byte a of this lane's vector: of it and of the next lane's
__device__ __forceinline__ uint4 joined(const uint4& w, int a)
{
    uint4 n;
    n.x = __shfl_down_sync(~0u, w.x, 1);
    n.y = __shfl_down_sync(~0u, w.y, 1);
    n.z = __shfl_down_sync(~0u, w.z, 1);
    n.w = __shfl_down_sync(~0u, w.w, 1);
    // by words, then by the bytes left
    const int words = a / 4, bits = a % 4 * 8;
    uint32_t v[5];
#pragma unroll
    for (int q = 0; q < 5; ++q) {
        const uint32_t two = q < 4 ? word_of(w, q) : n.x, three = q < 3 ? word_of(w, q + 1) : word_of(n, q - 3),
                       four = q < 2 ? word_of(w, q + 2) : word_of(n, q - 2), five = q < 1 ? w.w : word_of(n, q - 1);
        v[q] = words == 0 ? two : words == 1 ? three : words == 2 ? four : five;
    }
    return make_uint4(__funnelshift_r(v[0], v[1], bits), __funnelshift_r(v[1], v[2], bits),
                      __funnelshift_r(v[2], v[3], bits), __funnelshift_r(v[3], v[4], bits));
}

// The gradient of a slice whose ring comes to it the second time: f(pair of d, 2^d; d may be -inf in the groups that
// `masked` names, where it is clamped) -> pair.  Threads write what they read, so it may go over the logits.
template <typename E, bool FAST, typename R, typename F>
__device__ __forceinline__ void grad_slice_(R& ring, const uint4& edge, E* g, float m, float c, uint32_t masked, F f)
{
    const Slice<E>& s = ring.s;
    const float ref = FAST ? -rintf(m * c) : m == -INFINITY ? 0.f : -m;
    const uint64_t r2 = pair(ref, ref), c2 = pair(c, c);
    auto grad = [&](const uint4& x, auto clamp) {
        uint64_t v[EPV<E> / 2], y[EPV<E> / 2];
        Vec<E>::pairs(x, v);
#pragma unroll
        for (int q = 0; q < EPV<E> / 2; ++q) {
            const uint64_t d2 = FAST ? fma2(v[q], c2, r2) : mul2(add2(v[q], r2), c2);
            float a, z;
            unpair(d2, a, z);
            y[q] = f(decltype(clamp)::value ? pair(fmaxf(a, NONE), fmaxf(z, NONE)) : d2, pair(ex2_fast(a), ex2_fast(z)));
        }
        return Vec<E>::pack(y);
    };
    // streaming stores: L2 has better use for its lines
    auto store = [](char* to, const uint4& w) { __stcs((uint4*)to, w); };
    auto is_masked = [&](int b) { return masked >> min(b, 31) & 1; };
    auto any = [&](const uint4& x, int b) {
        return is_masked(b) ? grad(x, std::true_type()) : grad(x, std::false_type());
    };
    char* const out = (char*)(g + s.first);  // its element at the slice's start
    // elements q0 .. q1 - 1 of vector i
    auto elements = [&](const uint4& w, int i, int q0, int q1) {
        const int e = s.first + i * EPV<E>;
#pragma unroll
        for (int q = 0; q < EPV<E>; ++q)
            if (q >= q0 && q < q1 && e + q >= 0 && e + q < ring.V) ((Bits<E>*)g)[e + q] = bits_at<E>(w, q);
    };
    const int a = (int)((-(intptr_t)out) & 15);  // bytes from a vector's place to the next 16-byte boundary
    int i = threadIdx.x + ring.full * R::GROUP;
    ring.turn();
    if (a == 0) {
        char* to = out + (int64_t)i * 16;
        const uint4* last = ring.first();
        for (int j = 0; j < SC_GROUP; ++j)
            if (i + j * SC_NT >= s.lo && i + j * SC_NT < s.hi) store(to + j * SC_NT * 16, any(last[j * SC_NT], ring.full));
        ring.used_again();
#pragma unroll 1
        for (int b = ring.full - 1; b >= 0; --b) {
            i -= R::GROUP;
            to -= R::GROUP * 16;
            const uint4* v = ring.first();
            uint4 w[SC_GROUP];
            if (is_masked(b)) {
#pragma unroll
                for (int j = 0; j < SC_GROUP; ++j) w[j] = grad(v[j * SC_NT], std::true_type());
            } else {
#pragma unroll
                for (int j = 0; j < SC_GROUP; ++j) w[j] = grad(v[j * SC_NT], std::false_type());
            }
            if (b > 0 || i >= s.lo) store(to, w[0]);
            store(to + SC_NT * 16, w[1]);
            store(to + 2 * SC_NT * 16, w[2]);
            store(to + 3 * SC_NT * 16, w[3]);
            ring.used_again();
        }
    } else {
        // the gradient's rows begin elsewhere in a vector than the logits': lanes have neighbouring vectors, and join
        // them two by two to what lies between boundaries
        const int lane = threadIdx.x % 32, q = a / (int)sizeof(E);
        for (int b = ring.full; b >= 0; --b) {
            const uint4* v = ring.first();
            for (int j = 0; j < SC_GROUP; ++j) {
                const int i = threadIdx.x + b * R::GROUP + j * SC_NT;
                if (i - lane >= s.hi) continue;  // none of the warp's
                const bool in = i >= s.lo && i < s.hi;
                const uint4 w = in ? any(v[j * SC_NT], b) : no_vector<E>(), two = joined(w, a);
                if (!in) continue;
                if (lane < 31 && i + 1 < s.hi) store(out + (int64_t)i * 16 + a, two);
                else elements(w, i, q, EPV<E>);
                if (lane == 0 || i == s.lo) elements(w, i, 0, q);
            }
            ring.used_again();
        }
    }
    if (ring.has_edge()) elements(any(edge, ring.full), ring.edge_at(), 0, EPV<E>);
}
template <typename E, typename R, typename F>
__device__ __forceinline__ void grad_slice(R& ring, const uint4& edge, E* g, float m, float c, uint32_t masked, F f)
{
    if (plain_ref(m, c)) grad_slice_<E, true>(ring, edge, g, m, c, masked, f);
    else grad_slice_<E, false>(ring, edge, g, m, c, masked, f);
}

// ---- launches ------------------------------------------------------------------ //
// A kernel's launch set-up on each device, and the clusters of 1, 2, 4 .. CTAs that are resident there with the least of
// shared memory that it takes.
struct ScoreKernel {
    DeviceOnce once;
    int clusters[SV_MAX_DEVICES][4] = {};
};
struct ScoreLaunch {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[1];
    ScoreLaunch(int C, size_t smem, cudaStream_t s)
    {
        cfg.gridDim = dim3((unsigned)C);
        cfg.blockDim = dim3(SC_NT);
        cfg.dynamicSmemBytes = smem;
        cfg.stream = s;
        at[0].id = cudaLaunchAttributeClusterDimension;
        at[0].val.clusterDim.x = C;
        at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
        cfg.attrs = at;
        cfg.numAttrs = 1;
    }
};

// to be called before the others: `least` to `most` bytes of shared memory for the kernel
template <typename K>
cudaError_t score_ready(K kernel, ScoreKernel& sk, size_t least, size_t most)
{
    static_assert(SC_MAXC == 8, "four powers of two");
    return cuda_once(sk.once, nullptr, [&](int dev, int*) {
        cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
        for (int i = 0; i < 4 && e == cudaSuccess; ++i) {
            const ScoreLaunch l(1 << i, least, nullptr);
            e = cudaOccupancyMaxActiveClusters(&sk.clusters[dev][i], kernel, &l.cfg);
        }
        return e;
    });
}

// Launches a cluster of p.cluster CTAs for every row.
template <typename K> cudaError_t score_launch(K kernel, ScoreParams& p, size_t smem, cudaStream_t s)
{
    p.by_tokens = FastDiv(p.T);
    ScoreLaunch l(p.cluster, smem, s);
    l.cfg.gridDim = dim3((unsigned)p.rows * p.cluster);
    return cudaLaunchKernelEx(&l.cfg, kernel, p);
}

// vectors of a row, at any alignment
inline int score_vectors(const ScoreParams& p, size_t size) { return (int)(((size_t)p.V * size + 30) / 16); }

// CTAs of a row in a forward pass, by the time that each power of two would take: the rows that a resident cluster has
// one after another (and half a row for those that end last), each of a slice's vectors and a cost that does not shrink
// with it (`fixed`, in vectors of a thread).  smem_of: bytes for a slice, which may leave room for fewer CTAs on an SM.
template <typename F>
cudaError_t score_split_forward(const ScoreKernel& sk, ScoreParams& p, size_t size, int num_sms, int fixed, F smem_of)
{
    constexpr size_t SM_BYTES = 228 * 1024, AROUND = 2048;  // of an SM, and what a CTA takes besides
    const int row = score_vectors(p, size);
    int dev = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    double best = 0;
    for (int i = 0; i < 4 && (i == 0 || row >> i >= SC_NT); ++i) {
        const int C = 1 << i, per = (row + C - 1) / C;
        const int fit = num_sms * (int)(SM_BYTES / (smem_of(per) + AROUND)) / C;
        const int nc = max(1, min(sk.clusters[dev][i], fit));
        const double rounds = p.rows <= nc ? 1.0 : (double)p.rows / nc + 0.5, cost = rounds * ((double)per / SC_NT + fixed);
        if (C > 1 && cost >= best) continue;
        best = cost;
        p.cluster = C;
        p.per = per;
    }
    return cudaSuccess;
}
// CTAs of a row with a gradient, four of them an SM (their rings see to it): as many as it takes for the rows under way,
// as long as they are two passes over, to have room in L2 beside what else goes through it; and few rows are spread over
// more, for the SMs that would idle, while every thread has a vector or two.  What a ring holds at the turn, a third or
// more of a slice, is not read again at all: rings of 4, 5, 6 groups took 204, 201, 200 us for 2000 x 128256 bf16 and
// 174, 171, 169 for 777 x 128256 fp32.  With 140 MB instead of 100 under way 1500 x 100003 fp16 take 136 us, not 124
// (L2 loses more of what comes again), with 60 MB 143, and 777 x 128256 fp32 178, not 169 (more CTAs a row, each with
// its entries and joins).  Three CTAs an SM with rings of 8 take 190, 135, 169, and 28, not 24, for 300 x 32000 fp32.
constexpr size_t SC_GRAD_BYTES = SC_RING_GRAD * SC_GROUP_BYTES;
inline void score_split_gradient(ScoreParams& p, size_t size, int num_sms)
{
    const int row = score_vectors(p, size);
    const double under_way = 4.0 * num_sms < p.rows ? 4.0 * num_sms : p.rows;
    int C = 1;
    while (C < SC_MAXC && ((under_way / C) * row * 16 > SCORE_L2_ROWS ||
                           ((int64_t)p.rows * C < 2 * num_sms && row / (2 * C) >= SC_NT)))
        C *= 2;
    p.cluster = C;
    p.per = (row + C - 1) / C;
}

}  // namespace

}  // namespace sv
