// sv_score.cu -- the operators that score rows of logits: log probabilities of
// given tokens with entropy and top alternatives, the divergence from a
// teacher's top logits, and their gradients.
//
// One CTA per row, which reads it again for each step: the largest logit, the
// sums over exp, and (gradients, top alternatives) what follows from them.
#include "sv_score.cuh"

namespace sv {

namespace {

constexpr int SC_NT = 256;
constexpr uint32_t KEY_NEG_INF = 0x007FFFFFu;  // key_of(-inf)

template <typename E> __device__ __forceinline__ float widen(E x);
template <> __device__ __forceinline__ float widen(float x) { return x; }
template <> __device__ __forceinline__ float widen(__nv_bfloat16 x) { return __bfloat162float(x); }
template <> __device__ __forceinline__ float widen(__half x) { return __half2float(x); }
template <typename E> __device__ __forceinline__ E narrow(float x);
template <> __device__ __forceinline__ float narrow(float x) { return x; }
template <> __device__ __forceinline__ __nv_bfloat16 narrow(float x) { return __float2bfloat16_rn(x); }
template <> __device__ __forceinline__ __half narrow(float x) { return __float2half_rn(x); }

template <typename E> __device__ const E* row_of(const ScoreParams& p, int r)
{
    return (const E*)p.x + (int64_t)(r / p.T) * p.x_seq + (int64_t)(r % p.T) * p.x_tok;
}
template <typename E> __device__ E* grad_of(const ScoreParams& p, int r)
{
    return (E*)p.grad + (int64_t)(r / p.T) * p.g_seq + (int64_t)(r % p.T) * p.g_tok;
}

// reductions over the CTA, in a fixed order; every thread gets the result
template <typename X, typename F> __device__ X block_reduce(X x, F op)
{
    __shared__ X part[SC_NT / 32];
    for (int d = 16; d; d >>= 1) x = op(x, __shfl_xor_sync(~0u, x, d));
    __syncthreads();
    if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = x;
    __syncthreads();
    x = part[0];
    for (int i = 1; i < SC_NT / 32; ++i) x = op(x, part[i]);
    return x;
}
template <typename X> __device__ X block_sum(X x)
{
    return block_reduce(x, [](X a, X b) { return a + b; });
}
__device__ float block_max(float x)
{
    return block_reduce(x, [](float a, float b) { return fmax_nan(a, b); });
}

template <typename E> __device__ void zero_grad(const ScoreParams& p, int r)
{
    if (!p.grad) return;
    E* g = grad_of<E>(p, r);
    for (int v = threadIdx.x; v < p.V; v += SC_NT) g[v] = narrow<E>(0.f);
}

// the distance of a logit from the largest, times c: 2 to that power is its share of Z.  The difference comes
// first: products with c may overflow where it does not (a row of the type's lowest values).
__device__ __forceinline__ float dist2(float l, float m, float c) { return (l - m) * c; }

// ---- log probabilities --------------------------------------------------- //
template <typename E> __device__ void top_of_row(const ScoreParams& p, int r, const E* x, float m, float logz)
{
    __shared__ uint32_t keys[SPEC_SCORE_MAX_TOP];
    __shared__ int32_t ids[SPEC_SCORE_MAX_TOP];
    __shared__ int count;
    auto key = [&](int v) { return key_of(widen(x[v])); };
    auto number = [&](auto pred) {
        int n = 0;
        for (int v = threadIdx.x; v < p.V; v += SC_NT) n += pred(v) ? 1 : 0;
        return block_sum(n);
    };
    const int unmasked = number([&](int v) { return key(v) > KEY_NEG_INF; });
    const int n = min(p.top_n, unmasked);
    // the n-th largest key, and the last id among its equals that belongs to the first n
    uint32_t lo = KEY_NEG_INF + 1, hi = 0xFF800000u;
    while (lo < hi) {
        const uint32_t mid = lo + (hi - lo + 1) / 2;
        if (number([&](int v) { return key(v) >= mid; }) >= n) lo = mid;
        else hi = mid - 1;
    }
    const int above = number([&](int v) { return key(v) > lo; });
    int first = -1, last = p.V - 1;
    while (first < last) {
        const int mid = first + (last - first) / 2;
        if (number([&](int v) { return v <= mid && key(v) == lo; }) >= n - above) last = mid;
        else first = mid + 1;
    }
    if (threadIdx.x == 0) count = 0;
    __syncthreads();
    for (int v = threadIdx.x; n > 0 && v < p.V; v += SC_NT) {
        const uint32_t k = key(v);
        if (k > lo || (k == lo && v <= last)) {
            const int at = atomicAdd(&count, 1);
            keys[at] = k;
            ids[at] = v;
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += SC_NT) {
        int at = 0;
        for (int j = 0; j < n; ++j) at += keys[j] > keys[i] || (keys[j] == keys[i] && ids[j] < ids[i]);
        p.top_ids[(int64_t)r * p.top_n + at] = ids[i];
        p.top_lp[(int64_t)r * p.top_n + at] = (val_of(keys[i]) - m) * p.inv_temp - logz;
    }
    for (int i = n + threadIdx.x; i < p.top_n; i += SC_NT) {
        p.top_ids[(int64_t)r * p.top_n + i] = -1;
        p.top_lp[(int64_t)r * p.top_n + i] = -INFINITY;
    }
}

template <typename E> __global__ void __launch_bounds__(SC_NT) k_score_logprobs(const ScoreParams p)
{
    const int r = blockIdx.x, tid = threadIdx.x;
    const int id = p.ids ? p.ids[r] : 0;
    const E* x = row_of<E>(p, r);
    int status = id < -1 || id >= p.V ? SPEC_ROW_BAD_TOKEN : SPEC_ROW_OK;
    float m = 0.f;
    if (id >= 0 && status == SPEC_ROW_OK) {
        m = -INFINITY;
        for (int v = tid; v < p.V; v += SC_NT) m = fmax_nan(m, widen(x[v]));
        m = block_max(m);
        if (!(m > -INFINITY && m < INFINITY)) status = SPEC_ROW_NONFINITE;
    }
    if (id == -1 || status != SPEC_ROW_OK) {
        const float none = status == SPEC_ROW_OK ? 0.f : __int_as_float(0x7FFFFFFF);
        if (tid == 0) {
            p.row_status[r] = status;
            if (p.logprob) p.logprob[r] = none;
            if (p.rank) p.rank[r] = -1;
            if (p.entropy) p.entropy[r] = none;
            if (p.lse) p.lse[r] = none;
        }
        for (int i = tid; i < p.top_n; i += SC_NT) {
            p.top_ids[(int64_t)r * p.top_n + i] = -1;
            p.top_lp[(int64_t)r * p.top_n + i] = status == SPEC_ROW_OK ? -INFINITY : none;
        }
        zero_grad<E>(p, r);
        return;
    }
    const float xt = widen(x[id]);
    float s = 0.f, t = 0.f;
    int ahead = 0;
    for (int v = tid; v < p.V; v += SC_NT) {
        const float l = widen(x[v]), d = dist2(l, m, p.c), e = exp2f(d);
        s += e;
        t += e > 0.f ? e * d : 0.f;
        ahead += l > xt || (l == xt && v < id && l > -INFINITY);
    }
    s = block_sum(s);
    t = block_sum(t);
    ahead = block_sum(ahead);
    const float logz = logf(s), ent = logz - 0.69314718f * (t / s);
    if (tid == 0) {
        p.row_status[r] = SPEC_ROW_OK;
        if (p.logprob) p.logprob[r] = (xt - m) * p.inv_temp - logz;
        if (p.rank) p.rank[r] = ahead;
        if (p.entropy) p.entropy[r] = ent;
        if (p.lse) p.lse[r] = m * p.inv_temp + logz;
    }
    if (p.top_n) top_of_row(p, r, x, m, logz);
    if (p.grad) {
        __syncthreads();
        E* g = grad_of<E>(p, r);
        const float gl = p.g_logprob ? p.g_logprob[r] : 0.f, gh = p.g_entropy ? p.g_entropy[r] : 0.f;
        for (int v = tid; v < p.V; v += SC_NT) {
            const float d = dist2(widen(x[v]), m, p.c), e = exp2f(d) / s;
            const float plp = e > 0.f ? e * (0.69314718f * d - logz + ent) : 0.f;
            g[v] = narrow<E>(((v == id && p.g_logprob ? gl : 0.f) - gl * e - gh * plp) * p.inv_temp);
        }
    }
}

// ---- distillation --------------------------------------------------------- //
__device__ float teacher_value(const ScoreParams& p, int64_t at)
{
    const float t = p.teacher_dtype == SPEC_F32 ? ((const float*)p.teacher)[at]
                    : p.teacher_dtype == SPEC_BF16 ? __bfloat162float(((const __nv_bfloat16*)p.teacher)[at])
                                                   : __half2float(((const __half*)p.teacher)[at]);
    return t;
}

template <typename E> __global__ void __launch_bounds__(SC_NT) k_score_distill(const ScoreParams p)
{
    extern __shared__ uint32_t in_s[];  // one bit a token: an entry's
    __shared__ int32_t ids[SPEC_SCORE_MAX_ENTRIES];
    const int r = blockIdx.x, tid = threadIdx.x, k = p.k;
    const int64_t at = (int64_t)r * k + tid;
    const E* x = row_of<E>(p, r);
    for (int w = tid; w < (p.V + 31) / 32; w += SC_NT) in_s[w] = 0;
    const int id = tid < k ? p.ids[at] : -1;
    const float tv = id >= 0 ? teacher_value(p, at) : -INFINITY;
    ids[tid] = id;
    __syncthreads();
    bool bad = id < -1 || id >= p.V;
    for (int j = 0; j < tid; ++j) bad |= id >= 0 && ids[j] == id;
    bad = __syncthreads_or(bad);
    const bool any = __syncthreads_or(id >= 0);
    const float tmax = block_max(tv), lse = p.teacher_lse && any ? p.teacher_lse[r] : 0.f;
    int status = bad ? SPEC_ROW_BAD_TOKEN : SPEC_ROW_OK;
    if (id >= 0 && !bad) atomicOr(in_s + id / 32, 1u << (id % 32));
    __syncthreads();
    auto inside = [&](int v) { return in_s[v / 32] >> (v % 32) & 1; };
    // the largest logit of the others, of the entries, of all: the others' mass can be far below the entries'
    float mr = -INFINITY, m = 0.f, l = -INFINITY;
    if (any && !bad) {
        for (int v = tid; v < p.V; v += SC_NT)
            if (!inside(v)) mr = fmax_nan(mr, widen(x[v]));
        mr = block_max(mr);
        if (id >= 0) l = widen(x[id]);
        m = fmax_nan(mr, block_max(l));
        if (!(m > -INFINITY && m < INFINITY) || !(tmax < INFINITY) || (!p.tail && tmax == -INFINITY) ||
            !(fabsf(lse) < INFINITY))
            status = SPEC_ROW_NONFINITE;
    }
    if (!any || status != SPEC_ROW_OK) {
        if (tid == 0) {
            p.row_status[r] = status;
            if (p.loss) p.loss[r] = status == SPEC_ROW_OK ? 0.f : __int_as_float(0x7FFFFFFF);
            if (p.accept) p.accept[r] = status == SPEC_ROW_OK ? 0.f : __int_as_float(0x7FFFFFFF);
        }
        zero_grad<E>(p, r);
        return;
    }
    if (mr == -INFINITY) mr = m;  // no others: their sum is 0 at any reference
    float rest = 0.f;
    for (int v = tid; v < p.V; v += SC_NT)
        if (!inside(v)) rest += exp2f(dist2(widen(x[v]), mr, p.c));
    const double zr = block_sum((double)rest);  // relative to mr, z to m
    const double dr = ((double)mr - m) / p.temp, scale = exp(dr);
    const float e = exp2f(dist2(l, m, p.c));
    const double z = zr * scale + block_sum((double)e);
    // the teacher: ln q_i = y_i - nq
    const double y = id >= 0 ? (double)tv / p.teacher_temp : 0.0;
    const double ymax = (double)tmax / p.teacher_temp;
    const float w = id >= 0 ? expf((float)(y - (p.tail ? (double)lse : ymax))) : 0.f;
    const double sum = block_sum((double)w);
    const double nq = p.tail ? (double)lse : ymax + log(sum);
    const float q = p.tail ? w : (float)(w / sum);
    const double mass_s = p.tail ? sum : 1.0, qr = p.tail ? fmax(0.0, 1.0 - sum) : 0.0;
    const double d = ((double)l - m) / p.temp;
    const double part = block_sum(q > 0.f ? q * (y - nq - d) : 0.0);
    const float acc = block_sum(fminf(q, (float)(e / z)));
    if (tid == 0) {
        p.row_status[r] = SPEC_ROW_OK;
        double loss = part + mass_s * log(z);
        if (qr > 0.0) loss += qr * (log(qr) - (dr + log(zr) - log(z)));
        if (p.loss) p.loss[r] = (float)loss;
        if (p.accept) p.accept[r] = acc;
    }
    if (p.grad) {
        E* g = grad_of<E>(p, r);
        const float gl = (p.g_loss ? p.g_loss[r] : 1.f) * p.inv_temp;
        const double mass = mass_s + qr;
        const float ps = (float)(mass / z), pr = (float)(mass * scale / z - (zr > 0.0 ? qr / zr : 0.0));
        __syncthreads();
        for (int v = tid; v < p.V; v += SC_NT)
            if (!inside(v)) g[v] = narrow<E>(gl * (pr * exp2f(dist2(widen(x[v]), mr, p.c))));
        if (id >= 0) g[id] = narrow<E>(gl * (ps * e - q));
    }
}

template <typename E> cudaError_t go_logprobs(const ScoreParams& p, cudaStream_t s)
{
    k_score_logprobs<E><<<p.rows, SC_NT, 0, s>>>(p);
    return cudaGetLastError();
}
template <typename E> cudaError_t go_distill(const ScoreParams& p, cudaStream_t s)
{
    static DeviceOnce once;
    const size_t most = (SCORE_MAX_ROW_BYTES / sizeof(E) + 31) / 32 * 4;
    const cudaError_t e = cuda_once(once, nullptr, [&](int, int*) {
        return cudaFuncSetAttribute(k_score_distill<E>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
    });
    if (e != cudaSuccess) return e;
    k_score_distill<E><<<p.rows, SC_NT, (size_t)(p.V + 31) / 32 * 4, s>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_score_logprobs(const ScoreParams& p, int dtype, int, cudaStream_t s)
{
    return dtype == SPEC_F32 ? go_logprobs<float>(p, s)
           : dtype == SPEC_BF16 ? go_logprobs<__nv_bfloat16>(p, s)
                                : go_logprobs<__half>(p, s);
}

cudaError_t launch_score_distill(const ScoreParams& p, int dtype, int, cudaStream_t s)
{
    return dtype == SPEC_F32 ? go_distill<float>(p, s)
           : dtype == SPEC_BF16 ? go_distill<__nv_bfloat16>(p, s)
                                : go_distill<__half>(p, s);
}

}  // namespace sv
