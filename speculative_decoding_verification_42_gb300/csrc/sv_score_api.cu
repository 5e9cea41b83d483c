// sv_score_api.cu -- the C ABI of include/spec_score.h: argument checks and
// launches.  Host code only.
#include <math.h>

#include "sv_host.h"
#include "sv_once.h"
#include "sv_score.cuh"

using namespace sv;

namespace {

bool dtype_ok(int32_t d) { return d == SPEC_F32 || d == SPEC_BF16 || d == SPEC_F16; }
size_t size_of(int32_t d) { return d == SPEC_F32 ? 4 : 2; }
bool temp_ok(float t) { return t >= 1e-30f && t <= 1e30f; }
bool strides_ok(const spec_score_rows& r) { return r.seq_stride >= 0 && r.token_stride >= 0; }
constexpr int64_t MAX_STRIDE = (int64_t)1 << 34;  // products with a number of rows stay below 2^63
bool strides_fit(const spec_score_rows& r) { return r.seq_stride < MAX_STRIDE && r.token_stride < MAX_STRIDE; }
// no two of the rows share an element (positions inside sequences, or the reverse)
bool apart(const spec_score_rows& r, int64_t B, int64_t T, int64_t V)
{
    const int64_t s = r.seq_stride, t = r.token_stride;
    if (T == 1) return B == 1 || s >= V;
    if (B == 1) return t >= V;
    return (t >= V && s >= (T - 1) * t + V) || (s >= V && t >= (B - 1) * s + V);
}
bool on(const void* p, size_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

// what both operators check of their rows; SPEC_OK with *empty for a no-op
spec_status check_rows(int32_t device, int32_t dtype, int32_t batch, int32_t tokens, int32_t vocab, float temp,
                       const spec_score_rows& x, const spec_score_rows& g, const int32_t* row_status, bool* empty)
{
    if (device < 0 || !dtype_ok(dtype) || batch < 0 || tokens < 0 || vocab < 1 || !temp_ok(temp) || !strides_ok(x) ||
        !strides_ok(g))
        return SPEC_ERR_INVALID_ARG;
    *empty = batch == 0 || tokens == 0;
    if (*empty) return SPEC_OK;
    if (!x.ptr || !row_status) return SPEC_ERR_INVALID_ARG;
    const size_t s = size_of(dtype);
    if ((int64_t)batch * tokens > INT32_MAX / 8 || (size_t)vocab * s > SCORE_MAX_ROW_BYTES || !strides_fit(x) ||
        !strides_fit(g) || !on(x.ptr, s) || !on(g.ptr, s) || !on(row_status, 4))
        return SPEC_ERR_UNSUPPORTED;
    // two rows of a gradient at one place would be a race, as would one over another row's logits
    if (g.ptr && (!apart(g, batch, tokens, vocab) ||
                  (g.ptr == x.ptr && ((batch > 1 && g.seq_stride != x.seq_stride) ||
                                      (tokens > 1 && g.token_stride != x.token_stride)))))
        return SPEC_ERR_INVALID_ARG;
    return SPEC_OK;
}

// SMs of a device
DeviceOnce g_sms;
spec_status sms_of(int device, int* sms)
{
    const cudaError_t e = device_once(g_sms, device, cudaSuccess, cudaErrorInvalidDevice, sms, [](int dev, int* v) {
        return cudaDeviceGetAttribute(v, cudaDevAttrMultiProcessorCount, dev);
    });
    return e == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

ScoreParams rows_of(int32_t batch, int32_t tokens, int32_t vocab, float temp, const spec_score_rows& x,
                    const spec_score_rows& g, int32_t* row_status)
{
    ScoreParams p = {};
    p.x = (const char*)x.ptr;
    p.x_seq = x.seq_stride;
    p.x_tok = x.token_stride;
    p.grad = (char*)g.ptr;
    p.g_seq = g.seq_stride;
    p.g_tok = g.token_stride;
    p.rows = batch * tokens;
    p.T = tokens;
    p.V = vocab;
    p.inv_temp = 1.f / temp;
    p.c = (float)(1.4426950408889634 / (double)temp);
    p.row_status = row_status;
    return p;
}

}  // namespace

extern "C" {

spec_status spec_score_logprobs(const spec_score_logprobs_args* a, void* stream)
{
    if (!a) return SPEC_ERR_INVALID_ARG;
    bool empty;
    const spec_status st = check_rows(a->device, a->dtype, a->batch, a->tokens, a->vocab, a->temperature, a->logits,
                                      a->grad, a->row_status, &empty);
    if (st != SPEC_OK) return st;
    if (a->top_n < 0 || ((a->logprob || a->rank || a->grad_logprob) && !a->ids && !empty) ||
        (a->top_n > 0 && a->top_n <= SPEC_SCORE_MAX_TOP && (!a->top_ids || !a->top_logprobs) && !empty) ||
        (!empty && (a->grad.ptr != nullptr) != (a->grad_logprob || a->grad_entropy)))
        return SPEC_ERR_INVALID_ARG;
    if (a->top_n > SPEC_SCORE_MAX_TOP || !on(a->ids, 4) || !on(a->grad_logprob, 4) || !on(a->grad_entropy, 4) ||
        !on(a->logprob, 4) || !on(a->rank, 4) || !on(a->entropy, 4) || !on(a->lse, 4) || !on(a->top_ids, 4) ||
        !on(a->top_logprobs, 4))
        return SPEC_ERR_UNSUPPORTED;
    if (empty) return SPEC_OK;
    DeviceGuard g(a->device);
    if (!g.ok) return SPEC_ERR_CUDA;
    int sms = 0;
    if (sms_of(a->device, &sms) != SPEC_OK) return SPEC_ERR_CUDA;
    ScoreParams p = rows_of(a->batch, a->tokens, a->vocab, a->temperature, a->logits, a->grad, a->row_status);
    p.ids = a->ids;
    p.g_logprob = a->grad_logprob;
    p.g_entropy = a->grad_entropy;
    p.top_n = a->top_n;
    p.logprob = a->logprob;
    p.rank = a->rank;
    p.entropy = a->entropy;
    p.lse = a->lse;
    p.top_ids = a->top_ids;
    p.top_lp = a->top_logprobs;
    return launch_score_logprobs(p, a->dtype, sms, (cudaStream_t)stream) == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

spec_status spec_score_distill(const spec_score_distill_args* a, void* stream)
{
    if (!a) return SPEC_ERR_INVALID_ARG;
    bool empty;
    const spec_status st = check_rows(a->device, a->dtype, a->batch, a->tokens, a->vocab, a->temperature, a->student,
                                      a->grad, a->row_status, &empty);
    if (st != SPEC_OK) return st;
    if (!dtype_ok(a->teacher_dtype) || a->entries < 1 || !temp_ok(a->teacher_temperature) ||
        (!empty && (!a->ids || !a->teacher)) || (a->teacher_lse && !a->tail) || (a->grad_loss && !a->grad.ptr && !empty))
        return SPEC_ERR_INVALID_ARG;
    if (a->entries > SPEC_SCORE_MAX_ENTRIES || !on(a->ids, 4) || !on(a->teacher, size_of(a->teacher_dtype)) ||
        !on(a->teacher_lse, 4) || !on(a->grad_loss, 4) || !on(a->loss, 4) || !on(a->accept, 4))
        return SPEC_ERR_UNSUPPORTED;
    if (empty) return SPEC_OK;
    DeviceGuard g(a->device);
    if (!g.ok) return SPEC_ERR_CUDA;
    int sms = 0;
    if (sms_of(a->device, &sms) != SPEC_OK) return SPEC_ERR_CUDA;
    ScoreParams p = rows_of(a->batch, a->tokens, a->vocab, a->temperature, a->student, a->grad, a->row_status);
    p.ids = a->ids;
    p.k = a->entries;
    p.tail = a->tail ? 1 : 0;
    p.teacher = a->teacher;
    p.teacher_dtype = a->teacher_dtype;
    const double inv_tt = 1.0 / (double)a->teacher_temperature;
    p.inv_tt = (float)inv_tt;
    p.inv_tt_lo = (float)(inv_tt - (double)p.inv_tt);
    p.teacher_lse = a->teacher_lse;
    p.g_loss = a->grad_loss;
    p.loss = a->loss;
    p.accept = a->accept;
    return launch_score_distill(p, a->dtype, sms, (cudaStream_t)stream) == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

}  // extern "C"
