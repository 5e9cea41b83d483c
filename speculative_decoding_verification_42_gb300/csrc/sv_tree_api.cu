// sv_tree_api.cu -- the C ABI of include/spec_tree.h: argument checks, the
// workspace and the launches.  Host code only.
#include <math.h>
#include <string.h>

#include <new>

#include "sv_host.h"
#include "sv_tree.cuh"

using namespace sv;

struct spec_tree {
    spec_tree_config cfg;
    int page_log2;
    int num_sms;
    int fault;  // spec_tree_inject_fault: the fault armed for the next attend
    Workspace mem;
    unsigned* err;   // bounded waits that ran out (0 = none)
    void* parts;     // partial sums of spec_tree_attend
};

namespace {

bool batch_ok(const spec_tree* h, int32_t batch, int32_t tokens)
{
    // rows of all tensors are counted in 32 bits
    return batch >= 0 && batch <= h->cfg.max_batch && tokens >= 1 && tokens <= h->cfg.max_tokens &&
           (int64_t)batch * tokens <= INT32_MAX / (int64_t)h->cfg.q_heads;
}

TreeShape shape(const spec_tree* h, int32_t batch, int32_t tokens, const int32_t* ctx, const int32_t* n)
{
    const spec_tree_config& c = h->cfg;
    return TreeShape{batch, tokens, c.q_heads, c.kv_heads, c.head_dim, h->page_log2, c.table_width, c.num_pages,
                     ctx, n};
}

// strides of 16-byte loads and of tensor maps: multiples of 8 elements, 0 <= stride < 2^36
bool stride_ok(int64_t s) { return s >= 0 && s % 8 == 0 && s < ((int64_t)1 << 36); }
bool rows_ok(const spec_tree_rows& r)
{
    return aligned16(r.ptr) && stride_ok(r.seq_stride) && stride_ok(r.token_stride) && stride_ok(r.head_stride);
}
// a stride of 0 only where there is one element: two writers would meet at one place, and tensor maps take none
bool cache_ok(const spec_tree* h, const spec_tree_cache& c)
{
    return aligned16(c.k) && aligned16(c.v) && stride_ok(c.page_stride) && stride_ok(c.token_stride) &&
           stride_ok(c.head_stride) && (h->cfg.num_pages == 1 || c.page_stride) &&
           (h->cfg.page_size == 1 || c.token_stride) && (h->cfg.kv_heads == 1 || c.head_stride);
}
TreeRows rows(const spec_tree_rows& r) { return TreeRows{r.ptr, r.seq_stride, r.token_stride, r.head_stride}; }
TreeCachePtrs cache(const spec_tree_cache& c)
{
    return TreeCachePtrs{c.k, c.v, c.page_stride, c.token_stride, c.head_stride, c.layer_stride, c.layers};
}
spec_status launched(cudaError_t e) { return e == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA; }

}  // namespace

extern "C" {

spec_status spec_tree_create(const spec_tree_config* cfg, spec_tree_t* out)
{
    if (!out) return SPEC_ERR_INVALID_ARG;
    *out = nullptr;
    if (!cfg || cfg->device < 0 || cfg->max_batch < 1 || cfg->max_tokens < 1 || cfg->q_heads < 1 ||
        cfg->kv_heads < 1 || cfg->q_heads % cfg->kv_heads || cfg->head_dim < 1 || cfg->page_size < 1 ||
        cfg->num_pages < 1 || cfg->table_width < 1 || cfg->dtype < SPEC_F32 || cfg->dtype > SPEC_F16)
        return SPEC_ERR_INVALID_ARG;
    if ((int64_t)cfg->num_pages * cfg->page_size > INT32_MAX ||
        (int64_t)cfg->table_width * cfg->page_size > INT32_MAX)
        return SPEC_ERR_INVALID_ARG;
    if (cfg->dtype == SPEC_F32 || cfg->head_dim % 16 || cfg->head_dim > 256 || cfg->page_size < 8 ||
        cfg->page_size > 1024 || (cfg->page_size & (cfg->page_size - 1)) || cfg->q_heads / cfg->kv_heads > 128)
        return SPEC_ERR_UNSUPPORTED;
    DeviceGuard g(cfg->device);
    if (!g.ok) return SPEC_ERR_CUDA;
    spec_tree* h = new (std::nothrow) spec_tree();
    if (!h) return SPEC_ERR_OOM;
    h->cfg = *cfg;
    while ((1 << h->page_log2) < cfg->page_size) ++h->page_log2;
    spec_status st = SPEC_ERR_CUDA;
    size_t at;
    if (cudaDeviceGetAttribute(&h->num_sms, cudaDevAttrMultiProcessorCount, cfg->device) == cudaSuccess)
        st = workspace_take(&h->mem, cfg->device, 256 + tree_attend_bytes(cfg->head_dim, h->num_sms, &at, &at));
    if (st != SPEC_OK) {
        delete h;
        return st;
    }
    h->err = (unsigned*)h->mem.base;
    h->parts = (char*)h->mem.base + 256;
    *out = h;
    return SPEC_OK;
}

spec_status spec_tree_destroy(spec_tree_t h)
{
    if (!h) return SPEC_ERR_INVALID_ARG;
    spec_status st = SPEC_OK;
    {
        DeviceGuard g(h->cfg.device);
        if (!g.ok) st = SPEC_ERR_CUDA;
        if (workspace_give(&h->mem, h->cfg.device) != SPEC_OK) st = SPEC_ERR_CUDA;
    }
    delete h;
    return st;
}

spec_status spec_tree_check(spec_tree_t h, void* stream)
{
    if (!h) return SPEC_ERR_INVALID_ARG;
    DeviceGuard g(h->cfg.device);
    if (!g.ok) return SPEC_ERR_CUDA;
    cudaStream_t cs = (cudaStream_t)stream;
    unsigned word = 0;
    if (cudaMemcpyAsync(&word, h->err, sizeof word, cudaMemcpyDeviceToHost, cs) != cudaSuccess ||
        cudaStreamSynchronize(cs) != cudaSuccess ||
        (word && (cudaMemsetAsync(h->err, 0, sizeof word, cs) != cudaSuccess ||
                  cudaStreamSynchronize(cs) != cudaSuccess))) {
        cudaGetLastError();
        return SPEC_ERR_CUDA;
    }
    return word ? SPEC_ERR_TIMEOUT : SPEC_OK;
}

spec_status spec_tree_inject_fault(spec_tree_t h, int32_t fault)
{
    if (!h || (fault != SPEC_FAULT_NONE && fault != SPEC_FAULT_STALL_STREAM)) return SPEC_ERR_INVALID_ARG;
    h->fault = fault;
    return SPEC_OK;
}

spec_status spec_tree_plan(spec_tree_t h, const spec_tree_plan_args* a, void* stream)
{
    if (!h || !a || !batch_ok(h, a->batch, a->tokens) || !a->ring || !a->ring_out || a->ring == a->ring_out)
        return SPEC_ERR_INVALID_ARG;
    if (a->batch > 0 && (!a->ctx_len || !a->held || !a->free_pages || !a->block_table || !a->held_out ||
                         !a->slot_map || !a->positions || !a->row_status || a->held == a->held_out ||
                         (a->parents && (!a->tree_mask || a->tokens > SPEC_TREE_MAX_NODES))))
        return SPEC_ERR_INVALID_ARG;
    DeviceGuard g(h->cfg.device);
    if (!g.ok) return SPEC_ERR_CUDA;
    TreePlanParams p = {};
    p.s = shape(h, a->batch, a->tokens, a->ctx_len, a->n_tokens);
    p.parents = a->parents;
    p.held = a->held;
    p.ring = a->ring;
    p.free_pages = a->free_pages;
    p.table = a->block_table;
    p.held_out = a->held_out;
    p.ring_out = a->ring_out;
    p.slot_map = a->slot_map;
    p.positions = a->positions;
    p.mask = a->tree_mask;
    p.row_status = a->row_status;
    p.words = (a->tokens + 31) / 32;
    return launched(launch_tree_plan(p, h->num_sms, (cudaStream_t)stream));
}

spec_status spec_tree_append(spec_tree_t h, const spec_tree_append_args* a, void* stream)
{
    if (!h || !a || !batch_ok(h, a->batch, a->tokens) || !(a->eps >= 0.f) || isinf(a->eps))
        return SPEC_ERR_INVALID_ARG;
    if (a->batch == 0) return SPEC_OK;
    if (!a->q.ptr || !a->k.ptr || !a->v.ptr || !a->cache.k || !a->cache.v || !a->slot_map || !a->q_out ||
        (a->cos_sin && (!a->positions || a->table_len < 1 || a->rot_dim < 0)))
        return SPEC_ERR_INVALID_ARG;
    if (!rows_ok(a->q) || !rows_ok(a->k) || !rows_ok(a->v) || !cache_ok(h, a->cache) || !aligned16(a->q_out) ||
        !aligned16(a->q_weight) || !aligned16(a->k_weight) || !aligned16(a->cos_sin) ||
        (a->cos_sin && (a->rot_dim % 16 || a->rot_dim > h->cfg.head_dim)))
        return SPEC_ERR_UNSUPPORTED;
    DeviceGuard g(h->cfg.device);
    if (!g.ok) return SPEC_ERR_CUDA;
    TreeAppendParams p = {};
    p.s = shape(h, a->batch, a->tokens, nullptr, a->n_tokens);
    p.q = rows(a->q);
    p.k = rows(a->k);
    p.v = rows(a->v);
    p.c = cache(a->cache);
    p.slot_map = a->slot_map;
    p.positions = a->positions;
    p.qw = a->q_weight;
    p.kw = a->k_weight;
    p.cos_sin = a->cos_sin;
    p.table_len = a->table_len;
    p.rot = a->cos_sin ? a->rot_dim : 0;
    p.interleaved = a->interleaved ? 1 : 0;
    p.eps = a->eps;
    p.q_out = a->q_out;
    return launched(launch_tree_append(p, h->cfg.dtype, h->num_sms, (cudaStream_t)stream));
}

spec_status spec_tree_attend(spec_tree_t h, const spec_tree_attend_args* a, void* stream)
{
    if (!h || !a || !batch_ok(h, a->batch, a->tokens) || !(a->scale > 0.f) || isinf(a->scale))
        return SPEC_ERR_INVALID_ARG;
    if (a->batch == 0) return SPEC_OK;
    if (!a->q.ptr || !a->cache.k || !a->cache.v || !a->block_table || !a->ctx_len || !a->out ||
        (a->tree_mask && a->tokens > SPEC_TREE_MAX_NODES))
        return SPEC_ERR_INVALID_ARG;
    if (!rows_ok(a->q) || !cache_ok(h, a->cache) || !aligned16(a->out) || !aligned16(a->lse))
        return SPEC_ERR_UNSUPPORTED;
    // tensor maps: a stride of 0 only where there is one element
    const spec_tree_config& c = h->cfg;
    if ((a->batch > 1 && !a->q.seq_stride) || (a->tokens > 1 && !a->q.token_stride) ||
        (c.q_heads > 1 && !a->q.head_stride))
        return SPEC_ERR_UNSUPPORTED;
    DeviceGuard g(h->cfg.device);
    if (!g.ok) return SPEC_ERR_CUDA;
    TreeAttendParams p = {};
    p.s = shape(h, a->batch, a->tokens, a->ctx_len, a->n_tokens);
    if (!tree_attend_fits(p.s)) return SPEC_ERR_UNSUPPORTED;
    p.q = rows(a->q);
    p.c = cache(a->cache);
    p.table = a->block_table;
    p.mask = a->tree_mask;
    p.words = (a->tokens + 31) / 32;
    p.scale = a->scale;
    p.out = a->out;
    p.lse = a->lse;
    const bool stall = h->fault == SPEC_FAULT_STALL_STREAM;
    h->fault = SPEC_FAULT_NONE;
    return launched(launch_tree_attend(p, h->cfg.dtype, h->num_sms, h->parts, h->err, stall, (cudaStream_t)stream));
}

spec_status spec_tree_keep(spec_tree_t h, const spec_tree_keep_args* a, void* stream)
{
    if (!h || !a || !batch_ok(h, a->batch, a->tokens)) return SPEC_ERR_INVALID_ARG;
    if (a->batch == 0) return SPEC_OK;
    if (!a->cache.k || !a->cache.v || a->cache.layers < 1 || a->cache.layers > 65535 || !a->block_table ||
        !a->ctx_len || !a->path || !a->path_len || !a->ctx_out || a->ctx_out == a->ctx_len)
        return SPEC_ERR_INVALID_ARG;
    if (!cache_ok(h, a->cache) || !stride_ok(a->cache.layer_stride) ||
        (a->cache.layers > 1 && !a->cache.layer_stride))
        return SPEC_ERR_UNSUPPORTED;
    DeviceGuard g(h->cfg.device);
    if (!g.ok) return SPEC_ERR_CUDA;
    TreeKeepParams p = {};
    p.s = shape(h, a->batch, a->tokens, a->ctx_len, a->n_tokens);
    p.c = cache(a->cache);
    p.table = a->block_table;
    p.path = a->path;
    p.path_len = a->path_len;
    p.plan_status = a->plan_status;
    p.ctx_out = a->ctx_out;
    p.row_status = a->row_status;
    return launched(launch_tree_keep(p, (cudaStream_t)stream));
}

}  // extern "C"
