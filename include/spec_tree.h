/*
 * spec_tree.h -- C ABI of the operators around a verify step: the drafted
 * tokens of B sequences, a chain or a tree each, go through the target
 * model's attention over a paged cache of keys and values, and the accepted
 * ones stay in that cache (GB300, sm_103a).
 *
 * One round, per sequence b with ctx_b tokens in the cache and n_b drafted
 * tokens ("nodes" 0 .. n_b - 1, each node's parent before it):
 *   spec_tree_plan    pages for ctx_b + n_b tokens from a ring of free pages,
 *                     the node's slots in the cache, their positions and their
 *                     ancestor masks (once a round);
 *   spec_tree_append  per layer: RMS norm of every query and key head, the
 *                     position rotation, keys and values into their slots;
 *   spec_tree_attend  per layer: attention of every node over the context and
 *                     its ancestors;
 *   (the LM head and spec_verify_run choose the accepted path)
 *   spec_tree_keep    the accepted nodes' keys and values moved together
 *                     behind the context, in all layers, and the new lengths.
 * A prompt is a round too: a chain of n_b tokens, no parents.  n_b = 1 is
 * ordinary decoding.
 *
 * The cache.  num_pages pages of page_size tokens; token i of sequence b lies
 * in page block_table[b][i / page_size] at i % page_size, its slot being
 * page * page_size + i % page_size.  K and V are two tensors of one layout
 * [pages, tokens, heads, head_dim] with free strides (spec_tree_cache); the
 * last dimension is contiguous.  Node j of sequence b is token ctx_b + j.
 *
 * Conventions are those of spec_verify.h: device pointers owned by the caller,
 * asynchronous calls on the given stream without synchronisation or
 * allocation, host-side errors launch nothing, one handle on one stream at a
 * time.  Sequences are padded to T nodes (n_tokens[b] <= T of them count;
 * n_tokens NULL: all T).  Offsets into the cache are 64-bit.
 */
#ifndef SPEC_TREE_H
#define SPEC_TREE_H

#include <stdint.h>

#include "spec_verify.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct spec_tree* spec_tree_t; /* opaque handle */

/* the 16-bit types of queries, keys, values and outputs: SPEC_BF16 of
 * spec_dtype, and IEEE half precision */
enum { SPEC_F16 = 2 };

/* per-sequence row_status values of this header (0 is SPEC_ROW_OK) */
enum {
    SPEC_ROW_BAD_LEN = 5,  /* ctx < 0, n outside [0, T], held outside [0, table_width], */
                           /* ctx + n beyond the table, or a path longer than n          */
    SPEC_ROW_BAD_TREE = 6, /* a parent outside [-1, j) for node j; a path not ascending  */
    SPEC_ROW_NO_PAGES = 7  /* the ring of free pages is too short for this sequence;     */
                           /* keep: a token's page is not in the cache                   */
};

/* largest T of a tree (chains, i.e. calls without parents or masks, have no
 * limit but the handle's max_tokens) */
#define SPEC_TREE_MAX_NODES 256

typedef struct {
    int32_t device;      /* CUDA device ordinal                                          */
    int32_t max_batch;   /* largest B of any call                                        */
    int32_t max_tokens;  /* largest T of any call                                        */
    int32_t q_heads;     /* Hq, a multiple of kv_heads                                   */
    int32_t kv_heads;    /* Hkv                                                          */
    int32_t head_dim;    /* D: a multiple of 16, 16 <= D <= 256                          */
    int32_t dtype;       /* SPEC_BF16 or SPEC_F16                                        */
    int32_t page_size;   /* tokens per page: a power of two, 8 <= page_size <= 1024      */
    int32_t num_pages;   /* pages of the cache (and places of the ring of free pages)    */
    int32_t table_width; /* pages per row of a block table                               */
} spec_tree_config;

/* Create / destroy a handle: it owns the workspace of spec_tree_attend's
 * partial sums (from the allocator of spec_verify_set_allocator when one is
 * set).  SPEC_ERR_INVALID_ARG for sizes < 1, q_heads not a multiple of
 * kv_heads, num_pages * page_size or table_width * page_size beyond 2^31 - 1;
 * SPEC_ERR_UNSUPPORTED for a dtype (SPEC_F32 included), head_dim or page_size
 * outside the table above, or more than 128 query heads per key head. */
spec_status spec_tree_create(const spec_tree_config* cfg, spec_tree_t* out);
spec_status spec_tree_destroy(spec_tree_t h);

/* As spec_verify_check: waits for `stream`, then reads and clears the record
 * of device-side waits that ran out in spec_tree_attend. */
spec_status spec_tree_check(spec_tree_t h, void* stream);

/* As spec_verify_inject_fault (host side only): after SPEC_FAULT_STALL_STREAM
 * the next spec_tree_attend issues no copy, so that its bounded waits run out
 * and the record is set; its outputs are undefined. */
spec_status spec_tree_inject_fault(spec_tree_t h, int32_t fault);

/* ------------------------------------------------------------------------ */
/* plan                                                                      */
/* ------------------------------------------------------------------------ */
/* The free pages are a ring of num_pages places: pages free_pages[i mod
 * num_pages] for ring[0] <= i < ring[1] are free.  Sequence b holds the first
 * held[b] pages of its table row and needs need_b = ceil((ctx_b + n_b) /
 * page_size).
 *  - need_b > held_b: the next need_b - held_b pages of the ring, sequences
 *    in order, are written to its table row.  A sequence whose pages, those
 *    of the sequences before it included, go past the ring's end gets none and
 *    SPEC_ROW_NO_PAGES (and so do all behind it that need any), and -1 in the
 *    entries of its row that the missing pages would have filled: what they
 *    held may be another sequence's page by now.  Pages returned by this call
 *    are free from the next call on.
 *  - need_b < held_b: its last held_b - need_b pages go to the ring's end, in
 *    the order of the sequences.  ctx = n = 0 returns all pages of a sequence.
 * Inputs and outputs are separate buffers where both exist (held, ring): a
 * call whose inputs are unchanged can be repeated and gives the same result.
 * block_table and free_pages are updated in place; other entries of a row
 * beyond held_out are left as they are.
 * slot_map[b][j] and positions[b][j] (ctx_b + the node's depth; a root, parent
 * -1, has depth 0) are -1 for j >= n_b, for sequences whose status is not 0, and
 * for a node whose page, as the table has it, is not in the cache.
 * tree_mask[b][j] has bit i set iff node i is node j or an ancestor of it (bit i
 * of a row is bit i % 32 of word i / 32), and is 0 where slot_map is -1.  A
 * sequence with SPEC_ROW_BAD_TREE has its pages as its lengths ask. */
typedef struct {
    const int32_t* ctx_len;  /* [B]                                                   */
    const int32_t* n_tokens; /* [B] or NULL (T each)                                  */
    const int32_t* parents;  /* [B, T], parents[b][j] in [-1, j), or NULL: chains     */
    const int32_t* held;     /* [B]                                                   */
    const int64_t* ring;     /* [2]: head, tail; 0 <= tail - head <= num_pages        */
    int32_t* free_pages;     /* [num_pages], updated                                  */
    int32_t* block_table;    /* [B, table_width], updated                             */
    int32_t batch;           /* B, 0 <= B <= max_batch (0 copies the ring)            */
    int32_t tokens;          /* T, 1 <= T <= max_tokens (256 with parents)            */
    int32_t* held_out;       /* [B], not held                                         */
    int64_t* ring_out;       /* [2], not ring                                         */
    int32_t* slot_map;       /* [B, T]                                                */
    int32_t* positions;      /* [B, T]                                                */
    uint32_t* tree_mask;     /* [B, T, ceil(T / 32)]; required with parents, else NULL */
    int32_t* row_status;     /* [B]                                                   */
} spec_tree_plan_args;
spec_status spec_tree_plan(spec_tree_t h, const spec_tree_plan_args* a, void* stream);

/* a tensor [B, T, heads, head_dim] with free strides (in elements); the last
 * dimension is contiguous */
typedef struct {
    const void* ptr;
    int64_t seq_stride, token_stride, head_stride;
} spec_tree_rows;

/* the cache of one layer (or, for spec_tree_keep, of all): strides in
 * elements, the same for K and V */
typedef struct {
    void* k;
    void* v;
    int64_t page_stride, token_stride, head_stride;
    int64_t layer_stride; /* spec_tree_keep only                                      */
    int32_t layers;       /* spec_tree_keep only: >= 1                                */
} spec_tree_cache;

/* ------------------------------------------------------------------------ */
/* append                                                                    */
/* ------------------------------------------------------------------------ */
/* y = x * w / sqrt(mean(x^2) + eps) over each head of q (w = q_weight) and k
 * (k_weight), no norm where the weight is NULL; then, when cos_sin is given,
 * the pairs (a, b) of the first rot_dim elements of y become (a cos - b sin,
 * b cos + a sin), row `position` of cos_sin holding rot_dim / 2 cosines and
 * then rot_dim / 2 sines.  Pair i is elements (i, i + rot_dim / 2), or
 * (2 i, 2 i + 1) when interleaved.  All in fp32, rounded once.  q goes to
 * q_out, k and v (as it is) to their slots.  A node j >= n_b or with a slot
 * outside the cache gets a zero row in q_out and writes nothing to the cache;
 * one whose position cos_sin does not hold gets NaN in the first rot_dim elements
 * of q_out and k.
 * SPEC_ERR_UNSUPPORTED when a pointer to q, k, v, q_out, the weights or the
 * cache is not on 16 bytes, a stride is not a multiple of 8 elements (or is
 * beyond 2^36), a stride of the cache is 0 for a dimension larger than 1, or
 * rot_dim is not a multiple of 16 within [0, head_dim]. */
typedef struct {
    spec_tree_rows q, k, v;
    spec_tree_cache cache;
    const int32_t* slot_map;  /* [B, T]                                               */
    const int32_t* positions; /* [B, T], used with cos_sin                            */
    const int32_t* n_tokens;  /* [B] or NULL                                          */
    const void* q_weight;     /* [head_dim] of the handle's dtype, or NULL            */
    const void* k_weight;
    const float* cos_sin;     /* [table_len, rot_dim], on 16 bytes, or NULL           */
    int32_t table_len, rot_dim;
    int32_t interleaved;      /* 0 or 1                                               */
    float eps;                /* >= 0                                                 */
    int32_t batch, tokens;
    void* q_out;              /* [B, T, q_heads, head_dim], contiguous                */
} spec_tree_append_args;
spec_status spec_tree_append(spec_tree_t h, const spec_tree_append_args* a, void* stream);

/* ------------------------------------------------------------------------ */
/* attend                                                                    */
/* ------------------------------------------------------------------------ */
/* out[b][j][h] = sum_k p_k V[k], p = softmax over the keys that node j sees of
 * scale * (q[b][j][h] . K[k]) with key head h / (q_heads / kv_heads).  Node j
 * sees the tokens below ctx_b and those nodes i < n_b whose bit is set in
 * tree_mask[b][j] (any bits: a node need not see itself); without a mask the
 * nodes i <= j.  What a node does not see has no effect on its row, whatever
 * its values; an infinite value that it sees gives that infinity, or NaN where
 * its probability rounds to 0.  lse is the natural logarithm of the sum of exp
 * over the scores.  A node that sees nothing, whose finite sum is 0, or with
 * j >= n_b has a zero row and lse = -inf; so has every node of a sequence with
 * ctx < 0, n outside [0, T] or ctx + n beyond the table.  Keys and values of a
 * page outside the cache are zeros (a sequence that spec_tree_plan left without
 * pages: its rows have no meaning, and its status says so).  Scores, sums and
 * outputs accumulate in fp32; the probabilities are rounded to the 16-bit type
 * (in f16 in units of 2^-7 of the largest so far) before they meet V.
 * SPEC_ERR_UNSUPPORTED when q, the cache, out or lse is not on 16 bytes, a
 * stride is not a multiple of 8 elements (or is beyond 2^36), or is 0 for a
 * dimension larger than 1; or when the key tiles of the call could pass 2^31:
 * B * kv_heads * ceil(T / R) * (ceil(table_width * page_size / 64) + 4), where
 * R = 2 floor(128 / G) nodes for head_dim <= 128 and floor(128 / G) above, G =
 * q_heads / kv_heads.  T and the table count there, not the lengths in use. */
typedef struct {
    spec_tree_rows q;
    spec_tree_cache cache;
    const int32_t* block_table; /* [B, table_width]                                   */
    const int32_t* ctx_len;     /* [B]                                                */
    const int32_t* n_tokens;    /* [B] or NULL                                        */
    const uint32_t* tree_mask;  /* [B, T, ceil(T / 32)] or NULL; T <= 256 with a mask */
    float scale;                /* finite, > 0                                        */
    int32_t batch, tokens;
    void* out;                  /* [B, T, q_heads, head_dim], contiguous              */
    float* lse;                 /* [B, T, q_heads] or NULL                            */
} spec_tree_attend_args;
spec_status spec_tree_attend(spec_tree_t h, const spec_tree_attend_args* a, void* stream);

/* ------------------------------------------------------------------------ */
/* keep                                                                      */
/* ------------------------------------------------------------------------ */
/* For every sequence, layer and i < path_len[b]: token ctx_b + i of K and V
 * becomes token ctx_b + path[b][i]; ctx_out[b] = ctx_b + path_len[b].  A path
 * is strictly ascending within [0, n_b) (a node's parent comes before it, so
 * a path from a root is).  A sequence with a path that is not, or with lengths
 * outside their ranges, keeps its cache and length and gets SPEC_ROW_BAD_TREE
 * or SPEC_ROW_BAD_LEN, and so does one whose table row gives no page of the
 * cache for a token of the path or its new place, with SPEC_ROW_NO_PAGES.
 * plan_status is the row_status of the round's spec_tree_plan: a sequence with
 * a status there keeps its cache, its length and that status, as append has
 * written none of its nodes.  Pages of different sequences must be different.
 * SPEC_ERR_UNSUPPORTED when the cache is not on 16 bytes, a stride is not a
 * multiple of 8 elements (or is beyond 2^36), or is 0 for a dimension larger
 * than 1. */
typedef struct {
    spec_tree_cache cache;
    const int32_t* block_table; /* [B, table_width]                                   */
    const int32_t* ctx_len;     /* [B]                                                */
    const int32_t* n_tokens;    /* [B] or NULL                                        */
    const int32_t* path;        /* [B, T]                                             */
    const int32_t* path_len;    /* [B], 0 <= path_len <= n_b                          */
    int32_t batch, tokens;
    int32_t* ctx_out;           /* [B], not ctx_len                                   */
    int32_t* row_status;        /* [B] or NULL                                        */
    const int32_t* plan_status; /* [B] or NULL (every sequence was planned)           */
} spec_tree_keep_args;
spec_status spec_tree_keep(spec_tree_t h, const spec_tree_keep_args* a, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* SPEC_TREE_H */
