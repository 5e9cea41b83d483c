/*
 * spec_score.h -- C ABI of the operators that score rows of logits beside a
 * verify step (GB300, sm_103a): what a server reports about the emitted tokens,
 * and what a draft model learns from.
 *
 *   spec_score_logprobs  the log probability and rank of a given token of every
 *                        row, the row's entropy and its likeliest tokens; and
 *                        the gradient of log probability and entropy;
 *   spec_score_distill   the divergence of a row's distribution (the student's,
 *                        the draft's) from a teacher's of which the top logits
 *                        are known, and its gradient.  spec_score_logprobs over
 *                        the target's rows records such a teacher.
 *
 * Rows.  Logits are [B, T, V] (spec_score_rows): V contiguous elements of bf16,
 * f16 or fp32 per row, free strides between sequences and positions, any
 * alignment of the element type.  Everything else a row has (tokens, values,
 * results) is contiguous, row b * T + t.  Row offsets are 64-bit.
 * For logits l and temperature t: M = max l, Z = sum exp((l_v - M) / t), p_v =
 * exp((l_v - M) / t) / Z, and lse = M / t + ln Z.  Sums are held in 32 bits or
 * more, results are fp32, a gradient is rounded once to the type of the logits.
 *
 * Masked tokens are logits of -inf: probability 0.  The type's lowest value is
 * a value like any other.  A NaN or +inf logit, or a row without a finite one,
 * is SPEC_ROW_NONFINITE.  A row with a status other than 0 has NaN results, ids
 * and ranks of -1, and a gradient of 0: it trains nothing.
 *
 * Conventions are those of spec_verify.h: device pointers owned by the caller,
 * asynchronous calls on the given stream, errors found on the host launch
 * nothing.  There is no handle and no workspace: calls share nothing, may
 * overlap on any streams, and can be captured.  B = 0 or T = 0 is a no-op.
 * Results do not depend on the order in which the SMs work.
 *
 * Limits: V elements of at most 8 * 208 KB (425984 of fp32, 851968 of 16 bits),
 * B * T * 8 below 2^31; beyond them SPEC_ERR_UNSUPPORTED.
 */
#ifndef SPEC_SCORE_H
#define SPEC_SCORE_H

#include <stdint.h>

#include "spec_tree.h" /* SPEC_F16 */
#include "spec_verify.h"

#ifdef __cplusplus
extern "C" {
#endif

#define SPEC_SCORE_MAX_TOP 128     /* largest top_n of spec_score_logprobs              */
#define SPEC_SCORE_MAX_ENTRIES 256 /* largest number of teacher entries of a row        */

typedef struct {
    void* ptr;            /* element [0][0][0], aligned to its type                     */
    int64_t seq_stride;   /* elements from a sequence to the next                       */
    int64_t token_stride; /* elements from a position to the next                       */
} spec_score_rows;

typedef struct {
    int32_t device;       /* CUDA device ordinal                                        */
    int32_t dtype;        /* SPEC_BF16, SPEC_F16 or SPEC_F32: logits and gradient       */
    int32_t batch;        /* B                                                          */
    int32_t tokens;       /* T                                                          */
    int32_t vocab;        /* V                                                          */
    int32_t top_n;        /* likeliest tokens to report, 0 <= top_n <= MAX_TOP          */
    float temperature;    /* 1e-30 to 1e30                                              */
    spec_score_rows logits;
    const int32_t* ids;        /* [B, T] tokens, -1: row not scored; or NULL            */
    const float* grad_logprob; /* [B, T] upstream gradient of logprob, or NULL: 0       */
    const float* grad_entropy; /* [B, T] upstream gradient of entropy, or NULL: 0       */
    float* logprob;            /* [B, T] ln p_x, or NULL                                */
    int32_t* rank;             /* [B, T] number of tokens before x in the order (logit  */
                               /* desc, id asc), all masked tokens being last and none  */
                               /* before another; or NULL                               */
    float* entropy;            /* [B, T] - sum p ln p, in nats; or NULL                 */
    float* lse;                /* [B, T] or NULL                                        */
    int32_t* top_ids;          /* [B, T, top_n] the first tokens in that order, -1      */
                               /* where no unmasked one is left                         */
    float* top_logprobs;       /* [B, T, top_n] their ln p, -inf where there is none    */
    int32_t* row_status;       /* [B, T] SPEC_ROW_OK, _NONFINITE or _BAD_TOKEN          */
    spec_score_rows grad;      /* [B, T, V] of the logits' type, or ptr NULL            */
} spec_score_logprobs_args;

/* Log probabilities of given tokens, with entropy and top alternatives.
 * Without ids every row is scored, without logprob and rank.  With ids, a row
 * of -1 is neither read nor scored: logprob, entropy and lse 0 (sums over a
 * padded batch are the sums of its tokens), rank and top_ids -1, top_logprobs
 * -inf, status 0, gradient 0.  Another id outside [0, V) is
 * SPEC_ROW_BAD_TOKEN.
 * The gradient, of sum over rows of grad_logprob ln p_x + grad_entropy H:
 *   (grad_logprob (1[v = x] - p_v) - grad_entropy p_v (ln p_v + H)) / t
 * and 0 for masked tokens other than x.  It may be written over the logits
 * (the same pointer and strides); otherwise the two must not overlap, and no
 * two rows of the gradient may.
 * SPEC_ERR_INVALID_ARG: a NULL where one is needed (row_status; logits; ids of
 * logprob, rank or grad_logprob; top_ids and top_logprobs of top_n; grad of an
 * upstream gradient and the reverse), sizes < 0, V < 1, a bad temperature or
 * dtype, a negative stride.  SPEC_ERR_UNSUPPORTED: the limits above, top_n
 * beyond SPEC_SCORE_MAX_TOP, a pointer off its type's alignment. */
spec_status spec_score_logprobs(const spec_score_logprobs_args* args, void* stream);

typedef struct {
    int32_t device;        /* CUDA device ordinal                                       */
    int32_t dtype;         /* of student and gradient                                   */
    int32_t teacher_dtype; /* SPEC_BF16, SPEC_F16 or SPEC_F32                           */
    int32_t batch;         /* B                                                         */
    int32_t tokens;        /* T                                                         */
    int32_t vocab;         /* V                                                         */
    int32_t entries;       /* k teacher entries a row, 1 <= k <= MAX_ENTRIES            */
    int32_t tail;          /* 0: renormalised; 1: what is left is an outcome of its own */
    float temperature;         /* of the student's logits, 1e-30 to 1e30                */
    float teacher_temperature; /* of the teacher's values, 1e-30 to 1e30                */
    spec_score_rows student;
    const int32_t* ids;        /* [B, T, k] the entries' tokens, -1: no entry           */
    const void* teacher;       /* [B, T, k] the entries' logits, or log probabilities   */
    const float* teacher_lse;  /* [B, T] log-sum-exp of the teacher's logits over their */
                               /* temperature, all tokens; NULL: 0, i.e. the values     */
                               /* are log probabilities.  Only with tail.               */
    const float* grad_loss;    /* [B, T] upstream gradient of the loss, or NULL: 1      */
    float* loss;               /* [B, T] or NULL                                        */
    float* accept;             /* [B, T] or NULL                                        */
    int32_t* row_status;       /* [B, T] SPEC_ROW_OK, _NONFINITE or _BAD_TOKEN          */
    spec_score_rows grad;      /* [B, T, V] of the student's type, or ptr NULL          */
} spec_score_distill_args;

/* Distillation from a teacher's top logits.  With y_i = teacher_i /
 * teacher_temperature, S the tokens of the row's entries and p the student's
 * distribution:
 *   tail = 0: q = softmax(y) over the entries (the teacher with its top-k knob)
 *   tail = 1: q_i = exp(y_i - teacher_lse), q_r = max(0, 1 - sum q_i), p_r =
 *             sum of p_v, v not in S
 *   loss   = sum q_i (ln q_i - ln p_i)  [+ q_r (ln q_r - ln p_r)]
 *   accept = sum min(q_i, p_i): with tail = 0 the acceptance statistic alpha of
 *            spec_verify_outputs at these rows, with tail = 1 a lower bound
 *   gradient, times grad_loss: (m p_v - q_v) / temperature for v in S, (m p_v -
 *            q_r p_v / p_r) / temperature for the others (m p_v without tail),
 *            m = sum q_i [+ q_r]
 * A term with q = 0 is 0, one with q > 0 and p = 0 +inf (its gradient stays
 * finite; for p_r = 0 the others' is 0).  A row without an entry is neither read
 * nor scored: loss, accept and gradient 0, status 0.  A token twice in a row, or
 * one outside [-1, V), is SPEC_ROW_BAD_TOKEN; a NaN or +inf among the teacher's
 * values or a NaN or infinite teacher_lse, or, without tail, no finite value,
 * SPEC_ROW_NONFINITE.  The gradient may be written over the student's logits, as
 * in spec_score_logprobs.  Errors as there; teacher_lse without tail and entries
 * < 1 are SPEC_ERR_INVALID_ARG, entries beyond SPEC_SCORE_MAX_ENTRIES
 * SPEC_ERR_UNSUPPORTED. */
spec_status spec_score_distill(const spec_score_distill_args* args, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* SPEC_SCORE_H */
