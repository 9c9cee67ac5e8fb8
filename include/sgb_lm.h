/*
 * sgb_lm.h -- C ABI of the token-model operators (libsgb_lm.so): what stands
 * around an embedding table's rows in a language model that is trained or
 * served with them.
 *
 *  - block norms: the norm of a block's output, its gate, the scaled residual
 *    and the norm before the next block, in one pass; forward and backward;
 *  - distillation from a teacher's top logits: loss and gradient of the
 *    student's logits, with the teacher's tail mass and the labels'
 *    cross-entropy;
 *  - logits penalties before sampling: repetition, frequency and presence,
 *    biases, grammar masks.
 *
 * Conventions are those of sgb.h: plain C, status codes and element types
 * (SGB_F32, SGB_BF16, SGB_F16) from there, device pointers owned by the
 * caller and kept alive until the work enqueued on `stream` has finished
 * (a hipStream_t as void*, NULL = the null stream).  Host-detected errors
 * return before anything is enqueued.  Nothing is allocated, no memset is
 * recorded and the host never waits, except in sgb_lm_device_status(), so
 * every call can be captured into a HIP graph.  A plan belongs to the device
 * current at its creation and every call on it runs there; one made where
 * there is no device checks arguments and ends every valid call with
 * SGB_ERR_HIP.  Results do not
 * depend on timing: no floating-point atomics.
 *
 * A matrix argument is a pointer to row 0 and a row stride in elements (>= its
 * width; the elements of a row are adjacent).  Pointers need no more than their
 * element's alignment, but for stats, four floats a row that are read at once:
 * 16 bytes, where they are written too.  Rows may be 0: nothing is enqueued,
 * and gradient sums over rows are then written as zeros; the most are 2^31 - 1
 * for block norms, and for the others what one launch of fewer than 2^32
 * threads takes (SGB_ERR_UNSUPPORTED past it): 2^24 - 1 rows of up to 32 KB of
 * logits for distillation, 2^23 - 1 rows of up to 1024 logits for penalties,
 * fewer the longer.  Outputs must not overlap inputs or each other except where
 * a line here says so.  Refused are overlaps among the matrices of D, V or
 * vocab columns, and of the parameters' gradients with other outputs; the rest
 * (stats, losses, lists) is the caller's care.
 *
 * `workspace` is a device buffer, 256-byte aligned, of at least the size that
 * the operator's *_workspace_bytes() gives for that many rows or for more; its
 * contents need no initialisation.  Two calls that may run at the same time
 * need one each.
 */
#ifndef SGB_LM_H
#define SGB_LM_H

#include <stddef.h>
#include <stdint.h>

#include "sgb.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * sgb_lm_device_status -- synchronises `stream`, then stores in *out the
 * first error the kernels of the last call with rows that used `workspace`
 * recorded (SGB_OK if none; the replays of a captured call count as one call).
 * Distillation and penalties record
 * SGB_ERR_INDEX_OUT_OF_RANGE (an entry, label, token, bias id or mask index
 * at or past its range; it is left out and the rest computed) and
 * SGB_ERR_BAD_OFFSETS (a length outside its range; it is clamped).
 */
sgb_status sgb_lm_device_status(const void* workspace, void* stream, int32_t* out);

/* ------------------------------------------------------------ block norms
 *
 * For each row r, with gate row r / rows_per_gate:
 *     z     = post(h[r])                      post, pre: none (the identity),
 *     x_out = res_scale * x[r] + gate * z     rms: v / sqrt(mean(v^2) + eps) * weight,
 *     y     = pre(x_out)                      layer: (v - mean(v)) / sqrt(var(v) + eps)
 * each norm's product plus its bias where there is one (layer or rms).
 * Everything is computed in fp32 and rounded once per output; y comes from
 * the unrounded x_out.
 */
typedef enum { SGB_NORM_NONE = 0, SGB_NORM_RMS = 1, SGB_NORM_LAYER = 2 } sgb_norm_kind;

typedef struct sgb_block_norm_s* sgb_block_norm;

/* D: 1..8192 columns; eps >= 0. */
sgb_status sgb_block_norm_create(sgb_block_norm* out, int32_t D, int32_t post, int32_t pre,
                                 float post_eps, float pre_eps, float res_scale);
void sgb_block_norm_destroy(sgb_block_norm plan);
sgb_status sgb_block_norm_workspace_bytes(sgb_block_norm plan, int64_t rows, size_t* bytes);

/* The norms' parameters, [D] each: a weight for each norm that is not none
 * (NULL for none), a bias or NULL.  All of one type. */
typedef struct {
  const void* post_weight;
  const void* post_bias;
  const void* pre_weight;
  const void* pre_bias;
  int32_t dtype;                    /* F32, BF16 or F16                     */
} sgb_norm_params;

typedef struct {
  const void* x;                    /* [rows][D], res_dtype                 */
  const void* h;                    /* [rows][D], dtype                     */
  void* x_out;                      /* [rows][D], res_dtype; may be x       */
  void* y;                          /* [rows][D], dtype; NULL iff pre none;
                                       may be h                             */
  const void* gate;                 /* [ceil(rows / rows_per_gate)][D],
                                       dtype, or NULL (a gate of one)       */
  float* stats;                     /* [rows][4] or NULL: mean and 1/deviation
                                       of h, then of x_out, as the backward
                                       reads them (mean 0 for rms; 0 and 1
                                       for none)                            */
  int64_t x_stride, h_stride, x_out_stride, y_stride, gate_stride;
  int64_t rows;
  int64_t rows_per_gate;            /* >= 1 with a gate                     */
  int32_t dtype;                    /* F32, BF16, F16                       */
  int32_t res_dtype;                /* F32 or dtype                         */
} sgb_norm_forward_args;

sgb_status sgb_block_norm_forward(sgb_block_norm plan, const sgb_norm_params* params,
                                  const sgb_norm_forward_args* args, void* stream);

/*
 * Gradients of all of the above from dx_out (of x_out as the next layers see
 * it) and dy.  x_out, h, gate and stats are the forward's.  dx may be dx_out,
 * dh may be dy or h, d_gate has gate's type; sums over rows (d_gate over a
 * gate's rows, the parameters' over all) are fp32 sums in a fixed order.
 * Any of d_gate, d_post_*, d_pre_* may be NULL: not wanted.  rows = 0 writes
 * zeros into the parameters' gradients.
 */
typedef struct {
  const void* dx_out;               /* [rows][D], res_dtype                 */
  const void* dy;                   /* [rows][D], dtype; NULL iff pre none  */
  const void* x_out;                /* [rows][D], res_dtype (not read where
                                       pre is none)                         */
  const void* h;                    /* [rows][D], dtype (not read where post
                                       is none and d_gate NULL)             */
  const float* stats;               /* [rows][4]                            */
  const void* gate;                 /* as in the forward                    */
  void* dx;                         /* [rows][D], res_dtype                 */
  void* dh;                         /* [rows][D], dtype                     */
  void* d_gate;                     /* gate's shape and type                */
  float* d_post_weight;             /* [D] each                             */
  float* d_post_bias;
  float* d_pre_weight;
  float* d_pre_bias;
  int64_t dx_out_stride, dy_stride, x_out_stride, h_stride, gate_stride, dx_stride, dh_stride,
      d_gate_stride;
  int64_t rows;
  int64_t rows_per_gate;
  int32_t dtype;
  int32_t res_dtype;
} sgb_norm_backward_args;

sgb_status sgb_block_norm_backward(sgb_block_norm plan, const sgb_norm_params* params,
                                   const sgb_norm_backward_args* args, void* workspace,
                                   size_t workspace_bytes, void* stream);

/* ----------------------------------------------------------- distillation
 *
 * Row r has the student's logits x[V] and the teacher's K listed logits
 * v_k at ids_k (an id < 0: not listed).  With q = softmax(x / T):
 *  without teacher_lse  p = softmax(v / T) over the listed entries,
 *      KL = sum_k p_k (log p_k - log q[ids_k]);
 *  with it (the teacher's log-sum-exp of logits / T over its whole
 *      vocabulary)  p_k = exp(v_k / T - lse), the rest p' = max(0, 1 - sum p)
 *      against the student's mass q' outside the listed ids:
 *      KL = sum_k p_k (log p_k - log q[ids_k]) + p' (log p' - log q');
 *      p' is 0 where every id is listed, and where it is no more than what
 *      the rounding of an fp32 lse leaves, 2^-20 (1 + |lse|), while every
 *      logit outside is -inf or 150 T ln 2 below the largest listed (q' below
 *      2^-126): tokens barred for teacher and student alike;
 *  KL = 0 where nothing is listed.
 *      loss = weight * (kd_weight * T^2 * KL + ce_weight * CE),
 * CE the cross-entropy of softmax(x) at the label (0 for a label < 0).
 * The gradient is grad_scale * grad_loss * d loss / d x, in the logits' type.
 *
 * A row of weight 0 (padding) is not read: its loss and gradient are 0 whatever
 * it holds.  -inf logits have q = 0; any other row of nothing else has no
 * distribution, and whatever is listed its loss and gradient are NaN.  An id
 * listed twice counts twice in the sums over k and once in q'.
 */
typedef struct sgb_distill_s* sgb_distill;

/* V: 1..2^23; K: 1..1024; T > 0 with log2(e) / T finite in fp32; the weights finite. */
sgb_status sgb_distill_create(sgb_distill* out, int64_t V, int32_t K, float temperature,
                              float kd_weight, float ce_weight);
void sgb_distill_destroy(sgb_distill plan);
sgb_status sgb_distill_workspace_bytes(sgb_distill plan, int64_t rows, size_t* bytes);

typedef struct {
  const void* logits;               /* [rows][V], dtype                     */
  const int64_t* ids;               /* [rows][K]                            */
  const float* values;              /* [rows][K] teacher logits             */
  const float* teacher_lse;         /* [rows] or NULL                       */
  const int64_t* labels;            /* [rows]; NULL iff ce_weight is 0      */
  const float* row_weights;         /* [rows] or NULL (1)                   */
  float* loss;                      /* [rows] (not written by backward)     */
  float* stats;                     /* [rows][4] or NULL: written by forward,
                                       read by backward                     */
  const float* grad_loss;           /* [rows] or NULL (1); backward only    */
  void* grad;                       /* [rows][V], dtype                     */
  int64_t logits_stride, ids_stride, values_stride, grad_stride;
  int64_t rows;
  int32_t dtype;                    /* F32, BF16, F16                       */
  float grad_scale;
} sgb_distill_args;

/* loss (and stats); grad, grad_loss and grad_scale are not looked at. */
sgb_status sgb_distill_forward(sgb_distill plan, const sgb_distill_args* args, void* workspace,
                               size_t workspace_bytes, void* stream);
/* grad, from a forward's stats on the same inputs. */
sgb_status sgb_distill_backward(sgb_distill plan, const sgb_distill_args* args, void* workspace,
                                size_t workspace_bytes, void* stream);
/* loss and grad in one go (grad_loss and stats are not looked at). */
sgb_status sgb_distill_loss_grad(sgb_distill plan, const sgb_distill_args* args, void* workspace,
                                 size_t workspace_bytes, void* stream);

/* -------------------------------------------------------- logits penalties
 *
 * Row r has the tokens so far, tokens[0 .. len): a prompt of prompt_len, then
 * what was generated.  For each token v of the vocabulary, in this order:
 *  1. seen anywhere in the sequence: x = x > 0 ? x / repetition : x * repetition;
 *  2. generated n > 0 times: x -= frequency * n + presence;
 *  3. x += the sum of the row's biases at v;
 *  4. a mask row is chosen and its bit for v is 0: x = -inf.
 * In fp32, rounded once; a token that none of them touches keeps its bits (but a
 * signalling NaN of 16 bits may come out quiet).
 */
typedef struct sgb_penalty_s* sgb_penalty;

/* vocab: 1..2^31-1. */
sgb_status sgb_penalty_create(sgb_penalty* out, int64_t vocab);
void sgb_penalty_destroy(sgb_penalty plan);
sgb_status sgb_penalty_workspace_bytes(sgb_penalty plan, int64_t rows, size_t* bytes);

typedef struct {
  const void* logits;               /* [rows][vocab], dtype                 */
  void* out;                        /* [rows][vocab], dtype; may be logits  */
  const int32_t* tokens;            /* [rows][max_tokens]; tokens < 0 stand
                                       for nothing                          */
  const int32_t* prompt_lens;       /* [rows] or NULL (0): of lens          */
  const int32_t* lens;              /* [rows] or NULL (max_tokens)          */
  const float* repetition;          /* [rows] or NULL (1)                   */
  const float* frequency;           /* [rows] or NULL (0)                   */
  const float* presence;            /* [rows] or NULL (0)                   */
  const int32_t* bias_ids;          /* [rows][num_biases], < 0: none; or NULL */
  const float* bias_values;         /* [rows][num_biases]; NULL iff bias_ids */
  const int32_t* mask;              /* [num_masks][mask_stride] words, bit
                                       v % 32 of word v / 32 set: allowed;
                                       or NULL                              */
  const int32_t* mask_index;        /* [rows], < 0: no mask; or NULL: row r
                                       has mask r (num_masks = rows)        */
  int64_t logits_stride, out_stride, tokens_stride, bias_ids_stride, bias_values_stride,
      mask_stride;
  int64_t rows;
  int32_t max_tokens;               /* 0..2^21-1; 0: tokens may be NULL     */
  int32_t num_biases;               /* 0..1023                              */
  int32_t num_masks;
  int32_t dtype;                    /* F32, BF16, F16                       */
} sgb_penalty_args;

sgb_status sgb_penalty_apply(sgb_penalty plan, const sgb_penalty_args* args, void* workspace,
                             size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SGB_LM_H */
