/*
 * sgb_lm_step.h -- C ABI of further token-model operators of libsgb_lm.so: what
 * a training or serving step has next to those of sgb_lm.h.
 *
 *  - vocabulary cross-entropy: loss and gradients of the head's product over a
 *    large vocabulary, without a matrix of logits (with gradients, a chunk of
 *    rows has its exponentials in the workspace);
 *  - dropout from a counter-based generator, with the residual's addition:
 *    the mask is never stored;
 *  - quantising norm: root-mean-square norm with the residual's addition and
 *    an output in 8 bits with scales.
 *
 * Conventions are those of sgb_lm.h: status codes, element types, streams,
 * plans and their devices, matrices with row strides, workspaces
 * (sgb_lm_device_status() reads theirs), no allocation, no memset and no host
 * wait in a call, no floating-point atomics.  Pointers need no more than their
 * element's alignment.  An output, the workspace among them, that overlaps
 * anything else of the call is refused, but where a line here allows it.  Rows
 * may be 0: nothing is enqueued, but that a weight gradient that is not
 * accumulated is written as zeros.
 */
#ifndef SGB_LM_STEP_H
#define SGB_LM_STEP_H

#include <stddef.h>
#include <stdint.h>

#include "sgb_lm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------ vocabulary cross-entropy
 *
 * Row r has the hidden state h_r [D] and a label; w_v [D] is the head's row of
 * token v of V:
 *     x_rv = <h_r, w_v>,   lse_r = log sum_v exp(x_rv),
 *     loss_r = f_r (lse_r - x_r,label),   f_r the row weight, or 1;
 *  a row of weight 0 or with a label < 0 does not count: its loss and gradients
 *  are 0 whatever it holds.  Gradients of grad_scale * sum_r grad_loss_r loss_r:
 *     g_rv = grad_scale grad_loss_r f_r (exp(x_rv - lse_r) - [v = label_r]),
 *     d_hidden_r = sum_v g_rv w_v,   d_weight_v (+)= sum_r g_rv h_r.
 * Products of 16-bit types are summed in fp32; g (over grad_scale and the
 * row's factor, or the largest of these) is rounded to the operands' type for
 * the two products that follow: gradients are off by sqrt(2) times their own
 * rounding where many rows average it.  What g's rounding leaves is multiplied
 * too in calls of up to 128 rows, and in calls that ask for exact gradients: they
 * are off by their own rounding alone, and these two products take twice as
 * long.  fp32 operands are multiplied as they are, or,
 * where there are many rows, as three bf16 parts each and the six products of them
 * that an fp32 result can tell.
 * A row whose logits are all -inf, or hold +inf or NaN, has NaN for its loss and
 * gradients, and so has d_weight if the row counts.  Of fp32 operands a row of h
 * or w that holds an infinity may count as one that holds a NaN.
 * Weights and gradients from above have to be finite.
 *
 * The work goes by chunks of rows: the workspace does not grow past a chunk's,
 * at most 2 GiB of exponentials and 2.5 GiB of copies, gradients and sums.  A
 * 16-bit d_weight of more than one chunk adds 4 V D bytes for its sums, and weight
 * rows that may have to be copied, those of fp32 and of 16-bit elements whose D is
 * no multiple of 8, their copy, up to 4 GiB.  For D = 4096 and V = 131072, in GiB:
 * loss alone 0.6 (fp32 3.4); with gradients 0.35 for 8 rows of bf16, 3.0 for 8192,
 * 5.0 for any more; 5.1 for 8192 or more of fp16, 5.7 of fp32; for exact
 * gradients at most 0.2 more.
 */
typedef struct sgb_vocab_ce_s* sgb_vocab_ce;

/* D: 1..16384; V: 1..2^23. */
sgb_status sgb_vocab_ce_create(sgb_vocab_ce* out, int32_t D, int64_t V);
void sgb_vocab_ce_destroy(sgb_vocab_ce plan);

/* For calls of up to `rows` rows (below 2^31) of that type; gradient: 0 for
 * forward alone, 1 for all of the calls but those for exact gradients, 2 for
 * these too. */
sgb_status sgb_vocab_ce_workspace_bytes(sgb_vocab_ce plan, int64_t rows, int32_t dtype,
                                        int32_t gradient, size_t* bytes);

enum { SGB_VOCAB_CE_ACCUMULATE = 1, SGB_VOCAB_CE_EXACT = 2 };

typedef struct {
  const void* hidden;               /* [rows][D], dtype                     */
  const void* weight;               /* [V][D], dtype                        */
  const int64_t* labels;            /* [rows]                               */
  const float* row_weights;         /* [rows] or NULL (1)                   */
  float* loss;                      /* [rows] (not written by backward)     */
  float* lse;                       /* [rows]; written for every row by forward
                                       and loss_grad unless NULL; read by
                                       backward                             */
  const float* grad_loss;           /* [rows] or NULL (1); backward only    */
  void* d_hidden;                   /* [rows][D], dtype, or NULL: not wanted */
  void* d_weight;                   /* [V][D], d_weight_dtype, or NULL      */
  int64_t hidden_stride, weight_stride, d_hidden_stride, d_weight_stride;
  int64_t rows;
  int32_t dtype;                    /* F32, BF16, F16                       */
  int32_t d_weight_dtype;           /* F32 or dtype                         */
  int32_t accumulate;               /* SGB_VOCAB_CE_ACCUMULATE: d_weight is
                                       added to; SGB_VOCAB_CE_EXACT: exact
                                       gradients, see above; or their sum   */
  float grad_scale;
} sgb_vocab_ce_args;

/* loss (and lse). */
sgb_status sgb_vocab_ce_forward(sgb_vocab_ce plan, const sgb_vocab_ce_args* args, void* workspace,
                                size_t workspace_bytes, void* stream);
/* d_hidden, d_weight, from a forward's lse on the same inputs. */
sgb_status sgb_vocab_ce_backward(sgb_vocab_ce plan, const sgb_vocab_ce_args* args, void* workspace,
                                 size_t workspace_bytes, void* stream);
/* All of it in one go (grad_loss is not looked at): one product less. */
sgb_status sgb_vocab_ce_loss_grad(sgb_vocab_ce plan, const sgb_vocab_ce_args* args,
                                  void* workspace, size_t workspace_bytes, void* stream);

/* ----------------------------------------------------------------- dropout
 *
 *     out[r][c] = residual[r][c] + (kept(r, c) ? x[r][c] * scale : 0)
 * With t = round(p * 2^16), an element is kept iff its 16 random bits are at
 * least t, and scale = 2^16 / (2^16 - t) (t = 2^16: nothing is kept).  Bits
 * c mod 8 (the low half of a word before its high half) are of the four words of
 *     Philox4x32-10(counter = (c / 8, R mod 2^32, 2^31 + R / 2^32, offset mod 2^32),
 *                   key = (seed mod 2^32, seed / 2^32)),   R = first_row + r,
 * so they depend on the row and the column and on no stride, slice or launch:
 * the backward draws the same ones.  (Bit 31 of the third counter word keeps
 * them apart from those of the embedding update's stochastic rounding.)
 * With `state`, two 64-bit words on the device, the seed is state[0] and
 * state[1] is added to the offset: a captured call draws new masks when the
 * words change.  Everything is computed in fp32 and rounded once.  What is
 * dropped is not looked at: infinities and NaN there leave the residual.
 */
typedef struct sgb_dropout_s* sgb_dropout;

/* p: 0..1. */
sgb_status sgb_dropout_create(sgb_dropout* out, double p);
void sgb_dropout_destroy(sgb_dropout plan);

typedef struct {
  const void* x;                    /* [rows][cols], dtype                  */
  const void* residual;             /* [rows][cols], out_dtype, or NULL (0) */
  void* out;                        /* [rows][cols], out_dtype; may be x or
                                       residual (then of its type and stride) */
  const uint64_t* state;            /* [2] on the device, or NULL           */
  int64_t x_stride, residual_stride, out_stride;
  int64_t rows, first_row;          /* first_row >= 0, the sum at most 2^62 */
  uint64_t seed;                    /* not looked at with state             */
  uint64_t offset;
  int32_t cols;                     /* 1..2^24                              */
  int32_t dtype;                    /* F32, BF16, F16                       */
  int32_t out_dtype;                /* F32 or dtype; dtype without residual */
  int32_t reserved;                 /* 0                                    */
} sgb_dropout_args;

/* The backward is the same call on d_out, without residual (the residual's
 * gradient is d_out itself). */
sgb_status sgb_dropout_apply(sgb_dropout plan, const sgb_dropout_args* args, void* stream);

/* --------------------------------------------------------- quantising norm
 *
 * For each row, with M = 127 (int8) or 448 (e4m3):
 *     x_out = x + h,   v = x_out / sqrt(mean(x_out^2) + eps) * weight,
 *     scale_g = max over group g of |v| / M,   code = round(v / scale_g),
 * to nearest even, clamped to +-M.  v comes from the unrounded x_out; all in fp32.
 * A group whose scale would be below 2^-126 has scale 0 and codes 0.  A group
 * that holds a NaN has scale NaN and codes 0; one with an infinity in h or x
 * has a NaN there (the row's other groups are 0).  A v or an x_out * weight past
 * fp32's range (a weight's doing) makes its group's scale infinite and its codes
 * 0.  A row whose squares' sum is past it has codes 0 and scales 0, as next to an
 * infinity (NaN where a product is past it too); none below 2^64 / sqrt(D) has.
 */
typedef enum { SGB_CODE_INT8 = 0, SGB_CODE_E4M3 = 1 } sgb_code_kind;

typedef struct sgb_quant_norm_s* sgb_quant_norm;

/* D: 1..8192; group: 0 (one scale a row), 32, 64, 128, 256 or 512 columns. */
sgb_status sgb_quant_norm_create(sgb_quant_norm* out, int32_t D, int32_t code, int32_t group,
                                 float eps);
void sgb_quant_norm_destroy(sgb_quant_norm plan);

typedef struct {
  const void* h;                    /* [rows][D], dtype                     */
  const void* x;                    /* [rows][D], res_dtype, or NULL (0)    */
  void* x_out;                      /* [rows][D], res_dtype, or NULL: not
                                       wanted; may be x, or h if of its type */
  const void* weight;               /* [D], weight_dtype                    */
  uint8_t* q;                       /* [rows][D] codes, a byte each         */
  float* scales;                    /* [rows][ceil(D / group)]              */
  float* stats;                     /* [rows][4] or NULL: 0, 1, 0 and
                                       1 / sqrt(mean + eps): what the
                                       backward of a block norm without post
                                       norm reads; 16-byte aligned          */
  int64_t h_stride, x_stride, x_out_stride, q_stride, scales_stride;
  int64_t rows;                     /* below 2^31                           */
  int32_t dtype;                    /* F32, BF16, F16                       */
  int32_t res_dtype;                /* F32 or dtype                         */
  int32_t weight_dtype;             /* F32, BF16, F16                       */
  int32_t reserved;                 /* 0                                    */
} sgb_quant_norm_args;

sgb_status sgb_quant_norm_forward(sgb_quant_norm plan, const sgb_quant_norm_args* args,
                                  void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SGB_LM_STEP_H */
