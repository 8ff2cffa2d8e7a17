/*
 * vsa_block.h -- C ABI of the operators that make a whole transformer block of the attention layer
 * (libvsa.so, with vsa.h and vsa_layer.h):
 *   - vsa_gate_norm: the end of one branch and the start of the next in one pass: the branch's
 *     output, normalised or not, times its gate goes onto the residual stream, and the stream's
 *     norm with weight, bias and modulation is the next branch's input; and its backward;
 *   - vsa_linear: a matrix product with bias, activation and residual in its epilogue, and its
 *     backward, which can go on through the activation that made the input.
 *
 * Conventions are those of vsa_layer.h (ownership, streams, workspaces, status codes, graph
 * capture, the shared device error word, results that are a pure function of the inputs):
 *   - Data pointers of tensors are multiples of 16 bytes, and so are the strides of dimensions
 *     longer than 1; the last dimension is contiguous.  Strides count elements.  Input strides of
 *     the batch, of tokens and of modulation rows may be 0.  An output must not overlap itself or
 *     another tensor of the call, but for the two places that say so.
 *   - Vectors (weights, biases) are contiguous and 16-byte aligned.
 */
#ifndef VSA_BLOCK_H
#define VSA_BLOCK_H

#include "vsa_layer.h"

#ifdef __cplusplus
extern "C" {
#endif

/* A [batch, tokens, channels] tensor. */
typedef struct vsa_tokens {
  void* data; /* NULL: the tensor is absent (only where stated) */
  int64_t batch_stride;
  int64_t token_stride;
} vsa_tokens;

/* A [batch, groups, channels] modulation. */
typedef struct vsa_modulation {
  const void* data; /* NULL: absent */
  int64_t batch_stride;
  int64_t group_stride;
} vsa_modulation;

typedef enum vsa_norm_kind { VSA_LAYER_NORM = 0, VSA_RMS_NORM = 1 } vsa_norm_kind;

/*
 * One call.  For token t of a batch entry, with the modulation row g = t / (tokens / groups):
 *   u  = y, or with post_weight  y / sqrt(mean(y^2) + post_eps) * post_weight
 *   x' = x + gate_g u                                     (x' = x without y)
 *   n  = (x' - mean(x')) / sqrt(var(x') + eps), or for VSA_RMS_NORM  x' / sqrt(mean(x'^2) + eps)
 *   h  = (n weight + bias) (1 + scale_g) + shift_g        (absent: 1, 0, 0, 0)
 * Arithmetic is in fp32; x' is rounded once where it is stored, and h is computed from the
 * unrounded x' and rounded once.
 */
typedef struct vsa_gate_norm {
  int32_t batch;        /* >= 1; batch * tokens at most 2^30 */
  int32_t tokens;       /* >= 1 */
  int32_t channels;     /* a multiple of 8, 8 .. 8192 */
  int32_t groups;       /* modulation rows of a batch entry, a divisor of tokens; 1 without modulation */
  int32_t kind;         /* vsa_norm_kind */
  int32_t dtype;        /* vsa_dtype of the stream: x, x' and their gradients */
  int32_t branch_dtype; /* of y, h and their gradients: dtype, or 16-bit where dtype is VSA_F32 */
  int32_t mod_dtype;    /* of gate, scale, shift and their gradients: VSA_F32 or branch_dtype */
  int32_t weight_dtype; /* of the weights, bias and their gradients: VSA_F32 or branch_dtype */
  float eps, post_eps;  /* finite, >= 0 */
  vsa_modulation gate, scale, shift;
  const void *post_weight, *weight, *bias; /* [channels] or NULL; gate and post_weight only with y */
} vsa_gate_norm;

/* x_out = x', h.  y and x_out come together or are both absent.  x_out may be x itself (the same
 * data and strides). */
vsa_status vsa_gate_norm_fwd(const vsa_gate_norm* op, const vsa_tokens* x, const vsa_tokens* y,
                             const vsa_tokens* x_out, const vsa_tokens* h, void* stream);

/* Places of the parameters' gradients, contiguous and 16-byte aligned: [batch, groups, channels] of
 * the modulation, [channels] of the others; NULL where not wanted.  Absent with their parameter. */
typedef struct vsa_gate_norm_grads {
  void *gate, *scale, *shift, *post_weight, *weight, *bias;
} vsa_gate_norm_grads;

/* Bytes of device workspace vsa_gate_norm_bwd needs where gradients of op's parameters are wanted (0: none is
 * needed, or invalid arguments).  Where those of the modulations alone are wanted it may need none, as it
 * says of an op without weights and bias: for modulation rows of few tokens it is large with, 0 without. */
size_t vsa_gate_norm_bwd_workspace_bytes(const vsa_gate_norm* op);

/*
 * Gradients of vsa_gate_norm_fwd from dh, dx_out (absent: zero), and x_out and y as the forward
 * left them; the norm's statistics are taken again from x_out.  With a = (1 + scale) weight:
 *   dx = dx_out + (dh a - mean(dh a) - n mean(dh a n)) / sqrt(..)      (VSA_RMS_NORM: no mean(dh a))
 *   du = gate dx, through the post norm to dy; the parameters' gradients are sums of dx u, dh and
 *   dh n over their tokens, in fp32.
 * y and dy come together.  Without y, dx is the whole gradient of x.  dx may be dx_out itself.
 */
vsa_status vsa_gate_norm_bwd(const vsa_gate_norm* op, const vsa_tokens* dh,
                             const vsa_tokens* dx_out, const vsa_tokens* x_out,
                             const vsa_tokens* y, const vsa_tokens* dx, const vsa_tokens* dy,
                             const vsa_gate_norm_grads* grads, void* workspace,
                             size_t workspace_bytes, void* stream);

/* A matrix of contiguous rows. */
typedef struct vsa_matrix {
  void* data; /* NULL: absent (only where stated) */
  int64_t row_stride;
} vsa_matrix;

typedef enum vsa_act {
  VSA_ACT_NONE = 0,
  VSA_GELU = 1,      /* z Phi(z) */
  VSA_GELU_TANH = 2, /* z / 2 (1 + tanh(sqrt(2 / pi) (z + 0.044715 z^3))) */
  VSA_SILU = 3       /* z / (1 + exp(-z)) */
} vsa_act;

/* One product: z = x weight^T + bias, out = act(z) + residual.  Products are of 16-bit operands with
 * fp32 sums; the epilogue is in fp32 and each output is rounded once. */
typedef struct vsa_linear {
  int32_t rows;         /* of x and out, 1 .. 2^30; each matrix of 2^44 elements at most */
  int32_t in_features;  /* a multiple of 8, 8 .. 2^24 */
  int32_t out_features; /* a multiple of 8, 8 .. 2^24 */
  int32_t dtype;        /* of every matrix: VSA_BF16 or VSA_F16 */
  int32_t bias_dtype;   /* of bias and its gradient: VSA_F32 or dtype */
  int32_t act;          /* vsa_act */
  vsa_matrix weight;    /* [out_features, in_features]; rows must not be broadcast, nor those of
                         * the other matrices */
  const void* bias;     /* [out_features] or NULL */
} vsa_linear;

/* Bytes of device workspace of the two calls (0: none is needed, or invalid arguments). */
size_t vsa_linear_fwd_workspace_bytes(const vsa_linear* op);
size_t vsa_linear_bwd_workspace_bytes(const vsa_linear* op);

/* out [rows, out_features]; residual of the same shape, or absent; pre (the same shape, or absent)
 * takes z, for the backward of an activation. */
vsa_status vsa_linear_fwd(const vsa_linear* op, const vsa_matrix* x, const vsa_matrix* residual,
                          const vsa_matrix* out, const vsa_matrix* pre, void* workspace,
                          size_t workspace_bytes, void* stream);

/*
 * Gradients of vsa_linear_fwd; dout is also the residual's.  dz = dout act'(pre) is rounded to dtype as
 * an operand of the products where there is an activation:
 *   dx = dz weight,  dweight = dz^T x,  dbias = sum dz (fp32 sums).
 * With x_act, x is x_act(x_pre) and dx the gradient of x_pre: dx = (dz weight) x_act'(x_pre).
 * pre is present with an activation, x_pre with x_act.  dx, dweight, dbias: absent where not wanted.
 */
vsa_status vsa_linear_bwd(const vsa_linear* op, int32_t x_act, const vsa_matrix* dout,
                          const vsa_matrix* x, const vsa_matrix* pre, const vsa_matrix* x_pre,
                          const vsa_matrix* dx, const vsa_matrix* dweight, void* dbias,
                          void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* VSA_BLOCK_H */
