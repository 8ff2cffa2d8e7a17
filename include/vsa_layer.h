/*
 * vsa_layer.h -- C ABI of the operators around the block-sparse attention in a video transformer
 * layer (libvsa.so, with vsa.h):
 *   - vsa_norm_rope: the RMS norm of every query and key head with the position rotation, in the
 *     pass that moves q, k and v from the projection's token order into the attention's rows
 *     (cube by cube for video), and its backward;
 *   - vsa_cross: attention to an encoder's states of another length, and its backward.
 *
 * Conventions are those of vsa.h (ownership, streams, workspaces, status codes, graph capture),
 * with these additions:
 *   - Tensors are described by vsa_heads: any strides with unit stride inside a head; the data
 *     pointer and the strides of dimensions longer than 1 must be multiples of 16 bytes.
 *     Strides count elements.  Input strides may be 0 (a broadcast dimension; in vsa_cross
 *     that of the batch only); an output must not overlap itself or an input.
 *   - Problems only visible on the device never trap: they are clamped or skipped and set a bit
 *     in a device error word.  These operators share one word per device inside the library,
 *     which collects bits until vsa_layer_device_error reads and clears it (with
 *     VSA_DEVERR_TIMEOUT set, the outputs of some call since the last read are invalid).  The
 *     first call on each device looks up the word's address; make it before a stream capture.
 *   - Every result is a pure function of the inputs: sums that are split over CTAs are joined in
 *     a fixed order.
 */
#ifndef VSA_LAYER_H
#define VSA_LAYER_H

#include "vsa.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Further bits of the device error word. */
#define VSA_DEVERR_ORDER 0x40u  /* an order entry outside [-1, n) was read as -1, or `inverse`
                                 * does not name it back */
#define VSA_DEVERR_KV_LEN 0x80u /* a kv_len entry outside [0, kv_tokens] was clamped */

typedef enum vsa_dtype { VSA_BF16 = 0, VSA_F16 = 1, VSA_F32 = 2 } vsa_dtype;

/* A [batch, heads, tokens, head_dim] tensor, in any memory order. */
typedef struct vsa_heads {
  void* data; /* NULL: the tensor is absent (only where stated) */
  int64_t batch_stride;
  int64_t head_stride;
  int64_t token_stride;
  int32_t heads;
} vsa_heads;

/*
 * The norm and rotation of one call.  For every token t and head x of q or k:
 *   n = x / sqrt(mean(x^2) + eps),   y = R_t (n * w),
 * where R_t turns the pairs of the first `rot` elements of a head by the angles of token t:
 *   (a, b) -> (a cos - b sin, b cos + a sin),
 * pair i being elements (2i, 2i + 1), or (i, i + rot/2) with `halves` set.  v is only moved.
 * Every head is normalised by itself, with one weight for all heads of q and one for all of k: a
 * model that takes the mean over all heads together, with a weight for each of their elements, is
 * not served.  Arithmetic is in fp32, the sums of the weights' gradients included; each output is
 * rounded once.
 */
typedef struct vsa_norm_rope {
  int32_t batch;        /* >= 1; batch * tokens and batch * rows below 2^31 */
  int32_t tokens;       /* tokens of q, k, v (the projection's order), >= 1 */
  int32_t rows;         /* rows of the outputs (the attention's order), >= 1 */
  int32_t head_dim;     /* a multiple of 8, 8 .. 256 */
  int32_t dtype;        /* vsa_dtype of the activations */
  int32_t weight_dtype; /* vsa_dtype of the weights and their gradients: VSA_F32 or dtype */
  int32_t rot;          /* elements turned: 0 .. head_dim, a multiple of 8 (halves: of 16) */
  int32_t halves;
  float eps;            /* finite, >= 0 */
  const void* q_weight; /* [head_dim], or NULL: ones */
  const void* k_weight;
  const float* cosines; /* [tokens][rot / 2], 16-byte aligned; unused if rot is 0 */
  const float* sines;
  int64_t table_batch_stride; /* elements from one batch entry's table to the next; 0: shared */
  /* Forward: [rows], the token each row takes, -1 for a row of zeros.  Backward: [tokens], the
   * row each token went to, -1 for none (its gradients are zero).  NULL: row t is token t, and
   * rows == tokens.  A forward may take a token for several rows, but a backward follows one row
   * of each token: its gradients are the forward's only where the two orders name each other. */
  const int32_t* order;
  /* The order of the other direction, to have that checked, or NULL.  An entry of `order` that it
   * does not name back raises VSA_DEVERR_ORDER; the outputs are those of `order` all the same. */
  const int32_t* inverse;
} vsa_norm_rope;

/*
 * vsa_norm_rope_fwd -- q_out = norm_rope(q, q_weight), k_out = norm_rope(k, k_weight), v_out = v,
 * each [batch, heads, rows, head_dim].  Any of the three pairs may be absent.
 */
vsa_status vsa_norm_rope_fwd(const vsa_norm_rope* op, const vsa_heads* q, const vsa_heads* k,
                             const vsa_heads* v, const vsa_heads* q_out, const vsa_heads* k_out,
                             const vsa_heads* v_out, void* stream);

/* Bytes of device workspace vsa_norm_rope_bwd needs (0 for invalid arguments). */
size_t vsa_norm_rope_bwd_workspace_bytes(const vsa_norm_rope* op);

/*
 * vsa_norm_rope_bwd -- gradients of vsa_norm_rope_fwd, from the gradients of its outputs (rows)
 * and its inputs q, k (tokens): with u = R_t^T dy,
 *   dw = sum u n,   dx = (u w - n mean(u w n)) / sqrt(mean(x^2) + eps),   dv = dv_out moved back.
 * dq_weight, dk_weight: [head_dim] weight_dtype, or NULL where not wanted (absent with their
 * tensor).  `order` lists the tokens' rows.
 */
vsa_status vsa_norm_rope_bwd(const vsa_norm_rope* op, const vsa_heads* dq_out,
                             const vsa_heads* dk_out, const vsa_heads* dv_out, const vsa_heads* q,
                             const vsa_heads* k, const vsa_heads* dq, const vsa_heads* dk,
                             const vsa_heads* dv, void* dq_weight, void* dk_weight,
                             void* workspace, size_t workspace_bytes, void* stream);

/*
 * Cross attention: query head h reads key head h / (heads / kv_heads), the first
 * kv_len[b] of kv_tokens keys.  Rows at or past kv_len[b] of k and v may hold anything.
 */
typedef struct vsa_cross {
  int32_t batch;          /* >= 1 */
  int32_t heads;          /* a multiple of kv_heads; batch * heads <= 65535 */
  int32_t kv_heads;       /* >= 1 */
  int32_t q_tokens;       /* >= 1; batch * heads * q_tokens below 2^30 */
  int32_t kv_tokens;      /* >= 1; batch * kv_heads * kv_tokens below 2^30 */
  int32_t head_dim;       /* must be 128 */
  float sm_scale;         /* finite */
  const int32_t* kv_len;  /* [batch], or NULL: every key */
} vsa_cross;

/* Bytes of device workspace of the two calls (0: none is needed, or invalid arguments). */
size_t vsa_cross_fwd_workspace_bytes(const vsa_cross* op);
size_t vsa_cross_bwd_workspace_bytes(const vsa_cross* op);

/*
 * vsa_cross_fwd -- O = softmax(q k^T sm_scale) v, bf16, and lse [batch, heads, q_tokens] fp32
 * contiguous, base 2 in the M form of vsa_fwd.  Without a visible key O = 0 and lse = -inf.
 * With more than two query rows per key head (heads / kv_heads * q_tokens) the softmax's weights
 * are rounded to bf16 as an operand of the tensor cores (2^-8 at most; O is off by 0.0023 of its norm
 * on random inputs, where its own rounding makes 0.0017); up to two rows they stay fp32.  Sums, lse
 * and the statistics are fp32 everywhere.
 */
vsa_status vsa_cross_fwd(const vsa_cross* op, const vsa_heads* q, const vsa_heads* k,
                         const vsa_heads* v, const vsa_heads* o, float* lse, void* workspace,
                         size_t workspace_bytes, void* stream);

/*
 * vsa_cross_bwd -- with P = exp2(q k^T sm_scale log2e - lse) on the visible keys and
 * dS = P (dO v^T - rowsum(O dO)):
 *   dV = P^T dO,   dK = sm_scale dS^T q  (each summed over the query heads that share the key
 *   head),   dQ = sm_scale dS k.
 * o and lse as vsa_cross_fwd wrote them.  Rows at or past kv_len[b] of dK and dV are exact zeros.
 * P and dS are rounded to bf16 as operands (gradients off by 0.0024 of their norm, likewise).
 */
vsa_status vsa_cross_bwd(const vsa_cross* op, const vsa_heads* dout, const vsa_heads* q,
                         const vsa_heads* k, const vsa_heads* v, const vsa_heads* o,
                         const float* lse, const vsa_heads* dq, const vsa_heads* dk,
                         const vsa_heads* dv, void* workspace, size_t workspace_bytes,
                         void* stream);

/* Synchronise `stream`, copy the current device's error word of these operators to *bits and
 * clear it (0 if none has run on this device yet). */
vsa_status vsa_layer_device_error(uint32_t* bits, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* VSA_LAYER_H */
