// layer_internal.cuh -- definitions shared by the translation units of the layer operators
// (include/vsa_layer.h): kernel arguments and the host-side launch functions.
#pragma once

#include "../../include/vsa_layer.h"
#include "vsa_internal.cuh"

namespace vsa {

// A tensor as the kernels see it: element (b, h, t, d) at data[b * batch + h * head + t * token + d].
struct HeadsView {
  void* data;
  int64_t batch, head, token;
  int heads;  // 0: absent
};

// The device error word of the layer operators on the current device.
vsa_status layer_error_word(uint32_t** word);

// ---------------------------------------------------------------------------- norm_rope

struct NormRopeArgs {
  HeadsView in[3];   // q, k, v (forward: tokens; backward: the gradients of the outputs, rows)
  HeadsView out[3];  // forward: rows; backward: the gradients of the inputs, tokens
  HeadsView x[2];    // backward: q, k (tokens)
  const void* weight[2];
  void* dweight[2];
  const float *cosines, *sines;
  int64_t table_batch;
  const int32_t *order, *inverse;
  float* partial;  // backward: one [2][head_dim] fp32 sum per CTA
  uint32_t* err;
  int batch, tokens, rows, head_dim, rot;
  int dtype, weight_dtype;
  bool halves;
  float eps;
};

cudaError_t launch_norm_rope_fwd(const NormRopeArgs& a, cudaStream_t stream);
cudaError_t launch_norm_rope_bwd(const NormRopeArgs& a, cudaStream_t stream);
size_t norm_rope_bwd_workspace(int head_dim);

// ---------------------------------------------------------------------------- cross attention

struct CrossArgs {
  HeadsView q, k, v, o, dout, dq, dk, dv;
  const int32_t* kv_len;
  float* lse;  // written by the forward, read by the backward
  uint8_t* workspace;
  uint32_t* err;
  int batch, heads, kv_heads, q_tokens, kv_tokens;
  float sm_scale;
  uint64_t wait_ns;
};

cudaError_t launch_cross_fwd(const CrossArgs& a, cudaStream_t stream);
cudaError_t launch_cross_bwd(const CrossArgs& a, cudaStream_t stream);
// The forward for a few query rows per key head, and whether it is the one to use.
cudaError_t launch_cross_token(const CrossArgs& a, cudaStream_t stream);
bool use_cross_token(int heads, int kv_heads, int q_tokens);
size_t cross_token_workspace(int batch, int heads, int kv_heads, int q_tokens, int kv_tokens);
size_t cross_fwd_workspace(int batch, int heads, int kv_heads, int q_tokens, int kv_tokens);
size_t cross_bwd_workspace(int batch, int heads, int kv_heads, int q_tokens, int kv_tokens);

// Keys of batch entry b that take part, clamped to [0, kv_tokens].
__device__ __forceinline__ int visible_keys(const int32_t* kv_len, int b, int kv_tokens,
                                            uint32_t* err) {
  if (!kv_len) return kv_tokens;
  const int n = kv_len[b];
  if (n >= 0 && n <= kv_tokens) return n;
  atomicOr(err, VSA_DEVERR_KV_LEN);
  return n < 0 ? 0 : kv_tokens;
}

}  // namespace vsa
