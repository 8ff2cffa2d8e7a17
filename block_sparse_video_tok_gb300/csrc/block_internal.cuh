// block_internal.cuh -- definitions shared by the translation units of the block operators
// (include/vsa_block.h): kernel arguments and the host-side launch functions.
#pragma once

#include "../../include/vsa_block.h"
#include "layer_internal.cuh"

namespace vsa {

// ---------------------------------------------------------------------------- gate_norm

// Element (b, t, c) at data[b * batch + t * token + c]; data null: absent.
struct TokensView {
  void* data;
  int64_t batch, token;
};
struct ModView {
  const void* data;
  int64_t batch, group;
};

struct GateNormArgs {
  TokensView x, y, x_out, h;     // forward: x, y in, x_out, h out; backward: x_out, y in
  TokensView dh, dx_out, dx, dy;
  ModView gate, scale, shift;
  const void *post_weight, *weight, *bias;
  void *dgate, *dscale, *dshift, *dpost, *dweight, *dbias;
  float* workspace;
  int batch, tokens, channels, groups;
  int kind, dtype, branch_dtype, mod_dtype, weight_dtype;
  float eps, post_eps;
};

cudaError_t launch_gate_norm_fwd(const GateNormArgs& a, cudaStream_t stream);
cudaError_t launch_gate_norm_bwd(const GateNormArgs& a, cudaStream_t stream);
// Of the gradients that a has places for.
size_t gate_norm_bwd_workspace(const GateNormArgs& a);

// ---------------------------------------------------------------------------- linear

struct MatrixView {
  void* data;  // null: absent
  int64_t stride;
};

struct LinearArgs {
  MatrixView x, weight, residual, out, pre;        // forward
  MatrixView dout, x_pre, dx, dweight;             // backward (with x, weight, pre)
  const void* bias;
  void* dbias;
  uint8_t* workspace;
  uint32_t* err;
  int rows, in, out_features;
  int dtype, bias_dtype, act, x_act;
  uint64_t wait_ns;
};

cudaError_t launch_linear_fwd(const LinearArgs& a, cudaStream_t stream);
cudaError_t launch_linear_bwd(const LinearArgs& a, cudaStream_t stream);
size_t linear_fwd_workspace(int rows, int in, int out);
size_t linear_bwd_workspace(int rows, int in, int out, int act);

}  // namespace vsa
