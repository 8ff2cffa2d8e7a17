// gemm.cuh -- the matrix products of vsa_linear: arguments of the tensor-core kernel (gemm.cu) and
// what plans it on the host.
#pragma once

#include "block_internal.cuh"

namespace vsa {

// What a product computes, with the layout of its operands (16-bit, fp32 sums):
//   GEMM_FWD  out[m][n] = act(sum_k A[m][k] B[n][k] + bias[n]) + aux[m][n]; pre takes the value before act
//   GEMM_DX   out[m][n] = sum_k A[m][k] B[k][n], times act'(aux[m][n]) where aux is given
//   GEMM_DW   out[m][n] = sum_k A[k][m] B[k][n]
enum GemmOp : int { GEMM_FWD = 0, GEMM_DX = 1, GEMM_DW = 2 };

struct GemmArgs {
  MatrixView a, b, out, pre, aux;
  const void* bias;
  bool bias_f32;
  int m, n, k;
  int act;    // of GEMM_FWD; GEMM_DX: the activation whose slope is taken at aux
  int dtype;
  uint8_t* workspace;
  uint32_t* err;
  uint64_t wait_ns;
};

cudaError_t launch_gemm(GemmOp op, const GemmArgs& a, cudaStream_t stream);
size_t gemm_workspace(int m, int n, int k);

// The same for small products (no workspace), and whether it is the one to use.
cudaError_t launch_gemm_small(GemmOp op, const GemmArgs& a, cudaStream_t stream);
bool use_gemm_small(int m, int n, int k);
// Two of them in one launch, of one type and independent of each other, and whether that is offered.
cudaError_t launch_gemm_small_pair(GemmOp op_a, const GemmArgs& a, GemmOp op_b, const GemmArgs& b, cudaStream_t stream);
bool use_gemm_small_pair(const GemmArgs& a, const GemmArgs& b);
// About what gemm.cu's own kernels take.
double gemm_microseconds(int m, int n, int k);

// The forward for a few rows, and whether it is the one to use.
cudaError_t launch_linear_rows(const LinearArgs& a, cudaStream_t stream);
bool use_linear_rows(int rows, int in, int out);

// 2-D tensor map of a 16-bit matrix of `columns` x `rows`, box 64 columns x box_rows, 128-byte swizzle; narrow: 32
// columns, 64-byte swizzle.
cudaError_t make_tmap_matrix(CUtensorMap* map, const MatrixView& x, int columns, int rows, int box_rows, bool bf16,
                             bool narrow = false);

}  // namespace vsa
