// Argument block and launcher of the grouped products (csrc/grouped_gemm.cu).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/moe.h"

namespace moe {

// The four products.  "Rows" are activation rows in expert order, "channels"
// the long side of an expert's matrix.
enum GroupedKind {
  kGgForward = 0,  // out[r][n] = sum_k x[r][k] w[e][n][k], 16-bit operands
  kGgGradX = 1,    // dx[r][k]  = sum_n dy[r][n] w[e][n][k]
  kGgGradW = 2,    // dw[e][n][k] = sum_{r in e} dy[r][n] x[r][k]
  kGgInt8 = 3,     // out[r][n] = sx[r] sw[e][n] sum_k x[r][k] w[e][n][k], int8 operands
};

struct GroupedProblem {
  int kind;
  int rows, E, N, K;
  int dtype;      // moe_dtype of the 16-bit operands (ignored for int8)
  int out_dtype;  // moe_dtype
  const void* a;  // weights [E][N][K] (grad_w: dy [rows][N])
  const void* b;  // x [rows][K], grad_x: dy [rows][N], grad_w: x [rows][K]
  int64_t lda_bytes, ldb_bytes;  // row pitch
  int64_t stride_w_bytes;        // between experts (not grad_w)
  const int32_t* offsets;
  const int32_t* slot_map;
  int n_phys;
  const float* x_scale;
  const float* w_scale;
  void* out;
  int64_t ldo;       // elements
  int64_t stride_o;  // elements between experts (grad_w)
  int accumulate;    // grad_w, fp32
};

cudaError_t launch_grouped_gemm(const GroupedProblem& p, int n_sms, int smem_max, cudaStream_t st,
                                int* unsupported);

// The status word of these kernels, and 0 to it.
cudaError_t take_grouped_gemm_status(int* status);

// The same products (forward, int8) for few rows: csrc/grouped_gemv.cu, and
// whether that kernel is the faster one.
bool grouped_gemv_pays(const GroupedProblem& p, int n_sms);
cudaError_t launch_grouped_gemv(const GroupedProblem& p, int n_sms, cudaStream_t st);

}  // namespace moe
