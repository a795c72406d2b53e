// Launchers of the row operators around the grouped products (csrc/expert_rows.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/moe.h"

namespace moe {

cudaError_t launch_swiglu(int dtype, int rows, int F, const void* gu, int64_t ldg, void* h, int64_t ldh,
                          cudaStream_t st);
cudaError_t launch_swiglu_grad(int dtype, int rows, int F, const void* gu, int64_t ldg, const void* dh, int64_t ldh,
                               void* dgu, int64_t ldd, cudaStream_t st);
// int8 codes and one fp32 scale per row, of the rows themselves or (swiglu) of
// silu(g) u of gate/up rows.  row_token: source row of each output row, or null.
cudaError_t launch_quant_rows(int dtype, bool swiglu, int rows, int K, const void* x, int64_t ldx,
                              const int32_t* row_token, int n_tokens, int8_t* q, int64_t ldq, float* scale,
                              cudaStream_t st);

}  // namespace moe
