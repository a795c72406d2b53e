// C entry points of the expert operators: argument checks, then one launch each.
#include "devinfo.cuh"
#include "expert_rows.cuh"
#include "grouped_gemm.cuh"

using namespace moe;

namespace {

constexpr int kMaxExtent = 1 << 20;   // N, K: byte coordinates of a row stay far below 2^31
constexpr int kMaxDepthI8 = 131071;   // 128 * 128 * K < 2^31: the int32 sum cannot overflow
constexpr int kMaxGradRows = 1 << 26;  // one tile sums a group's rows: far below the limit of a device-side wait
constexpr int64_t kMaxPitch = (int64_t)1 << 36;  // elements: byte strides stay below the tensor maps' 2^40

bool on(const void* p, int bytes) { return (reinterpret_cast<uintptr_t>(p) & (uintptr_t)(bytes - 1)) == 0; }
bool is16(int t) { return t == MOE_T_BF16 || t == MOE_T_FP16; }
int size_of(int t) { return t == MOE_T_FP32 ? 4 : t == MOE_T_INT8 ? 1 : 2; }
// a matrix that is read: base and pitch in whole 16 bytes
bool operand(const void* p, int64_t ld, int elem) { return p && on(p, 16) && (ld * elem) % 16 == 0; }

struct Pitch {
  int64_t x, y, w, stride;
};

// own_matrices: expert e's matrix is matrix e of w (no slot_map says otherwise)
moe_status check_gemm(const moe_gemm_desc* d, bool int8, bool own_matrices, Pitch* t) {
  if (!d) return MOE_ERR_INVALID_ARG;
  if (d->rows < 0 || d->n_experts <= 0 || d->N <= 0 || d->K <= 0 || d->n_physical < 0) return MOE_ERR_INVALID_ARG;
  if (own_matrices && d->n_physical && d->n_physical < d->n_experts) return MOE_ERR_INVALID_ARG;
  if (int8 ? d->dtype != MOE_T_INT8 : !is16(d->dtype)) return MOE_ERR_INVALID_ARG;
  if (!is16(d->out_dtype) && d->out_dtype != MOE_T_FP32) return MOE_ERR_INVALID_ARG;
  if (d->n_experts > 1024 || d->N > kMaxExtent || d->K > kMaxExtent || (int8 && d->K > kMaxDepthI8) ||
      d->rows > (1 << 30))
    return MOE_ERR_UNSUPPORTED;
  t->x = d->ld_x ? d->ld_x : d->K;
  t->y = d->ld_y ? d->ld_y : d->N;
  t->w = d->ld_w ? d->ld_w : d->K;
  if (t->x < d->K || t->y < d->N || t->w < d->K) return MOE_ERR_INVALID_ARG;
  if (t->x > kMaxPitch || t->y > kMaxPitch || t->w > ((int64_t)1 << 30)) return MOE_ERR_UNSUPPORTED;
  const int64_t one = (int64_t)(d->N - 1) * t->w + d->K;
  t->stride = d->stride_w ? d->stride_w : (int64_t)d->N * t->w;
  if (t->stride < one) return MOE_ERR_INVALID_ARG;
  if (t->stride > kMaxPitch) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

moe_status run(const GroupedProblem& p, void* stream) {
  const DevInfo di = dev_info();
  int unsupported = 0;
  if (grouped_gemv_pays(p, di.sms)) {
    const cudaError_t err = launch_grouped_gemv(p, di.sms, static_cast<cudaStream_t>(stream));
    return err == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
  }
  const cudaError_t err = launch_grouped_gemm(p, di.sms, di.smem_optin, static_cast<cudaStream_t>(stream),
                                              &unsupported);
  if (unsupported) return MOE_ERR_UNSUPPORTED;
  return err == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

GroupedProblem problem(int kind, const moe_gemm_desc& d, const Pitch& t) {
  GroupedProblem p{};
  p.kind = kind;
  p.rows = d.rows;
  p.E = d.n_experts;
  p.N = d.N;
  p.K = d.K;
  p.dtype = d.dtype;
  p.out_dtype = d.out_dtype;
  p.n_phys = d.n_physical ? d.n_physical : d.n_experts;
  p.stride_w_bytes = t.stride * size_of(d.dtype);
  return p;
}

moe_status check_rows(int rows, int width, int dtype) {
  if (rows < 0 || width <= 0 || !is16(dtype)) return MOE_ERR_INVALID_ARG;
  if (width > kMaxExtent || rows > (1 << 30)) return MOE_ERR_UNSUPPORTED;
  if ((int64_t)rows * width > (int64_t)1 << 40) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

moe_status from(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

}  // namespace

extern "C" {

moe_status moe_grouped_gemm(const moe_gemm_desc* desc, const void* x, const void* w, const int32_t* slot_map,
                            const int32_t* offsets, void* out, void* stream) {
  Pitch t;
  moe_status s = check_gemm(desc, false, !slot_map, &t);
  if (s != MOE_OK || desc->rows == 0) return s;
  if (!operand(x, t.x, 2) || !operand(w, t.w, 2) || t.stride % 8 || !offsets || !out ||
      !on(out, size_of(desc->out_dtype)))
    return MOE_ERR_INVALID_ARG;
  GroupedProblem p = problem(kGgForward, *desc, t);
  p.a = w;
  p.b = x;
  p.lda_bytes = t.w * 2;
  p.ldb_bytes = t.x * 2;
  p.slot_map = slot_map;
  p.offsets = offsets;
  p.out = out;
  p.ldo = t.y;
  return run(p, stream);
}

moe_status moe_grouped_gemm_grad_x(const moe_gemm_desc* desc, const void* dy, const void* w,
                                   const int32_t* slot_map, const int32_t* offsets, void* dx, void* stream) {
  Pitch t;
  moe_status s = check_gemm(desc, false, !slot_map, &t);
  if (s != MOE_OK || desc->rows == 0) return s;
  if (!operand(dy, t.y, 2) || !operand(w, t.w, 2) || t.stride % 8 || !offsets || !dx ||
      !on(dx, size_of(desc->out_dtype)))
    return MOE_ERR_INVALID_ARG;
  GroupedProblem p = problem(kGgGradX, *desc, t);
  p.a = w;
  p.b = dy;
  p.lda_bytes = t.w * 2;
  p.ldb_bytes = t.y * 2;
  p.slot_map = slot_map;
  p.offsets = offsets;
  p.out = dx;
  p.ldo = t.x;
  return run(p, stream);
}

moe_status moe_grouped_gemm_grad_w(const moe_gemm_desc* desc, const void* dy, const void* x,
                                   const int32_t* offsets, void* dw, int accumulate, void* stream) {
  Pitch t;
  moe_status s = check_gemm(desc, false, false, &t);
  if (s != MOE_OK) return s;
  if (accumulate && desc->out_dtype != MOE_T_FP32) return MOE_ERR_INVALID_ARG;
  if (desc->rows > kMaxGradRows) return MOE_ERR_UNSUPPORTED;
  if (!offsets || !dw || !on(dw, size_of(desc->out_dtype))) return MOE_ERR_INVALID_ARG;
  if (desc->rows > 0 && (!operand(dy, t.y, 2) || !operand(x, t.x, 2))) return MOE_ERR_INVALID_ARG;
  GroupedProblem p = problem(kGgGradW, *desc, t);
  p.a = dy;
  p.b = x;
  p.lda_bytes = t.y * 2;
  p.ldb_bytes = t.x * 2;
  p.offsets = offsets;
  p.out = dw;
  p.ldo = t.w;
  p.stride_o = t.stride;
  p.accumulate = accumulate ? 1 : 0;
  return run(p, stream);
}

moe_status moe_grouped_gemm_i8(const moe_gemm_desc* desc, const int8_t* x, const float* x_scale, const int8_t* w,
                               const float* w_scale, const int32_t* slot_map, const int32_t* offsets, void* out,
                               void* stream) {
  Pitch t;
  moe_status s = check_gemm(desc, true, !slot_map, &t);
  if (s != MOE_OK || desc->rows == 0) return s;
  if (!operand(x, t.x, 1) || !operand(w, t.w, 1) || t.stride % 16 || !offsets || !out ||
      !on(out, size_of(desc->out_dtype)) || !x_scale || !on(x_scale, 4) || !w_scale || !on(w_scale, 4))
    return MOE_ERR_INVALID_ARG;
  GroupedProblem p = problem(kGgInt8, *desc, t);
  p.a = w;
  p.b = x;
  p.lda_bytes = t.w;
  p.ldb_bytes = t.x;
  p.slot_map = slot_map;
  p.offsets = offsets;
  p.x_scale = x_scale;
  p.w_scale = w_scale;
  p.out = out;
  p.ldo = t.y;
  return run(p, stream);
}

moe_status moe_quant_rows_i8(int32_t rows, int32_t K, int32_t dtype, const void* x, int64_t ld_x,
                             const int32_t* row_token, int32_t n_tokens, int8_t* q, int64_t ld_q, float* scale,
                             void* stream) {
  moe_status s = check_rows(rows, K, dtype);
  if (s != MOE_OK) return s;
  if (!ld_x) ld_x = K;
  if (!ld_q) ld_q = K;
  if (ld_x < K || ld_q < K || (row_token && n_tokens < 0)) return MOE_ERR_INVALID_ARG;
  if (rows == 0) return MOE_OK;
  if (!x && !(row_token && n_tokens == 0)) return MOE_ERR_INVALID_ARG;  // (without tokens no source is read)
  if (!on(x, 2) || !q || !scale || !on(scale, 4) || (row_token && !on(row_token, 4))) return MOE_ERR_INVALID_ARG;
  return from(launch_quant_rows(dtype, false, rows, K, x, ld_x, row_token, n_tokens, q, ld_q, scale,
                                static_cast<cudaStream_t>(stream)));
}

moe_status moe_swiglu(int32_t rows, int32_t F, int32_t dtype, const void* gate_up, int64_t ld_gu, void* h,
                      int64_t ld_h, void* stream) {
  moe_status s = check_rows(rows, F, dtype);
  if (s != MOE_OK) return s;
  if (!ld_gu) ld_gu = 2 * (int64_t)F;
  if (!ld_h) ld_h = F;
  if (ld_gu < 2 * (int64_t)F || ld_h < F) return MOE_ERR_INVALID_ARG;
  if (rows == 0) return MOE_OK;
  if (!gate_up || !on(gate_up, 2) || !h || !on(h, 2)) return MOE_ERR_INVALID_ARG;
  return from(launch_swiglu(dtype, rows, F, gate_up, ld_gu, h, ld_h, static_cast<cudaStream_t>(stream)));
}

moe_status moe_swiglu_quant_i8(int32_t rows, int32_t F, int32_t dtype, const void* gate_up, int64_t ld_gu,
                               int8_t* q, int64_t ld_q, float* scale, void* stream) {
  moe_status s = check_rows(rows, F, dtype);
  if (s != MOE_OK) return s;
  if (!ld_gu) ld_gu = 2 * (int64_t)F;
  if (!ld_q) ld_q = F;
  if (ld_gu < 2 * (int64_t)F || ld_q < F) return MOE_ERR_INVALID_ARG;
  if (rows == 0) return MOE_OK;
  if (!gate_up || !on(gate_up, 2) || !q || !scale || !on(scale, 4)) return MOE_ERR_INVALID_ARG;
  return from(launch_quant_rows(dtype, true, rows, F, gate_up, ld_gu, nullptr, 0, q, ld_q, scale,
                                static_cast<cudaStream_t>(stream)));
}

moe_status moe_swiglu_grad(int32_t rows, int32_t F, int32_t dtype, const void* gate_up, int64_t ld_gu,
                           const void* dh, int64_t ld_h, void* dgate_up, int64_t ld_d, void* stream) {
  moe_status s = check_rows(rows, F, dtype);
  if (s != MOE_OK) return s;
  if (!ld_gu) ld_gu = 2 * (int64_t)F;
  if (!ld_d) ld_d = 2 * (int64_t)F;
  if (!ld_h) ld_h = F;
  if (ld_gu < 2 * (int64_t)F || ld_d < 2 * (int64_t)F || ld_h < F) return MOE_ERR_INVALID_ARG;
  if (rows == 0) return MOE_OK;
  if (!gate_up || !on(gate_up, 2) || !dh || !on(dh, 2) || !dgate_up || !on(dgate_up, 2)) return MOE_ERR_INVALID_ARG;
  if (dgate_up == gate_up && ld_d != ld_gu) return MOE_ERR_INVALID_ARG;
  return from(launch_swiglu_grad(dtype, rows, F, gate_up, ld_gu, dh, ld_h, dgate_up, ld_d,
                                 static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
