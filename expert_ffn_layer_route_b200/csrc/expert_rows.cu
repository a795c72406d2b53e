// Row operators around the grouped products: SwiGLU, its gradient, and the
// 8-bit integer rows the int8 product reads (from activation rows, or straight
// from the gate/up product through SwiGLU).
//
//   silu(g) = g s, s = 1 / (1 + e^-g);   h = silu(g) u
//   dg = dh u s (1 + g (1 - s));         du = dh silu(g)
//   codes of a row v: amax = max|v|, scale = amax / 127, inv = 127 / amax (two
//   fp32 divisions), q = round-to-nearest-even(v inv) clamped to +-127
// All sums, products and statistics are fp32.  Every value is read once and
// written once: these kernels are bound by HBM (8192 x 14336: SwiGLU 110 us, its
// gradient 167 us, 6.4 and 7.0 TB/s), the int8 rows by the latencies of a row.
#include "expert_rows.cuh"

#include <type_traits>

#include "common.cuh"
#include "launch.cuh"
#include "profile.cuh"

namespace moe {

namespace {

constexpr int kRowThreads = 256;
constexpr float kCodeFloor = 7.52316385e-37f;  // 2^-120: below it a row is stored as zeros (127 / amax would overflow)

template <typename T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) {
  return __bfloat162float(v);
}
template <>
__device__ __forceinline__ float to_f32<__half>(__half v) {
  return __half2float(v);
}
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) {
  return __float2half_rn(v);
}

// W values of one access: 8 (16 bytes) where rows allow it, else 1.
template <typename T, int W>
__device__ __forceinline__ void load(const T* p, float (&v)[W]) {
  if constexpr (W == 8) {
    const uint4 u = __ldg(reinterpret_cast<const uint4*>(p));
    const T* e = reinterpret_cast<const T*>(&u);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = to_f32(e[i]);
  } else {
    v[0] = to_f32(*p);
  }
}
template <typename T, int W>
__device__ __forceinline__ void store(T* p, const float (&v)[W]) {
  if constexpr (W == 8) {
    uint4 u;
    T* e = reinterpret_cast<T*>(&u);
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = from_f32<T>(v[i]);
    *reinterpret_cast<uint4*>(p) = u;
  } else {
    *p = from_f32<T>(v[0]);
  }
}

// exp and the quotient by the fast approximations (a few fp32 ulps): their
// error is far below half a step of the 16-bit results and of the codes.
__device__ __forceinline__ float sigmoid(float g) { return __fdividef(1.f, 1.f + __expf(-g)); }

__device__ __forceinline__ uint32_t low_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}

}  // namespace

template <typename T, int W>
__global__ void __launch_bounds__(kRowThreads)
    swiglu_kernel(const T* __restrict__ gu, int64_t ldg, T* __restrict__ h, int64_t ldh, int F, int chunks) {
  pdl_wait_and_trigger();
  const int row = blockIdx.x / chunks;
  const int c = ((blockIdx.x - row * chunks) * kRowThreads + threadIdx.x) * W;
  if (c >= F) return;
  const T* p = gu + (int64_t)row * ldg + c;
  float g[W], u[W], o[W];
  load<T, W>(p, g);
  load<T, W>(p + F, u);
#pragma unroll
  for (int i = 0; i < W; ++i) o[i] = g[i] * sigmoid(g[i]) * u[i];
  store<T, W>(h + (int64_t)row * ldh + c, o);
}

template <typename T, int W>
__global__ void __launch_bounds__(kRowThreads)
    swiglu_grad_kernel(const T* gu, int64_t ldg, const T* __restrict__ dh, int64_t ldh, T* dgu, int64_t ldd, int F,
                       int chunks) {
  pdl_wait_and_trigger();
  const int row = blockIdx.x / chunks;
  const int c = ((blockIdx.x - row * chunks) * kRowThreads + threadIdx.x) * W;
  if (c >= F) return;
  const T* p = gu + (int64_t)row * ldg + c;
  float g[W], u[W], d[W], dg[W], du[W];
  load<T, W>(dh + (int64_t)row * ldh + c, d);
  // plain loads: dgate_up may be gate_up itself (each thread reads its own values first)
  if constexpr (W == 8) {
    const uint4 a = *reinterpret_cast<const uint4*>(p), b = *reinterpret_cast<const uint4*>(p + F);
    const T *ea = reinterpret_cast<const T*>(&a), *eb = reinterpret_cast<const T*>(&b);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      g[i] = to_f32(ea[i]);
      u[i] = to_f32(eb[i]);
    }
  } else {
    g[0] = to_f32(p[0]);
    u[0] = to_f32(p[F]);
  }
#pragma unroll
  for (int i = 0; i < W; ++i) {
    const float s = sigmoid(g[i]);
    du[i] = d[i] * (g[i] * s);
    dg[i] = d[i] * u[i] * (s * fmaf(g[i], 1.f - s, 1.f));
  }
  T* o = dgu + (int64_t)row * ldd + c;
  store<T, W>(o, dg);
  store<T, W>(o + F, du);
}

// One block of NT threads per row.  V > 0: the row's values stay in registers
// between the maximum and the codes (V vectors of W per thread); V = 0: rows too
// long for that are read (and SwiGLU computed) twice, the second time from
// L1/L2.  A row's loads, its maximum and its stores come one after the other, so
// what fills an SM is rows side by side: small blocks, 8 of 128 threads (3 of 384
// for long rows).  Measured: 8192 rows of 4096, 34 us against 45 with 2 blocks of
// 512; SwiGLU of 8192 x 14336 into codes 134 us (4.4 TB/s) against 154.  A
// persistent block that copies rows ahead into shared memory took 60 and 140 us.
template <typename T, bool kSwiglu, int W, int V, int NT>
__global__ void __launch_bounds__(NT, NT == 384 ? 3 : 1024 / NT)
    quant_rows_kernel(const T* __restrict__ x, int64_t ldx, const int32_t* __restrict__ row_token, int n_tokens,
                      int8_t* __restrict__ q, int64_t ldq, float* __restrict__ scale, int K) {
  pdl_wait_and_trigger();
  __shared__ float red[NT / 32];
  __shared__ int bad_any;
  const int row = blockIdx.x, tid = threadIdx.x;
  int64_t src = row;
  if (row_token) {
    const int t = __ldg(row_token + row);
    src = (unsigned)t < (unsigned)n_tokens ? t : -1;  // a pair the permutation dropped: a row of zeros
  }
  if (tid == 0) bad_any = 0;
  const T* p = x + (src < 0 ? 0 : src * ldx);
  auto value = [&](int c, float (&v)[W]) {
    load<T, W>(p + c, v);
    if constexpr (kSwiglu) {
      float u[W];
      load<T, W>(p + K + c, u);
#pragma unroll
      for (int i = 0; i < W; ++i) v[i] = v[i] * sigmoid(v[i]) * u[i];
    }
  };
  float keep[V > 0 ? V : 1][W];
  float amax = 0.f;
  float odd = 0.f;  // 0, and NaN once a NaN or an infinity was among the values
  auto take = [&](const float (&v)[W]) {
#pragma unroll
    for (int i = 0; i < W; ++i) {
      odd = fmaf(v[i], 0.f, odd);
      amax = fmaxf(amax, fabsf(v[i]));
    }
  };
  if (src >= 0) {
    if constexpr (V > 0) {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int c = (j * NT + tid) * W;
        if (c < K) {
          value(c, keep[j]);
          take(keep[j]);
        }
      }
    } else {
      for (int c = tid * W; c < K; c += NT * W) {
        float v[W];
        value(c, v);
        take(v);
      }
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  if ((tid & 31) == 0) red[tid >> 5] = amax;
  __syncthreads();
  if (odd != 0.f) bad_any = 1;  // (NaN)
#pragma unroll
  for (int w = 0; w < NT / 32; ++w) amax = fmaxf(amax, red[w]);
  __syncthreads();
  const bool live = amax >= kCodeFloor && !bad_any;
  const float inv = live ? __fdiv_rn(127.f, amax) : 0.f;
  if (tid == 0) scale[row] = bad_any ? __int_as_float(0x7fc00000) : live ? __fdiv_rn(amax, 127.f) : 0.f;
  int8_t* o = q + (int64_t)row * ldq;
  auto put = [&](int c, const float (&v)[W]) {
    // |v inv| < 127.5: adding 1.5 * 2^23 rounds it to an integer, ties to even,
    // whose two's complement is the sum's low byte
    uint32_t b[W];
#pragma unroll
    for (int i = 0; i < W; ++i)
      b[i] = live ? __float_as_uint(__fadd_rn(__fmul_rn(v[i], inv), 12582912.f)) : 0u;
    if constexpr (W == 8)
      *reinterpret_cast<uint2*>(o + c) = make_uint2(low_bytes(b[0], b[1], b[2], b[3]), low_bytes(b[4], b[5], b[6], b[7]));
    else
      o[c] = (int8_t)b[0];
  };
  if constexpr (V > 0) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int c = (j * NT + tid) * W;
      if (c < K) put(c, keep[j]);
    }
  } else {
    for (int c = tid * W; c < K; c += NT * W) {
      float v[W];
#pragma unroll
      for (int i = 0; i < W; ++i) v[i] = 0.f;
      if (src >= 0) value(c, v);
      put(c, v);
    }
  }
}

// ------------------------------------------------------------------ host side
static bool on16(const void* p, int64_t ld, int elem) {
  return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && (ld * elem) % 16 == 0;
}

template <typename T>
static cudaError_t swiglu_t(int rows, int F, const void* gu, int64_t ldg, void* h, int64_t ldh, cudaStream_t st) {
  ProfScope prof("swiglu", st);
  const bool wide = F % 8 == 0 && on16(gu, ldg, 2) && on16(h, ldh, 2);
  const int chunks = (F + kRowThreads * (wide ? 8 : 1) - 1) / (kRowThreads * (wide ? 8 : 1));
  const dim3 grid((unsigned)((int64_t)rows * chunks));
  return launch_pdl(wide ? swiglu_kernel<T, 8> : swiglu_kernel<T, 1>, grid, dim3(kRowThreads), 0, st,
                    static_cast<const T*>(gu), ldg, static_cast<T*>(h), ldh, F, chunks);
}

cudaError_t launch_swiglu(int dtype, int rows, int F, const void* gu, int64_t ldg, void* h, int64_t ldh,
                          cudaStream_t st) {
  return dtype == MOE_T_BF16 ? swiglu_t<__nv_bfloat16>(rows, F, gu, ldg, h, ldh, st)
                             : swiglu_t<__half>(rows, F, gu, ldg, h, ldh, st);
}

template <typename T>
static cudaError_t swiglu_grad_t(int rows, int F, const void* gu, int64_t ldg, const void* dh, int64_t ldh, void* dgu,
                                 int64_t ldd, cudaStream_t st) {
  ProfScope prof("swiglu_grad", st);
  const bool wide = F % 8 == 0 && on16(gu, ldg, 2) && on16(dh, ldh, 2) && on16(dgu, ldd, 2);
  const int chunks = (F + kRowThreads * (wide ? 8 : 1) - 1) / (kRowThreads * (wide ? 8 : 1));
  const dim3 grid((unsigned)((int64_t)rows * chunks));
  return launch_pdl(wide ? swiglu_grad_kernel<T, 8> : swiglu_grad_kernel<T, 1>, grid, dim3(kRowThreads), 0, st,
                    static_cast<const T*>(gu), ldg, static_cast<const T*>(dh), ldh, static_cast<T*>(dgu), ldd, F,
                    chunks);
}

cudaError_t launch_swiglu_grad(int dtype, int rows, int F, const void* gu, int64_t ldg, const void* dh, int64_t ldh,
                               void* dgu, int64_t ldd, cudaStream_t st) {
  return dtype == MOE_T_BF16 ? swiglu_grad_t<__nv_bfloat16>(rows, F, gu, ldg, dh, ldh, dgu, ldd, st)
                             : swiglu_grad_t<__half>(rows, F, gu, ldg, dh, ldh, dgu, ldd, st);
}

template <typename T, bool kSwiglu>
static cudaError_t quant_t(int rows, int K, const void* x, int64_t ldx, const int32_t* row_token, int n_tokens,
                           int8_t* q, int64_t ldq, float* scale, cudaStream_t st) {
  ProfScope prof(kSwiglu ? "swiglu_quant_i8" : "quant_rows_i8", st);
  const bool wide = K % 8 == 0 && on16(x, ldx, 2) && (reinterpret_cast<uintptr_t>(q) & 7) == 0 && ldq % 8 == 0;
  auto go = [&](auto w, auto v, auto nt) {
    constexpr int W = decltype(w)::value, V = decltype(v)::value, NT = decltype(nt)::value;
    return launch_pdl(quant_rows_kernel<T, kSwiglu, W, V, NT>, dim3(rows), dim3(NT), 0, st, static_cast<const T*>(x),
                      ldx, row_token, n_tokens, q, ldq, scale, K);
  };
  using std::integral_constant;
  const integral_constant<int, 0> twice;
  const integral_constant<int, 1> v1;
  const integral_constant<int, 2> v2;
  const integral_constant<int, 3> v3;
  const integral_constant<int, 4> v4;
  const integral_constant<int, 5> v5;
  const integral_constant<int, 8> w8;
  const integral_constant<int, 128> t128;
  const integral_constant<int, 256> t256;
  const integral_constant<int, 384> t384;
  const integral_constant<int, 512> t512;
  if (!wide) return go(v1, twice, t512);
  switch ((K + 1023) / 1024) {  // vectors of 8 for each of 128 threads
    case 1: return go(w8, v1, t128);
    case 2: return go(w8, v2, t128);
    case 3: return go(w8, v3, t128);
    case 4: return go(w8, v4, t128);
    case 5:
    case 6:
    case 7:
    case 8: return go(w8, v4, t256);
    default: break;
  }
  return K <= 8 * 384 * 5 ? go(w8, v5, t384) : go(w8, twice, t512);
}

cudaError_t launch_quant_rows(int dtype, bool swiglu, int rows, int K, const void* x, int64_t ldx,
                              const int32_t* row_token, int n_tokens, int8_t* q, int64_t ldq, float* scale,
                              cudaStream_t st) {
  if (dtype == MOE_T_BF16)
    return swiglu ? quant_t<__nv_bfloat16, true>(rows, K, x, ldx, row_token, n_tokens, q, ldq, scale, st)
                  : quant_t<__nv_bfloat16, false>(rows, K, x, ldx, row_token, n_tokens, q, ldq, scale, st);
  return swiglu ? quant_t<__half, true>(rows, K, x, ldx, row_token, n_tokens, q, ldq, scale, st)
                : quant_t<__half, false>(rows, K, x, ldx, row_token, n_tokens, q, ldq, scale, st);
}

}  // namespace moe
