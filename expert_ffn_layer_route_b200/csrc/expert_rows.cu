// Row operators around the grouped products: SwiGLU, its gradient, and the
// 8-bit integer rows the int8 product reads (from activation rows, or straight
// from the gate/up product through SwiGLU).
//
//   silu(g) = g s, s = 1 / (1 + e^-g);   h = silu(g) u
//   dg = dh u s (1 + g (1 - s));         du = dh silu(g)
//   codes of a row v: amax = max|v|, scale = amax / 127, inv = 127 / amax (two
//   fp32 divisions), q = round-to-nearest-even(v inv) clamped to +-127
// All sums, products and statistics are fp32.  Every value is read once and
// written once.  SwiGLU and its gradient are bound by HBM (8192 x 14336: 109 and
// 168 us, 6.5 and 7.0 TB/s); the int8 rows by the latencies of a row (8192 x 4096:
// 34 us, 3.0 TB/s), those from SwiGLU also by their exactly rounded steps (8192 x
// 14336: 180 us, 3.3 TB/s).
#include "expert_rows.cuh"

#include <algorithm>
#include <initializer_list>
#include <type_traits>
#include <utility>

#include "common.cuh"
#include "devinfo.cuh"
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

// W values of one access: 8 (16 bytes) or 2 (4 bytes) where rows allow it, else 1.
template <typename T, int W>
__device__ __forceinline__ void unpack(const T* e, float (&v)[W]) {
#pragma unroll
  for (int i = 0; i < W; ++i) v[i] = to_f32(e[i]);
}
template <typename T, int W>
__device__ __forceinline__ void load(const T* p, float (&v)[W]) {
  if constexpr (W == 8) {
    const uint4 u = __ldg(reinterpret_cast<const uint4*>(p));
    unpack<T, W>(reinterpret_cast<const T*>(&u), v);
  } else if constexpr (W == 2) {
    const uint32_t u = __ldg(reinterpret_cast<const uint32_t*>(p));
    unpack<T, W>(reinterpret_cast<const T*>(&u), v);
  } else {
    v[0] = to_f32(*p);
  }
}
template <typename T, int W>
__device__ __forceinline__ void load_plain(const T* p, float (&v)[W]) {  // (what this kernel may write too)
  if constexpr (W == 8) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    unpack<T, W>(reinterpret_cast<const T*>(&u), v);
  } else if constexpr (W == 2) {
    const uint32_t u = *reinterpret_cast<const uint32_t*>(p);
    unpack<T, W>(reinterpret_cast<const T*>(&u), v);
  } else {
    v[0] = to_f32(*p);
  }
}
template <typename T, int W>
__device__ __forceinline__ void store(T* p, const float (&v)[W]) {
  if constexpr (W == 1) {
    *p = from_f32<T>(v[0]);
  } else {
    typename std::conditional<W == 8, uint4, uint32_t>::type u;
    T* e = reinterpret_cast<T*>(&u);
#pragma unroll
    for (int i = 0; i < W; ++i) e[i] = from_f32<T>(v[i]);
    *reinterpret_cast<decltype(u)*>(p) = u;
  }
}

// exp and the quotient by the fast approximations.  The first is off by 2 + 1.173
// |g| units in the last place (some 100 at g = -87), the second by 2: 1e-5 at most,
// well below half a step of the 16-bit results.  Codes are not made this way, as
// it turns over those that lie next to a border (row_values).  Below g = -87.3 the
// quotient is 0; to keep e^g in factors there costs what would else be HBM's time
// (the gradient included, 8192 x 14336: 335 us, 287 where only vectors with such a
// value do it, 267).
__device__ __forceinline__ float sigmoid(float g) { return __fdividef(1.f, 1.f + __expf(-g)); }

__device__ __forceinline__ uint32_t low_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}

}  // namespace

// Vectors of all rows in one line, U of them a thread (a block's threads side by
// side): short rows fill blocks too, and narrow vectors still have U loads in
// flight.
template <typename T, int W, int U>
__global__ void __launch_bounds__(kRowThreads)
    swiglu_kernel(const T* __restrict__ gu, int64_t ldg, T* __restrict__ h, int64_t ldh, int F, uint32_t per_row,
                  uint32_t total) {
  pdl_wait_and_trigger();
  float g[U][W], u[U][W];
  const uint32_t first = blockIdx.x * (kRowThreads * U) + threadIdx.x;
#pragma unroll
  for (int k = 0; k < U; ++k) {
    const uint32_t i = first + k * kRowThreads;
    if (i < total) {
      const uint32_t row = i / per_row;
      const T* p = gu + row * ldg + (i - row * per_row) * W;
      load<T, W>(p, g[k]);
      load<T, W>(p + F, u[k]);
    }
  }
#pragma unroll
  for (int k = 0; k < U; ++k) {
    const uint32_t i = first + k * kRowThreads;
    if (i < total) {
      const uint32_t row = i / per_row;
      float o[W];
#pragma unroll
      for (int e = 0; e < W; ++e) o[e] = g[k][e] * sigmoid(g[k][e]) * u[k][e];
      store<T, W>(h + row * ldh + (i - row * per_row) * W, o);
    }
  }
}

template <typename T, int W, int U>
__global__ void __launch_bounds__(kRowThreads)
    swiglu_grad_kernel(const T* gu, int64_t ldg, const T* __restrict__ dh, int64_t ldh, T* dgu, int64_t ldd, int F,
                       uint32_t per_row, uint32_t total) {
  pdl_wait_and_trigger();
  float g[U][W], u[U][W], d[U][W];
  const uint32_t first = blockIdx.x * (kRowThreads * U) + threadIdx.x;
#pragma unroll
  for (int k = 0; k < U; ++k) {
    const uint32_t i = first + k * kRowThreads;
    if (i < total) {
      const uint32_t row = i / per_row, c = (i - row * per_row) * W;
      load<T, W>(dh + row * ldh + c, d[k]);
      // (dgate_up may be gate_up itself: each thread reads its own values first)
      load_plain<T, W>(gu + row * ldg + c, g[k]);
      load_plain<T, W>(gu + row * ldg + c + F, u[k]);
    }
  }
#pragma unroll
  for (int k = 0; k < U; ++k) {
    const uint32_t i = first + k * kRowThreads;
    if (i < total) {
      const uint32_t row = i / per_row, c = (i - row * per_row) * W;
      float dg[W], du[W];
#pragma unroll
      for (int e = 0; e < W; ++e) {
        const float s = sigmoid(g[k][e]);
        du[e] = d[k][e] * (g[k][e] * s);
        dg[e] = d[k][e] * u[k][e] * (s * fmaf(g[k][e], 1.f - s, 1.f));
      }
      T* o = dgu + row * ldd + c;
      store<T, W>(o, dg);
      store<T, W>(o + F, du);
    }
  }
}

// W values of a row from element c on: of the row itself, or of silu(g) u.  Past
// the row's end: zeros.
template <typename T, bool kSwiglu, int W>
__device__ __forceinline__ void row_values(const T* p, int c, int K, float (&v)[W]) {
  if (W == 1 || kSwiglu || c + W <= K) {  // (SwiGLU rows are only read W at a time where W divides them)
    load<T, W>(p + c, v);
    if constexpr (kSwiglu) {
      float u[W];
      load<T, W>(p + K + c, u);
#pragma unroll
      for (int i = 0; i < W; ++i)  // exactly rounded steps: approximate ones turn codes over that lie next to a border
        v[i] = __fmul_rn(__fdiv_rn(v[i], __fadd_rn(1.f, expf(-v[i]))), u[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < W; ++i) v[i] = c + i < K ? to_f32(p[c + i]) : 0.f;
  }
}

template <bool kWhole, int W>
__device__ __forceinline__ void put_codes(int8_t* o, int c, int K, const float (&v)[W], float inv, bool live) {
  // |v inv| < 127.5: adding 1.5 * 2^23 rounds it to an integer, ties to even,
  // whose two's complement is the sum's low byte
  uint32_t b[W];
#pragma unroll
  for (int i = 0; i < W; ++i) b[i] = live ? __float_as_uint(__fadd_rn(__fmul_rn(v[i], inv), 12582912.f)) : 0u;
  if (W > 1 && !kWhole && c + W > K) {
#pragma unroll
    for (int i = 0; i < W; ++i)
      if (c + i < K) o[c + i] = (int8_t)b[i];
  } else if constexpr (W == 8) {
    *reinterpret_cast<uint2*>(o + c) = make_uint2(low_bytes(b[0], b[1], b[2], b[3]), low_bytes(b[4], b[5], b[6], b[7]));
  } else if constexpr (W == 2) {
    *reinterpret_cast<uint16_t*>(o + c) = (uint16_t)__byte_perm(b[0], b[1], 0x0040);
  } else {
    o[c] = (int8_t)b[0];
  }
}

// Short rows: one warp each, V vectors of W a lane in registers.
template <typename T, bool kSwiglu, int W, int V>
__global__ void __launch_bounds__(kRowThreads, 4)
    quant_short_rows_kernel(const T* __restrict__ x, int64_t ldx, const int32_t* __restrict__ row_token, int n_tokens,
                            int8_t* __restrict__ q, int64_t ldq, float* __restrict__ scale, int K, int rows) {
  pdl_wait_and_trigger();
  const int lane = threadIdx.x & 31, row = blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5);
  if (row >= rows) return;
  int64_t src = row;
  if (row_token) {
    const int t = __ldg(row_token + row);
    src = (unsigned)t < (unsigned)n_tokens ? t : -1;  // a pair the permutation dropped: a row of zeros
  }
  const T* p = x + (src < 0 ? 0 : src * ldx);
  float keep[V][W], amax = 0.f, odd = 0.f;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int c = (j * 32 + lane) * W;
    if (src >= 0 && c < K) {
      row_values<T, kSwiglu, W>(p, c, K, keep[j]);
#pragma unroll
      for (int i = 0; i < W; ++i) {
        odd = fmaf(keep[j][i], 0.f, odd);
        amax = fmaxf(amax, fabsf(keep[j][i]));
      }
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  const bool bad = __any_sync(0xffffffffu, odd != 0.f);  // (NaN)
  const bool live = amax >= kCodeFloor && !bad;
  const float inv = live ? __fdiv_rn(127.f, amax) : 0.f;
  if (lane == 0) scale[row] = bad ? __int_as_float(0x7fc00000) : live ? __fdiv_rn(amax, 127.f) : 0.f;
  int8_t* o = q + (int64_t)row * ldq;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int c = (j * 32 + lane) * W;
    if (c < K) put_codes<kSwiglu, W>(o, c, K, keep[j], inv, live);
  }
}

// One block of NT threads per row.  V > 0: the row's values stay in registers
// between the maximum and the codes (V vectors of W per thread); V = 0: rows too
// long for that are read (and SwiGLU computed) twice, the second time from
// L1/L2.  A row's loads, its maximum and its stores come one after the other, so
// what fills an SM is rows side by side: small blocks, 8 of 128 threads (3 of 384
// for long rows).  Measured: 8192 rows of 4096, 34 us against 45 with 2 blocks of
// 512; SwiGLU of 8192 x 14336 into codes 180 us (by fast steps, that turn some codes
// over, 134 against 154; 48 bytes a thread of that instance go through local
// memory).  A persistent block that copies rows ahead into shared memory took 60
// and, by fast steps, 140 us.
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
  auto value = [&](int c, float (&v)[W]) { row_values<T, kSwiglu, W>(p, c, K, v); };
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
  auto put = [&](int c, const float (&v)[W]) { put_codes<kSwiglu, W>(o, c, K, v, inv, live); };
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
// Widest access that F values a row, bases and pitches allow: 8, 2 or 1 values.
static int width_of(int F, std::initializer_list<std::pair<const void*, int64_t>> all) {
  uint64_t place = (uint64_t)F * 2;
  for (const auto& p : all) place |= reinterpret_cast<uintptr_t>(p.first) | (uint64_t)p.second * 2;
  return place % 16 == 0 ? 8 : place % 4 == 0 ? 2 : 1;
}

// Vectors a thread takes: 8 narrow ones once that still leaves every SM four
// blocks (12096 x 315 with gradient 51 -> 30 us), else one (667 x 69: 3.0 us, 8.4
// with 8).
static int unroll_of(int64_t rows, int F, int w) {
  return w < 8 && rows * (F / w) >= (int64_t)8 * kRowThreads * 4 * dev_info().sms ? 8 : 1;
}

// launch(first row, grid, vectors a row, vectors) over all rows: at once, as long
// as 31 bits number the vectors.
template <typename L>
static cudaError_t by_rows(int rows, int F, int w, int u, L launch) {
  const int64_t per_row = F / w, most = 0x7fffffff / per_row;
  const int per_block = kRowThreads * u;
  for (int64_t r = 0; r < rows; r += most) {
    const int64_t total = std::min(most, rows - r) * per_row;
    const cudaError_t err = launch(r, dim3((unsigned)((total + per_block - 1) / per_block)), (uint32_t)per_row, (uint32_t)total);
    if (err != cudaSuccess) return err;
  }
  return cudaSuccess;
}

template <typename T>
static cudaError_t swiglu_t(int rows, int F, const void* gu, int64_t ldg, void* h, int64_t ldh, cudaStream_t st) {
  ProfScope prof("swiglu", st);
  const int w = width_of(F, {{gu, ldg}, {h, ldh}});
  const int u = unroll_of(rows, F, w);
  auto k = w == 8   ? swiglu_kernel<T, 8, 1>
           : w == 2 ? (u == 8 ? swiglu_kernel<T, 2, 8> : swiglu_kernel<T, 2, 1>)
                    : (u == 8 ? swiglu_kernel<T, 1, 8> : swiglu_kernel<T, 1, 1>);
  return by_rows(rows, F, w, u, [&](int64_t r, dim3 grid, uint32_t per_row, uint32_t total) {
    return launch_pdl(k, grid, dim3(kRowThreads), 0, st, static_cast<const T*>(gu) + r * ldg, ldg,
                      static_cast<T*>(h) + r * ldh, ldh, F, per_row, total);
  });
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
  const int w = width_of(F, {{gu, ldg}, {dh, ldh}, {dgu, ldd}});
  const int u = unroll_of(rows, F, w);
  auto k = w == 8   ? swiglu_grad_kernel<T, 8, 1>
           : w == 2 ? (u == 8 ? swiglu_grad_kernel<T, 2, 8> : swiglu_grad_kernel<T, 2, 1>)
                    : (u == 8 ? swiglu_grad_kernel<T, 1, 8> : swiglu_grad_kernel<T, 1, 1>);
  return by_rows(rows, F, w, u, [&](int64_t r, dim3 grid, uint32_t per_row, uint32_t total) {
    return launch_pdl(k, grid, dim3(kRowThreads), 0, st, static_cast<const T*>(gu) + r * ldg, ldg,
                      static_cast<const T*>(dh) + r * ldh, ldh, static_cast<T*>(dgu) + r * ldd, ldd, F, per_row, total);
  });
}

cudaError_t launch_swiglu_grad(int dtype, int rows, int F, const void* gu, int64_t ldg, const void* dh, int64_t ldh,
                               void* dgu, int64_t ldd, cudaStream_t st) {
  return dtype == MOE_T_BF16 ? swiglu_grad_t<__nv_bfloat16>(rows, F, gu, ldg, dh, ldh, dgu, ldd, st)
                             : swiglu_grad_t<__half>(rows, F, gu, ldg, dh, ldh, dgu, ldd, st);
}

template <int N>
using Int = std::integral_constant<int, N>;

template <typename T, bool kSwiglu>
static cudaError_t quant_t(int rows, int K, const void* x, int64_t ldx, const int32_t* row_token, int n_tokens,
                           int8_t* q, int64_t ldq, float* scale, cudaStream_t st) {
  ProfScope prof(kSwiglu ? "swiglu_quant_i8" : "quant_rows_i8", st);
  // widest access: 8 or 2 values, as the rows, the half rows of SwiGLU and the codes lie
  const uint64_t in = reinterpret_cast<uintptr_t>(x) | (uint64_t)ldx * 2 | (kSwiglu ? (uint64_t)K * 2 : 0);
  const uint64_t out = reinterpret_cast<uintptr_t>(q) | (uint64_t)ldq;
  const int w = in % 16 == 0 && out % 8 == 0 ? 8 : in % 4 == 0 && out % 2 == 0 ? 2 : 1;
  auto block = [&](auto wc, auto v, auto nt) {
    constexpr int W = decltype(wc)::value, V = decltype(v)::value, NT = decltype(nt)::value;
    return launch_pdl(quant_rows_kernel<T, kSwiglu, W, V, NT>, dim3(rows), dim3(NT), 0, st, static_cast<const T*>(x),
                      ldx, row_token, n_tokens, q, ldq, scale, K);
  };
  auto warp = [&](auto wc, auto v) {
    constexpr int W = decltype(wc)::value, V = decltype(v)::value;
    constexpr int kPer = kRowThreads / 32;
    return launch_pdl(quant_short_rows_kernel<T, kSwiglu, W, V>, dim3((rows - 1) / kPer + 1), dim3(kRowThreads), 0, st,
                      static_cast<const T*>(x), ldx, row_token, n_tokens, q, ldq, scale, K, rows);
  };
  if (w == 8) {
    const Int<8> w8;
    if (K <= 256) return warp(w8, Int<1>{});
    if (K <= 512) return warp(w8, Int<2>{});
    if (K <= 1024) return warp(w8, Int<4>{});
    switch ((K + 1023) / 1024) {  // vectors of 8 for each of 128 threads
      case 2: return block(w8, Int<2>{}, Int<128>{});
      case 3: return block(w8, Int<3>{}, Int<128>{});
      case 4: return block(w8, Int<4>{}, Int<128>{});
      case 5:
      case 6:
      case 7:
      case 8: return block(w8, Int<4>{}, Int<256>{});
      default: break;
    }
    return K <= 8 * 384 * 5 ? block(w8, Int<5>{}, Int<384>{}) : block(w8, Int<0>{}, Int<512>{});
  }
  if (w == 2) {
    const Int<2> w2;
    if (K <= 256) return warp(w2, Int<4>{});
    if (K <= 1024) return warp(w2, Int<16>{});
    if (K <= 4096) return block(w2, Int<8>{}, Int<256>{});
    return K <= 8192 ? block(w2, Int<16>{}, Int<256>{}) : block(w2, Int<0>{}, Int<512>{});
  }
  const Int<1> w1;
  if (K <= 256) return warp(w1, Int<8>{});
  if (K <= 1024) return warp(w1, Int<32>{});
  if (K <= 2048) return block(w1, Int<8>{}, Int<256>{});
  return K <= 4096 ? block(w1, Int<16>{}, Int<256>{}) : block(w1, Int<0>{}, Int<512>{});
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
