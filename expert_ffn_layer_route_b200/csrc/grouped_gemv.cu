// The grouped products for a handful of rows (single-token decode), forward
// and int8: see grouped_gemm.cu for the mathematics.
//
// With so few rows the time is that of the weights' bytes and of getting
// started; 128-channel tensor-core tiles are too coarse to spread one token's
// experts evenly over 148 SMs.  Here a warp takes 4 channels of one expert and
// all of the expert's rows: each lane streams 16-byte pieces of the 4 weight
// rows past the activations (L1 keeps those), in fp32 (int8: exact int32 by
// 4-way dot products), and a butterfly adds the lanes.  Nothing is staged and
// nothing waits, so the loads in flight are only bounded by the resident
// warps: 8 x 16 bytes per lane.
#include <type_traits>

#include "grouped_gemm.cuh"

#include "common.cuh"
#include "launch.cuh"
#include "profile.cuh"
#include "row_tail.cuh"

namespace moe {

namespace {

// 24 warps of 80 registers on an SM, in int8 20 of 96: with 80 some 100 bytes a
// thread go through local memory there (gpt-oss-shaped gate/up with its
// quantisation, one token / two tokens 16.5 / 28.3 us, 17.9 / 31.5; 10 rows of 84
// experts, [2145][3555], 16.0, 17.3), in 16 bits nothing does (5 rows, [1275][10201],
// 18.3 us, by 96 registers 19.9).  Blocks of 128 threads: gate/up in bf16, one token /
// two tokens, and one expert alone in int8 24.0 / 45.5, 6.3 us; 3 blocks of 256 24.4
// / 46.4, 6.3; 10 blocks of 128 (fewer registers) 24.4 / 43.8, 7.6.
constexpr int kGvThreads = 128;
constexpr int gv_min_blocks(int type) { return type == MOE_T_INT8 ? 5 : 6; }
constexpr int kGvChan = 4;                             // channels per warp
constexpr int kGvWarps = kGvThreads / 32;

struct GemvArgs {
  const uint8_t* w;
  const uint8_t* x;
  const int32_t* offsets;
  const int32_t* slot_map;
  const float* x_scale;
  const float* w_scale;
  void* out;
  int64_t lda, ldb, stride_w;  // bytes
  int64_t ldo;                 // elements
  int E, rows, n_phys, channels, depth_bytes;
  int out_dtype;
};

enum { kBf16 = MOE_T_BF16, kFp16 = MOE_T_FP16, kI8 = MOE_T_INT8 };

// Weights pass once: they need no place in L1.
__device__ __forceinline__ uint4 load_stream(const uint8_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

struct LoadTail {  // (predicated: 0 where nothing is to be read)
  __device__ __forceinline__ uint32_t u32(const uint8_t* p, bool on) const {
    uint32_t v;
    asm volatile("{\n .reg .pred q;\n setp.ne.u32 q, %2, 0;\n mov.u32 %0, 0;\n @q ld.global.nc.u32 %0, [%1];\n}\n"
                 : "=&r"(v) : "l"(p), "r"((uint32_t)on));
    return v;
  }
  __device__ __forceinline__ uint32_t u16(const uint8_t* p, bool on) const {
    uint32_t v;
    asm volatile("{\n .reg .pred q;\n setp.ne.u32 q, %2, 0;\n mov.u32 %0, 0;\n @q ld.global.nc.u16 %0, [%1];\n}\n"
                 : "=&r"(v) : "l"(p), "r"((uint32_t)on));
    return v;
  }
  __device__ __forceinline__ uint32_t u8(const uint8_t* p, bool on) const {
    uint32_t v;
    asm volatile("{\n .reg .pred q;\n setp.ne.u32 q, %2, 0;\n mov.u32 %0, 0;\n @q ld.global.nc.u8 %0, [%1];\n}\n"
                 : "=&r"(v) : "l"(p), "r"((uint32_t)on));
    return v;
  }
};
// The last n < 16 bytes of a row, zeros behind them, and no read behind them.
__device__ __forceinline__ uint4 load_tail(const uint8_t* p, int n) {
  const LoadTail load;
  return make_uint4(tail_word(p, n, load), tail_word(p + 4, n - 4, load), tail_word(p + 8, n - 8, load),
                    tail_word(p + 12, n - 12, load));
}
// The first n bytes of a 16-byte piece, zeros behind them (what lies behind a
// row's end may be anything, a NaN too).
__device__ __forceinline__ uint4 keep(uint4 v, int n) {
  uint32_t* e = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int b = n - 4 * i;
    e[i] = b >= 4 ? e[i] : b <= 0 ? 0u : e[i] & (0xffffffffu >> (32 - 8 * b));
  }
  return v;
}

template <int kType>
struct Sum {
  using T = float;
};
template <>
struct Sum<kI8> {
  using T = int;
};

template <int kType>
__device__ __forceinline__ void unpack(const uint4& v, float (&f)[8]) {
  const uint32_t e[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (kType == kBf16) {
      f[2 * i] = __uint_as_float(e[i] << 16);
      f[2 * i + 1] = __uint_as_float(e[i] & 0xffff0000u);
    } else {
      const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&e[i]));
      f[2 * i] = h.x;
      f[2 * i + 1] = h.y;
    }
  }
}

// acc[c][r] += the dot product of 16 bytes of channel c's and row r's values.
template <int kType, int R>
__device__ __forceinline__ void dot(const uint4 (&w)[kGvChan], const uint4 (&x)[R],
                                    typename Sum<kType>::T (&acc)[kGvChan][R]) {
  if constexpr (kType == kI8) {
#pragma unroll
    for (int c = 0; c < kGvChan; ++c)
#pragma unroll
      for (int r = 0; r < R; ++r) {
        acc[c][r] = __dp4a((int)w[c].x, (int)x[r].x, acc[c][r]);
        acc[c][r] = __dp4a((int)w[c].y, (int)x[r].y, acc[c][r]);
        acc[c][r] = __dp4a((int)w[c].z, (int)x[r].z, acc[c][r]);
        acc[c][r] = __dp4a((int)w[c].w, (int)x[r].w, acc[c][r]);
      }
  } else {
    float xf[R][8];
#pragma unroll
    for (int r = 0; r < R; ++r) unpack<kType>(x[r], xf[r]);
#pragma unroll
    for (int c = 0; c < kGvChan; ++c) {
      float wf[8];
      unpack<kType>(w[c], wf);
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[c][r] = fmaf(wf[i], xf[r][i], acc[c][r]);
    }
  }
}

// R rows from `row` on, the warp's channels from ch0 on.  kSplit: the block's
// warps share the channels, each takes every kGvWarps-th piece of the depth, and
// the first one adds their sums in order.  kTail: rows do not end on 16 bytes (the
// code for that costs the others 3%: one gpt-oss-shaped token 24.0, 24.7 us).
template <int kType, int R, bool kSplit, bool kTail>
__device__ __forceinline__ void rows_of(const GemvArgs& a, int64_t row, int ch0, int phys, int warp, int lane) {
  constexpr int kStep = kSplit ? 512 * kGvWarps : 512;
  using S = typename Sum<kType>::T;
  const uint8_t* w[kGvChan];
  const uint8_t* x[R];
#pragma unroll
  for (int c = 0; c < kGvChan; ++c)  // (past the last channel: the last again, not stored)
    w[c] = a.w + phys * a.stride_w + min(ch0 + c, a.channels - 1) * a.lda;
#pragma unroll
  for (int r = 0; r < R; ++r) x[r] = a.x + (row + r) * a.ldb;
  S acc[kGvChan][R];
#pragma unroll
  for (int c = 0; c < kGvChan; ++c)
#pragma unroll
    for (int r = 0; r < R; ++r) acc[c][r] = 0;
  const int whole = kTail ? a.depth_bytes & ~15 : a.depth_bytes;
  int b = lane * 16 + (kSplit ? warp * 512 : 0);
  for (; b + kStep < whole; b += 2 * kStep) {
    uint4 w0[kGvChan], w1[kGvChan], x0[R], x1[R];
#pragma unroll
    for (int c = 0; c < kGvChan; ++c) w0[c] = load_stream(w[c] + b);
#pragma unroll
    for (int c = 0; c < kGvChan; ++c) w1[c] = load_stream(w[c] + b + kStep);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      x0[r] = __ldg(reinterpret_cast<const uint4*>(x[r] + b));
      x1[r] = __ldg(reinterpret_cast<const uint4*>(x[r] + b + kStep));
    }
    dot<kType, R>(w0, x0, acc);
    dot<kType, R>(w1, x1, acc);
  }
  // A row's last bytes, fewer than 16 (kTail), come with the bytes up to the next 16, which every row but a buffer's
  // last one has behind it by its pitch; those of a last one by themselves.
  const bool w_ends = kTail && phys == a.n_phys - 1 && ch0 + kGvChan >= a.channels;
  const bool x_ends = kTail && row + R == a.rows;
  for (; b < a.depth_bytes; b += kStep) {
    const int n = a.depth_bytes - b;
    uint4 w0[kGvChan], x0[R];
    if (kTail && w_ends && n < 16) {
#pragma unroll
      for (int c = 0; c < kGvChan; ++c) w0[c] = load_tail(w[c] + b, n);
    } else {
#pragma unroll
      for (int c = 0; c < kGvChan; ++c) w0[c] = load_stream(w[c] + b);
    }
    if (kTail && x_ends && n < 16) {
#pragma unroll
      for (int r = 0; r < R; ++r) x0[r] = load_tail(x[r] + b, n);
    } else {
#pragma unroll
      for (int r = 0; r < R; ++r) x0[r] = __ldg(reinterpret_cast<const uint4*>(x[r] + b));
    }
    if (kTail && n < 16) {
#pragma unroll
      for (int c = 0; c < kGvChan; ++c) w0[c] = keep(w0[c], n);
#pragma unroll
      for (int r = 0; r < R; ++r) x0[r] = keep(x0[r], n);
    }
    dot<kType, R>(w0, x0, acc);
  }
#pragma unroll
  for (int c = 0; c < kGvChan; ++c)
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) acc[c][r] += __shfl_xor_sync(0xffffffffu, acc[c][r], o);
  S s = 0;
#pragma unroll
  for (int c = 0; c < kGvChan; ++c)
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (r * kGvChan + c == lane) s = acc[c][r];
  if constexpr (kSplit) {
    __shared__ S part[kGvWarps][kGvChan * R];
    if (lane < kGvChan * R) part[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && lane < kGvChan * R) {
#pragma unroll
      for (int o = 1; o < kGvWarps; ++o) s += part[o][lane];
    }
    __syncthreads();  // (the next rows' sums come to the same place)
    if (warp != 0) return;
  }
  if (lane < kGvChan * R) {
    const int lr = lane / kGvChan, ch = ch0 + lane % kGvChan;
    if (ch < a.channels) {
      float f = (float)s;
      if constexpr (kType == kI8)
        f *= __ldg(a.x_scale + row + lr) * __ldg(a.w_scale + (int64_t)phys * a.channels + ch);
      const int64_t o = (row + lr) * a.ldo + ch;
      if (a.out_dtype == MOE_T_FP32)
        static_cast<float*>(a.out)[o] = f;
      else if (a.out_dtype == MOE_T_BF16)
        static_cast<__nv_bfloat16*>(a.out)[o] = __float2bfloat16_rn(f);
      else
        static_cast<__half*>(a.out)[o] = __float2half_rn(f);
    }
  }
}

}  // namespace

// Grid: (channel blocks, rows); the blocks of a group's first row serve the
// whole group, those of its other rows end at once, so that a group's weights
// are read once whatever the routing.
template <int kType, bool kSplit, bool kTail>
__global__ void __launch_bounds__(kGvThreads, gv_min_blocks(kType)) grouped_gemv_kernel(const GemvArgs a) {
  // The group that starts at the block's row, its expert and rows in one word: the lowest resident expert's, where
  // offsets that go back and forth claim the row for several.
  constexpr int kRowBits = 8, kNone = 0x7fffffff;
  __shared__ int s_group;
  const int tid = threadIdx.x, lane = tid & 31;
  const int row = blockIdx.y;
  if (tid == 0) s_group = kNone;
  pdl_wait_and_trigger();
  __syncthreads();
  for (int e = tid; e < a.E; e += kGvThreads) {
    const int lo = __ldg(a.offsets + e), hi = __ldg(a.offsets + e + 1);
    if (lo < 0 || hi < lo || hi > a.rows) {
      set_status(MOE_ERR_DEVICE_INDEX);
    } else if (lo == row && hi > lo) {
      const int p = a.slot_map ? __ldg(a.slot_map + e) : e;
      if (p >= 0 && p < a.n_phys)
        atomicMin(&s_group, e << kRowBits | (hi - lo));
      else if (p != -1)  // (-1: not resident, its rows are left as they are)
        set_status(MOE_ERR_DEVICE_INDEX);
    }
  }
  __syncthreads();
  const int group = s_group, warp = tid >> 5;
  if (group == kNone) return;
  const int n = group & ((1 << kRowBits) - 1), expert = group >> kRowBits;
  const int phys = a.slot_map ? __ldg(a.slot_map + expert) : expert;
  const int ch0 = (kSplit ? blockIdx.x : blockIdx.x * kGvWarps + warp) * kGvChan;
  if (ch0 >= a.channels) return;
  int r = 0;
  for (; r + 2 <= n; r += 2) rows_of<kType, 2, kSplit, kTail>(a, row + r, ch0, phys, warp, lane);
  if (r < n) rows_of<kType, 1, kSplit, kTail>(a, row + r, ch0, phys, warp, lane);
}

namespace {

int64_t groups_of(const GroupedProblem& p) { return p.E < p.rows ? p.E : p.rows; }
int depth_bytes_of(const GroupedProblem& p) { return p.K * (p.kind == kGgInt8 ? 1 : 2); }
int64_t blocks_of(const GroupedProblem& p) { return ((int64_t)p.N + kGvWarps * kGvChan - 1) / (kGvWarps * kGvChan); }

// Few channels: a block to 4 of them, its warps along the depth, where whole
// warps would leave SMs idle (one expert, bf16, one row: [1275][10200] 17.2 us,
// split 7.6; [2080][3488] 5.5, 4.9; [5760][2880] 9.6, 8.9, but with half the
// depth's bytes, in int8, 8.2, 9.7).
bool split_depth(const GroupedProblem& p, int n_sms) {
  const int64_t blocks = groups_of(p) * blocks_of(p);
  return blocks < n_sms || (blocks < 3 * n_sms && depth_bytes_of(p) >= 4096);
}

}  // namespace

// Up to 12 rows (int8: 16) and about two per expert in use; measured against the
// tensor-core kernel (us, this kernel first): gpt-oss-shaped bf16 gate/up, 128
// experts, 4 / 8 / 12 / 16 rows 24.6 / 46.6 / 62.7 / 78.0 against 33.6 / 50.5 /
// 67.9 / 77.5, int8 with its quantisation 16.3 / 28.3 / 37.6 / 45.8 against
// 24.6 / 39.0 / 43.8 / 50.0; one such expert, 1 / 2 / 4 rows 9.6 / 12.4 / 17.8
// against 14.2 / 13.9 / 14.1; the tiny layer's 16 / 32 rows 5.0 / 6.7 against
// 4.9 / 4.9.
// With few channels 128-channel tiles leave most SMs idle: then up to six rows
// per expert ([1275][10200] with 5 / 12 rows 16.0 / 32.2 against 36.3 / 36.9,
// [2080][3488] with 5 / 8 rows 11.6 / 15.1 against 13.0).
bool grouped_gemv_pays(const GroupedProblem& p, int n_sms) {
  if (p.kind != kGgForward && p.kind != kGgInt8) return false;
  const int64_t per_expert = split_depth(p, n_sms) ? 6 : 2;
  return p.rows <= (p.kind == kGgInt8 ? 16 : 12) && p.rows <= per_expert * groups_of(p);
}

cudaError_t launch_grouped_gemv(const GroupedProblem& p, int n_sms, cudaStream_t st) {
  GemvArgs a;
  a.w = static_cast<const uint8_t*>(p.a);
  a.x = static_cast<const uint8_t*>(p.b);
  a.offsets = p.offsets;
  a.slot_map = p.slot_map;
  a.x_scale = p.x_scale;
  a.w_scale = p.w_scale;
  a.out = p.out;
  a.lda = p.lda_bytes;
  a.ldb = p.ldb_bytes;
  a.stride_w = p.stride_w_bytes;
  a.ldo = p.ldo;
  a.E = p.E;
  a.rows = p.rows;
  a.n_phys = p.n_phys;
  a.channels = p.N;
  a.depth_bytes = depth_bytes_of(p);
  a.out_dtype = p.out_dtype;
  ProfScope prof(p.kind == kGgInt8 ? "grouped_gemm_i8" : "grouped_gemm", st);
  const bool split = split_depth(p, n_sms);
  const dim3 grid((unsigned)(split ? (p.N + kGvChan - 1) / kGvChan : blocks_of(p)), p.rows);
  auto launch = [&](auto type) {
    constexpr int kType = decltype(type)::value;
    const bool tail = a.depth_bytes % 16 != 0;
    auto k = split ? (tail ? grouped_gemv_kernel<kType, true, true> : grouped_gemv_kernel<kType, true, false>)
                   : (tail ? grouped_gemv_kernel<kType, false, true> : grouped_gemv_kernel<kType, false, false>);
    return launch_pdl(k, grid, dim3(kGvThreads), 0, st, a);
  };
  if (p.kind == kGgInt8) return launch(std::integral_constant<int, kI8>{});
  return p.dtype == MOE_T_BF16 ? launch(std::integral_constant<int, kBf16>{})
                               : launch(std::integral_constant<int, kFp16>{});
}

}  // namespace moe
