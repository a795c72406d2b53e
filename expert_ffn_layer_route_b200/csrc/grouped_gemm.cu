// Products of ragged expert groups with each expert's matrix, forward and for
// both gradients, in 16-bit floats; and the forward product in 8-bit integers.
//
// Rows r in [offsets[e], offsets[e+1]) belong to expert e:
//   forward  out[r][n]   = sum_k x[r][k] w[e][n][k]
//   grad_x   dx[r][k]    = sum_n dy[r][n] w[e][n][k]
//   grad_w   dw[e][n][k] = sum_{r in e} dy[r][n] x[r][k]      (zeros for an empty group)
//   int8     out[r][n]   = x_scale[r] w_scale[e][n] sum_k x[r][k] w[e][n][k]
// All four run as D[channel][column] on the 5th-generation tensor cores, with
// the 128 tensor-memory lanes on the matrix's channels (n, k, n, n) and the
// columns on the ragged rows (grad_w: on k).  A group's rows are the N
// dimension of the MMA, which goes in steps of 16 and is chosen per tile at
// run time, so a group of 3 rows costs 16 columns, not a 128-row tile: small
// groups then run at the speed their weights arrive, and a ragged group wastes
// at most 15 columns.
#include <cstring>

#include "grouped_gemm.cuh"

#include "common.cuh"
#include "launch.cuh"
#include "profile.cuh"
#include "tc_ptx.cuh"
#include "tmap.cuh"

namespace moe {

namespace {

constexpr int kChan = 128;             // channels per tile = TMEM lanes
constexpr int kStageK = 128;           // bytes of the contraction per stage (one swizzle line)
constexpr int kABytes = kChan * kStageK;
constexpr int kSlabBytes = 64 * 128;   // 64 contraction rows x 64 channels of 16 bits
constexpr int kMaxStages = 12;
constexpr int kEpiWarps = 4;
constexpr int kEpiBytes = 2560;        // transposition buffer of one epilogue warp
constexpr int kGgThreads = 32 * (2 + kEpiWarps);

struct alignas(64) GgArgs {
  CUtensorMap tm_a;
  CUtensorMap tm_b;
  const int32_t* offsets;
  const int32_t* slot_map;
  const float* x_scale;
  const float* w_scale;
  void* out;
  int64_t ldo, stride_o;
  int E, rows, n_phys;
  int channels;  // M extent: N (forward, grad_w, int8) or K (grad_x)
  int depth;     // contraction extent in elements (grad_w: unused)
  int cols;      // grad_w: K
  int col_cap;   // widest column tile
  int box_rows;  // rows of one TMA box of B (K-major kinds)
  int stages, stage_bytes, tmem_cols;
  uint32_t idesc;  // instruction descriptor without N
  int out_dtype;
  int vec_ok;  // output rows start on 16-byte boundaries
  int accumulate;
};

// One group's entry in the shared-memory table.
struct Group {
  int tile0;  // first tile
  int row0, n;
  int expert, phys;
};

struct Tile {
  int m0;            // first channel
  int c0, nc;        // first column (row inside the group; grad_w: k) and columns that exist
  int ncols;         // MMA N: nc rounded up to 16
  int row0, n;       // the group's rows
  int expert, phys;
};

__device__ __forceinline__ void store_one(void* out, int dtype, int64_t i, float v) {
  if (dtype == MOE_T_FP32)
    static_cast<float*>(out)[i] = v;
  else if (dtype == MOE_T_BF16)
    static_cast<__nv_bfloat16*>(out)[i] = __float2bfloat16_rn(v);
  else
    static_cast<__half*>(out)[i] = __float2half_rn(v);
}

__device__ __forceinline__ uint32_t pack16(int dtype, float lo, float hi) {
  if (dtype == MOE_T_BF16) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&p);
  }
  const __half2 p = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&p);
}

// The last stage of a grad_w group holds rows of the next group, or none: the
// rows from `left` up to the next multiple of 16 (as far as the MMA reads) are
// cleared in both operands, so that neither their values nor a NaN among them
// reaches the sum.  A contraction row is one 128-byte line of each 64-channel
// slab, whatever the swizzle.
__device__ __forceinline__ void clear_tail(uint8_t* stage, int left, int ncols, int lane) {
  const int per_slab = (16 - (left & 15)) * 8;  // 16-byte pieces
  const int slabs = 2 + ceil_div(ncols, 64);
  for (int i = lane; i < slabs * per_slab; i += 32) {
    const int sl = i / per_slab, w = i - sl * per_slab;
    reinterpret_cast<uint4*>(stage + sl * kSlabBytes + left * 128)[w] = make_uint4(0, 0, 0, 0);
  }
  fence_proxy_async_smem();
  __syncwarp();
}

}  // namespace

template <int kKind>
__global__ void __launch_bounds__(kGgThreads, 1) grouped_gemm_kernel(const __grid_constant__ GgArgs a) {
  constexpr bool kAChanMajor = kKind == kGgGradX || kKind == kGgGradW;  // A rows run along the channels
  constexpr bool kBChanMajor = kKind == kGgGradW;
  constexpr int kElem = kKind == kGgInt8 ? 1 : 2;
  constexpr int kDepthStage = kAChanMajor ? 64 : kStageK / kElem;  // contraction elements per stage
  constexpr int kDepthMma = kKind == kGgInt8 ? 32 : 16;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* ring = smem;
  uint8_t* epi = ring + (size_t)a.stages * a.stage_bytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(epi + kEpiWarps * kEpiBytes);
  uint64_t* empty = full + kMaxStages;
  uint64_t* acc_full = empty + kMaxStages;
  uint64_t* acc_empty = acc_full + 2;
  uint64_t* drain = acc_empty + 2;
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* s_abort = reinterpret_cast<volatile int*>(s_tmem + 1);
  int* s_ngroups = reinterpret_cast<int*>(s_tmem + 2);
  Group* grp = reinterpret_cast<Group*>(s_tmem + 4);  // [E + 1], the groups that have tiles

  if (tid == 0) {
    for (int i = 0; i < a.stages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], kEpiWarps);
    }
    mbar_init(drain, 1);
    *s_abort = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tc::tmem_alloc(s_tmem, a.tmem_cols);
    tc::tmem_relinquish();
  }
  pdl_wait_and_trigger();
  // Group table.  Every thread loads the offsets of some experts (one round of
  // global latency for all of them), then warp 0 compacts and numbers them.
  for (int e = tid; e < a.E; e += kGgThreads) {
    const int lo = __ldg(a.offsets + e), hi = __ldg(a.offsets + e + 1);
    int n = hi - lo, p = e;
    if (lo < 0 || hi < lo || hi > a.rows) {
      set_status(MOE_ERR_DEVICE_INDEX);
      n = 0;
    }
    if (kKind != kGgGradW && a.slot_map) {
      p = __ldg(a.slot_map + e);
      if (n > 0 && (p < 0 || p >= a.n_phys)) {
        if (p != -1) set_status(MOE_ERR_DEVICE_INDEX);
        n = 0;  // not resident: its rows are left as they are
      }
    }
    grp[e].row0 = lo;
    grp[e].n = n;
    grp[e].phys = p;
  }
  __syncthreads();
  const int m_tiles = ceil_div(a.channels, kChan);
  if (warp == 0) {
    int ng = 0, tiles = 0;
    for (int base = 0; base < a.E; base += 32) {
      const int e = base + lane;
      int row0 = 0, n = 0, p = 0, t = 0;
      if (e < a.E) {
        row0 = grp[e].row0;
        n = grp[e].n;
        p = grp[e].phys;
        t = m_tiles * (kKind == kGgGradW ? ceil_div(a.cols, a.col_cap) : ceil_div(n, a.col_cap));
      }
      const uint32_t on = __ballot_sync(0xffffffffu, t > 0);
      int incl = t;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += o;
      }
      if (t > 0) {  // slots at or before this expert's own: already read above
        Group g;
        g.tile0 = tiles + incl - t;
        g.row0 = row0;
        g.n = n;
        g.expert = e;
        g.phys = p;
        grp[ng + __popc(on & ((1u << lane) - 1u))] = g;
      }
      ng += __popc(on);
      tiles += __shfl_sync(0xffffffffu, incl, 31);
      __syncwarp();
    }
    if (lane == 0) {
      grp[ng].tile0 = tiles;
      *s_ngroups = ng;
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem_base = *s_tmem;
  const int ngroups = *s_ngroups;
  const int total_tiles = grp[ngroups].tile0;

  auto decode = [&](int t) {
    int lo = 0, hi = ngroups - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (grp[mid].tile0 <= t) lo = mid; else hi = mid - 1;
    }
    const Group g = grp[lo];
    Tile ti;
    ti.row0 = g.row0;
    ti.n = g.n;
    ti.expert = g.expert;
    ti.phys = g.phys;
    const int local = t - g.tile0;
    const int width = kKind == kGgGradW ? a.cols : g.n;
    const int ct = ceil_div(width, a.col_cap);                 // column tiles, as even as 16 allows
    const int w = (ceil_div(width, ct) + 15) & ~15;
    const int mi = local / ct;                                  // column tiles of one channel tile run side by side
    ti.m0 = mi * kChan;
    ti.c0 = (local - mi * ct) * w;
    ti.nc = min(w, width - ti.c0);
    ti.ncols = (ti.nc + 15) & ~15;
    return ti;
  };
  auto steps_of = [&](const Tile& ti) {
    return ceil_div(kKind == kGgGradW ? ti.n : a.depth, kDepthStage);
  };

  if (warp == 0) {
    // ================================================================ TMA producer
    if (lane == 0) {
      if (a.rows > 0) {
        prefetch_tmap(&a.tm_a);
        prefetch_tmap(&a.tm_b);
      }
      const uint64_t pol = l2_evict_normal_policy();
      uint32_t s = 0, par = 1, cnt = 0;
      for (int t = blockIdx.x; t < total_tiles && !*s_abort; t += gridDim.x) {
        const Tile ti = decode(t);
        const int steps = steps_of(ti);
        const int boxes = kBChanMajor ? ceil_div(ti.ncols, 64) : ceil_div(ti.ncols, a.box_rows);
        const uint32_t bytes = kABytes + boxes * (kBChanMajor ? kSlabBytes : a.box_rows * kStageK);
        for (int ks = 0; ks < steps; ++ks) {
          if (!mbar_wait(&empty[s], par)) {
            *s_abort = 1;
            break;
          }
          uint8_t* sa = ring + (size_t)s * a.stage_bytes;
          uint8_t* sb = sa + kABytes;
          mbar_arrive_expect_tx(&full[s], bytes);
          if (kKind == kGgGradW) {
            const int r = ti.row0 + ks * 64;
            for (int i = 0; i < 2; ++i)
              tma_load_2d(sa + i * kSlabBytes, &a.tm_a, (ti.m0 + 64 * i) * 2, r, &full[s], pol);
            for (int i = 0; i < boxes; ++i)
              tma_load_2d(sb + i * kSlabBytes, &a.tm_b, (ti.c0 + 64 * i) * 2, r, &full[s], pol);
          } else {
            if (kKind == kGgGradX) {
              for (int i = 0; i < 2; ++i)
                tma_load_3d(sa + i * kSlabBytes, &a.tm_a, (ti.m0 + 64 * i) * 2, ks * 64, ti.phys, &full[s], pol);
            } else {
              tma_load_3d(sa, &a.tm_a, ks * kStageK, ti.m0, ti.phys, &full[s], pol);
            }
            for (int i = 0; i < boxes; ++i)
              tma_load_2d(sb + i * a.box_rows * kStageK, &a.tm_b, ks * kStageK,
                          ti.row0 + ti.c0 + i * a.box_rows, &full[s], pol);
          }
          ++cnt;
          if (++s == (uint32_t)a.stages) {
            s = 0;
            par ^= 1;
          }
        }
      }
      // every copy has landed before the block may leave
      const uint32_t first = cnt > (uint32_t)a.stages ? cnt - a.stages : 0;
      for (uint32_t c = first; c < cnt; ++c) mbar_wait(&full[c % a.stages], (c / a.stages) & 1u);
    }
  } else if (warp == 1) {
    // ================================================================ MMA issuer
    // (the whole warp follows the ring; lane 0 issues)
    uint32_t s = 0, par = 0;
    int i = 0;
    for (int t = blockIdx.x; t < total_tiles; t += gridDim.x, ++i) {
      const Tile ti = decode(t);
      const int buf = i & 1;
      if (*s_abort || !mbar_wait(&acc_empty[buf], ((uint32_t)(i >> 1) & 1u) ^ 1u)) {
        *s_abort = 1;
        break;
      }
      tc::fence_after_sync();
      const uint32_t d_tmem = tmem_base + (uint32_t)(buf * a.col_cap);
      const uint32_t idesc = a.idesc | ((uint32_t)(ti.ncols >> 3) << 17);
      const int steps = steps_of(ti);
      const int depth = kKind == kGgGradW ? ti.n : a.depth;
      for (int ks = 0; ks < steps; ++ks) {
        if (!mbar_wait(&full[s], par)) {
          *s_abort = 1;
          break;
        }
        uint8_t* stage = ring + (size_t)s * a.stage_bytes;
        const int left = depth - ks * kDepthStage;
        if (kKind == kGgGradW && left < kDepthStage && (left & 15)) clear_tail(stage, left, ti.ncols, lane);
        tc::fence_after_sync();
        if (lane == 0) {
          const int kmax = min(kDepthStage / kDepthMma, ceil_div(left, kDepthMma));
          const uint32_t sa = smem_u32(stage);
          const uint32_t sb = sa + kABytes;
          for (int kk = 0; kk < kmax; ++kk) {
            const uint64_t da = kAChanMajor ? tc::mnmajor_sw128_desc(sa + kk * 2048, kSlabBytes)
                                            : tc::kmajor_sw128_desc(sa + kk * 32);
            const uint64_t db = kBChanMajor ? tc::mnmajor_sw128_desc(sb + kk * 2048, kSlabBytes)
                                            : tc::kmajor_sw128_desc(sb + kk * 32);
            if (kKind == kGgInt8)
              tc::mma_i8(d_tmem, da, db, idesc, (ks | kk) != 0 ? 1u : 0u);
            else
              tc::mma_bf16(d_tmem, da, db, idesc, (ks | kk) != 0 ? 1u : 0u);
          }
          tc::commit(&empty[s]);
        }
        __syncwarp();
        if (++s == (uint32_t)a.stages) {
          s = 0;
          par ^= 1;
        }
      }
      if (*s_abort) break;
      if (lane == 0) {
        if (steps > 0)
          tc::commit(&acc_full[buf]);
        else
          mbar_arrive(&acc_full[buf]);  // an empty group: the epilogue writes zeros
      }
      __syncwarp();
    }
    if (lane == 0) {  // every MMA of this CTA has completed before TMEM is freed
      tc::commit(drain);
      mbar_wait(drain, 0);
    }
    __syncwarp();
  } else {
    // ================================================================ epilogue
    const int q = warp & 3;  // TMEM lane quadrant of this warp
    uint8_t* buf_t = epi + (warp - 2) * kEpiBytes;
    int i = 0;
    for (int t = blockIdx.x; t < total_tiles; t += gridDim.x, ++i) {
      const Tile ti = decode(t);
      const int buf = i & 1;
      if (*s_abort || !mbar_wait(&acc_full[buf], (uint32_t)(i >> 1) & 1u)) {
        *s_abort = 1;
        break;
      }
      tc::fence_after_sync();
      const uint32_t taddr = tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(buf * a.col_cap);
      const int ch0 = ti.m0 + q * 32;
      if (kKind == kGgGradW) {
        // one row n of dw per thread, 16 columns k at a time
        const int n = ch0 + lane;
        const bool zero = ti.n == 0;
        for (int j0 = 0; j0 < ti.ncols; j0 += 16) {
          uint32_t v[16];
          tc::ld_32x32b_x16(taddr + j0, v);
          tc::ld_wait();
          if (zero) {
#pragma unroll
            for (int j = 0; j < 16; ++j) v[j] = 0u;
          }
          if (n < a.channels) {
            const int64_t o = (int64_t)ti.expert * a.stride_o + (int64_t)n * a.ldo + ti.c0 + j0;
            const bool whole = a.vec_ok && j0 + 16 <= ti.nc && !a.accumulate;
            if (whole && a.out_dtype == MOE_T_FP32) {
              uint4* d = reinterpret_cast<uint4*>(static_cast<float*>(a.out) + o);
#pragma unroll
              for (int j = 0; j < 4; ++j) d[j] = make_uint4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
            } else if (whole) {
              uint32_t p[8];
#pragma unroll
              for (int j = 0; j < 8; ++j)
                p[j] = pack16(a.out_dtype, __uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1]));
              uint4* d = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + o);
              d[0] = make_uint4(p[0], p[1], p[2], p[3]);
              d[1] = make_uint4(p[4], p[5], p[6], p[7]);
            } else {
#pragma unroll
              for (int j = 0; j < 16; ++j) {
                if (j0 + j >= ti.nc) break;
                float f = __uint_as_float(v[j]);
                if (a.accumulate) f += static_cast<float*>(a.out)[o + j];
                store_one(a.out, a.out_dtype, o + j, f);
              }
            }
          }
        }
      } else {
        // 16 rows x 32 channels at a time through shared memory, so that a
        // row's 32 channels leave as 16-byte stores
        float sw = 0.f;
        if (kKind == kGgInt8 && ch0 + lane < a.channels)
          sw = __ldg(a.w_scale + (int64_t)ti.phys * a.channels + ch0 + lane);
        const int64_t row0 = (int64_t)ti.row0 + ti.c0;
        const bool f32 = a.out_dtype == MOE_T_FP32;
        for (int j0 = 0; j0 < ti.ncols; j0 += 16) {
          uint32_t v[16];
          tc::ld_32x32b_x16(taddr + j0, v);
          tc::ld_wait();
          if (kKind == kGgInt8) {
            float sx = 0.f;
            if (lane < 16 && j0 + lane < ti.nc) sx = __ldg(a.x_scale + row0 + j0 + lane);
#pragma unroll
            for (int j = 0; j < 16; ++j)
              v[j] = __float_as_uint((float)(int)v[j] * (__shfl_sync(0xffffffffu, sx, j) * sw));
          }
          if (ch0 >= a.channels) continue;
          __syncwarp();
          if (f32) {
            float* b = reinterpret_cast<float*>(buf_t);
#pragma unroll
            for (int j = 0; j < 16; ++j) b[j * 36 + lane] = __uint_as_float(v[j]);
          } else {
            uint16_t* b = reinterpret_cast<uint16_t*>(buf_t);
#pragma unroll
            for (int j = 0; j < 16; ++j)
              b[j * 40 + lane] = (uint16_t)pack16(a.out_dtype, __uint_as_float(v[j]), 0.f);
          }
          __syncwarp();
          const int per = f32 ? 4 : 8;  // channels per 16-byte store
          const int chunks = 32 / per;
          for (int i2 = lane; i2 < 16 * chunks; i2 += 32) {
            const int j = i2 / chunks, c = (i2 - j * chunks) * per;
            if (j0 + j >= ti.nc || ch0 + c >= a.channels) continue;
            const int64_t o = (row0 + j0 + j) * a.ldo + ch0 + c;
            const uint8_t* src = buf_t + (f32 ? (j * 36 + c) * 4 : (j * 40 + c) * 2);
            if (a.vec_ok && ch0 + c + per <= a.channels) {
              const uint4 w = *reinterpret_cast<const uint4*>(src);
              *reinterpret_cast<uint4*>(static_cast<uint8_t*>(a.out) + o * (f32 ? 4 : 2)) = w;
            } else {
              for (int z = 0; z < per && ch0 + c + z < a.channels; ++z) {
                if (f32)
                  static_cast<float*>(a.out)[o + z] = reinterpret_cast<const float*>(src)[z];
                else
                  static_cast<uint16_t*>(a.out)[o + z] = reinterpret_cast<const uint16_t*>(src)[z];
              }
            }
          }
        }
      }
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&acc_empty[buf]);
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (warp == 1) tc::tmem_dealloc(tmem_base, a.tmem_cols);
}

// ------------------------------------------------------------------ host side
template <int kKind>
static cudaError_t launch_kind(const GgArgs& a, int grid, size_t smem, cudaStream_t st) {
  cudaError_t err = set_dyn_smem_once<grouped_gemm_kernel<kKind>>(smem);
  if (err != cudaSuccess) return err;
  static const char* const names[4] = {"grouped_gemm", "grouped_gemm_grad_x", "grouped_gemm_grad_w",
                                       "grouped_gemm_i8"};
  ProfScope prof(names[kKind], st);
  return launch_pdl(grouped_gemm_kernel<kKind>, dim3(grid), dim3(kGgThreads), smem, st, a);
}

cudaError_t launch_grouped_gemm(const GroupedProblem& p, int n_sms, int smem_max, cudaStream_t st,
                                int* unsupported) {
  *unsupported = 0;
  GgArgs a;
  const int elem = p.kind == kGgInt8 ? 1 : 2;
  const bool gw = p.kind == kGgGradW, gx = p.kind == kGgGradX;
  a.offsets = p.offsets;
  a.slot_map = p.slot_map;
  a.x_scale = p.x_scale;
  a.w_scale = p.w_scale;
  a.out = p.out;
  a.ldo = p.ldo;
  a.stride_o = p.stride_o;
  a.E = p.E;
  a.rows = p.rows;
  a.n_phys = p.n_phys;
  a.channels = gx ? p.K : p.N;
  a.depth = gx ? p.N : p.K;
  a.cols = p.K;
  a.out_dtype = p.out_dtype;
  a.accumulate = p.accumulate;
  const int osz = p.out_dtype == MOE_T_FP32 ? 4 : 2;
  a.vec_ok = (reinterpret_cast<uintptr_t>(p.out) & 15) == 0 && (p.ldo * osz) % 16 == 0 &&
             (!gw || (p.stride_o * osz) % 16 == 0);
  // Widest column tile: twice the rows an expert has on average, as tiles of
  // 256 columns cost shared memory that small groups would rather have as
  // more stages of weights in flight.
  const int64_t groups = p.E < p.rows ? p.E : (p.rows > 0 ? p.rows : 1);
  const int64_t avg2 = 2 * (((int64_t)p.rows + groups - 1) / groups);
  const int64_t width = gw ? p.K : avg2;
  a.col_cap = width <= 32 ? 32 : width <= 64 ? 64 : width <= 128 ? 128 : 256;
  a.box_rows = 32;
  a.stage_bytes = kABytes + a.col_cap * (gw && a.col_cap < 64 ? 256 : 128);
  a.tmem_cols = 2 * a.col_cap;
  const size_t table = (size_t)(p.E + 1) * sizeof(Group);
  const size_t fixed_bytes = 1024 + kEpiWarps * kEpiBytes + (2 * kMaxStages + 8) * 8 + 32 + table;
  int stages = (int)(((size_t)smem_max - fixed_bytes) / a.stage_bytes);
  if (stages > kMaxStages) stages = kMaxStages;
  if (stages < 2) {
    *unsupported = 1;
    return cudaSuccess;
  }
  a.stages = stages;
  const size_t smem = fixed_bytes + (size_t)stages * a.stage_bytes;
  if (p.kind == kGgInt8)
    a.idesc = tc::idesc_i8_s32(kChan);
  else
    a.idesc = tc::idesc_16_f32(kChan, p.dtype == MOE_T_BF16, gx || gw, gw);
  // tensor maps (dimensions in bytes along the rows)
  if (gw && p.rows == 0) {  // nothing to load, every group is empty
    std::memset(&a.tm_a, 0, sizeof(a.tm_a));
    std::memset(&a.tm_b, 0, sizeof(a.tm_b));
  } else if (gw) {
    const uint64_t da[2] = {(uint64_t)p.N * 2, (uint64_t)p.rows}, sa[1] = {(uint64_t)p.lda_bytes};
    const uint64_t db[2] = {(uint64_t)p.K * 2, (uint64_t)p.rows}, sb[1] = {(uint64_t)p.ldb_bytes};
    const uint32_t box[2] = {128, 64};
    if (!encode_tmap_u8(&a.tm_a, p.a, 2, da, sa, box, true) || !encode_tmap_u8(&a.tm_b, p.b, 2, db, sb, box, true)) {
      *unsupported = 1;
      return cudaSuccess;
    }
  } else {
    const uint64_t da[3] = {(uint64_t)p.K * elem, (uint64_t)p.N, (uint64_t)p.n_phys};
    const uint64_t sa[2] = {(uint64_t)p.lda_bytes, (uint64_t)p.stride_w_bytes};
    const uint32_t box_a[3] = {128, gx ? 64u : (uint32_t)kChan, 1};
    const uint64_t db[2] = {(uint64_t)(gx ? p.N : p.K) * elem, (uint64_t)p.rows}, sb[1] = {(uint64_t)p.ldb_bytes};
    const uint32_t box_b[2] = {128, (uint32_t)a.box_rows};
    if (!encode_tmap_u8(&a.tm_a, p.a, 3, da, sa, box_a, true) ||
        !encode_tmap_u8(&a.tm_b, p.b, 2, db, sb, box_b, true)) {
      *unsupported = 1;
      return cudaSuccess;
    }
  }
  const int64_t m_tiles = (a.channels + kChan - 1) / kChan;
  const int64_t col_tiles = gw ? (int64_t)p.E * ((p.K + a.col_cap - 1) / a.col_cap)
                               : groups + p.rows / a.col_cap;
  const int64_t max_tiles = m_tiles * col_tiles;
  if (max_tiles > (int64_t)1 << 30) {
    *unsupported = 1;
    return cudaSuccess;
  }
  const int grid = (int)(max_tiles < n_sms ? max_tiles : n_sms);
  switch (p.kind) {
    case kGgForward: return launch_kind<kGgForward>(a, grid, smem, st);
    case kGgGradX: return launch_kind<kGgGradX>(a, grid, smem, st);
    case kGgGradW: return launch_kind<kGgGradW>(a, grid, smem, st);
    default: return launch_kind<kGgInt8>(a, grid, smem, st);
  }
}

}  // namespace moe
