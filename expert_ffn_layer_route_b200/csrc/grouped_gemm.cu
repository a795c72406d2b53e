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
// at most 15 columns (31 in pairs of CTAs).
//
// Roles of a CTA: warp 0 brings the operands (TMA, a ring of stages), warp 1
// issues the MMAs, 4 warps (8 in tiles of more than 64 columns) take the sums and
// write results, and in grad_w one more clears the ragged ends of groups; two
// accumulators, so that one is read under the next one's products.
// Measured (B200, HBM copy 6.56 TB/s, cuBLAS bf16 1.61 PFLOP/s in short runs, 1.37
// at the power limit): 2048 x 28672 x 4096 bf16 314 us cold (1530 TFLOP/s); 8192
// ragged rows of 8 experts, the same matrices, 1.39-1.44 ms (1335-1385), 1.59 at
// the power limit; fp32 results 1.29-1.45 ms for even groups (of 16 bits 1.25-1.29);
// 256 rows of 128 experts, [5760][2880], 0.52 ms (6.8 TB/s); int8, 1024 rows of 384
// experts, [4096][7168], 0.98 ms (6.9 TB/s); grad_w in fp32, 8192 rows of 128
// experts, [2880][2880], 0.77-0.88 ms, added 2.2 ms.
#include <atomic>
#include <cstring>

#include "grouped_gemm.cuh"

#include "common.cuh"
#include "launch.cuh"
#include "profile.cuh"
#include "tc_ptx.cuh"
#include "tmap.cuh"

namespace moe {

namespace {

constexpr int kChan = 128;             // channels per CTA and tile: the TMEM lanes
constexpr int kLine = 128;             // bytes of the contraction per K-major block (one swizzle line)
constexpr int kSlabBytes = 64 * 128;   // channel-major block: 64 contraction rows x 64 channels of 16 bits
constexpr int kABlock = kChan * kLine;  // the channels' operand of a block, either way
// The tensor cores cut their fp32 additions short (they do not round them): left
// to one accumulator, a sum over 3500 products comes out 4e-6 off, over 28672
// 3e-5, over 400000 half a step of fp16.  So a sum is taken in pieces of 640
// products, each by its own accumulator, which the epilogue adds in registers with
// rounded fp32 additions (under 1e-6 up to some 10^5 products).  int8 sums are exact.
constexpr int kPiece = 640;  // contraction elements (a multiple of a step's, 64 or 128)
constexpr int kMaxStages = 12;
constexpr int64_t kMaxTiles = (int64_t)1 << 30;
// A warp reads the 32 TMEM lanes of its quadrant.  Tiles of more than 64 columns
// have two warps to a quadrant, which take its columns in turn: the sums of 256
// columns then fit a thread's registers, 128 of them each; and with few rows to
// a group a grad_w tile is all epilogue, most of it latencies (fp32 gradients of
// 128 experts with 64 rows each: 868 us with 4 warps, 793 with 8).
constexpr int epi_warps(int kind, bool pair) { return pair || kind == kGgGradW ? 8 : 4; }
// Warps before the epilogue's: TMA, MMA; grad_w: the clearing one and an idle one
// too, a warpgroup, which leaves the epilogue's two some of its registers.
constexpr int first_epi(int kind) { return kind == kGgGradW ? 4 : 2; }
constexpr int gg_threads(int kind, bool pair) { return 32 * (first_epi(kind) + epi_warps(kind, pair)); }
// grad_w is launched with 384 threads of 168 registers (65536 / 384, in steps of
// 8).  Its epilogue wants more, for the sums of 256 columns next to the way out of
// a tile of one piece; what does not fit would live in local memory, which has no
// cache worth the name beside this shared memory (fp32 gradients of 128 experts
// with 64 rows each: 1500 us).
constexpr int kLaunchRegs = 168, kIssueRegs = 56, kEpiRegs = 224;
static_assert(kIssueRegs + 2 * kEpiRegs == 3 * kLaunchRegs, "the warpgroups have what they were launched with");
constexpr int kSingleCols = 64;  // widest tile of one CTA (but grad_w)
enum { k16, kF32Out, kF32Add };  // result: a 16-bit type, fp32, (grad_w) fp32 added to what is there
constexpr int kBoxBig = 64, kBoxSmall = 16;  // rows of the two TMA boxes of the ragged operand

// Staging buffer of one epilogue warp: 32 rows x 32 channels (forward, grad_x,
// int8), or 32 lines of 128 bytes, their 16-byte pieces swizzled (grad_w).
constexpr int epi_bytes(int kind, bool f32) { return kind == kGgGradW || f32 ? 32 * 128 : 32 * 64; }

struct alignas(64) GgArgs {
  CUtensorMap tm_a;
  CUtensorMap tm_b;    // 64-row boxes
  CUtensorMap tm_b16;  // 16-row boxes
  const int32_t* offsets;
  const int32_t* slot_map;
  const float* x_scale;
  const float* w_scale;
  void* out;
  int64_t ldo, stride_o;
  int E, rows, n_phys;
  int channels;  // M extent: N (forward, grad_w, int8) or K (grad_x)
  int depth;     // contraction extent in elements (grad_w: the group's rows)
  int cols;      // grad_w: K
  int col_cap;   // widest column tile
  int col_step;  // column tiles start on multiples of this
  int blocks;    // 128-byte contraction blocks per stage
  int stages, b_block, stage_bytes, tmem_cols;
  uint32_t idesc;  // instruction descriptor without N
  int out_dtype;
  int vec;        // widest store the result's address and pitches allow (bytes)
  int accumulate;
};

// One group's entry in the shared-memory table.  The divisions that a tile's
// place needs are made once, when the table is built.
struct alignas(16) Group {
  int tile0;  // first tile
  int ct, w;  // column tiles, and their width
  float per_ct;  // 1 / ct
  int row0, n;
  int expert, phys;
};

struct Tile {
  int m0;            // first channel (of the pair)
  int c0, nc;        // first column (row inside the group; grad_w: k) and columns that exist
  int row0, n;       // the group's rows
  int expert, phys;
};

// A role's walk through the tiles t, t + units, ...: the group is looked for
// from the last one on.
struct Walk {
  int g = 0;
  __device__ __forceinline__ Tile at(int t, const Group* grp, int ngroups, int width_all, int tile_chan) {
    if (g + 1 < ngroups && grp[g + 1].tile0 <= t) {
      int lo = g + 1, hi = ngroups - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (grp[mid].tile0 <= t) lo = mid; else hi = mid - 1;
      }
      g = lo;
    }
    const int4 p = *reinterpret_cast<const int4*>(&grp[g]);
    const int4 r = *(reinterpret_cast<const int4*>(&grp[g]) + 1);
    const int local = t - p.x, ct = p.y;
    // column tiles of one channel tile run side by side: local = mi * ct + ci
    int mi = __float2int_rd((float)local * __int_as_float(p.w)), ci = local - mi * ct;
    if (ci < 0) {
      --mi;
      ci += ct;
    } else if (ci >= ct) {
      ++mi;
      ci -= ct;
    }
    Tile ti;
    ti.m0 = mi * tile_chan;
    ti.c0 = ci * p.z;
    ti.nc = min(p.z, (width_all ? width_all : r.y) - ti.c0);
    ti.row0 = r.x;
    ti.n = r.y;
    ti.expert = r.z;
    ti.phys = r.w;
    return ti;
  }
};

// A whole warp's wait: every lane polls, and all leave with the same answer, so
// that a wait that was given up cannot part lanes that the warp's next
// instructions (elections, tensor-memory loads) need together.
template <bool kCluster = false>
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity) {
  return __all_sync(0xffffffffu, mbar_wait<kCluster>(bar, parity));
}
__device__ __forceinline__ bool warp_any(int v) { return __any_sync(0xffffffffu, v); }

// A value that is the same in all lanes, in a register the compiler knows to
// be: what TMA and MMA instructions take their operands from.
__device__ __forceinline__ int uni(int v) { return (int)__reduce_or_sync(0xffffffffu, (unsigned)v); }

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
__device__ __forceinline__ void clear_tail(uint8_t* block, int left, int slabs, int lane) {
  const int per_slab = (16 - (left & 15)) * 8;  // 16-byte pieces
  for (int i = lane; i < slabs * per_slab; i += 32) {
    const int sl = i / per_slab, w = i - sl * per_slab;
    reinterpret_cast<uint4*>(block + sl * kSlabBytes + left * 128)[w] = make_uint4(0, 0, 0, 0);
  }
  fence_proxy_async_smem();
  __syncwarp();
}

__device__ __forceinline__ void st_global16(uint8_t* p, const uint4& v) {
  asm volatile("st.global.v4.b32 [%0], {%1,%2,%3,%4};" ::"l"(p), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// Staged lines to global memory, every lane 16 bytes of a row at a time, kBatch
// loads before their stores: kPieces 16-byte pieces a row, rows [0, n) of
// 32, all of a row's pieces wanted.  at(row, piece): the staged address.
template <int kPieces, int kBatch, typename At>
__device__ __forceinline__ void store_lines(uint8_t* out, int64_t pitch, int n, int lane, At at) {
  constexpr int kRows = 32 / kPieces;  // rows a warp stores at once
  const int piece = lane % kPieces, r0 = lane / kPieces;
  uint8_t* d = out + r0 * pitch + piece * 16;
#pragma unroll
  for (int b = 0; b < kPieces; b += kBatch) {
    uint4 t[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) t[i] = lds128(at(r0 + (b + i) * kRows, piece));
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (r0 + (b + i) * kRows < n) st_global16(d, t[i]);
      d += kRows * pitch;
    }
  }
}

__device__ __forceinline__ void lds_words(uint32_t addr, uint32_t (&v)[1]) { v[0] = lds32(addr); }
__device__ __forceinline__ void lds_words(uint32_t addr, uint32_t (&v)[2]) {
  asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(v[0]), "=r"(v[1]) : "r"(addr));
}
__device__ __forceinline__ void lds_words(uint32_t addr, uint32_t (&v)[4]) {
  const uint4 u = lds128(addr);
  v[0] = u.x;
  v[1] = u.y;
  v[2] = u.z;
  v[3] = u.w;
}

// The same for whatever does not fit that: results that lie on kVec bytes only,
// edges (bytes [0, width) of each row), and (kAdd, fp32) sums added to what is
// there.  Staged rows of kRowBytes, kPitch apart, their 16-byte pieces swizzled
// or not; a lane keeps its place in the row and steps through the rows.
template <int kVec, int kRowBytes, int kPitch, bool kSwizzled, bool kAdd, int kMost>
__device__ __forceinline__ void store_pieces(uint8_t* out, int64_t pitch, uint32_t staged, int n, int width, int lane) {
  constexpr int kBytes = kVec < 4 ? 4 : kVec, kWords = kBytes / 4;  // per lane and row
  constexpr int kPieces = kRowBytes / kBytes, kRows = 32 / kPieces;
  constexpr int kBatch = kMost < kPieces ? kMost : kPieces;  // loads before their stores
  const int r0 = lane / kPieces, b = lane % kPieces * kBytes;
  const uint32_t s = staged + r0 * kPitch + (kSwizzled ? (((b >> 4) ^ r0) << 4 | (b & 15)) : b);
  uint8_t* d = out + r0 * pitch + b;
  static_assert(!kAdd || kWords != 2, "sums are added 4 or 16 bytes at a time");
  auto put = [&](uint8_t* p, const uint32_t(&t)[kWords], const float(&old)[kWords]) {
    if constexpr (kAdd && kWords == 4)
      *reinterpret_cast<float4*>(p) = make_float4(old[0] + __uint_as_float(t[0]), old[1] + __uint_as_float(t[1]),
                                                  old[2] + __uint_as_float(t[2]), old[3] + __uint_as_float(t[3]));
    else if constexpr (kAdd)
      *reinterpret_cast<float*>(p) = old[0] + __uint_as_float(t[0]);
    else if constexpr (kWords == 4)
      st_global16(p, make_uint4(t[0], t[1], t[2], t[3]));
    else if constexpr (kWords == 2)
      *reinterpret_cast<uint2*>(p) = make_uint2(t[0], t[1]);
    else if constexpr (kVec == 4)
      *reinterpret_cast<uint32_t*>(p) = t[0];
    else {
      reinterpret_cast<uint16_t*>(p)[0] = (uint16_t)t[0];
      reinterpret_cast<uint16_t*>(p)[1] = (uint16_t)(t[0] >> 16);
    }
  };
  if (b + kBytes <= width) {
    static_assert(!kSwizzled || kBatch * kRows % 8 == 0, "the swizzle goes by a row's place in its batch");
#pragma unroll 1
    for (int i0 = 0; i0 * kRows < n; i0 += kBatch) {
      uint32_t t[kBatch][kWords];
      float old[kBatch][kWords];
      uint8_t* p[kBatch];
      const int left = n - r0 - i0 * kRows;  // rows from this lane's first on
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        lds_words((kSwizzled ? s ^ ((i * kRows & 7) << 4) : s) + (i0 + i) * kRows * kPitch, t[i]);
        p[i] = d;
        d += kRows * pitch;
        if (kAdd && i * kRows < left) {
          if constexpr (kWords == 4) {
            const float4 f = *reinterpret_cast<const float4*>(p[i]);
            old[i][0] = f.x;
            old[i][1] = f.y;
            old[i][2] = f.z;
            old[i][3] = f.w;
          } else if constexpr (kWords == 1) {
            old[i][0] = *reinterpret_cast<const float*>(p[i]);
          }
        }
      }
      if (left >= (kBatch - 1) * kRows + 1) {
#pragma unroll
        for (int i = 0; i < kBatch; ++i) put(p[i], t[i], old[i]);
      } else {
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
          if (i * kRows < left) put(p[i], t[i], old[i]);
      }
    }
  } else if (b < width) {  // the row's end inside a lane's piece
#pragma unroll 1
    for (int r = r0, i = 0; r < n; r += kRows, ++i, d += kRows * pitch) {
      uint32_t t[kWords];
      lds_words((kSwizzled ? s ^ ((i * kRows & 7) << 4) : s) + i * kRows * kPitch, t);
      if constexpr (kAdd) {
#pragma unroll
        for (int z = 0; z < kWords; ++z)
          if (b + 4 * z < width) *reinterpret_cast<float*>(d + 4 * z) += __uint_as_float(t[z]);
      } else {
#pragma unroll
        for (int z = 0; z < kBytes; z += 2)
          if (b + z < width) *reinterpret_cast<uint16_t*>(d + z) = (uint16_t)(t[z >> 2] >> (8 * (z & 2)));
      }
    }
  }
}

// rows of kRow bytes (kSwizzled: lines of 128, their 16-byte pieces swizzled), values of kElem bytes (in line: a
// call would have to save the sums that the thread still holds)
template <int kElem, int kRow, bool kSwizzled, bool kAdd, bool kVec16, int kMost>
__device__ __forceinline__ void store_any(uint8_t* out, int64_t pitch, uint32_t staged, int n, int width, int vec,
                                          int lane) {
  if constexpr (kVec16)
    store_pieces<16, kRow, kRow, kSwizzled, kAdd, kAdd ? 2 : kMost>(out, pitch, staged, n, width, lane);
  else if (!kAdd && vec == 8)
    store_pieces<8, kRow, kRow, kSwizzled, false, kMost>(out, pitch, staged, n, width, lane);
  else if (vec >= 4 || kElem == 4)
    store_pieces<4, kRow, kRow, kSwizzled, kAdd, 8>(out, pitch, staged, n, width, lane);
  else
    store_pieces<2, kRow, kRow, kSwizzled, false, 8>(out, pitch, staged, n, width, lane);
}

// grad_w's way out: 32 rows n of dw, 128 bytes of k at a time.  A thread holds
// one row's line; through shared memory the lines leave 8 lanes to a line.
struct LineOut {
  uint8_t* out;    // first row and column of the warp's part of the tile
  int64_t pitch;   // bytes
  int n, nc;       // rows; columns of the tile that exist
  uint8_t* stage;  // the warp's buffer
  int dtype, vec;
};

// 32 values to the lane's line, from its 16-byte piece `at` on.
template <bool kF32>
__device__ __forceinline__ void put_line(const LineOut& w, int at, const uint32_t (&v)[32], int lane) {
  uint4* line = reinterpret_cast<uint4*>(w.stage + lane * 128);
  if constexpr (kF32) {
#pragma unroll
    for (int z = 0; z < 8; ++z)
      line[(at + z) ^ (lane & 7)] = make_uint4(v[4 * z], v[4 * z + 1], v[4 * z + 2], v[4 * z + 3]);
  } else {
    auto put = [&](int dtype) {
      auto two = [&](int j) { return pack16(dtype, __uint_as_float(v[j]), __uint_as_float(v[j + 1])); };
#pragma unroll
      for (int z = 0; z < 4; ++z)
        line[(at + z) ^ (lane & 7)] = make_uint4(two(8 * z), two(8 * z + 2), two(8 * z + 4), two(8 * z + 6));
    };
    if (w.dtype == MOE_T_BF16)
      put(MOE_T_BF16);
    else
      put(MOE_T_FP16);
  }
}

// The staged lines of column j0.
template <int kOut, bool kVec16, int kMost, typename F>
__device__ __forceinline__ void store_line(const LineOut& w, int j0, int lane, F between) {
  constexpr bool kAdd = kOut == kF32Add;
  constexpr int osz = kOut == k16 ? 2 : 4;
  const uint32_t staged = smem_u32(w.stage);
  __syncwarp();
  const int width = min(128, (w.nc - j0) * osz);
  if (!kAdd && kVec16 && width == 128) {
    between();
    store_lines<8, kMost>(w.out + j0 * osz, w.pitch, w.n, lane,
                          [&](int r, int p) { return staged + r * 128 + ((p ^ (r & 7)) << 4); });
  } else {
    store_any<osz, 128, true, kAdd, kVec16, kMost>(w.out + j0 * osz, w.pitch, staged, w.n, width, w.vec, lane);
    __syncwarp();
    between();
  }
  __syncwarp();
}

// Zeros, for an expert without rows (out of line: there is nothing to keep in registers).
template <int kOut, bool kVec16>
__device__ __noinline__ void store_zeros(const LineOut w, int half, int lane) {
  constexpr int kPerLine = kOut == k16 ? 64 : 32;
#pragma unroll
  for (int z = 0; z < 8; ++z) reinterpret_cast<uint4*>(w.stage + lane * 128)[z ^ (lane & 7)] = make_uint4(0, 0, 0, 0);
#pragma unroll 1
  for (int j0 = half * kPerLine; j0 < w.nc; j0 += 2 * kPerLine) store_line<kOut, kVec16, 8>(w, j0, lane, [] {});
}

// What sums will be added to, on its way to L2 while the tile's products run:
// a lane's row, the warp's lines of 32 columns.
__device__ __forceinline__ void prefetch_lines(const LineOut& w, int first, int step, int lane) {
  if (lane >= w.n) return;
  for (int j0 = first; j0 < w.nc; j0 += step)
    asm volatile("prefetch.global.L2 [%0];" ::"l"(w.out + lane * w.pitch + j0 * 4));
}

// The accumulators as an epilogue warp takes them, one after the other.
template <bool kPair>
struct Accumulators {
  uint64_t *full, *empty;
  volatile int* abort;
  uint32_t lanes;  // tensor-memory address of the warp's quadrant
  int col_cap;
  int i;  // taken so far

  __device__ __forceinline__ bool take() {  // waits for the next one (false: given up)
    const bool got = !warp_any(*abort) && warp_wait(&full[i & 1], (uint32_t)(i >> 1) & 1u);
    if (!got) *abort = 1;
    tc::fence_after_sync();
    return got;
  }
  __device__ __forceinline__ uint32_t addr() const { return lanes + (uint32_t)((i & 1) * col_cap); }
  __device__ __forceinline__ void release(int lane) {  // it has been read
    tc::fence_before_sync();
    __syncwarp();
    if (lane == 0) {
      if (kPair)
        mbar_arrive_cluster_relaxed(cluster_addr(&empty[i & 1], 0));
      else
        mbar_arrive(&empty[i & 1]);
    }
    ++i;
  }
};

// A tile's sums to registers, the pieces (kPiece products or fewer) added one
// after the other: kChunks times 32 columns, from column(c) on where that is
// below nc.  wanted: whether the warp's channels exist.  False: given up.
template <bool kInPieces, bool kPair, int kChunks, typename Column>
__device__ __forceinline__ bool take_sums(Accumulators<kPair>& acc, uint32_t (&sum)[kChunks][32], int depth, int nc,
                                          bool wanted, int lane, Column column) {
  if (!acc.take()) return false;
  if (wanted) {
    // (no branch between a load and its wait; what lies past the tile's columns is read somewhere inside)
    const int last = max(acc.col_cap - 32, 0);
#pragma unroll
    for (int c = 0; c < kChunks; ++c) tc::ld_issue32(acc.addr() + min(column(c), last), sum[c]);
#pragma unroll
    for (int c = 0; c < kChunks; ++c) tc::ld_wait32(sum[c]);
  }
  acc.release(lane);
  if constexpr (kInPieces) {
#pragma unroll 1
    for (int d0 = kPiece; d0 < depth; d0 += kPiece) {
      if (!acc.take()) return false;
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        if (!wanted || column(c) >= nc) continue;
#pragma unroll
        for (int h = 0; h < 32; h += 16) {
          uint32_t v[16];
          tc::ld_32x32b_x16(acc.addr() + column(c) + h, v);
          tc::ld_wait16(v);
#pragma unroll
          for (int j = 0; j < 16; ++j)
            sum[c][h + j] = __float_as_uint(__uint_as_float(sum[c][h + j]) + __uint_as_float(v[j]));
        }
      }
      acc.release(lane);
    }
  }
  return true;
}

// grad_w, a tile of several pieces: the accumulators taken so far, or -1 (given up).
template <bool kPair, int kOut, bool kVec16>
__device__ __forceinline__ int store_by_sums(Accumulators<kPair> acc, const LineOut w, int depth, int half, bool mine,
                                             int lane) {
  constexpr bool kF32 = kOut != k16;
  constexpr int kPerLine = kF32 ? 32 : 64, kChunks = 4, kChunkLine = kPerLine / 32;
  uint32_t sum[kChunks][32];
  if (!take_sums<true, kPair, kChunks>(acc, sum, depth, w.nc, mine, lane, [&](int c) {
        return (half + 2 * (c / kChunkLine)) * kPerLine + c % kChunkLine * 32;
      }))
    return -1;
  if (mine) {
#pragma unroll 1
    for (int l = 0, j0 = half * kPerLine; l < kChunks / kChunkLine && j0 < w.nc; ++l, j0 += 2 * kPerLine) {
#pragma unroll
      for (int c = 0; c < kChunks; ++c)  // (registers have no index: the line's chunks by comparison)
        if (c / kChunkLine == l) put_line<kF32>(w, c % kChunkLine * 4, sum[c], lane);
      store_line<kOut, kVec16, 4>(w, j0, lane, [] {});
    }
  }
  return acc.i;
}

// fp32 results take it by a call: in line its registers cost the tiles of one piece
// 7% (128 experts of 64 rows 770, 825 us; a 16-bit result leaves half the bytes).
template <bool kPair, int kOut, bool kVec16>
__device__ __noinline__ int store_by_sums_out_of_line(Accumulators<kPair> acc, const LineOut w, int depth, int half,
                                                      bool mine, int lane) {
  return store_by_sums<kPair, kOut, kVec16>(acc, w, depth, half, mine, lane);
}

}  // namespace

// kPair: two CTAs (a cluster, on neighbouring SMs) share one tile of 256
// channels: each loads its 128 channels of A and half of the columns of B, the
// even CTA issues one MMA for both, and each keeps its 128 channels of D.  Each
// operand byte then crosses L2 -> SM half as often as with tiles of one CTA.
template <int kKind, bool kPair, int kOut, bool kVec16>
__global__ void __launch_bounds__(gg_threads(kKind, kPair), 1) grouped_gemm_kernel(const __grid_constant__ GgArgs a) {
  constexpr bool kAChanMajor = kKind == kGgGradX || kKind == kGgGradW;  // A rows run along the channels
  constexpr bool kBChanMajor = kKind == kGgGradW;
  constexpr int kElem = kKind == kGgInt8 ? 1 : 2;
  constexpr int kDepthBlock = kLine / kElem;  // contraction elements per block
  constexpr int kDepthMma = 32 / kElem;
  constexpr int kColRound = kPair ? 32 : 16;
  constexpr int kEpiBytes = epi_bytes(kKind, kOut != k16), kEpiWarps = epi_warps(kKind, kPair);
  constexpr int kFirstEpi = first_epi(kKind);
  constexpr int kTileChan = kPair ? 2 * kChan : kChan;
  constexpr bool kInPieces = kKind != kGgInt8, kF32 = kOut != k16, kAdd = kOut == kF32Add;

  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = uni(tid >> 5);
  const int rank = kPair ? (int)(blockIdx.x & 1) : 0;
  const int unit = kPair ? (int)(blockIdx.x >> 1) : (int)blockIdx.x;
  const int units = kPair ? (int)(gridDim.x >> 1) : (int)gridDim.x;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + (-smem_u32(smem_raw) & 1023u);  // (an offset: the compiler goes on knowing the space)
  uint8_t* ring = smem;
  uint8_t* epi = ring + (size_t)a.stages * a.stage_bytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(epi + kEpiWarps * kEpiBytes);
  uint64_t* empty = full + kMaxStages;
  uint64_t* tail = empty + kMaxStages;  // grad_w: this CTA's half of a group's ragged last stage has landed
  uint64_t* acc_full = tail + kMaxStages;
  uint64_t* acc_empty = acc_full + 2;
  uint64_t* drain = acc_empty + 2;
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* s_abort = reinterpret_cast<volatile int*>(s_tmem + 1);
  int* s_ngroups = reinterpret_cast<int*>(s_tmem + 2);
  volatile int* s_tile = reinterpret_cast<volatile int*>(s_tmem + 3);  // grad_w: the tile that is being brought
  Group* grp = reinterpret_cast<Group*>(s_tmem + 6);  // [E + 1], the groups that have tiles

  if (tid == 0) {
    for (int i = 0; i < a.stages; ++i) {
      // (grad_w in pairs: two arrivals, as a ragged stage is handed over by each CTA's clearing warp)
      mbar_init(&full[i], kKind == kGgGradW && kPair ? 2 : 1);
      mbar_init(&empty[i], 1);
      mbar_init(&tail[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], kPair ? 2 * kEpiWarps : kEpiWarps);
    }
    mbar_init(drain, 1);
    *s_abort = 0;
    *s_tile = -1;
    fence_barrier_init();
  }
  if (warp == 1) tc::tmem_alloc_g<kPair>(s_tmem, a.tmem_cols);
  pdl_wait_and_trigger();
  // Group table.  Every thread loads the offsets of some experts (one round of
  // global latency for all of them), then warp 0 compacts and numbers them.
  for (int e = tid; e < a.E; e += gg_threads(kKind, kPair)) {
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
  if (warp == 0) {
    const int m_tiles = ceil_div(a.channels, kTileChan);
    int ng = 0, tiles = 0;
    for (int base = 0; base < a.E; base += 32) {
      const int e = base + lane;
      int row0 = 0, n = 0, p = 0, t = 0, ct = 0;
      if (e < a.E) {
        row0 = grp[e].row0;
        n = grp[e].n;
        p = grp[e].phys;
        // (grad_w: a group without rows has zeros to write, unless they would be added)
        ct = kKind != kGgGradW ? ceil_div(n, a.col_cap) : n == 0 && a.accumulate ? 0 : ceil_div(a.cols, a.col_cap);
        t = m_tiles * ct;
      }
      int64_t end = t;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int64_t o = __shfl_up_sync(0xffffffffu, end, off);
        if (lane >= off) end += o;
      }
      end += tiles;
      if (t > 0 && end > kMaxTiles) {  // more tiles than rows allow: offsets that go back and forth
        set_status(MOE_ERR_DEVICE_INDEX);
        t = 0;
      }
      const uint32_t on = __ballot_sync(0xffffffffu, t > 0);
      if (t > 0) {  // slots at or before this expert's own: already read above
        Group g;
        g.tile0 = (int)end - t;
        g.ct = ct;
        g.w = ceil_div(ceil_div(kKind == kGgGradW ? a.cols : n, ct), a.col_step) * a.col_step;  // as even as the step allows
        g.per_ct = 1.f / (float)ct;
        g.row0 = row0;
        g.n = n;
        g.expert = e;
        g.phys = p;
        grp[ng + __popc(on & ((1u << lane) - 1u))] = g;
      }
      ng += __popc(on);
      tiles = (int)__reduce_max_sync(0xffffffffu, (unsigned)(t > 0 ? (int)end : tiles));
      __syncwarp();
    }
    if (lane == 0) {
      grp[ng].tile0 = tiles;
      *s_ngroups = ng;
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  if constexpr (kPair) cluster_sync_all();  // the peer's barriers are initialised
  tc::fence_after_sync();
  const uint32_t tmem_base = uni(*s_tmem);
  const int ngroups = uni(*s_ngroups);
  const int total_tiles = uni(grp[ngroups].tile0);

  Walk walk;
  auto tile_at = [&](int t) { return walk.at(t, grp, ngroups, kKind == kGgGradW ? a.cols : 0, kTileChan); };
  auto mma_cols = [](const Tile& ti) { return (ti.nc + kColRound - 1) & ~(kColRound - 1); };
  const int step_depth = kDepthBlock * a.blocks;
  auto depth_of = [&](const Tile& ti) { return kKind == kGgGradW ? ti.n : a.depth; };
  // grad_w: whether a step ends inside a group of 16 contraction rows
  auto ragged = [&](int left) { return kKind == kGgGradW && left < kDepthBlock && (left & 15) != 0; };

  if constexpr (kKind == kGgGradW) {
    if (warp < kFirstEpi) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kIssueRegs));
  }
  if (warp == 0) {
    // ================================================================ TMA producer
    // (the whole warp runs the loops, one lane is elected to issue: see the MMA warp)
    if (a.rows > 0 && tc::elect_one()) {
      prefetch_tmap(&a.tm_a);
      prefetch_tmap(&a.tm_b);
      if (!kBChanMajor) prefetch_tmap(&a.tm_b16);
    }
    // Large groups read every operand tile several times, from pairs that run side by side (Mixtral-shaped
    // gate/up in a long loop at the power limit: 1576 us, 1532 with evict_last; dx 1715, 1690)
    const uint64_t pol = kPair ? l2_evict_last_policy() : l2_evict_normal_policy();
    uint32_t s = 0, par = 1, cnt = 0, tails = 0, tail_use = 0;
    for (int t = unit; t < total_tiles; t += units) {
      if (warp_any(*s_abort)) break;
      if (kKind == kGgGradW) *s_tile = t;
      const Tile ti = tile_at(t);
      const int depth = uni(depth_of(ti));
      const int ncols = uni(mma_cols(ti));
      const int bc = kPair ? ncols >> 1 : ncols;  // columns this CTA loads
      const int ch = uni(ti.m0) + rank * kChan;
      const int col = uni(ti.c0) + rank * bc;
      const int row0 = uni(ti.row0);
      const int phys = uni(ti.phys);
      const int b_bytes = kBChanMajor ? ceil_div(bc, 64) * kSlabBytes : bc * kLine;
      for (int d0 = 0; d0 < depth; d0 += step_depth) {
        if (!warp_wait(&empty[s], par)) {
          *s_abort = 1;
          break;
        }
        uint8_t* st = ring + s * (uint32_t)a.stage_bytes;
        const int left = depth - d0;
        const int nb = left >= step_depth ? a.blocks : ceil_div(left, kDepthBlock);
        const bool rag = ragged(left);
        if (rag) {
          tails |= 1u << s;
          tail_use ^= 1u << s;
        } else {
          tails &= ~(1u << s);
        }
        if (tc::elect_one()) {
          const uint32_t bytes = nb * (kABlock + b_bytes);
          uint64_t* bar = rag ? &tail[s] : &full[s];
          // the pair's copies are counted together on the even CTA's barrier (a ragged stage's on each CTA's own)
          if (rag) {
            mbar_arrive_expect_tx(bar, bytes);
          } else if (rank == 0) {
            mbar_arrive_expect_tx(bar, kPair ? 2 * bytes : bytes);
            if (kKind == kGgGradW && kPair) mbar_arrive(bar);
          }
          const uint32_t bar_pair = kPair ? cluster_addr(bar, rag ? rank : 0) : 0;
          auto load2 = [&](uint8_t* dst, const CUtensorMap* m, int c0, int c1) {
            if constexpr (kPair) tma_load_2d_pair(dst, m, c0, c1, bar_pair, pol);
            else tma_load_2d(dst, m, c0, c1, bar, pol);
          };
          auto load3 = [&](uint8_t* dst, const CUtensorMap* m, int c0, int c1, int c2) {
            if constexpr (kPair) tma_load_3d_pair(dst, m, c0, c1, c2, bar_pair, pol);
            else tma_load_3d(dst, m, c0, c1, c2, bar, pol);
          };
          for (int b = 0; b < nb; ++b) {
            uint8_t* sa = st + b * kABlock;
            uint8_t* sb = st + a.blocks * kABlock + b * a.b_block;
            const int d = d0 + b * kDepthBlock;
            if constexpr (kKind == kGgGradW) {
              for (int i = 0; i < 2; ++i) load2(sa + i * kSlabBytes, &a.tm_a, (ch + 64 * i) * 2, row0 + d);
              for (int i = 0; i * 64 < bc; ++i) load2(sb + i * kSlabBytes, &a.tm_b, (col + 64 * i) * 2, row0 + d);
            } else {
              if constexpr (kKind == kGgGradX) {
                for (int i = 0; i < 2; ++i) load3(sa + i * kSlabBytes, &a.tm_a, (ch + 64 * i) * 2, d, phys);
              } else {
                load3(sa, &a.tm_a, d * kElem, ch, phys);
              }
              int i = 0;
              for (; i + kBoxBig <= bc; i += kBoxBig) load2(sb + i * kLine, &a.tm_b, d * kElem, row0 + col + i);
              for (; i < bc; i += kBoxSmall) load2(sb + i * kLine, &a.tm_b16, d * kElem, row0 + col + i);
            }
          }
        }
        __syncwarp();
        ++cnt;
        if (++s == (uint32_t)a.stages) {
          s = 0;
          par ^= 1;
        }
      }
    }
    // Before the block may leave, every copy has landed and every arrival at
    // this CTA's barriers has come: the last uses of the stages are free again.
    bool fine = !warp_any(*s_abort);
    const uint32_t first = cnt > (uint32_t)a.stages ? cnt - a.stages : 0;
    for (uint32_t c = first; fine && c < cnt; ++c) fine = warp_wait(&empty[c % a.stages], (c / a.stages) & 1u);
    if (!fine) {  // given up somewhere: the copies alone
      for (uint32_t c = first; rank == 0 && c < cnt; ++c)
        if (!mbar_wait(&full[c % a.stages], (c / a.stages) & 1u)) break;
      for (int i = 0; i < a.stages; ++i)
        if ((tails >> i & 1u) && !mbar_wait(&tail[i], (tail_use >> i & 1u) ^ 1u)) break;
    }
  } else if (warp == 1) {
    // ================================================================ MMA issuer
    // (of the even CTA)
    uint32_t s = 0, par = 0;
    int i = 0;
    const uint32_t sa0 = smem_u32(ring), sb0 = sa0 + a.blocks * kABlock;
    const uint64_t a_desc0 = kAChanMajor ? tc::mnmajor_sw128_desc(sa0, kSlabBytes) : tc::kmajor_sw128_desc(sa0);
    const uint64_t b_desc0 = kBChanMajor ? tc::mnmajor_sw128_desc(sb0, kSlabBytes) : tc::kmajor_sw128_desc(sb0);
    for (int t = unit; t < total_tiles && rank == 0; t += units, ++i) {
      const Tile ti = tile_at(t);
      const int depth = uni(depth_of(ti));
      const int ncols = uni(mma_cols(ti));
      const uint32_t idesc = a.idesc | ((uint32_t)(ncols >> 3) << 17);
      uint32_t d_tmem = 0;
      int d0 = 0, in_piece = 0;  // (in_piece: what the accumulator holds already)
      do {
        if ((kInPieces ? in_piece : d0) == 0) {  // the next accumulator
          if (warp_any(*s_abort) || !warp_wait<kPair>(&acc_empty[i & 1], ((uint32_t)(i >> 1) & 1u) ^ 1u)) {
            *s_abort = 1;
            break;
          }
          tc::fence_after_sync();
          d_tmem = tmem_base + (uint32_t)((i & 1) * a.col_cap);
        }
        const int left = depth - d0;
        if (left <= 0) break;  // an empty group
        if (!warp_wait<kPair>(&full[s], par)) {
          *s_abort = 1;
          break;
        }
        tc::fence_after_sync();
        // Descriptors count in 16 bytes: the next MMA's operands lie 32 bytes (K-major) or 16 lines
        // (channel-major) on, the next block's kABlock and b_block.  The whole warp runs this loop and
        // one lane is elected at the instructions: with values the compiler knows to be the same in all
        // lanes it keeps them in uniform registers, where the MMA wants them.
        constexpr int kStepA = kAChanMajor ? 128 : 2, kStepB = kBChanMajor ? 128 : 2;
        uint64_t da = a_desc0 + (uint64_t)(s * (uint32_t)(a.stage_bytes >> 4));
        uint64_t db = b_desc0 + (uint64_t)(s * (uint32_t)(a.stage_bytes >> 4));
        uint32_t more = (kInPieces ? in_piece : d0) != 0;
        for (int l = left; l > 0 && l > left - step_depth; l -= kDepthBlock) {
          if (l >= kDepthBlock) {
            if (tc::elect_one()) {
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                tc::mma_g<kPair, kKind == kGgInt8>(d_tmem, da + kk * kStepA, db + kk * kStepB, idesc,
                                                   kk == 0 ? more : 1u);
            }
          } else if (tc::elect_one()) {
            for (int kk = 0; kk * kDepthMma < l; ++kk)
              tc::mma_g<kPair, kKind == kGgInt8>(d_tmem, da + kk * kStepA, db + kk * kStepB, idesc,
                                                 kk == 0 ? more : 1u);
          }
          more = 1;
          da += kABlock >> 4;
          db += (uint32_t)a.b_block >> 4;
        }
        if (tc::elect_one()) tc::commit_g<kPair>(&empty[s]);  // frees the stage once these MMAs have read it
        __syncwarp();
        if (++s == (uint32_t)a.stages) {
          s = 0;
          par ^= 1;
        }
        d0 += step_depth;
        if constexpr (kInPieces) {
          in_piece += step_depth;
          if (in_piece >= kPiece && d0 < depth) {  // a piece of the sum is complete
            if (tc::elect_one()) tc::commit_g<kPair>(&acc_full[i & 1]);
            ++i;
            in_piece = 0;
          }
        }
      } while (d0 < depth);
      if (warp_any(*s_abort)) break;
      if (tc::elect_one()) tc::commit_g<kPair>(&acc_full[i & 1]);  // (an empty group: at once)
      __syncwarp();
    }
    if (rank == 0) {  // every MMA has completed before TMEM is freed
      if (tc::elect_one()) tc::commit_own<kPair>(drain);
      mbar_wait(drain, 0);
    }
    __syncwarp();
  } else if (warp >= kFirstEpi) {
    if constexpr (kKind == kGgGradW) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kEpiRegs));
    // ================================================================ epilogue
    const int q = warp & 3;                    // TMEM lane quadrant of this warp
    const int half = (warp - kFirstEpi) >> 2;  // of two warps to a quadrant: which
    uint8_t* stage_o = epi + (warp - kFirstEpi) * kEpiBytes;
    const uint32_t staged = smem_u32(stage_o);
    constexpr int osz = kF32 ? 4 : 2;
    Accumulators<kPair> acc{acc_full, acc_empty, s_abort, tmem_base + ((uint32_t)(q * 32) << 16), a.col_cap, 0};
    for (int t = unit; t < total_tiles; t += units) {
      const Tile ti = tile_at(t);
      const int ch0 = ti.m0 + rank * kChan + q * 32;
      const bool mine = ch0 < a.channels;
      if constexpr (kKind == kGgGradW) {
        LineOut w;
        w.out = static_cast<uint8_t*>(a.out) +
                ((int64_t)ti.expert * a.stride_o + (int64_t)ch0 * a.ldo + ti.c0) * osz;
        w.pitch = a.ldo * osz;
        w.n = min(32, a.channels - ch0);
        w.nc = ti.nc;
        w.stage = stage_o;
        w.dtype = a.out_dtype;
        w.vec = a.vec;
        // 128-byte lines, which the two warps of a quadrant take in turn
        constexpr int kPerLine = kF32 ? 32 : 64;
        if (kAdd && mine) prefetch_lines(w, half * kPerLine, 2 * kPerLine, lane);
        if (!kAdd && ti.n == 0) {  // (with sums to add there is no such tile)
          if (!acc.take()) break;
          acc.release(lane);
          if (mine) store_zeros<kOut, kVec16>(w, half, lane);
          continue;
        }
        if (ti.n <= kPiece) {
          // One piece: straight from the accumulator, the next line's values on their way while one leaves.  With few
          // rows to a group the epilogue is all there is.
          if (!acc.take()) break;
          if (mine) {
            const int first = half * kPerLine;
            uint32_t v[32];
            if (first < ti.nc) tc::ld_issue32(acc.addr() + first, v);
#pragma unroll 1
            for (int j0 = first; j0 < ti.nc; j0 += 2 * kPerLine) {
              tc::ld_wait32(v);
              put_line<kF32>(w, 0, v, lane);
              if constexpr (!kF32) {
                tc::ld_issue32(acc.addr() + j0 + 32, v);
                tc::ld_wait32(v);
                put_line<kF32>(w, 4, v, lane);
              }
              // (8 loads at a time where the registers allow it)
              store_line<kOut, kVec16, kOut == kF32Out && kVec16 ? 4 : 8>(w, j0, lane, [&] {
                if (j0 + 2 * kPerLine < ti.nc) tc::ld_issue32(acc.addr() + j0 + 2 * kPerLine, v);
              });
            }
          }
          acc.release(lane);
          continue;
        }
        if constexpr (kF32)
          acc.i = store_by_sums_out_of_line<kPair, kOut, kVec16>(acc, w, ti.n, half, mine, lane);
        else
          acc.i = store_by_sums<kPair, kOut, kVec16>(acc, w, ti.n, half, mine, lane);
        if (acc.i < 0) break;
      } else {
        // 32 rows x 32 channels at a time: a thread holds one channel of 32
        // rows; through shared memory a row's channels leave side by side.
        // Two warps to a quadrant take turns at 32 rows.
        constexpr int kHalves = kEpiWarps / 4, kChunks = (kPair ? 256 : kSingleCols) / 32 / kHalves;
        const int64_t row0 = (int64_t)ti.row0 + ti.c0;
        // (the scales come while the products run)
        float sw = 0.f, sx[kChunks] = {};
        if constexpr (kKind == kGgInt8) {
          if (ch0 + lane < a.channels) sw = __ldg(a.w_scale + (int64_t)ti.phys * a.channels + ch0 + lane);
#pragma unroll
          for (int c = 0; c < kChunks; ++c) {
            const int j = (half + kHalves * c) * 32 + lane;
            if (j < ti.nc) sx[c] = __ldg(a.x_scale + row0 + j);
          }
        }
        uint32_t sum[kChunks][32];
        if (!take_sums<kInPieces, kPair, kChunks>(acc, sum, a.depth, ti.nc, mine, lane,
                                                  [&](int c) { return (half + kHalves * c) * 32; }))
          break;
        if (!mine) continue;
        constexpr int kRow = 32 * osz;
        const int width = min(32, a.channels - ch0) * osz;
        const int64_t op = a.ldo * osz;
#pragma unroll 1
        for (int l = 0, j0 = half * 32; l < kChunks && j0 < ti.nc; ++l, j0 += 32 * kHalves) {
          const int n = min(32, ti.nc - j0);
#pragma unroll
          for (int c = 0; c < kChunks; ++c) {  // (registers have no index: the chunk by comparison)
            if (c != l) continue;
#pragma unroll
            for (int g = 0; g < 32; g += 8) {
              if (g >= n) break;
#pragma unroll
              for (int j = g; j < g + 8; ++j) {
                float f = __uint_as_float(sum[c][j]);
                if constexpr (kKind == kGgInt8) f = (float)(int)sum[c][j] * (__shfl_sync(0xffffffffu, sx[c], j) * sw);
                if constexpr (osz == 4)
                  *reinterpret_cast<float*>(stage_o + j * kRow + lane * 4) = f;
                else
                  *reinterpret_cast<uint16_t*>(stage_o + j * kRow + lane * 2) = (uint16_t)pack16(a.out_dtype, f, 0.f);
              }
            }
          }
          __syncwarp();
          uint8_t* o = static_cast<uint8_t*>(a.out) + ((row0 + j0) * a.ldo + ch0) * osz;
          if (kVec16 && width == kRow)
            store_lines<kRow / 16, 4>(o, op, n, lane, [&](int r, int p) { return staged + r * kRow + p * 16; });
          else
            store_any<osz, kRow, false, false, kVec16, 2>(o, op, staged, n, width, a.vec, lane);
          __syncwarp();
        }
      }
    }
  }
  if (kKind == kGgGradW && warp == 2) {
    // ================================================================ clears the ragged stages
    uint32_t cnt = 0, uses = 0;
    for (int t = unit; t < total_tiles; t += units) {
      const Tile ti = tile_at(t);
      cnt += ceil_div(ti.n, kDepthBlock);
      const int left = ti.n % kDepthBlock;
      if ((left & 15) == 0) continue;
      const uint32_t s = (cnt - 1) % a.stages;
      // (any number of tiles without a ragged stage may come before this one)
      if (warp_any(*s_abort) || !mbar_wait_moving(&tail[s], (uses >> s) & 1u, s_tile)) {
        *s_abort = 1;
        break;
      }
      uses ^= 1u << s;
      clear_tail(ring + s * (uint32_t)a.stage_bytes, left, 2 + ceil_div(kPair ? mma_cols(ti) >> 1 : mma_cols(ti), 64), lane);
      if (lane == 0) {
        if (kPair)
          mbar_arrive_cluster(cluster_addr(&full[s], 0));
        else
          mbar_arrive(&full[s]);
      }
    }
  }
  __syncwarp();
  tc::fence_before_sync();
  __syncthreads();
  if constexpr (kPair) cluster_sync_all();  // the peer's arrivals and copies need this CTA's shared memory until here
  tc::fence_after_sync();
  __syncwarp();
  if (warp == 1) tc::tmem_dealloc_g<kPair>(tmem_base, a.tmem_cols);
}

// ------------------------------------------------------------------ host side
namespace {

template <int kKind, bool kPair, int kOut, bool kVec16>
cudaError_t launch_as(const GgArgs& a, int grid, size_t smem, cudaStream_t st) {
  cudaError_t err = set_dyn_smem_once<grouped_gemm_kernel<kKind, kPair, kOut, kVec16>>(smem);
  if (err != cudaSuccess) return err;
  if (kKind == kGgGradW) {  // a warp would wait for registers for good if the compiler had given it fewer than that
    static std::atomic<bool> as_planned{false};
    if (!as_planned.load(std::memory_order_relaxed)) {
      cudaFuncAttributes at;
      err = cudaFuncGetAttributes(&at, grouped_gemm_kernel<kKind, kPair, kOut, kVec16>);
      if (err != cudaSuccess) return err;
      if (at.numRegs != kLaunchRegs) return cudaErrorLaunchOutOfResources;
      as_planned.store(true, std::memory_order_relaxed);
    }
  }
  static const char* const names[4] = {"grouped_gemm", "grouped_gemm_grad_x", "grouped_gemm_grad_w",
                                       "grouped_gemm_i8"};
  ProfScope prof(names[kKind], st);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(gg_threads(kKind, kPair));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  int n = 0;
  if (pdl_enabled()) {
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n++].val.programmaticStreamSerializationAllowed = 1;
  }
  if (kPair) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = 2;
    attr[n].val.clusterDim.y = 1;
    attr[n++].val.clusterDim.z = 1;
  }
  cfg.attrs = attr;
  cfg.numAttrs = n;
  return cudaLaunchKernelEx(&cfg, grouped_gemm_kernel<kKind, kPair, kOut, kVec16>, a);
}

template <int kKind, bool kPair, int kOut>
cudaError_t launch_vec(const GgArgs& a, int grid, size_t smem, cudaStream_t st) {
  return a.vec == 16 ? launch_as<kKind, kPair, kOut, true>(a, grid, smem, st)
                     : launch_as<kKind, kPair, kOut, false>(a, grid, smem, st);
}

template <int kKind, bool kPair>
cudaError_t launch_out(const GgArgs& a, int grid, size_t smem, cudaStream_t st) {
  if (a.out_dtype != MOE_T_FP32) return launch_vec<kKind, kPair, k16>(a, grid, smem, st);
  if constexpr (kKind == kGgGradW)
    if (a.accumulate) return launch_vec<kKind, kPair, kF32Add>(a, grid, smem, st);
  return launch_vec<kKind, kPair, kF32Out>(a, grid, smem, st);
}

template <int kKind>
cudaError_t launch_kind(const GgArgs& a, bool pair, int grid, size_t smem, cudaStream_t st) {
  return pair ? launch_out<kKind, true>(a, grid, smem, st) : launch_out<kKind, false>(a, grid, smem, st);
}

int64_t div_up(int64_t a, int64_t b) { return (a + b - 1) / b; }

}  // namespace

cudaError_t take_grouped_gemm_status(int* status) {
  const int zero = 0;
  const cudaError_t err = cudaMemcpyFromSymbol(status, g_status, sizeof(int));
  return err != cudaSuccess || *status == 0 ? err : cudaMemcpyToSymbol(g_status, &zero, sizeof(int));
}

cudaError_t launch_grouped_gemm(const GroupedProblem& p, int n_sms, int smem_max, cudaStream_t st,
                                int* unsupported) {
  *unsupported = 0;
  GgArgs a;
  std::memset(&a, 0, sizeof(a));
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
  const uint64_t place = reinterpret_cast<uint64_t>(p.out) | (uint64_t)p.ldo * osz | (gw ? (uint64_t)p.stride_o * osz : 0);
  a.vec = place & 1 ? 1 : place & 2 ? 2 : place & 4 ? 4 : place & 8 ? 8 : 16;

  // Tiles.  cap: the widest column tile, twice the rows an expert has on
  // average, so that small groups leave the shared memory to stages of weights
  // (three times: Mixtral-shaped groups of 25 and 50 rows 3% slower, 128 experts
  // of 64 rows 4%; one and a half: 1% faster to 1% slower).  Pairs of CTAs from
  // 128 columns on: from 256 on costs groups of 64 rows 3% (354, 365 us), from 64
  // on int8 groups of 28 rows 6% (176, 186 us); two blocks a stage in tiles of
  // one CTA (one: e.g. 16 experts in use, 85.6 us, two 80.6, four 84.3).
  // A product that would leave a quarter of the SMs (or pairs) without a tile
  // takes narrower ones, its time being that of one tile: down to 128 columns,
  // or to 64 where the depth is short and the epilogue most of a tile (int8, 905
  // rows, [1216][384], with its quantisation: 14.3 us, 11.3 at 128, 10.1 at 64;
  // both gradients of 2282 rows, two experts, [20128][416]: 142 us, 127 at 128,
  // 152 at 64).  A grad_w of up to 128 channels takes tiles of one CTA, as half a
  // pair would have nothing to do (24 rows, 40 experts, [96][7168], both
  // gradients: 40, 31 us).
  const int64_t groups = p.rows <= 0 ? 1 : p.E < p.rows ? p.E : p.rows;
  const int64_t width = gw ? p.K : 2 * div_up(p.rows, groups);
  int cap = width <= 16 ? 16 : width <= 32 ? 32 : width <= 64 ? 64 : width <= 128 ? 128 : 256;
  if (gw && cap < 64) cap = 64;
  bool pair = cap >= 128 && !(gw && p.N <= kChan);
  auto col_tiles_about = [&](int c) { return gw ? p.E * div_up(p.K, c) : div_up(p.rows, c) + groups / 2; };
  const int least = gw || a.depth * elem <= 16 * kLine ? 64 : 128;
  while (cap > least && 4 * div_up(a.channels, pair ? 2 * kChan : kChan) * col_tiles_about(cap) <
                            3 * (pair ? n_sms / 2 : n_sms)) {
    cap /= 2;
    pair = pair && cap >= 128;
  }
  if (!gw && !pair && cap > kSingleCols) cap = kSingleCols;  // (as the rules above have it: a thread holds no more)
  a.col_cap = cap;
  a.col_step = gw ? 64 : pair ? 32 : 16;
  const int64_t col_tiles = gw ? p.E * div_up(p.K, cap) : groups + p.rows / cap;
  a.blocks = pair || gw ? 1 : 2;
  a.b_block = (pair ? cap / 2 : cap) * kLine;
  a.stage_bytes = a.blocks * (kABlock + a.b_block);
  a.tmem_cols = cap < 32 ? 64 : 2 * cap;  // (the epilogue reads 32 columns at a time)
  const size_t table = (size_t)(p.E + 1) * sizeof(Group);
  const size_t fixed_bytes = 1024 + epi_warps(p.kind, pair) * epi_bytes(p.kind, osz == 4) + (4 * kMaxStages + 8) * 8 + 32 + table;
  int stages = (smem_max - (int)fixed_bytes) / a.stage_bytes;
  if (stages > kMaxStages) stages = kMaxStages;
  if (stages < 2) {
    *unsupported = 1;
    return cudaSuccess;
  }
  a.stages = stages;
  const size_t smem = fixed_bytes + (size_t)stages * a.stage_bytes;
  const int m = pair ? 256 : 128;
  a.idesc = p.kind == kGgInt8 ? tc::idesc_i8_s32(m) : tc::idesc_16_f32(m, p.dtype == MOE_T_BF16, gx || gw, gw);

  // tensor maps (operands in bytes along the rows)
  bool ok = true;
  if (gw) {
    if (p.rows > 0) {
      const uint64_t da[2] = {(uint64_t)p.N * 2, (uint64_t)p.rows}, sa[1] = {(uint64_t)p.lda_bytes};
      const uint64_t db[2] = {(uint64_t)p.K * 2, (uint64_t)p.rows}, sb[1] = {(uint64_t)p.ldb_bytes};
      const uint32_t box[2] = {128, 64};
      ok = encode_tmap_u8(&a.tm_a, p.a, 2, da, sa, box, true) && encode_tmap_u8(&a.tm_b, p.b, 2, db, sb, box, true);
    }
  } else {
    const uint64_t da[3] = {(uint64_t)p.K * elem, (uint64_t)p.N, (uint64_t)p.n_phys};
    const uint64_t sa[2] = {(uint64_t)p.lda_bytes, (uint64_t)p.stride_w_bytes};
    const uint32_t box_a[3] = {128, gx ? 64u : (uint32_t)kChan, 1};
    const uint64_t db[2] = {(uint64_t)(gx ? p.N : p.K) * elem, (uint64_t)p.rows}, sb[1] = {(uint64_t)p.ldb_bytes};
    const uint32_t box_b[2] = {128, kBoxBig}, box_b16[2] = {128, kBoxSmall};
    ok = encode_tmap_u8(&a.tm_a, p.a, 3, da, sa, box_a, true) && encode_tmap_u8(&a.tm_b, p.b, 2, db, sb, box_b, true) &&
         encode_tmap_u8(&a.tm_b16, p.b, 2, db, sb, box_b16, true);
  }
  const int64_t max_tiles = div_up(a.channels, pair ? 2 * kChan : kChan) * col_tiles;
  if (!ok || max_tiles > kMaxTiles) {
    *unsupported = 1;
    return cudaSuccess;
  }
  const int grid = pair ? 2 * (int)(max_tiles < n_sms / 2 ? max_tiles : n_sms / 2)
                        : (int)(max_tiles < n_sms ? max_tiles : n_sms);
  switch (p.kind) {
    case kGgForward: return launch_kind<kGgForward>(a, pair, grid, smem, st);
    case kGgGradX: return launch_kind<kGgGradX>(a, pair, grid, smem, st);
    case kGgGradW: return launch_kind<kGgGradW>(a, pair, grid, smem, st);
    default: return launch_kind<kGgInt8>(a, pair, grid, smem, st);
  }
}

}  // namespace moe
