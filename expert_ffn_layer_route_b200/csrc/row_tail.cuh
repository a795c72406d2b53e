// The end of a row, value bytes [0, left) of a 16-byte piece, without a read
// behind them: a row may end where its buffer ends.  Plain C++ too, so that the
// reads can be looked over on the host.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define MOE_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define MOE_HOST_DEVICE inline
#endif

namespace moe {

// Bytes [0, left) of the 4-byte word at p (any left), zeros behind them, by
// load.u32, .u16 and .u8(address, whether to read: 0 if not), each at a multiple
// of its size if p is one of 4.  No branches: a thread's reads are on their way
// together.
template <typename Load>
MOE_HOST_DEVICE uint32_t tail_word(const uint8_t* p, int left, const Load& load) {
  const bool part = left > 0 && left < 4;
  return load.u32(p, left >= 4) | load.u16(p, part && (left & 2)) |
         load.u8(p + (left & 2), part && (left & 1)) << (8 * (left & 2));
}

}  // namespace moe
