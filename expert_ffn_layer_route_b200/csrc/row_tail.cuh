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

// Bytes [0, left) of the 4-byte word at p (any left), zeros behind them; read by
// load.u32, .u16 and .u8, each at an address that is a multiple of its size if p is.
template <typename Load>
MOE_HOST_DEVICE uint32_t tail_word(const uint8_t* p, int left, const Load& load) {
  if (left >= 4) return load.u32(p);
  uint32_t v = 0;
  if (left > 0) {
    if (left & 2) v = load.u16(p);
    if (left & 1) v |= (uint32_t)load.u8(p + (left & 2)) << (8 * (left & 2));
  }
  return v;
}

}  // namespace moe
