// i8.cuh -- loads of 8-bit rows that start anywhere (i8_rows.cu, i8_tiles.cu).
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace gb300 {

// 16 bytes from any address, of which the first n (1 to 16) are the operand's:
// the aligned 16-byte units that hold these, shifted together.  (A unit that
// holds a byte of an allocation is within it.)
__device__ __forceinline__ uint4 load16_at(const int8_t* p, int n) {
  const uint32_t s = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p) & 15u);
  const uint4* const unit = reinterpret_cast<const uint4*>(p - s);
  const uint4 a = __ldg(unit);
  uint4 b = make_uint4(0u, 0u, 0u, 0u);
  if (static_cast<int>(s) + n > 16) b = __ldg(unit + 1);
  const bool by8 = s & 8u, by4 = s & 4u;
  const uint32_t w[6] = {by8 ? a.z : a.x, by8 ? a.w : a.y, by8 ? b.x : a.z,
                         by8 ? b.y : a.w, by8 ? b.z : b.x, by8 ? b.w : b.y};
  const uint32_t v[5] = {by4 ? w[1] : w[0], by4 ? w[2] : w[1], by4 ? w[3] : w[2],
                         by4 ? w[4] : w[3], by4 ? w[5] : w[4]};
  const uint32_t sh = 8u * (s & 3u);
  return make_uint4(__funnelshift_r(v[0], v[1], sh), __funnelshift_r(v[1], v[2], sh),
                    __funnelshift_r(v[2], v[3], sh), __funnelshift_r(v[3], v[4], sh));
}

// The first n of a word's bytes, zeros after them.
__device__ __forceinline__ uint32_t first_bytes(uint32_t w, int n) {
  return n >= 4 ? w : n <= 0 ? 0u : w & (0xFFFFFFFFu >> (32 - 8 * n));
}

}  // namespace gb300
