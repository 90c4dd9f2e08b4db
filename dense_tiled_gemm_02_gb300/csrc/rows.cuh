// rows.cuh -- what the kernels on rows share: vectors of elements, sums over a
// row's threads, and the two 8-bit forms.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <type_traits>

#include "moe.h"
#include "ptx.cuh"
#include "rows.h"
#include "tc_launch.h"

namespace gb300 {

// VEC consecutive elements, moved by one load or store of at most 16 bytes each.
template <typename T, int VEC>
struct alignas(sizeof(T) * VEC > 16 ? 16 : sizeof(T) * VEC) Vec {
  T v[VEC];
};

template <typename T, int VEC>
__device__ __forceinline__ Vec<T, VEC> load_vec(const T* p) {
  return *reinterpret_cast<const Vec<T, VEC>*>(p);
}
template <typename T, int VEC>
__device__ __forceinline__ void store_vec(T* p, const Vec<T, VEC>& x) {
  *reinterpret_cast<Vec<T, VEC>*>(p) = x;
}

// The largest finite value of a type.
template <typename T>
__device__ __forceinline__ float largest() {
  if constexpr (std::is_same_v<T, __half>) return 65504.f;
  if constexpr (std::is_same_v<T, __nv_bfloat16>) return __uint_as_float(0x7F7F0000u);
  return __uint_as_float(0x7F7FFFFFu);
}

// Rounded to T; what is beyond the finite values becomes the largest of them,
// NaN stays (no comparison with it holds).
template <typename T>
__device__ __forceinline__ void narrow_finite(float v, T& x) {
  if (fabsf(v) > largest<T>()) v = copysignf(largest<T>(), v);
  narrow(v, x);
}

// Magnitudes are compared as integers: NaN then counts as above infinity,
// which fmaxf would let pass.
__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// Sum (and largest) over the threads of a row: one warp, or `warps` of them
// with the partial results in `part`, which no later call may still be reading:
// callers take two in turn.  In a fixed order, and the same in every thread.
__device__ __forceinline__ void row_reduce(float& sum, uint32_t& top, int warps, float2* part) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) {
    sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
    top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
  }
  if (warps == 1) return;
  const int lane = threadIdx.x & 31;
  if (lane == 0) part[threadIdx.x >> 5] = make_float2(sum, __uint_as_float(top));
  __syncthreads();
  const float2 x = lane < warps ? part[lane] : make_float2(0.f, 0.f);
  sum = x.x;
  top = __float_as_uint(x.y);
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) {
    sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
    top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
  }
}

// ---------------------------------------------------------------- scaled rows
// From the largest magnitude of a row: v * pre * inv are its integers, and
// scale * integer its values times `unit`.  Where 127 / top would overflow, v
// is brought up first.  A scale that is not finite has integers of 0.
struct RowScale {
  float scale, pre, inv;
};
__device__ __forceinline__ RowScale row_scale(float top, float unit) {
  RowScale r;
  r.scale = top * unit / 127.f;
  r.pre = top < 1e-30f ? 0x1p80f : 1.f;
  r.inv = top > 0.f && magnitude(r.scale) < 0x7F800000u ? 127.f / (top * r.pre) : 0.f;
  return r;
}
// (inv 0: also what is infinite or NaN in v gives 0)
__device__ __forceinline__ int8_t row_integer(float v, const RowScale& r) {
  return static_cast<int8_t>(r.inv > 0.f ? __float2int_rn(v * r.pre * r.inv) : 0);
}

// ---------------------------------------------------------------- block rows
// The exponent's byte for a block whose largest magnitude has these bits:
// the least power of two of which 127 reach it.  127 / 64 = 1.984375, so a
// mantissa above that (0x7E0000) takes one step more than k - 6.
__device__ __forceinline__ uint32_t block_exponent(uint32_t top, uint32_t least) {
  const int k = static_cast<int>(top >> 23);
  if (k == 255) return 255u;
  const int e = k - 6 + ((top & 0x7FFFFFu) > 0x7E0000u ? 1 : 0);
  return static_cast<uint32_t>(max(e, static_cast<int>(least)));
}
// fp16's last bit is 2^-24: steps below it would not come back exactly.
template <typename T>
__device__ __forceinline__ uint32_t least_exponent() {
  return std::is_same_v<T, __half> ? 103u : 0u;
}
// 2^(e - 127) (NaN for 255) and 2^(127 - e); e is at most 249 for the latter
__device__ __forceinline__ float block_step(uint32_t e) {
  return __uint_as_float(e == 255u ? 0x7FC00000u : e == 0u ? 0x00400000u : e << 23);
}
__device__ __forceinline__ float block_inverse(uint32_t e) {
  return e == 255u ? 0.f : __uint_as_float((254u - e) << 23);
}
__device__ __forceinline__ int8_t block_integer(float v, float inverse) {
  return static_cast<int8_t>(inverse > 0.f ? __float2int_rn(v * inverse) : 0);
}

}  // namespace gb300
