// rows.cuh -- what the kernels on rows share: vectors of elements, sums over a
// row's threads, and the two 8-bit forms.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstring>
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

// ---------------------------------------------------------------- rows of any alignment
// Rows whose length or place allows no vectors: a thread's VEC elements are read
// as the aligned words around them, shifted together, and stored as aligned
// words with the neighbouring lane's bytes in front, since an access for each
// element is bound by the number of accesses (8525 x 7723 of fp16 to scaled rows
// and back 283 us, this way 113; the norm of 8192 x 5001 of bf16 150 and 80 us, its
// gradients 473 and 153).  What is left above the floor is instructions.
template <typename T, int VEC>
struct Around {
  static constexpr int S = sizeof(T), BYTES = VEC * S, WORD = BYTES < 16 ? BYTES : 16;
  static constexpr int N = BYTES / WORD, Q = WORD / 4;
  uint32_t w[(N + 1) * Q];
  uint32_t shift;
};

// Of the VEC elements from i on (with LEAD i may be negative), those of a row of
// H: [from, to), to = 0 for none.
struct Range {
  int from, to;
};
template <int VEC, bool LEAD = false>
__device__ __forceinline__ Range elements_at(int i, int H) {
  return {LEAD ? max(0, -i) : 0, max(0, min(VEC, H - i))};
}

// Whether the words around the VEC elements at `at` lie within T rows of H
// elements, ld apart.
template <int VEC>
__device__ __forceinline__ bool inside(long long at, long long T, long long ld, int H) {
  return at >= VEC && at + 2 * VEC <= (T - 1) * ld + H;
}

// Elements `n` of those from p on, of which there are some; one by one where the
// words around are not all the operand's.
template <typename T, int VEC>
__device__ __forceinline__ void fetch(Around<T, VEC>& x, const T* p, const Range& n, bool words) {
  using A = Around<T, VEC>;
  const uint32_t a = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p)) & (A::WORD - 1);
#pragma unroll
  for (int j = 0; j < (A::N + 1) * A::Q; ++j) x.w[j] = 0u;
  x.shift = words ? a : 0u;
  if (words) {
    const uint8_t* const from = reinterpret_cast<const uint8_t*>(p) - a;
#pragma unroll
    for (int k = 0; k <= A::N; ++k)
      if (k * A::WORD < static_cast<int>(a) + n.to * A::S) {
        const auto v = load_vec<uint32_t, A::Q>(reinterpret_cast<const uint32_t*>(from + k * A::WORD));
#pragma unroll
        for (int j = 0; j < A::Q; ++j) x.w[k * A::Q + j] = v.v[j];
      }
  } else {
#pragma unroll
    for (int j = 0; j < VEC; ++j)
      if (j >= n.from && j < n.to) {
        using Bits = std::conditional_t<A::S == 4, uint32_t, std::conditional_t<A::S == 2, uint16_t, uint8_t>>;
        const uint32_t bits = reinterpret_cast<const Bits*>(p)[j];
        x.w[j * A::S / 4] |= bits << (j * A::S % 4 * 8);
      }
  }
}

// What was fetched; zeros for the other elements.  OFTEN: a branch passes by the
// shift where there is none (which costs rows that nearly all have one a tenth).
template <bool OFTEN, typename T, int VEC>
__device__ __forceinline__ Vec<T, VEC> shifted(const Around<T, VEC>& x, const Range& n) {
  using A = Around<T, VEC>;
  constexpr int W = (A::N + 1) * A::Q;
  uint32_t w[W];
#pragma unroll
  for (int j = 0; j < W; ++j) w[j] = x.w[j];
  if (!OFTEN || x.shift != 0u) {
    if constexpr (A::Q >= 4) {
#pragma unroll
      for (int j = 0; j + 2 < W; ++j) w[j] = x.shift & 8u ? w[j + 2] : w[j];
    }
    if constexpr (A::Q >= 2) {
#pragma unroll
      for (int j = 0; j + 1 < W; ++j) w[j] = x.shift & 4u ? w[j + 1] : w[j];
    }
    if constexpr (A::S < 4) {
#pragma unroll
      for (int j = 0; j + 1 < W; ++j) w[j] = __funnelshift_r(w[j], w[j + 1], 8u * (x.shift & 3u));
    }
  }
  Vec<T, VEC> o;
  memcpy(&o, w, A::BYTES);
  if (n.from > 0 || n.to < VEC) {
    Vec<T, VEC> zeros;
    memset(&zeros, 0, sizeof zeros);
#pragma unroll
    for (int j = 0; j < VEC; ++j)
      if (j < n.from || j >= n.to) o.v[j] = zeros.v[j];
  }
  return o;
}

// Elements `n` of each lane's vector to p on, which is element i of a row.  All
// lanes of a warp call; each one's elements follow those of the lane before, but
// where a row begins.
template <bool OFTEN, typename T, int VEC>
__device__ __forceinline__ void store_shifted(T* p, int i, const Range& n, const Vec<T, VEC>& x) {
  using A = Around<T, VEC>;
  constexpr int N = A::N, Q = A::Q, WORD = A::WORD, S = A::S;
  const int a = static_cast<int>(reinterpret_cast<uintptr_t>(p)) & (WORD - 1);
  const int end = a + n.to * S;
  uint32_t w[(N + 1) * Q];
  memcpy(w + Q, &x, A::BYTES);
  bool takes = false, given = false;
  if (!OFTEN || !__all_sync(0xFFFFFFFFu, a == 0)) {
    const int lane = threadIdx.x & 31;
    // a lane with a whole word takes the bytes in front of its own into it
    takes = lane > 0 && i >= VEC && end >= WORD && n.to > 0;
    given = __shfl_down_sync(0xFFFFFFFFu, static_cast<int>(takes), 1) && lane < 31;
#pragma unroll
    for (int j = 0; j < Q; ++j) w[j] = __shfl_up_sync(0xFFFFFFFFu, w[N * Q + j], 1);
    if constexpr (Q >= 4) {
#pragma unroll
      for (int j = (N + 1) * Q - 1; j >= 2; --j) w[j] = a & 8 ? w[j - 2] : w[j];
    }
    if constexpr (Q >= 2) {
#pragma unroll
      for (int j = (N + 1) * Q - 1; j >= 1; --j) w[j] = a & 4 ? w[j - 1] : w[j];
    }
    if constexpr (S < 4) {
#pragma unroll
      for (int j = (N + 1) * Q - 1; j >= Q; --j) w[j] = __funnelshift_l(w[j - 1], w[j], 8u * (a & 3));
    }
  }
  const int begin = takes ? 0 : a + n.from * S;
  uint8_t* const to = reinterpret_cast<uint8_t*>(p) - a;
#pragma unroll
  for (int k = 0; k < N; ++k)
    if (k * WORD >= begin && (k + 1) * WORD <= end) {
      Vec<uint32_t, Q> v;
#pragma unroll
      for (int j = 0; j < Q; ++j) v.v[j] = w[(k + 1) * Q + j];
      store_vec(reinterpret_cast<uint32_t*>(to + k * WORD), v);
    }
  // the elements of words that are not whole
  const int head = (begin + WORD - 1) / WORD * WORD, tail = given ? end : end / WORD * WORD;
  if (n.to > 0 && (begin < head || tail < end)) {
#pragma unroll
    for (int j = 0; j < VEC; ++j)
      if (j >= n.from && j < n.to && (a + j * S < head || a + j * S >= tail)) p[j] = x.v[j];
  }
}

// The largest finite value of a type.
template <typename T>
__device__ __forceinline__ float largest() {
  if constexpr (std::is_same_v<T, __half>) return 65504.f;
  if constexpr (std::is_same_v<T, __nv_bfloat16>) return __uint_as_float(0x7F7F0000u);
  return __uint_as_float(0x7F7FFFFFu);
}

// What is beyond the finite values becomes the largest of them, NaN stays (no
// comparison with it holds).
__device__ __forceinline__ float finite(float v, float most) {
  return fabsf(v) > most ? copysignf(most, v) : v;
}

// Rounded to T, two at a time: one instruction for both, and no byte permutes to
// put them together.
template <typename T, int VEC>
__device__ __forceinline__ Vec<T, VEC> narrowed(const float (&v)[VEC]) {
  Vec<T, VEC> o;
  if constexpr (std::is_same_v<T, float>) {
#pragma unroll
    for (int j = 0; j < VEC; ++j) o.v[j] = v[j];
  } else {
#pragma unroll
    for (int j = 0; j < VEC; j += 2) {
      if constexpr (std::is_same_v<T, __half>) {
        const __half2 p = __floats2half2_rn(v[j], v[j + 1]);
        memcpy(&o.v[j], &p, 4);
      } else {
        const __nv_bfloat162 p = __floats2bfloat162_rn(v[j], v[j + 1]);
        memcpy(&o.v[j], &p, 4);
      }
    }
  }
  return o;
}

// Magnitudes are compared as integers: NaN then counts as above infinity,
// which fmaxf would let pass.
__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// (SUM) sum and (TOP) largest over the threads of a row: one warp, or `warps` of them
// with the partial results in `part`, which no later call may still be reading:
// callers take two in turn.  In a fixed order, and the same in every thread.
template <bool SUM, bool TOP>
__device__ __forceinline__ void row_reduce(float& sum, uint32_t& top, int warps, float2* part) {
  auto over_warp = [&] {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
      if constexpr (SUM) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
      if constexpr (TOP) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
    }
  };
  over_warp();
  if (warps == 1) return;
  const int lane = threadIdx.x & 31;
  if (lane == 0) part[threadIdx.x >> 5] = make_float2(sum, __uint_as_float(top));
  __syncthreads();
  const float2 x = lane < warps ? part[lane] : make_float2(0.f, 0.f);
  sum = x.x;
  top = __float_as_uint(x.y);
  over_warp();
}

// The largest magnitude of a vector, as the bits of an fp32 number.  Those of
// 16-bit types are compared two at a time before they are widened.
template <typename T, int VEC>
__device__ __forceinline__ uint32_t vec_top(const Vec<T, VEC>& x) {
  if constexpr (sizeof(T) == 2 && VEC >= 2) {
    const uint32_t* const w = reinterpret_cast<const uint32_t*>(&x);
    uint32_t top = w[0] & 0x7FFF7FFFu;
#pragma unroll
    for (int j = 1; j < VEC / 2; ++j)
      asm("max.u16x2 %0, %0, %1;" : "+r"(top) : "r"(w[j] & 0x7FFF7FFFu));
    const unsigned short one = static_cast<unsigned short>(max(top & 0xFFFFu, top >> 16));
    T t;
    memcpy(&t, &one, 2);
    return __float_as_uint(widen(t));
  } else {
    uint32_t top = 0u;
#pragma unroll
    for (int j = 0; j < VEC; ++j) top = max(top, magnitude(widen(x.v[j])));
    return top;
  }
}

// ---------------------------------------------------------------- integers
// v * inverse to the nearest integer, ties to even: the last bits of its sum with
// 1.5 * 2^23, whose unit in the last place is 1 (a conversion instruction has a
// quarter of the rate).  The last byte is the integer's.
constexpr float INTEGERS = 12582912.f;
__device__ __forceinline__ uint32_t nearest(float v, float inverse) {
  return __float_as_uint(fmaf(v, inverse, INTEGERS));
}

// The last bytes of n, or zeros.
template <int VEC>
__device__ __forceinline__ Vec<int8_t, VEC> last_bytes(const uint32_t (&n)[VEC], bool zero) {
  Vec<uint32_t, VEC / 4> w;
#pragma unroll
  for (int j = 0; j < VEC / 4; ++j) {
    const uint32_t v = __byte_perm(__byte_perm(n[4 * j], n[4 * j + 1], 0x0040),
                                   __byte_perm(n[4 * j + 2], n[4 * j + 3], 0x0040), 0x5410);
    w.v[j] = zero ? 0u : v;
  }
  Vec<int8_t, VEC> q;
  memcpy(&q, &w, VEC);
  return q;
}

// 2^23 + 128 + the integer j of a vector: its byte, sign flipped, as the last of
// that fp32 number.
template <int VEC>
__device__ __forceinline__ float from_byte(const Vec<int8_t, VEC>& v, int j) {
  const uint32_t w = reinterpret_cast<const uint32_t*>(&v)[j >> 2] ^ 0x80808080u;
  return __uint_as_float(__byte_perm(w, 0x4B000000u, 0x7440u | (j & 3)));
}
constexpr float BYTE_BIAS = 8388736.f;

// ---------------------------------------------------------------- scaled rows
// Two fp32 operations by one instruction.
__device__ __forceinline__ uint64_t pair_of(float a, float b) {
  uint64_t p;
  asm("mov.b64 %0, {%1, %2};" : "=l"(p) : "f"(a), "f"(b));
  return p;
}
__device__ __forceinline__ void parts_of(uint64_t p, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(p));
}
__device__ __forceinline__ uint64_t mul_pair(uint64_t a, uint64_t b) {
  uint64_t p;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(p) : "l"(a), "l"(b));
  return p;
}
__device__ __forceinline__ uint64_t add_pair(uint64_t a, uint64_t b) {
  uint64_t p;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(p) : "l"(a), "l"(b));
  return p;
}
__device__ __forceinline__ uint64_t fma_pair(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t p;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(p) : "l"(a), "l"(b), "l"(c));
  return p;
}

// From the largest magnitude of a row: v * pre * (inv + low) are its integers, and
// scale * integer its values times `unit`.  inv + low is 127 / top / pre to twice
// fp32's bits, so that what is in the middle of two integers (top / 2 always is)
// comes out there and goes to the even one: by the reciprocal's 24 bits alone
// every second tie went astray.  pre keeps all of them in the normal range, 1 for a
// top between LEAST and MOST.  A scale that is not finite has integers of 0.
struct RowScale {
  float scale, pre, inv, low;
  static constexpr uint32_t LEAST = (127u - 100u) << 23, MOST = (127u + 100u) << 23;  // (bits)
};
__device__ __forceinline__ RowScale row_scale(float top, float unit) {
  RowScale r;
  r.scale = top * unit / 127.f;
  r.pre = top < __uint_as_float(RowScale::LEAST)  ? 0x1p80f
          : top > __uint_as_float(RowScale::MOST) ? 0x1p-80f
                                                  : 1.f;
  const float t = top * r.pre;
  const bool some = top > 0.f && magnitude(r.scale) < 0x7F800000u;
  r.inv = some ? 127.f / t : 0.f;
  r.low = some ? fmaf(-t, r.inv, 127.f) / t : 0.f;
  return r;
}
// The integers of VEC values: the nearest to 127 v / top rounded to fp32, ties to
// even (see nearest); 0 for a scale that is not finite.  For v and top of 16-bit
// types they are the nearest to the quotient itself, which is a middle or at least
// 2^-19 of its size off one (254 v and the odd multiple of top that it is compared
// with are multiples of v's last place, above 2^-11 v).  The same in 24 bits would
// take a second look at what rounds to a middle: by pairs 49 us instead of 31.6 for
// 16384 x 4096 bf16, in which middles are common, and the norm's 89 instead of 84.6.
// PRE: pre may not be 1.
template <bool PRE, int VEC>
__device__ __forceinline__ Vec<int8_t, VEC> row_integers(const float (&v)[VEC], const RowScale& r) {
  uint32_t n[VEC];
  float a[VEC];
  const uint64_t inv = pair_of(r.inv, r.inv), low = pair_of(r.low, r.low),
                 integers = pair_of(INTEGERS, INTEGERS);
#pragma unroll
  for (int j = 0; j < VEC; ++j) a[j] = v[j];
  if (PRE && r.pre != 1.f) {  // (the same for a row's threads, and rare)
#pragma unroll
    for (int j = 0; j < VEC; ++j) a[j] *= r.pre;
  }
#pragma unroll
  for (int j = 0; j < VEC; j += 2) {
    const uint64_t p = pair_of(a[j], a[j + 1]);
    float s0, s1;
    parts_of(add_pair(fma_pair(p, inv, mul_pair(p, low)), integers), s0, s1);
    n[j] = __float_as_uint(s0);
    n[j + 1] = __float_as_uint(s1);
  }
  return last_bytes(n, !(r.inv > 0.f));
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
// The integers of a vector times step.  POWER: a power of two (or NaN), of which
// the bias is an exact multiple, so that one operation does it; where that is finite.
template <bool POWER, int VEC>
__device__ __forceinline__ void times_step(const Vec<int8_t, VEC>& q, float step, float (&o)[VEC]) {
  if (POWER && step < 0x1p100f) {
    const float bias = step * -BYTE_BIAS;
#pragma unroll
    for (int j = 0; j < VEC; ++j) o[j] = fmaf(from_byte(q, j), step, bias);
  } else {
#pragma unroll
    for (int j = 0; j < VEC; ++j) o[j] = (from_byte(q, j) - BYTE_BIAS) * step;
  }
}
template <int VEC>
__device__ __forceinline__ Vec<int8_t, VEC> block_integers(const float (&v)[VEC], float inverse) {
  uint32_t n[VEC];
#pragma unroll
  for (int j = 0; j < VEC; ++j) n[j] = nearest(v[j], inverse);
  return last_bytes(n, !(inverse > 0.f));
}

// ---------------------------------------------------------------- items of rows
constexpr int DEAL_THREADS = 128;  // of a block whose threads take items in turn

// n / d for n < 2^31, by a multiplication and a shift: the division by an invariant
// integer of Granlund and Montgomery (1994), m = floor(2^32 (2^s - d) / d) + 1 with
// 2^s >= d the least (a 64-bit division would take longer than the rest of an item).
struct Divisor {
  uint32_t d, m, s;
};
inline Divisor divisor(int d) {
  uint32_t s = 0;
  while ((1ull << s) < static_cast<uint64_t>(d)) ++s;
  return {static_cast<uint32_t>(d),
          static_cast<uint32_t>(((1ull << 32) * ((1ull << s) - d)) / d + 1), s};
}
__device__ __forceinline__ uint32_t divide(uint32_t n, const Divisor& d) {
  return (__umulhi(n, d.m) + n) >> d.s;
}

// A block's items (`lanes` of them a row): `rows` whole rows,
// or one of the `parts` of a row.
struct Deal {
  int rows;
  uint32_t chunk;  // items of a part
  Divisor parts, lanes;
};
struct Items {
  long long row;
  uint32_t at, n;  // the first item within that row; items of the block
};
__device__ __forceinline__ Items block_items(long long T, const Deal& d, uint32_t block) {
  if (d.parts.d == 1) {
    const long long row = static_cast<long long>(block) * d.rows;
    return {row, 0u, static_cast<uint32_t>(min(static_cast<long long>(d.rows), T - row)) * d.lanes.d};
  }
  const uint32_t row = divide(block, d.parts), at = (block - row * d.parts.d) * d.chunk;
  return {row, at, min(d.chunk, d.lanes.d - at)};
}

// `items` a thread, fewer where that leaves SMs without work.  (A part is a
// multiple of DEAL_THREADS.)
inline Deal deal_of(long long T, int lanes, int items, int num_sms, dim3& grid) {
  uint32_t n = items * DEAL_THREADS;
  while (n > DEAL_THREADS && T * lanes < 2ll * num_sms * n) n /= 2;
  const uint32_t parts = (lanes + n - 1) / n;
  const int rows = parts > 1 ? 1 : static_cast<int>(n / lanes);
  grid = dim3(static_cast<unsigned>(parts > 1 ? T * parts : (T + rows - 1) / rows));
  return {rows, n, divisor(static_cast<int>(parts)), divisor(lanes)};
}

}  // namespace gb300
