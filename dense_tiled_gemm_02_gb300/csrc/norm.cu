// norm.cu -- a residual's addition and the root-mean-square norm of a row, out
// in its type or in 8 bits with a scale, and the gradients.
//
//   h = x + residual,  r = 1 / sqrt(mean h^2 + eps),  y = h r w
//   dx = r (w dy - h r^2 / H sum(w dy h)) + dresidual,  dw = sum over rows of dy h r
//
// Bound by HBM: each row is read once and stays in its threads' registers (the
// gradients': in shared memory).  The 8-bit form needs the largest |y| too, which
// is r max |h w|: known with the sum of squares, so that one reduction serves
// both, and r falls out of the integers y / scale = 127 h w / max |h w|.
//
// Measured (one GB300, 16384 x 4096 bf16 with a residual, us, in brackets the bytes
// at a copy's rate, which the forward pass beats because up to an L2 of what it
// writes goes to HBM after its end): 79 (80.3), to 8 bits 80 (70.3); the gradients
// 92 (80.3), from block rows 91 (70.6), of which 3 are the last sum of dweight; in
// fp32 154 (160.6), 125 (130.5), and the gradients of 8192 rows 86 (80.3).  Rows
// longer than the registers hold are read twice (2048 x 40000 bf16 149 (98), to 8
// bits 182 (86)), the gradients' past the ring, too (2048 x 20000 bf16 164 (49),
// 4096 x 16384 fp32 282 (161)).  A row's gradients held in registers between the
// passes, without the ring, 170 from block rows: a block that waits for its row's
// sum has nothing in flight.  16 x 4096 to 8 bits: 2.5 in a graph; a call's host
// side takes 5.0.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "rows.cuh"

namespace gb300 {

namespace {

constexpr int MAX_WARPS = 32;
constexpr int BACKWARD_BLOCKS = 8;  // per SM, at most
constexpr int RING_MOST = 4;        // stages of a block's ring
constexpr int RING_BYTES = 212 * 1024;  // of all blocks of an SM

// VEC weights of the rows' type or of fp32, from column i; with ANY of any
// alignment, from columns before the row's as well, and zeros outside it.
template <typename T, int VEC, bool ANY>
__device__ __forceinline__ void load_weight(const void* w, bool f32, int i, int H, float (&o)[VEC]) {
  auto load = [&](auto* p) {
    using W = std::remove_const_t<std::remove_pointer_t<decltype(p)>>;
    Vec<W, VEC> v;
    if constexpr (ANY) {
      Around<W, VEC> x;
      const Range n = elements_at<VEC, true>(i, H);
      fetch(x, p + i, n, inside<VEC>(i, 1, 0, H));
      v = shifted<true>(x, n);
    } else {
      v = load_vec<W, VEC>(p + i);
    }
#pragma unroll
    for (int j = 0; j < VEC; ++j) o[j] = widen(v.v[j]);
  };
  if (f32)
    load(static_cast<const float*>(w));
  else
    load(static_cast<const T*>(w));
}

// A row's sum of squares and (I8) largest |h w|; if KEEP with what the store needs
// of the weights: h w, or w.  SCALED (here and below): of h times `by`.
template <typename T, int VEC, bool I8, bool ANY, bool KEEP, bool SCALED>
__device__ __forceinline__ void row_sums(const NormParams& p, const Vec<T, VEC>& h, int i, float by,
                                         float& sum, uint32_t& top, float (&kept)[VEC]) {
  float w[VEC];
  if constexpr (I8 || KEEP) load_weight<T, VEC, ANY>(p.weight, p.weight_type == T_F32, i, p.H, w);
#pragma unroll
  for (int j = 0; j < VEC; ++j) {
    const float v = SCALED ? widen(h.v[j]) * by : widen(h.v[j]);
    sum = fmaf(v, v, sum);
    if constexpr (I8) top = max(top, magnitude(v * w[j]));
    if constexpr (KEEP) kept[j] = I8 ? v * w[j] : w[j];
  }
}

// What a thread's elements are loaded as.
template <typename T, int VEC, bool ANY>
using WordsOf = std::conditional_t<ANY, Around<T, VEC>, Vec<T, VEC>>;

template <typename T, int VEC>
__device__ __forceinline__ void add_residual(Vec<T, VEC>& h, const Vec<T, VEC>& r) {
  float v[VEC];
#pragma unroll
  for (int j = 0; j < VEC; ++j) v[j] = widen(h.v[j]) + widen(r.v[j]);
  h = narrowed<T, VEC>(v);
}

template <typename T, int VEC, bool ANY>
__device__ __forceinline__ void store_row(T* p, int i, int H, const Vec<T, VEC>& x) {
  if constexpr (ANY)
    store_shifted<true>(p, i, elements_at<VEC, true>(i, H), x);
  else if (i < H)
    store_vec(p, x);
}

template <typename T, int VEC, bool I8, bool ANY, bool KEEP, bool SCALED>
__device__ __forceinline__ void store_y(const NormParams& p, long long row, const Vec<T, VEC>& h,
                                        int i, float by, float r, const RowScale& q,
                                        const float (&kept)[VEC]) {
  auto value = [&](int j) { return SCALED ? widen(h.v[j]) * by : widen(h.v[j]); };
  float w[VEC];
  if (!KEEP && i < p.H) load_weight<T, VEC, ANY>(p.weight, p.weight_type == T_F32, i, p.H, w);
  if constexpr (I8) {
    float v[VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j) v[j] = KEEP ? kept[j] : value(j) * w[j];
    store_row<int8_t, VEC, ANY>(static_cast<int8_t*>(p.y) + row * p.ldy + i, i, p.H, row_integers<SCALED>(v, q));
  } else {
    float v[VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j) v[j] = value(j) * r * (KEEP ? kept[j] : w[j]);
    store_row<T, VEC, ANY>(static_cast<T*>(p.y) + row * p.ldy + i, i, p.H, narrowed<T, VEC>(v));
  }
}

// A row's blockDim.x threads hold NV vectors each, or with NV = 0 (rows too
// long for that) read them again, from h where there is a residual.  blockDim.y
// rows a block, more than one only with one warp a row.  ANY: rows of any
// alignment; a row's vectors then begin up to VEC - 1 elements before it, where
// x's words do, so that only operands aligned otherwise (the weight, 8-bit y) are
// shifted.
template <typename T, int VEC, int NV, bool I8, bool ANY>
__global__ void __launch_bounds__(1024) norm_kernel(const NormParams p) {
  __shared__ float2 part[2][MAX_WARPS];
  const int warps = blockDim.x >> 5;
  const long long row = static_cast<long long>(blockIdx.x) * blockDim.y + threadIdx.y;
  pdl_wait();
  pdl_trigger();
  if (row >= p.T) return;  // (a whole warp, which shares nothing)
  const int lead = ANY ? static_cast<int>(reinterpret_cast<uintptr_t>(static_cast<const T*>(p.x) + row * p.ldx) %
                                          (VEC * sizeof(T)) / sizeof(T))
                       : 0;
  const int step = blockDim.x * VEC, first = threadIdx.x * VEC - lead;
  const int warp_first = (threadIdx.x & ~31) * VEC - lead;  // whole warps store
  T* const hout = static_cast<T*>(p.h) + row * p.ldh;
  constexpr int N = NV > 0 ? NV : 1;
  using Words = WordsOf<T, VEC, ANY>;
  auto load = [&](const void* from, long long ld, int i, Words& v) {
    const Range n = elements_at<VEC, ANY>(i, p.H);
    const T* const at = static_cast<const T*>(from) + row * ld + i;
    if (n.to == 0) return;
    if constexpr (ANY)
      fetch(v, at, n, inside<VEC>(row * ld + i, p.T, ld, p.H));
    else
      v = load_vec<T, VEC>(at);
  };
  auto settle = [&](const Words& v, int i) {
    if constexpr (ANY)
      return shifted<true>(v, elements_at<VEC, true>(i, p.H));
    else
      return v;
  };
  // (shifted weights are fetched once, and before the barrier, where registers hold them)
  constexpr bool KEEP = ANY && NV > 0 && NV <= 2;
  Vec<T, VEC> h[N];
  float kept[N][VEC];
  float sum = 0.f;
  uint32_t top = 0u;
  if constexpr (NV > 0) {
    auto chunk = [&](int k, const Words& x, const Words& r) {
      const int i = first + k * step;
      h[k] = settle(x, i);
      if (p.residual) {
        add_residual(h[k], settle(r, i));
        store_row<T, VEC, ANY>(hout + i, i, p.H, h[k]);
      }
    };
    if constexpr (ANY && NV > 2) {  // (a vector's words take two vectors' registers)
#pragma unroll
      for (int k = 0; k < NV; ++k)
        if (warp_first + k * step < p.H) {
          Words x, r;
          load(p.x, p.ldx, first + k * step, x);
          if (p.residual) load(p.residual, p.ldr, first + k * step, r);
          chunk(k, x, r);
        }
    } else {
      Words x[NV];
#pragma unroll
      for (int k = 0; k < NV; ++k) load(p.x, p.ldx, first + k * step, x[k]);
      if (p.residual) {
        Words r[NV];
#pragma unroll
        for (int k = 0; k < NV; ++k) load(p.residual, p.ldr, first + k * step, r[k]);
#pragma unroll
        for (int k = 0; k < NV; ++k)
          if ((ANY ? warp_first : first) + k * step < p.H) chunk(k, x[k], r[k]);
      } else {
#pragma unroll
        for (int k = 0; k < NV; ++k) h[k] = settle(x[k], first + k * step);
      }
    }
  } else {
    for (int i = first, i0 = warp_first; i0 < p.H; i += step, i0 += step) {
      Words v;
      load(p.x, p.ldx, i, v);
      h[0] = settle(v, i);
      if (p.residual) {
        load(p.residual, p.ldr, i, v);
        add_residual(h[0], settle(v, i));
        store_row<T, VEC, ANY>(hout + i, i, p.H, h[0]);
      }
      if (i < p.H) row_sums<T, VEC, I8, ANY, KEEP, false>(p, h[0], i, 1.f, sum, top, kept[0]);
    }
  }
  // f(h, i, kept) for all of this thread's vectors in the row, or (whole_warps) its
  // warp's.  NV = 0: h's or x's row again (with ANY a thread reads what its warp's
  // lanes and, one word at either end, other warps stored before the barrier of
  // the sum).
  auto each = [&](bool whole_warps, auto f) {
    if constexpr (NV > 0) {
#pragma unroll
      for (int k = 0; k < NV; ++k)
        if ((whole_warps ? warp_first : first) + k * step < p.H) f(h[k], first + k * step, kept[k]);
    } else {
      for (int i = first, i0 = warp_first; (whole_warps ? i0 : i) < p.H; i += step, i0 += step) {
        Words v;
        load(p.residual ? p.h : p.x, p.residual ? p.ldh : p.ldx, i, v);
        f(settle(v, i), i, kept[0]);
      }
    }
  };
  if constexpr (NV > 0)
    each(false, [&](const Vec<T, VEC>& v, int i, float(&k)[VEC]) {
      row_sums<T, VEC, I8, ANY, KEEP, false>(p, v, i, 1.f, sum, top, k);
    });
  row_reduce<true, I8>(sum, top, warps, part[0]);
  auto finish = [&](auto scaled, float by, float r, float rstd) {  // r: of h times `by`
    const RowScale q = I8 ? row_scale(__uint_as_float(top), r) : RowScale{};
    if (threadIdx.x == 0) {
      if (p.rstd) p.rstd[row] = rstd;
      if constexpr (I8) p.scales[row] = q.scale;
    }
    each(ANY || NV == 0, [&](const Vec<T, VEC>& v, int i, const float(&k)[VEC]) {
      store_y<T, VEC, I8, ANY, KEEP, decltype(scaled)::value>(p, row, v, i, by, r, q, k);
    });
  };
  // Squares of values beyond 2^64 overflow, those below 2^-50 underflow (which
  // matters where eps is as small), and so may h w: then once more with h times
  // a power of two that brings its largest magnitude to one.  (Not fp16 by itself.)
  float by = 1.f, r = 0.f, rstd = 0.f;
  uint32_t most = 0u;
  if (!(sum < INFINITY) || (sum < 0x1p-90f && p.eps < 0x1p-100f) ||
      (I8 && (top < RowScale::LEAST || top > RowScale::MOST))) {
    each(false, [&](const Vec<T, VEC>& v, int, const float(&)[VEC]) { most = max(most, vec_top(v)); });
    float none = 0.f;
    row_reduce<false, true>(none, most, warps, part[1]);
  }
  const bool scaled = most != 0u && most < 0x7F800000u;  // (the same for all of a row's threads)
  if (scaled) {
    const uint32_t up = min(253u, max(1u, 254u - (most >> 23)));
    by = __uint_as_float(up << 23);
    sum = 0.f;
    top = 0u;
    each(false, [&](const Vec<T, VEC>& v, int i, float(&k)[VEC]) {
      row_sums<T, VEC, I8, ANY, KEEP, true>(p, v, i, by, sum, top, k);
    });
    row_reduce<true, I8>(sum, top, warps, part[0]);
    const float eps = p.eps * by * by;
    if (eps < 0x1p40f) {
      r = 1.f / sqrtf(sum / static_cast<float>(p.H) + eps);
      rstd = r * by;
    } else {  // the squares are nothing beside eps
      rstd = 1.f / sqrtf(p.eps);
      r = rstd * __uint_as_float((254u - up) << 23);
    }
  } else {
    r = rstd = 1.f / sqrtf(sum / static_cast<float>(p.H) + p.eps);
  }
  // (for rows that are read again, one loop for both: 173 us instead of 148 with two
  // for 2048 x 40000 bf16 with a residual; for those in registers, two: 54 us instead
  // of 58 with one for 16384 x 4096 bf16 to 8 bits)
  if (NV == 0 || scaled)
    finish(std::true_type{}, by, r, rstd);
  else
    finish(std::false_type{}, by, r, rstd);
}

// ---------------------------------------------------------------- backward
template <typename T, int VEC>
__device__ __forceinline__ Vec<T, VEC> dx_of(const float (&dy)[VEC], const float (&h)[VEC],
                                             const float (&w)[VEC], float r, float c,
                                             const Vec<T, VEC>& res, bool residual) {
  float v[VEC];
#pragma unroll
  for (int j = 0; j < VEC; ++j) {
    v[j] = r * (dy[j] * w[j] - h[j] * c);
    if (residual) v[j] += widen(res.v[j]);
  }
  return narrowed<T, VEC>(v);
}

// Threads of an SM that the ring kernels' registers are for: by the sums of
// dweight, and by what is shifted with ANY.
constexpr int ring_room(bool any, int nv, int sums) {
  return any ? (nv == 1 ? 640 : 512) : sums > 8 ? 512 : 1024;
}

// Bytes of a row's slot in the ring.
template <bool ANY>
__host__ __device__ constexpr uint32_t ring_slot(uint32_t bytes) {
  return ANY ? (bytes + 15u) / 16u * 16u + 16u : bytes;
}

// VEC values of h, of block rows in steps: the step is a power of two, which the
// factors r and c of a whole vector take instead, exactly.
template <typename T, int VEC>
__device__ __forceinline__ void widen_h(const Vec<T, VEC>& v, float (&h)[VEC]) {
#pragma unroll
  for (int j = 0; j < VEC; ++j) h[j] = widen(v.v[j]);
}
template <int VEC>
__device__ __forceinline__ void widen_h(const Vec<int8_t, VEC>& v, float (&h)[VEC]) {
#pragma unroll
  for (int j = 0; j < VEC; ++j) h[j] = from_byte(v, j) - BYTE_BIAS;
}

// Rows too long for the kernel below.  Blocks take rows in turn and read each
// twice; a thread's columns are the same in all of them, so that no two threads
// share a sum of dweight in the block's own row of `partial`.
template <typename T, int VEC, bool HELD, bool ANY>
__global__ void __launch_bounds__(512) norm_backward_kernel(const NormBackwardParams p) {
  using HT = std::conditional_t<HELD, int8_t, T>;
  __shared__ float2 part[2][MAX_WARPS];
  const int warps = blockDim.x >> 5;
  const int step = blockDim.x * VEC, first = threadIdx.x * VEC;
  const int warp_first = (threadIdx.x & ~31) * VEC;  // whole warps store
  const int blocks = (p.H + ROW_BLOCK - 1) / ROW_BLOCK;
  const bool w32 = p.weight_type == T_F32;
  float* const mine = p.partial + static_cast<long long>(blockIdx.x) * p.H;
  pdl_wait();
  pdl_trigger();
  if (p.dweight)
    for (int i = first; i < p.H; i += step)
      for (int j = 0; j < VEC; ++j)
        if (i + j < p.H) mine[i + j] = 0.f;
  int turn = 0;
  for (long long row = blockIdx.x; row < p.T; row += gridDim.x, turn ^= 1) {
    const float r = p.rstd[row];
    auto load = [&](auto* base, long long ld, int i) {
      using E = std::remove_const_t<std::remove_pointer_t<decltype(base)>>;
      if constexpr (ANY) {
        Around<E, VEC> v;
        const Range n = elements_at<VEC>(i, p.H);
        fetch(v, base + row * ld + i, n, inside<VEC>(row * ld + i, p.T, ld, p.H));
        return shifted<true>(v, n);
      } else {
        return load_vec<E, VEC>(base + row * ld + i);
      }
    };
    float dy[VEC], h[VEC], w[VEC], hstep = 1.f;
    auto load_row = [&](int i) {
      const auto dyv = load(static_cast<const T*>(p.dy), p.ldy, i);
      const auto hv = load(static_cast<const HT*>(p.h), p.ldh, i);
      widen_h(hv, h);
      if constexpr (HELD) hstep = block_step(p.E[row * blocks + i / ROW_BLOCK]);
#pragma unroll
      for (int j = 0; j < VEC; ++j) dy[j] = widen(dyv.v[j]);
      load_weight<T, VEC, ANY>(p.weight, w32, i, p.H, w);
    };
    float sum = 0.f;
    uint32_t top = 0u;
    for (int i = first; i < p.H; i += step) {
      load_row(i);
      const float rh = r * hstep;
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const float t = dy[j] * (h[j] * rh);
        sum = fmaf(t, w[j], sum);
        if (p.dweight && (!ANY || i + j < p.H)) mine[i + j] += t;
      }
    }
    row_reduce<true, false>(sum, top, warps, part[turn]);
    const float c = sum / static_cast<float>(p.H);
    for (int i = first, i0 = warp_first; i0 < p.H; i += step, i0 += step) {
      Vec<T, VEC> res{};
      if (i < p.H) {
        load_row(i);
        if (p.dresidual) res = load(static_cast<const T*>(p.dresidual), p.ldr, i);
      }
      store_row<T, VEC, ANY>(static_cast<T*>(p.dx) + row * p.ldx + i, i, p.H,
                             dx_of(dy, h, w, r, r * hstep * c, res, p.dresidual != nullptr));
    }
  }
}

// Rows whose dweight fits the threads' registers, on their way ahead: each block
// keeps the next rows of its turn in a ring in shared memory (bulk copies: dy, h
// and dresidual of a row are one stage), so that what is in flight does not
// depend on registers or on where a block is between its two passes over a row.
// The passes read the stage twice.  With LEAD (ANY, and 8-bit rows that are VEC
// apart, but not 16) the copies are of the aligned words around a row, less those
// that are not all the operand's, whose bytes the copying thread stores (for all
// 8-bit rows: 98 us instead of 89 for 16384 x 4096).
template <typename T, int NV, bool HELD, bool ANY, bool LEAD>
__global__ void __launch_bounds__(ring_room(ANY, NV, NV * 16 / static_cast<int>(sizeof(T))))
    norm_backward_ring_kernel(const NormBackwardParams p, const int stages) {
  constexpr int VEC = 16 / sizeof(T);
  using HT = std::conditional_t<HELD, int8_t, T>;
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ float2 part[2][MAX_WARPS];
  __shared__ uint64_t bars[RING_MOST];
  __shared__ int abort_flag;
  const int warps = blockDim.x >> 5;
  const int step = blockDim.x * VEC, first = threadIdx.x * VEC;
  const int warp_first = (threadIdx.x & ~31) * VEC;  // whole warps store
  const uint32_t dy_bytes = ring_slot<ANY>(p.H * sizeof(T)), h_bytes = ring_slot<LEAD>(p.H * sizeof(HT));
  const uint32_t stage_bytes = dy_bytes + h_bytes + (p.dresidual ? dy_bytes : 0u);
  const uint32_t bar0 = smem_u32(bars);
  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) mbar_init(bar0 + 8 * s, p.dresidual ? 3 : 2);
    abort_flag = 0;
    fence_mbar_init();
    fence_proxy_async_smem();
  }
  pdl_wait();
  pdl_trigger();
  __syncthreads();
  // bytes of a row's first word that are not its own
  auto lead = [&](const void* row) {
    return LEAD ? static_cast<int>(reinterpret_cast<uintptr_t>(row) & 15) : 0;
  };
  // lane l of the first warp copies operand l: dy, h, dresidual
  const int operands = p.dresidual ? 3 : 2;
  const uint8_t* const base =
      static_cast<const uint8_t*>(threadIdx.x == 0 ? p.dy : threadIdx.x == 1 ? p.h : p.dresidual);
  const int size = threadIdx.x == 1 ? sizeof(HT) : sizeof(T), length = p.H * size;
  const long long stride = (threadIdx.x == 0 ? p.ldy : threadIdx.x == 1 ? p.ldh : p.ldr) * size;
  const uint32_t slot = threadIdx.x == 0 ? 0u : threadIdx.x == 1 ? dy_bytes : dy_bytes + h_bytes;
  auto load_row = [&](long long row, int s) {
    if (threadIdx.x >= operands) return;
    const uint32_t bar = bar0 + 8 * s;
    uint8_t* const to = ring + s * stage_bytes + slot;
    const uint8_t* const from = base + row * stride;
    if constexpr (LEAD) {
      const int a = lead(from), end = a + length;
      // the words that are all the operand's: bytes [w0, w1) of the slot
      const int w0 = row * stride >= a ? 0 : 16;
      int w1 = (end + 15) & ~15;
      if ((p.T - 1 - row) * stride + end < w1) w1 -= 16;
      w1 = max(w0, w1);
      if (w0 > a)
        for (int i = a; i < min(w0, end); ++i) to[i] = from[i - a];
      for (int i = max(w1, a); i < end; ++i) to[i] = from[i - a];
      mbar_arrive_expect_tx(bar, w1 - w0);
      if (w1 > w0) bulk_load_1d(smem_u32(to) + w0, from - a + w0, w1 - w0, bar);
    } else {
      mbar_arrive_expect_tx(bar, length);
      bulk_load_1d(smem_u32(to), from, length, bar);
    }
  };
  const bool skip = (p.debug_flags & DBG_SKIP_FIRST_FILL) ||
                    ((p.debug_flags & DBG_SKIP_ONE_FILL) && blockIdx.x == 0);
  for (int s = skip ? 1 : 0; s < stages; ++s) {  // test hook: the wait for the first row expires
    const long long row = blockIdx.x + static_cast<long long>(s) * gridDim.x;
    if (row < p.T) load_row(row, s);
  }
  const int blocks = (p.H + ROW_BLOCK - 1) / ROW_BLOCK;
  float dw[NV][VEC] = {};
  float w[NV][VEC];
  uint32_t e_next[NV] = {};
  float r_next = 0.f;
  auto prefetch = [&](long long row) {  // what does not come by the ring
    if (row >= p.T) return;
    r_next = p.rstd[row];
    if constexpr (HELD) {
#pragma unroll
      for (int k = 0; k < NV; ++k)
        if (first + k * step < p.H) e_next[k] = p.E[row * blocks + (first + k * step) / ROW_BLOCK];
    }
  };
  prefetch(blockIdx.x);
#pragma unroll
  for (int k = 0; k < NV; ++k)
    if (first + k * step < p.H)
      load_weight<T, VEC, ANY>(p.weight, p.weight_type == T_F32, first + k * step, p.H, w[k]);
  int s = 0, turn = 0;
  uint32_t ph = 0;
  long long row = blockIdx.x;
  for (; row < p.T; row += gridDim.x, turn ^= 1) {
    const float r = r_next;
    float scale[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) scale[k] = HELD ? block_step(e_next[k]) : 1.f;
    prefetch(row + gridDim.x);
    // (a thread that gives up raises the flag before the barrier in row_reduce,
    // after which all see it)
    bounded_wait(bar0 + 8 * s, ph, &abort_flag, p.status, STATUS_TIMEOUT, p.timeout_ns);
    const uint8_t* const stage = ring + s * stage_bytes;
    const T* const dyrow = reinterpret_cast<const T*>(
        stage + lead(static_cast<const T*>(p.dy) + row * p.ldy));
    const HT* const hrow = reinterpret_cast<const HT*>(
        stage + dy_bytes + lead(static_cast<const HT*>(p.h) + row * p.ldh));
    const T* const resrow = reinterpret_cast<const T*>(
        stage + dy_bytes + h_bytes + lead(static_cast<const T*>(p.dresidual) + row * p.ldr));
    auto load = [&](auto* from, int i) {
      using E = std::remove_const_t<std::remove_pointer_t<decltype(from)>>;
      if constexpr (ANY) {
        Around<E, VEC> v;
        fetch(v, from + i, {0, VEC}, true);  // (its slot ends no earlier)
        return shifted<true>(v, elements_at<VEC>(i, p.H));
      } else {
        return load_vec<E, VEC>(from + i);
      }
    };
    float sum = 0.f;
    uint32_t top = 0u;
    // (a shifted row stays in registers for the second pass where there are enough)
    constexpr bool KEEP = ANY && NV == 1;
    Vec<HT, VEC> hv[NV];
    Vec<T, VEC> dyv[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k)
      if (first + k * step < p.H) {
        float h[VEC];
        const auto hk = load(hrow, first + k * step);
        widen_h(hk, h);
        const auto dy = load(dyrow, first + k * step);
        if constexpr (KEEP) {
          hv[k] = hk;
          dyv[k] = dy;
        }
        // (h r is about 1 whatever h is, dy h may be anything: h times its vector's r,
        // or of at most 127 steps the vector's sum)
        const float rh = HELD ? r * scale[k] : r;
        float vec = HELD ? 0.f : sum;
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          const float t = widen(dy.v[j]) * (HELD ? h[j] : h[j] * rh);
          dw[k][j] = HELD ? fmaf(t, rh, dw[k][j]) : dw[k][j] + t;
          vec = fmaf(t, w[k][j], vec);
        }
        sum = HELD ? fmaf(vec, rh, sum) : vec;
      }
    if (warps == 1) __syncwarp();
    row_reduce<true, false>(sum, top, warps, part[turn]);
    if (*const_cast<volatile int*>(&abort_flag)) break;
    // every thread is past its second pass over the previous row: its stage
    // takes the row after those under way
    if (row >= gridDim.x) {
      const long long next = row + static_cast<long long>(stages - 1) * gridDim.x;
      if (next < p.T) load_row(next, s == 0 ? stages - 1 : s - 1);
    }
    const float c = sum / static_cast<float>(p.H);
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int i = first + k * step;
      if (ANY ? warp_first + k * step < p.H : i < p.H) {
        float h[VEC], d[VEC];
        Vec<T, VEC> res{};
        if (i < p.H) {
          widen_h(KEEP ? hv[k] : load(hrow, i), h);
          const auto dy = KEEP ? dyv[k] : load(dyrow, i);
#pragma unroll
          for (int j = 0; j < VEC; ++j) d[j] = widen(dy.v[j]);
          if (p.dresidual) res = load(resrow, i);
        }
        store_row<T, VEC, ANY>(static_cast<T*>(p.dx) + row * p.ldx + i, i, p.H,
                               dx_of(d, h, w[k], r, HELD ? r * scale[k] * c : r * c, res, p.dresidual != nullptr));
      }
    }
    if (++s == stages) {
      s = 0;
      ph ^= 1u;
    }
  }
  if (p.dweight) {
    float* const mine = p.partial + static_cast<long long>(blockIdx.x) * p.H;
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
      for (int j = 0; j < VEC; ++j)
        if (first + k * step + (ANY ? j : 0) < p.H) mine[first + k * step + j] = dw[k][j];
  }
  // After a wait that ran out, at this block's row number m: copies under way land
  // before the block leaves (of rows m to m + stages - 2, at the first one more).
  if (row < p.T && threadIdx.x == 0) {
    const long long m = (row - blockIdx.x) / gridDim.x;
    for (long long n = m; n < m + stages - (m > 0); ++n)
      if (blockIdx.x + n * gridDim.x < p.T && !(skip && n == 0))
        drain_wait(bar0 + 8 * static_cast<uint32_t>(n % stages), static_cast<uint32_t>(n / stages) & 1u, 200000000ull);
  }
}

// dweight: the blocks' partial sums, 32 columns a block, added up by 32 warps
// in turn and then in warp order.  Eight loads in flight, a last batch's past the
// end of its last row again (predicated away instead, 16 of them take 5 us more for
// 1216 rows; a loop unrolled four times 1).
__global__ void __launch_bounds__(1024)
    norm_dweight_kernel(const float* partial, int rows, int H, float* dweight) {
  __shared__ float part[32][33];
  const int i = blockIdx.x * 32 + threadIdx.x;
  pdl_wait();
  pdl_trigger();
  float sum = 0.f;
  if (i < H) {
    for (int r0 = threadIdx.y; r0 < rows; r0 += 32 * 8) {
      float v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) v[u] = partial[static_cast<long long>(min(r0 + 32 * u, rows - 1)) * H + i];
#pragma unroll
      for (int u = 0; u < 8; ++u) sum += r0 + 32 * u < rows ? v[u] : 0.f;
    }
  }
  part[threadIdx.y][threadIdx.x] = sum;
  __syncthreads();
  if (threadIdx.y == 0 && i < H) {
    sum = 0.f;
#pragma unroll
    for (int y = 0; y < 32; ++y) sum += part[y][threadIdx.x];
    dweight[i] = sum;
  }
}

// ---------------------------------------------------------------- launches
int up32(long long n) { return static_cast<int>((n + 31) / 32 * 32); }

template <typename T, int VEC, bool I8, bool ANY>
cudaError_t launch_forward(const NormParams& p, int num_sms, cudaStream_t st) {
  const int n = (p.H + (ANY ? 2 : 1) * (VEC - 1)) / VEC;
  // Vectors a thread: four keep enough in flight where there are rows for all
  // SMs; few rows are spread over more threads.  With ANY, two as far as blocks
  // of 512 threads go, since four are loaded one after the other (8192 rows of
  // 5001 bf16 79 us with two, 98 with four; of 5001 fp32 224 with two in 640
  // threads, 139 with four).
  constexpr int MOST = 4;  // by the registers of 1024 threads
  const int most = p.T >= 4ll * num_sms ? MOST : p.T >= num_sms ? MOST / 2 : 1;
  int nv = 1;
  while (nv < most && n > (ANY && nv > 1 ? 512 : 32) * nv) nv *= 2;
  while (nv < MOST && n > 1024 * nv) nv *= 2;
  const bool again = n > 1024 * nv;
  const int threads = again ? 1024 : up32((n + nv - 1) / nv);
  const int rows = threads == 32 ? 4 : 1;
  const dim3 grid(static_cast<unsigned>((p.T + rows - 1) / rows)), block(threads, rows);
  if (again) return launch_pdl(norm_kernel<T, VEC, 0, I8, ANY>, grid, block, 0, st, p);
  if (nv == 4) return launch_pdl(norm_kernel<T, VEC, 4, I8, ANY>, grid, block, 0, st, p);
  if (nv == 2) return launch_pdl(norm_kernel<T, VEC, 2, I8, ANY>, grid, block, 0, st, p);
  return launch_pdl(norm_kernel<T, VEC, 1, I8, ANY>, grid, block, 0, st, p);
}

// Threads and vectors a thread of a ring block: as many vectors as its sums of
// dweight leave registers for (32 sums, 16 in fp32 whose values take twice the
// shared-memory reads), since every thread more lengthens the row's reduction
// (16384 x 4096 bf16: four vectors 90 us, two 119, one 115); 0: rows too long.
template <typename T>
int ring_threads(int H, int& nv) {
  constexpr int VEC = 16 / sizeof(T);
  const int n = (H + VEC - 1) / VEC;
  for (nv = 1; nv < 4 && n > 128 * nv;) nv *= 2;
  return n <= 512 * nv ? up32((n + nv - 1) / nv) : 0;
}

// A ring kernel's blocks an SM, by registers and shared memory, and stages a
// block; false where two stages do not fit.
bool ring_shape(int64_t stage_bytes, int threads, int room, int& blocks, int& stages) {
  for (blocks = std::min(BACKWARD_BLOCKS, room / threads); blocks > 0; --blocks) {
    stages = static_cast<int>(std::min<int64_t>(RING_MOST, RING_BYTES / blocks / stage_bytes));
    if (stages >= 2) return true;
  }
  return false;
}

// What a launch of the ring kernels needs once, for rows of H elements.
template <typename T, int NV>
cudaError_t allow_ring() {
  for (auto* const kernel :
       {norm_backward_ring_kernel<T, NV, false, false, false>, norm_backward_ring_kernel<T, NV, false, true, true>,
        norm_backward_ring_kernel<T, NV, true, false, false>, norm_backward_ring_kernel<T, NV, true, false, true>,
        norm_backward_ring_kernel<T, NV, true, true, true>}) {
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, RING_BYTES);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}
template <typename T>
cudaError_t prepare_typed(int H) {
  int nv;
  if (ring_threads<T>(H, nv) == 0) return cudaSuccess;
  return nv == 1 ? allow_ring<T, 1>() : nv == 2 ? allow_ring<T, 2>() : allow_ring<T, 4>();
}

template <typename T, bool HELD, bool ANY, bool LEAD>
cudaError_t launch_backward(const NormBackwardParams& p, int num_sms, int& blocks, cudaStream_t st) {
  constexpr int S = sizeof(T);
  int nv, per_sm, stages;
  const int threads = ring_threads<T>(p.H, nv);
  const uint32_t H = p.H;  // (four bytes of 2^30 elements and more pass an int)
  const int64_t stage_bytes =
      ring_slot<ANY>(H * S) * (p.dresidual ? 2ll : 1ll) + ring_slot<LEAD>(H * (HELD ? 1 : S));
  auto blocks_of = [&](int each) {
    return static_cast<int>(std::min<long long>(p.T, static_cast<long long>(num_sms) * each));
  };
  if (threads > 0 && ring_shape(stage_bytes, threads, ring_room(ANY, nv, nv * 16 / S), per_sm, stages)) {
    blocks = blocks_of(per_sm);
    auto* const kernel = nv == 1   ? norm_backward_ring_kernel<T, 1, HELD, ANY, LEAD>
                         : nv == 2 ? norm_backward_ring_kernel<T, 2, HELD, ANY, LEAD>
                                   : norm_backward_ring_kernel<T, 4, HELD, ANY, LEAD>;
    return launch_pdl(kernel, dim3(blocks), dim3(threads), stages * static_cast<size_t>(stage_bytes), st, p,
                      stages);
  }
  blocks = blocks_of(2);
  return launch_pdl(norm_backward_kernel<T, 16 / S, HELD, ANY>, dim3(blocks), dim3(512), 0, st, p);
}

// Whether rows (base, leading dimension in elements of `size` bytes) allow
// vectors of `bytes`.
bool rows_fit(const void* base, long long ld, int size, int bytes) {
  return reinterpret_cast<uintptr_t>(base) % bytes == 0 && ld * size % bytes == 0;
}

template <typename T>
cudaError_t forward_typed(const NormParams& p, int num_sms, cudaStream_t st) {
  constexpr int VEC = 16 / sizeof(T), S = sizeof(T);
  const bool vec = p.H % VEC == 0 && rows_fit(p.x, p.ldx, S, 16) &&
                   (!p.residual || (rows_fit(p.residual, p.ldr, S, 16) && rows_fit(p.h, p.ldh, S, 16))) &&
                   rows_fit(p.weight, 0, 1, 16) &&
                   (p.i8 ? rows_fit(p.y, p.ldy, 1, VEC) : rows_fit(p.y, p.ldy, S, 16));
  if (p.i8)
    return vec ? launch_forward<T, VEC, true, false>(p, num_sms, st)
               : launch_forward<T, VEC, true, true>(p, num_sms, st);
  return vec ? launch_forward<T, VEC, false, false>(p, num_sms, st)
             : launch_forward<T, VEC, false, true>(p, num_sms, st);
}

template <typename T, bool HELD>
cudaError_t backward_held(const NormBackwardParams& p, int num_sms, int& blocks, cudaStream_t st) {
  constexpr int VEC = 16 / sizeof(T), S = sizeof(T);
  const bool vec = p.H % VEC == 0 && rows_fit(p.dy, p.ldy, S, 16) &&
                   (HELD ? rows_fit(p.h, p.ldh, 1, VEC) : rows_fit(p.h, p.ldh, S, 16)) &&
                   (!p.dresidual || rows_fit(p.dresidual, p.ldr, S, 16)) &&
                   rows_fit(p.dx, p.ldx, S, 16) && rows_fit(p.weight, 0, 1, 16);
  if (!vec) return launch_backward<T, HELD, true, true>(p, num_sms, blocks, st);
  if constexpr (HELD)  // bulk copies are of 16 bytes
    if (p.H % 16 != 0 || !rows_fit(p.h, p.ldh, 1, 16))
      return launch_backward<T, HELD, false, true>(p, num_sms, blocks, st);
  return launch_backward<T, HELD, false, false>(p, num_sms, blocks, st);
}

template <typename T>
cudaError_t backward_typed(const NormBackwardParams& p, int num_sms, int& blocks, cudaStream_t st) {
  return p.E ? backward_held<T, true>(p, num_sms, blocks, st)
             : backward_held<T, false>(p, num_sms, blocks, st);
}

}  // namespace

cudaError_t launch_norm(const NormParams& p, int num_sms, cudaStream_t st) {
  return p.type == T_F32    ? forward_typed<float>(p, num_sms, st)
         : p.type == T_BF16 ? forward_typed<__nv_bfloat16>(p, num_sms, st)
                            : forward_typed<__half>(p, num_sms, st);
}

cudaError_t prepare_norm_backward(int H, int type) {
  return type == T_F32    ? prepare_typed<float>(H)
         : type == T_BF16 ? prepare_typed<__nv_bfloat16>(H)
                          : prepare_typed<__half>(H);
}

int norm_partial_rows(long long T, int H, int type, int num_sms) {
  int nv;
  const int threads = type == T_F32 ? ring_threads<float>(H, nv) : ring_threads<__half>(H, nv);
  const int sums = nv * (type == T_F32 ? 4 : 8);
  int blocks = 2;  // rows too long for the ring
  if (threads > 0)
    for (const bool any : {false, true})
      blocks = std::max(blocks, std::min(BACKWARD_BLOCKS, ring_room(any, nv, sums) / threads));
  return static_cast<int>(std::min<long long>(T, static_cast<long long>(num_sms) * blocks));
}

cudaError_t launch_norm_backward(const NormBackwardParams& p, int num_sms, cudaStream_t st) {
  int blocks = 0;
  const cudaError_t e = p.type == T_F32    ? backward_typed<float>(p, num_sms, blocks, st)
                        : p.type == T_BF16 ? backward_typed<__nv_bfloat16>(p, num_sms, blocks, st)
                                           : backward_typed<__half>(p, num_sms, blocks, st);
  if (e != cudaSuccess || !p.dweight) return e;
  return launch_pdl(norm_dweight_kernel, dim3((p.H + 31) / 32), dim3(32, 32), 0, st,
                    static_cast<const float*>(p.partial), blocks, p.H, p.dweight);
}

}  // namespace gb300
