// i8_rows.cu -- few rows times weights of 8-bit integers, with a scale for each
// row and each output; dense or grouped by expert.
//
//   D[r,n] = x_scales[r] w_scales[e,n] sum_k X[r,k] W_e[n,k]
//
// Bound by reading the weights once: N K bytes.  The integer matrix instruction
// (mma.sync.m16n8k32.s32.s8.s8.s32) takes the bytes as they are loaded, the
// weights as its 16-row operand and 8 rows of X as its columns, and its sums
// are exact.  Because a sum over K may take K in any order, the fragment's K
// positions are given to whatever the loads bring: thread (g, t) of a warp (g =
// lane / 4, t = lane % 4) loads the 16 bytes at 64 s + 16 t of weight rows g
// and g + 8 and of X's row g, which are two instructions' fragments.
//
// A block takes 16 outputs and 8 (16) rows; its warps share K and add their sums
// up in shared memory, as many warps as keep all SMs loading.  Past 8 rows the
// instruction's rate bounds it: 0.33 us a million weights and 16 rows.
//
// Measured (one GB300, us, the floor in brackets): 1 x 4096 x 4096 4.6 (2.5),
// 1 x 8192 x 8192 14.7 (10.0), 8 x 8192 x 8192 14.7, 16 rows 23.9; 64 rows over
// 40 of 64 experts of 4096 x 2048 55 (50.3: 6.1 TB/s of weights).  Below that a
// launch, one trip to HBM and the sum over warps bound it (1 x 1024 x 4096 2.4,
// 0.6).  An expert with most of the rows has its weights read, from L2, by every
// pass of 8: 64 rows on 2 of 64 experts 16.3 (2.6), 512 on one 70 (4.4); the host
// does not know the groups.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "i8.cuh"
#include "moe.h"
#include "ptx.cuh"
#include "rows.h"
#include "tc_launch.h"

namespace gb300 {

namespace {

constexpr int STEP = 64;  // K of a step
constexpr int SM_WARPS = 16;

__device__ __forceinline__ void mma_s8(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                       uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint4 load16(const int8_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

__device__ __forceinline__ void store_d(void* d, int type, long long i, float v) {
  if (type == T_F32)
    static_cast<float*>(d)[i] = v;
  else if (type == T_BF16)
    static_cast<__nv_bfloat16*>(d)[i] = __float2bfloat16_rn(v);
  else
    static_cast<__half*>(d)[i] = __float2half_rn(v);
}

__device__ __forceinline__ void prefetch_l2(const void* p) {
  asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
}

// Pass y of all experts' passes of `rows` rows, in their order: its expert, first
// and end row; empty past the last (every thread of the block calls it).
__device__ __forceinline__ int3 nth_pass(const int* offsets, int E, int R, uint32_t* status, int y,
                                         int rows) {
  __shared__ int sums[32];
  __shared__ int found[3];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  if (threadIdx.x == 0) found[1] = found[2] = 0;
  int before = 0;
  for (int e0 = 0; e0 < E && before <= y; e0 += blockDim.x) {
    const int e = e0 + threadIdx.x;
    int2 r = make_int2(0, 0);
    if (e < E) r = expert_rows(offsets, e, R, status);
    const int n = (r.y - r.x + rows - 1) / rows;
    int inc = n;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int u = __shfl_up_sync(0xFFFFFFFFu, inc, d);
      if (lane >= d) inc += u;
    }
    if (lane == 31) sums[warp] = inc;
    __syncthreads();
    int at = before + inc - n, all = before;
    for (int i = 0; i < warps; ++i) {
      if (i < warp) at += sums[i];
      all += sums[i];
    }
    if (y >= at && y < at + n) {
      found[0] = e;
      found[1] = r.x + (y - at) * rows;
      found[2] = min(r.y, found[1] + rows);
    }
    before = all;
    __syncthreads();
  }
  return make_int3(found[0], found[1], found[2]);
}

// 16 rows of weights against NT tiles of 8 rows of X; U steps in flight.  ALIGNED:
// rows of X and W are 16-byte multiples apart and start so.
template <int NT, bool ALIGNED>
__global__ void __launch_bounds__(32 * SM_WARPS, NT == 1 ? 2 : 1) i8_rows_kernel(const I8RowsParams p) {
  constexpr int U = 4;
  __shared__ int red[SM_WARPS][16][8 * NT + 1];
  const int warps = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int tiles = (p.N + 15) / 16;  // passes one after another, tiles fastest
  const int pass = blockIdx.x / tiles, n0 = (blockIdx.x - pass * tiles) * 16;
  if (!p.offsets && p.K <= warps * U * STEP) {
    // The weights on their way to L2 while the kernel before this one ends
    // (nothing is read before that), where a warp has a single run of them:
    // two lines of a row.  (1 x 4096 x 4096: 5.5 -> 4.9 us; with more runs it
    // is in the way, 1 x 8192 x 8192: 14.9 -> 16.8.)
    const int n = n0 + g, k = warp * U * STEP + 128 * t;
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (128 * t < U * STEP && k < p.K && n + 8 * i < p.N) prefetch_l2(p.W + (n + 8 * i) * p.ldw + k);
  }
  pdl_wait();
  pdl_trigger();
  int e = 0, rb = pass * 8 * NT, r1 = min(p.R, rb + 8 * NT);
  if (p.offsets) {
    const int3 rows = nth_pass(p.offsets, p.E, p.R, p.status, pass, 8 * NT);
    e = rows.x;
    rb = rows.y;
    r1 = rows.z;
    if (rb >= r1) return;
  }
  // this thread's first weight row, and how far on the others are; rows past
  // N read the first again and are not stored
  const int left = p.N - n0 - g;
  const int8_t* const w0 =
      p.W + (static_cast<long long>(e) * p.N + n0 + (left > 0 ? g : 0)) * p.ldw + 16 * t;
  auto rows_on = [&](int h) { return 8 * h < left ? 8 * h : 0; };
  const int steps = (p.K + STEP - 1) / STEP;
  {
    int acc[NT][4] = {};
    // the scales of the first output this thread will store, on their way
    // beside the sums (not multiplied here: that would wait for them)
    float first_x = 0.f, first_w = 0.f;
    {
      const int n = threadIdx.x % 16, m = threadIdx.x / 16;
      if (m < 8 * NT && rb + m < r1 && n0 + n < p.N) {
        first_x = p.x_scales[rb + m];
        first_w = p.w_scales[static_cast<long long>(e) * p.N + n0 + n];
      }
    }
    for (int s0 = warp * U; s0 < steps; s0 += warps * U) {
      uint4 w[2][U], x[NT][U];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int8_t* const src = w0 + rows_on(h) * p.ldw + s0 * STEP;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int k = (s0 + u) * STEP + 16 * t;
          w[h][u] = make_uint4(0u, 0u, 0u, 0u);
          if (k < p.K)
            w[h][u] = ALIGNED ? load16(src + u * STEP) : load16_at(src + u * STEP, min(16, p.K - k));
        }
      }
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const int r = rb + 8 * j + g;
        const int8_t* const src = p.X + (r < r1 ? r : rb) * p.ldx + s0 * STEP + 16 * t;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int k = (s0 + u) * STEP + 16 * t;
          uint4 v = make_uint4(0u, 0u, 0u, 0u);
          if (r < r1 && k < p.K) {
            if constexpr (ALIGNED) {
              v = ld_global_v4_pinned(src + u * STEP);
            } else {
              const int n = min(16, p.K - k);  // what follows in W meets zeros here
              v = load16_at(src + u * STEP, n);
              v = make_uint4(first_bytes(v.x, n), first_bytes(v.y, n - 4), first_bytes(v.z, n - 8),
                             first_bytes(v.w, n - 12));
            }
          }
          x[j][u] = v;
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          mma_s8(acc[j], w[0][u].x, w[1][u].x, w[0][u].y, w[1][u].y, x[j][u].x, x[j][u].y);
          mma_s8(acc[j], w[0][u].z, w[1][u].z, w[0][u].w, w[1][u].w, x[j][u].z, x[j][u].w);
        }
    }
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        red[warp][g + 8 * (q >> 1)][8 * j + 2 * t + (q & 1)] = acc[j][q];
    __syncthreads();
    for (int o = threadIdx.x; o < 16 * 8 * NT; o += blockDim.x) {
      const int n = o % 16, m = o / 16;
      if (rb + m < r1 && n0 + n < p.N) {
        int v = 0;
        for (int y = 0; y < warps; ++y) v += red[y][n][m];
        const bool first = o == threadIdx.x;
        const float sx = first ? first_x : p.x_scales[rb + m];
        const float sw = first ? first_w : p.w_scales[static_cast<long long>(e) * p.N + n0 + n];
        store_d(p.D, p.d_type, (rb + m) * p.ldd + n0 + n, static_cast<float>(v) * sx * sw);
      }
    }
  }
}

template <int NT, bool ALIGNED>
cudaError_t launch_as(const I8RowsParams& p, cudaStream_t st) {
  const int tiles = (p.N + 15) / 16;
  // passes: at most one that is not full for each expert with rows
  const int experts = p.offsets ? std::min(p.E, p.R) : 1;
  const int passes = p.offsets ? experts + p.R / (8 * NT) : (p.R + 8 * NT - 1) / (8 * NT);
  const int steps = (p.K + STEP - 1) / STEP;
  int warps = 4;
  while (warps < SM_WARPS && 2 * warps <= steps / 2 &&
         static_cast<long long>(tiles) * experts * warps < SM_WARPS * p.num_sms)
    warps *= 2;
  return launch_pdl(i8_rows_kernel<NT, ALIGNED>, dim3(static_cast<unsigned>(static_cast<long long>(tiles) * passes)), dim3(32 * warps), 0, st, p);
}

template <bool ALIGNED>
cudaError_t launch_rows(const I8RowsParams& p, cudaStream_t st) {
  const int rows = p.E > 1 ? (p.R + p.E - 1) / p.E : p.R;
  return rows <= 8 ? launch_as<1, ALIGNED>(p, st) : launch_as<2, ALIGNED>(p, st);
}

}  // namespace

cudaError_t launch_i8_rows(const I8RowsParams& p, cudaStream_t st) {
  const bool aligned = p.K % 16 == 0 && p.ldx % 16 == 0 && p.ldw % 16 == 0 &&
                       reinterpret_cast<uintptr_t>(p.X) % 16 == 0 &&
                       reinterpret_cast<uintptr_t>(p.W) % 16 == 0;
  return aligned ? launch_rows<true>(p, st) : launch_rows<false>(p, st);
}

}  // namespace gb300
