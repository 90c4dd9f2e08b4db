// w4.cu -- rows times 4-bit weights with a scale (and zero point) per group
// of K, for the few rows of a decode step; dense or grouped by expert.
//
//   D[r,n] = sum_groups s[n,G] * ( sum_{k in G} X[r,k] (q[n,k] - z[n,G]) )
//
// Bound by reading the weights once: N K / 2 bytes.  The integers q - z are
// exact in fp16 and bf16, so the inner sum goes to the tensor core
// (mma.sync.m16n8k16, fp32 accumulators) with the weights as its 16-row
// operand and 8 tokens as its columns, and the scale is applied to the fp32
// group sum: nothing is rounded before D.  (A tcgen05 tile would have to
// stage the expanded weights in shared memory, four times their bytes, for
// at most a handful of useful columns.)
//
// Because a sum over K may take K in any order, the fragment's K positions
// are given to whatever the loads bring: thread (g, t) of a warp (g = lane /
// 4, t = lane % 4) loads WPT words, 8 K each, of weight rows g and g + 8;
// the nibbles i and i + 4 of a word are one register of the fragment (one
// AND-OR puts both into the mantissas of 128 + q, or 1024 + q in fp16, and
// one packed subtraction of 128 + z is exact), and the X fragment pairs
// the same two k by a byte permute.  A step of a warp covers 32 WPT values
// of K and never crosses a group; the block's warps take steps in turn and
// add their sums in shared memory in warp order: deterministic.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "moe.h"
#include "ptx.cuh"
#include "tc_launch.h"

namespace gb300 {

namespace {

constexpr int WARPS = 8;
constexpr int THREADS = 32 * WARPS;

template <bool BF16>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  if constexpr (BF16) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
        "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  } else {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
        "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
}

// The exponent bits that make a small integer in the low mantissa bits the
// number BASE + integer: 128 in bf16, 1024 in fp16 (both halves).
template <bool BF16>
constexpr uint32_t kBase = BF16 ? 0x43004300u : 0x64006400u;

// Nibbles i and i + 4 of w minus the zero point, as two 16-bit floats.
template <bool BF16>
__device__ __forceinline__ uint32_t expand(uint32_t w, int i, uint32_t base_plus_zero) {
  const uint32_t v = ((w >> (4 * i)) & 0x000F000Fu) | kBase<BF16>;
  if constexpr (BF16) {
    const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&v),
                                     *reinterpret_cast<const __nv_bfloat162*>(&base_plus_zero));
    return *reinterpret_cast<const uint32_t*>(&d);
  } else {
    const __half2 d = __hsub2(*reinterpret_cast<const __half2*>(&v),
                              *reinterpret_cast<const __half2*>(&base_plus_zero));
    return *reinterpret_cast<const uint32_t*>(&d);
  }
}

template <int WPT>
__device__ __forceinline__ void load_words(const uint8_t* p, bool ok, uint32_t (&w)[WPT]) {
#pragma unroll
  for (int i = 0; i < WPT; ++i) w[i] = 0u;
  if (!ok) return;
  if constexpr (WPT == 4) {
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                 : "l"(p));
  } else if constexpr (WPT == 2) {
    asm volatile("ld.global.nc.v2.u32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "l"(p));
  } else {
    asm volatile("ld.global.nc.u32 %0, [%1];" : "=r"(w[0]) : "l"(p));
  }
}

__device__ __forceinline__ float load_scale(const void* s, int type, long long i) {
  if (type == T_F32) return static_cast<const float*>(s)[i];
  if (type == T_BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(s)[i]);
  return __half2float(static_cast<const __half*>(s)[i]);
}

__device__ __forceinline__ void store_d(void* d, int type, long long i, float v) {
  if (type == T_F32)
    static_cast<float*>(d)[i] = v;
  else if (type == T_BF16)
    static_cast<__nv_bfloat16*>(d)[i] = __float2bfloat16_rn(v);
  else
    static_cast<__half*>(d)[i] = __float2half_rn(v);
}

// The y-th expert that has rows, or -1 (every thread of the block calls it).
__device__ __forceinline__ int nth_expert(const W4Params& p, int y) {
  __shared__ uint32_t words[32];
  const int nw = (p.E + 31) / 32;
  for (int e0 = threadIdx.x & ~31; e0 < 32 * nw; e0 += THREADS) {
    const int e = e0 + (threadIdx.x & 31);
    bool any = false;
    if (e < p.E) {
      const int2 r = expert_rows(p.offsets, e, p.R, p.status);
      any = r.y > r.x;
    }
    const uint32_t b = __ballot_sync(0xFFFFFFFFu, any);
    if ((threadIdx.x & 31) == 0) words[e0 / 32] = b;
  }
  __syncthreads();
  for (int i = 0; i < nw; ++i) {
    const int n = __popc(words[i]);
    if (y < n) return 32 * i + __fns(words[i], 0, y + 1);
    y -= n;
  }
  return -1;
}

// RT: 16-row weight tiles a warp holds; NT: 8-token tiles.
template <bool BF16, int WPT, int RT, int NT>
__global__ void __launch_bounds__(THREADS) w4_kernel(const W4Params p) {
  constexpr int SPAN = 32 * WPT;  // K of one step
  __shared__ float red[WARPS][16 * RT][8 * NT + 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  pdl_wait();
  pdl_trigger();
  int e = 0, r0 = 0, r1 = p.R;
  if (p.offsets) {
    e = p.E > 1 ? nth_expert(p, blockIdx.y) : 0;
    if (e < 0) return;
    const int2 r = expert_rows(p.offsets, e, p.R, p.status);
    r0 = r.x;
    r1 = r.y;
  }
  const int n0 = blockIdx.x * 16 * RT;
  const long long row_bytes = p.K / 2;
  const uint8_t* wrow[RT][2];
  long long srow[RT][2];
  bool wok[RT][2];
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int n = n0 + 16 * i + 8 * h + g;
      wok[i][h] = n < p.N;
      const long long row = static_cast<long long>(e) * p.N + (wok[i][h] ? n : 0);
      wrow[i][h] = p.W + row * row_bytes;
      srow[i][h] = row * p.groups;
    }
  const uint16_t* const X = static_cast<const uint16_t*>(p.X);
  const int steps = (p.K + SPAN - 1) / SPAN;
  for (int rb = r0; rb < r1; rb += 8 * NT) {
    float acc[RT][NT][4];
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j) acc[i][j][0] = acc[i][j][1] = acc[i][j][2] = acc[i][j][3] = 0.f;
    for (int s = warp; s < steps; s += WARPS) {
      const int k = s * SPAN + t * 8 * WPT;
      const int G = s * SPAN / p.group;
      uint32_t w[RT][2][WPT], bz[RT][2];
      float sc[RT][2];
#pragma unroll
      for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          load_words<WPT>(wrow[i][h] + k / 2, wok[i][h] && k < p.K, w[i][h]);
          sc[i][h] = load_scale(p.scales, p.scale_type, srow[i][h] + G);
          const uint32_t z = p.zeros ? p.zeros[srow[i][h] + G] : 8u;
          bz[i][h] = kBase<BF16> + z * 0x00010001u;
        }
      float part[RT][NT][4];
#pragma unroll
      for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j)
          part[i][j][0] = part[i][j][1] = part[i][j][2] = part[i][j][3] = 0.f;
#pragma unroll
      for (int c = 0; c < WPT; ++c) {
        uint4 x[NT];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          x[j] = make_uint4(0u, 0u, 0u, 0u);
          const int r = rb + 8 * j + g;
          if (r < r1 && k < p.K)
            x[j] = *reinterpret_cast<const uint4*>(X + r * p.ldx + k + 8 * c);
        }
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t a[RT][4];
#pragma unroll
          for (int i = 0; i < RT; ++i) {
            a[i][0] = expand<BF16>(w[i][0][c], 2 * half, bz[i][0]);
            a[i][1] = expand<BF16>(w[i][1][c], 2 * half, bz[i][1]);
            a[i][2] = expand<BF16>(w[i][0][c], 2 * half + 1, bz[i][0]);
            a[i][3] = expand<BF16>(w[i][1][c], 2 * half + 1, bz[i][1]);
          }
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            const uint32_t lo = half ? x[j].y : x[j].x, hi = half ? x[j].w : x[j].z;
            const uint32_t b0 = __byte_perm(lo, hi, 0x5410), b1 = __byte_perm(lo, hi, 0x7632);
#pragma unroll
            for (int i = 0; i < RT; ++i) mma16816<BF16>(part[i][j], a[i], b0, b1);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int q = 0; q < 4; ++q)
            acc[i][j][q] = fmaf(sc[i][q >> 1], part[i][j][q], acc[i][j][q]);
    }
    __syncthreads();  // the previous rows' sums have been read
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          red[warp][16 * i + g + 8 * (q >> 1)][8 * j + 2 * t + (q & 1)] = acc[i][j][q];
    __syncthreads();
    for (int o = threadIdx.x; o < 16 * RT * 8 * NT; o += THREADS) {
      const int n = o % (16 * RT), m = o / (16 * RT);
      if (rb + m < r1 && n0 + n < p.N) {
        float v = 0.f;
#pragma unroll
        for (int x = 0; x < WARPS; ++x) v += red[x][n][m];
        store_d(p.D, p.d_type, (rb + m) * p.ldd + n0 + n, v);
      }
    }
  }
}

template <bool BF16, int WPT, int RT, int NT>
cudaError_t launch_as(const W4Params& p, cudaStream_t st) {
  const dim3 grid((p.N + 16 * RT - 1) / (16 * RT), p.E > 1 ? min(p.E, p.R) : 1);
  return launch_pdl(w4_kernel<BF16, WPT, RT, NT>, grid, dim3(THREADS), 0, st, p);
}

template <bool BF16, int WPT>
cudaError_t launch_wpt(const W4Params& p, cudaStream_t st) {
  // Tokens a pass covers: as many as an expert has on average.
  const int rows = p.E > 1 ? (p.R + p.E - 1) / p.E : p.R;
  if (rows <= 8) return launch_as<BF16, WPT, 1, 1>(p, st);
  if (rows <= 16) return launch_as<BF16, WPT, 1, 2>(p, st);
  return launch_as<BF16, WPT, 1, 4>(p, st);
}

template <bool BF16>
cudaError_t launch_type(const W4Params& p, cudaStream_t st) {
  // the widest load whose step stays within a group
  if (p.group % 128 == 0) return launch_wpt<BF16, 4>(p, st);
  if (p.group % 64 == 0) return launch_wpt<BF16, 2>(p, st);
  return launch_wpt<BF16, 1>(p, st);
}

}  // namespace

cudaError_t launch_w4(const W4Params& p, int num_sms, cudaStream_t st) {
  (void)num_sms;
  return p.x_type == T_BF16 ? launch_type<true>(p, st) : launch_type<false>(p, st);
}

}  // namespace gb300
