// w4.cu -- rows times 4-bit weights with a scale (and zero point) per group
// of K, for the few rows of a decode step; dense or grouped by expert.
//
//   D[r,n] = sum_groups s[n,G] * ( sum_{k in G} X[r,k] (q[n,k] - z[n,G]) )
//
// (a group's sum in steps of 128, 64 or 32 values, each scaled for itself)
//
// Bound by reading the weights once: N K / 2 bytes.  The integers q - z are
// exact in fp16 and bf16, so the inner sum goes to the tensor core
// (mma.sync.m16n8k16, fp32 accumulators) with the weights as its 16-row
// operand and 8 tokens as its columns, and the scale is applied to the fp32
// sums: nothing is rounded before D.  (A tcgen05 tile would have to
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
// of K and never crosses a group; the block's warps take runs of U steps in
// turn, X's fragments of a run staying in registers for both of a warp's
// 16-row tiles, and add their sums in shared memory in warp order:
// deterministic.
//
// Measured (one GB300): 4 x 8192 x 32768, groups of 128: 40 us (3.5 TB/s),
// 16 x 8192 x 8192, groups of 64: 21 us (45 with X loaded for every 16 rows),
// 64 rows over 40 experts of 4096 x 2048: 49 us (over 2 of 64 experts 34, on
// one 53: eight passes over its weights).  A prompt is not what this is for:
// 2048 x 4096 x 4096 takes 720 us, 64 passes.  No unit is more than half
// busy (logic 49%, L1 47%, issue 40% at the first case; the loads alone, with
// as many in flight, run at 6.2 TB/s): what bounds it is the time between a
// run's loads and its arithmetic, with 16 warps an SM to cover it (the
// next run's first tile on its way during this run's second: no gain, 39.8;
// the scales of eight steps by one load a row: 39.1, 19.9 and 50.4).  Measured
// against it on the same cases: a run's loads a run ahead in registers, by
// blocks that stay (55, 26 and 67 us: the registers of the second run cost as
// many instructions as the loads took), 24 and 32 warps an SM with half the
// loads each (50 and 56 us for the first case), four weight tiles against one
// X (48, 39 and 61), the weights expanded into tensor memory for tcgen05.mma
// (48, 29 and 64: four hand-overs a stage of 16 KB cost more than the
// instructions saved), X in registers for good with the weights through a
// bulk-copied ring (67, 31 and 101), and a ring of asynchronous copies per
// warp (43, 33 and 66).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "moe.h"
#include "ptx.cuh"
#include "tc_launch.h"

namespace gb300 {

namespace {

constexpr int SM_WARPS = 16;  // resident, by the registers


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

// Nibbles i and i + 4 of w minus the zero point, as two 16-bit floats.  mask
// (0x000F000F) and base (kBase) are kernel parameters: as constants the
// compiler spends two logic instructions on what is one of three registers,
// and the logic pipe is what bounds the expansion (805 -> 602 cycles for 128
// rows x 256 values on one SM).
template <bool BF16>
__device__ __forceinline__ uint32_t expand(uint32_t w, int i, uint32_t base_plus_zero,
                                           uint32_t mask, uint32_t base) {
  uint32_t v;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(v) : "r"(w >> (4 * i)), "r"(mask), "r"(base));
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
  if (!ok) return;  // what was there meets zeros of X
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

// A scale's bits, and the scale they are: what is loaded ahead of its use
// must not be looked at (not even to convert) in between.
__device__ __forceinline__ uint32_t scale_bits(const void* s, int type, long long i) {
  return type == T_F32 ? static_cast<const uint32_t*>(s)[i] : static_cast<const uint16_t*>(s)[i];
}
__device__ __forceinline__ float scale_value(uint32_t bits, int type) {
  if (type == T_F32) return __uint_as_float(bits);
  if (type == T_BF16) return __uint_as_float(bits << 16);
  return __half2float(__ushort_as_half(static_cast<unsigned short>(bits)));
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
  for (int e0 = threadIdx.x & ~31; e0 < 32 * nw; e0 += blockDim.x) {
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

constexpr int RT = 2;  // 16-row weight tiles a warp takes against one X

// NT: 8-token tiles.
template <int WPT, int NT>
constexpr int kRun = WPT * NT >= 8 ? 1 : (8 / (WPT * NT) > 4 ? 4 : 8 / (WPT * NT));  // steps of a run

// Most warps of a block (the sums of all of them in shared memory).
template <int NT>
constexpr int kMaxWarps = NT == 4 ? 8 : SM_WARPS;

template <bool BF16, int WPT, int NT>
__global__ void __launch_bounds__(32 * kMaxWarps<NT>, SM_WARPS / kMaxWarps<NT>)
    w4_kernel(const W4Params p) {
  constexpr int SPAN = 32 * WPT;  // K of one step
  constexpr int U = kRun<WPT, NT>;
  __shared__ float red[kMaxWarps<NT>][16 * RT][8 * NT + 1];
  const int warps = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const uint32_t mask = p.nibbles, base = p.nibble_base;
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
  // this thread's first weight row, and how far on the others are; rows past
  // N read the first again and are not stored
  const int left = p.N - n0 - g;
  const long long row0 = static_cast<long long>(e) * p.N + n0 + (left > 0 ? g : 0);
  const uint8_t* const w0 = p.W + row0 * (p.K / 2) + 4 * WPT * t;
  auto rows_on = [&](int i, int h) { return 16 * i + 8 * h < left ? 16 * i + 8 * h : 0; };
  const int steps = (p.K + SPAN - 1) / SPAN;
  const int group_steps = p.group / SPAN;  // steps that share a scale
  for (int rb = r0; rb < r1; rb += 8 * NT) {
    float acc[RT][NT][4];
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j) acc[i][j][0] = acc[i][j][1] = acc[i][j][2] = acc[i][j][3] = 0.f;
    for (int s0 = warp * U; s0 < steps; s0 += warps * U) {
      uint32_t w[2][U][2][WPT] = {};
      auto load_tile = [&](int i, uint32_t (&o)[U][2][WPT]) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint8_t* const src =
              w0 + static_cast<long long>(rows_on(i, h)) * (p.K / 2) + s0 * (SPAN / 2);
#pragma unroll
          for (int u = 0; u < U; ++u)
            load_words<WPT>(src + u * (SPAN / 2), (s0 + u) * SPAN + 8 * WPT * t < p.K, o[u][h]);
        }
      };
      load_tile(0, w[0]);
      // scales and zero points: thread t of a row's four holds step t's
      uint32_t sc[RT][2], z[RT][2];
      const int st = min(s0 + (t < U ? t : U - 1), steps - 1);
      const int G = group_steps == 1 ? st : st / group_steps;
#pragma unroll
      for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const long long at = row0 * p.groups + (rows_on(i, h) * p.groups + G);
          sc[i][h] = scale_bits(p.scales, p.scale_type, at);
          z[i][h] = p.zeros ? p.zeros[at] : 8u;
        }
      uint32_t xf[U][WPT][NT][4];
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const int r = rb + 8 * j + g;
        const uint16_t* const src =
            static_cast<const uint16_t*>(p.X) + (r < r1 ? r : rb) * p.ldx + s0 * SPAN + 8 * WPT * t;
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int c = 0; c < WPT; ++c) {
            uint4 x = make_uint4(0u, 0u, 0u, 0u);
            if (r < r1 && (s0 + u) * SPAN + 8 * WPT * t < p.K)
              x = *reinterpret_cast<const uint4*>(src + u * SPAN + 8 * c);
            xf[u][c][j][0] = __byte_perm(x.x, x.z, 0x5410);
            xf[u][c][j][1] = __byte_perm(x.x, x.z, 0x7632);
            xf[u][c][j][2] = __byte_perm(x.y, x.w, 0x5410);
            xf[u][c][j][3] = __byte_perm(x.y, x.w, 0x7632);
          }
      }
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        if (i + 1 < RT) load_tile(i + 1, w[(i + 1) & 1]);
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int from = (lane & ~3) | u;
          const uint32_t zl = base + __shfl_sync(0xFFFFFFFFu, z[i][0], from) * 0x00010001u;
          const uint32_t zh = base + __shfl_sync(0xFFFFFFFFu, z[i][1], from) * 0x00010001u;
          float sl = scale_value(__shfl_sync(0xFFFFFFFFu, sc[i][0], from), p.scale_type);
          float sh = scale_value(__shfl_sync(0xFFFFFFFFu, sc[i][1], from), p.scale_type);
          // past K: the sums are zeros, but the last group's scale may be infinite
          if (u > 0 && s0 + u >= steps) sl = sh = 0.f;
          float part[NT][4];
#pragma unroll
          for (int j = 0; j < NT; ++j) part[j][0] = part[j][1] = part[j][2] = part[j][3] = 0.f;
#pragma unroll
          for (int c = 0; c < WPT; ++c)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              const uint32_t lo = w[i & 1][u][0][c], hi = w[i & 1][u][1][c];
              const uint32_t a[4] = {expand<BF16>(lo, 2 * half, zl, mask, base),
                                     expand<BF16>(hi, 2 * half, zh, mask, base),
                                     expand<BF16>(lo, 2 * half + 1, zl, mask, base),
                                     expand<BF16>(hi, 2 * half + 1, zh, mask, base)};
#pragma unroll
              for (int j = 0; j < NT; ++j)
                mma16816<BF16>(part[j], a, xf[u][c][j][2 * half], xf[u][c][j][2 * half + 1]);
            }
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            acc[i][j][0] = fmaf(sl, part[j][0], acc[i][j][0]);
            acc[i][j][1] = fmaf(sl, part[j][1], acc[i][j][1]);
            acc[i][j][2] = fmaf(sh, part[j][2], acc[i][j][2]);
            acc[i][j][3] = fmaf(sh, part[j][3], acc[i][j][3]);
          }
        }
      }
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
    for (int o = threadIdx.x; o < 16 * RT * 8 * NT; o += blockDim.x) {
      const int n = o % (16 * RT), m = o / (16 * RT);
      if (rb + m < r1 && n0 + n < p.N) {
        float v = 0.f;
        for (int x = 0; x < warps; ++x) v += red[x][n][m];
        store_d(p.D, p.d_type, (rb + m) * p.ldd + n0 + n, v);
      }
    }
  }
}

template <bool BF16, int WPT, int NT>
cudaError_t launch_as(const W4Params& p, cudaStream_t st) {
  const int tiles = (p.N + 16 * RT - 1) / (16 * RT), experts = p.E > 1 ? std::min(p.E, p.R) : 1;
  const int run = 32 * WPT * kRun<WPT, NT>, runs = (p.K + run - 1) / run;
  // Warps that share a tile's K.  Few make better use of an SM, since its
  // blocks then wait for one another's loads and sums less (4 against 8 warps:
  // 4 x 8192 x 32768 39.4 against 42.4 us, 64 x 2048 x 1024 over 40 experts
  // 16.6 against 18.9; 2 against 4 at K = 1024: 16.9 against 17.9), but where
  // the tiles are few the SMs would be partly empty (8 against 4: 16 x 8192 x
  // 8192 20.9 against 27.5, 4 x 8192 x 10240 20.5 against 23.1, but 16 x 4096
  // x 16384 21.4 against 20.0; 16 against 8: 1 x 4096 x 4096 5.2 against 5.7).
  int warps = runs <= 4 ? 2 : 4;
  while (warps < kMaxWarps<NT> && warps < runs &&
         3ll * tiles * experts * warps < 2 * SM_WARPS * p.num_sms)
    warps *= 2;
  return launch_pdl(w4_kernel<BF16, WPT, NT>, dim3(tiles, experts), dim3(32 * warps), 0, st, p);
}

template <bool BF16, int WPT>
cudaError_t launch_wpt(const W4Params& p, cudaStream_t st) {
  // Tokens a pass covers: as many as an expert has on average (the host does
  // not know the groups).  Under skew the long groups take more passes, each
  // reading the expert's weights.
  const int rows = p.E > 1 ? (p.R + p.E - 1) / p.E : p.R;
  if (rows <= 8) return launch_as<BF16, WPT, 1>(p, st);
  if (rows <= 16) return launch_as<BF16, WPT, 2>(p, st);
  return launch_as<BF16, WPT, 4>(p, st);
}

template <bool BF16>
cudaError_t launch_type(const W4Params& p, cudaStream_t st) {
  // the widest loads whose step stays within a group
  if (p.group % 128 == 0) return launch_wpt<BF16, 4>(p, st);
  if (p.group % 64 == 0) return launch_wpt<BF16, 2>(p, st);
  return launch_wpt<BF16, 1>(p, st);
}

}  // namespace

cudaError_t launch_w4(const W4Params& params, cudaStream_t st) {
  W4Params p = params;
  p.nibbles = 0x000F000Fu;
  p.nibble_base = p.x_type == T_BF16 ? kBase<true> : kBase<false>;
  return p.x_type == T_BF16 ? launch_type<true>(p, st) : launch_type<false>(p, st);
}

}  // namespace gb300
