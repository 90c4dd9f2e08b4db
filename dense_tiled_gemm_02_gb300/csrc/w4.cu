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
#include <cstdlib>

#include "gemm.h"
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
          sc[i][h] = scale_value(scale_bits(p.scales, p.scale_type, srow[i][h] + G), p.scale_type);
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

// ---------------------------------------------------------------- tensor-memory form
// The same sums with the weights expanded into tensor memory, as the A operand
// of tcgen05.mma (128 weight rows x 256 K a stage), and up to 16 tokens as its
// N dimension: the warp-level form above spends as many instructions on X
// fragments, products and scales as on the weights (56 us at 4 x 8192 x
// 32768); here a thread does nothing per weight but expand it.
//
//   warp 0       TMA: 128 rows x 128 bytes of packed weights into the ring
//   warp 1       MMA issue: a block of GB values of K at a time into its own
//                accumulator columns (GB divides the group)
//   warps 2-3    X: 16 tokens x 256 K, permuted as the nibbles are, swizzled
//   warps 4-11   two groups of four, stages in turn: thread = weight row
//                reads its 128 bytes, expands them and stores 128 columns of
//                tensor memory
//   warps 12-15  thread = weight row: scales the blocks' sums in fp32
//
// Blocks take equal contiguous runs of stages over all (expert, row tile,
// token block) tiles; the pieces of a tile that several blocks share are
// added by whichever finishes last, in K order (as in grouped.cu).
constexpr int TC_THREADS = 512;
constexpr int TC_K = 256;                     // K of a stage
constexpr int TC_ROWS = 128;                  // weight rows of a tile
constexpr int TC_TOKENS = 16;
constexpr int TC_STAGES = 9;
constexpr int TC_MIN_RUN = 2;
constexpr uint32_t TC_W_BYTES = TC_ROWS * TC_K / 2;
constexpr uint32_t TC_X_BYTES = TC_TOKENS * TC_K * 2;

template <int GB>
struct TcCfg {
  static constexpr int BLOCKS = TC_K / GB;                // of a stage
  static constexpr int D_COLS = BLOCKS * TC_TOKENS;
  static constexpr int BUFS = GB == 128 ? 3 : 2;          // expanded stages in flight
  static constexpr uint32_t A_COL = 0;                    // BUFS x 128 columns
  static constexpr uint32_t D_COL = BUFS * (TC_K / 2);
  static_assert(D_COL + BUFS * D_COLS <= 512, "tensor memory");
  static constexpr uint32_t SMEM = 1024 + TC_STAGES * TC_W_BYTES + BUFS * TC_X_BYTES + 512 +
                                   4 * (2 * GEMM_MAX_EXPERTS + 2);
  static_assert(SMEM <= 227 * 1024, "shared memory of a block");
};

// D[tmem] (+)= A[tmem] * B[smem].
__device__ __forceinline__ void mma_f16_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                           uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}

// A run of stages of one tile: weight rows n0 .. n0 + 127 of expert e against
// its rows [r0, r1), stages [s0, s1).
struct TcPiece {
  int e, n0, r0, r1, s0, s1;
  int pieces, first, slot;
};

struct TcSchedule {
  const W4Params& p;
  const int* lo;      // [E + 1] offsets
  const int* prefix;  // [E + 1] tiles of the experts before
  int stages, row_tiles, c, units;
  int64_t total, at, end;

  __device__ __forceinline__ TcSchedule(const W4Params& p_, const int* lo_, const int* prefix_)
      : p(p_), lo(lo_), prefix(prefix_), c(blockIdx.x) {
    stages = max(1, (p.K + TC_K - 1) / TC_K);
    row_tiles = (p.N + TC_ROWS - 1) / TC_ROWS;
    total = static_cast<int64_t>(prefix[p.E]) * stages;
    // no run of fewer than TC_MIN_RUN stages (nor, above all, of none: the
    // pieces of a tile are counted by the runs it crosses)
    units = static_cast<int>(
        max(static_cast<int64_t>(1), min(static_cast<int64_t>(gridDim.x), total / TC_MIN_RUN)));
    at = c < units ? total * c / units : 0;
    end = c < units ? total * (c + 1) / units : 0;
  }
  __device__ __forceinline__ bool next(TcPiece& x) {
    if (at >= end) return false;
    const int64_t t = at / stages;
    int a = 0, b = p.E;  // prefix[a] <= t < prefix[b]
    while (b - a > 1) {
      const int m = (a + b) >> 1;
      if (prefix[m] <= t)
        a = m;
      else
        b = m;
    }
    const int i = static_cast<int>(t) - prefix[a];
    const int blocks = (prefix[a + 1] - prefix[a]) / row_tiles;  // of tokens
    const int rt = i / blocks;
    x.e = a;
    x.n0 = rt * TC_ROWS;
    x.r0 = lo[a] + (i - rt * blocks) * TC_TOKENS;
    x.r1 = min(lo[a + 1], x.r0 + TC_TOKENS);
    const int64_t t0 = t * stages, t1 = t0 + stages;
    x.s0 = static_cast<int>(at - t0);
    x.s1 = static_cast<int>(min(end, t1) - t0);
    x.first = static_cast<int>(((t0 + 1) * units - 1) / total);
    x.pieces = static_cast<int>((t1 * units - 1) / total) - x.first + 1;
    x.slot = c == x.first ? 1 : 0;
    at = min(end, t1);
    return true;
  }
};

template <bool BF16, int GB>
__global__ void __launch_bounds__(TC_THREADS, 1)
    w4_tc_kernel(const __grid_constant__ CUtensorMap tmW, const W4Params p) {
  using C = TcCfg<GB>;
  constexpr int BUFS = C::BUFS;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* const smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* const sW = smem;
  uint8_t* const sX = smem + TC_STAGES * TC_W_BYTES;
  uint64_t* const bars = reinterpret_cast<uint64_t*>(sX + BUFS * TC_X_BYTES);
  constexpr int NBARS = 2 * TC_STAGES + 4 * BUFS;
  static_assert(8 * NBARS + 16 <= 512, "barriers");
  uint32_t* const tmem_holder = reinterpret_cast<uint32_t*>(bars + NBARS);
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  volatile int* const ep_last = abort_flag + 1;
  int* const lo = reinterpret_cast<int*>(reinterpret_cast<uint8_t*>(bars) + 512);
  int* const prefix = lo + p.E + 1;
  const uint32_t bar0 = smem_u32(bars);
  auto w_full = [&](uint32_t s) { return bar0 + 8u * s; };
  auto w_empty = [&](uint32_t s) { return bar0 + 8u * (TC_STAGES + s); };
  auto a_full = [&](uint32_t b) { return bar0 + 8u * (2 * TC_STAGES + b); };       // weights expanded
  auto x_full = [&](uint32_t b) { return bar0 + 8u * (2 * TC_STAGES + BUFS + b); };
  auto done = [&](uint32_t b) { return bar0 + 8u * (2 * TC_STAGES + 2 * BUFS + b); };  // MMAs
  auto d_empty = [&](uint32_t b) { return bar0 + 8u * (2 * TC_STAGES + 3 * BUFS + b); };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < TC_STAGES; ++s) {
      mbar_init(w_full(s), 1);
      mbar_init(w_empty(s), 4);
    }
    for (int b = 0; b < BUFS; ++b) {
      mbar_init(a_full(b), 4);
      mbar_init(x_full(b), 2);
      mbar_init(done(b), 1);
      mbar_init(d_empty(b), 4);
    }
    *abort_flag = 0;
    fence_mbar_init();
    fence_proxy_async_smem();
  }
  if (warp == 0 && lane == 0) tma_prefetch_desc(&tmW);
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_holder), 512);
    tmem_relinquish();
  }
  pdl_wait();
  pdl_trigger();
  const int row_tiles = (p.N + TC_ROWS - 1) / TC_ROWS;
  for (int e = threadIdx.x; e <= p.E; e += TC_THREADS) {
    lo[e] = p.offsets ? p.offsets[e] : (e == 0 ? 0 : p.R);
    if (p.offsets && e < p.E) expert_rows(p.offsets, e, p.R, p.status);
  }
  __syncthreads();
  if (warp == 2) {
    auto tiles = [&](int e) {
      const bool ok = lo[e] >= 0 && lo[e + 1] >= lo[e] && lo[e + 1] <= p.R;
      return ok ? (lo[e + 1] - lo[e] + TC_TOKENS - 1) / TC_TOKENS * row_tiles : 0;
    };
    const int len = (p.E + 31) / 32, b = min(p.E, lane * len), e1 = min(p.E, b + len);
    int sum = 0;
    for (int e = b; e < e1; ++e) sum += tiles(e);
    int inc = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int u = __shfl_up_sync(0xFFFFFFFFu, inc, d);
      if (lane >= d) inc += u;
    }
    int at = inc - sum;
    for (int e = b; e < e1; ++e) {
      prefix[e] = at;
      at += tiles(e);
    }
    if (lane == 31) prefix[p.E] = inc;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;
  const uint64_t tmo = p.timeout_ns;
  TcSchedule work(p, lo, prefix);
  TcPiece x;
  // One lane waits for the warp; false after a timeout.
  auto wait = [&](uint32_t bar, uint32_t parity) {
    bool ok = true;
    if (lane == 0) ok = bounded_wait(bar, parity, abort_flag, p.status, STATUS_TIMEOUT, tmo);
    ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
    __syncwarp();
    return ok;
  };
  bool ok = true;

  if (warp == 0) {
    // -------------------------------------------------------------- W copies
    if (elect_one()) {
      uint32_t it = 0, s = 0, ph = 0;
      bool skipped = false;
      while (ok && work.next(x)) {
        for (int st = x.s0; st < x.s1; ++st) {
          ok = bounded_wait(w_empty(s), ph ^ 1u, abort_flag, p.status, STATUS_TIMEOUT, tmo);
          if (!ok) break;
          if ((p.debug_flags & DBG_SKIP_FIRST_FILL) && it == 0) {
            skipped = true;  // test hook: the first wait on the ring expires
          } else {
            mbar_arrive_expect_tx(w_full(s), TC_W_BYTES);
            tma_load_2d(smem_u32(sW + s * TC_W_BYTES), &tmW, st * (TC_K / 2), x.e * p.N + x.n0,
                        w_full(s));
          }
          ++it;
          if (++s == TC_STAGES) {
            s = 0;
            ph ^= 1u;
          }
        }
      }
      for (uint32_t j = it > TC_STAGES ? it - TC_STAGES : 0; j < it; ++j)
        if (!(skipped && j == 0)) drain_wait(w_full(j % TC_STAGES), (j / TC_STAGES) & 1u, 200000000ull);
    }
    __syncwarp();
  } else if (warp == 1) {
    // -------------------------------------------------------------- MMA issue
    if (elect_one()) {
      const uint32_t idesc = idesc_f16(BF16, 0, 0, TC_ROWS, TC_TOKENS);
      const uint32_t dhi = sdesc_hi_sw128(1024u);
      const uint32_t x_lo0 = sdesc_lo(smem_u32(sX), 16u);
      uint32_t b = 0, ph = 0;
      while (ok && work.next(x)) {
        for (int st = x.s0; st < x.s1; ++st) {
          ok = bounded_wait(d_empty(b), ph ^ 1u, abort_flag, p.status, STATUS_TIMEOUT, tmo) &&
               bounded_wait(x_full(b), ph, abort_flag, p.status, STATUS_TIMEOUT, tmo) &&
               bounded_wait(a_full(b), ph, abort_flag, p.status, STATUS_TIMEOUT, tmo);
          if (!ok) break;
          tc_fence_after();
          const uint32_t a = tmem_base + C::A_COL + b * (TC_K / 2);
          const uint32_t d = tmem_base + C::D_COL + b * C::D_COLS;
          const uint32_t x_lo = x_lo0 + b * (TC_X_BYTES >> 4);
          // the blocks in turn: a product into the accumulator of the one
          // before it waits for it, and at 16 columns that is most of its time
#pragma unroll
          for (int k = 0; k < GB; k += 16)
#pragma unroll
            for (int i = 0; i < C::BLOCKS; ++i) {
              const int at = i * GB + k;  // K of the stage
              mma_f16_ts(d + i * TC_TOKENS, a + at / 2,
                         sdesc(dhi, x_lo + (at / 64) * (TC_TOKENS * 128 / 16) + (at % 64) / 8), idesc,
                         k != 0);
            }
          mma_commit(done(b));
          if (++b == BUFS) {
            b = 0;
            ph ^= 1u;
          }
        }
      }
    }
    __syncwarp();
  } else if (warp < 4) {
    // -------------------------------------------------------------- X tiles
    // 16-byte unit (r, u): token r, K 8 u .. 8 u + 7 of the stage; this warp
    // takes units u of its parity, lane = 16 (u / 2 % 2) + r
    const uint16_t* const X = static_cast<const uint16_t*>(p.X);
    const int r = lane & 15, u0 = (warp & 1) + 2 * (lane >> 4);
    uint32_t b = 0, ph = 0;
    uint4 v[8];
    auto load = [&](const TcPiece& q, int st) {
      const uint16_t* const row = X + (q.r0 + r) * p.ldx + st * TC_K;
      const bool live = q.r0 + r < q.r1;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int k = 8 * (u0 + 4 * i);
        v[i] = make_uint4(0u, 0u, 0u, 0u);
        if (live && st * TC_K + k < p.K) v[i] = *reinterpret_cast<const uint4*>(row + k);
      }
    };
    bool more = work.next(x);
    if (more) load(x, x.s0);
    while (more) {
      for (int st = x.s0; st < x.s1; ++st) {
        ok = wait(done(b), ph ^ 1u);  // the MMAs have read the buffer
        if (!ok) break;
        uint8_t* const out = sX + b * TC_X_BYTES + r * 128;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int u = u0 + 4 * i;
          const uint4 w = make_uint4(__byte_perm(v[i].x, v[i].z, 0x5410), __byte_perm(v[i].x, v[i].z, 0x7632),
                                     __byte_perm(v[i].y, v[i].w, 0x5410), __byte_perm(v[i].y, v[i].w, 0x7632));
          *reinterpret_cast<uint4*>(out + (u >> 3) * (TC_TOKENS * 128) + (((u & 7) ^ (r & 7)) << 4)) = w;
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(x_full(b));
        if (++b == BUFS) {
          b = 0;
          ph ^= 1u;
        }
        // the next stage's tokens while this one is multiplied
        if (st + 1 < x.s1) {
          load(x, st + 1);
        } else {
          TcPiece n;
          more = work.next(n);
          if (more) load(n, n.s0);
          x = n;
          break;
        }
      }
      if (!ok) break;
    }
  } else if (warp < 12) {
    // -------------------------------------------------------------- expand the weights
    const int group = (warp >> 2) - 1;  // 0: even stages of this block, 1: odd ones
    const int row = (warp & 3) * 32 + lane;
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    uint32_t it = 0;
    while (ok && work.next(x)) {
      const int n = x.n0 + row;
      const long long at = (static_cast<long long>(x.e) * p.N + min(n, p.N - 1)) * p.groups;
      // zero points of this group's next stage, asked for a stage ahead
      uint32_t next_z[C::BLOCKS];
      auto ask = [&](int st) {
#pragma unroll
        for (int i = 0; i < C::BLOCKS; ++i)
          next_z[i] = p.zeros ? p.zeros[at + min((st * TC_K + i * GB) / p.group, p.groups - 1)] : 8u;
      };
      ask(x.s0 + static_cast<int>((it ^ static_cast<uint32_t>(group)) & 1u));
      for (int st = x.s0; st < x.s1; ++st, ++it) {
        if ((it & 1u) != static_cast<uint32_t>(group)) continue;
        const uint32_t s = it % TC_STAGES, b = it % BUFS;
        uint32_t bz[C::BLOCKS];
#pragma unroll
        for (int i = 0; i < C::BLOCKS; ++i) bz[i] = next_z[i];
        if (st + 2 < x.s1) ask(st + 2);
        ok = wait(w_full(s), (it / TC_STAGES) & 1u);
        if (!ok) break;
        const uint8_t* const in = sW + s * TC_W_BYTES + row * 128;
        const uint32_t out = tmem_base + lane_base + C::A_COL + b * (TC_K / 2);
#pragma unroll 1
        for (int h = 0; h < 4; ++h) {  // 64 K, 32 columns at a time
          uint32_t r[32];
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const uint4 w = *reinterpret_cast<const uint4*>(in + (((2 * h + c) ^ (row & 7)) << 4));
            uint32_t zero = bz[0];
#pragma unroll
            for (int i = 1; i < C::BLOCKS; ++i)
              if ((64 * h + 32 * c) / GB == i) zero = bz[i];
            const uint32_t z = kBase<BF16> + zero * 0x00010001u;
            const uint32_t q[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
              for (int j = 0; j < 4; ++j) r[16 * c + 4 * i + j] = expand<BF16>(q[i], j, z);
          }
          if (h == 0) {
            // the MMAs of the buffer's last stage have read it
            ok = wait(done(b), ((it / BUFS) & 1u) ^ 1u);
            if (!ok) break;
            tc_fence_after();
          }
          tmem_st_32x32b_x32(out + 32 * h, r);
        }
        if (!ok) break;
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(w_empty(s));
          mbar_arrive(a_full(b));
        }
      }
    }
  } else {
    // -------------------------------------------------------------- scale and store
    const int q = warp & 3;
    const uint32_t lane_base = static_cast<uint32_t>(q * 32) << 16;
    const bool leader = threadIdx.x == 384;
    uint32_t b = 0, ph = 0;
    while (ok && work.next(x)) {
      const int n = x.n0 + q * 32 + lane;
      const long long at = (static_cast<long long>(x.e) * p.N + min(n, p.N - 1)) * p.groups;
      float sum[TC_TOKENS];
#pragma unroll
      for (int j = 0; j < TC_TOKENS; ++j) sum[j] = 0.f;
      // Scales of AHEAD stages at a time, asked for AHEAD stages before they
      // are used: a stage is shorter than a trip to memory.
      constexpr int AHEAD = 2;
      uint32_t next_scale[AHEAD][C::BLOCKS], now_scale[AHEAD][C::BLOCKS];
      auto ask = [&](int st) {
#pragma unroll
        for (int a = 0; a < AHEAD; ++a)
#pragma unroll
          for (int i = 0; i < C::BLOCKS; ++i)
            next_scale[a][i] = scale_bits(
                p.scales, p.scale_type, at + min(((st + a) * TC_K + i * GB) / p.group, p.groups - 1));
      };
      ask(x.s0);
#pragma unroll 1
      for (int st0 = x.s0; ok && st0 < x.s1; st0 += AHEAD) {
#pragma unroll
      for (int a = 0; a < AHEAD; ++a)
#pragma unroll
        for (int i = 0; i < C::BLOCKS; ++i) now_scale[a][i] = next_scale[a][i];
      if (st0 + AHEAD < x.s1) ask(st0 + AHEAD);
#pragma unroll
      for (int a = 0; a < AHEAD; ++a) {
        if (st0 + a >= x.s1) break;
        float scale[C::BLOCKS];
#pragma unroll
        for (int i = 0; i < C::BLOCKS; ++i) scale[i] = scale_value(now_scale[a][i], p.scale_type);
        // all four warps take the same path through the barriers below
        if (leader) {
          const bool go = bounded_wait(done(b), ph, abort_flag, p.status, STATUS_TIMEOUT, tmo);
          *ep_last = go ? 1 : 0;
        }
        named_barrier_sync(1, 128);
        ok = *ep_last != 0;
        named_barrier_sync(1, 128);
        if (!ok) break;
        tc_fence_after();
        const uint32_t d = tmem_base + lane_base + C::D_COL + b * C::D_COLS;
#pragma unroll
        for (int i = 0; i < C::BLOCKS; ++i) {
          // past K: zeros in X, whatever the scale
          uint32_t v[16];
          tmem_ld_32x32b_x16(d + i * TC_TOKENS, v);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < TC_TOKENS; ++j) sum[j] = fmaf(scale[i], __uint_as_float(v[j]), sum[j]);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(d_empty(b));
        if (++b == BUFS) {
          b = 0;
          ph ^= 1u;
        }
      }
      }
      if (!ok) break;
      if (x.pieces > 1) {
        float* const mine = p.partial + (2 * static_cast<size_t>(blockIdx.x) + x.slot) * (TC_TOKENS * TC_ROWS) +
                            q * 32 + lane;
#pragma unroll
        for (int j = 0; j < TC_TOKENS; ++j) mine[j * TC_ROWS] = sum[j];
        __threadfence();
        named_barrier_sync(1, 128);
        if (leader) {
          unsigned* const count = p.counters + x.first;
          const bool last = atomicAdd(count, 1u) == static_cast<unsigned>(x.pieces) - 1u;
          if (last) *count = 0u;  // ready for the next call
          __threadfence();
          *ep_last = last ? 1 : 0;
        }
        named_barrier_sync(1, 128);
        const bool last = *ep_last != 0;
        named_barrier_sync(1, 128);
        if (!last) continue;
        __threadfence();
        float all[TC_TOKENS];
#pragma unroll
        for (int j = 0; j < TC_TOKENS; ++j) all[j] = 0.f;
        for (int i = 0; i < x.pieces; ++i) {  // in K order
          const float* const src =
              p.partial + (2 * static_cast<size_t>(x.first + i) + (i == 0 ? 1 : 0)) * (TC_TOKENS * TC_ROWS) +
              q * 32 + lane;
#pragma unroll
          for (int j = 0; j < TC_TOKENS; ++j) all[j] += __ldcg(src + j * TC_ROWS);
        }
#pragma unroll
        for (int j = 0; j < TC_TOKENS; ++j) sum[j] = all[j];
      }
      if (n < p.N) {
#pragma unroll
        for (int j = 0; j < TC_TOKENS; ++j)
          if (x.r0 + j < x.r1) store_d(p.D, p.d_type, (x.r0 + j) * p.ldd + n, sum[j]);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, 512);
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

template <bool BF16, int GB>
cudaError_t launch_tc(const W4Params& p, const CUtensorMap& w, int num_sms, cudaStream_t st) {
  const cudaError_t e =
      cudaFuncSetAttribute(w4_tc_kernel<BF16, GB>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           TcCfg<GB>::SMEM);
  if (e != cudaSuccess) return e;
  return launch_pdl(w4_tc_kernel<BF16, GB>, dim3(num_sms), dim3(TC_THREADS), TcCfg<GB>::SMEM, st, w, p);
}

template <bool BF16>
cudaError_t launch_type(const W4Params& p, const CUtensorMap* w, int num_sms, cudaStream_t st) {
  // the widest block (reads) whose step stays within a group
  static const int tcgb = getenv("TCGB") ? atoi(getenv("TCGB")) : 128;
  if (p.group % 128 == 0 && tcgb == 64 && w) return launch_tc<BF16, 64>(p, *w, num_sms, st);
  if (p.group % 64 == 0 && tcgb == 32 && w) return launch_tc<BF16, 32>(p, *w, num_sms, st);
  if (p.group % 128 == 0)
    return w ? launch_tc<BF16, 128>(p, *w, num_sms, st) : launch_wpt<BF16, 4>(p, st);
  if (p.group % 64 == 0)
    return w ? launch_tc<BF16, 64>(p, *w, num_sms, st) : launch_wpt<BF16, 2>(p, st);
  return w ? launch_tc<BF16, 32>(p, *w, num_sms, st) : launch_wpt<BF16, 1>(p, st);
}

}  // namespace

size_t w4_partial_bytes(int num_sms) {
  return sizeof(float) * 2 * num_sms * TC_TOKENS * TC_ROWS;
}

cudaError_t launch_w4(const W4Params& p, const CUtensorMap* w, int num_sms, cudaStream_t st) {
  return p.x_type == T_BF16 ? launch_type<true>(p, w, num_sms, st)
                            : launch_type<false>(p, w, num_sms, st);
}

}  // namespace gb300
