// grouped.cu -- matrix products grouped by expert over ragged row groups.
//
//   rows:  D[r,n]   = sum_k A[r,k] B_e[k,n] (+ C)         for the rows r of e
//   grad:  D_e[k,n] = sum over e's rows r of A[r,k] B[r,n] (+ C)
//
// tcgen05 with D's columns ("features") as the M dimension, 128 to a tile,
// and D's rows as the N dimension.  The M of an MMA is fixed while its N is
// any multiple of 32 up to 256, so the ragged side goes to N: a group of m
// rows is cut into ceil(m / 256) tiles of equal width and costs about m rows
// of tensor time, not m rounded up to a tile; a decode step's one or two rows
// cost a 32-wide MMA while the weights stream.  An accumulator's lanes are
// then consecutive features: lane-consecutive stores run along D's rows.
//
// Every CTA reads the offsets and counts the tiles of each expert into a
// prefix sum in shared memory; tile t of the persistent loop finds its expert
// by bisection.  No host knowledge of the groups, one launch.
//
// Nothing of another expert enters a sum, not even as 0 * NaN: rows past a
// group's end are columns of the accumulator that are not stored (rows), and
// K past its end is read as zeros on both sides because the tensor maps end
// there (an N-contiguous B gets a dimension per expert).  In grad the sum
// itself is ragged: the last slice's rows past the group are overwritten
// with zeros in shared memory, on both operands, before the MMA reads them.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "gemm.h"
#include "moe.h"
#include "ptx.cuh"
#include "tc_launch.h"

namespace gb300 {

namespace {

constexpr int FT = 128;              // features of a tile
constexpr int QT = 256;              // most D rows of a tile
constexpr int STAGES = 4;
constexpr uint32_t F_BYTES = FT * BK * 2;
constexpr uint32_t X_BYTES = QT * BK * 2;
constexpr int RASTER = 8;            // row tiles that share a features tile in L2

constexpr uint32_t grouped_smem() {
  return STAGES * (F_BYTES + X_BYTES) + 1024 /* alignment */ + 256 /* barriers */;
}
// after the barriers: first and end row of each expert, tile prefix
constexpr uint32_t smem_total() { return grouped_smem() + 4 * (3 * GEMM_MAX_EXPERTS + 1); }

// x, y, z: coordinates from the innermost dimension.
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const void* tmap, int32_t x, int32_t y,
                                            int32_t z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}

struct Tile {
  int e;
  int f0;         // first feature
  int q0, nq;     // first D row (rows: of all rows; grad: of the expert's K) and how many
  int k0, klen;   // the sum's range (rows: 0, K; grad: the expert's rows)
};

// Row tiles of an expert with m D rows, and their common width.
__device__ __forceinline__ int row_tiles(int m) { return (m + QT - 1) / QT; }
__device__ __forceinline__ int tile_width(int m, int tiles) {
  return ((m + tiles - 1) / tiles + 31) & ~31;
}

__device__ __forceinline__ Tile find_tile(const GroupedParams& p, const int* lo, const int* prefix,
                                          int t) {
  int a = 0, b = p.E;  // prefix[a] <= t < prefix[b]
  while (b - a > 1) {
    const int m = (a + b) >> 1;
    if (prefix[m] <= t)
      a = m;
    else
      b = m;
  }
  const int i = t - prefix[a];
  const int ft = (p.N + FT - 1) / FT;
  const int rows = lo[a + p.E] - lo[a];
  const int m = p.grad ? p.K : rows;
  const int rt = row_tiles(m), w = tile_width(m, rt);
  int64_t ri, fi;
  raster_tile(i, rt, ft, RASTER, ri, fi);
  Tile x;
  x.e = a;
  x.f0 = static_cast<int>(fi) * FT;
  const int q = static_cast<int>(ri) * w;
  x.nq = min(w, m - q);
  x.q0 = p.grad ? q : lo[a] + q;
  x.k0 = p.grad ? lo[a] : 0;
  x.klen = p.grad ? rows : p.K;
  return x;
}

__device__ __forceinline__ float load_c(const GroupedParams& p, long long i) {
  if (p.d_type == T_F32) return static_cast<const float*>(p.C)[i];
  if (p.d_type == T_BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(p.C)[i]);
  return __half2float(static_cast<const __half*>(p.C)[i]);
}
__device__ __forceinline__ void store_d(const GroupedParams& p, long long i, float v) {
  if (p.d_type == T_F32)
    static_cast<float*>(p.D)[i] = v;
  else if (p.d_type == T_BF16)
    static_cast<__nv_bfloat16*>(p.D)[i] = __float2bfloat16_rn(v);
  else
    static_cast<__half*>(p.D)[i] = __float2half_rn(v);
}

__global__ void __launch_bounds__(NUM_THREADS, 1)
    grouped_kernel(const __grid_constant__ CUtensorMap tmF, const __grid_constant__ CUtensorMap tmX128,
                   const __grid_constant__ CUtensorMap tmX32, const GroupedParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* const smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* const sF = smem;
  uint8_t* const sX = smem + STAGES * F_BYTES;
  uint64_t* const bars = reinterpret_cast<uint64_t*>(sX + STAGES * X_BYTES);
  constexpr int NBARS = 2 * STAGES + 5;
  uint32_t* const tmem_holder = reinterpret_cast<uint32_t*>(bars + NBARS);
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  volatile int* const ep_go = abort_flag + 1;
  int* const lo = reinterpret_cast<int*>(reinterpret_cast<uint8_t*>(bars) + 256);  // [2E]: first, end
  int* const prefix = lo + 2 * p.E;  // [E + 1]

  const uint32_t bar0 = smem_u32(bars);
  auto full = [&](uint32_t s) { return bar0 + 8u * s; };
  auto empty = [&](uint32_t s) { return bar0 + 8u * (STAGES + s); };
  auto acc_full = [&](uint32_t b) { return bar0 + 8u * (2 * STAGES + b); };
  auto acc_empty = [&](uint32_t b) { return bar0 + 8u * (2 * STAGES + 2 + b); };
  const uint32_t done_bar = bar0 + 8u * (2 * STAGES + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(acc_full(b), 1);
      mbar_init(acc_empty(b), 4);
    }
    mbar_init(done_bar, 1);
    *abort_flag = 0;
    fence_mbar_init();
    fence_proxy_async_smem();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_holder), 512);
    tmem_relinquish();
  }
  pdl_wait();
  pdl_trigger();
  const int ft = (p.N + FT - 1) / FT;
  for (int e = threadIdx.x; e < p.E; e += NUM_THREADS) {
    const int2 r = expert_rows(p.offsets, e, p.R, p.status);
    lo[e] = r.x;
    lo[e + p.E] = r.y;
  }
  __syncthreads();
  if (warp == 2) {  // the tile prefix: each lane a run of experts, then a warp scan
    const int len = (p.E + 31) / 32, b = min(p.E, lane * len), e1 = min(p.E, b + len);
    int sum = 0;
    for (int e = b; e < e1; ++e) sum += row_tiles(p.grad ? p.K : lo[e + p.E] - lo[e]) * ft;
    int inc = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int u = __shfl_up_sync(0xFFFFFFFFu, inc, d);
      if (lane >= d) inc += u;
    }
    int at = inc - sum;
    for (int e = b; e < e1; ++e) {
      prefix[e] = at;
      at += row_tiles(p.grad ? p.K : lo[e + p.E] - lo[e]) * ft;
    }
    if (lane == 31) prefix[p.E] = inc;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;
  const int tiles = prefix[p.E];
  const uint64_t tmo = p.timeout_ns;
  const int grid = gridDim.x;

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    if (lane == 0) {
      uint32_t it = 0, s = 0, ph = 0;
      bool stop = false, skipped = false;
      for (int t = blockIdx.x; t < tiles && !stop; t += grid) {
        const Tile x = find_tile(p, lo, prefix, t);
        for (int k = 0; k < x.klen; k += BK) {
          if (!bounded_wait(empty(s), ph ^ 1u, abort_flag, p.status, STATUS_TIMEOUT, tmo)) {
            stop = true;
            break;
          }
          const uint32_t fd = smem_u32(sF + s * F_BYTES), xd = smem_u32(sX + s * X_BYTES);
          if ((p.debug_flags & DBG_SKIP_FIRST_FILL) && it == 0) {
            skipped = true;  // test hook: the MMA's wait on the first stage expires
          } else if (p.grad) {
            const int xb = (x.nq + 63) / 64;
            mbar_arrive_expect_tx(full(s), F_BYTES + xb * 8192u);
            for (int i = 0; i < FT / 64; ++i)
              tma_load_2d(fd + i * 8192u, &tmF, x.f0 + 64 * i, x.k0 + k, full(s));
            for (int i = 0; i < xb; ++i)
              tma_load_2d(xd + i * 8192u, &tmX128, x.q0 + 64 * i, x.k0 + k, full(s));
          } else {
            const bool wide = x.nq > 64;
            const int xb = wide ? (x.nq + 127) / 128 : (x.nq + 31) / 32;
            mbar_arrive_expect_tx(full(s), F_BYTES + xb * (wide ? 16384u : 4096u));
            if (p.f_mn) {
              for (int i = 0; i < FT / 64; ++i)
                tma_load_3d(fd + i * 8192u, &tmF, x.f0 + 64 * i, k, x.e, full(s));
            } else {
              tma_load_2d(fd, &tmF, k, x.e * p.N + x.f0, full(s));
            }
            for (int i = 0; i < xb; ++i) {
              if (wide)
                tma_load_2d(xd + i * 16384u, &tmX128, k, x.q0 + 128 * i, full(s));
              else
                tma_load_2d(xd + i * 4096u, &tmX32, k, x.q0 + 32 * i, full(s));
            }
          }
          ++it;
          if (++s == STAGES) {
            s = 0;
            ph ^= 1u;
          }
        }
      }
      // copies in flight land before the CTA leaves
      for (uint32_t j = it > STAGES ? it - STAGES : 0; j < it; ++j) {
        if (skipped && j == 0) continue;
        drain_wait(full(j % STAGES), (j / STAGES) & 1u, 200000000ull);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    // All lanes walk the loop (they clear rows past a group together); lane 0
    // waits and issues.
    const bool x_mn = p.grad != 0;
    const uint32_t f_lo0 = sdesc_lo(smem_u32(sF), p.f_mn ? 8192u : 16u);
    const uint32_t x_lo0 = sdesc_lo(smem_u32(sX), x_mn ? 8192u : 16u);
    const uint32_t dhi = sdesc_hi_sw128(1024u);
    const uint32_t f_step = p.f_mn ? 128u : 2u, x_step = x_mn ? 128u : 2u;
    uint32_t s = 0, ph = 0, acc_it = 0;
    bool ok = true;
    for (int t = blockIdx.x; t < tiles && ok; t += grid) {
      const Tile x = find_tile(p, lo, prefix, t);
      if (x.klen == 0) continue;
      const uint32_t buf = acc_it & 1u;
      const uint32_t d_tmem = tmem_base + buf * QT;
      const uint32_t idesc = p.idesc | (static_cast<uint32_t>(((x.nq + 31) & ~31) >> 3) << 17);
      if (lane == 0)
        ok = bounded_wait(acc_empty(buf), ((acc_it >> 1) & 1u) ^ 1u, abort_flag, p.status,
                          STATUS_TIMEOUT, tmo);
      ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
      if (!ok) break;
      tc_fence_after();
      for (int k = 0; k < x.klen; k += BK) {
        if (lane == 0)
          ok = bounded_wait(full(s), ph, abort_flag, p.status, STATUS_TIMEOUT, tmo);
        ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
        if (!ok) break;
        const int left = min(BK, x.klen - k);
        const int chunks = (left + 15) / 16;
        if (p.grad && left < 16 * chunks) {
          // rows [left, 16 chunks) of the slice belong to another expert (or
          // to nobody): zero them in every 64-wide box of both operands
          const int n16 = (16 * chunks - left) * 8;  // 16-byte units per box
          const int boxes = FT / 64 + (x.nq + 63) / 64;
          for (int i = lane; i < n16 * boxes; i += 32) {
            const int b = i / n16, u = i - b * n16;
            uint8_t* const base = b < FT / 64 ? sF + s * F_BYTES + b * 8192
                                              : sX + s * X_BYTES + (b - FT / 64) * 8192;
            *reinterpret_cast<uint4*>(base + left * 128 + u * 16) = make_uint4(0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();
          __syncwarp();
        }
        if (lane == 0) {
          const uint32_t f_lo = f_lo0 + s * (F_BYTES >> 4), x_lo = x_lo0 + s * (X_BYTES >> 4);
          for (int c = 0; c < chunks; ++c)
            mma_f16_ss(d_tmem, sdesc(dhi, f_lo + c * f_step), sdesc(dhi, x_lo + c * x_step), idesc,
                       (k | c) != 0);
          mma_commit(empty(s));
        }
        __syncwarp();
        if (++s == STAGES) {
          s = 0;
          ph ^= 1u;
        }
      }
      if (!ok) break;
      if (lane == 0) mma_commit(acc_full(buf));
      ++acc_it;
    }
    if (lane == 0) {
      mma_commit(done_bar);
      drain_wait(done_bar, 0, 200000000ull);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3;
    const uint32_t lane_base = static_cast<uint32_t>(q * 32) << 16;
    const bool leader = threadIdx.x == 64;
    uint32_t acc_it = 0;
    for (int t = blockIdx.x; t < tiles; t += grid) {
      const Tile x = find_tile(p, lo, prefix, t);
      const uint32_t buf = acc_it & 1u;
      if (x.klen != 0) {
        if (leader)
          *ep_go = bounded_wait(acc_full(buf), (acc_it >> 1) & 1u, abort_flag, p.status,
                                STATUS_TIMEOUT, tmo) ? 1 : 0;
        named_barrier_sync(1, 128);
        const bool go = *ep_go != 0;
        named_barrier_sync(1, 128);
        if (!go) break;
        tc_fence_after();
      }
      const int f = x.f0 + q * 32 + lane;
      const long long row0 = p.grad ? static_cast<long long>(x.e) * p.K + x.q0 : x.q0;
#pragma unroll 1
      for (int c = 0; c < x.nq; c += 32) {
        uint32_t v[32];
        if (x.klen != 0) {
          tmem_ld_32x32b_x32(tmem_base + lane_base + buf * QT + c, v);
          tmem_ld_wait();
        } else {
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = 0u;
        }
        if (f < p.N) {
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            if (c + j >= x.nq) break;
            float d = __uint_as_float(v[j]);
            if (p.C) d += load_c(p, (row0 + c + j) * p.ldc + f);
            store_d(p, (row0 + c + j) * p.ldd + f, d);
          }
        }
        __syncwarp();
      }
      if (x.klen != 0) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(acc_empty(buf));
        ++acc_it;
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

}  // namespace

cudaError_t prepare_grouped() {
  return cudaFuncSetAttribute(grouped_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              smem_total());
}

cudaError_t launch_grouped(const CUtensorMap& f, const CUtensorMap& x128, const CUtensorMap& x32,
                           const GroupedParams& p, int grid, cudaStream_t st) {
  return launch_pdl(grouped_kernel, dim3(grid), dim3(NUM_THREADS), smem_total(), st, f, x128, x32, p);
}

}  // namespace gb300
