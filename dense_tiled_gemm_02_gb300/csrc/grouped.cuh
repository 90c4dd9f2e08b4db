// grouped.cuh -- what the grouped kernels share (grouped.cu, i8_tiles.cu): the
// schedule of tiles and K slices over the CTAs, and the instructions of their
// loads and epilogues.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "gemm.h"
#include "moe.h"
#include "ptx.cuh"
#include "tc_launch.h"

namespace gb300 {

namespace {

constexpr int FT = 128;                       // features of a CTA
constexpr int RASTER = 8;                     // row tiles that share a features tile in L2
constexpr int MIN_RUN = 8;                    // K slices (of 64): a shorter run costs more than it saves
constexpr uint32_t EPI_BYTES = 32 * 256;      // staged 32 rows x 128 features of 16 bits
// K slices (of 64) by which a split must shorten the busiest unit's work: what the
// exchange of partial sums costs (about 4 us at a quarter us a slice).  Three
// times as many for CTA pairs that share all of their tiles, whose 128 KB of
// partial sums a CTA nothing else hides (36 tiles of 47 slices on 76 pairs:
// 29.3 us split, 21.7 whole).
constexpr int SPLIT_GAIN = 16;
constexpr int EPI_WARPS = 8;
constexpr int QUEUE = 4;                      // pieces the schedule runs ahead

// ---------------------------------------------------------------- PTX these kernels add
template <int CG>
__device__ __forceinline__ void load_2d(uint32_t dst, const void* tmap, int32_t x, int32_t y,
                                        uint32_t bar) {
  if constexpr (CG == 2)
    tma_load_2d_pair(dst, tmap, x, y, bar);
  else
    tma_load_2d(dst, tmap, x, y, bar);
}

// x, y, z: coordinates from the innermost dimension.
template <int CG>
__device__ __forceinline__ void load_3d(uint32_t dst, const void* tmap, int32_t x, int32_t y,
                                        int32_t z, uint32_t bar) {
  if constexpr (CG == 2)
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}

template <int CG>
__device__ __forceinline__ void mma(uint32_t d, uint64_t f, uint64_t x, uint32_t idesc,
                                    uint32_t accumulate) {
  if constexpr (CG == 2)
    mma_f16_ss_pair(d, f, x, idesc, accumulate);
  else
    mma_f16_ss(d, f, x, idesc, accumulate);
}

// Arrive on `bar` (of both CTAs of a pair) when the MMAs so far are done.
template <int CG>
__device__ __forceinline__ void commit(uint32_t bar) {
  if constexpr (CG == 2)
    mma_commit_pair_both(bar);
  else
    mma_commit(bar);
}

// A tensor map that an earlier kernel wrote: before this thread's first copy by it.
__device__ __forceinline__ void acquire_map(const CUtensorMap* map) {
  asm volatile("fence.proxy.tensormap::generic.acquire.gpu [%0], 128;" ::"l"(map) : "memory");
}

// Store of a shared-memory box at (x, y, z), elements outside the tensor left
// out; tracked as a bulk group of this thread.
__device__ __forceinline__ void store_3d(const void* tmap, uint32_t src, int32_t x, int32_t y,
                                         int32_t z) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
                   reinterpret_cast<uint64_t>(tmap)),
               "r"(x), "r"(y), "r"(z), "r"(src)
               : "memory");
}

// Wait until at most N committed store groups still read shared memory.
template <int N>
__device__ __forceinline__ void bulk_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}

// 16 lanes x 32 columns as 16 x 8 fragments: of columns 8 i .. 8 i + 7, thread
// t receives lane t / 4, columns 2 (t % 4) and + 1 in r[4 i], r[4 i + 1], and
// lane t / 4 + 8 in r[4 i + 2], r[4 i + 3].
__device__ __forceinline__ void tmem_ld_16x256b_x4(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}

// Four 8 x 8 16-bit matrices, each stored transposed: lane 8 m + i gives the
// address of the 16-byte row that takes column i of matrix m.
__device__ __forceinline__ void stmatrix_x4_trans(uint32_t addr, uint32_t a, uint32_t b, uint32_t c,
                                                  uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr),
               "r"(a), "r"(b), "r"(c), "r"(d)
               : "memory");
}

// ---------------------------------------------------------------- schedule
// Row tiles of an expert with m D rows, and their common width.
template <int QT>
__device__ __forceinline__ int row_tiles(int m) {
  return (m + QT - 1) / QT;
}
__device__ __forceinline__ int tile_width(int m, int tiles) {
  return ((m + tiles - 1) / tiles + 31) & ~31;
}

// Rows of expert e; offsets that decrease or leave [0, R] bound none.
__device__ __forceinline__ int rows_of(const GroupedParams& p, const int* lo, int e) {
  return lo[e] < 0 || lo[e + 1] < lo[e] || lo[e + 1] > p.R ? 0 : lo[e + 1] - lo[e];
}

// K slices of a sum over len; an empty one counts as a slice without MMAs, so
// that its zeros (or C) are stored like any tile.
template <int SLICE = BK>
__device__ __forceinline__ int slices_of(int len) {
  return max(1, (len + SLICE - 1) / SLICE);
}

// A piece of work: a tile of D and the range [k, kend) of its sum.
struct alignas(16) Piece {
  int e, f0;         // expert, first feature
  int q0, nq;        // first D row (rows: of all rows; grad: of the expert's K) and how many
  int base, k, kend; // the sum's first row (grad) and this piece's range of it
  int pieces, first; // pieces of the tile and the unit that has its first
  int slot;          // partial sums: 1 for a tile's first piece, 0 for a later one
  int more;          // 0: the end of the work
};

// The work of unit c of `units`, in slices of SLICE values of K; a tile is split
// where that gains GAIN slices of 64.  prefix[e]: rows form, row tiles of the
// experts before e; grad, K slices of one tile of each of them.
template <int CG, int QT, int SLICE = BK, int GAIN = SPLIT_GAIN>
struct Schedule {
  const GroupedParams& p;
  const int* lo;      // [E + 1] offsets
  const int* prefix;  // [E + 1]
  int c, units;
  int ft, tiles_e, kb;      // feature tiles; grad: tiles of an expert; rows: slices of a tile
  int tiles, whole;         // all tiles; how many are dealt whole, round-robin
  int runs;
  int64_t s0, len;          // slices before the runs, and in them
  int i;                    // whole tiles taken
  int64_t at, end;          // this unit's run

  __device__ __forceinline__ Schedule(const GroupedParams& p_, const int* lo_, const int* prefix_,
                                      int c_, int units_)
      : p(p_), lo(lo_), prefix(prefix_), c(c_), units(units_) {
    ft = (p.N + FT * CG - 1) / (FT * CG);
    tiles_e = row_tiles<QT>(p.K) * ft;
    kb = slices_of<SLICE>(p.K);
    tiles = p.grad ? p.E * tiles_e : prefix[p.E] * ft;
    const int waves = tiles / units;
    const int64_t all = p.grad ? static_cast<int64_t>(prefix[p.E]) * tiles_e
                               : static_cast<int64_t>(tiles) * kb;
    // whole tiles take waves + 1 tiles of the busiest unit's time, equal runs
    // all / units slices
    const int64_t tile_kb = tiles > 0 ? all / tiles : 0;
    const int64_t gain = (waves + 1) * tile_kb - all / units;
    const bool split =
        tiles % units != 0 &&
        gain >= (CG == 2 && waves == 0 ? 3 * GAIN : GAIN) * BK / SLICE;
    whole = !split ? tiles : (waves > 1 ? waves - 1 : 0) * units;
    s0 = p.grad ? slices_before(whole) : static_cast<int64_t>(whole) * kb;
    len = all - s0;
    const int64_t most = min(static_cast<int64_t>(units), len * SLICE / (MIN_RUN * BK));
    runs = static_cast<int>(max(static_cast<int64_t>(min(tiles - whole, units)), most));
    i = 0;
    at = c < runs ? len * c / runs : 0;
    end = c < runs ? len * (c + 1) / runs : 0;
  }

  // grad: slices of all tiles before tile t
  __device__ __forceinline__ int64_t slices_before(int t) const {
    const int e = t / tiles_e;
    if (e >= p.E) return static_cast<int64_t>(prefix[p.E]) * tiles_e;
    return static_cast<int64_t>(prefix[e]) * tiles_e +
           static_cast<int64_t>(t - e * tiles_e) * (prefix[e + 1] - prefix[e]);
  }

  // The e with prefix[e] * scale <= v < prefix[e + 1] * scale.
  __device__ __forceinline__ int find(int64_t v, int scale) const {
    int a = 0, b = p.E;
    while (b - a > 1) {
      const int m = (a + b) >> 1;
      if (static_cast<int64_t>(prefix[m]) * scale <= v)
        a = m;
      else
        b = m;
    }
    return a;
  }

  __device__ __forceinline__ void place(Piece& x, int e, int tile_in_e) const {
    const int rows = rows_of(p, lo, e);
    const int m = p.grad ? p.K : rows;
    const int rt = row_tiles<QT>(m), w = tile_width(m, rt);
    int64_t ri, fi;
    raster_tile(tile_in_e, rt, ft, RASTER, ri, fi);
    const int q = static_cast<int>(ri) * w;
    x.e = e;
    x.f0 = static_cast<int>(fi) * FT * CG;
    x.nq = min(w, m - q);
    x.q0 = p.grad ? q : lo[e] + q;
    x.base = p.grad ? lo[e] : 0;
    x.kend = p.grad ? rows : p.K;
  }

  __device__ __forceinline__ bool next(Piece& x) {
    const int64_t t = c + static_cast<int64_t>(i) * units;
    if (t < whole) {
      ++i;
      const int e = p.grad ? static_cast<int>(t) / tiles_e : find(t, ft);
      place(x, e, static_cast<int>(t) - (p.grad ? e * tiles_e : prefix[e] * ft));
      x.k = 0;
      x.pieces = 1;
      x.first = c;
      x.slot = 0;
      return true;
    }
    if (at >= end) return false;
    const int64_t s = s0 + at;
    int64_t tile_s;  // the tile's first slice
    int n;           // its slices
    if (p.grad) {
      const int e = find(s, tiles_e);
      n = prefix[e + 1] - prefix[e];
      const int64_t before = static_cast<int64_t>(prefix[e]) * tiles_e;
      const int j = static_cast<int>((s - before) / n);
      tile_s = before + static_cast<int64_t>(j) * n;
      place(x, e, j);
    } else {
      n = kb;
      const int64_t tile = s / kb;
      tile_s = tile * kb;
      const int e = find(tile, ft);
      place(x, e, static_cast<int>(tile) - prefix[e] * ft);
    }
    const int64_t stop = min(end, tile_s - s0 + n);
    x.k = static_cast<int>(s - tile_s) * SLICE;
    x.kend = min(x.kend, static_cast<int>(stop + s0 - tile_s) * SLICE);
    const int64_t r0 = tile_s - s0, r1 = r0 + n - 1;
    x.first = static_cast<int>(((r0 + 1) * runs - 1) / len);
    x.pieces = static_cast<int>(((r1 + 1) * runs - 1) / len) - x.first + 1;
    x.slot = c == x.first ? 1 : 0;
    at = stop;
    return true;
  }
};

// ---------------------------------------------------------------- element types
template <int DT>
__device__ __forceinline__ float load_c(const void* c, long long i) {
  if constexpr (DT == T_F32) return static_cast<const float*>(c)[i];
  if constexpr (DT == T_BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(c)[i]);
  return __half2float(static_cast<const __half*>(c)[i]);
}
template <int DT>
__device__ __forceinline__ void store_d(void* d, long long i, float v) {
  if constexpr (DT == T_F32)
    static_cast<float*>(d)[i] = v;
  else if constexpr (DT == T_BF16)
    static_cast<__nv_bfloat16*>(d)[i] = __float2bfloat16_rn(v);
  else
    static_cast<__half*>(d)[i] = __float2half_rn(v);
}
template <int DT>
__device__ __forceinline__ uint32_t pack2(uint32_t lo, uint32_t hi) {
  if constexpr (DT == T_BF16) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(__uint_as_float(lo), __uint_as_float(hi));
    return *reinterpret_cast<const uint32_t*>(&v);
  } else {
    const __half2 v = __floats2half2_rn(__uint_as_float(lo), __uint_as_float(hi));
    return *reinterpret_cast<const uint32_t*>(&v);
  }
}

}  // namespace

}  // namespace gb300
