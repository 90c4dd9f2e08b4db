// i8_tiles.cu -- many rows times weights of 8-bit integers, with a scale for
// each row and each output; dense or grouped by expert.
//
//   D[r,n] = x_scales[r] w_scales[e,n] sum_k X[r,k] W_e[n,k]
//
// sm_103a has no 8-bit integer form of tcgen05.mma, so the integers go through
// the fp16 one, in which they and their products are exact and the fp32 sums
// are up to 2^24.  Schedule, tiles and epilogue are those of grouped.cu's narrow
// form (D's columns as the M dimension, D's rows as N); the weights are not
// widened in memory: they come to shared memory as bytes, converter warps turn
// them into fp16 and leave them in tensor memory, where the MMA reads its A
// operand.  So HBM gives a byte a weight, and shared memory takes one write and
// one read of it.  X, which every feature tile reads again, is widened once into
// the workspace.
//
// A byte b of the sign-flipped word beside 0x64 is the fp16 number 1024 + b:
// one byte permute makes two of them, one packed subtraction of 1152 the values.
//
// A stage goes round once: TMA, converters, MMA, TMA.  Its slot of tensor memory
// goes with it, so that the converters, who see the stage filled, know the slot
// free.  The converters' way through a stage is a chain of latencies (wait,
// load, convert, store, wait, arrive: about 600 cycles of which the instructions
// are a third), so two groups of warps take the stages in turn.  A third group, no
// loads from shared memory at all, halves of a stage a group and waits that spin
// changed the time by less than a twentieth.
//
// Fewer tiles than SMs: clusters of 2 to 8 CTAs take a tile each, a part of K a
// CTA, and add up through distributed shared memory.
//
// Measured (one GB300, us, the floor in brackets; X's widening included): 64 x
// 8192 x 8192 20.5 (10.3), 64 x 4096 x 4096 11.6 (2.6), 512 x 8192 x 8192 55 (35),
// 2048 x 8192 x 8192 185 (141), 1024 rows over 40 of 64 experts of 4096 x 2048 74
// (51).  What bounds it: with few rows the two launches, the first loads and the
// join (9 us around 11.5 of streaming); with many the converters (0.7-0.8 of the
// tensor rate).  From 6144 rows an expert, with tiles enough for all pairs, both
// operands are widened in HBM and go through grouped.cu's pairs instead: 8192 x
// 8192 x 8192 609-626 (564) against 711, 665 after seconds under the power cap.  W
// off the 16-byte grid is copied on each call: 64 x 8192 x 8191 43 (10.3).
// Not faster: X widened here as well (64 x 8192 x 8192 27 by the converters, 38 by
// the epilogue's warps); CTA pairs with the weights in tensor memory (8192^3 911,
// an arrival on the other CTA's barrier takes several times a local one's time).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "grouped.cuh"
#include "i8.cuh"
#include "rows.cuh"

namespace gb300 {

namespace {

constexpr int SLICE = 128;                    // K of a stage: a 128-byte row of W
constexpr uint32_t W_BYTES = FT * SLICE;
constexpr int TILE_EPI_WARPS = 4;
constexpr int CONV_GROUPS = 2;                // of four warps, taking stages in turn
constexpr int X_WARP = 7 + 4 * CONV_GROUPS;
// warp 0: W's loads, 1: MMA issue, 2-5: epilogue, 6: schedule, from 7: converters,
// last: X's loads
constexpr int I8_THREADS = 32 * (X_WARP + 1);

// WS stages of W on their way; XS of X, each with a slot of tensor memory for
// the W that meets it.
template <int QT>
struct Cfg {
  static constexpr int WS = QT == 64 ? 9 : 6, XS = 3;
  static constexpr uint32_t X_SUB = QT * BK * 2;  // 64 values of each row
  static constexpr uint32_t X_BYTES = 2 * X_SUB;
  // Tensor memory: two accumulators, then the slots.
  static constexpr uint32_t SLOT0 = 2 * QT;
  static_assert(SLOT0 + 64 * XS <= 512, "tensor memory");
  static constexpr uint32_t BAR_BYTES = 768;
  static constexpr uint32_t SMEM = 1024 + WS * W_BYTES + XS * X_BYTES + EPI_BYTES + BAR_BYTES +
                                   4 * (2 * GEMM_MAX_EXPERTS + 2);
  static_assert(SMEM <= 227 * 1024, "shared memory of a CTA");
  static_assert(X_SUB % 1024 == 0, "stage alignment");
};

// D[tmem] (+)= A[tmem] * B[smem]: A's rows in the lanes, two 16-bit values of K
// a column.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Bytes 0, 1 (HIGH: 2, 3) of a word whose sign bits are flipped, as fp16.
template <bool HIGH>
__device__ __forceinline__ uint32_t widen_pair(uint32_t flipped) {
  const uint32_t v = __byte_perm(flipped, 0x64646464u, HIGH ? 0x4342 : 0x4140);
  const __half2 d = __hsub2(*reinterpret_cast<const __half2*>(&v),
                            __half2half2(__ushort_as_half(0x6480)));
  return *reinterpret_cast<const uint32_t*>(&d);
}
__device__ __forceinline__ void widen4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  w ^= 0x80808080u;
  lo = widen_pair<false>(w);
  hi = widen_pair<true>(w);
}

// ---------------------------------------------------------------- kernel
// SPLIT: a cluster of `split` CTAs takes one tile, each its part of K, and they
// add their sums up through shared memory; else CTAs take tiles by the schedule.
template <int QT, int DT, bool SPLIT>
__global__ void __launch_bounds__(I8_THREADS, 1)
    i8_tiles_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                    const __grid_constant__ CUtensorMap tmX32,
                    const __grid_constant__ CUtensorMap tmD, const GroupedParams p,
                    const int split) {
  using C = Cfg<QT>;
  constexpr int WS = C::WS, XS = C::XS;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* const smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* const sW = smem;
  uint8_t* const sX = smem + WS * W_BYTES;
  uint8_t* const sE = sX + XS * C::X_BYTES;
  uint64_t* const bars = reinterpret_cast<uint64_t*>(sE + EPI_BYTES);
  constexpr int NBARS = 2 * WS + 3 * XS + 5 + 2 * QUEUE;
  uint32_t* const tmem_holder = reinterpret_cast<uint32_t*>(bars + NBARS);
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  volatile int* const ep_go = abort_flag + 1;  // two, taken in turn
  volatile int* const ep_last = abort_flag + 3;
  Piece* const queue = reinterpret_cast<Piece*>(reinterpret_cast<uint8_t*>(bars) + 512);
  static_assert(8 * NBARS + 20 <= 512 && 512 + QUEUE * sizeof(Piece) <= C::BAR_BYTES, "layout");
  int* const lo = reinterpret_cast<int*>(reinterpret_cast<uint8_t*>(bars) + C::BAR_BYTES);
  int* const prefix = lo + p.E + 1;

  const uint32_t bar0 = smem_u32(bars);
  auto w_full = [&](uint32_t s) { return bar0 + 8u * s; };
  auto w_empty = [&](uint32_t s) { return bar0 + 8u * (WS + s); };
  auto x_full = [&](uint32_t c) { return bar0 + 8u * (2 * WS + c); };
  auto ready = [&](uint32_t c) { return bar0 + 8u * (2 * WS + XS + c); };  // W in the slot
  auto done = [&](uint32_t c) { return bar0 + 8u * (2 * WS + 2 * XS + c); };
  constexpr uint32_t REST = 2 * WS + 3 * XS;
  auto acc_full = [&](uint32_t b) { return bar0 + 8u * (REST + b); };
  auto acc_empty = [&](uint32_t b) { return bar0 + 8u * (REST + 2 + b); };
  const uint32_t end_bar = bar0 + 8u * (REST + 4);
  auto q_full = [&](uint32_t i) { return bar0 + 8u * (REST + 5 + i); };
  auto q_empty = [&](uint32_t i) { return bar0 + 8u * (REST + 5 + QUEUE + i); };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < WS; ++s) {
      mbar_init(w_full(s), 1);
      mbar_init(w_empty(s), 4);  // a converter warp's arrival each
    }
    for (int c = 0; c < XS; ++c) {
      mbar_init(x_full(c), 1);
      mbar_init(ready(c), 4);
      mbar_init(done(c), 1);
    }
    for (int i = 0; i < QUEUE; ++i) {
      mbar_init(q_full(i), 1);
      mbar_init(q_empty(i), 3 + TILE_EPI_WARPS + 4 * CONV_GROUPS);  // a warp's arrival each
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(acc_full(b), 1);
      mbar_init(acc_empty(b), TILE_EPI_WARPS);
    }
    mbar_init(end_bar, 1);
    *abort_flag = 0;
    fence_mbar_init();
    fence_proxy_async_smem();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmW);
    tma_prefetch_desc(&tmX);
    tma_prefetch_desc(&tmX32);
    if (p.d_tma) tma_prefetch_desc(&tmD);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_holder), 512);
    tmem_relinquish();
  }
  if (!p.offsets) {  // one expert has all rows: nothing to read
    if (threadIdx.x == 0) {
      lo[0] = prefix[0] = 0;
      lo[1] = p.R;
      prefix[1] = row_tiles<QT>(p.R);
    }
  } else {
    pdl_wait();
    for (int e = threadIdx.x; e <= p.E; e += I8_THREADS) {
      lo[e] = p.offsets[e];
      if (e < p.E) expert_rows(p.offsets, e, p.R, p.status);
    }
    __syncthreads();
    if (warp == 2) {  // the prefix: each lane a run of experts, then a warp scan
      auto count = [&](int e) { return row_tiles<QT>(rows_of(p, lo, e)); };
      const int len = (p.E + 31) / 32, b = min(p.E, lane * len), e1 = min(p.E, b + len);
      int sum = 0;
      for (int e = b; e < e1; ++e) sum += count(e);
      int inc = sum;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int u = __shfl_up_sync(0xFFFFFFFFu, inc, d);
        if (lane >= d) inc += u;
      }
      int at = inc - sum;
      for (int e = b; e < e1; ++e) {
        prefix[e] = at;
        at += count(e);
      }
      if (lane == 31) prefix[p.E] = inc;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;
  const uint64_t tmo = p.timeout_ns;
  pdl_trigger();
  // The next piece of this CTA's work, taken by one warp for itself; false at
  // its end or after a timeout.
  uint32_t q_at = 0, q_ph = 0;
  const int rank = SPLIT ? static_cast<int>(cluster_ctarank()) : 0;
  bool taken = false;
  auto next_piece = [&](Piece& x) {
    if constexpr (SPLIT) {  // the cluster's tile, and this CTA's slices of it
      const int ft = (p.N + FT - 1) / FT, tile = blockIdx.x / split;
      if (taken || tile >= prefix[p.E] * ft) return false;
      taken = true;
      int a = 0, b = p.E;  // the expert: prefix[a] * ft <= tile < prefix[a + 1] * ft
      while (b - a > 1) {
        const int m = (a + b) >> 1;
        if (prefix[m] * ft <= tile)
          a = m;
        else
          b = m;
      }
      const int rows = rows_of(p, lo, a), rt = prefix[a + 1] - prefix[a], w = tile_width(rows, rt);
      const int t = tile - prefix[a] * ft, q = t % rt * w, slices = slices_of<SLICE>(p.K);
      x.e = a;
      x.f0 = t / rt * FT;
      x.q0 = lo[a] + q;
      x.nq = min(w, rows - q);
      x.k = rank * slices / split * SLICE;
      x.kend = min(p.K, (rank + 1) * slices / split * SLICE);
      return true;
    }
    bool ok = true;
    if (lane == 0)
      ok = bounded_wait(q_full(q_at), q_ph, abort_flag, p.status, STATUS_TIMEOUT, tmo);
    ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
    if (!ok) return false;
    __syncwarp();
    x = queue[q_at];
    __syncwarp();
    if (lane == 0) mbar_arrive(q_empty(q_at));
    if (++q_at == QUEUE) {
      q_at = 0;
      q_ph ^= 1u;
    }
    return x.more != 0;
  };
  Piece x;

  if (warp == 6 && SPLIT) {
    // (each warp finds its one piece itself)
  } else if (warp == 6) {
    // ------------------------------------------------------------ schedule
    // (384 x 4096 x 4096 in 96 tiles of 128 rows: 29.5 us split, 20.2 whole)
    Schedule<1, QT, SLICE, (QT == 128 ? 4 : 2) * SPLIT_GAIN> work(p, lo, prefix, blockIdx.x, gridDim.x);
    if (lane == 0) {
      for (bool more = true; more;) {
        more = work.next(x);
        x.more = more;
        if (!bounded_wait(q_empty(q_at), q_ph ^ 1u, abort_flag, p.status, STATUS_TIMEOUT, tmo)) break;
        queue[q_at] = x;
        mbar_arrive(q_full(q_at));
        if (++q_at == QUEUE) {
          q_at = 0;
          q_ph ^= 1u;
        }
      }
    }
    __syncwarp();
  } else if (warp == 0) {
    // ------------------------------------------------------------ loads of W
    uint32_t it = 0, s = 0, ph = 0;
    bool stop = false, skipped = false;
    const bool skip = (p.debug_flags & DBG_SKIP_FIRST_FILL) ||
                      ((p.debug_flags & DBG_SKIP_ONE_FILL) && blockIdx.x == 0);
    const uint32_t sW0 = smem_u32(sW);
    pdl_wait();
    while (next_piece(x)) {
      if (elect_one() && !stop) {
        const int wrow = x.e * p.N + x.f0;
        for (int k = x.k; k < x.kend; k += SLICE) {
          if (!bounded_wait(w_empty(s), ph ^ 1u, abort_flag, p.status, STATUS_TIMEOUT, tmo)) {
            stop = true;
            break;
          }
          if (it == 0 && skip) {
            skipped = true;  // test hook: the converters' wait on the first stage expires
          } else {
            mbar_arrive_expect_tx(w_full(s), W_BYTES);
            tma_load_2d(sW0 + s * W_BYTES, &tmW, k, wrow, w_full(s));
          }
          ++it;
          if (++s == WS) {
            s = 0;
            ph ^= 1u;
          }
        }
      }
      __syncwarp();
    }
    if (elect_one()) {
      // copies in flight land before the CTA leaves
      for (uint32_t j = it > WS ? it - WS : 0; j < it; ++j)
        if (!(skipped && j == 0)) drain_wait(w_full(j % WS), (j / WS) & 1u, 200000000ull);
    }
    __syncwarp();
  } else if (warp == X_WARP) {
    // ------------------------------------------------------------ loads of X
    uint32_t it = 0, c = 0, ph = 0;
    bool stop = false;
    const uint32_t sX0 = smem_u32(sX);
    pdl_wait();
    while (next_piece(x)) {
      if (elect_one() && !stop) {
        const bool big = x.nq > 32;
        const uint32_t bytes = 2u * (big ? C::X_SUB : 4096u);
        const CUtensorMap* const tm = big ? &tmX : &tmX32;
        for (int k = x.k; k < x.kend; k += SLICE) {
          if (!bounded_wait(done(c), ph ^ 1u, abort_flag, p.status, STATUS_TIMEOUT, tmo)) {
            stop = true;
            break;
          }
          mbar_arrive_expect_tx(x_full(c), bytes);
          tma_load_2d(sX0 + c * C::X_BYTES, tm, k, x.q0, x_full(c));
          tma_load_2d(sX0 + c * C::X_BYTES + C::X_SUB, tm, k + BK, x.q0, x_full(c));
          ++it;
          if (++c == XS) {
            c = 0;
            ph ^= 1u;
          }
        }
      }
      __syncwarp();
    }
    if (elect_one())
      for (uint32_t j = it > XS ? it - XS : 0; j < it; ++j)
        drain_wait(x_full(j % XS), (j / XS) & 1u, 200000000ull);
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    const uint32_t x_lo0 = sdesc_lo(smem_u32(sX), 16u);
    const uint32_t dhi = sdesc_hi_sw128(1024u);
    uint32_t c = 0, ph = 0, acc_it = 0;
    bool ok = true;
    while (next_piece(x)) {
      if (elect_one() && ok && x.k < x.kend) {
        const uint32_t buf = acc_it & 1u;
        const uint32_t d_tmem = tmem_base + buf * QT;
        const uint32_t idesc = p.idesc | (static_cast<uint32_t>(((x.nq + 31) & ~31) >> 3) << 17);
        ok = bounded_wait(acc_empty(buf), ((acc_it >> 1) & 1u) ^ 1u, abort_flag, p.status,
                          STATUS_TIMEOUT, tmo);
        uint32_t accumulate = 0;
        for (int k = x.k; ok && k < x.kend; k += SLICE) {
          ok = bounded_wait(x_full(c), ph, abort_flag, p.status, STATUS_TIMEOUT, tmo) &&
               bounded_wait(ready(c), ph, abort_flag, p.status, STATUS_TIMEOUT, tmo);
          if (!ok) break;
          tc_fence_after();
          const uint32_t a = tmem_base + C::SLOT0 + c * 64u;
          const uint32_t b = x_lo0 + c * (C::X_BYTES >> 4);
          // (values past K are zeros on both sides)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            mma_ts(d_tmem, a + 8u * i, sdesc(dhi, b + 2u * i), idesc, accumulate | i);
          if (x.kend - k > BK)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              mma_ts(d_tmem, a + 32u + 8u * i, sdesc(dhi, b + (C::X_SUB >> 4) + 2u * i), idesc, 1u);
          accumulate = 1;
          mma_commit(done(c));
          if (++c == XS) {
            c = 0;
            ph ^= 1u;
          }
        }
        if (ok) mma_commit(acc_full(buf));
        ++acc_it;
      }
      __syncwarp();
    }
    if (elect_one()) {
      mma_commit(end_bar);
      drain_wait(end_bar, 0, 200000000ull);
    }
    __syncwarp();
  } else if (warp > 6) {
    // ------------------------------------------------------------ converters
    // Lane = weight row = lane of tensor memory, of which a warp reaches its own
    // quarter: 128 bytes of the row as eight 16-byte units (unit u of row r at
    // u ^ r % 8: eight rows fall on all banks).
    const int q = warp & 3, group = (warp - 7) >> 2, row = 32 * q + lane;
    const uint32_t taddr = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + C::SLOT0;
    const uint8_t* const src0 = sW + row * SLICE;
    uint32_t s = 0, ph = 0, c = 0, cph = 0;
    int turn = 0;
    bool ok = true;
    while (next_piece(x)) {
      for (int k = x.k; ok && k < x.kend; k += SLICE) {
        if (turn == group) {
          ok = bounded_wait(w_full(s), ph, abort_flag, p.status, STATUS_TIMEOUT, tmo) &&
               bounded_wait(done(c), cph ^ 1u, abort_flag, p.status, STATUS_TIMEOUT, tmo);
          ok = __all_sync(0xFFFFFFFFu, ok);
          if (!ok) break;
          tc_fence_after();
          const uint8_t* const src = src0 + s * W_BYTES;
          auto convert = [&](int sub) {
            uint32_t v[32];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              const uint4 w = *reinterpret_cast<const uint4*>(
                  src + (((4 * sub + u) ^ (row & 7)) << 4));
              widen4(w.x, v[8 * u], v[8 * u + 1]);
              widen4(w.y, v[8 * u + 2], v[8 * u + 3]);
              widen4(w.z, v[8 * u + 4], v[8 * u + 5]);
              widen4(w.w, v[8 * u + 6], v[8 * u + 7]);
            }
            tmem_st_32x32b_x32(taddr + c * 64u + sub * 32u, v);
          };
          convert(0);
          if (x.kend - k > BK) convert(1);
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(ready(c));
            mbar_arrive(w_empty(s));
          }
        }
        turn = turn + 1 == CONV_GROUPS ? 0 : turn + 1;
        if (++s == WS) {
          s = 0;
          ph ^= 1u;
        }
        if (++c == XS) {
          c = 0;
          cph ^= 1u;
        }
      }
    }
  } else if constexpr (SPLIT) {
    // ------------------------------------------------------------ epilogue: below
  } else {
    // ------------------------------------------------------------ epilogue
    // As in grouped.cu, with the scales: of features one or four a thread, of
    // rows those of the chunk at hand.
    const int q = warp & 3;
    const uint32_t lane_base = static_cast<uint32_t>(q * 32) << 16;
    const bool ep_leader = threadIdx.x == 64;
    uint32_t acc_it = 0;
    const int unit = blockIdx.x;
    pdl_wait();
    for (;;) {
      const uint32_t buf = acc_it & 1u;
      // One thread decides for all four warps whether there is a piece, and
      // then whether it has its sums; the scales of its features and first rows
      // come in between.
      if (ep_leader)
        ep_go[0] = bounded_wait(q_full(q_at), q_ph, abort_flag, p.status, STATUS_TIMEOUT, tmo);
      named_barrier_sync(1, 32 * TILE_EPI_WARPS);
      if (!ep_go[0]) break;
      x = queue[q_at];
      __syncwarp();
      if (lane == 0) mbar_arrive(q_empty(q_at));
      if (++q_at == QUEUE) {
        q_at = 0;
        q_ph ^= 1u;
      }
      if (!x.more) break;
      auto release = [&] {  // the accumulator has been read
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(acc_empty(buf));
      };
      const int f0 = x.f0 + q * 32;  // this warp's features
      const int f = f0 + lane;
      const float* const fs = p.w_scales + static_cast<long long>(x.e) * p.N;
      const float* const rs = p.x_scales + x.q0;  // the tile's rows
      auto f_scale = [&](int i) { return i < p.N ? fs[i] : 0.f; };
      auto r_scale = [&](int i) { return i < x.nq ? rs[i] : 0.f; };
      // of features 8 i + lane / 4 of the warp's 32, and of rows 8 (i / 2) +
      // 2 (lane % 4) + i % 2 of a chunk: as the fragments of the accumulator lie
      float sf[4], sr[8];
      auto load_sr = [&](int c) {
#pragma unroll
        for (int i = 0; i < 8; ++i) sr[i] = r_scale(c + 8 * (i >> 1) + 2 * (lane & 3) + (i & 1));
      };
#pragma unroll
      for (int i = 0; i < 4; ++i) sf[i] = f_scale(f0 + 8 * i + (lane >> 2));
      load_sr(0);
      if (ep_leader)
        ep_go[1] = bounded_wait(acc_full(buf), (acc_it >> 1) & 1u, abort_flag, p.status,
                                STATUS_TIMEOUT, tmo);
      named_barrier_sync(1, 32 * TILE_EPI_WARPS);
      if (!ep_go[1]) break;
      tc_fence_after();
      const long long row0 = x.q0;
      const uint32_t taddr = tmem_base + lane_base + buf * QT;
      auto c_last = [&](int c) { return c + 32 >= x.nq; };
      const bool staged_store = DT != T_F32 && p.d_vec;
      auto stage_at = [&](int row, int u) {
        return sE + (u >> 3) * 4096 + row * 128 + (((u & 7) ^ (row & 7)) << 4);
      };
      auto stage_free = [&] {  // the buffer's last chunk has left it
        if (ep_leader) bulk_wait_read<0>();
        named_barrier_sync(1, 128);
      };
      auto copy_out = [&](int c) {  // rows c .. c + 31 of the tile
        const int fc = x.f0;
        const bool box = p.d_tma && c + 32 <= x.nq;
        if (box) fence_proxy_async_smem();
        named_barrier_sync(1, 128);
        if (box) {
          if (ep_leader) {
            const uint32_t src = smem_u32(sE);
            const int y = x.q0 + c;
            if (fc < p.N) store_3d(&tmD, src, fc, y, 0);
            if (fc + 64 < p.N) store_3d(&tmD, src + 4096u, fc + 64, y, 0);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int row = 8 * q + 2 * i + (lane >> 4), u = lane & 15;
            const int f8 = fc + 8 * u;
            const uint4 v = *reinterpret_cast<const uint4*>(stage_at(row, u));
            if (c + row < x.nq && f8 < p.N) {
              uint16_t* const d = static_cast<uint16_t*>(p.D) + (row0 + c + row) * p.ldd + f8;
              if (f8 + 8 <= p.N) {
                *reinterpret_cast<uint4*>(d) = v;
              } else {
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
                for (int j = 0; j < p.N - f8; ++j)
                  d[j] = static_cast<uint16_t>(w[j >> 1] >> (16 * (j & 1)));
              }
            }
          }
        }
        // one bulk group a chunk, empty where the threads stored it
        if (ep_leader) bulk_commit();
      };
      if (x.pieces == 1 && staged_store) {
        // fragments of 16 features x 8 rows, scaled, and transposed into rows by stmatrix
        if constexpr (DT != T_F32) {
#pragma unroll 1
          for (int c = 0; c < x.nq; c += 32) {
            if (c > 0) load_sr(c);
            uint32_t r[32];
            tmem_ld_16x256b_x4(taddr + c, r);
            tmem_ld_16x256b_x4(taddr + c + (16u << 16), r + 16);
            tmem_ld_wait();
            if (c_last(c)) release();
            const int m = lane >> 3;
            stage_free();
            auto pair = [&](int h, int i, int b) {  // rows 2 (lane % 4), + 1 of fragment i
              const uint32_t* const v = r + 16 * h + 4 * i + 2 * b;
              const float s = sf[2 * h + b];
              return pack2<DT>(__float_as_uint(__uint_as_float(v[0]) * sr[2 * i] * s),
                               __float_as_uint(__uint_as_float(v[1]) * sr[2 * i + 1] * s));
            };
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int i = 0; i < 4; i += 2)
                stmatrix_x4_trans(
                    smem_u32(stage_at(8 * (i + (m >> 1)) + (lane & 7), 4 * q + 2 * h + (m & 1))),
                    pair(h, i, 0), pair(h, i, 1), pair(h, i + 1, 0), pair(h, i + 1, 1));
            copy_out(c);
          }
        }
        ++acc_it;
        continue;
      }
      // Everything else: lane = feature, one D row at a time.  Partial sums of
      // a shared tile: float4 of four D rows of a feature, features adjacent.
      auto partial = [&](int piece_unit, int slot) {
        return reinterpret_cast<float4*>(
                   p.partial + static_cast<size_t>(2 * piece_unit + slot) * (QT * FT)) +
               q * 32 + lane;
      };
      if (x.pieces > 1) {
        // leave the sums, see who is last
        float4* const mine = partial(unit, x.slot);
#pragma unroll 1
        for (int c = 0; c < x.nq; c += 32) {
          uint32_t v[32];
          tmem_ld_32x32b_x32(taddr + c, v);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 8; ++j)
            mine[(c / 4 + j) * FT] =
                make_float4(__uint_as_float(v[4 * j]), __uint_as_float(v[4 * j + 1]),
                            __uint_as_float(v[4 * j + 2]), __uint_as_float(v[4 * j + 3]));
        }
        __threadfence();
        named_barrier_sync(1, 32 * TILE_EPI_WARPS);
        if (ep_leader) {
          unsigned* const count = p.counters + x.first;
          const bool last = atomicAdd(count, 1u) == static_cast<unsigned>(x.pieces) - 1u;
          if (last) *count = 0u;  // ready for the next call
          __threadfence();
          *ep_last = last ? 1 : 0;
        }
        named_barrier_sync(1, 32 * TILE_EPI_WARPS);
        const bool last = *ep_last != 0;
        named_barrier_sync(1, 32 * TILE_EPI_WARPS);
        if (!last) {
          release();
          ++acc_it;
          continue;
        }
        __threadfence();
      }
      const float s = f_scale(f);
#pragma unroll 1
      for (int c = 0; c < x.nq; c += 32) {
        float v[32];
        {
          uint32_t r[32];
          tmem_ld_32x32b_x32(taddr + c, r);
          tmem_ld_wait();
          if (c_last(c)) release();
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(r[j]);
        }
        if (x.pieces > 1) {
          // in K order, this unit's own sums among them: the same bits
          // whoever is last
          float t[32];
#pragma unroll
          for (int j = 0; j < 32; ++j) t[j] = 0.f;
#pragma unroll 1
          for (int i = 0; i < x.pieces; ++i) {
            if (x.first + i == unit) {
#pragma unroll
              for (int j = 0; j < 32; ++j) t[j] += v[j];
              continue;
            }
            const float4* const src = partial(x.first + i, i == 0 ? 1 : 0) + c / 4 * FT;
            float4 w[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) w[j] = __ldcg(src + j * FT);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              t[4 * j] += w[j].x;
              t[4 * j + 1] += w[j].y;
              t[4 * j + 2] += w[j].z;
              t[4 * j + 3] += w[j].w;
            }
          }
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = t[j];
        }
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = v[j] * r_scale(c + j) * s;
        if (staged_store) {
          stage_free();
          if constexpr (DT != T_F32) {
#pragma unroll
            for (int j = 0; j < 32; ++j)
              *reinterpret_cast<uint16_t*>(stage_at(j, 4 * q + (lane >> 3)) + 2 * (lane & 7)) =
                  static_cast<uint16_t>(pack2<DT>(__float_as_uint(v[j]), 0u));
          }
          copy_out(c);
        } else if (f < p.N) {
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if (c + j < x.nq) store_d<DT>(p.D, (row0 + c + j) * p.ldd + f, v[j]);
        }
        __syncwarp();
      }
      ++acc_it;
    }
    if (ep_leader) bulk_wait_read<0>();  // shared memory outlives the stores that read it
  }
  if constexpr (SPLIT) {
    // Each CTA finishes QT / split of the tile's rows and gets the others' sums
    // of them, [CTA][four rows][feature] float4, in what was the stages' shared
    // memory: all MMAs of the cluster are done and all copies have landed once
    // its threads meet.
    const int rows = QT / split, groups = rows / 4 * FT;
    float4* const sums = reinterpret_cast<float4*>(smem);
    taken = false;
    const bool tile = next_piece(x);
    pdl_wait();
    // the scales of this thread's first four outputs, on their way meanwhile
    const int f1 = x.f0 + threadIdx.x % FT, r1 = rank * rows + threadIdx.x / FT * 4;
    float sw = 0.f, sx[4] = {};
    if (tile && f1 < p.N) {
      sw = p.w_scales[static_cast<long long>(x.e) * p.N + f1];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (r1 + j < x.nq) sx[j] = p.x_scales[x.q0 + r1 + j];
    }
    __syncwarp();
    cluster_sync_all();
    tc_fence_after();
    const bool join = tile && *abort_flag == 0;
    if (join && warp >= 2 && warp != 6 && warp != X_WARP) {
      // twelve warps, three to a quarter of tensor memory, in turn over 16 rows
      const int q = warp & 3, part = warp < 6 ? 0 : (warp - 3) >> 2;
      const uint32_t taddr = tmem_base + (static_cast<uint32_t>(q * 32) << 16);
      const uint32_t mine = smem_u32(sums + rank * groups + q * 32 + lane);
#pragma unroll 1
      for (int c = 16 * part; c < x.nq; c += 48) {
        uint32_t v[16];
        tmem_ld_32x32b_x16(taddr + c, v);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int row = c + 4 * j;  // of the tile, of its owner's row % rows
          const uint32_t at = map_shared_rank(mine, row / rows) + row % rows / 4 * (FT * 16);
          asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(v[4 * j]),
                       "r"(v[4 * j + 1]), "r"(v[4 * j + 2]), "r"(v[4 * j + 3])
                       : "memory");
        }
      }
    }
    __syncwarp();
    cluster_sync_all();
    if (join) {
      for (int i = threadIdx.x; i < groups; i += I8_THREADS) {
        const int f = x.f0 + i % FT, r0 = rank * rows + i / FT * 4;
        if (f >= p.N || r0 >= x.nq) continue;
        float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int c = 0; c < split; ++c) {  // in K order
          const float4 v = sums[c * groups + i];
          t.x += v.x;
          t.y += v.y;
          t.z += v.z;
          t.w += v.w;
        }
        const bool first = i == threadIdx.x;
        const float s = first ? sw : p.w_scales[static_cast<long long>(x.e) * p.N + f];
        const float v[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (r0 + j < x.nq)
            store_d<DT>(p.D, static_cast<long long>(x.q0 + r0 + j) * p.ldd + f,
                        v[j] * (first ? sx[j] : p.x_scales[x.q0 + r0 + j]) * s);
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

// ---------------------------------------------------------------- copies of rows
// 16 values an item, as they are or widened to fp16.  A last unit that K ends in is padded with whatever
// follows: the tensor maps end at K.  Up to two jobs a launch (one after the
// other they take 3 us more of 4096 x 4096 x 4096), and two items a thread, one
// after the other (four, all in flight: 5 us more of 8192 x 8192 x 8192).
struct CopyJob {
  const int8_t* src;
  uint8_t* dst;
  long long ld_src, ld_dst, rows;
  int cols, aligned;  // rows of src are 16-byte multiples apart and start so
  bool widen;
  unsigned blocks;
  Deal deal;
};

__global__ void __launch_bounds__(DEAL_THREADS) i8_copy_kernel(const CopyJob first, const CopyJob second) {
  const bool two = blockIdx.x >= first.blocks;
  const CopyJob& job = two ? second : first;
  const Items all = block_items(job.rows, job.deal, blockIdx.x - (two ? first.blocks : 0u));
  pdl_wait();
  pdl_trigger();
  for (uint32_t at0 = threadIdx.x; at0 < all.n; at0 += DEAL_THREADS) {
    const uint32_t at = all.at + at0, r = divide(at, job.deal.lanes);
    const long long row = all.row + r;
    const int k = static_cast<int>(at - r * job.deal.lanes.d) * 16;
    const int8_t* const from = job.src + row * job.ld_src + k;
    const uint4 w = job.aligned ? *reinterpret_cast<const uint4*>(from) : load16_at(from, min(16, job.cols - k));
    uint4* const to = reinterpret_cast<uint4*>(job.dst + (job.widen ? 2 : 1) * (row * job.ld_dst + k));
    if (job.widen) {
      uint4 a, b;
      widen4(w.x, a.x, a.y);
      widen4(w.y, a.z, a.w);
      widen4(w.z, b.x, b.y);
      widen4(w.w, b.z, b.w);
      to[0] = a;
      to[1] = b;
    } else {
      to[0] = w;
    }
  }
}

CopyJob job_of(const I8Copy& c, int num_sms) {
  CopyJob j = {};
  if (c.rows == 0 || c.cols == 0) return j;
  j.src = c.src;
  j.dst = static_cast<uint8_t*>(c.dst);
  j.ld_src = c.ld_src;
  j.ld_dst = c.ld_dst;
  j.rows = c.rows;
  j.cols = c.cols;
  j.widen = c.widen;
  j.aligned = c.cols % 16 == 0 && c.ld_src % 16 == 0 && reinterpret_cast<uintptr_t>(c.src) % 16 == 0;
  dim3 grid;
  j.deal = deal_of(c.rows, (c.cols + 15) / 16, 2, num_sms, grid);
  j.blocks = grid.x;
  return j;
}

// ---------------------------------------------------------------- launches
template <int QT, int DT>
cudaLaunchConfig_t config(int units, int split, cudaStream_t st, cudaLaunchAttribute* attr) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(units * split));
  cfg.blockDim = dim3(I8_THREADS);
  cfg.dynamicSmemBytes = Cfg<QT>::SMEM;
  cfg.stream = st;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = split;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = split > 1 ? 2 : 1;
  return cfg;
}

template <int QT, int DT>
int prepare(int split, int num_sms) {
  auto* const kernel = split > 1 ? i8_tiles_kernel<QT, DT, true> : i8_tiles_kernel<QT, DT, false>;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<QT>::SMEM) !=
      cudaSuccess)
    return 0;
  if (split == 1) return num_sms;
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg = config<QT, DT>(1, split, nullptr, attr);
  int n = 0;
  return cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) == cudaSuccess ? n : 0;
}
template <int QT, int DT>
cudaError_t launch(const CUtensorMap& w, const CUtensorMap& x, const CUtensorMap& x32,
                   const CUtensorMap& d, const GroupedParams& p, int units, int split,
                   cudaStream_t st) {
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg = config<QT, DT>(units, split, st, attr);
  return split > 1 ? cudaLaunchKernelEx(&cfg, i8_tiles_kernel<QT, DT, true>, w, x, x32, d, p, split)
                   : cudaLaunchKernelEx(&cfg, i8_tiles_kernel<QT, DT, false>, w, x, x32, d, p, split);
}

template <int DT>
int prepare_typed(int rows, int split, int num_sms) {
  return rows == 128 ? prepare<128, DT>(split, num_sms) : prepare<64, DT>(split, num_sms);
}
template <int DT>
cudaError_t launch_typed(int rows, const CUtensorMap& w, const CUtensorMap& x,
                         const CUtensorMap& x32, const CUtensorMap& d, const GroupedParams& p,
                         int units, int split, cudaStream_t st) {
  return rows == 128 ? launch<128, DT>(w, x, x32, d, p, units, split, st)
                     : launch<64, DT>(w, x, x32, d, p, units, split, st);
}

}  // namespace

int prepare_i8_tiles(int rows, int d_type, int split, int num_sms) {
  return d_type == T_F32    ? prepare_typed<T_F32>(rows, split, num_sms)
         : d_type == T_BF16 ? prepare_typed<T_BF16>(rows, split, num_sms)
                            : prepare_typed<T_F16>(rows, split, num_sms);
}

size_t i8_tiles_partial_bytes(int rows, int units) {
  return sizeof(float) * 2 * units * FT * rows;
}

cudaError_t launch_i8_tiles(int rows, const CUtensorMap& w, const CUtensorMap& x,
                            const CUtensorMap& x32, const CUtensorMap& d, const GroupedParams& p,
                            int units, int split, cudaStream_t st) {
  return p.d_type == T_F32    ? launch_typed<T_F32>(rows, w, x, x32, d, p, units, split, st)
         : p.d_type == T_BF16 ? launch_typed<T_BF16>(rows, w, x, x32, d, p, units, split, st)
                              : launch_typed<T_F16>(rows, w, x, x32, d, p, units, split, st);
}

cudaError_t launch_i8_copies(const I8Copy& first, const I8Copy& second, int num_sms, cudaStream_t st) {
  const CopyJob a = job_of(first, num_sms), b = job_of(second, num_sms);
  if (a.blocks + b.blocks == 0) return cudaSuccess;
  return launch_pdl(i8_copy_kernel, dim3(a.blocks + b.blocks), dim3(DEAL_THREADS), 0, st, a, b);
}

}  // namespace gb300
