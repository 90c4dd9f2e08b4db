// grouped.cu -- matrix products grouped by expert over ragged row groups.
//
//   rows:  D[r,n]   = sum_k A[r,k] B_e[k,n] (+ C)         for the rows r of e
//   grad:  D_e[k,n] = sum over e's rows r of A[r,k] B[r,n] (+ C)
//
// tcgen05 with D's columns ("features") as the M dimension, 128 to a CTA,
// and D's rows as the N dimension.  The M of an MMA is fixed while its N is
// any multiple of 32 up to 256, so the ragged side goes to N: a group of m
// rows is cut into ceil(m / QT) tiles of equal width and costs about m rows
// of tensor time, not m rounded up to a tile; a decode step's one or two rows
// cost a 32-wide MMA while the weights stream.
//
// Two forms of one kernel:
//   wide    CTA pairs (cta_group::2), 256 features x up to 256 rows; each CTA
//           stages its 128 features and half of the rows, five 32 KB stages
//           (a sixth queued more loads in front of D's stores: 247 us against
//           239 for 32 x 2048 x 4096 gradients of 512 rows).  Bound by the
//           tensor pipe.
//   narrow  single CTAs, 128 features x up to 64 rows, eight 24 KB stages: for
//           groups of few rows, where reading the weights is the bound and
//           bytes in flight count.
//
// Every CTA reads the offsets and counts the row tiles of each expert into a
// prefix sum in shared memory, from which any tile or K slice finds its
// expert by bisection: no host knowledge of the groups, one launch.  Tiles
// are dealt round-robin; what would be a partial last wave (with one full
// wave before it) is dealt as equal runs of K slices instead.  The pieces of
// a tile that several units then share leave fp32 partial sums, and whichever
// of them finishes last adds them up in K order and stores D: no unit waits
// for another, and the result does not depend on who is last.
//
// Nothing of another expert enters a sum, not even as 0 * NaN: rows past a
// group's end are columns of the accumulator that are not stored (rows), and
// K past its end is read as zeros on both sides because the tensor maps end
// there (an N-contiguous B gets a dimension per expert).  In grad the sum
// itself is ragged: a small kernel before this one writes, per expert, copies
// of both operands' tensor maps whose rows end where the group does, so that
// rows past it are read as zeros too.  (Overwriting them with zeros in shared
// memory instead put the clearing, and the odd CTA's word that it had been
// done, between the last copy and the last MMA of every tile: 1.6 us a tile,
// 338 us against 254 for 32 experts of 513 and of 528 rows, 2048 x 4096.)
//
// Measured (one GB300, bf16): 32768 rows x 4096 over 32 experts of 4096 x 4096
// 625 us in the first 60 calls (1759 TFLOP/s, tensor-bound), 725 us after
// seconds of them (1517 TFLOP/s, SM clock 1.41 GHz under the 1400 W cap; a
// cuBLAS product loses as much); with an N-contiguous B 681, with fp32 D 707
// against 640 in the same run; weight gradients of 16384 rows, 32 of 2048 x
// 4096, 229 and 241 us (1200, 1140 TFLOP/s; 174 without D's stores, which take
// the same road as the next tile's operands: 537 MB of D); 64 rows over 48 of
// 64 experts of 4096 x 2048 126 us (6.4 TB/s of weights); 1000 rows, 1000 x
// 1000 over 7 of 8 experts 11.5-13.5 us (launch, first loads and epilogue, 168
// tiles on 152 SMs).  C and fp32 D are read and stored by the threads, a row of
// D at a time: the first case with C takes 1916 us, the gradients into fp32 D
// 418, and added up there (C = D) 3217.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "grouped.cuh"

namespace gb300 {

namespace {

constexpr uint32_t F_BYTES = FT * BK * 2;
// warp 0: TMA loads, 1: MMA issue, 2-9: epilogue (two groups of four, taking
// 32-row chunks of a tile in turn), 10: schedule
constexpr int GROUPED_THREADS = 352;

template <int CG, int QT, int STAGES>
struct Cfg {
  // Buffers of an epilogue group: D's stores wait their turn behind the loads.
  static constexpr int BUFS = CG == 2 ? 2 : 1;
  static constexpr uint32_t X_BYTES = (QT / CG) * BK * 2;
  static constexpr uint32_t STAGE_BYTES = F_BYTES + X_BYTES;
  static constexpr uint32_t TMEM_COLS = 2 * QT;
  static constexpr uint32_t BAR_BYTES = 768;  // barriers, flags, queue of pieces
  static constexpr uint32_t SMEM = 1024 + STAGES * STAGE_BYTES + 2 * BUFS * EPI_BYTES + BAR_BYTES +
                                   4 * (2 * GEMM_MAX_EXPERTS + 2);
  static_assert(SMEM <= 227 * 1024, "shared memory of a CTA");
};

// ---------------------------------------------------------------- kernel
// SCALED (rows form, no C): D[r, f] times x_scales[r] and the expert's w_scales[f],
// two multiplications of the fp32 sums on their way to the store (8192 x 8192 x
// 8192 548 us, as without).
template <int CG, int QT, int STAGES, int DT, bool SCALED>
__global__ void __launch_bounds__(GROUPED_THREADS, 1)
    grouped_kernel(const __grid_constant__ CUtensorMap tmF, const __grid_constant__ CUtensorMap tmX128,
                   const __grid_constant__ CUtensorMap tmX32,
                   const __grid_constant__ CUtensorMap tmD, const GroupedParams p) {
  using C = Cfg<CG, QT, STAGES>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* const smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* const sF = smem;
  uint8_t* const sX = smem + STAGES * F_BYTES;
  uint8_t* const sE = sX + STAGES * C::X_BYTES;  // epilogue: BUFS buffers a group
  uint64_t* const bars = reinterpret_cast<uint64_t*>(sE + 2 * C::BUFS * EPI_BYTES);
  constexpr int NBARS = 2 * STAGES + 5 + 2 * QUEUE;
  uint32_t* const tmem_holder = reinterpret_cast<uint32_t*>(bars + NBARS);
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  volatile int* const ep_go = abort_flag + 1;  // two, taken in turn
  volatile int* const ep_last = abort_flag + 3;
  Piece* const queue = reinterpret_cast<Piece*>(reinterpret_cast<uint8_t*>(bars) + 512);
  static_assert(8 * NBARS + 20 <= 512 && 512 + QUEUE * sizeof(Piece) <= C::BAR_BYTES, "layout");
  int* const lo = reinterpret_cast<int*>(reinterpret_cast<uint8_t*>(bars) + C::BAR_BYTES);
  int* const prefix = lo + p.E + 1;

  const uint32_t bar0 = smem_u32(bars);
  auto full = [&](uint32_t s) { return bar0 + 8u * s; };
  auto empty = [&](uint32_t s) { return bar0 + 8u * (STAGES + s); };
  auto acc_full = [&](uint32_t b) { return bar0 + 8u * (2 * STAGES + b); };
  auto acc_empty = [&](uint32_t b) { return bar0 + 8u * (2 * STAGES + 2 + b); };
  const uint32_t done_bar = bar0 + 8u * (2 * STAGES + 4);
  auto q_full = [&](uint32_t i) { return bar0 + 8u * (2 * STAGES + 5 + i); };
  auto q_empty = [&](uint32_t i) { return bar0 + 8u * (2 * STAGES + 5 + QUEUE + i); };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = CG == 2 ? cluster_ctarank() : 0u;
  const bool leader = rank == 0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    for (int i = 0; i < QUEUE; ++i) {
      mbar_init(q_full(i), 1);
      mbar_init(q_empty(i), 2 + EPI_WARPS);  // one arrival per warp that reads a piece
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(acc_full(b), 1);
      mbar_init(acc_empty(b), EPI_WARPS * CG);
    }
    mbar_init(done_bar, 1);
    *abort_flag = 0;
    fence_mbar_init();
    fence_proxy_async_smem();
  }
  if (warp == 0 && lane == 0) {
    if (!p.grad && p.K > 0) {  // the maps of operands that are not read are not made
      tma_prefetch_desc(&tmF);
      tma_prefetch_desc(&tmX128);
      tma_prefetch_desc(&tmX32);
    }
    if (p.d_tma) tma_prefetch_desc(&tmD);
  }
  if (warp == 1) {
    if constexpr (CG == 2) {
      tmem_alloc_pair(smem_u32(tmem_holder), C::TMEM_COLS);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(smem_u32(tmem_holder), C::TMEM_COLS);
      tmem_relinquish();
    }
  }
  pdl_wait();
  pdl_trigger();
  for (int e = threadIdx.x; e <= p.E; e += GROUPED_THREADS) {
    if constexpr (SCALED) {  // without offsets all rows are the one expert's
      if (!p.offsets) {
        lo[e] = e * p.R;
        continue;
      }
    }
    lo[e] = p.offsets[e];
    if (e < p.E) expert_rows(p.offsets, e, p.R, p.status);
  }
  __syncthreads();
  if (warp == 2) {  // the prefix: each lane a run of experts, then a warp scan
    auto count = [&](int e) {
      const int rows = rows_of(p, lo, e);
      return p.grad ? slices_of(rows) : row_tiles<QT>(rows);
    };
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
  tc_fence_before();
  __syncthreads();
  if constexpr (CG == 2) cluster_sync_all();  // both CTAs' barriers exist
  tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;
  const uint64_t tmo = p.timeout_ns;
  // The next piece of this CTA's work, taken by one warp for itself; false at
  // its end or after a timeout.
  uint32_t q_at = 0, q_ph = 0;
  auto next_piece = [&](Piece& x) {
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

  if (warp == 10) {
    // ------------------------------------------------------------ schedule (each CTA)
    // A piece costs a few hundred instructions (bisection, divisions); taken
    // by the MMA warp itself they held the tensor pipe up at every tile.
    Schedule<CG, QT> work(p, lo, prefix, blockIdx.x / CG, gridDim.x / CG);
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
    // ------------------------------------------------------------ TMA producer (each CTA)
    // The slice loop is kept tight, one copy of it per kind of operand: at
    // 512 tensor cycles a slice, the 650 that a general loop took to issue
    // one (branches and box loops inside) set the speed of the whole kernel.
    uint32_t it = 0, s = 0, ph = 0;
    int mapped = -1;  // grad: the expert whose tensor maps have been acquired
    bool stop = false, skipped = false;
    const bool skip = leader && ((p.debug_flags & DBG_SKIP_FIRST_FILL) ||
                                 ((p.debug_flags & DBG_SKIP_ONE_FILL) && blockIdx.x < CG));
    const uint32_t sF0 = smem_u32(sF), sX0 = smem_u32(sX);
    const uint32_t full0 = CG == 2 ? map_shared_rank(full(0), 0) : full(0);
    while (next_piece(x)) {
      if (elect_one() && !stop) {
        const int half = ((x.nq + 31) & ~31) / CG;  // this CTA's rows of the tile
        const int q0 = x.q0 + static_cast<int>(rank) * half, f0 = x.f0 + static_cast<int>(rank) * FT;
        const bool big = half > 64;
        const int boxes = p.grad ? (half + 63) / 64 : (big ? 1 : (half + 31) / 32);
        const uint32_t bytes = F_BYTES + boxes * (p.grad ? 8192u : (big ? 16384u : 4096u));
        const uint32_t both = CG * bytes;
        const int frow = x.e * p.N + f0;
        auto slices = [&](auto copies) {
          for (int k = x.k; k < x.kend; k += BK) {
            if (!bounded_wait(empty(s), ph ^ 1u, abort_flag, p.status, STATUS_TIMEOUT, tmo)) {
              stop = true;
              return;
            }
            if (it == 0 && skip) {
              skipped = true;  // test hook: the MMA's wait on the first stage expires
            } else {
              if (leader) mbar_arrive_expect_tx(full(s), both);
              copies(k, sF0 + s * F_BYTES, sX0 + s * C::X_BYTES, full0 + 8u * s);
            }
            ++it;
            if (++s == STAGES) {
              s = 0;
              ph ^= 1u;
            }
          }
        };
        const CUtensorMap* const mf = p.maps + x.e;  // grad: the maps that end with the group
        const CUtensorMap* const mx = mf + p.E;
        if (p.grad && x.k < x.kend && mapped != x.e) {
          acquire_map(mf);
          acquire_map(mx);
          mapped = x.e;
        }
        auto grad_copies = [&](int k, uint32_t fd, uint32_t xd, uint32_t bar) {
          const int r = x.base + k;
          load_2d<CG>(fd, mf, f0, r, bar);
          load_2d<CG>(fd + 8192u, mf, f0 + 64, r, bar);
          load_2d<CG>(xd, mx, q0, r, bar);
          if (boxes > 1) load_2d<CG>(xd + 8192u, mx, q0 + 64, r, bar);
        };
        auto f_copies = [&](int k, uint32_t fd, uint32_t bar) {  // N-contiguous B
          load_3d<CG>(fd, &tmF, f0, k, x.e, bar);
          load_3d<CG>(fd + 8192u, &tmF, f0 + 64, k, x.e, bar);
        };
        auto x_copies = [&](int k, uint32_t xd, uint32_t bar) {  // up to 64 rows
          load_2d<CG>(xd, &tmX32, k, q0, bar);
          if (boxes > 1) load_2d<CG>(xd + 4096u, &tmX32, k, q0 + 32, bar);
        };
        if (p.grad) {
          slices(grad_copies);
        } else if (p.f_mn && big) {
          slices([&](int k, uint32_t fd, uint32_t xd, uint32_t bar) {
            f_copies(k, fd, bar);
            load_2d<CG>(xd, &tmX128, k, q0, bar);
          });
        } else if (p.f_mn) {
          slices([&](int k, uint32_t fd, uint32_t xd, uint32_t bar) {
            f_copies(k, fd, bar);
            x_copies(k, xd, bar);
          });
        } else if (big) {
          slices([&](int k, uint32_t fd, uint32_t xd, uint32_t bar) {
            load_2d<CG>(fd, &tmF, k, frow, bar);
            load_2d<CG>(xd, &tmX128, k, q0, bar);
          });
        } else {
          slices([&](int k, uint32_t fd, uint32_t xd, uint32_t bar) {
            load_2d<CG>(fd, &tmF, k, frow, bar);
            x_copies(k, xd, bar);
          });
        }
      }
      __syncwarp();
    }
    if (elect_one()) {
      // Copies in flight land before the CTA leaves.  The even CTA's barriers
      // count both CTAs' (after giving up, the odd CTA gives its own time).
      if (leader) {
        for (uint32_t j = it > STAGES ? it - STAGES : 0; j < it; ++j) {
          if (skipped && j == 0) continue;
          drain_wait(full(j % STAGES), (j / STAGES) & 1u, 200000000ull);
        }
      } else if (*abort_flag) {
        const uint64_t t0 = global_timer_ns();
        while (global_timer_ns() - t0 < 1000000ull) __nanosleep(1000);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer (even CTA)
    const uint32_t f_lo0 = sdesc_lo(smem_u32(sF), p.f_mn ? 8192u : 16u);
    const uint32_t x_lo0 = sdesc_lo(smem_u32(sX), p.grad ? 8192u : 16u);
    const uint32_t dhi = sdesc_hi_sw128(1024u);
    // K steps of a slice, in 16-byte units: 32 bytes along a K-major row, 16
    // rows of an MN-major tile
    const uint32_t f_step = p.f_mn ? 128u : 2u, x_step = p.grad ? 128u : 2u;
    const uint32_t f_off[4] = {0u, f_step, 2 * f_step, 3 * f_step};
    const uint32_t x_off[4] = {0u, x_step, 2 * x_step, 3 * x_step};
    uint32_t s = 0, ph = 0, acc_it = 0;
    bool ok = true;
    while (next_piece(x)) {
      if (elect_one() && leader && ok && x.k < x.kend) {
        const uint32_t buf = acc_it & 1u;
        const uint32_t d_tmem = tmem_base + buf * QT;
        const uint32_t idesc = p.idesc | (static_cast<uint32_t>(((x.nq + 31) & ~31) >> 3) << 17);
        ok = bounded_wait(acc_empty(buf), ((acc_it >> 1) & 1u) ^ 1u, abort_flag, p.status,
                          STATUS_TIMEOUT, tmo);
        tc_fence_after();
        const int nfull = (x.kend - x.k) / BK;
        uint32_t accumulate = 0;
        for (int i = 0; ok && i < nfull; ++i) {
          ok = bounded_wait(full(s), ph, abort_flag, p.status, STATUS_TIMEOUT, tmo);
          if (!ok) break;
          const uint32_t f_lo = f_lo0 + s * (F_BYTES >> 4), x_lo = x_lo0 + s * (C::X_BYTES >> 4);
#pragma unroll
          for (int c = 0; c < 4; ++c)
            mma<CG>(d_tmem, sdesc(dhi, f_lo + f_off[c]), sdesc(dhi, x_lo + x_off[c]), idesc,
                    accumulate | c);
          accumulate = 1;
          commit<CG>(empty(s));
          if (++s == STAGES) {
            s = 0;
            ph ^= 1u;
          }
        }
        const int left = x.kend - x.k - nfull * BK;  // a last slice that is not whole
        if (ok && left > 0) {
          ok = bounded_wait(full(s), ph, abort_flag, p.status, STATUS_TIMEOUT, tmo);
          if (ok) {
            const uint32_t f_lo = f_lo0 + s * (F_BYTES >> 4), x_lo = x_lo0 + s * (C::X_BYTES >> 4);
            for (int c = 0; c < (left + 15) / 16; ++c)
              mma<CG>(d_tmem, sdesc(dhi, f_lo + c * f_step), sdesc(dhi, x_lo + c * x_step), idesc,
                      accumulate | c);
            commit<CG>(empty(s));
          }
          if (++s == STAGES) {
            s = 0;
            ph ^= 1u;
          }
        }
        if (ok) commit<CG>(acc_full(buf));
        ++acc_it;
      }
      __syncwarp();
    }
    if (elect_one() && leader) {
      commit<CG>(done_bar);
      drain_wait(done_bar, 0, 200000000ull);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ epilogue (each CTA)
    const int q = warp & 3, group = (warp - 2) >> 2;
    const uint32_t lane_base = static_cast<uint32_t>(q * 32) << 16;
    const bool ep_leader = threadIdx.x == 64, group_leader = threadIdx.x == 64 + 128 * group;
    uint32_t acc_it = 0;
    int buffer = 0;  // of the next chunk
    const int unit = blockIdx.x / CG;
    for (uint32_t turn = 0;; turn ^= 1u) {
      const uint32_t buf = acc_it & 1u;
      // One thread decides for all eight warps whether there is a piece and
      // its sums: after a timeout a warp that found the last piece would wait
      // for ever in the barriers below for one that had given up.  (Of the two
      // flags the other is written before the next barrier, this one after it.)
      if (ep_leader) {
        bool go = bounded_wait(q_full(q_at), q_ph, abort_flag, p.status, STATUS_TIMEOUT, tmo);
        if (go && queue[q_at].more && queue[q_at].k < queue[q_at].kend)
          go = bounded_wait(acc_full(buf), (acc_it >> 1) & 1u, abort_flag, p.status,
                            STATUS_TIMEOUT, tmo);
        ep_go[turn] = go ? 1 : 0;
      }
      named_barrier_sync(1, 32 * EPI_WARPS);
      if (!ep_go[turn]) break;
      x = queue[q_at];
      __syncwarp();
      if (lane == 0) mbar_arrive(q_empty(q_at));
      if (++q_at == QUEUE) {
        q_at = 0;
        q_ph ^= 1u;
      }
      if (!x.more) break;
      const bool sum = x.k < x.kend;
      if (sum) tc_fence_after();
      auto release = [&] {  // the accumulator has been read
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if constexpr (CG == 2)
            mbar_arrive_cluster(map_shared_rank(acc_empty(buf), 0));
          else
            mbar_arrive(acc_empty(buf));
        }
      };
      const int f = x.f0 + static_cast<int>(rank) * FT + q * 32 + lane;
      const long long row0 = p.grad ? static_cast<long long>(x.e) * p.K + x.q0 : x.q0;
      auto f_scale = [&](int i) {
        return i < p.N ? p.w_scales[static_cast<long long>(x.e) * p.N + i] : 0.f;
      };
      auto r_scale = [&](int i) { return i < x.nq ? p.x_scales[x.q0 + i] : 0.f; };
      const uint32_t taddr = tmem_base + lane_base + buf * QT;
      // This warp's last chunk of the tile; a tile of one chunk leaves the
      // second group without any.
      const int c_first = 32 * group;
      auto c_last = [&](int c) { return c + 64 >= x.nq; };
      if (sum && c_first >= x.nq) release();
      // 16-bit D with 16-byte rows and no C leaves through shared memory, 32
      // rows x 128 features at a time: a group's four warps put their features
      // side by side (two boxes of 64 features, unit u of row r at u ^ r % 8,
      // which is the TMA's swizzle and spares bank conflicts) and one thread
      // stores the boxes by TMA.  The box that a group of rows ends in (rows
      // form), or an N off the 16-byte grid, is stored by the threads.
      const bool staged_store = DT != T_F32 && p.d_vec && !p.C;
      const uint32_t gbar = 2 + group;
      auto stage_at = [&](int row, int u) {
        return sE + (C::BUFS * group + buffer) * EPI_BYTES + (u >> 3) * 4096 + row * 128 + (((u & 7) ^ (row & 7)) << 4);
      };
      auto stage_free = [&] {  // the buffer's last chunk has left it
        if (group_leader) bulk_wait_read<C::BUFS - 1>();
        named_barrier_sync(gbar, 128);
      };
      auto copy_out = [&](int c) {  // rows c .. c + 31 of the tile
        const int fc = x.f0 + static_cast<int>(rank) * FT;
        const bool box = p.d_tma && (p.grad || c + 32 <= x.nq);
        if (box) fence_proxy_async_smem();
        named_barrier_sync(gbar, 128);
        if (box) {
          if (group_leader) {
            const uint32_t src = smem_u32(sE + (C::BUFS * group + buffer) * EPI_BYTES);
            const int y = x.q0 + c, z = p.grad ? x.e : 0;
            if (fc < p.N) store_3d(&tmD, src, fc, y, z);
            if (fc + 64 < p.N) store_3d(&tmD, src + 4096u, fc + 64, y, z);
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
        // One bulk group a chunk, empty where the threads stored it: stage_free
        // counts groups, and a chunk without one would let it pass a buffer
        // whose store is still reading.
        if (group_leader) bulk_commit();
        buffer = buffer + 1 == C::BUFS ? 0 : buffer + 1;
      };
      // An empty sum: zeros, 16 bytes a lane, need no staging (gradients of 25
      // experts of 4272 x 2816, 7 of them with a row: 110 us, 206 through it).
      if (!sum && staged_store) {
        const int f8 = x.f0 + static_cast<int>(rank) * FT + 8 * (lane & 15);
        for (int r = 2 * (warp - 2) + (lane >> 4); r < x.nq && f8 < p.N; r += 2 * EPI_WARPS) {
          uint16_t* const d = static_cast<uint16_t*>(p.D) + (row0 + r) * p.ldd + f8;
          if (f8 + 8 <= p.N) {
            *reinterpret_cast<uint4*>(d) = make_uint4(0u, 0u, 0u, 0u);
          } else {
            for (int j = 0; j < p.N - f8; ++j) d[j] = 0;
          }
        }
        continue;
      }
      if (sum && x.pieces == 1 && staged_store) {
        // fragments of 16 features x 8 rows, transposed into rows by stmatrix
        if constexpr (DT != T_F32) {
          float sf[4];  // SCALED: of features 8 i + lane / 4 of the warp's 32
          if constexpr (SCALED) {
#pragma unroll
            for (int i = 0; i < 4; ++i) sf[i] = f_scale(f - lane + 8 * i + (lane >> 2));
          }
#pragma unroll 1
          for (int c = c_first; c < x.nq; c += 64) {
            uint32_t r[32];
            float sr[8];  // and of rows 8 (i / 2) + 2 (lane % 4) + i % 2 of the chunk
            if constexpr (SCALED) {
#pragma unroll
              for (int i = 0; i < 8; ++i)
                sr[i] = r_scale(c + 8 * (i >> 1) + 2 * (lane & 3) + (i & 1));
            }
            tmem_ld_16x256b_x4(taddr + c, r);
            tmem_ld_16x256b_x4(taddr + c + (16u << 16), r + 16);
            tmem_ld_wait();
            if (c_last(c)) release();
            const int m = lane >> 3;
            if constexpr (SCALED) {
#pragma unroll
              for (int i = 0; i < 32; ++i)  // r[16 h + 4 j + 2 b + k]: feature 2 h + b, row 2 j + k
                r[i] = __float_as_uint(__uint_as_float(r[i]) * sr[2 * ((i >> 2) & 3) + (i & 1)] *
                                       sf[2 * (i >> 4) + ((i >> 1) & 1)]);
            }
            stage_free();
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int i = 0; i < 4; i += 2) {
                const uint32_t* const v = r + 16 * h + 4 * i;
                stmatrix_x4_trans(
                    smem_u32(stage_at(8 * (i + (m >> 1)) + (lane & 7), 4 * q + 2 * h + (m & 1))),
                    pack2<DT>(v[0], v[1]), pack2<DT>(v[2], v[3]), pack2<DT>(v[4], v[5]),
                    pack2<DT>(v[6], v[7]));
              }
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
                   p.partial + (static_cast<size_t>(2 * piece_unit + slot) * CG + rank) * (QT * FT)) +
               q * 32 + lane;
      };
      if (x.pieces > 1) {
        // leave the sums, see who is last
        float4* const mine = partial(unit, x.slot);
#pragma unroll 1
        for (int c = c_first; c < x.nq; c += 64) {
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
        named_barrier_sync(1, 32 * EPI_WARPS);
        if (ep_leader) {
          unsigned* const count = p.counters + x.first * CG + rank;
          const bool last = atomicAdd(count, 1u) == static_cast<unsigned>(x.pieces) - 1u;
          if (last) *count = 0u;  // ready for the next call
          __threadfence();
          *ep_last = last ? 1 : 0;
        }
        named_barrier_sync(1, 32 * EPI_WARPS);
        const bool last = *ep_last != 0;
        named_barrier_sync(1, 32 * EPI_WARPS);
        if (!last) {
          if (c_first < x.nq) release();
          ++acc_it;
          continue;
        }
        __threadfence();
      }
#pragma unroll 1
      for (int c = c_first; c < x.nq; c += 64) {
        float v[32];
        if (sum) {
          uint32_t r[32];
          tmem_ld_32x32b_x32(taddr + c, r);
          tmem_ld_wait();
          if (c_last(c)) release();
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(r[j]);
        } else {
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = 0.f;
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
        if constexpr (SCALED) {
          const float s = f_scale(f);
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = v[j] * r_scale(c + j) * s;
        }
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
          if (p.C) {
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (c + j < x.nq) v[j] += load_c<DT>(p.C, (row0 + c + j) * p.ldc + f);
          }
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if (c + j < x.nq) store_d<DT>(p.D, (row0 + c + j) * p.ldd + f, v[j]);
        }
        __syncwarp();
      }
      if (sum) ++acc_it;
    }
    if (group_leader) bulk_wait_all();  // shared memory outlives the stores that read it
  }
  tc_fence_before();
  if constexpr (CG == 2)
    cluster_sync_all();
  else
    __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    if constexpr (CG == 2)
      tmem_dealloc_pair(tmem_base, C::TMEM_COLS);
    else
      tmem_dealloc(tmem_base, C::TMEM_COLS);
  }
}

// ---------------------------------------------------------------- tensor maps of grad
// One warp per expert: copies of the two maps whose second dimension (rows)
// ends where the expert's group does.  (An empty group's are not used.)
__global__ void __launch_bounds__(32)
    group_maps_kernel(const __grid_constant__ CUtensorMap f, const __grid_constant__ CUtensorMap x,
                      const int* offsets, int E, int R, CUtensorMap* maps, uint32_t* status) {
  __shared__ __align__(128) CUtensorMap sm[2];
  const int e = blockIdx.x;
  pdl_wait();
  pdl_trigger();
  const int2 r = expert_rows(offsets, e, R, status);
  if (threadIdx.x < 16) {
    const uint4* const src = reinterpret_cast<const uint4*>(threadIdx.x < 8 ? &f : &x);
    reinterpret_cast<uint4*>(sm)[threadIdx.x] = src[threadIdx.x & 7];
  }
  __syncwarp();
  if (threadIdx.x < 2)
    asm volatile("tensormap.replace.tile.global_dim.shared::cta.b1024.b32 [%0], 1, %1;" ::"r"(
                     smem_u32(sm + threadIdx.x)),
                 "r"(max(r.y, 1))
                 : "memory");
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 2; ++i)
    asm volatile(
        "tensormap.cp_fenceproxy.global.shared::cta.tensormap::generic.release.gpu.sync.aligned "
        "[%0], [%1], 128;" ::"l"(maps + i * E + e),
        "r"(smem_u32(sm + i))
        : "memory");
}

// ---------------------------------------------------------------- launches
constexpr int WIDE_QT = 256, WIDE_STAGES = 5;
constexpr int NARROW_QT = 64, NARROW_STAGES = 8;

template <int CG, int QT, int STAGES>
cudaLaunchConfig_t config(int units, cudaStream_t st, cudaLaunchAttribute* attr) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(units * CG));
  cfg.blockDim = dim3(GROUPED_THREADS);
  cfg.dynamicSmemBytes = Cfg<CG, QT, STAGES>::SMEM;
  cfg.stream = st;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = CG;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = CG == 2 ? 2 : 1;
  return cfg;
}

// Sets the kernel's shared memory limit; how many units run at once.
template <int CG, int QT, int STAGES, int DT, bool SCALED = false>
int prepare(int num_sms) {
  auto* kernel = grouped_kernel<CG, QT, STAGES, DT, SCALED>;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           Cfg<CG, QT, STAGES>::SMEM) != cudaSuccess)
    return 0;
  if (CG == 1) return num_sms;
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg = config<CG, QT, STAGES>(1, nullptr, attr);
  int n = 0;
  return cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) == cudaSuccess ? n : 0;
}

template <int CG, int QT, int STAGES, int DT, bool SCALED = false>
cudaError_t launch(const CUtensorMap& f, const CUtensorMap& x128, const CUtensorMap& x32,
                   const CUtensorMap& d, const GroupedParams& p, int units, cudaStream_t st) {
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg = config<CG, QT, STAGES>(units, st, attr);
  return cudaLaunchKernelEx(&cfg, grouped_kernel<CG, QT, STAGES, DT, SCALED>, f, x128, x32, d, p);
}

template <int DT>
int prepare_typed(bool wide, int num_sms) {
  return wide ? prepare<2, WIDE_QT, WIDE_STAGES, DT>(num_sms)
              : prepare<1, NARROW_QT, NARROW_STAGES, DT>(num_sms);
}
template <int DT>
cudaError_t launch_typed(bool wide, const CUtensorMap& f, const CUtensorMap& x128,
                         const CUtensorMap& x32, const CUtensorMap& d, const GroupedParams& p,
                         int units, cudaStream_t st) {
  return wide ? launch<2, WIDE_QT, WIDE_STAGES, DT>(f, x128, x32, d, p, units, st)
              : launch<1, NARROW_QT, NARROW_STAGES, DT>(f, x128, x32, d, p, units, st);
}

}  // namespace

int prepare_grouped(bool wide, int d_type, int num_sms) {
  return d_type == T_F32    ? prepare_typed<T_F32>(wide, num_sms)
         : d_type == T_BF16 ? prepare_typed<T_BF16>(wide, num_sms)
                            : prepare_typed<T_F16>(wide, num_sms);
}

int prepare_scaled(int d_type, int num_sms) {
  return d_type == T_F32    ? prepare<2, WIDE_QT, WIDE_STAGES, T_F32, true>(num_sms)
         : d_type == T_BF16 ? prepare<2, WIDE_QT, WIDE_STAGES, T_BF16, true>(num_sms)
                            : prepare<2, WIDE_QT, WIDE_STAGES, T_F16, true>(num_sms);
}

cudaError_t launch_scaled(const CUtensorMap& f, const CUtensorMap& x128, const CUtensorMap& x32,
                          const CUtensorMap& d, const GroupedParams& p, int units,
                          cudaStream_t st) {
  return p.d_type == T_F32
             ? launch<2, WIDE_QT, WIDE_STAGES, T_F32, true>(f, x128, x32, d, p, units, st)
         : p.d_type == T_BF16
             ? launch<2, WIDE_QT, WIDE_STAGES, T_BF16, true>(f, x128, x32, d, p, units, st)
             : launch<2, WIDE_QT, WIDE_STAGES, T_F16, true>(f, x128, x32, d, p, units, st);
}

size_t grouped_partial_bytes(bool wide, int units) {
  return sizeof(float) * 2 * units * FT * (wide ? 2 * WIDE_QT : NARROW_QT);
}

cudaError_t launch_grouped(bool wide, const CUtensorMap& f, const CUtensorMap& x128,
                           const CUtensorMap& x32, const CUtensorMap& d, const GroupedParams& p,
                           int units, cudaStream_t st) {
  if (p.grad && p.R > 0) {
    const cudaError_t e = launch_pdl(group_maps_kernel, dim3(p.E), dim3(32), 0, st, f, x128,
                                     p.offsets, p.E, p.R, p.maps, p.status);
    if (e != cudaSuccess) return e;
  }
  return p.d_type == T_F32    ? launch_typed<T_F32>(wide, f, x128, x32, d, p, units, st)
         : p.d_type == T_BF16 ? launch_typed<T_BF16>(wide, f, x128, x32, d, p, units, st)
                              : launch_typed<T_F16>(wide, f, x128, x32, d, p, units, st);
}

}  // namespace gb300
