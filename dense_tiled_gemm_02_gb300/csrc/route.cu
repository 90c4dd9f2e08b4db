// route.cu -- token routing: the k largest logits of each token, their
// softmax gates, and the stable sort of the chosen slots by expert.
//
//   g[t,j] = exp(x[t,e_j] - m) / Z,   m = max, Z = sum of exp(x - m) over the
//            chosen logits (normalize) or over all of them
//   dx[t,e_j] = g_j (dg_j - s), s = sum_i g_i dg_i; without normalize every
//            e gets p_e ([e = e_j] dg_j - s), p the softmax over all E
//
// The forward pass must read T x E logits once and write 20 bytes a slot: at
// 32768 x 256, k = 8, fp32, 5.8 us of traffic.  The k rounds of a warp-wide
// maximum bound it, not HBM: 23.7 us (1.6 TB/s), instructions issued in 64% of
// the cycles; the sort takes about 7 us more and the backward pass 8 us (a
// token to a warp, with a trip of its own for its choices, took 11.7), 38.3
// together; by the softmax over all E 33.9 forward and 21.6 backward, where a
// warp reads the rows of its tokens one after the other (4096 x 64, k = 1, whose
// 32 tokens a warp fill 16 blocks: 17.0 us, k = 2: 9.4).  A warp owns a token:
// lane l holds the logits e = 32 i + l as order-preserving 32-bit keys and its
// own largest; a round takes the warp's largest key (one warp reduction) and,
// where several lanes hold it, the lowest expert, and only the winning lane
// looks for its next one.
//
// The sort is a counting sort without atomics on its order, so equal inputs
// give equal outputs: every warp counts a contiguous run of tokens per expert,
// the counts are summed up in slot order, and the second walk over the run
// hands out rows.
// One block does all of it for small calls (one launch); otherwise blocks
// take contiguous tokens and leave their counts, and a second kernel, in which
// every block sums up all of them for itself, hands out the rows.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "moe.h"
#include "ptx.cuh"
#include "tc_launch.h"

namespace gb300 {

namespace {

constexpr uint32_t KEY_NEG_INF = 0x007FFFFFu;  // the key of -inf: not chosen, nor any below
constexpr int ONE_BLOCK_SLOTS = 4096;
constexpr int ONE_BLOCK_TOKENS = 64;
constexpr int TOKEN_STEP = 5;  // least k that the sort walks by tokens
constexpr int RANK_THREADS = 1024;
constexpr int RANK_STRIPS = 16;    // at most so many threads sum up one column of counts
constexpr int RANK_SLOTS = 8192;   // slots whose experts are in shared memory at a time

// fp32 as an unsigned key in the same order, -0 equal to +0, NaN on top (the
// addition gives every NaN as the positive 0x7FFFFFFF).
__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);
  return b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
  return v;
}

// A token's logits as they are in memory; -inf, never chosen, past the last.
template <typename T, int VPL>
__device__ __forceinline__ void load_row(const T* x, int E, int lane, T (&v)[VPL]) {
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int e = 32 * i + lane;
    if (e < E)
      v[i] = x[e];
    else
      narrow(-INFINITY, v[i]);
  }
}
template <typename T, int VPL>
__device__ __forceinline__ void to_keys(const T (&v)[VPL], uint32_t (&key)[VPL]) {
#pragma unroll
  for (int i = 0; i < VPL; ++i) key[i] = order_key(widen(v[i]));
}

// The token's choices: lane j < n (returned) holds the j-th key and expert;
// chosen: the warp's place for them in shared memory.
// A lane keeps its largest two and looks through its keys again only when it
// wins a third time; looking at every win made that search most of the work
// (59 us against 36 for 32768 x 256, k = 8).
template <int VPL>
__device__ __forceinline__ int top_k(const uint32_t (&key)[VPL], int k, int lane, uint2* chosen,
                                     uint32_t& my_key, int& my_expert) {
  uint32_t best, second, taken = 0u;
  int bi, si;
  bool spare;  // second is there
  auto look = [&] {
    best = second = 0u;
    bi = si = 0;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const uint32_t v = (taken >> i) & 1u ? 0u : key[i];
      if (v > best) {
        second = best;
        si = bi;
        best = v;
        bi = i;
      } else if (v > second) {
        second = v;
        si = i;
      }
    }
    spare = true;
  };
  look();
  int n = k;
  for (int j = 0; j < k; ++j) {
    const uint32_t m = __reduce_max_sync(0xFFFFFFFFu, best);
    if (m <= KEY_NEG_INF) {
      n = j;
      break;
    }
    bool mine = best == m;
    const uint32_t holders = __ballot_sync(0xFFFFFFFFu, mine);
    if (holders & (holders - 1u)) {  // equal logits: the lowest expert
      const uint32_t e = mine ? static_cast<uint32_t>(32 * bi + lane) : ~0u;
      mine = __reduce_min_sync(0xFFFFFFFFu, e) == e;
    }
    if (mine) {
      chosen[j] = make_uint2(m, static_cast<uint32_t>(32 * bi + lane));
      taken |= 1u << bi;
      if (spare) {
        best = second;
        bi = si;
        spare = false;
      } else {
        look();
      }
    }
  }
  __syncwarp();
  const uint2 c = lane < n ? chosen[lane] : make_uint2(0u, ~0u);
  __syncwarp();
  my_key = c.x;
  my_expert = static_cast<int>(c.y);
  return n;
}

// Counting sort of the slots of `tokens` tokens (k each) from slot s0 by a
// block's warps.  expert(i) is the expert of the block's i-th slot or -1; cnt:
// [warps][E] in shared memory.  count_slots leaves each warp's counts;
// hand_out_rows walks the same runs, cnt[w][e] then holding the first row of
// warp w's slots of expert e.  A step is one token, whose experts differ, so
// its lanes go their own ways; or 32 slots, where lanes of one expert find
// each other by a match (32768 x 256, k = 8: 42.3 us by tokens against 48.8
// by matches; k = 4: 36.5 against 35.6; k = 2: 33.4 against 29.6).
__device__ __forceinline__ bool by_token(int k) { return k >= TOKEN_STEP; }

template <typename Visit>
__device__ __forceinline__ void walk_run(int tokens, int k, Visit visit) {
  const int warps = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int len = (tokens + warps - 1) / warps;
  const int begin = min(tokens, warp * len) * k, end = min(tokens, (warp + 1) * len) * k;
  const int step = by_token(k) ? k : 32;
  for (int i = begin; i < end; i += step) {
    visit(lane < min(step, end - i) ? i + lane : -1);
    __syncwarp();
  }
}

template <typename ExpertOf>
__device__ __forceinline__ void count_slots(int tokens, int k, int E, int* cnt, ExpertOf expert) {
  const int warps = blockDim.x >> 5, lane = threadIdx.x & 31;
  int* const mine = cnt + (threadIdx.x >> 5) * E;
  for (int i = threadIdx.x; i < warps * E; i += blockDim.x) cnt[i] = 0;
  __syncthreads();
  walk_run(tokens, k, [&](int i) {
    const int e = i >= 0 ? expert(i) : -1;
    if (by_token(k)) {
      if (e >= 0) ++mine[e];
    } else {
      const uint32_t same = __match_any_sync(0xFFFFFFFFu, e);
      if (e >= 0 && lane == __ffs(same) - 1) mine[e] += __popc(same);
    }
  });
  __syncthreads();
}

template <typename ExpertOf>
__device__ __forceinline__ void hand_out_rows(int tokens, int k, int E, int s0, int* cnt,
                                              ExpertOf expert, int* row_slot, int* slot_row) {
  const int lane = threadIdx.x & 31;
  int* const mine = cnt + (threadIdx.x >> 5) * E;
  walk_run(tokens, k, [&](int i) {
    const int e = i >= 0 ? expert(i) : -1;
    int row = -1;
    if (by_token(k)) {
      if (e >= 0) row = mine[e]++;
    } else {
      const uint32_t same = __match_any_sync(0xFFFFFFFFu, e);
      const uint32_t below = same & ((1u << lane) - 1u);
      if (e >= 0) row = mine[e] + __popc(below);
      __syncwarp();
      if (e >= 0 && below == 0u) mine[e] += __popc(same);
    }
    if (row >= 0) row_slot[row] = s0 + i;
    if (i >= 0) slot_row[s0 + i] = row;
  });
}

// Exclusive prefix of v[0..E) into out[0..E], by one warp.
__device__ __forceinline__ void warp_prefix(const int* v, int E, int lane, int* out) {
  const int len = (E + 31) / 32, b = min(E, lane * len), e = min(E, b + len);
  int sum = 0;
  for (int i = b; i < e; ++i) sum += v[i];
  int inc = sum;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int u = __shfl_up_sync(0xFFFFFFFFu, inc, d);
    if (lane >= d) inc += u;
  }
  int at = inc - sum;
  for (int i = b; i < e; ++i) {
    out[i] = at;
    at += v[i];
  }
  if (lane == 31) out[E] = inc;
}

// Shared memory of the route kernel: cnt[warps][E], total[E], first[E + 1] and,
// in the one-block form, the experts of all slots.  (The several-block form
// touches total alone.  With room for no more than that, 32768 x 256, k = 8,
// fp32 took 30.1 us against 29.5, and the other sizes tried the same.)
size_t route_smem(int threads, int E, bool one_block) {
  return sizeof(int) * (static_cast<size_t>(threads / 32) * E + 2 * E + 1) +
         (one_block ? sizeof(short) * ONE_BLOCK_SLOTS : 0);
}

template <int VPL>
__host__ __device__ constexpr int route_threads() {
  return VPL <= 8 ? 1024 : 512;  // registers: the logits of DEPTH + 1 tokens a lane
}
// Tokens of a warp whose logits are on their way.  They stay in their own type
// until they are used: turned into keys at the load they were waited for there.
template <int VPL>
__host__ __device__ constexpr int route_depth() {
  return VPL <= 2 ? 4 : VPL <= 16 ? 2 : 1;
}

template <typename T, int VPL, bool ONE_BLOCK>
__global__ void __launch_bounds__(route_threads<VPL>()) route_kernel(const RouteParams p) {
  extern __shared__ int sm[];
  __shared__ uint2 chosen[route_threads<VPL>() / 32][32];
  const int warps = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int* const cnt = sm;
  int* const total = sm + warps * p.E;
  int* const first = total + p.E;
  short* const slots = reinterpret_cast<short*>(first + p.E + 1);
  const int t0 = blockIdx.x * p.tokens_per_block;
  const int tokens = min(p.T - t0, p.tokens_per_block);
  if (!ONE_BLOCK) {
    for (int e = threadIdx.x; e < p.E; e += blockDim.x) total[e] = 0;
    __syncthreads();
  }
  pdl_wait();
  pdl_trigger();
  const T* const logits = static_cast<const T*>(p.logits) + t0 * p.ld;
  constexpr int DEPTH = route_depth<VPL>();
  T next[DEPTH][VPL];
#pragma unroll
  for (int d = 0; d < DEPTH; ++d)
    if (warp + d * warps < tokens)
      load_row<T, VPL>(logits + (warp + d * warps) * p.ld, p.E, lane, next[d]);
  auto one_token = [&](int t, const uint32_t (&key)[VPL]) {
    float z = 0.f;
    if (!p.normalize) {
      uint32_t m = key[0];
#pragma unroll
      for (int i = 1; i < VPL; ++i) m = max(m, key[i]);
      m = __reduce_max_sync(0xFFFFFFFFu, m);
      const float top = key_value(m);
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        if (key[i] > KEY_NEG_INF) z += expf(key_value(key[i]) - top);
      z = warp_sum(z);
    }
    uint32_t my_key;
    int my_expert;
    const int n = top_k<VPL>(key, p.k, lane, chosen[warp], my_key, my_expert);
    const float top = key_value(__shfl_sync(0xFFFFFFFFu, my_key, 0));
    const float ex = lane < n ? expf(key_value(my_key) - top) : 0.f;
    if (p.normalize) z = warp_sum(ex);
    if (lane < p.k) {
      const int s = (t0 + t) * p.k + lane;
      p.experts[s] = my_expert;
      p.gates[s] = lane < n ? ex / z : 0.f;
      if (ONE_BLOCK)
        slots[s] = static_cast<short>(my_expert);
      else if (my_expert >= 0)
        atomicAdd(&total[my_expert], 1);  // a count: the order does not matter
    }
  };
  for (int t = warp; t < tokens; t += DEPTH * warps) {
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) {
      const int at = t + d * warps, then = at + DEPTH * warps;
      if (at >= tokens) break;
      uint32_t key[VPL];
      to_keys<T, VPL>(next[d], key);
      if (then < tokens) load_row<T, VPL>(logits + then * p.ld, p.E, lane, next[d]);
      one_token(at, key);
    }
  }
  __syncthreads();
  if constexpr (ONE_BLOCK) {
    const int n = p.T * p.k;
    auto expert = [&](int i) { return static_cast<int>(slots[i]); };
    count_slots(p.T, p.k, p.E, cnt, expert);
    for (int e = threadIdx.x; e < p.E; e += blockDim.x) {
      int sum = 0;
      for (int w = 0; w < warps; ++w) sum += cnt[w * p.E + e];
      total[e] = sum;
    }
    __syncthreads();
    if (warp == 0) warp_prefix(total, p.E, lane, first);
    __syncthreads();
    for (int e = threadIdx.x; e <= p.E; e += blockDim.x) {
      int at = first[e];
      p.offsets[e] = at;
      if (e < p.E)
        for (int w = 0; w < warps; ++w) {
          const int c = cnt[w * p.E + e];
          cnt[w * p.E + e] = at;
          at += c;
        }
    }
    __syncthreads();
    hand_out_rows(p.T, p.k, p.E, 0, cnt, expert, p.row_slot, p.slot_row);
    for (int r = first[p.E] + threadIdx.x; r < n; r += blockDim.x) p.row_slot[r] = -1;
  } else {
    for (int e = threadIdx.x; e < p.E; e += blockDim.x) p.hist[blockIdx.x * p.ld_hist + e] = total[e];
  }
}

// Block b hands out the rows of block b's slots.  It sums up the counts of all
// blocks and of those before it (from L2, 16 bytes a thread and load, a column
// of four experts split over up to RANK_STRIPS threads).  That is blocks^2 x E
// counts in all; a last block of the first kernel that did it once for all
// left the others idle for two trips over the counts, and took longer (a call
// 42.3 us against 31.9 at 32768 x 256, k = 8, bf16).  The experts are read
// ahead into
// shared memory: read by each walk, a trip to L2 for every step was most of
// this kernel.
__global__ void __launch_bounds__(RANK_THREADS) route_rank_kernel(const RouteParams p) {
  // cnt[warps][ld_hist], base[ld_hist], total[ld_hist], first[ld_hist + 1], experts
  extern __shared__ __align__(16) int cnt[];
  constexpr int WARPS = RANK_THREADS / 32;
  const int E4 = p.ld_hist / 4, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int* const base = cnt + WARPS * p.ld_hist;
  int* const total = base + p.ld_hist;
  int* const first = total + p.ld_hist;
  short* const slots = reinterpret_cast<short*>(first + p.ld_hist + 1);
  const int t0 = blockIdx.x * p.tokens_per_block, tokens = min(p.T - t0, p.tokens_per_block);
  const int chunk = RANK_SLOTS / p.k;  // tokens
  pdl_wait();
  pdl_trigger();
  auto read_experts = [&](int t) {
    const int s0 = (t0 + t) * p.k, n = min(tokens - t, chunk) * p.k;
#pragma unroll 8
    for (int i = threadIdx.x; i < n; i += RANK_THREADS)
      slots[i] = static_cast<short>(p.experts[s0 + i]);
  };
  const int strips = min(min(RANK_STRIPS, WARPS / 2), RANK_THREADS / E4);
  int4* const before4 = reinterpret_cast<int4*>(cnt);
  int4* const all4 = before4 + strips * E4;
  if (threadIdx.x < strips * E4) {
    const int s = threadIdx.x / E4, c = threadIdx.x - s * E4;
    const int4* const h = reinterpret_cast<const int4*>(p.hist) + c;
    int4 before = make_int4(0, 0, 0, 0), all = before;
#pragma unroll 8
    for (int b = s; b < p.blocks; b += strips) {
      const int4 v = __ldcg(h + static_cast<size_t>(b) * E4);
      all.x += v.x, all.y += v.y, all.z += v.z, all.w += v.w;
      if (b < static_cast<int>(blockIdx.x))
        before.x += v.x, before.y += v.y, before.z += v.z, before.w += v.w;
    }
    before4[threadIdx.x] = before;
    all4[threadIdx.x] = all;
  }
  read_experts(0);
  __syncthreads();
  for (int e = threadIdx.x; e < p.E; e += RANK_THREADS) {
    int before = 0, all = 0;
    for (int s = 0; s < strips; ++s) {
      before += cnt[s * p.ld_hist + e];
      all += cnt[(strips + s) * p.ld_hist + e];
    }
    base[e] = before;
    total[e] = all;
  }
  __syncthreads();
  if (warp == 0) warp_prefix(total, p.E, lane, first);
  __syncthreads();
  for (int e = threadIdx.x; e <= p.E; e += RANK_THREADS) {
    if (e < p.E) base[e] += first[e];
    if (blockIdx.x == 0) p.offsets[e] = first[e];
  }
  auto expert = [&](int i) { return static_cast<int>(slots[i]); };
  for (int t = 0; t < tokens; t += chunk) {
    if (t > 0) {
      __syncthreads();  // the last chunk's walk is over
      read_experts(t);
    }
    const int now = min(tokens - t, chunk);
    count_slots(now, p.k, p.E, cnt, expert);
    for (int e = threadIdx.x; e < p.E; e += RANK_THREADS) {
      int at = base[e];
      for (int w0 = 0; w0 < WARPS; w0 += 8) {
        int c[8];  // read together, as none depends on a store before it
#pragma unroll
        for (int w = 0; w < 8; ++w) c[w] = cnt[(w0 + w) * p.E + e];
#pragma unroll
        for (int w = 0; w < 8; ++w) {
          cnt[(w0 + w) * p.E + e] = at;
          at += c[w];
        }
      }
      base[e] = at;
    }
    __syncthreads();
    hand_out_rows(now, p.k, p.E, (t0 + t) * p.k, cnt, expert, p.row_slot, p.slot_row);
  }
  for (int i = threadIdx.x; i < tokens * p.k; i += RANK_THREADS)
    if (t0 * p.k + i >= first[p.E]) p.row_slot[t0 * p.k + i] = -1;
}

// A warp takes 32 / K tokens together, K the power of two that holds k: lane
// K i + j has choice j of the i-th, so all their choices come in one trip and
// one butterfly sums each token's.  Then it writes their rows whole, one after
// the other, and last all chosen entries (stores of one warp to one address
// stay in order across __syncwarp).  VPL: 0 for normalized gates, where the
// rest of a row is zeros.
template <typename T, int VPL>
__global__ void __launch_bounds__(256, VPL == 0 ? 6 : 1)
    route_backward_kernel(const RouteBackwardParams p) {
  const int lane = threadIdx.x & 31;
  const int K = p.k <= 1 ? 1 : 1 << (32 - __clz(p.k - 1));
  const int per = 32 / K, mine = lane / K, j = lane & (K - 1);
  pdl_wait();
  pdl_trigger();
  // 16-byte zeros where the rows allow it
  constexpr int V = 16 / sizeof(T);
  const bool wide = p.E % V == 0 && p.ld % V == 0 &&
                    (reinterpret_cast<uintptr_t>(p.dlogits) & 15u) == 0;
  T* const dlogits = static_cast<T*>(p.dlogits);
  const long long stride = static_cast<long long>(gridDim.x) * 8 * per;
  for (long long t0 = (blockIdx.x * 8ll + (threadIdx.x >> 5)) * per; t0 < p.T; t0 += stride) {
    const long long t = t0 + mine;
    int chosen = -1;
    float gate = 0.f, dgate = 0.f;
    if (t < p.T && j < p.k) {
      const long long at = t * p.k + j;
      chosen = p.experts[at];
      gate = p.gates[at];
      dgate = p.dgates[at];
    }
    if (chosen < 0 || chosen >= p.E) {
      chosen = -1;
      gate = dgate = 0.f;
    }
    float s = gate * dgate;
    for (int d = K / 2; d > 0; d >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, d);
    for (int q = 0; q < per && t0 + q < p.T; ++q) {
      T* const dx = dlogits + (t0 + q) * p.ld;
      if constexpr (VPL == 0) {
        if (wide) {
          for (int i = V * lane; i < p.E; i += 32 * V)
            *reinterpret_cast<uint4*>(dx + i) = make_uint4(0u, 0u, 0u, 0u);
        } else {
          for (int i = lane; i < p.E; i += 32) narrow(0.f, dx[i]);
        }
      } else {
        const float sum = __shfl_sync(0xFFFFFFFFu, s, q * K);
        uint32_t key[VPL];
        T row[VPL];
        load_row<T, VPL>(static_cast<const T*>(p.logits) + (t0 + q) * p.ld, p.E, lane, row);
        to_keys<T, VPL>(row, key);
        uint32_t m = key[0];
#pragma unroll
        for (int i = 1; i < VPL; ++i) m = max(m, key[i]);
        const float top = key_value(__reduce_max_sync(0xFFFFFFFFu, m));
        float ex[VPL], z = 0.f;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
          ex[i] = key[i] > KEY_NEG_INF ? expf(key_value(key[i]) - top) : 0.f;
          z += ex[i];
        }
        z = warp_sum(z);
#pragma unroll
        for (int i = 0; i < VPL; ++i)
          if (32 * i + lane < p.E)
            narrow(key[i] > KEY_NEG_INF ? -(ex[i] / z) * sum : 0.f, dx[32 * i + lane]);
      }
    }
    __syncwarp();
    if (chosen >= 0) narrow(gate * (dgate - s), dlogits[t * p.ld + chosen]);
    __syncwarp();
  }
}

template <typename T, int VPL, bool ONE_BLOCK>
cudaError_t launch_fwd(const RouteParams& p, cudaStream_t st) {
  const int threads = route_threads<VPL>();
  const size_t smem = route_smem(threads, p.E, ONE_BLOCK);
  auto* kernel = route_kernel<T, VPL, ONE_BLOCK>;
  if (smem + sizeof(uint2) * threads > 48 * 1024) {  // with the static part
    const cudaError_t e = cudaFuncSetAttribute(
        kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(kernel, dim3(p.blocks), dim3(threads), smem, st, p);
}

template <typename T, int VPL>
cudaError_t launch_bwd(const RouteBackwardParams& p, cudaStream_t st) {
  int per = 32;  // tokens of a warp
  while (per > 1 && per * p.k > 32) per /= 2;
  const long long blocks = (p.T + 8ll * per - 1) / (8 * per);
  return launch_pdl(route_backward_kernel<T, VPL>,
                    dim3(static_cast<unsigned>(std::min<long long>(blocks, 6ll * p.num_sms))),
                    dim3(256), 0, st, p);
}

template <typename T>
cudaError_t fwd_by_width(const RouteParams& p, cudaStream_t st) {
  const bool one = p.blocks == 1;
#define GB_ROUTE(V) \
  if (p.E <= 32 * V) return one ? launch_fwd<T, V, true>(p, st) : launch_fwd<T, V, false>(p, st);
  GB_ROUTE(1) GB_ROUTE(2) GB_ROUTE(4) GB_ROUTE(8) GB_ROUTE(16) GB_ROUTE(32)
#undef GB_ROUTE
  return cudaErrorInvalidValue;
}

template <typename T>
cudaError_t bwd_by_width(const RouteBackwardParams& p, cudaStream_t st) {
  if (p.normalize) return launch_bwd<T, 0>(p, st);
#define GB_ROUTE(V) \
  if (p.E <= 32 * V) return launch_bwd<T, V>(p, st);
  GB_ROUTE(1) GB_ROUTE(2) GB_ROUTE(4) GB_ROUTE(8) GB_ROUTE(16) GB_ROUTE(32)
#undef GB_ROUTE
  return cudaErrorInvalidValue;
}

}  // namespace

int route_blocks(long long T, int k, int num_sms) {
  if (T <= ONE_BLOCK_TOKENS && T * k <= ONE_BLOCK_SLOTS) return 1;
  // a block an SM; fewer than a token for each of its warps would only add counts
  const long long tokens = std::max<long long>((T + num_sms - 1) / num_sms, 32);
  return static_cast<int>((T + tokens - 1) / tokens);
}

cudaError_t launch_route(const RouteParams& p, cudaStream_t st) {
  cudaError_t e = p.type == T_F32    ? fwd_by_width<float>(p, st)
                  : p.type == T_BF16 ? fwd_by_width<__nv_bfloat16>(p, st)
                                     : fwd_by_width<__half>(p, st);
  if (e != cudaSuccess || p.blocks == 1) return e;
  const size_t smem = sizeof(int) * ((RANK_THREADS / 32 + 3) * static_cast<size_t>(p.ld_hist) + 1) +
                      sizeof(short) * RANK_SLOTS;
  if (smem > 48 * 1024) {
    e = cudaFuncSetAttribute(route_rank_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(smem));
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(route_rank_kernel, dim3(p.blocks), dim3(RANK_THREADS), smem, st, p);
}

cudaError_t launch_route_backward(const RouteBackwardParams& p, cudaStream_t st) {
  return p.type == T_F32    ? bwd_by_width<float>(p, st)
         : p.type == T_BF16 ? bwd_by_width<__nv_bfloat16>(p, st)
                            : bwd_by_width<__half>(p, st);
}

}  // namespace gb300
