// route.cu -- token routing: the k largest logits of each token, their
// softmax gates, and the stable sort of the chosen slots by expert.
//
//   g[t,j] = exp(x[t,e_j] - m) / Z,   m = max, Z = sum of exp(x - m) over the
//            chosen logits (normalize) or over all of them
//   dx[t,e_j] = g_j (dg_j - s), s = sum_i g_i dg_i; without normalize every
//            e gets p_e ([e = e_j] dg_j - s), p the softmax over all E
//
// The forward pass must read T x E logits once and write 20 bytes a slot;
// the k rounds of a warp-wide maximum bound it (see below), not HBM.  A warp
// owns a token: lane l holds the logits e = 32 i + l as order-preserving
// 32-bit keys and its own largest; a round takes the warp's largest key and,
// among its holders, the lowest expert (two warp reductions), and only the
// winning lane looks for its next one.
//
// The sort is a counting sort without atomics on its order, so equal inputs
// give equal outputs: every warp counts a contiguous run of slots per expert
// (lanes with the same expert find each other by a match), the counts are
// summed up in slot order, and the second walk over the run hands out rows.
// One block does all of it for small calls (one launch); otherwise blocks
// take contiguous tokens, the last one to finish turns the block counts into
// first rows, and a second kernel hands out the rows.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "moe.h"
#include "ptx.cuh"
#include "tc_launch.h"

namespace gb300 {

namespace {

constexpr uint32_t KEY_NEG_INF = 0x007FFFFFu;  // the key of -inf: not chosen, nor any below
constexpr int ONE_BLOCK_SLOTS = 4096;
constexpr int ONE_BLOCK_TOKENS = 64;

// fp32 as an unsigned key in the same order, -0 equal to +0, NaN on top.
__device__ __forceinline__ uint32_t order_key(float x) {
  if (x != x) return 0xFFFFFFFFu;
  const uint32_t b = __float_as_uint(x + 0.f);
  return b ^ ((b >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}

__device__ __forceinline__ float widen(float x) { return x; }
__device__ __forceinline__ float widen(__half x) { return __half2float(x); }
__device__ __forceinline__ float widen(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void narrow(float v, float& x) { x = v; }
__device__ __forceinline__ void narrow(float v, __half& x) { x = __float2half_rn(v); }
__device__ __forceinline__ void narrow(float v, __nv_bfloat16& x) { x = __float2bfloat16_rn(v); }

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
  return v;
}

template <typename T, int VPL>
__device__ __forceinline__ void load_keys(const T* x, int E, int lane, uint32_t (&key)[VPL]) {
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int e = 32 * i + lane;
    key[i] = e < E ? order_key(widen(x[e])) : 0u;
  }
}

// The token's choices: lane j < n (returned) holds the j-th key and expert.
template <int VPL>
__device__ __forceinline__ int top_k(uint32_t (&key)[VPL], int k, int lane, uint32_t& my_key,
                                     int& my_expert) {
  uint32_t best = key[0];
  int bi = 0;
#pragma unroll
  for (int i = 1; i < VPL; ++i)
    if (key[i] > best) {
      best = key[i];
      bi = i;
    }
  my_key = 0u;
  my_expert = -1;
  for (int j = 0; j < k; ++j) {
    const uint32_t m = __reduce_max_sync(0xFFFFFFFFu, best);
    if (m <= KEY_NEG_INF) return j;
    const uint32_t e =
        __reduce_min_sync(0xFFFFFFFFu, best == m ? static_cast<uint32_t>(32 * bi + lane) : ~0u);
    if (lane == j) {
      my_key = m;
      my_expert = static_cast<int>(e);
    }
    if ((e & 31u) == static_cast<uint32_t>(lane)) {
      best = 0u;
      const int gone = bi;
      bi = 0;
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        if (i == gone) key[i] = 0u;
        if (key[i] > best) {
          best = key[i];
          bi = i;
        }
      }
    }
  }
  return k;
}

// Counting sort of n slots from slot s0 by a block's warps.  expert(i) is the
// expert of the block's i-th slot or -1; cnt: [warps][E] in shared memory.
// count_slots leaves each warp's counts; hand_out_rows walks the same runs,
// cnt[w][e] then holding the first row of warp w's slots of expert e.
__device__ __forceinline__ int run_length(int n, int warps) {
  return ((n + warps - 1) / warps + 31) / 32 * 32;
}

template <typename ExpertOf, typename Visit>
__device__ __forceinline__ void walk_run(int n, int warps, int warp, int lane, ExpertOf expert,
                                         Visit visit) {
  const int len = run_length(n, warps);
  const int end = min(n, (warp + 1) * len);
  for (int i0 = warp * len; i0 < end; i0 += 32) {
    const int i = i0 + lane;
    const int e = i < end ? expert(i) : -1;
    const uint32_t same = __match_any_sync(0xFFFFFFFFu, e);
    visit(i, e, same);
    __syncwarp();
  }
}

template <typename ExpertOf>
__device__ __forceinline__ void count_slots(int n, int E, int* cnt, ExpertOf expert) {
  const int warps = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int i = threadIdx.x; i < warps * E; i += blockDim.x) cnt[i] = 0;
  __syncthreads();
  walk_run(n, warps, warp, lane, expert, [&](int, int e, uint32_t same) {
    if (e >= 0 && lane == __ffs(same) - 1) cnt[warp * E + e] += __popc(same);
  });
  __syncthreads();
}

template <typename ExpertOf>
__device__ __forceinline__ void hand_out_rows(int n, int E, int s0, int* cnt, ExpertOf expert,
                                              int* row_slot, int* slot_row) {
  const int warps = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  walk_run(n, warps, warp, lane, expert, [&](int i, int e, uint32_t same) {
    const uint32_t below = same & ((1u << lane) - 1u);
    int row = -1;
    if (e >= 0) {
      row = cnt[warp * E + e] + __popc(below);
      row_slot[row] = s0 + i;
    }
    __syncwarp();
    if (e >= 0 && below == 0u) cnt[warp * E + e] += __popc(same);
    if (i < n && i < (warp + 1) * run_length(n, warps)) slot_row[s0 + i] = row;
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

// Shared memory of the route kernels: cnt[warps][E], total[E], first[E + 1]
// and, in the one-block form, the experts of all slots.
size_t route_smem(int threads, int E, bool one_block) {
  return sizeof(int) * (static_cast<size_t>(threads / 32) * E + 2 * E + 1) +
         (one_block ? sizeof(short) * ONE_BLOCK_SLOTS : 0);
}

// The several-block form's end: each block leaves its counts, and the last
// one to do so turns them into the first row of each block's slots of each
// expert, and writes the offsets.
__device__ __forceinline__ void finish_blocks(const RouteParams& p, int* cnt, int* total,
                                              int* first) {
  const int warps = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int e = threadIdx.x; e < p.E; e += blockDim.x) p.hist[blockIdx.x * p.E + e] = total[e];
  __shared__ int last;
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) last = atomicAdd(p.ticket, 1u) == gridDim.x - 1;
  __syncthreads();
  if (!last) return;
  __threadfence();
  // Each expert's column of block counts becomes the rows before each block.
  // blockDim / E threads share a column, each a run of blocks; cnt holds the
  // runs' sums.
  const int strips = max(1, min(warps, static_cast<int>(blockDim.x) / p.E));
  const int per = (p.blocks + strips - 1) / strips;
  for (int i = threadIdx.x; i < strips * p.E; i += blockDim.x) {
    const int s = i / p.E, e = i - s * p.E;
    int sum = 0;
#pragma unroll 8
    for (int b = s * per; b < min(p.blocks, (s + 1) * per); ++b) sum += __ldcg(p.hist + b * p.E + e);
    cnt[i] = sum;
  }
  __syncthreads();
  for (int e = threadIdx.x; e < p.E; e += blockDim.x) {
    int sum = 0;
    for (int s = 0; s < strips; ++s) {
      const int c = cnt[s * p.E + e];
      cnt[s * p.E + e] = sum;
      sum += c;
    }
    total[e] = sum;
  }
  __syncthreads();
  if (warp == 0) warp_prefix(total, p.E, lane, first);
  __syncthreads();
  for (int e = threadIdx.x; e <= p.E; e += blockDim.x) p.offsets[e] = first[e];
  for (int i = threadIdx.x; i < strips * p.E; i += blockDim.x) {
    const int s = i / p.E, e = i - s * p.E;
    int at = first[e] + cnt[i];
#pragma unroll 8
    for (int b = s * per; b < min(p.blocks, (s + 1) * per); ++b) {
      const int c = __ldcg(p.hist + b * p.E + e);
      p.hist[b * p.E + e] = at;
      at += c;
    }
  }
  if (threadIdx.x == 0) *p.ticket = 0u;  // ready for the next call
}

template <typename T, int VPL>
constexpr int route_threads() {
  return VPL <= 8 ? 1024 : 512;  // registers: the keys of two tokens a lane
}

template <typename T, int VPL, bool ONE_BLOCK>
__global__ void __launch_bounds__(route_threads<T, VPL>()) route_kernel(const RouteParams p) {
  extern __shared__ int sm[];
  const int warps = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int* const cnt = sm;
  int* const total = sm + warps * p.E;
  int* const first = total + p.E;
  short* const slots = reinterpret_cast<short*>(first + p.E + 1);
  const int t0 = blockIdx.x * p.tokens_per_block;
  const int t1 = min(p.T, t0 + p.tokens_per_block);
  if (!ONE_BLOCK) {
    for (int e = threadIdx.x; e < p.E; e += blockDim.x) total[e] = 0;
    __syncthreads();
  }
  pdl_wait();
  pdl_trigger();
  const T* const logits = static_cast<const T*>(p.logits);
  uint32_t next[VPL];
  if (t0 + warp < t1) load_keys<T, VPL>(logits + (t0 + warp) * p.ld, p.E, lane, next);
  for (int t = t0 + warp; t < t1; t += warps) {
    uint32_t key[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) key[i] = next[i];
    if (t + warps < t1) load_keys<T, VPL>(logits + (t + warps) * p.ld, p.E, lane, next);
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
    const int n = top_k<VPL>(key, p.k, lane, my_key, my_expert);
    const float top = key_value(__shfl_sync(0xFFFFFFFFu, my_key, 0));
    const float ex = lane < n ? expf(key_value(my_key) - top) : 0.f;
    if (p.normalize) z = warp_sum(ex);
    if (lane < p.k) {
      const int s = t * p.k + lane;
      p.experts[s] = my_expert;
      p.gates[s] = lane < n ? ex / z : 0.f;
      if (ONE_BLOCK)
        slots[s] = static_cast<short>(my_expert);
      else if (my_expert >= 0)
        atomicAdd(&total[my_expert], 1);  // a count: the order does not matter
    }
  }
  __syncthreads();
  if constexpr (ONE_BLOCK) {
    const int n = p.T * p.k;
    auto expert = [&](int i) { return static_cast<int>(slots[i]); };
    count_slots(n, p.E, cnt, expert);
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
    hand_out_rows(n, p.E, 0, cnt, expert, p.row_slot, p.slot_row);
    for (int r = first[p.E] + threadIdx.x; r < n; r += blockDim.x) p.row_slot[r] = -1;
  } else {
    finish_blocks(p, cnt, total, first);
  }
}

__global__ void __launch_bounds__(512) route_rank_kernel(const RouteParams p) {
  extern __shared__ int cnt[];
  pdl_wait();
  pdl_trigger();
  const int warps = blockDim.x >> 5;
  const int s0 = blockIdx.x * p.tokens_per_block * p.k;
  const int n = min(p.T * p.k, s0 + p.tokens_per_block * p.k) - s0;
  auto expert = [&](int i) { return p.experts[s0 + i]; };
  count_slots(n, p.E, cnt, expert);
  for (int e = threadIdx.x; e < p.E; e += blockDim.x) {
    int at = p.hist[blockIdx.x * p.E + e];
    for (int w = 0; w < warps; ++w) {
      const int c = cnt[w * p.E + e];
      cnt[w * p.E + e] = at;
      at += c;
    }
  }
  __syncthreads();
  hand_out_rows(n, p.E, s0, cnt, expert, p.row_slot, p.slot_row);
  const int routed = p.offsets[p.E];
  for (int r = s0 + threadIdx.x; r < s0 + n; r += blockDim.x)
    if (r >= routed) p.row_slot[r] = -1;
}

// One warp per token: the row is written whole, then its k chosen entries
// (stores of one warp to one address stay in order across __syncwarp).
template <typename T, int VPL>
__global__ void __launch_bounds__(256) route_backward_kernel(const RouteBackwardParams p) {
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * 8 + (threadIdx.x >> 5);
  pdl_wait();
  pdl_trigger();
  if (t >= p.T) return;
  int e = -1;
  float g = 0.f, dg = 0.f;
  if (lane < p.k) {
    e = p.experts[static_cast<long long>(t) * p.k + lane];
    if (e >= p.E) e = -1;
    if (e >= 0) {
      g = p.gates[static_cast<long long>(t) * p.k + lane];
      dg = p.dgates[static_cast<long long>(t) * p.k + lane];
    }
  }
  const float s = warp_sum(g * dg);
  T* const dx = static_cast<T*>(p.dlogits) + t * p.ld;
  if (p.normalize) {
    T zero;
    narrow(0.f, zero);
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (32 * i + lane < p.E) dx[32 * i + lane] = zero;
  } else {
    uint32_t key[VPL];
    load_keys<T, VPL>(static_cast<const T*>(p.logits) + t * p.ld, p.E, lane, key);
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
        narrow(key[i] > KEY_NEG_INF ? -(ex[i] / z) * s : 0.f, dx[32 * i + lane]);
  }
  __syncwarp();
  if (e >= 0) narrow(g * (dg - s), dx[e]);
}

template <typename T, int VPL, bool ONE_BLOCK>
cudaError_t launch_fwd(const RouteParams& p, cudaStream_t st) {
  const int threads = route_threads<T, VPL>();
  const size_t smem = route_smem(threads, p.E, ONE_BLOCK);
  auto* kernel = route_kernel<T, VPL, ONE_BLOCK>;
  if (smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(
        kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(kernel, dim3(p.blocks), dim3(threads), smem, st, p);
}

template <typename T, int VPL>
cudaError_t launch_bwd(const RouteBackwardParams& p, cudaStream_t st) {
  return launch_pdl(route_backward_kernel<T, VPL>, dim3((p.T + 7) / 8), dim3(256), 0, st, p);
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
#define GB_ROUTE(V) \
  if (p.E <= 32 * V) return launch_bwd<T, V>(p, st);
  GB_ROUTE(1) GB_ROUTE(2) GB_ROUTE(4) GB_ROUTE(8) GB_ROUTE(16) GB_ROUTE(32)
#undef GB_ROUTE
  return cudaErrorInvalidValue;
}

}  // namespace

int route_blocks(long long T, int k, int num_sms) {
  if (T <= ONE_BLOCK_TOKENS && T * k <= ONE_BLOCK_SLOTS) return 1;
  const long long tokens = (T + num_sms - 1) / num_sms;
  return static_cast<int>((T + tokens - 1) / tokens);
}

cudaError_t launch_route(const RouteParams& p, cudaStream_t st) {
  cudaError_t e = p.type == T_F32    ? fwd_by_width<float>(p, st)
                  : p.type == T_BF16 ? fwd_by_width<__nv_bfloat16>(p, st)
                                     : fwd_by_width<__half>(p, st);
  if (e != cudaSuccess || p.blocks == 1) return e;
  const size_t smem = sizeof(int) * 16 * static_cast<size_t>(p.E);
  if (smem > 48 * 1024) {
    e = cudaFuncSetAttribute(route_rank_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(smem));
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(route_rank_kernel, dim3(p.blocks), dim3(512), smem, st, p);
}

cudaError_t launch_route_backward(const RouteBackwardParams& p, cudaStream_t st) {
  return p.type == T_F32    ? bwd_by_width<float>(p, st)
         : p.type == T_BF16 ? bwd_by_width<__nv_bfloat16>(p, st)
                            : bwd_by_width<__half>(p, st);
}

}  // namespace gb300
