// permute.cu -- rows of tokens into expert order and back, and their
// gradients.
//
//   gather            Xs[slot_row[t,j]] = X[t]; rows without a slot are zero
//   combine           Y[t] = sum_j g[t,j] Ys[slot_row[t,j]]   (g absent: 1)
//   combine_backward  dYs[slot_row[t,j]] = g[t,j] dY[t],
//                     dg[t,j] = sum_h dY[t,h] Ys[slot_row[t,j],h]
//
// All three are bound by HBM: they move each row once.  Threads are laid out
// by token, not by sorted row, so that X[t] and dY[t] are read once for all
// k rows that use them, and the k sums need no atomics: a fixed order, the
// same bits every time.  Rows move in 16-byte units where their addresses
// allow it, else element by element.  16384 tokens x 4 rows of 4096 bf16, both
// ways with gradients: 511 us for 2.7 GB (5.3 TB/s).  A decode step (16 tokens
// x 8 rows) is bound by its two calls.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "moe.h"
#include "ptx.cuh"
#include "tc_launch.h"

namespace gb300 {

namespace {

constexpr int THREADS = 256;
// KU, a template parameter: slots of a token in flight together, the smallest
// of 1, 2, 4, 8 that holds k (a larger k is walked in eights).  With 8 for
// every k the combine of k = 4 held 102 registers a thread, and two blocks an
// SM kept too little in flight: 230 us against 121 (16384 tokens x 4 rows of
// 4096 bf16).

// V consecutive elements of type T as one load or store (V = 1: one element).
template <typename T, int V>
struct alignas(sizeof(T) * V) Pack {
  T v[V];
};

// The sorted rows of slots j0 .. j0 + KU - 1 of token t, -1 for none (or no
// such slot).  All indices are loaded before any is looked at: a check
// between them (its atomic orders memory) left one index and one row load in
// flight at a time (that combine: 355 us against 230).
// clear, where given: sorted rows t * k + j0 .. + KU - 1 have no slot and become
// zeros.
template <int KU>
__device__ __forceinline__ void rows_of(const PermuteParams& p, long long t, int j0,
                                        int (&row)[KU], bool* clear = nullptr) {
  int slot[KU];
  const unsigned n = static_cast<unsigned>(p.T * p.k);
#pragma unroll
  for (int u = 0; u < KU; ++u) {
    row[u] = j0 + u < p.k ? p.slot_row[t * p.k + j0 + u] : -1;
    slot[u] = clear && j0 + u < p.k ? p.row_slot[t * p.k + j0 + u] : 0;
  }
  // an index is right when it is below n, or -1: then index + 1 is at most n
  bool bad = false;
#pragma unroll
  for (int u = 0; u < KU; ++u) {
    bad |= static_cast<unsigned>(row[u]) + 1u > n;
    bad |= static_cast<unsigned>(slot[u]) + 1u > n;
    if (static_cast<unsigned>(row[u]) >= n) row[u] = -1;
    if (clear) clear[u] = static_cast<unsigned>(slot[u]) >= n;
  }
  if (bad) atomicOr(p.status, STATUS_BAD_INDEX);
}

template <typename T, int V>
__device__ __forceinline__ Pack<T, V> zeros() {
  Pack<T, V> z;
#pragma unroll
  for (int i = 0; i < V; ++i) narrow(0.f, z.v[i]);
  return z;
}

// blockIdx.x: token and chunk of THREADS * V columns.  16384 tokens x 4 rows
// of 4096 bf16: 99 us (6.8 TB/s).
template <typename T, int V, int KU>
__global__ void __launch_bounds__(THREADS) gather_kernel(const PermuteParams p, int chunks) {
  using P = Pack<T, V>;
  const long long t = blockIdx.x / chunks;
  const long long h = (static_cast<long long>(blockIdx.x % chunks) * THREADS + threadIdx.x) * V;
  pdl_wait();
  pdl_trigger();
  if (h >= p.H) return;
  const P x = *reinterpret_cast<const P*>(static_cast<const T*>(p.tokens) + t * p.ld_tokens + h);
  T* const out = static_cast<T*>(p.rows_out) + h;
  for (int j0 = 0; j0 < p.k; j0 += KU) {
    int row[KU];
    bool clear[KU];
    rows_of(p, t, j0, row, clear);
#pragma unroll
    for (int u = 0; u < KU; ++u) {
      if (row[u] >= 0) *reinterpret_cast<P*>(out + row[u] * p.ld_rows) = x;
      if (clear[u])
        *reinterpret_cast<P*>(out + (t * p.k + j0 + u) * p.ld_rows) = zeros<T, V>();
    }
  }
}

// blockIdx.x: chunk of THREADS * V columns and every `stride`-th token.  The
// next token's rows and gates are asked for before this token's data is
// used: an index and the row it names are two trips to memory, one after the
// other.  16384 tokens x 4 rows of 4096 bf16: 118 us (5.7 TB/s) with gates,
// 102 (6.6 TB/s) without, from 121 and 119 with a block per token.
template <typename T, int V, int KU>
__global__ void __launch_bounds__(THREADS, KU <= 4 ? 4 : 3)
    combine_kernel(const PermuteParams p, int chunks) {
  using P = Pack<T, V>;
  const long long stride = gridDim.x / chunks;
  long long t = blockIdx.x / chunks;
  const long long h = (static_cast<long long>(blockIdx.x % chunks) * THREADS + threadIdx.x) * V;
  pdl_wait();
  pdl_trigger();
  if (h >= p.H) return;
  const T* const rows = static_cast<const T*>(p.rows) + h;
  int row[KU];
  float g[KU];
  auto ask = [&](long long token, int j0) {
    rows_of(p, token, j0, row);
#pragma unroll
    for (int u = 0; u < KU; ++u)
      g[u] = p.gates && j0 + u < p.k ? p.gates[token * p.k + j0 + u] : 1.f;
  };
  ask(t, 0);
  for (; t < p.T; t += stride) {
    float acc[V];
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = 0.f;
    for (int j0 = 0; j0 < p.k; j0 += KU) {
      P x[KU];
      float f[KU];
      bool live[KU];
#pragma unroll
      for (int u = 0; u < KU; ++u) {
        live[u] = row[u] >= 0;
        f[u] = g[u];
        if (live[u]) x[u] = *reinterpret_cast<const P*>(rows + row[u] * p.ld_rows);
      }
      const bool more = j0 + KU < p.k;
      if (more || t + stride < p.T) ask(more ? t : t + stride, more ? j0 + KU : 0);
      // an unrouted slot adds nothing, whatever its gate holds
#pragma unroll
      for (int u = 0; u < KU; ++u)
        if (live[u])
#pragma unroll
          for (int i = 0; i < V; ++i) acc[i] = fmaf(f[u], widen(x[u].v[i]), acc[i]);
    }
    P y;
#pragma unroll
    for (int i = 0; i < V; ++i) narrow(acc[i], y.v[i]);
    *reinterpret_cast<P*>(static_cast<T*>(p.tokens_out) + t * p.ld_tokens + h) = y;
  }
}

// One block per token: dY[t] goes out scaled to its k rows while the k dot
// products are summed, per thread over its columns, then over the warp by a
// fixed butterfly, then over the warps in order.  16384 tokens x 4 rows of
// 4096 bf16: 198 us (6.1 TB/s; 241 at 128 registers a thread).
template <typename T, int V, int KU>
__global__ void __launch_bounds__(THREADS, V > 1 && KU <= 4 ? 3 : 2)
    combine_backward_kernel(const PermuteParams p) {
  using P = Pack<T, V>;
  __shared__ float part[THREADS / 32][KU];
  const long long t = blockIdx.x;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  pdl_trigger();
  const T* const dY = static_cast<const T*>(p.tokens) + t * p.ld_tokens;
  T* const out = static_cast<T*>(p.rows_out);
  for (int j0 = 0; j0 < p.k; j0 += KU) {
    int row[KU];
    float g[KU], dot[KU];
    bool clear[KU];
    rows_of(p, t, j0, row, clear);
#pragma unroll
    for (int u = 0; u < KU; ++u) {
      dot[u] = 0.f;
      g[u] = row[u] >= 0 ? p.gates[t * p.k + j0 + u] : 0.f;
    }
    for (long long h = static_cast<long long>(threadIdx.x) * V; h < p.H; h += THREADS * V) {
      const P d = *reinterpret_cast<const P*>(dY + h);
      P y[KU];
#pragma unroll
      for (int u = 0; u < KU; ++u)
        if (row[u] >= 0)
          y[u] = *reinterpret_cast<const P*>(static_cast<const T*>(p.rows) + row[u] * p.ld_rows + h);
#pragma unroll
      for (int u = 0; u < KU; ++u) {
        if (row[u] >= 0) {
          P o;
#pragma unroll
          for (int i = 0; i < V; ++i) {
            const float f = widen(d.v[i]);
            dot[u] = fmaf(f, widen(y[u].v[i]), dot[u]);
            narrow(g[u] * f, o.v[i]);
          }
          *reinterpret_cast<P*>(out + row[u] * p.ld_rows + h) = o;
        }
        if (clear[u])
          *reinterpret_cast<P*>(out + (t * p.k + j0 + u) * p.ld_rows + h) = zeros<T, V>();
      }
    }
#pragma unroll
    for (int u = 0; u < KU; ++u) {
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) dot[u] += __shfl_xor_sync(0xFFFFFFFFu, dot[u], d);
      if (lane == 0) part[warp][u] = dot[u];
    }
    __syncthreads();
    if (threadIdx.x < KU && j0 + threadIdx.x < p.k) {
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < THREADS / 32; ++w) s += part[w][threadIdx.x];
      p.dgates[t * p.k + j0 + threadIdx.x] = s;
    }
    __syncthreads();
  }
}

enum class Op { kGather, kCombine, kBackward };

template <typename T, int V, int KU>
cudaError_t launch_as(Op op, const PermuteParams& p, int num_sms, cudaStream_t st) {
  const int chunks = static_cast<int>((p.H + THREADS * V - 1) / (THREADS * V));
  const dim3 block(THREADS);
  if (op == Op::kBackward)
    return launch_pdl(combine_backward_kernel<T, V, KU>, dim3(static_cast<unsigned>(p.T)), block, 0,
                      st, p);
  if (op == Op::kCombine) {
    // as many blocks as the SMs hold, each with several tokens
    const long long tokens = std::min(p.T, std::max(1ll, 4ll * num_sms / chunks));
    return launch_pdl(combine_kernel<T, V, KU>, dim3(static_cast<unsigned>(tokens * chunks)), block,
                      0, st, p, chunks);
  }
  const long long grid = p.T * chunks;
  if (grid > 0x7FFFFFFFll) return cudaErrorInvalidValue;
  return launch_pdl(gather_kernel<T, V, KU>, dim3(static_cast<unsigned>(grid)), block, 0, st, p,
                    chunks);
}

template <typename T, int V>
cudaError_t launch_k(Op op, const PermuteParams& p, int num_sms, cudaStream_t st) {
  return p.k <= 1   ? launch_as<T, V, 1>(op, p, num_sms, st)
         : p.k <= 2 ? launch_as<T, V, 2>(op, p, num_sms, st)
         : p.k <= 4 ? launch_as<T, V, 4>(op, p, num_sms, st)
                    : launch_as<T, V, 8>(op, p, num_sms, st);
}

template <typename T>
cudaError_t launch_typed(Op op, const PermuteParams& p, int num_sms, cudaStream_t st) {
  constexpr int V = 16 / sizeof(T);
  uintptr_t bits = 0;
  for (const void* q : {p.tokens, static_cast<const void*>(p.tokens_out), p.rows,
                        static_cast<const void*>(p.rows_out)})
    bits |= reinterpret_cast<uintptr_t>(q);
  const bool wide = bits % 16 == 0 && p.H % V == 0 && p.ld_tokens % V == 0 && p.ld_rows % V == 0;
  return wide ? launch_k<T, V>(op, p, num_sms, st) : launch_k<T, 1>(op, p, num_sms, st);
}

cudaError_t launch_op(Op op, const PermuteParams& p, int num_sms, cudaStream_t st) {
  return p.type == T_F32    ? launch_typed<float>(op, p, num_sms, st)
         : p.type == T_BF16 ? launch_typed<__nv_bfloat16>(op, p, num_sms, st)
                            : launch_typed<__half>(op, p, num_sms, st);
}

}  // namespace

cudaError_t launch_gather(const PermuteParams& p, int num_sms, cudaStream_t st) {
  return launch_op(Op::kGather, p, num_sms, st);
}
cudaError_t launch_combine(const PermuteParams& p, int num_sms, cudaStream_t st) {
  return launch_op(Op::kCombine, p, num_sms, st);
}
cudaError_t launch_combine_backward(const PermuteParams& p, int num_sms, cudaStream_t st) {
  return launch_op(Op::kBackward, p, num_sms, st);
}

}  // namespace gb300
