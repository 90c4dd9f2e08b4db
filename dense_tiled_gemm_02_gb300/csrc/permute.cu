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
// allow it, else element by element.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "moe.h"
#include "ptx.cuh"
#include "tc_launch.h"

namespace gb300 {

namespace {

constexpr int THREADS = 256;
constexpr int KU = 8;  // slots of a token in flight together

// V consecutive elements of type T as one load or store (V = 1: one element).
template <typename T, int V>
struct alignas(sizeof(T) * V) Pack {
  T v[V];
};

__device__ __forceinline__ float widen(float x) { return x; }
__device__ __forceinline__ float widen(__half x) { return __half2float(x); }
__device__ __forceinline__ float widen(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void narrow(float v, float& x) { x = v; }
__device__ __forceinline__ void narrow(float v, __half& x) { x = __float2half_rn(v); }
__device__ __forceinline__ void narrow(float v, __nv_bfloat16& x) { x = __float2bfloat16_rn(v); }

// The sorted row of a slot, -1 when it has none or the index is out of range.
__device__ __forceinline__ int row_of(const PermuteParams& p, long long slot) {
  const int r = p.slot_row[slot];
  if (r < -1 || r >= p.T * p.k) {
    atomicOr(p.status, STATUS_BAD_INDEX);
    return -1;
  }
  return r;
}

template <typename T, int V>
__device__ __forceinline__ Pack<T, V> zeros() {
  Pack<T, V> z;
#pragma unroll
  for (int i = 0; i < V; ++i) narrow(0.f, z.v[i]);
  return z;
}

// blockIdx.x: token and chunk of THREADS * V columns.
template <typename T, int V>
__global__ void __launch_bounds__(THREADS) gather_kernel(const PermuteParams p, int chunks) {
  using P = Pack<T, V>;
  const long long t = blockIdx.x / chunks;
  const long long h = (static_cast<long long>(blockIdx.x % chunks) * THREADS + threadIdx.x) * V;
  pdl_wait();
  pdl_trigger();
  if (h >= p.H) return;
  const P x = *reinterpret_cast<const P*>(static_cast<const T*>(p.tokens) + t * p.ld_tokens + h);
  T* const out = static_cast<T*>(p.rows_out) + h;
  for (int j = 0; j < p.k; ++j) {
    const long long slot = t * p.k + j;
    const int r = row_of(p, slot);
    if (r >= 0) *reinterpret_cast<P*>(out + r * p.ld_rows) = x;
    if (p.row_slot[slot] < 0) *reinterpret_cast<P*>(out + slot * p.ld_rows) = zeros<T, V>();
  }
}

template <typename T, int V>
__global__ void __launch_bounds__(THREADS) combine_kernel(const PermuteParams p, int chunks) {
  using P = Pack<T, V>;
  const long long t = blockIdx.x / chunks;
  const long long h = (static_cast<long long>(blockIdx.x % chunks) * THREADS + threadIdx.x) * V;
  pdl_wait();
  pdl_trigger();
  if (h >= p.H) return;
  const T* const rows = static_cast<const T*>(p.rows) + h;
  float acc[V];
#pragma unroll
  for (int i = 0; i < V; ++i) acc[i] = 0.f;
  for (int j0 = 0; j0 < p.k; j0 += KU) {
    P x[KU];
    float g[KU];
#pragma unroll
    for (int u = 0; u < KU; ++u) {
      g[u] = 0.f;
      if (j0 + u >= p.k) continue;
      const long long slot = t * p.k + j0 + u;
      const int r = row_of(p, slot);
      x[u] = r >= 0 ? *reinterpret_cast<const P*>(rows + r * p.ld_rows) : zeros<T, V>();
      // an unrouted slot adds nothing, whatever its gate holds
      if (r >= 0) g[u] = p.gates ? p.gates[slot] : 1.f;
    }
#pragma unroll
    for (int u = 0; u < KU; ++u)
      if (j0 + u < p.k)
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] = fmaf(g[u], widen(x[u].v[i]), acc[i]);
  }
  P y;
#pragma unroll
  for (int i = 0; i < V; ++i) narrow(acc[i], y.v[i]);
  *reinterpret_cast<P*>(static_cast<T*>(p.tokens_out) + t * p.ld_tokens + h) = y;
}

// One block per token: dY[t] goes out scaled to its k rows while the k dot
// products are summed, per thread over its columns, then over the warp by a
// fixed butterfly, then over the warps in order.
template <typename T, int V>
__global__ void __launch_bounds__(THREADS) combine_backward_kernel(const PermuteParams p) {
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
#pragma unroll
    for (int u = 0; u < KU; ++u) {
      row[u] = -1;
      g[u] = dot[u] = 0.f;
      clear[u] = false;
      if (j0 + u < p.k) {
        const long long slot = t * p.k + j0 + u;
        row[u] = row_of(p, slot);
        if (row[u] >= 0) g[u] = p.gates[slot];
        clear[u] = p.row_slot[slot] < 0;
      }
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

template <typename T, int V>
cudaError_t launch_as(Op op, const PermuteParams& p, cudaStream_t st) {
  const int chunks = static_cast<int>((p.H + THREADS * V - 1) / (THREADS * V));
  const dim3 block(THREADS);
  if (op == Op::kBackward)
    return launch_pdl(combine_backward_kernel<T, V>, dim3(static_cast<unsigned>(p.T)), block, 0, st,
                      p);
  const long long grid = p.T * chunks;
  if (grid > 0x7FFFFFFFll) return cudaErrorInvalidValue;
  return op == Op::kGather
             ? launch_pdl(gather_kernel<T, V>, dim3(static_cast<unsigned>(grid)), block, 0, st, p,
                          chunks)
             : launch_pdl(combine_kernel<T, V>, dim3(static_cast<unsigned>(grid)), block, 0, st, p,
                          chunks);
}

template <typename T>
cudaError_t launch_typed(Op op, const PermuteParams& p, cudaStream_t st) {
  constexpr int V = 16 / sizeof(T);
  uintptr_t bits = 0;
  for (const void* q : {p.tokens, static_cast<const void*>(p.tokens_out), p.rows,
                        static_cast<const void*>(p.rows_out)})
    bits |= reinterpret_cast<uintptr_t>(q);
  const bool wide = bits % 16 == 0 && p.H % V == 0 && p.ld_tokens % V == 0 && p.ld_rows % V == 0;
  return wide ? launch_as<T, V>(op, p, st) : launch_as<T, 1>(op, p, st);
}

cudaError_t launch_op(Op op, const PermuteParams& p, cudaStream_t st) {
  return p.type == T_F32    ? launch_typed<float>(op, p, st)
         : p.type == T_BF16 ? launch_typed<__nv_bfloat16>(op, p, st)
                            : launch_typed<__half>(op, p, st);
}

}  // namespace

cudaError_t launch_gather(const PermuteParams& p, cudaStream_t st) {
  return launch_op(Op::kGather, p, st);
}
cudaError_t launch_combine(const PermuteParams& p, cudaStream_t st) {
  return launch_op(Op::kCombine, p, st);
}
cudaError_t launch_combine_backward(const PermuteParams& p, cudaStream_t st) {
  return launch_op(Op::kBackward, p, st);
}

}  // namespace gb300
