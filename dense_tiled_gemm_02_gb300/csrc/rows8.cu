// rows8.cu -- rows to 8 bits and back: blocks of 32 values with a power of two,
// and whole rows with one fp32 scale.
//
// Bound by HBM: 16 values a thread and turn (two or four 16-byte loads, one
// 16-byte store, or the reverse), so that two threads share a block's exponent
// and one shuffle finds its largest magnitude.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "rows.cuh"

namespace gb300 {

namespace {

constexpr int THREADS = 256;

// ---------------------------------------------------------------- block rows
// VEC 16: two lanes a block.  VEC 1 (rows that do not allow vectors): a warp.
template <typename T, int VEC>
__global__ void __launch_bounds__(THREADS) pack_blocks_kernel(const Rows8Params p) {
  const int blocks = (p.H + ROW_BLOCK - 1) / ROW_BLOCK;
  constexpr int LANES = ROW_BLOCK / VEC;
  const long long all = p.T * blocks * LANES;
  pdl_wait();
  pdl_trigger();
  // (whole warps stay together: `all` counts lanes of whole blocks, and the
  // last warp's lanes past it load nothing but shuffle)
  for (long long at = static_cast<long long>(blockIdx.x) * THREADS + threadIdx.x;
       at - (threadIdx.x & 31) < all; at += static_cast<long long>(gridDim.x) * THREADS) {
    const long long item = at / LANES, row = item / blocks;
    const int b = static_cast<int>(item - row * blocks);
    const int i = b * ROW_BLOCK + static_cast<int>(at % LANES) * VEC;
    const bool ok = at < all && i < p.H;
    Vec<T, VEC> x{};
    if (ok) x = load_vec<T, VEC>(static_cast<const T*>(p.X) + row * p.ldx + i);
    uint32_t top = 0u;
#pragma unroll
    for (int j = 0; j < VEC; ++j) top = max(top, magnitude(widen(x.v[j])));
#pragma unroll
    for (int d = LANES / 2; d > 0; d >>= 1) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
    const uint32_t e = block_exponent(top, least_exponent<T>());
    const float inverse = block_inverse(e);
    if (ok) {
      Vec<int8_t, VEC> q;
#pragma unroll
      for (int j = 0; j < VEC; ++j) q.v[j] = block_integer(widen(x.v[j]), inverse);
      store_vec(p.q_out + row * p.ldq + i, q);
      if (at % LANES == 0) static_cast<uint8_t*>(p.scales_out)[row * blocks + b] = e;
    }
  }
}

template <typename T, int VEC, bool BLOCKS>
__global__ void __launch_bounds__(THREADS) unpack_kernel(const Rows8Params p) {
  const int blocks = (p.H + ROW_BLOCK - 1) / ROW_BLOCK, n = p.H / VEC;
  const long long all = p.T * n;
  pdl_wait();
  pdl_trigger();
  for (long long at = static_cast<long long>(blockIdx.x) * THREADS + threadIdx.x; at < all;
       at += static_cast<long long>(gridDim.x) * THREADS) {
    const long long row = at / n;
    const int i = static_cast<int>(at - row * n) * VEC;
    const auto q = load_vec<int8_t, VEC>(p.q + row * p.ldq + i);
    const float step =
        BLOCKS ? block_step(static_cast<const uint8_t*>(p.scales)[row * blocks + i / ROW_BLOCK])
               : static_cast<const float*>(p.scales)[row];
    Vec<T, VEC> x;
#pragma unroll
    for (int j = 0; j < VEC; ++j) narrow_finite(static_cast<float>(q.v[j]) * step, x.v[j]);
    store_vec(static_cast<T*>(p.X_out) + row * p.ldx + i, x);
  }
}

// ---------------------------------------------------------------- scaled rows
// A block (or, blockDim.x = 32, a warp) a row, which is read a second time for
// its integers, from L1 or L2.
template <typename T, int VEC>
__global__ void __launch_bounds__(1024) pack_rows_kernel(const Rows8Params p) {
  __shared__ float2 part[32];
  const long long row = static_cast<long long>(blockIdx.x) * blockDim.y + threadIdx.y;
  const int step = blockDim.x * VEC, first = threadIdx.x * VEC;
  pdl_wait();
  pdl_trigger();
  if (row >= p.T) return;
  const T* const X = static_cast<const T*>(p.X) + row * p.ldx;
  uint32_t top = 0u;
  float sum = 0.f;
#pragma unroll 2
  for (int i = first; i < p.H; i += step) {
    const auto x = load_vec<T, VEC>(X + i);
#pragma unroll
    for (int j = 0; j < VEC; ++j) top = max(top, magnitude(widen(x.v[j])));
  }
  row_reduce(sum, top, blockDim.x >> 5, part);
  const RowScale s = row_scale(__uint_as_float(top), 1.f);
  if (threadIdx.x == 0) static_cast<float*>(p.scales_out)[row] = s.scale;
#pragma unroll 2
  for (int i = first; i < p.H; i += step) {
    const auto x = load_vec<T, VEC>(X + i);
    Vec<int8_t, VEC> q;
#pragma unroll
    for (int j = 0; j < VEC; ++j) q.v[j] = row_integer(widen(x.v[j]), s);
    store_vec(p.q_out + row * p.ldq + i, q);
  }
}

// ---------------------------------------------------------------- launches
// Blocks of a grid-stride kernel over n threads' items.
dim3 stride_grid(long long n, int num_sms) {
  return dim3(static_cast<unsigned>(std::min<long long>((n + THREADS - 1) / THREADS, 16ll * num_sms)));
}

template <typename T, int VEC>
cudaError_t pack_as(const Rows8Params& p, int num_sms, cudaStream_t st) {
  if (p.block) {
    const long long n = p.T * ((p.H + ROW_BLOCK - 1) / ROW_BLOCK) * (ROW_BLOCK / VEC);
    return launch_pdl(pack_blocks_kernel<T, VEC>, stride_grid(n, num_sms), dim3(THREADS), 0, st, p);
  }
  const int n = (p.H + VEC - 1) / VEC;
  const int threads = std::min(1024, (n + 31) / 32 * 32), rows = threads == 32 ? 4 : 1;
  return launch_pdl(pack_rows_kernel<T, VEC>, dim3(static_cast<unsigned>((p.T + rows - 1) / rows)),
                    dim3(threads, rows), 0, st, p);
}
template <typename T, int VEC>
cudaError_t unpack_as(const Rows8Params& p, int num_sms, cudaStream_t st) {
  const dim3 grid = stride_grid(p.T * (p.H / VEC), num_sms);
  return p.block ? launch_pdl(unpack_kernel<T, VEC, true>, grid, dim3(THREADS), 0, st, p)
                 : launch_pdl(unpack_kernel<T, VEC, false>, grid, dim3(THREADS), 0, st, p);
}

template <typename T>
cudaError_t typed(const Rows8Params& p, bool pack, int num_sms, cudaStream_t st) {
  const void* const X = pack ? p.X : p.X_out;
  const void* const q = pack ? p.q_out : p.q;
  const bool vec = p.H % 16 == 0 && p.ldq % 16 == 0 && p.ldx * sizeof(T) % 16 == 0 &&
                   reinterpret_cast<uintptr_t>(X) % 16 == 0 && reinterpret_cast<uintptr_t>(q) % 16 == 0;
  if (pack) return vec ? pack_as<T, 16>(p, num_sms, st) : pack_as<T, 1>(p, num_sms, st);
  return vec ? unpack_as<T, 16>(p, num_sms, st) : unpack_as<T, 1>(p, num_sms, st);
}

cudaError_t launch(const Rows8Params& p, bool pack, int num_sms, cudaStream_t st) {
  return p.type == T_F32    ? typed<float>(p, pack, num_sms, st)
         : p.type == T_BF16 ? typed<__nv_bfloat16>(p, pack, num_sms, st)
                            : typed<__half>(p, pack, num_sms, st);
}

}  // namespace

cudaError_t launch_rows8_pack(const Rows8Params& p, int num_sms, cudaStream_t st) {
  return launch(p, true, num_sms, st);
}
cudaError_t launch_rows8_unpack(const Rows8Params& p, int num_sms, cudaStream_t st) {
  return launch(p, false, num_sms, st);
}

}  // namespace gb300
