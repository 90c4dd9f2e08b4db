// rows8.cu -- rows to 8 bits and back: blocks of 32 values with a power of two,
// and whole rows with one fp32 scale.
//
// Bound by HBM: 16 values a thread and turn (16-byte accesses on both sides:
// with 8 of a 16-bit type, 8-byte ones on the 8-bit side, unpacking takes 44
// instead of 33 us), several turns in flight; two lanes share a block's exponent
// and find its largest magnitude by a shuffle.  Integers are made and read by
// additions in the last place and byte permutes, since conversion instructions,
// at a quarter of the rate, bounded the first form (40 us; 64-bit divisions for
// an item's row another 5).
//
// Measured (one GB300, 16384 x 4096 bf16, floor 30.1 us each way): block rows 30
// us and back 33, scaled rows 29 and back 34.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "rows.cuh"

namespace gb300 {

namespace {

constexpr int THREADS = DEAL_THREADS;

// ---------------------------------------------------------------- block rows
// LANES lanes to 32 values; VEC 1 (rows that do not allow vectors): a warp.
template <typename T, int VEC>
__global__ void __launch_bounds__(THREADS)
    pack_blocks_kernel(const Rows8Params p, const Deal deal) {
  const int blocks = (p.H + ROW_BLOCK - 1) / ROW_BLOCK;
  constexpr int LANES = ROW_BLOCK / VEC, U = 4;
  const Items all = block_items(p.T, deal, blockIdx.x);
  const Divisor& lanes = deal.lanes;
  pdl_wait();
  pdl_trigger();
  // (whole warps stay together: lanes past the last item load nothing but shuffle)
  for (uint32_t at0 = threadIdx.x; at0 - (threadIdx.x & 31) < all.n; at0 += U * THREADS) {
    Vec<T, VEC> x[U];
    long long row[U];
    int i[U];
    bool ok[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t at = all.at + at0 + u * THREADS, r = divide(at, lanes);
      row[u] = all.row + r;
      i[u] = static_cast<int>(at - r * lanes.d) * VEC;
      ok[u] = at0 + u * THREADS < all.n && i[u] < p.H;
      x[u] = Vec<T, VEC>{};
      if (ok[u]) x[u] = load_vec<T, VEC>(static_cast<const T*>(p.X) + row[u] * p.ldx + i[u]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      uint32_t top = vec_top(x[u]);
#pragma unroll
      for (int d = LANES / 2; d > 0; d >>= 1) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
      const uint32_t e = block_exponent(top, least_exponent<T>());
      const float inverse = block_inverse(e);
      if (ok[u]) {
        float v[VEC];
#pragma unroll
        for (int j = 0; j < VEC; ++j) v[j] = widen(x[u].v[j]);
        store_block_integers(p.q_out + row[u] * p.ldq + i[u], v, inverse);
        if (i[u] % ROW_BLOCK == 0)
          static_cast<uint8_t*>(p.scales_out)[row[u] * blocks + i[u] / ROW_BLOCK] = e;
      }
    }
  }
}

template <typename T, int VEC, bool BLOCKS>
__global__ void __launch_bounds__(THREADS)
    unpack_kernel(const Rows8Params p, const Deal deal) {
  const int blocks = (p.H + ROW_BLOCK - 1) / ROW_BLOCK;
  const Items all = block_items(p.T, deal, blockIdx.x);
  const Divisor& lanes = deal.lanes;
  pdl_wait();
  pdl_trigger();
  constexpr int U = 2;
  for (uint32_t at0 = threadIdx.x; at0 < all.n; at0 += U * THREADS) {
    Vec<int8_t, VEC> q[U];
    float step[U];
    T* to[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t at = all.at + at0 + u * THREADS, r = divide(at, lanes);
      const long long row = all.row + r;
      const int i = static_cast<int>(at - r * lanes.d) * VEC;
      to[u] = static_cast<T*>(p.X_out) + row * p.ldx + i;
      if (at0 + u * THREADS < all.n) {
        q[u] = load_vec<int8_t, VEC>(p.q + row * p.ldq + i);
        step[u] = BLOCKS ? block_step(static_cast<const uint8_t*>(p.scales)[row * blocks + i / ROW_BLOCK])
                         : static_cast<const float*>(p.scales)[row];
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (at0 + u * THREADS < all.n) {
        float v[VEC];
        integers(q[u], v);
        Vec<T, VEC> x;
        if (step[u] < largest<T>() / 256.f) {  // nothing can round past the finite values
#pragma unroll
          for (int j = 0; j < VEC; ++j) narrow(v[j] * step[u], x.v[j]);
        } else {
#pragma unroll
          for (int j = 0; j < VEC; ++j) narrow_finite(v[j] * step[u], x.v[j]);
        }
        store_vec(to[u], x);
      }
  }
}

// ---------------------------------------------------------------- scaled rows
// A block (or, blockDim.x = 32, a warp) a row, whose threads hold NV vectors
// each, or with NV = 0 (rows too long) read them again.
template <typename T, int VEC, int NV>
__global__ void __launch_bounds__(1024) pack_rows_kernel(const Rows8Params p) {
  __shared__ float2 part[32];
  const long long row = static_cast<long long>(blockIdx.x) * blockDim.y + threadIdx.y;
  const int step = blockDim.x * VEC, first = threadIdx.x * VEC;
  pdl_wait();
  pdl_trigger();
  if (row >= p.T) return;
  const T* const X = static_cast<const T*>(p.X) + row * p.ldx;
  constexpr int N = NV > 0 ? NV : 1;
  Vec<T, VEC> x[N];
  uint32_t top = 0u;
  float sum = 0.f;
  auto largest_of = [&](const Vec<T, VEC>& v) { top = max(top, vec_top(v)); };
  if constexpr (NV > 0) {
#pragma unroll
    for (int k = 0; k < NV; ++k)
      if (first + k * step < p.H) x[k] = load_vec<T, VEC>(X + first + k * step);
#pragma unroll
    for (int k = 0; k < NV; ++k)
      if (first + k * step < p.H) largest_of(x[k]);
  } else {
    for (int i = first; i < p.H; i += step) largest_of(load_vec<T, VEC>(X + i));
  }
  row_reduce(sum, top, blockDim.x >> 5, part);
  const RowScale s = row_scale(__uint_as_float(top), 1.f);
  if (threadIdx.x == 0) static_cast<float*>(p.scales_out)[row] = s.scale;
  auto store = [&](const Vec<T, VEC>& v, int i) {
    float f[VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j) f[j] = widen(v.v[j]);
    store_row_integers(p.q_out + row * p.ldq + i, f, s);
  };
  if constexpr (NV > 0) {
#pragma unroll
    for (int k = 0; k < NV; ++k)
      if (first + k * step < p.H) store(x[k], first + k * step);
  } else {
    for (int i = first; i < p.H; i += step) store(load_vec<T, VEC>(X + i), i);
  }
}

// ---------------------------------------------------------------- launches
template <typename T, int VEC>
cudaError_t pack_as(const Rows8Params& p, int num_sms, cudaStream_t st) {
  if (p.block) {
    const int lanes = (p.H + ROW_BLOCK - 1) / ROW_BLOCK * (ROW_BLOCK / VEC);
    dim3 grid;
    const Deal deal = deal_of(p.T, lanes, num_sms, grid);
    return launch_pdl(pack_blocks_kernel<T, VEC>, grid, dim3(THREADS), 0, st, p, deal);
  }
  // few rows are spread over more threads
  constexpr int MOST = VEC == 1 ? 8 : VEC == 16 ? 2 : 4;
  const int n = (p.H + VEC - 1) / VEC;
  int nv = p.T >= num_sms ? MOST : 1;
  while (nv > 1 && n <= 16 * nv) nv /= 2;
  if (nv == 1 && n > 1024) nv = MOST;
  const bool again = n > 1024 * nv;
  const int threads = again ? 1024 : (((n + nv - 1) / nv) + 31) / 32 * 32, rows = threads == 32 ? 4 : 1;
  const dim3 grid(static_cast<unsigned>((p.T + rows - 1) / rows)), block(threads, rows);
  if (again) return launch_pdl(pack_rows_kernel<T, VEC, 0>, grid, block, 0, st, p);
  if (nv == 1) return launch_pdl(pack_rows_kernel<T, VEC, 1>, grid, block, 0, st, p);
  if constexpr (MOST == 8)
    if (nv == 8) return launch_pdl(pack_rows_kernel<T, VEC, 8>, grid, block, 0, st, p);
  if constexpr (MOST >= 4)
    if (nv == 4) return launch_pdl(pack_rows_kernel<T, VEC, 4>, grid, block, 0, st, p);
  return launch_pdl(pack_rows_kernel<T, VEC, 2>, grid, block, 0, st, p);
}
template <typename T, int VEC>
cudaError_t unpack_as(const Rows8Params& p, int num_sms, cudaStream_t st) {
  const int lanes = p.H / VEC;
  dim3 grid;
  const Deal deal = deal_of(p.T, lanes, num_sms, grid);
  return p.block ? launch_pdl(unpack_kernel<T, VEC, true>, grid, dim3(THREADS), 0, st, p, deal)
                 : launch_pdl(unpack_kernel<T, VEC, false>, grid, dim3(THREADS), 0, st, p, deal);
}

template <typename T>
cudaError_t typed(const Rows8Params& p, bool pack, int num_sms, cudaStream_t st) {
  const void* const X = pack ? p.X : p.X_out;
  const void* const q = pack ? p.q_out : p.q;
  // values a thread, by what the rows' lengths and places allow
  auto fits = [&](int vec, int bytes) {  // bytes: of an access to X
    return p.H % vec == 0 && p.ldq % vec == 0 && p.ldx * sizeof(T) % bytes == 0 &&
           reinterpret_cast<uintptr_t>(X) % bytes == 0 && reinterpret_cast<uintptr_t>(q) % vec == 0;
  };
  constexpr int HALF = 16 / sizeof(T);
  if (fits(16, 16)) return pack ? pack_as<T, 16>(p, num_sms, st) : unpack_as<T, 16>(p, num_sms, st);
  if (fits(HALF, 16)) return pack ? pack_as<T, HALF>(p, num_sms, st) : unpack_as<T, HALF>(p, num_sms, st);
  return pack ? pack_as<T, 1>(p, num_sms, st) : unpack_as<T, 1>(p, num_sms, st);
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
