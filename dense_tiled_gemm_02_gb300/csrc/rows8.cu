// rows8.cu -- rows to 8 bits and back: blocks of 32 values with a power of two,
// and whole rows with one fp32 scale.
//
// Bound by HBM: 16 values a thread and turn, 16-byte accesses on both sides
// (with 8 of a 16-bit type, 8-byte ones on the 8-bit side, unpacking takes 36
// instead of 34.6 us).  Packing has four turns in flight (two: 36 us instead of
// 30), unpacking takes two, one after the other (four, two in flight: 34.6 instead
// of 31.5; all in flight: 40).  Two lanes share a block's exponent and find its
// largest magnitude by a shuffle.  Integers are made and read by additions in
// the last place and byte permutes, since conversion instructions, at a quarter
// of the rate, bounded the first form (40 us; 64-bit divisions for an item's row
// another 5).
//
// Measured (one GB300, 16384 x 4096 bf16, floor 30.1 us each way): block rows 30.6
// us and back 31.9, scaled rows 31.5 and back 31.9; in fp32 (50.2) 49 and 69, 48
// and 69; 16384 x 4095, whose rows are of any alignment, 57 and 53, 60 and 52 (an
// access an element: 174 and 137, 94 and 132), scaled rows in fp32 84 and 66.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "rows.cuh"

namespace gb300 {

namespace {

constexpr int THREADS = DEAL_THREADS;

// ---------------------------------------------------------------- block rows
// LANES lanes to 32 values.  ANY: rows of any alignment.
template <typename T, int VEC, bool ANY>
__global__ void __launch_bounds__(THREADS)
    pack_blocks_kernel(const Rows8Params p, const Deal deal) {
  const int blocks = (p.H + ROW_BLOCK - 1) / ROW_BLOCK;
  constexpr int LANES = ROW_BLOCK / VEC, U = ANY ? 2 : 4;
  const Items all = block_items(p.T, deal, blockIdx.x);
  const Divisor& lanes = deal.lanes;
  pdl_wait();
  pdl_trigger();
  // (whole warps stay together: lanes past the last item load nothing but shuffle)
  for (uint32_t at0 = threadIdx.x; at0 - (threadIdx.x & 31) < all.n; at0 += U * THREADS) {
    Vec<T, VEC> x[U];
    Around<T, VEC> around[ANY ? U : 1];
    long long row[U];
    int i[U];
    Range n[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t at = all.at + at0 + u * THREADS, r = divide(at, lanes);
      row[u] = all.row + r;
      i[u] = static_cast<int>(at - r * lanes.d) * VEC;
      n[u] = at0 + u * THREADS < all.n ? elements_at<VEC>(i[u], p.H) : Range{0, 0};
      const long long from_at = row[u] * p.ldx + i[u];
      const T* const from = static_cast<const T*>(p.X) + from_at;
      if constexpr (ANY) {
        if (n[u].to > 0) fetch(around[u], from, n[u], inside<VEC>(from_at, p.T, p.ldx, p.H));
      } else {
        x[u] = Vec<T, VEC>{};
        if (n[u].to > 0) x[u] = load_vec<T, VEC>(from);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if constexpr (ANY) x[u] = shifted<false>(around[u], n[u]);
      uint32_t top = vec_top(x[u]);
#pragma unroll
      for (int d = LANES / 2; d > 0; d >>= 1) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
      const uint32_t e = block_exponent(top, least_exponent<T>());
      const float inverse = block_inverse(e);
      float v[VEC];
#pragma unroll
      for (int j = 0; j < VEC; ++j) v[j] = widen(x[u].v[j]);
      const auto q = block_integers(v, inverse);
      int8_t* const to = p.q_out + row[u] * p.ldq + i[u];
      if constexpr (ANY)
        store_shifted<false>(to, i[u], n[u], q);
      else if (n[u].to > 0)
        store_vec(to, q);
      if (n[u].to > 0 && i[u] % ROW_BLOCK == 0)
        static_cast<uint8_t*>(p.scales_out)[row[u] * blocks + i[u] / ROW_BLOCK] = e;
    }
  }
}

template <typename T, int VEC, bool BLOCKS, bool ANY>
__global__ void __launch_bounds__(THREADS)
    unpack_kernel(const Rows8Params p, const Deal deal) {
  const int blocks = (p.H + ROW_BLOCK - 1) / ROW_BLOCK;
  const Items all = block_items(p.T, deal, blockIdx.x);
  const Divisor& lanes = deal.lanes;
  pdl_wait();
  pdl_trigger();
  for (uint32_t at0 = threadIdx.x; at0 - (threadIdx.x & 31) < all.n; at0 += THREADS) {
    const uint32_t at = all.at + at0, r = divide(at, lanes);
    const long long row = all.row + r;
    const int i = static_cast<int>(at - r * lanes.d) * VEC;
    const Range n = at0 < all.n ? elements_at<VEC>(i, p.H) : Range{0, 0};
    Vec<int8_t, VEC> q{};
    Around<int8_t, VEC> around;
    float step = 0.f;
    if (n.to > 0) {
      const long long from_at = row * p.ldq + i;
      if constexpr (ANY)
        fetch(around, p.q + from_at, n, inside<VEC>(from_at, p.T, p.ldq, p.H));
      else
        q = load_vec<int8_t, VEC>(p.q + from_at);
      step = BLOCKS ? block_step(static_cast<const uint8_t*>(p.scales)[row * blocks + i / ROW_BLOCK])
                    : static_cast<const float*>(p.scales)[row];
    }
    if constexpr (ANY) q = shifted<false>(around, n);
    float v[VEC];
    times_step<BLOCKS>(q, step, v);
    if (!(fabsf(step) < largest<T>() / 256.f)) {  // else nothing can round past the finite values
#pragma unroll
      for (int j = 0; j < VEC; ++j) v[j] = finite(v[j], largest<T>());
    }
    const Vec<T, VEC> x = narrowed<T, VEC>(v);
    T* const to = static_cast<T*>(p.X_out) + row * p.ldx + i;
    if constexpr (ANY)
      store_shifted<false>(to, i, n, x);
    else if (n.to > 0)
      store_vec(to, x);
  }
}

// ---------------------------------------------------------------- scaled rows
// A block (or, blockDim.x = 32, a warp) a row, whose threads hold NV vectors
// each, or with NV = 0 (rows too long) read them again.
// Registers: what 1024 threads have; those that hold fp32 of any alignment keep to
// 48, at which five blocks of 256 threads fit an SM (16384 x 4095 84 us; with 52, so
// that four fit, 91).
template <typename T, int VEC, int NV, bool ANY>
__global__ void __maxnreg__(ANY && sizeof(T) == 4 ? 48 : 64) pack_rows_kernel(const Rows8Params p) {
  __shared__ float2 part[32];
  const long long row = static_cast<long long>(blockIdx.x) * blockDim.y + threadIdx.y;
  const int step = blockDim.x * VEC, first = threadIdx.x * VEC;
  const int warp_first = (threadIdx.x & ~31) * VEC;  // whole warps stay together
  pdl_wait();
  pdl_trigger();
  if (row >= p.T) return;
  const T* const X = static_cast<const T*>(p.X) + row * p.ldx;
  constexpr int N = NV > 0 ? NV : 1;
  Vec<T, VEC> x[N];
  Around<T, VEC> around[ANY ? N : 1];
  uint32_t top = 0u;
  float sum = 0.f;
  auto load = [&](int k, int i) {
    const Range n = elements_at<VEC>(i, p.H);
    if (n.to == 0) return;
    if constexpr (ANY)
      fetch(around[k], X + i, n, inside<VEC>(row * p.ldx + i, p.T, p.ldx, p.H));
    else
      x[k] = load_vec<T, VEC>(X + i);
  };
  auto settle = [&](int k, int i) {
    if constexpr (ANY) x[k] = shifted<false>(around[k], elements_at<VEC>(i, p.H));
  };
  if constexpr (NV > 0) {
#pragma unroll
    for (int k = 0; k < NV; ++k) load(k, first + k * step);
#pragma unroll
    for (int k = 0; k < NV; ++k)
      if (first + k * step < p.H) {
        settle(k, first + k * step);
        top = max(top, vec_top(x[k]));
      }
  } else {
    for (int i = first; i < p.H; i += step) {
      load(0, i);
      settle(0, i);
      top = max(top, vec_top(x[0]));
    }
  }
  row_reduce<false, true>(sum, top, blockDim.x >> 5, part);
  const RowScale s = row_scale(__uint_as_float(top), 1.f);
  if (threadIdx.x == 0) static_cast<float*>(p.scales_out)[row] = s.scale;
  auto store = [&](const Vec<T, VEC>& v, int i) {
    float f[VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j) f[j] = widen(v.v[j]);
    const auto q = row_integers<true>(f, s);
    int8_t* const to = p.q_out + row * p.ldq + i;
    if constexpr (ANY)
      store_shifted<false>(to, i, elements_at<VEC>(i, p.H), q);
    else if (i < p.H)
      store_vec(to, q);
  };
  if constexpr (NV > 0) {
#pragma unroll
    for (int k = 0; k < NV; ++k)
      if (warp_first + k * step < p.H) store(x[k], first + k * step);
  } else {
    for (int i = first, i0 = warp_first; i0 < p.H; i += step, i0 += step) {
      load(0, i);
      settle(0, i);
      store(x[0], i);
    }
  }
}

// ---------------------------------------------------------------- launches
template <typename T, int VEC, bool ANY>
cudaError_t pack_as(const Rows8Params& p, int num_sms, cudaStream_t st) {
  if (p.block) {
    const int lanes = (p.H + ROW_BLOCK - 1) / ROW_BLOCK * (ROW_BLOCK / VEC);
    dim3 grid;
    const Deal deal = deal_of(p.T, lanes, 4, num_sms, grid);
    return launch_pdl(pack_blocks_kernel<T, VEC, ANY>, grid, dim3(THREADS), 0, st, p, deal);
  }
  // few rows are spread over more threads
  constexpr int MOST = VEC == 16 || ANY ? 2 : 4;
  const int n = (p.H + VEC - 1) / VEC;
  int nv = p.T >= num_sms ? MOST : 1;
  while (nv > 1 && n <= 16 * nv) nv /= 2;
  if (nv == 1 && n > 1024) nv = MOST;
  const bool again = n > 1024 * nv;
  const int threads = again ? 1024 : (((n + nv - 1) / nv) + 31) / 32 * 32, rows = threads == 32 ? 4 : 1;
  const dim3 grid(static_cast<unsigned>((p.T + rows - 1) / rows)), block(threads, rows);
  if (again) return launch_pdl(pack_rows_kernel<T, VEC, 0, ANY>, grid, block, 0, st, p);
  if (nv == 1) return launch_pdl(pack_rows_kernel<T, VEC, 1, ANY>, grid, block, 0, st, p);
  if constexpr (MOST >= 4)
    if (nv == 4) return launch_pdl(pack_rows_kernel<T, VEC, 4, ANY>, grid, block, 0, st, p);
  return launch_pdl(pack_rows_kernel<T, VEC, 2, ANY>, grid, block, 0, st, p);
}
template <typename T, int VEC, bool ANY>
cudaError_t unpack_as(const Rows8Params& p, int num_sms, cudaStream_t st) {
  const int lanes = (p.H + VEC - 1) / VEC;
  dim3 grid;
  const Deal deal = deal_of(p.T, lanes, 2, num_sms, grid);
  return p.block ? launch_pdl(unpack_kernel<T, VEC, true, ANY>, grid, dim3(THREADS), 0, st, p, deal)
                 : launch_pdl(unpack_kernel<T, VEC, false, ANY>, grid, dim3(THREADS), 0, st, p, deal);
}
template <typename T, int VEC, bool ANY>
cudaError_t either_way(const Rows8Params& p, bool pack, int num_sms, cudaStream_t st) {
  return pack ? pack_as<T, VEC, ANY>(p, num_sms, st) : unpack_as<T, VEC, ANY>(p, num_sms, st);
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
  if (fits(16, 16)) return either_way<T, 16, false>(p, pack, num_sms, st);
  if (fits(HALF, 16)) return either_way<T, HALF, false>(p, pack, num_sms, st);
  return either_way<T, 32 / sizeof(T), true>(p, pack, num_sms, st);
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
