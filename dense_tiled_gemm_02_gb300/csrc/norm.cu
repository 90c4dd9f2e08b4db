// norm.cu -- a residual's addition and the root-mean-square norm of a row, out
// in its type or in 8 bits with a scale, and the gradients.
//
//   h = x + residual,  r = 1 / sqrt(mean h^2 + eps),  y = h r w
//   dx = r (w dy - h r^2 / H sum(w dy h)) + dresidual,  dw = sum over rows of dy h r
//
// Bound by HBM: each row is read once and stays in its threads' registers.
// The 8-bit form needs the largest |y| too, which is r max |h w|: known with
// the sum of squares, so that one reduction serves both, and r falls out of the
// integers y / scale = 127 h w / max |h w|.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "rows.cuh"

namespace gb300 {

namespace {

constexpr int MAX_WARPS = 32;
constexpr int BACKWARD_BLOCKS = 8;  // per SM, at most
constexpr int RING_MOST = 4;        // stages of a block's ring
constexpr int RING_BYTES = 212 * 1024;  // of all blocks of an SM
constexpr uint64_t RING_TIMEOUT_NS = 2000000000ull;

// VEC weights of the rows' type or of fp32, from column i.
template <typename T, int VEC>
__device__ __forceinline__ void load_weight(const void* w, bool f32, int i, float (&o)[VEC]) {
  if (f32) {
    const auto v = load_vec<float, VEC>(static_cast<const float*>(w) + i);
#pragma unroll
    for (int j = 0; j < VEC; ++j) o[j] = v.v[j];
  } else {
    const auto v = load_vec<T, VEC>(static_cast<const T*>(w) + i);
#pragma unroll
    for (int j = 0; j < VEC; ++j) o[j] = widen(v.v[j]);
  }
}

// h = x + residual in T, and its sum of squares and largest |h w|.
template <typename T, int VEC, bool I8>
__device__ __forceinline__ void row_sums(const NormParams& p, const Vec<T, VEC>& h, int i,
                                         float& sum, uint32_t& top) {
  float w[VEC];
  if constexpr (I8) load_weight<T, VEC>(p.weight, p.weight_type == T_F32, i, w);
#pragma unroll
  for (int j = 0; j < VEC; ++j) {
    const float v = widen(h.v[j]);
    sum = fmaf(v, v, sum);
    if constexpr (I8) top = max(top, magnitude(v * w[j]));
  }
}

template <typename T, int VEC>
__device__ __forceinline__ void add_residual(Vec<T, VEC>& h, const Vec<T, VEC>& r) {
#pragma unroll
  for (int j = 0; j < VEC; ++j) narrow(widen(h.v[j]) + widen(r.v[j]), h.v[j]);
}

template <typename T, int VEC, bool I8>
__device__ __forceinline__ void store_y(const NormParams& p, long long row, const Vec<T, VEC>& h,
                                        int i, float r, const RowScale& q) {
  float w[VEC];
  load_weight<T, VEC>(p.weight, p.weight_type == T_F32, i, w);
  if constexpr (I8) {
    float v[VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j) v[j] = widen(h.v[j]) * w[j];
    store_row_integers(static_cast<int8_t*>(p.y) + row * p.ldy + i, v, q);
  } else {
    Vec<T, VEC> y;
#pragma unroll
    for (int j = 0; j < VEC; ++j) narrow(widen(h.v[j]) * r * w[j], y.v[j]);
    store_vec(static_cast<T*>(p.y) + row * p.ldy + i, y);
  }
}

// A row's blockDim.x threads hold NV vectors each, or with NV = 0 (rows too
// long for that) read them again, from h where there is a residual.  blockDim.y
// rows a block, more than one only with one warp a row.
template <typename T, int VEC, int NV, bool I8>
__global__ void __launch_bounds__(1024) norm_kernel(const NormParams p) {
  __shared__ float2 part[MAX_WARPS];
  const int warps = blockDim.x >> 5;
  const long long row = static_cast<long long>(blockIdx.x) * blockDim.y + threadIdx.y;
  pdl_wait();
  pdl_trigger();
  if (row >= p.T) return;  // (a whole warp, which shares nothing)
  const T* const x = static_cast<const T*>(p.x) + row * p.ldx;
  const T* const res = p.residual ? static_cast<const T*>(p.residual) + row * p.ldr : nullptr;
  T* const hout = static_cast<T*>(p.h) + row * p.ldh;
  const int step = blockDim.x * VEC, first = threadIdx.x * VEC;
  constexpr int N = NV > 0 ? NV : 1;
  Vec<T, VEC> h[N];
  float sum = 0.f;
  uint32_t top = 0u;
  if constexpr (NV > 0) {
#pragma unroll
    for (int k = 0; k < NV; ++k)
      if (first + k * step < p.H) h[k] = load_vec<T, VEC>(x + first + k * step);
    if (res) {
      Vec<T, VEC> r[NV];
#pragma unroll
      for (int k = 0; k < NV; ++k)
        if (first + k * step < p.H) r[k] = load_vec<T, VEC>(res + first + k * step);
#pragma unroll
      for (int k = 0; k < NV; ++k)
        if (first + k * step < p.H) {
          add_residual(h[k], r[k]);
          store_vec(hout + first + k * step, h[k]);
        }
    }
#pragma unroll
    for (int k = 0; k < NV; ++k)
      if (first + k * step < p.H) row_sums<T, VEC, I8>(p, h[k], first + k * step, sum, top);
  } else {
    for (int i = first; i < p.H; i += step) {
      h[0] = load_vec<T, VEC>(x + i);
      if (res) {
        add_residual(h[0], load_vec<T, VEC>(res + i));
        store_vec(hout + i, h[0]);
      }
      row_sums<T, VEC, I8>(p, h[0], i, sum, top);
    }
  }
  row_reduce(sum, top, warps, part);
  const float r = 1.f / sqrtf(sum / static_cast<float>(p.H) + p.eps);
  const RowScale q = I8 ? row_scale(__uint_as_float(top), r) : RowScale{};
  if (threadIdx.x == 0) {
    if (p.rstd) p.rstd[row] = r;
    if constexpr (I8) p.scales[row] = q.scale;
  }
  if constexpr (NV > 0) {
#pragma unroll
    for (int k = 0; k < NV; ++k)
      if (first + k * step < p.H) store_y<T, VEC, I8>(p, row, h[k], first + k * step, r, q);
  } else {
    const T* const from = res ? hout : x;  // this thread's own stores
    for (int i = first; i < p.H; i += step)
      store_y<T, VEC, I8>(p, row, load_vec<T, VEC>(from + i), i, r, q);
  }
}

// ---------------------------------------------------------------- backward
// VEC values of h from column i of a row: of type T, or block rows.
template <typename T, int VEC, bool HELD>
struct HRow {
  const T* h;
  const int8_t* q;
  const uint8_t* e;
  __device__ __forceinline__ HRow(const NormBackwardParams& p, long long row) {
    if constexpr (HELD) {
      q = static_cast<const int8_t*>(p.h) + row * p.ldh;
      e = p.E + row * ((p.H + ROW_BLOCK - 1) / ROW_BLOCK);
    } else {
      h = static_cast<const T*>(p.h) + row * p.ldh;
    }
  }
  struct Raw {
    Vec<std::conditional_t<HELD, int8_t, T>, VEC> v;
    uint8_t e;
  };
  __device__ __forceinline__ void load(int i, Raw& r) const {
    if constexpr (HELD) {
      r.v = load_vec<int8_t, VEC>(q + i);
      r.e = e[i / ROW_BLOCK];
    } else {
      r.v = load_vec<T, VEC>(h + i);
    }
  }
  static __device__ __forceinline__ void widen_to(const Raw& r, float (&o)[VEC]) {
    if constexpr (HELD) {
      const float step = block_step(r.e);
#pragma unroll
      for (int j = 0; j < VEC; ++j) o[j] = static_cast<float>(r.v.v[j]) * step;
    } else {
#pragma unroll
      for (int j = 0; j < VEC; ++j) o[j] = widen(r.v.v[j]);
    }
  }
};

template <typename T, int VEC>
__device__ __forceinline__ void store_dx(const NormBackwardParams& p, long long row, int i,
                                         const float (&dy)[VEC], const float (&h)[VEC],
                                         const float (&w)[VEC], float r, float c,
                                         const Vec<T, VEC>& res) {
  Vec<T, VEC> o;
#pragma unroll
  for (int j = 0; j < VEC; ++j) {
    float v = r * (dy[j] * w[j] - h[j] * c);
    if (p.dresidual) v += widen(res.v[j]);
    narrow(v, o.v[j]);
  }
  store_vec(static_cast<T*>(p.dx) + row * p.ldx + i, o);
}

// Blocks take rows in turn; a thread's columns are the same in all of them, so
// that it sums their dweight in registers (NV = 0: in the block's own row of
// `partial`) and no two threads share a sum.
template <typename T, int VEC, int NV, bool HELD>
__global__ void __launch_bounds__(512) norm_backward_kernel(const NormBackwardParams p) {
  __shared__ float2 part[2][MAX_WARPS];
  constexpr int N = NV > 0 ? NV : 1;
  const int warps = blockDim.x >> 5;
  const int step = blockDim.x * VEC, first = threadIdx.x * VEC;
  const bool w32 = p.weight_type == T_F32;
  float* const mine = p.partial + static_cast<long long>(blockIdx.x) * p.H;
  float dw[N][VEC] = {};
  pdl_wait();
  pdl_trigger();
  if constexpr (NV == 0) {
    if (p.dweight)
      for (int i = first; i < p.H; i += step)
        for (int j = 0; j < VEC; ++j) mine[i + j] = 0.f;
  }
  int turn = 0;
  for (long long row = blockIdx.x; row < p.T; row += gridDim.x, turn ^= 1) {
    const HRow<T, VEC, HELD> hrow(p, row);
    const T* const dyrow = static_cast<const T*>(p.dy) + row * p.ldy;
    const T* const resrow = static_cast<const T*>(p.dresidual) + row * p.ldr;
    const float r = p.rstd[row];
    float sum = 0.f;
    uint32_t top = 0u;
    auto dot = [&](const float (&dy)[VEC], const float (&h)[VEC], int i) {
      float w[VEC];
      load_weight<T, VEC>(p.weight, w32, i, w);
#pragma unroll
      for (int j = 0; j < VEC; ++j) sum = fmaf(dy[j] * w[j], h[j], sum);
    };
    if constexpr (NV > 0) {
      Vec<T, VEC> dyv[NV], res[NV];
      typename HRow<T, VEC, HELD>::Raw hv[NV];
#pragma unroll
      for (int k = 0; k < NV; ++k)
        if (first + k * step < p.H) {
          dyv[k] = load_vec<T, VEC>(dyrow + first + k * step);
          hrow.load(first + k * step, hv[k]);
          if (p.dresidual) res[k] = load_vec<T, VEC>(resrow + first + k * step);
        }
      float dy[VEC], h[VEC], w[VEC];
#pragma unroll
      for (int k = 0; k < NV; ++k)
        if (first + k * step < p.H) {
          HRow<T, VEC, HELD>::widen_to(hv[k], h);
#pragma unroll
          for (int j = 0; j < VEC; ++j) {
            dy[j] = widen(dyv[k].v[j]);
            dw[k][j] = fmaf(dy[j], h[j] * r, dw[k][j]);
          }
          dot(dy, h, first + k * step);
        }
      row_reduce(sum, top, warps, part[turn]);
      const float c = r * r * (sum / static_cast<float>(p.H));
#pragma unroll
      for (int k = 0; k < NV; ++k)
        if (first + k * step < p.H) {
          HRow<T, VEC, HELD>::widen_to(hv[k], h);
#pragma unroll
          for (int j = 0; j < VEC; ++j) dy[j] = widen(dyv[k].v[j]);
          load_weight<T, VEC>(p.weight, w32, first + k * step, w);
          store_dx<T, VEC>(p, row, first + k * step, dy, h, w, r, c, res[k]);
        }
    } else {
      float dy[VEC], h[VEC], w[VEC];
      typename HRow<T, VEC, HELD>::Raw raw;
      auto load = [&](int i) {
        const Vec<T, VEC> v = load_vec<T, VEC>(dyrow + i);
        hrow.load(i, raw);
        HRow<T, VEC, HELD>::widen_to(raw, h);
#pragma unroll
        for (int j = 0; j < VEC; ++j) dy[j] = widen(v.v[j]);
      };
      for (int i = first; i < p.H; i += step) {
        load(i);
        dot(dy, h, i);
        if (p.dweight)
#pragma unroll
          for (int j = 0; j < VEC; ++j) mine[i + j] = fmaf(dy[j], h[j] * r, mine[i + j]);
      }
      row_reduce(sum, top, warps, part[turn]);
      const float c = r * r * (sum / static_cast<float>(p.H));
      for (int i = first; i < p.H; i += step) {
        load(i);
        load_weight<T, VEC>(p.weight, w32, i, w);
        Vec<T, VEC> res{};
        if (p.dresidual) res = load_vec<T, VEC>(resrow + i);
        store_dx<T, VEC>(p, row, i, dy, h, w, r, c, res);
      }
    }
  }
  if constexpr (NV > 0) {
    if (p.dweight) {
#pragma unroll
      for (int k = 0; k < NV; ++k)
        if (first + k * step < p.H)
#pragma unroll
          for (int j = 0; j < VEC; ++j) mine[first + k * step + j] = dw[k][j];
    }
  }
}

// The same with rows on their way: each block keeps the next rows of its turn in
// a ring in shared memory (bulk copies: dy, h and dresidual of a row are one
// stage), so that what is in flight does not depend on registers or on where a
// block is between its two passes over a row.  The passes read the stage twice.
template <typename T, int NV, bool HELD>
__global__ void __launch_bounds__(512)
    norm_backward_ring_kernel(const NormBackwardParams p, const int stages) {
  constexpr int VEC = 16 / sizeof(T);
  using HT = std::conditional_t<HELD, int8_t, T>;
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ float2 part[2][MAX_WARPS];
  __shared__ uint64_t bars[RING_MOST];
  __shared__ int abort_flag;
  const int warps = blockDim.x >> 5;
  const int step = blockDim.x * VEC, first = threadIdx.x * VEC;
  const uint32_t dy_bytes = p.H * sizeof(T), h_bytes = p.H * sizeof(HT);
  const uint32_t stage_bytes = dy_bytes + h_bytes + (p.dresidual ? dy_bytes : 0u);
  const uint32_t ring0 = smem_u32(ring), bar0 = smem_u32(bars);
  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) mbar_init(bar0 + 8 * s, 1);
    abort_flag = 0;
    fence_mbar_init();
    fence_proxy_async_smem();
  }
  pdl_wait();
  pdl_trigger();
  __syncthreads();
  auto load_row = [&](long long row, int s) {  // one thread
    const uint32_t bar = bar0 + 8 * s, to = ring0 + s * stage_bytes;
    mbar_arrive_expect_tx(bar, stage_bytes);
    bulk_load_1d(to, static_cast<const T*>(p.dy) + row * p.ldy, dy_bytes, bar);
    bulk_load_1d(to + dy_bytes, static_cast<const HT*>(p.h) + row * p.ldh, h_bytes, bar);
    if (p.dresidual)
      bulk_load_1d(to + dy_bytes + h_bytes, static_cast<const T*>(p.dresidual) + row * p.ldr,
                   dy_bytes, bar);
  };
  if (threadIdx.x == 0)
    for (int s = 0; s < stages; ++s) {
      const long long row = blockIdx.x + static_cast<long long>(s) * gridDim.x;
      if (row < p.T) load_row(row, s);
    }
  const int blocks = (p.H + ROW_BLOCK - 1) / ROW_BLOCK;
  float dw[NV][VEC] = {};
  float w[NV][VEC];
  uint32_t e_next[NV] = {};
  float r_next = 0.f;
  auto prefetch = [&](long long row) {  // what does not come by the ring
    if (row >= p.T) return;
    r_next = p.rstd[row];
    if constexpr (HELD) {
#pragma unroll
      for (int k = 0; k < NV; ++k)
        if (first + k * step < p.H) e_next[k] = p.E[row * blocks + (first + k * step) / ROW_BLOCK];
    }
  };
  prefetch(blockIdx.x);
#pragma unroll
  for (int k = 0; k < NV; ++k)
    if (first + k * step < p.H)
      load_weight<T, VEC>(p.weight, p.weight_type == T_F32, first + k * step, w[k]);
  int s = 0, turn = 0;
  uint32_t ph = 0;
  long long row = blockIdx.x;
  for (; row < p.T; row += gridDim.x, turn ^= 1) {
    const float r = r_next;
    float scale[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) scale[k] = HELD ? block_step(e_next[k]) : 1.f;
    prefetch(row + gridDim.x);
    // (a thread that gives up raises the flag before the barrier in row_reduce,
    // after which all see it)
    bounded_wait(bar0 + 8 * s, ph, &abort_flag, p.status, STATUS_TIMEOUT, RING_TIMEOUT_NS);
    const T* const dyrow = reinterpret_cast<const T*>(ring + s * stage_bytes);
    const HT* const hrow = reinterpret_cast<const HT*>(ring + s * stage_bytes + dy_bytes);
    const T* const resrow = reinterpret_cast<const T*>(ring + s * stage_bytes + dy_bytes + h_bytes);
    auto widen_h = [&](int k, float (&h)[VEC]) {
      const auto v = load_vec<HT, VEC>(hrow + first + k * step);
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        if constexpr (HELD)
          h[j] = fmaf(from_byte(v, j), scale[k], scale[k] * -BYTE_BIAS);
        else
          h[j] = widen(v.v[j]);
      }
    };
    float sum = 0.f;
    uint32_t top = 0u;
#pragma unroll
    for (int k = 0; k < NV; ++k)
      if (first + k * step < p.H) {
        float h[VEC];
        widen_h(k, h);
        const auto dy = load_vec<T, VEC>(dyrow + first + k * step);
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          const float t = widen(dy.v[j]) * h[j];
          dw[k][j] = fmaf(t, r, dw[k][j]);
          sum = fmaf(t, w[k][j], sum);
        }
      }
    if (warps == 1) __syncwarp();
    row_reduce(sum, top, warps, part[turn]);
    if (*const_cast<volatile int*>(&abort_flag)) break;
    // every thread is past its second pass over the previous row: its stage
    // takes the row after those under way
    if (threadIdx.x == 0 && row >= gridDim.x) {
      const long long next = row + static_cast<long long>(stages - 1) * gridDim.x;
      if (next < p.T) load_row(next, s == 0 ? stages - 1 : s - 1);
    }
    const float c = r * r * (sum / static_cast<float>(p.H));
#pragma unroll
    for (int k = 0; k < NV; ++k)
      if (first + k * step < p.H) {
        float h[VEC], d[VEC];
        widen_h(k, h);
        const auto dy = load_vec<T, VEC>(dyrow + first + k * step);
#pragma unroll
        for (int j = 0; j < VEC; ++j) d[j] = widen(dy.v[j]);
        Vec<T, VEC> res{};
        if (p.dresidual) res = load_vec<T, VEC>(resrow + first + k * step);
        store_dx<T, VEC>(p, row, first + k * step, d, h, w[k], r, c, res);
      }
    if (++s == stages) {
      s = 0;
      ph ^= 1u;
    }
  }
  if (p.dweight) {
    float* const mine = p.partial + static_cast<long long>(blockIdx.x) * p.H;
#pragma unroll
    for (int k = 0; k < NV; ++k)
      if (first + k * step < p.H)
#pragma unroll
        for (int j = 0; j < VEC; ++j) mine[first + k * step + j] = dw[k][j];
  }
  // after a wait that ran out: copies still under way land before the block leaves
  if (row < p.T && threadIdx.x == 0) {
    const uint64_t t0 = global_timer_ns();
    while (global_timer_ns() - t0 < 1000000ull) __nanosleep(1000);
  }
}

// dweight: the blocks' partial sums, 32 columns a block, added up by 32 warps
// in turn and then in warp order.
__global__ void __launch_bounds__(1024)
    norm_dweight_kernel(const float* partial, int rows, int H, float* dweight) {
  __shared__ float part[32][33];
  const int i = blockIdx.x * 32 + threadIdx.x;
  pdl_wait();
  pdl_trigger();
  float sum = 0.f;
  if (i < H) {
#pragma unroll 4
    for (int r = threadIdx.y; r < rows; r += 32) sum += partial[static_cast<long long>(r) * H + i];
  }
  part[threadIdx.y][threadIdx.x] = sum;
  __syncthreads();
  if (threadIdx.y == 0 && i < H) {
    sum = 0.f;
#pragma unroll
    for (int y = 0; y < 32; ++y) sum += part[y][threadIdx.x];
    dweight[i] = sum;
  }
}

// ---------------------------------------------------------------- launches
int up32(long long n) { return static_cast<int>((n + 31) / 32 * 32); }

template <typename T, int VEC, bool I8>
cudaError_t launch_forward(const NormParams& p, int num_sms, cudaStream_t st) {
  const int n = (p.H + VEC - 1) / VEC;
  // Vectors a thread: four keep enough in flight where there are rows for all
  // SMs; few rows are spread over more threads.
  constexpr int MOST = VEC == 1 ? 8 : 4;  // by the registers of 1024 threads
  const int most = p.T >= 4ll * num_sms ? MOST : p.T >= num_sms ? MOST / 2 : 1;
  int nv = 1;
  while (nv < most && n > 32 * nv) nv *= 2;
  while (nv < MOST && n > 1024 * nv) nv *= 2;
  const bool again = n > 1024 * nv;
  const int threads = again ? 1024 : up32((n + nv - 1) / nv);
  const int rows = threads == 32 ? 4 : 1;
  const dim3 grid(static_cast<unsigned>((p.T + rows - 1) / rows)), block(threads, rows);
  if (again) return launch_pdl(norm_kernel<T, VEC, 0, I8>, grid, block, 0, st, p);
  if constexpr (MOST >= 8)
    if (nv == 8) return launch_pdl(norm_kernel<T, VEC, 8, I8>, grid, block, 0, st, p);
  if (nv == 4) return launch_pdl(norm_kernel<T, VEC, 4, I8>, grid, block, 0, st, p);
  if (nv == 2) return launch_pdl(norm_kernel<T, VEC, 2, I8>, grid, block, 0, st, p);
  return launch_pdl(norm_kernel<T, VEC, 1, I8>, grid, block, 0, st, p);
}

// Threads and vectors a thread of a ring block: as many vectors as its sums of
// dweight leave registers for (32 sums, 16 in fp32 whose values take twice the
// shared-memory reads), since every thread more lengthens the row's reduction
// (16384 x 4096 bf16: four vectors 90 us, two 119, one 115); 0: rows too long.
template <typename T>
int ring_threads(int H, int& nv) {
  constexpr int VEC = 16 / sizeof(T);
  const int n = H / VEC;
  for (nv = 1; nv < 4 && n > 128 * nv;) nv *= 2;
  return n <= 512 * nv ? up32((n + nv - 1) / nv) : 0;
}

// A ring kernel's blocks an SM, by registers and shared memory, and stages a
// block; false where two stages do not fit.
bool ring_shape(int stage_bytes, int threads, int sums, int& blocks, int& stages) {
  for (blocks = std::min(BACKWARD_BLOCKS, (sums > 8 ? 512 : 1024) / threads); blocks > 0; --blocks) {
    stages = std::min(RING_MOST, RING_BYTES / blocks / stage_bytes);
    if (stages >= 2) return true;
  }
  return false;
}

template <typename T, int NV, bool HELD>
cudaError_t launch_ring(const NormBackwardParams& p, int threads, int blocks, int stages,
                        int stage_bytes, cudaStream_t st) {
  auto* const kernel = norm_backward_ring_kernel<T, NV, HELD>;
  const int bytes = stages * stage_bytes;
  const cudaError_t e =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, RING_BYTES);
  if (e != cudaSuccess) return e;
  return launch_pdl(kernel, dim3(blocks), dim3(threads), bytes, st, p, stages);
}

// Rows that allow vectors and fit the ring; launched (with *blocks set) or not.
template <typename T, bool HELD>
bool try_ring(const NormBackwardParams& p, int num_sms, int& blocks, cudaError_t& e,
              cudaStream_t st) {
  constexpr int S = sizeof(T);
  if (HELD && p.H % 16 != 0) return false;  // bulk copies are of 16 bytes
  int nv, per_sm, stages;
  const int threads = ring_threads<T>(p.H, nv);
  const int stage_bytes = p.H * (S + (HELD ? 1 : S) + (p.dresidual ? S : 0));
  if (threads == 0 || !ring_shape(stage_bytes, threads, nv * 16 / S, per_sm, stages)) return false;
  blocks = static_cast<int>(std::min<long long>(p.T, static_cast<long long>(num_sms) * per_sm));
  e = nv == 1   ? launch_ring<T, 1, HELD>(p, threads, blocks, stages, stage_bytes, st)
      : nv == 2 ? launch_ring<T, 2, HELD>(p, threads, blocks, stages, stage_bytes, st)
                : launch_ring<T, 4, HELD>(p, threads, blocks, stages, stage_bytes, st);
  return true;
}

// Rows the ring does not take: of any alignment, with their values in registers
// up to 8192 of them, else read twice.
template <typename T, int VEC, bool HELD>
cudaError_t launch_backward(const NormBackwardParams& p, int blocks, cudaStream_t st) {
  const dim3 grid(blocks);
  if constexpr (VEC == 1) {
    const int nv = p.H <= 2048 ? 8 : 16;
    if (p.H <= 512 * nv) {
      const dim3 block(up32((p.H + nv - 1) / nv));
      return nv == 8 ? launch_pdl(norm_backward_kernel<T, VEC, 8, HELD>, grid, block, 0, st, p)
                     : launch_pdl(norm_backward_kernel<T, VEC, 16, HELD>, grid, block, 0, st, p);
    }
  }
  return launch_pdl(norm_backward_kernel<T, VEC, 0, HELD>, grid, dim3(512), 0, st, p);
}

// Whether rows (base, leading dimension in elements of `size` bytes) allow
// vectors of `bytes`.
bool rows_fit(const void* base, long long ld, int size, int bytes) {
  return reinterpret_cast<uintptr_t>(base) % bytes == 0 && ld * size % bytes == 0;
}

template <typename T>
cudaError_t forward_typed(const NormParams& p, int num_sms, cudaStream_t st) {
  constexpr int VEC = 16 / sizeof(T), S = sizeof(T);
  const bool vec = p.H % VEC == 0 && rows_fit(p.x, p.ldx, S, 16) &&
                   (!p.residual || (rows_fit(p.residual, p.ldr, S, 16) && rows_fit(p.h, p.ldh, S, 16))) &&
                   rows_fit(p.weight, 0, 1, 16) &&
                   (p.i8 ? rows_fit(p.y, p.ldy, 1, VEC) : rows_fit(p.y, p.ldy, S, 16));
  if (p.i8)
    return vec ? launch_forward<T, VEC, true>(p, num_sms, st) : launch_forward<T, 1, true>(p, num_sms, st);
  return vec ? launch_forward<T, VEC, false>(p, num_sms, st) : launch_forward<T, 1, false>(p, num_sms, st);
}

template <typename T, bool HELD>
cudaError_t backward_held(const NormBackwardParams& p, int num_sms, int& blocks, cudaStream_t st) {
  constexpr int VEC = 16 / sizeof(T), S = sizeof(T);
  const bool vec = p.H % VEC == 0 && rows_fit(p.dy, p.ldy, S, 16) &&
                   (HELD ? rows_fit(p.h, p.ldh, 1, VEC) : rows_fit(p.h, p.ldh, S, 16)) &&
                   (!p.dresidual || rows_fit(p.dresidual, p.ldr, S, 16)) &&
                   rows_fit(p.dx, p.ldx, S, 16) && rows_fit(p.weight, 0, 1, 16);
  cudaError_t e = cudaSuccess;
  if (vec && (!HELD || rows_fit(p.h, p.ldh, 1, 16)) && try_ring<T, HELD>(p, num_sms, blocks, e, st))
    return e;
  blocks = norm_partial_rows(p.T, num_sms);
  return vec ? launch_backward<T, VEC, HELD>(p, blocks, st) : launch_backward<T, 1, HELD>(p, blocks, st);
}

template <typename T>
cudaError_t backward_typed(const NormBackwardParams& p, int num_sms, int& blocks, cudaStream_t st) {
  return p.E ? backward_held<T, true>(p, num_sms, blocks, st)
             : backward_held<T, false>(p, num_sms, blocks, st);
}

}  // namespace

cudaError_t launch_norm(const NormParams& p, int num_sms, cudaStream_t st) {
  return p.type == T_F32    ? forward_typed<float>(p, num_sms, st)
         : p.type == T_BF16 ? forward_typed<__nv_bfloat16>(p, num_sms, st)
                            : forward_typed<__half>(p, num_sms, st);
}

int norm_partial_rows(long long T, int num_sms) {
  return static_cast<int>(std::min<long long>(T, static_cast<long long>(num_sms) * BACKWARD_BLOCKS));
}

cudaError_t launch_norm_backward(const NormBackwardParams& p, int num_sms, cudaStream_t st) {
  int blocks = 0;
  const cudaError_t e = p.type == T_F32    ? backward_typed<float>(p, num_sms, blocks, st)
                        : p.type == T_BF16 ? backward_typed<__nv_bfloat16>(p, num_sms, blocks, st)
                                           : backward_typed<__half>(p, num_sms, blocks, st);
  if (e != cudaSuccess || !p.dweight) return e;
  return launch_pdl(norm_dweight_kernel, dim3((p.H + 31) / 32), dim3(32, 32), 0, st,
                    static_cast<const float*>(p.partial), blocks, p.H, p.dweight);
}

}  // namespace gb300
