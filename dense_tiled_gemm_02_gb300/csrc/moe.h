// moe.h -- parameters and launches of the mixture-of-experts and 4-bit-weight
// kernels (route.cu, permute.cu, grouped.cu, w4.cu), used by moe_host.cu.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "common.h"

namespace gb300 {

// The driver's cuTensorMapEncodeTiled, or null (gemm_host.cu).
void* tensor_map_encoder();

// Status bit beside STATUS_TIMEOUT: offsets or row indices out of range.
constexpr uint32_t STATUS_BAD_INDEX = 2u;
// Debug flag beside DBG_SKIP_FIRST_FILL: the same in the first unit alone.
constexpr int DBG_SKIP_ONE_FILL = 2;

// True in one lane, always the same, of a converged warp.  The branch of a
// thread that issues tcgen05 or TMA instructions is taken on this and not on
// a lane number: the compiler then knows that one thread runs it and keeps
// the operands in uniform registers, where the instructions read them.
// (16 tcgen05.mma of 128 x 16 x 16 from tensor memory: 290 cycles to issue
// against 1780 behind `lane == 0`.)
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "elect.sync _|q, 0xffffffff;\n\t"
      "selp.b32 %0, 1, 0, q;\n\t}"
      : "=r"(one));
  return one != 0u;
}

// Element types to fp32 and back.
__device__ __forceinline__ float widen(float x) { return x; }
__device__ __forceinline__ float widen(__half x) { return __half2float(x); }
__device__ __forceinline__ float widen(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void narrow(float v, float& x) { x = v; }
__device__ __forceinline__ void narrow(float v, __half& x) { x = __float2half_rn(v); }
__device__ __forceinline__ void narrow(float v, __nv_bfloat16& x) { x = __float2bfloat16_rn(v); }

// The rows [lo, hi) of expert e; empty, with the status set, when the offsets
// decrease or leave [0, R].
__device__ __forceinline__ int2 expert_rows(const int* offsets, int e, int R, uint32_t* status) {
  int2 r = make_int2(offsets[e], offsets[e + 1]);
  if (r.x < 0 || r.y < r.x || r.y > R) {
    atomicOr(status, STATUS_BAD_INDEX);
    r.y = r.x = 0;
  }
  return r;
}

// ---------------------------------------------------------------- routing (route.cu)
struct RouteParams {
  int T, E, k, type, normalize;
  long long ld;
  const void* logits;
  int* experts;
  float* gates;
  int* offsets;
  int* row_slot;
  int* slot_row;
  int blocks, tokens_per_block;  // several-block form
  int* hist;                     // [blocks][ld_hist]: the blocks' slots of each expert
  int ld_hist;                   // E up to a multiple of four
};
// Blocks of the forward kernel; 1: one block does the whole call.
int route_blocks(long long T, int k, int num_sms);
cudaError_t launch_route(const RouteParams& p, cudaStream_t st);

struct RouteBackwardParams {
  int T, E, k, type, normalize;
  long long ld;
  const void* logits;
  const int* experts;
  const float* gates;
  const float* dgates;
  void* dlogits;
  int num_sms;
};
cudaError_t launch_route_backward(const RouteBackwardParams& p, cudaStream_t st);

// ---------------------------------------------------------------- row movement (permute.cu)
struct PermuteParams {
  long long T, H;
  int k, type;
  long long ld_tokens, ld_rows;
  const void* tokens;  // X, or dY
  void* tokens_out;    // Y
  const void* rows;    // Ys
  void* rows_out;      // Xs, or dYs
  const int* row_slot;
  const int* slot_row;
  const float* gates;
  float* dgates;
  uint32_t* status;
};
cudaError_t launch_gather(const PermuteParams& p, int num_sms, cudaStream_t st);
cudaError_t launch_combine(const PermuteParams& p, int num_sms, cudaStream_t st);
cudaError_t launch_combine_backward(const PermuteParams& p, int num_sms, cudaStream_t st);

// ---------------------------------------------------------------- grouped products (grouped.cu)
struct GroupedParams {
  int grad;            // GEMM_GROUPED_GRAD: the sum runs over an expert's rows
  int E, R, K, N;
  int f_mn;            // features operand MN-major (B row-major)
  uint32_t idesc;      // instruction descriptor without its N field
  const int* offsets;
  const void* C;
  int d_type;          // also C's
  int d_vec;           // 16-bit D whose rows start on 16-byte boundaries
  int d_tma;           // and N a multiple of 8: stored by TMA
  long long ldc, ldd;
  void* D;
  float* partial;      // grouped_partial_bytes()
  unsigned* counters;  // one per CTA, zero between calls (cleared by the host after a timeout)
  CUtensorMap* maps;   // grad: the experts' maps of the features, then of the rows operand
  uint32_t* status;
  unsigned long long timeout_ns;
  int debug_flags;
};
// Sets the kernel up on the current device; how many of its units (CTA pairs
// when wide, else CTAs) run at once, 0 on failure.
int prepare_grouped(bool wide, int d_type, int num_sms);
size_t grouped_partial_bytes(bool wide, int units);
// Tensor maps: the features operand; the rows operand in boxes of 128 rows
// and of 32 (rows form; in grad x128 has 64 x 64 boxes, x32 is not read, and
// both are copied into p.maps per expert);
// D in boxes of 64 columns x 32 rows (when d_tma).
cudaError_t launch_grouped(bool wide, const CUtensorMap& f, const CUtensorMap& x128,
                           const CUtensorMap& x32, const CUtensorMap& d, const GroupedParams& p,
                           int units, cudaStream_t st);

// ---------------------------------------------------------------- 4-bit weights (w4.cu)
struct W4Params {
  int E, R, K, N, group, groups;
  int x_type, scale_type, d_type;
  long long ldx, ldd;
  const void* X;
  const uint8_t* W;
  const void* scales;
  const uint8_t* zeros;  // null: 8
  const int* offsets;    // null: all rows to expert 0
  void* D;
  uint32_t* status;
  int num_sms;
  uint32_t nibbles, nibble_base;  // set by launch_w4 (see expand in w4.cu)
};
cudaError_t launch_w4(const W4Params& p, cudaStream_t st);

}  // namespace gb300
