// rows.h -- parameters and launches of the operators on rows held in 8 bits
// (norm.cu, rows8.cu, i8_rows.cu), used by rows_host.cu.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "common.h"
#include "moe.h"

namespace gb300 {

constexpr int ROW_BLOCK = 32;  // values that share an exponent

// ---------------------------------------------------------------- norm (norm.cu)
struct NormParams {
  long long T;
  int H, type, weight_type, i8;
  float eps;
  long long ldx, ldr, ldh, ldy;
  const void* x;
  const void* residual;  // null: h is x
  const void* weight;
  void* h;
  void* y;
  float* scales;
  float* rstd;  // may be null
};
cudaError_t launch_norm(const NormParams& p, int num_sms, cudaStream_t st);

struct NormBackwardParams {
  long long T;
  int H, type, weight_type;
  long long ldy, ldh, ldr, ldx;  // dy, h, dresidual, dx
  const void* dy;
  const void* h;      // of type, or int8 when E
  const uint8_t* E;   // null: h is of type
  const void* weight;
  const float* rstd;
  const void* dresidual;  // may be null
  void* dx;
  float* dweight;     // may be null
  float* partial;     // norm_partial_rows() x H
  uint32_t* status;
  unsigned long long timeout_ns;
  int debug_flags;
};
// Blocks of the backward kernel, at most, each of which leaves a row of partial
// sums of dweight.
int norm_partial_rows(long long T, int H, int type, int num_sms);
// Once, before any of the launches.
cudaError_t prepare_norm_backward(int H, int type);
cudaError_t launch_norm_backward(const NormBackwardParams& p, int num_sms, cudaStream_t st);

// ---------------------------------------------------------------- rows to 8 bits (rows8.cu)
struct Rows8Params {
  long long T;
  int H, type, block;
  long long ldx, ldq;
  const void* X;
  void* X_out;
  const int8_t* q;
  int8_t* q_out;
  const void* scales;
  void* scales_out;
};
cudaError_t launch_rows8_pack(const Rows8Params& p, int num_sms, cudaStream_t st);
cudaError_t launch_rows8_unpack(const Rows8Params& p, int num_sms, cudaStream_t st);

// ---------------------------------------------------------------- products of few rows (i8_rows.cu)
struct I8RowsParams {
  int E, R, K, N, d_type;
  long long ldx, ldw, ldd;
  const int8_t* X;
  const float* x_scales;
  const int8_t* W;
  const float* w_scales;
  const int* offsets;  // null: all rows to expert 0
  void* D;
  uint32_t* status;
  int num_sms;
};
cudaError_t launch_i8_rows(const I8RowsParams& p, cudaStream_t st);

// ---------------------------------------------------------------- products of many rows (i8_tiles.cu)
// Tiles of up to `rows` (64 or 128) rows of X.  Sets the kernel up on the
// current device; how many of its CTAs (split 1) or clusters of `split` CTAs run
// at once, 0 on failure.
int prepare_i8_tiles(int rows, int d_type, int split, int num_sms);
size_t i8_tiles_partial_bytes(int rows, int units);
// Tensor maps: the weights' bytes in boxes of 128 x 128; X in fp16 in boxes of
// 64 values x `rows` rows and x 32; D as for launch_grouped.  p: the rows form
// with scales, offsets null for one expert with all rows.  split 1: `units` CTAs
// share out the tiles (and p.partial, p.counters are needed); split 2, 4 or 8:
// `units` clusters of as many CTAs, which must be at least as many as the tiles.
cudaError_t launch_i8_tiles(int rows, const CUtensorMap& w, const CUtensorMap& x,
                            const CUtensorMap& x32, const CUtensorMap& d, const GroupedParams& p,
                            int units, int split, cudaStream_t st);
// rows x cols bytes to 16-byte aligned rows of ld_dst elements, as they are or
// widened to fp16 (two operands in one launch; an empty one is left out).
struct I8Copy {
  const int8_t* src;
  long long ld_src;
  void* dst;
  long long ld_dst, rows;
  int cols;
  bool widen;  // to fp16
};
// Both (a job without rows is none) in one launch.
cudaError_t launch_i8_copies(const I8Copy& first, const I8Copy& second, int num_sms, cudaStream_t st);

}  // namespace gb300
