// op.h -- the handle behind gemm_op_t, and what the files that create and run
// such handles share (moe_host.cu, rows_host.cu).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <cstdlib>
#include <cstring>
#include <initializer_list>
#include <new>

#include "clear.h"
#include "common.h"
#include "gemm.h"
#include "moe.h"

namespace gb300 {

enum class Kind { kRoute, kPermute, kGrouped, kW4, kNorm, kRows8, kRows8Grad, kI8 };

constexpr uint64_t kDefaultTimeoutNs = 2000000000ull;  // 2 s per device-side wait
constexpr size_t kStatusBytes = 256;

inline bool is_16bit(int t) { return t == T_F16 || t == T_BF16; }
inline bool is_float(int t) { return is_16bit(t) || t == T_F32; }
inline int64_t elem_size(int t) { return t == T_F32 ? 4 : 2; }
inline int64_t up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }
inline bool aligned(const void* p, int64_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// GEMM_OK when every pointer is present and aligned to n bytes.
inline int check_pointers(std::initializer_list<const void*> ptrs, int64_t n) {
  for (const void* q : ptrs)
    if (!q) return GEMM_ERR_INVALID_ARG;
  for (const void* q : ptrs)
    if (!aligned(q, n)) return GEMM_ERR_MISALIGNED;
  return GEMM_OK;
}

}  // namespace gb300

struct gemm_op {
  gb300::Kind kind;
  int device = 0, num_sms = 0;
  gemm_route_desc_t route{};
  gemm_permute_desc_t permute{};
  gemm_grouped_desc_t grouped{};
  gemm_w4_desc_t w4{};
  gemm_norm_desc_t norm{};
  gemm_rows8_desc_t rows8{};
  gemm_rows8_grad_desc_t rows8_grad{};
  gemm_i8_desc_t i8{};
  void* ws = nullptr;
  size_t ws_bytes = 0;
  uint32_t* status = nullptr;
  uint64_t timeout_ns = gb300::kDefaultTimeoutNs;
  int debug_flags = 0;
  char plan[192] = "";  // not a string: its allocation could throw out of a C entry
  // grouped: operands copied to workspace rows the TMA unit can read
  bool copy_a = false, copy_b = false;
  int64_t a_rows = 0, a_cols = 0, b_rows = 0, b_cols = 0;
  int64_t ws_lda = 0, ws_ldb = 0;
  size_t ws_b_off = 0, ws_partial_off = 0, ws_counters_off = 0, ws_maps_off = 0;
  size_t counters_bytes = 0;
  bool wide = false;
  bool tiles = false;  // i8: on the tensor cores (wide, or tiles of tile_rows rows)
  int tile_rows = 0, split = 1;
  CUtensorMap map_x{}, map_x32{}, map_w{};  // i8: of the workspace's operands
  int units = 0;
  int grid = 0;  // route: blocks
  gemm_op* inner = nullptr;  // rows8_grad: the grouped product it ends in
};

namespace gb300 {

// Handle of a kind on the current device with `ws_bytes` of workspace, of which
// [zero_off, zero_off + zero_bytes) starts as zeros.
inline int make_op(Kind kind, size_t ws_bytes, size_t zero_off, size_t zero_bytes, gemm_op** out) {
  int dev = 0, major = 0, minor = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    cudaGetLastError();
    return GEMM_ERR_NO_DEVICE;
  }
  if (major != 10 || minor != 3) return GEMM_ERR_NO_DEVICE;
  gemm_op* op = new (std::nothrow) gemm_op();
  if (!op) return GEMM_ERR_ALLOC_FAILED;
  op->kind = kind;
  op->device = dev;
  op->num_sms = sms;
  op->ws_bytes = ws_bytes;
  if (cudaMalloc(&op->status, kStatusBytes) != cudaSuccess ||
      (ws_bytes && cudaMalloc(&op->ws, ws_bytes) != cudaSuccess) ||
      clear_now({{op->status, kStatusBytes},
                 {static_cast<uint8_t*>(op->ws) + zero_off, zero_bytes}}) != cudaSuccess) {
    cudaGetLastError();
    if (op->ws) cudaFree(op->ws);
    if (op->status) cudaFree(op->status);
    delete op;
    return GEMM_ERR_ALLOC_FAILED;
  }
  *out = op;
  return GEMM_OK;
}

inline bool usable(const gemm_op* op, Kind kind) {
  int dev = -1;
  return op && op->kind == kind && cudaGetDevice(&dev) == cudaSuccess && dev == op->device;
}

inline int launched(cudaError_t e) {
  if (e == cudaSuccess) return GEMM_OK;
  cudaGetLastError();
  return GEMM_ERR_CUDA;
}

// The plan's choice for `key`, unless GEMM_FORCE_PLAN="key=0|1,..." names it.
inline bool planned(const char* key, bool choice) {
  const char* env = std::getenv("GEMM_FORCE_PLAN");
  const size_t n = std::strlen(key);
  for (const char* s = env; s && *s; s = std::strchr(s, ',')) {
    if (*s == ',') ++s;
    if (std::strncmp(s, key, n) == 0 && s[n] == '=') return s[n + 1] != '0';
  }
  return choice;
}

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                              const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                              const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// Map of a row-major 16-bit operand, 128-byte swizzled boxes of box_cols x
// box_rows, zeros outside.  depth > 0: that many matrices of `rows` rows one
// after another, as a third dimension.
inline bool encode_rows(CUtensorMap* tm, const void* base, int64_t ld, int64_t cols, int64_t rows,
                        int64_t depth, int box_cols, int box_rows) {
  EncodeFn enc = reinterpret_cast<EncodeFn>(tensor_map_encoder());
  if (!enc) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)depth};
  const cuuint64_t strides[2] = {(cuuint64_t)ld * 2, (cuuint64_t)(ld * rows) * 2};
  const cuuint32_t box[3] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows, 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  return enc(tm, CU_TENSOR_MAP_DATA_TYPE_UINT16, depth > 0 ? 3 : 2, const_cast<void*>(base), dims,
             strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Map of a row-major 8-bit operand in 128-byte swizzled boxes of 128 x 128, zeros outside.
inline bool encode_bytes(CUtensorMap* tm, const void* base, int64_t ld, int64_t cols, int64_t rows) {
  EncodeFn enc = reinterpret_cast<EncodeFn>(tensor_map_encoder());
  if (!enc) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)ld};
  const cuuint32_t box[2] = {128, 128};
  const cuuint32_t estr[2] = {1, 1};
  return enc(tm, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box,
             estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace gb300
