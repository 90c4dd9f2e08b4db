// moe_host.cu -- C ABI of the mixture-of-experts and 4-bit-weight operators:
// validation, handles, tensor maps and launches.  See include/gemm.h for the
// contract of each entry.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cstdio>
#include <cstring>

#include "common.h"
#include "gemm.h"
#include "moe.h"
#include "op.h"
#include "tc_launch.h"

using namespace gb300;

extern "C" {

int gemm_op_status(gemm_op_t op, gemm_stream_t stream) {
  if (!op) return GEMM_ERR_INVALID_ARG;
  if (op->inner) return gemm_op_status(op->inner, stream);  // what it ends in has the kernels that report
  // all on the caller's stream: what was cleared on another one could be
  // cleared after the next run had set it
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  uint32_t word = 0;
  if (cudaMemcpyAsync(&word, op->status, sizeof word, cudaMemcpyDeviceToHost, st) != cudaSuccess ||
      cudaStreamSynchronize(st) != cudaSuccess)
    return GEMM_ERR_CUDA;
  // Units that gave up left the counters of the tiles they shared part-way:
  // the next call would take such a tile for finished too early.
  if ((word & STATUS_TIMEOUT) && op->counters_bytes &&
      cudaMemsetAsync(static_cast<uint8_t*>(op->ws) + op->ws_counters_off, 0, op->counters_bytes,
                      st) != cudaSuccess)
    return GEMM_ERR_CUDA;
  if (word != 0 && (cudaMemsetAsync(op->status, 0, sizeof word, st) != cudaSuccess ||
                    cudaStreamSynchronize(st) != cudaSuccess))
    return GEMM_ERR_CUDA;
  if (word & STATUS_TIMEOUT) return GEMM_ERR_DEVICE_TIMEOUT;
  return (word & STATUS_BAD_INDEX) ? GEMM_ERR_INVALID_ARG : GEMM_OK;
}

int gemm_op_destroy(gemm_op_t op) {
  if (!op) return GEMM_OK;
  const int rc = cudaDeviceSynchronize() == cudaSuccess ? GEMM_OK : GEMM_ERR_CUDA;
  gemm_op_destroy(op->inner);
  if (op->ws) cudaFree(op->ws);
  if (op->status) cudaFree(op->status);
  delete op;
  return rc;
}

int64_t gemm_op_workspace_bytes(gemm_op_t op) {
  if (!op) return -1;
  return static_cast<int64_t>(op->ws_bytes + (op->inner ? op->inner->ws_bytes : 0));
}

int gemm_op_plan_string(gemm_op_t op, char* buf, size_t n) {
  if (!op) return GEMM_ERR_INVALID_ARG;
  if (buf && n) std::snprintf(buf, n, "%s", op->plan);
  return static_cast<int>(std::strlen(op->plan));
}

int gemm_op_debug_set(gemm_op_t op, int flags, uint64_t timeout_ns) {
  if (!op) return GEMM_ERR_INVALID_ARG;
  if (op->inner) return gemm_op_debug_set(op->inner, flags, timeout_ns);
  op->debug_flags = flags;
  op->timeout_ns = timeout_ns ? timeout_ns : kDefaultTimeoutNs;
  return GEMM_OK;
}

// ---------------------------------------------------------------- routing
int gemm_route_create(gemm_op_t* out, const gemm_route_desc_t* desc) {
  if (!out || !desc) return GEMM_ERR_INVALID_ARG;
  gemm_route_desc_t d = *desc;
  if (d.ld == 0) d.ld = d.E;
  if (d.T < 0 || d.E < 1 || d.E > GEMM_MAX_EXPERTS || d.k < 1 ||
      d.k > std::min(d.E, GEMM_MAX_TOP_K) || d.ld < d.E || d.T > INT_MAX / d.k)
    return GEMM_ERR_INVALID_ARG;
  if (!is_float(d.type)) return GEMM_ERR_UNSUPPORTED;
  int dev = 0, sms = 1;
  if (cudaGetDevice(&dev) == cudaSuccess)
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  cudaGetLastError();
  const int blocks = route_blocks(d.T, d.k, std::max(sms, 1));
  gemm_op* op = nullptr;
  const size_t ws = blocks > 1 ? sizeof(int) * static_cast<size_t>(blocks) * up(d.E, 4) : 0;
  const int rc = make_op(Kind::kRoute, ws, 0, ws, &op);
  if (rc != GEMM_OK) return rc;
  op->route = d;
  op->grid = blocks;
  std::snprintf(op->plan, sizeof op->plan, "route T=%lld E=%d k=%d blocks=%d",
                static_cast<long long>(d.T), d.E, d.k, blocks);
  *out = op;
  return GEMM_OK;
}

int gemm_route_run(gemm_op_t op, const void* logits, int32_t* experts, float* gates,
                   int32_t* offsets, int32_t* row_slot, int32_t* slot_row, gemm_stream_t stream) {
  if (!usable(op, Kind::kRoute) || !offsets) return GEMM_ERR_INVALID_ARG;
  const gemm_route_desc_t& d = op->route;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (!aligned(offsets, 4)) return GEMM_ERR_MISALIGNED;
  if (d.T == 0) return launched(cudaMemsetAsync(offsets, 0, sizeof(int32_t) * (d.E + 1), st));
  if (!logits || !experts || !gates || !row_slot || !slot_row) return GEMM_ERR_INVALID_ARG;
  if (!aligned(logits, elem_size(d.type)) || !aligned(experts, 4) || !aligned(gates, 4) ||
      !aligned(row_slot, 4) || !aligned(slot_row, 4))
    return GEMM_ERR_MISALIGNED;
  RouteParams p{};
  p.T = static_cast<int>(d.T);
  p.E = d.E;
  p.k = d.k;
  p.type = d.type;
  p.normalize = d.normalize != 0;
  p.ld = d.ld;
  p.logits = logits;
  p.experts = experts;
  p.gates = gates;
  p.offsets = offsets;
  p.row_slot = row_slot;
  p.slot_row = slot_row;
  p.blocks = op->grid;
  p.tokens_per_block = static_cast<int>((d.T + op->grid - 1) / op->grid);
  p.hist = static_cast<int*>(op->ws);
  p.ld_hist = static_cast<int>(up(d.E, 4));
  return launched(launch_route(p, st));
}

int gemm_route_backward(gemm_op_t op, const void* logits, const int32_t* experts,
                        const float* gates, const float* dgates, void* dlogits,
                        gemm_stream_t stream) {
  if (!usable(op, Kind::kRoute)) return GEMM_ERR_INVALID_ARG;
  const gemm_route_desc_t& d = op->route;
  if (d.T == 0) return GEMM_OK;
  if (!logits || !experts || !gates || !dgates || !dlogits) return GEMM_ERR_INVALID_ARG;
  if (!aligned(logits, elem_size(d.type)) || !aligned(dlogits, elem_size(d.type)) ||
      !aligned(experts, 4) || !aligned(gates, 4) || !aligned(dgates, 4))
    return GEMM_ERR_MISALIGNED;
  RouteBackwardParams p{};
  p.T = static_cast<int>(d.T);
  p.E = d.E;
  p.k = d.k;
  p.type = d.type;
  p.normalize = d.normalize != 0;
  p.ld = d.ld;
  p.logits = logits;
  p.experts = experts;
  p.gates = gates;
  p.dgates = dgates;
  p.dlogits = dlogits;
  p.num_sms = op->num_sms;
  return launched(launch_route_backward(p, static_cast<cudaStream_t>(stream)));
}

// ---------------------------------------------------------------- row movement
int gemm_permute_create(gemm_op_t* out, const gemm_permute_desc_t* desc) {
  if (!out || !desc) return GEMM_ERR_INVALID_ARG;
  gemm_permute_desc_t d = *desc;
  if (d.ld_tokens == 0) d.ld_tokens = std::max<int64_t>(d.H, 1);
  if (d.ld_rows == 0) d.ld_rows = std::max<int64_t>(d.H, 1);
  if (d.T < 0 || d.H < 0 || d.H > INT_MAX / 2 || d.k < 1 || d.k > GEMM_MAX_TOP_K ||
      d.ld_tokens < d.H || d.ld_rows < d.H || d.T > INT_MAX / d.k)
    return GEMM_ERR_INVALID_ARG;
  if (!is_float(d.type)) return GEMM_ERR_UNSUPPORTED;
  gemm_op* op = nullptr;
  const int rc = make_op(Kind::kPermute, 0, 0, 0, &op);
  if (rc != GEMM_OK) return rc;
  op->permute = d;
  std::snprintf(op->plan, sizeof op->plan, "permute T=%lld k=%d H=%lld",
                static_cast<long long>(d.T), d.k, static_cast<long long>(d.H));
  *out = op;
  return GEMM_OK;
}

}  // extern "C"

namespace {

PermuteParams permute_params(const gemm_op* op) {
  const gemm_permute_desc_t& d = op->permute;
  PermuteParams p{};
  p.T = d.T;
  p.H = d.H;
  p.k = d.k;
  p.type = d.type;
  p.ld_tokens = d.ld_tokens;
  p.ld_rows = d.ld_rows;
  p.status = op->status;
  return p;
}

}  // namespace

extern "C" {

int gemm_permute_gather(gemm_op_t op, const void* X, const int32_t* row_slot,
                        const int32_t* slot_row, void* Xs, gemm_stream_t stream) {
  if (!usable(op, Kind::kPermute)) return GEMM_ERR_INVALID_ARG;
  if (op->permute.T == 0 || op->permute.H == 0) return GEMM_OK;
  int rc = check_pointers({X, Xs}, elem_size(op->permute.type));
  if (rc == GEMM_OK) rc = check_pointers({row_slot, slot_row}, 4);
  if (rc != GEMM_OK) return rc;
  PermuteParams p = permute_params(op);
  p.tokens = X;
  p.rows_out = Xs;
  p.row_slot = row_slot;
  p.slot_row = slot_row;
  return launched(launch_gather(p, op->num_sms, static_cast<cudaStream_t>(stream)));
}

int gemm_permute_combine(gemm_op_t op, const void* Ys, const int32_t* slot_row, const float* gates,
                         void* Y, gemm_stream_t stream) {
  if (!usable(op, Kind::kPermute)) return GEMM_ERR_INVALID_ARG;
  if (op->permute.T == 0 || op->permute.H == 0) return GEMM_OK;
  int rc = check_pointers({Ys, Y}, elem_size(op->permute.type));
  if (rc == GEMM_OK) rc = check_pointers({slot_row}, 4);
  if (rc != GEMM_OK) return rc;
  if (!aligned(gates, 4)) return GEMM_ERR_MISALIGNED;
  PermuteParams p = permute_params(op);
  p.rows = Ys;
  p.tokens_out = Y;
  p.slot_row = slot_row;
  p.gates = gates;
  return launched(launch_combine(p, op->num_sms, static_cast<cudaStream_t>(stream)));
}

int gemm_permute_combine_backward(gemm_op_t op, const void* dY, const void* Ys,
                                  const int32_t* row_slot, const int32_t* slot_row,
                                  const float* gates, void* dYs, float* dgates,
                                  gemm_stream_t stream) {
  if (!usable(op, Kind::kPermute)) return GEMM_ERR_INVALID_ARG;
  if (op->permute.T == 0) return GEMM_OK;
  int rc = check_pointers({row_slot, slot_row, gates, dgates}, 4);
  if (rc == GEMM_OK && op->permute.H > 0)
    rc = check_pointers({dY, Ys, dYs}, elem_size(op->permute.type));
  if (rc != GEMM_OK) return rc;
  PermuteParams p = permute_params(op);
  p.tokens = dY;
  p.rows = Ys;
  p.rows_out = dYs;
  p.row_slot = row_slot;
  p.slot_row = slot_row;
  p.gates = gates;
  p.dgates = dgates;
  return launched(launch_combine_backward(p, op->num_sms, static_cast<cudaStream_t>(stream)));
}

// ---------------------------------------------------------------- grouped products
int gemm_grouped_create(gemm_op_t* out, const gemm_grouped_desc_t* desc) {
  if (!out || !desc) return GEMM_ERR_INVALID_ARG;
  gemm_grouped_desc_t d = *desc;
  const bool grad = d.form == GEMM_GROUPED_GRAD;
  if ((!grad && d.form != GEMM_GROUPED_ROWS) || d.E < 1 || d.E > GEMM_MAX_EXPERTS || d.R < 0 ||
      d.K < 0 || d.N < 0 || d.R > INT_MAX / 2)
    return GEMM_ERR_INVALID_ARG;
  // row numbers of B and D (all experts) are 32-bit TMA coordinates
  if (d.K > INT_MAX / 2 / d.E || d.N > INT_MAX / 2 / d.E) return GEMM_ERR_INVALID_ARG;
  if (d.layout_b != GEMM_ROW_MAJOR && d.layout_b != GEMM_COL_MAJOR) return GEMM_ERR_INVALID_ARG;
  if (!is_16bit(d.ab_type) || !is_float(d.d_type) ||
      (static_cast<int>(d.c_type) != 0 && d.c_type != d.d_type) ||
      (grad && d.layout_b != GEMM_ROW_MAJOR))
    return GEMM_ERR_UNSUPPORTED;
  const bool b_kcontig = !grad && d.layout_b == GEMM_COL_MAJOR;
  const int64_t b_cols = b_kcontig ? d.K : d.N;
  const int64_t b_rows = grad ? d.R : d.E * (b_kcontig ? d.N : d.K);
  if (d.lda == 0) d.lda = std::max<int64_t>(d.K, 1);
  if (d.ldb == 0) d.ldb = std::max<int64_t>(b_cols, 1);
  if (d.ldc == 0) d.ldc = std::max<int64_t>(d.N, 1);
  if (d.ldd == 0) d.ldd = std::max<int64_t>(d.N, 1);
  if (d.lda < d.K || d.ldb < b_cols || d.ldc < d.N || d.ldd < d.N) return GEMM_ERR_INVALID_ARG;
  // tile numbers are 32-bit: the most there can be (each expert may add a
  // partial tile to the rows')
  const int64_t ft = (d.N + 127) / 128;
  const int64_t qt = grad ? d.E * ((d.K + 63) / 64) : d.R / 64 + d.E;
  if (ft > 0 && qt > INT_MAX / ft) return GEMM_ERR_INVALID_ARG;

  const bool copy_a = d.lda % 8 != 0 && d.R > 0 && d.K > 0;
  const bool copy_b = d.ldb % 8 != 0 && b_rows > 0 && b_cols > 0;
  const int64_t ws_lda = up(d.K, 64), ws_ldb = up(b_cols, 64);
  const size_t a_bytes = copy_a ? static_cast<size_t>(d.R) * ws_lda * 2 : 0;
  const size_t b_bytes = copy_b ? static_cast<size_t>(b_rows) * ws_ldb * 2 : 0;
  int sms = 0, dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    cudaGetLastError();
  // The wide form needs D rows to fill a tile's columns (more than 64 an
  // expert, on average) and a wave of tiles; or, with sums long enough to make
  // up for its slower ends, so many tiles that the narrow form would take a
  // second wave (narrow against wide, us: 2000 rows over 2 of 4096 x 2048 50.1,
  // 28.0; 1024 over 8 of 4096 x 2048 42.6, 32.5; 1024 over 4 of 2048 x 2048
  // 18.7, 16.7; but 8 slices, 4096 over 2 of 512 x 512, 10.3, 11.5; and in one
  // wave, 400 over 4 of 4096 x 2048, 18.6, 27.2).
  const int64_t m = grad ? d.K : d.R / d.E;
  const int64_t wide_tiles = d.E * ((m + 255) / 256) * ((d.N + 255) / 256);
  const int64_t narrow_tiles = d.E * ((m + 63) / 64) * ft;
  const int64_t slices = ((grad ? d.R / d.E : d.K) + BK - 1) / BK;
  const bool wide = planned(
      "wide", m > 64 && (wide_tiles >= sms / 2 || (2 * narrow_tiles > 3 * sms && slices >= 16)));
  const int most_units = std::max(1, wide ? sms / 2 : sms);
  const size_t partial = grouped_partial_bytes(wide, most_units);
  const size_t counters = 4 * static_cast<size_t>(most_units) * (wide ? 2 : 1);
  const size_t p_off = static_cast<size_t>(up(static_cast<int64_t>(a_bytes + b_bytes), 256));
  gemm_op* op = nullptr;
  const size_t maps_off = static_cast<size_t>(up(static_cast<int64_t>(p_off + partial + counters), 256));
  const size_t maps = grad ? 2 * sizeof(CUtensorMap) * d.E : 0;
  const int rc = make_op(Kind::kGrouped, maps_off + maps, p_off + partial, counters, &op);
  if (rc != GEMM_OK) return rc;
  op->units = std::min(most_units, prepare_grouped(wide, d.d_type, op->num_sms));
  if (op->units <= 0) {
    cudaGetLastError();
    gemm_op_destroy(op);
    return GEMM_ERR_CUDA;
  }
  op->wide = wide;
  op->ws_partial_off = p_off;
  op->ws_counters_off = p_off + partial;
  op->counters_bytes = counters;
  op->ws_maps_off = maps_off;
  op->grouped = d;
  op->copy_a = copy_a;
  op->copy_b = copy_b;
  op->a_rows = d.R;
  op->a_cols = d.K;
  op->b_rows = b_rows;
  op->b_cols = b_cols;
  op->ws_lda = copy_a ? ws_lda : d.lda;
  op->ws_ldb = copy_b ? ws_ldb : d.ldb;
  op->ws_b_off = a_bytes;
  std::snprintf(op->plan, sizeof op->plan, "grouped form=%s E=%d R=%lld K=%lld N=%lld wide=%d copy=%d%d units=%d",
                grad ? "grad" : "rows", d.E, static_cast<long long>(d.R),
                static_cast<long long>(d.K), static_cast<long long>(d.N), wide, copy_a, copy_b,
                op->units);
  *out = op;
  return GEMM_OK;
}

int gemm_grouped_run(gemm_op_t op, const void* A, const void* B, const int32_t* offsets,
                     const void* C, void* D, gemm_stream_t stream) {
  if (!usable(op, Kind::kGrouped)) return GEMM_ERR_INVALID_ARG;
  const gemm_grouped_desc_t& d = op->grouped;
  const bool grad = d.form == GEMM_GROUPED_GRAD;
  // an empty D: nothing to do
  if (d.N == 0 || (grad ? d.K == 0 : d.R == 0)) return GEMM_OK;
  const bool reads = grad ? d.R > 0 : d.K > 0;  // otherwise D = C
  if (!D || !offsets || (reads && (!A || !B)) || (C && static_cast<int>(d.c_type) == 0))
    return GEMM_ERR_INVALID_ARG;
  const int64_t ds = elem_size(d.d_type);
  if (!aligned(D, ds) || !aligned(C, ds) || !aligned(offsets, 4) ||
      (reads && (!aligned(A, op->copy_a ? 2 : 16) || !aligned(B, op->copy_b ? 2 : 16))))
    return GEMM_ERR_MISALIGNED;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const void *a = A, *b = B;
  if (reads && (op->copy_a || op->copy_b)) {
    CopyJob16 jobs[2] = {};
    uint16_t* const ws = static_cast<uint16_t*>(op->ws);
    uint16_t* const wsb = ws + op->ws_b_off / 2;
    if (op->copy_a) {
      jobs[0] = {static_cast<const uint16_t*>(A), d.lda, ws, op->ws_lda, op->a_rows, op->a_cols};
      a = ws;
    }
    if (op->copy_b) {
      jobs[1] = {static_cast<const uint16_t*>(B), d.ldb, wsb, op->ws_ldb, op->b_rows, op->b_cols};
      b = wsb;
    }
    const int rc = launched(launch_copy16(jobs, 2, op->num_sms, st));
    if (rc != GEMM_OK) return rc;
  }
  GroupedParams p{};
  CUtensorMap f{}, x128{}, x32{}, dm{};
  if (reads) {
    bool ok;
    if (grad) {
      ok = encode_rows(&f, b, op->ws_ldb, d.N, d.R, 0, 64, BK) &&
           encode_rows(&x128, a, op->ws_lda, d.K, d.R, 0, 64, BK);
    } else {
      ok = (d.layout_b == GEMM_COL_MAJOR
                ? encode_rows(&f, b, op->ws_ldb, d.K, op->b_rows, 0, BK, 128)
                : encode_rows(&f, b, op->ws_ldb, d.N, d.K, d.E, 64, BK)) &&
           encode_rows(&x128, a, op->ws_lda, d.K, d.R, 0, BK, 128) &&
           encode_rows(&x32, a, op->ws_lda, d.K, d.R, 0, BK, 32);
    }
    if (!ok) return GEMM_ERR_CUDA;
  }
  p.grad = grad;
  p.E = d.E;
  p.R = static_cast<int>(d.R);
  p.K = static_cast<int>(d.K);
  p.N = static_cast<int>(d.N);
  p.f_mn = grad || d.layout_b == GEMM_ROW_MAJOR;
  p.idesc = idesc_f16(d.ab_type == GEMM_BF16, p.f_mn, grad, op->wide ? 256 : 128, 0);
  p.offsets = offsets;
  p.C = C;
  p.d_type = d.d_type;
  p.d_vec = is_16bit(d.d_type) && d.ldd % 8 == 0 && aligned(D, 16);
  p.d_tma = p.d_vec && d.N % 8 == 0 && !C;
  if (p.d_tma && !(grad ? encode_rows(&dm, D, d.ldd, d.N, d.K, d.E, 64, 32)
                        : encode_rows(&dm, D, d.ldd, d.N, d.R, 1, 64, 32)))
    return GEMM_ERR_CUDA;
  p.ldc = d.ldc;
  p.ldd = d.ldd;
  p.D = D;
  uint8_t* const ws = static_cast<uint8_t*>(op->ws);
  p.partial = reinterpret_cast<float*>(ws + op->ws_partial_off);
  p.counters = reinterpret_cast<unsigned*>(ws + op->ws_counters_off);
  p.maps = reinterpret_cast<CUtensorMap*>(ws + op->ws_maps_off);
  p.status = op->status;
  p.timeout_ns = op->timeout_ns;
  p.debug_flags = op->debug_flags;
  op->debug_flags = 0;
  return launched(launch_grouped(op->wide, f, x128, x32, dm, p, op->units, st));
}

// ---------------------------------------------------------------- 4-bit weights
int gemm_w4_create(gemm_op_t* out, const gemm_w4_desc_t* desc) {
  if (!out || !desc) return GEMM_ERR_INVALID_ARG;
  gemm_w4_desc_t d = *desc;
  if (d.ldx == 0) d.ldx = std::max<int64_t>(d.K, 1);
  if (d.ldd == 0) d.ldd = std::max<int64_t>(d.N, 1);
  if (d.E < 1 || d.E > GEMM_MAX_EXPERTS || d.R < 0 || d.K < 0 || d.N < 0 || d.R > INT_MAX / 2 ||
      d.K > INT_MAX / 2 || d.N > INT_MAX / 2 || d.group < 32 || d.group % 32 != 0 ||
      d.K % 32 != 0 || d.ldx < d.K || d.ldd < d.N)
    return GEMM_ERR_INVALID_ARG;
  if (!is_16bit(d.x_type) || !is_float(d.scale_type) || !is_float(d.d_type))
    return GEMM_ERR_UNSUPPORTED;
  if (d.ldx % 8 != 0) return GEMM_ERR_MISALIGNED;
  gemm_op* op = nullptr;
  const int rc = make_op(Kind::kW4, 0, 0, 0, &op);
  if (rc != GEMM_OK) return rc;
  op->w4 = d;
  std::snprintf(op->plan, sizeof op->plan, "w4 E=%d R=%lld K=%lld N=%lld group=%d zeros=%d", d.E,
                static_cast<long long>(d.R), static_cast<long long>(d.K),
                static_cast<long long>(d.N), d.group, d.has_zeros != 0);
  *out = op;
  return GEMM_OK;
}

int gemm_w4_run(gemm_op_t op, const void* X, const uint8_t* W, const void* scales,
                const uint8_t* zeros, const int32_t* offsets, void* D, gemm_stream_t stream) {
  if (!usable(op, Kind::kW4)) return GEMM_ERR_INVALID_ARG;
  const gemm_w4_desc_t& d = op->w4;
  if (d.R == 0 || d.N == 0) return GEMM_OK;
  if (!D || (d.K > 0 && (!X || !W || !scales || (d.has_zeros != 0) != (zeros != nullptr))) ||
      (d.E > 1 && !offsets))
    return GEMM_ERR_INVALID_ARG;
  if (!aligned(D, elem_size(d.d_type)) || !aligned(X, 16) || !aligned(W, 16) ||
      !aligned(scales, elem_size(d.scale_type)) || !aligned(offsets, 4))
    return GEMM_ERR_MISALIGNED;
  W4Params p{};
  p.E = d.E;
  p.R = static_cast<int>(d.R);
  p.K = static_cast<int>(d.K);
  p.N = static_cast<int>(d.N);
  p.group = d.group;
  p.groups = static_cast<int>((d.K + d.group - 1) / d.group);
  p.x_type = d.x_type;
  p.scale_type = d.scale_type;
  p.d_type = d.d_type;
  p.ldx = d.ldx;
  p.ldd = d.ldd;
  p.X = X;
  p.W = W;
  p.scales = scales;
  p.zeros = zeros;
  p.offsets = offsets;
  p.D = D;
  p.status = op->status;
  p.num_sms = op->num_sms;
  return launched(launch_w4(p, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
