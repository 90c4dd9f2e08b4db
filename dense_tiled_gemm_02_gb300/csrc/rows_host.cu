// rows_host.cu -- C ABI of the operators on rows held in 8 bits: validation,
// handles and launches.  See include/gemm.h for the contract of each entry.
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdio>

#include "op.h"
#include "rows.h"
#include "tc_launch.h"

using namespace gb300;

namespace {

// Leading dimension 0 is packed; false for one below that.
bool settle(int64_t& ld, int64_t cols) {
  if (ld == 0) ld = std::max<int64_t>(cols, 1);
  return ld >= cols;
}

int64_t blocks_of(int64_t n) { return (n + ROW_BLOCK - 1) / ROW_BLOCK; }

}  // namespace

extern "C" {

// ---------------------------------------------------------------- norm
int gemm_norm_create(gemm_op_t* out, const gemm_norm_desc_t* desc) {
  if (!out || !desc) return GEMM_ERR_INVALID_ARG;
  gemm_norm_desc_t d = *desc;
  d.residual = d.residual != 0;
  if (d.T < 0 || d.H < 0 || d.T > INT_MAX / 2 || d.H > INT_MAX / 2 || !settle(d.ldx, d.H) ||
      !settle(d.ldr, d.H) || !settle(d.ldh, d.H) || !settle(d.ldy, d.H) || !std::isfinite(d.eps) ||
      d.eps < 0)
    return GEMM_ERR_INVALID_ARG;
  if (!is_float(d.type) || (d.weight_type != d.type && d.weight_type != GEMM_F32) ||
      (d.y_type != d.type && d.y_type != GEMM_I8))
    return GEMM_ERR_UNSUPPORTED;
  if (!d.residual) d.ldr = d.ldh = d.ldx;  // h is x
  int sms = 1, dev = 0;
  if (cudaGetDevice(&dev) == cudaSuccess)
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  cudaGetLastError();
  // partial sums of dweight; a norm out in 8 bits has no backward pass
  const size_t partial =
      d.y_type == GEMM_I8
          ? 0
          : sizeof(float) * static_cast<size_t>(d.H) *
                norm_partial_rows(d.T, static_cast<int>(d.H), d.type, std::max(sms, 1));
  gemm_op* op = nullptr;
  const int rc = make_op(Kind::kNorm, partial, 0, 0, &op);
  if (rc != GEMM_OK) return rc;
  if (d.y_type != GEMM_I8 && prepare_norm_backward(static_cast<int>(d.H), d.type) != cudaSuccess) {
    cudaGetLastError();
    gemm_op_destroy(op);
    return GEMM_ERR_CUDA;
  }
  op->norm = d;
  std::snprintf(op->plan, sizeof op->plan, "norm T=%lld H=%lld residual=%d out=%s",
                static_cast<long long>(d.T), static_cast<long long>(d.H), d.residual,
                d.y_type == GEMM_I8 ? "i8" : "x");
  *out = op;
  return GEMM_OK;
}

int gemm_norm_run(gemm_op_t op, const void* x, const void* residual, const void* weight, void* h,
                  void* y, float* scales, float* rstd, gemm_stream_t stream) {
  if (!usable(op, Kind::kNorm)) return GEMM_ERR_INVALID_ARG;
  const gemm_norm_desc_t& d = op->norm;
  const bool i8 = d.y_type == GEMM_I8;
  if (d.T == 0 || d.H == 0) return GEMM_OK;
  const int64_t s = elem_size(d.type);
  int rc = check_pointers({x}, s);
  if (rc == GEMM_OK) rc = check_pointers({weight}, elem_size(d.weight_type));
  if (rc == GEMM_OK) rc = check_pointers({y}, i8 ? 1 : s);
  if (rc == GEMM_OK && d.residual) rc = check_pointers({residual, h}, s);
  if (rc == GEMM_OK && i8) rc = check_pointers({scales}, 4);
  if (rc != GEMM_OK) return rc;
  if (!aligned(rstd, 4)) return GEMM_ERR_MISALIGNED;
  NormParams p{};
  p.T = d.T;
  p.H = static_cast<int>(d.H);
  p.type = d.type;
  p.weight_type = d.weight_type;
  p.i8 = i8;
  p.eps = d.eps;
  p.ldx = d.ldx;
  p.ldr = d.ldr;
  p.ldh = d.ldh;
  p.ldy = d.ldy;
  p.x = x;
  p.residual = d.residual ? residual : nullptr;
  p.weight = weight;
  p.h = d.residual ? h : nullptr;
  p.y = y;
  p.scales = scales;
  p.rstd = rstd;
  return launched(launch_norm(p, op->num_sms, static_cast<cudaStream_t>(stream)));
}

int gemm_norm_backward(gemm_op_t op, const void* dy, const void* h, const uint8_t* E,
                       const void* weight, const float* rstd, const void* dresidual, void* dx,
                       float* dweight, gemm_stream_t stream) {
  if (!usable(op, Kind::kNorm) || op->norm.y_type == GEMM_I8) return GEMM_ERR_INVALID_ARG;
  const gemm_norm_desc_t& d = op->norm;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (d.H == 0) return GEMM_OK;
  if (!aligned(dweight, 4)) return GEMM_ERR_MISALIGNED;
  if (d.T == 0)
    return dweight ? launched(cudaMemsetAsync(dweight, 0, sizeof(float) * d.H, st)) : GEMM_OK;
  const int64_t s = elem_size(d.type);
  int rc = check_pointers({dy, dx}, s);
  if (rc == GEMM_OK) rc = check_pointers({h}, E ? 1 : s);
  if (rc == GEMM_OK) rc = check_pointers({weight}, elem_size(d.weight_type));
  if (rc == GEMM_OK) rc = check_pointers({rstd}, 4);
  if (rc != GEMM_OK) return rc;
  if (!aligned(dresidual, s)) return GEMM_ERR_MISALIGNED;
  NormBackwardParams p{};
  p.T = d.T;
  p.H = static_cast<int>(d.H);
  p.type = d.type;
  p.weight_type = d.weight_type;
  p.ldy = d.ldy;
  p.ldh = E ? d.H : d.ldh;
  p.ldr = d.ldh;
  p.ldx = d.ldx;
  p.dy = dy;
  p.h = h;
  p.E = E;
  p.weight = weight;
  p.rstd = rstd;
  p.dresidual = dresidual;
  p.dx = dx;
  p.dweight = dweight;
  p.partial = static_cast<float*>(op->ws);
  p.status = op->status;
  p.timeout_ns = op->timeout_ns;
  p.debug_flags = op->debug_flags;
  op->debug_flags = 0;
  return launched(launch_norm_backward(p, op->num_sms, st));
}

// ---------------------------------------------------------------- rows to 8 bits
int gemm_rows8_create(gemm_op_t* out, const gemm_rows8_desc_t* desc) {
  if (!out || !desc) return GEMM_ERR_INVALID_ARG;
  gemm_rows8_desc_t d = *desc;
  if (d.T < 0 || d.H < 0 || d.T > INT_MAX / 2 || d.H > INT_MAX / 2 || !settle(d.ldx, d.H) ||
      !settle(d.ldq, d.H) || (d.block != 0 && d.block != ROW_BLOCK))
    return GEMM_ERR_INVALID_ARG;
  if (!is_float(d.type)) return GEMM_ERR_UNSUPPORTED;
  gemm_op* op = nullptr;
  const int rc = make_op(Kind::kRows8, 0, 0, 0, &op);
  if (rc != GEMM_OK) return rc;
  op->rows8 = d;
  std::snprintf(op->plan, sizeof op->plan, "rows8 T=%lld H=%lld block=%d",
                static_cast<long long>(d.T), static_cast<long long>(d.H), d.block);
  *out = op;
  return GEMM_OK;
}

}  // extern "C"

namespace {

int run_rows8(gemm_op_t op, const void* X_in, void* X_out, const int8_t* q_in, int8_t* q_out,
              const void* scales_in, void* scales_out, gemm_stream_t stream) {
  if (!usable(op, Kind::kRows8)) return GEMM_ERR_INVALID_ARG;
  const gemm_rows8_desc_t& d = op->rows8;
  const bool pack = q_out != nullptr;
  if (d.T == 0 || d.H == 0) return GEMM_OK;
  int rc = check_pointers({pack ? X_in : X_out}, elem_size(d.type));
  if (rc == GEMM_OK) rc = check_pointers({pack ? q_out : q_in}, 1);
  if (rc == GEMM_OK) rc = check_pointers({pack ? scales_out : scales_in}, d.block ? 1 : 4);
  if (rc != GEMM_OK) return rc;
  Rows8Params p{};
  p.T = d.T;
  p.H = static_cast<int>(d.H);
  p.type = d.type;
  p.block = d.block;
  p.ldx = d.ldx;
  p.ldq = d.ldq;
  p.X = X_in;
  p.X_out = X_out;
  p.q = q_in;
  p.q_out = q_out;
  p.scales = scales_in;
  p.scales_out = scales_out;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return launched(pack ? launch_rows8_pack(p, op->num_sms, st)
                       : launch_rows8_unpack(p, op->num_sms, st));
}

}  // namespace

extern "C" {

int gemm_rows8_pack(gemm_op_t op, const void* X, int8_t* q, void* scales, gemm_stream_t stream) {
  if (!q && usable(op, Kind::kRows8) && op->rows8.T > 0 && op->rows8.H > 0)
    return GEMM_ERR_INVALID_ARG;
  return run_rows8(op, X, nullptr, nullptr, q, nullptr, scales, stream);
}

int gemm_rows8_unpack(gemm_op_t op, const int8_t* q, const void* scales, void* X,
                      gemm_stream_t stream) {
  return run_rows8(op, nullptr, X, q, nullptr, scales, nullptr, stream);
}

// ---------------------------------------------------------------- gradients from block rows
int gemm_rows8_grad_create(gemm_op_t* out, const gemm_rows8_grad_desc_t* desc) {
  if (!out || !desc) return GEMM_ERR_INVALID_ARG;
  gemm_rows8_grad_desc_t d = *desc;
  if (d.R < 0 || d.K < 0 || d.K > INT_MAX / 2 || !settle(d.ldq, d.K)) return GEMM_ERR_INVALID_ARG;
  gemm_grouped_desc_t g{};
  g.form = GEMM_GROUPED_GRAD;
  g.E = d.E;
  g.R = d.R;
  g.K = d.K;
  g.N = d.N;
  g.ab_type = d.b_type;
  g.c_type = d.c_type;
  g.d_type = d.d_type;
  g.layout_b = GEMM_ROW_MAJOR;
  g.lda = up(std::max<int64_t>(d.K, 1), 64);
  g.ldb = d.ldb;
  g.ldc = d.ldc;
  g.ldd = d.ldd;
  gemm_op* inner = nullptr;
  int rc = gemm_grouped_create(&inner, &g);
  if (rc != GEMM_OK) return rc;
  // the rows in B's type, and the offsets of a single group
  const size_t rows = static_cast<size_t>(up(2 * d.R * g.lda, 256));
  gemm_op* op = nullptr;
  rc = make_op(Kind::kRows8Grad, rows + 256, rows, 256, &op);
  if (rc != GEMM_OK) {
    gemm_op_destroy(inner);
    return rc;
  }
  op->inner = inner;
  op->rows8_grad = d;
  op->ws_lda = g.lda;
  op->ws_b_off = rows;
  const int32_t one[2] = {0, static_cast<int32_t>(d.R)};
  if (write_now(static_cast<uint8_t*>(op->ws) + rows, one, sizeof one) != cudaSuccess) {
    cudaGetLastError();
    gemm_op_destroy(op);
    return GEMM_ERR_CUDA;
  }
  std::snprintf(op->plan, sizeof op->plan, "rows8_grad: %s", inner->plan);
  *out = op;
  return GEMM_OK;
}

int gemm_rows8_grad_run(gemm_op_t op, const int8_t* q, const uint8_t* E, const void* B,
                        const int32_t* offsets, const void* C, void* D, gemm_stream_t stream) {
  if (!usable(op, Kind::kRows8Grad)) return GEMM_ERR_INVALID_ARG;
  const gemm_rows8_grad_desc_t& d = op->rows8_grad;
  if (d.N == 0 || d.K == 0) return GEMM_OK;
  if (!D || (d.R > 0 && (!q || !E || !B)) || (d.E > 1 && !offsets)) return GEMM_ERR_INVALID_ARG;
  const int32_t* const groups =
      offsets ? offsets
              : reinterpret_cast<const int32_t*>(static_cast<uint8_t*>(op->ws) + op->ws_b_off);
  if (d.R > 0) {
    Rows8Params p{};
    p.T = d.R;
    p.H = static_cast<int>(d.K);
    p.type = d.b_type;
    p.block = ROW_BLOCK;
    p.ldx = op->ws_lda;
    p.ldq = d.ldq;
    p.X_out = op->ws;
    p.q = q;
    p.scales = E;
    const int rc = launched(launch_rows8_unpack(p, op->num_sms, static_cast<cudaStream_t>(stream)));
    if (rc != GEMM_OK) return rc;
  }
  return gemm_grouped_run(op->inner, op->ws, B, groups, C, D, stream);
}

// ---------------------------------------------------------------- scaled products
int gemm_i8_create(gemm_op_t* out, const gemm_i8_desc_t* desc) {
  if (!out || !desc) return GEMM_ERR_INVALID_ARG;
  gemm_i8_desc_t d = *desc;
  if (d.E < 1 || d.E > GEMM_MAX_EXPERTS || d.R < 0 || d.K < 0 || d.N < 0 || d.R > INT_MAX / 2 ||
      d.K >= 1 << 17 || d.N > INT_MAX / 2 / d.E || !settle(d.ldx, d.K) || !settle(d.ldw, d.K) ||
      !settle(d.ldd, d.N))
    return GEMM_ERR_INVALID_ARG;
  if (!is_float(d.d_type)) return GEMM_ERR_UNSUPPORTED;
  int sms = 1, dev = 0;
  if (cudaGetDevice(&dev) == cudaSuccess)
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  cudaGetLastError();
  // Which kernel, by the rows of an expert on average (the host does not know
  // the groups).  The few-rows kernel takes eight rows a pass for the weights'
  // bytes, and nine to sixteen at the rate of the integer instruction: 2 us and
  // 0.33 us a million weights and pass, against 6.5 and 0.19 of the tiles (16
  // rows of 4096 x 4096 8.4 and 10.9 us, of 8192 x 8192 23.7 and 19.0; 32 of
  // 1024 x 4096 5.3 and 7.6, of 4096 x 4096 14.4 and 10.9).  Tiles of 128 rows
  // against the wide form, N x K: 4096 rows of 8192 x 8192 363 and 362 us, 6144 of
  // 4096 x 4096 147 and 141, 8192 of 8192 x 8192 714 and 625, of 8192 x 1024 108 and
  // 89.  That is with at least four of the wide form's tiles for each of its CTA
  // pairs: with fewer its last round costs more than the converters do (8192 rows of
  // 2048 x 2048 59 and 70, of 256 x 8192 78 and 89, of 1024 x 8192 147 and 164;
  // 16384 of 1024 x 8192 are an exception, 263 and 242).
  const bool some = d.K > 0 && d.R > 0 && d.N > 0;
  const int64_t mean = (d.R + d.E - 1) / d.E, passes = (mean + 15) / 16;
  const double weights = static_cast<double>(d.E) * d.N * d.K;
  const bool few = mean <= 8 || (passes <= 2 && (0.33 * passes - 0.19) * weights < 4.5e6);
  const int64_t wide_tiles = d.E * ((mean + 255) / 256) * ((d.N + 255) / 256);
  const bool wide = some && planned("wide", d.R >= 6144ll * d.E && wide_tiles >= 4ll * (sms / 2));
  const bool tiles = wide || (some && planned("tiles", !few));
  const int rows = wide ? 0 : planned("tall", mean > 64) ? 128 : 64;
  // X in fp16; W in fp16 (wide), or a copy where the TMA unit cannot read its
  // rows; partial sums and counters of shared tiles
  const bool copy_w = wide || (tiles && d.ldw % 16 != 0);
  const int most_units = std::max(1, wide ? sms / 2 : sms);
  const int64_t ws_ldx = up(d.K, 64), ws_ldw = wide ? ws_ldx : up(d.K, 128);
  const size_t x_bytes = tiles ? static_cast<size_t>(up(2 * d.R * ws_ldx, 256)) : 0;
  const size_t w_bytes = copy_w ? static_cast<size_t>(d.E * d.N * ws_ldw * (wide ? 2 : 1)) : 0;
  const size_t p_off = static_cast<size_t>(up(static_cast<int64_t>(x_bytes + w_bytes), 256));
  // Fewer tiles than CTAs: clusters of CTAs share one each, all tiles in one
  // wave.  (The groups' tiles are not known: at most one more for each expert
  // with rows.)
  const int64_t experts = std::min<int64_t>(d.E, d.R);
  const int64_t row_tiles = rows ? (d.E == 1 ? (d.R + rows - 1) / rows : d.R / rows + experts) : 0;
  const int64_t most_tiles = row_tiles * ((d.N + 127) / 128);
  int split = 1;
  if (tiles && !wide && planned("csk", true)) {
    while (split < 8 && 2 * split * most_tiles <= sms && 2 * split <= (d.K + 127) / 128) split *= 2;
    // a cluster's CTAs are neighbours: fewer of them fit than CTAs alone
    while (split > 1 && prepare_i8_tiles(rows, d.d_type, split, sms) < most_tiles) split /= 2;
    cudaGetLastError();
  }
  const size_t partial = wide                  ? grouped_partial_bytes(true, most_units)
                         : tiles && split == 1 ? i8_tiles_partial_bytes(rows, most_units)
                                               : 0;
  const size_t counters = tiles && split == 1 ? 4 * static_cast<size_t>(most_units) * (wide ? 2 : 1) : 0;
  gemm_op* op = nullptr;
  const int rc = make_op(Kind::kI8, p_off + partial + counters, p_off + partial, counters, &op);
  if (rc != GEMM_OK) return rc;
  op->i8 = d;
  if (tiles) {
    if (wide)
      op->units = std::min(most_units, prepare_scaled(d.d_type, op->num_sms));
    else if (prepare_i8_tiles(rows, d.d_type, split, op->num_sms) > 0)
      op->units = split > 1 ? static_cast<int>(most_tiles) : most_units;
    if (op->units <= 0) {
      cudaGetLastError();
      gemm_op_destroy(op);
      return GEMM_ERR_CUDA;
    }
  }
  if (tiles) {
    uint8_t* const ws = static_cast<uint8_t*>(op->ws);
    const int64_t w_rows = d.E * d.N;
    if (!encode_rows(&op->map_x, ws, ws_ldx, d.K, d.R, 0, BK, wide ? 128 : rows) ||
        !encode_rows(&op->map_x32, ws, ws_ldx, d.K, d.R, 0, BK, 32) ||
        (wide && !encode_rows(&op->map_w, ws + x_bytes, ws_ldw, d.K, w_rows, 0, BK, 128)) ||
        (copy_w && !wide && !encode_bytes(&op->map_w, ws + x_bytes, ws_ldw, d.K, w_rows))) {
      gemm_op_destroy(op);
      return GEMM_ERR_CUDA;
    }
  }
  op->tiles = tiles;
  op->wide = wide;
  op->tile_rows = rows;
  op->split = split;
  op->copy_b = copy_w;
  op->ws_lda = ws_ldx;
  op->ws_ldb = copy_w ? ws_ldw : d.ldw;
  op->ws_b_off = x_bytes;
  op->ws_partial_off = p_off;
  op->ws_counters_off = p_off + partial;
  op->counters_bytes = counters;
  std::snprintf(op->plan, sizeof op->plan, "i8 E=%d R=%lld K=%lld N=%lld form=%s rows=%d split=%d copy=%d units=%d",
                d.E, static_cast<long long>(d.R), static_cast<long long>(d.K),
                static_cast<long long>(d.N), wide ? "wide" : tiles ? "tiles" : "rows", rows, split,
                copy_w, op->units);
  *out = op;
  return GEMM_OK;
}

}  // extern "C"

namespace {

int run_i8_tiles(gemm_op_t op, const int8_t* X, const float* x_scales, const int8_t* W,
                 const float* w_scales, const int32_t* offsets, void* D, cudaStream_t st) {
  const gemm_i8_desc_t& d = op->i8;
  const bool wide = op->wide;
  const int K = static_cast<int>(d.K);
  const int64_t w_rows = d.E * d.N;
  uint8_t* const ws = static_cast<uint8_t*>(op->ws);
  const I8Copy copy_x = {X, d.ldx, ws, op->ws_lda, d.R, K, true};
  const I8Copy copy_w = {W, d.ldw, ws + op->ws_b_off, op->ws_ldb, w_rows, K, wide};
  const int rc = launched(launch_i8_copies(copy_x, op->copy_b ? copy_w : I8Copy{}, op->num_sms, st));
  if (rc != GEMM_OK) return rc;
  // (the maps of what the caller owns; the others are the handle's)
  CUtensorMap wm{}, dm{};
  if (!op->copy_b && !encode_bytes(&wm, W, op->ws_ldb, d.K, w_rows)) return GEMM_ERR_CUDA;
  GroupedParams p{};
  p.E = d.E;
  p.R = static_cast<int>(d.R);
  p.K = K;
  p.N = static_cast<int>(d.N);
  p.idesc = idesc_f16(0, 0, 0, wide ? 256 : 128, 0);
  p.offsets = offsets;
  p.d_type = d.d_type;
  p.d_vec = is_16bit(d.d_type) && d.ldd % 8 == 0 && aligned(D, 16);
  p.d_tma = p.d_vec && d.N % 8 == 0 && op->split == 1;  // (clusters' threads store)
  if (p.d_tma && !encode_rows(&dm, D, d.ldd, d.N, d.R, 1, 64, 32)) return GEMM_ERR_CUDA;
  p.ldd = d.ldd;
  p.D = D;
  p.partial = reinterpret_cast<float*>(ws + op->ws_partial_off);
  p.counters = reinterpret_cast<unsigned*>(ws + op->ws_counters_off);
  p.status = op->status;
  p.timeout_ns = op->timeout_ns;
  p.debug_flags = op->debug_flags;
  op->debug_flags = 0;
  p.x_scales = x_scales;
  p.w_scales = w_scales;
  const CUtensorMap& w = op->copy_b ? op->map_w : wm;
  return launched(wide ? launch_scaled(w, op->map_x, op->map_x32, dm, p, op->units, st)
                       : launch_i8_tiles(op->tile_rows, w, op->map_x, op->map_x32, dm, p, op->units,
                                         op->split, st));
}

}  // namespace

extern "C" {

int gemm_i8_run(gemm_op_t op, const int8_t* X, const float* x_scales, const int8_t* W,
                const float* w_scales, const int32_t* offsets, void* D, gemm_stream_t stream) {
  if (!usable(op, Kind::kI8)) return GEMM_ERR_INVALID_ARG;
  const gemm_i8_desc_t& d = op->i8;
  if (d.R == 0 || d.N == 0) return GEMM_OK;
  if (!D || !x_scales || !w_scales || (d.K > 0 && (!X || !W)) || (d.E > 1 && !offsets))
    return GEMM_ERR_INVALID_ARG;
  if (!aligned(D, elem_size(d.d_type)) || !aligned(x_scales, 4) || !aligned(w_scales, 4) ||
      !aligned(offsets, 4) || (d.ldw % 16 == 0 && !aligned(W, 16)))
    return GEMM_ERR_MISALIGNED;
  if (op->tiles)
    return run_i8_tiles(op, X, x_scales, W, w_scales, offsets, D, static_cast<cudaStream_t>(stream));
  I8RowsParams p{};
  p.E = d.E;
  p.R = static_cast<int>(d.R);
  p.K = static_cast<int>(d.K);
  p.N = static_cast<int>(d.N);
  p.d_type = d.d_type;
  p.ldx = d.ldx;
  p.ldw = d.ldw;
  p.ldd = d.ldd;
  p.X = X;
  p.x_scales = x_scales;
  p.W = W;
  p.w_scales = w_scales;
  p.offsets = offsets;
  p.D = D;
  p.status = op->status;
  p.num_sms = op->num_sms;
  return launched(launch_i8_rows(p, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
