// C ABI of the 8-bit chain: argument checks and launches of the norm, the block
// quantisers and the products (scaled_rows.cu, scaled_product.cu).
#include <math.h>
#include <stdlib.h>
#include <string.h>

#include "../../include/ar.h"
#include "ar_internal.h"
#include "ar_scaled.h"

namespace {

constexpr int64_t kMaxRows = 1ll << 30;  // row indices, and their tiles' ends, in 32 bits
// Row quantisers: the most 128-column blocks whose grid has below 2^31 CTAs of 8 warps, at two a warp (unaligned rows).
constexpr int64_t kMaxRowBlocks = 16 * ((1ll << 31) - 1);

bool aligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

int64_t blocks_of(int64_t n) { return (n + 127) / 128; }

bool fault_is(const char* kind) {  // the AR_FAULT test hook (see ar.h)
  const char* f = getenv("AR_FAULT");
  return f && !strcmp(f, kind);
}

bool dtype_ok(ar_dtype t) { return t == AR_F32 || t == AR_BF16; }

ar_status from_cuda(cudaError_t e) { return e == cudaSuccess ? AR_OK : AR_ECUDA; }

// AR_FAULT=wait: the tile kernel's waits run out, after 2 ms.
void wait_hook(ar::ProductArgs& a) {
  if (!fault_is("wait")) return;
  a.starve = 1;
  a.timeout_ns = 2000000;
}

// The checks that the three products share.  el: bytes per operand element.
ar_status check_product(const void* X, int64_t ldx, int64_t n, int64_t in, const void* W, int64_t ldw, int64_t experts,
                        int64_t out, const void* Y, int64_t ldy, int el) {
  if (fault_is("param")) return AR_EINVAL;
  if (n < 0 || in <= 0 || out <= 0 || experts <= 0) return AR_EINVAL;
  if (in % (16 / el) != 0 || ldx % (16 / el) != 0 || ldw % (16 / el) != 0) return AR_EINVAL;
  if (ldx < in || ldw < in || ldy < out) return AR_EINVAL;
  if (n > kMaxRows || in >= (1ll << 30) || experts > ar::kMaxExperts || out > kMaxRows || experts * out > kMaxRows)
    return AR_EUNSUPPORTED;
  if (ldx >= (1ll << 38) || ldw >= (1ll << 38)) return AR_EUNSUPPORTED;  // the tensor maps' pitches
  if (n == 0) return AR_OK;
  if (!X || !W || !Y || !aligned(X, 16) || !aligned(W, 16) || !aligned(Y, 2)) return AR_EINVAL;
  return AR_OK;
}

}  // namespace

extern "C" {

ar_status ar_rms_norm(const void* x, ar_dtype x_dtype, int64_t ldx, int64_t rows, int64_t cols, const void* residual,
                      ar_dtype r_dtype, int64_t ldr, const void* weight, ar_dtype w_dtype, float eps, void* sum,
                      int64_t lds, uint16_t* y, int64_t ldy, uint8_t* q, int64_t ldq, float* scale, void* stream) {
  if (fault_is("param")) return AR_EINVAL;
  if (rows < 0 || cols < 0 || !dtype_ok(x_dtype) || !dtype_ok(r_dtype) || !dtype_ok(w_dtype)) return AR_EINVAL;
  if (!(eps >= 0.0f) || !isfinite(eps)) return AR_EINVAL;
  if (rows == 0 || cols == 0) return AR_OK;
  if (!x || (sum && !residual) || (q && !scale) || (!y && !q && !sum)) return AR_EINVAL;
  if (ldx < cols || (residual && ldr < cols) || (sum && lds < cols) || (y && ldy < cols) || (q && ldq < cols))
    return AR_EINVAL;
  const uintptr_t xa = x_dtype == AR_F32 ? 4 : 2, ra = r_dtype == AR_F32 ? 4 : 2, wa = w_dtype == AR_F32 ? 4 : 2;
  if (!aligned(x, xa) || !aligned(residual, ra) || !aligned(sum, ra) || !aligned(weight, wa) || !aligned(y, 2) ||
      !aligned(scale, 4))
    return AR_EINVAL;
  if (cols > ar::kNormMaxCols || rows > kMaxRows) return AR_EUNSUPPORTED;
  if (fault_is("launch")) return AR_ECUDA;
  ar::RmsNormArgs a;
  a.x = x;
  a.x_bf16 = x_dtype == AR_BF16;
  a.ldx = ldx;
  a.rows = rows;
  a.cols = static_cast<int>(cols);
  a.blocks = static_cast<int>(blocks_of(cols));
  a.residual = residual;
  a.r_bf16 = r_dtype == AR_BF16;
  a.ldr = ldr;
  a.weight = weight;
  a.w_bf16 = w_dtype == AR_BF16;
  a.eps = eps;
  a.sum = sum;
  a.lds = lds;
  a.y = y;
  a.ldy = ldy;
  a.q = q;
  a.ldq = ldq;
  a.scale = scale;
  return from_cuda(ar::launch_rms_norm(a, static_cast<cudaStream_t>(stream)));
}

ar_status ar_quant_scaled(const void* x, ar_dtype x_dtype, int64_t ldx, int64_t count, int64_t rows, int64_t cols,
                          int32_t block_rows, uint8_t* q, int64_t ldq, float* scale, void* stream) {
  if (fault_is("param")) return AR_EINVAL;
  if (count < 0 || rows < 0 || cols < 0 || !dtype_ok(x_dtype)) return AR_EINVAL;
  if (block_rows != 1 && block_rows != 128) return AR_EINVAL;
  if (count == 0 || rows == 0 || cols == 0) return AR_OK;
  if (!x || !q || !scale || ldx < cols || ldq < cols) return AR_EINVAL;
  if (!aligned(x, x_dtype == AR_F32 ? 4 : 2) || !aligned(scale, 4)) return AR_EINVAL;
  if (rows > kMaxRows || cols > kMaxRows || count > kMaxRows) return AR_EUNSUPPORTED;
  if (count * rows > (1ll << 40) / blocks_of(cols)) return AR_EUNSUPPORTED;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (block_rows == 1) {
    // rows of every matrix follow one another: one matrix of count * rows rows
    if (count * rows > kMaxRowBlocks / blocks_of(cols)) return AR_EUNSUPPORTED;
    if (fault_is("launch")) return AR_ECUDA;
    ar::RowQuantArgs a;
    a.x = x;
    a.x_bf16 = x_dtype == AR_BF16;
    a.ldx = ldx;
    a.rows = count * rows;
    a.cols = static_cast<int>(cols);
    a.blocks = static_cast<int>(blocks_of(cols));
    a.q = q;
    a.ldq = ldq;
    a.scale = scale;
    return from_cuda(ar::launch_row_quant(a, st));
  }
  if (count * blocks_of(rows) * blocks_of(cols) >= (1ll << 31)) return AR_EUNSUPPORTED;  // grid size
  if (fault_is("launch")) return AR_ECUDA;
  ar::TileQuantArgs a;
  a.x = x;
  a.x_bf16 = x_dtype == AR_BF16;
  a.ldx = ldx;
  a.count = count;
  a.rows = rows;
  a.cols = static_cast<int>(cols);
  a.blocks = static_cast<int>(blocks_of(cols));
  a.row_blocks = static_cast<int>(blocks_of(rows));
  a.q = q;
  a.ldq = ldq;
  a.scale = scale;
  return from_cuda(ar::launch_tile_quant(a, st));
}

ar_status ar_silu_mul_scaled(const uint16_t* a, int64_t lda, const uint16_t* b, int64_t ldb, int64_t rows, int64_t cols,
                             uint8_t* q, int64_t ldq, float* scale, void* stream) {
  if (fault_is("param")) return AR_EINVAL;
  if (rows < 0 || cols < 0) return AR_EINVAL;
  if (rows == 0 || cols == 0) return AR_OK;
  if (!a || !b || !q || !scale || lda < cols || ldb < cols || ldq < cols) return AR_EINVAL;
  if (!aligned(a, 2) || !aligned(b, 2) || !aligned(scale, 4)) return AR_EINVAL;
  if (rows > kMaxRows || cols > kMaxRows || rows > kMaxRowBlocks / blocks_of(cols)) return AR_EUNSUPPORTED;
  if (fault_is("launch")) return AR_ECUDA;
  ar::RowQuantArgs r;
  r.x = a;
  r.x_bf16 = 1;
  r.ldx = lda;
  r.gate = b;
  r.ldg = ldb;
  r.rows = rows;
  r.cols = static_cast<int>(cols);
  r.blocks = static_cast<int>(blocks_of(cols));
  r.q = q;
  r.ldq = ldq;
  r.scale = scale;
  return from_cuda(ar::launch_row_quant(r, static_cast<cudaStream_t>(stream)));
}

ar_status ar_linear_scaled(const uint8_t* X, int64_t ldx, const float* x_scale, int64_t n, int64_t in, const uint8_t* W,
                           int64_t ldw, const float* w_scale, int64_t out, const uint16_t* add, int64_t ldadd,
                           uint16_t* Y, int64_t ldy, int32_t* status, void* stream) {
  const ar_status s = check_product(X, ldx, n, in, W, ldw, 1, out, Y, ldy, 1);
  if (s != AR_OK || n == 0) return s;
  if (!x_scale || !w_scale || !aligned(x_scale, 4) || !aligned(w_scale, 4)) return AR_EINVAL;
  if (add && (ldadd < out || !aligned(add, 2))) return AR_EINVAL;
  if (fault_is("launch")) return AR_ECUDA;
  ar::ProductArgs a;
  a.f8 = 1;
  a.X = X;
  a.ldx = ldx;
  a.W = W;
  a.ldw = ldw;
  a.n = static_cast<int>(n);
  a.in = static_cast<int>(in);
  a.out = static_cast<int>(out);
  a.nkb = static_cast<int>(blocks_of(in));
  a.out_blocks = static_cast<int>(blocks_of(out));
  a.xs = x_scale;
  a.ws = w_scale;
  a.add = add;
  a.ldadd = ldadd;
  a.Y = Y;
  a.ldy = ldy;
  a.vec_y = aligned(Y, 16) && ldy % 8 == 0 && (!add || (aligned(add, 16) && ldadd % 8 == 0));
  a.status = status;
  wait_hook(a);
  return from_cuda(ar::launch_product(a, static_cast<cudaStream_t>(stream)));
}

ar_status ar_grouped_linear(const uint16_t* X, int64_t ldx, int64_t n, int64_t in, const int32_t* offsets,
                            int64_t experts, const uint16_t* W_hi, const uint16_t* W_lo, int64_t ldw, int64_t out,
                            uint16_t* Y, int64_t ldy, int32_t* status, void* stream) {
  const ar_status s = check_product(X, ldx, n, in, W_hi, ldw, experts, out, Y, ldy, 2);
  if (s != AR_OK || n == 0) return s;
  if (!offsets || !aligned(offsets, 4) || !aligned(W_lo, 16)) return AR_EINVAL;
  if (fault_is("launch")) return AR_ECUDA;
  ar::ProductArgs a;
  a.X = X;
  a.ldx = ldx * 2;
  a.W = W_hi;
  a.W_lo = W_lo;
  a.ldw = ldw * 2;
  a.n = static_cast<int>(n);
  a.in = static_cast<int>(in);
  a.out = static_cast<int>(out);
  a.nkb = static_cast<int>(blocks_of(in * 2));
  a.out_blocks = static_cast<int>(blocks_of(out));
  a.experts = static_cast<int>(experts);
  a.offsets = offsets;
  a.Y = Y;
  a.ldy = ldy;
  a.vec_y = aligned(Y, 16) && ldy % 8 == 0;
  a.status = status;
  wait_hook(a);
  return from_cuda(ar::launch_product(a, static_cast<cudaStream_t>(stream)));
}

ar_status ar_grouped_linear_scaled(const uint8_t* X, int64_t ldx, const float* x_scale, int64_t n, int64_t in,
                                   const int32_t* offsets, int64_t experts, const uint8_t* W, int64_t ldw,
                                   const float* w_scale, int64_t out, uint16_t* Y, int64_t ldy, int32_t* status,
                                   void* stream) {
  const ar_status s = check_product(X, ldx, n, in, W, ldw, experts, out, Y, ldy, 1);
  if (s != AR_OK || n == 0) return s;
  if (!offsets || !aligned(offsets, 4) || !x_scale || !w_scale || !aligned(x_scale, 4) || !aligned(w_scale, 4))
    return AR_EINVAL;
  if (fault_is("launch")) return AR_ECUDA;
  ar::ProductArgs a;
  a.f8 = 1;
  a.X = X;
  a.ldx = ldx;
  a.W = W;
  a.ldw = ldw;
  a.n = static_cast<int>(n);
  a.in = static_cast<int>(in);
  a.out = static_cast<int>(out);
  a.nkb = static_cast<int>(blocks_of(in));
  a.out_blocks = static_cast<int>(blocks_of(out));
  a.experts = static_cast<int>(experts);
  a.offsets = offsets;
  a.xs = x_scale;
  a.ws = w_scale;
  a.Y = Y;
  a.ldy = ldy;
  a.vec_y = aligned(Y, 16) && ldy % 8 == 0;
  a.status = status;
  wait_hook(a);
  return from_cuda(ar::launch_product(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
