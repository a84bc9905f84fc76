// Row kernels of the 8-bit chain: the root-mean-square norm with the residual's
// addition, and the e4m3 quantisers (rows, silu(a)*b, 128 x 128 weight tiles).
//
// All are bound by HBM: every input element is read once, every output written
// once, and the row (norm) or the block (quantisers) stays in registers between
// the reduction and the store.  A thread owns 8 consecutive columns (one 16-byte
// bf16 load, one 8-byte e4m3 store), so the 16 lanes of a half warp own one
// 128-column scale block and its maximum is four shuffles.
#include <cuda_fp8.h>
#include <math.h>

#include "ar_device.cuh"
#include "ar_scaled.h"

namespace ar {

namespace {

constexpr float kE4m3Max = 448.0f;

// ---------------------------------------------------------------------------
// Eight consecutive columns, raw as loaded (kept raw until every load of the
// thread is issued) and as fp32.
// ---------------------------------------------------------------------------

struct Bf16Oct {
  uint4 v;
};
struct F32Oct {
  float4 a, b;
};

template <bool kBf16>
struct OctOf {
  using type = F32Oct;
};
template <>
struct OctOf<true> {
  using type = Bf16Oct;
};

__device__ __forceinline__ uint4 ldg_stream(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// Columns [col, col + 8) of the row at element offset `row0`; those at or past
// `cols` read as 0.  kVec: 16-byte loads (the caller checked alignment and that
// cols is a multiple of 8).  The plain ld (not .nc) is for inputs that may be the
// buffer the same kernel writes (kAlias).
template <bool kVec, bool kAlias = false>
__device__ __forceinline__ Bf16Oct load_oct(const uint16_t* p, int64_t row0, int col, int cols) {
  Bf16Oct o;
  o.v = make_uint4(0, 0, 0, 0);
  if (col >= cols) return o;
  if (kVec) {
    o.v = kAlias ? *reinterpret_cast<const uint4*>(p + row0 + col) : ldg_stream(p + row0 + col);
  } else {
    uint32_t e[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = col + i < cols ? p[row0 + col + i] : 0u;
    o.v = make_uint4(e[0] | (e[1] << 16), e[2] | (e[3] << 16), e[4] | (e[5] << 16), e[6] | (e[7] << 16));
  }
  return o;
}

template <bool kVec, bool kAlias = false>
__device__ __forceinline__ F32Oct load_oct(const float* p, int64_t row0, int col, int cols) {
  F32Oct o;
  o.a = make_float4(0.f, 0.f, 0.f, 0.f);
  o.b = o.a;
  if (col >= cols) return o;
  if (kVec) {
    if (kAlias) {
      o.a = *reinterpret_cast<const float4*>(p + row0 + col);
      o.b = *reinterpret_cast<const float4*>(p + row0 + col + 4);
    } else {
      const uint4 x = ldg_stream(p + row0 + col), y = ldg_stream(p + row0 + col + 4);
      o.a = make_float4(__uint_as_float(x.x), __uint_as_float(x.y), __uint_as_float(x.z), __uint_as_float(x.w));
      o.b = make_float4(__uint_as_float(y.x), __uint_as_float(y.y), __uint_as_float(y.z), __uint_as_float(y.w));
    }
  } else {
    float e[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = col + i < cols ? p[row0 + col + i] : 0.f;
    o.a = make_float4(e[0], e[1], e[2], e[3]);
    o.b = make_float4(e[4], e[5], e[6], e[7]);
  }
  return o;
}

__device__ __forceinline__ void unpack(const Bf16Oct& o, float (&f)[8]) {
  const uint32_t w[4] = {o.v.x, o.v.y, o.v.z, o.v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ void unpack(const F32Oct& o, float (&f)[8]) {
  f[0] = o.a.x, f[1] = o.a.y, f[2] = o.a.z, f[3] = o.a.w;
  f[4] = o.b.x, f[5] = o.b.y, f[6] = o.b.z, f[7] = o.b.w;
}

template <bool kVec>
__device__ __forceinline__ void store_oct(uint16_t* p, int64_t row0, int col, int cols, const float (&f)[8]) {
  if (col >= cols) return;
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  if (kVec) {
    *reinterpret_cast<uint4*>(p + row0 + col) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (col + i < cols) p[row0 + col + i] = static_cast<uint16_t>(w[i / 2] >> (16 * (i & 1)));
  }
}

template <bool kVec>
__device__ __forceinline__ void store_oct(float* p, int64_t row0, int col, int cols, const float (&f)[8]) {
  if (col >= cols) return;
  if (kVec) {
    *reinterpret_cast<float4*>(p + row0 + col) = make_float4(f[0], f[1], f[2], f[3]);
    *reinterpret_cast<float4*>(p + row0 + col + 4) = make_float4(f[4], f[5], f[6], f[7]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (col + i < cols) p[row0 + col + i] = f[i];
  }
}

// ---------------------------------------------------------------------------
// The e4m3 quantiser of one block: s = max|x| / 448 (1 if that is 0), q = e4m3(x/s),
// every operation rounded to nearest even.
//
// x/s is the correctly rounded fp32 quotient.  Where 2^-80 <= s <= 2^100 it comes
// from the correctly rounded reciprocal and one residual correction (div_rn_by): a
// quotient that e4m3 does not round to 0 is at least 2^-10, so |x| >= 2^-91 and the
// residual, at least 2^-24 of it, is a normal number; smaller quotients round to 0
// whatever their last bits.  Any other s (an infinite or a denormal block among
// them) takes the full division.
//
// The maximum ignores NaN (fmaxf), so a NaN stays in its own place; an infinity
// makes s infinite and its block NaN where the infinity is and 0 * inf elsewhere
// when read back: the block as a whole is lost, as it is in the formula.
// ---------------------------------------------------------------------------

struct BlockScale {
  float s, rcp;
  bool fast;
};

__device__ __forceinline__ BlockScale block_scale(float amax) {
  BlockScale b;
  b.s = __fdiv_rn(amax, kE4m3Max);
  if (b.s == 0.0f) b.s = 1.0f;
  b.rcp = __frcp_rn(b.s);
  b.fast = b.s >= 0x1p-80f && b.s <= 0x1p100f;
  return b;
}

__device__ __forceinline__ uint2 quant_oct(const float (&f)[8], const BlockScale& b) {
  float u[8];
  if (b.fast) {
#pragma unroll
    for (int i = 0; i < 8; ++i) u[i] = div_rn_by(f[i], b.s, b.rcp);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) u[i] = __fdiv_rn(f[i], b.s);
  }
  uint32_t w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(u[4 * h], u[4 * h + 1]), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(u[4 * h + 2], u[4 * h + 3]), __NV_SATFINITE, __NV_E4M3);
    w[h] = lo | (hi << 16);
  }
  return make_uint2(w[0], w[1]);
}

template <bool kVec>
__device__ __forceinline__ void store_q(uint8_t* p, int64_t row0, int col, int cols, uint2 q) {
  if (col >= cols) return;
  if (kVec) {
    *reinterpret_cast<uint2*>(p + row0 + col) = q;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (col + i < cols) p[row0 + col + i] = static_cast<uint8_t>((i < 4 ? q.x : q.y) >> (8 * (i & 3)));
  }
}

__device__ __forceinline__ float oct_amax(const float (&f)[8]) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(f[i]));
  return m;
}

// Maximum over the 16 lanes of a half warp (one 128-column block).
__device__ __forceinline__ float half_warp_max(float m) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  return m;
}

// ---------------------------------------------------------------------------
// RMS norm.  One row per "team" of blockDim.x threads; blockDim.y rows per CTA when
// the team is one warp.  The row stays in registers (kOcts octs a thread), so x and
// the residual are read once and the residual may be updated in place.
// ---------------------------------------------------------------------------

template <bool kXBf16, int kRes, int kOcts, bool kVec>  // kRes: 0 none, 1 fp32, 2 bf16
__global__ void __launch_bounds__(1024) rms_norm_kernel(RmsNormArgs a) {
  using XT = typename OctOf<kXBf16>::type;
  using RT = typename OctOf<kRes == 2>::type;
  __shared__ float partial[32];
  const int64_t row = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
  if (row >= a.rows) return;  // whole warps (blockDim.y > 1 only for one-warp teams)
  const int cols = a.cols;
  XT xr[kOcts];
  RT rr[kOcts];
  Bf16Oct wr[kOcts];
#pragma unroll
  for (int i = 0; i < kOcts; ++i) {
    const int col = (threadIdx.x + i * blockDim.x) * 8;
    if constexpr (kXBf16)
      xr[i] = load_oct<kVec>(static_cast<const uint16_t*>(a.x), row * a.ldx, col, cols);
    else
      xr[i] = load_oct<kVec>(static_cast<const float*>(a.x), row * a.ldx, col, cols);
    if constexpr (kRes == 2)
      rr[i] = load_oct<kVec, true>(static_cast<const uint16_t*>(a.residual), row * a.ldr, col, cols);
    else if constexpr (kRes == 1)
      rr[i] = load_oct<kVec, true>(static_cast<const float*>(a.residual), row * a.ldr, col, cols);
  }
  if (a.weight && a.w_bf16) {
#pragma unroll
    for (int i = 0; i < kOcts; ++i)
      wr[i] = load_oct<kVec, true>(static_cast<const uint16_t*>(a.weight), 0, (threadIdx.x + i * blockDim.x) * 8, cols);
  }
  float h[kOcts][8];
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < kOcts; ++i) {
    unpack(xr[i], h[i]);
    if constexpr (kRes != 0) {
      float r[8];
      unpack(rr[i], r);
#pragma unroll
      for (int k = 0; k < 8; ++k) h[i][k] = __fadd_rn(h[i][k], r[k]);
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) ss = fmaf(h[i][k], h[i][k], ss);
  }
  if constexpr (kRes != 0) {
    if (a.sum) {
#pragma unroll
      for (int i = 0; i < kOcts; ++i) {
        const int col = (threadIdx.x + i * blockDim.x) * 8;
        if constexpr (kRes == 2)
          store_oct<kVec>(static_cast<uint16_t*>(a.sum), row * a.lds, col, cols, h[i]);
        else
          store_oct<kVec>(static_cast<float*>(a.sum), row * a.lds, col, cols, h[i]);
      }
    }
  }
  if (!a.y && !a.q) return;  // the sum alone
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  if (blockDim.x > 32) {
    // One partial per warp; every warp adds them in the same order.
    if ((threadIdx.x & 31) == 0) partial[threadIdx.x >> 5] = ss;
    __syncthreads();
    const int lane = threadIdx.x & 31;
    ss = lane < static_cast<int>(blockDim.x >> 5) ? partial[lane] : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  }
  const float inv = 1.0f / sqrtf(ss / static_cast<float>(cols) + a.eps);
#pragma unroll
  for (int i = 0; i < kOcts; ++i) {
    const int col = (threadIdx.x + i * blockDim.x) * 8;
#pragma unroll
    for (int k = 0; k < 8; ++k) h[i][k] = __fmul_rn(h[i][k], inv);
    if (a.weight) {
      float w[8];
      if (a.w_bf16)
        unpack(wr[i], w);
      else
        unpack(load_oct<kVec, true>(static_cast<const float*>(a.weight), 0, col, cols), w);
#pragma unroll
      for (int k = 0; k < 8; ++k) h[i][k] = __fmul_rn(h[i][k], w[k]);
    }
    if (a.y) store_oct<kVec>(a.y, row * a.ldy, col, cols, h[i]);
    if (a.q) {
      const BlockScale b = block_scale(half_warp_max(oct_amax(h[i])));
      store_q<kVec>(a.q, row * a.ldq, col, cols, quant_oct(h[i], b));
      if ((threadIdx.x & 15) == 0 && col < cols)
        a.scale[row * a.blocks + (col >> 7)] = b.s;
    }
  }
}

template <bool kXBf16, int kRes, int kOcts>
cudaError_t launch_norm_octs(const RmsNormArgs& a, bool vec, dim3 grid, dim3 block, cudaStream_t st) {
  if (vec)
    rms_norm_kernel<kXBf16, kRes, kOcts, true><<<grid, block, 0, st>>>(a);
  else
    rms_norm_kernel<kXBf16, kRes, kOcts, false><<<grid, block, 0, st>>>(a);
  return cudaGetLastError();
}

template <bool kXBf16, int kRes>
cudaError_t launch_norm(const RmsNormArgs& a, bool vec, cudaStream_t st) {
  const int octs = (a.cols + 7) / 8;
  if (octs <= 128) {  // up to 1024 columns: a warp per row, no shared memory
    const dim3 block(32, a.rows >= 8 ? 8 : static_cast<unsigned>(a.rows));
    const dim3 grid(static_cast<unsigned>((a.rows + block.y - 1) / block.y));
    if (octs <= 32) return launch_norm_octs<kXBf16, kRes, 1>(a, vec, grid, block, st);
    if (octs <= 64) return launch_norm_octs<kXBf16, kRes, 2>(a, vec, grid, block, st);
    return launch_norm_octs<kXBf16, kRes, 4>(a, vec, grid, block, st);
  }
  const dim3 grid(static_cast<unsigned>(a.rows));
  const int per = octs <= 1024 ? (octs <= 512 && a.rows > 296 ? 2 : 1) : octs <= 2048 ? 2 : 4;
  const dim3 block(static_cast<unsigned>(((octs + per - 1) / per + 31) / 32 * 32));
  if (per == 1) return launch_norm_octs<kXBf16, kRes, 1>(a, vec, grid, block, st);
  if (per == 2) return launch_norm_octs<kXBf16, kRes, 2>(a, vec, grid, block, st);
  return launch_norm_octs<kXBf16, kRes, 4>(a, vec, grid, block, st);
}

bool aligned_to(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

// ---------------------------------------------------------------------------
// Row quantiser: a half warp per (row, 128-column block), kUnits consecutive blocks
// each, so a thread has kUnits 16-byte loads in flight (twice that with the gate).
// ---------------------------------------------------------------------------

constexpr int kUnits = 4;

template <bool kXBf16, bool kGated, bool kVec>
__global__ void __launch_bounds__(256) row_quant_kernel(RowQuantArgs a) {
  using XT = typename OctOf<kXBf16>::type;
  const int64_t half = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 4;
  const int lane = threadIdx.x & 15;
  const int64_t units = a.rows * a.blocks;
  const int64_t first = half * kUnits;
  if ((half & ~int64_t(1)) * kUnits >= units) return;  // both halves of the warp are past the end
  int64_t row = first / a.blocks;
  int blk = static_cast<int>(first - row * a.blocks);
  XT xr[kUnits];
  Bf16Oct br[kUnits];
  int64_t rows[kUnits];
  int cols[kUnits];
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    rows[i] = row;
    // past the end: a column that no load or store takes
    cols[i] = first + i < units ? blk * 128 + lane * 8 : a.cols;
    if constexpr (kXBf16)
      xr[i] = load_oct<kVec>(static_cast<const uint16_t*>(a.x), row * a.ldx, cols[i], a.cols);
    else
      xr[i] = load_oct<kVec>(static_cast<const float*>(a.x), row * a.ldx, cols[i], a.cols);
    if constexpr (kGated) br[i] = load_oct<kVec>(a.gate, row * a.ldg, cols[i], a.cols);
    if (++blk == a.blocks) {
      blk = 0;
      ++row;
    }
  }
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    float f[8];
    unpack(xr[i], f);
    if constexpr (kGated) {
      float g[8];
      unpack(br[i], g);
      // silu(f) = f / (1 + exp(-f)): exp(-f) = inf gives -0, as the limit is
#pragma unroll
      for (int k = 0; k < 8; ++k) f[k] = __fmul_rn(__fdividef(f[k], 1.0f + expf(-f[k])), g[k]);
    }
    const BlockScale b = block_scale(half_warp_max(oct_amax(f)));
    store_q<kVec>(a.q, rows[i] * a.ldq, cols[i], a.cols, quant_oct(f, b));
    if (lane == 0 && cols[i] < a.cols) a.scale[first + i] = b.s;
  }
}

// ---------------------------------------------------------------------------
// Weight quantiser: a CTA per 128 x 128 tile.  Thread t owns the oct t % 16 of the
// rows t / 16 + 16 i, i < 8, in registers between the tile's maximum and the store.
// ---------------------------------------------------------------------------

template <bool kXBf16, bool kVec>
__global__ void __launch_bounds__(256) tile_quant_kernel(TileQuantArgs a) {
  using XT = typename OctOf<kXBf16>::type;
  __shared__ float partial[8];
  const int64_t tile = blockIdx.x;
  const int64_t per_mat = static_cast<int64_t>(a.row_blocks) * a.blocks;
  const int64_t mat = tile / per_mat;
  const int rb = static_cast<int>((tile - mat * per_mat) / a.blocks);
  const int cb = static_cast<int>(tile - mat * per_mat - static_cast<int64_t>(rb) * a.blocks);
  const int col = cb * 128 + (threadIdx.x & 15) * 8;
  XT xr[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t r = static_cast<int64_t>(rb) * 128 + (threadIdx.x >> 4) + 16 * i;
    const int c = r < a.rows ? col : a.cols;  // a row past the end reads as 0
    const int64_t row0 = (mat * a.rows + r) * a.ldx;
    if constexpr (kXBf16)
      xr[i] = load_oct<kVec>(static_cast<const uint16_t*>(a.x), row0, c, a.cols);
    else
      xr[i] = load_oct<kVec>(static_cast<const float*>(a.x), row0, c, a.cols);
  }
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float f[8];
    unpack(xr[i], f);
    m = fmaxf(m, oct_amax(f));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if ((threadIdx.x & 31) == 0) partial[threadIdx.x >> 5] = m;
  __syncthreads();
  m = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, partial[i]);
  const BlockScale b = block_scale(m);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t r = static_cast<int64_t>(rb) * 128 + (threadIdx.x >> 4) + 16 * i;
    if (r >= a.rows) continue;
    float f[8];
    unpack(xr[i], f);
    store_q<kVec>(a.q, (mat * a.rows + r) * a.ldq, col, a.cols, quant_oct(f, b));
  }
  if (threadIdx.x == 0) a.scale[tile] = b.s;
}

}  // namespace

cudaError_t launch_rms_norm(const RmsNormArgs& a, cudaStream_t st) {
  const int xe = a.x_bf16 ? 8 : 4, re = a.r_bf16 ? 8 : 4;  // elements per 16 bytes
  const bool vec = a.cols % 8 == 0 && aligned_to(a.x, 16) && a.ldx % xe == 0 &&
                   (!a.residual || (aligned_to(a.residual, 16) && a.ldr % re == 0)) &&
                   (!a.sum || (aligned_to(a.sum, 16) && a.lds % re == 0)) &&
                   (!a.weight || aligned_to(a.weight, 16)) && (!a.y || (aligned_to(a.y, 16) && a.ldy % 8 == 0)) &&
                   (!a.q || (aligned_to(a.q, 8) && a.ldq % 8 == 0));
  const int res = !a.residual ? 0 : a.r_bf16 ? 2 : 1;
  if (a.x_bf16) {
    if (res == 0) return launch_norm<true, 0>(a, vec, st);
    if (res == 1) return launch_norm<true, 1>(a, vec, st);
    return launch_norm<true, 2>(a, vec, st);
  }
  if (res == 0) return launch_norm<false, 0>(a, vec, st);
  if (res == 1) return launch_norm<false, 1>(a, vec, st);
  return launch_norm<false, 2>(a, vec, st);
}

cudaError_t launch_row_quant(const RowQuantArgs& a, cudaStream_t st) {
  const bool vec = a.cols % 8 == 0 && aligned_to(a.x, 16) && a.ldx % (a.x_bf16 ? 8 : 4) == 0 &&
                   (!a.gate || (aligned_to(a.gate, 16) && a.ldg % 8 == 0)) && aligned_to(a.q, 8) && a.ldq % 8 == 0;
  const int64_t halves = (a.rows * a.blocks + kUnits - 1) / kUnits;
  const unsigned grid = static_cast<unsigned>((halves + 15) / 16);
#define AR_ROW_QUANT(BF, GATED)                                   \
  do {                                                            \
    if (vec)                                                      \
      row_quant_kernel<BF, GATED, true><<<grid, 256, 0, st>>>(a);  \
    else                                                          \
      row_quant_kernel<BF, GATED, false><<<grid, 256, 0, st>>>(a); \
  } while (0)
  if (a.gate)
    AR_ROW_QUANT(true, true);
  else if (a.x_bf16)
    AR_ROW_QUANT(true, false);
  else
    AR_ROW_QUANT(false, false);
#undef AR_ROW_QUANT
  return cudaGetLastError();
}

cudaError_t launch_tile_quant(const TileQuantArgs& a, cudaStream_t st) {
  const bool vec = a.cols % 8 == 0 && aligned_to(a.x, 16) && a.ldx % (a.x_bf16 ? 8 : 4) == 0 && aligned_to(a.q, 8) &&
                   a.ldq % 8 == 0;
  const unsigned grid = static_cast<unsigned>(a.count * a.row_blocks * a.blocks);
  if (a.x_bf16) {
    if (vec)
      tile_quant_kernel<true, true><<<grid, 256, 0, st>>>(a);
    else
      tile_quant_kernel<true, false><<<grid, 256, 0, st>>>(a);
  } else {
    if (vec)
      tile_quant_kernel<false, true><<<grid, 256, 0, st>>>(a);
    else
      tile_quant_kernel<false, false><<<grid, 256, 0, st>>>(a);
  }
  return cudaGetLastError();
}

}  // namespace ar
