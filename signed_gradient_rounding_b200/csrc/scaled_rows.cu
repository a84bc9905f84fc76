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
struct Bf16Raw {  // loaded one by one: packing them would wait for the loads
  uint16_t e[8];
};
struct F32Oct {
  float4 a, b;
};

template <bool kBf16, bool kVec>
struct OctOf {
  using type = F32Oct;
};
template <>
struct OctOf<true, true> {
  using type = Bf16Oct;
};
template <>
struct OctOf<true, false> {
  using type = Bf16Raw;
};

// Read once.  (Not .nc: see chain_wait.)
__device__ __forceinline__ uint4 ld_stream(const void* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// Eight elements of a lane: where they are.  With 16-byte accesses (kVec: aligned rows,
// cols a multiple of 8) they are eight consecutive columns.  Without, element k is column
// col + 32 (k % 4) of one of two 128-column blocks (k < 4, k >= 4), so that a load or store
// instruction of the warp covers consecutive elements: eight consecutive columns per lane
// would touch 16 sectors per instruction instead of 2, and ran four times longer.
struct Place {
  int64_t row0, row1;  // element offsets of the rows of k < 4 and k >= 4 (kVec: row0)
  int col0, col1;      // first column (kVec: of all eight; else of the lane)
};

__device__ __forceinline__ int place_col(const Place& p, int k) { return (k < 4 ? p.col0 : p.col1) + 32 * (k & 3); }
__device__ __forceinline__ int64_t place_at(const Place& p, int k) { return (k < 4 ? p.row0 : p.row1) + place_col(p, k); }

// Elements at or past `cols` read as 0.  kAlias: loads that the compiler orders with the stores
// around them, for inputs that may be the buffer the same kernel writes.
template <bool kVec, bool kAlias = false>
__device__ __forceinline__ typename OctOf<true, kVec>::type load_oct(const uint16_t* p, const Place& at, int cols) {
  typename OctOf<true, kVec>::type o;
  if constexpr (kVec) {
    o.v = make_uint4(0, 0, 0, 0);
    if (at.col0 < cols)
      o.v = kAlias ? *reinterpret_cast<const uint4*>(p + at.row0 + at.col0) : ld_stream(p + at.row0 + at.col0);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) o.e[k] = place_col(at, k) < cols ? p[place_at(at, k)] : uint16_t(0);
  }
  return o;
}

template <bool kVec, bool kAlias = false>
__device__ __forceinline__ F32Oct load_oct(const float* p, const Place& at, int cols) {
  F32Oct o;
  o.a = make_float4(0.f, 0.f, 0.f, 0.f);
  o.b = o.a;
  if (kVec) {
    if (at.col0 >= cols) return o;
    const float* q = p + at.row0 + at.col0;
    if (kAlias) {
      o.a = *reinterpret_cast<const float4*>(q);
      o.b = *reinterpret_cast<const float4*>(q + 4);
    } else {
      const uint4 x = ld_stream(q), y = ld_stream(q + 4);
      o.a = make_float4(__uint_as_float(x.x), __uint_as_float(x.y), __uint_as_float(x.z), __uint_as_float(x.w));
      o.b = make_float4(__uint_as_float(y.x), __uint_as_float(y.y), __uint_as_float(y.z), __uint_as_float(y.w));
    }
  } else {
    float e[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) e[k] = place_col(at, k) < cols ? p[place_at(at, k)] : 0.f;
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

__device__ __forceinline__ void unpack(const Bf16Raw& o, float (&f)[8]) {
#pragma unroll
  for (int k = 0; k < 8; ++k) f[k] = bf16_bits_to_f32(o.e[k]);
}

__device__ __forceinline__ void unpack(const F32Oct& o, float (&f)[8]) {
  f[0] = o.a.x, f[1] = o.a.y, f[2] = o.a.z, f[3] = o.a.w;
  f[4] = o.b.x, f[5] = o.b.y, f[6] = o.b.z, f[7] = o.b.w;
}

template <bool kVec>
__device__ __forceinline__ void store_oct(uint16_t* p, const Place& at, int cols, const float (&f)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  if (kVec) {
    if (at.col0 < cols) *reinterpret_cast<uint4*>(p + at.row0 + at.col0) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (place_col(at, k) < cols) p[place_at(at, k)] = static_cast<uint16_t>(w[k / 2] >> (16 * (k & 1)));
  }
}

template <bool kVec>
__device__ __forceinline__ void store_oct(float* p, const Place& at, int cols, const float (&f)[8]) {
  if (kVec) {
    if (at.col0 >= cols) return;
    float* q = p + at.row0 + at.col0;
    *reinterpret_cast<float4*>(q) = make_float4(f[0], f[1], f[2], f[3]);
    *reinterpret_cast<float4*>(q + 4) = make_float4(f[4], f[5], f[6], f[7]);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (place_col(at, k) < cols) p[place_at(at, k)] = f[k];
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

// The scale and its reciprocal cost as much as the block's quotients if they come from full
// divisions, so in the fast range they do not either: amax / 448 by div_rn_by with the
// constant's reciprocal, and 1/s from the hardware's approximation (within one unit) by one
// Newton step with fma, which gives the correctly rounded reciprocal of every s whose
// significand is not all ones (Markstein 1990, as div_rn_by); those take the slow path.
__device__ __forceinline__ BlockScale block_scale(float amax) {
  BlockScale b;
  b.fast = amax >= 0x1p-70f && amax <= 0x1p100f;
  b.s = div_rn_by(amax, kE4m3Max, 1.0f / kE4m3Max);
  b.fast = b.fast && (__float_as_uint(b.s) & 0x7FFFFFu) != 0x7FFFFFu;
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(b.s));
  b.rcp = __fmaf_rn(__fmaf_rn(-b.s, y, 1.0f), y, y);
  if (!b.fast) {
    b.s = __fdiv_rn(amax, kE4m3Max);
    if (b.s == 0.0f) {
      b.s = 1.0f;
      b.rcp = 1.0f;
      b.fast = amax == 0.0f;  // (past the end of rows, for one: every quotient is 0)
    }
  }
  return b;
}

__device__ __forceinline__ uint2 quant_oct(const float (&f)[8], const BlockScale& b0, const BlockScale& b1) {
  float u[8];
  if (b0.fast && b1.fast) {
#pragma unroll
    for (int i = 0; i < 8; ++i) u[i] = div_rn_by(f[i], (i < 4 ? b0 : b1).s, (i < 4 ? b0 : b1).rcp);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) u[i] = __fdiv_rn(f[i], (i < 4 ? b0 : b1).s);
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
__device__ __forceinline__ void store_q(uint8_t* p, const Place& at, int cols, uint2 q) {
  if (kVec) {
    if (at.col0 < cols) *reinterpret_cast<uint2*>(p + at.row0 + at.col0) = q;
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (place_col(at, k) < cols) p[place_at(at, k)] = static_cast<uint8_t>((k < 4 ? q.x : q.y) >> (8 * (k & 3)));
  }
}

// Scales of the block (kVec) or the two blocks of a lane's elements.  kVec: the 16 lanes of a
// half warp own a block; else the whole warp owns both.
template <bool kVec>
__device__ __forceinline__ void lane_scales(const float (&f)[8], BlockScale& b0, BlockScale& b1) {
  if (kVec) {
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(f[i]));
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    b0 = block_scale(m);
    b1 = b0;
  } else {
    float m0 = 0.f, m1 = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      m0 = fmaxf(m0, fabsf(f[i]));
      m1 = fmaxf(m1, fabsf(f[i + 4]));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      m0 = fmaxf(m0, __shfl_xor_sync(0xffffffffu, m0, o));
      m1 = fmaxf(m1, __shfl_xor_sync(0xffffffffu, m1, o));
    }
    b0 = block_scale(m0);
    b1 = block_scale(m1);
  }
}

// ---------------------------------------------------------------------------
// RMS norm.  One row per "team" of blockDim.x threads; blockDim.y rows per CTA when
// the team is one warp.  The row stays in registers (kOcts octs a thread), so x and
// the residual are read once and the residual may be updated in place.
// ---------------------------------------------------------------------------

// Threads of a CTA with two octs each, two CTAs an SM: the most for which the register file leaves a
// thread 40 registers (at 800 the compiler has 32, and spills two to five times as much).
constexpr int kTwoOctThreads = 768;

// Spills: up to 48 bytes a thread at two octs and 144 at four, mostly of addresses; 1024 threads of
// four octs, or two CTAs of two, leave no more registers.
template <bool kXBf16, int kRes, int kOcts, bool kVec>  // kRes: 0 none, 1 fp32, 2 bf16
__global__ void __launch_bounds__(kOcts == 2 ? kTwoOctThreads : 1024, kOcts == 2 ? 2 : 1) rms_norm_kernel(RmsNormArgs a) {
  using XT = typename OctOf<kXBf16, kVec>::type;
  using RT = typename OctOf<kRes == 2, kVec>::type;
  __shared__ float partial[32];
  chain_next();
  chain_wait();
  const int64_t row = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
  if (row >= a.rows) return;  // whole warps (blockDim.y > 1 only for one-warp teams)
  const int cols = a.cols;
  const int lane = threadIdx.x & 31;
  // Octs i * blockDim.x + threadIdx.x of the row, or (not kVec) the warp's 256 columns.
  auto place = [&](int64_t ld, int i) {
    Place p;
    const int oct = threadIdx.x + i * blockDim.x;
    p.row0 = p.row1 = row * ld;
    p.col0 = kVec ? oct * 8 : (oct - lane) * 8 + lane;
    p.col1 = p.col0 + 128;
    return p;
  };
  // Every load of the thread is issued before the first value is used (unaligned rows take eight
  // loads an oct: there an oct's are).
  constexpr int kAhead = kVec ? kOcts : 1;
  XT xr[kAhead];
  RT rr[kAhead];
  auto load = [&](int i, int at) {
    if constexpr (kXBf16)
      xr[at] = load_oct<kVec>(static_cast<const uint16_t*>(a.x), place(a.ldx, i), cols);
    else
      xr[at] = load_oct<kVec>(static_cast<const float*>(a.x), place(a.ldx, i), cols);
    if constexpr (kRes == 2)
      rr[at] = load_oct<kVec, true>(static_cast<const uint16_t*>(a.residual), place(a.ldr, i), cols);
    else if constexpr (kRes == 1)
      rr[at] = load_oct<kVec, true>(static_cast<const float*>(a.residual), place(a.ldr, i), cols);
  };
  if constexpr (kVec) {
#pragma unroll
    for (int i = 0; i < kOcts; ++i) load(i, i);
  }
  Place col_place[kOcts];
#pragma unroll
  for (int i = 0; i < kOcts; ++i) col_place[i] = place(0, i);
  Bf16Oct wr[kOcts];
  if constexpr (kVec) if (a.weight && a.w_bf16) {
#pragma unroll
    for (int i = 0; i < kOcts; ++i)
      wr[i] = load_oct<kVec, true>(static_cast<const uint16_t*>(a.weight), col_place[i], cols);
  }
  float h[kOcts][8];
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < kOcts; ++i) {
    if constexpr (!kVec) load(i, 0);
    unpack(xr[kVec ? i : 0], h[i]);
    if constexpr (kRes != 0) {
      float r[8];
      unpack(rr[kVec ? i : 0], r);
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
        if constexpr (kRes == 2)
          store_oct<kVec>(static_cast<uint16_t*>(a.sum), place(a.lds, i), cols, h[i]);
        else
          store_oct<kVec>(static_cast<float*>(a.sum), place(a.lds, i), cols, h[i]);
      }
    }
  }
  if (!a.y && !a.q) return;  // the sum alone
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  if (blockDim.x > 32) {
    // One partial per warp; every warp adds them in the same order.
    if (lane == 0) partial[threadIdx.x >> 5] = ss;
    __syncthreads();
    ss = lane < static_cast<int>(blockDim.x >> 5) ? partial[lane] : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  }
  const float inv = rsqrtf(fmaf(ss, a.inv_cols, a.eps));  // rsqrtf: within 2 units
#pragma unroll
  for (int i = 0; i < kOcts; ++i) {
#pragma unroll
    for (int k = 0; k < 8; ++k) h[i][k] = __fmul_rn(h[i][k], inv);
    if (a.weight) {
      float w[8];
      if (kVec && a.w_bf16)
        unpack(wr[i], w);
      else if (a.w_bf16)
        unpack(load_oct<kVec, true>(static_cast<const uint16_t*>(a.weight), col_place[i], cols), w);
      else
        unpack(load_oct<kVec, true>(static_cast<const float*>(a.weight), col_place[i], cols), w);
#pragma unroll
      for (int k = 0; k < 8; ++k) h[i][k] = __fmul_rn(h[i][k], w[k]);
    }
    if (a.y) store_oct<kVec>(a.y, place(a.ldy, i), cols, h[i]);
    if (a.q) {
      BlockScale b0, b1;
      lane_scales<kVec>(h[i], b0, b1);
      const Place p = place(a.ldq, i);
      store_q<kVec>(a.q, p, cols, quant_oct(h[i], b0, b1));
      if ((lane & 15) == 0) {
        // kVec: lanes 0 and 16 hold the two blocks' scales; else both do
        const int col = kVec ? p.col0 : p.col0 - lane + 8 * lane;
        if (col < cols) a.scale[row * a.blocks + (col >> 7)] = kVec || lane == 0 ? b0.s : b1.s;
      }
    }
  }
}

template <bool kXBf16, int kRes, int kOcts>
cudaError_t launch_norm_octs(const RmsNormArgs& a, bool vec, dim3 grid, dim3 block, cudaStream_t st) {
  if (vec)
    return launch_chained(rms_norm_kernel<kXBf16, kRes, kOcts, true>, grid, block, 0, 1, st, a);
  else
    return launch_chained(rms_norm_kernel<kXBf16, kRes, kOcts, false>, grid, block, 0, 1, st, a);
}

template <bool kXBf16, int kRes>
cudaError_t launch_norm(RmsNormArgs a, bool vec, cudaStream_t st) {
  a.inv_cols = 1.0f / static_cast<float>(a.cols);
  const int octs = (a.cols + 7) / 8;
  if (octs <= 128) {  // up to 1024 columns: a warp per row, no shared memory
    const dim3 block(32, a.rows >= 8 ? 8 : static_cast<unsigned>(a.rows));
    const dim3 grid(static_cast<unsigned>((a.rows + block.y - 1) / block.y));
    if (octs <= 32) return launch_norm_octs<kXBf16, kRes, 1>(a, vec, grid, block, st);
    if (octs <= 64) return launch_norm_octs<kXBf16, kRes, 2>(a, vec, grid, block, st);
    return launch_norm_octs<kXBf16, kRes, 4>(a, vec, grid, block, st);
  }
  // A CTA per row.  Octs a thread, with both sides timed in us (bf16 residual and e4m3 out; fp32 residual
  // and bf16 out):
  //   up to 4096 columns, more rows than two CTAs on every SM: two.  8000 x 4096: 41 with two, 44 with one (64, 59);
  //     8000 x 2048: 20.3, 20.5 (34, 31).  Of fewer rows each wants its latency short: one.
  //   up to 8192 columns: one.  8000 x 5120: 56 with one, 53 with two (73, 79); 1000 x 8192: 11.9, 12.6 (14.6, 18.2).
  //   up to what two CTAs of two octs hold: two.  5000 x 12288: 81.5 with two, 86 with four (119, 119).
  //   above: four.  (A pair of CTAs per row, to have two rows an SM there too, was no faster: 2000 x 29568 103 us for 95.)
  DeviceInfo d;
  const cudaError_t e = device_info(&d);
  if (e != cudaSuccess) return e;
  const dim3 grid(static_cast<unsigned>(a.rows));
  const int per = octs <= 1024 ? (octs <= 512 && a.rows > 2 * d.sms ? 2 : 1) : octs <= 2 * kTwoOctThreads ? 2 : 4;
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

// Units in flight per half warp.  Unaligned rows are loaded element by element, eight loads a
// step: one step, and as many warps as fit, keep more of them in flight than four.
template <bool kVec>
constexpr int kUnitsOf = kVec ? 4 : 1;

// silu(f) = f / (1 + exp(-f)), from the hardware's exponential and reciprocal, as (f / 128) times
// 1 / (1/128 + exp(-f) / 128): so the reciprocal is a normal number wherever silu is one (down to
// f = -91.9; of the plain sum it is subnormal from -87.3 on, and the approximation gives 0 for
// those).  f / 128 is exact for every bf16.  Relative error below 2^-20 + |f| 2^-23: the argument
// f log2(e) - 7 is rounded once, ex2 and rcp are within 2 units.  With the library's expf and
// division the kernel was bound by its instructions: 33 per element, 217 us for 16384 x 11008
// where the memory takes 139; so it takes 182 (180 with the plain sum).  exp(-f) = inf gives f * 0 = -0, the limit.
__device__ __forceinline__ float silu(float f) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(__fmaf_rn(f, -1.44269504088896341f, -7.0f)));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(__fadd_rn(0x1p-7f, e)));
  return __fmul_rn(__fmul_rn(f, 0x1p-7f), r);
}

template <bool kXBf16, bool kGated, bool kVec>
__global__ void __launch_bounds__(256, kVec ? 4 : 1) row_quant_kernel(RowQuantArgs a) {
  using XT = typename OctOf<kXBf16, kVec>::type;
  constexpr int kUnits = kUnitsOf<kVec>;
  chain_next();
  chain_wait();
  // Unit u is block u % blocks of row u / blocks.  A warp takes 2 kUnits consecutive units;
  // step i of its lanes: kVec, unit first + i of its half; else units first + 2 i and + 2 i + 1.
  const int64_t warp = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  const int64_t units = a.rows * a.blocks;
  const int64_t warp_first = warp * (2 * kUnits);
  if (warp_first >= units) return;
  const int64_t first = warp_first + (kVec ? (lane >> 4) * kUnits : 0);
  int64_t row;
  if (units < (1ll << 31))
    row = static_cast<uint32_t>(first) / static_cast<uint32_t>(a.blocks);
  else
    row = first / a.blocks;
  int blk = static_cast<int>(first - row * a.blocks);
  auto next = [&](int64_t& r, int& b) {
    if (++b == a.blocks) {
      b = 0;
      ++r;
    }
  };
  XT xr[kUnits];
  typename OctOf<true, kVec>::type gr[kUnits];
  int64_t rows0[kUnits], rows1[kUnits];
  int cols0[kUnits], cols1[kUnits];
  const int off = kVec ? (lane & 15) * 8 : lane;
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    // past the end: a column that no load or store takes
    const int64_t u = first + (kVec ? i : 2 * i);
    rows0[i] = row;
    cols0[i] = u < units ? blk * 128 + off : a.cols;
    next(row, blk);
    if (!kVec) {
      rows1[i] = row;
      cols1[i] = u + 1 < units ? blk * 128 + off : a.cols;
      next(row, blk);
    } else {
      rows1[i] = rows0[i];
      cols1[i] = cols0[i];
    }
    const Place px = {rows0[i] * a.ldx, rows1[i] * a.ldx, cols0[i], cols1[i]};
    if constexpr (kXBf16)
      xr[i] = load_oct<kVec>(static_cast<const uint16_t*>(a.x), px, a.cols);
    else
      xr[i] = load_oct<kVec>(static_cast<const float*>(a.x), px, a.cols);
    if constexpr (kGated) {
      const Place pg = {rows0[i] * a.ldg, rows1[i] * a.ldg, cols0[i], cols1[i]};
      gr[i] = load_oct<kVec>(a.gate, pg, a.cols);
    }
  }
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    float f[8];
    unpack(xr[i], f);
    if constexpr (kGated) {
      float g[8];
      unpack(gr[i], g);
#pragma unroll
      for (int k = 0; k < 8; ++k) f[k] = __fmul_rn(silu(f[k]), g[k]);
    }
    BlockScale b0, b1;
    lane_scales<kVec>(f, b0, b1);
    const Place pq = {rows0[i] * a.ldq, rows1[i] * a.ldq, cols0[i], cols1[i]};
    store_q<kVec>(a.q, pq, a.cols, quant_oct(f, b0, b1));
    if (kVec) {
      if ((lane & 15) == 0 && cols0[i] < a.cols) a.scale[first + i] = b0.s;
    } else if ((lane & 15) == 0) {
      const int64_t u = first + 2 * i + (lane >> 4);
      if (u < units) a.scale[u] = lane == 0 ? b0.s : b1.s;
    }
  }
}

// ---------------------------------------------------------------------------
// Weight quantiser: a CTA per 128 x 128 tile.  Thread t owns the oct t % 16 of the
// rows t / 16 + 32 i, i < 4, in registers between the tile's maximum and the store.
// (fp32 input, and unaligned rows; two CTAs an SM leave 64 registers, of which 24 to 104 bytes spill.)
// ---------------------------------------------------------------------------

template <bool kXBf16, bool kVec>
__global__ void __launch_bounds__(512, 2) tile_quant_kernel(TileQuantArgs a) {
  using XT = typename OctOf<kXBf16, kVec>::type;
  __shared__ float partial[16];
  chain_next();
  chain_wait();
  const int64_t tile = blockIdx.x;
  const int64_t per_mat = static_cast<int64_t>(a.row_blocks) * a.blocks;
  const int64_t mat = tile / per_mat;
  const int rb = static_cast<int>((tile - mat * per_mat) / a.blocks);
  const int cb = static_cast<int>(tile - mat * per_mat - static_cast<int64_t>(rb) * a.blocks);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // kVec: oct t % 16 of row t / 16 + 32 i; else rows 2 warp and 2 warp + 1 (+ 32 i), strided columns
  auto place = [&](int64_t ld, int i) {
    const int64_t r0 = static_cast<int64_t>(rb) * 128 + 32 * i + (kVec ? static_cast<int>(threadIdx.x >> 4) : 2 * warp);
    const int col = cb * 128 + (kVec ? static_cast<int>(threadIdx.x & 15) * 8 : lane);
    Place p;  // a row past the end: a column that no load or store takes
    p.row0 = (mat * a.rows + r0) * ld;
    p.row1 = p.row0 + ld;
    p.col0 = r0 < a.rows ? col : a.cols;
    p.col1 = r0 + 1 < a.rows ? col : a.cols;
    return p;
  };
  XT xr[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (kXBf16)
      xr[i] = load_oct<kVec>(static_cast<const uint16_t*>(a.x), place(a.ldx, i), a.cols);
    else
      xr[i] = load_oct<kVec>(static_cast<const float*>(a.x), place(a.ldx, i), a.cols);
  }
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float f[8];
    unpack(xr[i], f);
#pragma unroll
    for (int k = 0; k < 8; ++k) m = fmaxf(m, fabsf(f[k]));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (lane == 0) partial[warp] = m;
  __syncthreads();
  m = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) m = fmaxf(m, partial[i]);
  const BlockScale b = block_scale(m);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float f[8];
    unpack(xr[i], f);
    store_q<kVec>(a.q, place(a.ldq, i), a.cols, quant_oct(f, b, b));
  }
  if (threadIdx.x == 0) a.scale[tile] = b.s;
}

// The same for aligned bf16 rows, the tile in shared memory: a thread copies its eight octs
// there asynchronously and reads them back twice, so the tile in flight takes no registers
// and six CTAs share an SM.  (Each thread reads only what it copied.)
__global__ void __launch_bounds__(256, 6) tile_quant_async_kernel(TileQuantArgs a) {
  __shared__ uint4 buf[8 * 256];
  __shared__ float partial[8];
  chain_next();
  chain_wait();
  const int64_t tile = blockIdx.x;
  const int64_t per_mat = static_cast<int64_t>(a.row_blocks) * a.blocks;
  const int64_t mat = tile / per_mat;
  const int rb = static_cast<int>((tile - mat * per_mat) / a.blocks);
  const int cb = static_cast<int>(tile - mat * per_mat - static_cast<int64_t>(rb) * a.blocks);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t r0 = static_cast<int64_t>(rb) * 128 + (threadIdx.x >> 4);
  const int col = cb * 128 + (threadIdx.x & 15) * 8;
  const bool col_ok = col < a.cols;
  const uint16_t* x = static_cast<const uint16_t*>(a.x) + (mat * a.rows + r0) * a.ldx + col;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const bool ok = col_ok && r0 + 16 * i < a.rows;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(&buf[i * 256 + threadIdx.x])),
                 "l"(ok ? x + 16 * i * a.ldx : static_cast<const uint16_t*>(a.x)), "r"(ok ? 16 : 0)
                 : "memory");
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float f[8];
    unpack(Bf16Oct{buf[i * 256 + threadIdx.x]}, f);
#pragma unroll
    for (int k = 0; k < 8; ++k) m = fmaxf(m, fabsf(f[k]));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (lane == 0) partial[warp] = m;
  __syncthreads();
  m = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, partial[i]);
  const BlockScale b = block_scale(m);
  uint8_t* q = a.q + (mat * a.rows + r0) * a.ldq + col;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float f[8];
    unpack(Bf16Oct{buf[i * 256 + threadIdx.x]}, f);
    const uint2 v = quant_oct(f, b, b);
    if (col_ok && r0 + 16 * i < a.rows) *reinterpret_cast<uint2*>(q + 16 * i * a.ldq) = v;
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
  const int per_warp = 2 * (vec ? kUnitsOf<true> : kUnitsOf<false>);
  const int64_t warps = (a.rows * a.blocks + per_warp - 1) / per_warp;
  const unsigned grid = static_cast<unsigned>((warps + 7) / 8);
  const dim3 block(256);
  if (a.gate) {
    if (vec) return launch_chained(row_quant_kernel<true, true, true>, grid, block, 0, 1, st, a);
    return launch_chained(row_quant_kernel<true, true, false>, grid, block, 0, 1, st, a);
  }
  if (a.x_bf16) {
    if (vec) return launch_chained(row_quant_kernel<true, false, true>, grid, block, 0, 1, st, a);
    return launch_chained(row_quant_kernel<true, false, false>, grid, block, 0, 1, st, a);
  }
  if (vec) return launch_chained(row_quant_kernel<false, false, true>, grid, block, 0, 1, st, a);
  return launch_chained(row_quant_kernel<false, false, false>, grid, block, 0, 1, st, a);
}

cudaError_t launch_tile_quant(const TileQuantArgs& a, cudaStream_t st) {
  const bool vec = a.cols % 8 == 0 && aligned_to(a.x, 16) && a.ldx % (a.x_bf16 ? 8 : 4) == 0 && aligned_to(a.q, 8) &&
                   a.ldq % 8 == 0;
  const unsigned grid = static_cast<unsigned>(a.count * a.row_blocks * a.blocks);
  if (a.x_bf16) {
    if (vec) return launch_chained(tile_quant_async_kernel, grid, dim3(256), 0, 1, st, a);
    return launch_chained(tile_quant_kernel<true, false>, grid, dim3(512), 0, 1, st, a);
  }
  if (vec) return launch_chained(tile_quant_kernel<false, true>, grid, dim3(512), 0, 1, st, a);
  return launch_chained(tile_quant_kernel<false, false>, grid, dim3(512), 0, 1, st, a);
}

}  // namespace ar
