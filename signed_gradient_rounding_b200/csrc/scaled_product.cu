// Products of the 8-bit chain: Y = X W^T with e4m3 operands and one fp32 scale per
// block of 128 along K (per row of X, per 128 rows of W), and with bf16 operands,
// dense or with the rows of X grouped by expert.
//
//   Y[n, o] = sum_kb xs[n, kb] ws[o / 128, kb] sum_{k in kb} X[n, k] W[o, k]  (+ add)
//
// The inner sum (128 products of e4m3 values) is one tensor-core accumulation in
// fp32; the outer one runs in fp32 registers, one fma per block, and the result is
// rounded once, to bf16.  (The scales are arbitrary fp32 numbers, so the tensor
// cores' own block scaling, which takes powers of two, does not apply.)
//
// Two kernels:
//   * tile_kernel: tcgen05 tiles, TMA-fed, accumulators in tensor memory; rows of X
//     are the tile's M side.  A K block of 128 bytes is one row of the 128-byte
//     swizzle, so both operand types share one pipeline.
//   * skinny_kernel: few rows per expert, bound by the weight's bytes; each weight
//     byte goes from HBM straight into the registers of the warp that multiplies it.
#include <atomic>

#include "ar_device.cuh"
#include "ar_internal.h"
#include "ar_scaled.h"

namespace ar {

namespace {

// Rows [r0, r1) of X that belong to expert e, clamped to the tensor: whatever the
// offsets hold, no access leaves it.
__device__ __forceinline__ void expert_rows(const ProductArgs& a, int e, int& r0, int& r1) {
  if (!a.offsets) {
    r0 = 0;
    r1 = a.n;
    return;
  }
  r0 = min(max(__ldg(a.offsets + e), 0), a.n);
  r1 = min(max(__ldg(a.offsets + e + 1), r0), a.n);
}

// ---------------------------------------------------------------------------
// Tile kernel
// ---------------------------------------------------------------------------

constexpr int kTileWarps = 10;  // producer, MMA issuer, 8 epilogue warps
constexpr int kTileThreads = 32 * kTileWarps;
constexpr int kMaxStages = 8;
constexpr int kRowTile = 128;     // rows per CTA: tensor-memory lanes
constexpr int kRasterM = 8;       // row blocks that share a sweep over the weight's columns
constexpr int kKBytes = 128;      // bytes of K per stage and row

struct TileSmem {
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t tfull[2], tempty[2];
  uint64_t drain;
  uint32_t tmem_base;
  int abort_flag;
  int cum[kMaxExperts + 1];  // row blocks of the experts before e
};

template <bool kPair, int kBN>
struct TileCfg {
  static constexpr int kBRows = kPair ? kBN / 2 : kBN;  // weight rows this CTA stages
  static constexpr int kABytes = kRowTile * kKBytes;
  static constexpr int kStageBytes = kABytes + kBRows * kKBytes;
  static constexpr int kStages = kStageBytes <= 32768 ? 6 : 4;
  static constexpr int kBM = kPair ? 2 * kRowTile : kRowTile;  // rows per unit (CTA or pair)
  static constexpr int kTmemCols = 2 * kBN;                    // two accumulators
  static constexpr int kBarOffset = kStages * kStageBytes;
  static constexpr int kSmemBytes = 1024 + kBarOffset + static_cast<int>(sizeof(TileSmem));
  static_assert(kSmemBytes <= 232448, "shared memory per CTA");
  static_assert(kTmemCols <= 512, "tensor memory");
};

struct Unit {
  int e;       // expert
  int m0, r1;  // first row of X of the unit, end of the expert's rows
  int n0;      // first column of Y
};

// Unit t in order: experts in turn; inside an expert groups of kRasterM row blocks,
// each sweeping the weight's column blocks with the row blocks innermost (the
// group's rows of X stay in L2 while the weight passes by).
__device__ __forceinline__ Unit find_unit(const ProductArgs& a, const int* cum, int64_t t, int num_n, int bm, int bn) {
  Unit u;
  const int mb = static_cast<int>(t / num_n);
  int e = 0;
  if (a.offsets) {
    int lo = 0, hi = a.experts;  // the last e with cum[e] <= mb
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (cum[mid] <= mb)
        lo = mid;
      else
        hi = mid;
    }
    e = lo;
  }
  int r0;
  expert_rows(a, e, r0, u.r1);
  const int64_t r = t - static_cast<int64_t>(cum[e]) * num_n;
  const int num_m = cum[e + 1] - cum[e];
  const int64_t per = static_cast<int64_t>(kRasterM) * num_n;
  const int grp = static_cast<int>(r / per);
  const int in_grp = static_cast<int>(r - grp * per);
  const int gm = min(kRasterM, num_m - grp * kRasterM);
  const int n_blk = in_grp / gm;
  u.e = e;
  u.m0 = r0 + (grp * kRasterM + in_grp - n_blk * gm) * bm;
  u.n0 = n_blk * bn;
  return u;
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Columns [col, col + 8) of row `row` of Y: + add, one rounding to bf16.
__device__ __forceinline__ void store8(const ProductArgs& a, int64_t row, int col, float (&x)[8]) {
  if (col >= a.out) return;
  uint16_t* y = a.Y + row * a.ldy + col;
  const uint16_t* add = a.add ? a.add + row * a.ldadd + col : nullptr;
  if (a.vec_y && col + 8 <= a.out) {
    if (add) {
      const uint4 v = *reinterpret_cast<const uint4*>(add);
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[2 * i] += __uint_as_float(w[i] << 16);
        x[2 * i + 1] += __uint_as_float(w[i] & 0xFFFF0000u);
      }
    }
    *reinterpret_cast<uint4*>(y) =
        make_uint4(pack2(x[0], x[1]), pack2(x[2], x[3]), pack2(x[4], x[5]), pack2(x[6], x[7]));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (col + i >= a.out) break;
      const float v = add ? x[i] + bf16_bits_to_f32(add[i]) : x[i];
      y[i] = static_cast<uint16_t>(pack2(v, 0.f) & 0xFFFFu);
    }
  }
}

// acc += s * v, two columns at a time.
__device__ __forceinline__ void fma2(uint64_t& acc, uint32_t v0, uint32_t v1, uint64_t s2) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "r"(v0), "r"(v1));
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(acc) : "l"(v), "l"(s2));
}

__device__ __forceinline__ void unpack2(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}

// e4m3 operands, fp32 accumulation (format fields 0 = e4m3), issued by one thread.
__device__ __forceinline__ void umma_f8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                        uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void umma_f8_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                             uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

__host__ __device__ constexpr uint32_t umma_idesc_f8(int M, int N) {
  return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);  // f32 D, e4m3 A and B
}

template <bool kF8, bool kPair, int kBN>
__global__ void __launch_bounds__(kTileThreads, 1)
    tile_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW,
                const __grid_constant__ CUtensorMap tmWlo, const __grid_constant__ ProductArgs args) {
  using C = TileCfg<kPair, kBN>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  TileSmem* sm = reinterpret_cast<TileSmem*>(smem + C::kBarOffset);
  volatile int* abort_flag = &sm->abort_flag;
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = kPair ? cluster_ctarank() : 0u;

  if (warp == 1 && lane == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&sm->full[s], 1);
      mbar_init(&sm->empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&sm->tfull[b], 1);
      mbar_init(&sm->tempty[b], (kPair ? 2 : 1) * 8);  // one arrive per epilogue warp
    }
    mbar_init(&sm->drain, 1);
    sm->abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0) {
    if (kPair) {
      tmem_alloc_pair(&sm->tmem_base, C::kTmemCols);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(&sm->tmem_base, C::kTmemCols);
      tmem_relinquish();
    }
    if (lane == 0) {
      tma_prefetch_desc(&tmX);
      tma_prefetch_desc(&tmW);
      if (args.W_lo) tma_prefetch_desc(&tmWlo);
    }
  }
  if (warp == 2) {
    // Row blocks before each expert.  Capped at what monotone offsets can give, so
    // that no offsets overflow the count.
    if (!args.offsets) {
      if (lane == 0) {
        sm->cum[0] = 0;
        sm->cum[1] = (args.n + C::kBM - 1) / C::kBM;
      }
    } else {
      const int limit = args.n / C::kBM + args.experts;
      int carry = 0;
      if (lane == 0) sm->cum[0] = 0;
      for (int e0 = 0; e0 < args.experts; e0 += 32) {
        int r0 = 0, r1 = 0;
        if (e0 + lane < args.experts) expert_rows(args, e0 + lane, r0, r1);
        int v = (r1 - r0 + C::kBM - 1) / C::kBM;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int up = __shfl_up_sync(0xffffffffu, v, o);
          if (lane >= o) v += up;
        }
        v = min(carry + v, limit);
        if (e0 + lane < args.experts) sm->cum[e0 + lane + 1] = v;
        carry = __shfl_sync(0xffffffffu, v, 31);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (kPair) cluster_sync_all();  // the peer's barriers are initialised before any remote arrive
  tc_fence_after();
  const uint32_t tmem_base = sm->tmem_base;
  const int num_n = (args.out + kBN - 1) / kBN;
  const int64_t num_units = static_cast<int64_t>(sm->cum[args.experts]) * num_n;
  const int64_t unit0 = kPair ? blockIdx.x >> 1 : blockIdx.x;
  const int64_t stride = kPair ? gridDim.x >> 1 : gridDim.x;
  const int nkb = args.nkb;
  const int k_total = (!kF8 && args.W_lo) ? 2 * nkb : nkb;
  // e4m3: the accumulator is handed over after every K block; bf16: after the last.
  const int k_chunk = kF8 ? 1 : k_total;

  if (warp == 0) {
    if (lane == 0) {
      // ------------------------------------------------------------ producer
      int stage = 0;
      uint32_t phase = 0, issued_mask = 0, issued_parity = 0;
      bool ok = true;
      for (int64_t t = unit0; ok && t < num_units; t += stride) {
        const Unit u = find_unit(args, sm->cum, t, num_n, C::kBM, kBN);
        const int x_row = u.m0 + static_cast<int>(rank) * kRowTile;
        const int w_row = u.e * args.out + u.n0 + static_cast<int>(rank) * C::kBRows;
        for (int kb = 0; kb < k_total; ++kb) {
          if (!mbar_wait<kPair>(&sm->empty[stage], phase ^ 1, abort_flag, args.status, args.timeout_ns)) {
            ok = false;
            break;
          }
          uint8_t* sx = smem + stage * C::kStageBytes;
          uint8_t* sw = sx + C::kABytes;
          const bool lo = !kF8 && kb >= nkb;
          const int k = (lo ? kb - nkb : kb) * kKBytes;  // bytes: the maps are byte maps
          const CUtensorMap* mw = lo ? &tmWlo : &tmW;
          if (kPair) {
            if (rank == 0) mbar_arrive_expect_tx(&sm->full[stage], 2 * C::kStageBytes);
            const uint32_t leader = mapa_shared(smem_u32(&sm->full[stage]), 0);
            tma_load_2d_pair(sx, &tmX, k, x_row, leader);
            tma_load_2d_pair(sw, mw, k, w_row, leader);
          } else {
            mbar_arrive_expect_tx(&sm->full[stage], C::kStageBytes);
            tma_load_2d(sx, &tmX, k, x_row, &sm->full[stage]);
            tma_load_2d(sw, mw, k, w_row, &sm->full[stage]);
          }
          issued_mask |= 1u << stage;
          issued_parity = (issued_parity & ~(1u << stage)) | (phase << stage);
          if (++stage == C::kStages) {
            stage = 0;
            phase ^= 1;
          }
        }
      }
      if (!ok) {
        if (kPair) {
          // The copies' completion is counted on the leader's barriers, which this
          // CTA cannot wait on: give anything in flight time to land.
          const uint64_t t0 = globaltimer_ns();
          while (globaltimer_ns() - t0 < 10000000ull) {
          }
        } else {
          for (int s = 0; s < C::kStages; ++s)
            if (issued_mask & (1u << s)) mbar_wait_drain(&sm->full[s], (issued_parity >> s) & 1u, args.timeout_ns);
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) {
      // ------------------------------------------------------------ MMA issuer
      constexpr int kM = kPair ? 2 * kRowTile : kRowTile;
      constexpr uint32_t idesc = kF8 ? umma_idesc_f8(kM, kBN) : umma_idesc_bf16(kM, kBN);
      int stage = 0, acc = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool ok = true;
      for (int64_t t = unit0; ok && t < num_units; t += stride) {
        for (int kb0 = 0; ok && kb0 < k_total; kb0 += k_chunk) {
          if (!mbar_wait<kPair>(&sm->tempty[acc], acc_phase ^ 1, abort_flag, args.status, args.timeout_ns)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t d_tmem = tmem_base + acc * kBN;
          for (int kb = kb0; kb < kb0 + k_chunk; ++kb) {
            if (!mbar_wait<kPair>(&sm->full[stage], phase, abort_flag, args.status, args.timeout_ns)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint32_t addr = smem_u32(smem + stage * C::kStageBytes);
            const uint64_t a_desc = umma_desc_sw128(addr), b_desc = umma_desc_sw128(addr + C::kABytes);
#pragma unroll
            for (int k = 0; k < 4; ++k) {  // 32 bytes of K each: 2 descriptor units
              const uint32_t accum = ((kb - kb0) | k) != 0 ? 1u : 0u;
              if (kF8 && kPair)
                umma_f8_pair(d_tmem, a_desc + 2 * k, b_desc + 2 * k, idesc, accum);
              else if (kF8)
                umma_f8(d_tmem, a_desc + 2 * k, b_desc + 2 * k, idesc, accum);
              else if (kPair)
                umma_bf16_pair(d_tmem, a_desc + 2 * k, b_desc + 2 * k, idesc, accum);
              else
                umma_bf16(d_tmem, a_desc + 2 * k, b_desc + 2 * k, idesc, accum);
            }
            if (kPair)
              umma_commit_pair_both(&sm->empty[stage]);
            else
              umma_commit(&sm->empty[stage]);
            if (++stage == C::kStages) {
              stage = 0;
              phase ^= 1;
            }
          }
          if (!ok) break;
          if (kPair)
            umma_commit_pair_both(&sm->tfull[acc]);
          else
            umma_commit(&sm->tfull[acc]);
          acc ^= 1;
          if (acc == 0) acc_phase ^= 1;
        }
      }
      // Every MMA this thread issued has completed once `drain` flips.
      if (kPair)
        umma_commit_pair_local(&sm->drain);
      else
        umma_commit(&sm->drain);
      mbar_wait_drain(&sm->drain, 0, args.timeout_ns);
    }
  } else {
    // -------------------------------------------------------------- epilogue
    constexpr int kNC = kBN / 2;       // columns per thread
    const int quarter = warp & 3;      // tensor-memory lanes this warp may access
    const int half = (warp - 2) >> 2;  // column half of the tile
    const uint32_t t_lane = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + half * kNC;
    const uint32_t leader_tempty0 = kPair ? mapa_shared(smem_u32(&sm->tempty[0]), 0) : 0u;
    const uint32_t leader_tempty1 = kPair ? mapa_shared(smem_u32(&sm->tempty[1]), 0) : 0u;
    auto release = [&](int buf) {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (kPair)
          mbar_arrive_cluster(buf ? leader_tempty1 : leader_tempty0);
        else
          mbar_arrive(&sm->tempty[buf]);
      }
    };
    int acc_buf = 0;
    uint32_t acc_phase = 0;
    bool ok = true;
    for (int64_t t = unit0; ok && t < num_units; t += stride) {
      const Unit u = find_unit(args, sm->cum, t, num_n, C::kBM, kBN);
      const int row = u.m0 + static_cast<int>(rank) * kRowTile + quarter * 32 + lane;
      const bool row_ok = row < u.r1;
      const int col0 = u.n0 + half * kNC;
      if constexpr (kF8) {
        uint64_t acc[kNC / 2];
#pragma unroll
        for (int i = 0; i < kNC / 2; ++i) acc[i] = 0ull;
        // Row and weight scales of four K blocks at a time, loaded one group ahead.
        const float* xs = args.xs + static_cast<int64_t>(row_ok ? row : u.r1 - 1) * nkb;
        const float* ws =
            args.ws + (static_cast<int64_t>(u.e) * args.out_blocks + min(col0 >> 7, args.out_blocks - 1)) * nkb;
        float xn[4], wn[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          xn[i] = __ldg(xs + min(i, nkb - 1));
          wn[i] = __ldg(ws + min(i, nkb - 1));
        }
        for (int kb0 = 0; ok && kb0 < nkb; kb0 += 4) {
          float s[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            s[i] = __fmul_rn(xn[i], wn[i]);
            xn[i] = __ldg(xs + min(kb0 + 4 + i, nkb - 1));
            wn[i] = __ldg(ws + min(kb0 + 4 + i, nkb - 1));
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (kb0 + i >= nkb) break;
            if (!mbar_wait<kPair>(&sm->tfull[acc_buf], acc_phase, abort_flag, args.status, args.timeout_ns, false)) {
              ok = false;
              break;
            }
            tc_fence_after();
            uint64_t s2;
            asm("mov.b64 %0, {%1, %1};" : "=l"(s2) : "f"(s[i]));
#pragma unroll
            for (int g = 0; g < kNC / 32; ++g) {
              uint32_t r[32];
              tmem_ld_32cols(t_lane + acc_buf * kBN + g * 32, r);
              tmem_ld_wait();
              if (g == kNC / 32 - 1) release(acc_buf);
#pragma unroll
              for (int j = 0; j < 16; ++j) fma2(acc[g * 16 + j], r[2 * j], r[2 * j + 1], s2);
            }
            acc_buf ^= 1;
            if (acc_buf == 0) acc_phase ^= 1;
          }
        }
        if (!ok) break;
        if (row_ok) {
#pragma unroll
          for (int c = 0; c < kNC / 8; ++c) {
            float x[8];
#pragma unroll
            for (int j = 0; j < 4; ++j) unpack2(acc[c * 4 + j], x[2 * j], x[2 * j + 1]);
            store8(args, row, col0 + c * 8, x);
          }
        }
      } else {
        if (!mbar_wait<kPair>(&sm->tfull[acc_buf], acc_phase, abort_flag, args.status, args.timeout_ns, false)) break;
        tc_fence_after();
#pragma unroll 1
        for (int g = 0; g < kNC / 32; ++g) {
          uint32_t r[32];
          __syncwarp();
          tmem_ld_32cols(t_lane + acc_buf * kBN + g * 32, r);
          tmem_ld_wait();
          if (g == kNC / 32 - 1) release(acc_buf);
          if (!row_ok) continue;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            float x[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = __uint_as_float(r[c * 8 + j]);
            store8(args, row, col0 + g * 32 + c * 8, x);
          }
        }
        acc_buf ^= 1;
        if (acc_buf == 0) acc_phase ^= 1;
      }
    }
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (kPair) cluster_sync_all();  // the leader's MMAs into this CTA's tensor memory are done
  tc_fence_after();
  if (warp == 0) {
    if (kPair)
      tmem_dealloc_pair(tmem_base, C::kTmemCols);
    else
      tmem_dealloc(tmem_base, C::kTmemCols);
  }
}

// ---------------------------------------------------------------------------
// Skinny kernel: 16 rows of W per CTA, the K blocks dealt to its 8 warps.
//
// A K block (128 bytes) of a warp is two 64-byte pieces; lane (g, q) holds bytes
// 16 q .. 16 q + 15 of each piece for weight rows g and g + 8 and for row g of each
// 8-row tile of X.  The m16n8 instructions take, from lane (g, q), two 4-byte
// registers per operand row; which columns of K they stand for does not matter as
// long as W and X agree, so the four registers of a 16-byte load feed two
// instructions as they are.
// ---------------------------------------------------------------------------

template <bool kF8>
__device__ __forceinline__ void mma_16x8(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  if (kF8)
    asm("mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

constexpr int kSkinnyWarps = 8;
constexpr int kSkinnyRows = 16;

template <bool kF8, int kNT>  // kNT tiles of 8 rows of X per pass
__global__ void __launch_bounds__(32 * kSkinnyWarps) skinny_kernel(const __grid_constant__ ProductArgs a) {
  constexpr int kU = 2;           // K blocks in flight per warp
  constexpr int kTok = 8 * kNT;
  __shared__ float red[kSkinnyWarps][kTok][kSkinnyRows + 1];
  const int e = blockIdx.y;
  int r0, r1;
  expert_rows(a, e, r0, r1);
  if (r0 >= r1) return;
  const int o0 = blockIdx.x * kSkinnyRows;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, q = lane & 3;
  const int in_bytes = a.in * (kF8 ? 1 : 2);  // a multiple of 16
  const bool w_ok[2] = {o0 + g < a.out, o0 + g + 8 < a.out};
  const int64_t w_off = (static_cast<int64_t>(e) * a.out + o0 + g) * a.ldw + q * 16;
  const float* ws = kF8 ? a.ws + (static_cast<int64_t>(e) * a.out_blocks + (o0 >> 7)) * a.nkb : nullptr;
  const int segs = (!kF8 && a.W_lo) ? 2 : 1;

  for (int t0 = r0; t0 < r1; t0 += kTok) {
    float acc[kNT][4];
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[nt][i] = 0.f;
    for (int seg = 0; seg < segs; ++seg) {
      const uint8_t* wp = static_cast<const uint8_t*>(seg ? a.W_lo : a.W) + w_off;
      for (int kb0 = warp; kb0 < a.nkb; kb0 += kU * kSkinnyWarps) {
        uint4 w[kU][2][2], x[kU][2][kNT];
        float sx[kU][kNT][2], sw[kU];
#pragma unroll
        for (int j = 0; j < kU; ++j) {
          const int kb = kb0 + j * kSkinnyWarps;
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int k = kb * kKBytes + c * 64;
            const bool k_ok = k + q * 16 < in_bytes;  // also false for kb past the end
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              w[j][c][h] = make_uint4(0, 0, 0, 0);
              if (k_ok && w_ok[h]) {
                const uint8_t* p = wp + h * 8 * a.ldw + k;
                asm("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                    : "=r"(w[j][c][h].x), "=r"(w[j][c][h].y), "=r"(w[j][c][h].z), "=r"(w[j][c][h].w)
                    : "l"(p));
              }
            }
#pragma unroll
            for (int nt = 0; nt < kNT; ++nt) {
              x[j][c][nt] = make_uint4(0, 0, 0, 0);
              const int row = t0 + nt * 8 + g;
              if (k_ok && row < r1)
                x[j][c][nt] = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(a.X) +
                                                                   static_cast<int64_t>(row) * a.ldx + q * 16 + k));
            }
          }
          if (kF8) {
            const bool kb_ok = kb < a.nkb;
            sw[j] = kb_ok ? __ldg(ws + kb) : 0.f;
#pragma unroll
            for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const int row = t0 + nt * 8 + q * 2 + h;
                sx[j][nt][h] = kb_ok && row < r1 ? __ldg(a.xs + static_cast<int64_t>(row) * a.nkb + kb) : 0.f;
              }
          }
        }
#pragma unroll
        for (int j = 0; j < kU; ++j) {
#pragma unroll
          for (int nt = 0; nt < kNT; ++nt) {
            float part[4] = {0.f, 0.f, 0.f, 0.f};
            float(&c4)[4] = kF8 ? part : acc[nt];
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const uint4 lo = w[j][c][0], hi = w[j][c][1], xx = x[j][c][nt];
              mma_16x8<kF8>(c4, lo.x, hi.x, lo.y, hi.y, xx.x, xx.y);
              mma_16x8<kF8>(c4, lo.z, hi.z, lo.w, hi.w, xx.z, xx.w);
            }
            if (kF8 && kb0 + j * kSkinnyWarps < a.nkb) {
              const float s0 = __fmul_rn(sx[j][nt][0], sw[j]), s1 = __fmul_rn(sx[j][nt][1], sw[j]);
              acc[nt][0] = fmaf(part[0], s0, acc[nt][0]);
              acc[nt][1] = fmaf(part[1], s1, acc[nt][1]);
              acc[nt][2] = fmaf(part[2], s0, acc[nt][2]);
              acc[nt][3] = fmaf(part[3], s1, acc[nt][3]);
            }
          }
        }
      }
    }
    // c0, c1: weight row g, rows 2q and 2q + 1 of X; c2, c3: weight row g + 8.
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt) {
      red[warp][nt * 8 + q * 2][g] = acc[nt][0];
      red[warp][nt * 8 + q * 2 + 1][g] = acc[nt][1];
      red[warp][nt * 8 + q * 2][g + 8] = acc[nt][2];
      red[warp][nt * 8 + q * 2 + 1][g + 8] = acc[nt][3];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < kTok * kSkinnyRows; i += 32 * kSkinnyWarps) {
      const int o = i % kSkinnyRows, tok = i / kSkinnyRows;
      if (t0 + tok < r1 && o0 + o < a.out) {
        float v = 0.f;
#pragma unroll
        for (int k = 0; k < kSkinnyWarps; ++k) v += red[k][tok][o];  // the same order on every call
        if (a.add) v += bf16_bits_to_f32(a.add[static_cast<int64_t>(t0 + tok) * a.ldadd + o0 + o]);
        a.Y[static_cast<int64_t>(t0 + tok) * a.ldy + o0 + o] = static_cast<uint16_t>(pack2(v, 0.f) & 0xFFFFu);
      }
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------
// Launch
// ---------------------------------------------------------------------------

struct DeviceInfo {
  int dev = 0, sms = 0;
};

cudaError_t device_info(DeviceInfo* d) {
  static std::atomic<int> sms[64];  // 0: not yet known
  cudaError_t e = cudaGetDevice(&d->dev);
  if (e != cudaSuccess) return e;
  if (d->dev < 0 || d->dev >= 64) return cudaErrorInvalidDevice;
  d->sms = sms[d->dev].load(std::memory_order_relaxed);
  if (d->sms == 0) {
    int major = 0;
    e = cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, d->dev);
    if (e != cudaSuccess) return e;
    if (major != 10) return cudaErrorNoKernelImageForDevice;
    e = cudaDeviceGetAttribute(&d->sms, cudaDevAttrMultiProcessorCount, d->dev);
    if (e != cudaSuccess) return e;
    sms[d->dev].store(d->sms, std::memory_order_relaxed);
  }
  return cudaSuccess;
}

template <bool kF8, bool kPair, int kBN>
cudaError_t launch_tile(const ProductArgs& a, const DeviceInfo& d, cudaStream_t st) {
  using C = TileCfg<kPair, kBN>;
  auto* fn = tile_kernel<kF8, kPair, kBN>;
  // Per kernel and device: the resident units (CTAs or pairs), once its
  // shared-memory limit is raised.  0: not yet done.
  static std::atomic<int> resident[64];
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kTileThreads);
  cfg.dynamicSmemBytes = C::kSmemBytes;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kPair ? 2 : 1;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int units = resident[d.dev].load(std::memory_order_relaxed);
  if (units == 0) {
    cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
    if (e != cudaSuccess) return e;
    units = d.sms;
    if (kPair) {
      cfg.gridDim = dim3(2 * (d.sms / 2));
      e = cudaOccupancyMaxActiveClusters(&units, fn, &cfg);
      if (e != cudaSuccess) return e;
      units = units < d.sms / 2 ? units : d.sms / 2;
    }
    if (units <= 0) return cudaErrorInvalidConfiguration;
    resident[d.dev].store(units, std::memory_order_relaxed);
  }
  // At most this many units have work; with offsets on the device the exact number is not known here.
  const int64_t most = (static_cast<int64_t>(a.n) / C::kBM + (a.offsets ? a.experts : 1)) * ((a.out + kBN - 1) / kBN);
  if (most < units) units = static_cast<int>(most);
  CUtensorMap mx, mw, mlo;
  const uint64_t bytes = static_cast<uint64_t>(a.in) * (kF8 ? 1 : 2);
  const uint64_t w_rows = static_cast<uint64_t>(a.experts) * a.out;
  cudaError_t e = make_tmap_bytes(&mx, a.X, a.n, bytes, a.ldx, kRowTile);
  if (e == cudaSuccess) e = make_tmap_bytes(&mw, a.W, w_rows, bytes, a.ldw, C::kBRows);
  if (e != cudaSuccess) return e;
  mlo = mw;
  if (a.W_lo) e = make_tmap_bytes(&mlo, a.W_lo, w_rows, bytes, a.ldw, C::kBRows);
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3(static_cast<unsigned>(kPair ? 2 * units : units));
  return cudaLaunchKernelEx(&cfg, fn, mx, mw, mlo, a);
}

template <bool kF8>
cudaError_t launch_type(const ProductArgs& a, const DeviceInfo& d, cudaStream_t st) {
  const int64_t per = (static_cast<int64_t>(a.n) + a.experts - 1) / a.experts;  // rows per expert, on average
  if (per <= 32) {
    const dim3 grid((a.out + kSkinnyRows - 1) / kSkinnyRows, a.experts);
    if (per <= 8)
      skinny_kernel<kF8, 1><<<grid, 32 * kSkinnyWarps, 0, st>>>(a);
    else if (per <= 16)
      skinny_kernel<kF8, 2><<<grid, 32 * kSkinnyWarps, 0, st>>>(a);
    else
      skinny_kernel<kF8, 4><<<grid, 32 * kSkinnyWarps, 0, st>>>(a);
    return cudaGetLastError();
  }
  return launch_tile<kF8, false, 128>(a, d, st);
}

}  // namespace

cudaError_t launch_product(const ProductArgs& a, cudaStream_t st) {
  DeviceInfo d;
  const cudaError_t e = device_info(&d);
  if (e != cudaSuccess) return e;
  return a.f8 ? launch_type<true>(a, d, st) : launch_type<false>(a, d, st);
}

}  // namespace ar
