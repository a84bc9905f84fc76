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
#include <type_traits>

#include "ar_device.cuh"
#include "ar_internal.h"
#include "ar_scaled.h"
#include "ar_units.h"

namespace ar {

namespace {

// Where bounded waits report when the caller passes no status word.
__device__ int g_product_status;

// ---------------------------------------------------------------------------
// Tile kernel
// ---------------------------------------------------------------------------

// Three warpgroups: producer, one or two MMA issuers and a scale loader; two of epilogue.
constexpr int kTileWarps = 12;
constexpr int kLoaderWarp = 3;
constexpr int kEpiWarp0 = 4;
constexpr int kTileThreads = 32 * kTileWarps;
constexpr int kMaxStages = 8;
constexpr int kRowTile = 128;     // rows per CTA: tensor-memory lanes
constexpr int kKBytes = 128;      // bytes of K per stage and row

constexpr int kScaleKb = 4;     // K blocks per slot of the scale ring
constexpr int kScaleSlots = 4;

struct TileSmem {
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t tfull[4], tempty[4];  // accumulator b of column half h: kHalves b + h
  uint64_t sfull[kScaleSlots], sempty[kScaleSlots];
  uint64_t drain[2];
  uint32_t tmem_base;
  int abort_flag;
  // e4m3: the scale ring.  A slot holds 16 bytes per row of the tile -- the aligned four of
  // the row's scales, so the K block that a slot starts with differs from row to row by
  // up to three -- and the weight's scales of four K blocks of each column half.
  alignas(16) float xs[kScaleSlots][kRowTile][kScaleKb];
  float ws[kScaleSlots][kScaleKb][2];
  int cum[kMaxExperts + 1];  // row blocks of the experts before e
};

template <bool kF8, bool kPair, int kBN>
struct TileCfg {
  // e4m3 tiles of 256 columns are two column halves of 128, each with its own MMAs,
  // accumulators and issuing warp: the hand-over of a half after every K block then
  // overlaps the other half's MMAs.
  static constexpr int kHalves = kF8 && kBN == 256 ? 2 : 1;
  static constexpr int kMmaN = kBN / kHalves;
  static constexpr int kBRows = kPair ? kBN / 2 : kBN;  // weight rows this CTA stages
  static constexpr int kWBoxes = kPair ? kHalves : 1;   // ... in so many loads (a pair's half: 64 rows in each CTA)
  static constexpr int kABytes = kRowTile * kKBytes;
  static constexpr int kStageBytes = kABytes + kBRows * kKBytes;
  static constexpr int kStages = kBN == 128 ? 5 : kPair ? 4 : 3;
  static constexpr int kNC = kBN / 2;               // columns per epilogue thread
  static constexpr int kRowPitch = kNC * 2 + 16;    // a row's part of Y on its way out; + 16: no bank conflicts
  static constexpr int kAccs = 512 / kBN;           // accumulators in tensor memory
  static constexpr int kBM = kPair ? 2 * kRowTile : kRowTile;  // rows per unit (CTA or pair)
  static constexpr int kTmemCols = 512;
  static constexpr int kOutOffset = kStages * kStageBytes;
  static constexpr int kBarOffset = kOutOffset + 8 * 32 * kRowPitch;
  static constexpr int kSmemBytes = 1024 + kBarOffset + static_cast<int>(sizeof(TileSmem));
  static_assert(kSmemBytes <= 232448, "shared memory per CTA");
  static_assert(kBarOffset % 16 == 0 && offsetof(TileSmem, xs) % 16 == 0, "16-byte asynchronous copies");
  static_assert(kAccs * kHalves <= 4, "accumulator barriers");
  // the shares of a split K, 128 x 128 fp32, pass through the operand stages
  static constexpr bool kCanSplit = !kPair && kBN == 128;
  static_assert(!kCanSplit || kStages * kStageBytes >= 128 * 128 * 4, "split-K exchange");
};

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// 16 bytes from byte `off` (even, below 16) of the 32 bytes a, b.
__device__ __forceinline__ uint4 bytes_at(uint4 a, uint4 b, int off) {
  uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
  for (int j = 0; j < 6; ++j) w[j] = off & 8 ? w[j + 2] : w[j];
#pragma unroll
  for (int j = 0; j < 5; ++j) w[j] = off & 4 ? w[j + 1] : w[j];
#pragma unroll
  for (int j = 0; j < 4; ++j) w[j] = __funnelshift_r(w[j], w[j + 1], off & 2 ? 16 : 0);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// 2, 4 or 8 bytes at an address that is a multiple of as many.
template <int kBytes>
__device__ __forceinline__ uint2 read_piece(const uint8_t* p) {
  if constexpr (kBytes == 8) return *reinterpret_cast<const uint2*>(p);
  if constexpr (kBytes == 4) return make_uint2(*reinterpret_cast<const uint32_t*>(p), 0);
  return make_uint2(*reinterpret_cast<const uint16_t*>(p), 0);
}
template <int kBytes>
__device__ __forceinline__ void write_piece(uint8_t* p, uint2 v) {
  if constexpr (kBytes == 8)
    *reinterpret_cast<uint2*>(p) = v;
  else if constexpr (kBytes == 4)
    *reinterpret_cast<uint32_t*>(p) = v.x;
  else
    *reinterpret_cast<uint16_t*>(p) = static_cast<uint16_t>(v.x);
}

// The way out of a warp's 32 rows x up to kNC columns (lane = row; rows from r1 on belong to
// others): each lane rounds its row's values into its own line of shared memory (put8), and
// the lines go to Y (send), each by one bulk copy, which runs while the warp goes on with the
// next unit.  The residual comes the same way back, asked for at the unit's start (begin).
// (Stored from registers, 16 bytes of 32 rows per instruction, the columns of a 256 x 256 tile
// kept the warps for 7500 cycles; through shared memory with coalesced stores for 3700, since
// every SM writes at the same time.)
//
// Where rows or widths are not multiples of 16 bytes, a line is brought as far from a 16-byte
// boundary as its row in memory is, so that the whole units of the row still leave by one bulk copy (and
// come, for the residual, by 16-byte copies); the up to 7 elements before and after them are moved
// in pieces of 2, 4 and 8 bytes.  (All elements one by one, by the whole warp: 4574 rows, 608 ->
// 2785: 36 us; so, 26; 20 with aligned rows.)  This form (not kWhole) has a kernel of its own:
// within the aligned one, its code slowed the loop over K (76 rows, 4096 -> 11008: 21.8 us for 19.2).
template <int kNC, bool kWhole>
struct RowsOut {
  static constexpr int kPitch = kNC * 2 + 16;
  uint8_t* lines;    // the warp's lines
  int row0, r1, col; // first row, end of the rows that exist, first column
  int cols;          // columns that exist (0 or fewer: none)
  int lane;

  __device__ __forceinline__ const uint16_t* add_row(const ProductArgs& a, int r) const {
    return a.add + static_cast<int64_t>(row0 + r) * a.ldadd + col;
  }
  static __device__ __forceinline__ int off16(const void* p) { return static_cast<int>(reinterpret_cast<uintptr_t>(p) & 15); }

  __device__ __forceinline__ void begin(const ProductArgs& a, uint8_t* warp_lines, int row0_, int r1_, int col_,
                                        int width, int lane_) {
    lines = warp_lines;
    row0 = row0_;
    r1 = r1_;
    col = col_;
    lane = lane_;
    cols = min(width, a.out - col);
    asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");  // the last unit's copies have read the lines
    __syncwarp();  // (every lane's: the residual is brought in by the whole warp)
    if (!a.add) return;
    constexpr int kUnits = kNC / 8;  // 16-byte units per row, at most
    const int unit = lane % kUnits;
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      const int r = i * (32 / kUnits) + lane / kUnits;
      if (row0 + r >= r1 || cols <= 0) continue;
      const uint16_t* from = add_row(a, r);
      const int off = kWhole ? 0 : off16(from);
      if (unit >= (off != 0) && unit < (off + cols * 2) / 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(lines + r * kPitch + unit * 16)),
                     "l"(reinterpret_cast<const uint8_t*>(from) - off + unit * 16)
                     : "memory");
    }
    if (!kWhole && row0 + lane < r1 && cols > 0) {
      const uint16_t* from = add_row(a, lane);
      const int off = off16(from);
      const uint8_t* unit0 = reinterpret_cast<const uint8_t*>(from) - off;
      uint2 v[12];
      edges(off, [&](auto j, auto size, int b) { v[decltype(j)::value] = read_piece<decltype(size)::value>(unit0 + b); });
      edges(off, [&](auto j, auto size, int b) { write_piece<decltype(size)::value>(lines + lane * kPitch + b, v[decltype(j)::value]); });
    }
  }

  // f(piece, size, byte of the line) for pieces of 2, 4 or 8 bytes, as long as their addresses allow, of
  // what of a row at `off` lies in no whole unit.
  template <class F>
  __device__ __forceinline__ void edges(int off, F f) const {
    const int end = off + cols * 2;
    if (off) pieces<0>(off, min(end, 16), f);
    pieces<6>(max(end & ~15, off ? 16 : 0), end, f);
  }

  template <int kFirst, class F>
  static __device__ __forceinline__ void pieces(int b, int end, F f) {
    auto piece = [&](auto index, auto size) {
      constexpr int kIndex = decltype(index)::value, kBytes = decltype(size)::value;
      if ((kIndex >= 3 || (b & kBytes)) && b + kBytes <= end) {
        f(std::integral_constant<int, kFirst + kIndex>{}, size, b);
        b += kBytes;
      }
    };
    piece(std::integral_constant<int, 0>{}, std::integral_constant<int, 2>{});
    piece(std::integral_constant<int, 1>{}, std::integral_constant<int, 4>{});
    piece(std::integral_constant<int, 2>{}, std::integral_constant<int, 8>{});
    piece(std::integral_constant<int, 3>{}, std::integral_constant<int, 8>{});
    piece(std::integral_constant<int, 4>{}, std::integral_constant<int, 4>{});
    piece(std::integral_constant<int, 5>{}, std::integral_constant<int, 2>{});
  }

  // Before the first put8: the residual is there, from the start of the lines.
  __device__ __forceinline__ void ready(const ProductArgs& a, int width) {
    if (!a.add) return;
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncwarp();
    const int off = kWhole ? 0 : off16(add_row(a, lane));
    if (off == 0) return;
    uint4* line = reinterpret_cast<uint4*>(lines + lane * kPitch);
    uint4 now = line[0];
#pragma unroll 2
    for (int u = 0; u < width / 8; ++u) {
      const uint4 next = line[u + 1];
      line[u] = bytes_at(now, next, off);
      now = next;
    }
  }

  // Columns c .. c + 7.
  __device__ __forceinline__ void put8(const ProductArgs& a, int c, float (&x)[8]) {
    uint4* p = reinterpret_cast<uint4*>(lines + lane * kPitch + c * 2);
    if (a.add) {
      const uint4 v = *p;
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        x[2 * j] += __uint_as_float(w[j] << 16);
        x[2 * j + 1] += __uint_as_float(w[j] & 0xFFFF0000u);
      }
    }
    *p = make_uint4(pack2(x[0], x[1]), pack2(x[2], x[3]), pack2(x[4], x[5]), pack2(x[6], x[7]));
  }

  // After the last put8.
  __device__ __forceinline__ void send(const ProductArgs& a, int width) {
    uint8_t* line = lines + lane * kPitch;
    int off = 0, lo = 0, hi = cols * 2;
    if (!kWhole) {
      off = off16(a.Y + static_cast<int64_t>(row0 + lane) * a.ldy + col);
      lo = off ? 16 : 0;
      hi = (off + cols * 2) & ~15;
      if (off) {  // to the row's own distance from a boundary
        uint4* units = reinterpret_cast<uint4*>(line);
        uint4 now = make_uint4(0, 0, 0, 0);
#pragma unroll 2
        for (int u = width / 8; u > 0; --u) {
          const uint4 before = units[u - 1];
          units[u] = bytes_at(before, now, 16 - off);
          now = before;
        }
        units[0] = bytes_at(now, now, 16 - off);
      }
    }
    if (row0 + lane < r1 && cols > 0) {
      uint8_t* to = reinterpret_cast<uint8_t*>(a.Y + static_cast<int64_t>(row0 + lane) * a.ldy + col) - off;
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      if (hi > lo)
        asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(to + lo),
                     "r"(smem_u32(line + lo)), "r"(hi - lo)
                     : "memory");
      if (!kWhole)
        edges(off, [&](auto, auto size, int b) { write_piece<decltype(size)::value>(to + b, read_piece<decltype(size)::value>(line + b)); });
    }
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
  }
};

// tcgen05 and TMA instructions issued by the whole warp with a predicate that holds in
// one lane (elect_one).  In a branch of one lane the compiler can neither keep their
// operands in uniform registers nor compute them there, which cost about 70 cycles per
// instruction; a K block of the tile kernel has 8 of them.
template <bool kF8, bool kPair>
__device__ __forceinline__ void umma(uint32_t leader, uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                     uint32_t accumulate) {
#define AR_UMMA(GROUP, KIND)                                                                     \
  asm volatile(                                                                                  \
      "{\n\t.reg .pred p, q;\n\t"                                                                \
      "setp.ne.b32 p, %4, 0;\n\t"                                                                \
      "setp.ne.b32 q, %5, 0;\n\t"                                                                \
      "@q tcgen05.mma.cta_group::" GROUP ".kind::" KIND " [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem), \
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(leader)                         \
      : "memory")
  if (kF8 && kPair)
    AR_UMMA("2", "f8f6f4");
  else if (kF8)
    AR_UMMA("1", "f8f6f4");
  else if (kPair)
    AR_UMMA("2", "f16");
  else
    AR_UMMA("1", "f16");
#undef AR_UMMA
}

// Arrive on `bar` (pair: on the barrier at this offset in both CTAs) once the MMAs issued so far are done.
template <bool kPair>
__device__ __forceinline__ void umma_commit_if(uint32_t leader, uint32_t bar) {
  if (kPair)
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\t"
        "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}" ::"r"(
            bar),
        "h"((uint16_t)3), "r"(leader)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar),
        "r"(leader)
        : "memory");
}

__device__ __forceinline__ void expect_tx_if(uint32_t leader, uint32_t bar, uint32_t bytes) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\t"
      "@q mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n\t}" ::"r"(bar),
      "r"(bytes), "r"(leader)
      : "memory");
}

template <bool kPair>
__device__ __forceinline__ void tma_load_if(uint32_t leader, uint32_t dst, const CUtensorMap* map, int32_t x, int32_t y,
                                            uint32_t bar) {
  if (kPair)
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "@q cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3}], [%4];\n\t}" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar), "r"(leader)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "@q cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3}], [%4];\n\t}" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar), "r"(leader)
        : "memory");
}

__device__ __forceinline__ float ld_shared(uint32_t addr) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

__device__ __forceinline__ float4 ld_cluster(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// Wait for the phase of `bar` with this parity (whole warps).  After timeout_ns, or once
// another role has given up (*abort), it records kDevTimeout in *status, raises *abort and
// returns false.  The test is one instruction of the warp, so its lanes leave together.
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, volatile int* abort, int* status,
                                         uint64_t timeout_ns) {
  uint32_t polls = 0;
  uint64_t t0 = 0;
  while (!mbar_try_wait(bar, parity)) {
    if ((++polls & 255u) == 0) {
      const uint64_t now = globaltimer_ns();
      if (t0 == 0) t0 = now;
      if (__any_sync(__activemask(), now - t0 > timeout_ns || *abort)) {
        atomicCAS(status, kDevOk, kDevTimeout);
        *abort = 1;
        return false;
      }
    }
  }
  return true;
}

// Slots of the scale ring that a share of `blocks` K blocks takes (rows start up to three
// blocks into their first).
__device__ __forceinline__ int scale_slots(int blocks) { return (blocks + 3 + kScaleKb - 1) / kScaleKb; }

// A 16-byte asynchronous copy of which the first `bytes` are read and the rest is zero.
__device__ __forceinline__ void cp_async16(float* dst, const float* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(bytes) : "memory");
}

// A 4-byte asynchronous copy, and an arrive once the thread's copies so far are done.
__device__ __forceinline__ void cp_async4(float* dst, const float* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}

__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// Arrive on the pair leader's barrier (a shared::cluster address).  No memory is handed
// over with it: the accumulator's values are in registers (tcgen05.wait::ld) and
// tcgen05.fence orders the loads, so the release stays at CTA scope; at cluster scope it
// waits for every outstanding access of the thread, and the hand-off took four times as long.
__device__ __forceinline__ void mbar_arrive_remote(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// 1 in one lane of the (converged) warp, the same on every call.
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p;
}

__host__ __device__ constexpr uint32_t umma_idesc_f8(int M, int N) {
  return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);  // f32 D, e4m3 A and B
}

template <bool kF8, bool kPair, int kBN, bool kWhole>
__global__ void __launch_bounds__(kTileThreads, 1)
    tile_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW,
                const __grid_constant__ CUtensorMap tmWlo, const __grid_constant__ ProductArgs args) {
  using C = TileCfg<kF8, kPair, kBN>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  TileSmem* sm = reinterpret_cast<TileSmem*>(smem + C::kBarOffset);
  volatile int* abort_flag = &sm->abort_flag;
  int* status = args.status ? args.status : &g_product_status;
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0);  // warp-uniform
  const int lane = threadIdx.x & 31;
  // A cluster is a pair of CTAs that share a 256-row tile, or args.split CTAs that share K.
  const bool split = C::kCanSplit && args.split > 1;
  const uint32_t cta = kPair || split ? cluster_ctarank() : 0u;
  const uint32_t rank = kPair ? cta : 0u;

  chain_next();
  if (warp == 1 && lane == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&sm->full[s], 1);
      mbar_init(&sm->empty[s], C::kHalves);  // one commit per issuer
    }
    for (int b = 0; b < C::kAccs * C::kHalves; ++b) {
      mbar_init(&sm->tfull[b], 1);
      mbar_init(&sm->tempty[b], (kPair ? 2 : 1) * 8 / C::kHalves);  // one arrive per epilogue warp that reads it
    }
    for (int b = 0; b < kScaleSlots; ++b) {
      mbar_init(&sm->sfull[b], 32);  // every thread of the loader warp
      mbar_init(&sm->sempty[b], 8);
    }
    mbar_init(&sm->drain[0], 1);
    mbar_init(&sm->drain[1], 1);
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
  chain_wait();  // (barriers and tensor memory, above, are this block's own)
  if (warp == 2) {
    // Row blocks before each expert.
    if (!args.offsets) {
      if (lane == 0) {
        sm->cum[0] = 0;
        sm->cum[1] = (args.n + C::kBM - 1) / C::kBM;
      }
    } else {
      const int limit = most_row_blocks(args, C::kBM);
      int carry = 0;
      if (lane == 0) sm->cum[0] = 0;
      for (int e0 = 0; e0 < args.experts; e0 += 32) {
        int v = e0 + lane < args.experts ? row_blocks(args, e0 + lane, C::kBM) : 0;
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
  const int64_t unit0 = kPair ? blockIdx.x >> 1 : split ? blockIdx.x / args.split : blockIdx.x;
  const int64_t stride = kPair ? gridDim.x >> 1 : split ? num_units : gridDim.x;  // split: one unit per cluster
  const int nkb = args.nkb;
  const int k_total = (!kF8 && args.W_lo) ? 2 * nkb : nkb;
  // This CTA's share of K (not empty: split <= nkb).
  const int k_begin = split ? static_cast<int>(static_cast<int64_t>(k_total) * cta / args.split) : 0;
  const int k_end = split ? static_cast<int>(static_cast<int64_t>(k_total) * (cta + 1) / args.split) : k_total;
  const uint32_t bar_full = smem_u32(sm->full), bar_empty = smem_u32(sm->empty);
  const uint32_t bar_tfull = smem_u32(sm->tfull), bar_tempty = smem_u32(sm->tempty);

  // Registers: the launch's 12 warps at 168 become 4 at 56 and 8 at 224.  The compiler allots 168 to all: the
  // e4m3 forms (128 sums, 64 columns in flight) spill 44 to 104 bytes a thread there, the bf16 ones none.
  if (warp < kEpiWarp0) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    if (warp == 0) {
      // -------------------------------------------------------------- producer
      const uint32_t leader = elect_one();
      const uint32_t leader_full = kPair ? mapa_shared(bar_full, 0) : 0u;  // completion counts on the pair leader's
      int stage = 0;
      uint32_t phase = 0, issued_mask = 0, issued_parity = 0;
      bool ok = true;
      for (int64_t t = unit0; ok && t < num_units && !args.starve; t += stride) {
        const Unit u = find_unit(args, sm->cum, t, num_n, C::kBM, kBN);
        const int x_row = u.m0 + static_cast<int>(rank) * kRowTile;
        const int w_row = u.e * args.out + u.n0 + static_cast<int>(rank) * (C::kBRows / C::kWBoxes);
        for (int kb = k_begin; kb < k_end; ++kb) {
          if (!wait_bar(bar_empty + 8 * stage, phase ^ 1, abort_flag, status, args.timeout_ns)) {
            ok = false;
            break;
          }
          const uint32_t sx = smem_u32(smem) + stage * C::kStageBytes;
          const bool lo = !kF8 && kb >= nkb;
          const int k = (lo ? kb - nkb : kb) * kKBytes;  // bytes: the maps are byte maps
          if (!kPair || rank == 0) expect_tx_if(leader, bar_full + 8 * stage, (kPair ? 2 : 1) * C::kStageBytes);
          const uint32_t bar = (kPair ? leader_full : bar_full) + 8 * stage;
          tma_load_if<kPair>(leader, sx, &tmX, k, x_row, bar);
#pragma unroll
          for (int b = 0; b < C::kWBoxes; ++b)
            tma_load_if<kPair>(leader, sx + C::kABytes + b * (C::kBRows / C::kWBoxes) * kKBytes, lo ? &tmWlo : &tmW, k,
                               w_row + b * C::kMmaN, bar);
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
    } else if (warp <= C::kHalves) {
      if (rank == 0) {
        // ------------------------------------------------------------ MMA issuers
        constexpr int kM = kPair ? 2 * kRowTile : kRowTile;
        constexpr uint32_t idesc = kF8 ? umma_idesc_f8(kM, C::kMmaN) : umma_idesc_bf16(kM, C::kMmaN);
        const int half = warp - 1;
        const uint32_t leader = elect_one();
        const uint64_t desc0 = umma_desc_sw128(smem_u32(smem));
        const uint32_t b_off = C::kABytes + half * (C::kBRows / C::kHalves) * kKBytes;
        int stage = 0, acc = 0;
        uint32_t phase = 0, acc_phase = 0;
        bool ok = true;
        for (int64_t t = unit0; ok && t < num_units; t += stride) {
          for (int kb = k_begin; kb < k_end; ++kb) {
            const uint32_t bar_acc = 8 * (acc * C::kHalves + half);
            const bool first = kF8 || kb == k_begin, last = kF8 || kb == k_end - 1;
            // both tests in flight at once: each takes over 100 cycles, passed or not
            const bool free = !first || mbar_try_wait(bar_tempty + bar_acc, acc_phase ^ 1);
            const bool here = mbar_try_wait(bar_full + 8 * stage, phase);
            if (!free) ok = wait_bar(bar_tempty + bar_acc, acc_phase ^ 1, abort_flag, status, args.timeout_ns);
            if (ok && !here) ok = wait_bar(bar_full + 8 * stage, phase, abort_flag, status, args.timeout_ns);
            if (!ok) break;
            tc_fence_after();
            const uint32_t d_tmem = tmem_base + acc * kBN + half * C::kMmaN;
            const uint64_t a_desc = desc0 + stage * (C::kStageBytes >> 4);
            const uint64_t b_desc = a_desc + (b_off >> 4);
#pragma unroll
            for (int k = 0; k < 4; ++k)  // 32 bytes of K each: 2 descriptor units
              umma<kF8, kPair>(leader, d_tmem, a_desc + 2 * k, b_desc + 2 * k, idesc, !first || k > 0);
            umma_commit_if<kPair>(leader, bar_empty + 8 * stage);
            if (last) {
              umma_commit_if<kPair>(leader, bar_tfull + bar_acc);
              if (++acc == C::kAccs) {
                acc = 0;
                acc_phase ^= 1;
              }
            }
            if (++stage == C::kStages) {
              stage = 0;
              phase ^= 1;
            }
          }
        }
        // Every MMA this warp's leader issued has completed once `drain` flips.
        if (leader) {
          if (kPair)
            umma_commit_pair_local(&sm->drain[half]);
          else
            umma_commit(&sm->drain[half]);
        }
        __syncwarp();
        mbar_wait_drain(&sm->drain[half], 0, args.timeout_ns);
      }
    } else if (kF8 && warp == kLoaderWarp) {
      // ---------------------------------------------------------- scale loader
      // Four rows per lane, one 16-byte asynchronous copy per row and slot (a row's scales are
      // contiguous along K), slots ahead of the epilogue.  Single 4-byte copies, a line
      // each, kept the load path busy for a third of the kernel's time; they remain for scales
      // that do not start on 16 bytes.
      const bool vec = (reinterpret_cast<uintptr_t>(args.xs) & 15) == 0;
      const int64_t total = static_cast<int64_t>(args.n) * nkb;
      uint32_t slots = 0;  // slots filled so far: slot slots % kScaleSlots is next
      bool ok = true;
      for (int64_t t = unit0; ok && t < num_units; t += stride) {
        const Unit u = find_unit(args, sm->cum, t, num_n, C::kBM, kBN);
        int64_t x[4];  // first aligned scale of the lane's rows; rows past the expert's end: past the tensor's
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int row = u.m0 + static_cast<int>(rank) * kRowTile + lane + 32 * r;
          x[r] = row < u.r1 ? (static_cast<int64_t>(row) * nkb + k_begin) & ~int64_t(3) : total;
        }
        // lanes 0 .. 7 also bring the weight's scales: block lane / 2 of half lane % 2
        const int nb = min((u.n0 + (lane & 1) * (kBN / 2)) >> 7, args.out_blocks - 1);
        const float* w = args.ws + (static_cast<int64_t>(u.e) * args.out_blocks + nb) * nkb;
        const int fills = scale_slots(k_end - k_begin);
        for (int j = 0; j < fills; ++j, ++slots) {
          const int slot = slots % kScaleSlots;
          if (!wait_bar(smem_u32(&sm->sempty[slot]), (slots / kScaleSlots & 1) ^ 1, abort_flag, status,
                        args.timeout_ns)) {
            ok = false;
            break;
          }
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int64_t left = total - (x[r] + 4 * j);  // scales from here to the tensor's end
            float* dst = sm->xs[slot][lane + 32 * r];
            const float* src = args.xs + (left > 0 ? x[r] + 4 * j : 0);
            if (vec) {
              cp_async16(dst, src, left >= 4 ? 16 : left > 0 ? static_cast<int>(left) * 4 : 0);
            } else {
#pragma unroll
              for (int i = 0; i < 4; ++i)
                if (i < left) cp_async4(dst + i, src + i);
            }
          }
          if (lane < 2 * kScaleKb)
            cp_async4(&sm->ws[slot][lane >> 1][lane & 1], w + min(k_begin + 4 * j + (lane >> 1), nkb - 1));
          cp_async_arrive(&sm->sfull[slot]);
        }
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
    }
    if (split) {
      __syncwarp();
      cluster_sync_all();
      cluster_sync_all();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
    // -------------------------------------------------------------- epilogue
    constexpr int kNC = C::kNC;
    const int quarter = warp & 3;      // tensor-memory lanes this warp may access
    const int half = (warp - kEpiWarp0) >> 2;  // column half of the tile
    const uint32_t t_lane = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + half * kNC;
    uint8_t* out_buf = smem + C::kOutOffset + (warp - kEpiWarp0) * 32 * C::kRowPitch;
    // This warp's accumulator barriers (the empty one is the pair leader's): + 8 kHalves for the second buffer.
    const uint32_t my_tfull = bar_tfull + (C::kHalves == 2 ? 8 * half : 0);
    const uint32_t my_tempty =
        (kPair ? mapa_shared(bar_tempty, 0) : bar_tempty) + (C::kHalves == 2 ? 8 * half : 0);
    const uint32_t xs_base = smem_u32(sm->xs[0][quarter * 32 + lane]), ws_base = smem_u32(&sm->ws[0][0][half]);
    auto release = [&](int buf) {  // (tcgen05.wait::ld, before it, is the whole warp's)
      tc_fence_before();
      if (lane == 0) mbar_arrive_remote(my_tempty + 8 * C::kHalves * buf);
    };
    int acc_buf = 0;
    uint32_t acc_phase = 0;
    uint32_t slots = 0;  // slots of the scale ring that earlier units took
    bool ok = true;
    for (int64_t t = unit0; ok && t < num_units; t += stride) {
      const Unit u = find_unit(args, sm->cum, t, num_n, C::kBM, kBN);
      const int row0 = u.m0 + static_cast<int>(rank) * kRowTile + quarter * 32;  // the warp's 32 rows
      const int col0 = u.n0 + half * kNC;
      if constexpr (kF8) {
        RowsOut<kNC, kWhole> rows_out;
        if (!split) rows_out.begin(args, out_buf, row0, u.r1, col0, kNC, lane);
        float acc[kNC];
#pragma unroll
        for (int i = 0; i < kNC; ++i) acc[i] = 0.f;
        // The row's scales start `skew` into its 16-byte pieces: block k is in slot (skew + k) / 4.
        // Byte offsets that move with k, and 64 columns in flight: 876 -> 867 us at n = 16384, 4096 -> 11008.
        const int blocks = k_end - k_begin;
        const uint32_t skew = (static_cast<uint32_t>(row0 + lane) * static_cast<uint32_t>(nkb) + k_begin) % kScaleKb;
        constexpr uint32_t kSlotBytes = kRowTile * kScaleKb * 4;
        uint32_t x_off = slots % kScaleSlots * kSlotBytes + skew * 4;
        uint32_t w_off = slots % kScaleSlots * (kScaleKb * 8);
        uint32_t next_slot = slots;  // to wait for
#pragma unroll 1
        for (int k = 0; k < blocks; ++k) {
          if (k == 0 || k % kScaleKb == 1) {  // a slot that is new to the rows that are furthest ahead
            if (!wait_bar(smem_u32(&sm->sfull[next_slot % kScaleSlots]), next_slot / kScaleSlots & 1, abort_flag, status,
                          args.timeout_ns)) {
              ok = false;
              break;
            }
            ++next_slot;
          }
          const float s = __fmul_rn(ld_shared(xs_base + x_off), ld_shared(ws_base + w_off));
          x_off += 4;
          if ((x_off & 15) == 0) x_off = (x_off + kSlotBytes - 16) % (kScaleSlots * kSlotBytes);
          w_off = (w_off + 8) % (kScaleSlots * kScaleKb * 8);
          if (k % kScaleKb == kScaleKb - 1) {  // no row needs slot k / 4 any more
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm->sempty[(slots + k / kScaleKb) % kScaleSlots]);
          }
          if (!wait_bar(my_tfull + 8 * C::kHalves * acc_buf, acc_phase, abort_flag, status, args.timeout_ns)) {
            ok = false;
            break;
          }
          tc_fence_after();
#pragma unroll
          for (int g = 0; g < kNC / 64; ++g) {
            uint32_t r[32], q[32];
            tmem_ld_32cols(t_lane + acc_buf * kBN + g * 64, r);
            tmem_ld_32cols(t_lane + acc_buf * kBN + g * 64 + 32, q);
            tmem_ld_wait();
            if (g == kNC / 64 - 1) release(acc_buf);
#pragma unroll
            for (int j = 0; j < 32; ++j) acc[g * 64 + j] = fmaf(__uint_as_float(r[j]), s, acc[g * 64 + j]);
#pragma unroll
            for (int j = 0; j < 32; ++j) acc[g * 64 + 32 + j] = fmaf(__uint_as_float(q[j]), s, acc[g * 64 + 32 + j]);
          }
          if (++acc_buf == C::kAccs) {
            acc_buf = 0;
            acc_phase ^= 1;
          }
        }
        if (!ok) break;
        __syncwarp();
        if (lane == 0)
          for (int j = blocks / kScaleKb; j < scale_slots(blocks); ++j)
            mbar_arrive(&sm->sempty[(slots + j) % kScaleSlots]);
        slots += scale_slots(blocks);
        if (split) {
          // This share's sums, for the exchange below: [column / 4][row], 16 bytes each.
          float4* part = reinterpret_cast<float4*>(smem) + half * (kNC / 4) * kRowTile + quarter * 32 + lane;
#pragma unroll
          for (int c = 0; c < kNC / 4; ++c)
            part[c * kRowTile] = make_float4(acc[4 * c], acc[4 * c + 1], acc[4 * c + 2], acc[4 * c + 3]);
          break;
        }
        rows_out.ready(args, kNC);
#pragma unroll
        for (int c = 0; c < kNC; c += 8) {
          float x[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) x[j] = acc[c + j];
          rows_out.put8(args, c, x);
        }
        rows_out.send(args, kNC);
      } else {
        RowsOut<kNC, kWhole> rows_out;
        if (!split) rows_out.begin(args, out_buf, row0, u.r1, col0, kNC, lane);
        if (!wait_bar(my_tfull + 8 * C::kHalves * acc_buf, acc_phase, abort_flag, status, args.timeout_ns)) {
          ok = false;  // (a share of K that is not there is not added up)
          break;
        }
        tc_fence_after();
        if (!split) rows_out.ready(args, kNC);
#pragma unroll 1
        for (int g = 0; g < kNC / 32; ++g) {
          uint32_t r[32];
          tmem_ld_32cols(t_lane + acc_buf * kBN + g * 32, r);
          tmem_ld_wait();
          if (g == kNC / 32 - 1) release(acc_buf);
          if (split) {
            float4* part =
                reinterpret_cast<float4*>(smem) + (half * (kNC / 4) + g * 8) * kRowTile + quarter * 32 + lane;
#pragma unroll
            for (int c = 0; c < 8; ++c)
              part[c * kRowTile] = make_float4(__uint_as_float(r[4 * c]), __uint_as_float(r[4 * c + 1]),
                                               __uint_as_float(r[4 * c + 2]), __uint_as_float(r[4 * c + 3]));
          } else {
#pragma unroll
            for (int c = 0; c < 32; c += 8) {
              float x[8];
#pragma unroll
              for (int j = 0; j < 8; ++j) x[j] = __uint_as_float(r[c + j]);
              rows_out.put8(args, g * 32 + c, x);
            }
          }
        }
        if (split) break;
        rows_out.send(args, kNC);
        if (++acc_buf == C::kAccs) {
          acc_buf = 0;
          acc_phase ^= 1;
        }
      }
    }
    if (split) {
      // Every CTA of the cluster adds its columns of the tile over the shares, in order.
      // (The operand stages are free: the accumulator's last hand-over follows every MMA.)
      const bool work = ok && unit0 < num_units;
      const int per = kBN / (2 * args.split);  // columns per thread: 32 or 16
      const int c0 = static_cast<int>(cta) * 2 * per + half * per;
      RowsOut<kNC, kWhole> rows_out;
      if (work) {
        const Unit u = find_unit(args, sm->cum, unit0, num_n, C::kBM, kBN);
        rows_out.begin(args, out_buf, u.m0 + quarter * 32, u.r1, u.n0 + c0, per, lane);
      }
      cluster_sync_all();
      if (work) {
        rows_out.ready(args, per);
        const uint32_t mine = smem_u32(smem) + (c0 / 4 * kRowTile + quarter * 32 + lane) * 16;
        auto put = [&](auto shares) {
          constexpr int kShares = decltype(shares)::value, kPer = kBN / (2 * kShares);
          float4 v[kPer / 4][kShares];  // all in flight at once
#pragma unroll
          for (int c = 0; c < kPer / 4; ++c)
#pragma unroll
            for (int k = 0; k < kShares; ++k) v[c][k] = ld_cluster(mapa_shared(mine + c * kRowTile * 16, k));
#pragma unroll
          for (int c = 0; c < kPer / 4; c += 2) {
            float x[8];
#pragma unroll
            for (int k = 0; k < kShares; ++k) {
              const float4 a = v[c][k], b = v[c + 1][k];
              const float y[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
              for (int j = 0; j < 8; ++j) x[j] = k == 0 ? y[j] : __fadd_rn(x[j], y[j]);
            }
            rows_out.put8(args, c * 4, x);
          }
        };
        if (args.split == 2)
          put(std::integral_constant<int, 2>{});
        else
          put(std::integral_constant<int, 4>{});
        rows_out.send(args, per);
      }
      cluster_sync_all();  // no CTA leaves while another reads its shares
    }
    asm volatile("cp.async.wait_all;\n\tcp.async.bulk.wait_group.read 0;" ::: "memory");
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
// Skinny kernel: 16 kMR rows of W per CTA, the K blocks dealt to its 8 warps.
//
// A K block (128 bytes) of a warp is two 64-byte pieces; lane (g, q) holds bytes
// 16 q .. 16 q + 15 of each piece for weight rows g and g + 8 of each 16-row tile and for
// row g of each 8-row tile of X.  The m16n8k16 instructions take, from lane (g, q), two
// 4-byte registers (pairs of 16-bit values) per operand row; which columns of K they stand
// for does not matter as long as W and X agree.  So bf16 registers feed them as they are,
// and a register of four e4m3 values becomes the two halves of an fp16 operand (exact:
// e4m3 is a subset of fp16).  The e4m3 form of the instruction does the same conversion
// for every product anew; converting each operand once is what makes several tiles cheap.
// ---------------------------------------------------------------------------

template <bool kF8>
__device__ __forceinline__ void mma_16x8(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  if (kF8)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Four e4m3 values as two fp16 pairs (exact; NaN stays NaN).
__device__ __forceinline__ void e4m3_to_f16(uint32_t v, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(v));
}

// A 16-byte piece as the operand registers of the instructions it feeds: 8 of fp16 pairs (4 k16
// steps of two), or the 4 it has (2 steps of two).
template <bool kF8>
struct Piece {
  static constexpr int kSteps = kF8 ? 4 : 2;
  uint32_t r[kSteps][2];
  __device__ __forceinline__ explicit Piece(const uint4& v) {
    if constexpr (kF8) {
      e4m3_to_f16(v.x, r[0][0], r[0][1]);
      e4m3_to_f16(v.y, r[1][0], r[1][1]);
      e4m3_to_f16(v.z, r[2][0], r[2][1]);
      e4m3_to_f16(v.w, r[3][0], r[3][1]);
    } else {
      r[0][0] = v.x, r[0][1] = v.y, r[1][0] = v.z, r[1][1] = v.w;
    }
  }
};

constexpr int kSkinnyWarps = 8;

// A lane's 16-byte asynchronous copy into its own place (zeros instead where `ok` is false).
__device__ __forceinline__ void cp_async_own(uint4* dst, const uint8_t* src, bool ok) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(ok ? 16 : 0) : "memory");
}

// kNT tiles of 8 rows of X per pass, kMR strips of 16 rows of W per CTA.  Each warp keeps the
// operands of kS K blocks in flight, in its own part of shared memory: asynchronous copies
// that each lane makes for itself and reads back itself, so nothing but its own
// cp.async groups orders them, and the bytes in flight (80 to 160 KB an SM) cost no registers.
// (With the same loads into registers, one or two blocks ahead, 64 experts of one row each, 4096 ->
// 2048, took 58.5 us; so they take 51, 90% of the measured copy bandwidth.)
template <bool kF8, int kNT, int kMR, int kS>
struct SkinnyCfg {
  static constexpr int kTok = 8 * kNT, kRows = 16 * kMR;
  static constexpr int kPieces = kMR * 4 + kNT * 2;  // 16-byte pieces per lane and K block
  static constexpr int kRing = kSkinnyWarps * kS * kPieces * 32 * 16;
  static constexpr int kRed = kSkinnyWarps * kTok * (kRows + 1) * 4;  // takes the ring's place after the last block
  static constexpr int kSmemBytes = kRing > kRed ? kRing : kRed;
};

template <bool kF8, int kNT, int kMR, int kS>
__global__ void __launch_bounds__(32 * kSkinnyWarps) skinny_kernel(const __grid_constant__ ProductArgs a) {
  using C = SkinnyCfg<kF8, kNT, kMR, kS>;
  constexpr int kTok = C::kTok, kRows = C::kRows;
  extern __shared__ uint4 skinny_smem[];
  chain_next();
  chain_wait();
  const int e = blockIdx.y;
  int r0, r1;
  expert_rows(a, e, r0, r1);
  r0 += blockIdx.z * kTok;  // passes blockIdx.z, + gridDim.z, ...
  if (r0 >= r1) return;
  const int o0 = blockIdx.x * kRows;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, q = lane & 3;
  const int in_bytes = a.in * (kF8 ? 1 : 2);  // a multiple of 16
  const int64_t w_off = (static_cast<int64_t>(e) * a.out + o0 + g) * a.ldw + q * 16;
  // (the rows of a CTA lie in one 128-row scale block: kRows divides 128)
  const float* ws = kF8 ? a.ws + (static_cast<int64_t>(e) * a.out_blocks + (o0 >> 7)) * a.nkb : nullptr;
  const int blocks = (!kF8 && a.W_lo) ? 2 * a.nkb : a.nkb;  // the lo half's follow the hi half's
  // [stage][piece][lane] of this warp
  uint4* ring = skinny_smem + warp * (kS * C::kPieces * 32) + lane;
  auto red = reinterpret_cast<float(*)[kTok][kRows + 1]>(skinny_smem);

  for (int t0 = r0; t0 < r1; t0 += gridDim.z * kTok) {
    float acc[kMR][kNT][4];
#pragma unroll
    for (int m = 0; m < kMR; ++m)
#pragma unroll
      for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[m][nt][i] = 0.f;
    float sx[kS][kNT][2], sw[kS];  // the scales of the stages' blocks
    // Block b into stage j: the copies, and the scales into registers; one group, empty past the end.
    auto load = [&](int b, int j) {
      if (b < blocks) {
        const bool lo = !kF8 && b >= a.nkb;
        const uint8_t* wp = static_cast<const uint8_t*>(lo ? a.W_lo : a.W) + w_off;
        const int kb = lo ? b - a.nkb : b;
        uint4* dst = ring + j * (C::kPieces * 32);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int k = kb * kKBytes + c * 64;
          const bool k_ok = k + q * 16 < in_bytes;
#pragma unroll
          for (int m = 0; m < kMR; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const bool ok = k_ok && o0 + m * 16 + h * 8 + g < a.out;
              cp_async_own(dst + ((m * 2 + c) * 2 + h) * 32,
                           ok ? wp + static_cast<int64_t>(m * 16 + h * 8) * a.ldw + k : static_cast<const uint8_t*>(a.W), ok);
            }
#pragma unroll
          for (int nt = 0; nt < kNT; ++nt) {
            const int row = t0 + nt * 8 + g;
            const bool ok = k_ok && row < r1;
            const uint8_t* x = static_cast<const uint8_t*>(a.X);
            cp_async_own(dst + (kMR * 4 + nt * 2 + c) * 32, ok ? x + static_cast<int64_t>(row) * a.ldx + q * 16 + k : x, ok);
          }
        }
        if (kF8) {
          sw[j] = ws[kb];
#pragma unroll
          for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int row = t0 + nt * 8 + q * 2 + h;
              sx[j][nt][h] = row < r1 ? a.xs[static_cast<int64_t>(row) * a.nkb + kb] : 0.f;
            }
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int j = 0; j < kS; ++j) load(warp + j * kSkinnyWarps, j);
    for (int b0 = warp; b0 < blocks; b0 += kS * kSkinnyWarps) {
#pragma unroll
      for (int j = 0; j < kS; ++j) {
        const int b = b0 + j * kSkinnyWarps;
        if (b >= blocks) break;
        asm volatile("cp.async.wait_group %0;" ::"n"(kS - 1) : "memory");  // the oldest group: stage j's
        const uint4* src = ring + j * (C::kPieces * 32);
        float part[kMR][kNT][4];
        if (kF8) {
#pragma unroll
          for (int m = 0; m < kMR; ++m)
#pragma unroll
            for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
              for (int i = 0; i < 4; ++i) part[m][nt][i] = 0.f;
        }
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint4 xv[kNT];
#pragma unroll
          for (int nt = 0; nt < kNT; ++nt) xv[nt] = src[(kMR * 4 + nt * 2 + c) * 32];
#pragma unroll
          for (int m = 0; m < kMR; ++m) {
            const Piece<kF8> lo(src[((m * 2 + c) * 2) * 32]), hi(src[((m * 2 + c) * 2 + 1) * 32]);
#pragma unroll
            for (int nt = 0; nt < kNT; ++nt) {
              const Piece<kF8> xx(xv[nt]);
#pragma unroll
              for (int s = 0; s < Piece<kF8>::kSteps; ++s)
                mma_16x8<kF8>(kF8 ? part[m][nt] : acc[m][nt], lo.r[s][0], hi.r[s][0], lo.r[s][1], hi.r[s][1],
                              xx.r[s][0], xx.r[s][1]);
            }
          }
        }
        if (kF8) {
#pragma unroll
          for (int nt = 0; nt < kNT; ++nt) {
            const float s0 = __fmul_rn(sx[j][nt][0], sw[j]), s1 = __fmul_rn(sx[j][nt][1], sw[j]);
#pragma unroll
            for (int m = 0; m < kMR; ++m) {
              acc[m][nt][0] = fmaf(part[m][nt][0], s0, acc[m][nt][0]);
              acc[m][nt][1] = fmaf(part[m][nt][1], s1, acc[m][nt][1]);
              acc[m][nt][2] = fmaf(part[m][nt][2], s0, acc[m][nt][2]);
              acc[m][nt][3] = fmaf(part[m][nt][3], s1, acc[m][nt][3]);
            }
          }
        }
        load(b + kS * kSkinnyWarps, j);
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();  // every warp is done with the ring
    // c0, c1: weight row g, rows 2q and 2q + 1 of X; c2, c3: weight row g + 8.
#pragma unroll
    for (int m = 0; m < kMR; ++m)
#pragma unroll
      for (int nt = 0; nt < kNT; ++nt) {
        red[warp][nt * 8 + q * 2][m * 16 + g] = acc[m][nt][0];
        red[warp][nt * 8 + q * 2 + 1][m * 16 + g] = acc[m][nt][1];
        red[warp][nt * 8 + q * 2][m * 16 + g + 8] = acc[m][nt][2];
        red[warp][nt * 8 + q * 2 + 1][m * 16 + g + 8] = acc[m][nt][3];
      }
    __syncthreads();
    for (int i = threadIdx.x; i < kTok * kRows; i += 32 * kSkinnyWarps) {
      const int o = i % kRows, tok = i / kRows;
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

template <bool kF8, int kNT, int kMR, int kS>
cudaError_t launch_skinny(const ProductArgs& a, const DeviceInfo& d, cudaStream_t st) {
  using C = SkinnyCfg<kF8, kNT, kMR, kS>;
  auto* fn = skinny_kernel<kF8, kNT, kMR, kS>;
  static std::atomic<int> ready[64];  // per device: the shared-memory limit is raised
  if (!ready[d.dev].load(std::memory_order_relaxed)) {
    const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
    if (e != cudaSuccess) return e;
    ready[d.dev].store(1, std::memory_order_relaxed);
  }
  // The passes over X side by side while there are few CTAs (up to 8 an SM): one whose expert has no such
  // rows leaves at once.
  const int strips = (a.out + C::kRows - 1) / C::kRows;
  const int64_t passes = (static_cast<int64_t>(a.n) + C::kTok - 1) / C::kTok;
  const int64_t room = 8 * d.sms / (static_cast<int64_t>(strips) * a.experts);
  const int64_t z = passes < room ? passes : room;
  const dim3 grid(strips, a.experts, static_cast<unsigned>(z > 1 ? z : 1));
  return launch_chained(fn, grid, dim3(32 * kSkinnyWarps), C::kSmemBytes, 1, st, a);
}

// Units of bm rows x bn columns that can have work (exact for one expert).
int64_t units_at_most(const ProductArgs& a, int bm, int bn) {
  return ((static_cast<int64_t>(a.n) + bm - 1) / bm + a.experts - 1) * ((a.out + bn - 1) / bn);
}

template <bool kF8, bool kPair, int kBN, bool kWhole>
cudaError_t launch_tile_as(ProductArgs a, const DeviceInfo& d, cudaStream_t st, int split) {
  using C = TileCfg<kF8, kPair, kBN>;
  auto* fn = tile_kernel<kF8, kPair, kBN, kWhole>;
  // Per kernel and device: the resident units (CTAs or pairs), once its
  // shared-memory limit is raised.  0: not yet done.
  static std::atomic<int> resident[64];
  int units = resident[d.dev].load(std::memory_order_relaxed);
  if (units == 0) {
    cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
    if (e != cudaSuccess) return e;
    units = d.sms;
    if (kPair) {
      cudaLaunchAttribute attr[1];
      attr[0].id = cudaLaunchAttributeClusterDimension;
      attr[0].val.clusterDim.x = 2;
      attr[0].val.clusterDim.y = 1;
      attr[0].val.clusterDim.z = 1;
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3(2 * (d.sms / 2));
      cfg.blockDim = dim3(kTileThreads);
      cfg.dynamicSmemBytes = C::kSmemBytes;
      cfg.attrs = attr;
      cfg.numAttrs = 1;
      e = cudaOccupancyMaxActiveClusters(&units, fn, &cfg);
      if (e != cudaSuccess) return e;
      units = units < d.sms / 2 ? units : d.sms / 2;
    }
    if (units <= 0) return cudaErrorInvalidConfiguration;
    resident[d.dev].store(units, std::memory_order_relaxed);
  }
  // At most this many units have work; with offsets on the device the exact number is not known here.
  const int64_t most = units_at_most(a, C::kBM, kBN);
  while (split > a.nkb) split /= 2;  // 1, 2 or 4
  a.split = split;
  // A bf16 accumulator is handed over after all of K, so the waits' limit grows with it: 1 us a K block, of which
  // 17 rows take 55 ns and 300 rows x 1000 columns 210.  (2^25 blocks, the longest, take 1.8 s.)
  a.timeout_ns += 1000ull * (a.W_lo ? 2 : 1) * static_cast<uint64_t>(a.nkb);
  if (most < units || split > 1) units = static_cast<int>(most);
  CUtensorMap mx, mw, mlo;
  const uint64_t bytes = static_cast<uint64_t>(a.in) * (kF8 ? 1 : 2);
  const uint64_t w_rows = static_cast<uint64_t>(a.experts) * a.out;
  cudaError_t e = make_tmap_bytes(&mx, a.X, a.n, bytes, a.ldx, kRowTile);
  if (e == cudaSuccess) e = make_tmap_bytes(&mw, a.W, w_rows, bytes, a.ldw, C::kBRows / C::kWBoxes);
  if (e != cudaSuccess) return e;
  mlo = mw;
  if (a.W_lo) e = make_tmap_bytes(&mlo, a.W_lo, w_rows, bytes, a.ldw, C::kBRows / C::kWBoxes);
  if (e != cudaSuccess) return e;
  const int cluster = kPair ? 2 : split;
  return launch_chained(fn, dim3(static_cast<unsigned>(cluster * units)), dim3(kTileThreads), C::kSmemBytes, cluster, st,
                        mx, mw, mlo, a);
}

template <bool kF8, bool kPair, int kBN>
cudaError_t launch_tile(const ProductArgs& a, const DeviceInfo& d, cudaStream_t st, int split = 1) {
  return a.vec_y && a.out % 8 == 0 ? launch_tile_as<kF8, kPair, kBN, true>(a, d, st, split)
                                   : launch_tile_as<kF8, kPair, kBN, false>(a, d, st, split);
}

// Which kernel.  Both operand types, times on one B200 in us (e4m3 unless said).
//
// Rows per expert (on average) decide between the two kernels.  The skinny one has no
// fixed cost but walks W again for every kTok rows; the tile one starts at 8 us (tensor
// memory, barriers, descriptors, the first loads) and then takes 128 rows for the price of one.
//   n = 8,  29568 -> 8192: skinny 43, tile 62         n = 16, 29568 -> 8192: skinny 48, tile 50
//   n = 32, 29568 -> 8192: skinny 87, tile 49         n = 32, 4096 -> 11008: skinny 21, tile 18
// Several experts are taken to be uneven (some have several times the average):
//   64 experts, 4096 -> 2048, 4 rows each: 83 and 115; 8: 102 and 107; 12: 117 and 108
//   the same in bf16, 8 rows each: 187 and 183; 12: 220 and 184
// Only the average is known here: an expert with many more rows walks its W once per 8 or 16 of them, alone.
//   256 experts, 2048 -> 1024, 1024 rows: 108 drawn evenly (10 rows at most), 178 with 411 in one expert.
// Of the skinny kernel's shapes, two strips of W per CTA and two blocks per warp in flight won
// over one strip (51 and 69 for 64 experts with 64 rows) and over more blocks (three: 70;
// shared memory then holds fewer CTAs); 8 rows of X per pass while there are no more, 16 up to 16.
//
// Among the tiles, 128 x 128 on one SM, 128 x 256 on one SM and 256 x 256 on a pair, the
// fewest waves times the cost of a wave: e4m3, K = 4096: 16, 26.5 and 25 us a wave (n = 16384,
// 4096 -> 11008: 1157, 1022, 933 in all; n = 333: 35, 28, 56; n = 512, 4096 -> 4096: 19, 26, 25);
// bf16: 13, 21 and 20 for 2048 columns of K.  With half the SMs idle or more, 128 x 128
// tiles share their K blocks among a cluster of 2 or 4 CTAs (n = 64, 4096 -> 4096: 17.5 alone,
// 13.8 and 12.2 shared; 29568 -> 8192: 85, 50).  A cluster of 8 gained nothing more (7.6 for
// 7.7 at 1024 -> 1000) and lost up to twice the time.
template <bool kF8>
cudaError_t launch_type(const ProductArgs& a, const DeviceInfo& d, cudaStream_t st) {
  const int64_t per = (static_cast<int64_t>(a.n) + a.experts - 1) / a.experts;
  const int64_t strips = (a.out + 15) / 16;  // 16-row strips of one W
  const bool one = a.experts == 1;
  if (per <= (one ? 8 : 4)) return launch_skinny<kF8, 1, 2, 2>(a, d, st);
  if (per <= (one ? 16 : 8)) return launch_skinny<kF8, 2, 2, 2>(a, d, st);
  // Small products of more rows, 32 a pass and the passes side by side: the work in blocks of 16 x 32 x 128
  // bytes, one of each of the CTA's 8 warps at least.  Times of the two kernels: 64 rows, 1024 -> 1000: 3.8 and 9.3; 32, 4096 -> 4096: 9.7 and 13.6;
  // 3802, 128 -> 1026: 49 and 13.6; 8 experts, 96 rows in all, 1024 -> 1024: 7.7 and 11.3.
  const int64_t active = a.experts < a.n ? a.experts : a.n;
  const int64_t passes = one ? (per + 31) / 32 : a.n / 32 + active;
  if (passes * strips * (a.nkb > 8 ? a.nkb : 8) <= 8192) return launch_skinny<kF8, 4, 1, 2>(a, d, st);
  // Row blocks: exact for one expert, else half a block more per expert, and one at least.
  auto waves = [&](int bm, int bn, int resident) {
    const int64_t cols = (a.out + bn - 1) / bn;
    if (a.experts == 1) return static_cast<double>(((a.n + bm - 1) / bm * cols + resident - 1) / resident);
    const double rows = static_cast<double>(a.n) / bm + 0.5 * active;
    const double units = (rows > active ? rows : active) * cols;
    return units > resident ? units / resident : 1.0;
  };
  const double small = waves(128, 128, d.sms) * (kF8 ? 16.0 : 13.0);
  const double wide = waves(128, 256, d.sms) * (kF8 ? 26.5 : 21.0);
  const double pair = waves(256, 256, d.sms / 2) * (kF8 ? 25.0 : 20.0);
  if (small <= wide && small <= pair) {
    const int64_t units = units_at_most(a, 128, 128);
    return launch_tile<kF8, false, 128>(a, d, st, units * 4 <= d.sms ? 4 : units * 2 <= d.sms ? 2 : 1);
  }
  if (wide <= pair) return launch_tile<kF8, false, 256>(a, d, st);
  return launch_tile<kF8, true, 256>(a, d, st);
}

}  // namespace

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

cudaError_t launch_product(const ProductArgs& a, cudaStream_t st) {
  DeviceInfo d;
  const cudaError_t e = device_info(&d);
  if (e != cudaSuccess) return e;
  return a.f8 ? launch_type<true>(a, d, st) : launch_type<false>(a, d, st);
}

}  // namespace ar
