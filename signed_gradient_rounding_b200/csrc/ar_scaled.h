// Launch interfaces of the 8-bit chain: e4m3 tensors with one fp32 scale per block of
// 128 columns (rows: per row; weights: per 128 rows), the norm and quantisers that
// make them, and the products, dense or grouped by expert, that read them.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace ar {

// The current device (one of sm_100) and its SMs.
struct DeviceInfo {
  int dev = 0, sms = 0;
};
cudaError_t device_info(DeviceInfo* d);

struct RmsNormArgs {
  const void* x = nullptr;  // [rows, cols] fp32 or bf16, row pitch ldx (elements, as every pitch here)
  int x_bf16 = 1;
  int64_t ldx = 0;
  int64_t rows = 0;
  int cols = 0, blocks = 0;         // blocks = ceil(cols / 128)
  const void* residual = nullptr;   // fp32 or bf16; null: none
  int r_bf16 = 1;
  int64_t ldr = 0;
  const void* weight = nullptr;     // [cols]; null: ones
  int w_bf16 = 1;
  float eps = 0.f;
  float inv_cols = 0.f;             // 1 / cols (set by the launch)
  void* sum = nullptr;              // the residual's type; may be the residual itself
  int64_t lds = 0;
  uint16_t* y = nullptr;
  int64_t ldy = 0;
  uint8_t* q = nullptr;
  int64_t ldq = 0;
  float* scale = nullptr;           // [rows, blocks]
};
constexpr int kNormMaxCols = 32768;  // 1024 threads x 4 octs of 8 columns in registers

struct RowQuantArgs {
  const void* x = nullptr;
  int x_bf16 = 1;
  int64_t ldx = 0;
  const uint16_t* gate = nullptr;  // set: the value is silu(x) * gate (x bf16)
  int64_t ldg = 0;
  int64_t rows = 0;
  int cols = 0, blocks = 0;
  uint8_t* q = nullptr;
  int64_t ldq = 0;
  float* scale = nullptr;  // [rows, blocks]
};

struct TileQuantArgs {
  const void* x = nullptr;  // [count, rows, cols], row pitch ldx, matrices rows * ldx apart
  int x_bf16 = 1;
  int64_t ldx = 0;
  int64_t count = 1, rows = 0;
  int cols = 0, blocks = 0, row_blocks = 0;
  uint8_t* q = nullptr;
  int64_t ldq = 0;
  float* scale = nullptr;  // [count, row_blocks, blocks]
};

// Launches of the chain overlap their own start with the end of the launch before them
// (programmatic dependent launch): a kernel lets the next one start as soon as all of its
// own blocks have (chain_next), and waits for the one before it to complete, its writes
// visible, before it touches memory (chain_wait, by every thread of every block, first of
// all).  A launch without the attribute before or after it is ordered as ever.
//
// So a kernel is already running while the one before it writes what it will read.  The read-only
// path (.nc loads, the ldg intrinsic) promises data that does not change while the kernel
// runs, and leaves the compiler free to move the load across the wait: no kernel of the chain uses it.
#ifdef __CUDACC__
__device__ __forceinline__ void chain_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void chain_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

template <class... P, class... A>
cudaError_t launch_chained(void (*fn)(P...), dim3 grid, dim3 block, size_t smem, int cluster, cudaStream_t st, A&&... args) {
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, fn, static_cast<P>(args)...);
}
#endif

cudaError_t launch_rms_norm(const RmsNormArgs& a, cudaStream_t st);
cudaError_t launch_row_quant(const RowQuantArgs& a, cudaStream_t st);
cudaError_t launch_tile_quant(const TileQuantArgs& a, cudaStream_t st);

// Y = X W^T, dense or by expert.  Operand rows are sequences of 128-byte K blocks
// (128 e4m3 or 64 bf16 elements).
struct ProductArgs {
  int f8 = 0;                        // e4m3 operands with scales; else bf16
  const void* X = nullptr;           // [n, in]
  int64_t ldx = 0;                   // bytes
  const void* W = nullptr;           // [experts * out, in]
  const void* W_lo = nullptr;        // bf16 only: the second half of a hi + lo pair
  int64_t ldw = 0;                   // bytes
  int n = 0, in = 0, out = 0;
  int nkb = 0;                       // K blocks: ceil(in * element size / 128)
  int out_blocks = 0;                // ceil(out / 128)
  int experts = 1;
  const int32_t* offsets = nullptr;  // [experts + 1] first row of each expert; null: one expert, all rows
  const float* xs = nullptr;         // [n, nkb]
  const float* ws = nullptr;         // [experts, out_blocks, nkb]
  const uint16_t* add = nullptr;     // [n, out] bf16, pitch ldadd
  int64_t ldadd = 0;
  uint16_t* Y = nullptr;             // [n, out] bf16, pitch ldy
  int64_t ldy = 0;
  int vec_y = 0;                     // Y and add take 16-byte accesses at multiples of 8 columns
  int split = 1;                     // CTAs of a cluster that share K (set by the launch)
  int* status = nullptr;             // null: a word of the library's
  uint64_t timeout_ns = 1000000000ull;  // of one wait; the launch adds to it for K
  int starve = 0;                    // test hook: the tiles' producers bring nothing, so every wait behind them runs out
};
constexpr int kMaxExperts = 1024;

cudaError_t launch_product(const ProductArgs& a, cudaStream_t st);

}  // namespace ar
