// ops.cu - C entry points of the norm and dropout operators (declared in
// include/moe_ffn.h): argument checks, kernel choice and launch. Nothing here
// synchronises the host or allocates device memory.
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstdio>

#include "dropout.cuh"
#include "moe_ffn.h"
#include "norm.cuh"
#include "ops_host.h"

namespace {

using moe::launch_overlapped;
using moe::set_error;

int dtype_size(int dtype) {
  return dtype == MOE_DTYPE_FP32 ? 4 : dtype == MOE_DTYPE_BF16 || dtype == MOE_DTYPE_FP16 ? 2 : 0;
}

bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

int launch_status(cudaError_t e, const char* what) {
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e == cudaSuccess) return MOE_OK;
  char buf[256];
  snprintf(buf, sizeof(buf), "%s launch failed: %s", what, cudaGetErrorString(e));
  cudaGetLastError();
  return set_error(MOE_CUDA_ERROR, buf);
}

// Shape and stride checks shared by the row operators; null when they pass.
const char* check_rows(int64_t rows, int64_t cols) {
  if (rows < 0) return "rows must be >= 0";
  if (cols < 1) return "cols must be >= 1";
  return nullptr;
}
bool bad_stride(int64_t rows, int64_t cols, int64_t ld) { return rows > 1 && ld < cols; }

// SMs of a B200, for the thresholds below (measured on one); grids ask the device.
constexpr int kB200Sms = 148;

constexpr int64_t kMaxRows = (1LL << 31) - 1;
constexpr int64_t kMaxCols = 1LL << 24;

// ------------------------------------------------------------------ norm
constexpr int kNormBlocks = 2 * kB200Sms;   // blocks (partial rows) of a backward pass at most

int round32(int64_t v) { return static_cast<int>((v + 31) / 32 * 32); }

template <typename T, int VEC, int VPT>
cudaError_t launch_norm_forward(const moe::NormParams& P, int group, cudaStream_t st) {
  const int per_block = group == 32 ? 4 : 1;
  const int64_t blocks = (P.rows + per_block - 1) / per_block;
  return launch_overlapped(moe::norm_forward_kernel<T, VEC, VPT>, dim3(unsigned(blocks)),
                           dim3(group * per_block), 0, st, 1, P, group);
}

// Rows from which the tile kernels run. In general when every SM has four; with two for
// rows of 4097 to 8192 (forward, 300 x 7168 bf16: 6.3 us, 7.8 with a block a row) and for
// unaligned rows above 4096 (300 x 7001 bf16: 10.1 and 14.9).
int64_t tile_rows_forward(int cols, bool vec) {
  return (cols > 4096 && (cols <= 8192 || !vec) ? 2 : 4) * kB200Sms;
}
// Backward: with two also from 256 to 1024 vectors a row (300 x 2048 bf16: 11.8 us, 13.7 with
// a block a row), and always for unaligned rows of 4097 to 8192 (1 x 7001 bf16: 9.6 us; a
// block a row would hold so many elements a thread that they spill, 20.6).
int64_t tile_rows_backward(int cols, bool vec, int vectors) {
  if (vec) return (vectors >= 256 && vectors <= 1024 ? 2 : 4) * kB200Sms;
  return cols > 4096 && cols <= 8192 ? 1 : 4 * kB200Sms;
}
constexpr size_t kTileSmem = 208 * 1024;
// 16 column warps beside the 8 row warps (with 8, 4096 x 7168 bf16 forward took 36 us
// where it took 26 and the backward pass up to 30% longer).
constexpr int kColumnWarps = 16;

// Rows a tile and slots, for `planes` matrices (x, and dy in the backward pass): three
// tiles of as many rows as fit (4096 x 7168 bf16 forward: 27 us with 4 rows and 3 slots, 34
// with 2 and 7), more tiles when they are small; no more rows a tile than a block has, so
// that with few rows several row warps share one.
bool tile_shape(moe::NormTile* L, const moe::NormParams& P, int vec, int vpt, int column_warps,
                size_t esize, int planes, bool contiguous, int sms, size_t* smem) {
  const int n = P.cols / vec;
  L->group = round32((n + vpt - 1) / vpt);
  if (L->group > column_warps * 32) return false;
  L->contiguous = contiguous;
  L->test_withhold = 0;
  L->weight_bytes = planes == 2 ? uint32_t((size_t(P.cols) * 4 + 127) / 128 * 128) : 0;
  if (L->weight_bytes >= kTileSmem) return false;
  const size_t room = kTileSmem - L->weight_bytes;
  const size_t extra = vec == 1 ? 32 : 0;         // a run of bytes widened to 16-byte boundaries
  for (int rows = moe::kTileMaxRows; rows >= 1; rows /= 2) {
    if (rows > 1 && int64_t(rows) * sms > P.rows + sms - 1) continue;
    const size_t slot = (size_t(P.cols) * esize * rows + extra + 127) / 128 * 128;
    const size_t tile = slot * planes;
    if (rows > 1 && tile * 3 > room) continue;
    if (tile * 2 > room) return false;
    size_t slots = room / tile;
    if (slots > moe::kTileMaxSlots) slots = moe::kTileMaxSlots;
    L->rows = rows;
    L->slots = int(slots);
    L->slot_bytes = uint32_t(slot);
    *smem = L->weight_bytes + tile * slots;
    return true;
  }
  return false;
}

// Raise a tile kernel's shared-memory limit, once a device (`done`: the kernel's own bits).
template <typename K>
cudaError_t tile_attribute(K kernel, std::atomic<uint64_t>* done, int device) {
  const uint64_t bit = 1ull << device;
  if (done->load(std::memory_order_acquire) & bit) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(
      kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kTileSmem));
  if (e == cudaSuccess) done->fetch_or(bit, std::memory_order_release);
  return e;
}

template <typename T, int VEC, int VPT, bool RMS>
cudaError_t launch_norm_forward_tile(const moe::NormParams& P, moe::NormTile L, size_t smem,
                                     const moe::OpsDevice& d, cudaStream_t st) {
  static std::atomic<uint64_t> done{0};
  const auto kernel = moe::norm_forward_tile_kernel<T, VEC, VPT, kColumnWarps, RMS>;
  const cudaError_t e = tile_attribute(kernel, &done, d.index);
  if (e != cudaSuccess) return e;
  L.test_withhold = moe::take_test_timeout();
  const int64_t blocks = P.rows < d.sms ? P.rows : d.sms;
  return launch_overlapped(kernel, dim3(unsigned(blocks)),
                           dim3(moe::tile_threads(kColumnWarps)), smem, st, 1, P, L, d.status);
}

// Runs the tile kernel with the fewest vectors a column thread that cover the columns; false
// when none does.
template <typename T, int VEC, bool RMS, int VPT, int MAX>
bool norm_forward_tile(const moe::NormParams& P, bool contiguous, const moe::OpsDevice& d,
                       cudaStream_t st, cudaError_t* e) {
  moe::NormTile L;
  size_t smem;
  if (tile_shape(&L, P, VEC, VPT, kColumnWarps, sizeof(T), 1, contiguous, d.sms, &smem)) {
    *e = launch_norm_forward_tile<T, VEC, VPT, RMS>(P, L, smem, d, st);
    return true;
  }
  if constexpr (VPT < MAX) return norm_forward_tile<T, VEC, RMS, VPT * 2, MAX>(P, contiguous, d, st, e);
  return false;
}

template <typename T>
cudaError_t norm_forward_any(const moe::NormParams& P, bool vec, bool contiguous,
                             const moe::OpsDevice& d, cudaStream_t st) {
  constexpr int V = 16 / sizeof(T);
  // Few rows: as many threads a row as it has vectors (latency). Many unaligned rows that
  // are not contiguous: short ones a warp each, no block barrier in the statistics.
  const bool few = P.rows < tile_rows_forward(P.cols, vec);
  if (!few && (vec || contiguous)) {
    cudaError_t e;
    if (vec ? (P.rms ? norm_forward_tile<T, V, true, 1, 4>(P, contiguous, d, st, &e)
                     : norm_forward_tile<T, V, false, 1, 4>(P, contiguous, d, st, &e))
            : (P.rms ? norm_forward_tile<T, 1, true, 4, 32>(P, contiguous, d, st, &e)
                     : norm_forward_tile<T, 1, false, 4, 32>(P, contiguous, d, st, &e)))
      return e;
  }
  if (vec) {
    const int n = P.cols / V;
    if (n <= 32) return launch_norm_forward<T, V, 1>(P, 32, st);
    if (n <= 1024) return launch_norm_forward<T, V, 1>(P, round32(n), st);
    if (n <= 2048) return launch_norm_forward<T, V, 4>(P, round32((n + 3) / 4), st);
    if (n <= 8192) return launch_norm_forward<T, V, 8>(P, round32((n + 7) / 8), st);
  } else {
    if (P.cols <= 32) return launch_norm_forward<T, 1, 1>(P, 32, st);
    if (!few && P.cols <= 128) return launch_norm_forward<T, 1, 4>(P, 32, st);
    if (!few && P.cols <= 512) return launch_norm_forward<T, 1, 16>(P, 32, st);
    if (P.cols <= 4096) return launch_norm_forward<T, 1, 4>(P, round32((P.cols + 3) / 4), st);
    if (P.cols <= 16384)
      return launch_norm_forward<T, 1, 16>(P, round32((P.cols + 15) / 16), st);
  }
  const int64_t blocks = P.rows < 592 ? P.rows : 592;
  return launch_overlapped(moe::norm_forward_long_kernel<T>, dim3(unsigned(blocks)), dim3(1024), 0,
                           st, 1, P);
}

template <typename T, int VEC, int VPT, bool RMS, bool GRADW>
cudaError_t launch_norm_backward(const moe::NormParams& P, int group, int* blocks,
                                 cudaStream_t st) {
  int groups = 512 / group;
  if (groups < 1) groups = 1;
  if (groups > 8) groups = 8;
  const size_t smem = groups > 1 ? size_t(RMS ? 1 : 2) * P.cols * sizeof(float) : 0;
  int64_t n = (P.rows + groups - 1) / groups;
  const int cap = group * groups > 512 ? kNormBlocks / 2 : kNormBlocks;
  if (n > cap) n = cap;
  *blocks = static_cast<int>(n);
  return launch_overlapped(moe::norm_backward_kernel<T, VEC, VPT, RMS, GRADW>, dim3(unsigned(n)),
                           dim3(group * groups), smem, st, 1, P, group);
}

template <typename T, int VEC, int VPT, bool RMS, bool GRADW>
cudaError_t launch_norm_backward_tile(const moe::NormParams& P, moe::NormTile L, size_t smem,
                                      const moe::OpsDevice& d, int* blocks, cudaStream_t st) {
  static std::atomic<uint64_t> done{0};
  const auto kernel = moe::norm_backward_tile_kernel<T, VEC, VPT, kColumnWarps, RMS, GRADW>;
  const cudaError_t e = tile_attribute(kernel, &done, d.index);
  if (e != cudaSuccess) return e;
  L.test_withhold = moe::take_test_timeout();
  // no more blocks than partial rows in the workspace: min(rows, kNormBlocks)
  *blocks = d.sms < kNormBlocks ? d.sms : kNormBlocks;
  if (P.rows < *blocks) *blocks = static_cast<int>(P.rows);
  return launch_overlapped(kernel, dim3(*blocks), dim3(moe::tile_threads(kColumnWarps)), smem, st, 1, P, L,
                           d.status);
}

template <typename T, int VEC, bool RMS, bool GRADW, int VPT, int MAX>
bool norm_backward_tile(const moe::NormParams& P, bool contiguous, const moe::OpsDevice& d,
                        int* blocks, cudaStream_t st, cudaError_t* e) {
  moe::NormTile L;
  size_t smem;
  if (tile_shape(&L, P, VEC, VPT, kColumnWarps, sizeof(T), 2, contiguous, d.sms, &smem)) {
    // the groups' sums meet in the ring: two planes of fp32 columns
    const bool meet = kColumnWarps * 32 / L.group > 1;
    if (meet && smem - L.weight_bytes < size_t(P.cols) * 8) return false;
    *e = launch_norm_backward_tile<T, VEC, VPT, RMS, GRADW>(P, L, smem, d, blocks, st);
    return true;
  }
  if constexpr (VPT < MAX)
    return norm_backward_tile<T, VEC, RMS, GRADW, VPT * 2, MAX>(P, contiguous, d, blocks, st, e);
  return false;
}

template <typename T, bool RMS, bool GRADW>
cudaError_t norm_backward_any(const moe::NormParams& P, bool vec, bool contiguous,
                              const moe::OpsDevice& d, int* blocks, cudaStream_t st) {
  constexpr int V = 16 / sizeof(T);
  if (P.rows >= tile_rows_backward(P.cols, vec, P.cols / V) && (vec || contiguous)) {
    cudaError_t e;
    if (vec ? norm_backward_tile<T, V, RMS, GRADW, 1, 4>(P, contiguous, d, blocks, st, &e)
            : norm_backward_tile<T, 1, RMS, GRADW, 4, 32>(P, contiguous, d, blocks, st, &e))
      return e;
  }
  if (vec) {
    const int n = P.cols / V;
    if (n <= 1024) return launch_norm_backward<T, V, 1, RMS, GRADW>(P, round32(n), blocks, st);
  } else if (P.cols <= 4096) {
    return launch_norm_backward<T, 1, 4, RMS, GRADW>(P, round32((P.cols + 3) / 4), blocks, st);
  }
  // Wider rows from global memory, three passes, element by element (300 x 16384 fp32: 40 us;
  // held in the registers of a block, spilling, 90. 3000 x 16384 fp32: 275 us, 600 x 70000: 316,
  // where reading x and dy and writing dx once would be 90 and 77).
  cudaError_t e = cudaSuccess;
  if (GRADW) {                          // before dx, which may overwrite dy
    *blocks = static_cast<int>(P.rows < 32 ? P.rows : 32);
    e = launch_overlapped(moe::norm_backward_long_sum_kernel<T>,
                          dim3(unsigned((P.cols + 255) / 256), *blocks), dim3(256), 0, st, 1, P);
  }
  if (P.y && e == cudaSuccess) {
    const int64_t n = P.rows < 592 ? P.rows : 592;
    e = launch_overlapped(moe::norm_backward_long_kernel<T>, dim3(unsigned(n)), dim3(1024), 0, st,
                          1, P);
  }
  return e;
}

template <typename T>
cudaError_t norm_backward_typed(const moe::NormParams& P, bool vec, bool contiguous, bool gradw,
                                const moe::OpsDevice& d, int* blocks, cudaStream_t st) {
  if (P.rms)
    return gradw ? norm_backward_any<T, true, true>(P, vec, contiguous, d, blocks, st)
                 : norm_backward_any<T, true, false>(P, vec, contiguous, d, blocks, st);
  return gradw ? norm_backward_any<T, false, true>(P, vec, contiguous, d, blocks, st)
               : norm_backward_any<T, false, false>(P, vec, contiguous, d, blocks, st);
}

// Whether rows of this tensor can be read as 16-byte vectors.
bool vector_rows(const void* p, int64_t rows, int64_t ld, int esize) {
  return aligned(p, 16) && (rows <= 1 || (ld * esize) % 16 == 0);
}

int check_norm(int kind, int dtype, int wdtype, int64_t rows, int64_t cols) {
  if (kind != MOE_NORM_LAYER && kind != MOE_NORM_RMS)
    return set_error(MOE_INVALID_ARG, "kind must be MOE_NORM_LAYER or MOE_NORM_RMS");
  if (!dtype_size(dtype)) return set_error(MOE_INVALID_ARG, "unknown dtype");
  if (wdtype != dtype && wdtype != MOE_DTYPE_FP32)
    return set_error(MOE_INVALID_ARG, "weights must have x's dtype or fp32");
  if (const char* m = check_rows(rows, cols)) return set_error(MOE_INVALID_ARG, m);
  if (rows > kMaxRows || cols > kMaxCols)
    return set_error(MOE_UNSUPPORTED, "norm needs rows < 2^31 and cols <= 2^24");
  return MOE_OK;
}

// ------------------------------------------------------------------ dropout
template <typename T, bool RES, int MODE>
cudaError_t launch_dropout(moe::DropoutParams P, bool flat, cudaStream_t st) {
  if (!flat) {
    int64_t blocks = (P.n + 1023) / 1024;
    if (blocks > (1 << 20)) blocks = 1 << 20;      // the rest of a larger tensor by stride
    return launch_overlapped(moe::dropout_strided_kernel<T, RES, MODE>, dim3(unsigned(blocks)),
                             dim3(256), 0, st, 1, P);
  }
  const int64_t n = P.n;
  const char *x = static_cast<const char*>(P.x), *res = static_cast<const char*>(P.residual);
  char* out = static_cast<char*>(P.out);
  for (int64_t e0 = 0; e0 < n; e0 += moe::kDropSlice) {
    P.n = n - e0 < moe::kDropSlice ? n - e0 : moe::kDropSlice;
    P.x = x + e0 * sizeof(T);
    P.residual = RES ? res + e0 * sizeof(T) : nullptr;
    P.out = out + e0 * sizeof(T);
    P.block_lo = static_cast<uint32_t>(e0 >> 2);
    P.block_hi = static_cast<uint32_t>((e0 >> 2) >> 32);
    const int64_t vecs = P.n * sizeof(T) / 16;
    // Four vectors a thread once that still leaves two rounds of blocks for every SM; below,
    // one each (128 x 2048 bf16: 1.5 us against 2.3 with four).
    cudaError_t e;
    if (vecs >= int64_t(8) * kB200Sms * 1024)
      e = launch_overlapped(moe::dropout_flat_kernel<T, RES, MODE, 4>,
                            dim3(unsigned((vecs + 1023) / 1024)), dim3(256), 0, st, 1, P);
    else
      e = launch_overlapped(moe::dropout_flat_kernel<T, RES, MODE, 1>,
                            dim3(unsigned(vecs < 256 ? 1 : (vecs + 255) / 256)), dim3(256), 0, st,
                            1, P);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

template <typename T>
cudaError_t dropout_typed(const moe::DropoutParams& P, int mode, bool flat, cudaStream_t st) {
  if (P.residual)
    return mode == moe::kDropNone   ? launch_dropout<T, true, moe::kDropNone>(P, flat, st)
           : mode == moe::kDropDraw ? launch_dropout<T, true, moe::kDropDraw>(P, flat, st)
                                    : launch_dropout<T, true, moe::kDropAll>(P, flat, st);
  return mode == moe::kDropNone   ? launch_dropout<T, false, moe::kDropNone>(P, flat, st)
         : mode == moe::kDropDraw ? launch_dropout<T, false, moe::kDropDraw>(P, flat, st)
                                  : launch_dropout<T, false, moe::kDropAll>(P, flat, st);
}

int dropout_run(int dtype, int64_t rows, int64_t cols, const void* x, int64_t ldx,
                const void* residual, int64_t ldr, double p, const uint64_t* rng, void* out,
                int64_t ldo, void* stream) {
  const int es = dtype_size(dtype);
  if (!es) return set_error(MOE_INVALID_ARG, "unknown dtype");
  if (const char* m = check_rows(rows, cols)) return set_error(MOE_INVALID_ARG, m);
  if (!(p >= 0.0 && p <= 1.0)) return set_error(MOE_INVALID_ARG, "p must lie in [0, 1]");
  if (rows > (1LL << 40) || cols > (1LL << 40) || (rows > 0 && cols > (1LL << 45) / rows))
    return set_error(MOE_UNSUPPORTED, "dropout needs at most 2^45 elements");
  if (rows == 0) return MOE_OK;
  if (!x || !out) return set_error(MOE_INVALID_ARG, "input and output must be non-null");
  if (bad_stride(rows, cols, ldx) || bad_stride(rows, cols, ldo) ||
      (residual && bad_stride(rows, cols, ldr)))
    return set_error(MOE_INVALID_ARG, "a row stride is smaller than cols");
  if (!aligned(x, es) || !aligned(out, es) || (residual && !aligned(residual, es)))
    return set_error(MOE_INVALID_ARG, "a tensor is not aligned to its elements");
  if (rows == 1) ldx = ldo = ldr = cols;
  moe::DropoutParams P = {};
  P.x = x;
  P.residual = residual;
  P.out = out;
  P.n = rows * cols;
  P.cols = cols;
  P.ldx = ldx;
  P.ldr = ldr;
  P.ldo = ldo;
  P.rng = reinterpret_cast<const unsigned long long*>(rng);
  const double t = std::nearbyint(p * 4294967296.0);
  const int mode = t >= 4294967296.0 ? moe::kDropAll : t > 0.0 ? moe::kDropDraw : moe::kDropNone;
  P.threshold = mode == moe::kDropDraw ? static_cast<uint32_t>(t) : 0u;
  P.scale = p < 1.0 ? static_cast<float>(1.0 / (1.0 - p)) : 0.0f;
  if (mode == moe::kDropDraw && (!rng || !aligned(rng, 8)))
    return set_error(MOE_INVALID_ARG, "rng must point to two uint64 on the device when p > 0");
  const bool flat = ldx == cols && ldo == cols && (!residual || ldr == cols) && aligned(x, 16) &&
                    aligned(out, 16) && (!residual || aligned(residual, 16));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = dtype == MOE_DTYPE_BF16
                            ? dropout_typed<__nv_bfloat16>(P, mode, flat, st)
                        : dtype == MOE_DTYPE_FP16 ? dropout_typed<__half>(P, mode, flat, st)
                                                  : dropout_typed<float>(P, mode, flat, st);
  return launch_status(e, "dropout");
}

}  // namespace

extern "C" {

int moe_norm_forward(int kind, int dtype, int wdtype, int64_t rows, int64_t cols, const void* x,
                     int64_t ldx, const void* weight, const void* bias, double eps, void* y,
                     int64_t ldy, float* mean, float* rstd, void* stream) {
  if (int s = check_norm(kind, dtype, wdtype, rows, cols)) return s;
  if (!(eps >= 0.0) || !std::isfinite(eps))
    return set_error(MOE_INVALID_ARG, "eps must be finite and >= 0");
  if (kind == MOE_NORM_RMS && (bias || mean))
    return set_error(MOE_INVALID_ARG, "an RMS norm has no bias and no mean");
  if (rows == 0) return MOE_OK;
  if (!x || !y) return set_error(MOE_INVALID_ARG, "x and y must be non-null");
  if (bad_stride(rows, cols, ldx) || bad_stride(rows, cols, ldy))
    return set_error(MOE_INVALID_ARG, "a row stride is smaller than cols");
  const int es = dtype_size(dtype), ws = dtype_size(wdtype);
  if (!aligned(x, es) || !aligned(y, es) || !aligned(weight, ws) || !aligned(bias, ws) ||
      !aligned(mean, 4) || !aligned(rstd, 4))
    return set_error(MOE_INVALID_ARG, "a tensor is not aligned to its elements");
  moe::NormParams P = {};
  P.x = x;
  P.weight = weight;
  P.bias = bias;
  P.y = y;
  P.mean = mean;
  P.rstd = rstd;
  P.rows = rows;
  P.ldx = ldx;
  P.ldy = ldy;
  P.cols = static_cast<int>(cols);
  P.eps = static_cast<float>(eps);
  P.rms = kind == MOE_NORM_RMS;
  P.wf32 = wdtype == MOE_DTYPE_FP32;
  const bool vec = cols % (16 / es) == 0 && vector_rows(x, rows, ldx, es) &&
                   vector_rows(y, rows, ldy, es) && aligned(weight, 16) && aligned(bias, 16);
  const bool contiguous = ldx == cols && aligned(x, 16);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  moe::OpsDevice d;
  if (int s = moe::ops_device(&d)) return s;
  const cudaError_t e = dtype == MOE_DTYPE_BF16
                            ? norm_forward_any<__nv_bfloat16>(P, vec, contiguous, d, st)
                        : dtype == MOE_DTYPE_FP16
                            ? norm_forward_any<__half>(P, vec, contiguous, d, st)
                            : norm_forward_any<float>(P, vec, contiguous, d, st);
  return launch_status(e, "norm forward");
}

size_t moe_norm_workspace_bytes(int kind, int64_t rows, int64_t cols) {
  if (check_norm(kind, MOE_DTYPE_FP32, MOE_DTYPE_FP32, rows, cols) != MOE_OK) return 0;
  const int64_t blocks = rows < kNormBlocks ? rows : kNormBlocks;
  return size_t(blocks) * (kind == MOE_NORM_RMS ? 1 : 2) * size_t(cols) * sizeof(float);
}

int moe_norm_backward(int kind, int dtype, int wdtype, int64_t rows, int64_t cols, const void* dy,
                      int64_t lddy, const void* x, int64_t ldx, const void* weight,
                      const float* mean, const float* rstd, void* dx, int64_t lddx, void* dweight,
                      void* dbias, void* workspace, size_t workspace_bytes, void* stream) {
  if (int s = check_norm(kind, dtype, wdtype, rows, cols)) return s;
  if (kind == MOE_NORM_RMS && (dbias || mean))
    return set_error(MOE_INVALID_ARG, "an RMS norm has no bias and no mean");
  if (!dx && !dweight && !dbias) return MOE_OK;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int es = dtype_size(dtype), ws = dtype_size(wdtype);
  if (!aligned(dweight, ws) || !aligned(dbias, ws))
    return set_error(MOE_INVALID_ARG, "a tensor is not aligned to its elements");
  if (rows == 0) {                     // sums over no rows
    cudaError_t e = cudaSuccess;
    if (dweight) e = cudaMemsetAsync(dweight, 0, size_t(cols) * ws, st);
    if (dbias && e == cudaSuccess) e = cudaMemsetAsync(dbias, 0, size_t(cols) * ws, st);
    return launch_status(e, "norm backward");
  }
  if (!dy || !x || !rstd || (kind == MOE_NORM_LAYER && !mean))
    return set_error(MOE_INVALID_ARG, "dy, x, rstd and (layer norm) mean must be non-null");
  if (bad_stride(rows, cols, lddy) || bad_stride(rows, cols, ldx) ||
      (dx && bad_stride(rows, cols, lddx)))
    return set_error(MOE_INVALID_ARG, "a row stride is smaller than cols");
  if (!aligned(dy, es) || !aligned(x, es) || !aligned(dx, es) || !aligned(weight, ws) ||
      !aligned(mean, 4) || !aligned(rstd, 4))
    return set_error(MOE_INVALID_ARG, "a tensor is not aligned to its elements");
  const bool gradw = dweight || dbias;
  if (gradw) {
    if (workspace_bytes < moe_norm_workspace_bytes(kind, rows, cols))
      return set_error(MOE_WORKSPACE_TOO_SMALL, "norm backward: workspace too small");
    if (!workspace || !aligned(workspace, 16))
      return set_error(MOE_INVALID_ARG, "workspace must be non-null and 16-byte aligned");
  }
  moe::NormParams P = {};
  P.x = x;
  P.dy = dy;
  P.weight = weight;
  P.y = dx;
  P.mean = const_cast<float*>(mean);
  P.rstd = const_cast<float*>(rstd);
  P.partial = static_cast<float*>(workspace);
  P.rows = rows;
  P.ldx = ldx;
  P.lddy = lddy;
  P.ldy = lddx;
  P.cols = static_cast<int>(cols);
  P.rms = kind == MOE_NORM_RMS;
  P.wf32 = wdtype == MOE_DTYPE_FP32;
  const bool vec = cols % (16 / es) == 0 && vector_rows(x, rows, ldx, es) &&
                   vector_rows(dy, rows, lddy, es) && (!dx || vector_rows(dx, rows, lddx, es)) &&
                   aligned(weight, 16);
  const bool contiguous = ldx == cols && lddy == cols && aligned(x, 16) && aligned(dy, 16);
  int blocks = 0;
  moe::OpsDevice d;
  if (int s = moe::ops_device(&d)) return s;
  cudaError_t e = dtype == MOE_DTYPE_BF16
                      ? norm_backward_typed<__nv_bfloat16>(P, vec, contiguous, gradw, d, &blocks, st)
                  : dtype == MOE_DTYPE_FP16
                      ? norm_backward_typed<__half>(P, vec, contiguous, gradw, d, &blocks, st)
                      : norm_backward_typed<float>(P, vec, contiguous, gradw, d, &blocks, st);
  if (e == cudaSuccess && gradw) {
    const dim3 grid(unsigned((cols + 31) / 32), dbias ? 2 : 1);
    const int planes = P.rms ? 1 : 2;
    if (wdtype == MOE_DTYPE_FP32)
      e = launch_overlapped(moe::norm_reduce_kernel<float>, grid, dim3(512), 0, st, 1,
                            P.partial, blocks, planes, P.cols, static_cast<float*>(dweight),
                            static_cast<float*>(dbias));
    else if (wdtype == MOE_DTYPE_BF16)
      e = launch_overlapped(moe::norm_reduce_kernel<__nv_bfloat16>, grid, dim3(512), 0, st, 1,
                            P.partial, blocks, planes, P.cols,
                            static_cast<__nv_bfloat16*>(dweight),
                            static_cast<__nv_bfloat16*>(dbias));
    else
      e = launch_overlapped(moe::norm_reduce_kernel<__half>, grid, dim3(512), 0, st, 1, P.partial,
                            blocks, planes, P.cols, static_cast<__half*>(dweight),
                            static_cast<__half*>(dbias));
  }
  return launch_status(e, "norm backward");
}

int moe_dropout_forward(int dtype, int64_t rows, int64_t cols, const void* x, int64_t ldx,
                        const void* residual, int64_t ldr, double p, const uint64_t* rng,
                        void* out, int64_t ldo, void* stream) {
  return dropout_run(dtype, rows, cols, x, ldx, residual, ldr, p, rng, out, ldo, stream);
}

int moe_dropout_backward(int dtype, int64_t rows, int64_t cols, const void* dout, int64_t lddout,
                         double p, const uint64_t* rng, void* dx, int64_t lddx, void* stream) {
  return dropout_run(dtype, rows, cols, dout, lddout, nullptr, 0, p, rng, dx, lddx, stream);
}

}  // extern "C"
