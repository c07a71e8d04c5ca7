// norm.cuh - layer norm and RMS norm over the rows of a matrix, forward and backward.
//
//   layer:  xh = (x - mean) * rstd,  rstd = 1 / sqrt(mean((x - mean)^2) + eps)
//   rms:    xh = x * rstd,           rstd = 1 / sqrt(mean(x^2) + eps)
//   y  = xh * weight + bias                       (weight, bias optional)
//   g  = dy * weight
//   dx = rstd * (g - mean(g) - xh * mean(g * xh)) (rms: without mean(g))
//   dweight = sum over rows of dy * xh,   dbias = sum over rows of dy
//
// Both passes are to be bound by memory: the forward reads x and writes y, the backward
// reads x and dy and writes dx, once each. A row is held in registers (few rows) or shared
// memory (many) between its statistics and its output; only rows too long for either are
// read again. Statistics, products and sums are fp32. The mean is summed as differences
// from an element of the row, p, the median of its first, middle and last (so that one element
// far from the others is not taken): mean = p + sum(x - p) / cols. A sum of the elements
// themselves is off by several steps of a large mean, and of a constant row of 123456.79 made
// 0.93 instead of 0; the differences' sum is off by parts of the row's spread only, so the
// mean is, but for that, the nearest fp32 value. The variance is the mean of squared
// differences from the mean (not a difference of two large sums). Results are rounded once,
// on the store. No atomics: the weight's gradient is summed per thread
// over the rows a block walks, then over the blocks in a fixed order, so equal inputs
// give equal bits.
#pragma once

#include "ops_types.cuh"
#include "ptx_sm100.cuh"

namespace moe {

struct NormParams {
  const void* x;
  const void* dy;
  const void* weight;   // null: 1
  const void* bias;     // null: 0
  void* y;              // y (forward) or dx (backward; null: not wanted)
  float* mean;          // forward: written when non-null; backward: read (layer)
  float* rstd;
  float* partial;       // backward: (blocks, 2, cols) or, for rms, (blocks, 1, cols)
  long long rows, ldx, lddy, ldy;
  int cols;
  float eps;
  int rms;
  int wf32;             // weight and bias are fp32 (else of x's type)
};

// VEC consecutive weights (or biases) as fp32.
template <typename T, int VEC>
__device__ __forceinline__ void load_weight(float (&w)[VEC], const void* p, int wf32, int col,
                                            float none) {
  if (!p) {
#pragma unroll
    for (int j = 0; j < VEC; ++j) w[j] = none;
  } else if (wf32) {
    const float* q = static_cast<const float*>(p) + col;
    if constexpr (VEC % 4 == 0) {
#pragma unroll
      for (int j = 0; j < VEC; j += 4) {
        const float4 v = *reinterpret_cast<const float4*>(q + j);
        w[j] = v.x;
        w[j + 1] = v.y;
        w[j + 2] = v.z;
        w[j + 3] = v.w;
      }
    } else {
#pragma unroll
      for (int j = 0; j < VEC; ++j) w[j] = q[j];
    }
  } else {
    const Pack<T, VEC> v = load_pack<T, VEC>(static_cast<const T*>(p) + col);
#pragma unroll
    for (int j = 0; j < VEC; ++j) w[j] = to_f32(v.v[j]);
  }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// The value that a row's elements are taken from while its mean is summed: the median of three
// of them (0 where that is no number, so that the mean of a row with an infinity is what its sum
// says).
__device__ __forceinline__ float row_pivot(float a, float b, float c) {
  const float p = fmaxf(fminf(a, b), fminf(fmaxf(a, b), c));
  return isfinite(p) ? p : 0.0f;
}
template <typename T>
__device__ __forceinline__ float row_pivot(const T* x, int cols) {
  return row_pivot(to_f32(x[0]), to_f32(x[cols >> 1]), to_f32(x[cols - 1]));
}

// Sum over the `threads` threads of one row group (a multiple of 32; named barrier
// `bar`). `slot` holds one float a warp and is used once per barrier, so two calls in a
// row take two slots.
__device__ __forceinline__ float group_sum(float v, float* slot, int warp_in_group, int threads,
                                           int bar) {
  v = warp_sum(v);
  if (threads == 32) return v;
  const int lane = threadIdx.x & 31;
  if (lane == 0) slot[warp_in_group] = v;
  asm volatile("bar.sync %0, %1;" ::"r"(bar), "r"(threads) : "memory");
  v = lane < (threads >> 5) ? slot[lane] : 0.0f;
  return warp_sum(v);
}

// Forward, one row per group of `group` threads (a warp or the block), its columns in
// registers: VPT packs of VEC elements a thread.
template <typename T, int VEC, int VPT>
__global__ void __launch_bounds__(1024) norm_forward_kernel(const NormParams P, int group) {
  __shared__ float s_sum[2][32];
  pdl_launch_dependents();
  pdl_wait();
  const int per_block = blockDim.x / group;
  const int tid = threadIdx.x % group;
  const int warp = tid >> 5;
  const long long row = static_cast<long long>(blockIdx.x) * per_block + threadIdx.x / group;
  if (row >= P.rows) return;          // whole groups leave together
  const T* x = static_cast<const T*>(P.x) + row * P.ldx;
  Pack<T, VEC> a[VPT];
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int col = (i * group + tid) * VEC;
    if (col < P.cols) a[i] = load_pack<T, VEC>(x + col);
  }
  float mean = 0.0f;
  const float n = static_cast<float>(P.cols);
  if (!P.rms) {
    const float pivot = row_pivot(x, P.cols);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int col = (i * group + tid) * VEC;
      if (col < P.cols) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) sum += to_f32(a[i].v[j]) - pivot;
      }
    }
    mean = pivot + group_sum(sum, s_sum[0], warp, group, 1) / n;
  }
  float sq = 0.0f;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int col = (i * group + tid) * VEC;
    if (col < P.cols) {
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const float c = to_f32(a[i].v[j]) - mean;
        sq += c * c;
      }
    }
  }
  const float rstd = 1.0f / sqrtf(group_sum(sq, s_sum[1], warp, group, 1) / n + P.eps);
  if (tid == 0) {
    if (P.mean) P.mean[row] = mean;
    if (P.rstd) P.rstd[row] = rstd;
  }
  T* y = static_cast<T*>(P.y) + row * P.ldy;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int col = (i * group + tid) * VEC;
    if (col < P.cols) {
      float w[VEC], b[VEC];
      load_weight<T, VEC>(w, P.weight, P.wf32, col, 1.0f);
      load_weight<T, VEC>(b, P.bias, P.wf32, col, 0.0f);
      Pack<T, VEC> o;
#pragma unroll
      for (int j = 0; j < VEC; ++j)
        o.v[j] = from_f32<T>((to_f32(a[i].v[j]) - mean) * rstd * w[j] + b[j]);
      store_pack<T, VEC>(y + col, o);
    }
  }
}

// Forward for rows too long for registers: three passes over the row, any alignment.
template <typename T>
__global__ void __launch_bounds__(1024) norm_forward_long_kernel(const NormParams P) {
  __shared__ float s_sum[2][32];
  pdl_launch_dependents();
  pdl_wait();
  const int warp = threadIdx.x >> 5;
  const float n = static_cast<float>(P.cols);
  for (long long row = blockIdx.x; row < P.rows; row += gridDim.x) {
    const T* x = static_cast<const T*>(P.x) + row * P.ldx;
    T* y = static_cast<T*>(P.y) + row * P.ldy;
    float mean = 0.0f;
    if (!P.rms) {
      float sum = 0.0f;
      const float pivot = row_pivot(x, P.cols);
      for (int c = threadIdx.x; c < P.cols; c += blockDim.x) sum += to_f32(x[c]) - pivot;
      mean = pivot + group_sum(sum, s_sum[0], warp, blockDim.x, 1) / n;
    }
    float sq = 0.0f;
    for (int c = threadIdx.x; c < P.cols; c += blockDim.x) {
      const float v = to_f32(x[c]) - mean;
      sq += v * v;
    }
    // divided before the threads' sums meet: the sum of a long row's squares may pass fp32's
    // range where their mean does not
    const float rstd = 1.0f / sqrtf(group_sum(sq / n, s_sum[1], warp, blockDim.x, 1) + P.eps);
    if (threadIdx.x == 0) {
      if (P.mean) P.mean[row] = mean;
      if (P.rstd) P.rstd[row] = rstd;
    }
    for (int c = threadIdx.x; c < P.cols; c += blockDim.x) {
      float w[1], b[1];
      load_weight<T, 1>(w, P.weight, P.wf32, c, 1.0f);
      load_weight<T, 1>(b, P.bias, P.wf32, c, 0.0f);
      y[c] = from_f32<T>((to_f32(x[c]) - mean) * rstd * w[0] + b[0]);
    }
    __syncthreads();                  // s_sum is free for the next row
  }
}

// Backward. A block holds blockDim.x / group row groups; each walks rows group-wise with
// a fixed set of columns a thread, so the weight's and the bias's gradients are sums in
// registers. The next row's x and dy are loaded before the current row is reduced. At the
// end the groups add their sums in order in shared memory and the block writes one
// partial row.
template <typename T, int VEC, int VPT, bool RMS, bool GRADW>
__global__ void __launch_bounds__(1024) norm_backward_kernel(const NormParams P, int group) {
  __shared__ float s_sum[2][2][32];
  extern __shared__ float s_acc[];    // [1 + !RMS][cols] when the block has several groups
  pdl_launch_dependents();
  pdl_wait();
  const int groups = blockDim.x / group;
  const int g = threadIdx.x / group, tid = threadIdx.x - g * group;
  const int warp = tid >> 5;
  const int first_slot = (g * group) >> 5;
  float dw[GRADW ? VPT : 1][VEC], db[GRADW && !RMS ? VPT : 1][VEC];
  float w[VPT][VEC];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int col = (i * group + tid) * VEC;
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      if (GRADW) dw[i][j] = 0.0f;
      if (GRADW && !RMS) db[i][j] = 0.0f;
      w[i][j] = 0.0f;
    }
    if (col < P.cols) load_weight<T, VEC>(w[i], P.weight, P.wf32, col, 1.0f);
  }
  const float inv = 1.0f / static_cast<float>(P.cols);
  const long long step = static_cast<long long>(gridDim.x) * groups;
  long long row = static_cast<long long>(blockIdx.x) * groups + g;
  Pack<T, VEC> xa[VPT], ya[VPT];
  float mean = 0.0f, rstd = 0.0f;
  auto load_row = [&](long long r) {
    const T* x = static_cast<const T*>(P.x) + r * P.ldx;
    const T* dy = static_cast<const T*>(P.dy) + r * P.lddy;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int col = (i * group + tid) * VEC;
      if (col < P.cols) {
        xa[i] = load_pack<T, VEC>(x + col);
        ya[i] = load_pack<T, VEC>(dy + col);
      }
    }
    if (!RMS) mean = P.mean[r];
    rstd = P.rstd[r];
  };
  if (row < P.rows) load_row(row);
  for (int it = 0; row < P.rows; row += step, it ^= 1) {
    float xh[VPT][VEC], gy[VPT][VEC];
    float c1 = 0.0f, c2 = 0.0f;
    const float r_std = rstd;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int col = (i * group + tid) * VEC;
      const bool ok = col < P.cols;
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        xh[i][j] = ok ? (to_f32(xa[i].v[j]) - mean) * rstd : 0.0f;
        const float d = ok ? to_f32(ya[i].v[j]) : 0.0f;
        if (GRADW) dw[i][j] += d * xh[i][j];
        if (GRADW && !RMS) db[i][j] += d;
        gy[i][j] = d * w[i][j];
        c1 += gy[i][j];
        c2 += gy[i][j] * xh[i][j];
      }
    }
    if (row + step < P.rows) load_row(row + step);
    if (!P.y) continue;               // uniform: dx is not wanted
    // two values through one barrier; the slots of alternate rows differ, so a warp that
    // is one row ahead does not overwrite what a slower one still reads
    c2 = warp_sum(c2);
    if (!RMS) c1 = warp_sum(c1);
    if (group > 32) {
      const int lane = threadIdx.x & 31;
      if (lane == 0) {
        s_sum[it][0][first_slot + warp] = c2;
        if (!RMS) s_sum[it][1][first_slot + warp] = c1;
      }
      asm volatile("bar.sync %0, %1;" ::"r"(g + 1), "r"(group) : "memory");
      c2 = lane < (group >> 5) ? s_sum[it][0][first_slot + lane] : 0.0f;
      if (!RMS) c1 = lane < (group >> 5) ? s_sum[it][1][first_slot + lane] : 0.0f;
      c2 = warp_sum(c2);
      if (!RMS) c1 = warp_sum(c1);
    }
    c2 *= inv;
    c1 = RMS ? 0.0f : c1 * inv;
    T* dx = static_cast<T*>(P.y) + row * P.ldy;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int col = (i * group + tid) * VEC;
      if (col < P.cols) {
        Pack<T, VEC> o;
#pragma unroll
        for (int j = 0; j < VEC; ++j)
          o.v[j] = from_f32<T>(r_std * (gy[i][j] - c1 - xh[i][j] * c2));
        store_pack<T, VEC>(dx + col, o);
      }
    }
  }
  if (!GRADW) return;
  float* out = P.partial + static_cast<size_t>(blockIdx.x) * (RMS ? 1 : 2) * P.cols;
  for (int k = 0; k < groups; ++k) {
    if (g == k) {
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int col = (i * group + tid) * VEC;
        if (col < P.cols) {
#pragma unroll
          for (int j = 0; j < VEC; ++j) {
            float a = dw[GRADW ? i : 0][j];
            float b = RMS ? 0.0f : db[GRADW && !RMS ? i : 0][j];
            if (k > 0) {
              a += s_acc[col + j];
              if (!RMS) b += s_acc[P.cols + col + j];
            }
            float* dst = k == groups - 1 ? out : s_acc;
            dst[col + j] = a;
            if (!RMS) dst[P.cols + col + j] = b;
          }
        }
      }
    }
    if (groups > 1) __syncthreads();
  }
}

// Backward for rows too long for a block's registers: dx (the row is read twice)...
template <typename T>
__global__ void __launch_bounds__(1024) norm_backward_long_kernel(const NormParams P) {
  __shared__ float s_sum[2][32];
  pdl_launch_dependents();
  pdl_wait();
  const int warp = threadIdx.x >> 5;
  const float inv = 1.0f / static_cast<float>(P.cols);
  for (long long row = blockIdx.x; row < P.rows; row += gridDim.x) {
    const T* x = static_cast<const T*>(P.x) + row * P.ldx;
    const T* dy = static_cast<const T*>(P.dy) + row * P.lddy;
    T* dx = static_cast<T*>(P.y) + row * P.ldy;
    const float mean = P.rms ? 0.0f : P.mean[row], rstd = P.rstd[row];
    float c1 = 0.0f, c2 = 0.0f;
    for (int c = threadIdx.x; c < P.cols; c += blockDim.x) {
      float w[1];
      load_weight<T, 1>(w, P.weight, P.wf32, c, 1.0f);
      const float gy = to_f32(dy[c]) * w[0];
      c1 += gy;
      c2 += gy * (to_f32(x[c]) - mean) * rstd;
    }
    c1 = P.rms ? 0.0f : group_sum(c1, s_sum[0], warp, blockDim.x, 1) * inv;
    c2 = group_sum(c2, s_sum[1], warp, blockDim.x, 1) * inv;
    for (int c = threadIdx.x; c < P.cols; c += blockDim.x) {
      float w[1];
      load_weight<T, 1>(w, P.weight, P.wf32, c, 1.0f);
      const float xh = (to_f32(x[c]) - mean) * rstd;
      dx[c] = from_f32<T>(rstd * (to_f32(dy[c]) * w[0] - c1 - xh * c2));
    }
    __syncthreads();
  }
}
// ... and the partial sums of dweight and dbias: a thread a column, blockIdx.y a set of rows.
template <typename T>
__global__ void __launch_bounds__(256) norm_backward_long_sum_kernel(const NormParams P) {
  pdl_launch_dependents();
  pdl_wait();
  const long long c = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (c >= P.cols) return;
  float dw = 0.0f, db = 0.0f;
  for (long long row = blockIdx.y; row < P.rows; row += gridDim.y) {
    const float d = to_f32(static_cast<const T*>(P.dy)[row * P.lddy + c]);
    const float mean = P.rms ? 0.0f : P.mean[row];
    dw += d * (to_f32(static_cast<const T*>(P.x)[row * P.ldx + c]) - mean) * P.rstd[row];
    db += d;
  }
  float* out = P.partial + static_cast<size_t>(blockIdx.y) * (P.rms ? 1 : 2) * P.cols;
  out[c] = dw;
  if (!P.rms) out[P.cols + c] = db;
}

// ------------------------------------------------------------------ tile kernels
// Many rows: one persistent block an SM walks its share of the rows in tiles of 1 to 32
// rows, as a pipeline of warps over a ring of shared-memory slots:
//   one thread brings tiles in with bulk copies (cp.async.bulk), as far ahead as there are
//     slots, so that the loads in flight depend neither on registers nor on occupancy;
//   8 row warps sum what a row needs along it (8 / rows warps a row, or rows / 8 rows a
//     warp; a lane holds many elements, so shuffles are few) and leave the row's finished
//     statistics in shared memory;
//   the column warps keep their columns' weights, and in the backward pass their
//     gradients, in registers over all rows, and write the output. They are the longer
//     stage and all work on one tile, so nothing that could be done before is left to them.
// Barriers of the ring order them tile by tile (full, summed, free); there is no block-wide
// barrier, so no part waits for another's latency. (With the row spread over a block and
// two block reductions a row, 8192 x 2048 bf16 took 36 us forward; with tiles worked first
// along rows and then along columns by all warps, 18.)
//
// VEC = 16 bytes of elements: rows start on 16-byte boundaries. VEC = 1: contiguous rows of
// any width; a tile is then one run of bytes that is copied from the 16-byte boundary at or
// before it, and its elements are read one by one.
constexpr int kRowWarps = 8;
constexpr int kTileMaxSlots = 8;
constexpr int kTileMaxRows = 32;
constexpr int tile_threads(int column_warps) { return (kRowWarps + column_warps + 1) * 32; }

struct NormTile {
  int rows;                // a tile: 1, 2, 4, 8, 16 or 32
  int slots;
  int group;               // column threads that cover the columns once
  int contiguous;          // rows follow one another: one copy a tile
  uint32_t slot_bytes;     // of one matrix
  uint32_t weight_bytes;   // backward: the weight staged in front of the ring
  int test_withhold;       // test hook: block 0 withholds its first tile's copies
};

struct TileShared {
  uint64_t full[kTileMaxSlots], summed[kTileMaxSlots], free[kTileMaxSlots];
  // a row's finished values: mean and rstd; backward: and the means of g and of g * xh
  float4 stat[kTileMaxSlots][kTileMaxRows];
  float2 part[2][kRowWarps];          // what several row warps sum of one row; alternate tiles
  int abort;
};

// Row warps that share rows meet here between their sums and the rows' statistics.
__device__ __forceinline__ void row_warps_meet() {
  asm volatile("bar.sync 3, %0;" ::"n"(kRowWarps * 32) : "memory");
}

// Wait for a phase of a ring barrier, suspended in the hardware for up to 0.1 ms a try (25
// warps that poll would take the issue slots of those that work). A wait that gives up
// (2 s) marks the block; what follows is garbage in bounds, reported through the status
// word.
__device__ __forceinline__ void tile_wait(uint64_t* bar, uint32_t parity, volatile int* abort,
                                          int* status) {
  const uint32_t addr = smem_u32(bar);
  uint64_t t0 = 0;
  for (;;) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.b32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(addr), "r"(parity), "r"(100000u)
        : "memory");
    if (ok || *abort) return;
    const uint64_t now = global_timer_ns();
    if (t0 == 0) t0 = now;
    if (now - t0 > kWaitLimitNs) {
      *abort = 1;
      atomicExch(status, 6);          // MOE_DEVICE_TIMEOUT
      return;
    }
  }
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes,
                                          uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
          "r"(dst),
      "l"(__cvta_generic_to_global(src)), "r"(bytes), "r"(bar)
      : "memory");
}

// Bytes a tile's first row lies past the start of its slot.
template <typename T, int VEC>
__device__ __forceinline__ uint32_t tile_shift(const NormParams& P, long long row) {
  return VEC == 1 ? static_cast<uint32_t>(row * P.cols * sizeof(T)) & 15u : 0u;
}

// Copies of one matrix's rows [row, row + n) into a slot; returns the bytes that will be
// counted on `bar`. One thread. VEC == 1: the run of bytes is widened to 16-byte
// boundaries, inside the matrix; what lies past the last boundary at its very end (fewer
// than 16 bytes) is copied by hand, before this thread's arrival on the barrier.
template <typename T, int VEC, bool ISSUE>
__device__ __forceinline__ uint32_t tile_copy(const NormParams& P, const NormTile& L,
                                              const void* base, long long ld, long long row, int n,
                                              uint8_t* slot, uint32_t bar) {
  const uint32_t row_bytes = static_cast<uint32_t>(P.cols) * sizeof(T);
  if (VEC == 1) {
    const unsigned long long b0 = static_cast<unsigned long long>(row) * row_bytes;
    const unsigned long long b1 = b0 + static_cast<unsigned long long>(n) * row_bytes;
    const unsigned long long all = static_cast<unsigned long long>(P.rows) * row_bytes;
    const unsigned long long from = b0 & ~15ull;
    const unsigned long long up = (b1 + 15) & ~15ull, last = all & ~15ull;
    const unsigned long long to = up < last ? up : last;
    const uint32_t bytes = to > from ? static_cast<uint32_t>(to - from) : 0u;
    if (ISSUE) {
      const char* src = static_cast<const char*>(base);
      if (bytes) bulk_load(smem_u32(slot), src + from, bytes, bar);
    } else {
      const char* src = static_cast<const char*>(base);
      for (unsigned long long i = to > from ? to : from; i < b1; i += sizeof(T))
        *reinterpret_cast<T*>(slot + (i - from)) = *reinterpret_cast<const T*>(src + i);
    }
    return bytes;
  }
  if (ISSUE) {
    const T* src = static_cast<const T*>(base) + row * ld;
    if (L.contiguous) {
      bulk_load(smem_u32(slot), src, n * row_bytes, bar);
    } else {
      for (int r = 0; r < n; ++r)
        bulk_load(smem_u32(slot) + r * row_bytes, src + r * ld, row_bytes, bar);
    }
  }
  return n * row_bytes;
}

// A thread's VEC elements as pairs of fp32 values (VEC = 1: one pair, its second value 0),
// read from a slot by shared-memory address.
template <int VEC>
constexpr int pairs() {
  return VEC == 1 ? 1 : VEC / 2;
}
template <typename T, int VEC>
__device__ __forceinline__ void ld_tile(f32x2 (&f)[pairs<VEC>()], uint32_t addr) {
  if constexpr (VEC == 1 && sizeof(T) == 4) {
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr));
    f[0] = make2(v, 0.0f);
  } else if constexpr (VEC == 1) {
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr));
    f[0] = make2(unpack2<T>(static_cast<uint32_t>(v)).x, 0.0f);
  } else if constexpr (sizeof(T) == 4) {
    asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];"
                 : "=f"(f[0].x), "=f"(f[0].y), "=f"(f[1].x), "=f"(f[1].y)
                 : "r"(addr));
  } else {
    uint32_t w[4];
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                 : "r"(addr));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 v = unpack2<T>(w[i]);
      f[i] = make2(v.x, v.y);
    }
  }
}
// The pivot of the row that starts at a shared-memory address.
template <typename T>
__device__ __forceinline__ float tile_pivot(uint32_t row, int cols) {
  f32x2 a[1], b[1], c[1];
  ld_tile<T, 1>(a, row);
  ld_tile<T, 1>(b, row + (cols >> 1) * static_cast<uint32_t>(sizeof(T)));
  ld_tile<T, 1>(c, row + (cols - 1) * static_cast<uint32_t>(sizeof(T)));
  return row_pivot(a[0].x, b[0].x, c[0].x);
}
template <typename T, int VEC>
__device__ __forceinline__ void st_out(T* p, const f32x2 (&f)[pairs<VEC>()]) {
  if constexpr (VEC == 1) {
    *p = from_f32<T>(f[0].x);
  } else if constexpr (sizeof(T) == 4) {
    *reinterpret_cast<float4*>(p) = make_float4(f[0].x, f[0].y, f[1].x, f[1].y);
  } else {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      w[i] = pack2<T>(f[i].x, f[i].y);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}
// VEC weights (or biases) as pairs.
template <typename T, int VEC>
__device__ __forceinline__ void load_weight2(f32x2 (&f)[pairs<VEC>()], const void* p, int wf32,
                                             int col, float none) {
  float w[VEC];
  load_weight<T, VEC>(w, p, wf32, col, none);
  if constexpr (VEC == 1) {
    f[0] = make2(w[0], 0.0f);
  } else {
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) f[i] = make2(w[2 * i], w[2 * i + 1]);
  }
}

// This block's rows: [lo, hi).
__device__ __forceinline__ void tile_range(const NormParams& P, long long* lo, long long* hi) {
  *lo = P.rows * blockIdx.x / gridDim.x;
  *hi = P.rows * (blockIdx.x + 1) / gridDim.x;
}

// 1 / sqrt(v), v > 0 (or 0: infinity): rsqrtf (off by at most 2 units in the last place) and one
// step of Newton's method on f(y) = 1 / y^2 - v, y' = y + y (1 - v y^2) / 2, whose own roundings
// then count: at most 4 * 2^-24 in all. The step is left out where v y y could leave the normal
// numbers. (1.0f / sqrtf(v) in its place: 16384 x 128 bf16 RMS forward 8.5 us instead of 7.7.)
__device__ __forceinline__ float inv_sqrt(float v) {
  const float y = rsqrtf(v);
  const float e = fmaf(-0.5f * v * y, y, 0.5f);
  return v > 1e-37f && v < 3e38f ? fmaf(y, e, y) : y;
}

// Vectors of part q of a row of n vectors that wpr warps share in rounds of 32 each.
__device__ __forceinline__ int part_vectors(int n, int wpr, int q) {
  const int round = wpr * 32;
  const int rem = n % round - q * 32;
  return n / round * 32 + min(max(rem, 0), 32);
}

// The block's part of the pipeline that brings tiles in; PLANES matrices (x, and dy) a
// slot. One thread. Returns once every tile has landed.
template <typename T, int VEC, int PLANES>
__device__ __forceinline__ void tile_producer(const NormParams& P, const NormTile& L, uint8_t* ring,
                                              TileShared& sh, long long lo, long long hi, int tiles,
                                              int* status) {
  int s = 0;
  uint32_t ph = 0, issued = 0, last = 0;           // slots in use, parity of their last copy
  for (int t = 0; t < tiles; ++t) {
    tile_wait(&sh.free[s], ph ^ 1u, &sh.abort, status);
    if (*static_cast<volatile int*>(&sh.abort)) break;
    if (t == 0 && L.test_withhold && blockIdx.x == 0) {     // slot 0 never fills: all roles give up
      s = 1;
      continue;
    }
    const long long row = lo + static_cast<long long>(t) * L.rows;
    const int n = static_cast<int>(hi - row < L.rows ? hi - row : L.rows);
    uint8_t* slot = ring + static_cast<size_t>(s) * PLANES * L.slot_bytes;
    const uint32_t bar = smem_u32(&sh.full[s]);
    uint32_t bytes = tile_copy<T, VEC, false>(P, L, P.x, P.ldx, row, n, slot, bar);
    if (PLANES == 2)
      bytes += tile_copy<T, VEC, false>(P, L, P.dy, P.lddy, row, n, slot + L.slot_bytes, bar);
    mbar_arrive_expect_tx(bar, bytes);
    tile_copy<T, VEC, true>(P, L, P.x, P.ldx, row, n, slot, bar);
    if (PLANES == 2)
      tile_copy<T, VEC, true>(P, L, P.dy, P.lddy, row, n, slot + L.slot_bytes, bar);
    issued |= 1u << s;
    last = (last & ~(1u << s)) | (ph << s);
    if (++s == L.slots) {
      s = 0;
      ph ^= 1u;
    }
  }
  // the block keeps its shared memory until the copies have landed, given up or not
  for (int i = 0; i < L.slots; ++i)
    if (issued >> i & 1u) {
      int never = 0;
      tile_wait(&sh.full[i], last >> i & 1u, &never, status);
    }
}

__device__ __forceinline__ void tile_init(const NormTile& L, TileShared& sh, int column_warps) {
  if (threadIdx.x == 0) {
    for (int s = 0; s < L.slots; ++s) {
      mbar_init(smem_u32(&sh.full[s]), 1);
      mbar_init(smem_u32(&sh.summed[s]), L.rows < kRowWarps ? L.rows : kRowWarps);
      mbar_init(smem_u32(&sh.free[s]), column_warps);
    }
    sh.abort = 0;
    fence_mbar_init();
  }
  __syncthreads();
}

template <typename T, int VEC, int VPT, int CW, bool RMS>
__global__ void __launch_bounds__(tile_threads(CW), 1)
    norm_forward_tile_kernel(const NormParams P, const NormTile L, int* status) {
  constexpr int kVecBytes = VEC * static_cast<int>(sizeof(T));
  constexpr int kPairs = pairs<VEC>();
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ TileShared sh;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  tile_init(L, sh, CW);
  pdl_wait();
  pdl_launch_dependents();
  long long lo, hi;
  tile_range(P, &lo, &hi);
  const int tiles = static_cast<int>((hi - lo + L.rows - 1) / L.rows);
  const uint32_t row_bytes = static_cast<uint32_t>(P.cols) * sizeof(T);
  const int n_vec = P.cols / VEC;
  const int wpr = L.rows < kRowWarps ? kRowWarps / L.rows : 1;
  int s = 0;
  uint32_t ph = 0;
  if (warp == kRowWarps + CW) {
    if (lane == 0) tile_producer<T, VEC, 1>(P, L, ring, sh, lo, hi, tiles, status);
  } else if (warp < kRowWarps) {
    // ---- row warps: the sum of this warp's part of its row (as differences from the row's
    // pivot), and the squared differences from the part's own mean. Sums are multiplied by
    // the counts' reciprocals: being differences, they need no exact division.
    const int my_row = warp / wpr, q = warp - my_row * wpr;
    const float inv_n = 1.0f / static_cast<float>(P.cols);
    const float own_n = static_cast<float>(part_vectors(n_vec, wpr, q) * VEC);
    const float own_inv = own_n > 0.0f ? 1.0f / own_n : 0.0f;
    // the elements that the warp lane / q' of this row sums (lane < wpr)
    const float lane_n =
        lane < wpr ? static_cast<float>(part_vectors(n_vec, wpr, lane) * VEC) : 0.0f;
    const float lane_inv = lane_n > 0.0f ? 1.0f / lane_n : 0.0f;
    auto finish = [&](long long row, int r, int slot, float mean, float m2) {
      const float rstd = inv_sqrt(fmaf(m2, inv_n, P.eps));
      if (lane == 0) {
        sh.stat[slot][r] = make_float4(mean, rstd, 0.0f, 0.0f);
        if (!RMS && P.mean) P.mean[row] = mean;
        if (P.rstd) P.rstd[row] = rstd;
      }
    };
    const uint32_t base = smem_u32(ring) + (q * 32 + lane) * kVecBytes;
    const uint32_t step = wpr * 32 * kVecBytes;
    // every lane reads the same number of vectors, the last perhaps beyond the row: masked
    const int rounds = (n_vec + wpr * 32 - 1) / (wpr * 32);
    const bool last = (rounds - 1) * wpr * 32 + q * 32 + lane < n_vec;
    for (int t = 0; t < tiles; ++t) {
      const long long row0 = lo + static_cast<long long>(t) * L.rows;
      tile_wait(&sh.full[s], ph, &sh.abort, status);
      float pivot = 0.0f;
      for (int r = my_row; r < L.rows && row0 + r < hi; r += kRowWarps) {
        const uint32_t x = base + s * L.slot_bytes + tile_shift<T, VEC>(P, row0) + r * row_bytes;
        float sum = 0.0f, part_mean = 0.0f;
        if (!RMS) {
          pivot = tile_pivot<T>(x - (q * 32 + lane) * kVecBytes, P.cols);
          const f32x2 from = make2(-pivot, VEC == 1 ? 0.0f : -pivot);
          f32x2 acc[2] = {{0.0f, 0.0f}, {0.0f, 0.0f}};
          auto add = [&](int k) {
            f32x2 a[kPairs];
            ld_tile<T, VEC>(a, x + k * step);
#pragma unroll
            for (int j = 0; j < kPairs; ++j) acc[j & 1] = add2(acc[j & 1], add2(a[j], from));
          };
#pragma unroll 4
          for (int k = 0; k < rounds - 1; ++k) add(k);
          if (last) add(rounds - 1);
          const f32x2 both = add2(acc[0], acc[1]);
          sum = warp_sum(both.x + both.y);
          part_mean = fmaf(sum, own_inv, pivot);
        }
        const f32x2 shift = make2(-part_mean, VEC == 1 ? 0.0f : -part_mean);
        f32x2 acc[2] = {{0.0f, 0.0f}, {0.0f, 0.0f}};
        auto add = [&](int k) {
          f32x2 a[kPairs];
          ld_tile<T, VEC>(a, x + k * step);
#pragma unroll
          for (int j = 0; j < kPairs; ++j) {
            const f32x2 c = RMS ? a[j] : add2(a[j], shift);
            acc[j & 1] = fma2(c, c, acc[j & 1]);
          }
        };
#pragma unroll 4
        for (int k = 0; k < rounds - 1; ++k) add(k);
        if (last) add(rounds - 1);
        const f32x2 both = add2(acc[0], acc[1]);
        float sq = both.x + both.y;
        sq = warp_sum(sq);
        if (wpr == 1) {
          finish(row0 + r, r, s, part_mean, sq);
        } else if (lane == 0) {
          sh.part[t & 1][warp] = make_float2(sum, sq);
        }
      }
      if (wpr > 1) {
        row_warps_meet();
        if (q == 0 && row0 + my_row < hi) {
          // sum (x - m)^2 = sum (x - m_w)^2 + n_w (m_w - m)^2 over the row's warps w; both
          // means less the pivot
          const float2 p = lane < wpr ? sh.part[t & 1][warp + lane] : make_float2(0.0f, 0.0f);
          const float off = RMS ? 0.0f : warp_sum(p.x) * inv_n;
          const float d = RMS ? 0.0f : p.x * lane_inv - off;
          // (this warp's pivot is that of row my_row, the only row it summed)
          finish(row0 + my_row, my_row, s, off + pivot, warp_sum(fmaf(lane_n * d, d, p.y)));
        }
      }
      __syncwarp();
      if (lane == 0 && q == 0) mbar_arrive(smem_u32(&sh.summed[s]));
      if (++s == L.slots) {
        s = 0;
        ph ^= 1u;
      }
    }
  } else {
    // ---- column warps
    const int ct = threadIdx.x - kRowWarps * 32;
    const int groups = CW * 32 / L.group;
    const int g = ct / L.group, tid = ct - g * L.group;
    f32x2 w[VPT][kPairs], b[RMS ? 1 : VPT][kPairs];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int col = (i * L.group + tid) * VEC;
      if (g < groups && col < P.cols) {
        load_weight2<T, VEC>(w[i], P.weight, P.wf32, col, 1.0f);
        if (!RMS) load_weight2<T, VEC>(b[RMS ? 0 : i], P.bias, P.wf32, col, 0.0f);
      }
    }
    for (int t = 0; t < tiles; ++t) {
      const long long row0 = lo + static_cast<long long>(t) * L.rows;
      const int valid = static_cast<int>(hi - row0 < L.rows ? hi - row0 : L.rows);
      tile_wait(&sh.full[s], ph, &sh.abort, status);
      tile_wait(&sh.summed[s], ph, &sh.abort, status);
      uint32_t x = smem_u32(ring) + s * L.slot_bytes + tile_shift<T, VEC>(P, row0) +
                   g * row_bytes + tid * kVecBytes;
      T* y = static_cast<T*>(P.y) + (row0 + g) * P.ldy + tid * VEC;
#pragma unroll 2
      for (int r0 = 0; r0 < valid; r0 += groups, x += groups * row_bytes, y += groups * P.ldy) {
        const int r = r0 + g;
        if (g < groups && r < valid) {
          const float4 st = sh.stat[s][r];
          const f32x2 shift = make2(-st.x, -st.x), scale = make2(st.y, st.y);
#pragma unroll
          for (int i = 0; i < VPT; ++i) {
            const int col = (i * L.group + tid) * VEC;
            if (col < P.cols) {
              f32x2 a[kPairs];
              ld_tile<T, VEC>(a, x + i * L.group * kVecBytes);
#pragma unroll
              for (int j = 0; j < kPairs; ++j) {
                const f32x2 xh = mul2(RMS ? a[j] : add2(a[j], shift), scale);
                a[j] = RMS ? mul2(xh, w[i][j]) : fma2(xh, w[i][j], b[RMS ? 0 : i][j]);
              }
              st_out<T, VEC>(y + i * L.group * VEC, a);
            }
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&sh.free[s]));
      if (++s == L.slots) {
        s = 0;
        ph ^= 1u;
      }
    }
  }
}

template <typename T, int VEC, int VPT, int CW, bool RMS, bool GRADW>
__global__ void __launch_bounds__(tile_threads(CW), 1)
    norm_backward_tile_kernel(const NormParams P, const NormTile L, int* status) {
  constexpr bool kHold = VPT * VEC <= 8;           // column warps: weights in registers
  constexpr int kVecBytes = VEC * static_cast<int>(sizeof(T));
  constexpr int kPairs = pairs<VEC>();
  extern __shared__ __align__(128) uint8_t smem_tile[];
  __shared__ TileShared sh;
  uint8_t* ring = smem_tile + L.weight_bytes;
  float* ws = reinterpret_cast<float*>(smem_tile);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  tile_init(L, sh, CW);
  pdl_wait();
  pdl_launch_dependents();
  long long lo, hi;
  tile_range(P, &lo, &hi);
  const int tiles = static_cast<int>((hi - lo + L.rows - 1) / L.rows);
  // the weight in shared memory, fp32; the first tiles are on their way meanwhile
  if (warp < kRowWarps + CW) {
    for (int c = threadIdx.x; c < P.cols; c += (kRowWarps + CW) * 32) {
      float v[1];
      load_weight<T, 1>(v, P.weight, P.wf32, c, 1.0f);
      ws[c] = v[0];
    }
    asm volatile("bar.sync 1, %0;" ::"n"((kRowWarps + CW) * 32) : "memory");
  }
  const uint32_t row_bytes = static_cast<uint32_t>(P.cols) * sizeof(T);
  const int n_vec = P.cols / VEC;
  const int wpr = L.rows < kRowWarps ? kRowWarps / L.rows : 1;
  int s = 0;
  uint32_t ph = 0;
  if (warp == kRowWarps + CW) {
    if (lane == 0) tile_producer<T, VEC, 2>(P, L, ring, sh, lo, hi, tiles, status);
    return;
  }
  if (warp < kRowWarps) {
    // ---- row warps: their part of the sums of g * (x - mean) and of g
    const int my_row = warp / wpr, q = warp - my_row * wpr;
    const float inv_n = 1.0f / static_cast<float>(P.cols);
    // lane l holds the statistics of row l of the tile, loaded one tile ahead
    float next_mean = 0.0f, next_rstd = 0.0f;
    auto load_stats = [&](long long row) {
      if (lane < L.rows && row + lane < hi) {
        if (!RMS) next_mean = P.mean[row + lane];
        next_rstd = P.rstd[row + lane];
      }
    };
    load_stats(lo);
    const uint32_t base = smem_u32(ring) + (q * 32 + lane) * kVecBytes;
    const uint32_t step = wpr * 32 * kVecBytes;
    const uint32_t w_base = smem_u32(ws) + (q * 32 + lane) * (VEC * 4);
    const int rounds = (n_vec + wpr * 32 - 1) / (wpr * 32);
    const bool last = (rounds - 1) * wpr * 32 + q * 32 + lane < n_vec;
    for (int t = 0; t < tiles; ++t) {
      const long long row0 = lo + static_cast<long long>(t) * L.rows;
      const float means = next_mean, rstds = next_rstd;
      load_stats(row0 + L.rows);
      tile_wait(&sh.full[s], ph, &sh.abort, status);
      for (int r = my_row; r < L.rows && row0 + r < hi; r += kRowWarps) {
        const float mean = RMS ? 0.0f : __shfl_sync(0xffffffffu, means, r);
        const float rstd = __shfl_sync(0xffffffffu, rstds, r);
        const uint32_t x =
            base + s * 2 * L.slot_bytes + tile_shift<T, VEC>(P, row0) + r * row_bytes;
        const f32x2 shift = make2(-mean, -mean);
        f32x2 s1[2] = {{0.0f, 0.0f}, {0.0f, 0.0f}}, s2[2] = {{0.0f, 0.0f}, {0.0f, 0.0f}};
        auto add = [&](int k) {
          f32x2 a[kPairs], d[kPairs], wv[kPairs];
          ld_tile<T, VEC>(a, x + k * step);
          ld_tile<T, VEC>(d, x + L.slot_bytes + k * step);
          const uint32_t wa = w_base + k * wpr * (32 * VEC * 4);
          if constexpr (VEC == 1) {
            ld_tile<float, 1>(wv, wa);
          } else {
#pragma unroll
            for (int j = 0; j < kPairs; j += 2)
              ld_tile<float, 4>(*reinterpret_cast<f32x2(*)[2]>(wv + j), wa + j * 8);
          }
#pragma unroll
          for (int j = 0; j < kPairs; ++j) {
            const f32x2 gy = mul2(d[j], wv[j]);
            s2[j & 1] = fma2(gy, RMS ? a[j] : add2(a[j], shift), s2[j & 1]);
            if (!RMS) s1[j & 1] = add2(s1[j & 1], gy);
          }
        };
#pragma unroll 2
        for (int k = 0; k < rounds - 1; ++k) add(k);
        if (last) add(rounds - 1);
        const f32x2 b1 = add2(s1[0], s1[1]), b2 = add2(s2[0], s2[1]);
        float c1 = b1.x + b1.y, c2 = b2.x + b2.y;
        c2 = warp_sum(c2) * rstd;
        if (!RMS) c1 = warp_sum(c1);
        if (lane == 0) {
          if (wpr == 1)
            sh.stat[s][r] = make_float4(mean, rstd, c1 * inv_n, c2 * inv_n);
          else
            sh.part[t & 1][warp] = make_float2(c1, c2);
        }
      }
      if (wpr > 1) {
        row_warps_meet();
        if (q == 0 && row0 + my_row < hi) {
          const float2 p = lane < wpr ? sh.part[t & 1][warp + lane] : make_float2(0.0f, 0.0f);
          const float c1 = RMS ? 0.0f : warp_sum(p.x), c2 = warp_sum(p.y);
          const float mean = RMS ? 0.0f : __shfl_sync(0xffffffffu, means, my_row);
          const float rstd = __shfl_sync(0xffffffffu, rstds, my_row);
          if (lane == 0)
            sh.stat[s][my_row] = make_float4(mean, rstd, c1 * inv_n, c2 * inv_n);
        }
      }
      __syncwarp();
      if (lane == 0 && q == 0) mbar_arrive(smem_u32(&sh.summed[s]));
      if (++s == L.slots) {
        s = 0;
        ph ^= 1u;
      }
    }
    return;
  }
  // ---- column warps
  const int ct = threadIdx.x - kRowWarps * 32;
  const int groups = CW * 32 / L.group;
  const int g = ct / L.group, tid = ct - g * L.group;
  const uint32_t w_at = smem_u32(ws) + tid * (VEC * 4);
  auto weights = [&](f32x2 (&f)[kPairs], int i) {
    const uint32_t at = w_at + i * L.group * (VEC * 4);
    if constexpr (VEC == 1) {
      ld_tile<float, 1>(f, at);
    } else {
#pragma unroll
      for (int j = 0; j < kPairs; j += 2)
        ld_tile<float, 4>(*reinterpret_cast<f32x2(*)[2]>(f + j), at + j * 8);
    }
  };
  f32x2 w[kHold ? VPT : 1][kPairs], dw[GRADW ? VPT : 1][kPairs],
      db[GRADW && !RMS ? VPT : 1][kPairs];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    if (kHold && (i * L.group + tid) * VEC < P.cols) weights(w[kHold ? i : 0], i);
#pragma unroll
    for (int j = 0; j < kPairs; ++j) {
      if (GRADW) dw[GRADW ? i : 0][j] = make2(0.0f, 0.0f);
      if (GRADW && !RMS) db[GRADW && !RMS ? i : 0][j] = make2(0.0f, 0.0f);
    }
  }
  for (int t = 0; t < tiles; ++t) {
    const long long row0 = lo + static_cast<long long>(t) * L.rows;
    const int valid = static_cast<int>(hi - row0 < L.rows ? hi - row0 : L.rows);
    tile_wait(&sh.full[s], ph, &sh.abort, status);
    tile_wait(&sh.summed[s], ph, &sh.abort, status);
    uint32_t x = smem_u32(ring) + s * 2 * L.slot_bytes + tile_shift<T, VEC>(P, row0) +
                 g * row_bytes + tid * kVecBytes;
    T* dx = static_cast<T*>(P.y) + (row0 + g) * P.ldy + tid * VEC;
    for (int r0 = 0; r0 < valid; r0 += groups, x += groups * row_bytes, dx += groups * P.ldy) {
      const int r = r0 + g;
      if (g < groups && r < valid) {
        const float4 st = sh.stat[s][r];
        const f32x2 shift = make2(-st.x, -st.x), scale = make2(st.y, st.y);
        const f32x2 minus_c1 = make2(-st.z, -st.z), minus_c2 = make2(-st.w, -st.w);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
          const int col = (i * L.group + tid) * VEC;
          if (col < P.cols) {
            f32x2 a[kPairs], d[kPairs];
            ld_tile<T, VEC>(a, x + i * L.group * kVecBytes);
            ld_tile<T, VEC>(d, x + L.slot_bytes + i * L.group * kVecBytes);
            if (!kHold) weights(w[0], i);
#pragma unroll
            for (int j = 0; j < kPairs; ++j) {
              const f32x2 xh = mul2(RMS ? a[j] : add2(a[j], shift), scale);
              if (GRADW) dw[GRADW ? i : 0][j] = fma2(d[j], xh, dw[GRADW ? i : 0][j]);
              if (GRADW && !RMS) db[GRADW && !RMS ? i : 0][j] = add2(db[GRADW && !RMS ? i : 0][j], d[j]);
              const f32x2 gc = RMS ? mul2(d[j], w[kHold ? i : 0][j])
                                   : fma2(d[j], w[kHold ? i : 0][j], minus_c1);
              a[j] = mul2(scale, fma2(xh, minus_c2, gc));
            }
            if (P.y) st_out<T, VEC>(dx + i * L.group * VEC, a);
          }
        }
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&sh.free[s]));
    if (++s == L.slots) {
      s = 0;
      ph ^= 1u;
    }
  }
  if (!GRADW) return;
  // The groups add their sums in order in shared memory (the ring is free: the column warps
  // have read every tile), and the last writes the block's partial row.
  asm volatile("bar.sync 2, %0;" ::"n"(CW * 32) : "memory");
  float* acc = reinterpret_cast<float*>(ring);
  float* out = P.partial + static_cast<size_t>(blockIdx.x) * (RMS ? 1 : 2) * P.cols;
  for (int k = 0; k < groups; ++k) {
    if (g == k) {
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int col = (i * L.group + tid) * VEC;
        if (col < P.cols) {
#pragma unroll
          for (int j = 0; j < VEC; ++j) {
            const float2 pw = dw[GRADW ? i : 0][j / 2];
            const float2 pb = RMS ? make_float2(0.0f, 0.0f) : db[GRADW && !RMS ? i : 0][j / 2];
            float p = j & 1 ? pw.y : pw.x;
            float q2 = j & 1 ? pb.y : pb.x;
            if (k > 0) {
              p += acc[col + j];
              if (!RMS) q2 += acc[P.cols + col + j];
            }
            float* dst = k == groups - 1 ? out : acc;
            dst[col + j] = p;
            if (!RMS) dst[P.cols + col + j] = q2;
          }
        }
      }
    }
    asm volatile("bar.sync 2, %0;" ::"n"(CW * 32) : "memory");
  }
}

// Sum of the blocks' partial rows: 32 columns a block, 16 threads a column that each walk
// every 16th partial row, added in a fixed order. blockIdx.y picks dweight or dbias.
template <typename W>
__global__ void __launch_bounds__(512) norm_reduce_kernel(const float* partial, int blocks,
                                                          int planes, int cols, W* dweight,
                                                          W* dbias) {
  __shared__ float s[16][33];
  pdl_launch_dependents();
  pdl_wait();
  W* out = blockIdx.y == 0 ? dweight : dbias;
  if (!out) return;                   // uniform over the block
  const int c = threadIdx.x & 31, r = threadIdx.x >> 5;
  const long long col = static_cast<long long>(blockIdx.x) * 32 + c;
  float sum = 0.0f;
  if (col < cols)
    for (int b = r; b < blocks; b += 16)
      sum += partial[(static_cast<size_t>(b) * planes + blockIdx.y) * cols + col];
  s[r][c] = sum;
  __syncthreads();
  if (r == 0 && col < cols) {
#pragma unroll
    for (int k = 1; k < 16; ++k) sum += s[k][c];
    out[col] = from_f32<W>(sum);
  }
}

}  // namespace moe
