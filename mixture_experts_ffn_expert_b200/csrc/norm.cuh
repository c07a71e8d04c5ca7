// norm.cuh - layer norm and RMS norm over the rows of a matrix, forward and backward.
//
//   layer:  xh = (x - mean) * rstd,  rstd = 1 / sqrt(mean((x - mean)^2) + eps)
//   rms:    xh = x * rstd,           rstd = 1 / sqrt(mean(x^2) + eps)
//   y  = xh * weight + bias                       (weight, bias optional)
//   g  = dy * weight
//   dx = rstd * (g - mean(g) - xh * mean(g * xh)) (rms: without mean(g))
//   dweight = sum over rows of dy * xh,   dbias = sum over rows of dy
//
// Both passes are bound by memory: the forward reads x and writes y, the backward reads
// x and dy and writes dx, once each. A row is held in registers between its statistics
// and its output. Statistics, products and sums are fp32; the variance is the mean of
// squared differences from the mean (not a difference of two large sums). Results are
// rounded once, on the store. No atomics: the weight's gradient is summed per thread
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
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int col = (i * group + tid) * VEC;
      if (col < P.cols) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) sum += to_f32(a[i].v[j]);
      }
    }
    mean = group_sum(sum, s_sum[0], warp, group, 1) / n;
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
      for (int c = threadIdx.x; c < P.cols; c += blockDim.x) sum += to_f32(x[c]);
      mean = group_sum(sum, s_sum[0], warp, blockDim.x, 1) / n;
    }
    float sq = 0.0f;
    for (int c = threadIdx.x; c < P.cols; c += blockDim.x) {
      const float v = to_f32(x[c]) - mean;
      sq += v * v;
    }
    const float rstd = 1.0f / sqrtf(group_sum(sq, s_sum[1], warp, blockDim.x, 1) / n + P.eps);
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

// Backward for rows too long for registers: dx (three reads of the row)...
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
