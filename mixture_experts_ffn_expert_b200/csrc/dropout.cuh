// dropout.cuh - dropout with the residual add, its mask drawn from a counter-based
// generator and never stored.
//
//   forward:   out[e] = residual[e] + (keep(e) ? x[e] / (1 - p) : 0)
//   backward:  dx[e]  = keep(e) ? dout[e] / (1 - p) : 0
//   keep(e):   word e % 4 of Philox-4x32-10(counter = (e / 4, offset), key = seed)
//              is at least round(p * 2^32),      e = row * cols + column
//
// Philox-4x32-10 is the generator of Salmon, Moraes, Dror and Shaw, "Parallel
// random numbers: as easy as 1, 2, 3" (SC 2011): ten rounds of two 32 x 32 -> 64 bit
// products and exclusive ors. e / 4 fills the counter's low 64 bits and the offset the
// high 64, so draws with different offsets never share a counter. A dropped element
// contributes exactly zero, whatever it holds (also NaN or an infinity).
#pragma once

#include "ops_types.cuh"
#include "ptx_sm100.cuh"

namespace moe {

__device__ __forceinline__ uint4 philox_4x32_10(uint64_t block, uint64_t offset, uint64_t seed) {
  uint32_t c0 = static_cast<uint32_t>(block), c1 = static_cast<uint32_t>(block >> 32);
  uint32_t c2 = static_cast<uint32_t>(offset), c3 = static_cast<uint32_t>(offset >> 32);
  uint32_t k0 = static_cast<uint32_t>(seed), k1 = static_cast<uint32_t>(seed >> 32);
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t p0 = static_cast<uint64_t>(c0) * 0xD2511F53u;
    const uint64_t p1 = static_cast<uint64_t>(c2) * 0xCD9E8D57u;
    c0 = static_cast<uint32_t>(p1 >> 32) ^ c1 ^ k0;
    c1 = static_cast<uint32_t>(p1);
    c2 = static_cast<uint32_t>(p0 >> 32) ^ c3 ^ k1;
    c3 = static_cast<uint32_t>(p0);
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return make_uint4(c0, c1, c2, c3);
}

struct DropoutParams {
  const void* x;          // x (forward) or dout (backward)
  const void* residual;   // null: none
  void* out;
  long long n, cols;      // rows * cols elements
  long long ldx, ldr, ldo;
  const unsigned long long* rng;   // device: seed, offset
  uint32_t threshold;     // a word below it drops its element (p < 1)
  float scale;            // 1 / (1 - p)
  int mode;               // 0: p = 0, nothing dropped; 1: draw; 2: p = 1, all dropped
};

// Contiguous tensors (each row stride equal to cols): the batch is one line of n
// elements, whatever cols is. A thread takes one 16-byte vector (2 Philox blocks of a
// 16-bit type, 1 of fp32) per step.
template <typename T, bool RES>
__global__ void __launch_bounds__(256) dropout_flat_kernel(const DropoutParams P) {
  constexpr int V = 16 / sizeof(T);
  pdl_launch_dependents();
  pdl_wait();
  const T* x = static_cast<const T*>(P.x);
  const T* res = static_cast<const T*>(P.residual);
  T* out = static_cast<T*>(P.out);
  const uint64_t seed = P.mode == 1 ? P.rng[0] : 0, offset = P.mode == 1 ? P.rng[1] : 0;
  const long long nvec = P.n / V;
  const long long stride = static_cast<long long>(gridDim.x) * blockDim.x;
  const long long first = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x;
  for (long long i = first; i < nvec; i += stride) {
    const Pack<T, V> a = load_pack<T, V>(x + i * V);
    Pack<T, V> r;
    if (RES) r = load_pack<T, V>(res + i * V);
    Pack<T, V> o;
#pragma unroll
    for (int b = 0; b < V / 4; ++b) {
      uint4 w = make_uint4(0, 0, 0, 0);
      if (P.mode == 1) w = philox_4x32_10(i * (V / 4) + b, offset, seed);
      const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const bool keep = P.mode == 0 || (P.mode == 1 && ws[j] >= P.threshold);
        float v = keep ? to_f32(a.v[4 * b + j]) * P.scale : 0.0f;
        if (RES) v += to_f32(r.v[4 * b + j]);
        o.v[4 * b + j] = from_f32<T>(v);
      }
    }
    store_pack<T, V>(out + i * V, o);
  }
  // the last n % V elements, one a thread
  const long long tail = nvec * V + first;
  if (tail < P.n) {
    uint4 w = make_uint4(0, 0, 0, 0);
    if (P.mode == 1) w = philox_4x32_10(tail >> 2, offset, seed);
    const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
    const bool keep = P.mode == 0 || (P.mode == 1 && ws[tail & 3] >= P.threshold);
    float v = keep ? to_f32(x[tail]) * P.scale : 0.0f;
    if (RES) v += to_f32(res[tail]);
    out[tail] = from_f32<T>(v);
  }
}

// Any strides and alignment: a thread takes the four elements of one Philox block,
// element by element.
template <typename T, bool RES>
__global__ void __launch_bounds__(256) dropout_strided_kernel(const DropoutParams P) {
  pdl_launch_dependents();
  pdl_wait();
  const T* x = static_cast<const T*>(P.x);
  const T* res = static_cast<const T*>(P.residual);
  T* out = static_cast<T*>(P.out);
  const uint64_t seed = P.mode == 1 ? P.rng[0] : 0, offset = P.mode == 1 ? P.rng[1] : 0;
  const long long nblk = (P.n + 3) / 4;
  const long long stride = static_cast<long long>(gridDim.x) * blockDim.x;
  for (long long i = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x; i < nblk;
       i += stride) {
    uint4 w = make_uint4(0, 0, 0, 0);
    if (P.mode == 1) w = philox_4x32_10(i, offset, seed);
    const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
    long long row = (4 * i) / P.cols, col = 4 * i - row * P.cols;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (4 * i + j >= P.n) break;
      const bool keep = P.mode == 0 || (P.mode == 1 && ws[j] >= P.threshold);
      float v = keep ? to_f32(x[row * P.ldx + col]) * P.scale : 0.0f;
      if (RES) v += to_f32(res[row * P.ldr + col]);
      out[row * P.ldo + col] = from_f32<T>(v);
      if (++col == P.cols) {
        col = 0;
        ++row;
      }
    }
  }
}

}  // namespace moe
