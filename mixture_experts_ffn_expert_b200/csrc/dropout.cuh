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

// Seed and offset, the same in every thread: told to the compiler by the shuffle, so that
// the key schedule is uniform arithmetic and not part of each thread's.
struct PhiloxKey {
  uint32_t k0, k1, o0, o1;
};
__device__ __forceinline__ PhiloxKey load_philox_key(const unsigned long long* rng) {
  const unsigned long long seed = rng[0], offset = rng[1];
  PhiloxKey k;
  k.k0 = __shfl_sync(0xffffffffu, static_cast<uint32_t>(seed), 0);
  k.k1 = __shfl_sync(0xffffffffu, static_cast<uint32_t>(seed >> 32), 0);
  k.o0 = __shfl_sync(0xffffffffu, static_cast<uint32_t>(offset), 0);
  k.o1 = __shfl_sync(0xffffffffu, static_cast<uint32_t>(offset >> 32), 0);
  return k;
}

__device__ __forceinline__ uint4 philox_4x32_10(uint32_t c0, uint32_t c1, const PhiloxKey& key) {
  uint32_t c2 = key.o0, c3 = key.o1;
  uint32_t k0 = key.k0, k1 = key.k1;
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
  long long n, cols;      // rows * cols elements (of this launch)
  uint32_t block_lo, block_hi;     // flat: Philox block of the launch's first element
  long long ldx, ldr, ldo;
  const unsigned long long* rng;   // device: seed, offset
  uint32_t threshold;     // a word below it drops its element (kDropDraw)
  float scale;            // 1 / (1 - p)
};

// p = 0 keeps all, p = 1 drops all; only what lies between draws.
enum { kDropNone = 0, kDropDraw = 1, kDropAll = 2 };

template <int MODE>
__device__ __forceinline__ bool drop_keeps(uint32_t word, uint32_t threshold) {
  return MODE == kDropNone || (MODE == kDropDraw && word >= threshold);
}

// One element, any type and mode.
template <typename T, bool RES, int MODE>
__device__ __forceinline__ T drop_element(const DropoutParams& P, T x, T res, uint32_t word) {
  const float v = drop_keeps<MODE>(word, P.threshold) ? to_f32(x) : 0.0f;
  return from_f32<T>(RES ? fmaf(v, P.scale, to_f32(res)) : v * P.scale);
}

// One 16-byte vector: its mask, product and sum.
template <typename T, bool RES, int MODE>
__device__ __forceinline__ uint4 drop_vector(const DropoutParams& P, uint32_t i,
                                             const PhiloxKey& key, const uint4& a,
                                             const uint4& r) {
  const uint32_t av[4] = {a.x, a.y, a.z, a.w}, rv[4] = {r.x, r.y, r.z, r.w};
  uint32_t ov[4];
  if constexpr (sizeof(T) == 4) {
    uint4 w = make_uint4(0, 0, 0, 0);
    if (MODE == kDropDraw) w = philox_4x32_10(P.block_lo + i, P.block_hi, key);
    const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int j = 0; j < 4; ++j)
      ov[j] = __float_as_uint(drop_element<float, RES, MODE>(
          P, __uint_as_float(av[j]), __uint_as_float(RES ? rv[j] : 0u), ws[j]));
  } else {
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      uint4 w = make_uint4(0, 0, 0, 0);
      if (MODE == kDropDraw) w = philox_4x32_10(P.block_lo + 2 * i + b, P.block_hi, key);
      const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float2 x2 = unpack2<T>(av[2 * b + h]);
        const float lo = drop_keeps<MODE>(ws[2 * h], P.threshold) ? x2.x : 0.0f;
        const float hi = drop_keeps<MODE>(ws[2 * h + 1], P.threshold) ? x2.y : 0.0f;
        float2 r2 = make_float2(0.0f, 0.0f);
        if (RES) r2 = unpack2<T>(rv[2 * b + h]);
        ov[2 * b + h] = RES ? pack2<T>(fmaf(lo, P.scale, r2.x), fmaf(hi, P.scale, r2.y))
                            : pack2<T>(lo * P.scale, hi * P.scale);
      }
    }
  }
  return make_uint4(ov[0], ov[1], ov[2], ov[3]);
}

// Contiguous tensors (each row stride equal to cols): the batch is one line of n
// elements, whatever cols is. A launch covers at most 2^33 of them, so that the Philox
// block's high word is one number for the launch: with it and the offset uniform, the
// first two rounds have one product a thread each instead of two. A block of 256 threads
// takes VPT * 256 consecutive 16-byte vectors, a thread VPT of them 256 apart, all loaded
// before the first is used. The kernel is bound by the integer and fp32 pipes about as
// much as by memory (18 wide products and 20 exclusive ors for 4 elements): 8192 x 7168
// bf16 forward and backward took 155 us at one vector a thread with the key schedule in
// every thread, 113 us at four with it uniform.
constexpr long long kDropSlice = 1LL << 33;
template <typename T, bool RES, int MODE, int VPT>
__global__ void __launch_bounds__(256, 4) dropout_flat_kernel(const DropoutParams P) {
  constexpr int V = 16 / sizeof(T);
  pdl_wait();
  pdl_launch_dependents();
  const T* x = static_cast<const T*>(P.x);
  const T* res = static_cast<const T*>(P.residual);
  T* out = static_cast<T*>(P.out);
  PhiloxKey key = {};
  if (MODE == kDropDraw) key = load_philox_key(P.rng);
  const uint32_t nvec = static_cast<uint32_t>(P.n / V);
  const uint32_t base = blockIdx.x * (256 * VPT) + threadIdx.x;
  uint4 a[VPT], r[VPT];
#pragma unroll
  for (int k = 0; k < VPT; ++k) {
    const uint32_t i = base + k * 256;
    if (i < nvec) {
      a[k] = reinterpret_cast<const uint4*>(x)[i];
      if (RES) r[k] = reinterpret_cast<const uint4*>(res)[i];
    }
  }
#pragma unroll
  for (int k = 0; k < VPT; ++k) {
    const uint32_t i = base + k * 256;
    if (i < nvec)
      reinterpret_cast<uint4*>(out)[i] = drop_vector<T, RES, MODE>(P, i, key, a[k], r[k]);
  }
  // the last n % V elements, by the first block
  const long long tail = static_cast<long long>(nvec) * V + threadIdx.x;
  if (blockIdx.x == 0 && tail < P.n) {
    uint4 w = make_uint4(0, 0, 0, 0);
    if (MODE == kDropDraw)
      w = philox_4x32_10(P.block_lo + static_cast<uint32_t>(tail >> 2), P.block_hi, key);
    const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
    out[tail] = drop_element<T, RES, MODE>(P, x[tail], RES ? res[tail] : x[tail], ws[tail & 3]);
  }
}

// Any strides and alignment: a thread takes the four elements of one Philox block,
// element by element, with one 64-bit division for the block's row (8192 x 7168 bf16, rows
// padded or starting at an odd element: 178 us forward and 154 backward, where the contiguous
// kernel takes 55 and 51; 777 x 1001 fp32 4.7 and 2.7). It is there so that no layout is refused;
// a program that draws over large padded tensors is better off with contiguous ones.
template <typename T, bool RES, int MODE>
__global__ void __launch_bounds__(256) dropout_strided_kernel(const DropoutParams P) {
  pdl_wait();
  pdl_launch_dependents();
  const T* x = static_cast<const T*>(P.x);
  const T* res = static_cast<const T*>(P.residual);
  T* out = static_cast<T*>(P.out);
  PhiloxKey key = {};
  if (MODE == kDropDraw) key = load_philox_key(P.rng);
  const long long nblk = (P.n + 3) / 4;
  const long long stride = static_cast<long long>(gridDim.x) * blockDim.x;
  for (long long i = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x; i < nblk;
       i += stride) {
    uint4 w = make_uint4(0, 0, 0, 0);
    if (MODE == kDropDraw) w = philox_4x32_10(static_cast<uint32_t>(i), static_cast<uint32_t>(i >> 32), key);
    const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
    long long row = (4 * i) / P.cols, col = 4 * i - row * P.cols;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (4 * i + j >= P.n) break;
      const T a = x[row * P.ldx + col];
      out[row * P.ldo + col] =
          drop_element<T, RES, MODE>(P, a, RES ? res[row * P.ldr + col] : a, ws[j]);
      if (++col == P.cols) {
        col = 0;
        ++row;
      }
    }
  }
}

}  // namespace moe
