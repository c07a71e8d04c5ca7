// dense_gemm_sm100.cuh - tcgen05 products of the gated feed-forward block, forward and
// backward: D[M, N] = sum over k of A[m, k] B[n, k], where each operand lies in memory
// either with k contiguous (a weight or an activation read along its rows) or with m or n
// contiguous (read along its columns: the transposed operands of the backward pass). Both
// are loaded by TMA with 128-byte swizzle into 64-element slabs; the operand's major-ness
// is a bit of the instruction descriptor and the strides of the shared-memory descriptor,
// so no operand is ever transposed in memory.
//
// One launch runs a list of products (a persistent kernel walks all their tiles):
//   forward   gate/up  A = x (k), B = W1 and W3 (k)     epilogue act(gate) * up; gate, up saved
//             down     A = h (k), B = W2 (k)            plain
//   backward  dh       A = dout (k), B = W2 (n)         epilogue dgate, dup, h
//             dx       A = dgate then dup (k), B = W1 then W3 (n); one reduction over 2f
//             dW1, dW3 A = dgate / dup (m), B = x (n)
//             dW2      A = dout (m), B = h (n)
//
// h, dgate and dup are rounded to 16 bits between the products because they are operands of the
// next. gate and up are none: they are saved in fp32, so that a gradient has one rounding on its
// way beside its own (saved in 16 bits, which takes 470 MB less traffic for 4096 tokens and
// f=14336, the gradients' errors were twice a rounding's). The backward pass computes h again
// from them instead of keeping a third matrix. In fp16 what passes 65504 is infinite.
//
// Warp roles: warp 0 loads A, warp 6 loads B, one thread of warp 1 issues the MMAs,
// warps 2-5 run the epilogue from TMEM while the next tile's MMAs fill the other
// accumulator. PAIR: a cluster of two CTAs computes a 256 x 256 tile (cta_group::2, each
// CTA loads half of A and half of B); otherwise one CTA computes a 128 x 128 tile.
// All waits are bounded (see ptx_sm100.cuh); no load uses cluster multicast.
#pragma once

#include <type_traits>

#include "ops_types.cuh"
#include "ptx_sm100.cuh"

namespace moe {

enum { kGemmPlain = 0, kGemmGluForward = 1, kGemmGluBackward = 2, kGemmGluForwardSave = 3 };
enum { kActSilu = 0, kActGelu = 1 };

constexpr int kDgThreads = 224;
constexpr int kDgMaxProblems = 4;
constexpr int kDgMaxMaps = 14;
constexpr int kDgTileBytes = 16384;                 // one operand's 128 x 64 stage
constexpr int kDgStageBytes = 2 * kDgTileBytes;

// Outputs leave through shared memory: the epilogue warps write a chunk of their tile
// there (swizzled, so that a thread's row does not collide with its neighbours') and one
// thread stores it with TMA, which writes whole lines and clips what lies outside the
// matrix. (Stored from registers, a warp's 16-byte stores went to 32 different rows; the
// dh product of a 4096 x 4096 x 14336 step, which reads two and writes three matrices in
// its epilogue, took 490 us that way.) Plain products use chunks of 64 columns and four
// buffers (with a short reduction, as of the weights' gradients over few tokens, the stores
// are the kernel), gate/up 32 columns and four, with the pre-activations saved 16 columns (one
// buffer of 16 and two of 32 bits) and three, dh 32 columns of three outputs and two.
template <int EPI>
struct DenseCfg {
  static constexpr bool kGlu = EPI == kGemmGluForward || EPI == kGemmGluForwardSave;
  static constexpr bool kSave = EPI == kGemmGluForwardSave;
  static constexpr int kChunk = EPI == kGemmPlain ? 64 : kSave ? 16 : 32;
  static constexpr int kOuts = EPI == kGemmPlain || EPI == kGemmGluForward ? 1 : 3;
  static constexpr int kSets = EPI == kGemmGluBackward ? 2 : kSave ? 3 : 4;
  static constexpr int kStages = 5;
  static constexpr int kBufBytes = 128 * kChunk * 2;            // one 16-bit output's chunk
  // start of output o's chunk in a set (saved ones are twice as large as the first)
  static constexpr int out_at(int o) { return o == 0 ? 0 : kSave ? (2 * o - 1) * kBufBytes : o * kBufBytes; }
  static constexpr int kSetBytes = kSave ? 5 * kBufBytes : kOuts * kBufBytes;
  static constexpr size_t kSmem =
      1024 + size_t(kStages) * kDgStageBytes + kSets * size_t(kSetBytes) + 256;
  static_assert(kSmem <= 227 * 1024, "one block's shared memory");
};

struct DenseProblem {
  int m_tiles, n_tiles, tile0;      // tile0: tiles of the problems before it
  int M, N;                         // rows and columns of D (N: of one of gate / up)
  int kb[2];                        // k-blocks of 64 in the two segments of the reduction
  int map_a[2], map_b[2];           // tensor maps of the segments
  int a_mn, b_mn;                   // 1: m (n) is the contiguous dimension
  int map_out[3];                   // plain: D; gate/up: h, gate, up; dh: h, dgate, dup
};

struct DenseParams {
  DenseProblem p[kDgMaxProblems];
  int n_problems, total_tiles, n_maps;
  int first_tiles;                  // tiles of problem 0 (the costly ones)
  int extra;                        // see tile_of
  const float *gate, *up;           // dh: the saved pre-activations (M, N)
  int act;
  int test_withhold;                // test hook: worker 0 withholds its first stage's copy of A
  int* status;
};

struct DenseMaps {
  CUtensorMap m[kDgMaxMaps];
};

__device__ __forceinline__ void raise_abort(volatile int* s_abort, int* status) {
  *s_abort = 1;
  atomicExch(status, 6);            // MOE_DEVICE_TIMEOUT
}

// The it-th tile of worker w of n. Problem 0's tiles are dealt round-robin; workers left
// with one tile fewer then take `extra` tiles each of the (cheaper) rest, and what remains
// is dealt round-robin again, so a launch whose first product has few, long tiles still
// ends evenly.
__device__ __forceinline__ int tile_of(const DenseParams& P, int w, int n, int it) {
  const int t1 = P.first_tiles;
  const int mine = w < t1 ? (t1 - w + n - 1) / n : 0;
  if (it < mine) return w + it * n;
  int j = it - mine;
  const int rem = t1 % n;
  int base = t1;
  if (P.extra > 0 && rem > 0) {
    const int late = n - rem;       // workers with one long tile fewer
    if (w >= rem) {
      if (j < P.extra) return base + (w - rem) + j * late;
      j -= P.extra;
    }
    base += late * P.extra;
  }
  return base + w + j * n;
}

struct DenseTile {
  int p, m, n;
};

// Tiles of a problem are walked in bands of 8 m-tiles, n outer and m inner, so that the
// tiles running at one time share their operands' slabs through L2.
__device__ __forceinline__ DenseTile decode_dense(const DenseParams& P, int tile) {
  DenseTile t;
  t.p = 0;
#pragma unroll
  for (int i = 1; i < kDgMaxProblems; ++i)
    if (i < P.n_problems && tile >= P.p[i].tile0) t.p = i;
  const DenseProblem& q = P.p[t.p];
  const int local = tile - q.tile0;
  const int band = local / (8 * q.n_tiles);
  const int rows = min(8, q.m_tiles - band * 8);
  const int in_band = local - band * 8 * q.n_tiles;
  t.n = in_band / rows;
  t.m = band * 8 + in_band - t.n * rows;
  return t;
}

// Shared-memory descriptors of 128-byte swizzled slabs, the low and the high word. The
// high word is the same for both orders: stride byte offset 1024 >> 4 (the next 8 rows of
// a k-major tile, the next 8 k of an mn-major one), descriptor version 1, 128-byte
// swizzle. Low word: address >> 4 and the leading byte offset >> 4, which a swizzled
// k-major tile does not use and which in an mn-major tile is the distance of two slabs of
// 64 m or n (64 k x 128 bytes).
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint64_t dense_desc(uint32_t addr, int mn) {
  const uint32_t lo = ((addr & 0x3FFFFu) >> 4) | ((mn ? (8192u >> 4) : 1u) << 16);
  return (static_cast<uint64_t>(kDescHi) << 32) | lo;
}
// Step of the descriptor's address field for the next 16 k.
__device__ __forceinline__ uint32_t dense_kstep(int mn) { return mn ? (2048u >> 4) : (32u >> 4); }

// kind::f16 instruction descriptor: fp32 accumulator (bit 4), A and B format (0 fp16,
// 1 bf16) at 7 and 10, transpose bits 15 (A) and 16 (B) for mn-major operands.
template <typename T>
__device__ __forceinline__ uint32_t dense_idesc(uint32_t M, uint32_t N, int a_mn, int b_mn) {
  constexpr uint32_t fmt = std::is_same<T, __nv_bfloat16>::value ? 1u : 0u;
  return (1u << 4) | (fmt << 7) | (fmt << 10) | (uint32_t(a_mn) << 15) | (uint32_t(b_mn) << 16) |
         ((N >> 3) << 17) | ((M >> 4) << 24);
}

__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.b32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}

// The gate's activation and its derivative, fp32.
//   SiLU: a s(a), s(1 + a (1 - s));   GELU (tanh form): with q = sqrt(2/pi) (a + 0.044715 a^3)
//   and s = 1 / (1 + exp(-2q)) = (1 + tanh q) / 2:  a s,  s + 2 a s (1 - s) q'
__device__ __forceinline__ float act_value(float a, int act) {
  const float z = act == kActSilu ? a : 1.5957691216057308f * (a + 0.044715f * a * a * a);
  return a * __fdividef(1.0f, 1.0f + __expf(-z));
}
// A gate may be as large as fp32 holds, or infinite: below -1e12 it is taken as -1e12, and for
// the derivative above 1e12 as 1e12 (s is exactly 0 or 1 long before), so that 0 times infinity
// does not make a NaN of a gradient that is 0 or 1.
__device__ __forceinline__ void act_value_grad(float a, int act, float& v, float& d) {
  a = a < -1e12f ? -1e12f : a;
  const float b = a > 1e12f ? 1e12f : a;
  const float b2 = b * b;
  const float z = act == kActSilu ? b : 1.5957691216057308f * (b + 0.044715f * b * b2);
  const float dz = act == kActSilu ? 1.0f : 1.5957691216057308f * (1.0f + 0.134145f * b2);
  const float s = __fdividef(1.0f, 1.0f + __expf(-z));
  v = a * s;
  d = s + b * s * (1.0f - s) * dz;
}

template <typename T>
__device__ __forceinline__ uint4 pack8(const float* v) {
  return make_uint4(pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3]), pack2<T>(v[4], v[5]),
                    pack2<T>(v[6], v[7]));
}

// TMA store of one staged chunk, and its bookkeeping (by one thread).
__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, uint32_t src, int32_t x,
                                             int32_t y) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(src), "r"(x), "r"(y)
               : "memory");
}
__device__ __forceinline__ void bulk_commit() {
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void bulk_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void bulk_wait_all() {
  asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}
// Barrier of the four epilogue warps.
__device__ __forceinline__ void epilogue_barrier() {
  asm volatile("bar.sync 1, 128;" ::: "memory");
}

// Byte offset of the 16-byte piece c of row r in a staged chunk (the 128-, 64- or 32-byte TMA
// swizzle for rows of as many bytes).
template <int ROW_BYTES>
__device__ __forceinline__ uint32_t staged(int r, int c) {
  static_assert(ROW_BYTES == 128 || ROW_BYTES == 64 || ROW_BYTES == 32, "a swizzle's row");
  return ROW_BYTES == 128  ? r * 128 + ((c ^ (r & 7)) << 4)
         : ROW_BYTES == 64 ? r * 64 + ((c ^ ((r >> 1) & 3)) << 4)
                           : r * 32 + ((c ^ ((r >> 2) & 1)) << 4);
}
__device__ __forceinline__ void st_shared_16(uint32_t addr, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z),
               "r"(v.w)
               : "memory");
}

template <typename T, int EPI, bool PAIR>
__global__ void __launch_bounds__(kDgThreads, 1)
    dense_gemm_kernel(const __grid_constant__ DenseMaps maps,
                      const __grid_constant__ DenseParams P) {
  using Cfg = DenseCfg<EPI>;
  constexpr int kS = Cfg::kStages;
  constexpr int kTileM = PAIR ? 256 : 128;
  constexpr int kAcc = PAIR ? 256 : 128;            // accumulator columns of a tile
  constexpr int kTmem = 2 * kAcc;
  constexpr bool kGlu = Cfg::kGlu;
  constexpr int kOutCols = kGlu ? kAcc / 2 : kAcc;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* staging = smem + size_t(kS) * kDgStageBytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(staging + Cfg::kSets * Cfg::kSetBytes);
  uint64_t* full_bar = bars;
  uint64_t* empty_bar = bars + kS;
  uint64_t* tfull_bar = bars + 2 * kS;
  uint64_t* tempty_bar = tfull_bar + 2;
  uint64_t* drain_bar = tempty_bar + 2;
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(drain_bar + 1);
  volatile int* s_abort = reinterpret_cast<volatile int*>(s_tmem + 1);
  static_assert((2 * kS + 5) * 8 + 8 <= 256, "barriers fit their 256 bytes");

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = PAIR ? cluster_ctarank() : 0u;
  const bool leader = rank == 0u;
  const int half = PAIR ? static_cast<int>(rank) : 0;
  const int worker = PAIR ? blockIdx.x >> 1 : blockIdx.x;
  const int workers = PAIR ? gridDim.x >> 1 : gridDim.x;

  pdl_launch_dependents();
  if (threadIdx.x == 0) {
    for (int s = 0; s < kS; ++s) {
      mbar_init(smem_u32(&full_bar[s]), 1);
      mbar_init(smem_u32(&empty_bar[s]), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(smem_u32(&tfull_bar[b]), 1);
      mbar_init(smem_u32(&tempty_bar[b]), PAIR ? 256 : 128);
    }
    mbar_init(smem_u32(drain_bar), 1);
    *s_abort = 0;
    fence_mbar_init();
  }
  // the descriptors' first use would otherwise wait for them after the predecessor's end
  if (warp == 6 && lane < P.n_maps) tma_prefetch_desc(&maps.m[lane]);
  if (warp == 1) {
    if (PAIR) {
      tmem_alloc_pair(smem_u32(s_tmem), kTmem);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(smem_u32(s_tmem), kTmem);
      tmem_relinquish();
    }
  }
  tc_fence_before_sync();
  if (PAIR)
    cluster_sync();
  else
    __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem_base = *s_tmem;
  pdl_wait();

  if (warp == 0 || warp == 6) {
    // ------------------------------------------------------------ TMA producers
    if (elect_one()) {
      const bool is_a = warp == 0;
      int s = 0;
      uint32_t ph = 0, issued_mask = 0, issued_par = 0;
      bool ok = true, withhold = P.test_withhold && worker == 0 && leader && is_a;
      for (int it = 0; ok; ++it) {
        const int tile = tile_of(P, worker, workers, it);
        if (tile >= P.total_tiles) break;
        const DenseTile tc = decode_dense(P, tile);
        const DenseProblem& q = P.p[tc.p];
        const int mn = is_a ? q.a_mn : q.b_mn;
        // first m or n of this CTA's 128 rows of the operand
        int row0 = is_a ? tc.m * kTileM + half * 128 : tc.n * kOutCols;
        if (!is_a && PAIR && !kGlu) row0 += half * 128;
        for (int seg = 0; seg < 2 && ok; ++seg) {
          const int nkb = q.kb[seg];
          const CUtensorMap* map =
              &maps.m[is_a ? q.map_a[seg]
                           : (PAIR && kGlu ? q.map_b[half] : q.map_b[seg])];
          const CUtensorMap* map1 = &maps.m[q.map_b[1]];
          for (int kb = 0; kb < nkb; ++kb) {
            ok = mbar_wait(smem_u32(&empty_bar[s]), ph ^ 1u, s_abort);
            if (!ok) break;
            if (withhold) {           // the stage's barrier never completes: all roles give up
              withhold = false;
              s = 1;
              continue;
            }
            uint32_t fb = smem_u32(&full_bar[s]);
            if (is_a && leader) mbar_arrive_expect_tx(fb, (PAIR ? 2 : 1) * kDgStageBytes);
            if (PAIR) fb = mapa_shared(fb, 0);
            const uint32_t dst =
                smem_u32(smem + size_t(s) * kDgStageBytes) + (is_a ? 0 : kDgTileBytes);
            const int k0 = kb * 64;
            if (PAIR) {
              if (mn) {
                tma_load_2d_pair(dst, map, fb, row0, k0);
                tma_load_2d_pair(dst + 8192, map, fb, row0 + 64, k0);
              } else {
                tma_load_2d_pair(dst, map, fb, k0, row0);
              }
            } else if (mn) {
              tma_load_2d(dst, map, fb, row0, k0);
              tma_load_2d(dst + 8192, map, fb, row0 + 64, k0);
            } else if (kGlu && !is_a) {
              tma_load_2d(dst, map, fb, k0, row0);          // 64 rows of W1, 64 of W3
              tma_load_2d(dst + 8192, map1, fb, k0, row0);
            } else {
              tma_load_2d(dst, map, fb, k0, row0);
            }
            issued_mask |= 1u << s;
            issued_par = (issued_par & ~(1u << s)) | (ph << s);
            if (++s == kS) {
              s = 0;
              ph ^= 1u;
            }
          }
        }
      }
      if (!ok) raise_abort(s_abort, P.status);
      // The block keeps its shared memory until its copies have landed, given up or not (also by
      // another role, after this one issued its last): a bounded time. The leader's barriers
      // count both CTAs' copies.
      if (leader)
        for (int i = 0; i < kS; ++i)
          if (issued_mask & (1u << i)) {
            int never = 0;
            mbar_wait(smem_u32(&full_bar[i]), (issued_par >> i) & 1u, &never);
          }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (leader && elect_one()) {
      int s = 0, acc = 0;
      uint32_t ph = 0, acc_ph = 0;
      bool ok = true;
      for (int it = 0; ok; ++it) {
        const int tile = tile_of(P, worker, workers, it);
        if (tile >= P.total_tiles) break;
        const DenseTile tc = decode_dense(P, tile);
        const DenseProblem& q = P.p[tc.p];
        const int a_mn = q.a_mn, b_mn = q.b_mn;
        const uint32_t idesc = dense_idesc<T>(kTileM, kAcc, a_mn, b_mn);
        const uint32_t a_step = dense_kstep(a_mn), b_step = dense_kstep(b_mn);
        const int nkb = q.kb[0] + q.kb[1];
        ok = mbar_wait(smem_u32(&tempty_bar[acc]), acc_ph ^ 1u, s_abort);
        if (!ok) break;
        tc_fence_after_sync();
        const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * kAcc);
        for (int kb = 0; kb < nkb; ++kb) {
          ok = mbar_wait(smem_u32(&full_bar[s]), ph, s_abort);
          if (!ok) break;
          tc_fence_after_sync();
          const uint32_t a_base = smem_u32(smem + size_t(s) * kDgStageBytes);
          const uint64_t a_desc = dense_desc(a_base, a_mn);
          const uint64_t b_desc = dense_desc(a_base + kDgTileBytes, b_mn);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if (PAIR)
              umma_bf16_pair(d_tmem, a_desc + k * a_step, b_desc + k * b_step, idesc,
                             (kb > 0 || k > 0) ? 1u : 0u);
            else
              umma_bf16(d_tmem, a_desc + k * a_step, b_desc + k * b_step, idesc,
                        (kb > 0 || k > 0) ? 1u : 0u);
          }
          if (PAIR)
            umma_commit_pair(smem_u32(&empty_bar[s]));
          else
            umma_commit(smem_u32(&empty_bar[s]));
          if (++s == kS) {
            s = 0;
            ph ^= 1u;
          }
        }
        if (!ok) break;
        if (PAIR)
          umma_commit_pair(smem_u32(&tfull_bar[acc]));
        else
          umma_commit(smem_u32(&tfull_bar[acc]));
        if (++acc == 2) {
          acc = 0;
          acc_ph ^= 1u;
        }
      }
      if (!ok) {
        raise_abort(s_abort, P.status);
        if (PAIR)
          umma_commit_pair(smem_u32(drain_bar));
        else
          umma_commit(smem_u32(drain_bar));
        int never = 0;
        mbar_wait(smem_u32(drain_bar), 0, &never);
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ epilogue
    const int quarter = warp & 3;
    const int r = quarter * 32 + lane;
    const uint32_t lane_base = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16);
    const uint32_t stage0 = smem_u32(staging);
    constexpr int kCh = Cfg::kChunk;
    const bool storer = threadIdx.x == 64;            // first thread of warp 2
    int acc = 0, set = 0;
    uint32_t acc_ph = 0;
    for (int it = 0;; ++it) {
      const int tile = tile_of(P, worker, workers, it);
      if (tile >= P.total_tiles) break;
      const DenseTile tc = decode_dense(P, tile);
      const DenseProblem& q = P.p[tc.p];
      const int rows0 = tc.m * kTileM + half * 128;   // first row of this CTA's part
      const long long row = static_cast<long long>(rows0) + r;
      const bool row_ok = row < q.M;
      const int col0 = tc.n * kOutCols;
      const uint32_t tbase = lane_base + static_cast<uint32_t>(acc * kAcc);
      const int cols = min(kOutCols, q.N - col0);
      // dh: the saved pre-activations of a chunk are loaded one chunk ahead, after the present
      // chunk's have all been used
      float4 g4[8], u4[8];
      auto load_saved = [&](int c, int v) {
        const long long at = row * q.N + col0 + c + v * 8;
        const bool in = row_ok && c + v * 8 < cols;
#pragma unroll
        for (int i = 2 * v; i < 2 * v + 2; ++i) {
          const long long e = at + (i & 1) * 4;
          g4[i] = in ? *reinterpret_cast<const float4*>(P.gate + e) : make_float4(0, 0, 0, 0);
          u4[i] = in ? *reinterpret_cast<const float4*>(P.up + e) : make_float4(0, 0, 0, 0);
        }
      };
      if (EPI == kGemmGluBackward) {
#pragma unroll
        for (int v = 0; v < 4; ++v) load_saved(0, v);
      }
      bool ok = mbar_wait(smem_u32(&tfull_bar[acc]), acc_ph, s_abort);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok && lane == 0) raise_abort(s_abort, P.status);
      // The four warps leave together (they meet at named barriers below): the vote is
      // carried by the barrier itself.
      int all_ok;
      asm volatile(
          "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %1, 0;\n\t"
          "barrier.cta.red.and.pred q, 1, 128, p;\n\tselp.b32 %0, 1, 0, q;\n\t}"
          : "=r"(all_ok)
          : "r"(ok ? 1 : 0)
          : "memory");
      if (!all_ok) break;
      tc_fence_after_sync();
#pragma unroll 1
      for (int c = 0; c < cols; c += kCh) {
        const uint32_t buf = stage0 + set * Cfg::kSetBytes;
        constexpr int kRowBytes = kCh * 2;
        // this set's previous stores (kSets chunks ago) have read it
        auto set_free = [&] {
          if (storer) bulk_wait_read<Cfg::kSets - 1>();
          __syncwarp();
          epilogue_barrier();
        };
        // after the last chunk's loads the accumulator is read: the next tile may have it
        auto release = [&] {
          if (c + kCh < cols) return;
          tc_fence_before_sync();
          if (PAIR && !leader)
            mbar_arrive_cluster(mapa_shared(smem_u32(&tempty_bar[acc]), 0));
          else
            mbar_arrive(smem_u32(&tempty_bar[acc]));
        };
        if constexpr (EPI == kGemmGluForward) {
          uint32_t a[32], u[32];
          tmem_ld_32cols(tbase + c, a);
          tmem_ld_32cols(tbase + kOutCols + c, u);
          tmem_ld_wait();
          release();
          uint4 packed[4];
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            float h[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
              h[j] = act_value(__uint_as_float(a[v * 8 + j]), P.act) *
                     __uint_as_float(u[v * 8 + j]);
            packed[v] = pack8<T>(h);
          }
          set_free();
#pragma unroll
          for (int v = 0; v < 4; ++v) st_shared_16(buf + staged<kRowBytes>(r, v), packed[v]);
        } else if constexpr (EPI == kGemmGluForwardSave) {
          uint32_t a[2][8], u[2][8];
#pragma unroll
          for (int v = 0; v < 2; ++v) {
            tmem_ld_8cols(tbase + c + v * 8, a[v]);
            tmem_ld_8cols(tbase + kOutCols + c + v * 8, u[v]);
          }
          tmem_ld_wait();
          release();
          uint4 packed[2];
#pragma unroll
          for (int v = 0; v < 2; ++v) {
            float h[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
              h[j] = act_value(__uint_as_float(a[v][j]), P.act) * __uint_as_float(u[v][j]);
            packed[v] = pack8<T>(h);
          }
          set_free();
#pragma unroll
          for (int v = 0; v < 2; ++v) st_shared_16(buf + staged<kRowBytes>(r, v), packed[v]);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t* ga = &a[i >> 1][(i & 1) * 4];
            const uint32_t* ua = &u[i >> 1][(i & 1) * 4];
            const uint32_t at = buf + staged<2 * kRowBytes>(r, i);
            st_shared_16(at + Cfg::out_at(1), make_uint4(ga[0], ga[1], ga[2], ga[3]));
            st_shared_16(at + Cfg::out_at(2), make_uint4(ua[0], ua[1], ua[2], ua[3]));
          }
        } else if constexpr (EPI == kGemmGluBackward) {
          uint32_t a[32];
          tmem_ld_32cols(tbase + c, a);
          tmem_ld_wait();
          release();
          uint4 pk[3][4];
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            float dg[8], du[8], h[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float4 gp = g4[2 * v + (j >> 2)], upv = u4[2 * v + (j >> 2)];
              const int k = j & 3;
              const float g = k == 0 ? gp.x : k == 1 ? gp.y : k == 2 ? gp.z : gp.w;
              const float u = k == 0 ? upv.x : k == 1 ? upv.y : k == 2 ? upv.z : upv.w;
              const float dh = __uint_as_float(a[v * 8 + j]);
              float val, der;
              act_value_grad(g, P.act, val, der);
              dg[j] = dh * u * der;
              du[j] = dh * val;
              h[j] = val * u;
            }
            pk[0][v] = pack8<T>(h);
            pk[1][v] = pack8<T>(dg);
            pk[2][v] = pack8<T>(du);
          }
          if (c + kCh < cols) {
#pragma unroll
            for (int v = 0; v < 4; ++v) load_saved(c + kCh, v);
          }
          set_free();
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            const uint32_t at = buf + staged<kRowBytes>(r, v);
            st_shared_16(at, pk[0][v]);
            st_shared_16(at + Cfg::out_at(1), pk[1][v]);
            st_shared_16(at + Cfg::out_at(2), pk[2][v]);
          }
        } else {
          uint4 packed[8];
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
            uint32_t a[32];
            tmem_ld_32cols(tbase + c + hh * 32, a);
            tmem_ld_wait();
#pragma unroll
            for (int v = 0; v < 4; ++v)
              packed[hh * 4 + v] = pack8<T>(reinterpret_cast<const float*>(a) + v * 8);
          }
          release();
          set_free();
#pragma unroll
          for (int v = 0; v < 8; ++v) st_shared_16(buf + staged<kRowBytes>(r, v), packed[v]);
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        epilogue_barrier();
        if (storer) {
          if (rows0 < q.M) {
#pragma unroll
            for (int o = 0; o < Cfg::kOuts; ++o)
              tma_store_2d(&maps.m[q.map_out[o]], buf + Cfg::out_at(o), col0 + c, rows0);
          }
          bulk_commit();
        }
        __syncwarp();
        if (++set == Cfg::kSets) set = 0;
      }
      if (++acc == 2) {
        acc = 0;
        acc_ph ^= 1u;
      }
    }
    if (storer) bulk_wait_all();
    __syncwarp();
  }

  tc_fence_before_sync();
  if (PAIR)
    cluster_sync();
  else
    __syncthreads();
  tc_fence_after_sync();
  if (warp == 1) {
    if (PAIR)
      tmem_dealloc_pair(tmem_base, kTmem);
    else
      tmem_dealloc(tmem_base, kTmem);
  }
}

}  // namespace moe
