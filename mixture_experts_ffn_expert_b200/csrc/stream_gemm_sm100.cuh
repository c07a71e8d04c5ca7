// stream_gemm_sm100.cuh - products of the gated feed-forward block for few tokens, where the
// time is that of reading the weights, and for more tokens where the other kernels' tiles
// would leave SMs idle (a long reduction over few tiles).
//
// The weights are the 128-row operand of tcgen05.mma and the tokens its N columns (16, 32,
// 64 or 128, padded with zeros by TMA; more than 128 tokens are tiled by 128), so up to 128
// tokens a weight tile is read once and the tensor work does not grow with a padded token
// tile. The reduction is split over the CTAs
// of a cluster (1, 2, 4 or 8), as many as it takes to give every SM a stream of its own:
// two CTAs share an SM, each with its own ring of TMA stages, which keeps about 200 KB of
// loads in flight an SM. Every rank finishes an equal share of the tile's rows: each CTA
// stores its fp32 partial rows from TMEM straight into the shared memory of the rank that
// owns them (distributed shared memory), and after a cluster barrier that rank adds them
// in rank order and runs the epilogue (so sums are the same bits every time and no partial
// result goes through global memory). Stores, not loads, cross the cluster: with 128
// tokens the ranks' loads of each other's partial tiles took 4 of the kernel's 11 us.
//
//   gate/up  A = W1 rows 0-63, W3 rows 64-127 of the tile    epilogue act(gate) * up
//   down     A = W2                                          plain
//   dh       A = W2 read along its columns                   epilogue dgate, dup, h
//   dx       A = W1 then W3 read along their columns         plain, one reduction over 2f
#pragma once

#include "dense_gemm_sm100.cuh"

namespace moe {

constexpr int kStreamThreads = 224;
constexpr int kStreamTokens = 128;          // a token tile

template <int NB>
struct StreamCfg {
  static constexpr int kStageBytes = kDgTileBytes + NB * 128;
  static constexpr int kStages = NB <= 16 ? 5 : NB <= 32 ? 4 : 3;
  // Partial rows received from the ranks: an area of their own, or for 128 tokens (where
  // that would leave no room for the stages of a second CTA) the stages, once every rank
  // has finished its MMAs.
  static constexpr bool kOverStages = NB == 128;
  static constexpr int kRedBytes = 128 * NB * 4;
  static constexpr int kTmem = NB < 32 ? 32 : NB;
  static constexpr size_t kSmem =
      1024 + size_t(kStages) * kStageBytes + (kOverStages ? 0 : kRedBytes) + 256;
  static_assert(!kOverStages || kRedBytes <= kStages * kStageBytes, "they fit the stages");
};

struct StreamParams {
  int T, N;                 // tokens; rows of the weights (columns of the output)
  int t_tiles;              // token tiles
  int kb[2];                // k-blocks of 64 in the two segments of the reduction
  int a_mn;                 // weights read along their columns
  int early;                // weights may be loaded before the predecessor has finished
  int act;
  void* out;                // plain: (T, N), rows ldo apart
  long long ldo;
  float *gate, *up;         // the saved pre-activations (T, N); gate/up: null to save none
  void *hidden, *dgate, *dup;
  int test_withhold;        // test hook: block 0 withholds its first stage's weights
  int* status;
};

struct StreamMaps {
  CUtensorMap a[2], b[2];
};

__device__ __forceinline__ void st_cluster_f32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

__device__ __forceinline__ uint32_t cluster_nctarank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}

template <typename T, int EPI, int NB>
__global__ void __launch_bounds__(kStreamThreads, 2)
    stream_gemm_kernel(const __grid_constant__ StreamMaps maps,
                       const __grid_constant__ StreamParams P) {
  using Cfg = StreamCfg<NB>;
  constexpr int kS = Cfg::kStages;
  constexpr int kRows = EPI == kGemmGluForward ? 64 : 128;     // output columns of a tile
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  float* red = reinterpret_cast<float*>(
      smem + (Cfg::kOverStages ? 0 : size_t(kS) * Cfg::kStageBytes));
  uint64_t* full_bar = reinterpret_cast<uint64_t*>(
      smem + size_t(kS) * Cfg::kStageBytes + (Cfg::kOverStages ? 0 : Cfg::kRedBytes));
  uint64_t* empty_bar = full_bar + kS;
  uint64_t* done_bar = empty_bar + kS;
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(done_bar + 1);
  volatile int* s_abort = reinterpret_cast<volatile int*>(s_tmem + 1);
  static_assert((2 * kS + 1) * 8 + 8 <= 256, "barriers fit their 256 bytes");

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int ranks = static_cast<int>(cluster_nctarank());
  const int rank = static_cast<int>(cluster_ctarank());
  // clusters that share a weight tile are neighbours
  const int tile = blockIdx.x / ranks;
  const int row0 = tile / P.t_tiles * kRows;
  const int token0 = tile % P.t_tiles * kStreamTokens;
  const int tokens = min(P.T - token0, kStreamTokens);

  if (threadIdx.x == 0) {
    for (int s = 0; s < kS; ++s) {
      mbar_init(smem_u32(&full_bar[s]), 2);       // the two producers
      mbar_init(smem_u32(&empty_bar[s]), 1);
    }
    mbar_init(smem_u32(done_bar), 1);
    *s_abort = 0;
    fence_mbar_init();
    tma_prefetch_desc(&maps.a[0]);
    tma_prefetch_desc(&maps.b[0]);
    if (EPI == kGemmGluForward || P.kb[1] > 0) tma_prefetch_desc(&maps.a[1]);
    if (P.kb[1] > 0) tma_prefetch_desc(&maps.b[1]);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(s_tmem), Cfg::kTmem);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  cluster_sync();                  // the ranks' shared memory may be written from here on
  tc_fence_after_sync();
  const uint32_t tmem_base = *s_tmem;

  const int total = P.kb[0] + P.kb[1];
  const int kb_lo = static_cast<int>(static_cast<long long>(total) * rank / ranks);
  const int kb_hi = static_cast<int>(static_cast<long long>(total) * (rank + 1) / ranks);

  if (warp == 0 || warp == 6) {
    // ------------------------------------------------------------ TMA producers
    // warp 0 streams the weights, warp 6 the tokens (which the predecessor may have written)
    const bool weights = warp == 0;
    if (!weights || !P.early) pdl_wait();
    if (elect_one()) {
      int s = 0;
      uint32_t ph = 0, issued_mask = 0, issued_par = 0;
      bool ok = true, withhold = P.test_withhold && weights && blockIdx.x == 0;
      for (int kb = kb_lo; kb < kb_hi; ++kb) {
        // the ring is full: its first stage is free only when the tokens have come, and the
        // bounded wait for that must not begin while the predecessor runs
        if (weights && P.early && kb == kb_lo + kS) pdl_wait();
        ok = mbar_wait(smem_u32(&empty_bar[s]), ph ^ 1u, s_abort);
        if (!ok) break;
        if (withhold) {               // the stage's barrier never completes: all roles give up
          withhold = false;
          s = 1;
          continue;
        }
        const int seg = kb >= P.kb[0];
        const int k0 = (seg ? kb - P.kb[0] : kb) * 64;
        const uint32_t fb = smem_u32(&full_bar[s]);
        const uint32_t dst = smem_u32(smem + size_t(s) * Cfg::kStageBytes);
        if (weights) {
          mbar_arrive_expect_tx(fb, kDgTileBytes);
          if (EPI == kGemmGluForward) {
            tma_load_2d(dst, &maps.a[0], fb, k0, row0);
            tma_load_2d(dst + 8192, &maps.a[1], fb, k0, row0);
          } else if (P.a_mn) {
            tma_load_2d(dst, &maps.a[seg], fb, row0, k0);
            tma_load_2d(dst + 8192, &maps.a[seg], fb, row0 + 64, k0);
          } else {
            tma_load_2d(dst, &maps.a[seg], fb, k0, row0);
          }
        } else {
          mbar_arrive_expect_tx(fb, NB * 128);
          tma_load_2d(dst + kDgTileBytes, &maps.b[seg], fb, k0, token0);
        }
        issued_mask |= 1u << s;
        issued_par = (issued_par & ~(1u << s)) | (ph << s);
        if (++s == kS) {
          s = 0;
          ph ^= 1u;
        }
      }
      if (!ok) raise_abort(s_abort, P.status);
      if (weights && P.early) pdl_wait();       // the stages fill only with the tokens
      // The block keeps its shared memory until its copies have landed, given up or not (also by
      // the MMA issuer, after this role issued its last): a bounded time.
      for (int i = 0; i < kS; ++i)
        if (issued_mask & (1u << i)) {
          int never = 0;
          mbar_wait(smem_u32(&full_bar[i]), (issued_par >> i) & 1u, &never);
        }
    }
    __syncwarp();
    if (weights && P.early) pdl_wait();
  } else {
    pdl_wait();
    if (warp == 1 && elect_one()) {
      // ---------------------------------------------------------- MMA issuer
      const uint32_t idesc = dense_idesc<T>(128, NB, P.a_mn, 0);
      const uint32_t a_step = dense_kstep(P.a_mn), b_step = dense_kstep(0);
      int s = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int kb = kb_lo; kb < kb_hi; ++kb) {
        ok = mbar_wait(smem_u32(&full_bar[s]), ph, s_abort);
        if (!ok) break;
        tc_fence_after_sync();
        const uint32_t base = smem_u32(smem + size_t(s) * Cfg::kStageBytes);
        const uint64_t a_desc = dense_desc(base, P.a_mn);
        const uint64_t b_desc = dense_desc(base + kDgTileBytes, 0);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          umma_bf16(tmem_base, a_desc + k * a_step, b_desc + k * b_step, idesc,
                    (kb > kb_lo || k > 0) ? 1u : 0u);
        umma_commit(smem_u32(&empty_bar[s]));
        if (++s == kS) {
          s = 0;
          ph ^= 1u;
        }
      }
      if (!ok) raise_abort(s_abort, P.status);
      umma_commit(smem_u32(done_bar));
    }
    __syncwarp();
  }
  // Dependents may start only now. The trigger fires with a block's first thread here, and any
  // thread that has passed its wait proves that what came before this kernel is complete, so a
  // dependent may read the weights early. (Warp 0 of an early launch may be before its wait.)
  pdl_launch_dependents();

  // ------------------------------------------------------------ partial rows to their owners
  const int share = kRows / ranks;                 // output columns a rank finishes
  const int rows_each = 128 / ranks;               // accumulator rows of those
  const bool finisher = warp >= 2 && warp < 6;
  bool done = false;
  if (finisher) {
    int never = 0;
    done = mbar_wait(smem_u32(done_bar), 0, &never);
    done = __all_sync(0xffffffffu, done);
    if (!done && lane == 0) raise_abort(s_abort, P.status);
    tc_fence_after_sync();
  }
  if (Cfg::kOverStages) cluster_sync();            // all ranks' stages have been read
  if (finisher) {
    if (done) {
      const int quarter = warp & 3;
      const int r = quarter * 32 + lane;           // accumulator row
      const uint32_t lane_base = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16);
      // gate/up: rows 64-127 are the up rows of the owners of rows 0-63
      const int out_row = EPI == kGemmGluForward ? (r & 63) : r;
      const int owner = out_row / share;
      const int local = out_row - owner * share + (EPI == kGemmGluForward && r >= 64 ? share : 0);
      // token by token, so that a warp's store is one run of consecutive words for every
      // owner (16-byte stores of four tokens a lane, a row apart, took twice as long)
      const uint32_t dst =
          mapa_shared(smem_u32(red), owner) + (rank * tokens * rows_each + local) * 4;
#pragma unroll 1
      for (int c = 0; c < tokens; c += 16) {
        uint32_t v[16];
        tmem_ld_8cols(lane_base + c, *reinterpret_cast<uint32_t(*)[8]>(v));
        tmem_ld_8cols(lane_base + c + 8, *reinterpret_cast<uint32_t(*)[8]>(v + 8));
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 16; ++j)
          if (c + j < tokens) st_cluster_f32(dst + (c + j) * rows_each * 4, v[j]);
      }
    }
    tc_fence_before_sync();
  }
  cluster_sync();

  // ------------------------------------------------------------ reduction and epilogue
  // This rank's share of the tile's output columns, four at a time.
  const int quads = share / 4;
  for (int i = threadIdx.x; i < tokens * quads; i += kStreamThreads) {
    const int t = i / quads;
    const int local = (i - t * quads) * 4;
    const int n = row0 + rank * share + local;
    if (n >= P.N) continue;
    const float* part = red + t * rows_each + local;
    float v[4] = {0, 0, 0, 0}, u[4] = {0, 0, 0, 0};
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if (k < ranks) {
        const float4 p = *reinterpret_cast<const float4*>(part + k * tokens * rows_each);
        v[0] += p.x;
        v[1] += p.y;
        v[2] += p.z;
        v[3] += p.w;
        if (EPI == kGemmGluForward) {
          const float4 w = *reinterpret_cast<const float4*>(part + k * tokens * rows_each + share);
          u[0] += w.x;
          u[1] += w.y;
          u[2] += w.z;
          u[3] += w.w;
        }
      }
    }
    if (EPI == kGemmPlain) {
      *reinterpret_cast<uint2*>(static_cast<T*>(P.out) + (token0 + t) * P.ldo + n) =
          make_uint2(pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3]));
    } else if (EPI == kGemmGluForward) {
      const long long at = static_cast<long long>(token0 + t) * P.N + n;
      float h[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) h[j] = act_value(v[j], P.act) * u[j];
      *reinterpret_cast<uint2*>(static_cast<T*>(P.hidden) + at) =
          make_uint2(pack2<T>(h[0], h[1]), pack2<T>(h[2], h[3]));
      if (P.gate) {
        *reinterpret_cast<float4*>(P.gate + at) = make_float4(v[0], v[1], v[2], v[3]);
        *reinterpret_cast<float4*>(P.up + at) = make_float4(u[0], u[1], u[2], u[3]);
      }
    } else {
      const long long at = static_cast<long long>(token0 + t) * P.N + n;
      const float4 g4 = *reinterpret_cast<const float4*>(P.gate + at);
      const float4 u4 = *reinterpret_cast<const float4*>(P.up + at);
      const float gg[4] = {g4.x, g4.y, g4.z, g4.w}, uu[4] = {u4.x, u4.y, u4.z, u4.w};
      float dg[4], du[4], h[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float val, der;
        act_value_grad(gg[j], P.act, val, der);
        dg[j] = v[j] * uu[j] * der;
        du[j] = v[j] * val;
        h[j] = val * uu[j];
      }
      *reinterpret_cast<uint2*>(static_cast<T*>(P.dgate) + at) =
          make_uint2(pack2<T>(dg[0], dg[1]), pack2<T>(dg[2], dg[3]));
      *reinterpret_cast<uint2*>(static_cast<T*>(P.dup) + at) =
          make_uint2(pack2<T>(du[0], du[1]), pack2<T>(du[2], du[3]));
      *reinterpret_cast<uint2*>(static_cast<T*>(P.hidden) + at) =
          make_uint2(pack2<T>(h[0], h[1]), pack2<T>(h[2], h[3]));
    }
  }
  if (warp == 1) tmem_dealloc(tmem_base, Cfg::kTmem);
}

}  // namespace moe
