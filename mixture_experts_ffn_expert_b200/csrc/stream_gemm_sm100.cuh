// stream_gemm_sm100.cuh - products of the gated feed-forward block for up to 128 tokens,
// where the time is that of reading the weights once.
//
// The weights are the 128-row operand of tcgen05.mma and the tokens its N columns (16, 32,
// 64 or 128, padded with zeros by TMA), so a weight tile is read by one CTA only and the
// tensor work does not grow with a padded token tile. The reduction is split over the CTAs
// of a cluster (1, 2, 4 or 8), as many as it takes to give every SM a stream of its own:
// two CTAs share an SM, each with its own ring of TMA stages, which keeps about 200 KB of
// loads in flight an SM. Each CTA leaves its fp32 partial tile in its own shared memory;
// after a cluster barrier every CTA adds an equal share of the rows over the ranks, in
// rank order, through distributed shared memory, and runs the epilogue on them (so sums
// are the same bits every time and no partial result goes through global memory).
//
//   gate/up  A = W1 rows 0-63, W3 rows 64-127 of the tile    epilogue act(gate) * up
//   down     A = W2                                          plain
//   dh       A = W2 read along its columns                   epilogue dgate, dup, h
//   dx       A = W1 then W3 read along their columns         plain, one reduction over 2f
#pragma once

#include "dense_gemm_sm100.cuh"

namespace moe {

constexpr int kStreamThreads = 224;
constexpr int kStreamMaxTokens = 128;

template <int NB>
struct StreamCfg {
  static constexpr int kStageBytes = kDgTileBytes + NB * 128;
  static constexpr int kStages = NB <= 16 ? 6 : NB <= 32 ? 5 : NB <= 64 ? 4 : 3;
  static constexpr int kRedBytes = 128 * NB * 4;          // partial tile, over the stages
  static constexpr int kTmem = NB < 32 ? 32 : NB;
  static constexpr size_t kSmem = 1024 + size_t(kStages) * kStageBytes + 256;
  static_assert(kRedBytes <= kStages * kStageBytes, "the partial tile fits the stages");
};

struct StreamParams {
  int T, N;                 // tokens; rows of the weights (columns of the output)
  int kb[2];                // k-blocks of 64 in the two segments of the reduction
  int a_mn;                 // weights read along their columns
  int early;                // weights may be loaded before the predecessor has finished
  int act;
  void* out;                // plain: (T, N), rows ldo apart
  long long ldo;
  void *gate, *up, *hidden, *dgate, *dup;
  int* status;
};

struct StreamMaps {
  CUtensorMap a[2], b[2];
};

__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
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
  uint64_t* full_bar = reinterpret_cast<uint64_t*>(smem + size_t(kS) * Cfg::kStageBytes);
  uint64_t* empty_bar = full_bar + kS;
  uint64_t* done_bar = empty_bar + kS;
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(done_bar + 1);
  volatile int* s_abort = reinterpret_cast<volatile int*>(s_tmem + 1);
  static_assert((2 * kS + 1) * 8 + 8 <= 256, "barriers fit their 256 bytes");

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int ranks = static_cast<int>(cluster_nctarank());
  const int rank = static_cast<int>(cluster_ctarank());
  const int tile = blockIdx.x / ranks;
  const int row0 = tile * kRows;

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
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(s_tmem), Cfg::kTmem);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
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
      bool ok = true;
      for (int kb = kb_lo; kb < kb_hi; ++kb) {
        ok = mbar_wait(smem_u32(&empty_bar[s]), ph ^ 1u, s_abort);
        if (!ok) break;
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
          tma_load_2d(dst + kDgTileBytes, &maps.b[seg], fb, k0, 0);
        }
        issued_mask |= 1u << s;
        issued_par = (issued_par & ~(1u << s)) | (ph << s);
        if (++s == kS) {
          s = 0;
          ph ^= 1u;
        }
      }
      if (!ok) {
        raise_abort(s_abort, P.status);
        for (int i = 0; i < kS; ++i)      // copies in flight get a bounded time to land
          if (issued_mask & (1u << i)) {
            int never = 0;
            mbar_wait(smem_u32(&full_bar[i]), (issued_par >> i) & 1u, &never);
          }
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
  // Dependents may start only now: every thread is past its wait, so what came before this
  // kernel is complete and a dependent may read the weights early.
  pdl_launch_dependents();

  // ------------------------------------------------------------ partial tile to shared memory
  // All MMAs are done, so all stages have been read; the tile is stored column (token) by
  // column, 128 rows each: consecutive lanes write consecutive words.
  if (warp >= 2 && warp < 6) {
    int never = 0;
    bool ok = mbar_wait(smem_u32(done_bar), 0, &never);
    ok = __all_sync(0xffffffffu, ok);
    if (!ok && lane == 0) raise_abort(s_abort, P.status);
    tc_fence_after_sync();
    if (ok) {
      const int quarter = warp & 3;
      const uint32_t lane_base = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16);
      float* red = reinterpret_cast<float*>(smem) + quarter * 32 + lane;
#pragma unroll 1
      for (int c = 0; c < NB; c += 8) {
        if (c >= P.T) break;
        uint32_t v[8];
        tmem_ld_8cols(lane_base + c, v);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 8; ++j) red[(c + j) * 128] = __uint_as_float(v[j]);
      }
    }
    tc_fence_before_sync();
  }
  cluster_sync();

  // ------------------------------------------------------------ reduction and epilogue
  // This CTA's share: rows r_lo .. r_lo + share - 1 of the tile's outputs, four at a time.
  const int share = kRows / ranks;
  const int r_lo = rank * share;
  const int quads = share / 4;
  const uint32_t red0 = smem_u32(smem);
  for (int i = threadIdx.x; i < P.T * quads; i += kStreamThreads) {
    const int t = i / quads;
    const int r = r_lo + (i - t * quads) * 4;
    const int n = row0 + r;
    if (n >= P.N) continue;
    float v[4] = {0, 0, 0, 0}, u[4] = {0, 0, 0, 0};
    float4 p[8], w[8];               // all ranks' loads in flight before the first addition
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if (k < ranks) {
        const uint32_t base = mapa_shared(red0, k) + (t * 128 + r) * 4;
        p[k] = ld_cluster_f4(base);
        if (EPI == kGemmGluForward) w[k] = ld_cluster_f4(base + 64 * 4);
      }
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if (k < ranks) {
        v[0] += p[k].x;
        v[1] += p[k].y;
        v[2] += p[k].z;
        v[3] += p[k].w;
        if (EPI == kGemmGluForward) {
          u[0] += w[k].x;
          u[1] += w[k].y;
          u[2] += w[k].z;
          u[3] += w[k].w;
        }
      }
    }
    if (EPI == kGemmPlain) {
      *reinterpret_cast<uint2*>(static_cast<T*>(P.out) + t * P.ldo + n) =
          make_uint2(pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3]));
    } else if (EPI == kGemmGluForward) {
      const long long at = static_cast<long long>(t) * P.N + n;
      float h[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) h[j] = act_value(v[j], P.act) * u[j];
      *reinterpret_cast<uint2*>(static_cast<T*>(P.hidden) + at) =
          make_uint2(pack2<T>(h[0], h[1]), pack2<T>(h[2], h[3]));
      if (P.gate) {
        *reinterpret_cast<uint2*>(static_cast<T*>(P.gate) + at) =
            make_uint2(pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3]));
        *reinterpret_cast<uint2*>(static_cast<T*>(P.up) + at) =
            make_uint2(pack2<T>(u[0], u[1]), pack2<T>(u[2], u[3]));
      }
    } else {
      const long long at = static_cast<long long>(t) * P.N + n;
      const uint2 g2 = *reinterpret_cast<const uint2*>(static_cast<const T*>(P.gate) + at);
      const uint2 u2 = *reinterpret_cast<const uint2*>(static_cast<const T*>(P.up) + at);
      const float2 ga = unpack2<T>(g2.x), gb = unpack2<T>(g2.y);
      const float2 ua = unpack2<T>(u2.x), ub = unpack2<T>(u2.y);
      const float gg[4] = {ga.x, ga.y, gb.x, gb.y}, uu[4] = {ua.x, ua.y, ub.x, ub.y};
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
  cluster_sync();                  // the other ranks have read this CTA's partial tile
  if (warp == 1) tmem_dealloc(tmem_base, Cfg::kTmem);
}

}  // namespace moe
