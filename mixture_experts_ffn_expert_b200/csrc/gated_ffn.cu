// gated_ffn.cu - C entry points of the gated feed-forward block with its backward pass
// (declared in include/moe_ffn.h): argument checks, tensor maps, tile choice, launches.
// Nothing here synchronises the host (moe_ops_device_status apart) or allocates device
// memory.
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>
#include <cstdio>

#include "dense_gemm_sm100.cuh"
#include "moe_ffn.h"
#include "ops_host.h"
#include "stream_gemm_sm100.cuh"

namespace {

using moe::launch_overlapped;
using moe::set_error;

// Set by a kernel that gave up a bounded wait; one word a device.
__device__ int g_ops_status;

// Launches of this host thread until the one whose first copy is withheld (0: none).
thread_local int t_test_timeout = 0;

constexpr int kMaxDevices = 64;

struct DeviceInfo {
  std::atomic<int> ready{0};
  int sms = 0;
  int* status = nullptr;
};
DeviceInfo g_devices[kMaxDevices];

int cuda_error(cudaError_t e, const char* what) {
  char buf[256];
  snprintf(buf, sizeof(buf), "%s: %s", what, cudaGetErrorString(e));
  cudaGetLastError();
  return set_error(MOE_CUDA_ERROR, buf);
}

template <typename T, int EPI, int NB>
cudaError_t set_stream_smem_one() {
  return cudaFuncSetAttribute(moe::stream_gemm_kernel<T, EPI, NB>,
                              cudaFuncAttributeMaxDynamicSharedMemorySize,
                              int(moe::StreamCfg<NB>::kSmem));
}

template <typename T, int EPI>
cudaError_t set_stream_smem() {
  cudaError_t e = set_stream_smem_one<T, EPI, 16>();
  if (e == cudaSuccess) e = set_stream_smem_one<T, EPI, 32>();
  if (e == cudaSuccess) e = set_stream_smem_one<T, EPI, 64>();
  if (e == cudaSuccess) e = set_stream_smem_one<T, EPI, 128>();
  return e;
}

template <typename T, int EPI>
cudaError_t set_dense_smem() {
  cudaError_t e = cudaFuncSetAttribute(moe::dense_gemm_kernel<T, EPI, true>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       int(moe::DenseCfg<EPI>::kSmem));
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(moe::dense_gemm_kernel<T, EPI, false>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                             int(moe::DenseCfg<EPI>::kSmem));
  return e;
}

template <typename T>
cudaError_t set_smem() {
  cudaError_t e = set_dense_smem<T, moe::kGemmPlain>();
  if (e == cudaSuccess) e = set_dense_smem<T, moe::kGemmGluForward>();
  if (e == cudaSuccess) e = set_dense_smem<T, moe::kGemmGluForwardSave>();
  if (e == cudaSuccess) e = set_dense_smem<T, moe::kGemmGluBackward>();
  if (e == cudaSuccess) e = set_stream_smem<T, moe::kGemmPlain>();
  if (e == cudaSuccess) e = set_stream_smem<T, moe::kGemmGluForward>();
  if (e == cudaSuccess) e = set_stream_smem<T, moe::kGemmGluBackward>();
  return e;
}

// Properties of the current device; the first call on a device also raises the kernels'
// shared-memory limits there (repeating that is harmless, so two first calls may race).
int device_info(DeviceInfo** out) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_error(e, "no usable CUDA device");
  if (dev >= kMaxDevices) return set_error(MOE_UNSUPPORTED, "device index above 63");
  DeviceInfo& d = g_devices[dev];
  if (!d.ready.load(std::memory_order_acquire)) {
    int major = 0, minor = 0, sms = 0;
    void* status = nullptr;
    if ((e = cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev)) ||
        (e = cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev)) ||
        (e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)))
      return cuda_error(e, "device query");
    if (major != 10 || minor != 0)
      return set_error(MOE_UNSUPPORTED, "this library is built for sm_100a only");
    if ((e = cudaGetSymbolAddress(&status, g_ops_status)) ||
        (e = set_smem<__nv_bfloat16>()) || (e = set_smem<__half>()))
      return cuda_error(e, "kernel attributes");
    if (!moe::tensor_map_encoder())
      return set_error(MOE_CUDA_ERROR, "cuTensorMapEncodeTiled is not available from the driver");
    d.sms = sms;
    d.status = static_cast<int*>(status);
    d.ready.store(1, std::memory_order_release);
  }
  *out = &d;
  return MOE_OK;
}

bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
size_t align_up(size_t v) { return (v + 255) / 256 * 256; }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Matrix (rows, cols) of a type (an MOE_DTYPE_), rows `ld` elements apart, in boxes of box_cols
// columns x box_rows rows, swizzled over a box row's 128, 64 or 32 bytes; what a box covers
// beyond the matrix reads as zero and is not written.
bool encode_map(CUtensorMap* m, int dtype, const void* base, int64_t rows, int64_t cols, int64_t ld,
                int box_rows, int box_cols = 64) {
  const int size = dtype == MOE_DTYPE_FP32 ? 4 : 2;
  cuuint64_t dims[2] = {cuuint64_t(cols), cuuint64_t(rows)};
  cuuint64_t strides[1] = {cuuint64_t(ld) * size};
  cuuint32_t box[2] = {cuuint32_t(box_cols), cuuint32_t(box_rows)};
  cuuint32_t estr[2] = {1, 1};
  return moe::tensor_map_encoder()(
             m,
             dtype == MOE_DTYPE_FP32   ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
             : dtype == MOE_DTYPE_FP16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                       : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
             2, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             box_cols * size == 128  ? CU_TENSOR_MAP_SWIZZLE_128B
             : box_cols * size == 64 ? CU_TENSOR_MAP_SWIZZLE_64B
                                     : CU_TENSOR_MAP_SWIZZLE_32B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// One launch being put together: tensor maps and products.
struct GemmLaunch {
  moe::DenseMaps maps;
  moe::DenseParams P = {};
  int n_maps = 0;
  int dtype;                // MOE_DTYPE_BF16 or MOE_DTYPE_FP16
  bool ok = true;

  int map(const void* base, int64_t rows, int64_t cols, int64_t ld, int box_rows,
          int box_cols = 64) {
    ok = ok && encode_map(&maps.m[n_maps], dtype, base, rows, cols, ld, box_rows, box_cols);
    return n_maps++;
  }
  // A saved pre-activation, fp32, stored in chunks of 16 columns.
  int map_saved(const void* base, int64_t rows, int64_t cols) {
    ok = ok && encode_map(&maps.m[n_maps], MOE_DTYPE_FP32, base, rows, cols, cols, 128, 16);
    return n_maps++;
  }

  void product(int M, int N, int tile_m, int tile_n, int64_t k0, int64_t k1, int a0, int a1,
               int b0, int b1, int a_mn, int b_mn, int out0, int out1 = 0, int out2 = 0) {
    moe::DenseProblem& q = P.p[P.n_problems++];
    q.M = M;
    q.N = N;
    q.m_tiles = int(ceil_div(M, tile_m));
    q.n_tiles = int(ceil_div(N, tile_n));
    q.tile0 = P.total_tiles;
    q.kb[0] = int(ceil_div(k0, 64));
    q.kb[1] = int(ceil_div(k1, 64));
    q.map_a[0] = a0;
    q.map_a[1] = a1;
    q.map_b[0] = b0;
    q.map_b[1] = b1;
    q.a_mn = a_mn;
    q.b_mn = b_mn;
    q.map_out[0] = out0;
    q.map_out[1] = out1;
    q.map_out[2] = out2;
    P.total_tiles += q.m_tiles * q.n_tiles;
  }
};

template <typename T, int EPI, bool PAIR>
cudaError_t launch(GemmLaunch& L, const DeviceInfo& d, cudaStream_t st) {
  int workers = PAIR ? d.sms / 2 : d.sms;
  if (workers > L.P.total_tiles) workers = L.P.total_tiles;
  const moe::DenseProblem& q0 = L.P.p[0];
  L.P.first_tiles = q0.m_tiles * q0.n_tiles;
  L.P.extra = 0;
  if (L.P.n_problems > 1) {
    const int late = workers - L.P.first_tiles % workers;   // == workers: no remainder
    const int rest = L.P.total_tiles - L.P.first_tiles;
    // a tile costs its k-blocks, and at least its epilogue (about 2 us of a pair, 1 us of a
    // single CTA)
    const int least = PAIR ? 7 : 5;
    int k0 = q0.kb[0] + q0.kb[1], k1 = L.P.p[1].kb[0] + L.P.p[1].kb[1];
    if (k0 < least) k0 = least;
    if (k1 < least) k1 = least;
    int extra = (k0 + k1 / 2) / k1;
    if (late < workers && extra > rest / late) extra = rest / late;
    if (late < workers) L.P.extra = extra;
  }
  L.P.status = d.status;
  L.P.test_withhold = moe::take_test_timeout();
  L.P.n_maps = L.n_maps;
  return launch_overlapped(moe::dense_gemm_kernel<T, EPI, PAIR>,
                           dim3(PAIR ? 2 * workers : workers), dim3(moe::kDgThreads),
                           moe::DenseCfg<EPI>::kSmem, st, PAIR ? 2 : 1, L.maps, L.P);
}

template <int EPI>
cudaError_t launch_any(GemmLaunch& L, bool pair, const DeviceInfo& d, cudaStream_t st) {
  if (!L.ok) return cudaErrorInvalidValue;         // a tensor map could not be encoded
  if (L.dtype == MOE_DTYPE_FP16)
    return pair ? launch<__half, EPI, true>(L, d, st) : launch<__half, EPI, false>(L, d, st);
  return pair ? launch<__nv_bfloat16, EPI, true>(L, d, st)
              : launch<__nv_bfloat16, EPI, false>(L, d, st);
}

// How a product of `tokens` rows, `n` columns (of one of gate / up) and `kb` k-blocks runs:
// on CTA pairs, on single CTAs, or streaming its weights with a split reduction. Estimates in
// microseconds, from measurements on B200: a k-block of 64 takes about 0.3 us in a 256 x 256
// tile of a pair, 0.21 in a 128 x 128 tile of one CTA (32 KB of operands from L2 an SM),
// and the split reduction ends with about 3.5 us of exchange more. Up to 128 tokens the
// weights are streamed, small forwards of more than 64 excepted (small_forward).
enum Shape { kPairs, kSingle, kStream };

int stream_ranks(int64_t tiles, int64_t kb, int sms) {
  int ranks = 1;
  while (ranks < 8 && tiles * ranks * 2 <= 2 * sms && ranks * 2 <= kb) ranks *= 2;
  return ranks;
}

// The weights' gradients run on CTA pairs once there are enough tiles for every pair of SMs
// and a tile's reduction over the tokens is longer than its epilogue. The whole backward pass on
// pairs and on single CTAs, us, for 384, 448, 512 and 640 tokens:
//   d=4096 f=14336   311 and 326   324 and 381   324 and 399   400 and 463
//   d=4096 f=4096    103 and 107   105 and 118   103 and 122   128 and 146
//   d=2048 f=2816     56 and 48     56 and 50     57 and 53     57 and 59
// so one switch point for all sizes lies between what wide and what narrow blocks would take.
bool use_pairs(int64_t f, int64_t d, int64_t tokens, const DeviceInfo& dev) {
  return tokens > 448 && 3 * ceil_div(f, 256) * ceil_div(d, 256) >= dev.sms / 2;
}

Shape choose(int64_t tokens, int64_t n, int64_t kb, bool glu, const DeviceInfo& d) {
  if (tokens <= moe::kStreamTokens) return kStream;
  const int64_t cols = glu ? 2 * n : n;
  const int64_t t256 = ceil_div(tokens, 256) * ceil_div(cols, 256);
  const int64_t t128 = ceil_div(tokens, 128) * ceil_div(cols, 128);
  const int ranks = stream_ranks(t128, kb, d.sms);
  const double pairs = ceil_div(t256, d.sms / 2) * kb * 0.30;
  const double single = ceil_div(t128, d.sms) * kb * 0.21;
  const double stream = ceil_div(t128 * ranks, d.sms) * ceil_div(kb, ranks) * 0.21 + 3.5;
  if (stream < pairs && stream < single) return kStream;
  return pairs <= single ? kPairs : kSingle;
}

// Whether a forward over 65 to 128 tokens runs on single CTAs: its matrices are so small that
// the exchange after both split reductions, 0.045 us a token each, costs more than they save
// (128 tokens, d=f=1024: 14.5 us, 17.9 streamed; d=2048 f=1408: 20.3 and 23.7; d=7168, f=2048:
// 43.9 and 36.6). The estimate must be 1 us ahead: where the two come out equal, streaming is the
// faster (128 tokens, d=2048, f=2816: 26.0 us, 23.9 streamed). It holds for the 128-column tile
// only: up to 64 tokens the rows received have an area of their own, and streaming is ahead at
// every size measured (64 tokens, d=f=512: 9.8 us, 8.2 streamed; d=f=1024: 14.1 and 11.2).
bool small_forward(int64_t tokens, int64_t d, int64_t f, const DeviceInfo& dev) {
  if (tokens <= 64 || tokens > moe::kStreamTokens) return false;
  double single = 0.0, stream = 0.0;
  const int64_t shape[2][2] = {{2 * f, d}, {d, f}};        // columns and reduction
  for (const auto& s : shape) {
    const int64_t tiles = ceil_div(s[0], 128), kb = ceil_div(s[1], 64);
    const int ranks = stream_ranks(tiles, kb, dev.sms);
    single += ceil_div(tiles, dev.sms) * kb * 0.21;
    stream += ceil_div(tiles * ranks, dev.sms) * ceil_div(kb, ranks) * 0.21 + 0.045 * tokens;
  }
  return single + 1.0 < stream;
}

// One product whose weights are streamed by clusters that split the reduction until there
// are about two CTAs an SM.
struct StreamLaunch {
  moe::StreamMaps maps;
  moe::StreamParams P = {};
  int dtype;                // MOE_DTYPE_BF16 or MOE_DTYPE_FP16
  bool ok = true;

  int columns() const { return P.T <= 16 ? 16 : P.T <= 32 ? 32 : P.T <= 64 ? 64 : 128; }
  void weights(int i, const void* base, int64_t rows, int64_t cols, int box_rows) {
    ok = ok && encode_map(&maps.a[i], dtype, base, rows, cols, cols, box_rows);
  }
  void tokens(int i, const void* base, int64_t cols, int64_t ld) {
    ok = ok && encode_map(&maps.b[i], dtype, base, P.T, cols, ld, columns());
  }
};

template <typename T, int EPI, int NB>
cudaError_t launch_stream_columns(StreamLaunch& L, const DeviceInfo& d, cudaStream_t st) {
  L.P.t_tiles = int(ceil_div(L.P.T, moe::kStreamTokens));
  const int64_t tiles = L.P.t_tiles * ceil_div(L.P.N, EPI == moe::kGemmGluForward ? 64 : 128);
  const int ranks = stream_ranks(tiles, L.P.kb[0] + L.P.kb[1], d.sms);
  L.P.status = d.status;
  L.P.test_withhold = moe::take_test_timeout();
  return launch_overlapped(moe::stream_gemm_kernel<T, EPI, NB>, dim3(unsigned(tiles * ranks)),
                           dim3(moe::kStreamThreads), moe::StreamCfg<NB>::kSmem, st, ranks, L.maps,
                           L.P);
}

template <int EPI>
cudaError_t launch_stream(StreamLaunch& L, const DeviceInfo& d, cudaStream_t st) {
  if (!L.ok) return cudaErrorInvalidValue;         // a tensor map could not be encoded
  const int nb = L.columns();
  if (L.dtype == MOE_DTYPE_FP16) {
    if (nb == 16) return launch_stream_columns<__half, EPI, 16>(L, d, st);
    if (nb == 32) return launch_stream_columns<__half, EPI, 32>(L, d, st);
    if (nb == 64) return launch_stream_columns<__half, EPI, 64>(L, d, st);
    return launch_stream_columns<__half, EPI, 128>(L, d, st);
  }
  if (nb == 16) return launch_stream_columns<__nv_bfloat16, EPI, 16>(L, d, st);
  if (nb == 32) return launch_stream_columns<__nv_bfloat16, EPI, 32>(L, d, st);
  if (nb == 64) return launch_stream_columns<__nv_bfloat16, EPI, 64>(L, d, st);
  return launch_stream_columns<__nv_bfloat16, EPI, 128>(L, d, st);
}

int check_shape(int act, int dtype, int64_t T, int64_t d, int64_t f) {
  if (act != MOE_ACT_SILU && act != MOE_ACT_GELU)
    return set_error(MOE_INVALID_ARG, "activation must be MOE_ACT_SILU or MOE_ACT_GELU");
  if (dtype != MOE_DTYPE_BF16 && dtype != MOE_DTYPE_FP16)
    return set_error(MOE_INVALID_ARG, "the gated feed-forward block takes bf16 or fp16");
  if (T < 0) return set_error(MOE_INVALID_ARG, "T must be >= 0");
  if (d < 1 || f < 1) return set_error(MOE_INVALID_CONFIG, "d and f must be >= 1");
  if (d % 8 || f % 8 || d > (1 << 20) || f > (1 << 20) || T > (1 << 24))
    return set_error(MOE_UNSUPPORTED,
                     "d and f must be multiples of 8 up to 2^20, T at most 2^24");
  return MOE_OK;
}

int check_rows(const void* p, int64_t T, int64_t cols, int64_t ld, const char* what) {
  char buf[128];
  if (!p || !aligned(p, 16)) {
    snprintf(buf, sizeof(buf), "%s must be non-null and 16-byte aligned", what);
    return set_error(MOE_INVALID_ARG, buf);
  }
  if (T > 1 && (ld < cols || ld % 8 || ld > (1LL << 31))) {
    snprintf(buf, sizeof(buf), "%s: the row stride must be a multiple of 8 and >= its width",
             what);
    return set_error(MOE_INVALID_ARG, buf);
  }
  return MOE_OK;
}

}  // namespace

namespace moe {
int ops_device(OpsDevice* out) {
  DeviceInfo* d;
  if (int s = device_info(&d)) return s;
  out->index = static_cast<int>(d - g_devices);
  out->sms = d->sms;
  out->status = d->status;
  return MOE_OK;
}

int take_test_timeout() {
  if (t_test_timeout == 0) return 0;
  return --t_test_timeout == 0;
}
}  // namespace moe

extern "C" {

size_t moe_gated_ffn_workspace_bytes(int64_t T, int64_t d, int64_t f, int backward) {
  if (check_shape(MOE_ACT_SILU, MOE_DTYPE_BF16, T, d, f) != MOE_OK) return 0;
  return (backward ? 3 : 1) * align_up(size_t(T) * f * 2);
}

int moe_gated_ffn_forward(int act, int dtype, int64_t T, int64_t d, int64_t f, const void* x,
                          int64_t ldx, const void* W1, const void* W3, const void* W2, void* out,
                          int64_t ldo, float* gate, float* up, void* workspace,
                          size_t workspace_bytes, void* stream) {
  if (int s = check_shape(act, dtype, T, d, f)) return s;
  if (T == 0) return MOE_OK;
  if (int s = check_rows(x, T, d, ldx, "x")) return s;
  if (int s = check_rows(out, T, d, ldo, "out")) return s;
  if (int s = check_rows(W1, 1, d, d, "W1")) return s;
  if (int s = check_rows(W3, 1, d, d, "W3")) return s;
  if (int s = check_rows(W2, 1, f, f, "W2")) return s;
  if ((gate == nullptr) != (up == nullptr) || !aligned(gate, 16) || !aligned(up, 16))
    return set_error(MOE_INVALID_ARG, "gate and up must be both null or both 16-byte aligned");
  if (workspace_bytes < moe_gated_ffn_workspace_bytes(T, d, f, 0))
    return set_error(MOE_WORKSPACE_TOO_SMALL, "gated feed-forward: workspace too small");
  if (!workspace || !aligned(workspace, 256))
    return set_error(MOE_INVALID_ARG, "workspace must be non-null and 256-byte aligned");
  if (T == 1) ldx = ldo = d;
  DeviceInfo* dev;
  if (int s = device_info(&dev)) return s;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int m = int(T);
  cudaError_t e;
  bool overlapped = false;       // the first kernel lets the second load weights early
  const bool small = small_forward(T, d, f, *dev);
  const Shape first = small ? kSingle : choose(T, f, ceil_div(d, 64), true, *dev);
  if (first == kStream) {
    StreamLaunch L;
    L.dtype = dtype;
    L.P.T = m;
    L.P.N = int(f);
    L.P.kb[0] = int(ceil_div(d, 64));
    L.P.act = act;
    L.P.hidden = workspace;
    L.P.gate = gate;
    L.P.up = up;
    L.weights(0, W1, f, d, 64);
    L.weights(1, W3, f, d, 64);
    L.tokens(0, x, d, ldx);
    e = launch_stream<moe::kGemmGluForward>(L, *dev, st);
    overlapped = true;
  } else {
    GemmLaunch L;
    L.dtype = dtype;
    const bool pair = first == kPairs;
    const int a = L.map(x, T, d, ldx, 128);
    const int b1 = L.map(W1, f, d, d, pair ? 128 : 64);
    const int b3 = L.map(W3, f, d, d, pair ? 128 : 64);
    const int o0 = L.map(workspace, T, f, f, 128, gate ? 16 : 32);
    const int o1 = gate ? L.map_saved(gate, T, f) : o0;
    const int o2 = gate ? L.map_saved(up, T, f) : o0;
    L.product(m, int(f), pair ? 256 : 128, pair ? 128 : 64, d, 0, a, a, b1, b3, 0, 0, o0, o1, o2);
    L.P.act = act;
    e = gate ? launch_any<moe::kGemmGluForwardSave>(L, pair, *dev, st)
             : launch_any<moe::kGemmGluForward>(L, pair, *dev, st);
  }
  if (e != cudaSuccess) return cuda_error(e, "gated feed-forward gate/up launch");
  const Shape second = small ? kSingle : choose(T, d, ceil_div(f, 64), false, *dev);
  if (second == kStream) {
    StreamLaunch L;
    L.dtype = dtype;
    L.P.T = m;
    L.P.N = int(d);
    L.P.kb[0] = int(ceil_div(f, 64));
    L.P.early = overlapped;
    L.P.out = out;
    L.P.ldo = ldo;
    L.weights(0, W2, d, f, 128);
    L.tokens(0, workspace, f, f);
    e = launch_stream<moe::kGemmPlain>(L, *dev, st);
  } else {
    GemmLaunch L;
    L.dtype = dtype;
    const bool pair = second == kPairs;
    const int tile = pair ? 256 : 128;
    const int a = L.map(workspace, T, f, f, 128), b = L.map(W2, d, f, f, 128);
    L.product(m, int(d), tile, tile, f, 0, a, a, b, b, 0, 0, L.map(out, T, d, ldo, 128));
    e = launch_any<moe::kGemmPlain>(L, pair, *dev, st);
  }
  if (e != cudaSuccess) return cuda_error(e, "gated feed-forward down launch");
  return MOE_OK;
}

int moe_gated_ffn_backward(int act, int dtype, int64_t T, int64_t d, int64_t f, const void* dout,
                           int64_t lddout, const void* x, int64_t ldx, const void* W1,
                           const void* W3, const void* W2, const float* gate, const float* up,
                           void* dx, int64_t lddx, void* dW1, void* dW3, void* dW2,
                           void* workspace, size_t workspace_bytes, void* stream) {
  if (int s = check_shape(act, dtype, T, d, f)) return s;
  if (!dx && !dW1 && !dW3 && !dW2) return MOE_OK;
  if (!aligned(dW1, 16) || !aligned(dW3, 16) || !aligned(dW2, 16))
    return set_error(MOE_INVALID_ARG, "dW1, dW3 and dW2 must be 16-byte aligned");
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (T == 0) {                        // sums over no tokens
    void* grads[3] = {dW1, dW3, dW2};
    for (void* g : grads)
      if (g) {
        const cudaError_t e = cudaMemsetAsync(g, 0, size_t(d) * f * 2, st);
        if (e != cudaSuccess) return cuda_error(e, "gated feed-forward backward");
      }
    return MOE_OK;
  }
  if (int s = check_rows(dout, T, d, lddout, "dout")) return s;
  if (int s = check_rows(x, T, d, ldx, "x")) return s;
  if (dx)
    if (int s = check_rows(dx, T, d, lddx, "dx")) return s;
  if (int s = check_rows(W1, 1, d, d, "W1")) return s;
  if (int s = check_rows(W3, 1, d, d, "W3")) return s;
  if (int s = check_rows(W2, 1, f, f, "W2")) return s;
  if (int s = check_rows(gate, 1, f, f, "gate")) return s;
  if (int s = check_rows(up, 1, f, f, "up")) return s;
  if (workspace_bytes < moe_gated_ffn_workspace_bytes(T, d, f, 1))
    return set_error(MOE_WORKSPACE_TOO_SMALL, "gated feed-forward backward: workspace too small");
  if (!workspace || !aligned(workspace, 256))
    return set_error(MOE_INVALID_ARG, "workspace must be non-null and 256-byte aligned");
  if (T == 1) ldx = lddx = lddout = d;
  DeviceInfo* dev;
  if (int s = device_info(&dev)) return s;
  const size_t plane = align_up(size_t(T) * f * 2);
  char* ws = static_cast<char*>(workspace);
  void *dgate = ws, *dup = ws + plane, *hidden = ws + 2 * plane;
  const int m = int(T);
  cudaError_t e;
  bool overlapped = false;       // the first kernel lets the second load weights early
  const Shape first = choose(T, f, ceil_div(d, 64), false, *dev);
  if (first == kStream) {
    StreamLaunch L;
    L.dtype = dtype;
    L.P.T = m;
    L.P.N = int(f);
    L.P.kb[0] = int(ceil_div(d, 64));
    L.P.a_mn = 1;
    L.P.act = act;
    L.P.gate = const_cast<float*>(gate);
    L.P.up = const_cast<float*>(up);
    L.P.dgate = dgate;
    L.P.dup = dup;
    L.P.hidden = hidden;
    L.weights(0, W2, d, f, 64);
    L.tokens(0, dout, d, lddout);
    e = launch_stream<moe::kGemmGluBackward>(L, *dev, st);
    overlapped = true;
  } else {
    GemmLaunch L;
    L.dtype = dtype;
    const bool pair = first == kPairs;
    const int tile = pair ? 256 : 128;
    const int a = L.map(dout, T, d, lddout, 128), b = L.map(W2, d, f, f, 64);
    const int o0 = L.map(hidden, T, f, f, 128, 32), o1 = L.map(dgate, T, f, f, 128, 32);
    const int o2 = L.map(dup, T, f, f, 128, 32);
    L.product(m, int(f), tile, tile, d, 0, a, a, b, b, 0, 1, o0, o1, o2);
    L.P.gate = gate;
    L.P.up = up;
    L.P.act = act;
    e = launch_any<moe::kGemmGluBackward>(L, pair, *dev, st);
  }
  if (e != cudaSuccess) return cuda_error(e, "gated feed-forward dh launch");
  const bool weights = dW1 || dW3 || dW2;
  const Shape third = choose(T, d, 2 * ceil_div(f, 64), false, *dev);
  // dx runs in one launch with the weights' gradients, its long tiles beside their short
  // ones, unless there are so few tokens that reading W1 and W3 is all it does. The backward pass
  // streamed and together, us, for 16, 32, 64 and 128 tokens:
  //   d=4096 f=14336   173 and 180   170 and 181   182 and 184   194 and 192
  //   d=7168 f=2048     54 and 58     55 and 53     59 and 56     68 and 61
  //   d=2048 f=1408     18 and 19     19 and 19     22 and 21     30 and 24
  const bool stream_dx = dx && third == kStream && (!weights || T <= 32);
  if (stream_dx) {
    StreamLaunch L;
    L.dtype = dtype;
    L.P.T = m;
    L.P.N = int(d);
    L.P.kb[0] = L.P.kb[1] = int(ceil_div(f, 64));
    L.P.a_mn = 1;
    L.P.early = overlapped;
    L.P.out = dx;
    L.P.ldo = lddx;
    L.weights(0, W1, f, d, 64);
    L.weights(1, W3, f, d, 64);
    L.tokens(0, dgate, f, f);
    L.tokens(1, dup, f, f);
    e = launch_stream<moe::kGemmPlain>(L, *dev, st);
    if (e != cudaSuccess) return cuda_error(e, "gated feed-forward dx launch");
    if (!weights) return MOE_OK;
  }
  GemmLaunch L;
  L.dtype = dtype;
  const bool pair = weights ? use_pairs(f, d, T, *dev) : third == kPairs;
  const int tile = pair ? 256 : 128;
  if (dx && !stream_dx) {
    const int a0 = L.map(dgate, T, f, f, 128), a1 = L.map(dup, T, f, f, 128);
    const int b0 = L.map(W1, f, d, d, 64), b1 = L.map(W3, f, d, d, 64);
    L.product(m, int(d), tile, tile, f, f, a0, a1, b0, b1, 0, 1, L.map(dx, T, d, lddx, 128));
  }
  const int xm = dW1 || dW3 ? L.map(x, T, d, ldx, 64) : 0;
  if (dW1) {
    const int a = L.map(dgate, T, f, f, 64);
    L.product(int(f), int(d), tile, tile, T, 0, a, a, xm, xm, 1, 1,
              L.map(dW1, f, d, d, 128));
  }
  if (dW3) {
    const int a = L.map(dup, T, f, f, 64);
    L.product(int(f), int(d), tile, tile, T, 0, a, a, xm, xm, 1, 1,
              L.map(dW3, f, d, d, 128));
  }
  if (dW2) {
    const int a = L.map(dout, T, d, lddout, 64), b = L.map(hidden, T, f, f, 64);
    L.product(int(d), int(f), tile, tile, T, 0, a, a, b, b, 1, 1, L.map(dW2, d, f, f, 128));
  }
  if (!L.ok) return set_error(MOE_CUDA_ERROR, "tensor map encoding failed");
  e = launch_any<moe::kGemmPlain>(L, pair, *dev, st);
  if (e != cudaSuccess) return cuda_error(e, "gated feed-forward gradient launch");
  return MOE_OK;
}

int moe_ops_test_wait_timeout(int launch) {
  if (launch < 0) return set_error(MOE_INVALID_ARG, "launch must be >= 0");
  t_test_timeout = launch;
  return MOE_OK;
}

int moe_ops_device_status(void) {
  DeviceInfo* dev;
  if (int s = device_info(&dev)) return s;
  int v = 0;
  cudaError_t e = cudaMemcpy(&v, dev->status, sizeof(int), cudaMemcpyDeviceToHost);
  if (e == cudaSuccess && v != 0) e = cudaMemset(dev->status, 0, sizeof(int));
  if (e != cudaSuccess) return cuda_error(e, "device status read");
  if (v != MOE_OK) return set_error(v, "an operator's kernel gave up a bounded wait");
  return MOE_OK;
}

}  // extern "C"
