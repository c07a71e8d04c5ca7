// ops_host.h - host-side pieces shared by the library's translation units.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <utility>

namespace moe {

// Record a failure for moe_last_error() / moe_last_status(); returns `status`.
int set_error(int status, const char* message);

// cuTensorMapEncodeTiled of the running driver (null when it has none).
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn tensor_map_encoder();

// The current device, its SM count and its status word (device memory); checks that it is
// an sm_100 device with an index below 64. MOE_OK or a recorded failure.
struct OpsDevice {
  int index, sms;
  int* status;
};
int ops_device(OpsDevice* out);

// Test hook (moe_ops_test_wait_timeout): whether the launch being put together on this host
// thread is the armed one; counts the launch.
int take_test_timeout();

// Launch with programmatic stream serialisation, optionally as clusters of `cluster` CTAs:
// the kernel may start its prologue while its predecessor in the stream finishes, and
// waits (griddepcontrol.wait) before it touches global memory.
template <typename... KArgs, typename... Args>
cudaError_t launch_overlapped(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem,
                              cudaStream_t st, int cluster, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cluster > 1) {
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
  }
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

}  // namespace moe
