// Host helpers shared by the files that define entry points.
#pragma once

#include <cstdint>
#include <utility>

#include <cuda.h>
#include <cuda_runtime.h>

namespace qlora {

// Operators whose kernels' attributes are set together, by the first call of
// one of them in a context: nobody else's first call pays for it (all three
// together took a first NF4 call from 7.0 to 7.8 ms) or fails with it.
enum class OpFamily : int { kFp8 = 0, kNorm = 1, kAdamw = 2 };

// Device check of the current device (see check_current_device_status), with
// its SM count and how many CTA pairs of one CTA a SM fit on it at once.
int check_current_device(OpFamily family, int* sms, int* pairs = nullptr);

// What the check does for each family: the shared-memory limits of its kernels,
// and how many clusters of the 8-bit product's split kernel fit on the device.
cudaError_t set_fp8_attributes(int dev);    // fp8.cu
cudaError_t set_norm_attributes();          // norm.cu
cudaError_t set_adamw_attributes();         // optim_multi.cu

// Device address of the status word (ptx.cuh) on the current device, after a
// successful device check of the 8-bit product's family.
unsigned int* device_status_word();

// Counts a launch and returns its status (a qlora_status_t).
int launch_done();

// 2-D tensor map of a row-major matrix (see map2d in api.cu).
bool encode_map2d(CUtensorMap* m, CUtensorMapDataType dt, const void* ptr, uint64_t inner, uint64_t outer,
                  uint64_t row_bytes, uint32_t box_inner, uint32_t box_outer, CUtensorMapSwizzle sw);

namespace host {

inline bool aligned(const void* p, unsigned bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }
inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline int64_t rup(int64_t a, int64_t b) { return cdiv(a, b) * b; }
inline size_t al256(size_t b) { return (b + 255) & ~static_cast<size_t>(255); }

// Launch as a programmatic dependent of the kernel in front on the stream
// (and, with `cluster` > 1, in clusters of that many CTAs): the kernel waits
// for that grid itself before it touches global memory.
template <typename... KArgs, typename... Args>
int launch_pdl(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t st, unsigned cluster,
               Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
  return launch_done();
}

}  // namespace host
}  // namespace qlora
