// Host-side helpers: launch accounting and event timing, tensor-map encoding,
// argument checks. Used by the .cu files that launch kernels.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <cmath>

#include "adaspark.h"

namespace adaspark {

// Records a begin/end event pair around a launch when the timer is enabled and
// counts every launch.
void timer_begin(const char* name, cudaStream_t s);
void timer_end(cudaStream_t s);
void count_launch();

#ifdef __CUDACC__
template <typename... KArgs, typename... Args>
inline cudaError_t launch(const char* name, void (*kernel)(KArgs...), dim3 grid, dim3 block,
                          size_t smem, cudaStream_t s, Args&&... args) {
  timer_begin(name, s);
  kernel<<<grid, block, smem, s>>>(static_cast<KArgs>(args)...);
  cudaError_t e = cudaGetLastError();
  timer_end(s);
  count_launch();
  return e;
}

// Lets `kernel` use `bytes` of dynamic shared memory on the current device; asked
// of the runtime once per kernel and device.
int allow_smem(const void* kernel, int bytes);
template <typename... KArgs>
inline int allow_smem(void (*kernel)(KArgs...), int bytes) {
  return allow_smem(reinterpret_cast<const void*>(kernel), bytes);
}

// launch() of a kernel whose blocks may come up while the stream's previous
// kernel still runs: it must call dependency_wait() (common.cuh) before it
// touches anything that kernel writes. `cluster`: blocks per cluster along x.
template <typename... KArgs, typename... Args>
inline cudaError_t launch_after(const char* name, void (*kernel)(KArgs...), dim3 grid, dim3 block,
                                size_t smem, cudaStream_t s, int cluster, Args&&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2] = {};
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {(unsigned)cluster, 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  timer_begin(name, s);
  cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...);
  if (e == cudaSuccess) e = cudaGetLastError();
  timer_end(s);
  count_launch();
  return e;
}
#endif

// cuTensorMapEncodeTiled through the runtime's driver entry point (no -lcuda).
// 2D or 3D maps of 16-bit elements (bf16 or fp16), 128-byte swizzle, zero fill
// out of bounds. dims/strides are innermost first; strides in bytes for dims
// 1.. (dim 0 is dense).
bool encode_tmap_16(CUtensorMap* map, const void* base, int rank, const uint64_t* dims,
                    const uint64_t* strides_bytes, const uint32_t* box, bool fp16);
inline bool encode_tmap_bf16(CUtensorMap* map, const void* base, int rank, const uint64_t* dims,
                             const uint64_t* strides_bytes, const uint32_t* box) {
  return encode_tmap_16(map, base, rank, dims, strides_bytes, box, false);
}

inline bool p_valid(float p) { return p > 0.0f && p <= 1.0f; }  // false for NaN

inline bool aligned(const void* ptr, size_t a) {
  return (reinterpret_cast<uintptr_t>(ptr) % a) == 0;
}

int device_is_sm100();  // 1 yes, 0 no, -1 query failed

// ADASPARK_OK when the current device is an sm_100 GPU; *sms (if not NULL) gets
// its SM count. Looked up once per device.
int current_device(int* sms);

}  // namespace adaspark
