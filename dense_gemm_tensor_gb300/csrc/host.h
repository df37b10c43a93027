// What the C entry points of the library share on the host side: the current
// device's record, memory checks, tensor-map encoding and launch accounting.
// The definitions are in gemm_host.cu.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace dgt {

// One call's device and the launch-wide numbers its kernels take (the device
// status words, a fresh epoch, and the debug hook's settings).
struct CallContext {
  int dev;
  int sm_count;
  uint32_t* status;
  uint32_t epoch;
  uint32_t debug;
  uint64_t wait_limit_ns;
};

// Fills `out` for the current device; a GEMM_* code.
int begin_call(CallContext* out);

// Device (or managed) memory of the current device `dev`?
bool on_device(const void* ptr, int dev);

// Tiled tensor maps with x innermost; box box_inner x box_outer. 3-D: z
// matrices mat_bytes apart, box_depth of them to a box. 2-D: rows only (the
// form row gathers take).
bool encode_map_3d(CUtensorMap* m, CUtensorMapDataType dt, const void* base, uint64_t inner, uint64_t outer,
                   uint64_t row_bytes, uint64_t depth, uint64_t mat_bytes, uint32_t box_inner, uint32_t box_outer,
                   CUtensorMapSwizzle swizzle, uint32_t box_depth = 1);
bool encode_map_2d(CUtensorMap* m, CUtensorMapDataType dt, const void* base, uint64_t inner, uint64_t outer,
                   uint64_t row_bytes, uint32_t box_inner, uint32_t box_outer, CUtensorMapSwizzle swizzle);

// Counts kernels launched by the library (gemm_launch_count).
void count_launches(int n);

// Launches `kern` as a programmatic dependent of the previous kernel on the
// stream (the kernel itself waits, griddepcontrol.wait, before it touches
// memory); clusters of `cluster` CTAs where that is above 1.
template <class... P, class... A>
cudaError_t launch_dependent(void (*kern)(P...), int grid, int block, size_t smem, cudaStream_t stream, int cluster,
                             A... args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.gridDim = dim3(grid, 1, 1);
  cfg.blockDim = dim3(block, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  const cudaError_t launched = cudaLaunchKernelEx(&cfg, kern, P(args)...);
  const cudaError_t last = cudaGetLastError();  // also clears a refused launch's error for the next call
  const cudaError_t e = launched != cudaSuccess ? launched : last;
  if (e == cudaSuccess) count_launches(1);
  return e;
}

}  // namespace dgt
