// Host helpers of the language-model kernels' launches.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace grape {

// bf16 row-major [rows][cols] with a row pitch of `ld` elements as a 2-D tensor map of
// (box_cols x box_rows) boxes, 128-byte swizzle.
bool lm_map_2d(CUtensorMap* m, const void* ptr, uint64_t rows, uint64_t cols, uint64_t ld, uint32_t box_cols,
               uint32_t box_rows);
// SM count of the current device, and the opt-in to `smem` bytes of dynamic shared memory for
// `kernel` on it; both are taken once per device.
int lm_sm_count();
cudaError_t lm_configure_kernel(const void* kernel, int smem);

// A launch, as a programmatic dependent of the kernel before it in the stream when `pdl` (the kernel
// itself waits with griddepcontrol.wait before it reads that kernel's outputs).
template <class Kern, class... Args>
cudaError_t lm_launch(bool pdl, Kern kernel, dim3 grid, unsigned block, size_t smem, cudaStream_t st, Args... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute a[1];
  a[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = a;
  cfg.numAttrs = pdl ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace grape
