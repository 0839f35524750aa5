// cache.cuh -- what the kernels of the 8-bit serving cache share: the cache as
// the device sees it, E4M3 conversions and the block scale rule.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "common.cuh"
#include "launch.h"

namespace csa {

// Smallest e >= -126 with amax <= 448 * 2^e, for a finite amax >= 0.  448 is
// 1.75 * 2^8, so e is amax's exponent - 8, one more when its mantissa is above
// 1.75: adding 2^23 - 1 - 0x600000 to the bits carries exactly then.
__device__ __forceinline__ int e4m3_scale_exponent(float amax) {
  return max((int)((__float_as_uint(amax) + 0x1fffffu) >> 23) - 135, -126);
}
__device__ __forceinline__ float pow2i(int e) {  // e in [-126, 127]
  return __uint_as_float((uint32_t)(e + 127) << 23);
}

// Two E4M3 codes (low byte first) as halves: exact, NaN stays NaN.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint16_t v) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(v));
  return r;
}
__device__ __forceinline__ float2 f16x2_to_float2(uint32_t v) {
  return __half22float2(*reinterpret_cast<const __half2*>(&v));
}
// Two floats as E4M3 codes, rounded to nearest even (lo in the low byte); the
// callers' values are within 448, and NaN stays NaN.
__device__ __forceinline__ uint16_t e4m3x2_from_floats(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// Block of sequence b that holds row `pos` (pos within the table), or -1 with
// the status raised for a number out of range.
__device__ __forceinline__ int cache_block(const CacheView& c, int b, int pos, int* status) {
  const int blk = __ldg(c.table + (int64_t)b * c.max_blocks + (pos >> c.log_block));
  if (blk >= 0 && blk < c.n_blocks) return blk;
  raise_status(status, CSA_ERR_DEVICE_BOUNDS);
  return -1;
}

// Launches a kernel whose first act is griddepcontrol.wait: its launch overlaps
// the end of what runs before it on the stream.
template <typename... P, typename... A>
cudaError_t launch_after(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream, A... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, P(args)...);
}

}  // namespace csa
