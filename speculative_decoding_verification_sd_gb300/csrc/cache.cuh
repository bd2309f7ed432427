// cache.cuh -- device-side access to the paged key-value cache and to the
// step's row ranges, shared by the append and attention kernels.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "sd_device.cuh"
#include "serving.h"

namespace sdk {

// Row range of request i: first packed row and row count.  A range that is
// not a compaction of at most k_max + 1 rows below bs * (k_max + 1) is
// refused: count -1.
struct RowRange {
  int first, n;
};
__device__ __forceinline__ RowRange row_range(const int* cu, int i, int bs, int k_max) {
  const int a = __ldg(cu + i), b = __ldg(cu + i + 1);
  const bool ok = a >= 0 && b >= a && static_cast<long long>(b) - a <= k_max + 1 &&
                  b <= static_cast<long long>(bs) * (k_max + 1);
  return ok ? RowRange{a, b - a} : RowRange{0, -1};
}

// A request's length as attention takes it.  Kernels step past the last token by up
// to a tile, so lengths stop short of 2^31.
__device__ __forceinline__ int attended_len(const CacheView& c, int given) {
  const long long room = static_cast<long long>(c.max_pages) * c.page_size;
  return min(max(given, 0), static_cast<int>(min(room, static_cast<long long>(SD_MAX_LEN))));
}

// Element offset of (page, slot) in the cache tensors.
__device__ __forceinline__ long long slot_offset(const CacheView& c, int page, int slot) {
  return page * c.page_stride + slot * c.token_stride;
}

__device__ __forceinline__ float e4m3_to_float(uint8_t b) {
  __nv_fp8_e4m3 x;
  x.__x = b;
  return static_cast<float>(x);
}
__device__ __forceinline__ float bf16_to_float(uint16_t b) {
  return __uint_as_float(static_cast<uint32_t>(b) << 16);
}
__device__ __forceinline__ uint16_t float_to_bf16(float x) {
  return __bfloat16_as_ushort(__float2bfloat16_rn(x));
}

}  // namespace sdk
