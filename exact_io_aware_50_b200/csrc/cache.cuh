// cache.cuh -- device helpers of the paged E4M3 cache kernels.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"
#include "launch.h"

namespace fa {

// Two E4M3 codes -> two halves; every E4M3 value is a half, so this is exact.
__device__ __forceinline__ uint32_t e4m3x2_to_half2(uint32_t codes) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((unsigned short)codes));
  return r;
}

__device__ __forceinline__ float2 e4m3x2_to_float2(uint32_t codes) {
  const uint32_t h = e4m3x2_to_half2(codes);
  return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}

// Scale of a block of tokens: the least power of two s >= 2^-112 with
// amax <= 448 s (448 = 0.875 * 2^9 is the largest E4M3 value).  amax finite.
__device__ __forceinline__ float e4m3_block_scale(float amax) {
  const uint32_t b = __float_as_uint(amax);
  const int e = (int)(b >> 23) - 126;        // amax = m 2^e with m in [1/2, 1) (normal numbers)
  const int k = e - 9 + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0);   // m > 0.875
  return __uint_as_float((uint32_t)(max(k, -112) + 127) << 23);
}

// Whether a scale is a power of two, as every scale is that an append has chosen.
__device__ __forceinline__ bool power_of_two(float s) { return (__float_as_uint(s) & 0x7FFFFFu) == 0; }

// The E4M3 code of x, rounded once: x is cut to float32 with its last bit set where
// something was cut off, which no tie between two codes has.
__device__ __forceinline__ uint32_t e4m3_code(double x) {
  const float f = __double2float_rz(x);
  return pack_e4m3x2((double)f == x ? f : __uint_as_float(__float_as_uint(f) | 1u), 0.f) & 0xFFu;
}

// Page number of a sequence's page-th page, or -1 when it is not in the cache.
__device__ __forceinline__ int checked_page(const int *table, long long at, int num_pages,
                                            unsigned *err) {
  const int pg = table[at];
  if ((unsigned)pg < (unsigned)num_pages) return pg;
  atomicOr(err, kErrPage);
  return -1;
}

// Tokens of sequence b that the cache can hold: its length, at least 0 and at
// most the table's max_pages pages.
__device__ __forceinline__ int checked_len(const int *lens, int b, int max_pages, int page,
                                           unsigned *err) {
  const int n = lens[b], most = max_pages * page;
  if (n >= 0 && n <= most) return n;
  atomicOr(err, kErrPage);
  return n < 0 ? 0 : most;
}

}  // namespace fa
