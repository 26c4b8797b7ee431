// Device helpers of the paged-cache kernels.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"
#include "paged.h"

namespace infllmv2 {

constexpr uint32_t kStatusBadPage = 0x8u;

// A sequence's length, or 0 (flagged) where it is outside [0, cap].
__device__ __forceinline__ int paged_len(const int32_t* kv_lens, int b, int cap, uint32_t* status) {
  const int n = kv_lens[b];
  if (n >= 0 && n <= cap) return n;
  atomicOr(status, kStatusBadKvLen);
  return 0;
}

// Index of (page, head, row) in weights / positions.
__device__ __forceinline__ long long paged_meta(int page, int h, int row, int Hkv, int ps) {
  return (static_cast<long long>(page) * Hkv + h) * ps + row;
}

}  // namespace infllmv2
