// Pieces shared by the kernels over the paged e4m3 KV cache.
#pragma once

#include <cuda_fp16.h>

#include "ssv_internal.cuh"

namespace ssv {

// A record without rows (an ended or refused request): skipped without an error.
__host__ __device__ __forceinline__ bool seq_idle(const ssv_seq& s) { return s.new_len == 0 && s.block == 0; }

__host__ __device__ __forceinline__ bool page_size_ok(int ps) { return ps == 16 || ps == 32 || ps == 64 || ps == 128; }

inline int ilog2(int x) {
  int n = 0;
  while ((1 << n) < x) ++n;
  return n;
}

// two e4m3 codes (low byte first) -> two fp16 values, exact
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint16_t c) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(c));
  return r;
}

// two fp32 values -> two e4m3 codes (lo in the low byte), nearest even, clamped to +-448, NaN to NaN
__device__ __forceinline__ uint16_t f32_to_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

}  // namespace ssv
