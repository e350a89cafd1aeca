// q4_common.cuh -- device helpers of the 4-bit table kernels.
//
// A table entry is scale * (q - zero), q in 0..15 (include/lmh.h, lmh_q4_table).
// Eight entries fill a 32-bit word, entry j in bits 4j..4j+3.
#pragma once

#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "lmh.h"

namespace lmh {

// The table as the kernels take it (by value).
struct Q4View {
  const unsigned char* packed;
  int64_t packed_row_bytes;
  const void* scales;
  int scale_dtype;  // lmh_dtype
  int64_t scale_row_stride;
  const unsigned char* zeros;  // or null: every zero is 8
  int64_t zero_row_stride;
  int V, H;
};

inline Q4View q4_view(const lmh_q4_table& t) {
  return Q4View{static_cast<const unsigned char*>(t.packed), t.packed_row_bytes, t.scales,
                static_cast<int>(t.scale_dtype), t.scale_row_stride, t.zeros, t.zero_row_stride, t.V, t.H};
}

__device__ __forceinline__ float load_as_f32(const void* p, int dtype, int64_t i) {
  if (dtype == LMH_BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
  if (dtype == LMH_F16) return __half2float(static_cast<const __half*>(p)[i]);
  return static_cast<const float*>(p)[i];
}

// Zero point of group `g` of row `v` (the low four bits of its byte).
__device__ __forceinline__ int q4_zero(const Q4View& t, int64_t v, int g) {
  return t.zeros ? (t.zeros[v * t.zero_row_stride + g] & 15) : 8;
}

}  // namespace lmh
