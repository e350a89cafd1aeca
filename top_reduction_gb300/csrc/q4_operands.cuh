// q4_operands.cuh -- what the two kernels of lmh_project_q4 share: their tiles and
// arguments, and the way the hidden rows are held.
#pragma once

#include <cmath>

#include "device_common.cuh"
#include "lmh_internal.h"
#include "q4_common.cuh"
#include "tma.cuh"

namespace lmh {

constexpr int kQ4TileRows = 128;
constexpr int kQ4RowGroups = kQ4TileRows / 32;
constexpr int kQ4BoxBytes = 128;                       // of a row
constexpr int kQ4BoxEntries = 2 * kQ4BoxBytes;
constexpr int kQ4BoxBlocks = kQ4BoxEntries / 32;
constexpr int kQ4StageBytes = kQ4TileRows * kQ4BoxBytes;
constexpr int kQ4MaxStages = 12;
constexpr size_t kQ4SmemMax = 227 * 1024;

struct Q4ProjectArgs {
  const void* hidden;
  int64_t hidden_stride;
  int num_tokens;
  const int32_t* row_idx;
  int rows;
  bool vec;  // hidden rows can be read 16 bytes at a time
  Q4View t;
  float logit_scale;
  void* out;
  bool out_f32;
  int64_t out_stride;
  uint32_t* dev_status;
  int stages;       // of the ring
  int slab;         // boxes of hidden rows in shared memory at once
  bool scale_vec;   // a row's scales can be read eight at a time
  uint64_t wait_ns;
};

__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }

// Eight hidden values (from 16-byte vectors, or one by one).
template <typename T>
__device__ __forceinline__ void load_hidden(const T* src, bool vec, float (&x)[8]) {
  alignas(16) T v[8];
  if (vec) {
    *reinterpret_cast<uint4*>(v) = __ldg(reinterpret_cast<const uint4*>(src));
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = src[e];
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] = to_f32(v[e]);
}

__device__ __forceinline__ uint32_t half2_bits(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// 2^e for e in [-149, 127]
__device__ __forceinline__ float pow2(int e) {
  return e >= -126 ? __int_as_float((e + 127) << 23) : __int_as_float(1 << (e + 149));
}

}  // namespace lmh
