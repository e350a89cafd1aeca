// q4_table.cu -- making a 4-bit table (lmh_quantize_q4) and looking rows of it
// up (lmh_lookup_q4).
//
// Both walk the table eight entries (one 32-bit word) at a time: a thread that
// owns a word reads 16 bytes of bf16 and writes 4, or reads 4 bytes and writes
// 16 (or 32) bytes of output, so that a warp's reads and writes are each one
// contiguous piece of a row.
#include <cmath>

#include "device_common.cuh"
#include "lmh_internal.h"
#include "q4_common.cuh"

namespace lmh {

namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ void store_scale(void* p, int dtype, int64_t i, float s) {
  if (dtype == LMH_BF16)
    static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(s);
  else if (dtype == LMH_F16)
    static_cast<__half*>(p)[i] = __float2half_rn(s);
  else
    static_cast<float*>(p)[i] = s;
}

// The value a scale has once it is stored.
__device__ __forceinline__ float round_to(float s, int dtype) {
  if (dtype == LMH_BF16) return __bfloat162float(__float2bfloat16_rn(s));
  if (dtype == LMH_F16) return __half2float(__float2half_rn(s));
  return s;
}

// One word (eight entries) per thread; the group / 8 threads of a group are
// neighbours in a warp and share their extremes by shuffles.  Words are numbered
// over the whole table; H is a multiple of the group, so a group never splits.
// 151936 x 2560 bf16, group 64: 516 us with cold L2 (145 at the copy rate), 553 with zero
// points; done once per table, and not worked on.
__global__ void __launch_bounds__(kThreads)
    quantize_q4_kernel(const __nv_bfloat16* __restrict__ W, int64_t w_stride, bool vec, int V, int H, int group,
                       uint8_t* packed, int64_t packed_row_bytes, void* scales, int scale_dtype,
                       int64_t scale_row_stride, uint8_t* zeros, int64_t zero_row_stride) {
  pdl_wait();
  const int words = H / 8;
  const int64_t total = static_cast<int64_t>(V) * words;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kThreads;
  for (int64_t base = static_cast<int64_t>(blockIdx.x) * kThreads; base < total; base += stride) {
    const int64_t i = base + threadIdx.x;
    const bool in = i < total;
    const int64_t v = in ? i / words : 0;
    const int j = in ? static_cast<int>(i - v * words) : 0;
    float w[8];
    float hi = 0.0f, lo = 0.0f;  // the extremes, with 0 among them
    if (in) {
      const __nv_bfloat16* src = W + v * w_stride + 8 * j;
      if (vec) {
        const uint4 x = *reinterpret_cast<const uint4*>(src);
        const uint32_t u[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          w[2 * e] = __uint_as_float(u[e] << 16);
          w[2 * e + 1] = __uint_as_float(u[e] & 0xFFFF0000u);
        }
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = __bfloat162float(src[e]);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        hi = fmaxf(hi, w[e]);
        lo = fminf(lo, w[e]);
      }
    }
    for (int o = group / 16; o > 0; o >>= 1) {
      hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
      lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    }
    if (!in) continue;
    const float s = round_to(zeros ? (hi - lo) / 15.0f : fmaxf(hi, -lo) / 7.0f, scale_dtype);
    float zero = 8.0f;
    if (zeros) zero = s > 0.0f ? fminf(fmaxf(rintf(-lo / s), 0.0f), 15.0f) : 0.0f;
    uint32_t q = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float r = s > 0.0f ? rintf(w[e] / s) : 0.0f;
      q |= static_cast<uint32_t>(fminf(fmaxf(r + zero, 0.0f), 15.0f)) << (4 * e);
    }
    *reinterpret_cast<uint32_t*>(packed + v * packed_row_bytes + 4 * j) = q;
    if ((8 * j) % group == 0) {
      const int g = 8 * j / group;
      store_scale(scales, scale_dtype, v * scale_row_stride + g, s);
      if (zeros) zeros[v * zero_row_stride + g] = static_cast<uint8_t>(zero);
    }
  }
}

template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) {
  return x;
}
template <>
__device__ __forceinline__ __half from_f32<__half>(float x) {
  return __float2half_rn(x);
}
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) {
  return __float2bfloat16_rn(x);
}

// One thread per word of an output row.  Reads H/2 bytes and a row's scales, writes H
// elements.  A decode batch is launch latency; for prompts it is mostly the instructions
// (issue slots 73% busy, about 165 for a warp's words: an id, a scale, a zero point and
// their addresses for every eight entries), beside the chain of two loads (the id, then word,
// scale and zero): 16384 rows of 1024 entries take 16.4 us with cold L2 (13.4 in a row of
// calls: 3.3 TB/s).  64-bit
// divisions per word and conversions of q - zero took 0.4 us more.  Measured and dropped:
// two or four words of a thread in flight at once on fewer blocks (18.4 and 24.6 us), 128
// or 512 threads a block, or a block for every 256 words (22.5, 20.5 and 18.4 us).
template <typename T>
__global__ void __launch_bounds__(kThreads)
    lookup_q4_kernel(const int32_t* __restrict__ ids, int n, Q4View t, int group_shift, float scale, T* __restrict__ out,
                     int64_t out_stride, bool vec, uint32_t* dev_status) {
  pdl_wait();
  // The grid has fewer than 2^31 threads, so a thread's first word is found by one
  // 32-bit division, and the next ones by adding the step's rows and words.
  const uint32_t words = t.H / 8;
  const uint32_t first = blockIdx.x * kThreads + threadIdx.x, step = gridDim.x * kThreads;
  const uint32_t step_rows = step / words;
  const int step_words = static_cast<int>(step - step_rows * words);
  int64_t row = first / words;
  int j = static_cast<int>(first - static_cast<uint32_t>(row) * words);
  for (; row < n; row += step_rows, j += step_words) {
    if (j >= static_cast<int>(words)) {
      j -= static_cast<int>(words);
      if (++row >= n) break;
    }
    const int id = ids[row];
    alignas(16) T y[8];
    if (id >= 0 && id < t.V) {
      const int64_t v = id;
      const int g = 8 * j >> group_shift;
      const uint32_t q = *reinterpret_cast<const uint32_t*>(t.packed + v * t.packed_row_bytes + 4 * j);
      const float s = load_as_f32(t.scales, t.scale_dtype, v * t.scale_row_stride + g);
      // 2^23 + q less 2^23 + zero, in place of a conversion of q - zero
      const float zero = 8388608.0f + static_cast<float>(q4_zero(t, v, g));
#pragma unroll
      for (int e = 0; e < 8; ++e)
        y[e] = from_f32<T>(__fmul_rn(
            __fmul_rn(__uint_as_float(0x4B000000u | ((q >> (4 * e)) & 15u)) - zero, s), scale));
    } else {
      if (j == 0 && id != -1) set_status(dev_status, LMH_DS_SEL_OUT_OF_RANGE);
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = from_f32<T>(0.0f);
    }
    T* dst = out + row * out_stride + 8 * j;
    if (vec) {
      const uint4* src = reinterpret_cast<const uint4*>(y);
#pragma unroll
      for (int e = 0; e < static_cast<int>(sizeof(y) / 16); ++e) reinterpret_cast<uint4*>(dst)[e] = src[e];
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) dst[e] = y[e];
    }
  }
}

template <typename T>
cudaError_t launch_lookup(const int32_t* ids, int n, const lmh_q4_table& t, float scale, void* out, int64_t out_stride,
                          uint32_t* dev_status, int num_sms, cudaStream_t stream) {
  const bool vec = reinterpret_cast<uintptr_t>(out) % 16 == 0 && (out_stride * sizeof(T)) % 16 == 0;
  const int64_t words = static_cast<int64_t>(n) * (t.H / 8);
  int64_t blocks = (words + kThreads - 1) / kThreads;
  const int64_t cap = static_cast<int64_t>(num_sms) * 32;
  if (blocks > cap) blocks = cap;
  return launch_kernel(lookup_q4_kernel<T>, dim3(static_cast<unsigned>(blocks)), dim3(kThreads), 0, stream, true, ids,
                       n, q4_view(t), t.group == 32 ? 5 : t.group == 64 ? 6 : 7, scale, static_cast<T*>(out), out_stride, vec,
                       dev_status);
}

}  // namespace

cudaError_t launch_quantize_q4(const void* W, int64_t w_stride, const lmh_q4_table& t, cudaStream_t stream) {
  const bool vec = reinterpret_cast<uintptr_t>(W) % 16 == 0 && w_stride % 8 == 0;
  const int64_t words = static_cast<int64_t>(t.V) * (t.H / 8);
  int64_t blocks = (words + kThreads - 1) / kThreads;
  if (blocks > (1 << 20)) blocks = 1 << 20;
  return launch_kernel(quantize_q4_kernel, dim3(static_cast<unsigned>(blocks)), dim3(kThreads), 0, stream, true,
                       static_cast<const __nv_bfloat16*>(W), w_stride, vec, static_cast<int>(t.V),
                       static_cast<int>(t.H), static_cast<int>(t.group),
                       static_cast<uint8_t*>(const_cast<void*>(t.packed)), t.packed_row_bytes,
                       const_cast<void*>(t.scales), static_cast<int>(t.scale_dtype), t.scale_row_stride,
                       const_cast<uint8_t*>(t.zeros), t.zero_row_stride);
}

cudaError_t launch_lookup_q4(const int32_t* ids, int n, const lmh_q4_table& t, float scale, void* out,
                             lmh_dtype out_dtype, int64_t out_stride, uint32_t* dev_status, int num_sms,
                             cudaStream_t stream) {
  if (out_dtype == LMH_BF16)
    return launch_lookup<__nv_bfloat16>(ids, n, t, scale, out, out_stride, dev_status, num_sms, stream);
  if (out_dtype == LMH_F16) return launch_lookup<__half>(ids, n, t, scale, out, out_stride, dev_status, num_sms, stream);
  return launch_lookup<float>(ids, n, t, scale, out, out_stride, dev_status, num_sms, stream);
}

}  // namespace lmh
