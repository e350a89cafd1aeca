// logits_vec.cuh -- 16-byte vectors of logits (bf16, f16 or f32) widened to fp32.
#pragma once

#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cuda_runtime.h>

namespace lmh {

template <typename T>
struct Vec16;  // 16-byte vector of T widened to fp32

template <>
struct Vec16<__nv_bfloat16> {
  static constexpr int N = 8;
  static constexpr uint32_t kNegInfWord = 0xFF80FF80u;  // two bf16 -inf
  __device__ __forceinline__ static void load(const void* p, float* x) { unpack(*reinterpret_cast<const uint4*>(p), x); }
  __device__ __forceinline__ static void unpack(const uint4 w, float* x) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(u[i] << 16);
      x[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
    }
  }
  // maximum of 8 vectors, pairwise on packed bf16x2 (exact)
  __device__ __forceinline__ static float max8(const uint4* w) {
    __nv_bfloat162 m[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t* a = reinterpret_cast<const uint32_t*>(&w[2 * i]);
      const uint32_t* b = reinterpret_cast<const uint32_t*>(&w[2 * i + 1]);
      __nv_bfloat162 t0 = __hmax2(as2(a[0]), as2(a[1])), t1 = __hmax2(as2(a[2]), as2(a[3]));
      __nv_bfloat162 t2 = __hmax2(as2(b[0]), as2(b[1])), t3 = __hmax2(as2(b[2]), as2(b[3]));
      m[i] = __hmax2(__hmax2(t0, t1), __hmax2(t2, t3));
    }
    const __nv_bfloat162 r = __hmax2(__hmax2(m[0], m[1]), __hmax2(m[2], m[3]));
    return fmaxf(__low2float(r), __high2float(r));
  }
  // the vector as 4 pairs of fp32 values
  __device__ __forceinline__ static void pairs(const uint4 w, float2* p) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = make_float2(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xFFFF0000u));
  }
  __device__ __forceinline__ static __nv_bfloat162 as2(uint32_t u) {
    return *reinterpret_cast<const __nv_bfloat162*>(&u);
  }
  __device__ __forceinline__ static float at(const void* base, int64_t i) {
    const uint16_t b = reinterpret_cast<const uint16_t*>(base)[i];
    return __uint_as_float(static_cast<uint32_t>(b) << 16);
  }
};

template <>
struct Vec16<__half> {
  static constexpr int N = 8;
  static constexpr uint32_t kNegInfWord = 0xFC00FC00u;  // two f16 -inf
  __device__ __forceinline__ static void load(const void* p, float* x) { unpack(*reinterpret_cast<const uint4*>(p), x); }
  __device__ __forceinline__ static void unpack(const uint4 w, float* x) {
    const __half2* h = reinterpret_cast<const __half2*>(&w);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(h[i]);
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
  __device__ __forceinline__ static void pairs(const uint4 w, float2* p) {
    const __half2* h = reinterpret_cast<const __half2*>(&w);
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = __half22float2(h[i]);
  }
  __device__ __forceinline__ static float max8(const uint4* w) {
    const __half2* h = reinterpret_cast<const __half2*>(w);
    __half2 m[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2* p = h + 8 * i;
      m[i] = __hmax2(__hmax2(__hmax2(p[0], p[1]), __hmax2(p[2], p[3])),
                     __hmax2(__hmax2(p[4], p[5]), __hmax2(p[6], p[7])));
    }
    const __half2 r = __hmax2(__hmax2(m[0], m[1]), __hmax2(m[2], m[3]));
    return fmaxf(__low2float(r), __high2float(r));
  }
  __device__ __forceinline__ static float at(const void* base, int64_t i) {
    return __half2float(reinterpret_cast<const __half*>(base)[i]);
  }
};

template <>
struct Vec16<float> {
  static constexpr int N = 4;
  static constexpr uint32_t kNegInfWord = 0xFF800000u;
  __device__ __forceinline__ static void load(const void* p, float* x) { unpack(*reinterpret_cast<const uint4*>(p), x); }
  __device__ __forceinline__ static void unpack(const uint4 w, float* x) {
    x[0] = __uint_as_float(w.x);
    x[1] = __uint_as_float(w.y);
    x[2] = __uint_as_float(w.z);
    x[3] = __uint_as_float(w.w);
  }
  __device__ __forceinline__ static void pairs(const uint4 w, float2* p) {
    p[0] = make_float2(__uint_as_float(w.x), __uint_as_float(w.y));
    p[1] = make_float2(__uint_as_float(w.z), __uint_as_float(w.w));
  }
  __device__ __forceinline__ static float max8(const uint4* w) {
    float m[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint4 a = w[2 * i], b = w[2 * i + 1];
      m[i] = fmaxf(fmaxf(fmaxf(__uint_as_float(a.x), __uint_as_float(a.y)), fmaxf(__uint_as_float(a.z), __uint_as_float(a.w))),
                   fmaxf(fmaxf(__uint_as_float(b.x), __uint_as_float(b.y)), fmaxf(__uint_as_float(b.z), __uint_as_float(b.w))));
    }
    return fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
  }
  __device__ __forceinline__ static float at(const void* base, int64_t i) {
    return reinterpret_cast<const float*>(base)[i];
  }
};

template <typename T>
__device__ __forceinline__ T neg_inf();
template <>
__device__ __forceinline__ __nv_bfloat16 neg_inf<__nv_bfloat16>() {
  return __ushort_as_bfloat16(static_cast<unsigned short>(0xFF80u));
}
template <>
__device__ __forceinline__ __half neg_inf<__half>() {
  return __ushort_as_half(static_cast<unsigned short>(0xFC00u));
}
template <>
__device__ __forceinline__ float neg_inf<float>() {
  return -INFINITY;
}

}  // namespace lmh
