// q4_project.cu -- the head projection through a 4-bit table (lmh_project_q4).
//
//   out[n][v] = logit_scale * sum_g scale[v][g] * sum_{h in g} (q[v][h] - zero[v][g]) * x[n][h]
//
// For the batches of a decode step (up to a few dozen rows) the table is the
// traffic: V * H/2 bytes, read once.  The products run on mma.sync m16n8k16
// with 16 table rows as the A operand and 8 hidden rows as the B operand, so a
// single hidden row costs the same instructions as eight.  The A operand is
// built in registers: a pair of entries of a word becomes a pair of 16-bit
// floats by one logic operation (128 + q in bf16, 1024 + q in f16, both exact)
// and one packed subtraction of 128 + zero (exact: q - zero is a small whole
// number).  One group's sum stays in the MMA's fp32 accumulator; the group's
// scale is applied to it in fp32, so no product of scale and entry is rounded to
// 16 bits.
//
// The order of a group's entries within an MMA is free as long as A and B agree.
// Lane c of a row's four lanes takes the group / 4 consecutive entries
// c * group/4 .. of a group -- one 4, 8 or 16-byte load for groups of 32, 64
// and 128 -- and pair i of a word is its entries (i, i + 4).  The hidden rows lie
// in shared memory in exactly that order, 16 bytes per lane and word.
#include <cmath>

#include "device_common.cuh"
#include "lmh_internal.h"
#include "q4_common.cuh"

namespace lmh {

namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kRowsPerWarp = 16;
constexpr int kRowsPerTile = kRowsPerWarp * kWarps;
constexpr size_t kSmemMax = 200 * 1024;

template <typename T>
struct Half2;
template <>
struct Half2<__nv_bfloat16> {
  static constexpr uint32_t kMagic = 0x43004300u;  // 128 (+ q) in both halves
  static __device__ __forceinline__ uint32_t offset(int zero) { return 0x43004300u + 0x00010001u * zero; }
  static __device__ __forceinline__ uint32_t sub(uint32_t a, uint32_t b) {
    const __nv_bfloat162 r =
        __hsub2(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
  }
  static __device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
};
template <>
struct Half2<__half> {
  static constexpr uint32_t kMagic = 0x64006400u;  // 1024 (+ q) in both halves
  static __device__ __forceinline__ uint32_t offset(int zero) { return 0x64006400u + 0x00010001u * zero; }
  static __device__ __forceinline__ uint32_t sub(uint32_t a, uint32_t b) {
    const __half2 r = __hsub2(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
  }
  static __device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
};

// One lane's words of one group of one table row.
template <int W>
struct Words {
  uint32_t w[W];
};
template <int W>
__device__ __forceinline__ Words<W> load_words(const unsigned char* p) {
  Words<W> r;
  if constexpr (W == 1) {
    r.w[0] = __ldg(reinterpret_cast<const uint32_t*>(p));
  } else if constexpr (W == 2) {
    const uint2 x = __ldg(reinterpret_cast<const uint2*>(p));
    r.w[0] = x.x;
    r.w[1] = x.y;
  } else {
    const uint4 x = __ldg(reinterpret_cast<const uint4*>(p));
    r.w[0] = x.x;
    r.w[1] = x.y;
    r.w[2] = x.z;
    r.w[3] = x.w;
  }
  return r;
}

// W: words per lane and group (group / 32).  NT: tiles of 8 hidden rows per pass
// (blockIdx.y counts passes).  A warp owns 16 table rows at a time; a CTA's
// shared memory holds `slab` groups of its pass's hidden rows.
template <typename T, int W, int NT>
__global__ void __launch_bounds__(kThreads)
    project_q4_kernel(const T* __restrict__ hidden, int64_t hidden_stride, int num_tokens,
                      const int32_t* __restrict__ row_idx, int rows, Q4View t, int slab, float logit_scale,
                      void* __restrict__ out, int out_f32, int64_t out_stride, uint32_t* dev_status) {
  constexpr int G = 32 * W;
  extern __shared__ uint4 smem[];  // [slab groups][W][NT][32 lanes]
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int gid = lane >> 2, c = lane & 3;
  const int n0 = blockIdx.y * 8 * NT;
  const int groups = t.H / G;
  pdl_wait();
  pdl_launch_dependents();

  // Hidden rows n0.. of groups [g0, g0 + ng) into shared memory, in MMA order.
  auto stage = [&](int g0, int ng) {
    const int items = ng * W * NT * 32;
    for (int i = threadIdx.x; i < items; i += kThreads) {
      const int l = i & 31, nt = (i >> 5) % NT, wq = ((i >> 5) / NT) % W, g = (i >> 5) / (NT * W);
      const int n = n0 + nt * 8 + (l >> 2);
      const int h = (g0 + g) * G + (l & 3) * (G / 4) + wq * 8;
      uint32_t x[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = 0;
      if (n < rows) {
        const int r = row_idx ? row_idx[n] : n;
        if (r >= 0 && r < num_tokens) {
          const uint16_t* src = reinterpret_cast<const uint16_t*>(hidden) + r * hidden_stride + h;
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] = src[e];
        } else if (h == 0) {
          set_status(dev_status, LMH_DS_ROW_IDX_OUT_OF_RANGE);
        }
      }
      smem[i] = make_uint4(x[0] | (x[4] << 16), x[1] | (x[5] << 16), x[2] | (x[6] << 16), x[3] | (x[7] << 16));
    }
  };

  const bool resident = slab >= groups;
  if (resident) {
    stage(0, groups);
    __syncthreads();
  }
  const int tiles = (t.V + kRowsPerTile - 1) / kRowsPerTile;
  for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const int v0 = tile * kRowsPerTile + warp * kRowsPerWarp;
    const int va = min(v0 + gid, t.V - 1), vb = min(v0 + gid + 8, t.V - 1);  // rows past V repeat the last one
    const unsigned char* pa = t.packed + va * t.packed_row_bytes + c * 4 * W;
    const unsigned char* pb = t.packed + vb * t.packed_row_bytes + c * 4 * W;
    float acc[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[nt][e] = 0.0f;
    for (int g0 = 0; g0 < groups; g0 += slab) {
      const int ng = min(slab, groups - g0);
      if (!resident) {
        __syncthreads();
        stage(g0, ng);
        __syncthreads();
      }
      for (int g = 0; g < ng; ++g) {
        const Words<W> xa = load_words<W>(pa + (g0 + g) * (G / 2));
        const Words<W> xb = load_words<W>(pb + (g0 + g) * (G / 2));
        const float sa = load_as_f32(t.scales, t.scale_dtype, va * t.scale_row_stride + g0 + g);
        const float sb = load_as_f32(t.scales, t.scale_dtype, vb * t.scale_row_stride + g0 + g);
        const uint32_t za = Half2<T>::offset(q4_zero(t, va, g0 + g));
        const uint32_t zb = Half2<T>::offset(q4_zero(t, vb, g0 + g));
        float d[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) d[nt][e] = 0.0f;
#pragma unroll
        for (int wq = 0; wq < W; ++wq) {
          uint32_t a[2][4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t qa = ((xa.w[wq] >> (4 * i)) & 0x000F000Fu) | Half2<T>::kMagic;
            const uint32_t qb = ((xb.w[wq] >> (4 * i)) & 0x000F000Fu) | Half2<T>::kMagic;
            a[i >> 1][2 * (i & 1)] = Half2<T>::sub(qa, za);
            a[i >> 1][2 * (i & 1) + 1] = Half2<T>::sub(qb, zb);
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const uint4 b = smem[((g * W + wq) * NT + nt) * 32 + lane];
            Half2<T>::mma(d[nt], a[0], b.x, b.y);
            Half2<T>::mma(d[nt], a[1], b.z, b.w);
          }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          acc[nt][0] = fmaf(sa, d[nt][0], acc[nt][0]);
          acc[nt][1] = fmaf(sa, d[nt][1], acc[nt][1]);
          acc[nt][2] = fmaf(sb, d[nt][2], acc[nt][2]);
          acc[nt][3] = fmaf(sb, d[nt][3], acc[nt][3]);
        }
      }
    }
    // lane (gid, c) holds table rows gid and gid + 8 of hidden rows 2c and 2c + 1
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int n = n0 + nt * 8 + 2 * c + (e & 1), v = v0 + gid + 8 * (e >> 1);
        if (n < rows && v < t.V) {
          const float y = logit_scale * acc[nt][e];
          if (out_f32)
            static_cast<float*>(out)[n * out_stride + v] = y;
          else
            static_cast<T*>(out)[n * out_stride + v] = static_cast<T>(y);
        }
      }
  }
}

template <typename T, int W, int NT>
cudaError_t launch_one(const void* hidden, int64_t hidden_stride, int num_tokens, const int32_t* row_idx, int rows,
                       const lmh_q4_table& t, float logit_scale, void* out, bool out_f32, int64_t out_stride,
                       uint32_t* dev_status, int num_sms, cudaStream_t stream) {
  const int groups = t.H / (32 * W);
  const size_t group_bytes = static_cast<size_t>(W) * NT * 32 * 16;
  int slab = static_cast<int>(kSmemMax / group_bytes);
  if (slab > groups) slab = groups;
  const size_t smem = group_bytes * slab;
  const int per_sm = smem > 100 * 1024 ? 1 : (smem > 64 * 1024 ? 2 : 3);
  const int tiles = (t.V + kRowsPerTile - 1) / kRowsPerTile;
  const int passes = (rows + 8 * NT - 1) / (8 * NT);
  int grid = num_sms * per_sm;
  if (grid > tiles) grid = tiles;
  return launch_kernel(project_q4_kernel<T, W, NT>, dim3(grid, passes), dim3(kThreads), smem, stream, true,
                       static_cast<const T*>(hidden), hidden_stride, num_tokens, row_idx, rows, q4_view(t), slab,
                       logit_scale, out, out_f32 ? 1 : 0, out_stride, dev_status);
}

template <typename T, int W>
cudaError_t launch_rows(const void* hidden, int64_t hidden_stride, int num_tokens, const int32_t* row_idx, int rows,
                        const lmh_q4_table& t, float logit_scale, void* out, bool out_f32, int64_t out_stride,
                        uint32_t* dev_status, int num_sms, cudaStream_t stream) {
  if (rows <= 8)
    return launch_one<T, W, 1>(hidden, hidden_stride, num_tokens, row_idx, rows, t, logit_scale, out, out_f32,
                               out_stride, dev_status, num_sms, stream);
  if (rows <= 16)
    return launch_one<T, W, 2>(hidden, hidden_stride, num_tokens, row_idx, rows, t, logit_scale, out, out_f32,
                               out_stride, dev_status, num_sms, stream);
  return launch_one<T, W, 4>(hidden, hidden_stride, num_tokens, row_idx, rows, t, logit_scale, out, out_f32,
                             out_stride, dev_status, num_sms, stream);
}

template <typename T>
cudaError_t launch_group(const void* hidden, int64_t hidden_stride, int num_tokens, const int32_t* row_idx, int rows,
                         const lmh_q4_table& t, float logit_scale, void* out, bool out_f32, int64_t out_stride,
                         uint32_t* dev_status, int num_sms, cudaStream_t stream) {
  if (t.group == 32)
    return launch_rows<T, 1>(hidden, hidden_stride, num_tokens, row_idx, rows, t, logit_scale, out, out_f32,
                             out_stride, dev_status, num_sms, stream);
  if (t.group == 64)
    return launch_rows<T, 2>(hidden, hidden_stride, num_tokens, row_idx, rows, t, logit_scale, out, out_f32,
                             out_stride, dev_status, num_sms, stream);
  return launch_rows<T, 4>(hidden, hidden_stride, num_tokens, row_idx, rows, t, logit_scale, out, out_f32, out_stride,
                           dev_status, num_sms, stream);
}

template <typename T, int W, int NT>
cudaError_t set_one() {
  return cudaFuncSetAttribute(project_q4_kernel<T, W, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              static_cast<int>(kSmemMax));
}
template <typename T>
cudaError_t set_type() {
  cudaError_t e = cudaSuccess;
  if (e == cudaSuccess) e = set_one<T, 1, 1>();
  if (e == cudaSuccess) e = set_one<T, 1, 2>();
  if (e == cudaSuccess) e = set_one<T, 1, 4>();
  if (e == cudaSuccess) e = set_one<T, 2, 1>();
  if (e == cudaSuccess) e = set_one<T, 2, 2>();
  if (e == cudaSuccess) e = set_one<T, 2, 4>();
  if (e == cudaSuccess) e = set_one<T, 4, 1>();
  if (e == cudaSuccess) e = set_one<T, 4, 2>();
  if (e == cudaSuccess) e = set_one<T, 4, 4>();
  return e;
}

}  // namespace

cudaError_t q4_project_setup() {
  const cudaError_t e = set_type<__nv_bfloat16>();
  return e == cudaSuccess ? set_type<__half>() : e;
}

cudaError_t launch_project_q4(const void* hidden, lmh_dtype hidden_dtype, int64_t hidden_stride, int num_tokens,
                              const int32_t* row_idx, int rows, const lmh_q4_table& t, float logit_scale, void* out,
                              lmh_dtype out_dtype, int64_t out_stride, uint32_t* dev_status, int num_sms,
                              cudaStream_t stream) {
  const bool f32 = out_dtype == LMH_F32;
  if (hidden_dtype == LMH_BF16)
    return launch_group<__nv_bfloat16>(hidden, hidden_stride, num_tokens, row_idx, rows, t, logit_scale, out, f32,
                                       out_stride, dev_status, num_sms, stream);
  return launch_group<__half>(hidden, hidden_stride, num_tokens, row_idx, rows, t, logit_scale, out, f32, out_stride,
                              dev_status, num_sms, stream);
}

}  // namespace lmh
