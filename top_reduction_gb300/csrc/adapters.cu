// adapters.cu -- low-rank adapters of many requests beside a shared projection (lmh_add_adapters).
//
//   out[i][n] = y[i][n] + scale_l * sum_r up[l][n][r] * d[i][r],   d[i][r] = sum_h down[l][r][h] * x[i][h]
//
// with l = adapter_idx[i].  Three kernels: the rows are sorted by adapter and cut into tiles of up to
// kADTile rows of one adapter; d of every tile; the second product, added to y.
//
// Both products run on mma.sync m16n8k16 with 16 rows of the weights as the A operand and 8 rows of the
// batch as the B operand: a batch of one row costs the same weight reads as one of eight, and weights go
// from memory to the MMA's registers without a stop in shared memory.  The order of the entries along the
// inner dimension is free as long as A and B agree, so a lane takes 16 contiguous bytes of a weight row.
//
// d enters the second product as two 16-bit parts, high and low: 16 bits (bf16) or 22 (f16) of its fp32
// value, so that its rounding stays near that of the fp32 sums.
#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "device_common.cuh"
#include "lmh_internal.h"

namespace lmh {

constexpr int kADTile = 32;       // rows of a tile
constexpr int kADCols = kADTile / 8;
constexpr int kADPlanThreads = 1024;
constexpr int kADThreads = 256;   // both products
constexpr int kADWarps = kADThreads / 32;
constexpr int kADStep = 32;       // outputs n a warp takes at a time

struct AdapterTile {
  int adapter;  // -1: rows without one
  int first;    // in `order`
  int count;
  int pad;
};

struct AdapterArgs {
  const char* x;
  int64_t x_stride;  // elements
  int num_tokens;
  const int32_t* row_idx;
  const int32_t* adapter_idx;
  int rows;
  const char* down;
  int64_t down_adapter, down_row;  // strides in elements
  const char* up;
  int64_t up_adapter, up_row;
  const float* scales;
  const int32_t* ranks;
  int count, R, H, N;
  bool x_vec;  // rows of x are 16-byte aligned
  const char* y;
  int64_t y_stride;
  char* out;
  int64_t out_stride;
  bool in_place;
  int y_vec;  // outputs that may be read and written at once: 4, or 1
  // workspace
  int32_t* tile_count;
  AdapterTile* tiles;
  int32_t* order;
  float* d;    // [splits][rows][R]
  int splits;  // of H
  uint32_t* dev_status;
};

template <typename T>
__device__ __forceinline__ void mma16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1);
template <>
__device__ __forceinline__ void mma16<__nv_bfloat16>(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma16<__half>(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <typename T>
struct Half16;  // conversions of a 16-bit type
template <>
struct Half16<__nv_bfloat16> {
  __device__ __forceinline__ static uint16_t bits(float v) { return __bfloat16_as_ushort(__float2bfloat16_rn(v)); }
  __device__ __forceinline__ static float value(uint16_t b) { return __uint_as_float(static_cast<uint32_t>(b) << 16); }
};
template <>
struct Half16<__half> {
  __device__ __forceinline__ static uint16_t bits(float v) { return __half_as_ushort(__float2half_rn(v)); }
  __device__ __forceinline__ static float value(uint16_t b) { return __half2float(__ushort_as_half(b)); }
};

template <typename Y>
__device__ __forceinline__ float y_load(const char* p, int64_t i);
template <>
__device__ __forceinline__ float y_load<float>(const char* p, int64_t i) { return reinterpret_cast<const float*>(p)[i]; }
template <>
__device__ __forceinline__ float y_load<__nv_bfloat16>(const char* p, int64_t i) {
  return Half16<__nv_bfloat16>::value(reinterpret_cast<const uint16_t*>(p)[i]);
}
template <>
__device__ __forceinline__ float y_load<__half>(const char* p, int64_t i) {
  return Half16<__half>::value(reinterpret_cast<const uint16_t*>(p)[i]);
}
template <typename Y>
__device__ __forceinline__ void y_store(char* p, int64_t i, float v) {
  reinterpret_cast<uint16_t*>(p)[i] = Half16<Y>::bits(v);
}
template <>
__device__ __forceinline__ void y_store<float>(char* p, int64_t i, float v) { reinterpret_cast<float*>(p)[i] = v; }

// four neighbours at once (16 or 8 bytes)
template <typename Y>
__device__ __forceinline__ void y_load4(const char* p, int64_t i, float (&v)[4]) {
  const uint2 w = *reinterpret_cast<const uint2*>(p + 2 * i);
  v[0] = Half16<Y>::value(w.x & 0xFFFFu), v[1] = Half16<Y>::value(w.x >> 16);
  v[2] = Half16<Y>::value(w.y & 0xFFFFu), v[3] = Half16<Y>::value(w.y >> 16);
}
template <>
__device__ __forceinline__ void y_load4<float>(const char* p, int64_t i, float (&v)[4]) {
  const float4 w = *reinterpret_cast<const float4*>(p + 4 * i);
  v[0] = w.x, v[1] = w.y, v[2] = w.z, v[3] = w.w;
}
template <typename Y>
__device__ __forceinline__ void y_store4(char* p, int64_t i, const float (&v)[4]) {
  uint2 w;
  w.x = Half16<Y>::bits(v[0]) | static_cast<uint32_t>(Half16<Y>::bits(v[1])) << 16;
  w.y = Half16<Y>::bits(v[2]) | static_cast<uint32_t>(Half16<Y>::bits(v[3])) << 16;
  *reinterpret_cast<uint2*>(p + 2 * i) = w;
}
template <>
__device__ __forceinline__ void y_store4<float>(char* p, int64_t i, const float (&v)[4]) {
  *reinterpret_cast<float4*>(p + 4 * i) = make_float4(v[0], v[1], v[2], v[3]);
}

// ---------------------------------------------------------------------------
// plan: rows by adapter, cut into tiles
// ---------------------------------------------------------------------------
// One CTA.  Counts per adapter (slot `count` holds the rows without one), a scan, the rows' places.  The
// order of an adapter's rows is whatever the atomics make it: no row's result depends on it.
__global__ void __launch_bounds__(kADPlanThreads) adapter_plan_kernel(const AdapterArgs a) {
  extern __shared__ int32_t plan_smem[];
  const int L = a.count;
  int32_t* hist = plan_smem;            // [L + 1] counts, then the next free place
  __shared__ int32_t wsum[2][kADPlanThreads / 32];
  __shared__ int32_t carry[2];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_wait();
  for (int i = tid; i <= L; i += kADPlanThreads) hist[i] = 0;
  if (tid < 2) carry[tid] = 0;
  __syncthreads();
  bool bad = false;
  auto slot = [&](int i) {
    const int l = a.adapter_idx[i];
    if (l >= 0 && l < L) return l;
    bad |= l != -1;
    return L;
  };
  for (int i = tid; i < a.rows; i += kADPlanThreads) atomicAdd(&hist[slot(i)], 1);
  __syncthreads();
  // exclusive sums of rows and of tiles over the adapters
  for (int base = 0; base <= L; base += kADPlanThreads) {
    const int l = base + tid;
    const int n = l <= L ? hist[l] : 0;
    const int nt = l == L && a.in_place ? 0 : (n + kADTile - 1) / kADTile;
    int in = n, it = nt;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int p = __shfl_up_sync(0xffffffffu, in, o), t = __shfl_up_sync(0xffffffffu, it, o);
      if (lane >= o) in += p, it += t;
    }
    if (lane == 31) wsum[0][warp] = in, wsum[1][warp] = it;
    __syncthreads();
    int before_n = carry[0] + in - n, before_t = carry[1] + it - nt;
    for (int w = 0; w < warp; ++w) before_n += wsum[0][w], before_t += wsum[1][w];
    __syncthreads();
    if (tid == kADPlanThreads - 1) carry[0] = before_n + n, carry[1] = before_t + nt;
    if (l <= L) hist[l] = before_n;
    for (int j = 0; j < nt; ++j)
      a.tiles[before_t + j] = AdapterTile{l < L ? l : -1, before_n + j * kADTile, min(kADTile, n - j * kADTile), 0};
    __syncthreads();
  }
  if (tid == 0) *a.tile_count = carry[1];
  for (int i = tid; i < a.rows; i += kADPlanThreads) a.order[atomicAdd(&hist[slot(i)], 1)] = i;
  if (bad) set_status(a.dev_status, LMH_DS_ADAPTER_OUT_OF_RANGE);
}

// ---------------------------------------------------------------------------
// first product
// ---------------------------------------------------------------------------
// One CTA a (tile, share of H): its warps take blocks of 32 entries of H in turn; their sums meet in
// shared memory in a fixed order.  RT: tiles of 16 adapter rows.
template <typename T, int RT>
__global__ void __launch_bounds__(kADThreads) adapter_down_kernel(const AdapterArgs a) {
  extern __shared__ float down_smem[];  // [kADWarps][RT * 16][kADTile]
  __shared__ int32_t tok[kADTile];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  pdl_wait();
  pdl_launch_dependents();
  const int n_tiles = *a.tile_count;
  const int split = blockIdx.y;
  const int blocks = (a.H + 31) / 32;
  const int lo = static_cast<int>(static_cast<int64_t>(blocks) * split / a.splits);
  const int hi = static_cast<int>(static_cast<int64_t>(blocks) * (split + 1) / a.splits);
  for (int ti = blockIdx.x; ti < n_tiles; ti += gridDim.x) {
    const AdapterTile tile = a.tiles[ti];
    if (tile.adapter < 0) continue;  // (uniform)
    const int rank = a.ranks ? min(max(a.ranks[tile.adapter], 0), a.R) : a.R;
    if (tid < kADTile) {
      int tk = -1;
      if (tid < tile.count) {
        const int row = a.order[tile.first + tid];
        tk = a.row_idx ? a.row_idx[row] : row;
        if (tk < 0 || tk >= a.num_tokens) {
          tk = -1;  // reads zeros
          set_status(a.dev_status, LMH_DS_ROW_IDX_OUT_OF_RANGE);
        }
      }
      tok[tid] = tk;
    }
    __syncthreads();
    const int cols = (tile.count + 7) / 8;
    const T* down = reinterpret_cast<const T*>(a.down) + static_cast<int64_t>(tile.adapter) * a.down_adapter;
    float acc[RT][kADCols][4] = {};
    for (int kb = lo + warp; kb < hi; kb += kADWarps) {
      const int h = kb * 32 + t * 8;  // H is a multiple of 8
      uint4 xv[kADCols];
#pragma unroll
      for (int c = 0; c < kADCols; ++c) {
        xv[c] = make_uint4(0, 0, 0, 0);
        const int tk = tok[c * 8 + g];
        if (c < cols && tk >= 0 && h < a.H) {
          const T* p = reinterpret_cast<const T*>(a.x) + static_cast<int64_t>(tk) * a.x_stride + h;
          if (a.x_vec) {
            xv[c] = *reinterpret_cast<const uint4*>(p);
          } else {
            const uint16_t* e = reinterpret_cast<const uint16_t*>(p);
            xv[c] = make_uint4(e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6] | e[7] << 16);
          }
        }
      }
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        const int r0 = rt * 16 + g;
        uint4 w0 = make_uint4(0, 0, 0, 0), w1 = w0;
        if (h < a.H) {
          if (r0 < rank) w0 = *reinterpret_cast<const uint4*>(down + r0 * a.down_row + h);
          if (r0 + 8 < rank) w1 = *reinterpret_cast<const uint4*>(down + (r0 + 8) * a.down_row + h);
        }
        const uint32_t a0[4] = {w0.x, w1.x, w0.y, w1.y}, a1[4] = {w0.z, w1.z, w0.w, w1.w};
#pragma unroll
        for (int c = 0; c < kADCols; ++c) {
          if (c < cols) {
            mma16<T>(acc[rt][c], a0, xv[c].x, xv[c].y);
            mma16<T>(acc[rt][c], a1, xv[c].z, xv[c].w);
          }
        }
      }
    }
    float* mine = down_smem + warp * (RT * 16 * kADTile);
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
      for (int c = 0; c < kADCols; ++c)
        if (c < cols) {
          float* p = mine + (rt * 16 + g) * kADTile + c * 8 + 2 * t;
          *reinterpret_cast<float2*>(p) = make_float2(acc[rt][c][0], acc[rt][c][1]);
          *reinterpret_cast<float2*>(p + 8 * kADTile) = make_float2(acc[rt][c][2], acc[rt][c][3]);
        }
    __syncthreads();
    float* d = a.d + (static_cast<int64_t>(split) * a.rows + tile.first) * a.R;
    for (int i = tid; i < tile.count * a.R; i += kADThreads) {
      const int row = i / a.R, r = i - row * a.R;
      float s = 0.0f;
#pragma unroll
      for (int w = 0; w < kADWarps; ++w) s += down_smem[w * (RT * 16 * kADTile) + r * kADTile + row];
      d[i] = s;
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------
// second product, added to y
// ---------------------------------------------------------------------------
// A warp takes 32 outputs at a time, as two MMAs of 16 weight rows: rows n0 + 4g and n0 + 4g + 1 are row g and
// g + 8 of the first, n0 + 4g + 2 and + 3 of the second, so that a lane's results for a batch row are four
// neighbours.  KS: k16 steps (1: ranks to 16, lanes take 8 bytes of a weight row; else 16 bytes of 32 entries).
template <typename T, typename Y, int KS>
__global__ void __launch_bounds__(kADThreads) adapter_up_kernel(const AdapterArgs a, int chunk, int n_chunks) {
  __shared__ uint4 frag[KS][kADCols][32];  // d in MMA order: high parts (b0, b1), low parts (b0, b1)
  __shared__ int32_t rows[kADTile];
  __shared__ float unscale[kADTile];       // f16: the power of two that a row's d was divided by
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  pdl_wait();
  const int n_tiles = *a.tile_count;
  const int64_t items = static_cast<int64_t>(n_tiles) * n_chunks;
  // every CTA takes a contiguous share, so that it seldom changes tiles
  const int64_t i0 = items * blockIdx.x / gridDim.x, i1 = items * (blockIdx.x + 1) / gridDim.x;
  int held = -1;
  AdapterTile tile{};
  int rank = 0, cols = 0;
  for (int64_t it = i0; it < i1; ++it) {
    const int ti = static_cast<int>(it / n_chunks), ci = static_cast<int>(it - static_cast<int64_t>(ti) * n_chunks);
    if (ti != held) {
      __syncthreads();
      held = ti;
      tile = a.tiles[ti];
      cols = (tile.count + 7) / 8;
      rank = tile.adapter < 0 ? 0 : a.ranks ? min(max(a.ranks[tile.adapter], 0), a.R) : a.R;
      const float scale = tile.adapter < 0 ? 0.0f : a.scales ? a.scales[tile.adapter] : 1.0f;
      if (tid < tile.count) rows[tid] = a.order[tile.first + tid];
      // a warp takes a row: its d, summed over the shares of H
      for (int i = warp; i < cols * 8; i += kADWarps) {
        constexpr int PER = (KS * 16 + 31) / 32;  // entries a lane
        float v[PER];
        float most = 0.0f;
#pragma unroll
        for (int u = 0; u < PER; ++u) {
          const int r = u * 32 + lane;
          v[u] = 0.0f;
          if (i < tile.count && r < rank) {
            for (int s = 0; s < a.splits; ++s)
              v[u] += __ldcg(a.d + (static_cast<int64_t>(s) * a.rows + tile.first + i) * a.R + r);
            v[u] *= scale;
          }
          most = fmaxf(most, fabsf(v[u]));
        }
        float by = 1.0f;
        if constexpr (std::is_same<T, __half>::value) {
          // f16: the row's largest value goes into [2^13, 2^14), which is exact
          most = warp_max(most);
          if (most > 0.0f && most < INFINITY) {
            const int e = min(max(ilogbf(most), -112), 127);
            by = ldexpf(1.0f, 13 - e);
            if (lane == 0) unscale[i] = ldexpf(1.0f, e - 13);
          } else if (lane == 0) {
            unscale[i] = 1.0f;
          }
        } else if (lane == 0) {
          unscale[i] = 1.0f;
        }
#pragma unroll
        for (int u = 0; u < PER; ++u) {
          const int r = u * 32 + lane;
          if (r >= KS * 16) break;
          const float f = v[u] * by;
          const uint16_t high = Half16<T>::bits(f);
          const float hv = Half16<T>::value(high);
          const uint16_t low = Half16<T>::bits(fabsf(hv) < INFINITY ? f - hv : 0.0f);
          // where entry r stands: step, lane's t, register, half
          int ks, tt, reg;
          if (KS == 1) {
            ks = 0, tt = r >> 2, reg = (r >> 1) & 1;
          } else {
            const int e = r & 31;
            ks = (r >> 5) * 2 + ((e >> 2) & 1), tt = e >> 3, reg = (e >> 1) & 1;
          }
          uint16_t* f16p = reinterpret_cast<uint16_t*>(&frag[ks][i >> 3][(i & 7) * 4 + tt]);
          f16p[reg * 2 + (r & 1)] = high;
          f16p[4 + reg * 2 + (r & 1)] = low;
        }
      }
      __syncthreads();
    }
    const T* up = reinterpret_cast<const T*>(a.up) + static_cast<int64_t>(max(tile.adapter, 0)) * a.up_adapter;
    const int n_end = min(a.N, (ci + 1) * chunk);
    for (int n0 = ci * chunk + warp * kADStep; n0 < n_end; n0 += kADWarps * kADStep) {
      float acc[2][kADCols][4] = {};
      const int nb = n0 + 4 * g;  // this lane's weight rows and outputs: nb .. nb + 3
      if (rank > 0) {
        if constexpr (KS == 1) {
          uint2 w[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            w[q] = make_uint2(0, 0);
            if (nb + q < a.N && t * 4 < rank)
              w[q] = *reinterpret_cast<const uint2*>(up + static_cast<int64_t>(nb + q) * a.up_row + t * 4);
            const int nv = rank - t * 4;  // entries past the rank may hold anything
            if (nv < 4) {
              w[q].x &= nv >= 2 ? ~0u : nv == 1 ? 0xFFFFu : 0u;
              w[q].y &= nv == 3 ? 0xFFFFu : 0u;
            }
          }
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint32_t af[4] = {w[2 * j].x, w[2 * j + 1].x, w[2 * j].y, w[2 * j + 1].y};
#pragma unroll
            for (int c = 0; c < kADCols; ++c)
              if (c < cols) {
                const uint4 b = frag[0][c][lane];
                mma16<T>(acc[j][c], af, b.x, b.y);
                mma16<T>(acc[j][c], af, b.z, b.w);
              }
          }
        } else {
#pragma unroll
          for (int kb = 0; kb < KS / 2; ++kb) {
            const int nv = rank - kb * 32 - t * 8;
            uint4 w[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              w[q] = make_uint4(0, 0, 0, 0);
              if (nb + q < a.N && nv > 0)
                w[q] = *reinterpret_cast<const uint4*>(up + static_cast<int64_t>(nb + q) * a.up_row + kb * 32 + t * 8);
              if (nv < 8) {
                uint32_t* u = reinterpret_cast<uint32_t*>(&w[q]);
#pragma unroll
                for (int e = 0; e < 4; ++e) u[e] &= nv >= 2 * e + 2 ? ~0u : nv == 2 * e + 1 ? 0xFFFFu : 0u;
              }
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const uint4 u = w[2 * j], v = w[2 * j + 1];
              const uint32_t a0[4] = {u.x, v.x, u.y, v.y}, a1[4] = {u.z, v.z, u.w, v.w};
#pragma unroll
              for (int c = 0; c < kADCols; ++c)
                if (c < cols) {
                  const uint4 b0 = frag[2 * kb][c][lane], b1 = frag[2 * kb + 1][c][lane];
                  mma16<T>(acc[j][c], a0, b0.x, b0.y);
                  mma16<T>(acc[j][c], a0, b0.z, b0.w);
                  mma16<T>(acc[j][c], a1, b1.x, b1.y);
                  mma16<T>(acc[j][c], a1, b1.z, b1.w);
                }
            }
          }
        }
      }
#pragma unroll
      for (int c = 0; c < kADCols; ++c) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int i = c * 8 + 2 * t + u;
          if (i >= tile.count || nb >= a.N) continue;
          const float back = unscale[i];
          const float dv[4] = {acc[0][c][u] * back, acc[0][c][2 + u] * back, acc[1][c][u] * back, acc[1][c][2 + u] * back};
          const int64_t yi = static_cast<int64_t>(rows[i]) * a.y_stride + nb;
          const int64_t oi = static_cast<int64_t>(rows[i]) * a.out_stride + nb;
          if (a.y_vec == 4 && nb + 4 <= a.N) {
            float v[4];
            y_load4<Y>(a.y, yi, v);
#pragma unroll
            for (int q = 0; q < 4; ++q) v[q] += dv[q];
            y_store4<Y>(a.out, oi, v);
          } else {
#pragma unroll
            for (int q = 0; q < 4; ++q)
              if (nb + q < a.N) y_store<Y>(a.out, oi + q, y_load<Y>(a.y, yi + q) + dv[q]);
          }
        }
      }
    }
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
static size_t align_up(size_t n) { return (n + 255) & ~static_cast<size_t>(255); }

// Shares of H of the first product: enough CTAs for the GPU when the tiles are few, each with
// work for its warps.
static int adapter_splits(int rows, int count, int H, int num_sms) {
  const int blocks = (H + 31) / 32;
  const int64_t tiles = static_cast<int64_t>((rows + kADTile - 1) / kADTile) + (rows < count ? rows : count);
  int64_t s = num_sms / (tiles > 0 ? tiles : 1);
  const int most = blocks / (2 * kADWarps);  // two blocks of 32 a warp at least
  if (s > most) s = most;
  if (s > 8) s = 8;
  return s < 1 ? 1 : static_cast<int>(s);
}

static int64_t adapter_max_tiles(int rows, int count) {
  const int64_t by_rows = (rows + kADTile - 1) / kADTile;
  return by_rows + (rows < count + 1 ? rows : count + 1);
}

size_t adapters_workspace_bytes(int rows, int count, int rank, int H, int num_sms) {
  return 256 + align_up(static_cast<size_t>(adapter_max_tiles(rows, count)) * sizeof(AdapterTile)) +
         align_up(static_cast<size_t>(rows) * 4) +
         align_up(static_cast<size_t>(adapter_splits(rows, count, H, num_sms)) * static_cast<size_t>(rows) *
                  static_cast<size_t>(rank) * 4);
}

template <typename T, int RT>
static cudaError_t down_setup() {
  return cudaFuncSetAttribute(adapter_down_kernel<T, RT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              kADWarps * RT * 16 * kADTile * 4);
}
template <typename T>
static cudaError_t adapters_setup_one() {
  cudaError_t e = down_setup<T, 1>();
  if (e == cudaSuccess) e = down_setup<T, 2>();
  if (e == cudaSuccess) e = down_setup<T, 4>();
  if (e == cudaSuccess) e = down_setup<T, 8>();
  return e;
}
cudaError_t adapters_setup() {
  const cudaError_t e = adapters_setup_one<__nv_bfloat16>();
  return e == cudaSuccess ? adapters_setup_one<__half>() : e;
}

template <typename T, int RT>
static cudaError_t launch_down(const AdapterArgs& a, int grid, cudaStream_t stream) {
  return launch_kernel(adapter_down_kernel<T, RT>, dim3(grid, a.splits), dim3(kADThreads),
                       static_cast<size_t>(kADWarps * RT * 16 * kADTile * 4), stream, true, a);
}

template <typename T, typename Y>
static cudaError_t launch_up(const AdapterArgs& a, int grid, int chunk, int n_chunks, cudaStream_t stream) {
  const dim3 b(kADThreads), gr(grid);
  if (a.R <= 16) return launch_kernel(adapter_up_kernel<T, Y, 1>, gr, b, 0, stream, true, a, chunk, n_chunks);
  if (a.R <= 32) return launch_kernel(adapter_up_kernel<T, Y, 2>, gr, b, 0, stream, true, a, chunk, n_chunks);
  if (a.R <= 64) return launch_kernel(adapter_up_kernel<T, Y, 4>, gr, b, 0, stream, true, a, chunk, n_chunks);
  return launch_kernel(adapter_up_kernel<T, Y, 8>, gr, b, 0, stream, true, a, chunk, n_chunks);
}

template <typename T>
static cudaError_t launch_adapters(const AdapterArgs& a, lmh_dtype out_dtype, int num_sms, cudaStream_t stream) {
  const int64_t max_tiles = adapter_max_tiles(a.rows, a.count);
  trace_begin(kTraceAdapterPlan, stream);
  cudaError_t e = launch_kernel(adapter_plan_kernel, dim3(1), dim3(kADPlanThreads),
                                static_cast<size_t>(a.count + 1) * 4, stream, true, a);
  trace_end(kTraceAdapterPlan, stream);
  if (e != cudaSuccess) return e;
  const int grid = static_cast<int>(max_tiles < 4 * num_sms ? max_tiles : 4 * num_sms);
  trace_begin(kTraceAdapterDown, stream);
  if (a.R <= 16) e = launch_down<T, 1>(a, grid, stream);
  else if (a.R <= 32) e = launch_down<T, 2>(a, grid, stream);
  else if (a.R <= 64) e = launch_down<T, 4>(a, grid, stream);
  else e = launch_down<T, 8>(a, grid, stream);
  trace_end(kTraceAdapterDown, stream);
  if (e != cudaSuccess) return e;
  const int chunk = kADWarps * kADStep;
  const int n_chunks = (a.N + chunk - 1) / chunk;
  const int64_t items = max_tiles * n_chunks;
  const int up_grid = static_cast<int>(items < 4 * num_sms ? items : 4 * num_sms);
  trace_begin(kTraceAdapterUp, stream);
  e = out_dtype == LMH_F32 ? launch_up<T, float>(a, up_grid, chunk, n_chunks, stream)
                           : launch_up<T, T>(a, up_grid, chunk, n_chunks, stream);
  trace_end(kTraceAdapterUp, stream);
  return e;
}

cudaError_t launch_add_adapters(const void* x, int64_t x_stride, int num_tokens, const int32_t* row_idx, int rows,
                                const int32_t* adapter_idx, const lmh_adapters& t, const void* y, int64_t y_stride,
                                void* out, lmh_dtype out_dtype, int64_t out_stride, void* workspace,
                                uint32_t* dev_status, int num_sms, cudaStream_t stream) {
  AdapterArgs a{};
  a.x = static_cast<const char*>(x);
  a.x_stride = x_stride;
  a.num_tokens = num_tokens;
  a.row_idx = row_idx;
  a.adapter_idx = adapter_idx;
  a.rows = rows;
  a.down = static_cast<const char*>(t.down);
  a.down_adapter = t.down_adapter_stride;
  a.down_row = t.down_row_stride;
  a.up = static_cast<const char*>(t.up);
  a.up_adapter = t.up_adapter_stride;
  a.up_row = t.up_row_stride;
  a.scales = t.scales;
  a.ranks = t.ranks;
  a.count = t.count;
  a.R = t.rank;
  a.H = t.H;
  a.N = t.N;
  a.x_vec = reinterpret_cast<uintptr_t>(x) % 16 == 0 && x_stride % 8 == 0;
  a.y = static_cast<const char*>(y);
  a.y_stride = y_stride;
  a.out = static_cast<char*>(out);
  a.out_stride = out_stride;
  a.in_place = y == out && y_stride == out_stride;
  const size_t four = out_dtype == LMH_F32 ? 16 : 8;
  a.y_vec = reinterpret_cast<uintptr_t>(y) % four == 0 && reinterpret_cast<uintptr_t>(out) % four == 0 &&
                    y_stride % 4 == 0 && out_stride % 4 == 0 ? 4 : 1;
  a.splits = adapter_splits(rows, t.count, t.H, num_sms);
  char* p = static_cast<char*>(workspace);
  a.tile_count = reinterpret_cast<int32_t*>(p);
  p += 256;
  a.tiles = reinterpret_cast<AdapterTile*>(p);
  p += align_up(static_cast<size_t>(adapter_max_tiles(rows, t.count)) * sizeof(AdapterTile));
  a.order = reinterpret_cast<int32_t*>(p);
  p += align_up(static_cast<size_t>(rows) * 4);
  a.d = reinterpret_cast<float*>(p);
  a.dev_status = dev_status;
  return t.dtype == LMH_BF16 ? launch_adapters<__nv_bfloat16>(a, out_dtype, num_sms, stream)
                             : launch_adapters<__half>(a, out_dtype, num_sms, stream);
}

}  // namespace lmh
