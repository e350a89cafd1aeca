// adapters.cuh -- low-rank adapters of many requests beside a shared projection (lmh_add_adapters).
// Instantiated per type of the weights in adapters_*.cu; plan and host side: adapters.cu.
//
//   out[i][n] = y[i][n] + scale_l * sum_r up[l][n][r] * d[i][r],   d[i][r] = sum_h down[l][r][h] * x[i][h]
//
// with l = adapter_idx[i].  The rows are cut into tiles of up to kADTile rows of one adapter.  One kernel
// makes d of every tile, the next the second product, added to y.  Up to kADOwnPlan rows every CTA works out
// the tiles from the indices by itself; above, a kernel before the two sorts the rows by adapter.
//
// Both products run on mma.sync m16n8k16 with 16 rows of the weights as the A operand and 8 rows of the
// batch as the B operand: a batch of one row costs the same weight reads as one of eight, and weights go
// from memory to the MMA's registers without a stop in shared memory.  The order of the entries along the
// inner dimension is free as long as A and B agree, so a lane takes 16 contiguous bytes of a weight row.
//
// d enters the second product as two 16-bit parts, high and low: 16 bits (bf16) or 22 (f16) of its fp32
// value, so that its rounding stays near that of the fp32 sums.
#pragma once

#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "device_common.cuh"
#include "lmh_internal.h"

namespace lmh {

constexpr int kADTile = 64;       // rows of a tile
constexpr int kADCols = kADTile / 8;
constexpr int kADPlanThreads = 1024;
constexpr int kADThreads = 256;   // both products
constexpr int kADWarps = kADThreads / 32;
constexpr int kADStep = 32;       // outputs n a warp takes at a time
constexpr int kADOwnPlan = kADThreads;  // rows to which every CTA finds its tiles by itself

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
  // workspace
  int32_t* tile_count;  // written by the plan kernel, as are tiles and order
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

// ---------------------------------------------------------------------------
// a lane's own copies
// ---------------------------------------------------------------------------
// Weights, x and y come through rings in shared memory in which every lane copies (cp.async) what it will
// itself read, in the order of its registers: no barrier, no bank conflict, and as many bytes in flight as the
// ring holds, which registers do not (measured: DESIGN).
template <int BYTES>
__device__ __forceinline__ void lane_copy(void* smem_dst, const void* src) {
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(smem_dst)), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(smem_u32(smem_dst)), "l"(src), "n"(BYTES) : "memory");
}
__device__ __forceinline__ void lane_copies_end() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// All but the last N groups of this lane's copies have arrived.
template <int N>
__device__ __forceinline__ void lane_copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// ---------------------------------------------------------------------------
// tiles
// ---------------------------------------------------------------------------
// The tiles of a call as a CTA of kADThreads threads sees them.  With at most kADOwnPlan rows thread i
// takes row i: its place among the rows of the same adapter gives its tile and its place in it, and a tile's
// number is its first row's among the rows that are first in a tile.  Otherwise the plan kernel's results.
struct TileSmem {
  alignas(16) int32_t adapter_of[kADOwnPlan];
  int32_t rows[kADTile];  // of the current tile
  int32_t adapter, part, count, tiles;
};

struct TileFinder {
  int mine = -2;   // this thread's row's adapter (own plan); -2: no such row
  int place = 0;   // among the rows with the same
  int number = -1;  // of the tile that this thread's row is first in

  // All threads; the indices may be read.  Returns the number of tiles.
  __device__ int start(const AdapterArgs& a, TileSmem& sm) {
    if (a.rows > kADOwnPlan) return __ldcg(a.tile_count);
    const int i = threadIdx.x;
    if (i < a.rows) {
      mine = a.adapter_idx[i];
      if (mine < 0 || mine >= a.count) {
        if (mine != -1) set_status(a.dev_status, LMH_DS_ADAPTER_OUT_OF_RANGE);
        mine = -1;
      }
    }
    sm.adapter_of[i] = mine;
    if (i == 0) sm.tiles = 0;
    __syncthreads();
    if (i < a.rows) {
      int n = 0;
      for (int j = 0; j < i; j += 4) {  // (rows from i on are not counted)
        const int4 o = *reinterpret_cast<const int4*>(&sm.adapter_of[j]);
        n += o.x == mine;
        n += o.y == mine && j + 1 < i;
        n += o.z == mine && j + 2 < i;
        n += o.w == mine && j + 3 < i;
      }
      place = n;
    }
    const bool first = i < a.rows && place % kADTile == 0 && !(mine == -1 && a.in_place);
    const unsigned firsts = __ballot_sync(0xffffffffu, first);
    __syncthreads();
    // the warps' counts, in the place of the indices that nobody reads any more
    if ((i & 31) == 0) sm.adapter_of[i >> 5] = __popc(firsts);
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kADWarps; ++w) {
      const int c = sm.adapter_of[w];
      before += w < (i >> 5) ? c : 0;
      all += c;
    }
    if (first) number = before + __popc(firsts & ((1u << (i & 31)) - 1));
    return all;
  }

  // All threads: tile `t`'s rows, adapter and count into sm (behind a barrier of its own).
  __device__ void take(const AdapterArgs& a, TileSmem& sm, int t) {
    __syncthreads();  // nobody reads the tile before
    if (a.rows > kADOwnPlan) {
      const AdapterTile tile = a.tiles[t];
      if (threadIdx.x == 0) sm.adapter = tile.adapter, sm.count = tile.count;
      if (threadIdx.x < static_cast<unsigned>(tile.count)) sm.rows[threadIdx.x] = __ldcg(a.order + tile.first + threadIdx.x);
      __syncthreads();
      return;
    }
    if (number == t) sm.adapter = mine, sm.part = place / kADTile, sm.count = 0;
    __syncthreads();
    if (mine == sm.adapter && place / kADTile == sm.part) {  // (a thread without a row has mine = -2)
      sm.rows[place % kADTile] = threadIdx.x;
      atomicAdd(&sm.count, 1);
    }
    __syncthreads();
  }
};

__device__ __forceinline__ int adapter_rank(const AdapterArgs& a, int adapter) {
  return adapter < 0 ? 0 : a.ranks ? min(max(a.ranks[adapter], 0), a.R) : a.R;
}

// ---------------------------------------------------------------------------
// first product
// ---------------------------------------------------------------------------
// One CTA a (tile, share of H).  A warp takes 16 rows of a small tile (or what there is of them), 32 of a
// larger one, so one or two warps share the tile by rows and the others the blocks of 32 entries of H; their
// sums meet in shared memory in a fixed order.  RT: tiles of 16 adapter rows.
constexpr int adapter_down_depth(int rt) { return rt == 8 ? 2 : 4; }
constexpr int adapter_down_entry(int rt) { return (4 + 2 * rt) * 512; }  // a lane's 16 bytes of 4 x and 2 RT weights
constexpr int adapter_down_smem(int rt) {
  const int ring = kADWarps * adapter_down_depth(rt) * adapter_down_entry(rt), sums = kADWarps * rt * 16 * 32 * 4;
  return ring > sums ? ring : sums;
}

// A warp's share: blocks first, first + step, ... below hi of its C * 8 rows' x and the adapter's rows.
template <typename T, int RT, int C>
__device__ __forceinline__ void down_share(const AdapterArgs& a, const T* down, int rank, const int32_t* tok, int count,
                                           int first, int step, int hi, unsigned char* ring, float (&acc)[RT][C][4]) {
  constexpr int D = adapter_down_depth(RT), ENTRY = adapter_down_entry(RT);
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const T* xp[C];
  bool have[C];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int tk = tok[c * 8 + g];  // -1 for rows that are not there
    have[c] = tk >= 0;
    xp[c] = reinterpret_cast<const T*>(a.x) + static_cast<int64_t>(tk) * a.x_stride + t * 8;
  }
  auto issue = [&](int j) {
    const int kb = first + j * step;
    const int h = kb * 32 + t * 8;  // H is a multiple of 8
    uint4* e = reinterpret_cast<uint4*>(ring + (j % D) * ENTRY) + lane;
    if (kb < hi && h < a.H) {
#pragma unroll
      for (int rt = 0; rt < 2 * RT; ++rt)
        if (rt * 8 + g < rank) lane_copy<16>(e + rt * 32, down + (rt * 8 + g) * a.down_row + h);
      if (a.x_vec)
#pragma unroll
        for (int c = 0; c < C; ++c)
          if (have[c]) lane_copy<16>(e + (2 * RT + c) * 32, xp[c] + kb * 32);
    }
    lane_copies_end();
  };
  for (int j = 0; j < D - 1; ++j) issue(j);
  for (int j = 0; first + j * step < hi; ++j) {
    issue(j + D - 1);
    const int kb = first + j * step;
    const bool in = kb * 32 + t * 8 < a.H;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    lane_copies_wait<D - 1>();
    const uint4* e = reinterpret_cast<const uint4*>(ring + (j % D) * ENTRY) + lane;
    uint4 xv[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      xv[c] = zero;
      if (!in || !have[c]) continue;
      if (a.x_vec) {
        xv[c] = e[(2 * RT + c) * 32];
      } else {
        const uint16_t* p = reinterpret_cast<const uint16_t*>(xp[c] + kb * 32);
        xv[c] = make_uint4(p[0] | p[1] << 16, p[2] | p[3] << 16, p[4] | p[5] << 16, p[6] | p[7] << 16);
      }
    }
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      const uint4 w0 = in && rt * 16 + g < rank ? e[2 * rt * 32] : zero;
      const uint4 w1 = in && rt * 16 + 8 + g < rank ? e[(2 * rt + 1) * 32] : zero;
      const uint32_t a0[4] = {w0.x, w1.x, w0.y, w1.y}, a1[4] = {w0.z, w1.z, w0.w, w1.w};
#pragma unroll
      for (int c = 0; c < C; ++c)
        if (c * 8 < count) {
          mma16<T>(acc[rt][c], a0, xv[c].x, xv[c].y);
          mma16<T>(acc[rt][c], a1, xv[c].z, xv[c].w);
        }
    }
  }
  lane_copies_wait<0>();
}

template <typename T, int RT>
__global__ void __launch_bounds__(kADThreads) adapter_down_kernel(const AdapterArgs a) {
  extern __shared__ __align__(16) unsigned char down_smem[];  // the warps' rings, then their sums [warp][rows][RT * 16]
  __shared__ TileSmem ts;
  __shared__ int32_t tok[kADTile];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  pdl_wait();
  pdl_launch_dependents();
  TileFinder finder;
  const int n_tiles = finder.start(a, ts);
  const int split = blockIdx.y;
  const int blocks = (a.H + 31) / 32;
  const int lo = static_cast<int>(static_cast<int64_t>(blocks) * split / a.splits);
  const int hi = static_cast<int>(static_cast<int64_t>(blocks) * (split + 1) / a.splits);
  unsigned char* ring = down_smem + warp * (adapter_down_depth(RT) * adapter_down_entry(RT));
  float* sums = reinterpret_cast<float*>(down_smem);
  for (int ti = blockIdx.x; ti < n_tiles; ti += gridDim.x) {
    finder.take(a, ts, ti);
    if (ts.adapter < 0) continue;  // (uniform)
    const int count = ts.count, rank = adapter_rank(a, ts.adapter);
    if (tid < kADTile) {
      int tk = -1;
      if (tid < count) {
        tk = a.row_idx ? a.row_idx[ts.rows[tid]] : ts.rows[tid];
        if (tk < 0 || tk >= a.num_tokens) {
          tk = -1;  // reads zeros
          set_status(a.dev_status, LMH_DS_ROW_IDX_OUT_OF_RANGE);
        }
      }
      tok[tid] = tk;
    }
    __syncthreads();
    const T* down = reinterpret_cast<const T*>(a.down) + static_cast<int64_t>(ts.adapter) * a.down_adapter;
    // warps that share the tile by rows, and how many rows each takes
    const int by_rows = count <= 32 ? 1 : 2, per = count <= 16 ? 16 : 32;
    const int wk = kADWarps / by_rows, part = warp % by_rows, first = lo + warp / by_rows;
    auto share = [&](auto c_const) {
      constexpr int C = decltype(c_const)::value;
      float acc[RT][C][4] = {};
      down_share<T, RT, C>(a, down, rank, tok + part * per, count - part * per, first, wk, hi, ring, acc);
      __syncthreads();  // the rings are done with
      float* mine = sums + warp * (C * 8 * RT * 16);
#pragma unroll
      for (int rt = 0; rt < RT; ++rt)
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            mine[(c * 8 + 2 * t + (e & 1)) * (RT * 16) + rt * 16 + g + 8 * (e >> 1)] = acc[rt][c][e];
    };
    if (count <= 8) share(std::integral_constant<int, 1>{});
    else if (count <= 16) share(std::integral_constant<int, 2>{});
    else share(std::integral_constant<int, 4>{});
    __syncthreads();
    const int rows_of = count <= 8 ? 8 : per;  // rows of a warp's sums
    float* d = a.d + static_cast<int64_t>(split) * a.rows * a.R;
    for (int i = tid; i < count * (RT * 16); i += kADThreads) {
      const int row = i / (RT * 16), r = i % (RT * 16);
      if (r >= a.R) continue;
      const float* p = sums + ((row / rows_of) * rows_of + row % rows_of) * (RT * 16) + r;
      float s = 0.0f;
      for (int w = 0; w < wk; ++w) s += p[w * by_rows * rows_of * (RT * 16)];
      d[static_cast<int64_t>(ts.rows[row]) * a.R + r] = s;
    }
  }
}

// ---------------------------------------------------------------------------
// second product, added to y
// ---------------------------------------------------------------------------
// Four outputs of one row, as a lane holds them.  VEC: four neighbours, read and written at once; else outputs
// n, n + 8, n + 16 and n + 24, neighbouring lanes holding neighbours.
template <typename Y, bool VEC>
struct Outputs {
  static constexpr int ES = static_cast<int>(sizeof(Y));
  static constexpr bool kRing = VEC || ES == 4;  // (copies are of four bytes at least)
  // into the ring's place (16 bytes of ES 4, 8 of ES 2, a lane): out of the row's `left` outputs from n on
  __device__ __forceinline__ static void copy(unsigned char* to, const char* row, int left) {
    if constexpr (VEC) {
      lane_copy<4 * ES>(to, row);
    } else if constexpr (ES == 4) {
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (8 * q < left) lane_copy<4>(to + 4 * q, row + 32 * q);
    }
  }
  __device__ __forceinline__ static void add_and_store(const unsigned char* in, const char* y_row, char* row, int left,
                                                       const float (&d)[4]) {
    if constexpr (VEC && ES == 4) {
      const float4 v = *reinterpret_cast<const float4*>(in);
      *reinterpret_cast<float4*>(row) = make_float4(v.x + d[0], v.y + d[1], v.z + d[2], v.w + d[3]);
    } else if constexpr (VEC) {
      using C = Half16<Y>;
      const uint2 v = *reinterpret_cast<const uint2*>(in);
      uint2 w;
      w.x = C::bits(C::value(v.x & 0xFFFFu) + d[0]) | static_cast<uint32_t>(C::bits(C::value(v.x >> 16) + d[1])) << 16;
      w.y = C::bits(C::value(v.y & 0xFFFFu) + d[2]) | static_cast<uint32_t>(C::bits(C::value(v.y >> 16) + d[3])) << 16;
      *reinterpret_cast<uint2*>(row) = w;
    } else if constexpr (ES == 4) {
      const float4 v = *reinterpret_cast<const float4*>(in);
      const float f[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (8 * q < left) reinterpret_cast<float*>(row)[8 * q] = f[q] + d[q];
    } else {
      using C = Half16<Y>;
      uint16_t v[4] = {};
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (8 * q < left) v[q] = reinterpret_cast<const uint16_t*>(y_row)[8 * q];
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (8 * q < left) reinterpret_cast<uint16_t*>(row)[8 * q] = C::bits(C::value(v[q]) + d[q]);
    }
  }
};

// d in MMA order: the high parts (b0, b1) and the low parts (b0, b1) of a lane
template <int KS>
struct UpSmem {
  uint4 frag[KS][kADCols][32];
  float unscale[kADTile];  // f16: the power of two that a row's d was divided by
  int64_t y[kADTile], out[kADTile];  // the rows' first bytes
};

// All threads: a tile's d, scaled, into sm.
template <typename T, int KS>
__device__ void up_operand(const AdapterArgs& a, const TileSmem& ts, UpSmem<KS>& sm, int rank) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int count = ts.count, cols = (count + 7) / 8;
  const float scale = ts.adapter < 0 ? 0.0f : a.scales ? a.scales[ts.adapter] : 1.0f;
  constexpr int PER = (KS * 16 + 31) / 32;  // entries a lane; a warp takes a row at a time
  for (int i = warp; i < cols * 8; i += kADWarps) {
    float v[PER];
    float most = 0.0f;
#pragma unroll
    for (int u = 0; u < PER; ++u) {
      const int r = u * 32 + lane;
      v[u] = 0.0f;
      if (i < count && r < rank) {
        const float* d = a.d + static_cast<int64_t>(ts.rows[i]) * a.R + r;
        for (int s = 0; s < a.splits; ++s) v[u] += __ldcg(d + static_cast<int64_t>(s) * a.rows * a.R);
        v[u] *= scale;
      }
      most = fmaxf(most, fabsf(v[u]));
    }
    float by = 1.0f, back = 1.0f;
    if constexpr (std::is_same<T, __half>::value) {
      // f16: the row's largest value goes into [2^13, 2^14), which is exact
      most = warp_max(most);
      if (most > 0.0f && most < INFINITY) {
        const int e = min(max(ilogbf(most), -112), 127);
        by = ldexpf(1.0f, 13 - e);
        back = ldexpf(1.0f, e - 13);
      }
    }
    if (lane == 0) sm.unscale[i] = back;
#pragma unroll
    for (int u = 0; u < PER; ++u) {
      const int r = u * 32 + lane;
      if (r >= KS * 16) break;
      const float f = v[u] * by;
      const uint16_t high = Half16<T>::bits(f);
      const float hv = Half16<T>::value(high);
      const uint16_t low = Half16<T>::bits(fabsf(hv) < INFINITY ? f - hv : 0.0f);
      // where entry r stands: step, lane's t, register
      int ks, tt, reg;
      if (KS == 1) {
        ks = 0, tt = r >> 2, reg = (r >> 1) & 1;
      } else {
        const int e = r & 31;
        ks = (r >> 5) * 2 + ((e >> 2) & 1), tt = e >> 3, reg = (e >> 1) & 1;
      }
      uint16_t* p = reinterpret_cast<uint16_t*>(&sm.frag[ks][i >> 3][(i & 7) * 4 + tt]);
      p[reg * 2 + (r & 1)] = high;
      p[4 + reg * 2 + (r & 1)] = low;
    }
  }
}

// 16-bit entries from `n` on made 0 (entries past an adapter's rank may hold anything)
__device__ __forceinline__ void first_entries(uint2& w, int n) {
  w.x &= n >= 2 ? ~0u : n == 1 ? 0xFFFFu : 0u;
  w.y &= n >= 4 ? ~0u : n == 3 ? 0xFFFFu : 0u;
}
__device__ __forceinline__ void first_entries(uint4& w, int n) {
  uint2 a = make_uint2(w.x, w.y), b = make_uint2(w.z, w.w);
  first_entries(a, n);
  first_entries(b, n - 4);
  w = make_uint4(a.x, a.y, b.x, b.y);
}

// A warp's weights of 32 outputs: four rows of up a lane (q), as two MMAs' operands (q = 0, 1 and 2, 3).
// KS 1: ranks to 16, a lane takes 8 bytes of a weight row; else 16 bytes of every 32 entries.
template <typename T, int KS>
struct UpWeights {
  static constexpr int KB = KS == 1 ? 1 : KS / 2;
  static constexpr int E = KS == 1 ? 4 : 8;  // entries of a weight row that a lane takes of a block
  using Word = typename std::conditional<KS == 1, uint2, uint4>::type;
  Word w[KB][4];

  // The lane's words of rows `row`, row + step, ... (those below N) into the ring's place.
  __device__ __forceinline__ static void copy(unsigned char* to, const T* up, int64_t up_row, int row, int step, int N,
                                              int rank, int lane) {
    const int t = lane & 3;
    Word* e = reinterpret_cast<Word*>(to) + lane;
    const T* p = up + row * up_row + t * E;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      if (row + q * step < N) {
#pragma unroll
        for (int kb = 0; kb < KB; ++kb)
          if (kb * 32 + t * E < rank) lane_copy<static_cast<int>(sizeof(Word))>(e + (kb * 4 + q) * 32, p + kb * 32);
      }
      p += step * up_row;
    }
  }
  // Entries behind the rank become 0; rows behind N hold whatever they do: their results are not kept.
  __device__ __forceinline__ void read(const unsigned char* from, int rank, int lane) {
    const Word* e = reinterpret_cast<const Word*>(from) + lane;
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) {
      const int left = rank - kb * 32 - (lane & 3) * E;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        w[kb][q] = e[(kb * 4 + q) * 32];
        if (left < E) first_entries(w[kb][q], left);
      }
    }
  }
  // acc[j] += rows (2j, 2j + 1) times column tile c of d
  __device__ __forceinline__ void multiply(const UpSmem<KS>& sm, int c, int lane, float (&acc)[2][4]) const {
    if constexpr (KS == 1) {
      const uint4 b = sm.frag[0][c][lane];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint32_t f[4] = {w[0][2 * j].x, w[0][2 * j + 1].x, w[0][2 * j].y, w[0][2 * j + 1].y};
        mma16<T>(acc[j], f, b.x, b.y);
        mma16<T>(acc[j], f, b.z, b.w);
      }
    } else {
#pragma unroll
      for (int kb = 0; kb < KB; ++kb) {
        const uint4 b0 = sm.frag[2 * kb][c][lane], b1 = sm.frag[2 * kb + 1][c][lane];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint4 u = w[kb][2 * j], v = w[kb][2 * j + 1];
          const uint32_t f0[4] = {u.x, v.x, u.y, v.y}, f1[4] = {u.z, v.z, u.w, v.w};
          mma16<T>(acc[j], f0, b0.x, b0.y);
          mma16<T>(acc[j], f0, b0.z, b0.w);
          mma16<T>(acc[j], f1, b1.x, b1.y);
          mma16<T>(acc[j], f1, b1.z, b1.w);
        }
      }
    }
  }
};

// A warp's ring: entries of the weights of 32 outputs and of y for C tiles of 8 rows.
constexpr int up_entry(int ks, int es, int c) { return ks * 1024 + c * es * 256; }
constexpr int up_warp_bytes(int ks, int es) {
  const int two = 2 * up_entry(ks, es, 4), most = 13 * 1024;  // two entries of the larger kind at least
  return two > most ? two : most;
}
constexpr int up_depth(int ks, int es, int c) {
  const int n = up_warp_bytes(ks, es) / up_entry(ks, es, c);
  return n < 8 ? n : 8;
}
constexpr int up_ctas(int ks, int es) { return up_warp_bytes(ks, es) <= 13 * 1024 ? 2 : 1; }  // per SM

// A warp's part of a tile's outputs [n_begin, n_end): every kADWarps-th step of 32 from its first on.  C: column
// tiles of an entry; a tile of more rows has `halves` entries a step, of which the first brings the weights.
// start(): the copies that fill the ring; run(): the rest, once d stands in sm.
template <typename T, typename Y, int KS, bool VEC, int C>
struct UpShare {
  static constexpr int ES = static_cast<int>(sizeof(Y)), D = up_depth(KS, ES, C), ENTRY = up_entry(KS, ES, C);
  const AdapterArgs& a;
  const UpSmem<KS>& sm;
  const T* up;
  unsigned char* ring;
  int rank, count, n_first, n_end, halves;

  __device__ __forceinline__ int output(int step) const {  // the lane's first output of a step
    const int g = (threadIdx.x & 31) >> 2;
    return n_first + step * (kADWarps * kADStep) + (VEC ? 4 * g : g);
  }
  __device__ __forceinline__ void issue(int j) const {
    const int lane = threadIdx.x & 31, t = lane & 3;
    const int step = halves == 1 ? j : j >> 1, half = halves == 1 ? 0 : j & 1;
    const int n = output(step);
    unsigned char* e = ring + (j % D) * ENTRY;
    if (n_first + step * (kADWarps * kADStep) < n_end) {
      if (half == 0) UpWeights<T, KS>::copy(e, up, a.up_row, n, VEC ? 1 : 8, a.N, rank, lane);
      if (Outputs<Y, VEC>::kRing && n < n_end) {
#pragma unroll
        for (int c = 0; c < 2 * C; ++c) {
          const int i = half * 32 + (c >> 1) * 8 + 2 * t + (c & 1);
          if (i < count)
            Outputs<Y, VEC>::copy(e + KS * 1024 + (c * 32 + lane) * (4 * ES), a.y + sm.y[i] + static_cast<int64_t>(n) * ES, n_end - n);
        }
      }
    }
    lane_copies_end();
  }
  __device__ __forceinline__ void start() const {
#pragma unroll 1
    for (int j = 0; j < D - 1; ++j) issue(j);
  }
  __device__ __forceinline__ void run() const {
    const int lane = threadIdx.x & 31, t = lane & 3;
    UpWeights<T, KS> w;
#pragma unroll 1
    for (int j = 0;; ++j) {
      const int step = halves == 1 ? j : j >> 1, half = halves == 1 ? 0 : j & 1;
      if (n_first + step * (kADWarps * kADStep) >= n_end) break;
      issue(j + D - 1);
      lane_copies_wait<D - 1>();
      const unsigned char* e = ring + (j % D) * ENTRY;
      const int n = output(step);
      if (half == 0) w.read(e, rank, lane);
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int c0 = half * 4 + c;
        if (c0 * 8 >= count) break;
        float acc[2][4] = {};
        w.multiply(sm, c0, lane, acc);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int i = c0 * 8 + 2 * t + u;
          if (i >= count || n >= n_end) continue;
          const float back = sm.unscale[i];
          const float dv[4] = {acc[0][u] * back, acc[0][2 + u] * back, acc[1][u] * back, acc[1][2 + u] * back};
          Outputs<Y, VEC>::add_and_store(e + KS * 1024 + ((2 * c + u) * 32 + lane) * (4 * ES),
                                         a.y + sm.y[i] + static_cast<int64_t>(n) * ES,
                                         a.out + sm.out[i] + static_cast<int64_t>(n) * ES, n_end - n, dv);
        }
      }
    }
    lane_copies_wait<0>();
  }
};

// A warp takes 32 outputs at a time as two MMAs of 16 weight rows.  VEC: rows n0 + 4g and n0 + 4g + 1 are row g
// and g + 8 of the first, n0 + 4g + 2 and + 3 of the second, so that a lane's results for a batch row are four
// neighbours.  Else n0 + g + 8q: neighbouring lanes hold neighbours.
// The work is (tile, step of 32 outputs); every CTA takes a contiguous share, so that it seldom changes tiles.
template <typename T, typename Y, int KS, bool VEC>
__global__ void __launch_bounds__(kADThreads, up_ctas(KS, sizeof(Y))) adapter_up_kernel(const AdapterArgs a) {
  extern __shared__ __align__(16) unsigned char up_ring[];
  __shared__ UpSmem<KS> sm;
  __shared__ TileSmem ts;
  const int tid = threadIdx.x, warp = tid >> 5;
  // the kernel before this one is the first product, which has itself waited for all before it: only d has to
  // wait for its end, and what the plan kernel wrote has been waited for
  TileFinder finder;
  const int n_tiles = finder.start(a, ts);
  const int64_t steps = (a.N + kADStep - 1) / kADStep;
  const int64_t all = steps * n_tiles;
  int64_t at = all * blockIdx.x / gridDim.x;
  const int64_t end = all * (blockIdx.x + 1) / gridDim.x;
  bool waited = false;
  while (at < end) {
    const int ti = static_cast<int>(at / steps);
    const int s0 = static_cast<int>(at - ti * steps), s1 = static_cast<int>(min(steps, s0 + (end - at)));
    at += s1 - s0;
    finder.take(a, ts, ti);
    const int count = ts.count, rank = adapter_rank(a, ts.adapter);
    if (tid < count) {
      sm.y[tid] = ts.rows[tid] * a.y_stride * static_cast<int64_t>(sizeof(Y));
      sm.out[tid] = ts.rows[tid] * a.out_stride * static_cast<int64_t>(sizeof(Y));
    }
    __syncthreads();
    const T* up = reinterpret_cast<const T*>(a.up) + static_cast<int64_t>(max(ts.adapter, 0)) * a.up_adapter;
    unsigned char* ring = up_ring + warp * up_warp_bytes(KS, sizeof(Y));
    const int n_first = (s0 + warp) * kADStep, n_end = min(a.N, s1 * kADStep);
    auto share = [&](const auto& part) {
      part.start();
      if (!waited) pdl_wait();
      waited = true;
      up_operand<T, KS>(a, ts, sm, rank);
      __syncthreads();
      part.run();
    };
    if (count <= 8) share(UpShare<T, Y, KS, VEC, 1>{a, sm, up, ring, rank, count, n_first, n_end, 1});
    else share(UpShare<T, Y, KS, VEC, 4>{a, sm, up, ring, rank, count, n_first, n_end, count <= 32 ? 1 : 2});
  }
  // a CTA without work waits too: this grid is not to end before the one that makes d
  if (!waited) pdl_wait();
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
template <typename T, int RT>
cudaError_t down_setup() {
  return cudaFuncSetAttribute(adapter_down_kernel<T, RT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              adapter_down_smem(RT));
}

template <typename T, typename Y, int KS, bool VEC>
cudaError_t up_setup() {
  return cudaFuncSetAttribute(adapter_up_kernel<T, Y, KS, VEC>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              kADWarps * up_warp_bytes(KS, sizeof(Y)));
}

template <typename T, typename Y, bool VEC>
cudaError_t up_setup_of() {
  cudaError_t e = up_setup<T, Y, 1, VEC>();
  if (e == cudaSuccess) e = up_setup<T, Y, 2, VEC>();
  if (e == cudaSuccess) e = up_setup<T, Y, 4, VEC>();
  if (e == cudaSuccess) e = up_setup<T, Y, 8, VEC>();
  return e;
}

template <typename T>
cudaError_t adapters_setup_one() {
  cudaError_t e = down_setup<T, 1>();
  if (e == cudaSuccess) e = down_setup<T, 2>();
  if (e == cudaSuccess) e = down_setup<T, 4>();
  if (e == cudaSuccess) e = down_setup<T, 8>();
  if (e == cudaSuccess) e = up_setup_of<T, float, true>();
  if (e == cudaSuccess) e = up_setup_of<T, float, false>();
  if (e == cudaSuccess) e = up_setup_of<T, T, true>();
  if (e == cudaSuccess) e = up_setup_of<T, T, false>();
  return e;
}

template <typename T>
cudaError_t launch_down(const AdapterArgs& a, int grid, cudaStream_t stream) {
  const dim3 g(grid, a.splits), b(kADThreads);
  if (a.R <= 16) return launch_kernel(adapter_down_kernel<T, 1>, g, b, static_cast<size_t>(adapter_down_smem(1)), stream, true, a);
  if (a.R <= 32) return launch_kernel(adapter_down_kernel<T, 2>, g, b, static_cast<size_t>(adapter_down_smem(2)), stream, true, a);
  if (a.R <= 64) return launch_kernel(adapter_down_kernel<T, 4>, g, b, static_cast<size_t>(adapter_down_smem(4)), stream, true, a);
  return launch_kernel(adapter_down_kernel<T, 8>, g, b, static_cast<size_t>(adapter_down_smem(8)), stream, true, a);
}

template <typename T, typename Y, int KS, bool VEC>
cudaError_t launch_up_ks(const AdapterArgs& a, int64_t max_steps, int num_sms, cudaStream_t stream) {
  const int64_t most = static_cast<int64_t>(num_sms) * up_ctas(KS, sizeof(Y));  // one wave
  const int64_t few = (max_steps + kADWarps - 1) / kADWarps;
  return launch_kernel(adapter_up_kernel<T, Y, KS, VEC>, dim3(static_cast<unsigned>(few < most ? few : most)),
                       dim3(kADThreads), static_cast<size_t>(kADWarps * up_warp_bytes(KS, sizeof(Y))), stream, true, a);
}

template <typename T, typename Y, bool VEC>
cudaError_t launch_up_of(const AdapterArgs& a, int64_t max_steps, int num_sms, cudaStream_t stream) {
  if (a.R <= 16) return launch_up_ks<T, Y, 1, VEC>(a, max_steps, num_sms, stream);
  if (a.R <= 32) return launch_up_ks<T, Y, 2, VEC>(a, max_steps, num_sms, stream);
  if (a.R <= 64) return launch_up_ks<T, Y, 4, VEC>(a, max_steps, num_sms, stream);
  return launch_up_ks<T, Y, 8, VEC>(a, max_steps, num_sms, stream);
}

// max_steps: (tiles) x (steps of 32 outputs), at most
template <typename T>
cudaError_t launch_up(const AdapterArgs& a, lmh_dtype out_dtype, bool vec, int64_t max_steps, int num_sms,
                      cudaStream_t stream) {
  if (out_dtype == LMH_F32)
    return vec ? launch_up_of<T, float, true>(a, max_steps, num_sms, stream)
               : launch_up_of<T, float, false>(a, max_steps, num_sms, stream);
  return vec ? launch_up_of<T, T, true>(a, max_steps, num_sms, stream)
             : launch_up_of<T, T, false>(a, max_steps, num_sms, stream);
}

// The two types' kernels (adapters_bf16.cu, adapters_f16.cu).
cudaError_t adapters_setup_bf16();
cudaError_t adapters_setup_f16();
cudaError_t launch_down_bf16(const AdapterArgs& a, int grid, cudaStream_t stream);
cudaError_t launch_down_f16(const AdapterArgs& a, int grid, cudaStream_t stream);
cudaError_t launch_up_bf16(const AdapterArgs& a, lmh_dtype out_dtype, bool vec, int64_t max_steps, int num_sms,
                           cudaStream_t stream);
cudaError_t launch_up_f16(const AdapterArgs& a, lmh_dtype out_dtype, bool vec, int64_t max_steps, int num_sms,
                          cudaStream_t stream);

}  // namespace lmh
