// adapters.cuh -- low-rank adapters of many requests beside a shared projection (lmh_add_adapters).
// Instantiated per type of the weights in adapters_*.cu; plan and host side: adapters.cu.
//
//   out[i][n] = y[i][n] + scale_l * sum_r up[l][n][r] * d[i][r],   d[i][r] = sum_h down[l][r][h] * x[i][h]
//
// with l = adapter_idx[i].  The rows are cut into tiles of up to kADTile rows of one adapter.  One kernel makes d of
// every tile, the next the second product, added to y.
//
// To kADOwnPlan rows every CTA works out the tiles from the indices by itself.  Both products run on mma.sync
// m16n8k16 with 16 rows of the weights as the A operand and 8 rows of the batch as the B operand: a tile of one row
// costs the same weight reads as one of eight, and the weights' bytes bound calls of few rows (64 rows of 48 adapters
// of ranks to 32, f16, x 128256: the second product reads 411 MB from DRAM in 77 us, 0.82 of the copy rate; the ranks in
// use are half of it, but DRAM hands out 64 bytes at a time, a whole row of rank 32).  Above, a kernel before the
// two sorts the rows by adapter; the batch's rows are the A operand, 16 a warp, and a CTA shares the weights: rows'
// bytes bound these calls (packed prompts, 16384 rows of rank 64, 1024 -> 4096: 90 us for 304 MB, 0.50 of the copy rate).
//
// The order of the entries along the inner dimension is free as long as A and B agree, so in the first product a lane
// takes 16 contiguous bytes of a weight row and of x.
//
// d enters the second product as two 16-bit parts, high and low (16 bits of its value for bf16, 22 for f16), so that
// its rounding stays near that of the fp32 sums.  For 16-bit outputs too, whose y may take nearly all of the added part
// away.  (The second part doubles the MMAs and the operand's reads from shared memory: packed prompts as above take
// 84 us with one part and 90 so, 64 rows of 48 adapters 78 and 79.)
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
constexpr int kADThreads = 256;   // first product
constexpr int kADWarps = kADThreads / 32;
constexpr int kADStep = 32;       // outputs of the second product that a warp takes at a time
// Rows to which every CTA finds its tiles by itself, a thread a row.  The kernels of many rows took longer below (bf16 in
// a graph, H 4096, ranks 16 / 64 with 8 adapters): 64 rows x 4096 7.1 / 10.1 us here and 14.7 / 28.1 there, 256 rows
// 14.0 / 18.9 and 14.6 / 27.7, 256 x 151936 fp32 71.5 and 76.9; 256 rows of H 1024 x 28672 18.7 and 16.0, the one size
// of 28 that lost.  A packed batch of more rows has no such kernel here: its indices go beyond a CTA's threads.
constexpr int kADOwnPlan = 256;

struct alignas(16) AdapterTile {
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
  int piece;  // calls of many rows: bytes that rows of y and out can be read and written at a time (8, 16)
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

// d = a * b
template <typename T>
__device__ __forceinline__ void mma16_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1);
template <>
__device__ __forceinline__ void mma16_first<__nv_bfloat16>(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                                           uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
}
template <>
__device__ __forceinline__ void mma16_first<__half>(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
}

// Four 8 x 8 matrices of 16-bit entries, lane 8i + r giving row r of matrix i (16 bytes): an A operand.
__device__ __forceinline__ void load_matrices(uint32_t (&m)[4], uint32_t smem_row) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(m[0]), "=r"(m[1]), "=r"(m[2]), "=r"(m[3])
               : "r"(smem_row)
               : "memory");
}

template <typename T>
struct Half16;  // conversions of a 16-bit type
template <>
struct Half16<__nv_bfloat16> {
  __device__ __forceinline__ static float2 pair(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  }
  __device__ __forceinline__ static uint32_t pack(float x, float y) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&p);
  }
  __device__ __forceinline__ static uint16_t bits(float v) { return __bfloat16_as_ushort(__float2bfloat16_rn(v)); }
  __device__ __forceinline__ static float value(uint16_t b) { return __uint_as_float(static_cast<uint32_t>(b) << 16); }
};
template <>
struct Half16<__half> {
  __device__ __forceinline__ static float2 pair(uint32_t w) {
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
  }
  __device__ __forceinline__ static uint32_t pack(float x, float y) {
    const __half2 p = __floats2half2_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&p);
  }
  __device__ __forceinline__ static uint16_t bits(float v) { return __half_as_ushort(__float2half_rn(v)); }
  __device__ __forceinline__ static float value(uint16_t b) { return __half2float(__ushort_as_half(b)); }
};

// ---------------------------------------------------------------------------
// a lane's own copies
// ---------------------------------------------------------------------------
// Weights, x and y come through rings in shared memory in which every lane copies (cp.async) what it will
// itself read, in the order of its registers: no barrier, no bank conflict, and as many bytes in flight as the
// ring holds, which registers do not (33 rows of 8 adapters x 151936: 56 us with loads to registers, 21 so).
// (The form that fills up with zeros was measured slower: 17 million wavefronts of shared memory in place of 6.)
template <int BYTES>
__device__ __forceinline__ void lane_copy(uint32_t smem_dst, const void* src) {
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_dst), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(smem_dst), "l"(src), "n"(BYTES) : "memory");
}
// The same where `go` holds, without a branch.
template <int BYTES>
__device__ __forceinline__ void lane_copy_if(bool go, uint32_t smem_dst, const void* src) {
  if constexpr (BYTES == 16)
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.s32 p, %2, 0;\n\t@p cp.async.cg.shared.global [%0], [%1], 16;\n\t}" ::"r"(
                     smem_dst), "l"(src), "r"(static_cast<int>(go))
                 : "memory");
  else
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.s32 p, %2, 0;\n\t@p cp.async.ca.shared.global [%0], [%1], %3;\n\t}" ::"r"(
                     smem_dst), "l"(src), "r"(static_cast<int>(go)), "n"(BYTES)
                 : "memory");
}
__device__ __forceinline__ void lane_copies_end() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// All but the last N groups of this lane's copies have arrived.
template <int N>
__device__ __forceinline__ void lane_copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// ---------------------------------------------------------------------------
// tiles
// ---------------------------------------------------------------------------
// The tiles of a call as a CTA sees them.
struct TileSmem {
  int32_t rows[kADTile];  // of the current tile
  int32_t adapter, count;
};

// Calls of many rows: the plan kernel's results.
struct PlannedTiles {
  // Returns the number of tiles.
  __device__ __forceinline__ int start(const AdapterArgs& a, TileSmem&) { return __ldcg(a.tile_count); }
  // All threads: tile `t`'s rows, adapter and count into sm (behind a barrier of its own).
  __device__ __forceinline__ void take(const AdapterArgs& a, TileSmem& sm, int t) {
    __syncthreads();  // nobody reads the tile before
    const int4 tile4 = __ldcg(reinterpret_cast<const int4*>(a.tiles + t));
    const AdapterTile tile{tile4.x, tile4.y, tile4.z, tile4.w};
    if (threadIdx.x == 0) sm.adapter = tile.adapter, sm.count = tile.count;
    if (threadIdx.x < static_cast<unsigned>(tile.count)) sm.rows[threadIdx.x] = __ldcg(a.order + tile.first + threadIdx.x);
    __syncthreads();
  }
};

// To kADOwnPlan rows: found by each CTA, of at least as many threads.  Thread i takes row i: its place among the rows
// of the same adapter gives its tile and its place in it, and a tile's number is its first row's among the rows that
// are first in a tile.
struct OwnTileSmem : TileSmem {
  alignas(16) int32_t adapter_of[kADOwnPlan];
  int32_t part;
};

struct TileFinder {
  int mine = -2;   // this thread's row's adapter (own plan); -2: no such row
  int place = 0;   // among the rows with the same
  int number = -1;  // of the tile that this thread's row is first in

  // All threads; the indices may be read.  (Through L2: this grid may start before the kernel that writes them ends,
  // and an L1 line could be of before.)  Returns the number of tiles.
  __device__ int start(const AdapterArgs& a, OwnTileSmem& sm) {
    const int i = threadIdx.x;
    if (i < a.rows) {
      mine = __ldcg(a.adapter_idx + i);
      if (mine < 0 || mine >= a.count) {
        if (mine != -1) set_status(a.dev_status, LMH_DS_ADAPTER_OUT_OF_RANGE);
        mine = -1;
      }
    }
    if (i < kADOwnPlan) sm.adapter_of[i] = mine;
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
    if (i < kADOwnPlan && (i & 31) == 0) sm.adapter_of[i >> 5] = __popc(firsts);
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kADOwnPlan / 32; ++w) {
      const int c = sm.adapter_of[w];
      before += w < (i >> 5) ? c : 0;
      all += c;
    }
    if (first) number = before + __popc(firsts & ((1u << (i & 31)) - 1));
    return all;
  }

  // All threads: tile `t`'s rows, adapter and count into sm (behind a barrier of its own).
  __device__ void take(const AdapterArgs& a, OwnTileSmem& sm, int t) {
    __syncthreads();  // nobody reads the tile before
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
  return adapter < 0 ? 0 : a.ranks ? min(max(__ldcg(a.ranks + adapter), 0), a.R) : a.R;
}

// ---------------------------------------------------------------------------
// first product
// ---------------------------------------------------------------------------
// One CTA a (tile, share of H).  Few rows are bound by latency here (33 rows of 2560 x rank 16: 7 us alone, of which
// the weights' 0.7 MB take 0.1).  A warp takes 16 rows of a small tile (or what there is of them), 32 of a
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
        if (rt * 8 + g < rank) lane_copy<16>(smem_u32(e + rt * 32), down + (rt * 8 + g) * a.down_row + h);
      if (a.x_vec)
#pragma unroll
        for (int c = 0; c < C; ++c)
          if (have[c]) lane_copy<16>(smem_u32(e + (2 * RT + c) * 32), xp[c] + kb * 32);
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
  __shared__ OwnTileSmem ts;
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
        tk = a.row_idx ? __ldcg(a.row_idx + ts.rows[tid]) : ts.rows[tid];
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
// first product, calls of many rows
// ---------------------------------------------------------------------------
// The batch's rows are the MMA's A operand, 16 a warp, and 8 adapter rows the B operand: the tile's four row groups
// share the weights, which come in stages of 128 entries of H that the whole CTA copies; two warps share a row group
// by entries of H.  As above a lane takes 16 contiguous bytes of a row for two steps of 16, so the operands need no
// transposition: a lane's registers of x are its own loads, a stage ahead.  (16384 rows of 1024 x rank 64: 21 us alone,
// 31 MB from DRAM; a wave of 261 tiles that each wait for their own eight stages.  x two stages ahead, 2 or 5 stages
// of weights: the same or slower.)
constexpr int kADDownStage = 128;  // entries of H: four blocks of 32
constexpr int kADDownStages = 3;
constexpr int down_wide_stage_bytes(int rt) { return rt * 16 * kADDownStage * 2; }
constexpr int down_wide_smem(int rt) {
  const int ring = kADDownStages * down_wide_stage_bytes(rt), sums = 4 * 16 * (rt * 16 + 4) * 4;
  return ring > sums ? ring : sums;
}

template <typename T, int RT>
__global__ void __launch_bounds__(kADThreads, RT <= 4 ? 2 : 1) adapter_down_wide_kernel(const AdapterArgs a) {
  extern __shared__ __align__(128) unsigned char dw_ring[];  // [stages][block of 32][adapter row][64 bytes]
  __shared__ TileSmem ts;
  constexpr int S = kADDownStages, NT = 2 * RT;  // NT: tiles of 8 adapter rows
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  const int rgroup = warp & 3, half = warp >> 2;  // half: blocks 2 half, 2 half + 1 of a stage
  pdl_wait();
  pdl_launch_dependents();
  PlannedTiles finder;
  const int n_tiles = finder.start(a, ts);
  // this CTA's share of H (few tiles: several shares), in stages
  const int all = (a.H + kADDownStage - 1) / kADDownStage;
  const int lo = static_cast<int>(static_cast<int64_t>(all) * blockIdx.y / a.splits);
  const int hi = static_cast<int>(static_cast<int64_t>(all) * (blockIdx.y + 1) / a.splits);
  for (int ti = blockIdx.x; ti < n_tiles; ti += gridDim.x) {
    finder.take(a, ts, ti);
    if (ts.adapter < 0) continue;  // (uniform)
    const int count = ts.count, rank = adapter_rank(a, ts.adapter);
    const T* down = reinterpret_cast<const T*>(a.down) + static_cast<int64_t>(ts.adapter) * a.down_adapter;
    auto issue = [&](int st) {
      if (st < hi) {
        // pieces of 16 bytes: 16 of an adapter row's 128 entries
        const int c = tid % 16, h = st * kADDownStage + c * 8;
        const uint32_t to = smem_u32(dw_ring) + st % S * down_wide_stage_bytes(RT) + (c / 4) * (RT * 16 * 64) + (c % 4) * 16;
#pragma unroll
        for (int i = 0; i < RT; ++i) {
          const int r = tid / 16 + i * 16;
          lane_copy_if<16>(r < rank && h < a.H, to + r * 64, down + r * a.down_row + h);
        }
      }
      lane_copies_end();
    };
    for (int i = 0; i < S - 1; ++i) issue(lo + i);
    const char* x[2];
    bool have[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int i = rgroup * 16 + u * 8 + g;
      int tk = -1;
      if (i < count) {
        tk = a.row_idx ? __ldcg(a.row_idx + ts.rows[i]) : ts.rows[i];
        if (tk < 0 || tk >= a.num_tokens) {
          tk = -1;  // reads zeros
          set_status(a.dev_status, LMH_DS_ROW_IDX_OUT_OF_RANGE);
        }
      }
      have[u] = tk >= 0;
      x[u] = a.x + (static_cast<int64_t>(max(tk, 0)) * a.x_stride + t * 8) * 2;
    }
    uint4 xv[2][2];  // [block][row], of the stage to come
    auto load_x = [&](int st) {
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const int h = st * kADDownStage + (half * 2 + b) * 32;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          xv[b][u] = make_uint4(0, 0, 0, 0);
          if (!have[u] || st >= hi || h + t * 8 >= a.H) continue;
          const char* p = x[u] + static_cast<int64_t>(h) * 2;
          if (a.x_vec) {
            xv[b][u] = __ldcg(reinterpret_cast<const uint4*>(p));
          } else {
            const uint16_t* e = reinterpret_cast<const uint16_t*>(p);
            xv[b][u] = make_uint4(e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6] | e[7] << 16);
          }
        }
      }
    };
    float acc[NT][4] = {};
    load_x(lo);
    const bool work = rgroup * 16 < count;
    for (int st = lo; st < hi; ++st) {
      uint4 xc[2][2];
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int u = 0; u < 2; ++u) xc[b][u] = xv[b][u];
      load_x(st + 1);  // (behind the share: zeros)
      lane_copies_wait<S - 2>();
      __syncthreads();  // the stage is there, and the one before it has been read
      issue(st + S - 1);
      if (!work) continue;
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const int block = half * 2 + b;
        const bool in = st * kADDownStage + block * 32 + t * 8 < a.H;
        const unsigned char* w = dw_ring + st % S * down_wide_stage_bytes(RT) + block * (RT * 16 * 64) + g * 64 + t * 16;
        const uint32_t a0[4] = {xc[b][0].x, xc[b][1].x, xc[b][0].y, xc[b][1].y};
        const uint32_t a1[4] = {xc[b][0].z, xc[b][1].z, xc[b][0].w, xc[b][1].w};
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          if (n * 8 >= rank) break;
          uint4 v = *reinterpret_cast<const uint4*>(w + n * (8 * 64));
          if (!in || n * 8 + g >= rank) v = make_uint4(0, 0, 0, 0);  // (not copied)
          mma16<T>(acc[n], a0, v.x, v.y);
          mma16<T>(acc[n], a1, v.z, v.w);
        }
      }
    }
    lane_copies_wait<0>();
    __syncthreads();  // the ring is done with
    // the halves' sums meet in shared memory: [row group][16 rows][RT * 16, and 4 so that rows differ in bank]
    constexpr int PITCH = RT * 16 + 4;
    float* sums = reinterpret_cast<float*>(dw_ring) + rgroup * (16 * PITCH);
    if (half == 1)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int u = 0; u < 2; ++u)
          *reinterpret_cast<float2*>(sums + (g + 8 * u) * PITCH + n * 8 + 2 * t) = make_float2(acc[n][2 * u], acc[n][2 * u + 1]);
    __syncthreads();
    if (half == 0)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int i = rgroup * 16 + u * 8 + g;
        if (i >= count) continue;
        float* d = a.d + (static_cast<int64_t>(blockIdx.y) * a.rows + ts.rows[i]) * a.R;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          if (n * 8 >= a.R) break;
          const float2 s = *reinterpret_cast<const float2*>(sums + (g + 8 * u) * PITCH + n * 8 + 2 * t);
          *reinterpret_cast<float2*>(d + n * 8 + 2 * t) = make_float2(acc[n][2 * u] + s.x, acc[n][2 * u + 1] + s.y);
        }
      }
  }
}

// ---------------------------------------------------------------------------
// second product, added to y
// ---------------------------------------------------------------------------
// The four outputs of one row that a lane holds of a step of 32: output(g, e), e = 0..3.  VEC: neighbours, read and
// written at once (16 bytes, or 8 of 16-bit outputs); else every eighth, neighbouring lanes holding neighbours.
// FULL: all of them are the row's; else those below `left` (counted from the lane's first).
template <typename Y, bool VEC>
struct Outputs {
  static constexpr int ES = static_cast<int>(sizeof(Y));
  static constexpr int BYTES = 4 * ES;               // of a lane and row
  static constexpr int ROWS4 = ES == 4 ? 512 : 320;  // bytes in the ring of the four rows that the lanes copy at once
  __device__ __forceinline__ static int output(int g, int e) { return VEC ? 4 * g + e : g + 8 * e; }
  // A lane's place for its share of a row of its own: those of a row are neighbours, as in memory (whole sectors), and
  // the four rows of a copy do not meet in a bank when a quarter of a warp reads.
  // (16-bit outputs that do not align: a row's 32 take 16 or 17 words of four bytes, the least that a copy moves.)
  __device__ __forceinline__ static int place(int lane) {
    const int g = lane >> 2, t = lane & 3;
    if constexpr (!VEC && ES == 2) return t * 80;
    return t * (8 * BYTES) + (((g >> 1) ^ t) * 2 + (g & 1)) * BYTES;
  }
  template <bool FULL>
  __device__ __forceinline__ static void copy(uint32_t to, const char* row, bool have, int left) {
    if constexpr (VEC) {
      lane_copy_if<4 * ES>(have && (FULL || left > 0), to, row);
    } else if constexpr (ES == 4) {
#pragma unroll
      for (int e = 0; e < 4; ++e) lane_copy_if<4>(have && (FULL || 8 * e < left), to + e * 4, row + 32 * e);
    } else {  // words g, g + 8 and (lane group 0) 16 of those that hold the row's outputs of the step
      const int g = (static_cast<int>(threadIdx.x) & 31) >> 2;
      const uintptr_t first = reinterpret_cast<uintptr_t>(row) - 2 * g;
      const int skip = static_cast<int>(first >> 1) & 1;
      const char* p = reinterpret_cast<const char*>(first - 2 * skip) + 4 * g;
#pragma unroll
      for (int w = 0; w < 3; ++w)
        lane_copy_if<4>(have && (w < 2 || (g == 0 && skip)) && (FULL || 2 * (g + 8 * w) - skip < left + g), to + 4 * (g + 8 * w),
                        p + 32 * w);
    }
  }
  // d[e] times `by` is added to output e.
  template <bool FULL>
  __device__ __forceinline__ static void add_and_store(const unsigned char* in, const char* y_row, char* row, bool have,
                                                       int left, const float (&d)[4], float by) {
    if constexpr (ES == 4) {
      const float4 v = *reinterpret_cast<const float4*>(in);
      const float4 r = make_float4(fmaf(d[0], by, v.x), fmaf(d[1], by, v.y), fmaf(d[2], by, v.z), fmaf(d[3], by, v.w));
      if constexpr (VEC) {
        if (have && (FULL || left > 0)) *reinterpret_cast<float4*>(row) = r;
      } else {
        const float f[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (have && (FULL || 8 * e < left)) reinterpret_cast<float*>(row)[8 * e] = f[e];
      }
    } else {
      using C = Half16<Y>;
      if constexpr (VEC) {
        const uint2 v = *reinterpret_cast<const uint2*>(in);
        const float2 a = C::pair(v.x), b = C::pair(v.y);
        const uint2 w = make_uint2(C::pack(fmaf(d[0], by, a.x), fmaf(d[1], by, a.y)),
                                   C::pack(fmaf(d[2], by, b.x), fmaf(d[3], by, b.y)));
        if (have && (FULL || left > 0)) *reinterpret_cast<uint2*>(row) = w;
      } else {
        const int g = (static_cast<int>(threadIdx.x) & 31) >> 2;
        const int skip = static_cast<int>((reinterpret_cast<uintptr_t>(y_row) >> 1) - g) & 1;
        const uint16_t* v = reinterpret_cast<const uint16_t*>(in) + skip + g;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint16_t r = C::bits(fmaf(d[e], by, C::value(v[8 * e])));
          if (have && (FULL || 8 * e < left)) reinterpret_cast<uint16_t*>(row)[8 * e] = r;
        }
      }
    }
  }
};

template <int KS>
struct UpSmem {
  // d in MMA order, a lane's registers of a step: the 16-bit values (b0, b1) and what their rounding left (b0, b1)
  uint4 frag[KS][kADCols][32];
  float unscale[kADTile];  // f16: the power of two that a row's d was divided by
  int64_t y[kADTile], out[kADTile];  // the rows' first bytes
};

// All threads: a tile's d, scaled, into sm.  A warp takes every W-th row, four at a time, all of whose loads of a share
// of H are out before the first is used (128 rows of rank 64, 4096 -> 4096: 27 us with a row at a time, 17 so, which
// takes 8 warps in place of 16 for rank 64).
template <typename T, int KS, int W>
__device__ void up_operand(const AdapterArgs& a, const TileSmem& ts, UpSmem<KS>& sm, int rank) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int count = ts.count, cols = (count + 7) / 8;
  const float scale = ts.adapter < 0 ? 0.0f : a.scales ? __ldcg(a.scales + ts.adapter) : 1.0f;
  constexpr int PER = (KS * 16 + 31) / 32;  // entries a lane
  auto rows = [&](auto rows_const, int first) {  // of a warp
    constexpr int K = decltype(rows_const)::value;
    float v[K][PER] = {};
    const float* d[K];
#pragma unroll
    for (int k = 0; k < K; ++k) d[k] = a.d + static_cast<int64_t>(ts.rows[min(first + k * W, count - 1)]) * a.R;
    if (rank > 0 && first < count) {
#pragma unroll (K == 1 ? 4 : 2)
      for (int s = 0; s < a.splits; ++s) {
        const int64_t off = static_cast<int64_t>(s) * a.rows * a.R;
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
          for (int u = 0; u < PER; ++u) v[k][u] += __ldcg(d[k] + off + min(u * 32 + lane, a.R - 1));
      }
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int i = first + k * W;
      if (i >= cols * 8) break;
      float most = 0.0f;
#pragma unroll
      for (int u = 0; u < PER; ++u) {
        v[k][u] = i < count && u * 32 + lane < rank ? v[k][u] * scale : 0.0f;
        most = fmaxf(most, fabsf(v[k][u]));
      }
      float by = 1.0f;
      if constexpr (std::is_same<T, __half>::value) {
        // f16: the row's largest value goes into [2^13, 2^14), which is exact
        float back = 1.0f;
        most = warp_max(most);
        if (most > 0.0f && most < INFINITY) {
          const int e = min(max(ilogbf(most), -112), 127);
          by = ldexpf(1.0f, 13 - e);
          back = ldexpf(1.0f, e - 13);
        }
        if (lane == 0) sm.unscale[i] = back;
      }
#pragma unroll
      for (int u = 0; u < PER; ++u) {
        const int r = u * 32 + lane;
        if (r >= KS * 16) break;
        const float f = v[k][u] * by;
        const uint16_t high = Half16<T>::bits(f);
        const int reg = (r >> 3) & 1;  // of the step r / 16, in the lane of r's pair
        uint16_t* p = reinterpret_cast<uint16_t*>(&sm.frag[r >> 4][i >> 3][(i & 7) * 4 + ((r & 7) >> 1)]);
        p[reg * 2 + (r & 1)] = high;
        const float hv = Half16<T>::value(high);
        p[4 + reg * 2 + (r & 1)] = Half16<T>::bits(fabsf(hv) < INFINITY ? f - hv : 0.0f);
      }
    }
  };
  if (cols * 8 <= W) {
    rows(std::integral_constant<int, 1>{}, warp);
  } else {
#pragma unroll 1
    for (int first = warp; first < cols * 8; first += 4 * W) rows(std::integral_constant<int, 4>{}, first);
  }
}

// A warp's weights of a step: two MMAs' A operands, of 16 outputs each.  They come in 16-byte pieces of a row, CH to a
// row, neighbouring lanes copying neighbouring pieces.  The two pieces of a 32-byte sector stay together: copies of
// one sector to two places are two reads from L2 (measured: 2x the sectors, 110 us in place of 92 for 64 rows of 48
// adapters of rank 32).  A row stands at 32 KS times its number, its sectors' places within 128 bytes exclusive-ored
// with two bits of the number and the halves' places in a sector with a third, so that no two of a matrix's eight rows
// (ldmatrix) meet in a bank (64 rows of 48 adapters: 79 us with two to a bank, 77 so).
template <bool VEC, int KS>
struct UpPlaces {
  static constexpr int CH = 2 * KS;      // pieces of a row
  static constexpr int ROWS = 32 / CH;   // rows that the lanes copy at a time
  static constexpr int COPIES = kADStep / ROWS;
  __device__ __forceinline__ static int at(int row, int c) {
    const int x = VEC ? row >> 2 : KS == 1 ? 0 : KS == 2 ? (row >> 1) & 1 : row;
    return (row * (32 * KS) + c * 16) ^ ((x & 3) << 5) ^ ((row >> (VEC ? 4 : 2) & 1) << 4);
  }
};

// A warp's ring: entries of the weights of a step and of y for C tiles of 8 rows.  A CTA has an SM for itself, with as
// many warps as its registers allow (8 to 12 bytes spilled for ranks above 64, none below), each with a ring of at least
// two of the larger entries.
constexpr int kADUpCols = 2;                                                         // C of tiles of more than 8 rows
constexpr int up_entry(int ks, int es, int c) { return ks * 1024 + c * (es == 4 ? 1024 : 640); }
constexpr int kADUpStatic = 2900;  // (what else a CTA holds beside d)
constexpr int up_ring_bytes(int ks) { return 227 * 1024 - ks * kADCols * 32 * 16 - kADUpStatic; }
constexpr int up_warps(int ks) { return ks <= 2 ? 16 : 8; }
constexpr int up_warp_bytes(int ks) { return up_ring_bytes(ks) / up_warps(ks) / 512 * 512; }
constexpr int up_depth(int ks, int es, int c) {
  const int n = up_warp_bytes(ks) / up_entry(ks, es, c);
  return n < 8 ? n : 8;
}

// A tile's start (its rows, the first copies, d) takes a CTA about as long as this many steps: 33 rows of 8 adapters x
// 151936 take 20.5 us in a graph with equal shares, 19.3 so.  Not more than a part of a tile, as shares of small calls
// would be all start (5 rows x 4096: 4.5 us, 4.8 with 64 steps).
__device__ __forceinline__ int up_start(int64_t steps) { return static_cast<int>(min(static_cast<int64_t>(96), steps / 32)); }

// A warp's part of a tile's outputs [.., n_end): every step that is the warp's.  C: column tiles of an entry; a tile of
// more rows has several entries a step, of which the first brings the weights.
// start(): the copies that fill the ring; run(): the rest, once d stands in sm.
template <typename T, typename Y, int KS, bool VEC, int C>
struct UpShare {
  static constexpr int ES = static_cast<int>(sizeof(Y)), J = 2, STEP = kADStep;
  using O = Outputs<Y, VEC>;
  using P = UpPlaces<VEC, KS>;
  static constexpr int D = up_depth(KS, ES, C), ENTRY = up_entry(KS, ES, C);
  static constexpr int STRIDE = up_warps(KS) * STEP;  // outputs from a step to the warp's next
  static constexpr int W_BYTES = J * KS * 512, ROW_BYTES = O::ROWS4;
  static_assert(D >= 2, "a ring of two entries at least");
  const AdapterArgs& a;
  const UpSmem<KS>& sm;
  int rank, count, n_end, t, parts;  // parts: entries a step
  unsigned char* ring_y;       // the lane's place for y in the first entry
  uint32_t ring;               // the first entry
  bool in_rank;                // the lane's pieces of the weight rows are
  // the next entry to be copied
  const char* wp;              // the lane's first piece
  int64_t pitch, step;         // bytes from a piece to the lane's next, and to the warp's next step's
  const char* yp0;             // C 1: the lane's two rows of y, and of out, at its first output
  const char* yp1;
  char* op0;
  char* op1;
  int in_n0, in_part, in_at;   // the step's first output, the entry's number in it, its offset in the ring
  int lane_n;                  // the lane's first output, from the step's

  __device__ __forceinline__ UpShare(const AdapterArgs& args, const UpSmem<KS>& s, const T* up,
                                     unsigned char* warp_ring, int rank_, int count_, int n_first, int n_end_)
      : a(args), sm(s), rank(rank_), count(count_), n_end(n_end_) {
    const int lane = threadIdx.x & 31;
    t = lane & 3;
    parts = C == 1 ? 1 : (count + 8 * C - 1) / (8 * C);
    ring = smem_u32(warp_ring);
    ring_y = warp_ring + W_BYTES + O::place(lane);
    in_n0 = n_first;
    lane_n = O::output(lane >> 2, 0);
    in_at = in_part = 0;
    in_rank = (lane % P::CH) * 8 < rank;
    wp = reinterpret_cast<const char*>(up + (n_first + lane / P::CH) * a.up_row + (lane % P::CH) * 8);
    pitch = 2 * P::ROWS * a.up_row;
    step = 2 * STRIDE * a.up_row;
    if constexpr (C == 1) {
      const int64_t off = static_cast<int64_t>(n_first + lane_n) * ES;
      const int i0 = min(2 * t, count - 1), i1 = min(2 * t + 1, count - 1);
      yp0 = a.y + sm.y[i0] + off, yp1 = a.y + sm.y[i1] + off;
      op0 = a.out + sm.out[i0] + off, op1 = a.out + sm.out[i1] + off;
    }
  }
  template <bool FULL>
  __device__ __forceinline__ void copy_entry() {
    const int lane = threadIdx.x & 31;
    if ((C == 1 || in_part == 0) && rank > 0) {
      const char* p = wp;
#pragma unroll
      for (int i = 0; i < P::COPIES; ++i) {
        const int row = lane / P::CH + i * P::ROWS;
        const uint32_t to = ring + in_at + P::at(row, lane % P::CH);
        lane_copy_if<16>(in_rank && (FULL || in_n0 + row < n_end), to, p);
        p += pitch;
      }
    }
    const int left = n_end - in_n0 - lane_n;
    const uint32_t to = smem_u32(ring_y) + in_at;
    if constexpr (C == 1) {
      O::template copy<FULL>(to, yp0, 2 * t < count, left);
      O::template copy<FULL>(to + ROW_BYTES, yp1, 2 * t + 1 < count, left);
    } else {
      const char* y = a.y + static_cast<int64_t>(in_n0 + lane_n) * ES;
      const int row = in_part * (8 * C) + 2 * t;
#pragma unroll
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int u = 0; u < 2; ++u)  // (rows behind the last have offsets of it)
          O::template copy<FULL>(to + (2 * c + u) * ROW_BYTES, y + sm.y[row + c * 8 + u], row + c * 8 + u < count, left);
    }
  }
  __device__ __forceinline__ void issue() {
    if (in_n0 < n_end) {
      if (in_n0 + STEP <= n_end) copy_entry<true>();
      else copy_entry<false>();
      if (C == 1 || ++in_part == parts) {
        in_part = 0;
        in_n0 += STRIDE;
        wp += step;
        if constexpr (C == 1) yp0 += STRIDE * ES, yp1 += STRIDE * ES;
      }
      in_at = in_at == (D - 1) * ENTRY ? 0 : in_at + ENTRY;
    }
    lane_copies_end();
  }
  __device__ __forceinline__ void start() {
#pragma unroll 1
    for (int j = 0; j < D - 1; ++j) issue();
  }
  // The weights of the entry, as far as the rank goes.
  __device__ __forceinline__ void read_weights(uint32_t entry, uint32_t (&w)[KS][J][4]) const {
    const int lane = threadIdx.x & 31;
    // a rank that ends inside a step's 16 entries: the words of its two pieces that count
    const int rest = rank % 16 - 2 * t;
    const uint32_t keep0 = rank % 16 == 0 || rest >= 2 ? ~0u : rest == 1 ? 0xFFFFu : 0u;
    const uint32_t keep1 = rank % 16 == 0 || rest >= 10 ? ~0u : rest == 9 ? 0xFFFFu : 0u;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      if (ks * 16 >= rank) break;
#pragma unroll
      for (int j = 0; j < J; ++j) {
        // matrices of the tile: a lane group's outputs 2 j and 2 j + 1 (e) in piece 2 ks, the same in piece 2 ks + 1
        const int e = 2 * j + ((lane >> 3) & 1);
        load_matrices(w[ks][j], entry + P::at(O::output(lane & 7, e), 2 * ks + (lane >> 4)));
      }
      if (ks * 16 + 16 > rank) {
#pragma unroll
        for (int j = 0; j < J; ++j) w[ks][j][0] &= keep0, w[ks][j][1] &= keep0, w[ks][j][2] &= keep1, w[ks][j][3] &= keep1;
      }
    }
  }
  // acc[c][j] = the step's outputs 16 j .. times column tile c of the entry's part of d.
  __device__ __forceinline__ void multiply(const uint32_t (&w)[KS][J][4], int part,
                                           const uint4 (&kept)[KS], float (&acc)[C][J][4]) const {
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      if (ks * 16 >= rank) break;
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const uint4 b = C == 1 ? kept[ks] : sm.frag[ks][part * C + c][threadIdx.x & 31];
#pragma unroll
        for (int j = 0; j < J; ++j) {
          if (ks == 0) mma16_first<T>(acc[c][j], w[ks][j], b.x, b.y);
          else mma16<T>(acc[c][j], w[ks][j], b.x, b.y);
        }
#pragma unroll
        for (int j = 0; j < J; ++j) mma16<T>(acc[c][j], w[ks][j], b.z, b.w);
      }
    }
  }
  // A column tile's results: rows i and i + 1 of the tile.
  template <bool FULL>
  __device__ __forceinline__ void finish(const float (&acc)[J][4], int i, const unsigned char* in, int n) {
    const int64_t off = static_cast<int64_t>(n) * ES;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      float dv[2 * J];
#pragma unroll
      for (int e = 0; e < 2 * J; ++e) dv[e] = acc[e >> 1][(e & 1) * 2 + u];
      const float back = std::is_same<T, __half>::value ? sm.unscale[i + u] : 1.0f;
      const char* y = C == 1 ? (u ? yp1 : yp0) : a.y + off + sm.y[i + u];
      char* out = C == 1 ? (u ? op1 : op0) : a.out + off + sm.out[i + u];
      O::template add_and_store<FULL>(in + u * ROW_BYTES, y, out, i + u < count, n_end - n, dv, back);
    }
  }
  __device__ __forceinline__ void run(int n0) {
    const int lane = threadIdx.x & 31;
    int at = 0, part = 0;
    uint4 kept[KS];
    if constexpr (C == 1) {
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) kept[ks] = sm.frag[ks][0][lane];
    }
    uint32_t w[KS][J][4];
    while (n0 < n_end) {
      __syncwarp();  // the entry that is copied over has been read by all lanes
      issue();
      lane_copies_wait<D - 1>();
      __syncwarp();  // the weights are read by other lanes than copied them
      if (C == 1 || part == 0) read_weights(ring + at, w);
      float acc[C][J][4];
      multiply(w, part, kept, acc);
      if (rank == 0) {  // nothing is added: -0, which leaves a y of -0 too
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
          for (int j = 0; j < J; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[c][j][e] = -0.0f;
      }
      const bool full = n0 + STEP <= n_end;
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const unsigned char* in = ring_y + at + 2 * c * ROW_BYTES;
        const int i = (part * C + c) * 8 + 2 * t;
        if (full) finish<true>(acc[c], i, in, n0 + lane_n);
        else finish<false>(acc[c], i, in, n0 + lane_n);
      }
      if (C == 1 || ++part == parts) {
        part = 0;
        n0 += STRIDE;
        if constexpr (C == 1) {
          op0 += STRIDE * ES, op1 += STRIDE * ES;
        }
      }
      at = at == (D - 1) * ENTRY ? 0 : at + ENTRY;
    }
    lane_copies_wait<0>();
    __syncwarp();
  }
};

// The work is (tile, step of outputs); every CTA takes a contiguous share, so that it seldom changes tiles.
template <typename T, typename Y, int KS, bool VEC>
__global__ void __launch_bounds__(32 * up_warps(KS), 1) adapter_up_kernel(const AdapterArgs a) {
  extern __shared__ __align__(128) unsigned char up_ring[];
  __shared__ UpSmem<KS> sm;
  __shared__ OwnTileSmem ts;
  constexpr int STEP = kADStep;
  const int tid = threadIdx.x, warp = tid >> 5;
  // the kernel before this one is the first product, which has itself waited for all before it: only d has to
  // wait for its end, and what the plan kernel wrote has been waited for
  TileFinder finder;
  const int n_tiles = finder.start(a, ts);
  // a share that goes on in a second tile is shorter by what the tile's start takes
  const int start = up_start((a.N + STEP - 1) / STEP);
  const int64_t steps = (a.N + STEP - 1) / STEP + start;
  const int64_t all = steps * n_tiles;
  int64_t at = all * blockIdx.x / gridDim.x;
  const int64_t end = all * (blockIdx.x + 1) / gridDim.x;
  bool waited = false;
  while (at < end) {
    const int ti = static_cast<int>(at / steps);
    const int from = static_cast<int>(at - ti * steps), to = static_cast<int>(min(steps, from + (end - at)));
    at += to - from;
    const int s0 = max(0, from - start), s1 = max(0, to - start);
    if (s0 == s1) continue;
    finder.take(a, ts, ti);
    const int count = ts.count, rank = adapter_rank(a, ts.adapter);
    if (tid < kADTile) {
      const int row = ts.rows[min(tid, count - 1)];
      sm.y[tid] = row * a.y_stride * static_cast<int64_t>(sizeof(Y));
      sm.out[tid] = row * a.out_stride * static_cast<int64_t>(sizeof(Y));
    }
    __syncthreads();
    const T* up = reinterpret_cast<const T*>(a.up) + static_cast<int64_t>(max(ts.adapter, 0)) * a.up_adapter;
    unsigned char* ring = up_ring + warp * up_warp_bytes(KS);
    const int n_first = (s0 + warp) * STEP, n_end = min(a.N, s1 * STEP);
    auto share = [&](auto&& part) {
      part.start();
      if (!waited) pdl_wait();
      waited = true;
      up_operand<T, KS, up_warps(KS)>(a, ts, sm, rank);
      __syncthreads();
      part.run(n_first);
    };
    if (count <= 8) share(UpShare<T, Y, KS, VEC, 1>(a, sm, up, ring, rank, count, n_first, n_end));
    else share(UpShare<T, Y, KS, VEC, kADUpCols>(a, sm, up, ring, rank, count, n_first, n_end));
  }
  // a CTA without work waits too: this grid is not to end before the one that makes d
  if (!waited) pdl_wait();
}

// ---------------------------------------------------------------------------
// second product, calls of many rows
// ---------------------------------------------------------------------------
// Here the batch's rows are the MMA's A operand (16 a warp, held in registers for a whole tile) and 8 rows of the
// weights the B operand.  A lane's part of d and its two rows of y and out stay the same from step to step, which
// leaves about a fifth of the instructions of the kernel above per output (packed prompts, 16384 rows of rank 64 x
// 4096, with one part of d: 108 us there, 60 here; with both 66 here).  268 MB of rows make a floor of 40 us; issue
// slots are 35% busy, the tensor pipe 44% and DRAM 54%: what is left is latency, of a tile's start and of the stages'
// barriers, with 16 warps an SM.  For ranks of 33 to 64 some of the kernel's registers spill (up to 68 bytes; none
// for aligned bf16 outputs).
// The weights come in stages of kADWideStage outputs that the whole CTA copies and reads; warps share a stage by rows
// (one for every 16 of the tile's) and by outputs.  A block is 32 outputs; column c of its tile j stands for output
// 8 (c / 2) + 2 j + c % 2, so that a lane has eight neighbours of a row.
constexpr int kADWideThreads = 256;
constexpr int kADWideWarps = kADWideThreads / 32;
constexpr int kADWideStages = 3;
// Outputs of a stage: of 64-row tiles a warp takes two blocks.  (Four, and a ring twice as large, with one part of d for
// 16-bit outputs: 75 us for packed prompts' second product where this took 60, and 109 for 1257 fp32 rows of rank 64 x
// 23728 where this took 98.
// What is in flight queues then: even the copies' issue waited 1500 cycles a stage.)
constexpr int kADWideStage = 128;
constexpr int wide_stage_bytes(int ks) { return kADWideStage * 32 * ks; }

// Eight neighbouring outputs of a row, read and written in pieces of PIECE bytes: 16, or 8 where 16-bit rows align for
// no more (N a multiple of 4: 1591 rows of rank 16 x 42180 bf16 take 84 us so, 141 as unaligned rows).
template <typename Y, int PIECE>
struct Eight {
  static constexpr int ES = static_cast<int>(sizeof(Y)), PN = PIECE / ES;  // PN: outputs of a piece
  uint32_t w[2 * ES];
  // Outputs n .. n + 7 of the row at `row`; pieces that are not below `end` are read from its start.
  __device__ __forceinline__ void load(const char* row, int n, int end) {
#pragma unroll
    for (int p = 0; p < 8 / PN; ++p) {
      const int at = n + p * PN;
      const char* from = row + static_cast<int64_t>(at < end ? at : 0) * ES;
      if constexpr (PIECE == 16) {
        const uint4 v = *reinterpret_cast<const uint4*>(from);
        w[4 * p] = v.x, w[4 * p + 1] = v.y, w[4 * p + 2] = v.z, w[4 * p + 3] = v.w;
      } else {
        const uint2 v = *reinterpret_cast<const uint2*>(from);
        w[2 * p] = v.x, w[2 * p + 1] = v.y;
      }
    }
  }
  // d[e] times `by` is added to output e, and those below `left` are written.
  __device__ __forceinline__ void add_and_store(char* row, int left, const float (&d)[8], float by) const {
    if constexpr (ES == 4) {
#pragma unroll
      for (int p = 0; p < 2; ++p)
        if (left > 4 * p)
          *reinterpret_cast<float4*>(row + 16 * p) =
              make_float4(fmaf(d[4 * p], by, __uint_as_float(w[4 * p])), fmaf(d[4 * p + 1], by, __uint_as_float(w[4 * p + 1])),
                          fmaf(d[4 * p + 2], by, __uint_as_float(w[4 * p + 2])), fmaf(d[4 * p + 3], by, __uint_as_float(w[4 * p + 3])));
    } else {
      using C = Half16<Y>;
      uint32_t r[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 v = C::pair(w[i]);
        r[i] = C::pack(fmaf(d[2 * i], by, v.x), fmaf(d[2 * i + 1], by, v.y));
      }
      if constexpr (PIECE == 16) {
        if (left > 0) *reinterpret_cast<uint4*>(row) = make_uint4(r[0], r[1], r[2], r[3]);
      } else {
        if (left > 0) *reinterpret_cast<uint2*>(row) = make_uint2(r[0], r[1]);
        if (left > 4) *reinterpret_cast<uint2*>(row + 8) = make_uint2(r[2], r[3]);
      }
    }
  }
};

// Rows that do not align for that: a block's 16 rows x 32 outputs cross shared memory, and a lane reads and writes
// one output of each row, neighbouring lanes neighbours.
template <typename Y>
struct Sixteen {
  static constexpr int ES = static_cast<int>(sizeof(Y));
  uint32_t w[16];  // the lane's output of every row
  // Output n of the rows at base + off[i] (that of the row's start, if n is not below `end`).
  __device__ __forceinline__ void load(const char* base, const int64_t* off, int n, int end) {
    const int64_t at = static_cast<int64_t>(n < end ? n : 0) * ES;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const char* p = base + off[i] + at;
      if constexpr (ES == 4) w[i] = *reinterpret_cast<const uint32_t*>(p);
      else w[i] = *reinterpret_cast<const uint16_t*>(p);
    }
  }
  // delta[i * pitch] is added to the output of row i, of `rows` rows.
  __device__ __forceinline__ void add_and_store(char* base, const int64_t* off, int n, bool in, int rows, const float* delta,
                                                int pitch) const {
    const int64_t at = static_cast<int64_t>(n) * ES;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float d = delta[i * pitch];
      if (i >= rows || !in) continue;
      char* p = base + off[i] + at;
      if constexpr (ES == 4) *reinterpret_cast<float*>(p) = __uint_as_float(w[i]) + d;
      else *reinterpret_cast<uint16_t*>(p) = Half16<Y>::bits(Half16<Y>::value(static_cast<uint16_t>(w[i])) + d);
    }
  }
};

constexpr int wide_ctas(int ks) { return ks <= 4 ? 2 : 1; }

// PIECE: bytes of a row that are read and written at once, 0: its elements.
template <typename T, typename Y, int KS, int PIECE>
__global__ void __launch_bounds__(kADWideThreads, wide_ctas(KS)) adapter_wide_kernel(const AdapterArgs a) {
  extern __shared__ __align__(128) unsigned char wide_ring[];
  __shared__ TileSmem ts;
  constexpr bool VEC = PIECE != 0;
  constexpr int ES = static_cast<int>(sizeof(Y)), CH = 2 * KS, S = kADWideStages;
  constexpr int STAGE = kADWideStage, STAGE_BYTES = wide_stage_bytes(KS), MOST = STAGE / 64;  // MOST: blocks a warp
  constexpr int ROWS = kADWideThreads / CH;  // weight rows that the CTA copies at a time
  using Held = typename std::conditional<VEC, Eight<Y, VEC ? PIECE : 16>[2], Sixteen<Y>>::type;  // y of a lane and block
  constexpr int PITCH = 36;
  __shared__ float cross[VEC ? 1 : kADWideWarps][VEC ? 1 : 16 * PITCH];
  __shared__ int64_t offs[VEC ? 1 : 4][2][VEC ? 1 : 16];  // [16 rows of the tile][y, out]: the rows' first bytes
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  // (as in the kernel above: all but d was complete before this kernel started)
  PlannedTiles finder;
  const int n_tiles = finder.start(a, ts);
  const int64_t stages = (a.N + STAGE - 1) / STAGE;
  const int64_t all = stages * n_tiles;
  int64_t at = all * blockIdx.x / gridDim.x;
  const int64_t end = all * (blockIdx.x + 1) / gridDim.x;
  // where a weight row's piece stands in a stage: sectors stay whole, and no two of a matrix's eight rows meet in a
  // bank (packed prompts: 109 us with two to a bank, 102 so)
  auto place = [](int row, int c) { return (row * (32 * KS) + c * 16) ^ (((row >> 3) & 3) << 5) ^ ((row & 1) << 4); };
  bool waited = false;
  while (at < end) {
    const int ti = static_cast<int>(at / stages);
    const int s0 = static_cast<int>(at - ti * stages), s1 = static_cast<int>(min(stages, s0 + (end - at)));
    at += s1 - s0;
    finder.take(a, ts, ti);
    const int count = ts.count, rank = adapter_rank(a, ts.adapter);
    const int rg = count <= 16 ? 1 : count <= 32 ? 2 : 4, ng = kADWideWarps / rg;  // warps by rows and by outputs
    const int row0 = (warp % rg) * 16 + g;
    const int blocks = max(1, STAGE / 32 / ng), first_block = warp / rg * blocks;  // of a stage, the warp's: neighbours
    const bool idle = first_block * 32 >= STAGE;  // (fewer blocks than warps)
    const bool have[2] = {row0 < count, row0 + 8 < count};
    const int row[2] = {ts.rows[have[0] ? row0 : 0], ts.rows[have[1] ? row0 + 8 : 0]};
    const char* y[2];
    char* out[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      y[u] = a.y + (row[u] * a.y_stride + 8 * t) * ES;
      out[u] = a.out + (row[u] * a.out_stride + 8 * t) * ES;
    }
    const T* up = reinterpret_cast<const T*>(a.up) + static_cast<int64_t>(max(ts.adapter, 0)) * a.up_adapter;
    auto issue = [&](int st) {
      if (st < s1 && rank > 0) {
        const int n0 = st * STAGE;
        const uint32_t to = smem_u32(wide_ring) + (st - s0) % S * STAGE_BYTES;
        const int c = tid % CH;
        const T* p = up + (n0 + tid / CH) * a.up_row + c * 8;
#pragma unroll
        for (int i = 0; i < STAGE / ROWS; ++i) {
          const int r = tid / CH + i * ROWS;
          lane_copy_if<16>(c * 8 < rank && n0 + r < a.N, to + place(r, c), p);
          p += ROWS * a.up_row;
        }
      }
      lane_copies_end();
    };
    for (int i = 0; i < S - 1; ++i) issue(s0 + i);

    // y of a stage; a block's is replaced by the next stage's as soon as it is used.  No branch and no condition, so
    // that nothing waits for it before its use: rows that are not there have the first one's address, outputs behind
    // the row's end and stages behind the last the row's start.
    Held v[MOST];
    const int rset = warp % rg, rows_here = count - rset * 16;
    if constexpr (!VEC) {
      if (tid < kADTile) {
        const int64_t r = ts.rows[min(tid, count - 1)];
        offs[tid / 16][0][tid % 16] = r * a.y_stride * ES;
        offs[tid / 16][1][tid % 16] = r * a.out_stride * ES;
      }
      __syncthreads();
    }
    auto load_block = [&](int st, int b) {
      const int n = st * STAGE + (first_block + b) * 32, end = st < s1 ? a.N : 0;
      if constexpr (VEC) {
#pragma unroll
        for (int u = 0; u < 2; ++u) v[b][u].load(y[u] - 8 * t * ES, n + 8 * t, end);
      } else {
        v[b].load(a.y, offs[rset][0], n + lane, end);
      }
    };
#pragma unroll
    for (int b = 0; b < MOST; ++b)
      if (b < blocks) load_block(s0, b);
    if (!waited) pdl_wait();
    waited = true;

    // ---- the lane's part of d: rows row0 and row0 + 8, entries 2 t, 2 t + 1, 2 t + 8, 2 t + 9 of every 16 ----
    const float scale = ts.adapter < 0 ? 0.0f : a.scales ? __ldcg(a.scales + ts.adapter) : 1.0f;
    uint32_t hi[KS][4], lo[KS][4];
    float back[2] = {1.0f, 1.0f};
    {
      // (every load of a share of H is out before the first is used; what is not there is read from the row's start;
      // one after the other: 102 us for packed prompts, 97 so)
      float2 p[2][KS][2] = {};
      for (int i = 0; i < a.splits; ++i) {
        const float* d = a.d + static_cast<int64_t>(i) * a.rows * a.R + 2 * t;
        float2 q[2][KS][2];
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int e = 0; e < 2 * KS; ++e)  // (R is a multiple of 8)
            q[u][e >> 1][e & 1] =
                __ldcg(reinterpret_cast<const float2*>(d + static_cast<int64_t>(row[u]) * a.R + (e * 8 < a.R ? e * 8 : 0)));
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int e = 0; e < 2 * KS; ++e) {
            p[u][e >> 1][e & 1].x += q[u][e >> 1][e & 1].x;
            p[u][e >> 1][e & 1].y += q[u][e >> 1][e & 1].y;
          }
      }
      float v[2][KS][4];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        float most = 0.0f;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int r = ks * 16 + h * 8 + 2 * t;
            v[u][ks][2 * h] = have[u] && r < rank ? p[u][ks][h].x * scale : 0.0f;
            v[u][ks][2 * h + 1] = have[u] && r + 1 < rank ? p[u][ks][h].y * scale : 0.0f;
            most = fmaxf(most, fmaxf(fabsf(v[u][ks][2 * h]), fabsf(v[u][ks][2 * h + 1])));
          }
        if constexpr (std::is_same<T, __half>::value) {
          // f16: the row's largest value goes into [2^13, 2^14), which is exact
          most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 1));
          most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 2));
          if (most > 0.0f && most < INFINITY) {
            const int e = min(max(ilogbf(most), -112), 127);
            back[u] = ldexpf(1.0f, e - 13);
#pragma unroll
            for (int ks = 0; ks < KS; ++ks)
#pragma unroll
              for (int q = 0; q < 4; ++q) v[u][ks][q] *= ldexpf(1.0f, 13 - e);
          }
        }
      }
#pragma unroll
      for (int ks = 0; ks < KS; ++ks)
#pragma unroll
        for (int q = 0; q < 4; ++q) {  // registers (row, k), (row + 8, k), (row, k + 8), (row + 8, k + 8)
          const float x0 = v[q & 1][ks][(q >> 1) * 2], x1 = v[q & 1][ks][(q >> 1) * 2 + 1];
          hi[ks][q] = Half16<T>::pack(x0, x1);
          const float2 b = Half16<T>::pair(hi[ks][q]);
          lo[ks][q] = Half16<T>::pack(fabsf(b.x) < INFINITY ? x0 - b.x : 0.0f, fabsf(b.y) < INFINITY ? x1 - b.y : 0.0f);
        }
    }
    // a rank that ends inside a step's 16 entries: the words of its two pieces that count
    const int rest = rank % 16 - 2 * t;
    const uint32_t keep0 = rank % 16 == 0 || rest >= 2 ? ~0u : rest == 1 ? 0xFFFFu : 0u;
    const uint32_t keep1 = rank % 16 == 0 || rest >= 10 ? ~0u : rest == 9 ? 0xFFFFu : 0u;

    const int last = rank % 16 != 0 ? rank / 16 : -1;  // the step of 16 entries that is cut

    // lane 8 i + c gives the row of matrix i that column c stands for; its place in a stage's first block (tile j: 64 KS
    // bytes further on, block b: 1024 KS; KS 1: matrices of two tiles' two pieces, else of a tile's four of 32 entries)
    const int mc = lane & 7, mi = lane >> 3, mrow = 8 * (mc >> 1) + (mc & 1);
    uint32_t from[KS == 1 ? 1 : KS / 2];
    if constexpr (KS == 1) {
      from[0] = place(mrow + 2 * (mi >> 1), mi & 1);
    } else {
#pragma unroll
      for (int kp = 0; kp < KS / 2; ++kp) from[kp] = place(mrow, 4 * kp + mi);
    }

    // FULL: the stage's outputs are all the row's.  ALL: the rank is the whole of the KS steps.
    auto work = [&](int st, auto full_const, auto all_const) {
      constexpr bool FULL = decltype(full_const)::value, ALL = decltype(all_const)::value;
      const uint32_t stage = smem_u32(wide_ring) + (st - s0) % S * STAGE_BYTES;
#pragma unroll
      for (int b = 0; b < MOST; ++b) {
        if (b >= blocks || idle) break;
        const int block = first_block + b, n = st * STAGE + block * 32;
        const uint32_t bs = stage + block * (1024 * KS);
        float acc[4][4];
        if constexpr (!ALL) {  // (-0: where the rank is 0, y is left as it is, a -0 too)
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[j][e] = -0.0f;
        }
        auto multiply = [&](int j, int ks, uint32_t b0, uint32_t b1) {
          if (ALL && ks == 0) mma16_first<T>(acc[j], hi[0], b0, b1);
          else mma16<T>(acc[j], hi[ks], b0, b1);
          mma16<T>(acc[j], lo[ks], b0, b1);
        };
        if constexpr (KS == 1) {
          if (ALL || rank > 0) {
#pragma unroll
            for (int j = 0; j < 4; j += 2) {
              uint32_t w[4];
              load_matrices(w, bs + from[0] + j * 64);
              if constexpr (!ALL) w[0] &= keep0, w[1] &= keep1, w[2] &= keep0, w[3] &= keep1;
              multiply(j, 0, w[0], w[1]);
              multiply(j + 1, 0, w[2], w[3]);
            }
          }
        } else {
#pragma unroll
          for (int kp = 0; kp < KS / 2; ++kp) {
            if (!ALL && kp * 32 >= rank) break;
            const bool both = ALL || kp * 32 + 16 < rank;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              uint32_t w[4];
              load_matrices(w, bs + from[kp] + j * (64 * KS));
              if (!ALL && last == 2 * kp) w[0] &= keep0, w[1] &= keep1;
              multiply(j, 2 * kp, w[0], w[1]);
              if (both) {
                if (!ALL && last == 2 * kp + 1) w[2] &= keep0, w[3] &= keep1;
                multiply(j, 2 * kp + 1, w[2], w[3]);
              }
            }
          }
        }
        if constexpr (VEC) {
          const int left = FULL ? 8 : a.N - n - 8 * t;
          const int64_t off = static_cast<int64_t>(n) * ES;
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const float dv[8] = {acc[0][2 * u], acc[0][2 * u + 1], acc[1][2 * u], acc[1][2 * u + 1],
                                 acc[2][2 * u], acc[2][2 * u + 1], acc[3][2 * u], acc[3][2 * u + 1]};
            if (have[u]) v[b][u].add_and_store(out[u] + off, left, dv, back[u]);
          }
        } else {
          float* mine = cross[warp];
          __syncwarp();  // the block before has been read
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int j = 0; j < 4; ++j)
              *reinterpret_cast<float2*>(mine + (g + 8 * u) * PITCH + 8 * t + 2 * j) =
                  make_float2(acc[j][2 * u] * back[u], acc[j][2 * u + 1] * back[u]);
          __syncwarp();
          v[b].add_and_store(a.out, offs[rset][1], n + lane, FULL || n + lane < a.N, rows_here, mine + lane, PITCH);
        }
        if constexpr (FULL) load_block(st + 1, b);
      }
    };
    auto begin = [&](int st) {
      lane_copies_wait<S - 2>();
      __syncthreads();  // the stage is there, and the one before it has been read
      issue(st + S - 1);
    };
    const int whole = min(s1, a.N / STAGE);
#pragma unroll 1
    for (int st = s0; st < whole; ++st) {
      begin(st);
      if (rank == 16 * KS) work(st, std::true_type{}, std::true_type{});
      else work(st, std::true_type{}, std::false_type{});
    }
    if (whole < s1) {  // the row's last stage is a part of one
      begin(s1 - 1);
      work(s1 - 1, std::false_type{}, std::false_type{});
    }
    lane_copies_wait<0>();
  }
  if (!waited) pdl_wait();
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
template <typename T, int RT>
cudaError_t down_setup() {
  const cudaError_t e = cudaFuncSetAttribute(adapter_down_wide_kernel<T, RT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             down_wide_smem(RT));
  if (e != cudaSuccess) return e;
  return cudaFuncSetAttribute(adapter_down_kernel<T, RT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              adapter_down_smem(RT));
}

template <typename T, typename Y, int KS, bool VEC>
cudaError_t up_setup() {
  return cudaFuncSetAttribute(adapter_up_kernel<T, Y, KS, VEC>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              up_warps(KS) * up_warp_bytes(KS));
}

template <typename T, typename Y, int KS, int PIECE>
cudaError_t wide_setup_piece() {
  return cudaFuncSetAttribute(adapter_wide_kernel<T, Y, KS, PIECE>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              kADWideStages * wide_stage_bytes(KS));
}
template <typename T, typename Y, int KS, bool VEC>
cudaError_t wide_setup() {
  cudaError_t e = wide_setup_piece<T, Y, KS, VEC ? 16 : 0>();
  if constexpr (VEC && sizeof(Y) == 2)
    if (e == cudaSuccess) e = wide_setup_piece<T, Y, KS, 8>();
  return e;
}

template <typename T, typename Y, bool VEC>
cudaError_t up_setup_of() {
  cudaError_t e = wide_setup<T, Y, 1, VEC>();
  if (e == cudaSuccess) e = wide_setup<T, Y, 2, VEC>();
  if (e == cudaSuccess) e = wide_setup<T, Y, 4, VEC>();
  if (e == cudaSuccess) e = wide_setup<T, Y, 8, VEC>();
  if (e == cudaSuccess) e = up_setup<T, Y, 1, VEC>();
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

template <typename T, int RT>
cudaError_t launch_down_rt(const AdapterArgs& a, int grid, cudaStream_t stream) {
  if (a.rows > kADOwnPlan)
    return launch_kernel(adapter_down_wide_kernel<T, RT>, dim3(grid, a.splits), dim3(kADThreads),
                         static_cast<size_t>(down_wide_smem(RT)), stream, true, a);
  return launch_kernel(adapter_down_kernel<T, RT>, dim3(grid, a.splits), dim3(kADThreads),
                       static_cast<size_t>(adapter_down_smem(RT)), stream, true, a);
}

template <typename T>
cudaError_t launch_down(const AdapterArgs& a, int grid, cudaStream_t stream) {
  if (a.R <= 16) return launch_down_rt<T, 1>(a, grid, stream);
  if (a.R <= 32) return launch_down_rt<T, 2>(a, grid, stream);
  if (a.R <= 64) return launch_down_rt<T, 4>(a, grid, stream);
  return launch_down_rt<T, 8>(a, grid, stream);
}

template <typename T, typename Y, int KS, bool VEC>
cudaError_t launch_up_ks(const AdapterArgs& a, int64_t max_tiles, int num_sms, cudaStream_t stream) {
  if (a.rows > kADOwnPlan) {
    const int64_t most = static_cast<int64_t>(num_sms) * wide_ctas(KS);
    constexpr int STAGE = kADWideStage;
    const int64_t stages = max_tiles * ((a.N + STAGE - 1) / STAGE);
    const dim3 grid(static_cast<unsigned>(stages < most ? stages : most));
    constexpr size_t smem = kADWideStages * wide_stage_bytes(KS);
    if constexpr (VEC && sizeof(Y) == 2)
      if (a.piece == 8)
        return launch_kernel(adapter_wide_kernel<T, Y, KS, 8>, grid, dim3(kADWideThreads), smem, stream, true, a);
    return launch_kernel(adapter_wide_kernel<T, Y, KS, VEC ? 16 : 0>, grid, dim3(kADWideThreads), smem, stream, true, a);
  }
  constexpr int STEP = kADStep;
  const int64_t max_steps = max_tiles * ((a.N + STEP - 1) / STEP);
  const int64_t most = num_sms;  // one wave
  const int64_t few = (max_steps + up_warps(KS) - 1) / up_warps(KS);
  return launch_kernel(adapter_up_kernel<T, Y, KS, VEC>, dim3(static_cast<unsigned>(few < most ? few : most)),
                       dim3(32 * up_warps(KS)), static_cast<size_t>(up_warps(KS) * up_warp_bytes(KS)), stream, true, a);
}

template <typename T, typename Y, bool VEC>
cudaError_t launch_up_of(const AdapterArgs& a, int64_t max_tiles, int num_sms, cudaStream_t stream) {
  if (a.R <= 16) return launch_up_ks<T, Y, 1, VEC>(a, max_tiles, num_sms, stream);
  if (a.R <= 32) return launch_up_ks<T, Y, 2, VEC>(a, max_tiles, num_sms, stream);
  if (a.R <= 64) return launch_up_ks<T, Y, 4, VEC>(a, max_tiles, num_sms, stream);
  return launch_up_ks<T, Y, 8, VEC>(a, max_tiles, num_sms, stream);
}

template <typename T>
cudaError_t launch_up(const AdapterArgs& a, lmh_dtype out_dtype, bool vec, int64_t max_tiles, int num_sms,
                      cudaStream_t stream) {
  if (out_dtype == LMH_F32)
    return vec ? launch_up_of<T, float, true>(a, max_tiles, num_sms, stream)
               : launch_up_of<T, float, false>(a, max_tiles, num_sms, stream);
  return vec ? launch_up_of<T, T, true>(a, max_tiles, num_sms, stream)
             : launch_up_of<T, T, false>(a, max_tiles, num_sms, stream);
}

// The two types' kernels (adapters_bf16.cu, adapters_f16.cu).
cudaError_t adapters_setup_bf16();
cudaError_t adapters_setup_f16();
cudaError_t launch_down_bf16(const AdapterArgs& a, int grid, cudaStream_t stream);
cudaError_t launch_down_f16(const AdapterArgs& a, int grid, cudaStream_t stream);
cudaError_t launch_up_bf16(const AdapterArgs& a, lmh_dtype out_dtype, bool vec, int64_t max_tiles, int num_sms,
                           cudaStream_t stream);
cudaError_t launch_up_f16(const AdapterArgs& a, lmh_dtype out_dtype, bool vec, int64_t max_tiles, int num_sms,
                          cudaStream_t stream);

}  // namespace lmh
