// q4_project.cuh -- the head projection through a 4-bit table (lmh_project_q4): the kernel
// for up to 16 hidden rows a read of the table, and for more where there are zero points or
// the hidden rows are long (the others: q4_project_wide.cuh); the choice between the two.
// Instantiated per type of the hidden rows in q4_project_*.cu.
//
//   out[n][v] = logit_scale * sum_g scale[v][g] * sum_{h in g} (q[v][h] - zero[v][g]) * x[n][h]
//
// For the batches of a decode step (up to a few dozen rows) the table is the
// traffic: V * H/2 bytes and its scales, read once.  The products run on mma.sync
// m16n8k16 (f16) with 16 table rows as the A operand and 8 hidden rows as the B
// operand, so a single hidden row costs the same instructions as eight.
//
// Measured with cold L2 (2560 x 151936, group 64): 53 us for 1 row, of which the table's
// 207 MB at the copy rate are 30.5, 70 us for 16 rows (80 with zero points), 150 for 32 with
// zero points; 4096 x 128256, group 128 with zero points, 16 rows: 92 us (41 at the copy
// rate), 32 rows in two reads 172 (162 without zero points).  For one row the issue slots are busy 57% and the ALU 43%: what bounds it beside
// the reads is the unpacking.  For 16 and 32 rows it is the latency that the 12 or 8 warps
// whose sums fit in registers cannot cover, and loads that stay in flight only as far as
// the few stages go that the hidden rows leave.
//
// An f16 holds two nibbles' places in its ten mantissa bits: with exponent bits
// for 1024 put in, bits 0..3 make it 1024 + q and bits 4..7 make it 1024 + 16q.  One
// logic operation and one packed f16 operation give an operand of two entries
// q - zero, exact whole numbers: nine operations for a word of eight entries (in bf16,
// with seven bits, every nibble would have to be shifted to the bottom first: eleven).
// - So the hidden rows are held as f16, scaled by a power of two that brings the row's
//   largest finite value into [2^14, 2^15).  That is exact for bf16 and f16 values down
//   to 2^-28 of the row's largest, and off by at most 2^-39 of the largest below: less
//   than the fp32 sums round.
// - A group's sum stays in the MMA's fp32 accumulator and its scale is applied in
//   fp32, so no product of scale and entry is rounded to 16 bits.
// - Measured and dropped: no conversion at all, the nibble as a subnormal f16 (q *
//   2^-24) and the zero points in the accumulator's start.  The MMA aligns products by
//   their operands' exponents, and with the leading zeros of a subnormal in the operand
//   it drops seven bits of every product: errors of 6e-6 of the sum of magnitudes.
//
// - tcgen05 (the other kernel's way) with 16 hidden rows an MMA was measured and dropped for
//   up to 16 rows: 84, 49 and 123 us where this kernel took 53, 33 and 92 (1 row of 2560 and 8
//   of 1024 x 151936, 16 of 4096 x 128256).
//
// Work: a CTA takes tiles of 128 table rows.  Its producer warp streams a tile as
// boxes of 128 rows x 128 bytes (256 entries) into a ring of shared-memory stages
// (TMA, 128-byte swizzle).  A row group of 32 rows has KW consumer warps that take
// its boxes in turn, each a box of 32 rows whole: one read of the hidden rows serves
// two MMA row tiles, and the scales' addresses and the wait are paid once per 256
// entries.  At the end of a tile one of the KW warps, each in its turn, gets the
// others' sums through shared memory, adds them up in a fixed order and writes the
// logits; the others go on to the next tile at once.
// Measured and dropped, where the hidden rows leave few stages (16 rows of 4096 / 32 of
// 2560 without zero points; as it is: 92 / 129 us): pairs of CTAs that share a tile's
// entries, and so have half of the hidden rows each (113 / 147); no producer, the last
// reader of a stage loads its next box (96 / 127, and 2 us more for small calls); boxes of
// 64 bytes a row, for twice the stages (104 / 137); 16 table rows a warp and twice the
// warps (98 / 139).
//
// The order of a block's entries within an MMA is free as long as A and B agree:
// lane c of a row's four lanes takes word c of the block's four words (entries 8c
// .. 8c+7), and pair i of a word is its entries (i, i + 4).  Lane (row, c) reads
// the word at 16-byte chunk (block ^ row % 8) of its row, so a warp's reads touch
// every bank once.  The hidden rows lie in shared memory in MMA order, 16 bytes per
// lane and block.
#pragma once

#include "q4_operands.cuh"
#include "q4_project_wide.cuh"

namespace lmh {

// The shortest ring: a warp's next box must not wrap the ring twice.
constexpr int q4_min_stages(int nt) { return nt == 1 ? 4 : 3; }

// Consumer warps per row group for NT tiles of 8 hidden rows: as many as the
// registers that the sums need allow (96, 128 and 168 a thread).
constexpr int q4_kw(int nt) { return nt == 1 ? 4 : nt == 2 ? 3 : 2; }
constexpr int q4_threads(int nt) { return 32 * (kQ4RowGroups * q4_kw(nt) + 1); }  // one warp is the producer

// Shared memory: [ring][hidden rows][the warps' sums][rows' maxima and
// scales][barriers]; the ring at a 1024-byte boundary.
__host__ __device__ inline size_t q4_hidden_bytes(int boxes, int nt) {
  return static_cast<size_t>(boxes) * kQ4BoxBlocks * nt * 512;
}
constexpr size_t q4_sums_bytes(int nt) { return static_cast<size_t>(kQ4RowGroups) * (q4_kw(nt) - 1) * nt * 1024; }
constexpr size_t kQ4FixedBytes = 1024 + 64 * 4 + (2 * kQ4MaxStages + 1) * 8;

// The constants that take a row's zero point off: 1024 + zero and -(64 + zero), twice.
struct Q4Zero {
  uint32_t low, high;
};
__device__ __forceinline__ Q4Zero q4_zero_bits(uint32_t zero) {
  // in f16, 1024 + z is 0x6400 + z, and -(64 + z) is 0xD400 + 16z
  return Q4Zero{0x64006400u + 0x00010001u * zero, 0xD400D400u + 0x00100010u * zero};
}

// Operand registers of a word's eight entries: pair i is entries (i, i + 4), as q - zero.
__device__ __forceinline__ void q4_pairs(uint32_t w, const Q4Zero& z, uint32_t (&p)[4]) {
#pragma unroll
  for (int i = 0; i < 4; i += 2) {
    const uint32_t v = i ? w >> 8 : w;
    // (written out: as an expression of constants (v & mask) | 0x6400 becomes two operations)
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(p[i]) : "r"(v), "r"(0x000F000Fu), "r"(0x64006400u));
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(p[i + 1]) : "r"(v), "r"(0x00F000F0u), "r"(0x64006400u));
    asm("sub.rn.f16x2 %0, %0, %1;" : "+r"(p[i]) : "r"(z.low));
    asm("fma.rn.f16x2 %0, %0, %1, %2;" : "+r"(p[i + 1]) : "r"(0x2C002C00u), "r"(z.high));  // * 1/16
  }
}

// d += a * b: a 16 x 16 (rows gid and gid + 8 in alternating registers), b 16 x 8
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// d = a * b
__device__ __forceinline__ void mma_f16_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}

// G: entries per group.  NT: tiles of 8 hidden rows per pass (blockIdx.y counts
// passes).  ZP: the table has zero points.
template <typename T, int G, int NT, bool ZP>
__global__ void __launch_bounds__(q4_threads(NT), 1)
    project_q4_kernel(const __grid_constant__ CUtensorMap map, const Q4ProjectArgs a) {
  constexpr int KW = q4_kw(NT);
  constexpr int kConsumers = kQ4RowGroups * KW;
  constexpr int kGroups = kQ4BoxEntries / G;  // of a box: 8, 4 or 2
  constexpr int kLoads = kGroups > 4 ? 2 : 1;  // scales per lane and table row
  extern __shared__ unsigned char smem_raw[];
  unsigned char* ring = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  uint4* xs = reinterpret_cast<uint4*>(ring + a.stages * kQ4StageBytes);         // [block][NT][32 lanes]
  float* sums = reinterpret_cast<float*>(xs + a.slab * kQ4BoxBlocks * NT * 32);  // [group][KW - 1][2 * NT][4][32]
  int* row_max = reinterpret_cast<int*>(sums + kQ4RowGroups * (KW - 1) * 2 * NT * 4 * 32);  // [8 * NT], room for 32
  float* row_scale = reinterpret_cast<float*>(row_max + 32);                                // [8 * NT], room for 32
  uint64_t* full = reinterpret_cast<uint64_t*>(row_scale + 32);
  uint64_t* empty = full + kQ4MaxStages;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(empty + kQ4MaxStages);

  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int boxes = (a.t.H + kQ4BoxEntries - 1) / kQ4BoxEntries;
  const int tiles = (a.t.V + kQ4TileRows - 1) / kQ4TileRows;
  if (threadIdx.x == 0) {
    for (int s = 0; s < a.stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], kQ4RowGroups);  // one warp of every row group reads a stage
    }
    *abort_flag = 0;
    mbar_init_fence();
  }
  __syncthreads();

  if (warp == kConsumers) {
    // ------------------------- producer -------------------------
    if (lane == 0) {
      prefetch_tmap(&map);
      pdl_wait();  // (the kernel before this one may be quantize_q4_kernel, whose table this is)
      int s = 0;
      uint32_t ph = 0;
      bool ok = true;
      int issued = 0;
      for (int tile = blockIdx.x; ok && tile < tiles; tile += gridDim.x)
        for (int b = 0; b < boxes; ++b) {
          if (!wait_or_abort(&empty[s], ph ^ 1u, abort_flag, a.dev_status, a.wait_ns)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(&full[s], kQ4StageBytes);
          tma_load_2d(ring + s * kQ4StageBytes, &map, b * kQ4BoxBytes, tile * kQ4TileRows, &full[s]);
          issued = min(issued + 1, a.stages);
          if (++s == a.stages) {
            s = 0;
            ph ^= 1u;
          }
        }
      // every stage's last load lands before the CTA exits (after an abort nobody else waits for it)
      for (int i = 0; i < issued; ++i) {
        if (--s < 0) {
          s = a.stages - 1;
          ph ^= 1u;
        }
        mbar_wait(&full[s], ph);
      }
    }
    return;
  }

  // ------------------------- consumers -------------------------
  const int gid = lane >> 2, c = lane & 3;
  const int group = warp / KW, kw = warp % KW;
  const int n0 = blockIdx.y * 8 * NT;
  const int groups = a.t.H / G;
  const bool resident = a.slab >= boxes;
  const bool scale32 = a.t.scale_dtype == LMH_F32, scale_bf16 = a.t.scale_dtype == LMH_BF16;
  pdl_wait();
  // (no early launch of the next kernel: it may read the logits ahead of its wait, as logprobs_from_logits does)

  // named barriers: all consumers; per row group, a tile's sums are there, and are read
  // (of even and of odd tiles: the finisher skips the wait at the next tile, and may be
  // at the one after that while the others are still to pass the first)
  constexpr int kAllConsumers = 1, kSumsThere = 2, kSumsRead = kSumsThere + kQ4RowGroups;
  static_assert(kSumsRead + 2 * kQ4RowGroups <= 16, "sixteen named barriers");
  auto hidden_row = [&](int n) -> const T* {
    if (n0 + n >= a.rows) return nullptr;
    const int r = a.row_idx ? a.row_idx[n0 + n] : n0 + n;
    if (r < 0 || r >= a.num_tokens) return nullptr;
    return static_cast<const T*>(a.hidden) + r * a.hidden_stride;
  };
  // A thread's hidden rows are the same all along: item i is (block, nt, lane), and
  // its row is nt * 8 + lane / 4.
  const T* my_hidden[NT];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    my_hidden[nt] = hidden_row(nt * 8 + gid);
    if (!my_hidden[nt] && n0 + nt * 8 + gid < a.rows && warp == 0 && c == 0)
      set_status(a.dev_status, LMH_DS_ROW_IDX_OUT_OF_RANGE);
  }
  // The largest finite value of every row.
  if (threadIdx.x < 8 * NT) row_max[threadIdx.x] = 0;
  named_bar_sync(kAllConsumers, 32 * kConsumers);
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    float m = 0.0f;
    if (my_hidden[nt])
#pragma unroll 5
      for (int h = warp * 32 + c * 8; h < a.t.H; h += 32 * kConsumers) {
        float x[8];
        load_hidden(my_hidden[nt] + h, a.vec, x);
#pragma unroll
        for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(x[e]) < INFINITY ? fabsf(x[e]) : 0.0f);
      }
    atomicMax(&row_max[nt * 8 + gid], __float_as_int(m));  // (not negative: ordered as its bits)
  }
  named_bar_sync(kAllConsumers, 32 * kConsumers);
  float scale1[NT], scale2[NT];  // 2^(14 - exponent), in two exact steps: it may be no fp32 number
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const float m = __int_as_float(row_max[nt * 8 + gid]);
    const int k = 14 - (m > 0.0f ? ilogbf(m) : 0);
    scale1[nt] = pow2(k / 2);
    scale2[nt] = pow2(k - k / 2);
  }
  if (threadIdx.x < 8 * NT) {
    const float m = __int_as_float(row_max[threadIdx.x]);
    row_scale[threadIdx.x] = pow2(m > 0.0f ? ilogbf(m) : 0);
  }

  // Hidden rows n0.. of boxes [b0, b0 + slab) into shared memory, scaled, in MMA
  // order; zeros past the last row and the last entry.
  auto stage = [&](int b0) {
#pragma unroll 5
    for (int blk = warp; blk < a.slab * kQ4BoxBlocks; blk += kConsumers) {
      const int h = (b0 * kQ4BoxBlocks + blk) * 32 + c * 8;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        uint4 y = make_uint4(0, 0, 0, 0);
        if (my_hidden[nt] && h < a.t.H) {
          float x[8];
          load_hidden(my_hidden[nt] + h, a.vec, x);
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] = x[e] * scale1[nt] * scale2[nt];
          y = make_uint4(half2_bits(x[0], x[4]), half2_bits(x[1], x[5]), half2_bits(x[2], x[6]),
                         half2_bits(x[3], x[7]));
        }
        xs[(blk * NT + nt) * 32 + lane] = y;
      }
    }
    named_bar_sync(kAllConsumers, 32 * kConsumers);
  };
  if (resident) stage(0);

  // This warp's boxes are every KW-th of the CTA's sequence.  Their scales (and zero
  // points) are loaded one box ahead, as raw bits, and spread over a table row's four
  // lanes: lane c holds group c % kGroups and, with eight groups a box, group 4 + c.
  int next_tile = blockIdx.x, next_box = kw;
  const char* scale_row[4];
  const unsigned char* zero_row[4];
  const int scale_shift = scale32 ? 2 : 1;
  auto set_rows = [&]() {
    const int v0 = next_tile * kQ4TileRows + group * 32 + gid;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t v = min(v0 + 8 * i, a.t.V - 1);  // rows past V repeat the last one
      scale_row[i] = static_cast<const char*>(a.t.scales) + ((v * a.t.scale_row_stride) << scale_shift);
      if (ZP) zero_row[i] = a.t.zeros + v * a.t.zero_row_stride;
    }
  };
  uint32_t raw_s[4][kLoads], raw_z[4][kLoads];
  auto load_scales = [&]() {
#pragma unroll
    for (int j = 0; j < kLoads; ++j) {
      const int g = min(next_box * kGroups + c % kGroups + 4 * j, groups - 1);
      const int at = g << scale_shift;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        raw_s[i][j] = scale32 ? __ldg(reinterpret_cast<const uint32_t*>(scale_row[i] + at))
                              : __ldg(reinterpret_cast<const uint16_t*>(scale_row[i] + at));
        if (ZP) raw_z[i][j] = __ldg(zero_row[i] + g);
      }
    }
  };
  auto next_scales = [&]() {  // next_box has moved on
    if (next_box >= boxes) {
      do {
        next_box -= boxes;
        next_tile += gridDim.x;
      } while (next_box >= boxes);
      if (next_tile >= tiles) return;
      set_rows();
    }
    if (next_tile < tiles) load_scales();
  };
  set_rows();
  next_scales();

  // Offset within a stage of this lane's word of block 0 in the swizzled rows: bits 4..6
  // hold the 16-byte chunk, block ^ row % 8.
  const uint32_t my_word = (group * 32 + gid) * kQ4BoxBytes + (gid << 4) + c * 4;
  int box = kw;  // this warp's next box within the tile (boxes and more: in a later tile)
  int s = kw;    // its stage
  uint32_t ph = 0;
  bool later_lap = false;
  bool ok = true;
  auto wait = [&](uint64_t* bar, uint32_t parity) {  // (the whole warp agrees)
    return __all_sync(0xffffffffu, mbar_test_wait(bar, parity) ||
                                       wait_or_abort(bar, parity, abort_flag, a.dev_status, a.wait_ns));
  };
  int it = 0;  // tiles done
  int finisher = 0;
  for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x, ++it) {
    float acc[2][NT][4];
#pragma unroll
    for (int mt = 0; mt < 2; ++mt)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[mt][nt][e] = 0.0f;
    for (int b0 = 0; b0 < boxes; b0 += a.slab) {
      if (!resident) {
        named_bar_sync(kAllConsumers, 32 * kConsumers);
        stage(b0);
      }
      const int b1 = min(b0 + a.slab, boxes);
      for (; box < b1; box += KW) {
        float sv[4][kLoads];
        uint32_t zv[4][kLoads];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < kLoads; ++j) {
            sv[i][j] = scale32      ? __uint_as_float(raw_s[i][j])
                       : scale_bf16 ? __uint_as_float(raw_s[i][j] << 16)
                                    : __half2float(__ushort_as_half(static_cast<unsigned short>(raw_s[i][j])));
            if (ZP) zv[i][j] = raw_z[i][j];
          }
        if ((box + 1) * kGroups > groups) {
          // A group past the last one sums to 0, and its scale is 0 too: the last group's may be infinite.
#pragma unroll
          for (int j = 0; j < kLoads; ++j)
            if (box * kGroups + c % kGroups + 4 * j >= groups)
#pragma unroll
              for (int i = 0; i < 4; ++i) sv[i][j] = 0.0f;
        }
        next_box += KW;
        next_scales();
        // A stage's last box was another warp's where the ring is no multiple of KW: that one
        // has to be over first, or a wait for this one's parity would take the one before
        // the last for it.  (All row groups have left a box before the next is loaded.)
        if (ok && later_lap) ok = wait(&empty[s], ph ^ 1u);
        if (ok) ok = wait(&full[s], ph);
        if (ok) {
          const uint32_t rows = my_word + s * kQ4StageBytes;
          const uint4* x = xs + (box - b0) * kQ4BoxBlocks * NT * 32 + lane;
#pragma unroll
          for (int g = 0; g < kGroups; ++g) {
            float d[2][NT][4];
            Q4Zero zero[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
              zero[i] =
                  q4_zero_bits(ZP ? (__shfl_sync(0xffffffffu, zv[i][g / 4], (lane & 28) | (g & 3)) & 15u) : 8u);
#pragma unroll
            for (int j = 0; j < G / 32; ++j) {
              const int blk = g * (G / 32) + j;
              const unsigned char* w0 = ring + (rows ^ (blk << 4));
              uint32_t w[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) w[i] = *reinterpret_cast<const uint32_t*>(w0 + i * 8 * kQ4BoxBytes);
              uint4 b[NT];
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) b[nt] = x[(blk * NT + nt) * 32];
#pragma unroll
              for (int mt = 0; mt < 2; ++mt) {
                uint32_t fa[4], fb[4];
                q4_pairs(w[2 * mt], zero[2 * mt], fa);
                q4_pairs(w[2 * mt + 1], zero[2 * mt + 1], fb);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                  if (j == 0)
                    mma_f16_first(d[mt][nt], fa[0], fb[0], fa[1], fb[1], b[nt].x, b[nt].y);
                  else
                    mma_f16(d[mt][nt], fa[0], fb[0], fa[1], fb[1], b[nt].x, b[nt].y);
                  mma_f16(d[mt][nt], fa[2], fb[2], fa[3], fb[3], b[nt].z, b[nt].w);
                }
              }
            }
#pragma unroll
            for (int mt = 0; mt < 2; ++mt) {
              const float sa = __shfl_sync(0xffffffffu, sv[2 * mt][g / 4], (lane & 28) | (g & 3));
              const float sb = __shfl_sync(0xffffffffu, sv[2 * mt + 1][g / 4], (lane & 28) | (g & 3));
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[mt][nt][e] = fmaf(e < 2 ? sa : sb, d[mt][nt][e], acc[mt][nt][e]);
            }
          }
          // The stage is free once every lane's words are in registers.  An arrival under
          // `lane == 0` after __syncwarp() was seen to overtake the last block's loads, so
          // it hangs on sums that need them: either lane's arrival does.
          const bool none =
              __all_sync(0xffffffffu, __float_as_uint(acc[0][0][0] + acc[1][0][0]) != 0xFFFFFFFEu);
          if (lane == (none ? 0 : 1)) mbar_arrive(&empty[s]);
        }
        s += KW;
        if (s >= a.stages) {
          s -= a.stages;
          ph ^= 1u;
          later_lap = true;
        }
      }
    }
    box -= boxes;

    // The tile's sums: a warp that does not finish it leaves its own and goes on.  Every
    // warp passes these barriers at every tile, after an abort too.
    float* parts = sums + group * (KW - 1) * 2 * NT * 4 * 32 + lane;
    const int last_finisher = finisher == 0 ? KW - 1 : finisher - 1;
    __syncwarp();
    if (it > 0 && kw != last_finisher) named_bar_sync(kSumsRead + ((it - 1) & 1) * kQ4RowGroups + group, 32 * KW);
    if (kw != finisher) {
      float* mine = parts + (kw < finisher ? kw : kw - 1) * 2 * NT * 4 * 32;
#pragma unroll
      for (int mt = 0; mt < 2; ++mt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) mine[((mt * NT + nt) * 4 + e) * 32] = acc[mt][nt][e];
      __syncwarp();
      named_bar_arrive(kSumsThere + group, 32 * KW);
    } else {
      named_bar_sync(kSumsThere + group, 32 * KW);
#pragma unroll
      for (int w = 0; w < KW - 1; ++w)
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[mt][nt][e] += parts[((w * 2 * NT + mt * NT + nt) * 4 + e) * 32];
      if (tile + static_cast<int>(gridDim.x) < tiles) {
        __syncwarp();
        named_bar_arrive(kSumsRead + (it & 1) * kQ4RowGroups + group, 32 * KW);
      }
      if (ok) {
        const int v0 = tile * kQ4TileRows + group * 32 + gid;
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              // lane (gid, c) holds table rows gid and gid + 8 of hidden rows 2c and 2c + 1
              const int n = n0 + nt * 8 + 2 * c + (e & 1);
              const int v = v0 + mt * 16 + 8 * (e >> 1);
              if (n < a.rows && v < a.t.V) {
                // the sums are of x * 2^(14 - exponent)
                const float y = acc[mt][nt][e] * 6.103515625e-5f * row_scale[nt * 8 + 2 * c + (e & 1)] * a.logit_scale;
                if (a.out_f32)
                  static_cast<float*>(a.out)[n * a.out_stride + v] = y;
                else
                  static_cast<T*>(a.out)[n * a.out_stride + v] = static_cast<T>(y);
              }
            }
      }
    }
    if (++finisher == KW) finisher = 0;
  }
}

template <typename T, int G, int NT, bool ZP>
cudaError_t q4_launch_one(Q4ProjectArgs a, int num_sms, cudaStream_t stream) {
  const int boxes = (a.t.H + kQ4BoxEntries - 1) / kQ4BoxEntries;
  const int tiles = (a.t.V + kQ4TileRows - 1) / kQ4TileRows;
  const size_t fixed = kQ4FixedBytes + q4_sums_bytes(NT);
  // All the hidden rows in shared memory with the shortest ring, or as many boxes of
  // them as fit (restaged as a tile goes on).
  const size_t room = kQ4SmemMax - fixed - q4_min_stages(NT) * kQ4StageBytes;
  const int fit = static_cast<int>(room / q4_hidden_bytes(1, NT));
  a.slab = boxes < fit ? boxes : fit;
  a.stages = static_cast<int>((kQ4SmemMax - fixed - q4_hidden_bytes(a.slab, NT)) / kQ4StageBytes);
  if (a.stages > kQ4MaxStages) a.stages = kQ4MaxStages;
  const size_t smem = fixed + q4_hidden_bytes(a.slab, NT) + static_cast<size_t>(a.stages) * kQ4StageBytes;
  CUtensorMap map;
  cudaError_t e = make_tensor_map_2d(&map, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.t.packed, static_cast<uint64_t>(a.t.H / 2),
                                     static_cast<uint64_t>(a.t.V), static_cast<uint64_t>(a.t.packed_row_bytes),
                                     kQ4BoxBytes, kQ4TileRows);
  if (e != cudaSuccess) return e;
  const int passes = (a.rows + 8 * NT - 1) / (8 * NT);
  const int grid = tiles < num_sms ? tiles : num_sms;
  return launch_kernel(project_q4_kernel<T, G, NT, ZP>, dim3(grid, passes), dim3(q4_threads(NT)), smem, stream, true, map,
                       a);
}

// Hidden rows per pass: 8, 16 or 32, the fewest passes whose rows stay in shared
// memory (a second pass reads the table again; restaging the hidden rows at every
// tile reads them again from L2, and stops the tile for it).  32 without zero points
// are the other kernel's: 98 us for 32 rows of 2560 x 151936 where four tiles here took 129.
template <typename T, int G, bool ZP>
cudaError_t q4_launch_rows(const Q4ProjectArgs& a, int num_sms, cudaStream_t stream) {
  const int boxes = (a.t.H + kQ4BoxEntries - 1) / kQ4BoxEntries;
  auto fits = [&](int nt) {
    return kQ4FixedBytes + q4_sums_bytes(nt) + q4_hidden_bytes(boxes, nt) + q4_min_stages(nt) * kQ4StageBytes <= kQ4SmemMax;
  };
  if constexpr (ZP) {
    if (a.rows > 16 && fits(4)) return q4_launch_one<T, G, 4, ZP>(a, num_sms, stream);
  } else {
    if (a.rows > 16 && q4_wide_fits(a.t.H)) return q4_wide_launch<T, G>(a, num_sms, stream);
  }
  if (a.rows > 8 && fits(2)) return q4_launch_one<T, G, 2, ZP>(a, num_sms, stream);
  return q4_launch_one<T, G, 1, ZP>(a, num_sms, stream);
}

template <typename T>
cudaError_t q4_launch(const Q4ProjectArgs& a, int group, int num_sms, cudaStream_t stream) {
  const bool zp = a.t.zeros != nullptr;
  if (group == 32)
    return zp ? q4_launch_rows<T, 32, true>(a, num_sms, stream) : q4_launch_rows<T, 32, false>(a, num_sms, stream);
  if (group == 64)
    return zp ? q4_launch_rows<T, 64, true>(a, num_sms, stream) : q4_launch_rows<T, 64, false>(a, num_sms, stream);
  return zp ? q4_launch_rows<T, 128, true>(a, num_sms, stream) : q4_launch_rows<T, 128, false>(a, num_sms, stream);
}

template <typename T, int G, int NT, bool ZP>
cudaError_t q4_attr() {
  return cudaFuncSetAttribute(project_q4_kernel<T, G, NT, ZP>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              static_cast<int>(kQ4SmemMax));
}
template <typename T, int G>
cudaError_t q4_attr_group() {
  cudaError_t e = q4_attr<T, G, 1, false>();
  if (e == cudaSuccess) e = q4_attr<T, G, 1, true>();
  if (e == cudaSuccess) e = q4_attr<T, G, 2, false>();
  if (e == cudaSuccess) e = q4_attr<T, G, 2, true>();
  if (e == cudaSuccess) e = q4_attr<T, G, 4, true>();
  if (e == cudaSuccess) e = q4_wide_attr<T, G>();
  return e;
}
template <typename T>
cudaError_t q4_attr_type() {
  cudaError_t e = q4_attr_group<T, 32>();
  if (e == cudaSuccess) e = q4_attr_group<T, 64>();
  if (e == cudaSuccess) e = q4_attr_group<T, 128>();
  return e;
}

// One type's instances (q4_project_bf16.cu, q4_project_f16.cu).
cudaError_t q4_setup_bf16();
cudaError_t q4_setup_f16();
cudaError_t q4_launch_bf16(const Q4ProjectArgs& a, int group, int num_sms, cudaStream_t stream);
cudaError_t q4_launch_f16(const Q4ProjectArgs& a, int group, int num_sms, cudaStream_t stream);

}  // namespace lmh
