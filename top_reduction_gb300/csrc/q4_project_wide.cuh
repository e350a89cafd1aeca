// q4_project_wide.cuh -- lmh_project_q4 for 17 to 32 hidden rows a pass, without zero
// points: the products on tcgen05.
//
// A CTA takes tiles of 128 table rows, the M of an MMA, with 32 hidden rows as its N.
//
// - The producer streams a tile as boxes of 128 rows x 128 bytes (256 entries) into a
//   ring in shared memory (TMA, 128-byte swizzle).
// - Eight unpacking warps, a thread per table row (and half of a box), make f16
//   entries q - 8 and put them into tensor memory, where an MMA takes its A operand
//   from: in shared memory they would be four times the packed bytes, written and read
//   again, more than it can move in the time that HBM gives.
// - Two threads issue tcgen05.mma (kind::f16) for every other stage of 128 entries: A from
//   tensor memory, B (the hidden rows) resident in shared memory, one fp32 accumulator
//   per group of entries.  (MMAs this narrow cost their issuer more than the tensor
//   cores: one thread took 1.5 times as long.)  A stage's MMAs end on one barrier, which
//   frees its A operand and hands over its accumulators.
// - Eight warps, a thread per table row and half of the hidden rows, take a group's
//   accumulator from tensor memory, multiply it by the row's scale and add it up in
//   registers: no product of scale and entry is rounded to 16 bits, and a thread needs
//   its own row's scales alone.  At the end of a tile a warp writes 32 neighbouring
//   logits of its hidden rows.
//
// Unpacking and the hidden rows' form are those of project_q4_kernel, whose two entries
// of a pair have one constant here: the zero point is 8.  (Tables with zero points run on
// project_q4_kernel.  An unpacking thread owns one table row, so it could subtract the row's
// own zero points as that kernel does; such a form has not been built.)
//
// Measured with cold L2: 98 us for 32 rows of 2560 x 151936, group 64 (226 MB in and out: 33
// us at the copy rate), where mma.sync took 129; 94 for 17 rows, 59 for 24 of 1024, group 32;
// 174 for 33 rows, 186 for 64 and 709 for 256, which read and unpack the table once per 32.
// The unpacking and the sums' warps hold the issue slots 53% busy, the tensor pipe is 11%
// busy: what is left is the stages' hand-over between the roles, four times per 128 entries,
// with a ring of three stages beside the hidden rows.
#pragma once

#include "q4_operands.cuh"
#include "tcgen05.cuh"

namespace lmh {

constexpr int kWideRows = 32;
constexpr int kWideMinStages = 3;

// warps: 0 producer, 1 and 2 MMA, 4..11 unpacking, 12..19 sums (a warp reaches the lane
// quarter of tensor memory that its number mod 4 says)
constexpr int kWideThreads = 640;
constexpr int kQ4Issuers = 2;
constexpr int kQ4FirstUnpack = 4, kQ4Unpack = 8, kQ4FirstSum = 12, kQ4Sum = 8;

// tensor memory: four A stages of 128 entries (64 columns), then the accumulators of four
// stages' groups, or of two where four have no room
constexpr int kQ4AStages = 4, kQ4AEntries = 128, kQ4ACols = 64;
constexpr int kQ4AccCol = kQ4AStages * kQ4ACols;
constexpr int q4_bank_cols(int group) { return kQ4AEntries / group * kWideRows; }
constexpr int q4_banks(int group) { return 4 * q4_bank_cols(group) <= 256 ? 4 : 2; }

// Shared memory: [ring][hidden rows][row offsets, maxima, scales][barriers]; ring and
// hidden rows at 1024-byte boundaries.
__host__ __device__ inline size_t q4_wide_hidden_bytes(int boxes) {
  return static_cast<size_t>(boxes) * kQ4BoxEntries * kWideRows * 2;
}
constexpr int kWideBarriers = 2 * kQ4MaxStages + 3 * kQ4AStages + 1 + kQ4Issuers;
constexpr size_t kWideFixedBytes = 1024 + kWideRows * 16 + (kWideBarriers + 1) * 8;

// Operand registers of a word's eight entries: pair i is entries (i, i + 4), as q - 8.
__device__ __forceinline__ void q4_wide_pairs(uint32_t w, uint32_t* p) {
#pragma unroll
  for (int i = 0; i < 4; i += 2) {
    const uint32_t v = i ? w >> 8 : w;
    // (written out: as an expression of constants (v & mask) | 0x6400 becomes two operations)
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(p[i]) : "r"(v), "r"(0x000F000Fu), "r"(0x64006400u));
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(p[i + 1]) : "r"(v), "r"(0x00F000F0u), "r"(0x64006400u));
    asm("sub.rn.f16x2 %0, %0, %1;" : "+r"(p[i]) : "r"(0x64086408u));                                  // - 1032
    asm("fma.rn.f16x2 %0, %0, %1, %2;" : "+r"(p[i + 1]) : "r"(0x2C002C00u), "r"(0xD480D480u));  // / 16 - 72
  }
}

// 32 columns of this thread's tensor-memory lane.  Warp-collective.
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};" ::
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
        "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]),
        "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]),
        "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31]),
        "r"(taddr)
      : "memory");
}

// 16 columns of this thread's tensor-memory lane (the wait in the same statement, so that
// no use of the registers comes before it).  Warp-collective.
__device__ __forceinline__ void tmem_ld(uint32_t taddr, float (&v)[16]) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}

__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// d[128 x N] (+)= a[128 x 16] (tensor memory) * b[N x 16] (shared memory), f16 to fp32
__device__ __forceinline__ void umma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t accumulate,
                                            uint32_t idesc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// G: entries per group.  blockIdx.y counts passes of 32 hidden rows.
template <typename T, int G>
__global__ void __launch_bounds__(kWideThreads, 1)
    project_q4_wide_kernel(const __grid_constant__ CUtensorMap map, const Q4ProjectArgs a) {
  extern __shared__ unsigned char smem_raw[];
  unsigned char* ring = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  unsigned char* xs = ring + a.stages * kQ4StageBytes;  // [block of 64 entries][kWideRows rows of 128 bytes, swizzled]
  const int boxes = (a.t.H + kQ4BoxEntries - 1) / kQ4BoxEntries;
  const int groups = a.t.H / G;
  int64_t* row_off = reinterpret_cast<int64_t*>(xs + q4_wide_hidden_bytes(boxes));  // elements; -1: no such row
  float* row_max = reinterpret_cast<float*>(row_off + kWideRows);
  float* row_scale = row_max + kWideRows;  // 2^(exponent of row_max)
  uint64_t* full = reinterpret_cast<uint64_t*>(row_scale + kWideRows);
  uint64_t* empty = full + kQ4MaxStages;
  uint64_t* a_full = empty + kQ4MaxStages;
  uint64_t* stage_done = a_full + kQ4AStages;  // a stage's MMAs
  uint64_t* d_empty = stage_done + kQ4AStages;
  uint64_t* hidden_ready = d_empty + kQ4AStages;  // the hidden rows are there
  uint64_t* mma_drain = hidden_ready + 1;         // [issuer]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_drain + kQ4Issuers);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int tiles = (a.t.V + kQ4TileRows - 1) / kQ4TileRows;
  const int n0 = blockIdx.y * kWideRows;
  if (threadIdx.x == 0) {
    for (int s = 0; s < a.stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], kQ4Unpack);
    }
    for (int s = 0; s < kQ4AStages; ++s) {
      mbar_init(&a_full[s], 4);
      mbar_init(&stage_done[s], 1);
      mbar_init(&d_empty[s], kQ4Sum);
    }
    mbar_init(hidden_ready, 32 * kQ4Unpack);
    for (int i = 0; i < kQ4Issuers; ++i) mbar_init(&mma_drain[i], 1);
    *abort_flag = 0;
    mbar_init_fence();
  }
  if (warp == 1) tmem_alloc_all(tmem_slot);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  constexpr int kBanks = q4_banks(G), kBankCols = q4_bank_cols(G), kPerStage = kQ4AEntries / G;

  // A wait that the whole warp agrees on.
  auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
    return __all_sync(0xffffffffu, mbar_test_wait(bar, parity) ||
                                       wait_or_abort(bar, parity, abort_flag, a.dev_status, a.wait_ns));
  };

  if (warp == 0) {
    // ------------------------- producer -------------------------
    if (lane == 0) {
      prefetch_tmap(&map);
      pdl_wait();  // (the kernel before this one may be quantize_q4_kernel, whose table this is)
      int s = 0, issued = 0;
      uint32_t ph = 0;
      bool ok = true;
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
  } else if (warp <= kQ4Issuers) {
    // ------------------------- MMA issue -------------------------
    if (lane == 0) {
      constexpr uint32_t kIdesc = (1u << 4)                                          // D: f32; A, B: f16 (0)
                                  | (static_cast<uint32_t>(kWideRows >> 3) << 17)    // N / 8
                                  | (static_cast<uint32_t>(kQ4TileRows >> 4) << 24);  // M / 16
      constexpr int kSteps = G / 16;  // MMAs per group
      const int me = warp - 1;
      // What can be is worked out beforehand, and a stage's MMAs are written out.
      const uint64_t b_desc = sw128_kmajor_desc(smem_u32(xs));  // + bytes / 16
      auto wait1 = [&](uint64_t* bar, uint32_t parity) {
        return mbar_test_wait(bar, parity) || wait_or_abort(bar, parity, abort_flag, a.dev_status, a.wait_ns);
      };
      bool ok = wait1(hidden_ready, 0);
      uint32_t r = me;  // stage, of those of all tiles
      for (int tile = blockIdx.x; ok && tile < tiles; tile += gridDim.x) {
        for (int at = me; at < 2 * boxes; at += kQ4Issuers, r += kQ4Issuers) {
          ok = wait1(&a_full[r % kQ4AStages], (r / kQ4AStages) & 1u) &&
               wait1(&d_empty[r % kBanks], ((r / kBanks) & 1u) ^ 1u);
          if (!ok) break;
          tc_fence_after();
          const uint64_t desc = b_desc + static_cast<uint32_t>(at) * (kQ4AEntries / 64 * (kWideRows * 128 / 16));
          const uint32_t a_tmem = tmem + (r % kQ4AStages) * kQ4ACols;
          const uint32_t d_tmem = tmem + kQ4AccCol + (r % kBanks) * kBankCols;
#pragma unroll
          for (int k = 0; k < kQ4AEntries / 16; ++k) {
            if (k % kSteps == 0 && at * kQ4AEntries + 16 * k >= a.t.H) break;  // (no group past the last)
            umma_f16_ts(d_tmem + (k / kSteps) * kWideRows, a_tmem + 8 * k,
                        desc + (k / 4) * (kWideRows * 128 / 16) + (k % 4) * 2, k % kSteps != 0, kIdesc);
          }
          umma_commit(&stage_done[r % kQ4AStages]);
        }
      }
      // every MMA that was issued is done before the tensor memory is given back
      umma_commit(&mma_drain[me]);
      mbar_wait(&mma_drain[me], 0);
    }
  } else if (warp >= kQ4FirstUnpack && warp < kQ4FirstUnpack + kQ4Unpack) {
    // ------------------------- unpacking -------------------------
    const int uw = warp - kQ4FirstUnpack, quarter = warp & 3, half = uw >> 2;
    pdl_wait();  // (no early launch of the next kernel: it may read the logits ahead of its wait)
    // The hidden rows: where they are and their largest finite values (a warp per row).
    for (int n = uw; n < kWideRows; n += kQ4Unpack) {
      int64_t off = -1;
      if (n0 + n < a.rows) {
        const int row = a.row_idx ? a.row_idx[n0 + n] : n0 + n;
        if (row >= 0 && row < a.num_tokens)
          off = row * a.hidden_stride;
        else if (lane == 0)
          set_status(a.dev_status, LMH_DS_ROW_IDX_OUT_OF_RANGE);
      }
      const T* src = static_cast<const T*>(a.hidden) + off;
      float m = 0.0f;
      if (off >= 0)
#pragma unroll 5
        for (int h = lane * 8; h < a.t.H; h += 256) {
          float x[8];
          load_hidden(src + h, a.vec, x);
#pragma unroll
          for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(x[e]) < INFINITY ? fabsf(x[e]) : 0.0f);
        }
      m = warp_max(m);
      const int exponent = m > 0.0f ? ilogbf(m) : 0;
      if (lane == 0) {
        row_off[n] = off;
        row_max[n] = m;
        row_scale[n] = pow2(exponent);
      }
    }
    named_bar_sync(1, 32 * kQ4Unpack);

    // The hidden rows into shared memory, scaled, zeros past the last row and the last
    // entry.  Pair order within eight entries as in q4_wide_pairs().
    const int items = boxes * (kQ4BoxEntries / 8) * kWideRows;
#pragma unroll 4
    for (int i = uw * 32 + lane; i < items; i += 32 * kQ4Unpack) {
      const int chunk = i & 7, n = (i >> 3) % kWideRows, block = (i >> 3) / kWideRows;
      const int h = block * 64 + chunk * 8;
      uint4 y = make_uint4(0, 0, 0, 0);
      if (row_off[n] >= 0 && h < a.t.H) {
        float x[8];
        load_hidden(static_cast<const T*>(a.hidden) + row_off[n] + h, a.vec, x);
        // 2^(14 - exponent), in two exact steps: it may be no fp32 number
        const int k = 14 - (row_max[n] > 0.0f ? ilogbf(row_max[n]) : 0);
        const float f1 = pow2(k / 2), f2 = pow2(k - k / 2);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = x[e] * f1 * f2;
        y = make_uint4(half2_bits(x[0], x[4]), half2_bits(x[1], x[5]), half2_bits(x[2], x[6]),
                       half2_bits(x[3], x[7]));
      }
      *reinterpret_cast<uint4*>(xs + (block * kWideRows + n) * 128 + ((chunk ^ (n & 7)) << 4)) = y;
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the MMAs read them
    mbar_arrive(hidden_ready);

    const uint32_t lane_base = tmem + (static_cast<uint32_t>(quarter) << 21);  // lane 32 * quarter
    // byte offset in a box of this row's 16-byte chunk `half * 4`, swizzled; ^ (j << 4) for the next ones
    const uint32_t my_row = (quarter * 32 + lane) * kQ4BoxBytes + (((half * 4) ^ (lane & 7)) << 4);
    int s = 0;
    uint32_t ph = 0, r0 = 0;  // r0: A stages before this tile
    bool ok = true;
    for (int tile = blockIdx.x; ok && tile < tiles; tile += gridDim.x) {
      for (int b = 0; ok && b < boxes; ++b) {
        ok = wait(&full[s], ph);
        if (!ok) break;
        // A half has every other stage: where the last box has no second half, its stage is
        // handed on empty.  (Were it left out, the halves would change stages from tile to
        // tile, and a wait could take a phase of two laps ago for the one before.)
        const uint32_t r = r0 + 2 * b + half;
        ok = wait(&stage_done[r % kQ4AStages], ((r / kQ4AStages) & 1u) ^ 1u);
        if (!ok) break;
        if (b * kQ4BoxEntries + half * kQ4AEntries < a.t.H) {
          const unsigned char* row = ring + s * kQ4StageBytes;
          tc_fence_after();
          const uint32_t to = lane_base + (r % kQ4AStages) * kQ4ACols;
#pragma unroll
          for (int j = 0; j < 4; j += 2) {
            const uint4 w = *reinterpret_cast<const uint4*>(row + (my_row ^ (j << 4)));
            const uint4 x = *reinterpret_cast<const uint4*>(row + (my_row ^ ((j + 1) << 4)));
            uint32_t p[32];
            q4_wide_pairs(w.x, p);
            q4_wide_pairs(w.y, p + 4);
            q4_wide_pairs(w.z, p + 8);
            q4_wide_pairs(w.w, p + 12);
            q4_wide_pairs(x.x, p + 16);
            q4_wide_pairs(x.y, p + 20);
            q4_wide_pairs(x.z, p + 24);
            q4_wide_pairs(x.w, p + 28);
            tmem_st32(to + 16 * j, p);
          }
          tmem_st_wait();
          tc_fence_before();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&a_full[r % kQ4AStages]);
        // (behind the wait for the stores: the words that they were made of have been read)
        if (lane == 0) mbar_arrive(&empty[s]);
        if (++s == a.stages) {
          s = 0;
          ph ^= 1u;
        }
      }
      r0 += 2 * boxes;
    }
  } else if (warp >= kQ4FirstSum) {
    // ------------------------- sums -------------------------
    const int quarter = warp & 3, row = quarter * 32 + lane;
    constexpr int kMine = kWideRows / 2;  // hidden rows n1 .. n1 + kMine - 1 of the pass
    const int n1 = (warp - kQ4FirstSum) / 4 * kMine;
    pdl_wait();
    const bool scale32 = a.t.scale_dtype == LMH_F32, scale_bf16 = a.t.scale_dtype == LMH_BF16;
    // Eight groups' scales of this thread's row, as raw bits, loaded eight groups ahead.
    uint32_t raw[8];
    auto load_scales = [&](int tile, int g0) {
      const int64_t v = min(tile * kQ4TileRows + row, a.t.V - 1);  // (rows past V repeat the last one)
      const int64_t at = v * a.t.scale_row_stride + g0;
      if (a.scale_vec && g0 + 8 <= groups) {
        const uint4* p = reinterpret_cast<const uint4*>(static_cast<const char*>(a.t.scales) + at * (scale32 ? 4 : 2));
        const uint4 x = __ldg(p), y = scale32 ? __ldg(p + 1) : make_uint4(0, 0, 0, 0);
        raw[0] = x.x, raw[1] = x.y, raw[2] = x.z, raw[3] = x.w;
        raw[4] = y.x, raw[5] = y.y, raw[6] = y.z, raw[7] = y.w;
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int64_t to = at + min(i, groups - 1 - g0);
          raw[i] = scale32 ? __ldg(static_cast<const uint32_t*>(a.t.scales) + to)
                           : __ldg(static_cast<const uint16_t*>(a.t.scales) + to);
        }
      }
    };
    const uint32_t d_base = tmem + (static_cast<uint32_t>(quarter) << 21) + kQ4AccCol + n1;
    uint32_t r = 0;  // stages done
    if (static_cast<int>(blockIdx.x) < tiles) load_scales(blockIdx.x, 0);
    bool ok = wait(hidden_ready, 0);  // (row_scale is there, too)
    for (int tile = blockIdx.x; ok && tile < tiles; tile += gridDim.x) {
      float acc[kMine];
#pragma unroll
      for (int n = 0; n < kMine; ++n) acc[n] = 0.0f;
#pragma unroll 1
      for (int g0 = 0; ok && g0 < groups; g0 += 8) {
        const bool packed = a.scale_vec && !scale32 && g0 + 8 <= groups;
        float sc[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t bits = packed ? (i & 1 ? raw[i / 2] >> 16 : raw[i / 2] & 0xFFFFu) : raw[i];
          sc[i] = scale32      ? __uint_as_float(bits)
                  : scale_bf16 ? __uint_as_float(bits << 16)
                               : __half2float(__ushort_as_half(static_cast<unsigned short>(bits)));
        }
        const bool last = g0 + 8 >= groups;
        if (!last)
          load_scales(tile, g0 + 8);
        else if (tile + static_cast<int>(gridDim.x) < tiles)
          load_scales(tile + gridDim.x, 0);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (!ok || g0 + i >= groups) break;
          if (i % kPerStage == 0) {
            ok = wait(&stage_done[r % kQ4AStages], (r / kQ4AStages) & 1u);
            if (!ok) break;
            tc_fence_after();
          }
          float d[kMine];
          tmem_ld(d_base + (r % kBanks) * kBankCols + (i % kPerStage) * kWideRows, d);
          if (i % kPerStage == kPerStage - 1 || g0 + i == groups - 1) {  // the stage's last group
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&d_empty[r % kBanks]);
            ++r;
          }
#pragma unroll
          for (int n = 0; n < kMine; ++n) acc[n] = fmaf(sc[i], d[n], acc[n]);
        }
      }
      if (ok && (a.t.H + kQ4AEntries - 1) / kQ4AEntries % 2 != 0) {  // (the stage that was handed on empty)
        ok = wait(&stage_done[r % kQ4AStages], (r / kQ4AStages) & 1u);
        __syncwarp();
        if (lane == 0 && ok) mbar_arrive(&d_empty[r % kBanks]);
        ++r;
      }
      const int v = tile * kQ4TileRows + row;
      if (ok && v < a.t.V) {
#pragma unroll
        for (int n = 0; n < kMine; ++n) {
          if (n0 + n1 + n >= a.rows) break;
          // the sums are of x * 2^(14 - exponent)
          const float y = acc[n] * 6.103515625e-5f * row_scale[n1 + n] * a.logit_scale;
          const int64_t to = (n0 + n1 + n) * a.out_stride + v;
          if (a.out_f32)
            static_cast<float*>(a.out)[to] = y;
          else
            static_cast<T*>(a.out)[to] = static_cast<T>(y);
        }
      }
    }
  }

  __syncwarp();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_free_all(tmem);
  }
}

// Whether the hidden rows stay in shared memory beside the shortest ring.
inline bool q4_wide_fits(int H) {
  const int boxes = (H + kQ4BoxEntries - 1) / kQ4BoxEntries;
  return kWideFixedBytes + q4_wide_hidden_bytes(boxes) + kWideMinStages * kQ4StageBytes <= kQ4SmemMax;
}

template <typename T, int G>
cudaError_t q4_wide_launch(Q4ProjectArgs a, int num_sms, cudaStream_t stream) {
  const int boxes = (a.t.H + kQ4BoxEntries - 1) / kQ4BoxEntries;
  const int tiles = (a.t.V + kQ4TileRows - 1) / kQ4TileRows;
  const size_t fixed = kWideFixedBytes + q4_wide_hidden_bytes(boxes);
  a.stages = static_cast<int>((kQ4SmemMax - fixed) / kQ4StageBytes);
  if (a.stages > kQ4MaxStages) a.stages = kQ4MaxStages;
  const size_t smem = fixed + static_cast<size_t>(a.stages) * kQ4StageBytes;
  const size_t sb = a.t.scale_dtype == LMH_F32 ? 4 : 2;
  a.scale_vec = reinterpret_cast<uintptr_t>(a.t.scales) % 16 == 0 && a.t.scale_row_stride * sb % 16 == 0;
  CUtensorMap map;
  cudaError_t e = make_tensor_map_2d(&map, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.t.packed, static_cast<uint64_t>(a.t.H / 2),
                                     static_cast<uint64_t>(a.t.V), static_cast<uint64_t>(a.t.packed_row_bytes),
                                     kQ4BoxBytes, kQ4TileRows);
  if (e != cudaSuccess) return e;
  const int passes = (a.rows + kWideRows - 1) / kWideRows;
  return launch_kernel(project_q4_wide_kernel<T, G>, dim3(tiles < num_sms ? tiles : num_sms, passes),
                       dim3(kWideThreads), smem, stream, true, map, a);
}

template <typename T, int G>
cudaError_t q4_wide_attr() {
  return cudaFuncSetAttribute(project_q4_wide_kernel<T, G>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              static_cast<int>(kQ4SmemMax));
}

}  // namespace lmh
