// reorder_rows.cu -- the states of a batch follow the rows they come from (lmh_reorder_rows).
//
// Row r of every state gets what row parents[r] held, within groups of `beams` rows.  All rows of a group
// that others need are read into shared memory, a slice at a time, before any is written: in place, a row
// may be both a source and overwritten.  Rows that stay are neither read nor written; a row that several
// take is read once.
//
//   * reorder_bulk_kernel, for states whose rows and chunks begin on 16-byte boundaries: one warp a CTA, bulk
//     copies into a ring of stages and from there to the rows that take them; no byte passes a register.  Bound
//     by the bytes moved: caches of four layers (420 MB read, 420 written) take 153 us, 0.81 of the copy rate.
//   * reorder_rows_kernel, for the others and for calls that move little: plain loads and stores.  A step's
//     histories and block tables (256 rows, 4.9 MB read and written): 4.5 us in a graph, latency.
//     The caches take 273 us where their rows align to 8 bytes, 346 to 4, 501 to 2.
#include "device_common.cuh"
#include "lmh_internal.h"

namespace lmh {

constexpr int kRRThreads = 256;
constexpr int kRRStates = 24;       // states of one launch
constexpr int kRRSmem = 64 * 1024;  // staging
constexpr int kRRSliceMax = 8192;   // bytes of a row a CTA takes at a time, at most
// Bytes of the aligned states from which on bulk copies are taken.  Caches of 8 groups of 4 rows in place, half of whose
// rows move, plain / bulk in a graph: 2 MB 3.4 / 3.7 us, 8 MB 4.3 / 4.2, 17 MB 7.0 / 5.0, 34 MB 10.1 / 7.6, 268 MB
// 84 / 39; to other buffers 8 MB 4.6 / 4.6, 17 MB 8.1 / 6.1.
constexpr int64_t kRBLeast = 16ll << 20;

struct ReorderState {
  const char* src;
  char* dst;
  int64_t src_row, dst_row;          // strides in bytes
  int64_t src_outer[2], dst_outer[2];
  int64_t chunk;                     // contiguous bytes of a row
  int64_t position;                  // bytes of a position, 0: chunks are moved whole
  int32_t n1;                        // chunks of a row: n0 * n1
  int32_t slices;                    // of a chunk
  int64_t units_end;                 // running sum of n0 * n1 * slices
};

struct ReorderArgs {
  ReorderState st[kRRStates];
  int n_states;
  int groups, beams;
  int slice;  // bytes, a multiple of 16
  bool ragged;  // a state's chunks or positions are no multiple of 16 bytes
  uint64_t wait_ns;
  const int32_t* parents;
  const int32_t* lengths;
  uint32_t* dev_status;
};

// All threads: n bytes between shared memory (16-byte aligned) and global memory at `address`, in the widest units
// that it allows.
template <typename U>
__device__ __forceinline__ int copy_units(char* to, const char* from, int n) {
  const int units = n / static_cast<int>(sizeof(U));
#pragma unroll 4
  for (int j = threadIdx.x; j < units; j += kRRThreads) reinterpret_cast<U*>(to)[j] = reinterpret_cast<const U*>(from)[j];
  return units * static_cast<int>(sizeof(U));
}
__device__ __forceinline__ void copy_bytes(char* to, const char* from, int n, uintptr_t address) {
  const int done = address % 16 == 0  ? copy_units<uint4>(to, from, n)
                   : address % 8 == 0 ? copy_units<uint2>(to, from, n)
                   : address % 4 == 0 ? copy_units<uint32_t>(to, from, n)
                   : address % 2 == 0 ? copy_units<uint16_t>(to, from, n)
                                      : 0;
  for (int j = done + threadIdx.x; j < n; j += kRRThreads) to[j] = from[j];
}

__global__ void __launch_bounds__(kRRThreads) reorder_rows_kernel(const __grid_constant__ ReorderArgs a) {
  extern __shared__ __align__(16) unsigned char stage[];  // [sources][slice]
  __shared__ int16_t parent[kBeamsMaxRows], place[kBeamsMaxRows], source[kBeamsMaxRows];
  __shared__ int32_t length[kBeamsMaxRows];
  __shared__ int n_src;
  const int tid = threadIdx.x, B = a.beams;
  pdl_wait();
  const int64_t units = a.st[a.n_states - 1].units_end;
  // a CTA keeps its group: blockIdx.y, and every gridDim.y-th one after it
  for (int group = blockIdx.y; group < a.groups; group += gridDim.y) {
    const int row0 = group * B;
    __syncthreads();
    if (tid < B) {
      const int p = __ldcg(a.parents + row0 + tid);  // (through L2: the kernel before may have just written them)
      const bool ok = p >= row0 && p < row0 + B;
      if (!ok && p != -1) set_status(a.dev_status, LMH_DS_ROW_IDX_OUT_OF_RANGE);
      parent[tid] = static_cast<int16_t>(ok ? p - row0 : tid);
      length[tid] = a.lengths ? __ldcg(a.lengths + row0 + tid) : 0x7FFFFFFF;
    }
    __syncthreads();
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
      int si = 0;
      while (u >= a.st[si].units_end) ++si;
      const ReorderState& s = a.st[si];
      const int64_t in = u - (si ? a.st[si - 1].units_end : 0);
      const int64_t outer = in / s.slices;
      const int slice = static_cast<int>(in - outer * s.slices);
      const int64_t o0 = outer / s.n1, o1 = outer - o0 * s.n1;
      const int64_t off = static_cast<int64_t>(slice) * a.slice;
      const bool in_place = s.src == s.dst;
      const char* src = s.src + o0 * s.src_outer[0] + o1 * s.src_outer[1] + off;
      char* dst = s.dst + o0 * s.dst_outer[0] + o1 * s.dst_outer[1] + off;
      const int64_t left = min(s.chunk - off, static_cast<int64_t>(a.slice));
      // bytes of row p's slice that are in use
      auto used = [&](int p) -> int {
        if (s.position == 0) return static_cast<int>(left);
        const int64_t n = static_cast<int64_t>(max(length[p], 0)) * s.position - off;
        return static_cast<int>(max(static_cast<int64_t>(0), min(n, left)));
      };
      __syncthreads();
      if (tid == 0) n_src = 0;
      if (tid < B) place[tid] = -1;
      __syncthreads();
      if (tid < B && !(in_place && parent[tid] == tid)) place[parent[tid]] = 0;  // needed
      __syncthreads();
      if (tid < B && place[tid] == 0) {
        const int i = atomicAdd(&n_src, 1);
        place[tid] = static_cast<int16_t>(i);
        source[i] = static_cast<int16_t>(tid);
      }
      __syncthreads();
      for (int i = 0; i < n_src; ++i) {
        const int p = source[i];
        const char* from = src + (row0 + p) * s.src_row;
        unsigned char* to = stage + static_cast<size_t>(i) * a.slice;
        const int n = used(p);
        copy_bytes(reinterpret_cast<char*>(to), from, n, reinterpret_cast<uintptr_t>(from));
      }
      __syncthreads();
      for (int r = 0; r < B; ++r) {
        const int p = parent[r];
        if (in_place && p == r) continue;
        char* to = dst + (row0 + r) * s.dst_row;
        copy_bytes(to, reinterpret_cast<const char*>(stage + static_cast<size_t>(place[p]) * a.slice), used(p),
                   reinterpret_cast<uintptr_t>(to));
      }
    }
  }
}

// ---------------------------------------------------------------------------
// bulk copies
// ---------------------------------------------------------------------------
// (caches of four layers, 153 us; 4 stages of 24 KB: 162; 3 CTAs of 4 stages of 16 KB: 157, of 3 of 24 KB: 204;
// 1 CTA of 6 stages: 232)
constexpr int kRBStages = 3;
constexpr int kRBCtasPerSm = 2;
constexpr int kRBStageBytes = 32 * 1024;

// What a stage holds until its rows are written.
struct ReorderStage {
  char* dst;             // of the group's first row, at the slice
  int64_t dst_row;
  int slice;             // bytes from a source to the next in the stage
  int16_t place[kBeamsMaxRows];  // of row r's source in the stage, or -1: row r is not written
  int32_t bytes[kBeamsMaxRows];  // of row r
};

__device__ __forceinline__ void bulk_store(void* gmem_dst, const void* smem_src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(gmem_dst), "r"(smem_u32(smem_src)),
               "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void bulk_stores_end() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
// This lane's stores but for the last N groups have left shared memory.
template <int N>
__device__ __forceinline__ void bulk_stores_read() { asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory"); }
__device__ __forceinline__ void bulk_stores_done() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

__global__ void __launch_bounds__(32) reorder_bulk_kernel(const __grid_constant__ ReorderArgs a) {
  extern __shared__ __align__(128) unsigned char ring[];  // [stages][sources][slice], stages of kRBStageBytes
  __shared__ ReorderStage st[kRBStages];
  __shared__ uint64_t full[kRBStages];
  __shared__ int16_t parent[kBeamsMaxRows], slot[kBeamsMaxRows], source[kBeamsMaxRows];
  __shared__ int32_t used[kBeamsMaxRows];
  constexpr int S = kRBStages, W = kBeamsMaxRows / 32;
  const int lane = threadIdx.x, B = a.beams;
  if (lane == 0) {
    for (int s = 0; s < S; ++s) mbar_init(&full[s], 1);
    mbar_init_fence();
  }
  __syncwarp();
  pdl_wait();
  // Pass t is slice unit t / groups of group (t + t / groups) % groups: a CTA's passes go through the groups, whose
  // lengths differ, and through the chunks before the slices, whose last ones may be empty.
  const uint32_t units = static_cast<uint32_t>(a.st[a.n_states - 1].units_end);
  const uint64_t passes = static_cast<uint64_t>(units) * a.groups;
  auto group_of = [&](uint64_t t) { return static_cast<int>((t + t / a.groups) % a.groups); };
  int32_t par[W], len[W];  // the rows of the next pass, asked for a pass ahead
  auto ask = [&](uint64_t t) {
    if (t >= passes) return;
    const int row0 = group_of(t) * B;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const int r = w * 32 + lane;
      if (r >= B) continue;
      par[w] = __ldcg(a.parents + row0 + r);
      len[w] = a.lengths ? __ldcg(a.lengths + row0 + r) : 0x7FFFFFFF;
    }
  };
  // The stores of stage s, once its loads have arrived; false if they did not.
  auto finish = [&](uint32_t n) -> bool {
    const int s = static_cast<int>(n % S);
    const bool ok = mbar_wait_limit(&full[s], (n / S) & 1u, a.wait_ns);
    if (!__all_sync(0xffffffffu, ok)) return false;
    const ReorderStage& e = st[s];
    const unsigned char* stage = ring + s * kRBStageBytes;
    for (int r = lane; r < B; r += 32) {
      const int p = e.place[r], bytes = e.bytes[r] & ~15;
      if (p >= 0 && bytes > 0) bulk_store(e.dst + r * e.dst_row, stage + p * e.slice, static_cast<uint32_t>(bytes));
    }
    bulk_stores_end();
    if (a.ragged) {  // the last bytes of a run of positions
      for (int r = 0; r < B; ++r) {
        const int p = e.place[r], at = (e.bytes[r] & ~15) + lane;
        if (p >= 0 && at < e.bytes[r]) e.dst[r * e.dst_row + at] = static_cast<char>(stage[p * e.slice + at]);
      }
    }
    return true;
  };
  uint64_t t = blockIdx.x;
  ask(t);
  uint32_t issued = 0, finished = 0;
  bool ok = true;
  for (; t < passes && ok; t += gridDim.x) {
    const uint32_t u = static_cast<uint32_t>(t / a.groups);
    const int row0 = group_of(t) * B;
    int si = 0;
    while (u >= static_cast<uint64_t>(a.st[si].units_end)) ++si;
    const ReorderState& s = a.st[si];
    const uint32_t in = u - static_cast<uint32_t>(si ? a.st[si - 1].units_end : 0);
    const uint32_t chunks = static_cast<uint32_t>((s.units_end - (si ? a.st[si - 1].units_end : 0)) / s.slices);
    const uint32_t slice = in / chunks, outer = in - slice * chunks;
    const uint32_t o0 = outer / s.n1, o1 = outer - o0 * s.n1;
    const int64_t off = static_cast<int64_t>(slice) * a.slice;
    const bool in_place = s.src == s.dst;
    const int left = static_cast<int>(min(s.chunk - off, static_cast<int64_t>(a.slice)));
    // ---- the group's rows ----
    __syncwarp();
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const int r = w * 32 + lane;
      if (r >= B) continue;
      const bool good = par[w] >= row0 && par[w] < row0 + B;
      if (!good && par[w] != -1) set_status(a.dev_status, LMH_DS_ROW_IDX_OUT_OF_RANGE);
      parent[r] = static_cast<int16_t>(good ? par[w] - row0 : r);
      const int64_t n = s.position == 0 ? left : static_cast<int64_t>(max(len[w], 0)) * s.position - off;
      used[r] = static_cast<int32_t>(max(static_cast<int64_t>(0), min(n, static_cast<int64_t>(left))));
      slot[r] = -1;
    }
    __syncwarp();
    ask(t + gridDim.x);
    bool moves = false;
    for (int r = lane; r < B; r += 32) {
      const int p = parent[r];
      if (used[p] > 0 && !(in_place && p == r)) {
        slot[p] = 0;  // needed
        moves = true;
      }
    }
    if (!__any_sync(0xffffffffu, moves)) continue;  // (nothing in use here, or every row stays)
    __syncwarp();
    int n_src = 0;
    for (int w = 0; w * 32 < B; ++w) {
      const int r = w * 32 + lane;
      const bool need = r < B && slot[r] == 0;
      const unsigned m = __ballot_sync(0xffffffffu, need);
      if (need) {
        const int i = n_src + __popc(m & ((1u << lane) - 1));
        slot[r] = static_cast<int16_t>(i);
        source[i] = static_cast<int16_t>(r);
      }
      n_src += __popc(m);
    }
    __syncwarp();
    const char* src = s.src + o0 * s.src_outer[0] + o1 * s.src_outer[1] + off + row0 * s.src_row;
    char* dst = s.dst + o0 * s.dst_outer[0] + o1 * s.dst_outer[1] + off + row0 * s.dst_row;
    // A stage holds the slices of half the group's rows, which are seldom more; else the slice goes in halves.
    const bool halves = n_src * a.slice > kRBStageBytes;
    const int sub = halves ? a.slice / 2 : a.slice;
    for (int h = 0; h < (halves ? 2 : 1) && ok; ++h) {
      auto bytes_of = [&](int p) { return min(max(used[p] - h * sub, 0), sub); };
      // ---- the stage: its last stores have read it, then its loads ----
      const int sg = static_cast<int>(issued % S);
      bulk_stores_read<S - 2>();  // (a group of stores a stage: this one's were S - 1 stages ago)
      // a run's last bytes were written and read there by threads, before copies write to the same place
      if (a.ragged) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      ReorderStage& e = st[sg];
      if (lane == 0) e.dst = dst + h * sub, e.dst_row = s.dst_row, e.slice = sub;
      uint32_t bytes = 0;
      for (int i = lane; i < n_src; i += 32) bytes += static_cast<uint32_t>(bytes_of(source[i]) & ~15);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) bytes += __shfl_xor_sync(0xffffffffu, bytes, o);
      for (int r = lane; r < B; r += 32) {
        const int p = parent[r];
        const bool go = used[p] > 0 && !(in_place && p == r);
        e.place[r] = go ? slot[p] : static_cast<int16_t>(-1);
        e.bytes[r] = bytes_of(p);
      }
      unsigned char* stage = ring + sg * kRBStageBytes;
      if (a.ragged) {
        for (int i = 0; i < n_src; ++i) {
          const int p = source[i], n = bytes_of(p), at = (n & ~15) + lane;
          if (at < n) stage[i * sub + at] = static_cast<unsigned char>(__ldcg(src + h * sub + p * s.src_row + at));
        }
      }
      if (lane == 0) mbar_arrive_expect_tx(&full[sg], bytes);
      __syncwarp();
      for (int i = lane; i < n_src; i += 32) {
        const int p = source[i], n = bytes_of(p) & ~15;
        if (n > 0) bulk_load(stage + i * sub, src + h * sub + p * s.src_row, static_cast<uint32_t>(n), &full[sg]);
      }
      ++issued;
      if (issued - finished == static_cast<uint32_t>(S - 1)) ok = finish(finished++);
    }
  }
  while (ok && finished < issued) ok = finish(finished++);
  if (!ok) {  // the copies in flight land before the CTA exits
    if (lane == 0) set_status(a.dev_status, LMH_DS_TIMEOUT);
    for (uint32_t n = finished - 1; n < issued; ++n) mbar_wait(&full[n % S], (n / S) & 1u);
  }
  bulk_stores_done();
}

cudaError_t reorder_setup() {
  cudaError_t e = cudaFuncSetAttribute(reorder_rows_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kRRSmem);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(reorder_bulk_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kRBStages * kRBStageBytes);
  return e;
}

// Whether a state's rows, chunks and slices begin on 16-byte boundaries (and hold 16 bytes at least).
static bool state_aligned(const lmh_row_state& s) {
  const int64_t all = s.src_row_bytes | s.dst_row_bytes | s.src_outer_bytes[0] | s.src_outer_bytes[1] |
                      s.dst_outer_bytes[0] | s.dst_outer_bytes[1];
  return all % 16 == 0 && reinterpret_cast<uintptr_t>(s.src) % 16 == 0 && reinterpret_cast<uintptr_t>(s.dst) % 16 == 0 &&
         s.chunk_bytes >= 16;
}

cudaError_t launch_reorder_rows(const lmh_row_state* states, int num_states, int groups, int beams,
                                const int32_t* parents, const int32_t* lengths, uint32_t* dev_status, int num_sms,
                                cudaStream_t stream) {
  int64_t aligned_bytes = 0;
  for (int i = 0; i < num_states; ++i)
    if (states[i].n0 && states[i].n1 && states[i].chunk_bytes && state_aligned(states[i]))
      aligned_bytes += static_cast<int64_t>(states[i].n0) * states[i].n1 * states[i].chunk_bytes * groups * beams;
  for (int bulk = 0; bulk < 2; ++bulk) {
    // plain: every row of a group may be needed at once; bulk: half of them (see the kernel)
    int slice = (bulk ? kRBStageBytes / ((beams + 1) / 2) : kRRSmem / beams) / 128 * 128;
    if (!bulk && slice > kRRSliceMax) slice = kRRSliceMax;
    for (int at = 0; at < num_states;) {
      ReorderArgs a{};
      a.groups = groups;
      a.beams = beams;
      a.slice = slice;
      a.parents = parents;
      a.lengths = lengths;
      a.dev_status = dev_status;
      a.wait_ns = wait_limit_ns();
      int64_t units = 0;
      for (; at < num_states && a.n_states < kRRStates; ++at) {
        const lmh_row_state& s = states[at];
        if (s.n0 == 0 || s.n1 == 0 || s.chunk_bytes == 0) continue;
        if ((aligned_bytes >= kRBLeast && state_aligned(s)) != (bulk != 0)) continue;
        ReorderState& t = a.st[a.n_states++];
        t.src = static_cast<const char*>(s.src);
        t.dst = static_cast<char*>(s.dst);
        t.src_row = s.src_row_bytes;
        t.dst_row = s.dst_row_bytes;
        for (int i = 0; i < 2; ++i) t.src_outer[i] = s.src_outer_bytes[i], t.dst_outer[i] = s.dst_outer_bytes[i];
        t.chunk = s.chunk_bytes;
        t.position = lengths ? s.position_bytes : 0;
        t.n1 = s.n1;
        t.slices = static_cast<int32_t>((s.chunk_bytes + slice - 1) / slice);
        units += static_cast<int64_t>(s.n0) * s.n1 * t.slices;
        t.units_end = units;
        if (s.chunk_bytes % 16 != 0 || t.position % 16 != 0) a.ragged = true;
      }
      if (a.n_states == 0) continue;
      if (units > INT32_MAX) return cudaErrorInvalidValue;
      trace_begin(kTraceReorder, stream);
      cudaError_t e;
      if (bulk) {
        const int64_t passes = units * groups, ctas = static_cast<int64_t>(kRBCtasPerSm) * num_sms;
        e = launch_kernel(reorder_bulk_kernel, dim3(static_cast<unsigned>(passes < ctas ? passes : ctas)), dim3(32),
                          static_cast<size_t>(kRBStages * kRBStageBytes), stream, true, a);
      } else {
        const int64_t ctas = 3ll * num_sms;
        const int gy = static_cast<int>(groups < ctas ? groups : ctas);
        int64_t gx = (ctas + gy - 1) / gy;
        if (gx > units) gx = units;
        e = launch_kernel(reorder_rows_kernel, dim3(static_cast<unsigned>(gx), gy), dim3(kRRThreads),
                          static_cast<size_t>(slice) * beams, stream, true, a);
      }
      trace_end(kTraceReorder, stream);
      if (e != cudaSuccess) return e;
    }
  }
  return cudaSuccess;
}

}  // namespace lmh
