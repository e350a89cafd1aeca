// reorder_rows.cu -- the states of a batch follow the rows they come from (lmh_reorder_rows).
//
// Row r of every state gets what row parents[r] held, within groups of `beams` rows.  All rows of a group
// that others need are read into shared memory, a slice at a time, before any is written: in place, a row
// may be both a source and overwritten.  Rows that stay are neither read nor written; a row that several
// take is read once.
#include "device_common.cuh"
#include "lmh_internal.h"

namespace lmh {

constexpr int kRRThreads = 256;
constexpr int kRRStates = 24;       // states of one launch
constexpr int kRRSmem = 64 * 1024;  // staging
constexpr int kRRSliceMax = 8192;   // bytes of a row a CTA takes at a time, at most

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
  const int32_t* parents;
  const int32_t* lengths;
  uint32_t* dev_status;
};

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
        if (reinterpret_cast<uintptr_t>(from) % 16 == 0) {
          for (int j = tid * 16; j + 16 <= n; j += kRRThreads * 16)
            *reinterpret_cast<uint4*>(to + j) = *reinterpret_cast<const uint4*>(from + j);
          for (int j = (n & ~15) + tid; j < n; j += kRRThreads) to[j] = static_cast<unsigned char>(from[j]);
        } else {
          for (int j = tid; j < n; j += kRRThreads) to[j] = static_cast<unsigned char>(from[j]);
        }
      }
      __syncthreads();
      for (int r = 0; r < B; ++r) {
        const int p = parent[r];
        if (in_place && p == r) continue;
        const unsigned char* from = stage + static_cast<size_t>(place[p]) * a.slice;
        char* to = dst + (row0 + r) * s.dst_row;
        const int n = used(p);
        if (reinterpret_cast<uintptr_t>(to) % 16 == 0) {
          for (int j = tid * 16; j + 16 <= n; j += kRRThreads * 16)
            *reinterpret_cast<uint4*>(to + j) = *reinterpret_cast<const uint4*>(from + j);
          for (int j = (n & ~15) + tid; j < n; j += kRRThreads) to[j] = static_cast<char>(from[j]);
        } else {
          for (int j = tid; j < n; j += kRRThreads) to[j] = static_cast<char>(from[j]);
        }
      }
    }
  }
}

cudaError_t reorder_setup() {
  return cudaFuncSetAttribute(reorder_rows_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kRRSmem);
}

cudaError_t launch_reorder_rows(const lmh_row_state* states, int num_states, int groups, int beams,
                                const int32_t* parents, const int32_t* lengths, uint32_t* dev_status, int num_sms,
                                cudaStream_t stream) {
  int slice = kRRSmem / beams / 128 * 128;  // every row of a group may be needed
  if (slice > kRRSliceMax) slice = kRRSliceMax;
  for (int at = 0; at < num_states; at += kRRStates) {
    ReorderArgs a{};
    a.groups = groups;
    a.beams = beams;
    a.slice = slice;
    a.parents = parents;
    a.lengths = lengths;
    a.dev_status = dev_status;
    int64_t units = 0;
    for (int i = at; i < num_states && i < at + kRRStates; ++i) {
      const lmh_row_state& s = states[i];
      if (s.n0 == 0 || s.n1 == 0 || s.chunk_bytes == 0) continue;
      ReorderState& t = a.st[a.n_states++];
      t.src = static_cast<const char*>(s.src);
      t.dst = static_cast<char*>(s.dst);
      t.src_row = s.src_row_bytes;
      t.dst_row = s.dst_row_bytes;
      t.src_outer[0] = s.src_outer_bytes[0];
      t.src_outer[1] = s.src_outer_bytes[1];
      t.dst_outer[0] = s.dst_outer_bytes[0];
      t.dst_outer[1] = s.dst_outer_bytes[1];
      t.chunk = s.chunk_bytes;
      t.position = lengths ? s.position_bytes : 0;
      t.n1 = s.n1;
      t.slices = static_cast<int32_t>((s.chunk_bytes + slice - 1) / slice);
      units += static_cast<int64_t>(s.n0) * s.n1 * t.slices;
      t.units_end = units;
    }
    if (a.n_states == 0) continue;
    const int64_t ctas = 3ll * num_sms;
    const int gy = static_cast<int>(groups < ctas ? groups : ctas);
    int64_t gx = (ctas + gy - 1) / gy;
    if (gx > units) gx = units;
    trace_begin(kTraceReorder, stream);
    const cudaError_t e = launch_kernel(reorder_rows_kernel, dim3(static_cast<unsigned>(gx), gy), dim3(kRRThreads),
                                        static_cast<size_t>(slice) * beams, stream, true, a);
    trace_end(kTraceReorder, stream);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace lmh
