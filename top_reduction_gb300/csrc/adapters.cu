// adapters.cu -- the plan of a call with many rows (lmh_add_adapters), and the host side; the products: adapters.cuh.
#include "adapters.cuh"

namespace lmh {

// ---------------------------------------------------------------------------
// plan: rows by adapter, cut into tiles
// ---------------------------------------------------------------------------
// One CTA.  Counts per adapter (slot `count` holds the rows without one), a scan, the rows' places.  Lanes
// with the same adapter take their places with one atomic.  The order of an adapter's rows is whatever the
// atomics make it: no row's result depends on it.  16384 rows take 13 us alone, of one SM's latency and issue (0.66 of its
// slots); indices loaded one look ahead in place of 16 at once: 17 us.
__global__ void __launch_bounds__(kADPlanThreads) adapter_plan_kernel(const AdapterArgs a) {
  extern __shared__ int32_t plan_smem[];
  const int L = a.count;
  int32_t* next = plan_smem;              // [L + 1] counts, then the next free place
  int32_t* first_tile = plan_smem + L + 1;  // [L + 2]
  __shared__ int32_t wsum[2][kADPlanThreads / 32];
  __shared__ int32_t carry[2];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_wait();
  pdl_launch_dependents();
  for (int i = tid; i <= L; i += kADPlanThreads) next[i] = 0;
  if (tid < 2) carry[tid] = 0;
  __syncthreads();
  bool bad = false;
  constexpr int HELD = 16;  // rows a thread looks up at once
  // f(row, slot) for every row, a warp's lanes together; slot -1 behind the last
  auto for_rows = [&](auto f) {
    for (int base = 0; base < a.rows; base += HELD * kADPlanThreads) {
      int l[HELD];
#pragma unroll
      for (int u = 0; u < HELD; ++u) {
        const int i = base + u * kADPlanThreads + tid;
        l[u] = i < a.rows ? __ldcg(a.adapter_idx + i) : -2;
      }
#pragma unroll
      for (int u = 0; u < HELD; ++u) {
        if (base + u * kADPlanThreads >= a.rows) break;
        const bool in = l[u] >= 0 && l[u] < L;
        bad |= !in && l[u] != -1 && l[u] != -2;
        const int i = base + u * kADPlanThreads + tid;
        bad |= l[u] == -2 && i < a.rows;
        f(i, i >= a.rows ? -1 : in ? l[u] : L);
      }
    }
  };
  // The lanes with the same slot.  Packed prompts hand a warp rows of one adapter, which is seen at once.
  auto same_slot = [&](int l) {
    return __all_sync(0xffffffffu, l == __shfl_sync(0xffffffffu, l, 0)) ? 0xffffffffu : __match_any_sync(0xffffffffu, l);
  };
  for_rows([&](int, int l) {
    const unsigned same = same_slot(l);
    if (l >= 0 && lane == __ffs(same) - 1) atomicAdd(&next[l], __popc(same));
  });
  __syncthreads();
  // exclusive sums of rows and of tiles over the adapters
  for (int base = 0; base <= L; base += kADPlanThreads) {
    const int l = base + tid;
    const int n = l <= L ? next[l] : 0;
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
    if (l <= L) next[l] = before_n, first_tile[l] = before_t;
    __syncthreads();
  }
  const int tiles = carry[1];
  if (tid == 0) {
    *a.tile_count = tiles;
    first_tile[L + 1] = tiles;
  }
  __syncthreads();
  // a thread a tile: its adapter is the last whose first tile is not behind it and that has tiles
  for (int t = tid; t < tiles; t += kADPlanThreads) {
    int lo = 0, hi = L;
    while (lo < hi) {
      const int mid = (lo + hi + 1) / 2;
      if (first_tile[mid] <= t) lo = mid;
      else hi = mid - 1;
    }
    const int part = t - first_tile[lo];
    const int begin = next[lo], end = lo < L ? next[lo + 1] : a.rows;
    const int at = begin + part * kADTile;
    a.tiles[t] = AdapterTile{lo < L ? lo : -1, at, min(kADTile, end - at), 0};
  }
  __syncthreads();
  for_rows([&](int i, int l) {
    const unsigned same = same_slot(l);
    const int leader = __ffs(same) - 1;
    int at = 0;
    if (l >= 0 && lane == leader) at = atomicAdd(&next[l], __popc(same));
    at = __shfl_sync(0xffffffffu, at, leader);
    if (l >= 0) a.order[at + __popc(same & ((1u << lane) - 1))] = i;
  });
  if (bad) set_status(a.dev_status, LMH_DS_ADAPTER_OUT_OF_RANGE);
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
  // two blocks of 32 a warp at least; calls of many rows: four stages a CTA
  const int most = rows > kADOwnPlan ? (H + kADDownStage - 1) / kADDownStage / 4 : blocks / (2 * kADWarps);
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

cudaError_t adapters_setup() {
  const cudaError_t e = adapters_setup_bf16();
  return e == cudaSuccess ? adapters_setup_f16() : e;
}

static cudaError_t launch_adapters(const AdapterArgs& a, bool bf16, lmh_dtype out_dtype, bool vec, int num_sms,
                                   cudaStream_t stream) {
  const int64_t max_tiles = adapter_max_tiles(a.rows, a.count);
  cudaError_t e = cudaSuccess;
  if (a.rows > kADOwnPlan) {
    trace_begin(kTraceAdapterPlan, stream);
    e = launch_kernel(adapter_plan_kernel, dim3(1), dim3(kADPlanThreads), static_cast<size_t>(2 * a.count + 3) * 4,
                      stream, true, a);
    trace_end(kTraceAdapterPlan, stream);
    if (e != cudaSuccess) return e;
  }
  const int grid = static_cast<int>(max_tiles < 4 * num_sms ? max_tiles : 4 * num_sms);
  trace_begin(kTraceAdapterDown, stream);
  e = bf16 ? launch_down_bf16(a, grid, stream) : launch_down_f16(a, grid, stream);
  trace_end(kTraceAdapterDown, stream);
  if (e != cudaSuccess) return e;
  trace_begin(kTraceAdapterUp, stream);
  e = bf16 ? launch_up_bf16(a, out_dtype, vec, max_tiles, num_sms, stream)
           : launch_up_f16(a, out_dtype, vec, max_tiles, num_sms, stream);
  trace_end(kTraceAdapterUp, stream);
  return e;
}

// Whether rows of y or out can be read and written n neighbours at a time.
static bool adapter_rows_align(const void* p, int64_t stride, int N, lmh_dtype dtype, int n) {
  const int bytes = n * (dtype == LMH_F32 ? 4 : 2);
  return reinterpret_cast<uintptr_t>(p) % bytes == 0 && stride % n == 0 && N % n == 0;
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
  auto align = [&](int n) {
    return adapter_rows_align(y, y_stride, t.N, out_dtype, n) && adapter_rows_align(out, out_stride, t.N, out_dtype, n);
  };
  const bool vec = align(4);
  a.piece = out_dtype == LMH_F32 || align(8) ? 16 : 8;
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
  return launch_adapters(a, t.dtype == LMH_BF16, out_dtype, vec, num_sms, stream);
}

}  // namespace lmh
