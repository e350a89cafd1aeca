// sample_logits.cu -- one token per row with temperature, top-k, top-p and
// min-p from one given uniform number (lmh_sample_from_logits).
//
// A row belongs to a thread-block cluster.  Its CTAs hold the row in their
// shared memory (a contiguous slice of the ids each), so HBM is read once and
// every later pass -- the sum of the weights, the searches for the top-k and
// top-p thresholds, the draw -- runs on chip.
//
// Weights are whole numbers, w = rint(2^32 exp2(t)) with t = (z - max) * c: their
// sums are the same in any order, so neither the split over threads, warps and
// CTAs nor the batch changes a draw.  A sum costs no integer conversion per
// logit: adding 1.5 * 2^9 to p = exp2(t) leaves p rounded to 2^-14 in the
// mantissa's low bits, the rest p - that (exact) plus 1.5 * 2^-9 leaves it
// rounded to 2^-32 in the same way, and the two bit patterns are summed as
// integers (the constants' bits are taken off once at the end).
//
// Two ways to the kept tokens of a row with top-k or top-p:
// - A list.  Every lane knows the largest of its own logits.  A histogram of these
//   maxima over z gives a bound that at least k tokens reach (128 for top-p alone),
//   few more than that do, and only warps with such a lane look at their logits
//   again.  The tokens that reach it go to the cluster's first CTA, which ranks
//   them by counting: with n tokens, n^2 comparisons give every token its rank and the
//   mass before it.  This holds for k up to kListTarget, and for top-p wherever the
//   listed tokens have the mass that is asked for.
// - A threshold (z, id) otherwise: every token with a larger logit is kept, and those
//   equal to it up to that id.  It is the last token of the prefix of the order (z
//   descending, id ascending) that reaches a count (top-k) or a mass (top-p): a
//   histogram of all logits over t, one of the bin that holds the end over its 512th
//   parts, and a list of what is left there.  Where that is too long (many equal
//   logits), histograms over ever smaller intervals of z go on until one value is left,
//   whose tokens are counted off in id order.  The bins that the second histogram cuts
//   up come from a sample of the row, with a margin, in place of the first histogram: an
//   addition in shared memory for every logit costs more than all arithmetic on it.
//   Sums stay exact, so a sample that misses costs time, not the result.
// Tokens of weight 0 (t < -33) can be left out of either: no draw falls on them and no
// sum changes.
//
// What bounds it is latency: a row is a chain of steps, each a pass over what a thread
// holds (a microsecond or two) or an agreement of the cluster (one), and a decode batch is
// one wave of rows.  Measured with cold L2: 20 us for one row of 128256 f32 with top-k and
// top-p, 45 for 32 rows of 151936 f32 with mixed filters (half of them are done after 19
// us in the kernel; the longest chain, 43, is a top-p row whose tokens do not fit a list:
// loading 6 us, the list that does not do 12, the bracket 7, the parts 8, their list 5, the
// draw 6), 27 for 64 rows of 128256 bf16 with min-p and a mask, 147 for 256 rows of 248320
// bf16 (127 MB; 2048 CTAs, two to an SM).  HBM is not the bound in any of them: 13% of its
// time for the largest.  (The 32 rows take 33 to 43 us in a row of calls, by how many of them
// need a threshold.)  Top-k beyond a list and top-p after it are two searches: 51 us for one
// flat row of 151936 f32 with k 1000, 68 for 32 of them, 408 for 256 in bf16.
// The lists' bins lie over z as it is, so that no row's maximum is needed first.  A row whose
// logits are all above 64 or below -64, or most of them within a bin, overflows its list and
// takes the threshold's way after it: 113 us for one row of 128256 f32 with k 50 and p 0.95
// where 18 are usual, 164 for 32 of 151936 where 20 are.  Half the CTAs per row there, with twice the logits each, were
// slower (205 us where an earlier state of this kernel took 166).
// The next kernel is not let in early, although none of this library's reads ids ahead of its
// wait any more: that would let draws in a row overlap, and has not been measured in this form.
//
// A row's work is a chain of short steps, each run once by a CTA, so instructions come
// from far away more often than not: written out for every element of a vector in every
// pass, the kernel had 300 KB of them and spent most of its time fetching them.  Only
// the passes over all logits are unrolled; the steps of the searches take one element
// per lane, and what does not depend on the logits' type is a function of its own.
#include <cmath>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "device_common.cuh"
#include "lmh_internal.h"

namespace lmh {

namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kBins = 512;             // of every histogram: one per thread
constexpr int kListCap = 512;          // tokens in a list, and in one CTA's part of it
constexpr int kListTarget = 384;       // largest k that is tried with a list
constexpr int kListTargetTopP = 128;   // tokens asked for with top-p alone
constexpr float kMinT = -33.0f;        // below: weight 0
constexpr float kMaxBinsTop = 64.0f;   // the lanes' maxima: bins from this z down,
constexpr float kMaxBinsPer = 4.0f;    // so many to a unit
constexpr int kSampleFromV = 16384;    // vocabularies whose threshold searches begin with a sample
constexpr int kSampleStep = 16;        // of which one logit in so many is (8 and 32: no difference)
constexpr int kUnroll = 4;             // vectors of a lane whose mask words are in flight at once
constexpr float kHiAdd = 768.0f;             // 1.5 * 2^9: unit 2^-14
constexpr float kLoAdd = 0.0029296875f;      // 1.5 * 2^-9: unit 2^-32
constexpr uint32_t kHiBits = 0x44400000u;    // of kHiAdd
constexpr uint32_t kLoBits = 0x3B400000u;    // of kLoAdd
constexpr int kHiShift = 18;                 // 2^-14 in units of 2^-32

using u64 = unsigned long long;

// ---------------------------------------------------------------------------
// clusters
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
// All threads of all CTAs of the cluster; orders their shared-memory accesses.
__device__ __forceinline__ void cluster_arrive() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.aligned.release;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  __syncwarp();
  asm volatile("barrier.cluster.wait.aligned.acquire;" ::: "memory");
}
__device__ __forceinline__ void cluster_sync() {
  cluster_arrive();
  cluster_wait();
}
// Address of `p` (this CTA's shared memory) in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t cluster_addr(const void* p, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  return a;
}
__device__ __forceinline__ void st_cluster_u64(uint32_t a, u64 v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(a), "l"(v) : "memory");
}
__device__ __forceinline__ void st_cluster_u32(uint32_t a, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}
__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ u64 ld_cluster_u64(uint32_t a) {
  u64 v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(a) : "memory");
  return v;
}

// ---------------------------------------------------------------------------
// logits in 16-byte vectors
// ---------------------------------------------------------------------------
template <typename T>
struct Vec;  // kN elements a vector; to_float and widen are exact
template <>
struct Vec<float> {
  static constexpr int kN = 4;
  static constexpr int kZeroBits = 0;  // low bits of a widened value that are always 0
  static __device__ __forceinline__ void widen(const uint4& x, float (&z)[4]) {
    z[0] = __uint_as_float(x.x);
    z[1] = __uint_as_float(x.y);
    z[2] = __uint_as_float(x.z);
    z[3] = __uint_as_float(x.w);
  }
  static __device__ __forceinline__ float to_float(float x) { return x; }
  static __device__ __forceinline__ float from_float(float x) { return x; }
  // NaN becomes -inf
  static __device__ __forceinline__ uint4 clean(const uint4& x) {
    auto f = [](uint32_t u) { return __float_as_uint(fmaxf(__uint_as_float(u), -INFINITY)); };
    return make_uint4(f(x.x), f(x.y), f(x.z), f(x.w));
  }
  static __device__ __forceinline__ float max_of(const uint4& x) {
    return fmaxf(fmaxf(__uint_as_float(x.x), __uint_as_float(x.y)), fmaxf(__uint_as_float(x.z), __uint_as_float(x.w)));
  }
  // -inf in element e where bit e of `allowed` is clear
  static __device__ __forceinline__ uint4 masked(const uint4& x, uint32_t allowed) {
    return make_uint4((allowed & 1) ? x.x : 0xFF800000u, (allowed & 2) ? x.y : 0xFF800000u,
                      (allowed & 4) ? x.z : 0xFF800000u, (allowed & 8) ? x.w : 0xFF800000u);
  }
};
// The same for the 16-bit types: kNegInf twice in a word, packed maxima.
template <uint32_t kNegInf, typename Max2>
__device__ __forceinline__ uint4 clean16(const uint4& x, Max2 max2) {
  return make_uint4(max2(x.x, kNegInf), max2(x.y, kNegInf), max2(x.z, kNegInf), max2(x.w, kNegInf));
}
template <uint32_t kNegInf>
__device__ __forceinline__ uint4 masked16(const uint4& x, uint32_t allowed) {
  auto one = [&](uint32_t u, uint32_t bits) {
    const uint32_t keep = ((bits & 1) ? 0x0000FFFFu : 0u) | ((bits & 2) ? 0xFFFF0000u : 0u);
    return (u & keep) | (kNegInf & ~keep);
  };
  return make_uint4(one(x.x, allowed), one(x.y, allowed >> 2), one(x.z, allowed >> 4), one(x.w, allowed >> 6));
}
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t max_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int kN = 8;
  static constexpr int kZeroBits = 16;
  static __device__ __forceinline__ void widen(const uint4& x, float (&z)[8]) {
    const uint32_t u[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      z[2 * i] = __uint_as_float(u[i] << 16);
      z[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
    }
  }
  static __device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
  static __device__ __forceinline__ __nv_bfloat16 from_float(float x) { return __float2bfloat16_rn(x); }
  static __device__ __forceinline__ uint4 clean(const uint4& x) { return clean16<0xFF80FF80u>(x, max_bf16x2); }
  static __device__ __forceinline__ uint4 masked(const uint4& x, uint32_t allowed) {
    return masked16<0xFF80FF80u>(x, allowed);
  }
  static __device__ __forceinline__ float max_of(const uint4& x) {
    const uint32_t m = max_bf16x2(max_bf16x2(x.x, x.y), max_bf16x2(x.z, x.w));
    return fmaxf(__uint_as_float(m << 16), __uint_as_float(m & 0xFFFF0000u));
  }
};
template <>
struct Vec<__half> {
  static constexpr int kN = 8;
  static constexpr int kZeroBits = 13;
  static __device__ __forceinline__ void widen(const uint4& x, float (&z)[8]) {
    const uint32_t u[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
      z[2 * i] = f.x;
      z[2 * i + 1] = f.y;
    }
  }
  static __device__ __forceinline__ float to_float(__half x) { return __half2float(x); }
  static __device__ __forceinline__ __half from_float(float x) { return __float2half_rn(x); }
  static __device__ __forceinline__ uint4 clean(const uint4& x) { return clean16<0xFC00FC00u>(x, max_f16x2); }
  static __device__ __forceinline__ uint4 masked(const uint4& x, uint32_t allowed) {
    return masked16<0xFC00FC00u>(x, allowed);
  }
  static __device__ __forceinline__ float max_of(const uint4& x) {
    const uint32_t m = max_f16x2(max_f16x2(x.x, x.y), max_f16x2(x.z, x.w));
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&m));
    return fmaxf(f.x, f.y);
  }
};

// ---------------------------------------------------------------------------
// weights
// ---------------------------------------------------------------------------
__device__ __forceinline__ float tempered(float z, float zm, float c) { return __fmul_rn(__fsub_rn(z, zm), c); }

// The two parts of the weight of p = exp2(t), as bit patterns to be summed.
__device__ __forceinline__ void weight_bits(float p, uint32_t& hi, uint32_t& lo) {
  const float h = __fadd_rn(p, kHiAdd);
  const float rest = __fsub_rn(p, __fsub_rn(h, kHiAdd));
  hi = __float_as_uint(h);
  lo = __float_as_uint(__fadd_rn(rest, kLoAdd));
}
// Sum of n weights from the sums (mod 2^32) of their parts; n < 2^14.
__device__ __forceinline__ u64 weight_sum(uint32_t hi, uint32_t lo, uint32_t n) {
  const long long h = static_cast<int32_t>(hi - n * kHiBits), l = static_cast<int32_t>(lo - n * kLoBits);
  return static_cast<u64>((h << kHiShift) + l);
}
__device__ __forceinline__ u64 weight_of(float t) {
  uint32_t hi, lo;
  weight_bits(ex2_approx(t), hi, lo);
  return weight_sum(hi, lo, 1);
}

// f * mass for 0 < f < 1 and mass < 2^53, rounded to fp64, then down or up to a whole
// number.
__device__ __noinline__ u64 fp64_product(float f, u64 mass, bool up) {
  const double x = __dmul_rn(static_cast<double>(f), static_cast<double>(static_cast<long long>(mass)));
  return up ? __double2ull_ru(x) : __double2ull_rd(x);
}

// The mass that top-p asks for: max(1, ceil(p * mass)), p < 1.
__device__ __forceinline__ u64 mass_wanted(float top_p, u64 mass) {
  return top_p > 0.0f ? max(1ull, fp64_product(top_p, mass, true)) : 1ull;
}

// The point of a draw: floor(u * total), below total.
__device__ __forceinline__ u64 draw_point(float uniform, u64 total) {
  const float u = fminf(fmaxf(uniform, 0.0f), 0.99999994f);
  const u64 r = fp64_product(u, total, false);
  return r < total ? r : total - 1;
}

struct Params {
  const void* logits;
  int64_t row_stride;
  int rows, V;
  lmh_filters f;
  const float* uniforms;
  int32_t* ids;
  float* logprobs;
  uint32_t* dev_status;
  uint64_t wait_ns;  // limit of the wait for a row's copies
};

// What is kept: t >= min_t, and z > z_cut or (z == z_cut and id <= id_cut).
struct Kept {
  float min_t;
  float z_cut;
  int id_cut;
};

// A listed token: its key (z, id) as in device_common.cuh, and its weight.
struct __align__(16) Listed {
  u64 key;
  u64 w;
};

struct Shared {
  // read or written by the other CTAs of the cluster
  u64 slot[2][kMaxCluster];  // of a reduction: each CTA's value
  uint32_t list_hist[kBins];
  uint32_t list_n;
  int list_ok;
  u64 list_key, list_mass;
  u64 part_n[kMaxCluster], part_ends[kMaxCluster];  // each CTA's, as `slot`
  union {
    uint32_t hist[2][2][kBins];  // [which][high, low part or count][bin]
    struct {
      u64 part[kListCap];        // this CTA's part of a list: keys (over hist[0])
      Listed list[kListCap];     // the first CTA's list (over hist[1])
    };
  };
  // this CTA's own
  u64 scratch[kWarps];
  u64 warp_mass[kWarps];
  u64 found_above;
  int found_bin, found_hi;
  uint32_t extremes[2];
  int count;
  u64 kept, point;
  uint64_t arrived[kWarps];  // barriers: a warp's part of the row is there
};

__shared__ Shared sh;
extern __shared__ uint4 row_data[];

// ---------------------------------------------------------------------------
// steps that do not depend on the logits' type
// ---------------------------------------------------------------------------
__device__ __noinline__ u64 warp_sum_u64(u64 v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Inclusive sum over a warp's lanes.
__device__ __noinline__ u64 warp_scan_u64(u64 v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const u64 t = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += t;
  }
  return v;
}

// Sum over this CTA of every thread's value.
__device__ __noinline__ u64 block_sum_u64(u64 v) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  v = warp_sum_u64(v);
  __syncthreads();
  if (lane == 0) sh.scratch[warp] = v;
  __syncthreads();
  return warp_sum_u64(lane < kWarps ? sh.scratch[lane] : 0);
}

// The reductions over the cluster: one warp gives this CTA's value to every CTA, so
// that behind the barrier each reads its own shared memory.  `parity` alternates from
// one reduction to the next.
__device__ __noinline__ uint32_t cluster_max(uint32_t v, int parity) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int size = static_cast<int>(cluster_size());
  v = __reduce_max_sync(0xffffffffu, v);
  __syncthreads();
  if (lane == 0) sh.scratch[warp] = v;
  __syncthreads();
  if (warp == 0) {
    const uint32_t m = __reduce_max_sync(0xffffffffu, lane < kWarps ? static_cast<uint32_t>(sh.scratch[lane]) : 0u);
    if (lane < size) st_cluster_u64(cluster_addr(&sh.slot[parity][cluster_rank()], lane), m);
  }
  cluster_sync();
  return __reduce_max_sync(0xffffffffu, lane < size ? static_cast<uint32_t>(sh.slot[parity][lane]) : 0u);
}

// Sum over the cluster of one value per warp (the same in its lanes), and the sum over
// the CTAs before this one.  Leaves the warps' values in sh.warp_mass.
struct Sum {
  u64 all, before;
};
__device__ __noinline__ Sum cluster_sum(u64 v, int parity) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int size = static_cast<int>(cluster_size()), rank = static_cast<int>(cluster_rank());
  __syncthreads();
  if (lane == 0) sh.warp_mass[warp] = v;
  __syncthreads();
  if (warp == 0) {
    const u64 m = warp_sum_u64(lane < kWarps ? sh.warp_mass[lane] : 0);
    if (lane < size) st_cluster_u64(cluster_addr(&sh.slot[parity][rank], lane), m);
  }
  cluster_sync();
  Sum s{0, 0};
  for (int r = 0; r < size; ++r) {
    const u64 m = sh.slot[parity][r];
    s.all += m;
    if (r < rank) s.before += m;
  }
  return s;
}

// This thread's bin, summed over the cluster's CTAs: hist0 counts, or with hist1 the high
// and low parts of masses.
__device__ __noinline__ u64 gather_bin(const uint32_t* hist0, const uint32_t* hist1) {
  const int size = static_cast<int>(cluster_size());
  uint32_t a[kMaxCluster], b[kMaxCluster];
#pragma unroll
  for (int r = 0; r < kMaxCluster; ++r) {  // (all loads in flight before the first is used)
    a[r] = b[r] = 0;
    if (r < size) {
      a[r] = ld_cluster_u32(cluster_addr(hist0 + threadIdx.x, r));
      if (hist1) b[r] = ld_cluster_u32(cluster_addr(hist1 + threadIdx.x, r));
    }
  }
  u64 s = 0;
#pragma unroll
  for (int r = 0; r < kMaxCluster; ++r) s += hist1 ? (static_cast<u64>(a[r]) << 16) + b[r] : a[r];
  return s;
}

// The bin at which `above` and the bins' sums (one per thread, `mine`) first reach the
// target, or -1; its sum from the bins before it is in sh.found_above.
__device__ __noinline__ int find_bin(u64 mine, u64 target, u64 above) {
  static_assert(kBins == kThreads, "one bin per thread");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  u64 incl = warp_scan_u64(mine);
  __syncthreads();
  if (lane == 31) sh.scratch[warp] = incl;
  if (threadIdx.x == 0) sh.found_bin = -1;
  __syncthreads();
  incl += above;
#pragma unroll 1
  for (int w = 0; w < warp; ++w) incl += sh.scratch[w];
  if (incl >= target && incl - mine < target) {
    sh.found_bin = threadIdx.x;
    sh.found_above = incl - mine;
  }
  __syncthreads();
  return sh.found_bin;
}

// The bins, sh.found_bin to sh.found_hi, between which a prefix of the row should end by
// a sample's histogram (`mine` this thread's bin of it): where the sample's sums are
// within `margin` of `share` of its whole sum, or of `share` itself where it is above 1.
__device__ __noinline__ void find_bracket(u64 mine, float share, float margin) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, tid = threadIdx.x;
  u64 incl = warp_scan_u64(mine);
  __syncthreads();
  if (lane == 31) sh.scratch[warp] = incl;
  if (tid == 0) {
    sh.found_bin = 0;
    sh.found_hi = kBins - 1;
  }
  __syncthreads();
  u64 all = 0;
#pragma unroll 1
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) incl += sh.scratch[w];
    all += sh.scratch[w];
  }
  // (not so far up that a share near 1 takes in the whole tail)
  const float unit = share > 1.0f ? 1.0f : static_cast<float>(all);
  const float from = (share - margin) * unit;
  const float to = (share > 1.0f ? share + margin : fminf(share + margin, 1.0f - 0.125f * (1.0f - share))) * unit;
  const float below = static_cast<float>(incl - mine), upto = static_cast<float>(incl);
  if (below < from && upto >= from) sh.found_bin = tid;
  if (below < to && upto >= to) sh.found_hi = tid;
  __syncthreads();
}

// The first CTA fetches the CTAs' parts of a list: their tokens' number, or -1 if they
// are too many.  (Part of a longer agreement: a cluster barrier before and after.)
__device__ __noinline__ int fetch_list(float zm, float c) {
  static_assert(kListCap <= kThreads, "one thread per listed token");
  const int size = static_cast<int>(cluster_size()), tid = threadIdx.x;
  uint32_t n[kMaxCluster];
#pragma unroll
  for (int r = 0; r < kMaxCluster; ++r) n[r] = r < size ? ld_cluster_u32(cluster_addr(&sh.list_n, r)) : 0;
  int total = 0, cta = 0, at = 0;  // where this thread's token lies
#pragma unroll
  for (int r = 0; r < kMaxCluster; ++r) {
    const int m = static_cast<int>(min(n[r], kListCap + 1u));
    if (tid >= total && tid - total < m) {
      cta = r;
      at = tid - total;
    }
    total += m;
  }
  if (total > kListCap) return -1;
  if (tid < total) {
    const u64 key = ld_cluster_u64(cluster_addr(&sh.part[at], cta));
    sh.list[tid] = Listed{key, weight_of(tempered(key_value(key), zm, c))};
  }
  return total;
}

// Every listed token's rank (bits 48..) and the mass before it in the order (below
// 2^48) into sh.part, by comparing all with all, eight threads per token.
constexpr int kPerToken = 8;
__device__ __noinline__ void rank_list(int n) {
  const int lane = threadIdx.x & 31, sub = lane % kPerToken;
  __syncthreads();
#pragma unroll 1
  for (int i0 = (threadIdx.x >> 5) * (32 / kPerToken); i0 < n; i0 += kThreads / kPerToken) {  // (a warp's own share)
    const int i = i0 + lane / kPerToken;
    u64 above = 0;
    if (i < n) {
      const u64 key = sh.list[i].key;
#pragma unroll 4
      for (int j = sub; j < n; j += kPerToken) {
        const Listed o = sh.list[j];
        if (o.key > key) above += o.w + (1ull << 48);
      }
    }
#pragma unroll
    for (int o = 1; o < kPerToken; o <<= 1) above += __shfl_xor_sync(0xffffffffu, above, o);
    if (i < n && sub == 0) sh.part[i] = above;
  }
  __syncthreads();
}

__device__ __noinline__ void write_token(const Params& p, int row, int id, float t, u64 total) {
  p.ids[row] = id;
  if (p.logprobs) {
    const float k32 = __fmul_rn(__ll2float_rn(static_cast<long long>(total)), 2.3283064365386963e-10f);  // 2^-32
    p.logprobs[row] = __fsub_rn(__fmul_rn(t, 0.6931471805599453f), logf(k32));
  }
}

// The draw from the first CTA's list of n tokens.  top_k > 0: the mass that is wanted is
// worked out here, else it is `need`.
__device__ __noinline__ void draw_from_list(const Params& p, int row, int n, int top_k, float top_p, u64 need,
                                            float min_t, float uniform, float zm, float c) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  rank_list(n);
  if (warp == 0) {
    if (top_k > 0) {
      u64 mass = 0;
#pragma unroll 1
      for (int i = lane; i < n; i += 32)
        if (static_cast<int>(sh.part[i] >> 48) < top_k) mass += sh.list[i].w;
      mass = warp_sum_u64(mass);
      need = top_p < 1.0f ? mass_wanted(top_p, mass) : mass;
    }
    // the kept ones, closed up (each to a place at or before its own), and their mass
    u64 kept = 0;
    int m = 0;
#pragma unroll 1
    for (int i0 = 0; i0 < n; i0 += 32) {
      const int i = i0 + lane;
      Listed it{0, 0};
      bool keep = false;
      if (i < n) {
        it = sh.list[i];
        const u64 place = sh.part[i];
        keep = it.w > 0 && (place & 0xFFFFFFFFFFFFull) < need &&
               (top_k == 0 || static_cast<int>(place >> 48) < top_k) && tempered(key_value(it.key), zm, c) >= min_t;
      }
      const unsigned ones = __ballot_sync(0xffffffffu, keep);  // (every lane has read its token)
      if (keep) {
        kept += it.w;
        sh.list[m + __popc(ones & ((1u << lane) - 1u))] = it;
      }
      m += __popc(ones);
    }
    kept = warp_sum_u64(kept);
    const u64 r = draw_point(uniform, kept);
    if (lane == 0) {
      sh.count = m;
      sh.kept = kept;
      sh.point = r;
    }
  }
  __syncthreads();
  const int m = sh.count;
  const u64 r = sh.point;
  const int sub = lane % kPerToken;
#pragma unroll 1
  for (int i0 = warp * (32 / kPerToken); i0 < m; i0 += kThreads / kPerToken) {
    const int i = i0 + lane / kPerToken;
    u64 before = 0;
    Listed it{0, 0};
    if (i < m) {
      it = sh.list[i];
#pragma unroll 4
      for (int j = sub; j < m; j += kPerToken) {
        const Listed o = sh.list[j];
        // ids are complemented in the keys' low words
        if (static_cast<uint32_t>(o.key) > static_cast<uint32_t>(it.key)) before += o.w;
      }
    }
#pragma unroll
    for (int o = 1; o < kPerToken; o <<= 1) before += __shfl_xor_sync(0xffffffffu, before, o);
    if (i < m && sub == 0 && before <= r && r < before + it.w)
      write_token(p, row, key_id(it.key), tempered(key_value(it.key), zm, c), sh.kept);
  }
}

// Adds a logit to a histogram: its weight in two parts, or a count.
__device__ __forceinline__ void count_into(uint32_t (*hist)[kBins], int bin, bool by_mass, float t) {
  if (by_mass) {
    const u64 w = weight_of(t);
    atomicAdd(&hist[0][bin], static_cast<uint32_t>(w >> 16));
    atomicAdd(&hist[1][bin], static_cast<uint32_t>(w) & 0xFFFFu);
  } else {
    atomicAdd(&hist[0][bin], 1u);
  }
}

__device__ __forceinline__ void clear_hist(uint32_t (*hist)[kBins]) {
  __syncthreads();
  hist[0][threadIdx.x] = 0;
  hist[1][threadIdx.x] = 0;
  if (threadIdx.x == 0) sh.list_n = sh.extremes[0] = sh.extremes[1] = 0;
  __syncthreads();
}

// ---------------------------------------------------------------------------
// one row
// ---------------------------------------------------------------------------
template <typename T>
class RowSampler {
 public:
  static constexpr int kN = Vec<T>::kN;

  __device__ __forceinline__ RowSampler(const Params& p, int row) : p_(p), row_(row) {
    lane_ = threadIdx.x & 31;
    warp_ = threadIdx.x >> 5;
    parity_ = 0;
    sh.list_hist[threadIdx.x] = 0;
    if (threadIdx.x == 0) sh.list_n = 0;
    cluster_arrive();  // (waited for before these are counted up, or a word goes to another CTA)
    // (in flight while the row is loaded)
    temperature_ = p.f.temperature ? __ldg(p.f.temperature + row) : 1.0f;
    top_k_ = p.f.top_k ? __ldg(p.f.top_k + row) : 0;
    top_p_ = p.f.top_p ? __ldg(p.f.top_p + row) : 1.0f;
    min_p_ = p.f.min_p ? __ldg(p.f.min_p + row) : 0.0f;
    uniform_ = __ldg(p.uniforms + row);
    load();
  }

  // True: no CTA but the first has anything left to do or to be read.
  __device__ __forceinline__ bool run();

 private:
  const Params& p_;
  int row_, lane_, warp_, parity_;
  // this warp's part of the row: n_ vectors from data_, id0_ the id of their first element
  // (below 0 in a row's first vector)
  uint4* data_;
  int n_, id0_;
  float zm_, c_;
  float lane_max_;  // of this lane's logits
  float temperature_, top_p_, min_p_, uniform_;
  int top_k_;

  __device__ __forceinline__ void load();
  __device__ __forceinline__ float element(int j) const { return Vec<T>::to_float(reinterpret_cast<const T*>(data_)[j]); }
  __device__ __forceinline__ float t_of(float z) const { return tempered(z, zm_, c_); }
  __device__ __forceinline__ uint32_t max_over(uint32_t v) {
    parity_ ^= 1;
    return cluster_max(v, parity_);
  }
  __device__ __forceinline__ Sum sum_over(u64 v) {
    parity_ ^= 1;
    return cluster_sum(v, parity_);
  }
  // (no short cuts: these would be branches for every logit)
  static __device__ __forceinline__ bool kept_by(const Kept& k, float t, float z, int id) {
    return (t >= k.min_t) & ((z > k.z_cut) | ((z == k.z_cut) & (id <= k.id_cut)));
  }
  __device__ __forceinline__ bool is_kept(float z, int id, const Kept& k) const { return kept_by(k, t_of(z), z, id); }
  template <bool kEvery>
  __device__ __forceinline__ u64 warp_mass(const Kept& k);
  __device__ __forceinline__ void threshold(bool by_mass, u64 target, u64 total, float listed_t, u64 listed_mass,
                                            Kept* k);
  __device__ __forceinline__ void draw(const Kept& k);
  __device__ __forceinline__ void greedy();
  __device__ __forceinline__ bool from_list(int top_k, float top_p, float min_t, u64* mass, float* listed_t,
                                            u64* listed_mass);
  // Place of t on the scale of 0 .. kMinT, cut into kBins bins (kBins: no weight).
  __device__ __forceinline__ float place(float t) const {
    return t >= kMinT ? __fmul_rn(t, (kBins - 1) / kMinT) : kBins;
  }
  // Bin of a lane's maximum: over z itself, so that the histogram needs no maximum of the
  // row; the ends take what lies outside (kBins: -inf).
  static __device__ __forceinline__ int max_bin(float z) {
    const float x = fminf(fmaxf(kMaxBinsTop - z, 0.0f) * kMaxBinsPer, kBins - 1.0f);
    return z > -INFINITY ? static_cast<int>(x) : kBins;
  }
  __device__ __forceinline__ void count_max() {
    const int b = max_bin(lane_max_);
    if (b < kBins && (top_k_ > 0 || top_p_ < 1.0f)) atomicAdd(&sh.list_hist[b], 1u);
  }
  // The value whose order key without its constant low bits (kZeroBits) is `high`.
  static __device__ __forceinline__ float key_value_of(uint32_t high) {
    const uint32_t low = (1u << Vec<T>::kZeroBits) - 1u, key = high << Vec<T>::kZeroBits;
    return ord_f32(key & 0x80000000u ? key : key | low);
  }
  // f(z, j) for this warp's elements j, one per lane at a time; `kAtOnce` of them side by side
  template <int kAtOnce, typename F>
  __device__ __forceinline__ void for_each_element(F&& f) const {
    const int m = n_ * kN;
    int j = lane_;
    if (kAtOnce > 1) {
#pragma unroll 1
      for (; j + 32 * (kAtOnce - 1) < m; j += 32 * kAtOnce) {
        float z[kAtOnce];
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) z[u] = element(j + 32 * u);
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) f(z[u], j + 32 * u);
      }
    }
#pragma unroll 1
    for (; j < m; j += 32) f(element(j), j);
  }
};

// Copies this CTA's slice into shared memory: -inf stands for tokens that are
// not allowed, NaN, and the padding of the row's first and last vector.  A warp works
// on its own part of the slice alone.
template <typename T>
__device__ __forceinline__ void RowSampler<T>::load() {
  const int size = static_cast<int>(cluster_size()), rank = static_cast<int>(cluster_rank());
  const T* row = static_cast<const T*>(p_.logits) + static_cast<int64_t>(row_) * p_.row_stride;
  const int lead = static_cast<int>((reinterpret_cast<uintptr_t>(row) / sizeof(T)) % kN);  // elements before the row
  const uint4* base = reinterpret_cast<const uint4*>(row - lead);
  const int nvec = (lead + p_.V + kN - 1) / kN;
  const int per_cta = (nvec + size - 1) / size;
  const int cta0 = min(rank * per_cta, nvec), cta1 = min(cta0 + per_cta, nvec);
  const int per_warp = (cta1 - cta0 + kWarps - 1) / kWarps;
  const int v0 = min(cta0 + warp_ * per_warp, cta1), v1 = min(v0 + per_warp, cta1);
  data_ = row_data + (v0 - cta0);
  n_ = v1 - v0;
  id0_ = v0 * kN - lead;
  const uint32_t* mask =
      p_.f.allowed_mask ? p_.f.allowed_mask + static_cast<int64_t>(row_) * p_.f.mask_words : nullptr;
  // The vectors that lie in the row whole, [w0, w1) of this warp's, come by one bulk copy,
  // the first and the last of a row by element.
  const int w0 = lead > 0 && v0 == 0 ? 1 : 0, w1 = min(v1, (lead + p_.V) / kN) - v0;
  uint64_t* arrived = &sh.arrived[warp_];
  if (w1 > w0) {
    if (lane_ == 0) {
      const uint32_t bytes = static_cast<uint32_t>(w1 - w0) * 16u;
      mbar_init(arrived, 1);
      mbar_init_fence();
      mbar_arrive_expect_tx(arrived, bytes);
      bulk_load(data_ + w0, base + v0 + w0, bytes, arrived);
    }
    __syncwarp();
  }
  auto by_element = [&](int j) {
    const int v = id0_ + j;
    float z = -INFINITY;
    if (v >= 0 && v < p_.V && (!mask || ((mask[v >> 5] >> (v & 31)) & 1u))) z = Vec<T>::to_float(row[v]);
    reinterpret_cast<T*>(data_)[j] = Vec<T>::from_float(fmaxf(z, -INFINITY));  // (NaN becomes -inf)
  };
  const int after = max(w0, w1);  // vectors [w0, after) are whole, at most two are not
  if (lane_ < w0 * kN) by_element(lane_);
  if (after * kN + lane_ < n_ * kN) by_element(after * kN + lane_);
  __syncwarp();
  // A lane's maximum is that of its vectors: lane_, lane_ + 32, ...
  lane_max_ = -INFINITY;
  if (lane_ < w0) lane_max_ = Vec<T>::max_of(data_[lane_]);
#pragma unroll 1
  for (int i = after; i < n_; ++i)
    if (i % 32 == lane_) lane_max_ = fmaxf(lane_max_, Vec<T>::max_of(data_[i]));
  if (w1 <= w0) return;
  bool waited = false;
#pragma unroll 1
  for (int i0 = lane_; i0 < w1; i0 += 32 * kUnroll) {
    uint32_t allowed[kUnroll];  // the mask's words are in flight beside the logits
    if (mask) {
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int id = id0_ + (i0 + 32 * u) * kN, w = id >> 5;
        allowed[u] = 0;
        if (i0 + 32 * u >= w0 && i0 + 32 * u < w1)
          allowed[u] = __funnelshift_r(mask[w], (id & 31) + kN > 32 ? mask[w + 1] : 0u, id & 31);
      }
    }
    if (!waited) {
      if (!mbar_wait_limit(arrived, 0, p_.wait_ns)) {
        set_status(p_.dev_status, LMH_DS_TIMEOUT);
        mbar_wait(arrived, 0);  // (the copy lands before the CTA may leave)
      }
      waited = true;
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int i = i0 + 32 * u;
      if (i < w0 || i >= w1) continue;
      const uint4 x = data_[i];
      const uint4 y = Vec<T>::clean(mask ? Vec<T>::masked(x, allowed[u]) : x);
      if (x.x != y.x || x.y != y.y || x.z != y.z || x.w != y.w) data_[i] = y;
      lane_max_ = fmaxf(lane_max_, Vec<T>::max_of(y));
    }
  }
  __syncwarp();
}

// Sum of the weights of this warp's kept tokens (kEvery: of all), two logits an
// instruction where the arithmetic allows.
template <typename T>
template <bool kEvery>
__device__ __forceinline__ u64 RowSampler<T>::warp_mass(const Kept& k) {
  uint32_t hi = 0, lo = 0, n = 0;
  const float2 zm2 = make_float2(-zm_, -zm_), c2 = make_float2(c_, c_);
  const float2 minus = make_float2(-1.0f, -1.0f), add_hi = make_float2(kHiAdd, kHiAdd),
               sub_hi = make_float2(-kHiAdd, -kHiAdd), add_lo = make_float2(kLoAdd, kLoAdd);
#pragma unroll 1
  for (int i = lane_; i < n_; i += 32) {
    float z[kN];
    Vec<T>::widen(data_[i], z);
    const int id = id0_ + i * kN;
#pragma unroll
    for (int e = 0; e < kN; e += 2) {
      const float2 t = __fmul2_rn(__fadd2_rn(make_float2(z[e], z[e + 1]), zm2), c2);
      float2 w = make_float2(ex2_approx(t.x), ex2_approx(t.y));
      if (!kEvery) {
        w.x = kept_by(k, t.x, z[e], id + e) ? w.x : 0.0f;
        w.y = kept_by(k, t.y, z[e + 1], id + e + 1) ? w.y : 0.0f;
      }
      // weight_bits() of both
      const float2 h = __fadd2_rn(w, add_hi);
      const float2 l = __fadd2_rn(__ffma2_rn(__fadd2_rn(h, sub_hi), minus, w), add_lo);
      hi += __float_as_uint(h.x) + __float_as_uint(h.y);
      lo += __float_as_uint(l.x) + __float_as_uint(l.y);
    }
    n += kN;
  }
  return warp_sum_u64(weight_sum(hi, lo, n));
}

// Narrows k->z_cut, k->id_cut to the shortest prefix of the order whose count (or
// mass) reaches target >= 1.  A target above the total of the tokens with a weight
// leaves k alone.  By mass: `total` is that of the tokens that *k keeps so far (the sample
// is of these alone), of which the ones above listed_t (there or thereabouts: it is the
// sample that leaves them out) have listed_mass.
template <typename T>
__device__ __forceinline__ void RowSampler<T>::threshold(bool by_mass, u64 target, u64 total, float listed_t,
                                                         u64 listed_mass, Kept* k) {
  // The prefix ends at a t of [t0, t1], which is cut into kBins parts: by distinct values
  // where a 16-bit type has no more of them there, so that a part's mass is its count
  // times one weight, else linear in t.
  float t1 = INFINITY, t0 = kMinT, per_t = 0.0f;
  uint32_t key_top = 0;
  bool by_key = false;
  int part = -1;
  u64 above = 0;  // count or mass of what comes before the part
  auto inside = [&](float t) { return (t <= t1) & (t >= t0); };
  auto part_of = [&](float z, float t) -> int {
    const int b = by_key ? static_cast<int>(key_top - (f32_ord(z) >> Vec<T>::kZeroBits))
                         : static_cast<int>((fminf(t1, 0.0f) - t) * per_t);
    return min(max(b, 0), kBins - 1);
  };
  // The interval comes from a sample of the logits, with a margin; where that
  // was not enough (or the row is short), from all logits.
#pragma unroll 1
  for (int attempt = p_.V >= kSampleFromV ? 0 : 1; attempt < 2 && part < 0; ++attempt) {
    clear_hist(sh.hist[0]);
    const int step = attempt == 0 ? kSampleStep : 1;
#pragma unroll 1
    for (int j = lane_ * step; j < n_ * kN; j += 32 * step) {
      const float z = element(j), t = t_of(z);
      const int b = static_cast<int>(place(t));
      if (b < kBins && (attempt > 0 || ((t <= listed_t) & is_kept(z, id0_ + j, *k))))
        count_into(sh.hist[0], b, by_mass, t);
    }
    cluster_sync();
    const u64 bin_sum = gather_bin(sh.hist[0][0], by_mass ? sh.hist[0][1] : nullptr);
    int lo_bin, hi_bin;
    if (attempt == 0) {
      const float share = by_mass ? static_cast<float>(target - listed_mass) / static_cast<float>(total - listed_mass)
                                  : 1.0f + static_cast<float>(target) / kSampleStep;
      find_bracket(bin_sum, share, by_mass ? 0.08f : 16.0f + 0.05f * share);
      lo_bin = sh.found_bin;
      hi_bin = max(sh.found_hi, lo_bin);
    } else {
      lo_bin = hi_bin = find_bin(bin_sum, target, 0);
      if (lo_bin < 0) return;
    }
    // (a bin more on either side: the ends are not the bins' to the last bit)
    t1 = lo_bin <= 1 ? INFINITY : static_cast<float>(lo_bin - 1) * (kMinT / (kBins - 1));
    t0 = fmaxf(kMinT, static_cast<float>(hi_bin + 2) * (kMinT / (kBins - 1)));
    per_t = static_cast<float>(kBins) / (fminf(t1, 0.0f) - t0);
    if (Vec<T>::kZeroBits > 0) {
      // the interval in z, with room for the roundings of t: no z inside may miss the parts
      const float z1 = zm_ + fminf(t1, 0.0f) / c_, z0 = zm_ + t0 / c_;
      const float from = z0 - 1e-6f * (fabsf(zm_) + fabsf(z0));
      key_top = (f32_ord(z1 + 1e-6f * (fabsf(zm_) + fabsf(z1))) >> Vec<T>::kZeroBits) + 1;
      by_key = from > -INFINITY && key_top - (f32_ord(from) >> Vec<T>::kZeroBits) + 1 < kBins;
    }
    // The interval's parts, and the sum of what comes before it.
    clear_hist(sh.hist[1]);
    uint32_t hi = 0, lo = 0, n = 0;
#pragma unroll 1
    for (int i = lane_; i < n_; i += 32) {
      float z[kN];
      Vec<T>::widen(data_[i], z);
#pragma unroll
      for (int e = 0; e < kN; ++e) {
        const float t = t_of(z[e]);
        const float w = by_mass ? ex2_approx(t) : 1.0f;
        uint32_t h, l;
        weight_bits(t > t1 ? w : 0.0f, h, l);
        hi += h;
        lo += l;
        if (inside(t)) {
          const int b = part_of(z[e], t);
          if (by_mass && !by_key) {
            weight_bits(w, h, l);
            const u64 one = weight_sum(h, l, 1);
            atomicAdd(&sh.hist[1][0][b], static_cast<uint32_t>(one >> 16));
            atomicAdd(&sh.hist[1][1][b], static_cast<uint32_t>(one) & 0xFFFFu);
          } else {
            atomicAdd(&sh.hist[1][0][b], 1u);
          }
        }
      }
      n += kN;
    }
    u64 sum = weight_sum(hi, lo, n);
    if (!by_mass) sum >>= 32;
    above = sum_over(warp_sum_u64(sum)).all;
    if (above < target) {
      u64 mine = gather_bin(sh.hist[1][0], by_mass && !by_key ? sh.hist[1][1] : nullptr);
      if (by_mass && by_key) mine *= weight_of(t_of(key_value_of(key_top - threadIdx.x)));
      part = find_bin(mine, target, above);
      if (part >= 0) above = sh.found_above;
    }
  }
  if (part < 0) return;
  // The part's tokens: their number and extremes, and a list where they are not equals.
  uint32_t mine = 0, top = 0, bottom = 0;  // of the order keys, and of their complements
  if (by_key) {
    const float v = key_value_of(key_top - part);
#pragma unroll 1
    for (int i = lane_; i < n_; i += 32) {
      float z[kN];
      Vec<T>::widen(data_[i], z);
#pragma unroll
      for (int e = 0; e < kN; ++e) mine += z[e] == v ? 1 : 0;
    }
    top = f32_ord(v);
    bottom = ~top;
  } else {
    for_each_element<4>([&](float z, int j) {
      const float t = t_of(z);
      if (inside(t) && part_of(z, t) == part) {
        ++mine;
        top = max(top, f32_ord(z));
        bottom = max(bottom, ~f32_ord(z));
        const uint32_t at = atomicAdd(&sh.list_n, 1u);
        if (at < kListCap) sh.part[at] = make_key(z, id0_ + j);
      }
    });
  }
  mine = __reduce_add_sync(0xffffffffu, mine);
  top = __reduce_max_sync(0xffffffffu, top);
  bottom = __reduce_max_sync(0xffffffffu, bottom);
  if (lane_ == 0) {
    sh.warp_mass[warp_] = mine;
    if (by_key) atomicAdd(&sh.list_n, mine);
    atomicMax(&sh.extremes[0], top);
    atomicMax(&sh.extremes[1], bottom);
  }
  __syncthreads();
  const int size = static_cast<int>(cluster_size()), rank = static_cast<int>(cluster_rank());
  if (static_cast<int>(threadIdx.x) < size) {
    st_cluster_u64(cluster_addr(&sh.part_n[rank], threadIdx.x), sh.list_n);
    st_cluster_u64(cluster_addr(&sh.part_ends[rank], threadIdx.x),
                   (static_cast<u64>(sh.extremes[0]) << 32) | sh.extremes[1]);
  }
  cluster_sync();
  u64 n_all = 0, n_before = 0;
  top = bottom = 0;
#pragma unroll 1
  for (int r = 0; r < size; ++r) {
    n_all += sh.part_n[r];
    if (r < rank) n_before += sh.part_n[r];
    top = max(top, static_cast<uint32_t>(sh.part_ends[r] >> 32));
    bottom = max(bottom, static_cast<uint32_t>(sh.part_ends[r]));
  }
  float hi = ord_f32(top), lo = ord_f32(~bottom);
  if (lo < hi && n_all <= kListCap) {
    // The first CTA ranks the list and tells every CTA the last token of the prefix.
    if (rank == 0) {
      const int n = fetch_list(zm_, c_);
      rank_list(n);
      if (static_cast<int>(threadIdx.x) < n) {
        const u64 r = sh.part[threadIdx.x];
        const Listed it = sh.list[threadIdx.x];
        const u64 before = above + (by_mass ? r & 0xFFFFFFFFFFFFull : r >> 48);
        if (before < target && before + (by_mass ? it.w : 1) >= target)
          for (int q = 0; q < size; ++q) st_cluster_u64(cluster_addr(&sh.list_key, q), it.key);
      }
    }
    cluster_sync();
    k->z_cut = key_value(sh.list_key);
    k->id_cut = key_id(sh.list_key);
    return;
  }
  // Too many: go on with the interval of z between the extremes, or count off equals.
  const bool counted = !(lo < hi);
#pragma unroll 1
  for (int level = 0; lo < hi; ++level) {
    // Bins over [lo, hi], bin 0 at the top: linear in z first, which spreads a
    // row's logits evenly; linear in the order keys after eight levels or where
    // the width is no ordinary number (each such level takes 9 bits off the keys).
    const float width = __fsub_rn(hi, lo);
    const bool linear = level < 8 && width < 1e30f && width > 1e-30f;
    const float inv = linear ? __fdiv_rn(kBins - 1, width) : 0.0f;
    const uint32_t ord_hi = f32_ord(hi);
    const int shift = max(0, 32 - __clz(ord_hi - f32_ord(lo)) - 9);
    auto interval_bin = [&](float z) -> int {
      return linear ? min(static_cast<int>(__fmul_rn(__fsub_rn(hi, z), inv)), kBins - 1)
                    : static_cast<int>((ord_hi - f32_ord(z)) >> shift);
    };
    uint32_t(*hist)[kBins] = sh.hist[level & 1];
    clear_hist(hist);
    for_each_element<1>([&](float z, int) {
      if (z >= lo && z <= hi) count_into(hist, interval_bin(z), by_mass, t_of(z));
    });
    cluster_sync();
    const int b = find_bin(gather_bin(hist[0], by_mass ? hist[1] : nullptr), target, above);
    if (b < 0) return;  // (not reached: the target lies in [lo, hi])
    above = sh.found_above;
    // the bin's own extremes are the next interval
    top = bottom = 0;
    for_each_element<1>([&](float z, int) {
      if (z >= lo && z <= hi && interval_bin(z) == b) {
        top = max(top, f32_ord(z));
        bottom = max(bottom, ~f32_ord(z));
      }
    });
    hi = ord_f32(max_over(top));
    lo = ord_f32(~max_over(bottom));
  }
  // One value left, `hi`: of the tokens equal to it the first m in id order are kept.
  Sum ties{n_all, n_before};
  if (!counted) {
    mine = 0;
    for_each_element<1>([&](float z, int) { mine += z == hi ? 1 : 0; });
    mine = __reduce_add_sync(0xffffffffu, mine);
    ties = sum_over(mine);
  }
  u64 m = target - above;
  if (by_mass) {
    const u64 w = weight_of(t_of(hi));
    if (w == 0) return;  // (a target above the row's total)
    m = (m + w - 1) / w;
  }
  if (m > ties.all) return;
  // the warp that holds the m-th of them finds its id
  u64 before = ties.before;
#pragma unroll 1
  for (int w = 0; w < warp_; ++w) before += sh.warp_mass[w];
  uint32_t found = 0;
  if (before < m && m <= before + mine) {
    int left = static_cast<int>(m - before);
#pragma unroll 1
    for (int j0 = 0; j0 < n_ * kN; j0 += 32) {
      const bool tie = j0 + lane_ < n_ * kN && element(j0 + lane_) == hi;
      const unsigned ones = __ballot_sync(0xffffffffu, tie);
      if (tie && __popc(ones & ((2u << lane_) - 1u)) == left) found = static_cast<uint32_t>(id0_ + j0 + lane_) + 1;
      left -= __popc(ones);
      if (left <= 0) break;
    }
  }
  k->z_cut = hi;
  k->id_cut = static_cast<int>(max_over(found)) - 1;
}

// Draws from a list, if one can be made: true when the row is done.  With top-p alone
// *mass becomes the row's mass, and *listed_mass that of the tokens down to *listed_t
// (+inf and 0 when there are too many).
template <typename T>
__device__ __forceinline__ bool RowSampler<T>::from_list(int top_k, float top_p, float min_t, u64* mass,
                                                         float* listed_t, u64* listed_mass) {
  const u64 target = top_k > 0 ? top_k : kListTargetTopP;
  const int my_bin = max_bin(lane_max_);
  if (top_k == 0) *mass = sum_over(warp_mass<true>(Kept{})).all;
  // The last bin that is listed: the first at which the lanes' maxima reach the target.
  int last_bin = find_bin(gather_bin(sh.list_hist, nullptr), target, 0);
  if (last_bin < 0) last_bin = kBins - 1;  // (all there are)
  if (__any_sync(0xffffffffu, my_bin <= last_bin)) {
    // vectors whose maximum reaches it, then their elements side by side
#pragma unroll 1
    for (int i0 = 0; i0 < n_; i0 += 32) {
      const int i = i0 + lane_;
      unsigned hits = __ballot_sync(0xffffffffu, i < n_ && max_bin(i < n_ ? Vec<T>::max_of(data_[i]) : 0.0f) <= last_bin);
#pragma unroll 1
      for (; hits != 0; hits &= hits - 1) {
        const int j = (i0 + __ffs(hits) - 1) * kN + lane_;
        if (lane_ >= kN) continue;
        const float z = element(j);
        if (max_bin(z) > last_bin) continue;
        const uint32_t at = atomicAdd(&sh.list_n, 1u);
        if (at < kListCap) sh.part[at] = make_key(z, id0_ + j);
      }
    }
  }
  cluster_sync();
  // The first CTA fetches the parts and says whether they will do.
  if (cluster_rank() == 0) {
    u64 need = 0, have = 0;
    const int total = fetch_list(zm_, c_);
    bool ok = total >= 0;
    if (ok && top_k == 0) {
      need = mass_wanted(top_p, *mass);
      // (a thread's token is the one that it fetched)
      have = block_sum_u64(static_cast<int>(threadIdx.x) < total ? sh.list[threadIdx.x].w : 0);
      ok = have >= need;
    }
    // its word to every CTA; it does not wait for them where they have nothing left to do
    const int said = ok ? 1 : total < 0 ? 0 : 2;
    if (threadIdx.x < cluster_size()) {
      st_cluster_u64(cluster_addr(&sh.list_mass, threadIdx.x), have);
      st_cluster_u32(cluster_addr(&sh.list_ok, threadIdx.x), said);
    }
    cluster_arrive();
    if (ok) {
      draw_from_list(p_, row_, total, top_k, top_p, need, min_t, uniform_, zm_, c_);
      cluster_wait();
      return true;
    }
    cluster_wait();
  } else {
    cluster_sync();
  }
  if (sh.list_ok == 2) {
    *listed_t = t_of(kMaxBinsTop - static_cast<float>(last_bin + 1) / kMaxBinsPer);
    *listed_mass = sh.list_mass;
  }
  return sh.list_ok == 1;
}

// The token at the given point of the kept tokens' mass, in id order.
template <typename T>
__device__ __forceinline__ void RowSampler<T>::draw(const Kept& k) {
  const u64 mine =
      k.z_cut > -INFINITY || k.min_t > -INFINITY ? warp_mass<false>(k) : warp_mass<true>(k);
  const Sum sum = sum_over(mine);
  const u64 r = draw_point(uniform_, sum.all);
  u64 before = sum.before;
#pragma unroll 1
  for (int w = 0; w < warp_; ++w) before += sh.warp_mass[w];
  if (r < before || r >= before + mine) return;
  u64 left = r - before;  // mass to pass within this warp's vectors
#pragma unroll 1
  for (int i0 = 0; i0 < n_; i0 += 32) {
    const int i = i0 + lane_;
    u64 w = 0;
    if (i < n_)
#pragma unroll 2
      for (int j = i * kN; j < (i + 1) * kN; ++j) {
        const float z = element(j);
        if (is_kept(z, id0_ + j, k)) w += weight_of(t_of(z));
      }
    const u64 incl = warp_scan_u64(w);
    const u64 all = __shfl_sync(0xffffffffu, incl, 31);
    if (left < all) {
      if (incl - w <= left && left < incl) {
        u64 at = incl - w;
#pragma unroll 1
        for (int j = i * kN; j < (i + 1) * kN; ++j) {
          const float z = element(j);
          if (!is_kept(z, id0_ + j, k)) continue;
          at += weight_of(t_of(z));
          if (left < at) {
            write_token(p_, row_, id0_ + j, t_of(z), sum.all);
            break;
          }
        }
      }
      return;
    }
    left -= all;
  }
}

// The first token whose logit is the row's maximum.
template <typename T>
__device__ __forceinline__ void RowSampler<T>::greedy() {
  uint32_t first = 0;  // complemented id
  if (lane_max_ == zm_) {
#pragma unroll 1
    for (int i = lane_; i < n_ && first == 0; i += 32) {
      if (Vec<T>::max_of(data_[i]) != zm_) continue;
#pragma unroll 1
      for (int j = (i + 1) * kN - 1; j >= i * kN; --j)
        if (element(j) == zm_) first = ~static_cast<uint32_t>(id0_ + j);
    }
  }
  first = max_over(first);
  if (cluster_rank() == 0 && threadIdx.x == 0) {
    p_.ids[row_] = static_cast<int32_t>(~first);
    if (p_.logprobs) p_.logprobs[row_] = 0.0f;
  }
}

template <typename T>
__device__ __forceinline__ bool RowSampler<T>::run() {
  cluster_wait();  // every CTA of the cluster has started
  count_max();
  zm_ = ord_f32(max_over(f32_ord(lane_max_)));
  if (zm_ == -INFINITY) {
    if (cluster_rank() == 0 && threadIdx.x == 0) {
      p_.ids[row_] = -1;
      if (p_.logprobs) p_.logprobs[row_] = __int_as_float(0x7FC00000);
      set_status(p_.dev_status, LMH_DS_NO_ALLOWED_TOKEN);
    }
    return false;
  }
  if (zm_ == INFINITY) {  // only the +inf tokens are left, as equals
    float m = -INFINITY;
    for_each_element<1>([&](float z, int j) {
      const float y = z == INFINITY ? 0.0f : -INFINITY;
      reinterpret_cast<T*>(data_)[j] = Vec<T>::from_float(y);
      m = fmaxf(m, y);
    });
    __syncwarp();
    // (the lanes of a warp that holds one may all look for it)
    lane_max_ = __any_sync(0xffffffffu, m == 0.0f) ? 0.0f : -INFINITY;
    zm_ = 0.0f;
    __syncthreads();
    sh.list_hist[threadIdx.x] = 0;
    __syncthreads();
    count_max();
    cluster_sync();
  }
  if (!(temperature_ > 0.0f)) {
    greedy();
    return false;
  }
  c_ = fminf(fmaxf(__fmul_rn(__frcp_rn(temperature_), kLog2e), 1.1754944e-38f), 3.402823466e+38f);

  Kept k{-INFINITY, -INFINITY, INT32_MAX};
  const int top_k = top_k_ > 0 && top_k_ < p_.V ? top_k_ : 0;
  const float min_t = min_p_ > 0.0f ? fminf(log2f(min_p_), 0.0f) : -INFINITY;
  u64 mass = 0, listed_mass = 0;
  float listed_t = INFINITY;
  bool have_mass = false;
  if (top_k > 0 ? top_k <= kListTarget : top_p_ < 1.0f) {
    if (from_list(top_k, top_p_, min_t, &mass, &listed_t, &listed_mass)) return true;
    have_mass = top_k == 0;
  }
#pragma unroll 1
  for (int by_mass = top_k > 0 ? 0 : 1; by_mass < (top_p_ < 1.0f ? 2 : 1); ++by_mass) {
    if (by_mass && !have_mass) mass = sum_over(warp_mass<false>(k)).all;
    threshold(by_mass != 0, by_mass ? mass_wanted(top_p_, mass) : static_cast<u64>(top_k), mass, listed_t,
              listed_mass, &k);
  }
  k.min_t = min_t;
  draw(k);
  return false;
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 2) sample_logits_kernel(const __grid_constant__ Params p) {
  pdl_wait();
  // (no early launch of the next kernel)
  RowSampler<T> s(p, static_cast<int>(blockIdx.x / cluster_size()));
  const bool first_only = s.run();
  // No CTA leaves while another may still read its shared memory; after a draw from a
  // list the others need not wait for the first, and make room for the next row.
  cluster_arrive();
  if (!first_only || cluster_rank() == 0) cluster_wait();
}

template <typename T>
cudaError_t set_up() {
  cudaFuncAttributes a{};
  cudaError_t e = cudaFuncGetAttributes(&a, sample_logits_kernel<T>);
  if (e != cudaSuccess) return e;
  return cudaFuncSetAttribute(sample_logits_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              227 * 1024 - static_cast<int>(a.sharedSizeBytes));
}

template <typename T>
cudaError_t launch(const Params& p, int num_sms, cudaStream_t stream) {
  // Largest slice of a row in one CTA: as many vectors as the kernel's own split.
  auto slice_bytes = [&](int cl) {
    const int nvec = (p.V + 2 * Vec<T>::kN - 2) / Vec<T>::kN;
    return static_cast<size_t>((nvec + cl - 1) / cl) * 16;
  };
  // More CTAs per row until a slice leaves room for two or three CTAs per SM and,
  // while the rows do not fill the GPU, until a slice is down to 8 Ki logits.
  int cl = 1;
  while (cl < kMaxCluster && (slice_bytes(cl) > 64 * 1024 || (p.rows * cl < num_sms && p.V / cl > 8192))) cl *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.rows) * cl);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = slice_bytes(cl);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cl;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, sample_logits_kernel<T>, p);
}

}  // namespace

cudaError_t sample_logits_setup() {
  cudaError_t e = set_up<float>();
  if (e == cudaSuccess) e = set_up<__nv_bfloat16>();
  if (e == cudaSuccess) e = set_up<__half>();
  return e;
}

cudaError_t launch_sample_logits(const void* logits, lmh_dtype dtype, int rows, int V, int64_t row_stride,
                                 const lmh_filters& f, const float* uniforms, int32_t* ids, float* logprobs,
                                 uint32_t* dev_status, int num_sms, cudaStream_t stream) {
  const Params p{logits, row_stride, rows, V, f, uniforms, ids, logprobs, dev_status, wait_limit_ns()};
  if (dtype == LMH_F32) return launch<float>(p, num_sms, stream);
  if (dtype == LMH_BF16) return launch<__nv_bfloat16>(p, num_sms, stream);
  return launch<__half>(p, num_sms, stream);
}

}  // namespace lmh
