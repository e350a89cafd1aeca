// sample_logits.cu -- one token per row with temperature, top-k, top-p and
// min-p from one given uniform number (lmh_sample_from_logits).
//
// A row belongs to a thread-block cluster.  Its CTAs hold the row in their
// shared memory (a contiguous slice of the ids each), so HBM is read once and
// every later pass -- the maximum, the sum of the weights, the searches for the
// top-k and top-p thresholds, the draw -- runs on chip.
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
//   maxima over t gives a bound that at least k tokens reach (128 for top-p alone),
//   few more than that do, and only lanes whose maximum reaches it look at their
//   logits again.  The tokens that reach it go to the cluster's first CTA, which ranks
//   them by counting: with n tokens, n^2 comparisons give every token its rank and the
//   mass before it.  This holds for k up to kListTarget, and for top-p wherever the
//   listed tokens have the mass that is asked for.
// - A threshold (z, id) otherwise: every token with a larger logit is kept, and those
//   equal to it up to that id.  It is the last token of the prefix of the order (z
//   descending, id ascending) that reaches a count (top-k) or a mass (top-p): a
//   histogram of all logits over t, one of the bin that holds the end over its 512th
//   parts, and a list of what is left there.  Where that is too long (many equal
//   logits), histograms over ever smaller intervals of z go on until one value is left,
//   whose tokens are counted off in id order.
// Tokens of weight 0 (t < -33) can be left out of either: no draw falls on them and no
// sum changes.
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
constexpr int kUnroll = 4;             // vectors of a lane whose mask words are in flight at once
constexpr float kHiAdd = 768.0f;             // 1.5 * 2^9: unit 2^-14
constexpr float kLoAdd = 0.0029296875f;      // 1.5 * 2^-9: unit 2^-32
constexpr uint32_t kHiBits = 0x44400000u;    // of kHiAdd
constexpr uint32_t kLoBits = 0x3B400000u;    // of kLoAdd
constexpr int kHiShift = 18;                 // 2^-14 in units of 2^-32

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
__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ unsigned long long ld_cluster_u64(uint32_t a) {
  unsigned long long v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(a) : "memory");
  return v;
}

// f(rank, *p in CTA `rank`) for every CTA of the cluster, in rank order; all the loads
// are in flight before the first is used.
template <typename F>
__device__ __forceinline__ void for_each_cta(const uint32_t* p, uint32_t size, F&& f) {
  uint32_t v[kMaxCluster];
#pragma unroll
  for (int r = 0; r < kMaxCluster; ++r)
    if (r < static_cast<int>(size)) v[r] = ld_cluster_u32(cluster_addr(p, r));
#pragma unroll
  for (int r = 0; r < kMaxCluster; ++r)
    if (r < static_cast<int>(size)) f(static_cast<uint32_t>(r), v[r]);
}
template <typename F>
__device__ __forceinline__ void for_each_cta(const unsigned long long* p, uint32_t size, F&& f) {
  unsigned long long v[kMaxCluster];
#pragma unroll
  for (int r = 0; r < kMaxCluster; ++r)
    if (r < static_cast<int>(size)) v[r] = ld_cluster_u64(cluster_addr(p, r));
#pragma unroll
  for (int r = 0; r < kMaxCluster; ++r)
    if (r < static_cast<int>(size)) f(static_cast<uint32_t>(r), v[r]);
}

// ---------------------------------------------------------------------------
// logits in 16-byte vectors
// ---------------------------------------------------------------------------
template <typename T>
struct Vec;  // kN elements a vector; widen and narrow are exact
template <>
struct Vec<float> {
  static constexpr int kN = 4;
  static __device__ __forceinline__ void widen(const uint4& x, float (&z)[4]) {
    z[0] = __uint_as_float(x.x);
    z[1] = __uint_as_float(x.y);
    z[2] = __uint_as_float(x.z);
    z[3] = __uint_as_float(x.w);
  }
  static __device__ __forceinline__ uint4 narrow(const float (&z)[4]) {
    return make_uint4(__float_as_uint(z[0]), __float_as_uint(z[1]), __float_as_uint(z[2]), __float_as_uint(z[3]));
  }
  static __device__ __forceinline__ float to_float(float x) { return x; }
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
  static __device__ __forceinline__ void widen(const uint4& x, float (&z)[8]) {
    const uint32_t u[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      z[2 * i] = __uint_as_float(u[i] << 16);
      z[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
    }
  }
  static __device__ __forceinline__ uint4 narrow(const float (&z)[8]) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      u[i] = (__float_as_uint(z[2 * i]) >> 16) | (__float_as_uint(z[2 * i + 1]) & 0xFFFF0000u);
    return make_uint4(u[0], u[1], u[2], u[3]);
  }
  static __device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
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
  static __device__ __forceinline__ void widen(const uint4& x, float (&z)[8]) {
    const uint32_t u[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
      z[2 * i] = f.x;
      z[2 * i + 1] = f.y;
    }
  }
  static __device__ __forceinline__ uint4 narrow(const float (&z)[8]) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2 h = __floats2half2_rn(z[2 * i], z[2 * i + 1]);
      u[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return make_uint4(u[0], u[1], u[2], u[3]);
  }
  static __device__ __forceinline__ float to_float(__half x) { return __half2float(x); }
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
__device__ __forceinline__ long long weight_sum(uint32_t hi, uint32_t lo, uint32_t n) {
  const long long h = static_cast<int32_t>(hi - n * kHiBits), l = static_cast<int32_t>(lo - n * kLoBits);
  return (h << kHiShift) + l;
}
__device__ __forceinline__ long long weight_of(float t) {
  uint32_t hi, lo;
  weight_bits(ex2_approx(t), hi, lo);
  return weight_sum(hi, lo, 1);
}

__device__ __forceinline__ long long warp_sum_i64(long long v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

__device__ __forceinline__ unsigned long long warp_sum_u64(unsigned long long v) {
  return static_cast<unsigned long long>(warp_sum_i64(static_cast<long long>(v)));
}

// The mass that top-p asks for: max(1, ceil(p * mass)).
__device__ __forceinline__ unsigned long long mass_wanted(float top_p, unsigned long long mass) {
  const double x = ceil(__dmul_rn(static_cast<double>(top_p), static_cast<double>(static_cast<long long>(mass))));
  return x >= 1.0 ? static_cast<unsigned long long>(x) : 1ull;
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
  unsigned long long key;
  unsigned long long w;
};

struct Shared {
  // read by the other CTAs of the cluster
  uint32_t slot_u32[2];
  unsigned long long slot_u64[2];
  uint32_t list_hist[kBins];
  uint32_t list_n;
  int list_ok;
  unsigned long long list_key;
  union {
    uint32_t hist[2][2][kBins];            // [level parity][high, low part or count][bin]
    struct {
      unsigned long long part[kListCap];   // this CTA's part of a list: keys (over hist[0])
      Listed list[kListCap];               // the first CTA's list (over hist[1])
    };
  };
  // this CTA's own
  uint32_t scratch_u32[kWarps];
  unsigned long long scratch_u64[kWarps];
  unsigned long long warp_mass[kWarps];
  unsigned long long found_above;
  int found_bin;
  uint32_t count;
  unsigned long long kept, point;
  uint64_t arrived[kWarps];  // barriers: a warp's part of the row is there
};

// One row's slice in one CTA.
template <typename T>
struct Slice {
  uint4* data;        // this warp's vectors: data[i], i = lane, lane + 32, ...
  int n;              // vectors of this warp
  int id0;            // id of element 0 of data[0] (may be below 0 in a row's first vector)
  int lane;
};

template <typename T, typename F>
__device__ __forceinline__ void for_each_vector(const Slice<T>& s, F&& f) {
  for (int i = s.lane; i < s.n; i += 32) {
    float z[Vec<T>::kN];
    Vec<T>::widen(s.data[i], z);
    f(z, s.id0 + i * Vec<T>::kN);
  }
}

template <typename T>
class RowSampler {
 public:
  static constexpr int kN = Vec<T>::kN;

  __device__ RowSampler(const Params& p, Shared& sh, uint4* data, int row)
      : p_(p), sh_(sh), row_(row), rank_(cluster_rank()), size_(cluster_size()) {
    tid_ = threadIdx.x;
    lane_ = tid_ & 31;
    warp_ = tid_ >> 5;
    parity_ = 0;
    for (int b = tid_; b < kBins; b += kThreads) sh_.list_hist[b] = 0;
    if (tid_ == 0) sh_.list_n = 0;
    // (in flight while the row is loaded)
    temperature_ = p.f.temperature ? __ldg(p.f.temperature + row) : 1.0f;
    top_k_ = p.f.top_k ? __ldg(p.f.top_k + row) : 0;
    top_p_ = p.f.top_p ? __ldg(p.f.top_p + row) : 1.0f;
    min_p_ = p.f.min_p ? __ldg(p.f.min_p + row) : 0.0f;
    uniform_ = __ldg(p.uniforms + row);
    load(data);
  }

  // True: no CTA but the first has anything left to do or to be read.
  __device__ bool run();

 private:
  const Params& p_;
  Shared& sh_;
  int row_, tid_, lane_, warp_;
  uint32_t rank_, size_;
  int parity_;
  Slice<T> s_;
  float zm_, c_;
  float lane_max_;  // of this lane's logits
  float temperature_, top_p_, min_p_, uniform_;
  int top_k_;

  __device__ void load(uint4* data);
  // max / min / sum over the cluster (every thread gets the result)
  __device__ uint32_t reduce_max_u32(uint32_t v);
  __device__ unsigned long long reduce_sum_u64(unsigned long long v, unsigned long long* before);
  __device__ bool is_kept(float z, int id, const Kept& k) const {
    return tempered(z, zm_, c_) >= k.min_t && (z > k.z_cut || (z == k.z_cut && id <= k.id_cut));
  }
  enum { kAll, kMinTOnly, kThreshold };
  template <int kCase>
  __device__ unsigned long long warp_mass_case(const Kept& k);
  __device__ unsigned long long warp_kept_mass(const Kept& k);
  __device__ int find_bin(const uint32_t (*hist)[kBins], bool by_mass, unsigned long long target,
                          unsigned long long* above);
  __device__ void count_into(uint32_t (*hist)[kBins], int bin, bool by_mass, float z);
  __device__ int fetch_list();
  __device__ unsigned long long rank_list(int n);
  __device__ void threshold(bool by_mass, unsigned long long target, Kept* k);
  __device__ void draw(const Kept& k);
  __device__ void greedy();
  __device__ unsigned long long block_sum_u64(unsigned long long v);
  __device__ bool from_list(int top_k, float top_p, float min_t, unsigned long long* mass);
  __device__ void draw_from_list(int n, int top_k, unsigned long long need, float min_t);
  __device__ void write(int id, float z, unsigned long long total);
  // Place of z on the scale of t = 0 .. kMinT, cut into kBins parts (kBins and more:
  // no weight), and its part.
  __device__ float list_place(float z) const {
    const float t = tempered(z, zm_, c_);
    return t >= kMinT ? __fmul_rn(t, (kBins - 1) / kMinT) : kBins;
  }
  __device__ int list_bin(float z) const { return static_cast<int>(list_place(z)); }
};

// Copies this CTA's slice into shared memory: -inf stands for tokens that are
// not allowed, NaN, and the padding of the row's first and last vector.  A warp works
// on its own part of the slice alone, and a lane writes only what it reads back itself.
template <typename T>
__device__ void RowSampler<T>::load(uint4* data) {
  const T* row = static_cast<const T*>(p_.logits) + static_cast<int64_t>(row_) * p_.row_stride;
  const int lead = static_cast<int>((reinterpret_cast<uintptr_t>(row) / sizeof(T)) % kN);  // elements before the row
  const uint4* base = reinterpret_cast<const uint4*>(row - lead);
  const int nvec = (lead + p_.V + kN - 1) / kN;
  const int per_cta = (nvec + static_cast<int>(size_) - 1) / static_cast<int>(size_);
  const int cta0 = min(static_cast<int>(rank_) * per_cta, nvec), cta1 = min(cta0 + per_cta, nvec);
  const int per_warp = (cta1 - cta0 + kWarps - 1) / kWarps;
  const int v0 = min(cta0 + warp_ * per_warp, cta1), v1 = min(v0 + per_warp, cta1);
  s_.data = data + (v0 - cta0);
  s_.n = v1 - v0;
  s_.id0 = v0 * kN - lead;
  s_.lane = lane_;
  const uint32_t* mask =
      p_.f.allowed_mask ? p_.f.allowed_mask + static_cast<int64_t>(row_) * p_.f.mask_words : nullptr;
  // The vectors that lie in the row whole come by one bulk copy per warp, the first and
  // the last of a row by element.
  const int whole0 = max(v0, lead > 0 ? 1 : 0), whole1 = min(v1, (lead + p_.V) / kN);
  const uint32_t bytes = whole1 > whole0 ? static_cast<uint32_t>(whole1 - whole0) * 16u : 0u;
  uint64_t* arrived = &sh_.arrived[warp_];
  if (bytes > 0) {
    if (lane_ == 0) {
      mbar_init(arrived, 1);
      mbar_init_fence();
      mbar_arrive_expect_tx(arrived, bytes);
      bulk_load(s_.data + (whole0 - v0), base + whole0, bytes, arrived);
    }
    __syncwarp();
  }
  lane_max_ = -INFINITY;
  bool waited = bytes == 0;
  for (int i0 = lane_; i0 < s_.n; i0 += 32 * kUnroll) {
    uint32_t allowed[kUnroll];  // the mask's words are in flight beside the logits
    if (mask) {
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int i = i0 + 32 * u;
        const int id = s_.id0 + i * kN, w = id >> 5;
        allowed[u] = 0xFFFFFFFFu;
        if (i < s_.n && id >= 0 && id + kN <= p_.V)
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
      if (i >= s_.n) continue;
      const int id = s_.id0 + i * kN;
      uint4 x, y;
      if (id >= 0 && id + kN <= p_.V) {
        x = s_.data[i];
        y = Vec<T>::clean(mask ? Vec<T>::masked(x, allowed[u]) : x);
        if (x.x != y.x || x.y != y.y || x.z != y.z || x.w != y.w) s_.data[i] = y;
      } else {
        float z[kN];
#pragma unroll
        for (int e = 0; e < kN; ++e) {
          const int v = id + e;
          z[e] = -INFINITY;
          if (v >= 0 && v < p_.V && (!mask || ((mask[v >> 5] >> (v & 31)) & 1u))) z[e] = Vec<T>::to_float(row[v]);
        }
        y = Vec<T>::clean(Vec<T>::narrow(z));
        s_.data[i] = y;
      }
      lane_max_ = fmaxf(lane_max_, Vec<T>::max_of(y));
    }
  }
}

template <typename T>
__device__ uint32_t RowSampler<T>::reduce_max_u32(uint32_t v) {
  v = __reduce_max_sync(0xffffffffu, v);
  if (lane_ == 0) sh_.scratch_u32[warp_] = v;
  __syncthreads();
  if (warp_ == 0) {
    const uint32_t m = __reduce_max_sync(0xffffffffu, lane_ < kWarps ? sh_.scratch_u32[lane_] : 0u);
    if (lane_ == 0) sh_.slot_u32[parity_] = m;
  }
  cluster_sync();
  uint32_t m = 0;
  for_each_cta(&sh_.slot_u32[parity_], size_, [&](uint32_t, uint32_t v) { m = max(m, v); });
  parity_ ^= 1;
  return m;
}

// Sum over the cluster of one value per warp (lane 0's); *before: the sum over
// the CTAs of lower rank.  Leaves the warps' values in sh_.warp_mass.
template <typename T>
__device__ unsigned long long RowSampler<T>::reduce_sum_u64(unsigned long long v, unsigned long long* before) {
  __syncthreads();
  if (lane_ == 0) sh_.warp_mass[warp_] = v;
  __syncthreads();
  if (warp_ == 0) {
    const long long m = warp_sum_i64(lane_ < kWarps ? static_cast<long long>(sh_.warp_mass[lane_]) : 0);
    if (lane_ == 0) sh_.slot_u64[parity_] = static_cast<unsigned long long>(m);
  }
  cluster_sync();
  unsigned long long all = 0, b = 0;
  for_each_cta(&sh_.slot_u64[parity_], size_, [&](uint32_t r, unsigned long long m) {
    if (r < rank_) b += m;
    all += m;
  });
  parity_ ^= 1;
  *before = b;
  return all;
}

// Sum of the weights of this warp's kept tokens.  Two logits an instruction where the
// arithmetic allows; the three cases differ in what has to be compared.
template <typename T>
template <int kCase>
__device__ unsigned long long RowSampler<T>::warp_mass_case(const Kept& k) {
  uint32_t hi = 0, lo = 0, n = 0;
  const float2 zm2 = make_float2(-zm_, -zm_), c2 = make_float2(c_, c_);
  const float2 minus = make_float2(-1.0f, -1.0f), add_hi = make_float2(kHiAdd, kHiAdd),
               sub_hi = make_float2(-kHiAdd, -kHiAdd), add_lo = make_float2(kLoAdd, kLoAdd);
#pragma unroll 2
  for (int i = lane_; i < s_.n; i += 32) {
    float z[kN];
    Vec<T>::widen(s_.data[i], z);
    const int id = s_.id0 + i * kN;
#pragma unroll
    for (int e = 0; e < kN; e += 2) {
      const float2 t = __fmul2_rn(__fadd2_rn(make_float2(z[e], z[e + 1]), zm2), c2);
      float2 w = make_float2(ex2_approx(t.x), ex2_approx(t.y));
      if (kCase >= kMinTOnly) {
        if (!(t.x >= k.min_t)) w.x = 0.0f;
        if (!(t.y >= k.min_t)) w.y = 0.0f;
      }
      if (kCase == kThreshold) {
        if (!(z[e] > k.z_cut || (z[e] == k.z_cut && id + e <= k.id_cut))) w.x = 0.0f;
        if (!(z[e + 1] > k.z_cut || (z[e + 1] == k.z_cut && id + e + 1 <= k.id_cut))) w.y = 0.0f;
      }
      // weight_bits() of both
      const float2 h = __fadd2_rn(w, add_hi);
      const float2 l = __fadd2_rn(__ffma2_rn(__fadd2_rn(h, sub_hi), minus, w), add_lo);
      hi += __float_as_uint(h.x) + __float_as_uint(h.y);
      lo += __float_as_uint(l.x) + __float_as_uint(l.y);
    }
    n += kN;
  }
  return warp_sum_u64(static_cast<unsigned long long>(weight_sum(hi, lo, n)));
}

template <typename T>
__device__ unsigned long long RowSampler<T>::warp_kept_mass(const Kept& k) {
  if (k.z_cut > -INFINITY) return warp_mass_case<kThreshold>(k);
  return k.min_t > -INFINITY ? warp_mass_case<kMinTOnly>(k) : warp_mass_case<kAll>(k);
}

// The bin of the cluster's histograms at which `above` and the bins' counts (or
// masses) first reach the target, or -1; *above grows by the bins before it.  For all
// threads of all CTAs, each CTA for itself.
template <typename T>
__device__ int RowSampler<T>::find_bin(const uint32_t (*hist)[kBins], bool by_mass, unsigned long long target,
                                       unsigned long long* above) {
  static_assert(kBins == kThreads, "one bin per thread");
  unsigned long long mine = 0;
  for_each_cta(&hist[0][tid_], size_, [&](uint32_t, uint32_t h) {
    mine += by_mass ? static_cast<unsigned long long>(h) << 16 : h;
  });
  if (by_mass) for_each_cta(&hist[1][tid_], size_, [&](uint32_t, uint32_t h) { mine += h; });
  unsigned long long incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned long long t = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane_ >= o) incl += t;
  }
  if (lane_ == 31) sh_.scratch_u64[warp_] = incl;
  if (tid_ == 0) sh_.found_bin = -1;
  __syncthreads();
  incl += *above;
  for (int w = 0; w < warp_; ++w) incl += sh_.scratch_u64[w];
  if (incl >= target && incl - mine < target) {
    sh_.found_bin = tid_;
    sh_.found_above = incl - mine;
  }
  __syncthreads();
  if (sh_.found_bin >= 0) *above = sh_.found_above;
  return sh_.found_bin;
}

template <typename T>
__device__ void RowSampler<T>::count_into(uint32_t (*hist)[kBins], int bin, bool by_mass, float z) {
  if (by_mass) {
    const unsigned long long w = static_cast<unsigned long long>(weight_of(tempered(z, zm_, c_)));
    atomicAdd(&hist[0][bin], static_cast<uint32_t>(w >> 16));
    atomicAdd(&hist[1][bin], static_cast<uint32_t>(w) & 0xFFFFu);
  } else {
    atomicAdd(&hist[0][bin], 1u);
  }
}

// The first CTA fetches the CTAs' parts of a list: their tokens' number, or -1 if they
// are too many.  (Part of a longer agreement: a cluster barrier before and after.)
template <typename T>
__device__ int RowSampler<T>::fetch_list() {
  static_assert(kListCap <= kThreads, "one thread per listed token");
  uint32_t total = 0, cta = 0, at = 0;  // where this thread's token lies
  for_each_cta(&sh_.list_n, size_, [&](uint32_t r, uint32_t m) {
    if (static_cast<uint32_t>(tid_) >= total && static_cast<uint32_t>(tid_) - total < m) {
      cta = r;
      at = tid_ - total;
    }
    total += min(m, kListCap + 1u);
  });
  if (total > kListCap) return -1;
  if (static_cast<uint32_t>(tid_) < total) {
    const unsigned long long key = ld_cluster_u64(cluster_addr(&sh_.part[at], cta));
    sh_.list[tid_] = Listed{key, static_cast<unsigned long long>(weight_of(tempered(key_value(key), zm_, c_)))};
  }
  return static_cast<int>(total);
}

// Every listed token's rank (bits 48..) and the mass before it in the order (below
// 2^48), by comparing all with all: eight threads per token.  Token i's to its thread i.
constexpr int kPerToken = 8;
template <typename T>
__device__ unsigned long long RowSampler<T>::rank_list(int n) {
  static_assert(kListCap <= kThreads, "one thread per listed token at the end");
  const int sub = tid_ % kPerToken;
  __syncthreads();
  for (int i0 = warp_ * (32 / kPerToken); i0 < n; i0 += kThreads / kPerToken) {  // (a warp's share is its own)
    const int i = i0 + lane_ / kPerToken;
    unsigned long long above = 0;
    if (i < n) {
      const unsigned long long key = sh_.list[i].key;
      for (int j = sub; j < n; j += kPerToken) {
        const Listed o = sh_.list[j];
        if (o.key > key) above += o.w + (1ull << 48);
      }
    }
#pragma unroll
    for (int o = 1; o < kPerToken; o <<= 1) above += __shfl_xor_sync(0xffffffffu, above, o);
    if (i < n && sub == 0) sh_.part[i] = above;
  }
  __syncthreads();
  return tid_ < n ? sh_.part[tid_] : 0;
}

// Narrows k->z_cut, k->id_cut to the shortest prefix of the order whose count (or
// mass) reaches target >= 1.  A target above the total of the tokens with a weight
// leaves k alone.
template <typename T>
__device__ void RowSampler<T>::threshold(bool by_mass, unsigned long long target, Kept* k) {
  unsigned long long above = 0;  // count or mass of the bins before
  int bin[2] = {0, 0};
  // the part of bin bin[0] that z lies in, or kBins
  auto part_bin = [&](float z) -> int {
    const float x = list_place(z);
    return static_cast<int>(x) == bin[0] ? min(static_cast<int>((x - bin[0]) * kBins), kBins - 1) : kBins;
  };
#pragma unroll
  for (int level = 0; level < 2; ++level) {
    uint32_t(*hist)[kBins] = sh_.hist[level];
    __syncthreads();
    hist[0][tid_] = 0;
    hist[1][tid_] = 0;
    if (tid_ == 0) sh_.list_n = 0;
    __syncthreads();
    for_each_vector(s_, [&](const float(&z)[kN], int) {
#pragma unroll
      for (int e = 0; e < kN; ++e) {
        const int b = level == 0 ? list_bin(z[e]) : part_bin(z[e]);
        if (b < kBins) count_into(hist, b, by_mass, z[e]);
      }
    });
    cluster_sync();
    bin[level] = find_bin(hist, by_mass, target, &above);
    if (bin[level] < 0) return;
  }
  for_each_vector(s_, [&](const float(&z)[kN], int id) {
#pragma unroll
    for (int e = 0; e < kN; ++e)
      if (part_bin(z[e]) == bin[1]) {
        const uint32_t at = atomicAdd(&sh_.list_n, 1u);
        if (at < kListCap) sh_.part[at] = make_key(z[e], id + e);
      }
  });
  cluster_sync();
  if (rank_ == 0) {
    const int n = fetch_list();
    if (n >= 0) {
      const unsigned long long r = rank_list(n);
      if (tid_ < n) {
        const unsigned long long before = above + (by_mass ? r & 0xFFFFFFFFFFFFull : r >> 48);
        if (before < target && before + (by_mass ? sh_.list[tid_].w : 1) >= target) sh_.list_key = sh_.list[tid_].key;
      }
    }
    if (tid_ == 0) sh_.list_ok = n >= 0;
  }
  cluster_sync();
  if (ld_cluster_u32(cluster_addr(&sh_.list_ok, 0)) != 0) {
    const unsigned long long key = ld_cluster_u64(cluster_addr(&sh_.list_key, 0));
    k->z_cut = key_value(key);
    k->id_cut = key_id(key);
    return;
  }
  // Too many in one part of a bin: go on with its extremes.
  float hi, lo;
  {
    uint32_t top = 0, bottom = 0;  // of the order keys, and of their complements
    for_each_vector(s_, [&](const float(&z)[kN], int) {
#pragma unroll
      for (int e = 0; e < kN; ++e)
        if (part_bin(z[e]) == bin[1]) {
          top = max(top, f32_ord(z[e]));
          bottom = max(bottom, ~f32_ord(z[e]));
        }
    });
    __syncthreads();
    hi = ord_f32(reduce_max_u32(top));
    __syncthreads();
    lo = ord_f32(~reduce_max_u32(bottom));
  }
  for (int level = 0; lo < hi; ++level) {
    // Bins over [lo, hi], bin 0 at the top: linear in z first, which spreads a
    // row's logits evenly; linear in the order keys after eight levels or where
    // the width is no ordinary number (each such level takes 9 bits off the keys).
    const float width = __fsub_rn(hi, lo);
    const bool linear = level < 8 && width < 1e30f && width > 1e-30f;
    const float inv = linear ? __fdiv_rn(kBins - 1, width) : 0.0f;
    const uint32_t ord_hi = f32_ord(hi);
    const int shift = max(0, 32 - __clz(ord_hi - f32_ord(lo)) - 9);
    auto bin_of = [&](float z) -> int {
      return linear ? min(static_cast<int>(__fmul_rn(__fsub_rn(hi, z), inv)), kBins - 1)
                    : static_cast<int>((ord_hi - f32_ord(z)) >> shift);
    };
    uint32_t(*hist)[kBins] = sh_.hist[parity_];
    __syncthreads();
    hist[0][tid_] = 0;
    hist[1][tid_] = 0;
    __syncthreads();
    for_each_vector(s_, [&](const float(&z)[kN], int) {
#pragma unroll
      for (int e = 0; e < kN; ++e)
        if (z[e] >= lo && z[e] <= hi) count_into(hist, bin_of(z[e]), by_mass, z[e]);
    });
    cluster_sync();
    const int bin = find_bin(hist, by_mass, target, &above);
    if (bin < 0) return;  // (not reached: the target lies in [lo, hi])
    // the bin's own extremes are the next interval
    uint32_t top = 0, bottom = 0;
    for_each_vector(s_, [&](const float(&z)[kN], int) {
#pragma unroll
      for (int e = 0; e < kN; ++e)
        if (z[e] >= lo && z[e] <= hi && bin_of(z[e]) == bin) {
          top = max(top, f32_ord(z[e]));
          bottom = max(bottom, ~f32_ord(z[e]));
        }
    });
    parity_ ^= 1;
    __syncthreads();
    const uint32_t t = reduce_max_u32(top);
    __syncthreads();
    const uint32_t b = reduce_max_u32(bottom);
    hi = ord_f32(t);
    lo = ord_f32(~b);
  }
  // One value left, `hi`: of the tokens equal to it the first m in id order are kept.
  unsigned long long ties = 0, before = 0;
  for_each_vector(s_, [&](const float(&z)[kN], int) {
#pragma unroll
    for (int e = 0; e < kN; ++e) ties += z[e] == hi ? 1 : 0;
  });
  ties = static_cast<unsigned long long>(warp_sum_i64(static_cast<long long>(ties)));
  const unsigned long long all = reduce_sum_u64(ties, &before);
  unsigned long long m = target - above;
  if (by_mass) {
    const unsigned long long w = static_cast<unsigned long long>(weight_of(tempered(hi, zm_, c_)));
    if (w == 0) return;  // (a target above the row's total)
    m = (m + w - 1) / w;
  }
  if (m > all) return;
  // the CTA and warp that hold the m-th of them find its id
  unsigned long long b = before;
  for (int w = 0; w < warp_; ++w) b += sh_.warp_mass[w];
  uint32_t found = 0;
  if (b < m && m <= b + ties) {
    unsigned long long left = m - b;
    for (int i0 = 0; i0 < s_.n; i0 += 32) {
      const int i = i0 + lane_;
      float z[kN];
      int cnt = 0;
      if (i < s_.n) {
        Vec<T>::widen(s_.data[i], z);
#pragma unroll
        for (int e = 0; e < kN; ++e) cnt += z[e] == hi ? 1 : 0;
      }
      int incl = cnt;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane_ >= o) incl += t;
      }
      const int total = __shfl_sync(0xffffffffu, incl, 31);
      if (static_cast<unsigned long long>(total) >= left) {
        int need = static_cast<int>(left) - (incl - cnt);
        if (need >= 1 && need <= cnt) {
#pragma unroll
          for (int e = 0; e < kN; ++e)
            if (z[e] == hi && --need == 0) found = static_cast<uint32_t>(s_.id0 + i * kN + e) + 1;
        }
        break;
      }
      left -= total;
    }
  }
  __syncthreads();
  const uint32_t f = reduce_max_u32(found);
  k->z_cut = hi;
  k->id_cut = static_cast<int>(f) - 1;
}

template <typename T>
__device__ void RowSampler<T>::write(int id, float z, unsigned long long total) {
  p_.ids[row_] = id;
  if (p_.logprobs) {
    const float k32 = __fmul_rn(__ll2float_rn(static_cast<long long>(total)), 2.3283064365386963e-10f);  // 2^-32
    p_.logprobs[row_] = __fsub_rn(__fmul_rn(tempered(z, zm_, c_), 0.6931471805599453f), logf(k32));
  }
}

// The point of a draw: floor(u * total), below total.
__device__ __forceinline__ unsigned long long draw_point(float uniform, unsigned long long total) {
  const float u = fminf(fmaxf(uniform, 0.0f), 0.99999994f);
  const unsigned long long r = static_cast<unsigned long long>(
      floor(__dmul_rn(static_cast<double>(u), static_cast<double>(static_cast<long long>(total)))));
  return r < total ? r : total - 1;
}

// Sum over this CTA of every thread's value.
template <typename T>
__device__ unsigned long long RowSampler<T>::block_sum_u64(unsigned long long v) {
  v = static_cast<unsigned long long>(warp_sum_i64(static_cast<long long>(v)));
  __syncthreads();
  if (lane_ == 0) sh_.scratch_u64[warp_] = v;
  __syncthreads();
  return static_cast<unsigned long long>(
      warp_sum_i64(lane_ < kWarps ? static_cast<long long>(sh_.scratch_u64[lane_]) : 0));
}

// Draws from a list, if one can be made: true when the row is done.  With top-p alone
// *mass becomes the row's mass.
template <typename T>
__device__ bool RowSampler<T>::from_list(int top_k, float top_p, float min_t, unsigned long long* mass) {
  const unsigned target = top_k > 0 ? top_k : kListTargetTopP;
  const int my_bin = list_bin(lane_max_);
  if (my_bin < kBins) atomicAdd(&sh_.list_hist[my_bin], 1u);
  unsigned long long before;
  if (top_k == 0) {
    *mass = reduce_sum_u64(warp_kept_mass(Kept{-INFINITY, -INFINITY, INT32_MAX}), &before);
  } else {
    cluster_sync();
  }
  // The last bin that is listed: the first at which the lanes' maxima reach the target.
  uint32_t n = 0;
  for_each_cta(&sh_.list_hist[tid_], size_, [&](uint32_t, uint32_t h) { n += h; });
  uint32_t incl = n;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t t = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane_ >= o) incl += t;
  }
  if (lane_ == 31) sh_.scratch_u32[warp_] = incl;
  if (tid_ == 0) sh_.found_bin = kBins - 1;
  __syncthreads();
  for (int w = 0; w < warp_; ++w) incl += sh_.scratch_u32[w];
  if (incl >= target && incl - n < target) sh_.found_bin = tid_;
  __syncthreads();
  const int last_bin = sh_.found_bin;
  if (my_bin <= last_bin) {
    for (int i = lane_; i < s_.n; i += 32) {
      const uint4 x = s_.data[i];
      if (list_bin(Vec<T>::max_of(x)) > last_bin) continue;
      float z[kN];
      Vec<T>::widen(x, z);
#pragma unroll
      for (int e = 0; e < kN; ++e)
        if (list_bin(z[e]) <= last_bin) {
          const uint32_t at = atomicAdd(&sh_.list_n, 1u);
          if (at < kListCap) sh_.part[at] = make_key(z[e], s_.id0 + i * kN + e);
        }
    }
  }
  cluster_sync();
  // The first CTA fetches the parts and says whether they will do.
  unsigned long long need = 0;
  int total = 0;
  if (rank_ == 0) {
    total = fetch_list();
    bool ok = total >= 0;
    if (ok && top_k == 0) {
      need = mass_wanted(top_p, *mass);
      unsigned long long have = 0;
      __syncthreads();
      for (int i = tid_; i < total; i += kThreads) have += sh_.list[i].w;
      ok = block_sum_u64(have) >= need;
    }
    if (tid_ == 0) sh_.list_ok = ok;
  }
  cluster_sync();
  const bool ok = ld_cluster_u32(cluster_addr(&sh_.list_ok, 0)) != 0;
  if (ok && rank_ == 0) draw_from_list(total, top_k, need, min_t);
  return ok;
}

// The draw from the first CTA's list of n tokens.  top_k > 0: `need` is worked out here.
template <typename T>
__device__ void RowSampler<T>::draw_from_list(int n, int top_k, unsigned long long need, float min_t) {
  rank_list(n);
  if (warp_ == 0) {
    if (top_k > 0) {
      unsigned long long mass = 0;
      for (int i = lane_; i < n; i += 32)
        if (static_cast<int>(sh_.part[i] >> 48) < top_k) mass += sh_.list[i].w;
      mass = warp_sum_u64(mass);
      need = top_p_ < 1.0f ? mass_wanted(top_p_, mass) : mass;
    }
    // the kept ones, closed up (each to a place at or before its own), and their mass
    unsigned long long kept = 0;
    int m = 0;
    for (int i0 = 0; i0 < n; i0 += 32) {
      const int i = i0 + lane_;
      Listed it{0, 0};
      bool keep = false;
      if (i < n) {
        it = sh_.list[i];
        const unsigned long long place = sh_.part[i];
        keep = it.w > 0 && (place & 0xFFFFFFFFFFFFull) < need &&
               (top_k == 0 || static_cast<int>(place >> 48) < top_k) &&
               tempered(key_value(it.key), zm_, c_) >= min_t;
      }
      const unsigned ones = __ballot_sync(0xffffffffu, keep);  // (every lane has read its token)
      if (keep) {
        kept += it.w;
        sh_.list[m + __popc(ones & ((1u << lane_) - 1u))] = it;
      }
      m += __popc(ones);
    }
    kept = warp_sum_u64(kept);
    if (lane_ == 0) {
      sh_.count = m;
      sh_.kept = kept;
      sh_.point = draw_point(uniform_, kept);
    }
  }
  __syncthreads();
  const int m = static_cast<int>(sh_.count);
  const unsigned long long r = sh_.point;
  const int sub = tid_ % kPerToken;
  for (int i0 = warp_ * (32 / kPerToken); i0 < m; i0 += kThreads / kPerToken) {
    const int i = i0 + lane_ / kPerToken;
    unsigned long long before = 0;
    Listed it{0, 0};
    if (i < m) {
      it = sh_.list[i];
      for (int j = sub; j < m; j += kPerToken) {
        const Listed o = sh_.list[j];
        // ids are complemented in the keys' low words
        if (static_cast<uint32_t>(o.key) > static_cast<uint32_t>(it.key)) before += o.w;
      }
    }
#pragma unroll
    for (int o = 1; o < kPerToken; o <<= 1) before += __shfl_xor_sync(0xffffffffu, before, o);
    if (i < m && sub == 0 && before <= r && r < before + it.w) write(key_id(it.key), key_value(it.key), sh_.kept);
  }
}

// The token at the given point of the kept tokens' mass, in id order.
template <typename T>
__device__ void RowSampler<T>::draw(const Kept& k) {
  const unsigned long long mine = warp_kept_mass(k);
  unsigned long long before = 0;
  const unsigned long long total = reduce_sum_u64(mine, &before);
  const unsigned long long r = draw_point(uniform_, total);
  for (int w = 0; w < warp_; ++w) before += sh_.warp_mass[w];
  if (r < before || r >= before + mine) return;
  unsigned long long left = r - before;  // mass to pass within this warp's vectors
  for (int i0 = 0; i0 < s_.n; i0 += 32) {
    const int i = i0 + lane_;
    float z[kN];
    unsigned long long w[kN], sum = 0;
#pragma unroll
    for (int e = 0; e < kN; ++e) w[e] = 0;
    if (i < s_.n) {
      Vec<T>::widen(s_.data[i], z);
#pragma unroll
      for (int e = 0; e < kN; ++e) {
        if (is_kept(z[e], s_.id0 + i * kN + e, k))
          w[e] = static_cast<unsigned long long>(weight_of(tempered(z[e], zm_, c_)));
        sum += w[e];
      }
    }
    unsigned long long incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned long long t = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane_ >= o) incl += t;
    }
    const unsigned long long all = __shfl_sync(0xffffffffu, incl, 31);
    if (left < all) {
      unsigned long long at = incl - sum;
      if (at <= left && left < incl) {
        int id = -1;
        float zs = 0.0f;
#pragma unroll
        for (int e = 0; e < kN; ++e) {
          if (at <= left && left < at + w[e]) {
            id = s_.id0 + i * kN + e;
            zs = z[e];
          }
          at += w[e];
        }
        write(id, zs, total);
      }
      return;
    }
    left -= all;
  }
}

// The first token whose logit is the row's maximum.
template <typename T>
__device__ void RowSampler<T>::greedy() {
  uint32_t first = 0;  // complemented id
  for_each_vector(s_, [&](const float(&z)[kN], int id) {
#pragma unroll
    for (int e = 0; e < kN; ++e)
      if (z[e] == zm_) first = max(first, ~static_cast<uint32_t>(id + e));
  });
  __syncthreads();
  first = reduce_max_u32(first);
  if (rank_ == 0 && tid_ == 0) {
    p_.ids[row_] = static_cast<int32_t>(~first);
    if (p_.logprobs) p_.logprobs[row_] = 0.0f;
  }
}

template <typename T>
__device__ bool RowSampler<T>::run() {
  int top_k = top_k_;
  const float T_row = temperature_, min_p = min_p_;
  zm_ = ord_f32(reduce_max_u32(f32_ord(lane_max_)));
  if (zm_ == -INFINITY) {
    if (rank_ == 0 && tid_ == 0) {
      p_.ids[row_] = -1;
      if (p_.logprobs) p_.logprobs[row_] = __int_as_float(0x7FC00000);
      set_status(p_.dev_status, LMH_DS_NO_ALLOWED_TOKEN);
    }
    return false;
  }
  if (zm_ == INFINITY) {  // only the +inf tokens are left, as equals
    for (int i = lane_; i < s_.n; i += 32) {
      float z[kN];
      Vec<T>::widen(s_.data[i], z);
#pragma unroll
      for (int e = 0; e < kN; ++e) z[e] = z[e] == INFINITY ? 0.0f : -INFINITY;
      s_.data[i] = Vec<T>::narrow(z);
    }
    zm_ = 0.0f;
    lane_max_ = lane_max_ == INFINITY ? 0.0f : -INFINITY;
  }
  if (!(T_row > 0.0f)) {
    greedy();
    return false;
  }
  c_ = fminf(fmaxf(__fmul_rn(__frcp_rn(T_row), kLog2e), 1.1754944e-38f), 3.402823466e+38f);

  Kept k{-INFINITY, -INFINITY, INT32_MAX};
  if (top_k < 0 || top_k >= p_.V) top_k = 0;
  const float top_p = top_p_;
  const float min_t = min_p > 0.0f ? fminf(log2f(min_p), 0.0f) : -INFINITY;
  unsigned long long mass = 0;
  bool have_mass = false;
  if (top_k > 0 ? top_k <= kListTarget : top_p < 1.0f) {
    if (from_list(top_k, top_p, min_t, &mass)) return true;
    have_mass = top_k == 0;
  }
  if (top_k > 0) threshold(false, static_cast<unsigned long long>(top_k), &k);
  if (top_p < 1.0f) {
    unsigned long long before;
    if (!have_mass) mass = reduce_sum_u64(warp_kept_mass(k), &before);
    threshold(true, mass_wanted(top_p, mass), &k);
  }
  k.min_t = min_t;
  draw(k);
  return false;
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 2) sample_logits_kernel(Params p) {
  extern __shared__ uint4 data[];
  __shared__ Shared sh;
  pdl_wait();
  pdl_launch_dependents();
  RowSampler<T> s(p, sh, data, static_cast<int>(blockIdx.x / cluster_size()));
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
