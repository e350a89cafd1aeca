// beam_select.cu -- the best continuations of groups of beams (lmh_beam_select,
// lmh_beam_select_lists).
//
//   score(b, v) = cum[b] + z[b][v] - lse[b],  lse[b] = log sum_v exp(z[b][v])
//
// and of every group's beams x V scores the k largest, ties by beam, then token.  Scores are
// compared in 64 bits: two beams' scores differ by what their log-sum-exps differ by, which
// 32 bits would round to a step of the score (5e-7 at 8).
#include "device_common.cuh"
#include "lmh_internal.h"
#include "logits_vec.cuh"

namespace lmh {

constexpr int kBSThreads = 256;                       // stream kernel
constexpr int kBSBlocksPerWarp = 8;                   // 64-blocks a warp takes of a chunk
constexpr int kBSBlocks = kBSBlocksPerWarp * kBSThreads / 32;  // 64-blocks of a chunk
constexpr int kBGThreads = 512;                       // choice kernel: one CTA a group
constexpr int kBGWarps = kBGThreads / 32;
constexpr int kBGCand = 1024;                         // candidates held in shared memory
constexpr int kBGKept = 1024;                         // kept blocks listed
constexpr int kBeamsMax = LMH_K_MAX;

struct BeamArgs {
  const char* logits;
  int64_t row_stride;  // elements
  int rows, beams, V, nblk;
  int slots;  // (m, s) pairs a row
  const float* cum;
  const uint8_t* finished;
  int pad_id;
  const uint32_t* mask;
  int mask_words;
  int k;
  bool keep_slots;
  float* out_scores;
  int32_t* out_parents;
  int32_t* out_tokens;
  float2* part_ms;
  float* bmax;
  uint32_t* dev_status;
  // lists
  const int32_t* ids;
  const float* lps;
  int n;
};

__device__ __forceinline__ bool mask_allows(const uint32_t* words, int v) {
  return words == nullptr || ((__ldg(words + (v >> 5)) >> (v & 31)) & 1u);
}

// ---------------------------------------------------------------------------
// stream kernel: one chunk of kBSBlocks 64-blocks of one row a CTA
// ---------------------------------------------------------------------------
// Every thread holds its logits in registers: the block maxima (over allowed tokens) go to the
// workspace, the chunk's (m, s) over all tokens to one slot.  x - m is taken before the product with
// log2(e): the rounding of m * log2(e) would be common to a row's terms, and shift its lse.
template <typename T>
__global__ void __launch_bounds__(kBSThreads) beam_stream_kernel(const BeamArgs a) {
  using VT = Vec16<T>;
  __shared__ float red[32];
  pdl_wait();
  pdl_launch_dependents();
  const int row = blockIdx.x, chunk = blockIdx.y;
  if (a.finished && a.finished[row]) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const T* src = reinterpret_cast<const T*>(a.logits) + static_cast<int64_t>(row) * a.row_stride;
  const uint32_t* mrow = a.mask ? a.mask + static_cast<int64_t>(row) * a.mask_words : nullptr;
  const int b0 = chunk * kBSBlocks + warp;  // this warp's blocks: b0, b0 + 8, ...
  float x[2 * kBSBlocksPerWarp];
  float tm = -INFINITY;
#pragma unroll
  for (int i = 0; i < kBSBlocksPerWarp; ++i) {
    const int b = b0 + i * (kBSThreads / 32);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int v = b * kBlock + h * 32 + lane;
      float t = v < a.V ? VT::at(src, v) : -INFINITY;
      t = t == t ? t : -INFINITY;  // NaN counts as -inf
      x[2 * i + h] = t;
      tm = fmaxf(tm, t);
    }
  }
#pragma unroll
  for (int i = 0; i < kBSBlocksPerWarp; ++i) {
    const int b = b0 + i * (kBSThreads / 32);
    float m = -INFINITY;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int v = b * kBlock + h * 32 + lane;
      if (v < a.V && mask_allows(mrow, v)) m = fmaxf(m, x[2 * i + h]);
    }
    m = warp_max(m);
    if (lane == 0 && b < a.nblk) a.bmax[static_cast<int64_t>(row) * a.nblk + b] = m;
  }
  const float M = block_max(tm, red);
  float s = 0.0f;
  if (M == INFINITY) {
#pragma unroll
    for (int i = 0; i < 2 * kBSBlocksPerWarp; ++i) s += x[i] == INFINITY ? 1.0f : 0.0f;
  } else if (M > -INFINITY) {
#pragma unroll
    for (int i = 0; i < 2 * kBSBlocksPerWarp; ++i) s += ex2_approx((x[i] - M) * kLog2e);
  }
  s = block_sum(s, red);
  if (threadIdx.x == 0) a.part_ms[static_cast<int64_t>(row) * a.slots + chunk] = make_float2(M, s);
}

// ---------------------------------------------------------------------------
// choice of a group
// ---------------------------------------------------------------------------
struct Cand {
  double score;
  uint32_t at;  // beam * V + token (lists: beam * n + place)
};

// (score, at) goes before (score2, at2)
__device__ __forceinline__ bool before(double s, uint32_t at, double s2, uint32_t at2) {
  return s > s2 || (s == s2 && at < at2);
}

enum RowState : uint8_t { kRowNone = 0, kRowNormal = 1, kRowPlusInf = 2, kRowEnded = 3 };

template <int NT>
struct ChoiceSmem {
  double score[kBGCand];
  uint32_t at[kBGCand];
  double res_score[kBeamsMax];
  uint32_t res_at[kBeamsMax];
  double off[kBeamsMax];   // cum - log sum exp(z - M) of the group's rows
  float offf[kBeamsMax];
  float top_z[kBeamsMax];  // M, their largest logit
  uint8_t state[kBeamsMax];
  int first[kBeamsMax];    // keep_slots: the place of a candidate, or -1
  double wscore[NT / 32];
  uint32_t wat[NT / 32];
  uint32_t count, kept;
  float top[NT / 32 * 64];
  float bound;
  float off_max;
  uint32_t kept_blocks[kBGKept];
};

// Orders sm.score/at[0 .. cnt) into sm.res_*[0 .. min(cnt, k)): every thread counts those before its own.
template <int NT>
__device__ void rank_candidates(ChoiceSmem<NT>& sm, int cnt, int k) {
  for (int i = threadIdx.x; i < cnt; i += NT) {
    const double s = sm.score[i];
    const uint32_t at = sm.at[i];
    int rank = 0;
    for (int j = 0; j < cnt; ++j) rank += before(sm.score[j], sm.at[j], s, at);
    if (rank < k) {
      sm.res_score[rank] = s;
      sm.res_at[rank] = at;
    }
  }
}

// Writes the group's k results (the first `cnt` of sm.res_* are real).  `token(at, beam)` gives a token.
template <int NT, typename Token>
__device__ void write_results(const BeamArgs& a, ChoiceSmem<NT>& sm, int group, int cnt, int per_beam, Token token) {
  const int k = a.k;
  const int64_t base = static_cast<int64_t>(group) * k;
  auto beam_of = [&](int r) { return r < cnt ? static_cast<int>(sm.res_at[r] / static_cast<uint32_t>(per_beam)) : -1; };
  if (a.keep_slots) {  // k == beams <= NT
    const int r = threadIdx.x;
    if (r < k) sm.first[r] = -1;
    __syncthreads();
    bool first = false;
    if (r < cnt) {
      first = true;
      const int b = beam_of(r);
      for (int j = 0; j < r; ++j) first &= beam_of(j) != b;
      if (first) sm.first[b] = r;  // slot b is taken by candidate r
    }
    __syncthreads();
    if (r < k && !first) {  // the turn-th candidate that is no first child takes the turn-th free slot
      int turn = 0;
      for (int j = 0; j < r; ++j) {
        const int b = beam_of(j);
        turn += b < 0 || sm.first[b] != j;
      }
      int slot = 0;
      for (int t = 0; slot < k; ++slot)
        if (sm.first[slot] < 0 && t++ == turn) break;
      sm.kept_blocks[r] = static_cast<uint32_t>(slot);
    } else if (r < k) {
      sm.kept_blocks[r] = static_cast<uint32_t>(beam_of(r));
    }
    __syncthreads();
  }
  for (int r = threadIdx.x; r < k; r += NT) {
    const int64_t to = base + (a.keep_slots ? static_cast<int>(sm.kept_blocks[r]) : r);
    const int b = beam_of(r);
    a.out_scores[to] = b < 0 ? -INFINITY : static_cast<float>(sm.res_score[r]);
    a.out_parents[to] = b < 0 ? -1 : group * a.beams + b;
    a.out_tokens[to] = b < 0 ? -1 : (sm.state[b] == kRowEnded ? a.pad_id : token(sm.res_at[r], b));
  }
  if (cnt == 0 && threadIdx.x == 0) set_status(a.dev_status, LMH_DS_NO_ALLOWED_TOKEN);
}

// The k best by repeatedly taking the best that is left: exact for any number of ties, used where the
// candidates do not fit.  `scan(s, at, last_s, last_at)` puts the thread's best item behind (last_s, last_at)
// into (s, at), s = -inf for none.  Returns the number found.
template <int NT, typename Scan>
__device__ int take_in_turn(ChoiceSmem<NT>& sm, int k, Scan scan) {
  double last_s = INFINITY;
  uint32_t last_at = 0;
  double s = -INFINITY;
  uint32_t at = 0xFFFFFFFFu;
  bool stale = true;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int r = 0;
  for (; r < k; ++r) {
    if (stale) scan(s, at, last_s, last_at);
    double bs = s;
    uint32_t bat = at;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const double os = __shfl_xor_sync(0xffffffffu, bs, o);
      const uint32_t oat = __shfl_xor_sync(0xffffffffu, bat, o);
      if (before(os, oat, bs, bat)) bs = os, bat = oat;
    }
    __syncthreads();
    if (lane == 0) sm.wscore[warp] = bs, sm.wat[warp] = bat;
    __syncthreads();
    bs = sm.wscore[0], bat = sm.wat[0];
#pragma unroll
    for (int w = 1; w < NT / 32; ++w)
      if (before(sm.wscore[w], sm.wat[w], bs, bat)) bs = sm.wscore[w], bat = sm.wat[w];
    if (!(static_cast<float>(bs) > -INFINITY)) break;
    if (threadIdx.x == 0) sm.res_score[r] = bs, sm.res_at[r] = bat;
    last_s = bs, last_at = bat;
    stale = s == bs && at == bat;  // (the pair is one thread's alone)
  }
  __syncthreads();
  return r;
}

// z - M, first of a score's sums: rows far from 0 (all logits at a type's lowest value) keep the rest of the
// score.  A row with +inf logits has only these, as equals.
template <typename F>
__device__ __forceinline__ F below_top(uint8_t state, float z, float M) {
  if (state == kRowPlusInf) return z == INFINITY ? static_cast<F>(0) : static_cast<F>(-INFINITY);
  return static_cast<F>(z) - static_cast<F>(M);
}

template <typename T>
__global__ void __launch_bounds__(kBGThreads) beam_choose_kernel(const BeamArgs a) {
  using VT = Vec16<T>;
  constexpr int NT = kBGThreads;
  extern __shared__ __align__(16) unsigned char smem_raw[];
  ChoiceSmem<NT>& sm = *reinterpret_cast<ChoiceSmem<NT>*>(smem_raw);
  const int group = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int B = a.beams, nblk = a.nblk;
  const int row0 = group * B;
  pdl_wait();
  if (tid == 0) sm.count = 0, sm.kept = 0, sm.off_max = 0.0f;

  // ---- the rows' cum - lse ----
  for (int b = warp; b < B; b += kBGWarps) {
    const int row = row0 + b;
    const float cum = a.cum[row];
    const bool ended = a.finished && a.finished[row];
    const float2* ms = a.part_ms + static_cast<int64_t>(row) * a.slots;
    float M = -INFINITY;
    double S = 0.0;
    if (!ended) {
      for (int j = lane; j < a.slots; j += 32) M = fmaxf(M, __ldcg(ms + j).x);
      M = warp_max(M);
      for (int j = lane; j < a.slots; j += 32) {
        const float2 p = __ldcg(ms + j);
        if (p.x == M) S += p.y;
        else if (p.x > -INFINITY && M < INFINITY) S += static_cast<double>(p.y) * exp2(static_cast<double>(p.x - M) * 1.4426950408889634);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) S += __shfl_xor_sync(0xffffffffu, S, o);
    }
    if (lane == 0) {
      const bool fin = cum > -INFINITY && cum < INFINITY;  // (false for NaN)
      uint8_t st = kRowNone;
      double off = 0.0;
      if (fin && ended) {
        st = kRowEnded;
        off = cum;
      } else if (fin && M > -INFINITY) {
        st = M == INFINITY ? kRowPlusInf : kRowNormal;
        off = static_cast<double>(cum) - log(S);
      }
      sm.state[b] = st;
      sm.off[b] = off;
      sm.offf[b] = static_cast<float>(off);
      sm.top_z[b] = M;
    }
  }
  __syncthreads();
  if (tid < B) {
    if (sm.state[tid] == kRowEnded) {
      const uint32_t i = atomicAdd(&sm.count, 1u);
      sm.score[i] = sm.off[tid];
      sm.at[i] = static_cast<uint32_t>(tid) * static_cast<uint32_t>(a.V);
    }
    atomicMax(reinterpret_cast<int*>(&sm.off_max), __float_as_int(fabsf(sm.offf[tid])));
  }

  // ---- a bound that at least k blocks reach ----
  const float* bm = a.bmax + static_cast<int64_t>(row0) * nblk;
  const int nb = B * nblk;
  auto block_score = [&](int i) -> float {  // in fp32
    const int b = i / nblk;
    const uint8_t st = sm.state[b];
    return st == kRowNormal || st == kRowPlusInf ? below_top<float>(st, __ldcg(bm + i), sm.top_z[b]) + sm.offf[b]
                                                 : -INFINITY;
  };
  float m1 = -INFINITY, m2 = -INFINITY;
  for (int i = tid; i < nb; i += NT) {
    const float v = block_score(i);
    m2 = fmaxf(m2, fminf(m1, v));
    m1 = fmaxf(m1, v);
  }
  const int q = min(64, max(2, (a.k + 3) / 4));  // values of a warp that are looked at: 16 q >= k
  {
    uint32_t k1 = f32_ord(m1), k2 = f32_ord(m2);
    for (int r = 0; r < q; ++r) {
      const uint32_t m = __reduce_max_sync(0xffffffffu, k1);
      const unsigned holders = __ballot_sync(0xffffffffu, k1 == m);
      if (lane == __ffs(holders) - 1) {
        sm.top[warp * q + r] = m ? ord_f32(m) : -INFINITY;
        k1 = k2;
        k2 = 0;
      }
    }
  }
  __syncthreads();
  const int nv = kBGWarps * q;
  for (int i = tid; i < nv; i += NT) {
    const float v = sm.top[i];
    int rank = 0;
    for (int j = 0; j < nv; ++j) rank += sm.top[j] > v || (sm.top[j] == v && j < i);
    if (rank == a.k - 1) sm.bound = v;
  }
  __syncthreads();
  // The k-th best score is at least `bound` but for fp32's rounding of bound and of the sums compared
  // with it (2^-24 of each term): 2^-21 covers both.
  float t = sm.bound;
  if (t > -INFINITY) t -= ldexpf(fabsf(t) + sm.off_max, -21);

  // ---- the blocks that reach it ----
  for (int i = tid; i < nb; i += NT) {
    const float v = block_score(i);
    if (v >= t && v > -INFINITY) {
      const uint32_t p = atomicAdd(&sm.kept, 1u);
      if (p < kBGKept) sm.kept_blocks[p] = static_cast<uint32_t>(i);
    }
  }
  __syncthreads();
  const int nkept = static_cast<int>(sm.kept);
  auto logit = [&](int b, int v) -> float {  // -inf for a token that is not allowed
    const int row = row0 + b;
    if (a.mask && !mask_allows(a.mask + static_cast<int64_t>(row) * a.mask_words, v)) return -INFINITY;
    const float z = VT::at(a.logits, static_cast<int64_t>(row) * a.row_stride + v);
    return z == z ? z : -INFINITY;
  };
  auto score_of = [&](int b, float z) -> double {
    return sm.off[b] + below_top<double>(sm.state[b], z, sm.top_z[b]);
  };
  if (nkept <= kBGKept) {
    for (int j = tid; j < nkept * kBlock; j += NT) {
      const int i = static_cast<int>(sm.kept_blocks[j / kBlock]);
      const int b = i / nblk, v = (i - b * nblk) * kBlock + j % kBlock;
      if (v >= a.V) continue;
      const float z = logit(b, v);
      const float f = below_top<float>(sm.state[b], z, sm.top_z[b]) + sm.offf[b];
      if (!(f >= t) || !(f > -INFINITY)) continue;
      const uint32_t p = atomicAdd(&sm.count, 1u);
      if (p < kBGCand) {
        sm.score[p] = score_of(b, z);
        sm.at[p] = static_cast<uint32_t>(b) * static_cast<uint32_t>(a.V) + static_cast<uint32_t>(v);
      }
    }
  }
  __syncthreads();
  int cnt = static_cast<int>(sm.count);
  if (nkept <= kBGKept && cnt <= kBGCand) {
    rank_candidates(sm, cnt, a.k);
    cnt = min(cnt, a.k);
    __syncthreads();
  } else {
    // a thread's blocks are a contiguous share, looked through again only after its best is taken
    const int per = (nb + NT - 1) / NT;
    const int lo = min(nb, tid * per), hi = min(nb, lo + per);
    cnt = take_in_turn(sm, a.k, [&](double& s, uint32_t& at, double last_s, uint32_t last_at) {
      s = -INFINITY;
      at = 0xFFFFFFFFu;
      for (int i = lo; i < hi; ++i) {
        const int b = i / nblk, blk = i - b * nblk;
        const uint8_t st = sm.state[b];
        if (st == kRowNone) continue;
        if (st == kRowEnded) {
          const uint32_t e = static_cast<uint32_t>(b) * static_cast<uint32_t>(a.V);
          if (blk == 0 && before(last_s, last_at, sm.off[b], e) && before(sm.off[b], e, s, at)) s = sm.off[b], at = e;
          continue;
        }
        // (an equal score further on comes after the one that is held)
        const double most = score_of(b, __ldcg(bm + i));
        for (int v = blk * kBlock; most > s && v < min(a.V, (blk + 1) * kBlock); ++v) {
          const double c = score_of(b, logit(b, v));
          const uint32_t e = static_cast<uint32_t>(b) * static_cast<uint32_t>(a.V) + static_cast<uint32_t>(v);
          if (static_cast<float>(c) > -INFINITY && before(last_s, last_at, c, e) && c > s) s = c, at = e;
        }
      }
    });
  }
  write_results(a, sm, group, cnt, a.V,
                [&](uint32_t at, int b) { return static_cast<int32_t>(at - static_cast<uint32_t>(b) * static_cast<uint32_t>(a.V)); });
}

// ---------------------------------------------------------------------------
// from top-k lists
// ---------------------------------------------------------------------------
constexpr int kBLThreads = 256;

__global__ void __launch_bounds__(kBLThreads) beam_lists_kernel(const BeamArgs a) {
  constexpr int NT = kBLThreads;
  extern __shared__ __align__(16) unsigned char smem_raw[];
  ChoiceSmem<NT>& sm = *reinterpret_cast<ChoiceSmem<NT>*>(smem_raw);
  const int group = blockIdx.x, tid = threadIdx.x;
  const int B = a.beams, n = a.n, row0 = group * B;
  pdl_wait();
  if (tid == 0) sm.count = 0;
  if (tid < B) {
    const float cum = a.cum[row0 + tid];
    const bool fin = cum > -INFINITY && cum < INFINITY;
    sm.state[tid] = !fin ? kRowNone : (a.finished && a.finished[row0 + tid]) ? kRowEnded : kRowNormal;
    sm.off[tid] = cum;
  }
  __syncthreads();
  const int64_t e0 = static_cast<int64_t>(row0) * n;
  const int total = B * n;
  // the score of entry i of the group's lists; -inf for none
  auto entry = [&](int i) -> double {
    const int b = i / n;
    const uint8_t st = sm.state[b];
    if (st == kRowEnded) return i == b * n ? sm.off[b] : -INFINITY;
    if (st == kRowNone || a.ids[e0 + i] < 0) return -INFINITY;
    const float lp = a.lps[e0 + i];
    if (!(lp > -INFINITY && lp < INFINITY)) return -INFINITY;
    const double s = sm.off[b] + static_cast<double>(lp);
    return static_cast<float>(s) > -INFINITY ? s : -INFINITY;
  };
  for (int i = tid; i < total; i += NT) {
    const double s = entry(i);
    if (s > -INFINITY) {
      const uint32_t p = atomicAdd(&sm.count, 1u);
      if (p < kBGCand) sm.score[p] = s, sm.at[p] = static_cast<uint32_t>(i);
    }
  }
  __syncthreads();
  int cnt = static_cast<int>(sm.count);
  if (cnt <= kBGCand) {
    rank_candidates(sm, cnt, a.k);
    cnt = min(cnt, a.k);
    __syncthreads();
  } else {
    cnt = take_in_turn(sm, a.k, [&](double& s, uint32_t& at, double last_s, uint32_t last_at) {
      s = -INFINITY;
      at = 0xFFFFFFFFu;
      for (int i = tid; i < total; i += NT) {
        const double c = entry(i);
        const uint32_t e = static_cast<uint32_t>(i);
        if (c > -INFINITY && before(last_s, last_at, c, e) && before(c, e, s, at)) s = c, at = e;
      }
    });
  }
  write_results(a, sm, group, cnt, n, [&](uint32_t at, int) { return a.ids[e0 + at]; });
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
static size_t align_up(size_t n) { return (n + 255) & ~static_cast<size_t>(255); }

static int beam_slots(int V) { return ((V + kBlock - 1) / kBlock + kBSBlocks - 1) / kBSBlocks; }

size_t beam_workspace_bytes(int rows, int V) {
  const size_t nblk = (static_cast<size_t>(V) + kBlock - 1) / kBlock;
  return align_up(static_cast<size_t>(rows) * static_cast<size_t>(beam_slots(V)) * 8) +
         align_up(static_cast<size_t>(rows) * nblk * 4);
}

template <typename T>
static cudaError_t beam_setup_one() {
  return cudaFuncSetAttribute(beam_choose_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              sizeof(ChoiceSmem<kBGThreads>));
}

cudaError_t beam_setup() {
  cudaError_t e = beam_setup_one<__nv_bfloat16>();
  if (e == cudaSuccess) e = beam_setup_one<__half>();
  if (e == cudaSuccess) e = beam_setup_one<float>();
  return e;
}

static BeamArgs beam_args(const BeamCall& c) {
  BeamArgs a{};
  a.rows = c.groups * c.beams;
  a.beams = c.beams;
  a.V = c.V;
  a.cum = c.scores;
  a.finished = c.finished;
  a.pad_id = c.pad_id;
  a.k = c.k;
  a.keep_slots = c.keep_slots;
  a.out_scores = c.out_scores;
  a.out_parents = c.out_parents;
  a.out_tokens = c.out_tokens;
  a.dev_status = c.dev_status;
  return a;
}

template <typename T>
static cudaError_t launch_beams(const BeamArgs& a, int groups, cudaStream_t stream) {
  trace_begin(kTraceBeamStream, stream);
  cudaError_t e = launch_kernel(beam_stream_kernel<T>, dim3(a.rows, a.slots), dim3(kBSThreads), 0, stream, true, a);
  trace_end(kTraceBeamStream, stream);
  if (e != cudaSuccess) return e;
  trace_begin(kTraceBeamChoose, stream);
  e = launch_kernel(beam_choose_kernel<T>, dim3(groups), dim3(kBGThreads), sizeof(ChoiceSmem<kBGThreads>), stream, true, a);
  trace_end(kTraceBeamChoose, stream);
  return e;
}

cudaError_t launch_beam_select(const BeamCall& c, const void* logits, lmh_dtype dtype, int64_t row_stride,
                               const uint32_t* mask, int mask_words, void* workspace, int num_sms,
                               cudaStream_t stream) {
  BeamArgs a = beam_args(c);
  a.logits = static_cast<const char*>(logits);
  a.row_stride = row_stride;
  a.nblk = (c.V + kBlock - 1) / kBlock;
  a.slots = beam_slots(c.V);
  a.mask = mask;
  a.mask_words = mask_words;
  a.part_ms = static_cast<float2*>(workspace);
  a.bmax = reinterpret_cast<float*>(static_cast<char*>(workspace) +
                                    align_up(static_cast<size_t>(a.rows) * static_cast<size_t>(a.slots) * 8));
  switch (dtype) {
    case LMH_BF16: return launch_beams<__nv_bfloat16>(a, c.groups, stream);
    case LMH_F16: return launch_beams<__half>(a, c.groups, stream);
    default: return launch_beams<float>(a, c.groups, stream);
  }
}

cudaError_t launch_beam_select_lists(const BeamCall& c, const int32_t* ids, const float* logprobs, int n,
                                     cudaStream_t stream) {
  BeamArgs a = beam_args(c);
  a.ids = ids;
  a.lps = logprobs;
  a.n = n;
  trace_begin(kTraceBeamChoose, stream);
  const cudaError_t e = launch_kernel(beam_lists_kernel, dim3(c.groups), dim3(kBLThreads),
                                      sizeof(ChoiceSmem<kBLThreads>), stream, true, a);
  trace_end(kTraceBeamChoose, stream);
  return e;
}

}  // namespace lmh
