// beam_select.cu -- the best continuations of groups of beams (lmh_beam_select,
// lmh_beam_select_lists).
//
//   score(b, v) = cum[b] + z[b][v] - lse[b],  lse[b] = log sum_v exp(z[b][v])
//
// and of every group's beams x V scores the k largest, ties by beam, then token.  Scores are
// compared in 64 bits: two beams' scores differ by what their log-sum-exps differ by, which
// 32 bits would round to a step of the score (5e-7 at 8).  As whole numbers of the same order:
// this GPU's rate of 64-bit floating operations is low (two a clock and SM).
//
//   * beam_stream_kernel reads every logit once (persistent CTAs, bulk copies into a ring, a
//     thread 128 bytes): the largest allowed logit of every block of 64 and of every span of
//     32 threads, and the span's (max, sum of exponentials) go to the workspace.  Bound by the
//     logits' bytes: 256 x 248320 bf16 (127 MB) take 27 us, 0.70 of the copy rate; fp32 with a
//     mask, 64 x 128256 of which 52 rows have not ended (28 MB), 12.7 us, as long as its few
//     chunks a CTA take to start and drain.
//   * beam_choose_kernel, one CTA a group: the rows' lse from the spans' pairs; a bound t that at
//     least k spans reach, the blocks of the spans that reach it, a tighter bound from those, the
//     logits of the blocks that reach that, and their exact order.  7 us behind the stream in a
//     graph, all latency: its code runs once, and most of the time is its first reading.  So it is
//     kept short: what is used more than once is called, not inlined (with everything inlined it
//     took 2.6 us more).
#include <type_traits>

#include "device_common.cuh"
#include "lmh_internal.h"
#include "logits_vec.cuh"

namespace lmh {

// stream kernel
constexpr int kBSConsumerWarps = 4;
constexpr int kBSConsumers = kBSConsumerWarps * 32;
constexpr int kBSThreads = kBSConsumers + 32;        // + one producer warp
constexpr int kBSChunkBytes = kBSConsumers * 128;    // 128 bytes of a row a consumer
constexpr int kBSStageBytes = kBSChunkBytes + 128;   // (a chunk that begins off a 16-byte boundary takes 16 more)
constexpr int kBSStages = 3;
constexpr int kBSCtasPerSm = 4;
constexpr int kBSSmem = kBSStages * kBSStageBytes + kBSStages * 32 + 2 * kBSStages * 8 + 16;
// choice
constexpr int kBGThreads = 512;                       // one CTA a group
constexpr int kBGWarps = kBGThreads / 32;
constexpr int kBGHeld = 2;                            // spans or blocks a thread holds between its two looks at them
constexpr int kBGCand = 1024;                         // candidates held in shared memory
constexpr int kBGKept = 512;                          // spans, blocks listed
constexpr int kBLThreads = 256;                       // from lists

struct BeamArgs {
  const char* logits;
  int64_t row_stride;  // elements
  int rows, beams, V, nblk;
  int chunks;  // of a row
  int spans;   // of a row
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
  float2* part_ms;  // [rows][spans]
  float* smax;      // [rows][spans], with a mask: the largest allowed logit (without: part_ms.x)
  float* bmax;      // [rows][nblk]
  uint32_t* dev_status;
  uint64_t wait_ns;
  // lists
  const int32_t* ids;
  const float* lps;
  int n;
};

// Inputs are read through L2: this grid may start before the kernel that writes them ends, and an L1 line could be
// of before.
__device__ __forceinline__ bool mask_allows(const uint32_t* words, int v) {
  return (__ldcg(words + (v >> 5)) >> (v & 31)) & 1u;
}
template <typename T>
__device__ __forceinline__ float logit_at(const char* base, int64_t i) {
  if constexpr (sizeof(T) == 4) {
    return __ldcg(reinterpret_cast<const float*>(base) + i);
  } else {
    const uint16_t b = __ldcg(reinterpret_cast<const uint16_t*>(base) + i);
    return Vec16<T>::at(&b, 0);
  }
}

// ---------------------------------------------------------------------------
// stream kernel
// ---------------------------------------------------------------------------
// A chunk is 128 bytes of a row for each consumer.  Rows need not begin on 16-byte boundaries: the copy begins
// on the one before (inside the same 16 bytes of memory), `skip` elements ahead, and a consumer looks at nine
// vectors in place of eight, the first `skip` elements of its first and the others of its last left out.
struct BeamStage {
  int row;   // < 0: no more chunks
  int lb;    // first block of the chunk in the row
  int ne;    // logits in the chunk
  int skip;  // elements of the stage before the first logit
};

// 16 bytes of logits as they count: element e is kept where bit e of `keep` is set, else -inf.
template <typename T>
__device__ __forceinline__ uint4 keep_elements(uint4 w, uint32_t keep) {
  if constexpr (sizeof(T) == 4) {
    w.x = keep & 1u ? w.x : Vec16<T>::kNegInfWord;
    w.y = keep & 2u ? w.y : Vec16<T>::kNegInfWord;
    w.z = keep & 4u ? w.z : Vec16<T>::kNegInfWord;
    w.w = keep & 8u ? w.w : Vec16<T>::kNegInfWord;
  } else {
    uint32_t* u = reinterpret_cast<uint32_t*>(&w);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t m = ((keep >> (2 * i)) & 1u ? 0xFFFFu : 0u) | ((keep >> (2 * i + 1)) & 1u ? 0xFFFF0000u : 0u);
      u[i] = (u[i] & m) | (Vec16<T>::kNegInfWord & ~m);
    }
  }
  return w;
}

// The sum of exp(x - m) over a vector, in two lanes: 2^(x L + by) with by = -(m L rounded); the caller makes up for
// that rounding, which all terms share (it would shift the row's lse).  FAR: 2^((x + by) L) with by = -m, one operation
// more a pair, for an m whose m L is rounded by more than can be made up for.
template <typename T, bool FAR>
__device__ __forceinline__ void add_exps(const uint4& w, float2 L2, float2 by, float2 (&acc)[2]) {
  constexpr int EPV = Vec16<T>::N;
  float2 p[EPV / 2];
  Vec16<T>::pairs(w, p);
#pragma unroll
  for (int q = 0; q < EPV / 2; ++q) {
    const float2 y = FAR ? __fmul2_rn(__fadd2_rn(p[q], by), L2) : __ffma2_rn(p[q], L2, by);
    acc[q & 1] = __fadd2_rn(acc[q & 1], make_float2(ex2_approx(y.x), ex2_approx(y.y)));
  }
}

template <typename T, bool MASK>
__global__ void __launch_bounds__(kBSThreads, kBSCtasPerSm) beam_stream_kernel(const BeamArgs a) {
  using VT = Vec16<T>;
  constexpr int ES = static_cast<int>(sizeof(T));
  constexpr int EPV = VT::N;               // elements of a vector
  constexpr int EPT = 128 / ES;            // of a consumer
  constexpr int TPB = kBlock / EPT;        // consumers of a block of 64 (1, or 2 for fp32)
  constexpr int CH = kBSConsumers / TPB;   // blocks of a chunk
  constexpr int S = kBSStages;
  extern __shared__ __align__(128) unsigned char smem[];
  BeamStage* desc = reinterpret_cast<BeamStage*>(smem + S * kBSStageBytes);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + S * kBSStageBytes + S * 32);
  uint64_t* empty = full + S;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(empty + S);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], kBSConsumerWarps);
    }
    *abort_flag = 0;
    mbar_init_fence();
  }
  __syncthreads();
  pdl_launch_dependents();  // the choice may be scheduled; it waits for this grid's results

  if (warp == kBSConsumerWarps) {  // producer
    if (lane != 0) return;
    const int64_t total = static_cast<int64_t>(a.rows) * a.chunks;
    const uint64_t policy = l2_evict_first_policy();
    int64_t c = blockIdx.x;  // this CTA's chunks: every gridDim.x-th
    auto issue = [&](int s) {
      BeamStage& d = desc[s];
      if (c >= total) {
        d.row = -1;
        mbar_arrive(&full[s]);
        return false;
      }
      const int row = static_cast<int>(c / a.chunks);
      const int lb = static_cast<int>(c - static_cast<int64_t>(row) * a.chunks) * CH;
      const int ne = min(CH * kBlock, a.V - lb * kBlock);
      const char* src = a.logits + (static_cast<int64_t>(row) * a.row_stride + static_cast<int64_t>(lb) * kBlock) * ES;
      const uint32_t off = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(src) & 15u);
      d.row = row;
      d.lb = lb;
      d.ne = ne;
      d.skip = static_cast<int>(off) / ES;
      const uint32_t bytes = (off + static_cast<uint32_t>(ne * ES) + 15u) & ~15u;
      mbar_arrive_expect_tx(&full[s], bytes);
      bulk_load_hint(smem + s * kBSStageBytes, src - off, bytes, &full[s], policy);
      c += gridDim.x;
      return true;
    };
    // The first S chunks go out before the grid-dependency wait (they read logits only; see lmh.h), the others
    // behind it.  With ended beams all go out behind it, where the flags may be read: an ended beam's logits are not.
    uint32_t issued = 0;
    bool ended = false;
    const uint32_t ahead = a.finished ? 0u : static_cast<uint32_t>(S);
    for (; issued < ahead && !ended; ++issued) ended = !issue(static_cast<int>(issued));
    pdl_wait();
    for (; !ended; ++issued) {
      const int s = static_cast<int>(issued % S);
      if (!wait_or_abort(&empty[s], ((issued / S) & 1u) ^ 1u, abort_flag, a.dev_status, a.wait_ns)) break;
      if (a.finished)
        while (c < total && __ldcg(a.finished + c / a.chunks)) c += gridDim.x;
      ended = !issue(s);
    }
    // copies still in flight (after an abort) land before the CTA exits
    const uint32_t first = issued > static_cast<uint32_t>(S) ? issued - S : 0u;
    for (uint32_t i = first; i < issued; ++i) mbar_wait(&full[i % S], (i / S) & 1u);
    return;
  }

  const int rot = tid & 7;  // vector order turned by lane: no bank conflict
  const uint64_t keep_policy = l2_evict_last_policy();
  const float L = kLog2e;
  pdl_wait();  // the workspace may be written
  for (uint32_t i = 0;; ++i) {
    const int s = static_cast<int>(i % S);
    const bool ok = wait_or_abort(&full[s], (i / S) & 1u, abort_flag, a.dev_status, a.wait_ns);
    if (!__all_sync(0xffffffffu, ok)) break;
    const BeamStage d = desc[s];
    if (d.row < 0) break;
    const int ne_t = min(max(d.ne - tid * EPT, 0), EPT);  // this thread's logits
    uint64_t allowed = ~0ull;
    if constexpr (MASK) {  // (asked for before the stage is read)
      const uint32_t* m = a.mask + static_cast<int64_t>(d.row) * a.mask_words;
      const int word = (d.lb * kBlock + tid * EPT) / 32;
      allowed = 0;
      if (ne_t > 0) allowed = __ldcg(m + word);
      if (EPT == 64 && ne_t > 32) allowed |= static_cast<uint64_t>(__ldcg(m + word + 1)) << 32;
    }
    const unsigned char* mine = smem + s * kBSStageBytes + tid * 128;
    uint4 w[8], w8 = make_uint4(VT::kNegInfWord, VT::kNegInfWord, VT::kNegInfWord, VT::kNegInfWord);
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = *reinterpret_cast<const uint4*>(mine + ((j + rot) & 7) * 16);
    if (d.skip) w8 = *reinterpret_cast<const uint4*>(mine + 128);
    __syncwarp();
    if (lane == 0) mbar_arrive(&empty[s]);
    if (d.skip || ne_t < EPT) {  // element x of vector v is logit v * EPV + x - skip of the thread
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int first = ((j + rot) & 7) * EPV - d.skip;
        uint32_t keep = 0;
#pragma unroll
        for (int x = 0; x < EPV; ++x) keep |= (first + x >= 0 && first + x < ne_t ? 1u : 0u) << x;
        w[j] = keep_elements<T>(w[j], keep);
      }
      uint32_t keep = 0;
#pragma unroll
      for (int x = 0; x < EPV; ++x) keep |= (x < d.skip && EPT - d.skip + x < ne_t ? 1u : 0u) << x;
      w8 = keep_elements<T>(w8, keep);
    }
    float tail = -INFINITY;  // of the ninth vector
    if (d.skip) {
      float x[EPV];
      VT::unpack(w8, x);
#pragma unroll
      for (int e = 0; e < EPV; ++e) tail = fmaxf(tail, x[e]);
    }
    float vm = fmaxf(VT::max8(w), tail);  // (NaN is dropped)
    vm = vm == vm ? vm : -INFINITY;
    float bm = vm;
    if constexpr (MASK) {
      bm = -INFINITY;
      if (allowed) {
        uint4 k[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int first = ((j + rot) & 7) * EPV - d.skip;
          k[j] = keep_elements<T>(w[j], static_cast<uint32_t>(first >= 0 ? allowed >> first : allowed << -first));
        }
        bm = VT::max8(k);
        if (d.skip) {
          float x[EPV];
          VT::unpack(keep_elements<T>(w8, static_cast<uint32_t>(allowed >> (EPT - d.skip))), x);
#pragma unroll
          for (int e = 0; e < EPV; ++e) bm = fmaxf(bm, x[e]);
        }
        bm = bm == bm ? bm : -INFINITY;
      }
    }
    const float smx = MASK ? warp_max(bm) : 0.0f;
    const float M = warp_max(vm);
    if (TPB == 2) bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, 1));
    const int b = d.lb + tid / TPB;
    if (tid % TPB == 0 && b < a.nblk) st_keep(a.bmax + static_cast<int64_t>(d.row) * a.nblk + b, bm, keep_policy);
    float ts = 0.0f;  // sum of exp(x - vm) over this thread's logits
    if (vm > -INFINITY) {
      const float ml = vm * L, shift = fmaf(vm, L, -ml);  // what the rounding of ml left
      auto sum_of = [&](auto far_const, float by) {
        constexpr bool FAR = decltype(far_const)::value;
        const float2 L2 = make_float2(L, L), by2 = make_float2(by, by);
        float2 acc0[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
        float2 acc1[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
          add_exps<T, FAR>(w[j], L2, by2, acc0);
          add_exps<T, FAR>(w[j + 1], L2, by2, acc1);
        }
        if (d.skip) add_exps<T, FAR>(w8, L2, by2, acc0);
        const float2 r = __fadd2_rn(__fadd2_rn(acc0[0], acc0[1]), __fadd2_rn(acc1[0], acc1[1]));
        return r.x + r.y;
      };
      // 2^-shift as 1 - shift ln 2, off by 2^-26 at the limit (|vm| to 5678 is always within it; 1e9 has a shift of 18)
      if (fabsf(shift) <= 2.44140625e-4f) {
        ts = sum_of(std::false_type{}, -ml);
        ts = fmaf(ts, shift * -0.6931471805599453f, ts);
      } else {
        ts = sum_of(std::true_type{}, -vm);
      }
      if (!(ts < INFINITY)) {  // +inf or NaN among the logits: one by one
        ts = 0.0f;
#pragma unroll
        for (int j = 0; j < 9; ++j) {
          float x[EPV];
          VT::unpack(j < 8 ? w[j & 7] : w8, x);
#pragma unroll
          for (int e = 0; e < EPV; ++e) {
            if (vm == INFINITY) ts += x[e] == INFINITY ? 1.0f : 0.0f;
            else ts += x[e] == x[e] ? ex2_approx((x[e] - vm) * L) : 0.0f;
          }
        }
      }
    }
    // the span's pair
    const float sc = warp_sum(vm == -INFINITY ? 0.0f : vm == M ? ts : M == INFINITY ? 0.0f : ts * ex2_approx((vm - M) * L));
    const int span = d.lb / (CH / kBSConsumerWarps) + warp;
    if (lane == 0 && span < a.spans) {
      const int64_t at = static_cast<int64_t>(d.row) * a.spans + span;
      a.part_ms[at] = make_float2(M, sc);
      if constexpr (MASK) a.smax[at] = smx;
    }
  }
}

// ---------------------------------------------------------------------------
// choice of a group
// ---------------------------------------------------------------------------
// A score as a whole number of the same order (scores are above -inf and not NaN; 0 is none).
__device__ __forceinline__ uint64_t score_key(double s) {
  const uint64_t u = static_cast<uint64_t>(__double_as_longlong(s + 0.0));  // (-0 becomes +0)
  return (u >> 63) ? ~u : u | (1ull << 63);
}
__device__ __forceinline__ float key_score(uint64_t k) {
  return static_cast<float>(__longlong_as_double(static_cast<long long>((k >> 63) ? k & ~(1ull << 63) : ~k)));
}
// (key, at) goes before (key2, at2); at: beam * V + token (lists: beam * n + place)
__device__ __forceinline__ bool before(uint64_t k, uint32_t at, uint64_t k2, uint32_t at2) {
  return k > k2 || (k == k2 && at < at2);
}

enum RowState : uint8_t { kRowNone = 0, kRowNormal = 1, kRowPlusInf = 2, kRowEnded = 3 };

template <int NT>
struct ChoiceSmem {
  uint64_t key[kBGCand];
  uint32_t at[kBGCand];
  float z[kBGCand];        // the candidate's logit, until its key is made
  uint8_t beam[kBGCand];
  uint64_t res_key[kBeamsMaxRows];
  uint32_t res_at[kBeamsMaxRows];
  uint8_t res_beam[kBeamsMaxRows];
  double off[kBeamsMaxRows];   // cum - log sum exp(z - M) of the group's rows
  float offf[kBeamsMaxRows];
  float top_z[kBeamsMaxRows];  // M, their largest logit
  uint8_t state[kBeamsMaxRows];
  int first[kBeamsMaxRows];    // keep_slots: the candidate in a place, or -1
  int slot[kBeamsMaxRows];     // keep_slots: a candidate's place
  uint64_t wkey[NT / 32];
  uint32_t wat[NT / 32];
  uint32_t count, spans, blocks, real;
  alignas(16) uint32_t top[NT / 32 * 64];
  uint32_t bound;
  float off_max;  // the largest off of a row that goes on, if above 0
  uint32_t kept_spans[kBGKept];
  uint32_t kept_blocks[kBGKept];
};

// Orders sm.key/at[0 .. cnt) into sm.res_*[0 .. min(cnt, k)): eight threads a candidate count those before it.
template <int NT>
__device__ __noinline__ void rank_candidates(ChoiceSmem<NT>& sm, int cnt, int k) {
  const int sub = threadIdx.x % 8;
  for (int base = 0; base < cnt; base += NT / 8) {
    const int i = base + static_cast<int>(threadIdx.x) / 8;
    const uint64_t key = i < cnt ? sm.key[i] : 0;
    const uint32_t at = i < cnt ? sm.at[i] : 0;
    int rank = 0;
#pragma unroll 1
    for (int j = sub; j < cnt; j += 8) rank += before(sm.key[j], sm.at[j], key, at);
    rank += __shfl_xor_sync(0xffffffffu, rank, 1);
    rank += __shfl_xor_sync(0xffffffffu, rank, 2);
    rank += __shfl_xor_sync(0xffffffffu, rank, 4);
    if (i < cnt && sub == 0 && rank < k) {
      sm.res_key[rank] = key;
      sm.res_at[rank] = at;
      sm.res_beam[rank] = sm.beam[i];
    }
  }
}

// Writes the group's k results (the first `cnt` of sm.res_* are real).  `token(at, beam)` gives a token.
template <int NT, typename Token>
__device__ __forceinline__ void write_results(const BeamArgs& a, ChoiceSmem<NT>& sm, int group, int cnt, Token token) {
  const int k = a.k;
  const int64_t base = static_cast<int64_t>(group) * k;
  auto beam_of = [&](int r) { return r < cnt ? static_cast<int>(sm.res_beam[r]) : -1; };
  if (a.keep_slots) {  // k == beams <= NT
    const int r = threadIdx.x;
    if (r < k) sm.first[r] = -1;
    __syncthreads();
    bool first = false;
    if (r < cnt) {
      first = true;
      const int b = beam_of(r);
      for (int j = 0; j < r; ++j) first &= beam_of(j) != b;
      if (first) sm.first[b] = r;
    }
    __syncthreads();
    if (r < k && !first) {  // the turn-th candidate that is no first child takes the turn-th free place
      int turn = 0;
      for (int j = 0; j < r; ++j) {
        const int b = beam_of(j);
        turn += b < 0 || sm.first[b] != j;
      }
      int slot = 0;
      for (int t = 0; slot < k; ++slot)
        if (sm.first[slot] < 0 && t++ == turn) break;
      sm.slot[r] = slot;
    } else if (r < k) {
      sm.slot[r] = beam_of(r);
    }
    __syncthreads();
  }
  for (int r = threadIdx.x; r < k; r += NT) {
    const int64_t to = base + (a.keep_slots ? sm.slot[r] : r);
    const int b = beam_of(r);
    a.out_scores[to] = b < 0 ? -INFINITY : key_score(sm.res_key[r]);
    a.out_parents[to] = b < 0 ? -1 : group * a.beams + b;
    a.out_tokens[to] = b < 0 ? -1 : (sm.state[b] == kRowEnded ? a.pad_id : token(sm.res_at[r], b));
  }
  if (cnt == 0 && threadIdx.x == 0) set_status(a.dev_status, LMH_DS_NO_ALLOWED_TOKEN);
}

// The k best by repeatedly taking the best that is left: exact for any number of ties, used where the
// candidates do not fit.  `scan(key, at, last_key, last_at)` puts the thread's best item behind (last_key, last_at)
// into (key, at), key = 0 for none.  Returns the number found.
template <int NT, typename Scan>
__device__ __noinline__ int take_in_turn(ChoiceSmem<NT>& sm, int k, uint32_t per_beam, Scan scan) {
  uint64_t last = ~0ull, key = 0;
  uint32_t last_at = 0, at = 0xFFFFFFFFu;
  bool stale = true;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int r = 0;
  for (; r < k; ++r) {
    if (stale) scan(key, at, last, last_at);
    uint64_t bk = key;
    uint32_t bat = at;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const uint64_t ok = __shfl_xor_sync(0xffffffffu, bk, o);
      const uint32_t oat = __shfl_xor_sync(0xffffffffu, bat, o);
      if (before(ok, oat, bk, bat)) bk = ok, bat = oat;
    }
    __syncthreads();
    if (lane == 0) sm.wkey[warp] = bk, sm.wat[warp] = bat;
    __syncthreads();
    bk = sm.wkey[0], bat = sm.wat[0];
#pragma unroll
    for (int w = 1; w < NT / 32; ++w)
      if (before(sm.wkey[w], sm.wat[w], bk, bat)) bk = sm.wkey[w], bat = sm.wat[w];
    if (bk == 0) break;
    if (threadIdx.x == 0) sm.res_key[r] = bk, sm.res_at[r] = bat, sm.res_beam[r] = static_cast<uint8_t>(bat / per_beam);
    last = bk, last_at = bat;
    stale = key == bk && at == bat;  // (the pair is one thread's alone)
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

// a + b and what its rounding left
__device__ __forceinline__ void two_sum(float& s, float& c, float b) {
  const float t = s + b, z = t - s;
  c += (s - (t - z)) + (b - z);
  s = t;
}

// sm.bound = a value that at least k of the threads' values reach, or 0 if they are fewer (values: order-preserving
// whole numbers, 0 for none): of every warp the q largest of its threads' two largest (q warps >= k), of those the
// k-th, which every thread counts for a value.  Two barriers.
template <int NT>
__device__ __noinline__ void bound_of(ChoiceSmem<NT>& sm, uint32_t k1, uint32_t k2, int k) {
  constexpr int W = NT / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int q = min(64, max(2, (4 * k + W - 1) / W));
  for (int r = 0; r < q; ++r) {
    const uint32_t m = __reduce_max_sync(0xffffffffu, k1);
    const unsigned holders = __ballot_sync(0xffffffffu, k1 == m);
    if (lane == __ffs(holders) - 1) {
      sm.top[warp * q + r] = m;
      k1 = k2;
      k2 = 0;
    }
  }
  __syncthreads();
  const int nv = W * q;  // a multiple of 4
  for (int i = threadIdx.x; i < nv; i += NT) {
    const uint32_t v = sm.top[i];
    int rank = 0;
    for (int j = 0; j < nv; j += 4) {
      const uint4 o = *reinterpret_cast<const uint4*>(&sm.top[j]);
      rank += (o.x > v || (o.x == v && j < i)) + (o.y > v || (o.y == v && j + 1 < i)) +
              (o.z > v || (o.z == v && j + 2 < i)) + (o.w > v || (o.w == v && j + 3 < i));
    }
    if (rank == k - 1) sm.bound = v;
  }
  __syncthreads();
}

// Leaves, of the candidates sm.key/at[0 .. cnt), those that a bound on the upper halves of their keys lets through:
// hardly more than k.  Returns how many.
template <int NT>
__device__ __noinline__ int thin_candidates(ChoiceSmem<NT>& sm, int cnt, int k) {
  constexpr int MOST = kBGCand / NT;
  uint64_t key[MOST];
  uint32_t at[MOST], k1 = 0, k2 = 0;
  uint8_t beam[MOST];
#pragma unroll
  for (int u = 0; u < MOST; ++u) {
    const int i = u * NT + static_cast<int>(threadIdx.x);
    key[u] = i < cnt ? sm.key[i] : 0;
    at[u] = i < cnt ? sm.at[i] : 0;
    beam[u] = i < cnt ? sm.beam[i] : 0;
    const uint32_t h = static_cast<uint32_t>(key[u] >> 32);
    k2 = max(k2, min(k1, h));
    k1 = max(k1, h);
  }
  bound_of(sm, k1, k2, k);
  const uint32_t t = sm.bound;
  if (threadIdx.x == 0) sm.count = 0;
  __syncthreads();
#pragma unroll
  for (int u = 0; u < MOST; ++u)
    if (key[u] != 0 && static_cast<uint32_t>(key[u] >> 32) >= t) {
      const uint32_t p = atomicAdd(&sm.count, 1u);
      sm.key[p] = key[u];
      sm.at[p] = at[u];
      sm.beam[p] = beam[u];
    }
  __syncthreads();
  return static_cast<int>(sm.count);
}

template <typename T>
__global__ void __launch_bounds__(kBGThreads) beam_choose_kernel(const BeamArgs a) {
  constexpr int NT = kBGThreads;
  constexpr int SB = 32 / (kBlock / (128 / static_cast<int>(sizeof(T))));  // blocks of a span
  extern __shared__ __align__(16) unsigned char smem_raw[];
  ChoiceSmem<NT>& sm = *reinterpret_cast<ChoiceSmem<NT>*>(smem_raw);
  const int group = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int B = a.beams, nblk = a.nblk, P = a.spans;
  const int row0 = group * B;
  pdl_wait();
  if (tid == 0) sm.count = 0, sm.spans = 0, sm.blocks = 0, sm.real = 0, sm.off_max = 0.0f;

  // ---- the rows' cum - log sum exp(z - M) ----
  // 32 bits but for the last sum: the terms are good to 2^-23, the sum carries what its roundings leave, and
  // log S = e ln 2 + log f with f next to 1, whose 32-bit logarithm is off by 2^-25.
  for (int b = warp; b < B; b += kBGWarps) {
    const int row = row0 + b;
    const float cum = __ldcg(a.cum + row);
    const bool ended = a.finished && __ldcg(a.finished + row);
    const float2* ms = a.part_ms + static_cast<int64_t>(row) * P;
    float M = -INFINITY, S = 0.0f, c = 0.0f;
    if (!ended) {
      float2 p[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) p[u] = u * 32 + lane < P ? __ldcg(ms + u * 32 + lane) : make_float2(-INFINITY, 0.0f);
#pragma unroll
      for (int u = 0; u < 4; ++u) M = fmaxf(M, p[u].x);
      for (int j = 128 + lane; j < P; j += 32) M = fmaxf(M, __ldcg(ms + j).x);
      M = warp_max(M);
      auto add = [&](float2 q) {
        if (q.x == M) two_sum(S, c, q.x > -INFINITY ? q.y : 0.0f);
        else if (q.x > -INFINITY && M < INFINITY) two_sum(S, c, q.y * exp2f((q.x - M) * kLog2e));
      };
#pragma unroll
      for (int u = 0; u < 4; ++u) add(p[u]);
      for (int j = 128 + lane; j < P; j += 32) add(__ldcg(ms + j));
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const float s2 = __shfl_xor_sync(0xffffffffu, S, o), c2 = __shfl_xor_sync(0xffffffffu, c, o);
        two_sum(S, c, s2);
        c += c2;
      }
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
        int e;
        float f = frexpf(S, &e);
        if (f < 0.70710678f) f *= 2.0f, --e;
        off = static_cast<double>(cum) - (e * 0.69314718055994530942 + static_cast<double>(logf(f) + c / S));
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
      sm.z[i] = 0.0f;
      sm.beam[i] = static_cast<uint8_t>(tid);
      sm.at[i] = static_cast<uint32_t>(tid) * static_cast<uint32_t>(a.V);
    } else {
      atomicMax(reinterpret_cast<int*>(&sm.off_max), __float_as_int(fmaxf(sm.offf[tid], 0.0f)));
    }
  }
  auto score32 = [&](int b, float z) -> float {
    const uint8_t st = sm.state[b];
    return st == kRowNormal || st == kRowPlusInf ? below_top<float>(st, z, sm.top_z[b]) + sm.offf[b] : -INFINITY;
  };
  auto key_of = [&](int b, float z) -> uint64_t {  // 0: no continuation
    const uint8_t st = sm.state[b];
    const double s = st == kRowEnded ? sm.off[b] : sm.off[b] + below_top<double>(st, z, sm.top_z[b]);
    return static_cast<float>(s) > -INFINITY ? score_key(s) : 0;
  };
  const float* bm = a.bmax + static_cast<int64_t>(row0) * nblk;
  const int64_t span0 = static_cast<int64_t>(row0) * P;
  // Twice the same: items 0 .. n - 1, first the group's spans, then the blocks of the kept spans (item i: block i % SB
  // of kept span i / SB), of which those that reach a bound that k of them reach are listed.  A thread holds its first
  // values between its two looks.  The k-th best score is at least the bound t but for fp32's rounding of it and of the
  // sums compared with it.  A sum (z - M) + off is off by 2^-24 of its terms and of itself; z - M is not above 0, so that
  // is 2^-23 |score| for off <= 0, and 2^-23 (|score| + off) above.  Scores next to t have no other size than t, or
  // than the largest off above 0: 2^-21 (|t| + that off) is twice what both need.  (A beam far below, as those that
  // are not the first have when a search begins, widens nothing.  With its |off| in the margin, 4 beams of 151936 fp32
  // logits overflowed the lists: 1490 us for this kernel, 14 so.)
  float t = -INFINITY;
  bool fits = true;
  int n_blocks = 0;
#pragma unroll 1
  for (int level = 0; level < 2 && fits; ++level) {
    const int n = level == 0 ? B * P : static_cast<int>(sm.spans) * SB;
    auto value = [&](int i) -> float {
      int span = i, blk = 0;
      if (level) {
        span = static_cast<int>(sm.kept_spans[i / SB]);
        blk = i % SB;
      }
      const int b = span / P;
      const float* p = a.mask ? a.smax + span0 + span : &a.part_ms[span0 + span].x;
      if (level) {
        blk += (span - b * P) * SB;
        if (blk >= nblk) return -INFINITY;
        p = bm + static_cast<int64_t>(b) * nblk + blk;
      }
      return score32(b, __ldcg(p));
    };
    float m1 = -INFINITY, m2 = -INFINITY, held[kBGHeld];
#pragma unroll
    for (int u = 0; u < kBGHeld; ++u) held[u] = u * NT + tid < n ? value(u * NT + tid) : -INFINITY;
    auto top2 = [&](float v) {
      m2 = fmaxf(m2, fminf(m1, v));
      m1 = fmaxf(m1, v);
    };
#pragma unroll
    for (int u = 0; u < kBGHeld; ++u) top2(held[u]);
#pragma unroll 1
    for (int i = kBGHeld * NT + tid; i < n; i += NT) top2(value(i));
    bound_of(sm, m1 > -INFINITY ? f32_ord(m1) : 0u, m2 > -INFINITY ? f32_ord(m2) : 0u, a.k);
    t = sm.bound ? ord_f32(sm.bound) : -INFINITY;
    if (t > -INFINITY) t -= (fabsf(t) + sm.off_max) * 4.76837158203125e-7f;  // 2^-21
    uint32_t* list = level ? sm.kept_blocks : sm.kept_spans;
    uint32_t* count = level ? &sm.blocks : &sm.spans;
    auto keep = [&](int i, float v) {
      if (v >= t && v > -INFINITY) {
        const uint32_t p = atomicAdd(count, 1u);
        if (p < kBGKept) list[p] = static_cast<uint32_t>(i);
      }
    };
#pragma unroll
    for (int u = 0; u < kBGHeld; ++u) keep(u * NT + tid, held[u]);
#pragma unroll 1
    for (int i = kBGHeld * NT + tid; i < n; i += NT) keep(i, value(i));
    __syncthreads();
    n_blocks = static_cast<int>(*count);
    fits = n_blocks <= kBGKept;
  }
  auto logit = [&](int b, int v) -> float {  // -inf for a token that is not allowed
    const int row = row0 + b;
    if (a.mask && !mask_allows(a.mask + static_cast<int64_t>(row) * a.mask_words, v)) return -INFINITY;
    const float z = logit_at<T>(a.logits, static_cast<int64_t>(row) * a.row_stride + v);
    return z == z ? z : -INFINITY;
  };
  int cnt = 0;
  if (fits) {
#pragma unroll 1
    for (int j = tid; j < n_blocks * kBlock; j += NT) {
      const int i = static_cast<int>(sm.kept_blocks[j / kBlock]);
      const int span = static_cast<int>(sm.kept_spans[i / SB]), b = span / P;
      const int v = ((span - b * P) * SB + i % SB) * kBlock + j % kBlock;
      if (v >= a.V) continue;
      const float z = logit(b, v);
      const float f = score32(b, z);
      if (!(f >= t) || !(f > -INFINITY)) continue;
      const uint32_t p = atomicAdd(&sm.count, 1u);
      if (p < kBGCand) {
        sm.z[p] = z;
        sm.beam[p] = static_cast<uint8_t>(b);
        sm.at[p] = static_cast<uint32_t>(b) * static_cast<uint32_t>(a.V) + static_cast<uint32_t>(v);
      }
    }
    __syncthreads();
    cnt = static_cast<int>(sm.count);
    fits = cnt <= kBGCand;
  }
  if (fits) {
    // (64 bits only here, in few warps)
    for (int i = tid; i < cnt; i += NT) {
      const uint64_t key = key_of(sm.beam[i], sm.z[i]);
      sm.key[i] = key;
      if (key) atomicAdd(&sm.real, 1u);
    }
    __syncthreads();
    const int real = static_cast<int>(sm.real);
    if (cnt > 128 && cnt > a.k) cnt = thin_candidates(sm, cnt, a.k);
    rank_candidates(sm, cnt, a.k);
    cnt = min(real, a.k);
    __syncthreads();
  } else {
    // a thread's blocks are a contiguous share, looked through again only after its best is taken
    const int nb = B * nblk, per = (nb + NT - 1) / NT;
    const int lo = min(nb, tid * per), hi = min(nb, lo + per);
    cnt = take_in_turn(sm, a.k, static_cast<uint32_t>(a.V), [&](uint64_t& key, uint32_t& at, uint64_t last, uint32_t last_at) {
      key = 0;
      at = 0xFFFFFFFFu;
      for (int i = lo; i < hi; ++i) {
        const int b = i / nblk, blk = i - b * nblk;
        const uint8_t st = sm.state[b];
        const uint32_t e0 = static_cast<uint32_t>(b) * static_cast<uint32_t>(a.V);
        if (st == kRowNone) continue;
        if (st == kRowEnded) {
          const uint64_t c = score_key(sm.off[b]);
          if (blk == 0 && before(last, last_at, c, e0) && before(c, e0, key, at)) key = c, at = e0;
          continue;
        }
        // (an equal score further on comes after the one that is held)
        const uint64_t most = key_of(b, __ldcg(bm + i));
        for (int v = blk * kBlock; most > key && v < min(a.V, (blk + 1) * kBlock); ++v) {
          const uint64_t c = key_of(b, logit(b, v));
          const uint32_t e = e0 + static_cast<uint32_t>(v);
          if (c > key && before(last, last_at, c, e)) key = c, at = e;
        }
      }
    });
  }
  write_results(a, sm, group, cnt,
                [&](uint32_t at, int b) { return static_cast<int32_t>(at - static_cast<uint32_t>(b) * static_cast<uint32_t>(a.V)); });
}

// ---------------------------------------------------------------------------
// from top-k lists
// ---------------------------------------------------------------------------
// One CTA a group; 64 groups of 4 lists of 20: 5 us in a graph, 9 us alone, latency.
__global__ void __launch_bounds__(kBLThreads) beam_lists_kernel(const BeamArgs a) {
  constexpr int NT = kBLThreads;
  extern __shared__ __align__(16) unsigned char smem_raw[];
  ChoiceSmem<NT>& sm = *reinterpret_cast<ChoiceSmem<NT>*>(smem_raw);
  const int group = blockIdx.x, tid = threadIdx.x;
  const int B = a.beams, n = a.n, row0 = group * B;
  pdl_wait();
  const int64_t e0 = static_cast<int64_t>(row0) * n;
  const int total = B * n;
  // the first entries are on their way while the rows' scores arrive
  const int id0 = tid < total ? __ldcg(a.ids + e0 + tid) : -1;
  const float lp0 = tid < total ? __ldcg(a.lps + e0 + tid) : 0.0f;
  if (tid == 0) sm.count = 0;
  if (tid < B) {
    const float cum = __ldcg(a.cum + row0 + tid);
    const bool fin = cum > -INFINITY && cum < INFINITY;
    sm.state[tid] = !fin ? kRowNone : (a.finished && __ldcg(a.finished + row0 + tid)) ? kRowEnded : kRowNormal;
    sm.off[tid] = cum;
  }
  __syncthreads();
  // the key of entry i of the group's lists; 0 for none
  auto entry = [&](int i, int id, float lp) -> uint64_t {
    const int b = i / n;
    const uint8_t st = sm.state[b];
    if (st == kRowEnded) return i == b * n ? score_key(sm.off[b]) : 0;
    if (st == kRowNone || id < 0 || !(lp > -INFINITY && lp < INFINITY)) return 0;
    const double s = sm.off[b] + static_cast<double>(lp);
    return static_cast<float>(s) > -INFINITY ? score_key(s) : 0;
  };
  auto key_at = [&](int i) { return i == tid ? entry(i, id0, lp0) : entry(i, __ldcg(a.ids + e0 + i), __ldcg(a.lps + e0 + i)); };
  uint32_t least = 0;  // of a key's upper half
  if (total > kBGCand) {  // more than the list holds: those that a bound lets through
    uint32_t k1 = 0, k2 = 0;
    for (int i = tid; i < total; i += NT) {
      const uint32_t h = static_cast<uint32_t>(key_at(i) >> 32);
      k2 = max(k2, min(k1, h));
      k1 = max(k1, h);
    }
    bound_of(sm, k1, k2, a.k);
    least = sm.bound;
  }
  for (int i = tid; i < total; i += NT) {
    const uint64_t key = key_at(i);
    if (key && static_cast<uint32_t>(key >> 32) >= least) {
      const uint32_t p = atomicAdd(&sm.count, 1u);
      if (p < kBGCand) sm.key[p] = key, sm.at[p] = static_cast<uint32_t>(i), sm.beam[p] = static_cast<uint8_t>(i / n);
    }
  }
  __syncthreads();
  int cnt = static_cast<int>(sm.count);
  if (cnt <= kBGCand) {
    if (cnt > 128 && cnt > a.k) cnt = thin_candidates(sm, cnt, a.k);
    rank_candidates(sm, cnt, a.k);
    cnt = min(cnt, a.k);
    __syncthreads();
  } else {
    cnt = take_in_turn(sm, a.k, static_cast<uint32_t>(n), [&](uint64_t& key, uint32_t& at, uint64_t last, uint32_t last_at) {
      key = 0;
      at = 0xFFFFFFFFu;
      for (int i = tid; i < total; i += NT) {
        const uint64_t c = entry(i, __ldcg(a.ids + e0 + i), __ldcg(a.lps + e0 + i));
        const uint32_t e = static_cast<uint32_t>(i);
        if (c && before(last, last_at, c, e) && before(c, e, key, at)) key = c, at = e;
      }
    });
  }
  write_results(a, sm, group, cnt, [&](uint32_t at, int) { return __ldcg(a.ids + e0 + at); });
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
static size_t align_up(size_t n) { return (n + 255) & ~static_cast<size_t>(255); }

// Spans of a row: of 32 threads' 128 bytes; the workspace is sized for fp32's, the shortest.
static int beam_spans(int V, int es) { return static_cast<int>((static_cast<int64_t>(V) * es + 4095) / 4096); }

size_t beam_workspace_bytes(int rows, int V) {
  const size_t nblk = (static_cast<size_t>(V) + kBlock - 1) / kBlock;
  const size_t spans = static_cast<size_t>(rows) * static_cast<size_t>(beam_spans(V, 4));
  return align_up(spans * 8) + align_up(spans * 4) + align_up(static_cast<size_t>(rows) * nblk * 4);
}

template <typename T>
static cudaError_t beam_setup_one() {
  cudaError_t e = cudaFuncSetAttribute(beam_choose_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       sizeof(ChoiceSmem<kBGThreads>));
  for (auto* f : {beam_stream_kernel<T, false>, beam_stream_kernel<T, true>}) {
    if (e == cudaSuccess) e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, kBSSmem);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(f, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
  }
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(beam_choose_kernel<T>, cudaFuncAttributePreferredSharedMemoryCarveout,
                             cudaSharedmemCarveoutMaxShared);
  return e;
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
  a.wait_ns = wait_limit_ns();
  return a;
}

template <typename T>
static cudaError_t launch_beams(BeamArgs a, int groups, int num_sms, cudaStream_t stream) {
  constexpr int64_t per_chunk = kBSChunkBytes / static_cast<int>(sizeof(T));
  a.chunks = static_cast<int>((a.V + per_chunk - 1) / per_chunk);
  a.spans = beam_spans(a.V, sizeof(T));
  const int64_t chunks = static_cast<int64_t>(a.rows) * a.chunks, most = static_cast<int64_t>(num_sms) * kBSCtasPerSm;
  const dim3 grid(static_cast<unsigned>(chunks < most ? chunks : most));
  trace_begin(kTraceBeamStream, stream);
  cudaError_t e = launch_kernel(a.mask ? beam_stream_kernel<T, true> : beam_stream_kernel<T, false>, grid, dim3(kBSThreads),
                                static_cast<size_t>(kBSSmem), stream, true, a);
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
  a.mask = mask;
  a.mask_words = mask_words;
  const size_t spans = static_cast<size_t>(a.rows) * static_cast<size_t>(beam_spans(c.V, 4));
  char* p = static_cast<char*>(workspace);
  a.part_ms = reinterpret_cast<float2*>(p);
  p += align_up(spans * 8);
  a.smax = reinterpret_cast<float*>(p);
  p += align_up(spans * 4);
  a.bmax = reinterpret_cast<float*>(p);
  switch (dtype) {
    case LMH_BF16: return launch_beams<__nv_bfloat16>(a, c.groups, num_sms, stream);
    case LMH_F16: return launch_beams<__half>(a, c.groups, num_sms, stream);
    default: return launch_beams<float>(a, c.groups, num_sms, stream);
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
