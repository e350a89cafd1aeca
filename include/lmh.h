/*
 * lmh.h -- C ABI of liblmh, the LM-head logprob library for one NVIDIA GB300
 * GPU (sm_103a).
 *
 * The library computes the output-head hot path of LLM serving:
 *
 *   1. lmh_select_rows          pick the rows of a packed batch that are
 *                               sampled and emit compacted prefix sums;
 *   2. lmh_project_logprobs     gather those rows, project them through the
 *                               [hidden x vocab] head on the tensor cores and
 *                               reduce every row over the full vocabulary to
 *                               an O(k+1) result without writing the
 *                               [rows x vocab] logits to memory;
 *   3. lmh_logprobs_from_logits the same reduction for logits that already
 *                               exist (prompt scoring of logits chunks).
 *
 * lmh_project_partials and lmh_merge_records split step 2 over GPUs that each
 * hold a share of the vocabulary (a vocabulary-parallel head).
 *
 * For a decode step around a model body with a 4-bit head: lmh_lookup_q4 (the
 * input rows of token ids), lmh_project_q4 (the logits of the body's rows) and
 * lmh_sample_from_logits (the next ids, with temperature, top-k, top-p, min-p).
 *
 * For a step of beam search, or of requests with adapters of their own:
 * lmh_add_adapters (low-rank adapters of many requests beside a shared projection),
 * lmh_beam_select and lmh_beam_select_lists (each group's best continuations, from
 * logits or from the top-k lists of lmh_project_logprobs) and lmh_reorder_rows (the
 * beams' states follow their parents).
 *
 * The O(k+1) result of a row is: lse (fp32 log-sum-exp over the vocabulary),
 * the selected token's logprob, and the exact top-k (ids and logprobs),
 * sorted by logit descending with exact ties ordered by ascending token id.
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 * - Pointers named "device" are device memory owned by the caller (for
 *   example PyTorch tensors).  The library allocates no memory per call and
 *   keeps no per-call state; scratch memory is the caller's `workspace`.
 * - Every call is enqueued on `stream` and returns without waiting for the
 *   GPU: no host synchronisation and no device->host copy happens inside.
 * - Kernels are launched with programmatic dependent launch, so a call's
 *   first kernel may start while the kernel enqueued before it finishes.
 *   Before it waits for that kernel it reads only the head weights W (projection
 *   entry points) or the logits of its first chunks (logits entry points).  Those
 *   inputs must therefore not be written by a kernel enqueued right before the
 *   call that itself triggers programmatic dependent launch before writing them
 *   (ordinary kernels, and this library's own, do not).
 * - Host-side argument checks return an error status and launch nothing.
 *   Errors only visible on the device (bad cu_seqlens, an id out of range)
 *   set bits (LMH_DS_*) in the caller's optional `dev_status` word with an
 *   atomic OR; kernels never trap.  The caller zeroes that word.
 * - Matrices are row-major; `*_stride` arguments are in elements.
 * - The first call on a device of each family (head and reductions, draw, 4-bit
 *   projection, adapters, beams, states) performs a one-time set-up (kernel attributes, driver entry
 *   points) under a lock.
 */
#ifndef LMH_H
#define LMH_H

#include <stddef.h>
#include <stdint.h>

#include <cuda_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

#define LMH_VERSION 1

/* Largest k (top-k entries per row) any entry point accepts. */
#define LMH_K_MAX 128
/* Largest number of beams in a group. */
#define LMH_BEAMS_MAX 128
/* k_max = LMH_K_FULL asks for the full-vocabulary output: topk_logprobs
 * receives [rows x V] logprobs in token-id order and topk_ids is not written
 * (openinfer issue #719, "Acceptance criteria": the -1 behaviour is the
 * frontend's full-vocabulary contract). */
#define LMH_K_FULL (-1)

typedef enum lmh_status {
    LMH_OK = 0,
    LMH_ERR_INVALID_ARG = 1,         /* null required pointer, bad size, k > vocab, ... */
    LMH_ERR_UNSUPPORTED = 2,         /* valid request this version does not implement    */
    LMH_ERR_WORKSPACE_TOO_SMALL = 3, /* workspace_bytes < lmh_workspace_bytes(...)       */
    LMH_ERR_CUDA = 4,                /* a CUDA runtime/driver call failed                 */
    LMH_ERR_TIMEOUT = 5              /* reserved: device waits report LMH_DS_TIMEOUT      */
} lmh_status;

typedef enum lmh_dtype { LMH_BF16 = 0, LMH_F16 = 1, LMH_F32 = 2 } lmh_dtype;

/* Storage of the head weight W, whose math shape is [H x V]. */
typedef enum lmh_w_layout {
    LMH_W_VH = 0, /* stored [V x H] row-major: PyTorch lm_head.weight (H contiguous) */
    LMH_W_HV = 1  /* stored [H x V] row-major (V contiguous; V % 8 == 0)            */
} lmh_w_layout;

/* Which entry point a workspace is sized for. */
typedef enum lmh_path { LMH_PATH_PROJECT = 0, LMH_PATH_FROM_LOGITS = 1, LMH_PATH_PROBE = 2 } lmh_path;

/* Device status bits (OR-ed into *dev_status). */
#define LMH_DS_BAD_CU_SEQLENS 0x1u       /* cu[0] != 0, cu decreasing, or an empty prefill segment */
#define LMH_DS_SEL_OUT_OF_RANGE 0x2u     /* a selected id outside [0, V) other than -1 (row gets NaN) */
#define LMH_DS_ROWS_OVERFLOW 0x4u        /* more selected rows than max_out_rows (extra rows dropped) */
#define LMH_DS_ROW_IDX_OUT_OF_RANGE 0x8u /* a row index outside [0, num_tokens) (row reads zeros)   */
#define LMH_DS_TIMEOUT 0x10u             /* a bounded device-side wait gave up (kernel returned)     */
#define LMH_DS_NO_ALLOWED_TOKEN 0x20u    /* sampling: a row's mask allows no token (id -1, NaN); beams: a
                                            group has no continuation                               */
#define LMH_DS_ADAPTER_OUT_OF_RANGE 0x40u /* an adapter index outside [0, count) other than -1 (none is added) */

/*
 * lmh_select_rows -- which rows of a packed batch are sampled.
 *
 * Defined by the vllm-metal release v0.4.0.dev20260831, "Summary": decode
 * rows are kept; prefill segment j is sampled at its last row,
 * cu_seqlens[num_decode + j + 1] - 1; pure-decode steps are unchanged; since
 * logits are no longer row-aligned with the input, compacted prefix sums
 * (logits_cu_seqlens) are emitted while cu_seqlens itself stays valid for
 * other consumers.  Readings where the page is silent: a decode sequence of
 * several rows keeps all of them; all_rows_mask[s] != 0 keeps every row of
 * prefill segment s (prompt scoring of every position, openinfer issue #719,
 * "Description").
 *
 *   cu_seqlens        device int32 [num_seqs + 1], cu[0] = 0, non-decreasing.
 *   num_seqs          number of sequences S (>= 0).
 *   num_decode        sequences [0, num_decode) are decode sequences.
 *   all_rows_mask     device uint8 [num_seqs] or NULL (all zero).
 *   max_out_rows      capacity of row_idx.
 *   row_idx           device int32 [max_out_rows], out: selected rows, ascending.
 *   logits_cu_seqlens device int32 [num_seqs + 1], out: logits_cu[0] = 0,
 *                     logits_cu[s+1] = logits_cu[s] + rows taken from s.
 *   dev_status        device uint32 or NULL.
 * Bad cu_seqlens set LMH_DS_BAD_CU_SEQLENS; an offending sequence contributes
 * no row.  More than max_out_rows rows set LMH_DS_ROWS_OVERFLOW (the rows
 * beyond the capacity are dropped; logits_cu_seqlens keeps the full counts).
 * Errors: LMH_ERR_INVALID_ARG for null pointers, negative sizes or
 * num_decode > num_seqs.
 */
lmh_status lmh_select_rows(const int32_t* cu_seqlens, int32_t num_seqs, int32_t num_decode,
                           const uint8_t* all_rows_mask, int32_t max_out_rows, int32_t* row_idx,
                           int32_t* logits_cu_seqlens, uint32_t* dev_status, cudaStream_t stream);

/*
 * lmh_count_selected_rows -- host helper: the number of rows lmh_select_rows
 * selects, computed from a HOST copy of cu_seqlens / all_rows_mask, so that a
 * caller can size buffers and pass `rows` without a device synchronisation.
 * Returns -1 for an invalid batch (same rules as above).
 */
int32_t lmh_count_selected_rows(const int32_t* cu_seqlens_host, int32_t num_seqs,
                                int32_t num_decode, const uint8_t* all_rows_mask_host);

/*
 * lmh_workspace_bytes -- bytes of scratch the given entry point needs for
 * these sizes on the current device (the split of the vocabulary depends on
 * its SM count).  `hidden` is ignored for LMH_PATH_FROM_LOGITS.  Returns 0
 * for sizes the entry point rejects.  The workspace must be 256-byte aligned.
 */
size_t lmh_workspace_bytes(int32_t rows, int32_t hidden, int32_t vocab, int32_t k_max,
                           lmh_path path);

/*
 * lmh_project_logprobs -- selective head projection with a fused reduction.
 *
 * Defined by: vllm-metal release v0.4.0.dev20260831, "Summary" (gather the
 * sampled rows and run the head on those alone); mlxcel PR #1969 (the row
 * sliced before the head equals the full forward's row); MTPLX PR #532,
 * "Change" (one fp32 logsumexp per row, a 64-logit block-max prefilter for
 * the exact top-k, fp32(logit) - lse at the survivors and the scored token,
 * exact ties by ascending id); openinfer issue #719, "Suggested direction"
 * and "Acceptance criteria" (compute lse, the selected logprob and the top-k
 * on the device and return an O(k+1) result).
 *
 * For row i: A[i] = hidden[row_idx[i]] (or hidden[i] when row_idx is NULL),
 * z[i][v] = sum_h A[i][h] * W[h][v] with bf16 inputs and fp32 accumulation;
 * lse[i] = log sum_v exp(z[i][v]); sel_logprob[i] = z[i][sel] - lse[i];
 * topk_ids[i][r], topk_logprobs[i][r] for r < k_i = row_k[i] (or k_max):
 * the r-th best (z desc, id asc); ranks r >= k_i hold id -1 and -inf.
 *
 *   hidden            device bf16 [num_tokens x H], row stride hidden_row_stride
 *                     (>= H); 16-byte aligned base.
 *   num_tokens        rows of `hidden` (bounds for row_idx).
 *   row_idx           device int32 [rows] or NULL.
 *   rows, H, V        sizes; H % 8 == 0.
 *   W                 device bf16, layout w_layout, 16-byte aligned; with
 *                     LMH_W_HV, V % 8 == 0 (rows of V elements are 16-byte
 *                     multiples).  Both layouts run the same kernels at the
 *                     same speed: the [H x V] slices enter the tensor cores
 *                     vocabulary-major.
 *   sel_ids           device int32 [rows] or NULL; -1 = no selected token (NaN).
 *   row_k             device int32 [rows] or NULL (= k_max); values clamped to [0, k_max].
 *   k_max             0..LMH_K_MAX and <= V, or LMH_K_FULL.
 *   lse               device fp32 [rows], out.
 *   sel_logprob       device fp32 [rows], out (required when sel_ids != NULL).
 *   topk_ids          device int32 [rows x k_max], out (required when k_max > 0).
 *   topk_logprobs     device fp32 [rows x k_max], out (required when k_max > 0);
 *                     with k_max = LMH_K_FULL: device fp32 [rows x V], out,
 *                     16-byte aligned, entry [i][v] = fp32(z[i][v]) - lse[i]
 *                     (row_k and topk_ids are ignored).
 *   logits_out        device fp32 [rows x V] or NULL (16-byte aligned): when
 *                     given, the fp32 logits are also written (the
 *                     materializing arm and debugging); the reduction
 *                     results are unchanged.
 *   workspace         device, >= lmh_workspace_bytes(rows, H, V, k_max,
 *                     LMH_PATH_PROJECT) bytes, 256-byte aligned.
 * Errors: LMH_ERR_INVALID_ARG, LMH_ERR_UNSUPPORTED (k_max < -1 or > LMH_K_MAX,
 * LMH_W_HV with V % 8 != 0, H % 8 != 0, misaligned pointers),
 * LMH_ERR_WORKSPACE_TOO_SMALL, LMH_ERR_CUDA.  Device: LMH_DS_SEL_OUT_OF_RANGE,
 * LMH_DS_ROW_IDX_OUT_OF_RANGE, LMH_DS_TIMEOUT.
 */
lmh_status lmh_project_logprobs(const void* hidden, int64_t hidden_row_stride, int32_t num_tokens,
                                const int32_t* row_idx, int32_t rows, int32_t H, const void* W,
                                lmh_w_layout w_layout, int32_t V, const int32_t* sel_ids,
                                const int32_t* row_k, int32_t k_max, float* lse,
                                float* sel_logprob, int32_t* topk_ids, float* topk_logprobs,
                                float* logits_out, void* workspace, size_t workspace_bytes,
                                uint32_t* dev_status, cudaStream_t stream);

/*
 * lmh_project_logprobs_scaled -- lmh_project_logprobs with a head transform.
 *
 * Defined by: vllm-metal release v0.4.0.dev20260831, "Summary": some models
 * scale their head output (Cohere's logit_scale multiplies the logits,
 * Granite's logits_scaling divides them), and a head reproduced without the
 * scale gives silently wrong logits.  Here every logit is
 * fp32(logit_scale * (A . W)) before the reduction (and in logits_out):
 * pass logit_scale = s for Cohere, 1 / d for Granite's logits_scaling = d.
 *
 *   logit_scale       finite and > 0 (LMH_ERR_INVALID_ARG otherwise); 1 is
 *                     lmh_project_logprobs itself.
 * Every other argument, result and error as lmh_project_logprobs.
 */
lmh_status lmh_project_logprobs_scaled(const void* hidden, int64_t hidden_row_stride, int32_t num_tokens,
                                       const int32_t* row_idx, int32_t rows, int32_t H, const void* W,
                                       lmh_w_layout w_layout, int32_t V, const int32_t* sel_ids,
                                       const int32_t* row_k, int32_t k_max, float* lse, float* sel_logprob,
                                       int32_t* topk_ids, float* topk_logprobs, float* logits_out,
                                       void* workspace, size_t workspace_bytes, uint32_t* dev_status,
                                       float logit_scale, cudaStream_t stream);

/*
 * Device-side sampling (lmh_project_logprobs_sample), Gumbel-max over the
 * allowed tokens of each row; the grammar bitmask is given per selected row
 * (the compacted layout: vllm-metal release v0.4.0.dev20260831, "Testing",
 * bitmask application under the compacted layout).
 *
 * For row i, with z the (scaled) fp32 logits of lmh_project_logprobs:
 *   allowed(v)  = allowed_mask is NULL, or bit (v % 32) of
 *                 allowed_mask[i * mask_words + v / 32] is set;
 *   T           = temperature[i] (1 when temperature is NULL);
 *   score(v)    = z[i][v] / T + g(v) for T > 0, z[i][v] for T <= 0 (greedy);
 *   g(v)        = -log(-log u), u = ((w >> 9) + 0.5) * 2^-23, w = word (v & 3)
 *                 of Philox4x32-10 (Salmon et al., SC 2011) with counter
 *                 (v >> 2, lo(off), hi(off), 0x53414D50), key (lo(seed),
 *                 hi(seed)), off = offsets[i] (i when offsets is NULL);
 *   sampled_ids[i] = the allowed v with the largest score, ties to the
 *                 smaller id; -1 when no token is allowed (and
 *                 LMH_DS_NO_ALLOWED_TOKEN is set);
 *   sampled_logprob[i] = z[i][sampled] - lse[i] (the unmasked, untempered
 *                 distribution); NaN for -1.
 * The noise is computed with fast fp32 logarithms; a draw can differ from an
 * exact-arithmetic draw only when two scores are within the fp32 rounding of
 * the head and the noise.
 */
typedef struct lmh_sampling {
  const float* temperature;     /* device fp32 [rows] or NULL */
  const uint32_t* allowed_mask; /* device u32 [rows x mask_words] or NULL */
  int32_t mask_words;           /* >= ceil(V / 32) when allowed_mask is given */
  uint64_t seed;
  const int64_t* offsets;       /* device int64 [rows] or NULL */
  int32_t* sampled_ids;         /* device int32 [rows], out (required) */
  float* sampled_logprob;       /* device fp32 [rows], out, or NULL */
} lmh_sampling;

/*
 * lmh_project_logprobs_sample -- lmh_project_logprobs_scaled plus the
 * sampled token of every row (the same pass over W).  sampling may not be
 * NULL; its pointers are all device memory owned by the caller.
 * Errors: as lmh_project_logprobs_scaled, and LMH_ERR_INVALID_ARG for a
 * NULL sampling or sampled_ids, or mask_words < ceil(V / 32) with a mask.
 */
lmh_status lmh_project_logprobs_sample(const void* hidden, int64_t hidden_row_stride, int32_t num_tokens,
                                       const int32_t* row_idx, int32_t rows, int32_t H, const void* W,
                                       lmh_w_layout w_layout, int32_t V, const int32_t* sel_ids,
                                       const int32_t* row_k, int32_t k_max, float* lse, float* sel_logprob,
                                       int32_t* topk_ids, float* topk_logprobs, float* logits_out,
                                       void* workspace, size_t workspace_bytes, uint32_t* dev_status,
                                       float logit_scale, const lmh_sampling* sampling, cudaStream_t stream);

/*
 * lmh_probe_selective -- does this library's selective head reproduce the
 * model's own head output?
 *
 * Defined by: vllm-metal release v0.4.0.dev20260831, "Summary"
 * (supports_selective_logits probes once at load and demands bit-exact
 * equality with the model's own output; on a mismatch the engine keeps full
 * logits) and "Testing" (the probe rejects a model that scales its head
 * output when the scale is not reproduced).
 *
 *   hidden, hidden_row_stride, num_tokens, row_idx, rows, H, W, V:
 *                     as lmh_project_logprobs (row_idx = the rows to probe).
 *   logit_scale       the head transform to reproduce (1 = none; > 0).
 *   ref_logits        device f32 [rows x V] (row stride V): the model's own
 *                     logits of those rows.
 *   tolerance         an element mismatches when |ours - ref| > tolerance or
 *                     exactly one of them is NaN; 0 asks for bit-exact values
 *                     (except that +0 and -0 match).
 *   mismatches        device u32, out: the number of mismatching elements
 *                     (written, not accumulated).
 *   workspace         >= lmh_workspace_bytes(rows, H, V, 0, LMH_PATH_PROBE)
 *                     bytes, 256-byte aligned.
 * Errors: as lmh_project_logprobs, and LMH_ERR_INVALID_ARG for a null
 * ref_logits or mismatches, a negative or NaN tolerance, or a logit_scale
 * that is not finite and > 0.
 */
lmh_status lmh_probe_selective(const void* hidden, int64_t hidden_row_stride, int32_t num_tokens,
                               const int32_t* row_idx, int32_t rows, int32_t H, const void* W, int32_t V,
                               float logit_scale, const float* ref_logits, float tolerance,
                               uint32_t* mismatches, void* workspace, size_t workspace_bytes,
                               uint32_t* dev_status, cudaStream_t stream);

/*
 * lmh_logprobs_from_logits -- the same per-row reduction for logits that are
 * already in device memory (prompt scoring of logits chunks).
 *
 * Defined by MTPLX PR #532, "Summary" and "Change" (per 256-row chunk of
 * 248,320 logits: one fp32 logsumexp per row; top-k through the 64-logit
 * block-max prefilter that keeps the k blocks with the largest maxima and
 * selects the exact top-k among their entries; fp32(logit) - lse only at the
 * survivors and the scored token; exact ties by ascending id) and openinfer
 * issue #719 (reusable for decode rows and batches of prompt positions).
 *
 *   logits            device [rows x V] of dtype, row stride row_stride (>= V),
 *                     base aligned to sizeof(dtype).  When the base, the
 *                     row stride and the row length are multiples of 16
 *                     bytes the logits are streamed with bulk copies, else
 *                     with plain loads.
 *   sel_ids, row_k, k_max, lse, sel_logprob, topk_ids, topk_logprobs:
 *                     as for lmh_project_logprobs (logit = the given value
 *                     widened exactly to fp32).
 *   workspace         >= lmh_workspace_bytes(rows, 0, V, k_max,
 *                     LMH_PATH_FROM_LOGITS) bytes, 256-byte aligned.
 * Results for NaN or +inf logits are unspecified.  A row of only -inf gives
 * lse = -inf and NaN logprobs (ids 0..k-1).
 * Errors: as lmh_project_logprobs.
 */
lmh_status lmh_logprobs_from_logits(const void* logits, lmh_dtype dtype, int32_t rows, int32_t V,
                                    int64_t row_stride, const int32_t* sel_ids,
                                    const int32_t* row_k, int32_t k_max, float* lse,
                                    float* sel_logprob, int32_t* topk_ids, float* topk_logprobs,
                                    void* workspace, size_t workspace_bytes, uint32_t* dev_status,
                                    cudaStream_t stream);

/*
 * lmh_logprobs_from_logits_static -- lmh_logprobs_from_logits without a
 * caller workspace.
 *
 * The pages have no counterpart for this entry point.  It serves callers
 * that cannot allocate device memory when they need the reduction:
 * - an engine that gave all free HBM to its KV-cache pool at start-up;
 * - plain C code without access to the framework's allocator;
 * - a latency-critical loop where cudaMalloc/cudaFree would synchronise the
 *   device.
 * It runs the same kernels and returns the same results as
 * lmh_logprobs_from_logits. Instead of a caller workspace, it keeps its
 * partials in a fixed 8 MiB array in the library's own device memory, which
 * every GPU that loads the library holds until the process exits.  The call
 * allocates nothing.
 *
 * Arguments, results and errors are those of lmh_logprobs_from_logits,
 * minus workspace/workspace_bytes, with two differences:
 * - sizes whose partials need more than the 8 MiB are rejected with
 *   LMH_ERR_WORKSPACE_TOO_SMALL, and nothing is launched.  The partials take
 *   about rows * (4 * ceil(V / 64) + 8 * slots + 8) bytes, with slots =
 *   4 * ceil(ceil(V / 64) / 64) (whatever k_max and dtype): 256 rows x
 *   248320 need about 4.5 MB and fit; the largest batch is 479 rows at
 *   V = 248320 and 782 rows at V = 151936.
 * - the first call on each device does a one-time set-up with that device
 *   current: kernel attributes, and the array's device address via
 *   cudaGetSymbolAddress.  Make that first call before any stream capture.
 * Every call shares the one array, which keeps the previous call's contents.
 * Nothing in it needs to start at zero, but calls that overlap on the GPU
 * race on it: serialise them, on one stream or with events.
 */
lmh_status lmh_logprobs_from_logits_static(const void* logits, lmh_dtype dtype, int32_t rows,
                                           int32_t V, int64_t row_stride, const int32_t* sel_ids,
                                           const int32_t* row_k, int32_t k_max, float* lse,
                                           float* sel_logprob, int32_t* topk_ids,
                                           float* topk_logprobs, uint32_t* dev_status,
                                           cudaStream_t stream);

/*
 * Vocabulary-parallel head: several GPUs, each holding a share of the head's
 * vocabulary, together compute the same O(k+1) result as lmh_project_logprobs.
 *
 * Defined by openinfer issue #719, "Suggested direction" (a numerically sound
 * multi-stage reduction: per-part max and sum of exponentials combine exactly
 * into the log-sum-exp) and MTPLX PR #532, "Change" (the exact top-k of a row
 * lies among the union of the parts' own top-k lists; exact ties by ascending
 * token id).  Each rank calls lmh_project_partials on its share, the ranks
 * all-gather their records (any collective that concatenates equal-sized byte
 * buffers in rank order, e.g. an NCCL all-gather into the caller's device
 * memory), and every rank (or one) calls lmh_merge_records on the gathered
 * buffer.  The library itself makes no collective call.
 *
 * A record is lmh_record_bytes(k_max) bytes per row, 8-byte aligned:
 *   float m            the share's largest logit of the row (-inf: none)
 *   float s            sum over the share of exp(logit - m)
 *   float sel_logit    the selected token's logit, when it lies in the share
 *   uint32 flags       bit 0: sel_logit is set
 *   uint64 keys[k_max] the share's best k entries, best first: a key is
 *                      (order-preserving bits of the fp32 logit << 32) |
 *                      ~token_id, with global token ids; 0 = no entry.
 */
size_t lmh_record_bytes(int32_t k_max);

/*
 * lmh_project_partials -- one share of a vocabulary-parallel head.
 *
 * As lmh_project_logprobs (same hidden / row_idx / rows / H / sel_ids /
 * row_k / k_max meanings, the same fp32 accumulation and the same per-row
 * reduction), over the share's tokens [v_begin, v_begin + v_count) only:
 *   W_share    device bf16 [v_count x H], rows v_begin.. of lm_head.weight
 *              (LMH_W_VH; other layouts: LMH_ERR_UNSUPPORTED).
 *   V          the full vocabulary (sel_ids and returned ids are global).
 *   records    device [rows] records (lmh_record_bytes(k_max) each), out.
 *   workspace  >= lmh_workspace_bytes(rows, H, v_count, k_max, LMH_PATH_PROJECT).
 * k_max in [0, LMH_K_MAX] and <= v_count.  No logits are written.
 * Errors: as lmh_project_logprobs; LMH_ERR_INVALID_ARG also when the share is
 * empty or leaves [0, V).
 */
lmh_status lmh_project_partials(const void* hidden, int64_t hidden_row_stride, int32_t num_tokens,
                                const int32_t* row_idx, int32_t rows, int32_t H, const void* W_share,
                                lmh_w_layout w_layout, int32_t v_begin, int32_t v_count, int32_t V,
                                const int32_t* sel_ids, const int32_t* row_k, int32_t k_max, void* records,
                                void* workspace, size_t workspace_bytes, uint32_t* dev_status,
                                cudaStream_t stream);

/* Workspace of lmh_merge_records (bytes; 0 for invalid arguments). */
size_t lmh_merge_workspace_bytes(int32_t rows, int32_t num_parts, int32_t k_max);

/*
 * lmh_merge_records -- the rows' final results from the gathered records.
 *
 *   records     device [num_parts][rows] records, part p's rows contiguous
 *               (the layout of an all-gather of each rank's record buffer).
 *               The parts' shares must partition [0, V).
 *   V, sel_ids, row_k, k_max, lse, sel_logprob, topk_ids, topk_logprobs:
 *               as for lmh_project_logprobs (k_max must equal the k_max the
 *               records were made with).
 *   workspace   >= lmh_merge_workspace_bytes(rows, num_parts, k_max).
 * lse = M + log(sum_p s_p exp(m_p - M)), M = max_p m_p; the top-k is the best
 * k keys of the parts' lists; logprob = logit - lse.
 * Errors: as lmh_project_logprobs.
 */
lmh_status lmh_merge_records(const void* records, int32_t num_parts, int32_t rows, int32_t V,
                             const int32_t* sel_ids, const int32_t* row_k, int32_t k_max, float* lse,
                             float* sel_logprob, int32_t* topk_ids, float* topk_logprobs, void* workspace,
                             size_t workspace_bytes, uint32_t* dev_status, cudaStream_t stream);

/*
 * lmh_sample_from_logits -- one token per row from given logits, with
 * temperature, top-k, top-p and min-p, and one given random number per row.
 *
 * The filters a serving request asks for, applied to logits in device memory
 * (the full logits of lmh_project_logprobs, the output of lmh_project_q4, or a
 * model's own).  The pages name the selected token as an input and have no
 * counterpart for the filters; the definition is this one.  For row i:
 *   z_v      = the logit widened to fp32; -inf for a token that allowed_mask
 *              forbids (whatever value stands there) and for NaN.  zm = max z.
 *              Rows whose zm is +inf draw among their +inf tokens alone (these
 *              count as 0, every other token as -inf).
 *   T        = temperature[i] (1 when NULL).  T <= 0 or NaN is greedy: the
 *              token with the largest z, ties to the smallest id, logprob 0;
 *              the filters do not matter.
 *   c        = log2(e) * (1 / T) in fp32, two roundings, held in [2^-126, FLT_MAX].
 *   t_v      = fp32(fp32(z_v - zm) * c);  w_v = rint(2^32 * exp2f(t_v)), a whole
 *              number (exp2f is CUDA's).
 *   order    = z descending, exact ties by ascending id.
 *   top-k    keeps the first k tokens of the order (k <= 0 or k >= V: all); M is
 *            the sum of their w.
 *   top-p    keeps the shortest prefix of the order whose sum of w is at least
 *            max(1, ceil(p * M)), the product in fp64 (p >= 1 or NaN: all).
 *   min-p    keeps the tokens with t_v >= min(log2f(m), 0), that is of at least m
 *            times the best token's probability (m <= 0 or NaN: all).
 *   A token is kept when every filter keeps it; the best token always is.
 *   sampled_ids[i] = the smallest id whose sum of kept w over the ids up to and
 *            including it exceeds r = min(floor(u * K), K - 1): K the sum of all
 *            kept w, u = uniforms[i] held in [0, 1 - 2^-24] (NaN: 0), the product
 *            in fp64.
 *   sampled_logprob[i] = t * ln 2 - ln(K / 2^32): the token's log-probability in
 *            the distribution that it was drawn from.  (Its log-probability in
 *            the model's own distribution: lmh_logprobs_from_logits with sel_ids.)
 *   A row with no token above -inf gives id -1, a NaN logprob and
 *   LMH_DS_NO_ALLOWED_TOKEN.
 * The sums are of whole numbers, so a draw depends neither on the GPU's split of
 * a row nor on the batch that the row is in.
 *
 *   logits            device [rows x V] of dtype, row stride row_stride (>= V),
 *                     aligned to sizeof(dtype); V <= LMH_SAMPLE_V_MAX.
 *   filters           NULL: none, temperature 1.  Its pointers are device memory.
 *   uniforms          device fp32 [rows].
 *   sampled_ids       device int32 [rows], out.
 *   sampled_logprob   device fp32 [rows], out, or NULL.
 * No workspace is needed.  Errors: LMH_ERR_INVALID_ARG (null pointers, bad sizes,
 * mask_words < ceil(V / 32) with a mask), LMH_ERR_UNSUPPORTED (misaligned logits,
 * V > LMH_SAMPLE_V_MAX), LMH_ERR_CUDA.  Device: LMH_DS_NO_ALLOWED_TOKEN,
 * LMH_DS_TIMEOUT.
 */
#define LMH_SAMPLE_V_MAX 393216

typedef struct lmh_filters {
  const float* temperature;     /* device fp32 [rows] or NULL (1) */
  const int32_t* top_k;         /* device int32 [rows] or NULL (off) */
  const float* top_p;           /* device fp32 [rows] or NULL (off) */
  const float* min_p;           /* device fp32 [rows] or NULL (off) */
  const uint32_t* allowed_mask; /* device u32 [rows x mask_words] or NULL, as in lmh_sampling */
  int32_t mask_words;           /* >= ceil(V / 32) when allowed_mask is given */
} lmh_filters;

lmh_status lmh_sample_from_logits(const void* logits, lmh_dtype dtype, int32_t rows, int32_t V, int64_t row_stride,
                                  const lmh_filters* filters, const float* uniforms, int32_t* sampled_ids,
                                  float* sampled_logprob, uint32_t* dev_status, cudaStream_t stream);

/*
 * A [V x H] table (an LM head, or the embedding that is tied to it) held in 4
 * bits with one scale per group of `group` consecutive entries of a row:
 *   value[v][h] = scale[v][h / group] * (q[v][h] - zero[v][h / group])
 * with q in 0..15 and zero = 8 when `zeros` is NULL.  The pages leave quantised
 * heads to the model's own framework; this is the plain layout such checkpoints
 * are brought to: two entries a byte, the even h in the low half.
 */
typedef struct lmh_q4_table {
  const void* packed;       /* device u8 [V x H/2], 16-byte aligned */
  int64_t packed_row_bytes; /* >= H/2, a multiple of 16 */
  const void* scales;       /* device [V x H/group] of scale_dtype */
  lmh_dtype scale_dtype;    /* any lmh_dtype */
  int64_t scale_row_stride; /* elements, >= H/group */
  const uint8_t* zeros;     /* device u8 [V x H/group] (the low four bits count), or NULL */
  int64_t zero_row_stride;  /* elements, >= H/group */
  int32_t V, H;             /* H a multiple of group */
  int32_t group;            /* 32, 64 or 128 */
} lmh_q4_table;

/*
 * lmh_quantize_q4 -- round a bf16 table to 4 bits (once, when weights are loaded).
 *
 * Writes the arrays that `table` points to (its pointers are outputs here).  Per
 * group, in fp32 with the scale rounded once to scale_dtype (s below):
 *   zeros NULL:  s = max|w| / 7;              q = clamp(rint(w / s), -8, 7) + 8
 *   with zeros:  s = (max(w, 0) - min(w, 0)) / 15;  zero = clamp(rint(-min(w, 0) / s), 0, 15);
 *                q = clamp(rint(w / s) + zero, 0, 15)
 * A group whose s is 0 holds q = zero (8 without zeros).  Entries are finite.
 *
 *   W             device bf16 [V x H], row stride w_row_stride (>= H).
 * Errors: LMH_ERR_INVALID_ARG, LMH_ERR_UNSUPPORTED (a table outside the layout
 * above), LMH_ERR_CUDA.
 */
lmh_status lmh_quantize_q4(const void* W, int64_t w_row_stride, const lmh_q4_table* table, cudaStream_t stream);

/*
 * lmh_project_q4 -- the head projection through a 4-bit table.
 *
 *   out[i][v] = logit_scale * sum_h hidden[row_idx[i]][h] * value[v][h]
 * The products are of the 16-bit inputs and whole numbers (exact); a group's sum
 * is held in fp32, times its scale, and summed in fp32.  Rounded once, to
 * out_dtype.  Entries of a hidden row smaller than 2^-28 of the row's largest are
 * rounded to 2^-39 of it.  A row with an infinity or NaN gives infinities and NaN.
 * For batches of few rows (decode): the rows are taken in passes, each of which
 * reads the table once, of up to 32 rows where H is at most 2816 (with zero points
 * 2560), 16 up to 5120, 8 above.  Where a table is at hand in bf16 too,
 * lmh_project_logprobs takes less time from 33 rows on (2560 x 151936: 141 us for
 * 64 rows with the logits written, 186 here), less or about as much from 17 on with
 * zero points (32 rows: 137, 150 here) or longer rows (32 rows of 4096 x 128256: 168,
 * 162 here).
 *
 *   hidden            device [num_tokens x H] of hidden_dtype (LMH_BF16 or
 *                     LMH_F16), row stride hidden_row_stride (>= H), aligned to
 *                     its elements.
 *   row_idx           device int32 [rows] or NULL, as lmh_project_logprobs.
 *   logit_scale       finite and > 0 (a head transform, as
 *                     lmh_project_logprobs_scaled).
 *   out               device [rows x V] of out_dtype (LMH_F32 or hidden_dtype),
 *                     row stride out_row_stride (>= V).
 * The table is read only after the kernel enqueued before this one has ended, so
 * that may be the one that makes it.  No workspace is needed.
 * Errors: LMH_ERR_INVALID_ARG, LMH_ERR_UNSUPPORTED (dtypes, group, alignment, V above
 * 2^31 - 128, H above 2^31 - 16385), LMH_ERR_CUDA.  Device:
 * LMH_DS_ROW_IDX_OUT_OF_RANGE (the row reads zeros), LMH_DS_TIMEOUT.
 */
lmh_status lmh_project_q4(const void* hidden, lmh_dtype hidden_dtype, int64_t hidden_row_stride, int32_t num_tokens,
                          const int32_t* row_idx, int32_t rows, const lmh_q4_table* table, float logit_scale,
                          void* out, lmh_dtype out_dtype, int64_t out_row_stride, uint32_t* dev_status,
                          cudaStream_t stream);

/*
 * lmh_lookup_q4 -- the embedding rows of token ids, from a tied 4-bit table.
 *
 *   out[i][h] = (q - zero) * table scale * scale, in fp32 (the first product is
 *               exact for 16-bit scales), rounded once to out_dtype.
 *   ids               device int32 [n].  -1 (no token) gives a row of zeros; any
 *                     other id outside [0, V) does too and sets
 *                     LMH_DS_SEL_OUT_OF_RANGE.
 *   scale             finite (1, or a model's embedding multiplier).
 *   out               device [n x H] of out_dtype (any), row stride
 *                     out_row_stride (>= H).
 * Errors: as lmh_project_q4.
 */
lmh_status lmh_lookup_q4(const int32_t* ids, int32_t n, const lmh_q4_table* table, float scale, void* out,
                         lmh_dtype out_dtype, int64_t out_row_stride, uint32_t* dev_status, cudaStream_t stream);

/*
 * Low-rank adapters of several requests, in one array each: adapter l adds
 * scale[l] * up[l] . (down[l] . x) to a projection of x.
 */
#define LMH_ADAPTERS_MAX 4096
#define LMH_ADAPTER_RANK_MAX 128

typedef struct lmh_adapters {
  const void* down;            /* device [count x rank x H] of dtype, 16-byte aligned */
  int64_t down_adapter_stride; /* elements, a multiple of 8 */
  int64_t down_row_stride;     /* elements, >= H, a multiple of 8 */
  const void* up;              /* device [count x N x rank] of dtype, 16-byte aligned */
  int64_t up_adapter_stride;   /* elements, a multiple of 8 */
  int64_t up_row_stride;       /* elements, >= rank, a multiple of 8 */
  lmh_dtype dtype;             /* LMH_BF16 or LMH_F16 */
  const float* scales;         /* device fp32 [count], or NULL (1) */
  const int32_t* ranks;        /* device int32 [count], or NULL (rank): the ranks in use, held in
                                  [0, rank]; what stands behind them is not used */
  int32_t count;               /* 1..LMH_ADAPTERS_MAX */
  int32_t rank;                /* a multiple of 8, to LMH_ADAPTER_RANK_MAX */
  int32_t H, N;                /* H a multiple of 8 */
} lmh_adapters;

/* Workspace of lmh_add_adapters (bytes; 0 for sizes it rejects), 256-byte aligned.  The size
 * depends on the device's SM count. */
size_t lmh_adapters_workspace_bytes(int32_t rows, const lmh_adapters* table);

/*
 * lmh_add_adapters -- each row's adapter beside a shared projection.
 *
 *   out[i][n] = y[i][n] + scales[l] * sum_r up[l][n][r] * d[i][r],
 *   d[i][r]   = sum_h down[l][r][h] * x[row_idx[i]][h],      l = adapter_idx[i]
 *
 * y is the shared projection's result for the rows (a layer's, or the logits of
 * lmh_project_q4 or lmh_project_logprobs), so out is the projection with the
 * requests' adapters.  Sums are held in fp32.  d enters the second product as the sum of
 * two numbers of dtype: within 2^-16 of its value for LMH_BF16 and 2^-22 for LMH_F16 (f16
 * parts of a row's d below 2^-28 of its largest: within 2^-38 of the largest).  Rounded
 * once, to out_dtype.  A row of x with an infinity or NaN gives infinities and NaN, and so
 * does a row of up in the output that it makes.  The rows may come in any order, each with
 * any adapter; an adapter's weights are read about once per 64 rows that use it, and not at
 * all if none does.
 *
 *   x                 device [num_tokens x H] of the table's dtype, row stride
 *                     x_row_stride (>= H), aligned to its elements.
 *   row_idx           device int32 [rows] or NULL, as lmh_project_logprobs.
 *   adapter_idx       device int32 [rows]; -1: no adapter (out is y).  Any other index
 *                     outside [0, count) counts as -1 and sets
 *                     LMH_DS_ADAPTER_OUT_OF_RANGE.
 *   y                 device [rows x N] of out_dtype, row stride y_row_stride (>= N).
 *   out               device [rows x N] of out_dtype (LMH_F32 or the table's dtype), row
 *                     stride out_row_stride (>= N).  It may be y itself with the same
 *                     stride (rows without an adapter are not touched then); it
 *                     overlaps y in no other way, nor x.
 *   workspace         >= lmh_adapters_workspace_bytes(rows, table) bytes, 256-byte
 *                     aligned.
 * Errors: LMH_ERR_INVALID_ARG, LMH_ERR_UNSUPPORTED (dtypes, rank, count, alignment, sizes
 * near 2^31), LMH_ERR_WORKSPACE_TOO_SMALL, LMH_ERR_CUDA.  Device: LMH_DS_ADAPTER_OUT_OF_RANGE,
 * LMH_DS_ROW_IDX_OUT_OF_RANGE (the row reads zeros).
 */
lmh_status lmh_add_adapters(const void* x, int64_t x_row_stride, int32_t num_tokens, const int32_t* row_idx,
                            int32_t rows, const int32_t* adapter_idx, const lmh_adapters* table, const void* y,
                            int64_t y_row_stride, void* out, lmh_dtype out_dtype, int64_t out_row_stride,
                            void* workspace, size_t workspace_bytes, uint32_t* dev_status, cudaStream_t stream);

/*
 * Beam search: rows [g * beams, (g + 1) * beams) are group g's beams, each with a score
 * (the sum of its tokens' log-probabilities) in `scores`.
 *
 *   parents   the row that a continuation comes from (g * beams + beam), and
 *   tokens    the token that it adds; both -1, with a score of -inf, in places that no
 *             continuation is left for.
 *   finished  a beam whose flag is set has ended: it has one continuation, itself, with
 *             pad_id as its token and its score as it is.  Its logits are not read.
 *   k         continuations per group, best first.  Twice the beams leave enough for a
 *             step's ended ones to be taken out by the caller.
 *   keep_slots  (k == beams only) the continuations do not come best first: a parent's
 *             best one stands in the parent's own place, the others fill the places left
 *             over, best first from the lowest.  parents[parents[r]] == parents[r] then, so
 *             lmh_reorder_rows moves the fewest rows.
 */
typedef struct lmh_beams {
  int32_t groups, beams;    /* beams 1..LMH_BEAMS_MAX */
  int32_t k;                /* 1..LMH_K_MAX */
  int32_t keep_slots;       /* 0 or 1 */
  const float* scores;      /* device fp32 [groups x beams]; a beam whose score is not finite
                               has no continuation */
  const uint8_t* finished;  /* device u8 [groups x beams], or NULL */
  int32_t pad_id;
  float* out_scores;        /* device fp32 [groups x k], out; may not be `scores` */
  int32_t* out_parents;     /* device int32 [groups x k], out */
  int32_t* out_tokens;      /* device int32 [groups x k], out */
} lmh_beams;

/* Workspace of lmh_beam_select (bytes; 0 for sizes it rejects), 256-byte aligned. */
size_t lmh_beam_workspace_bytes(int32_t groups, int32_t beams, int32_t V);

/*
 * lmh_beam_select -- each group's k best continuations over its beams and the vocabulary.
 *
 *   score(b, v) = scores[b] + z[b][v] - lse[b],   lse[b] = log sum_v exp(z[b][v])
 *
 * The log-sum-exp is over all tokens; allowed_mask takes tokens out of the choice only (as
 * in lmh_project_logprobs_sample, a token's log-probability is the model's own).  Scores are
 * compared in 64 bits, as (scores[b] - log sum_v exp(z[b][v] - M)) + (z[b][v] - M) with M
 * the row's largest logit; equal ones are ordered by beam, then token.  A NaN logit counts as -inf, and -inf is no
 * continuation; a row with +inf logits has these alone, as equals.  A score that fp32
 * cannot hold is no continuation.
 *
 *   logits            device [groups * beams x V] of dtype, row stride row_stride (>= V),
 *                     aligned to sizeof(dtype); beams * V to 2^31 - 2^16 - 1.
 *   allowed_mask      device u32 [groups * beams x mask_words] or NULL, as in lmh_sampling.
 *   workspace         >= lmh_beam_workspace_bytes(groups, beams, V) bytes, 256-byte aligned.
 * Errors: LMH_ERR_INVALID_ARG, LMH_ERR_UNSUPPORTED (beams, k, misaligned logits or mask, beams * V),
 * LMH_ERR_WORKSPACE_TOO_SMALL, LMH_ERR_CUDA.  Device: LMH_DS_NO_ALLOWED_TOKEN (a group
 * without a continuation), LMH_DS_TIMEOUT.
 */
lmh_status lmh_beam_select(const lmh_beams* beams, const void* logits, lmh_dtype dtype, int32_t V,
                           int64_t row_stride, const uint32_t* allowed_mask, int32_t mask_words, void* workspace,
                           size_t workspace_bytes, uint32_t* dev_status, cudaStream_t stream);

/*
 * lmh_beam_select_lists -- the same from each beam's own best tokens (the top-k lists of
 * lmh_project_logprobs, whose logits never reach memory): lists of at least k entries give
 * what lmh_beam_select gives, up to the rounding of the lists' logprobs.
 *
 *   topk_ids, topk_logprobs  device [groups * beams x n], contiguous.  Entries with an id
 *                     below 0 or a logprob that is not finite are none.  Equal scores are
 *                     ordered by beam, then place in the list.
 * beams * n to 2^31 - 2^16 - 1.  No workspace is needed.  Errors: as lmh_beam_select.
 */
lmh_status lmh_beam_select_lists(const lmh_beams* beams, const int32_t* topk_ids, const float* topk_logprobs,
                                 int32_t n, uint32_t* dev_status, cudaStream_t stream);

/*
 * A state that has one row per row of the batch: token histories, block tables, caches.
 * Row r's bytes are n0 * n1 chunks of chunk_bytes each, chunk (i, j) at
 *   src + r * src_row_bytes + i * src_outer_bytes[0] + j * src_outer_bytes[1]
 * and in the same way at dst.  dst == src (with the same strides): in place.  With
 * position_bytes > 0, a chunk is a run of positions of that size.
 */
typedef struct lmh_row_state {
  const void* src;
  void* dst;
  int64_t src_row_bytes, dst_row_bytes;
  int64_t src_outer_bytes[2], dst_outer_bytes[2];
  int32_t n0, n1;
  int64_t chunk_bytes;
  int64_t position_bytes; /* 0: chunks are moved whole */
} lmh_row_state;

/*
 * lmh_reorder_rows -- every state's row r becomes what row parents[r] held.
 *
 * Rows [g * beams, (g + 1) * beams) are a group, and a row's parent is one of its group
 * (the out_parents of a selection with k == beams).  In place, rows that are their own
 * parents are not touched, and any other parents are right too (rows that swap, a row that
 * is taken and replaced).
 *
 *   states            host array [num_states].  Their strides are not negative; rows and
 *                     chunks of a dst do not overlap, nor do the states each other (in
 *                     place, dst and src are the same memory), parents or lengths.
 *   parents           device int32 [groups * beams]; -1 (no continuation): the row itself.
 *                     Any other row outside the group counts as -1 and sets
 *                     LMH_DS_ROW_IDX_OUT_OF_RANGE.
 *   lengths           device int32 [groups * beams] or NULL: positions in use of each row
 *                     as it is in src.  Of states with positions, a row's first
 *                     lengths[parent] are moved, and what stands behind them in dst is left
 *                     as it was.  NULL: all are moved.
 * No workspace is needed.  Errors: LMH_ERR_INVALID_ARG (null pointers, sizes, negative
 * strides, in place with other strides), LMH_ERR_UNSUPPORTED (beams, positions of
 * 2^31 bytes or more, states of some 2^39 bytes a row), LMH_ERR_CUDA.  Device:
 * LMH_DS_ROW_IDX_OUT_OF_RANGE, LMH_DS_TIMEOUT (rows may be partly moved then, in place too).
 */
lmh_status lmh_reorder_rows(const lmh_row_state* states, int32_t num_states, int32_t groups, int32_t beams,
                            const int32_t* parents, const int32_t* lengths, uint32_t* dev_status,
                            cudaStream_t stream);

/* Human-readable name of a status code (static storage). */
const char* lmh_status_string(lmh_status status);

/* LMH_VERSION of the loaded library. */
int32_t lmh_version(void);

/*
 * Kernel tracing (device time per kernel, measured with CUDA events recorded
 * on the launching stream around every launch while enabled).  Not for use
 * while a stream is being captured into a CUDA graph.
 *
 * lmh_trace_enable(1) starts recording, lmh_trace_enable(0) stops.
 * lmh_trace_read waits for the recorded events, then reports the launches
 * and total milliseconds of the named kernel ("select_rows", "gather_rows",
 * "head_logprobs", "merge_partials", "logits_reduce" (the streaming pass of
 * lmh_logprobs_from_logits), "logits_select" (its per-row selection),
 * "full_logprobs" (the pass that writes the k_max = LMH_K_FULL output),
 * "sample_logits", "project_q4", "lookup_q4", "quantize_q4", "adapter_plan",
 * "adapter_down", "adapter_up", "beam_stream", "beam_choose", "reorder_rows") since the
 * last reset.
 * lmh_trace_reset clears the totals.
 */
lmh_status lmh_trace_enable(int32_t enable);
lmh_status lmh_trace_read(const char* kernel, int64_t* launches, double* total_ms);
void lmh_trace_reset(void);

/*
 * lmh_debug_set_wait_limit -- test hook for the timeout path; not for
 * production use.  The pages have no counterpart.
 *
 * Inside a kernel, every wait on another role of the same CTA (a shared-memory
 * stage, an accumulator, a chunk) gives up after this limit: the kernel sets
 * LMH_DS_TIMEOUT in *dev_status, stops its loops, lets its copies and tensor-
 * core work in flight finish (those drain waits keep a fixed 2 s limit), frees
 * its tensor memory and returns, so the context stays usable.  The default is
 * 2 s, far above any legitimate wait; a test sets a limit shorter than the
 * latency of one load so that the first wait runs out, then calls with 0 to
 * restore the default.  The value applies to kernels launched after the call,
 * from any thread.  Always LMH_OK.
 */
lmh_status lmh_debug_set_wait_limit(uint64_t limit_ns);

#ifdef __cplusplus
}
#endif

#endif /* LMH_H */
