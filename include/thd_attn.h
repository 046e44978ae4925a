/*
 * thd_attn.h -- C ABI of libthdattn.so: causal softmax attention over packed
 * variable-length THD tensors, decomposed the way P2P (ring) context
 * parallelism decomposes it, with every CP rank emulated on one GPU.
 *
 * Sources (web pages), cited by page and section:
 *   [P1] TransformerEngine issue #2208, "thd format is not supported with
 *        hierarchical CP implementation yet" (traceback through
 *        AttnFuncWithCPAndKVP2P; maintainer reply on P2P vs A2A).
 *   [P2] TransformerEngine issue #3487, "THD P2P context-parallel regression
 *        when padded cu_seqlens are value-equal but not object-identical"
 *        ("Describe the bug", "Steps/Code to reproduce bug",
 *        "Expected behavior").
 *   [P3] "Hybrid / Hierarchical Context Parallel Skill" ("Contraintes
 *        requises": seq_length % (2 * context_parallel_size) == 0;
 *        "Pitfalls" item 5).
 *
 * Conventions for every entry point
 *   - THD layout: tensor [T, H, D] is row-major and contiguous, token-major:
 *     element (t, h, d) at ((t * H) + h) * D + d.  bf16 tensors are passed
 *     as `void*` to 2-byte IEEE bfloat16 storage.
 *   - cu_seqlens (int32, B+1 entries, cu[0] == 0) are exclusive prefix sums of
 *     the VALID lengths L_b.  cu_seqlens_padded (int32, B+1, may be NULL) are
 *     the buffer offsets: sequence b's valid tokens sit at rows
 *     [pad[b], pad[b] + L_b) and rows [pad[b] + L_b, pad[b+1]) are pad.
 *     NULL means no padding (pad = cu).
 *   - Each padded length P_b must be divisible by 2 * cp_size [P3
 *     "Contraintes requises"]; chunk length cb = P_b / (2 cp_size); emulated
 *     rank r owns chunks r and 2 cp_size - 1 - r.
 *   - All pointers are DEVICE pointers owned by the caller; the library never
 *     allocates device memory and never synchronises the host.  All work is
 *     enqueued on `stream` (a cudaStream_t; NULL = legacy default stream).
 *   - Return value: a host-side status (THD_OK or THD_ERR_*) for argument
 *     errors found without reading device memory, and launch failures.
 *   - Metadata errors can only be seen on the device (cu_seqlens live in
 *     device memory).  The first kernel of each call writes `*dev_status`
 *     (int32, device): 0 when the metadata is valid, else a THD_DEV_*
 *     code; every later kernel of the call reads it and returns without
 *     touching the outputs when it is nonzero.  Read it after the stream has
 *     synchronised.  Kernels that give up a bounded wait write
 *     THD_ERR_TIMEOUT there.
 *   - Workspace: caller-provided device memory of at least
 *     thd_workspace_size(...) bytes, 256-byte aligned; its contents need not be
 *     initialised and are not meaningful after the call.
 *   - Nothing is captured across calls except read-only state (driver entry
 *     points, per-device attributes); calls are safe to capture in a CUDA
 *     graph as long as the pointers stay valid.
 */
#ifndef THD_ATTN_H
#define THD_ATTN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st* thd_stream_t; /* identical to cudaStream_t */

#if defined(__GNUC__)
#define THD_API __attribute__((visibility("default")))
#else
#define THD_API
#endif

/* host-side status codes */
#define THD_OK 0
#define THD_ERR_INVALID_ARG 1 /* null pointer, bad size, misaligned pointer */
#define THD_ERR_UNSUPPORTED 2 /* head_dim not 64/128, unsupported mode */
#define THD_ERR_CUDA 3        /* a CUDA call or launch failed */
#define THD_ERR_TIMEOUT 4     /* (device) a bounded wait gave up */
#define THD_ERR_WORKSPACE 5   /* workspace too small or misaligned */

/* device-side status codes written to *dev_status */
#define THD_DEV_ERR_NONZERO_START 101  /* cu_seqlens[0] or padded[0] != 0 */
#define THD_DEV_ERR_NOT_MONOTONE 102   /* negative length */
#define THD_DEV_ERR_VALID_GT_PAD 103   /* L_b > P_b */
#define THD_DEV_ERR_NOT_DIVISIBLE 104  /* P_b % (2 cp_size) != 0 */
#define THD_DEV_ERR_EXCEEDS_BUF 105    /* pad[B] larger than the buffer rows */
#define THD_DEV_ERR_CAUSAL_LENGTHS 106 /* top-left causal with q and kv lengths differing */
#define THD_DEV_ERR_CAPACITY 107       /* internal schedule capacity exceeded */
#define THD_DEV_ERR_DOC_ORDER 108      /* document numbers decrease inside a sequence */
#define THD_DEV_ERR_PAGE 109           /* the block table names a page outside the cache */
#define THD_DEV_ERR_KV_LEN 110         /* a cached length below 0 or the new rows, or past the block table */

/* Kernel identifiers for the profiling hook. */
#define THD_KERNEL_PLAN 1
#define THD_KERNEL_FWD 2
#define THD_KERNEL_BWD_PREP 3
#define THD_KERNEL_BWD 4
#define THD_KERNEL_BWD_DQ 5
#define THD_KERNEL_LSE_MERGE 6
#define THD_KERNEL_TAIL_ZERO 7
#define THD_KERNEL_PARTITION 8
#define THD_KERNEL_A2A 9
#define THD_KERNEL_ROPE 10
#define THD_KERNEL_DROPOUT 11
#define THD_KERNEL_DOCS 12
#define THD_KERNEL_BWD_JOIN 13
#define THD_KERNEL_DECODE 14
#define THD_KERNEL_DECODE_JOIN 15
#define THD_KERNEL_CACHE_APPEND 16
#define THD_KERNEL_CACHE_EVICT 17
#define THD_KERNEL_DECODE_WEIGHTS 18

/* mask modes (the `causal` argument of the attention entry points) */
#define THD_CAUSAL_NONE 0
#define THD_CAUSAL_TOP_LEFT 1
#define THD_CAUSAL_BOTTOM_RIGHT 2

/* element types of the row-wise operators and of a key-value cache */
#define THD_DTYPE_BF16 0
#define THD_DTYPE_FP32 1
#define THD_DTYPE_E4M3 2 /* a cache's keys and values, with an exponent for each row */

/* thd_cp_a2a directions */
#define THD_A2A_TO_GROUPS 0 /* shards -> per-member head groups (the all-to-all in front of attention) */
#define THD_A2A_TO_SHARDS 1 /* per-member head groups -> shards (the all-to-all behind it) */

/* Human-readable text for any status above (host or device). Never NULL. */
THD_API const char* thd_status_string(int status);

/* Library ABI version (major * 100 + minor). */
THD_API int thd_version(void);

/*
 * Bytes of workspace thd_attn_fwd (for_bwd = 0) or thd_attn_bwd (for_bwd = 1)
 * needs for these sizes.  T_q / T_kv are the buffer rows of q and k/v.
 * Returns 0 for invalid sizes.
 */
THD_API size_t thd_workspace_size(int B, int64_t T_q, int64_t T_kv, int Hq, int Hkv, int D, int cp_size, int for_bwd);

/*
 * thd_cp_partition -- per-rank cu_seqlens for THD + P2P context parallelism,
 * for every emulated rank in ONE launch.
 *
 * [P2 "Describe the bug"] names the helper get_cu_seqlens_on_cp_rank, which
 * the padded path calls once per ring step; [P3 "Contraintes requises"]
 * fixes the 2*cp_size split.  For rank r and sequence b, with
 * cb = P_b / (2 cp_size):
 *     v1 = clamp(L_b - r cb, 0, cb)                (valid rows of chunk r)
 *     v2 = clamp(L_b - (2 cp_size - 1 - r) cb, 0, cb)
 *     cu_rank[r][b+1]        = cu_rank[r][b] + v1 + v2
 *     cu_rank_padded[r][b]   = pad[b] / cp_size
 *     cu_rank_half[r][0][b+1] = cu_rank_half[r][0][b] + v1
 *     cu_rank_half[r][1][b+1] = cu_rank_half[r][1][b] + v2
 *     token_map[r * (T / cp_size) + p] = global padded row of rank-local row p
 *       (rank-local rows of sequence b: chunk r then chunk 2cp-1-r), T = pad[B].
 * Arguments:
 *   cu_seqlens [B+1], cu_seqlens_padded [B+1] or NULL: device int32.
 *   pad_between_seqs: -1 decide from VALUES (padded iff some entry differs,
 *     never by pointer identity [P2 "Expected behavior"]), 0 ignore the
 *     padded array, 1 use it.
 *   cu_rank, cu_rank_padded: [cp_size][B+1] int32; cu_rank_half
 *     [cp_size][2][B+1] int32; token_map [token_map_capacity] int32.  Any
 *     output may be NULL (not written).  token_map needs capacity >= pad[B]
 *     (else THD_DEV_ERR_EXCEEDS_BUF).
 *   dev_status: device int32, always written.
 * Bit-exact (integer).
 */
THD_API int thd_cp_partition(const int32_t* cu_seqlens, const int32_t* cu_seqlens_padded, int B, int cp_size,
                     int pad_between_seqs, int32_t* cu_rank, int32_t* cu_rank_padded, int32_t* cu_rank_half,
                     int32_t* token_map, int64_t token_map_capacity, int32_t* dev_status, thd_stream_t stream);

/*
 * thd_attn_fwd -- O = softmax(scale q k^T + mask) v per sequence and head,
 * and lse = logsumexp of the masked scaled scores (natural log).
 *
 * Decomposition [P1 traceback: AttnFuncWithCPAndKVP2P; P3 "Contraintes
 * requises"]: work is split per emulated rank r (local query rows = chunk r
 * then chunk 2cp-1-r of each sequence) and ring step i, where rank r
 * holds the KV of rank s = (r - i) mod cp_size; per-step partials are merged
 * on chip by online-softmax (log-sum-exp) correction.  The merged result
 * equals plain attention.  Query and key sequences are chunked separately
 * (P_q / 2cp and P_kv / 2cp rows).
 *
 * Masks (`causal`; the pages train causal self-attention, the top-left mask
 * with equal lengths; the other two are the plainest completions):
 *   THD_CAUSAL_NONE (0): every valid key.
 *   THD_CAUSAL_TOP_LEFT (1): query i sees key j iff j <= i; needs equal q
 *     and kv valid and padded lengths per sequence (else the device status
 *     THD_DEV_ERR_CAUSAL_LENGTHS).
 *   THD_CAUSAL_BOTTOM_RIGHT (2): j <= i + L_kv - L_q, the last query aligned
 *     with the last key (a query block at the end of its keys); equal to
 *     top-left when the lengths agree.  With L_q > L_kv the first L_q - L_kv
 *     queries see no key: o = 0, lse = -inf (and zero gradients).
 *
 *   q   [T_q, Hq, D] bf16;  k, v [T_kv, Hkv, D] bf16 (Hq % Hkv == 0; query
 *       head h reads kv head h / (Hq/Hkv)).  16-byte aligned.
 *   o   [T_q, Hq, D] bf16 output; lse [Hq, T_q] fp32 output.  Rows that hold
 *       no valid token (pad rows and rows [pad_q[B], T_q)) get o = 0 and
 *       lse = -inf.
 *   D: 64 or 128.  causal: 0, 1 or 2 as above.  softmax_scale > 0.
 *   cp_size >= 1: the emulated CP degree.  pad_between_seqs as in
 *   thd_cp_partition (decided per side from values when -1).
 *   Pad rows inside tiles are read: they must hold finite values.
 */
THD_API int thd_attn_fwd(const void* q, const void* k, const void* v, void* o, float* lse, const int32_t* cu_seqlens_q,
                 const int32_t* cu_seqlens_kv, const int32_t* cu_seqlens_q_padded,
                 const int32_t* cu_seqlens_kv_padded, int B, int64_t T_q, int64_t T_kv, int Hq, int Hkv, int D,
                 int causal, float softmax_scale, int cp_size, int pad_between_seqs, void* workspace,
                 size_t workspace_bytes, int32_t* dev_status, thd_stream_t stream);

/*
 * thd_attn_fwd_step -- the partial of ONE ring step, materialised: for every
 * emulated rank r, the attention of its local queries against the KV it
 * holds at step `step` (rank s = (r - step) mod cp_size), written in fp32 at
 * the queries' global rows:
 *   o_part [T_q, Hq, D] fp32, lse_part [Hq, T_q] fp32 (natural log).
 * Rows that get no contribution at this step get o = 0, lse = -inf.  Merging
 * the cp_size step partials with thd_lse_merge gives thd_attn_fwd's result
 * (the ring with communication replaced by reads of rank s's rows).
 * Other arguments as thd_attn_fwd.
 */
THD_API int thd_attn_fwd_step(const void* q, const void* k, const void* v, float* o_part, float* lse_part,
                      const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_kv, const int32_t* cu_seqlens_q_padded,
                      const int32_t* cu_seqlens_kv_padded, int B, int64_t T_q, int64_t T_kv, int Hq, int Hkv,
                      int D, int causal, float softmax_scale, int cp_size, int pad_between_seqs, int step,
                      void* workspace, size_t workspace_bytes, int32_t* dev_status, thd_stream_t stream);

/*
 * thd_attn_fwd_step_bf16 -- thd_attn_fwd_step with the step's partial output
 * in bf16, the precision the ring keeps its per-step outputs in when they are
 * materialised [P1 traceback: AttnFuncWithCPAndKVP2P.forward, per-step
 * outputs corrected into the running output]:
 *   o_part [T_q, Hq, D] bf16 (16-byte aligned), lse_part [Hq, T_q] fp32.
 * Same rows, masks and -inf/0 conventions as thd_attn_fwd_step; merge the
 * steps with thd_lse_merge_bf16 into an fp32 accumulator.
 */
THD_API int thd_attn_fwd_step_bf16(const void* q, const void* k, const void* v, void* o_part, float* lse_part,
                                   const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_kv,
                                   const int32_t* cu_seqlens_q_padded, const int32_t* cu_seqlens_kv_padded, int B,
                                   int64_t T_q, int64_t T_kv, int Hq, int Hkv, int D, int causal,
                                   float softmax_scale, int cp_size, int pad_between_seqs, int step,
                                   void* workspace, size_t workspace_bytes, int32_t* dev_status,
                                   thd_stream_t stream);

/*
 * thd_attn_fwd_noalloc -- thd_attn_fwd for callers that cannot allocate device
 * memory where they call the library.  The pages have no counterpart to
 * this entry point; it exists for deployment.  Examples of such callers: a
 * plug-in that only receives input and output pointers from a host framework
 * whose own pool allocator owns the device memory; a serving loop with a
 * fixed, pre-planned memory budget; code that must not call cudaMalloc,
 * which can synchronise the device and is not allowed inside stream capture.
 *
 * Same arguments and results as thd_attn_fwd, minus the workspace: the
 * scratch lives in a static device array of THD_NOALLOC_SCRATCH_BYTES (1 MiB)
 * inside the library, which every GPU that loads the library keeps until the
 * process exits.  The entry point calls no cudaMalloc/cudaFree and no
 * allocating library routine.
 *   - Limit: returns THD_ERR_WORKSPACE, launching nothing, when
 *     thd_workspace_size(B, T_q, T_kv, Hq, Hkv, D, cp_size, 0) exceeds
 *     THD_NOALLOC_SCRATCH_BYTES (about T_q / 128 + cp_size * B < 65000 schedule
 *     entries, e.g. up to ~8M tokens for a few sequences).
 *   - Set-up: the first call on each device looks up the array's device
 *     address (cudaGetSymbolAddress) with that device current; make that first
 *     call before any stream capture.
 *   - Sharing: every call on a device uses the same array, which keeps the
 *     last call's contents (nothing in it needs clearing; each call rewrites
 *     what it reads).  Calls whose kernels overlap on the GPU (different
 *     streams, or host threads without ordering) race on it: serialise them.
 */
#define THD_NOALLOC_SCRATCH_BYTES (1 << 20)
THD_API int thd_attn_fwd_noalloc(const void* q, const void* k, const void* v, void* o, float* lse,
                                 const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_kv,
                                 const int32_t* cu_seqlens_q_padded, const int32_t* cu_seqlens_kv_padded, int B,
                                 int64_t T_q, int64_t T_kv, int Hq, int Hkv, int D, int causal, float softmax_scale,
                                 int cp_size, int pad_between_seqs, int32_t* dev_status, thd_stream_t stream);

/*
 * thd_attn_bwd -- gradients of thd_attn_fwd w.r.t. q, k, v.
 * [P2 "Steps/Code to reproduce bug"] runs forward/backward on this layout.
 *   q, k, v, o (forward output), dout: bf16 as in thd_attn_fwd; lse [Hq, T_q]
 *   fp32 from thd_attn_fwd.
 *   dq [dq_rows, Hq, D], dk/dv [dkv_rows, Hkv, D] bf16 outputs, with
 *   dq_rows >= T_q and dkv_rows >= T_kv.  Every row without a valid token,
 *   including the slack rows [pad[B], rows), is written with 0 (the THD
 *   gradient tail-zero of [P2 "Describe the bug"], done on the device with
 *   no extra launch and no work when there is no slack).
 * dK/dV of each kv head sum over its query-head group.  Two passes: a
 * key-stationary kernel for dK/dV and a query-stationary kernel for dQ (it
 * recomputes S and dP for its query tile); every output element is summed in
 * a fixed order, so dQ, dK and dV are bit-reproducible across runs.
 * Launches: the planner (both schedules in one launch), the Delta
 * preprocess, dQ, dK/dV.
 */
THD_API int thd_attn_bwd(const void* q, const void* k, const void* v, const void* o, const float* lse, const void* dout,
                 void* dq, void* dk, void* dv, int64_t dq_rows, int64_t dkv_rows, const int32_t* cu_seqlens_q,
                 const int32_t* cu_seqlens_kv, const int32_t* cu_seqlens_q_padded,
                 const int32_t* cu_seqlens_kv_padded, int B, int64_t T_q, int64_t T_kv, int Hq, int Hkv, int D,
                 int causal, float softmax_scale, int cp_size, int pad_between_seqs, void* workspace,
                 size_t workspace_bytes, int32_t* dev_status, thd_stream_t stream);

/*
 * thd_attn_score_fwd -- thd_attn_fwd with a score function and more masks:
 *     x_ij = softmax_scale q_i . k_j
 *     y_ij = softcap tanh(x_ij / softcap)            (softcap > 0; else x_ij)
 *     y_ij -= dist_slopes[h] |i + koff - j|          (dist_slopes given)
 *     O = softmax(y + mask) v,  lse = logsumexp(y + mask),
 * with koff = L_kv - L_q under THD_CAUSAL_BOTTOM_RIGHT and 0 otherwise (the
 * distance is between positions of the sequence).  Masks, all of which must
 * let a pair through:
 *   causal: as in thd_attn_fwd, except that with prefix_len the first
 *     prefix_len[b] keys of sequence b are visible to all of its queries
 *     (values below 0 count as 0, above L_kv as L_kv; without a causal mask
 *     it changes nothing);
 *   documents: query and key have the same number, doc_q[row] == doc_kv[row].
 * A query that sees no key gets o = 0, lse = -inf (and zero gradients).
 *   softcap: 0 (no cap), or positive with softmax_scale / softcap between
 *     2^-40 and 2^40; it and softmax_scale at most 2.3e38.
 *   dist_slopes: device fp32 [Hq] or NULL (constants: no gradient), of either
 *     sign; slope times distance must stay below 2^100.  Scores are fp32: a key's
 *     y, and a row's lse, are exact to 2^-22 of their size.
 *   doc_q [T_q], doc_kv [T_kv]: device int32 document number of every row, or
 *     both NULL.  They may be one array.  Inside a sequence the numbers of
 *     its valid rows must not decrease (else THD_DEV_ERR_DOC_ORDER); rows
 *     without a valid token are not looked at.
 *   prefix_len: device int32 [B] or NULL.
 * cp_size: padded lengths have to be divisible by 2 cp_size as in
 *   thd_attn_fwd.  Otherwise it changes nothing: with every rank's rows in the
 *   one buffer each sequence is walked as a whole, not by the ranks' chunks,
 *   and the outputs are those of any cp_size, bit for bit.
 * Key tiles that no query of a tile sees are skipped, whatever mask hides
 * them.  With none of the four given the call is thd_attn_fwd.  Every row
 * with a valid token must hold finite q, k, v, and so must up to 15 rows behind
 * a sequence's last one, pad rows, the next sequence's, or rows behind the last
 * (the backward: of dO too): a masked key's score counts nothing, but its row
 * of v is multiplied by 0.  With a softcap of at most 55.4, P is formed without a
 * running maximum, between 2^-80 and 2^80: elements of v have to be 0 or between
 * 2^-40 and 2^30 in magnitude, or they may be lost or overflow.
 * Other arguments as thd_attn_fwd; the workspace is larger:
 * thd_score_workspace_size(.., has_docs = doc_q != NULL, 0).
 * Launches: planner and forward; with documents two more (checks, extents).
 */
THD_API int thd_attn_score_fwd(const void* q, const void* k, const void* v, void* o, float* lse,
                               const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_kv,
                               const int32_t* cu_seqlens_q_padded, const int32_t* cu_seqlens_kv_padded, int B,
                               int64_t T_q, int64_t T_kv, int Hq, int Hkv, int D, int causal, float softmax_scale,
                               int cp_size, int pad_between_seqs, float softcap, const float* dist_slopes,
                               const int32_t* doc_q, const int32_t* doc_kv, const int32_t* prefix_len,
                               void* workspace, size_t workspace_bytes, int32_t* dev_status, thd_stream_t stream);

/*
 * thd_attn_score_bwd -- gradients of thd_attn_score_fwd w.r.t. q, k, v; with
 * P = exp(y - lse), dP = dO v^T, Delta = rowsum(dO * O):
 *     dx = P (dP - Delta) (1 - tanh^2(x / softcap)).
 * Arguments as thd_attn_bwd, with the modifications the forward was given;
 * workspace thd_score_workspace_size(.., has_docs, 1).  Bit-reproducible for a
 * workspace of the same size (a smaller one adds dK and dV up in other parts).
 * Delta, off by O's rounding to bf16, is corrected by the row sum of
 * P (dP - Delta): for dK always, for dQ with heads of 64 always, with heads of 128
 * in rows that see at most 128 keys and in heads with |dist_slopes[h]| >= 0.375.
 * Elsewhere dQ is as exact as plain
 * attention's: 2.4e-3 relative where the scores spread a row's weight, 3 to 4e-3
 * where they gather it on a few keys.  Launches: planner, preprocess, dQ and dK/dV; with documents
 * two more; with few key tiles to go round, one that joins dK/dV's parts.
 */
THD_API int thd_attn_score_bwd(const void* q, const void* k, const void* v, const void* o, const float* lse,
                               const void* dout, void* dq, void* dk, void* dv, int64_t dq_rows, int64_t dkv_rows,
                               const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_kv,
                               const int32_t* cu_seqlens_q_padded, const int32_t* cu_seqlens_kv_padded, int B,
                               int64_t T_q, int64_t T_kv, int Hq, int Hkv, int D, int causal, float softmax_scale,
                               int cp_size, int pad_between_seqs, float softcap, const float* dist_slopes,
                               const int32_t* doc_q, const int32_t* doc_kv, const int32_t* prefix_len,
                               void* workspace, size_t workspace_bytes, int32_t* dev_status, thd_stream_t stream);

/*
 * Bytes of workspace thd_attn_score_fwd (for_bwd = 0) or thd_attn_score_bwd
 * (for_bwd = 1) needs; has_docs: document numbers are given.  Returns 0 for
 * invalid sizes.  The backward of a call with few key tiles asks for more, to
 * share them among the SMs; what a call with more tokens asks for serves it too
 * (it then shares them less).
 */
THD_API size_t thd_score_workspace_size(int B, int64_t T_q, int64_t T_kv, int Hq, int Hkv, int D, int cp_size,
                                        int has_docs, int for_bwd);

/*
 * thd_lse_merge -- in place: (o_acc, lse_acc) <- merge((o_acc, lse_acc),
 * (o_part, lse_part)), the ring's per-step output correction
 * [P1 traceback].  Per (t, h), with a = lse_acc, b = lse_part:
 *     lse = max(a, b) + log1p(exp(-|a - b|))
 *     o   = exp(a - lse) o_acc + exp(b - lse) o_part
 * A side with lse = -inf contributes nothing; both -inf give (0, -inf).
 *   o_acc, o_part [T, H, D] fp32; lse_acc, lse_part [H, T] fp32; 16-byte
 *   aligned.  D a multiple of 4.  H at most 16384 (else THD_ERR_UNSUPPORTED).
 */
THD_API int thd_lse_merge(float* o_acc, float* lse_acc, const float* o_part, const float* lse_part, int64_t T, int H,
                  int D, thd_stream_t stream);

/*
 * thd_lse_merge_bf16 -- thd_lse_merge with the incoming partial o_part in
 * bf16 ([T, H, D], 8-byte aligned; thd_attn_fwd_step_bf16's output); the
 * accumulator (o_acc fp32, lse_acc) and lse_part are as in thd_lse_merge.
 */
THD_API int thd_lse_merge_bf16(float* o_acc, float* lse_acc, const void* o_part, const float* lse_part, int64_t T,
                               int H, int D, thd_stream_t stream);

/*
 * thd_grad_tail_zero -- zero gradient rows past the last padded endpoint:
 * rows [cu_seqlens_q_padded[B], dq_rows) of dq and [cu_seqlens_kv_padded[B],
 * dkv_rows) of dk and dv (bf16, [rows, H, D]).  [P2 "Describe the bug"]:
 * the THD tail-zero; [P2 "Expected behavior"]: no work when the valid
 * endpoint equals the buffer end.  The endpoint is read ON THE DEVICE (no
 * host sync, graph-safe); when the caller already knows there is no tail
 * (host_knows_no_tail = 1) nothing is launched.  Any of dq/dk/dv may be NULL.
 * An endpoint outside [0, rows] is invalid metadata: that buffer is left
 * untouched (no write ever falls outside [0, rows) of a buffer).
 */
THD_API int thd_grad_tail_zero(void* dq, void* dk, void* dv, int64_t dq_rows, int64_t dkv_rows, int Hq, int Hkv, int D,
                       const int32_t* cu_seqlens_q_padded, const int32_t* cu_seqlens_kv_padded, int B,
                       int host_knows_no_tail, thd_stream_t stream);

/*
 * ---- Ulysses (A2A) and hierarchical a2a+p2p context parallelism, emulated ----
 *
 * [P1, the maintainer's reply]: A2A (Ulysses) exchanges heads for sequence
 * and THD had no A2A path; [P3]: hierarchical CP runs A2A inside groups of
 * a2a_size ranks and the P2P ring across cp_size / a2a_size groups, with
 * prod(sizes) == cp_size.  Layouts (the pages print none; plainest reading):
 *   shards [cp_size][T/cp_size, H, D] bf16: CP rank r's THD shard, its rows
 *     in load-balanced order -- chunk r then chunk 2cp-1-r of every sequence,
 *     chunk = P_b / (2 cp_size) rows -- the rows thd_cp_partition's token map
 *     lists for rank r;
 *   groups [a2a_size][T, H/a2a_size, D] bf16: member i of the A2A groups
 *     holds heads [i H/a2a, (i+1) H/a2a) of every token at its global padded
 *     row.  Groups are runs of a2a_size consecutive ranks, so group j holds
 *     exactly p2p rank j's rows of the 2 * (cp/a2a) split.
 * a2a_size == cp_size is pure Ulysses; a2a_size == 1 is the plain P2P ring.
 * T is the global row count (shard stride T/cp_size rows, T % cp_size == 0);
 * rows past cu_seqlens_padded[B] are not moved.
 */

/*
 * thd_cp_a2a -- move one tensor between the two layouts, every rank and
 * group in one launch.  direction THD_A2A_TO_GROUPS reads shards from src
 * and writes groups to dst; THD_A2A_TO_SHARDS the reverse.
 *   src, dst: device bf16, 16-byte aligned, not overlapping.
 *   cu_seqlens_padded: device int32 [B+1]; checked on the device (starts at
 *     0, monotone, every P_b divisible by 2*cp_size, pad[B] <= T), else a
 *     THD_DEV_ERR_* code in *dev_status and nothing written.
 *   H % a2a_size == 0, cp_size % a2a_size == 0, D a multiple of 8.
 * Bit-exact (a permutation of rows).  Launches: the planner (checks only)
 * and the copy kernel.
 */
THD_API int thd_cp_a2a(const void* src, void* dst, const int32_t* cu_seqlens_padded, int B, int64_t T, int H, int D,
                       int cp_size, int a2a_size, int direction, int32_t* dev_status, thd_stream_t stream);

/*
 * Bytes of workspace thd_attn_fwd_a2a (for_bwd = 0) or thd_attn_bwd_a2a
 * (for_bwd = 1) needs: global-order copies of the moved tensors plus the
 * attention workspace.  Returns 0 for unsupported sizes.
 */
THD_API size_t thd_a2a_workspace_size(int B, int64_t T, int Hq, int Hkv, int D, int cp_size, int a2a_size,
                                      int for_bwd);

/*
 * thd_attn_fwd_a2a -- attention through the emulated A2A / hierarchical
 * decomposition: q, k, v shards -> the members' buffers (one launch); every
 * member runs the fused P2P ring of p2p = cp_size / a2a_size ranks over its
 * heads; O -> shards.  On one GPU the members' buffers are the head slices
 * of one tensor in global row order (the a2a_size = 1 layout of thd_cp_a2a),
 * so a single thd_attn_fwd launch with cp_size = p2p serves every member;
 * its work items are per head, so a member's result depends on its own
 * slice alone.  Equal to unsplit attention (tested).
 *   q [cp][T/cp, Hq, D], k, v [cp][T/cp, Hkv, D], o [cp][T/cp, Hq, D]: shards.
 *   lse: fp32 [Hq, T] in global row order (members' heads stacked).
 *   cu_seqlens, cu_seqlens_padded: device int32 [B+1], self-attention (the
 *     same for q and kv); the padded offsets define the shards.
 *   Hq, Hkv divisible by a2a_size; D 64 or 128.
 * Launches: 5 (checks, move in, planner, forward, move out).  Workspace:
 * thd_a2a_workspace_size(.., 0).
 */
THD_API int thd_attn_fwd_a2a(const void* q, const void* k, const void* v, void* o, float* lse,
                             const int32_t* cu_seqlens, const int32_t* cu_seqlens_padded, int B, int64_t T, int Hq,
                             int Hkv, int D, int causal, float softmax_scale, int cp_size, int a2a_size,
                             void* workspace, size_t workspace_bytes, int32_t* dev_status, thd_stream_t stream);

/*
 * thd_attn_bwd_a2a -- gradients through the same decomposition: q, k, v, o,
 * dO shards -> the members' buffers (one launch); the thd_attn_bwd path with
 * cp_size = p2p for every member at once; dQ, dK, dV -> shards (one launch).
 *   Shards as in thd_attn_fwd_a2a; lse [Hq, T] as it returns it; dq
 *   [cp][T/cp, Hq, D], dk, dv [cp][T/cp, Hkv, D].  Rows of each shard past
 *   cu_seqlens_padded[B] / cp_size are not written.
 * Launches: 7 (checks, move in, the four of thd_attn_bwd, move out).
 * Workspace: thd_a2a_workspace_size(.., 1).
 * Bit-reproducible.
 */
THD_API int thd_attn_bwd_a2a(const void* q, const void* k, const void* v, const void* o, const float* lse,
                             const void* dout, void* dq, void* dk, void* dv, const int32_t* cu_seqlens,
                             const int32_t* cu_seqlens_padded, int B, int64_t T, int Hq, int Hkv, int D, int causal,
                             float softmax_scale, int cp_size, int a2a_size, void* workspace, size_t workspace_bytes,
                             int32_t* dev_status, thd_stream_t stream);

/*
 * ---- operators on the rows around attention: rotary positions, dropout ----
 * They act on every one of the T rows they are given (a rank's shard, the
 * global buffer, or a part of either) and need no cu_seqlens, no workspace
 * and no device status: what can be wrong is seen on the host.
 */

/*
 * thd_rope -- rotary positions with several axes (for example time, height
 * and width) on queries and keys, one launch.  With f_i = inv_freq[i] and
 * a_i = axis_of[i] for i < rot_dim / 2, per row t and head the pair i,
 *     elements (i, i + rot_dim / 2)   (adjacent = 0)
 *     elements (2 i, 2 i + 1)         (adjacent = 1),
 * is turned by angle = positions[a_i][t] * f_i:
 *     (a, b) -> (a cos - b sin, b cos + a sin).
 * Elements past rot_dim are copied.  inverse = 1 turns by -angle: the
 * gradient of the inputs from the gradient of the outputs.  Angles are exact
 * to 2^-24 turns at any 32-bit position for |inv_freq| up to 2^40 (past that
 * the error grows with it); products and sums are fp32, rounded once.
 *   q_in, q_out: rows of [Hq, D]; k_in, k_out: rows of [Hkv, D] (NULL with
 *     Hkv = 0: queries alone).  `..._stride`: elements between rows, at least
 *     H * D (larger for a slice of a fused projection's output, as input or
 *     as output).  In place (out == in) needs equal strides; otherwise inputs
 *     and outputs must not overlap.  Aligned to the element size; 16-byte
 *     aligned rows with D a multiple of 8 and rot_dim of 16 (8 if adjacent)
 *     take 16-byte accesses.
 *   T rows, 0 <= T < 2^31; 1 <= D <= 1024; rot_dim even, 2 <= rot_dim <=
 *     min(D, 256).
 *   positions: device int32 [n_axes][T], any values; n_axes 1..16.
 *   inv_freq: HOST double [rot_dim / 2], finite; axis_of: HOST uint8
 *     [rot_dim / 2], each < n_axes.  Both are read before the call returns.
 *   dtype: THD_DTYPE_BF16 or THD_DTYPE_FP32 (inputs and outputs alike).
 */
THD_API int thd_rope(const void* q_in, const void* k_in, void* q_out, void* k_out, int64_t q_in_stride,
                     int64_t k_in_stride, int64_t q_out_stride, int64_t k_out_stride, int64_t T, int Hq, int Hkv,
                     int D, int rot_dim, const int32_t* positions, int n_axes, const double* inv_freq,
                     const uint8_t* axis_of, int adjacent, int inverse, int dtype, thd_stream_t stream);

/*
 * thd_dropout_add -- out = residual + keep(row, column) * x / (1 - p) on
 * [T, C] rows, the mask drawn from a counter-based generator and never
 * stored.  The gradient with respect to x is the same call on the output's
 * gradient, without a residual (that of the residual is the output's).
 *   Mask: Philox 4x32-10, key = rng[0], counter = (column / 8, id, rng[1]),
 *     16 bits an element (column 8 g + 2 w + h takes half h of word w); kept
 *     when they are >= round(65536 p), and scaled by 65536 / (65536 -
 *     round(65536 p)).  id is row_ids[row] when given, else the row's index:
 *     with a rank's token map as row_ids (thd_cp_partition), a shard draws
 *     what the unsplit buffer draws.
 *   x, out: [T, C], residual: [T, C] or NULL; out may be x or residual, else
 *     they must not overlap.  Aligned to the element size; 16-byte aligned
 *     tensors with C a multiple of 8 take 16-byte accesses.
 *   0 <= T < 2^31, 0 <= C < 2^31; 0 <= p, round(65536 p) < 65536.
 *   rng: DEVICE uint64 [2] = {seed, offset}, 8-byte aligned, read by the
 *     kernel: a captured graph draws a new mask when its owner changes them
 *     between replays.
 *   A dropped element gives the residual (or 0) whatever x holds.
 */
THD_API int thd_dropout_add(const void* x, const void* residual, void* out, int64_t T, int64_t C,
                            const int32_t* row_ids, double p, const uint64_t* rng, int dtype, thd_stream_t stream);

/*
 * ---- a paged key-value cache: what fills it, reads it and keeps it small ----
 *
 * A cache holds the keys and values of sequences in pages of page_size slots.
 * Sequence b's slot j is slot j % page_size of page block_table[b][j /
 * page_size]; its kv_len[b] first slots are held.  Entries of the table behind
 * those are not read.  The slots' order means nothing to attention: what a
 * slot's token was numbered is kept, where it matters, in `pos`.
 *   k, v: [num_pages][page_size][Hkv][D] in any order of the first three
 *     dimensions (kv_stride: elements from page to page, slot to slot and head
 *     to head, the same for both; rows contiguous).  16-byte aligned, strides a
 *     multiple of 16 bytes.  D 64 or 128.
 *   dtype THD_DTYPE_BF16, or THD_DTYPE_E4M3 with k_exp, v_exp: a uint8 for each
 *     slot and head (exp_stride, as kv_stride): the row stands for its e4m3
 *     numbers times 2^(exp - 127), 15 <= exp; 255: not a number.
 *   `weight` (fp32) and `pos` (int32) of the calls below are such arrays, a
 *     number for each slot and head, with weight_stride and pos_stride.
 *   num_pages < 2^31; max_pages * page_size <= 2^30; Hq / Hkv <= 512.
 *   A page may stand in several sequences' rows of the table while it is only
 *     read; what a call writes (append, evict, weights) lies in pages of one
 *     sequence, once.  Strides of 0 (one number for all heads, say) are for
 *     arrays that are only read, and for weight and pos of append.
 * The struct is read before a call returns; its pointers are device pointers.
 *
 * Device status of these calls: STICKY.  *dev_status is only ever raised, to
 * the largest code met; its owner zeroes it (once, before the first call, and
 * reads it when it likes: a captured graph of many steps keeps one word).  A
 * call that raises it neither reads nor writes outside the cache; what it writes
 * for the sequences concerned is unspecified.
 */
typedef struct thd_kv_cache {
  void* k;
  void* v;
  uint8_t* k_exp; /* NULL for THD_DTYPE_BF16 */
  uint8_t* v_exp;
  const int32_t* block_table; /* [B] rows of max_pages entries, table_stride entries apart */
  const int32_t* kv_len;      /* [B] */
  int64_t num_pages;
  int64_t table_stride;
  int64_t kv_stride[3]; /* page, slot, head: elements */
  int64_t exp_stride[3];
  int64_t weight_stride[3];
  int64_t pos_stride[3];
  int32_t page_size, max_pages, B, Hkv, D, dtype;
} thd_kv_cache;

/*
 * thd_cache_append -- the new rows of packed sequences into their caches, one
 * launch.  Sequence b's rows are [cu_seqlens[b], cu_seqlens[b+1]) of k and v,
 * m_b of them, and go to its slots [kv_len[b] - m_b, kv_len[b]): kv_len counts
 * them already, as for the attention that follows.  cu_seqlens NULL: one row a
 * sequence, T == B.  Rows behind cu_seqlens[B] are left out.
 *   k, v: bf16 rows of [Hkv, D], k_stride and v_stride elements apart (a
 *     slice of a fused projection's output), 16-byte aligned, strides too.
 *   e4m3: per row and head, with x the largest magnitude, the exponent is the
 *     smallest e with x <= 448 * 2^(e - 127), at least 67 (127 for a row of
 *     zeros); stored is the row times 2^(127 - e), rounded to nearest even.  A
 *     row with an infinity or NaN is stored as 255.
 *   weight, pos: NULL, or set for the new slots: 0, and the token's number
 *     tokens_seen[b] - m_b + i (tokens_seen NULL: kv_len).
 */
THD_API int thd_cache_append(const thd_kv_cache* cache, const void* k, const void* v, int64_t k_stride,
                             int64_t v_stride, int64_t T, const int32_t* cu_seqlens, float* weight, int32_t* pos,
                             const int32_t* tokens_seen, int32_t* dev_status, thd_stream_t stream);

/*
 * thd_attn_decode -- attention of one new token of each sequence over its
 * cache (which holds the token's own key and value: append first).  For
 * query head h of sequence b, over its visible slots j, kv_start[b] <= j <
 * kv_len[b] (kv_start NULL: 0, else clamped to [0, kv_len[b]]):
 *     x_j = softmax_scale q . k_j,  y_j = softcap tanh(x_j / softcap) (softcap 0: x_j)
 *           - dist_slopes[h] (tokens_seen[b] - 1 - pos_j)
 *     lse = log sum_j exp(y_j),  p_j = exp(y_j - lse),  o = sum_j p_j v_j
 * as thd_attn_score_fwd gives a sequence's last row.  No visible slot: o = 0,
 * lse = -inf.  Rows of several ranks' caches merge by thd_lse_merge.
 *   q: bf16 rows of [Hq, D], q_stride (even) elements apart, 4-byte aligned.
 *   o: bf16 [B, Hq, D], 16-byte aligned; lse: fp32 [Hq, B].  Neither overlaps
 *     an input.
 *   dist_slopes fp32 [Hq] or NULL.  pos NULL: a slot's token has the slot's
 *     number; tokens_seen NULL: kv_len.  Both are read with dist_slopes only.
 *   kv_start counts slots, not tokens: it is the start of the token's document
 *     while slots lie in their tokens' order, which is until thd_cache_evict
 *     moves some.  See there for what to do about documents then.
 *   weight_out NULL, or: weight_out = weight_in + the sum of p_j over the kv
 *     head's query heads, for the visible slots (weight_out may be weight_in,
 *     else they do not overlap).
 *   Lengths are read on the device: a captured graph serves growing ones.
 * Sums are fp32.  Probabilities meet bf16 values as two bf16 numbers each (to
 * 2^-16), above 16 query heads a kv head as one (2^-8); e4m3 values as fp16
 * (2^-11) after their row's scale is multiplied in, off by at most 2^-32 of the
 * largest such product (small ones keep fewer bits, below that none; rows of
 * zeros, whatever their scale, do not count as the largest).
 * Bit-reproducible on one kind of GPU.  Launches: 2 (1 for tables of at most 64
 * slots), with weights one more.  Workspace: thd_decode_workspace_size; calls that
 * may run at the same time need one each.
 */
THD_API int thd_attn_decode(const thd_kv_cache* cache, const void* q, int64_t q_stride, void* o, float* lse, int Hq,
                            float softmax_scale, float softcap, const float* dist_slopes, const int32_t* kv_start,
                            const int32_t* pos, const int32_t* tokens_seen, const float* weight_in,
                            float* weight_out, void* workspace, size_t workspace_bytes, int32_t* dev_status,
                            thd_stream_t stream);

/*
 * Bytes of workspace thd_attn_decode needs; capacity: max_pages * page_size
 * (it counts with weights alone: 4 bytes a slot and query head).  Returns 0
 * for invalid sizes.
 */
THD_API size_t thd_decode_workspace_size(int B, int Hq, int Hkv, int D, int64_t capacity, int has_weights);

/*
 * thd_cache_evict -- shrinks caches to `budget` slots, kv head by kv head, one
 * launch.  Of a sequence's n = kv_len[b] > budget slots the budget with the
 * largest weight stay, ties going to the lower slot; NaN counts as less than
 * all.  Slots whose token is among the first `sinks` (pos < sinks) or the last
 * `recent` (pos >= tokens_seen[b] - recent) stay before any weight, +infinity
 * too; where the budget holds fewer than those, the newest do (the largest pos;
 * those from tokens_seen[b] - 1 on count alike, and those 2^23 - 2 or more below).  Kept
 * slots in front of the budget stay where they are; the i-th kept slot behind
 * it moves into the i-th evicted slot in front of it: keys, values, exponents,
 * weight and pos.  Slots behind the budget are left as they were.
 *   new_len: int32 [B] = min(n, budget); neither kv_len nor tokens_seen.
 *   weight_out, pos_out: may be weight_in, pos_in (then only moved numbers are
 *     written), else they get those of all slots below new_len.
 *   0 < budget; sinks, recent >= 0.
 * Documents: slots leave their tokens' order, each kv head its own way, so no
 * kv_start of thd_attn_decode tells a document's tokens from earlier ones
 * afterwards.  Tokens that no later one may see are let go first, by a weight of
 * NaN in their slots (and sinks 0): where kv_len[b] - kv_start[b] >= budget, all
 * of them leave and the sequence goes on with kv_start 0.
 * Workspace: thd_evict_workspace_size.
 */
THD_API int thd_cache_evict(const thd_kv_cache* cache, const float* weight_in, float* weight_out,
                            const int32_t* pos_in, int32_t* pos_out, const int32_t* tokens_seen, int budget, int sinks,
                            int recent, int32_t* new_len, void* workspace, size_t workspace_bytes,
                            int32_t* dev_status, thd_stream_t stream);

/* Bytes of workspace thd_cache_evict needs; 0 for invalid sizes. */
THD_API size_t thd_evict_workspace_size(int B, int Hkv, int64_t capacity, int budget);

/*
 * Profiling hook (not needed for normal use): while enabled for `kernel_id`
 * (a THD_KERNEL_* value), every launch of that kernel is bracketed by a pair
 * of CUDA events recorded on its stream, up to `max_records` launches.
 * thd_profile_read synchronises those events and returns the durations in
 * milliseconds (oldest first) and their number.  kernel_id 0 disables.
 */
THD_API int thd_profile_enable(int kernel_id, int max_records);
THD_API int thd_profile_read(float* ms_out, int max_out, int* count_out);

/* Number of kernels this library has launched in this process. */
THD_API uint64_t thd_launch_count(void);

/*
 * Test hook for the failure path (not for normal use): the NEXT launch of
 * kernel_id (THD_KERNEL_FWD, THD_KERNEL_BWD or THD_KERNEL_BWD_DQ) runs no
 * work: every thread waits on a barrier that nothing completes, the bounded
 * wait gives up after its limit (2 s), each CTA frees its tensor memory and
 * the call's *dev_status reads THD_ERR_TIMEOUT.  That call's outputs are not
 * written.  The device stays usable for the next call.  kernel_id 0 disarms.
 * One-shot and process-wide.
 */
THD_API int thd_test_arm_stall(int kernel_id);

/*
 * Test hook (not for normal use): the forward has two kernels with the same
 * results up to rounding order -- one that runs a single work item per CTA
 * at a time (used when sequences average at least 16384 tokens) and one
 * with two items in flight per CTA (used otherwise).  which =
 * THD_FWD_KERNEL_SINGLE or THD_FWD_KERNEL_DUAL makes every later forward
 * call (fused or one-step) use that kernel, so tests can run both on any
 * workload; 0 restores the automatic choice.  Process-wide.  Returns
 * THD_ERR_INVALID_ARG for any other value.
 */
#define THD_FWD_KERNEL_SINGLE 1
#define THD_FWD_KERNEL_DUAL 2
THD_API int thd_test_select_fwd_kernel(int which);

#ifdef __cplusplus
}
#endif

#endif /* THD_ATTN_H */
