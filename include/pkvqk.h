/*
 * pkvqk — paged KV-cache decode attention for GB300 (sm_103a): C ABI.
 *
 * The decode step of an attention layer over a paged KV cache, in three
 * calls that follow the problem statement of InfiniLM PR #585 ("perf: Qwen3
 * offline inference — hybrid attention backend, fused rms_norm_rope, chunked
 * prefill + prompt-lookup spec decoding"), section "概述 / Summary":
 *
 *   1. pkvqk_norm_rope_append — item 2: fused per-head RMSNorm + full-rotary
 *      (neox rotate-half) RoPE on q and k; k and v then go into the paged
 *      BSHD cache (item 1) through a slot mapping.
 *   2. pkvqk_paged_decode     — item 1: split-KV paged decode attention with
 *      GQA read straight from the strided BSHD cache; with q_len > 1 it is
 *      the causal multi-query verify of item 4 (k + 1 tokens per sequence).
 *   3. pkvqk_lse_combine      — item 1 ("splitkv"): log-sum-exp merge of the
 *      split partials.
 *   4. pkvqk_paged_prefill    — item 4 (chunked prefill): the same causal
 *      attention for many new tokens per sequence (a prefill chunk after
 *      its prior context), on the tensor cores; pkvqk_paged_prefill_varlen
 *      takes a different number of new tokens per sequence (item 1's
 *      varlen prefill).
 *
 * Conventions shared by every call
 * --------------------------------
 * - Every buffer is owned by the caller; the library allocates no device
 *   memory and keeps no state beyond a per-thread error message, facts it
 *   caches per device (the SM count; each kernel's shared-memory limit, set
 *   once), the rotary sin/cos knot table it builds once on the host, and the
 *   fixed scratch of pkvqk_paged_decode_static_ws (below).
 * - Pointers marked "device" must be device (or managed) memory of the
 *   current device; they are checked with cudaPointerGetAttributes and a
 *   host pointer is rejected with PKVQK_ERR_POINTER_RESIDENCY.
 * - bf16 means IEEE bfloat16 (raw 16-bit storage).  Strides are in elements.
 * - Work is enqueued on `stream`; no call synchronises, reads device memory
 *   on the host, or allocates, so every call can be recorded into a CUDA
 *   graph.  Argument errors are detected on the host before any launch and
 *   leave all buffers untouched.
 * - `status_flags` (optional, may be NULL) is a device int32 into which the
 *   kernels OR the PKVQK_FLAG_* bits below when they meet bad data (an
 *   out-of-range block id or slot) or a pipeline wait that timed out.  The
 *   caller zeroes it and reads it back when convenient.
 * - On failure the call returns a non-zero pkvqk_status and
 *   pkvqk_last_error() describes it.
 */
#ifndef PKVQK_H
#define PKVQK_H

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define PKVQK_API __attribute__((visibility("default")))
#else
#define PKVQK_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

/* Same handle as cudaStream_t / CUstream; NULL is the legacy default stream. */
typedef struct CUstream_st* pkvqk_stream_t;

typedef enum pkvqk_status {
  PKVQK_OK = 0,
  PKVQK_ERR_INVALID_ARG = 1,          /* null pointer, bad size, misaligned   */
  PKVQK_ERR_UNSUPPORTED = 2,          /* valid but not implemented (e.g. D)   */
  PKVQK_ERR_WORKSPACE_TOO_SMALL = 3,
  PKVQK_ERR_POINTER_RESIDENCY = 4,    /* host pointer where device expected   */
  PKVQK_ERR_CUDA = 5                  /* a CUDA runtime/driver call failed    */
} pkvqk_status;

/* Bits OR-ed into *status_flags by the kernels. */
#define PKVQK_FLAG_BAD_SLOT      0x1  /* slot >= num_blocks*block_size: skipped */
#define PKVQK_FLAG_BAD_BLOCK_ID  0x2  /* block id outside [0, num_blocks): its keys read as zeros */
#define PKVQK_FLAG_WAIT_TIMEOUT  0x4  /* a pipeline wait gave up: output invalid */
#define PKVQK_FLAG_BAD_VALUE     0x8  /* 8-bit append: a k or v value that is not finite;
                                         drafts: a NaN or negative probability, or none above 0 */
#define PKVQK_FLAG_BAD_TOKEN     0x10 /* drafted token outside [0, vocab_size): not accepted */

/*
 * Layout of a paged cache, shared by the K and the V cache of a layer:
 * element (block, slot, head, d) lives at
 *     base + block*block_stride + slot*slot_stride + head*head_stride + d.
 * The default BSHD layout [num_blocks, block_size, num_kv_heads, head_dim]
 * has block_stride = block_size*num_kv_heads*head_dim,
 * slot_stride = num_kv_heads*head_dim, head_stride = head_dim; any strides
 * that are multiples of 8 elements (16 bytes) are accepted, so K and V may be
 * two views into one interleaved or stacked allocation (no copy is made).
 * block_size must be a multiple of 16 (16..256); head_dim must be 128.
 */
typedef struct pkvqk_cache_layout {
  int64_t num_blocks;
  int32_t block_size;
  int32_t num_kv_heads;
  int32_t head_dim;
  int32_t reserved;                  /* set to 0 */
  int64_t block_stride;
  int64_t slot_stride;
  int64_t head_stride;
} pkvqk_cache_layout;

/* Code formats of an 8-bit cache. */
typedef enum pkvqk_q8_format {
  PKVQK_Q8_E4M3 = 1,                 /* 1-4-3 floating point, largest value 448 */
  PKVQK_Q8_INT8 = 2                  /* two's complement, -127 .. 127 */
} pkvqk_q8_format;

/*
 * A layer's 8-bit K and V caches: one code a value, and one fp32 scale for
 * each group of 16 consecutive slots of a page and kv head, K and V apart;
 * the value is code * scale.  Codes follow `layout` (one byte an element; the
 * strides, in elements, are multiples of 16 here); the scale of (block, slot,
 * head) lives at
 *     scales + block*scale_block_stride + (slot / 16)*scale_group_stride
 *            + head*scale_head_stride
 * (positive strides; e.g. [num_blocks, block_size / 16, num_kv_heads]).
 * pkvqk_norm_rope_append_q8 writes powers of two from 2^-64 to 2^63; the
 * attention calls take any positive scale in that range and move others (0,
 * negative, NaN) to its nearest end, NaN to 2^-64.  Per key and kv head the
 * pair takes 2*(128 + 4/16) bytes, 0.501 of a bf16 cache.
 */
typedef struct pkvqk_q8_cache {
  void* k;                           /* device codes, 16-byte aligned */
  void* v;
  float* k_scales;                   /* device scales, 4-byte aligned */
  float* v_scales;
  pkvqk_cache_layout layout;
  int32_t format;                    /* pkvqk_q8_format, of K and of V */
  int32_t reserved;                  /* set to 0 */
  int64_t scale_block_stride;
  int64_t scale_group_stride;
  int64_t scale_head_stride;
} pkvqk_q8_cache;

/*
 * Rules that the scored attention calls (pkvqk_paged_decode_scored,
 * pkvqk_paged_prefill_scored, pkvqk_paged_prefill_varlen_scored) put on scores and on
 * what a row sees.  All zero: plain causal attention.  For the row at position
 * p = seq_len - q_len + t of sequence b, q head h and key n:
 *   s = scale * <q, K_n>
 *   s = softcap * tanh(s / softcap)          where softcap > 0
 *   s = s - slopes[h] * |p - n|              where slopes is given
 *   n is visible where lo <= n < hi:
 *     lo = max(0, p - window + 1 (where window > 0), first_keys[row])
 *     hi = max(p + 1, min(prefix_lens[b], seq_len))
 * So a window keeps the last `window` keys of a row, its own among them; first_keys
 * gives each token row the first key of its document (or of what is not padding); the
 * keys of a prefix are seen by every row of the sequence, also by those before them, from
 * the row's lo on.
 * first_keys bounds a row from below alone: what keeps a row from the documents after its
 * own is that they lie behind it, and a prefix lifts that.  With documents a prefix is the
 * first document's and must not reach past its end; a longer one shows the rows of every
 * document that it reaches past the keys of the next, and none of this is checked.  (Up to
 * that end it changes nothing for later documents: they stay causal.)
 */
typedef struct pkvqk_score_rules {
  float softcap;                     /* 0 (none) or 2^-20 .. 2^20 */
  int32_t window;                    /* keys; 0: none */
  const float* slopes;               /* device fp32 [num_q_heads] or NULL */
  const int32_t* first_keys;         /* device int32, one per token row of q, or NULL */
  const int32_t* prefix_lens;        /* device int32 [batch] or NULL */
} pkvqk_score_rules;

/* Message of the last failing call made on this thread ("" if none). */
PKVQK_API const char* pkvqk_last_error(void);

/* ABI version of this header: 1. */
PKVQK_API int32_t pkvqk_abi_version(void);

/*
 * Fused per-head RMSNorm + neox RoPE on q and k, then the k/v append.
 * Source: InfiniLM PR #585, "概述 / Summary" item 2 ("rms_norm_rope"), item 1
 * (BSHD paged cache).
 *
 * For each token t < num_tokens and head h, with x the head's D values:
 *   y = x / sqrt(mean(x^2) + eps) * gamma          (gamma_q for q, gamma_k for k)
 *   for i < D/2, a = positions[t] * theta^(-2i/D):
 *     y'[i]       = y[i] cos a - y[i + D/2] sin a
 *     y'[i + D/2] = y[i + D/2] cos a + y[i] sin a
 * rounded once to bf16 (round-to-nearest-even).  q is overwritten in place.
 * With s = slot_mapping[t] in [0, num_blocks*block_size), the rotated k and
 * the unchanged v of every kv head go to block s / block_size, slot
 * s % block_size of k_cache / v_cache.  s < 0 (padding) writes nothing; a
 * too-large s writes nothing and sets PKVQK_FLAG_BAD_SLOT.
 *
 *   q             device bf16, element (t, h, d) at q[t*q_stride_t + h*q_stride_h + d]
 *   k, v          device bf16, same form with their own strides, Hkv heads
 *   positions     device int64 [num_tokens]
 *   slot_mapping  device int64 [num_tokens]
 *   gamma_q/_k    device bf16 [head_dim]
 *   k_cache, v_cache  device bf16, layout as described by `layout`
 * Two tokens mapped to the same slot race (caller error).  Strides and base
 * pointers must be 16-byte aligned.
 */
PKVQK_API pkvqk_status pkvqk_norm_rope_append(
    void* q, int64_t q_stride_t, int64_t q_stride_h,
    const void* k, int64_t k_stride_t, int64_t k_stride_h,
    const void* v, int64_t v_stride_t, int64_t v_stride_h,
    const int64_t* positions, const int64_t* slot_mapping,
    const void* gamma_q, const void* gamma_k,
    float theta, float eps,
    int32_t num_tokens, int32_t num_q_heads,
    void* k_cache, void* v_cache, const pkvqk_cache_layout* layout,
    int32_t* status_flags, pkvqk_stream_t stream);

/*
 * Bytes of a rotary table for positions 0 .. max_positions-1: 1 KiB per
 * position.  0 when max_positions is outside 1 .. 2^21.
 */
PKVQK_API size_t pkvqk_rope_table_bytes(int32_t max_positions);

/*
 * Fills `table` with the rotary sin/cos that pkvqk_norm_rope_append computes
 * for a token at each position p < max_positions (same source, item 2): for
 * i < D/2 the angle p * theta^(-2i/D), reduced and evaluated exactly as that
 * call does, kept as float-float pairs.  Build once per model (theta and the
 * longest context), before the steps that read it; the table depends on
 * nothing else.
 *
 *   table          device, 16-byte aligned, pkvqk_rope_table_bytes(max_positions)
 *                  bytes, owned by the caller; written by a kernel on `stream`
 *   max_positions  0 .. 2^21 (0: nothing to do)
 * Errors: PKVQK_ERR_INVALID_ARG (max_positions out of range, theta not > 0,
 * table not a 16-byte aligned device pointer).
 */
PKVQK_API pkvqk_status pkvqk_rope_table_build(void* table, int32_t max_positions, float theta,
                                              pkvqk_stream_t stream);

/*
 * pkvqk_norm_rope_append with the angles of tokens at positions
 * 0 .. table_positions-1 read from a table built by pkvqk_rope_table_build
 * (with the same theta) instead of computed per token.  Tokens at other
 * positions compute theirs as pkvqk_norm_rope_append does.  The results are
 * bit-identical to pkvqk_norm_rope_append's.  Every other argument and error
 * as there; table_positions 0 .. 2^21 (0: no table is read).
 */
PKVQK_API pkvqk_status pkvqk_norm_rope_append_cached(
    void* q, int64_t q_stride_t, int64_t q_stride_h,
    const void* k, int64_t k_stride_t, int64_t k_stride_h,
    const void* v, int64_t v_stride_t, int64_t v_stride_h,
    const int64_t* positions, const int64_t* slot_mapping,
    const void* gamma_q, const void* gamma_k,
    float theta, float eps,
    int32_t num_tokens, int32_t num_q_heads,
    void* k_cache, void* v_cache, const pkvqk_cache_layout* layout,
    const void* rope_table, int32_t table_positions,
    int32_t* status_flags, pkvqk_stream_t stream);

/*
 * pkvqk_norm_rope_append with rotary positions of several axes, as the tokens of
 * images and videos have (time, height, width): frequency i < D/2 of token t
 * turns by the angle
 *     positions[freq_axes[i]*positions_stride_a + t] * theta^(-2i/D),
 * everything else as there.  Text tokens have the same position on every axis
 * and get what pkvqk_norm_rope_append gives them, bit for bit.
 *
 *   q, q_out           device bf16, own strides; q_out may be q, else they must not overlap
 *   positions          device int64, [num_axes][num_tokens], the axes positions_stride_a
 *                      elements apart, a token's neighbours adjacent
 *   num_axes           1 .. 4
 *   freq_axes          HOST uint8 [head_dim / 2], each below num_axes; read before the
 *                      call returns.  Contiguous sections and interleaved axes are both
 *                      such maps; where every four frequencies 4l .. 4l+3 share an axis a
 *                      token's angles are read from the table in 16-byte pieces
 *   rope_table, table_positions   as pkvqk_norm_rope_append_cached (0: no table is read); a
 *                      token is served by the table where it has the positions of all its axes
 */
PKVQK_API pkvqk_status pkvqk_norm_rope_append_axes(
    const void* q, int64_t q_stride_t, int64_t q_stride_h,
    void* q_out, int64_t q_out_stride_t, int64_t q_out_stride_h,
    const void* k, int64_t k_stride_t, int64_t k_stride_h,
    const void* v, int64_t v_stride_t, int64_t v_stride_h,
    const int64_t* positions, int64_t positions_stride_a,
    int32_t num_axes, const uint8_t* freq_axes,
    const int64_t* slot_mapping,
    const void* gamma_q, const void* gamma_k,
    float theta, float eps,
    int32_t num_tokens, int32_t num_q_heads,
    void* k_cache, void* v_cache, const pkvqk_cache_layout* layout,
    const void* rope_table, int32_t table_positions,
    int32_t* status_flags, pkvqk_stream_t stream);

/*
 * pkvqk_norm_rope_append into an 8-bit cache: the same norm and rotation of q
 * and k (angles from rope_table for positions 0 .. table_positions-1, computed
 * for others; table_positions 0: all computed), q written to q_out (which may
 * be q), rotated k and v quantised from fp32 with one rounding.
 *
 * For every group of 16 slots that the call writes, per kv head and for K and
 * V apart, with a the largest |value| that it writes there and M = 448 (e4m3)
 * or 127 (int8):
 *   2^e, e the smallest integer in -64 .. 63 with a <= M*2^e (at most 63)
 *   scale = 2^e                        where slot 0 of the group is written,
 *         = max(2^e, stored scale)     elsewhere: the group holds earlier tokens
 *   code  = value / scale, to the nearest code, ties to even (in calls of 2048
 *           tokens and more K's values come from an fp32 norm and rotation, and
 *           one within 2^-20 of itself of the middle between two codes may get
 *           either; so may, in any call, a subnormal e4m3 code)
 * In any call K's a comes from that norm and rotation: within 2^-20 of M*2^e it may
 * get that e or the next.  A stored scale that is no power of two is kept as it is
 * where it is the larger; value / scale is then rounded to fp32 before the code.
 * Where the stored scale grew, the codes of the group's other slots are
 * rescaled (code * old / new, to the nearest), so that earlier tokens keep
 * their values.  Writing slot 0 starts a group anew: what other slots of it
 * hold is free.  A stored scale outside 2^-64 .. 2^63 counts as 2^-64.
 * Values beyond M*scale (infinities, or a scale at its limit) become the
 * largest code, NaN becomes 0, and neither counts for a; PKVQK_FLAG_BAD_VALUE
 * reports values that are not finite.
 *
 * Tokens of one call whose slots lie in one group must be adjacent in token
 * order (as the consecutive tokens of a sequence are), with no other token and
 * no padding between them; otherwise, as when two tokens share a slot, the
 * group's contents are undefined.  Such near-ties aside, results do not depend
 * on how a sequence's other groups are spread over calls.
 *
 *   q, k, v, positions, slot_mapping, gamma_q/_k, theta, eps: as
 *   pkvqk_norm_rope_append; q_out as q (own strides); rope_table as
 *   pkvqk_norm_rope_append_cached
 */
PKVQK_API pkvqk_status pkvqk_norm_rope_append_q8(
    const void* q, int64_t q_stride_t, int64_t q_stride_h,
    void* q_out, int64_t q_out_stride_t, int64_t q_out_stride_h,
    const void* k, int64_t k_stride_t, int64_t k_stride_h,
    const void* v, int64_t v_stride_t, int64_t v_stride_h,
    const int64_t* positions, const int64_t* slot_mapping,
    const void* gamma_q, const void* gamma_k,
    float theta, float eps,
    int32_t num_tokens, int32_t num_q_heads,
    const pkvqk_q8_cache* cache,
    const void* rope_table, int32_t table_positions,
    int32_t* status_flags, pkvqk_stream_t stream);

/*
 * Schedule for pkvqk_paged_decode from host-side facts only (no device
 * read): batch, kv heads, rows per kv head (q_len * Hq/Hkv), the longest
 * sequence, the total key count and the SM count (0 = query the current
 * device).  Returns 0 (the balanced schedule: chosen for large batches whose
 * total keys are under half of batch x longest) or a split count in
 * [1, 256]; above 16 rows per kv head
 * (run on the tensor-core kernel, see pkvqk_paged_decode) it returns
 * pkvqk_choose_prefill_splits(batch, num_kv_heads, rows_per_kv_head, 1, ...).
 * Source: the "decode routing hint (host side, zero device sync)" of
 * InfiniLM PR #585, Summary item 3.
 */
PKVQK_API int32_t pkvqk_choose_num_splits(int32_t batch, int32_t num_kv_heads,
                                int32_t rows_per_kv_head, int32_t max_seq_len,
                                int64_t total_tokens, int32_t block_size,
                                int32_t sm_count);

/*
 * Workspace bytes pkvqk_paged_decode needs on the current device:
 * - num_splits == 1: 0;
 * - num_splits >= 2: batch*q_len*Hq*num_splits*(head_dim + 1)*4, rounded up
 *   to 256.  Layout: fp32 partial outputs [rows][num_splits][head_dim], then
 *   fp32 partial lse [rows][num_splits] (rows = (b*q_len + t)*Hq + h);
 * - num_splits == 0 (balanced): an upper bound for any kv-head count,
 *   ((SMs + batch)*q_len*Hq*(head_dim + 1)*4 + batch*Hq*8) rounded up, where
 *   SMs is the current device's multiprocessor count (internal layout).
 * Nothing in the workspace needs to start at zero, and calls of any shape and
 * schedule may share one (in stream order).
 */
PKVQK_API size_t pkvqk_decode_workspace_bytes(int32_t batch, int32_t q_len,
                                    int32_t num_q_heads, int32_t head_dim,
                                    int32_t num_splits);

/*
 * Split-KV paged decode attention with GQA; causal multi-query verify when
 * q_len > 1.  Source: InfiniLM PR #585, "概述 / Summary" items 1 and 4.
 *
 * For sequence b, query token t < q_len and q head h (kv head h / (Hq/Hkv)):
 *   visible keys  n < seq_lens[b] - q_len + t + 1, key n at block
 *                 block_tables[b*max_blocks_per_seq + n / block_size],
 *                 slot n % block_size
 *   s_n = scale * <q, K_n>   (scale <= 0 selects head_dim^-1/2)
 *   out = sum_n softmax(s)_n V_n,  lse = log sum_n exp(s_n)
 * A row with no visible key outputs 0 and lse = -inf; a row with a NaN score is
 * NaN, lse included.
 *
 * Schedules (the result does not depend on them, up to rounding):
 * - num_splits >= 1 (split-KV): with C = ceil(ceil(max_seq_len_hint /
 *   block_size) / num_splits) pages, split j < S-1 of a sequence covers pages
 *   [j*C, (j+1)*C) and split S-1 covers [(S-1)*C, end), so every key is
 *   covered whatever the hint.  Each split keeps an online softmax; for
 *   num_splits > 1 the partials go to the workspace and a log-sum-exp
 *   combine kernel that this call launches (as a programmatic dependent, so
 *   its launch overlaps the decode kernel's tail) merges them.
 *   pkvqk_choose_num_splits gives a host-side choice.
 * - num_splits == 0 (balanced): a persistent grid of 0.84 CTAs per SM; the
 *   pages of all (sequence, kv-head group) pairs are laid end to end and
 *   every CTA takes an equal contiguous share, crossing sequence boundaries;
 *   a sequence covered by one CTA is written directly, one cut across CTAs is
 *   merged by a combine kernel this call launches.  Balances any mix of
 *   lengths.
 *
 *   q             device bf16, element (b*q_len + t, h, d) at
 *                 q[(b*q_len + t)*q_stride_t + h*q_stride_h + d]
 *   block_tables  device int32 [batch, max_blocks_per_seq]
 *   seq_lens      device int32 [batch], counting the q_len new tokens
 *   num_splits    0 (balanced schedule) or 1..256 (split schedule)
 *   max_seq_len_hint  host int >= the longest seq_len (0 = max_blocks_per_seq*block_size)
 *   out           device bf16 [batch, q_len, Hq, head_dim], contiguous
 *   lse_out       device fp32 [batch, q_len, Hq] or NULL
 *   workspace     device, >= pkvqk_decode_workspace_bytes(batch, q_len, Hq,
 *                 head_dim, num_splits) on the current device (NULL if 0)
 * Supported: head_dim 128, Hq % Hkv == 0, q_len <= 16.  Up to 16 rows per
 * kv head (q_len*Hq/Hkv) run on the decode kernel; more (e.g. q_len 5 at
 * 8 q heads per kv head) run on the tensor-core multi-query kernel of
 * pkvqk_paged_prefill with the same split boundaries and partial layout,
 * and num_splits == 0 there becomes a split count whose partials fit the
 * balanced workspace bound.
 */
PKVQK_API pkvqk_status pkvqk_paged_decode(
    const void* q, int64_t q_stride_t, int64_t q_stride_h,
    const void* k_cache, const void* v_cache, const pkvqk_cache_layout* layout,
    const int32_t* block_tables, int32_t max_blocks_per_seq,
    const int32_t* seq_lens,
    int32_t batch, int32_t q_len, int32_t num_q_heads,
    int32_t num_splits, int32_t max_seq_len_hint, float scale,
    void* out, float* lse_out,
    void* workspace, size_t workspace_bytes,
    int32_t* status_flags, pkvqk_stream_t stream);

/*
 * pkvqk_paged_decode under score rules (pkvqk_score_rules), with the same schedules,
 * workspace and limits.  Of a sequence only the pages from its rows' first visible key
 * on are read, and splits are counted from the page of that key: block-table entries
 * before it may hold anything, and max_seq_len_hint bounds the keys from there to the
 * sequence's end (a window bounds them too, without a hint); give
 * pkvqk_choose_num_splits such spans in place of lengths.  The first visible key is that of
 * the rows that see any.  Slots past seq_lens[b] and before the first visible key may hold
 * anything, NaN included.  A V between them that is not finite, or of a magnitude of 2^46
 * and more, may make NaN or infinities of any row of its sequence and kv head.  A row with
 * no visible key outputs 0 and lse = -inf; a row with a NaN score is NaN, lse included.
 */
PKVQK_API pkvqk_status pkvqk_paged_decode_scored(
    const void* q, int64_t q_stride_t, int64_t q_stride_h,
    const void* k_cache, const void* v_cache, const pkvqk_cache_layout* layout,
    const int32_t* block_tables, int32_t max_blocks_per_seq,
    const int32_t* seq_lens,
    int32_t batch, int32_t q_len, int32_t num_q_heads,
    int32_t num_splits, int32_t max_seq_len_hint, float scale,
    const pkvqk_score_rules* rules,
    void* out, float* lse_out,
    void* workspace, size_t workspace_bytes,
    int32_t* status_flags, pkvqk_stream_t stream);

/*
 * pkvqk_paged_decode over an 8-bit cache: the same definition with K_n and V_n
 * = code * scale, the same schedules (the balanced one with a CTA per SM),
 * pkvqk_choose_num_splits and pkvqk_decode_workspace_bytes.  Codes and q enter
 * the products exactly (a q row is scaled by a power of two first; only what is
 * 2^-28 below its largest magnitude is rounded), sums are fp32, softmax weights
 * are rounded to 2^-11.  Slots at or past seq_lens[b] may hold any code and scale;
 * an e4m3 NaN code of a visible V makes NaN of every row of its sequence and
 * kv head.
 * More than 16 rows per kv head run as pkvqk_paged_prefill_q8 does.
 */
PKVQK_API pkvqk_status pkvqk_paged_decode_q8(
    const void* q, int64_t q_stride_t, int64_t q_stride_h,
    const pkvqk_q8_cache* cache,
    const int32_t* block_tables, int32_t max_blocks_per_seq,
    const int32_t* seq_lens,
    int32_t batch, int32_t q_len, int32_t num_q_heads,
    int32_t num_splits, int32_t max_seq_len_hint, float scale,
    void* out, float* lse_out,
    void* workspace, size_t workspace_bytes,
    int32_t* status_flags, pkvqk_stream_t stream);

/*
 * As pkvqk_paged_decode but stops after the split pass: the partials stay in
 * the workspace (layout above) and are not merged (pkvqk_lse_combine merges
 * them).  num_splits must be >= 2 (no heuristic).
 */
PKVQK_API pkvqk_status pkvqk_paged_decode_partials(
    const void* q, int64_t q_stride_t, int64_t q_stride_h,
    const void* k_cache, const void* v_cache, const pkvqk_cache_layout* layout,
    const int32_t* block_tables, int32_t max_blocks_per_seq,
    const int32_t* seq_lens,
    int32_t batch, int32_t q_len, int32_t num_q_heads,
    int32_t num_splits, int32_t max_seq_len_hint, float scale,
    void* workspace, size_t workspace_bytes,
    int32_t* status_flags, pkvqk_stream_t stream);

/*
 * pkvqk_paged_decode without a caller workspace.  The pages describe no such
 * call: it has no counterpart there and exists for callers that cannot
 * allocate device memory — e.g. a plugin that a host engine hands only input
 * and output pointers, or code running while an allocator refuses to
 * allocate — and so cannot pass the split workspace.
 *
 * Same arguments and results as pkvqk_paged_decode minus workspace and
 * workspace_bytes, except that num_splits == 0 here picks the split count
 * with pkvqk_choose_num_splits (the split schedule) instead of the balanced
 * schedule.  The split partials go to a fixed 16 MiB array inside the
 * library (pkvqk_static_workspace_capacity()), held on every GPU that loads
 * the library until the process exits.  A call whose partials need more
 * (pkvqk_decode_workspace_bytes for its split count) returns
 * PKVQK_ERR_WORKSPACE_TOO_SMALL and launches nothing; so does a
 * num_splits == 0 call whose chosen split count needs more.  Arguments that
 * pkvqk_paged_decode rejects are rejected the same way here.  The call
 * allocates nothing.  The first call on a device looks up the array's device
 * address (cudaGetSymbolAddress, with that device current) and caches it for
 * the CUDA context current at that time; a later call under another context
 * of the device (a driver context made current by the caller, or the primary
 * context re-created after cudaDeviceReset) looks it up again.  Make the
 * first call in each context before any stream capture.  All calls on a
 * device share the one array and it keeps the last call's partials: calls
 * that can overlap on the GPU (different streams, no ordering between them)
 * race and corrupt each other's results.  Nothing in it needs to start at
 * zero.
 */
PKVQK_API pkvqk_status pkvqk_paged_decode_static_ws(
    const void* q, int64_t q_stride_t, int64_t q_stride_h,
    const void* k_cache, const void* v_cache, const pkvqk_cache_layout* layout,
    const int32_t* block_tables, int32_t max_blocks_per_seq,
    const int32_t* seq_lens,
    int32_t batch, int32_t q_len, int32_t num_q_heads,
    int32_t num_splits, int32_t max_seq_len_hint, float scale,
    void* out, float* lse_out,
    int32_t* status_flags, pkvqk_stream_t stream);

/* Bytes of the array pkvqk_paged_decode_static_ws uses (16 MiB). */
PKVQK_API size_t pkvqk_static_workspace_capacity(void);

/*
 * Log-sum-exp merge of split partials.  Source: InfiniLM PR #585, Summary
 * item 1 ("splitkv").  For each row r < rows:
 *   M = max_j lse[r][j];  w_j = exp(lse[r][j] - M)
 *   out[r] = sum_j w_j o[r][j] / sum_j w_j,  lse_out[r] = M + log sum_j w_j
 * Splits with lse = -inf weigh 0; a row whose splits are all empty outputs
 * 0 and -inf, one with a split whose lse is NaN NaN.
 *   ws_o    device fp32 [rows][num_splits][head_dim]
 *   ws_lse  device fp32 [rows][num_splits]
 *   out     device bf16 [rows][head_dim];  lse_out device fp32 [rows] or NULL
 * head_dim must be 128.
 */
PKVQK_API pkvqk_status pkvqk_lse_combine(const float* ws_o, const float* ws_lse,
                               int32_t rows, int32_t head_dim,
                               int32_t num_splits, void* out, float* lse_out,
                               pkvqk_stream_t stream);

/* Types of the probabilities that pkvqk_verify_drafts reads. */
typedef enum pkvqk_prob_type {
  PKVQK_PROB_FP32 = 0,
  PKVQK_PROB_BF16 = 1,
  PKVQK_PROB_FP16 = 2
} pkvqk_prob_type;

/*
 * Verdict on drafted tokens, after a verify step (pkvqk_paged_decode with
 * q_len = drafts + 1, and the model's head) has given the target's probabilities.
 * Source: the speculative verify of InfiniLM PR #585, Summary item 4.
 *
 * Sequence b has n = draft_lens[b] drafts (max_drafts where draft_lens is NULL) x_i,
 * target rows p_i, i <= n, draft rows q_i, i < n, and uniforms u_i.  With
 * draft_probs NULL the drafts were certain (looked up in the prompt): q_i(x_i) is 1
 * and q_i is 0 elsewhere.
 *   draft i is accepted if all before it are and u_i * q_i(x_i) < p_i(x_i) (the
 *   product not rounded); j = the number accepted
 *   w(v) = max(p_j(v) - q_j(v), 0) where j < n; p_n(v) where j = n; where no w(v) is
 *   above 0, w = p_j
 *   y = the smallest v with w(0) + .. + w(v) > u_{max_drafts} * sum of w
 *   tokens[b] = x_0 .. x_{j-1}, y, then -1;  num_accepted[b] = j
 *   kept_lens[b] = seq_lens[b] - (n - j): the keys that stay, where seq_lens[b] counts
 *   the cached tokens of the verify step; what the cache holds past them is free
 * so that with independent u, uniform in [0, 1), the tokens are distributed as the
 * target's own.  For y probabilities count as multiples of 2^-44, to the nearest; sums of
 * them and u times the sum are exact.  Probabilities above 1 count as 1, NaN and negative
 * ones as 0, where drafts are judged and where y is drawn (reported by PKVQK_FLAG_BAD_VALUE
 * where y's rows hold them); a row without any weight gives y = -1 and the same flag.  A
 * draft outside [0, vocab_size) is not accepted, takes no weight away where draft_probs is
 * NULL, and is reported by PKVQK_FLAG_BAD_TOKEN.  u_{max_drafts} below 0 and NaN counts as
 * 0, from 1 on as just below 1; the other u_i are compared as they are.
 *
 *   target_probs  device, row (b, i) of vocab_size values at
 *                 b*target_stride_b + i*target_stride_t elements, i <= max_drafts
 *   draft_probs   device, the same type, i < max_drafts; or NULL
 *   type          pkvqk_prob_type of both; 16-byte rows (base, strides) are read fastest
 *   draft_tokens  device int32 [batch, max_drafts]   (may be NULL where max_drafts is 0)
 *   draft_lens    device int32 [batch] or NULL; values outside 0 .. max_drafts count as
 *                 the nearest of them
 *   uniforms      device fp32 [batch, max_drafts + 1]
 *   tokens        device int32 [batch, max_drafts + 1];  num_accepted device int32 [batch]
 *   seq_lens, kept_lens  device int32 [batch], both or neither; may be the same
 * Rows past n are not read.  max_drafts 0 .. 255 (0: y drawn from p_0), vocab_size
 * 1 .. 2^20 - 1, batch <= 65535.
 */
PKVQK_API pkvqk_status pkvqk_verify_drafts(
    const void* target_probs, int64_t target_stride_b, int64_t target_stride_t,
    const void* draft_probs, int64_t draft_stride_b, int64_t draft_stride_t,
    int32_t type,
    const int32_t* draft_tokens, const int32_t* draft_lens, const float* uniforms,
    int32_t batch, int32_t max_drafts, int32_t vocab_size,
    int32_t* tokens, int32_t* num_accepted,
    const int32_t* seq_lens, int32_t* kept_lens,
    int32_t* status_flags, pkvqk_stream_t stream);

/*
 * Split count for pkvqk_paged_prefill from host-side facts only: batch, kv
 * heads, q_len, group (Hq/Hkv), the longest sequence (keys, counting the new
 * tokens) and the SM count (0 = the current device's).  Returns 1..256: 1
 * when the row tiles alone fill the GPU, else enough splits of >= 256 keys
 * to give about one CTA per SM.
 */
PKVQK_API int32_t pkvqk_choose_prefill_splits(int32_t batch, int32_t num_kv_heads,
                                    int32_t q_len, int32_t group,
                                    int32_t max_seq_len, int32_t sm_count);

/*
 * Workspace bytes of pkvqk_paged_prefill: 0 for num_splits == 1, else
 * batch*q_len*Hq*num_splits*(head_dim + 1)*4 rounded up to 256: fp32 partial
 * outputs [rows][num_splits][head_dim] then fp32 partial lse
 * [rows][num_splits], rows = (b*q_len + t)*Hq + h (the layout
 * pkvqk_lse_combine reads).  Nothing in it needs to start at zero.
 */
PKVQK_API size_t pkvqk_prefill_workspace_bytes(int32_t batch, int32_t q_len,
                                     int32_t num_q_heads, int32_t head_dim,
                                     int32_t num_splits);

/*
 * Causal multi-query paged attention on the tensor cores: a chunked-prefill
 * step (q_len new tokens per sequence, appended to the cache beforehand,
 * attend to their prior context and causally to each other) or, with small
 * q_len, a speculative-verify step.  Source: InfiniLM PR #585, "概述 /
 * Summary" item 4 (chunked prefill; fixed b x (k+1) verify shape) and item 1
 * (paged cache read through the block table).
 *
 * Same definition as pkvqk_paged_decode: query token t of sequence b sees the
 * keys n < seq_lens[b] - q_len + t + 1; q head h reads kv head h / (Hq/Hkv);
 * scale <= 0 selects head_dim^-1/2; a row with no visible key outputs 0 and
 * lse = -inf.  The rows (t, h) of one kv head are packed t*group + h%group
 * into tiles of 128, so one CTA's tile covers 128/group tokens.
 *
 * num_splits >= 1: split j covers pages [j*C, (j+1)*C) of every sequence,
 * C = ceil(ceil(max_seq_len_hint / block_size) / num_splits), the last split
 * also everything past (S-1)*C pages.  With num_splits > 1 the normalised
 * partials go to the workspace and this call then launches the log-sum-exp
 * combine (pkvqk_lse_combine) on the same stream.
 *
 *   q, out, lse_out, block_tables, seq_lens: as pkvqk_paged_decode
 *   num_splits    1..256 (pkvqk_choose_prefill_splits gives a choice)
 *   max_seq_len_hint  host int >= the longest seq_len (0 = max_blocks_per_seq*block_size)
 *   workspace     device, >= pkvqk_prefill_workspace_bytes(...) (NULL if 0)
 * Supported: head_dim 128, Hq % Hkv == 0, 1 <= q_len <= 16384,
 * q_len*Hq/Hkv <= 65536.  One CTA per SM (197 KiB of shared memory and 512
 * tensor-memory columns each).
 */
PKVQK_API pkvqk_status pkvqk_paged_prefill(
    const void* q, int64_t q_stride_t, int64_t q_stride_h,
    const void* k_cache, const void* v_cache, const pkvqk_cache_layout* layout,
    const int32_t* block_tables, int32_t max_blocks_per_seq,
    const int32_t* seq_lens,
    int32_t batch, int32_t q_len, int32_t num_q_heads,
    int32_t num_splits, int32_t max_seq_len_hint, float scale,
    void* out, float* lse_out,
    void* workspace, size_t workspace_bytes,
    int32_t* status_flags, pkvqk_stream_t stream);

/*
 * Varlen form of pkvqk_paged_prefill: every sequence brings its own number of
 * new tokens, packed back to back (the FlashAttention-2 varlen convention the
 * pages use for prefill, Summary item 1).  Source: InfiniLM PR #585, "概述 /
 * Summary" items 1 (varlen prefill, paged cache) and 4 (chunked prefill).
 *
 * Sequence b's q_len_b = cu_seqlens_q[b+1] - cu_seqlens_q[b] new tokens are
 * rows cu_seqlens_q[b] .. cu_seqlens_q[b+1]-1 of q, out and lse_out; token t
 * of it sees the keys n < seq_lens[b] - q_len_b + t + 1 (seq_lens counting the
 * new tokens).  A fresh prompt has seq_lens[b] == q_len_b; a later chunk of a
 * prompt, or a verify step, has more keys than new tokens.
 *
 *   q              device bf16, row i at q[i*q_stride_t + h*q_stride_h + d]
 *   cu_seqlens_q   device int32 [batch + 1], non-decreasing, cu_seqlens_q[0] = 0
 *   max_q_len      host int >= every q_len_b (1..16384): sizes the grid (no
 *                  device read); tokens past it are not computed
 *   total_q        host: rows of q / out / lse_out (= cu_seqlens_q[batch]);
 *                  rows at or past it are never written
 *   out            device bf16 [total_q, Hq, head_dim], contiguous
 *   lse_out        device fp32 [total_q, Hq] or NULL
 *   workspace      num_splits > 1: >= pkvqk_prefill_workspace_bytes(1, total_q,
 *                  Hq, head_dim, num_splits)
 * Everything else as pkvqk_paged_prefill.
 */
PKVQK_API pkvqk_status pkvqk_paged_prefill_varlen(
    const void* q, int64_t q_stride_t, int64_t q_stride_h,
    const int32_t* cu_seqlens_q, int32_t max_q_len, int64_t total_q,
    const void* k_cache, const void* v_cache, const pkvqk_cache_layout* layout,
    const int32_t* block_tables, int32_t max_blocks_per_seq,
    const int32_t* seq_lens,
    int32_t batch, int32_t num_q_heads,
    int32_t num_splits, int32_t max_seq_len_hint, float scale,
    void* out, float* lse_out,
    void* workspace, size_t workspace_bytes,
    int32_t* status_flags, pkvqk_stream_t stream);

/*
 * pkvqk_paged_prefill and pkvqk_paged_prefill_varlen under score rules
 * (pkvqk_score_rules; first_keys has one entry per row of q), with the same split choice
 * and workspace.  Each row tile (256 / group tokens, at least one) reads the keys from its
 * rows' first visible one to their last, and its splits are counted from the page of the
 * first; hint, slots that no row sees and V that is not finite as for
 * pkvqk_paged_decode_scored.
 */
PKVQK_API pkvqk_status pkvqk_paged_prefill_scored(
    const void* q, int64_t q_stride_t, int64_t q_stride_h,
    const void* k_cache, const void* v_cache, const pkvqk_cache_layout* layout,
    const int32_t* block_tables, int32_t max_blocks_per_seq,
    const int32_t* seq_lens,
    int32_t batch, int32_t q_len, int32_t num_q_heads,
    int32_t num_splits, int32_t max_seq_len_hint, float scale,
    const pkvqk_score_rules* rules,
    void* out, float* lse_out,
    void* workspace, size_t workspace_bytes,
    int32_t* status_flags, pkvqk_stream_t stream);

PKVQK_API pkvqk_status pkvqk_paged_prefill_varlen_scored(
    const void* q, int64_t q_stride_t, int64_t q_stride_h,
    const int32_t* cu_seqlens_q, int32_t max_q_len, int64_t total_q,
    const void* k_cache, const void* v_cache, const pkvqk_cache_layout* layout,
    const int32_t* block_tables, int32_t max_blocks_per_seq,
    const int32_t* seq_lens,
    int32_t batch, int32_t num_q_heads,
    int32_t num_splits, int32_t max_seq_len_hint, float scale,
    const pkvqk_score_rules* rules,
    void* out, float* lse_out,
    void* workspace, size_t workspace_bytes,
    int32_t* status_flags, pkvqk_stream_t stream);

/*
 * pkvqk_paged_prefill and pkvqk_paged_prefill_varlen over an 8-bit cache: the same
 * definition with K_n and V_n = code * scale, the same split choice and
 * workspace; exactness, slots past the sequence's end and NaN codes as for
 * pkvqk_paged_decode_q8.
 */
PKVQK_API pkvqk_status pkvqk_paged_prefill_q8(
    const void* q, int64_t q_stride_t, int64_t q_stride_h,
    const pkvqk_q8_cache* cache,
    const int32_t* block_tables, int32_t max_blocks_per_seq,
    const int32_t* seq_lens,
    int32_t batch, int32_t q_len, int32_t num_q_heads,
    int32_t num_splits, int32_t max_seq_len_hint, float scale,
    void* out, float* lse_out,
    void* workspace, size_t workspace_bytes,
    int32_t* status_flags, pkvqk_stream_t stream);

PKVQK_API pkvqk_status pkvqk_paged_prefill_varlen_q8(
    const void* q, int64_t q_stride_t, int64_t q_stride_h,
    const int32_t* cu_seqlens_q, int32_t max_q_len, int64_t total_q,
    const pkvqk_q8_cache* cache,
    const int32_t* block_tables, int32_t max_blocks_per_seq,
    const int32_t* seq_lens,
    int32_t batch, int32_t num_q_heads,
    int32_t num_splits, int32_t max_seq_len_hint, float scale,
    void* out, float* lse_out,
    void* workspace, size_t workspace_bytes,
    int32_t* status_flags, pkvqk_stream_t stream);

#ifdef __cplusplus
}  /* extern "C" */
#endif

#endif /* PKVQK_H */
