/*
 * kvq.h -- C ABI of the GB300 (sm_103a) library for attention decode over a
 * quantized KV cache.
 *
 * What it computes (sources are the web pages the library follows):
 *  - Quantize-on-append of new K/V rows into the cache, as FP8 E4M3 with a
 *    static per-tensor scale (compressed-tensors PR 436, kv_cache_scheme:
 *    8-bit float, symmetric, strategy "tensor", dynamic false, minmax
 *    observer) or as NVFP4: E2M1 values in blocks of 16 along head_dim with a
 *    dynamic E4M3 block scale and an fp32 global scale (Model-Optimizer PR
 *    714, Testing: quantizers "(2, 1) bit ... block_sizes={-1: 16, 'type':
 *    'dynamic', 'scale_bits': (4, 3)}" with a calibrated amax).
 *  - Split-KV flash decode (Model-Optimizer PR 1832, notes under the latency
 *    tables): each (request, kv head) sequence is cut into s contiguous
 *    chunks; kvq_decode_partial runs one partial softmax (running max,
 *    denominator, weighted V) per chunk and kvq_decode_combine merges the s
 *    partials.  kvq_auto_splits picks s from the SM count and batch x heads.
 *  - Options: GQA/MHA head groups, paged blocks, FP8-quantized softmax
 *    probabilities with a prob scale and FP8 output with an out scale (vLLM
 *    PR 15734), and the MLA latent-cache variant (Model-Optimizer PR 714:
 *    kv_c_bmm_quantizer on the 512-wide latent cache, q_bmm_quantizer off).
 *
 * Conventions (all calls):
 *  - Every device buffer (cache, queries, outputs, workspace) is allocated
 *    and owned by the caller.  The library allocates no memory and keeps no
 *    per-call state; calls are re-entrant.  (It caches, per device, values
 *    that do not change: the number of MLA CTA clusters that fit at once.)
 *  - Pointers marked (device) must be device (or managed) memory of the
 *    current CUDA device; pointers marked (host) are read on the host.  The
 *    per-step inputs read with plain loads -- q, k_new, v_new, kpe_new --
 *    and the decode output may also be pinned host memory (page-locked and
 *    mapped, as cudaHostAlloc gives): the kernels then read and write it in
 *    place over the CPU-GPU link.  The cache, block table, seq_lens and the
 *    scratch must be device memory (the cache is read by TMA).
 *  - Calls are asynchronous on `stream` (a cudaStream_t passed as void*;
 *    NULL = the legacy default stream).  No call synchronizes.
 *  - Every call validates its arguments first and returns KVQ_ERR_INVALID or
 *    KVQ_ERR_UNSUPPORTED without launching anything.  After launching it
 *    returns KVQ_ERR_CUDA if the launch reported an error.
 *  - bf16 tensors are raw IEEE bfloat16 bit patterns (uint16).
 */
#ifndef KVQ_H
#define KVQ_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef int kvq_status;
#define KVQ_OK 0
#define KVQ_ERR_INVALID 1      /* bad pointer, size, scale or layout */
#define KVQ_ERR_UNSUPPORTED 2  /* valid but not implemented (dims, format) */
#define KVQ_ERR_WORKSPACE 3    /* a workspace or scratch area is too small */
#define KVQ_ERR_CUDA 4         /* the CUDA runtime reported an error */

/* Cache formats */
#define KVQ_FP8_E4M3 1
#define KVQ_NVFP4 2

/* Output types of kvq_decode_combine */
#define KVQ_OUT_F32 0
#define KVQ_OUT_BF16 1
#define KVQ_OUT_E4M3 2

/* Bits that kernels OR into kvq_decode_params.error_flag */
#define KVQ_DEVERR_WAIT_TIMEOUT 1   /* a pipeline wait gave up (results invalid) */
#define KVQ_DEVERR_SEQ_CLAMPED 2    /* seq_lens[b] exceeded the cache; clamped */
#define KVQ_DEVERR_BAD_PAGE 4       /* a block-table entry was out of range; page 0 read
                                       (kvq_rope_append: the token's rows are not written) */
#define KVQ_DEVERR_BAD_POSITION 8   /* a position past the rotation table; its rows are
                                       not written */
#define KVQ_DEVERR_REFUSED 16       /* kvq_plan_step: a request was not served */
#define KVQ_DEVERR_BAD_POOL 32      /* kvq_plan_step: the free pages' count is out of range */

/*
 * A paged quantized KV cache.  Caller-owned plain struct; the library only
 * reads it.
 *
 * Layout of one cache tensor (K or V), page-major then head-major, so one
 * (page, kv head) is a contiguous run of page_size rows:
 *   FP8:    codes  uint8 [num_pages][num_kv_heads][page_size][head_dim]
 *   NVFP4:  codes  uint8 [num_pages][num_kv_heads][page_size][head_dim/2]
 *                  (element 2i in the low nibble, 2i+1 in the high nibble)
 *           bscale uint8 [num_pages][num_kv_heads][page_size][head_dim/16]
 *                  (E4M3 block scales, one per 16 consecutive elements)
 * Token t of request b lives in page block_table[b*max_pages_per_seq + t /
 * page_size], row t % page_size.  A contiguous cache is the special case of
 * one page per request (page_size = capacity, block_table[b][0] = b).
 *
 * Dequantized values: FP8 x = dec(code) * scale; NVFP4 x = dec(e2m1) *
 * dec(bscale) * scale, where scale is k_scale or v_scale.
 *
 * MLA latent cache (rope_dim > 0): k_codes/k_bscale hold the NVFP4 latent
 * kv_c (num_kv_heads = 1, head_dim = 512), k_pe holds the bf16 rope keys
 * [num_pages][page_size][rope_dim], v_codes is NULL and v_is_k_latent = 1
 * (the values are the latent itself).
 */
typedef struct kvq_cache {
  int32_t fmt;               /* KVQ_FP8_E4M3 or KVQ_NVFP4 */
  int32_t num_pages;         /* >= 1 */
  int32_t page_size;         /* tokens per page, a multiple of 16 */
  int32_t num_kv_heads;      /* Hkv >= 1 */
  int32_t head_dim;          /* D: FP8 64 or 128; NVFP4 64, 128 or 256 (MLA 512) */
  void* k_codes;             /* (device) 16-byte aligned */
  void* v_codes;             /* (device) 16-byte aligned; NULL for MLA */
  void* k_bscale;            /* (device) NVFP4 only, 16-byte aligned */
  void* v_bscale;            /* (device) NVFP4 only, 16-byte aligned */
  float k_scale;             /* FP8 scale or NVFP4 global scale, finite > 0 */
  float v_scale;             /* as k_scale (ignored for MLA) */
                             /* (both ignored where per-head scales are given) */
  const int32_t* block_table;/* (device) [batch][max_pages_per_seq] */
  int32_t max_pages_per_seq; /* >= 1 */
  int32_t rope_dim;          /* MLA: 64; otherwise 0 */
  void* k_pe;                /* (device) MLA only: bf16 rope keys */
  int32_t v_is_k_latent;     /* MLA: 1; otherwise 0 */
  /*
   * Per-kv-head scales (compressed-tensors PR 436, "attn_head" strategy: one
   * static scale per attention head).  Optional, (device) float
   * [num_kv_heads] each: when non-NULL, kv head h of K (V) uses
   * k_head_scale[h] (v_head_scale[h]) wherever k_scale (v_scale) appears
   * above -- the FP8 scale or the NVFP4 global scale -- in the append and in
   * the decode, and k_scale (v_scale) is ignored.  Every entry must be
   * finite and > 0 (not checked: device memory).  They are read like the
   * block table, so nothing still running may write them (fresh_tokens).
   * Not for MLA (one latent kv head: use k_scale).
   */
  const float* k_head_scale;
  const float* v_head_scale;
} kvq_cache;

/* Parameters of one decode step (shared by partial and combine). */
typedef struct kvq_decode_params {
  int32_t batch;             /* B >= 0 (0 is a no-op) */
  int32_t num_q_heads;       /* Hq, a multiple of Hkv; Hq/Hkv <= 16 */
  int32_t qk_dim;            /* head_dim (MLA: 512 + 64 = 576) */
  int32_t v_dim;             /* head_dim (MLA: 512) */
  int32_t num_splits;        /* 1 <= s <= 64 (see kvq_auto_splits) */
  const int32_t* seq_lens;   /* (device) [batch] tokens per request */
  int32_t max_kv_len;        /* (host) upper bound of seq_lens[] */
  float sm_scale;            /* softmax scale (e.g. 1/sqrt(head_dim)) */
  float prob_scale;          /* > 0: FP8 softmax probabilities; 0: off */
  int32_t out_dtype;         /* KVQ_OUT_* (used by combine) */
  float out_scale;           /* KVQ_OUT_E4M3: output scale, finite > 0 */
  int32_t* error_flag;       /* (device, optional) KVQ_DEVERR_* bits OR-ed in */
  /*
   * Overlap with the append of this step (>= 0).  0: the decode waits for
   * the preceding kernel in the stream to finish before it reads any input
   * (always correct).  n > 0 declares that the work issued immediately
   * before on the same stream is one kvq_quantize_append call that wrote
   * only positions seq_lens[b] - n .. seq_lens[b] - 1 of each request, and
   * that q, seq_lens, the block table and every other cache position were
   * complete when that call was made (kvq_quantize_append starts after all
   * earlier work in the stream).  The decode then streams every other part
   * of the cache while the append runs and waits for it only before the
   * boxes that hold those positions.  q, seq_lens and the block table are
   * read before that wait, so the append (or anything else still running
   * when the decode starts) must not write them.  Not part of the pages'
   * method: a scheduling contract between two calls of this library.
   */
  int32_t fresh_tokens;
  /*
   * FP8 query (compressed-tensors PR 436: a query observer next to the K
   * and V ones, GSM8K rows "QKV-FP8-Tensor" / "QKV-FP8-Head"; vLLM PR 15734:
   * QK quantization in the attention loop).  q_fp8 = 0: q is bf16 (default).
   * q_fp8 = 1: q holds E4M3 codes [batch][Hq][qk_dim] (kvq_quantize_fp8
   * makes them) whose values are dec(code) * q_scale, or * q_head_scale[hq]
   * when that (device, [num_q_heads]) array is given.  With an FP8 cache the
   * scores run on E4M3 x E4M3 tensor-core MMAs straight from the cached
   * codes; with an NVFP4 cache the codes are widened exactly to f16.  Not
   * for MLA.
   */
  int32_t q_fp8;
  float q_scale;             /* q_fp8 without q_head_scale: finite > 0 */
  const float* q_head_scale; /* (device, optional) [num_q_heads] */
  /*
   * kvq_decode_shared and kvq_chunk_attention only (the other calls ignore it).
   * 0: the probabilities of the prefix (the chunks) enter the products with V in
   * two f16 parts, as kvq_decode's do.  1: in one, rounded by up to 2^-11 of a
   * weight where kvq_decode keeps 2^-22; a bf16 output, whose own rounding is 2^-8,
   * then differs here and there by one step, and the products with V take half the
   * tensor-core time.  Differential heads have two parts either way.
   */
  int32_t prefix_p_f16;
} kvq_decode_params;

/* Human-readable name of a status code (static string). */
const char* kvq_status_string(kvq_status s);

/*
 * Static per-tensor scale from a calibrated amax (the minmax observer of
 * compressed-tensors PR 436; the MaxCalibrator amax of Model-Optimizer PR
 * 714).  Host only.
 *   KVQ_FP8_E4M3: scale = fl32(amax / 448)   (448 = largest E4M3 value)
 *   KVQ_NVFP4:    scale = fl32(amax / 2688)  (2688 = 6 * 448: largest E2M1
 *                 value times largest E4M3 block scale)
 * amax == 0 gives 1.0.  Negative, NaN or infinite amax -> KVQ_ERR_INVALID.
 */
kvq_status kvq_tensor_scale(int fmt, float amax, float* scale_out /* host */);

/*
 * amax = max |x| over n bf16 values, written to *amax_out (device float).
 * The calibration step that feeds kvq_tensor_scale.  n may be 0 (gives 0).
 */
kvq_status kvq_amax_bf16(const void* x /* device bf16 [n] */, size_t n,
                         float* amax_out /* device */, void* stream);

/*
 * Quantize-on-append.  Writes n_tokens new rows per request into the cache:
 * row t of request b goes to position start_pos[b] + t.
 *   k_new   (device) bf16 [batch][n_tokens][num_kv_heads][head_dim]
 *   v_new   (device) bf16, same shape (NULL for MLA)
 *   kpe_new (device) bf16 [batch][n_tokens][rope_dim] (MLA only, else NULL)
 *   start_pos (device) int32 [batch]
 * FP8:   code = E4M3(fl32(x / scale)), round to nearest even, saturating at
 *        +-448 (the sign of zero is kept).
 * NVFP4, per 16-element block along head_dim:
 *        bamax = max |x|;  sc = E4M3(fl32(fl32(bamax / 6) / scale));
 *        es = fl32(dec(sc) * scale);  code = E2M1(fl32(x / es)) (all 0 when
 *        es == 0), round to nearest even, saturating at +-6.
 * The caller guarantees that the pages for positions start_pos[b] ..
 * start_pos[b] + n_tokens - 1 exist in the block table; positions past
 * max_pages_per_seq * page_size are skipped (not written).
 * Input pointers must be 16-byte aligned.  batch <= 32767, num_kv_heads <=
 * 65535 and n_tokens < 2^30 (else KVQ_ERR_UNSUPPORTED).
 */
kvq_status kvq_quantize_append(const kvq_cache* c, const void* k_new, const void* v_new,
                               const void* kpe_new, const int32_t* start_pos, int batch,
                               int n_tokens, void* stream);

/*
 * Norm and rotation of queries and keys.  Which the model applies, and with
 * what, is the same for every call of a layer:
 *   norm:     n_i = (x_i r) w_i,  r = 1 / sqrt(sum_j x_j^2 / head_dim + eps)
 *             over each head, where weights are given (q_norm for queries,
 *             k_norm for keys; each may be NULL on its own);
 *   rotation: of the head's first rot_dim elements, by the angles of the
 *             token's position, (a, b) -> (a cos - b sin, b cos + a sin) over
 *             the pairs (i, i + rot_dim/2) (interleaved = 0) or (2i, 2i + 1)
 *             (interleaved = 1), i < rot_dim/2; the rest passes unrotated.
 * All of it runs in fp32 on the bf16 input; a result is rounded once, to its
 * output type.  E4M3 codes whose fp32 quotient lies within 16 steps of a
 * rounding boundary are decided with some 48 bits, 43 where a norm is given (values that neither norm nor
 * rotation changes keep kvq_quantize_fp8's quotient).  A row's sum of squares
 * has to stay in the range of fp32.
 */
typedef struct kvq_rotary {
  const float* cos_sin;      /* (device) [num_positions][rot_dim]: the rot_dim/2
                                cosines of a position, then its sines; 16-byte
                                aligned (ignored where rot_dim is 0) */
  int32_t num_positions;     /* rows of the table */
  int32_t rot_dim;           /* 0 (no rotation) or a multiple of 32, <= head_dim */
  int32_t interleaved;       /* 0 or 1 */
  const float* q_norm;       /* (device, optional) [head_dim], 16-byte aligned */
  const float* k_norm;       /* (device, optional) [head_dim]; MLA: [512], the latent's */
  float eps;                 /* finite >= 0 (read where a norm is given) */
} kvq_rotary;

/*
 * Rows of heads, such as a slice of a packed projection: head h of token t is
 * the head_dim elements at data + t * token_stride + h * head_stride.  Strides
 * count elements (bytes where the rows hold codes), are multiples of 8 in [0,
 * 2^31) and data is 16-byte aligned.  Rows that a call writes may not overlap
 * one another.
 */
typedef struct kvq_heads {
  void* data;                /* (device, or pinned host memory like the inputs above) */
  int64_t token_stride;
  int64_t head_stride;
  int32_t num_heads;         /* >= 1 */
} kvq_heads;

/*
 * Norm and rotation of queries q and keys k (either may be NULL) in one pass:
 * token t of num_tokens is at positions[t] (device int32; may be NULL without
 * a rotation).
 *   q, k   bf16 rows;  head_dim 64, 128 or 256.
 *   q_out  bf16 rows, or with q_fp8 = 1 E4M3 codes for an FP8-query decode:
 *          E4M3(y / s), s = q_head_scale[h] (device) where given, else q_scale
 *          (finite > 0), rounded and saturating as kvq_quantize_fp8's.
 *   k_out  bf16 rows.
 * bf16 outputs may be the inputs themselves (same data and strides); otherwise
 * no output may overlap an input.  Tokens at negative positions are skipped
 * (their output rows stay as they were: the padding of a batch), and so are
 * tokens at positions past the table, which set KVQ_DEVERR_BAD_POSITION.
 * num_tokens times the number of heads < 2^31 (else KVQ_ERR_UNSUPPORTED).
 */
kvq_status kvq_norm_rope(const kvq_rotary* r, int head_dim, int num_tokens,
                         const int32_t* positions, const kvq_heads* q, const kvq_heads* q_out,
                         int q_fp8, float q_scale, const float* q_head_scale, const kvq_heads* k,
                         const kvq_heads* k_out, int32_t* error_flag, void* stream);

/*
 * kvq_quantize_append of keys that are normed and rotated on the way, and, in
 * the same launch, the norm and rotation of the step's queries.
 *   Token (b, t), t < n_tokens, of the padded batch is row b * n_tokens + t of
 *   k, v, kpe, q and q_out, and goes to position start_pos[b] + t, which also
 *   gives its angles.
 *   new_lens (device int32 [batch], optional): only the first new_lens[b]
 *   tokens of request b are real (all for n_tokens or more, none for 0 or
 *   less); the rest are neither read nor written, and their cache rows and
 *   q_out rows stay as they were.  Two real tokens may not share a cache row.
 *   k, v   bf16 rows of num_kv_heads heads;  head_dim 64, 128 or 256.
 *   q, q_out, q_fp8, q_scale, q_head_scale (q may be NULL): as in
 *          kvq_norm_rope.  A decode that reads q_out must not use
 *          fresh_tokens (q is not complete before this call); without q the
 *          call takes kvq_quantize_append's place in that contract.
 *   MLA cache (head_dim 512, rope_dim 64): k holds the latents (normed with
 *          k_norm where given, not rotated), kpe the rope keys (rotated, bf16);
 *          v and q are NULL, and rot_dim is at most 64.
 * The quantisers are kvq_quantize_append's on the fp32 values (V: the same
 * codes).  error_flag (device, optional) gets KVQ_DEVERR_BAD_POSITION for a
 * position past the rotation table and KVQ_DEVERR_BAD_PAGE for a page index
 * out of range.  A token at a negative position or past the rotation table is
 * skipped altogether; one whose page index is out of range, or that lies past
 * the block table (as in the plain append), gets no cache row, but its q_out
 * row is written.
 */
kvq_status kvq_rope_append(const kvq_cache* c, const kvq_rotary* r, int batch, int n_tokens,
                           const int32_t* start_pos, const int32_t* new_lens, const kvq_heads* k,
                           const kvq_heads* v, const kvq_heads* kpe, const kvq_heads* q,
                           const kvq_heads* q_out, int q_fp8, float q_scale,
                           const float* q_head_scale, int32_t* error_flag, void* stream);

/*
 * A step's paging on the GPU: what the appends, kvq_chunk_attention and the
 * decodes take -- block table, lengths, start positions, packed offsets, slots and
 * positions of the new tokens -- from the requests' lengths and their changes.
 *
 * Request b holds seq_lens[b] tokens in the first ceil(length / page_size) pages of
 * its block-table row.  add_lens[b] > 0 adds that many tokens; below zero takes the
 * last ones off again (all of them where there are fewer), so INT32_MIN ends a
 * request; 0 leaves it.  The free pages are a stack, free_pages[0 .. *free_count - 1]:
 *  - first the pages that are no longer needed go on it, in the order of the
 *    requests and, within one, of its block-table entries (those entries stay);
 *  - then the requests that grow take theirs from its top in the same order, each
 *    page into the next entry of the request's row.  A request is served whole or not
 *    at all: where the pages are not all there, it and every later request that needs
 *    a page get none; nor does one that would pass its block-table row, or whose
 *    tokens would pass max_tokens.  Such a request keeps its length and sets
 *    KVQ_DEVERR_REFUSED.
 * Lengths outside [0, max_pages_per_seq page_size] are clamped (KVQ_DEVERR_SEQ_CLAMPED),
 * a count outside [0, num_pages] too, and pages that come back beyond num_pages of them are
 * dropped (both KVQ_DEVERR_BAD_POOL).  A page whose index is out of range sets
 * KVQ_DEVERR_BAD_PAGE when it comes back and when it is taken, and is a page like any other
 * otherwise: it goes on the stack, and the request that takes it is served, but its tokens
 * there have no slots.  After that bit the tables and the free pages have to be made anew.
 *
 * Outputs (the last four may be NULL):
 *   seq_lens_out   [batch] the new lengths (may be seq_lens)
 *   free_count_out [1] the new count (may be free_count); free_pages at and above it
 *                  holds what was popped
 *   start_pos      [batch] the lengths before: where the new tokens go
 *   q_offsets      [batch + 1] request b's new tokens are rows q_offsets[b] ..
 *                  q_offsets[b + 1] - 1 of the packed step, whether it is served or
 *                  not; at most max_tokens
 *   slots          [max_tokens] of each new token, page * page_size + row; -1 for the
 *                  tokens of refused requests and rows past the last token, and (with
 *                  KVQ_DEVERR_BAD_PAGE) where the page is out of range
 *   positions      [max_tokens] of each new token; -1 as above, except for bad pages
 * counter is one word that is zero before the first call and left so.  No other two
 * of these arrays may overlap.  All of it runs on the GPU, in one launch: a captured
 * step replays with lengths that change.  batch <= 8192, max_tokens and num_pages <= 2^30
 * (else KVQ_ERR_UNSUPPORTED).
 * Calls that share the free pages or the counter must not overlap on the GPU.
 */
typedef struct kvq_page_plan {
  int32_t batch;             /* >= 0 (0: nothing is written but the rows past the last token,
                                the first offset and the count) */
  int32_t page_size;         /* >= 1 */
  int32_t num_pages;         /* >= 1, of the cache and of free_pages */
  int32_t max_pages_per_seq; /* >= 1, with page_size below 2^31 tokens */
  int32_t max_tokens;        /* >= 0, rows of the packed step */
  int32_t* block_table;      /* (device) [batch][max_pages_per_seq], updated */
  const int32_t* seq_lens;   /* (device) [batch] */
  int32_t* seq_lens_out;     /* (device) [batch] */
  const int32_t* add_lens;   /* (device) [batch] */
  int32_t* free_pages;       /* (device) [num_pages], updated */
  const int32_t* free_count; /* (device) [1] */
  int32_t* free_count_out;   /* (device) [1] */
  uint32_t* counter;         /* (device) [1] */
  int32_t* start_pos;        /* (device, optional) */
  int32_t* q_offsets;        /* (device, optional) */
  int64_t* slots;            /* (device, optional) */
  int32_t* positions;        /* (device, optional) */
  int32_t* error_flag;       /* (device, optional) KVQ_DEVERR_* bits OR-ed in */
} kvq_page_plan;

kvq_status kvq_plan_step(const kvq_page_plan* p, void* stream);

/*
 * kvq_rope_append for a packed step: row t of k, v, kpe, q and q_out is a token of
 * some request, at positions[t] (device int32; NULL where nothing is rotated), and its
 * cache row is slots[t] (device int64): row slots[t] % page_size of page slots[t] /
 * page_size.  The block table is not read.  Tokens at negative positions are skipped,
 * as are those past the rotation table (KVQ_DEVERR_BAD_POSITION); a token with a
 * negative slot, or with one past the cache (KVQ_DEVERR_BAD_PAGE), gets no cache row,
 * but its q_out row is written.  No two tokens may share a slot.  All else is
 * kvq_rope_append's, the codes too.
 */
kvq_status kvq_rope_append_slots(const kvq_cache* c, const kvq_rotary* r, int num_tokens,
                                 const int32_t* positions, const int64_t* slots,
                                 const kvq_heads* k, const kvq_heads* v, const kvq_heads* kpe,
                                 const kvq_heads* q, const kvq_heads* q_out, int q_fp8,
                                 float q_scale, const float* q_head_scale, int32_t* error_flag,
                                 void* stream);

/*
 * Split-count heuristic (host only, deterministic).  base = batch *
 * num_kv_heads (MLA: batch) CTAs per split; the partial kernel keeps
 * ctas_per_sm CTAs resident per SM (2: six-warp CTAs, or four-warp CTAs
 * with more than 8 query heads per kv head; 1 for the MLA shape:
 * KVQ_NVFP4, num_kv_heads 1, q_per_kv 16), so
 * s = floor(ctas_per_sm * num_sms / base) splits fill one wave; when that
 * is 0 (more groups than one wave holds), s = ceil(max_kv_len / 2048), so
 * that long or ragged requests are cut into chunks that balance across the
 * waves.  Above 32 splits with
 * chunks under 256 tokens (max_kv_len < 256 s), s becomes
 * max(32, ceil(max_kv_len / 256)).  s is then lowered so that every chunk
 * keeps at least 128 tokens and clamped to [1, 64].  num_sms is
 * the device's multiprocessor count (cudaDevAttrMultiProcessorCount).
 */
kvq_status kvq_auto_splits(int num_sms, int batch, int num_kv_heads, int q_per_kv,
                           int max_kv_len, int fmt, int* out_s /* host */);

/* Bytes of the split partials: part_o (fp32 [batch][Hq][s][v_dim]) plus
 * part_lse (fp32 [batch][Hq][s]). */
size_t kvq_partial_workspace_bytes(int batch, int num_q_heads, int num_splits, int v_dim);

/*
 * Split-KV partial.  For request b, query head hq (kv head hq / (Hq/Hkv))
 * and split j, over chunk j of the request's sequence (chunk length c =
 * ceil(L/s) rounded up to 16 tokens; chunk j = [j*c, min((j+1)*c, L))):
 *   S_i = sm_scale * q . k^_i;   m = max_i S_i;   l = sum_i exp(S_i - m)
 *   part_o[b][hq][j][:] = sum_i exp(S_i - m) v^_i / l
 *   part_lse[b][hq][j]  = m + ln l          (-inf and o = 0 for empty chunks)
 * With prob_scale > 0 (FP8 probabilities) the weight of v^_i is
 *   p_q = dec(E4M3(fl32(p~ / prob_scale))) * prob_scale, p~ = exp(S_i - m)
 * in fp32 with m the chunk max, while l sums the unquantized p~.
 *   q (device) bf16 [batch][Hq][qk_dim], 16-byte aligned.
 *   part_o, part_lse (device) as in kvq_partial_workspace_bytes; part_o
 *   16-byte aligned.
 * With prob_scale > 0 one chunk's scores must fit in on-chip memory:
 * ceil(max_kv_len / s) rounded up to 16, times Hq/Hkv, at most 16384;
 * larger chunks return KVQ_ERR_UNSUPPORTED (raise num_splits).
 * Otherwise the weights enter the products with v^ in two f16 parts: each off
 * by at most 2^-22 of itself, or by 2^-25 of the chunk's largest where that is
 * more.  A chunk's products add up in the matrix units' fp32 accumulators, which
 * cut off towards zero: where all values have one sign, 100000 tokens in one
 * chunk lose 9e-5 of their sum, in eight chunks 7e-6.
 */
kvq_status kvq_decode_partial(const kvq_cache* c, const kvq_decode_params* p, const void* q,
                              float* part_o, float* part_lse, void* stream);

/*
 * Combine of the s partials of kvq_decode_partial:
 *   M = max_j lse_j;  w_j = exp(lse_j - M);  O = sum_j w_j o_j / sum_j w_j
 * (partials with lse = -inf are skipped; O = 0 when all are empty), written
 * to out (device) [batch][Hq][v_dim] as fp32, bf16 (round to nearest even)
 * or E4M3 codes E4M3(fl32(O / out_scale)) per p->out_dtype.
 */
kvq_status kvq_decode_combine(const kvq_decode_params* p, const float* part_o,
                              const float* part_lse, void* out, void* stream);

/*
 * One decode step in a single launch: kvq_decode_partial followed by the
 * merge of kvq_decode_combine, which the last CTA to finish for each
 * (request, kv head) performs with the same arithmetic and output types.
 * MLA with 2..8 splits runs as thread-block clusters of a request's splits
 * when they fit the device in as many waves as single CTAs: the partials
 * then merge through distributed shared memory (part_o and part_lse are not
 * written, the counters not used), with the same results bit for bit.
 *   part_o, part_lse (device) split partials, as for kvq_decode_partial.
 *   counters (device) uint32 [batch * num_kv_heads] arrival counters.  They
 *   must be zero before the first call; every call leaves them at zero
 *   again, so one zero-filled array (sized for the largest batch *
 *   num_kv_heads) serves any number of later calls.  Calls that share
 *   counters or partials must not overlap on the GPU (stream-order them).
 *   out (device) [batch][Hq][v_dim] in p->out_dtype.
 */
kvq_status kvq_decode(const kvq_cache* c, const kvq_decode_params* p, const void* q,
                      float* part_o, float* part_lse, uint32_t* counters, void* out,
                      void* stream);

/*
 * kvq_decode for a batch whose requests share their first prefix_len tokens,
 * in the same pages (a system prompt, a document, the common past of sampled
 * answers): the shared tokens are read once for all requests, and their
 * scores and values are products of all query rows of a kv head, on the
 * tensor cores.  The result is kvq_decode's.
 *   c, p       as for kvq_decode, with each request's whole block table and
 *              length: tokens prefix_len .. seq_lens[b] - 1 are its own.  A
 *              request shorter than prefix_len (0 for a padded row) takes no
 *              part in the sharing and reads its own table only.
 *   prefix_len (host) a multiple of page_size, at most p->max_kv_len and
 *              2^31 - 4097; 0 is kvq_decode.
 *   prefix_table (device int32, optional) [prefix_len / page_size] the shared
 *              pages; NULL: the first entries of the block table's row of the
 *              first request that is at least prefix_len long.
 *   prefix_splits, p->num_splits: chunks of the prefix (at least one 128-token
 *              tile each: more are lowered) and of each request's own tokens;
 *              kvq_shared_splits picks both.  Together at most 64.
 *   part_o, part_lse, counters (device): as for kvq_decode, sized for
 *              p->num_splits + prefix_splits splits; part_o 32-byte aligned.
 * FP8 and NVFP4 caches with head_dim 64 or 128, bf16 or FP8 queries, per-head
 * scales; not MLA, and prob_scale must be 0 (KVQ_ERR_UNSUPPORTED).  It pays
 * from a few requests on: the prefix takes at least one pass of the tensor
 * cores over 128 rows, and kvq_decode reads a prefix that only one or two
 * requests share (or that is shorter than what each adds) in less time.
 * fresh_tokens is taken as 0 where prefix_len is positive.  The prefix's
 * probabilities enter the products with V in two f16 parts, as kvq_decode's do, or
 * in one where p->prefix_p_f16 asks for that: each off by at most 2^-22 (2^-11) of
 * itself, or by 2^-32 of the row's largest one where that is more, so that a token
 * below 2^-32 of the largest counts in the sum alone.  A split's products add up in
 * the matrix units' fp32 accumulators, which cut off towards zero: where all values
 * have one sign, a prefix of 131072 tokens loses 4e-4 of its sum in one split, 2.2e-5
 * in twelve.
 * Two or three launches on `stream` (three where not all own chunks fit on the
 * SMs beside the prefix); calls that share partials or counters must not
 * overlap on the GPU.
 */
kvq_status kvq_decode_shared(const kvq_cache* c, const kvq_decode_params* p, int prefix_len,
                             const int32_t* prefix_table, int prefix_splits, const void* q,
                             float* part_o, float* part_lse, uint32_t* counters, void* out,
                             void* stream);

/*
 * Split counts for kvq_decode_shared (host only, deterministic): the pair with
 * the shortest modelled step.  The prefix's grid has num_kv_heads x row tiles x
 * prefix_splits CTAs, one per SM (a row tile is 128 of the batch * q_per_kv
 * rows of a kv head, or 256 if there are more); the requests' own chunks
 * (batch * num_kv_heads * own_splits CTAs, two per SM) run beside it on the
 * SMs that it leaves free.  own_splits is a power of two up to 16 with at
 * least 128 tokens of max_own_len, the longest own part, per chunk;
 * prefix_splits has at least one 128-token tile per chunk; together at most 64.
 * The model's times are those of an FP8 cache with head_dim 128; fmt is checked
 * and changes nothing so far.
 */
kvq_status kvq_shared_splits(int num_sms, int batch, int num_kv_heads, int q_per_kv,
                             int prefix_len, int max_own_len, int fmt,
                             int* prefix_splits /* host */, int* own_splits /* host */);

/*
 * Differential attention: the difference of two softmax maps.  A head of head_dim D
 * has two queries and two keys of D / 2 elements, side by side in its row -- q = [q1
 * q2], and in the cache k = [k1 k2] -- and values of D:
 *   S1_i = sm_scale q1 . k1_i,  S2_i = sm_scale q2 . k2_i
 *   o = sum_i softmax_i(S1) v_i - lambda[hq] sum_i softmax_i(S2) v_i
 *   out = gain o                                             (norm NULL)
 *   out = gain norm o / sqrt(sum_j o_j^2 / D + eps)          (elementwise)
 * sm_scale is usually 1/sqrt(D / 2), and gain 1 - lambda_init.  Everything before the
 * output's rounding is fp32; an o of zeros gives zeros, whatever eps.  The two sums of
 * a request without tokens are zeros.
 * Models that turn each of q1, q2, k1 and k2 over its own D / 2 elements: kvq_rotary with
 * interleaved = 1, rot_dim = D and a table that has the D / 4 cosines of a half twice, then
 * its sines twice, does so in the appends and in kvq_norm_rope.  Where the model pairs the
 * elements (i, i + D/4) of a half, one permutation of its projections' rows, the same for
 * queries and keys, makes them (2i, 2i + 1) and leaves the scores as they are.  (interleaved
 * = 0 pairs elements of the whole head, across the two maps.)  Halves of 64 or 128 may also
 * be turned as heads of their own, by kvq_norm_rope with head_dim D / 2, before an append
 * with rot_dim 0; its keys are rounded to bf16 on the way.
 */
typedef struct kvq_diff {
  const float* lambda;       /* (device) [num_q_heads] */
  const float* norm;         /* (device, optional) [head_dim], 16-byte aligned */
  float eps;                 /* finite >= 0 (read where norm is given) */
  float gain;                /* finite */
} kvq_diff;

/*
 * kvq_decode with differential heads: a single token of each request, in one launch.
 * As for kvq_decode, with these differences: q, out and num_q_heads count
 * differential heads; part_o and part_lse hold two rows for each, so they are sized
 * for 2 * num_q_heads heads; num_q_heads / num_kv_heads is at most 8 and prob_scale is
 * 0 (else KVQ_ERR_UNSUPPORTED); not MLA.  The probabilities enter the products with V in two
 * f16 parts: each off by at most 2^-22 of itself, or by 2^-32 of the row's largest one where
 * that is more.  kvq_auto_splits with twice the query heads
 * per kv head picks num_splits (15 instead of 16 with head_dim up to 128: NVFP4's 16 on
 * one kv head are taken for MLA there).  With fresh_tokens lambda and norm, too, have to be
 * complete before the append.
 */
kvq_status kvq_decode_diff(const kvq_cache* c, const kvq_decode_params* p, const kvq_diff* d,
                           const void* q, float* part_o, float* part_lse, uint32_t* counters,
                           void* out, void* stream);

/*
 * Causal attention of a packed step over the cache: prompt chunks, single tokens and
 * idle requests in any mixture.  Request b's new tokens are rows q_offsets[b] ..
 * q_offsets[b + 1] - 1 of q and out (kvq_plan_step gives the offsets), and its
 * seq_lens[b] = L tokens, the new ones among them, are in the cache: with n new ones,
 * the i-th attends to tokens 0 .. L - n + i,
 *   out[t][hq][:] = sum_j softmax_j(sm_scale q . k_j) v_j
 * in p->out_dtype, or with d (optional) the differential attention above.  Tokens
 * before position 0 (n > L) attend to nothing and give 0.  Rows of q and out past
 * the last offset are neither read nor written.  Offsets are taken within [0,
 * num_tokens] and lengths within the block table (KVQ_DEVERR_SEQ_CLAMPED); a pair of
 * offsets that falls counts as no tokens.  No two requests may share a row: offsets with
 * more of it than num_tokens rows could hold leave the chunks' rows unwritten
 * (KVQ_DEVERR_SEQ_CLAMPED).
 *   q   (device) bf16, or E4M3 codes (p->q_fp8), [num_tokens][Hq][head_dim], 16-byte
 *       aligned
 *   out (device) [num_tokens][Hq][head_dim], 32-byte aligned
 *   workspace (device) kvq_chunk_workspace_bytes for the device's SMs, 32-byte aligned;
 *       nothing in it has to be kept or cleared between calls.
 * Uses batch, num_q_heads, qk_dim = v_dim = head_dim, seq_lens, max_kv_len, sm_scale,
 * out_dtype, out_scale, error_flag, prefix_p_f16 and the FP8 query of p (num_splits and fresh_tokens
 * have to be in their ranges and change nothing; prob_scale must be 0).  FP8 and NVFP4 caches with head_dim 64 or 128 and
 * any number of query heads per kv head, per-head scales; not MLA, batch <= 8192.
 * The chunks' work is cut by its size, over the keys too, so that all SMs get the same
 * share of it, whatever the lengths.  In a batch of more than one, requests with a single
 * new token are the split-KV decode's (at most 16 query rows per kv head, 8 differential
 * ones; with more they count as chunks), which runs before the chunks and cuts each
 * request's tokens into one number of chunks, made from batch and max_kv_len; those that are
 * far longer than the others count as chunks, so that no SM waits long for one request.
 * Three or four launches on `stream`.
 * The chunks' probabilities enter the products with V in two f16 parts: each off by at most
 * 2^-21 of itself, or by 2^-31 of the row's largest one where that is more (from 2^-10 of the
 * largest down); of plain heads and where p->prefix_p_f16 asks for it in one: 2^-11, or 2^-32
 * of the largest.  So a token below 2^-32 of the largest counts in the sum alone, and many
 * small ones of one size may be off in the same direction (131072 of them: 6e-5 of a row at
 * most).
 * Everything summed is fp32, but the matrix units' accumulators cut off: where all values
 * have one sign, long sums lose up to 6e-6 of themselves with fp32 outputs, 1.5e-5 with
 * differential heads and 5e-5 with bf16 and E4M3 outputs and with one part.
 * A NaN among a token's keys or values reaches the rows that attend to it and no others;
 * all dims of such a row may become NaN.
 * Calls that share a workspace must not overlap on the GPU.
 */
kvq_status kvq_chunk_attention(const kvq_cache* c, const kvq_decode_params* p, const kvq_diff* d,
                               int num_tokens, const int32_t* q_offsets, const void* q,
                               void* workspace, size_t workspace_bytes, void* out, void* stream);

/* Bytes of kvq_chunk_attention's workspace, for these heads, batch and max_kv_len (0 for
 * arguments below their range); d as in the call. */
size_t kvq_chunk_workspace_bytes(int num_sms, const kvq_cache* c, const kvq_decode_params* p,
                                 const kvq_diff* d);

/*
 * Prefill attention over the cache (Model-Optimizer PR 1832: the prefill
 * kernel of its latency tables, timed against split-KV decode): causal, no
 * KV split.  Request b holds seq_lens[b] = L tokens, the last q_len of them
 * the new ones whose queries are given: query i (position L - q_len + i)
 * attends to keys 0 .. L - q_len + i,
 *   out[b][i][hq][:] = sum_j softmax_j(sm_scale q . k^_j) v^_j
 * in p->out_dtype (as kvq_decode_combine writes it).  With q_len = 1 this
 * is one program per (request, kv head) over the whole sequence.
 *   q   (device) bf16 [batch][q_len][Hq][head_dim], 16-byte aligned.
 *   out (device) [batch][q_len][Hq][head_dim].
 * Uses batch, num_q_heads, qk_dim = v_dim = head_dim, seq_lens, max_kv_len,
 * sm_scale, out_dtype, out_scale and error_flag of p (num_splits and
 * fresh_tokens are ignored; prob_scale must be 0 and q_fp8 0).  FP8 or
 * NVFP4 caches with head_dim 64 or 128, per-kv-head scales allowed; not MLA.
 * Requests with L < q_len: queries before position 0 attend to nothing and
 * give 0.  q_len >= 1.  The products add up in the matrix units' fp32 accumulators,
 * which cut off towards zero: 60000 tokens whose values have one sign lose 3.6e-4 of
 * their sum (kvq_chunk_attention less than 6e-6 with fp32 outputs).
 */
kvq_status kvq_prefill(const kvq_cache* c, const kvq_decode_params* p, int q_len, const void* q,
                       void* out, void* stream);

/*
 * Allocation-free decode step (the pages have no counterpart; this is a
 * convenience of this library).  For callers that cannot allocate device
 * memory -- their device memory is owned by a host framework's fixed pool,
 * or a hard memory budget forbids another cudaMalloc -- this does what
 * kvq_decode does, but keeps the split partials and arrival counters in a
 * static device buffer inside the library: KVQ_NOALLOC_SCRATCH_BYTES (4 MiB)
 * that every GPU loading the library holds until the process exits.  The
 * caller passes only inputs and the output.
 *   Needs 256-aligned (4 * batch * num_kv_heads) + 256-aligned
 *   (4 * batch * Hq * num_splits) + 4 * batch * Hq * num_splits * v_dim
 *   bytes <= KVQ_NOALLOC_SCRATCH_BYTES; larger requests return
 *   KVQ_ERR_WORKSPACE (use kvq_decode with caller-owned buffers).
 *   Every call looks up the buffer's device address on the current device
 *   (cudaGetSymbolAddress); the first call on a device also loads the
 *   library's device code there, so make it before any stream capture.
 *   Every call clears the counters (an asynchronous memset on `stream`)
 *   and then launches the decode; it allocates and frees nothing.  The
 *   memset sits between a preceding kvq_quantize_append and the decode, so
 *   p->fresh_tokens > 0 is accepted but gives no overlap here: the decode
 *   starts after the append has finished.
 *   All calls share the one buffer: calls that overlap on the GPU (other
 *   streams, other host threads) race and must be serialized by the caller.
 */
#define KVQ_NOALLOC_SCRATCH_BYTES (4u << 20)
kvq_status kvq_decode_noalloc(const kvq_cache* c, const kvq_decode_params* p, const void* q,
                              void* out, void* stream);

/*
 * FP8 quantization of bf16 values (e.g. the query of an FP8-query decode):
 *   out[i] = E4M3(fl32(x[i] / s)), s = head_scale[(i / head_len) % num_heads]
 * when head_scale (device, [num_heads]) is given, else scale (finite > 0);
 * round to nearest even, saturating at +-448, the sign of zero kept -- the
 * arithmetic of the FP8 append.  x (device, bf16, 16-byte aligned) and out
 * (device) hold n elements; n and head_len multiples of 8 (head_len > 0
 * when head_scale is given).
 */
kvq_status kvq_quantize_fp8(const void* x, size_t n, float scale, const float* head_scale,
                            int head_len, int num_heads, uint8_t* out, void* stream);

/*
 * Elementwise fp32 -> code conversions with the device encoders the append
 * path uses: out[i] = E4M3(x[i]) (round to nearest even, saturating at
 * +-448) or the E2M1 nibble of x[i] (saturating at +-6) in the low 4 bits.
 * x and out (device), n >= 0.  NaN inputs give unspecified codes.
 */
kvq_status kvq_encode_e4m3(const float* x, uint8_t* out, size_t n, void* stream);
kvq_status kvq_encode_e2m1(const float* x, uint8_t* out, size_t n, void* stream);

/*
 * The FP8-probability quantizer of the decode kernels (vLLM PR 15734:
 * softmax(QK^T) quantized to FP8 with prob_output_scale), elementwise:
 *   out[i] = E4M3(fl32(p[i] / prob_scale))   (round to nearest even, +-448)
 * computed exactly as kvq_decode_partial computes it for probabilities in
 * [0, 1].  The division by prob_scale takes a precomputed reciprocal and one
 * fused correction when a host check shows that, for this prob_scale, it
 * gives the codes of the IEEE division for every p in [0, 1] (it always does
 * near the E4M3 rounding boundaries, where it is checked, and it is within
 * one fp32 step of the IEEE quotient everywhere); otherwise it is the IEEE
 * division.  *used_reciprocal (host, optional) tells which.  prob_scale
 * finite > 0; p and out (device), n >= 0 (n = 0 runs only the host check).
 * Codes for p outside [0, 1] are unspecified.
 */
kvq_status kvq_encode_prob_e4m3(const float* p, uint8_t* out, size_t n, float prob_scale,
                                int* used_reciprocal /* host */, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* KVQ_H */
