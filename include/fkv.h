/*
 * fkv.h -- C ABI of libfkv: FP8 paged-KV decode attention for sm_103a (GB300).
 *
 * The operations follow the description of Cloudflare's serving work in
 * "Cloudflare Workers AI Optimizes Large Model Serving with KV Cache
 * Quantization, Weight Compression, and Integrity Checks" (the extracted text
 * of the post "Smaller, faster, safer: running Kimi and GLM at scale") and
 * "Kimi and GLM Reasoning Slimming: Hands-On Test", section "Giving Every
 * Physical Cache Page a 'Generation Number'":
 *   - the KV cache is stored as FP8 e4m3 instead of BF16, halving its size;
 *   - the FP8 attention kernel converts cache values as it reads them;
 *   - every physical page has a tag that changes when it is reallocated; each
 *     request records the (page, tag) pairs it expects; a separate batch check
 *     (not fused into attention) runs before decode reads the cache, and a
 *     mismatching request is aborted (fail closed); deployments that do not
 *     enable the check pay nothing.
 *
 * Conventions for every call
 *   - All array arguments are DEVICE pointers owned by the caller; the library
 *     never allocates, frees or retains them.  `stream` is a cudaStream_t
 *     passed as void* (NULL = the legacy default stream).
 *   - Calls are asynchronous on `stream`: no host synchronisation, no
 *     device-to-host copy.  Host-side argument checks return
 *     FKV_ERR_INVALID_ARG / FKV_ERR_UNSUPPORTED synchronously and launch
 *     nothing; a failed launch returns FKV_ERR_CUDA.
 *   - Data-dependent problems found on the device never trap: they are
 *     recorded in a sticky per-device error word (see fkv_device_error) and
 *     the affected output is handled as documented per call.
 *   - head_dim must be 128.  Cache, q and out must be 16-byte aligned.
 *
 * Layouts
 *   KV pool (one per K and one per V, per layer):
 *       [num_pages][num_kv_heads][page_size][head_dim]
 *     one (page, head) tile is page_size * head_dim contiguous elements;
 *     elements are e4m3 codes (1 byte) or bf16 (2 bytes).
 *     The 4-bit pool (FKV_KV_FP4) is uint8
 *       [num_pages][num_kv_heads][page_size][FKV_FP4_ROW_BYTES]
 *     with one row of 72 bytes per (token, KV head): byte j < 64 holds the e2m1
 *     codes of dims 2j (low nibble) and 2j + 1 (high nibble), byte 64 + b the
 *     e4m3 scale s_b of dims 16b .. 16b + 15.  With g the KV head's fp32 scale
 *     (the same scale an FP8 cache of that head would use), dim d of the row
 *     stands for e2m1(code_d) * s_(d / 16) * g: 0.5625 of the FP8 cache's bytes.
 *   Page table (CSR): page_indptr int32[batch + 1], page_indices int32[nnz];
 *     token t of request r lives in page page_indices[page_indptr[r] + t /
 *     page_size] at offset t % page_size.
 *   Queries / outputs: bf16 [batch][num_q_heads][head_dim]; query head i
 *     attends with KV head i / (num_q_heads / num_kv_heads).
 */
#ifndef FKV_H_
#define FKV_H_

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define FKV_API __attribute__((visibility("default")))
#else
#define FKV_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    FKV_OK = 0,
    FKV_ERR_INVALID_ARG = 1,   /* null pointer, bad size, misalignment, small workspace */
    FKV_ERR_UNSUPPORTED = 2,   /* valid but not implemented (head_dim != 128, a group size that does not split into groups of <= 8, ...) */
    FKV_ERR_CUDA = 3,          /* a CUDA runtime call or launch failed */
    FKV_ERR_SCRATCH_LIMIT = 4  /* paged_decode_attn_noalloc: the shape needs more scratch than
                                  FKV_NOALLOC_SCRATCH_BYTES */
} fkv_status;

typedef enum {
    FKV_KV_FP8_E4M3 = 0,
    FKV_KV_BF16 = 1,
    FKV_KV_FP4 = 2      /* e2m1 codes with an e4m3 scale per 16 dims: rows of FKV_FP4_ROW_BYTES */
} fkv_kv_dtype;

#define FKV_FP4_ROW_BYTES 72   /* a token row of the 4-bit cache: 64 bytes of codes, 8 scales */

/* Bits of the sticky device error word. */
#define FKV_DEVERR_APPEND_SLOT   0x1u  /* kv_append_*: slot beyond the pool, token skipped */
#define FKV_DEVERR_ATTN_PAGE     0x2u  /* paged_*_attn: page id outside [0, num_pages), row zeroed */
#define FKV_DEVERR_TIMEOUT       0x4u  /* a bounded wait on a copy gave up; the call's output is not valid */
#define FKV_DEVERR_REALLOC_PAGE  0x8u  /* kv_page_realloc: a listed id is outside [0, num_pages), skipped */
#define FKV_DEVERR_GATHER_SLOT   0x10u /* kv_gather: slot beyond the pool, its rows written as zeros */
#define FKV_DEVERR_TABLES        0x20u /* kv_step_tables: a request was refused, or a free page id is outside [0, num_pages) */
#define FKV_DEVERR_ROPE_AXIS     0x40u /* qk_norm_rope, kv_append_rope: an axis_map entry is not below n_axes, its pair was not turned */
#define FKV_DEVERR_TREE          0x80u /* kv_tree_commit: a kept list or a drafted token's page is not valid (the request was left
                                          as it was), or the free list has no room (no page was given back) */

FKV_API const char *fkv_status_string(fkv_status s);

/*
 * kv_append_fp8 -- quantize new tokens' K and V to e4m3 and write them into
 * their page slots.  (Cloudflare post: the cache is stored as FP8 e4m3 instead
 * of BF16.)  For every token n with slot = slot_mapping[n] >= 0, KV head h and
 * element d:
 *     code = e4m3_rne_satfinite( fl32( fl32(x) / scale[h] ) )
 * i.e. an IEEE round-to-nearest fp32 division followed by one
 * round-to-nearest-even to e4m3; |values| > 448 and +-Inf saturate to +-448,
 * NaN stays NaN.  The code goes to cache[slot / page_size][h][slot %
 * page_size][d].
 *
 *   k_new, v_new   bf16 [n_tokens][num_kv_heads][head_dim]
 *   slot_mapping   int64 [n_tokens]; < 0 means "padding, skip"
 *   k_scale, v_scale  fp32 [num_kv_heads], positive and finite (this layer)
 *   k_cache, v_cache  uint8 pools (layout above)
 * A slot whose page is >= num_pages is skipped and sets FKV_DEVERR_APPEND_SLOT.
 * Bytes outside the written slots are never touched.  n_tokens == 0 is a no-op.
 */
FKV_API fkv_status kv_append_fp8(const void *k_new, const void *v_new,
                         const int64_t *slot_mapping, int32_t n_tokens,
                         const float *k_scale, const float *v_scale,
                         uint8_t *k_cache, uint8_t *v_cache,
                         int32_t num_pages, int32_t num_kv_heads,
                         int32_t page_size, int32_t head_dim, void *stream);

/*
 * kv_append_bf16 -- the BF16-cache counterpart of kv_append_fp8 (the
 * comparison baseline the Cloudflare post measures against): the same
 * placement, values stored unchanged.
 */
FKV_API fkv_status kv_append_bf16(const void *k_new, const void *v_new,
                          const int64_t *slot_mapping, int32_t n_tokens,
                          void *k_cache, void *v_cache,
                          int32_t num_pages, int32_t num_kv_heads,
                          int32_t page_size, int32_t head_dim, void *stream);

/*
 * kv_append_fp4 -- the 4-bit cache's counterpart of kv_append_fp8: the same
 * arguments and placement, pools of FKV_FP4_ROW_BYTES rows (layout above).
 * For each block of 16 dims of a row, with g = scale[h]:
 *     s    = e4m3_rne_satfinite( fl32( max|x| / fl32(6 g) ) )
 *     D    = fl32( s * g )
 *     code = e2m1_rne_satfinite( fl32( x / D ) );
 *            0 for the whole block when D is 0 or NaN
 * (IEEE divisions, ties to the even code; a zero code may carry either sign).  Scales of kv_calibrate_scales fit:
 * a block's s is then at most 74.7, so values up to six times the calibrated
 * maximum are still held without saturation.  An infinity saturates (its
 * block takes s = 448); a NaN makes its block's scale, and so its 16 values,
 * NaN.  A slot listed twice in one call ends with a mix of the two tokens' rows
 * (a block may hold one's codes under the other's scale): list each slot once.
 * num_kv_heads is at most 32767.
 */
FKV_API fkv_status kv_append_fp4(const void *k_new, const void *v_new,
                         const int64_t *slot_mapping, int32_t n_tokens,
                         const float *k_scale, const float *v_scale,
                         uint8_t *k_cache, uint8_t *v_cache,
                         int32_t num_pages, int32_t num_kv_heads,
                         int32_t page_size, int32_t head_dim, void *stream);

/*
 * kv_gather -- read cached tokens back as bf16 (a prompt's next chunk, or a
 * request that reuses a cached prefix, attends over them outside the decode
 * kernel).  For every n with slot = slots[n] >= 0, KV head h and element d:
 *     out[n][h][d] = bf16_rne( fl32( value * scale[h] ) )
 * with value the e4m3 code's value (FKV_KV_FP8_E4M3) or e2m1 code * block scale
 * (FKV_KV_FP4, exact before the product with scale[h]); FKV_KV_BF16 rows are
 * copied.  The rows of slot < 0 (padding) are zeros, as are those of a slot
 * whose page is >= num_pages, which sets FKV_DEVERR_GATHER_SLOT.
 *
 *   k_cache, v_cache  pools (layout above) of dtype kv_dtype
 *   k_scale, v_scale  fp32 [num_kv_heads]; ignored (may be NULL) for BF16
 *   slots          int64 [n_tokens], repeats allowed
 *   k_out, v_out   bf16 [n_tokens][num_kv_heads][head_dim], 16-byte aligned
 * num_kv_heads is at most 32767.  n_tokens == 0 is a no-op.
 */
FKV_API fkv_status kv_gather(const void *k_cache, const void *v_cache, int32_t kv_dtype,
                             const float *k_scale, const float *v_scale,
                             const int64_t *slots, int32_t n_tokens, void *k_out, void *v_out,
                             int32_t num_pages, int32_t num_kv_heads,
                             int32_t page_size, int32_t head_dim, void *stream);

/*
 * qk_norm_rope -- RMS norm of every query and key head and the rotation by the
 * token's position, in one pass, before the keys go into the cache.  For every
 * token n and head row x of 128 elements (fp32 arithmetic, one rounding to
 * bf16 at the end):
 *     y = x * rsqrt(mean(x^2) + eps) * weight     (y = x when weight is NULL)
 *     pair j < rotary_dim / 2:  theta = positions[axis_map[j]][n] * inv_freq[j]
 *         (a, b) -> (a cos - b sin, b cos + a sin), cos and sin times rot_scale
 *     with (a, b) = (y[j], y[j + rotary_dim / 2]), or (y[2j], y[2j + 1]) when
 *     interleaved != 0; elements from rotary_dim on are y unchanged.
 * The angle keeps its low bits at far positions: the product is formed in two
 * fp32 words and reduced to a fraction of a turn before sin and cos (|theta|
 * below 2^31; below 2^20 it is off by about 2^-23 of a turn).  A normed row's
 * sum of squares has to be a finite fp32 number (every |x| below 1.6e18 is),
 * and a normal one if eps is 0 (some |x| above 1.1e-19: squares of less vanish).
 *
 *   q, k           bf16, token n's heads at q + n * q_token_stride (elements):
 *                  num_q_heads (num_kv_heads) rows of 128, contiguous; token
 *                  strides are multiples of 8, so q and k may lie in one
 *                  projection's output.  k may be NULL with num_kv_heads 0.
 *   q_out, k_out   bf16, the same with their own token strides; they may be q
 *                  and k themselves (in place) but must not overlap otherwise
 *   q_weight, k_weight  bf16 [128], or NULL for no norm of those heads
 *   positions      int32 [n_axes][n_tokens]
 *   inv_freq       fp32 [rotary_dim / 2], finite
 *   axis_map       uint8 [rotary_dim / 2], each below n_axes (an entry that is
 *                  not leaves its pair unturned, cos 1 and sin 0 without
 *                  rot_scale, and sets FKV_DEVERR_ROPE_AXIS);
 *                  NULL: axis 0 for every pair.  n_axes is 1 .. 8
 *   rotary_dim     a multiple of 16, 16 .. 128
 * n_tokens == 0 is a no-op.
 */
FKV_API fkv_status qk_norm_rope(const void *q, int64_t q_token_stride, int32_t num_q_heads,
                                const void *k, int64_t k_token_stride, int32_t num_kv_heads,
                                void *q_out, int64_t q_out_token_stride,
                                void *k_out, int64_t k_out_token_stride, int32_t n_tokens,
                                const void *q_weight, const void *k_weight, float eps,
                                const int32_t *positions, int32_t n_axes, const float *inv_freq,
                                const uint8_t *axis_map, int32_t rotary_dim, int32_t interleaved,
                                float rot_scale, int32_t head_dim, void *stream);

/*
 * kv_step_tables -- the tables of one step made on the device from the
 * requests' lengths: page table, slots and positions of the new tokens, with
 * pages taken from a free list where a request grows into them.  Request r
 * holds c = cached_lens[r] tokens and gets n = new_lens[r] more (0: idle, 1:
 * decode, more: a prompt chunk).  With S = page_size, have = ceil(c / S),
 * pages = ceil((c + n) / S):
 *   - its CSR row has `pages` entries: block_table[r][0 .. have), then pages -
 *     have new pages, taken from the top of the free list (free_pages[*free_count
 *     - 1] first) in request order and stored in block_table[r] with their live
 *     tags in block_tags[r]; expected_tags is parallel to page_indices;
 *   - its new tokens are entries token_indptr[r] .. token_indptr[r] + n - 1 of
 *     slot_mapping (page * S + offset) and positions (c, c + 1, ...);
 *   - step_lens[r] = c + n is what paged_decode_attn attends over, and
 *     cached_lens_out[r] = c + n the length kept for the next step.
 * Refused requests (refused[r] = 1, and FKV_DEVERR_TABLES is set): c or n
 * negative or c + n over 2^31 - 1; pages > max_blocks; tokens past n_tokens or
 * entries past nnz; or not enough free pages, counted in request order.  Their
 * step_lens is 0, cached_lens_out[r] = c, their slots are -1 (appends skip
 * them), no page is taken.  A request refused for the first two reasons has an
 * empty CSR row; otherwise missing pages are -1 with tag 0, which
 * kv_page_tag_check and paged_decode_attn reject.  Prefix sums that pass
 * n_tokens or nnz are cut to it.  A listed page id outside [0, num_pages), taken
 * or existing, makes its entries -1 and the slots of tokens on it -1 and sets
 * FKV_DEVERR_TABLES (block_table gets the -1 of a taken one; an existing one's
 * cell and tags are left).  A refused request's positions are c, c + 1, ...,
 * or 0 where it was refused for one of the first two reasons.
 *
 *   cached_lens, new_lens  int32 [batch]
 *   block_table    int32 [batch][max_blocks], block_tags uint32, the same shape;
 *                  only the cells of newly taken pages are written
 *   free_pages     int32 [num_free]; free_count int32 [1] (at most num_free is used)
 *   page_tags      uint32 [num_pages] live tags (read only: kv_page_realloc bumps
 *                  a page's tag when it is given back)
 *   step_lens, cached_lens_out  int32 [batch]; cached_lens_out may be cached_lens
 *   refused        uint8 [batch]
 *   page_indptr    int32 [batch + 1]; page_indices int32 [nnz] and expected_tags
 *                  uint32 [nnz], entries past the last row left as they were
 *   token_indptr   int32 [batch + 1]; slot_mapping int64 [n_tokens] and positions
 *                  int32 [n_tokens], entries past the last token are -1 and 0
 *   free_left      int32 [1], pages still free; may be free_count
 *   workspace      kv_step_tables_workspace_size(batch) bytes, 256-byte aligned,
 *                  not shared by calls that overlap on the GPU
 * The result depends only on the inputs (its few atomics are integer maxima and
 * ORs, the same in any order), and a call repeated on the same inputs writes the
 * same bytes.  batch == 0 still fills slot_mapping
 * and positions, writes the two indptr's single 0 and free_left.
 */
FKV_API size_t kv_step_tables_workspace_size(int32_t batch);
FKV_API fkv_status kv_step_tables(const int32_t *cached_lens, const int32_t *new_lens, int32_t batch,
                                  int32_t *block_table, uint32_t *block_tags, int32_t max_blocks,
                                  const int32_t *free_pages, int32_t num_free, const int32_t *free_count,
                                  const uint32_t *page_tags, int32_t num_pages, int32_t page_size,
                                  int32_t *step_lens, int32_t *cached_lens_out, uint8_t *refused,
                                  int32_t *page_indptr, int32_t *page_indices, uint32_t *expected_tags,
                                  int32_t nnz, int32_t *token_indptr, int64_t *slot_mapping,
                                  int32_t *positions, int32_t n_tokens, int32_t *free_left,
                                  void *workspace, size_t workspace_bytes, void *stream);

/*
 * kv_calibrate_scales -- the per-KV-head scales for writing a whole prompt
 * into the FP8 cache (Cloudflare post: prefill keeps BF16, the cache decode
 * reads is FP8 e4m3).  For each KV head h, separately for K and for V:
 *     amax = max |x| over all n_tokens tokens and head_dim elements of head h
 *     scale[h] = fl32(amax / 448)  (IEEE division; 448 = largest e4m3 value),
 *                1 when amax is 0 (including n_tokens == 0)
 * then kv_append_fp8 with these scales quantizes the prompt (bulk write).
 *
 *   k, v      bf16 [n_tokens][num_kv_heads][head_dim], finite values
 *             (a NaN or Inf input gives a NaN or Inf scale)
 *   k_scale, v_scale  fp32 [num_kv_heads] outputs (also used as the
 *             reduction's scratch; nothing else is written)
 * Launches two kernels and two memsets on `stream`.
 */
FKV_API fkv_status kv_calibrate_scales(const void *k, const void *v, int64_t n_tokens,
                                       int32_t num_kv_heads, int32_t head_dim,
                                       float *k_scale, float *v_scale, void *stream);

/*
 * kv_page_tag_check -- the separate batched integrity pass ("Kimi and GLM
 * Reasoning Slimming: Hands-On Test", section "Giving Every Physical Cache
 * Page a 'Generation Number'"; Cloudflare post, integrity checking).  For each
 * request r:
 *     abort_mask[r] = 1  if its CSR row is malformed (indptr[r] < 0,
 *                        indptr[r+1] < indptr[r] or indptr[r+1] > nnz), or
 *                        for any j in [indptr[r], indptr[r+1]):
 *                        page_indices[j] outside [0, num_pages) or
 *                        page_tags[page_indices[j]] != expected_tags[j]
 *     abort_mask[r] = 0  otherwise.
 *
 *   page_tags      uint32 [num_pages]  live generation tags
 *   page_indptr    int32 [batch + 1], page_indices int32 [nnz]
 *   expected_tags  uint32 [nnz]  parallel to page_indices
 *   abort_mask     uint8 [batch]  output, stays on the device; pass it to
 *                  paged_decode_attn.  Not calling this function and passing
 *                  abort_mask = NULL there is the no-tracker path.
 * batch == 0 is a no-op.
 */
FKV_API fkv_status kv_page_tag_check(const uint32_t *page_tags, int32_t num_pages,
                             const int32_t *page_indptr, const int32_t *page_indices,
                             const uint32_t *expected_tags, int32_t batch, int64_t nnz,
                             uint8_t *abort_mask, void *stream);

/*
 * kv_append_fp8_tag_check -- kv_append_fp8 and kv_page_tag_check of one
 * decode step in a single launch.  (Cloudflare post, integrity checking: the
 * check runs as a separate batch pass before decode reads the cache, not
 * inside the attention kernel; this call keeps it a pass of its own and only
 * shares the append's launch.)
 *
 * Equivalent to kv_append_fp8(k_new ... head_dim) followed by
 * kv_page_tag_check(page_tags, num_pages, page_indptr, page_indices,
 * expected_tags, batch, nnz, abort_mask) on the same stream: the same cache
 * bytes, the same mask, the same argument checks and error codes.  The two
 * parts touch disjoint memory (the append writes only cache bytes, the check
 * reads tags and tables and writes only abort_mask), so the kernel runs them
 * side by side; the caller must not pass buffers that overlap across the two
 * parts.  page_tags has num_pages entries (the pool the append writes into).
 * n_tokens == 0 runs the check alone, batch == 0 the append alone.
 */
FKV_API fkv_status kv_append_fp8_tag_check(const void *k_new, const void *v_new,
                                   const int64_t *slot_mapping, int32_t n_tokens,
                                   const float *k_scale, const float *v_scale,
                                   uint8_t *k_cache, uint8_t *v_cache,
                                   int32_t num_pages, int32_t num_kv_heads,
                                   int32_t page_size, int32_t head_dim,
                                   const uint32_t *page_tags, const int32_t *page_indptr,
                                   const int32_t *page_indices, const uint32_t *expected_tags,
                                   int32_t batch, int64_t nnz, uint8_t *abort_mask, void *stream);

/*
 * kv_append_bf16_tag_check -- the same one-launch prologue for a BF16 cache:
 * kv_append_bf16 followed by kv_page_tag_check, with the same arguments,
 * results, argument checks and rules as kv_append_fp8_tag_check (no scales).
 */
FKV_API fkv_status kv_append_bf16_tag_check(const void *k_new, const void *v_new,
                                    const int64_t *slot_mapping, int32_t n_tokens,
                                    void *k_cache, void *v_cache,
                                    int32_t num_pages, int32_t num_kv_heads,
                                    int32_t page_size, int32_t head_dim,
                                    const uint32_t *page_tags, const int32_t *page_indptr,
                                    const int32_t *page_indices, const uint32_t *expected_tags,
                                    int32_t batch, int64_t nnz, uint8_t *abort_mask, void *stream);

/*
 * kv_append_fp4_tag_check -- the same one-launch prologue for a 4-bit cache:
 * kv_append_fp4 followed by kv_page_tag_check, with the arguments, results,
 * argument checks and rules of kv_append_fp8_tag_check.  It is made for a decode
 * step; thousands of tokens are written faster by the two calls.
 */
FKV_API fkv_status kv_append_fp4_tag_check(const void *k_new, const void *v_new,
                                   const int64_t *slot_mapping, int32_t n_tokens,
                                   const float *k_scale, const float *v_scale,
                                   uint8_t *k_cache, uint8_t *v_cache,
                                   int32_t num_pages, int32_t num_kv_heads,
                                   int32_t page_size, int32_t head_dim,
                                   const uint32_t *page_tags, const int32_t *page_indptr,
                                   const int32_t *page_indices, const uint32_t *expected_tags,
                                   int32_t batch, int64_t nnz, uint8_t *abort_mask, void *stream);

/*
 * kv_page_realloc -- hand pages to new owners on the device ("Kimi and GLM
 * Reasoning Slimming: Hands-On Test", section "Giving Every Physical Cache
 * Page a 'Generation Number'": a page's tag changes each time it is
 * reallocated, so holders of the old (page, tag) pair fail the check; the
 * same page names clearing GPU memory as a further defence).  For each j:
 *     p = pages[j]; page_tags[p] += 1 (modulo 2^32); new_tags[j] = page_tags[p]
 * and, when k_cache / v_cache are given, every byte of page p in both pools
 * is zeroed (all KV heads).  new_tags[j] is the tag the new owner records as
 * its expected tag.
 *
 *   page_tags   uint32 [num_pages], updated in place
 *   pages       int32 [n]; list each page at most once per call (a repeated
 *               page still ends with its tag bumped once per listing, but
 *               which listing receives which new tag is unspecified)
 *   new_tags    uint32 [n] output; 0 for an id outside [0, num_pages), which
 *               is skipped and sets FKV_DEVERR_REALLOC_PAGE
 *   k_cache, v_cache  both NULL (no scrub) or the pools of this layer, of
 *               dtype kv_dtype with num_kv_heads, page_size, head_dim = 128
 * n == 0 is a no-op.
 */
FKV_API fkv_status kv_page_realloc(uint32_t *page_tags, int32_t num_pages,
                                   const int32_t *pages, int32_t n, uint32_t *new_tags,
                                   void *k_cache, void *v_cache, int32_t kv_dtype,
                                   int32_t num_kv_heads, int32_t page_size, int32_t head_dim,
                                   void *stream);

/*
 * paged_decode_attn_workspace_size -- bytes of device workspace that
 * paged_decode_attn needs for this shape on the current device (it depends on
 * the device's SM count).  Returns 0 for unsupported shapes.
 */
FKV_API size_t paged_decode_attn_workspace_size(int32_t batch, int32_t num_q_heads,
                                        int32_t num_kv_heads, int32_t head_dim,
                                        int32_t kv_dtype);

/*
 * paged_decode_attn -- decode-phase attention over the paged cache, values
 * converted from the cache format as they are read (Cloudflare post: the FP8
 * attention kernel converts values as it reads them).  For each request r and
 * query head i (kv head h = i / G):
 *     out[r][i] = sum_t softmax_t( sm_scale * q[r][i] . k_t ) v_t
 * over the request's seq_lens[r] tokens, with k_t = code * k_scale[h] and
 * v_t = code * v_scale[h] for FP8 (the bf16 values for BF16; for FP4 code *
 * block scale * k_scale[h] or v_scale[h]).
 *
 *   q              bf16 [batch][num_q_heads][head_dim]
 *   k_cache, v_cache  pools (layout above) of dtype kv_dtype (fkv_kv_dtype)
 *   k_scale, v_scale  fp32 [num_kv_heads] for FP8 and FP4; ignored (may be NULL) for BF16
 *   page_indptr, page_indices  the CSR page table; nnz = length of page_indices
 *   seq_lens       int32 [batch]  tokens to attend per request
 *   abort_mask     uint8 [batch] from kv_page_tag_check, or NULL (no tracker)
 *   sm_scale       softmax scale, usually 1/sqrt(head_dim)
 *   out            bf16 [batch][num_q_heads][head_dim]
 *   workspace      device scratch of at least
 *                  paged_decode_attn_workspace_size(...) bytes, 256-byte
 *                  aligned; no initialisation needed; must not be shared by
 *                  calls that overlap on the GPU.
 * Fail closed: a request that is aborted, has a malformed CSR row (indptr[r]
 * < 0, indptr[r+1] < indptr[r] or indptr[r+1] > nnz), has seq_lens[r] <= 0,
 * has more tokens than its pages hold, or whose pages include an id outside
 * [0, num_pages), gets an all-zero output row, and no other row is affected.
 * The pages of the first four kinds are not read.  An id outside the pool is
 * never dereferenced: that tile is copied from page 0 instead, and the row is
 * written as zeros whatever those bytes hold (FKV_DEVERR_ATTN_PAGE is set).
 * Deterministic: the same call gives the same bytes every time (the split
 * over warps depends only on the live requests, and the merge of a split
 * (request, KV head) does not depend on which warp performs it or when).  The
 * 4-bit cache's split also depends on nnz: from 60000 tiles' worth of listed
 * pages on (a tile is 64 tokens of one KV head) a call is spread over more
 * warps, so the same rows under a longer page table may differ by rounding, and
 * short requests under a table with room for many take up to 6 us longer: pass
 * the nnz that a step can need, not the most that any may.
 * Softmax weights and their sums are fp32; the product with V takes them as f16
 * for FP8 and FP4 (each within 2^-11 of itself, down to 2^-29 of the largest
 * weight of its part) and as two bf16 words for BF16.
 * Supported: head_dim 128, page_size in {16, 32, 64, 128}, group size
 * G = num_q_heads / num_kv_heads in 1..8, or above 8 when G splits into R
 * equal groups of at most 8 with R a power of two up to 8 (10, 12, 16, 24,
 * 32, 64, ...): each group is then served as a virtual KV head that reads
 * the KV head's pages again, so such a call reads R times the K/V bytes.
 * Other G return FKV_ERR_UNSUPPORTED.
 */
FKV_API fkv_status paged_decode_attn(const void *q, int32_t batch, int32_t num_q_heads,
                             const void *k_cache, const void *v_cache, int32_t kv_dtype,
                             const float *k_scale, const float *v_scale,
                             int32_t num_pages, int32_t num_kv_heads,
                             int32_t page_size, int32_t head_dim,
                             const int32_t *page_indptr, const int32_t *page_indices,
                             int64_t nnz, const int32_t *seq_lens, const uint8_t *abort_mask,
                             float sm_scale, void *out,
                             void *workspace, size_t workspace_bytes, void *stream);

/*
 * paged_decode_attn_noalloc -- paged_decode_attn for callers that cannot
 * allocate device memory.  (The pages describe no such entry point; it has no
 * counterpart there.)
 *
 * Who needs it: code that has no allocator of its own -- a plugin inside a
 * host runtime that owns all device memory and passes the plugin only its
 * input and output buffers -- and serving loops that forbid cudaMalloc on the
 * hot path because it can synchronise the device and stall other streams.
 * Neither can hand paged_decode_attn its workspace.
 *
 * What it does: exactly paged_decode_attn (same arguments, same results,
 * same fail-closed rules) minus the workspace arguments.  Its scratch is one
 * fixed device array of FKV_NOALLOC_SCRATCH_BYTES compiled into the library;
 * every GPU that loads the library reserves that array until the process
 * exits.  The call itself allocates nothing (no cudaMalloc, no cudaFree, no
 * allocating library routine).
 *
 * Limits and rules:
 *   - A shape whose workspace (paged_decode_attn_workspace_size) exceeds
 *     FKV_NOALLOC_SCRATCH_BYTES is rejected with FKV_ERR_SCRATCH_LIMIT before
 *     anything is launched.  With 8 query heads per KV head, 16 MiB covers
 *     roughly batch * num_kv_heads up to 3000 on a 152-SM GB300.
 *   - The first call on a device looks up the array's device address
 *     (cudaGetSymbolAddress, with that device current); make that first call
 *     before any stream capture.  The address is kept together with the id
 *     of the CUDA context it was found in.  When the context changes --
 *     cudaDeviceReset, or the primary context released and created again,
 *     which loads the library's device code anew -- the kept address is
 *     dropped and the next call looks it up again (so that call, too, is a
 *     first call and belongs outside stream capture).
 *   - All calls on a device share the one array and it keeps whatever the
 *     last call left in it (each call clears what it needs cleared).  Calls
 *     that overlap on the GPU -- on different streams, or from different host
 *     threads without ordering -- race on it and give wrong results; order
 *     them on one stream or serialise them.
 */
#define FKV_NOALLOC_SCRATCH_BYTES (16u << 20)
FKV_API fkv_status paged_decode_attn_noalloc(const void *q, int32_t batch, int32_t num_q_heads,
                                     const void *k_cache, const void *v_cache, int32_t kv_dtype,
                                     const float *k_scale, const float *v_scale,
                                     int32_t num_pages, int32_t num_kv_heads,
                                     int32_t page_size, int32_t head_dim,
                                     const int32_t *page_indptr, const int32_t *page_indices,
                                     int64_t nnz, const int32_t *seq_lens, const uint8_t *abort_mask,
                                     float sm_scale, void *out, void *stream);

/*
 * kv_append_rope -- qk_norm_rope and the append in one pass: the query heads are
 * normed, turned and written as bf16, the key heads normed, turned and put into
 * the cache, the value heads put into the cache as they are.  Norm and rotation
 * are qk_norm_rope's; keys are quantised from their fp32 values, rounded once
 * (qk_norm_rope followed by kv_append_* rounds them to bf16 in between):
 *   FP8:  code = e4m3_rne_satfinite( x / scale[h] )
 *   FP4:  kv_append_fp4's blocks and codes, with x for the bf16 element
 *   BF16: bf16_rne(x)
 * (a key's quotient is within an fp32 ulp of x / scale[h]; the values' codes are
 * the bytes of kv_append_fp8, kv_append_bf16 or kv_append_fp4.)
 *
 *   q, k, v        bf16, token n's heads at q + n * q_token_stride (elements):
 *                  rows of 128, contiguous; token strides are multiples of 8, so
 *                  the three may lie in one projection's output.  q and q_out may
 *                  be NULL with num_q_heads 0
 *   q_out          bf16, with its own token stride; may be q itself (in place)
 *                  but must not overlap q, k or v otherwise
 *   q_weight ... rot_scale  as in qk_norm_rope
 *   slot_mapping, k_scale, v_scale, k_cache, v_cache  as in kv_append_fp8, with
 *                  pools of dtype kv_dtype; scales are ignored (may be NULL) for
 *                  BF16.  A token whose slot is < 0 or whose page is >= num_pages
 *                  (which sets FKV_DEVERR_APPEND_SLOT) still has its query heads
 *                  turned.  List each slot once.
 * num_kv_heads is at most 32767.  n_tokens == 0 is a no-op.
 */
FKV_API fkv_status kv_append_rope(const void *q, int64_t q_token_stride, int32_t num_q_heads,
                                  const void *k, int64_t k_token_stride,
                                  const void *v, int64_t v_token_stride, int32_t num_kv_heads,
                                  void *q_out, int64_t q_out_token_stride, int32_t n_tokens,
                                  const void *q_weight, const void *k_weight, float eps,
                                  const int32_t *positions, int32_t n_axes, const float *inv_freq,
                                  const uint8_t *axis_map, int32_t rotary_dim, int32_t interleaved,
                                  float rot_scale, const int64_t *slot_mapping, int32_t kv_dtype,
                                  const float *k_scale, const float *v_scale,
                                  void *k_cache, void *v_cache, int32_t num_pages, int32_t page_size,
                                  int32_t head_dim, void *stream);

/*
 * paged_tree_attn -- attention of drafted tokens over the paged cache.  Request r
 * has n = token_indptr[r + 1] - token_indptr[r] drafted tokens (kv_step_tables'
 * new tokens), already in the cache as the last n of its seq_lens[r] tokens; c =
 * seq_lens[r] - n tokens are committed.  Its i-th query row sees
 *   - drafted token j (position c + j) if bit j % 64 of word j / 64 of the row's
 *     tree_mask is set: its ancestors in the tree, and itself;
 *   - committed token t if window is 0, or t < sinks, or t > p - window with p =
 *     c + max(0, bits set in its mask - 1), the position of its depth in the tree.
 * and out = softmax(sm_scale * q . k) v over what it sees, as in paged_decode_attn.
 * The window says nothing of drafted tokens: they are seen by their bits alone.  For a
 * sliding window along a path deeper than it, leave out the bits of the ancestors that
 * the window (and sinks) leave out; each row is then paged_window_attn's of its token.
 * Bits of tokens that are not there (n and above) are ignored, in the count too.  A
 * row that sees nothing is zeros.  What a row does not see has no part in it, whatever
 * it holds (NaN, infinities; but infinite V that every row of a request sees may give NaN).  Query
 * elements down to 2^-32 of the largest among the rows of a KV head are exact over FP8
 * and FP4, BF16 ones always.  Any order of the drafted tokens is taken; positions (depths) of
 * siblings are the caller's, in kv_append_rope.
 *
 *   q, out         bf16 [n_tokens][num_q_heads][head_dim], rows of request r at
 *                  token_indptr[r] ..; rows that are no request's are not written
 *   token_indptr   int32 [batch + 1]
 *   tree_mask      uint64 [n_tokens][mask_words], mask_words 1 .. 4
 *   window, sinks  0 and 0: no window (sinks has no effect without one)
 *   workspace      paged_tree_attn_workspace_size(...) bytes, 256-byte aligned, no
 *                  initialisation needed, not shared by calls that overlap on
 *                  the GPU (two captured graphs that may run at once need two); one
 *                  of more tokens fits a call of fewer
 *   the others     as in paged_decode_attn
 * Fail closed: the rows of a request that is aborted, has a malformed CSR row, has
 * n > seq_lens[r], n > 64 * mask_words, more tokens than its pages hold, or a page
 * that it reads outside [0, num_pages) (FKV_DEVERR_ATTN_PAGE) are zeros.  It reads the
 * pages of all its tokens, with a window those of the first sinks tokens and from the
 * window of a row at depth 0 on, whatever the masks name of them.  token_indptr
 * entries that are negative, decreasing or past n_tokens leave the request's rows
 * unwritten.
 * Softmax weights and their sums are fp32; the product with V takes them as f16
 * for FP8 and FP4 (each within 2^-11 of itself, down to 2^-24 of the row's largest)
 * and as two bf16 words for BF16.  Logits may have any size that fp32 holds; tokens
 * times the largest |V| has to stay below 2^128.
 * Deterministic: the same call gives the same bytes every time.  Two launches.
 * Supported: head_dim 128, page_size in {16, 32, 64, 128}, up to 128 query heads
 * per KV head.  batch == 0 or n_tokens == 0 is a no-op.
 */
FKV_API size_t paged_tree_attn_workspace_size(int32_t n_tokens, int32_t batch, int32_t num_q_heads,
                                              int32_t num_kv_heads, int32_t head_dim, int32_t kv_dtype);
FKV_API fkv_status paged_tree_attn(const void *q, int32_t n_tokens, int32_t num_q_heads,
                                   const void *k_cache, const void *v_cache, int32_t kv_dtype,
                                   const float *k_scale, const float *v_scale,
                                   int32_t num_pages, int32_t num_kv_heads,
                                   int32_t page_size, int32_t head_dim,
                                   const int32_t *page_indptr, const int32_t *page_indices,
                                   int64_t nnz, const int32_t *seq_lens, int32_t batch,
                                   const int32_t *token_indptr, const uint64_t *tree_mask,
                                   int32_t mask_words, int32_t window, int32_t sinks,
                                   const uint8_t *abort_mask, float sm_scale, void *out,
                                   void *workspace, size_t workspace_bytes, void *stream);

/*
 * paged_window_attn -- decode attention over a sliding window and a few first
 * tokens: paged_decode_attn's arguments and results, over the tokens
 *     t < sinks  or  t >= seq_lens[r] - window
 * of request r, whose query is its last token.  window >= 1, sinks >= 0.  Pages
 * whose tokens are all outside are not read and their entries may hold any id (of
 * pages given back, say).  The workspace is paged_tree_attn_workspace_size(batch,
 * batch, ...) bytes; limits, failing closed and determinism are paged_tree_attn's.
 */
FKV_API fkv_status paged_window_attn(const void *q, int32_t batch, int32_t num_q_heads,
                                     const void *k_cache, const void *v_cache, int32_t kv_dtype,
                                     const float *k_scale, const float *v_scale,
                                     int32_t num_pages, int32_t num_kv_heads,
                                     int32_t page_size, int32_t head_dim,
                                     const int32_t *page_indptr, const int32_t *page_indices,
                                     int64_t nnz, const int32_t *seq_lens, int32_t window, int32_t sinks,
                                     const uint8_t *abort_mask, float sm_scale, void *out,
                                     void *workspace, size_t workspace_bytes, void *stream);

/*
 * kv_tree_commit -- after the drafted tokens of a step are verified: the kept ones'
 * cache rows move to where the next step expects them.  With n, c as in
 * paged_tree_attn and the kept path accepted[r][0 .. accepted_counts[r]) (indices of
 * drafted tokens, strictly increasing: parents come before children):
 *   - for i = 0, 1, ...: the K and V rows of position c + accepted[r][i] go to
 *     position c + i (all KV heads);
 *   - lens_out[r] = c + accepted_counts[r], the length kept for the next step;
 *   - with free_pages: the pages of its tokens past ceil(lens_out[r] / page_size) go
 *     back onto the free list, their live tags bumped by one if page_tags is given
 *     (holders of the old tag fail the check).  They are pushed so that the next
 *     kv_step_tables takes them in the order in which this step did: request 0's
 *     first one is on top.
 * An aborted request, one with a malformed CSR row or token_indptr, and one with n >
 * seq_lens[r] or more tokens than its pages hold is left as it is: no row moves,
 * lens_out[r] is not written, no page goes back.  So is one whose list is not strictly
 * increasing, leaves [0, n), or is longer than n or max_accepted, and one with a
 * drafted token's page outside [0, num_pages); these set FKV_DEVERR_TREE.
 *
 *   k_cache, v_cache  pools of dtype kv_dtype; bytes of other rows are not touched
 *   accepted       int32 [batch][max_accepted]; accepted_counts int32 [batch]
 *   lens_out       int32 [batch], not seq_lens, accepted or accepted_counts themselves
 *                  (kv_step_tables' cached_lens_out fits: it is already the length kept
 *                  for requests left as they are)
 *   free_pages     int32 [num_free], free_count int32 [1] (the entries in use), free_left
 *                  int32 [1] (in use afterwards; may be free_count), page_tags uint32
 *                  [num_pages] or NULL; or all NULL and num_free 0: no page goes back.
 *                  Without room for all pages none goes back (FKV_DEVERR_TREE).
 * A request's drafted positions must lie on pages of its own.  batch == 0 with a free
 * list still writes free_left.
 */
FKV_API fkv_status kv_tree_commit(void *k_cache, void *v_cache, int32_t kv_dtype, int32_t num_pages,
                                  int32_t num_kv_heads, int32_t page_size, int32_t head_dim,
                                  const int32_t *page_indptr, const int32_t *page_indices, int64_t nnz,
                                  const int32_t *seq_lens, int32_t batch, const int32_t *token_indptr,
                                  int32_t n_tokens, const int32_t *accepted, int32_t max_accepted,
                                  const int32_t *accepted_counts, const uint8_t *abort_mask,
                                  int32_t *lens_out, int32_t *free_pages, int32_t num_free,
                                  const int32_t *free_count, int32_t *free_left, uint32_t *page_tags,
                                  void *stream);

/*
 * fkv_device_error -- read (and optionally clear) the sticky device error word
 * of the current device.  Synchronises the device.  *flags receives the OR of
 * FKV_DEVERR_* bits recorded since the last clear.
 */
FKV_API fkv_status fkv_device_error(uint32_t *flags, int32_t clear);

/* Number of kernels one call launches (for launch accounting). */
FKV_API int32_t fkv_kernels_per_call(const char *entry_point);

/*
 * fkv_selftest_wait -- run the failure path of the kernels' bounded waits
 * (diagnostic; the pages have no counterpart).  Every wait in the library's
 * kernels is on an mbarrier that a copy or another warp completes, and gives
 * up after a time limit, recording FKV_DEVERR_TIMEOUT instead of hanging.
 * This launches one block whose three warps run those wait helpers (the
 * spinning one, the sleeping one, and that of tree and window attention) on an
 * mbarrier that nothing completes: each gives up after limit_ns nanoseconds,
 * sets FKV_DEVERR_TIMEOUT and the kernel ends normally.  With complete != 0 the
 * block completes the barrier first and all waits return at once (no error
 * bit).  result: NULL, or a device uint32[2] receiving 1 (the wait saw the
 * barrier complete) or 0 (it gave up): [0] of the first and third helper (2:
 * they do not agree, or waits of the third kind still wait after one gave up),
 * [1] of the sleeping one.  limit_ns above 10 s returns FKV_ERR_INVALID_ARG.
 * Asynchronous on `stream`; read the outcome with fkv_device_error.
 */
FKV_API fkv_status fkv_selftest_wait(uint64_t limit_ns, int32_t complete, uint32_t *result, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* FKV_H_ */
