/*
 * bi_kv_cache.h -- C ABI of the paged 8-bit key/value cache (libbigemm.so): the block tables and
 * slot maps, and the write into the cache.  bi_paged_attention.h holds the decode attention that
 * reads it.
 *
 * The pages' decode attention walks a sequence's cached keys and values ("DeepSeek V4的batch
 * invariance：大模型确定性推理的工程基石" (lshu.cn), section 4.1).  This cache holds them in pages of
 * page_size tokens, as e4m3 codes with one fp32 scale for each page and key/value head, keys and
 * values apart:
 *
 *   value(page p, token i, head h, d) = e4m3(code) * scale[p][h].
 *
 * Batch invariance reaches into the cache: a page's codes and scales are a function of the tokens
 * written to it since its first place was, alone.  They do not depend on the other sequences, on the
 * page's number, or on whether the tokens came one at a time, in pieces or all at once (see
 * bi_kv_append_e4m3, also for tokens that are discarded and written over).
 *
 * Pointers are device pointers of the current device, owned by the caller; calls are asynchronous
 * on `stream` and allocate nothing.  Status codes are those of bi_gemm.h; a refused call has
 * launched nothing.
 */
#ifndef BI_KV_CACHE_H
#define BI_KV_CACHE_H

#include <stddef.h>
#include <stdint.h>

#include <cuda_runtime_api.h>

#include "bi_gemm.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * A cache: two pools of pages and their scales.  Code (p, i, h, d) of keys and of values lies at
 * byte p * page_stride + i * token_stride + h * head_stride + d of its pool, so both [page][token]
 * [head][d] and [page][head][token][d] (whose (page, head) blocks are contiguous) are cache
 * layouts; a slot, the number of one token's place, is p * page_size + i.
 * Limits: page_size 16, 32, 64, 128 or 256; head_dim 64 or 128; num_pages * page_size < 2^31.
 * k, v 16-byte aligned, strides multiples of 16 and at least head_dim, page_stride at least the
 * bytes a page spans, and no two codes at one byte; scales 4-byte aligned, [num_pages][num_heads].
 */
typedef struct {
    void *k, *v;                 /* e4m3 codes */
    float *k_scale, *v_scale;    /* [num_pages][num_heads] */
    int64_t num_pages;
    int page_size;               /* tokens in a page */
    int num_heads;               /* key/value heads */
    int head_dim;
    int64_t page_stride, token_stride, head_stride;   /* bytes */
} bi_kv_cache_t;

/*
 * Block tables and slot maps of one step, from the requests' lengths.  Request b has ctx_lens[b]
 * tokens in the cache (in the pages block_table[b][0 .. ceil(ctx/page_size))) and gets
 * new_lens[b] >= 0 more; new_lens[b] = -1 ends it.  In this order:
 *   1. the pages of ended requests are pushed on the stack free_pages[0 .. *free_count), by
 *      request and then by position;
 *   2. every other request whose tokens reach past its last page gets pages from the top of the
 *      stack, by request and then by position, written to block_table[b] behind its present ones;
 *   3. seq_lens[b] = ctx + new (0 for an ended request); token_offsets[0 .. B], the exclusive sums
 *      of the new lengths; and for the j-th new token of request b, row t = token_offsets[b] + j,
 *      positions[t] = ctx + j and slot_map[t] = its slot.  The rows of slot_map and positions from
 *      token_offsets[B] to max_tokens are set to -1;
 *   4. *free_left = the pages left on the stack.
 * Entries of block_table that get no page keep what they held, as do those of free_pages that step 1
 * does not push to (a page that step 2 pops stays in its entry).  All of it is integer work in a fixed
 * order.
 *
 * *status (device) is set to BI_OK; to BI_ERR_INVALID_ARG for a length below 0 (new_lens: below
 * -1) or a *free_count outside [0, free_capacity]; or to BI_ERR_UNSUPPORTED_SHAPE when the call
 * does not fit: a request beyond max_pages pages, more than max_tokens new tokens, too few free
 * pages, or more returned pages than free_capacity holds.  In the last two cases nothing is assigned or
 * returned: seq_lens gets ctx_lens, token_offsets 0, slot_map and positions -1, *free_left
 * *free_count, and the table and the stack stay as they are.
 * Page numbers on the stack are the caller's (each page once); one that is negative or whose slots
 * would pass 2^31 gives -1 in slot_map.
 *
 * int32 device arrays: ctx_lens, new_lens, seq_lens [B]; free_pages [free_capacity]; free_count,
 * free_left, status [1]; block_table [B][ld_table], ld_table >= max_pages; token_offsets [B + 1];
 * slot_map, positions [max_tokens] (positions may be NULL).  seq_lens may be ctx_lens and
 * free_left may be free_count (a captured step that is replayed); other arrays must not overlap.
 * Limits: 0 <= B <= 8192, max_pages * page_size < 2^31, max_tokens and free_capacity <= 2^30.
 * Errors: BI_ERR_INVALID_ARG, BI_ERR_ALIGNMENT (4 bytes), BI_ERR_UNSUPPORTED_SHAPE,
 * BI_ERR_NO_DEVICE, BI_ERR_CUDA.
 */
bi_status_t bi_kv_block_tables(const int32_t *ctx_lens, const int32_t *new_lens, int64_t B,
                               int page_size, int32_t *free_pages, int64_t free_capacity,
                               const int32_t *free_count, int32_t *block_table, int64_t ld_table,
                               int64_t max_pages, int32_t *seq_lens, int32_t *token_offsets,
                               int32_t *slot_map, int32_t *positions, int64_t max_tokens,
                               int32_t *free_left, int32_t *status, cudaStream_t stream);

/*
 * Write T tokens into the cache: row t of K and V (bf16 [T][num_heads][head_dim], row pitches ldk
 * and ldv in elements, so slices of a fused projection's output will do) goes to slot slot_map[t];
 * rows with a slot outside [0, num_pages * page_size) are skipped.
 *
 * Scales.  2^E with one exponent for each page and head, E = max over the page's tokens of the
 * smallest e with amax <= 448 * 2^e, amax the token's largest finite magnitude in that head; e is
 * kept in [-64, 64] (a zero token has e = -64, magnitudes above 448 * 2^64 saturate).  A token in the
 * page's first place starts the page anew; any other joins the tokens in the places before it,
 * and when it raises E their codes are moved to the new scale.
 * Codes.  code = R(x / 2^E), R rounding to nearest even at 4 significant bits and, below the
 * smallest normal 2^-6, cutting to a multiple of 2^-9.  R(R(x / 2^E) / 2^D) = R(x / 2^(E + D)) for
 * every D >= 0 (rounding twice to the nearest subnormal would not give that), so a moved code is
 * the code the token would have got at once, and the page is a function of its tokens alone.  The
 * cut costs at most 2^-9 of the scale, 2^-16 of the head's largest magnitude.
 * Infinities and NaN are stored as NaN.
 * Writing a place again.  E only grows until the page is started anew, so the page then keeps the
 * exponent, and the rounding of the codes before that place, that the discarded token gave it: the codes
 * are those of R(x / 2^E) for that E, no finer.  A sequence whose length goes back (draft tokens that were
 * rejected) is the function of its final tokens that a sequence without them is only if the page of its
 * new end is written again from that page's first place; a page that is new since then always is.
 *
 * Contract: the slots of one page in one call are consecutive rows with consecutive slots, as
 * bi_kv_block_tables gives them (one run per page), and the places before a run's first slot hold
 * tokens that this call has written before, under a scale it has written.  Otherwise the page's
 * contents are unspecified (nothing is written outside the named pages).
 * K and V 16-byte aligned, ldk and ldv multiples of 8 and >= num_heads * head_dim; slot_map int32
 * [T], 4-byte aligned.  T = 0 is a no-op returning BI_OK.  T < 2^31.
 * Errors: BI_ERR_INVALID_ARG, BI_ERR_ALIGNMENT, BI_ERR_UNSUPPORTED_SHAPE, BI_ERR_NO_DEVICE,
 * BI_ERR_CUDA.
 */
bi_status_t bi_kv_append_e4m3(const bi_kv_cache_t *cache, const void *K, int64_t ldk, const void *V,
                              int64_t ldv, const int32_t *slot_map, int64_t T, cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* BI_KV_CACHE_H */
