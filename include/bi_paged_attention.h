/*
 * bi_paged_attention.h -- C ABI of the decode attention over the paged 8-bit cache (libbigemm.so).
 *
 * For each sequence b and query head h (grouped queries: head h reads key/value head
 * h / (Hq / num_heads)), with the cache of bi_kv_cache.h and L = seq_lens[b]:
 *   s_j = scale * (q . k_j)  for the positions j in [max(0, L - window), L)  (window 0: from 0),
 *   O[b][h] = sum_j softmax(s)_j v_j, rounded once to bf16;  lse[b][h] = log sum_j exp(s_j).
 * Position j lies in page block_table[b][j / page_size], place j % page_size.
 *
 * Batch invariance: the reduction order is fixed by (L, window) alone.  The positions are cut into
 * chunks at fixed places, each chunk is reduced in a fixed order by whichever CTA gets it, and the
 * chunks are added in ascending order, so a sequence's output does not depend on the batch, on the
 * page numbers or on the page size.  ("DeepSeek V4的batch invariance：大模型确定性推理的工程基石"
 * (lshu.cn), section 4.1, has one kernel that splits a sequence and one that does not, with equal
 * bits; here every call splits at the same places.)
 *
 * A sequence with L = 0 gets O = 0 and lse = -inf.  L outside [0, max_pages * page_size], a page
 * number outside [0, num_pages) or a scale outside [2^-64, 2^64] among the attended positions make
 * the sequence's outputs (a scale: its key/value head's) NaN, and nothing is read out of bounds.
 *
 * Accuracy: sums, softmax statistics and scores are fp32.  Entries of a query head below 2^-28 of its
 * largest are off by up to 2^-39 of that largest, all others exact.  In the sum over v_j the weights are fp16, off
 * by up to 2^-11 of themselves with signs that vary (weight times value scale below 2^-29 of the
 * sequence's largest: by 2^-40 of that), before O is rounded to bf16, up to 2^-8.  lse and the
 * denominator do not see it.  bi_decode_attention keeps fp32 weights.
 *
 * Codes behind position L - 1, NaN among them, and pages wholly before the window are never read
 * into a result.  Several query tokens of one sequence are sequences of their own that share a
 * table row's contents, each with its own length.
 */
#ifndef BI_PAGED_ATTENTION_H
#define BI_PAGED_ATTENTION_H

#include <stddef.h>
#include <stdint.h>

#include <cuda_runtime_api.h>

#include "bi_gemm.h"
#include "bi_kv_cache.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Bytes of workspace bi_paged_decode_attention needs for B sequences of up to max_len positions
 * (max_pages * page_size): one partial result per chunk, query head and sequence.  0 when no
 * sequence can have two chunks, and for sizes that the call refuses: below 1, B above 16384, B * Hq
 * from 2^31, D other than 64 and 128, max_len above 2^30. */
size_t bi_paged_decode_attention_workspace_bytes(int64_t B, int Hq, int D, int64_t max_len);

/*
 * One query token per sequence.  Device pointers:
 *   Q [B][ldq] bf16, the Hq * head_dim values of a row contiguous (a slice of a fused projection's
 *   output will do); O [B][ldo] bf16; lse fp32 [B][Hq] or NULL;
 *   block_table int32 [B][ld_table], ld_table >= max_pages; seq_lens int32 [B].
 * scale: any finite value.  window: 0, or the number of positions a query sees.
 * Hq a multiple of num_heads, at most 16 query heads per key/value head.  Q finite.  Where s_j log2 e
 * itself is beyond the fp32 range, the query head's outputs are NaN or those without position j.
 * workspace: at least bi_paged_decode_attention_workspace_bytes(B, Hq, head_dim, max_pages *
 * page_size) bytes, 16-byte aligned (NULL when that is 0).  The call overwrites it; calls that may
 * run at the same time need workspaces of their own.
 * Q and O 16-byte aligned, ldq and ldo multiples of 8 and >= Hq * head_dim; other arrays 4-byte
 * aligned.  B = 0 is a no-op returning BI_OK.  Limits: B <= 16384, max_pages * page_size <= 2^30, and at most
 * 2^30 partial results (B * num_heads * chunks, with at most 128 chunks).
 * Errors: BI_ERR_INVALID_ARG, BI_ERR_ALIGNMENT, BI_ERR_UNSUPPORTED_SHAPE, BI_ERR_NO_DEVICE,
 * BI_ERR_CUDA.
 */
bi_status_t bi_paged_decode_attention(const bi_kv_cache_t *cache, const void *Q, int64_t ldq,
                                      const int32_t *block_table, int64_t ld_table,
                                      int64_t max_pages, const int32_t *seq_lens, int64_t B, int Hq,
                                      float scale, int64_t window, void *workspace,
                                      size_t workspace_bytes, void *O, int64_t ldo, float *lse,
                                      cudaStream_t stream);

/*
 * The time limit, in nanoseconds, of every wait inside the attention kernels that this process launches
 * from now on (default 2e9, i.e. 2 s; 0 restores the default), counted as by bi_gemm_set_wait_timeout;
 * a captured call keeps the limit it was captured with.  A thread block whose wait runs out waits for
 * its copies in flight and ends: what it has not finished by then is NaN in O and lse, nothing is left
 * as it was, the other blocks' outputs are right and the context stays usable.  No status word
 * reports it.
 */
bi_status_t bi_paged_decode_attention_set_wait_timeout(uint64_t timeout_ns);

/*
 * Test-only fault injection on the host side of the launch, for the whole process: every thread block
 * leaves its n-th load out (counted from 1; 0: none), so that a wait for it must end by its time
 * limit.  Never set in production.
 */
bi_status_t bi_paged_decode_attention_debug_skip_load(uint32_t n);

#ifdef __cplusplus
}
#endif

#endif /* BI_PAGED_ATTENTION_H */
