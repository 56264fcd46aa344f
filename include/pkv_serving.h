/*
 * pkv_serving.h -- a cache held in 8 bits, cross attention to an encoder's
 * states, and page tables kept on the device.  Part of libpkv; the conventions
 * of pkv.h (ownership, streams, errors, layouts, pkv_problem) and of
 * pkv_context.h (views, runs of new tokens, workspaces, what is done about bad
 * lengths, offsets and page numbers) hold here too.
 *
 * 8-bit cache (kv8).  K and V share one pool, bytes
 *     kv8_pool [num_pool_pages][Hkv][32 d],  kv8_scales [num_pool_pages][Hkv][2],
 * the pool 16-byte, the scales 2-byte aligned.  A block is one page of one KV head,
 * K and V apart: 16 tokens by d channels of e4m3 codes (no infinities, 448 the
 * largest) and one scale 2^e, held as the byte e + 127 (K first).  Writing a run
 * gives a block the smallest e with max |x| <= 448 * 2^e over the finite elements
 * of the run's tokens in it, kept in [-15, 7] (PKV_F16) or [-117, 119] (PKV_BF16);
 * where the block holds earlier tokens of the row (the run starts inside the
 * page), e is not smaller than before, and where it grows those tokens' codes are
 * rounded again.  An element becomes x / 2^e rounded to the nearest code, ties to
 * even, saturating at 448; an infinity or a NaN becomes NaN, and reads back as
 * NaN.  The value that a code stands for is exact in the problem's type.  It is
 * off by at most 2^-4 of the element, or 2^(e - 10) where that is more; where the
 * block has grown since, these roundings add up, and it is off by less than 2^(e - 9)
 * where that is more than 2^-4 of the element.  (Elements whose magnitude passes 448 *
 * 2^7, PKV_BF16 448 * 2^119, saturate instead.)  Byte order of a page:
 * csrc/serving/kv8_common.h.  One pool serves one dtype.
 *
 * Cross attention.  Every query of row i sees all N_i = seq_lens[i] tokens of
 * the row's cache: states of an encoder, written once (pkv_store_kv,
 * pkv_kv4_store, pkv_kv8_store), of a length that has nothing to do with the
 * number of queries.  The problem's table and lengths are the encoder's.  Rows
 * may share pages; beams of one request are best passed as several queries of
 * one row, which reads its states once for sixteen of them (query heads of the
 * group times tokens) and more.
 *
 * Page tables.  A row owns the pages of its table up to its length; pages are
 * nobody's twice.  All on the device:
 *     lens        int32 [B]: tokens that a row holds
 *     block_table int32 [B][max_pages_per_row]
 *     free_pages  int32 [num_pool_pages]: a stack, its first state[0] entries valid
 *     state       int32 [4]: free pages; rows that the last pkv_pages_take turned
 *                 down; an arrival counter, zero between calls; reserved
 * Of the problem, batch, num_pool_pages and max_pages_per_row matter; the rest is
 * checked as ever.  Calls on the same tables must not overlap.
 */
#ifndef PKV_SERVING_H
#define PKV_SERVING_H

#include "pkv_context.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Bytes of one page of one KV head in the 8-bit cache (K and V): 32 d; 0 for
 * a head size that is neither 64 nor 128. */
size_t pkv_kv8_page_bytes(int32_t head_dim);

/*
 * Write a run of new tokens into the 8-bit cache, and read a run back: arguments
 * and errors as pkv_kv4_store and pkv_kv4_load, with the scales beside the pool.
 * Earlier tokens of a touched page keep their bytes unless the block's exponent
 * grows; tokens behind the run keep theirs, and mean nothing.  Rows of one call must
 * not write to the same page.
 */
pkv_status pkv_kv8_store(const pkv_problem* prob, const int32_t* tok_offsets, int32_t num_tokens,
                         const int32_t* seq_lens_dev, const void* k_new, int64_t k_stride,
                         const void* v_new, int64_t v_stride, const int32_t* block_table,
                         void* kv8_pool, void* kv8_scales, hipStream_t stream);
pkv_status pkv_kv8_load(const pkv_problem* prob, const int32_t* tok_offsets, int32_t num_tokens,
                        const int32_t* seq_lens_dev, const int32_t* block_table,
                        const void* kv8_pool, const void* kv8_scales, void* k_out, void* v_out,
                        hipStream_t stream);

/*
 * Decode and prompt attention over the 8-bit cache: pkv_attend_kv4 and
 * pkv_prompt_kv4 with the scales beside the pool.  Decode has their split caps
 * and workspaces too.  A prompt's max_splits is the number of workgroups of a KV head
 * that its tiles are spread over, by even shares of all the work there is, whatever
 * tiles that cuts (1: a workgroup for each tile; no more than fill the current
 * device, and of 8 steps of 64 keys or more each).  pkv_prompt_kv8_splits and
 * pkv_prompt_kv8_workspace_bytes give its caps and workspaces, on the terms of
 * pkv_prompt_splits and pkv_prompt_workspace_bytes.
 */
pkv_status pkv_attend_kv8(const pkv_problem* prob, const pkv_view* view,
                          const int32_t* seq_lens_dev, int32_t max_splits, const void* q,
                          const void* kv8_pool, const void* kv8_scales,
                          const int32_t* block_table, void* workspace, size_t workspace_bytes,
                          void* out, float* lse, hipStream_t stream);
pkv_status pkv_prompt_kv8(const pkv_problem* prob, const pkv_view* view,
                          const int32_t* tok_offsets, int32_t num_tokens,
                          const int32_t* seq_lens_dev, int32_t max_splits, const void* q,
                          const void* kv8_pool, const void* kv8_scales,
                          const int32_t* block_table, void* workspace, size_t workspace_bytes,
                          void* out, float* lse, hipStream_t stream);

size_t pkv_prompt_kv8_workspace_bytes(const pkv_problem* prob, int32_t num_tokens,
                                      int32_t one_per_row, int32_t max_splits);
int32_t pkv_prompt_kv8_splits(const pkv_problem* prob, const pkv_view* view, int32_t num_tokens,
                              int32_t one_per_row, int32_t num_cus);

/*
 * Cross attention of num_tokens queries, ragged over the rows as tok_offsets says
 * (NULL: one per row, num_tokens = B), over 16-bit pages, the 4-bit or the 8-bit
 * pool.  q, out [num_tokens][Hq][d], lse [num_tokens][Hq] (may be NULL).  A query
 * of a row without tokens gets out = 0, lse = -inf.
 *   Calls of few queries a row (by num_tokens, B, Hq and Hkv alone) keep 16 or more bits of
 *   a weight in the second product, as decode does; calls of many round it to the
 *   problem's type, as prompts do.  Statistics and sums are held in fp32.
 *   max_splits: few queries: a tile cuts its keys into up to this many ranges; many:
 *     as pkv_prompt_kv8's.  pkv_cross_splits gives a cap that fills num_cus compute
 *     units (0 on an invalid argument).
 *   workspace: pkv_cross_workspace_bytes device bytes (0 for one split and where
 *     the call would be refused), on the terms of pkv_attend_window's; one_per_row
 *     says that the call passes no tok_offsets.  The size falls where calls become ones
 *     of many queries.  A call of few queries takes no more ranges than its workspace
 *     holds, so that of a larger step of the same problem, in two splits or more, does
 *     for it too; with all of its ranges only if it has its own size, the largest over
 *     the steps.
 * Errors: as pkv_prompt_window's, PKV_ENOSPC of few queries where the workspace does
 * not hold two ranges; PKV_ERANGE also where tiles of sixteen queries,
 * (num_tokens * G / 16 + B) * Hkv, times max_splits pass 2^24 - 1, or 65536 in splits.
 */
size_t pkv_cross_workspace_bytes(const pkv_problem* prob, int32_t num_tokens, int32_t one_per_row,
                                 int32_t max_splits);
int32_t pkv_cross_splits(const pkv_problem* prob, int32_t num_tokens, int32_t one_per_row,
                         int32_t num_cus);
pkv_status pkv_cross(const pkv_problem* prob, const int32_t* tok_offsets, int32_t num_tokens,
                     const int32_t* seq_lens_dev, int32_t max_splits, const void* q,
                     const void* k_pool, const void* v_pool, const int32_t* block_table,
                     void* workspace, size_t workspace_bytes, void* out, float* lse,
                     hipStream_t stream);
pkv_status pkv_cross_kv4(const pkv_problem* prob, const int32_t* tok_offsets, int32_t num_tokens,
                         const int32_t* seq_lens_dev, int32_t max_splits, const void* q,
                         const void* kv4_pool, const int32_t* block_table, void* workspace,
                         size_t workspace_bytes, void* out, float* lse, hipStream_t stream);
pkv_status pkv_cross_kv8(const pkv_problem* prob, const int32_t* tok_offsets, int32_t num_tokens,
                         const int32_t* seq_lens_dev, int32_t max_splits, const void* q,
                         const void* kv8_pool, const void* kv8_scales,
                         const int32_t* block_table, void* workspace, size_t workspace_bytes,
                         void* out, float* lse, hipStream_t stream);

/*
 * Give a step's new tokens their pages: counts [B] tokens for every row (below 0:
 * none), one row's behind the other's in the step's token-major arrays of
 * num_tokens rows.
 *   A row is served when its length and its new one lie in [0, max_pages_per_row *
 *   P], its tokens in the arrays (a row without any is never outside them), and the
 *   pages that it and the rows before it ask for in the free list; a row that needs
 *   no page is never short of them.  Served
 *   rows take pages from the top of the stack, in row order, into their tables, and
 *   grow by their counts; the others stay as they are.
 *   Written for the step's calls:
 *     seq_lens [B]: the length after the tokens, 0 for a row turned down (so that
 *       its tokens are not stored and its queries see nothing)
 *     tok_offsets [B + 1]: sums of counts, no higher than num_tokens
 *     slots int64 [num_tokens] (may be NULL): page * P + place of each token, -1
 *       for tokens of rows turned down and where the page lies outside the pool
 *     positions int32 [num_tokens] (may be NULL): its position in the row, -1 for
 *       tokens of rows turned down
 *   Entries of slots and positions behind the last offset are left as they were.
 * Errors: PKV_EINVAL (null pointer, num_tokens < 0), PKV_ESHAPE, PKV_EDTYPE (problem),
 * PKV_ERANGE (num_tokens above 2^30), PKV_EHIP.
 */
pkv_status pkv_pages_take(const pkv_problem* prob, const int32_t* counts, int32_t num_tokens,
                          int32_t* lens, int32_t* block_table, const int32_t* free_pages,
                          int32_t* state, int32_t* seq_lens, int32_t* tok_offsets, int64_t* slots,
                          int32_t* positions, hipStream_t stream);

/*
 * Cut every row down to keep[i] tokens (0: the row is done): the pages behind go
 * back on the stack, the last row's last page first, and their table entries
 * become -1.  A row that is no longer than that, or whose keep is negative, is left
 * alone.  After a pkv_pages_take, giving back what it took restores the stack.
 * Entries outside [0, num_pool_pages) do not go on the stack.  Pages that it has no
 * room for, these entries counted, are dropped (it has, unless a page was in two
 * tables).  Errors as above.
 */
pkv_status pkv_pages_release(const pkv_problem* prob, const int32_t* keep, int32_t* lens,
                             int32_t* block_table, int32_t* free_pages, int32_t* state,
                             hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* PKV_SERVING_H */
