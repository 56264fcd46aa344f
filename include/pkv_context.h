/*
 * pkv_context.h -- what a decode engine reads besides the whole 16-bit
 * context: a sliding window with sinks, prompts, and a cache held in 4 bits.
 * Part of libpkv; the conventions of pkv.h (ownership, streams, errors,
 * layouts, pkv_problem) hold here too.
 *
 * View.  The query at position p (0-based) sees token t when t <= p and
 *     window == 0, or t > p - window, or t < sinks:
 * the last `window` tokens, its own included, and the first `sinks` tokens.
 * A null view sees everything up to p.
 *
 * Runs.  Calls that take tok_offsets handle several new tokens per row: row i
 * has n_i = tok_offsets[i+1] - tok_offsets[i] of them, stored one after the
 * other at rows tok_offsets[i] .. of the token-major arrays, at positions
 * N_i - n_i .. N_i - 1, with N_i = seq_lens[i] the length AFTER them.
 * tok_offsets: int32 [B + 1] on the device, non-decreasing, first entry 0,
 * last entry at most num_tokens; rows of the token-major arrays behind the
 * last offset are neither read nor written.
 *
 * On the device, where the host cannot check: a row whose length lies outside
 * [0, max_pages_per_row * P] is treated as empty; a new token at a negative
 * position is not stored, and as a query it sees nothing; a block-table entry
 * outside [0, num_pool_pages) holds no tokens (they are not stored, not seen,
 * and not read back); offsets outside [0, num_tokens] are clamped to it.  A
 * query that sees nothing gets out = 0, lse = -inf.  Tokens that no query of
 * a row sees may hold anything, NaN and infinities included; a NaN or an
 * infinity in a token that one query of a row sees may also reach other queries
 * of that row (never other rows).
 * Scores, scale <q, k>, are held in fp32 and have to stay below 2^23 in magnitude,
 * where neighbouring numbers are still 1/2 apart.
 *
 * 4-bit cache (kv4).  K and V share one pool, bytes
 *     kv4_pool [num_pool_pages][Hkv][17 d],
 * 16-byte aligned.  A block is 32 consecutive channels of one token and head.
 * With a = max |x| over the block, its scale is 2^e, e = floor(log2 a) - 2,
 * one more where a > 7 * 2^e, kept in [-23, 13] (PKV_F16) or [-120, 125]
 * (PKV_BF16); its elements are x / 2^e rounded to nearest-even among 0 .5 1
 * 1.5 2 3 4 6 and their negatives, saturating at 6: no element is off by more
 * than 2^e unless its magnitude passes 7 * 2^13 (7 * 2^125).  The value it
 * stands for is exact in the problem's type.  A block that holds an
 * infinity or a NaN reads back as NaN.  Byte order of a page: csrc/context/
 * kv4_common.h.  One pool serves one dtype.
 */
#ifndef PKV_CONTEXT_H
#define PKV_CONTEXT_H

#include "pkv.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct pkv_view {
  int32_t window; /* visible last tokens, 0 = all                        */
  int32_t sinks;  /* first tokens that stay visible, >= 0                */
} pkv_view;

/* Bytes of one page of one KV head in the 4-bit cache (K and V): 17 d; 0 for
 * a head size that is neither 64 nor 128. */
size_t pkv_kv4_page_bytes(int32_t head_dim);

/*
 * Write a run of new tokens: every row's tokens at positions N_i - n_i ..
 * N_i - 1 go through the block table into the 16-bit pools (pkv_store_kv) or,
 * quantised as they are written, into the 4-bit pool (pkv_kv4_store).
 *   k_new, v_new: [num_tokens] rows of Hkv * d elements, k_stride / v_stride
 *     elements apart (at least Hkv * d, a multiple of 8), 16-byte aligned:
 *     a slice of a fused projection's output can be passed in place.
 *   tok_offsets: NULL means one token per row (num_tokens = B).
 * Other tokens of a touched page keep their bytes.  Two tokens of one call
 * that share a page slot race.
 * Errors: PKV_EINVAL (null pointer, negative num_tokens, num_tokens != B
 * without tok_offsets), PKV_ESHAPE (problem; a stride or an alignment),
 * PKV_EDTYPE, PKV_ERANGE (more than 2^24 - 1 workgroups: (num_tokens / 16 + 2 B)
 * * Hkv), PKV_EHIP.  num_tokens = 0 does nothing.
 */
pkv_status pkv_store_kv(const pkv_problem* prob, const int32_t* tok_offsets, int32_t num_tokens,
                        const int32_t* seq_lens_dev, const void* k_new, int64_t k_stride,
                        const void* v_new, int64_t v_stride, const int32_t* block_table,
                        void* k_pool, void* v_pool, hipStream_t stream);
pkv_status pkv_kv4_store(const pkv_problem* prob, const int32_t* tok_offsets, int32_t num_tokens,
                         const int32_t* seq_lens_dev, const void* k_new, int64_t k_stride,
                         const void* v_new, int64_t v_stride, const int32_t* block_table,
                         void* kv4_pool, hipStream_t stream);

/*
 * Read a run back: the values the 4-bit cache stands for, in the problem's
 * type, k_out, v_out: [num_tokens][Hkv][d].  Arguments and errors as
 * pkv_kv4_store; rows of tokens that are not in the cache (above) are left as
 * they were.
 */
pkv_status pkv_kv4_load(const pkv_problem* prob, const int32_t* tok_offsets, int32_t num_tokens,
                        const int32_t* seq_lens_dev, const int32_t* block_table,
                        const void* kv4_pool, void* k_out, void* v_out, hipStream_t stream);

/*
 * Decode attention of one query token per row (position N_i - 1) over the
 * visible part of the cache: pkv_attend_window reads 16-bit pages,
 * pkv_attend_kv4 the 4-bit pool.  Only pages that hold a visible token are
 * read.  Each row's list of visible pages is cut into up to max_splits equal
 * ranges, ceil(T_max / s) pages each with T_max the longest row's list and s the
 * least of max_splits and what pkv_attend_splits gives where a table holds T_max
 * pages (so short rows under a wide table stay whole), or more pages where the
 * ranges then fill the compute units of the current device evenly.
 *   workspace: at least pkv_attend_workspace_bytes(prob, max_splits) bytes of
 *     device memory, 16-byte aligned, the first 256 KiB (one counter for each of
 *     65536 pairs of row and KV head) zero before the first call that uses it;
 *     every call leaves them zero.  Calls of any problems, prompts included, may use
 *     one workspace in turn; calls that overlap on it race, two replays of
 *     captured graphs included.
 *   out [B][Hq][d], lse [B][Hq] (may be NULL) as in pkv.h; softmax statistics
 *     and sums are held in fp32.
 * pkv_problem.kernel is ignored.  Every G <= 16 is covered at both head sizes.
 * Errors: PKV_EINVAL (null pointer, a window or sinks < 0, max_splits outside
 * [1, 65535]), PKV_ESHAPE (problem, a misaligned pointer), PKV_EDTYPE,
 * PKV_ENOSPC (workspace too small), PKV_ERANGE (B or Hq above 65535, more than
 * 2^24 - 1 tasks B * Hkv * max_splits, or more than 65536 pairs B * Hkv in more
 * than one split), PKV_EHIP.  pkv_attend_workspace_bytes gives 0 where the call would be refused.
 */
size_t pkv_attend_workspace_bytes(const pkv_problem* prob, int32_t max_splits);
pkv_status pkv_attend_window(const pkv_problem* prob, const pkv_view* view,
                             const int32_t* seq_lens_dev, int32_t max_splits, const void* q,
                             const void* k_pool, const void* v_pool, const int32_t* block_table,
                             void* workspace, size_t workspace_bytes, void* out, float* lse,
                             hipStream_t stream);
pkv_status pkv_attend_kv4(const pkv_problem* prob, const pkv_view* view,
                          const int32_t* seq_lens_dev, int32_t max_splits, const void* q,
                          const void* kv4_pool, const int32_t* block_table, void* workspace,
                          size_t workspace_bytes, void* out, float* lse, hipStream_t stream);

/*
 * Split cap for the two calls above: enough ranges to fill num_cus compute
 * units with the batch's (row, KV head) pairs when every row is as long as
 * the block table (or the view) lets it be.  Host only; 0 on an invalid
 * argument (num_cus 1..1024).
 */
int32_t pkv_attend_splits(const pkv_problem* prob, const pkv_view* view, int32_t num_cus);

/*
 * Prompt attention: every new token of every row is a query, causal, with the
 * view applied at its own position; keys and values, the new tokens' included,
 * come from the cache (store them first).
 *   q, out [num_tokens][Hq][d], lse [num_tokens][Hq] (may be NULL), token-major
 *   as tok_offsets says (NULL: one token per row, num_tokens = B).
 * P enters the second product rounded to the problem's type; statistics and
 * sums are held in fp32.
 *   max_splits: a tile of 128 query rows (tokens times heads of a group) cuts
 *     its keys into up to this many ranges, for few queries over long contexts:
 *     no more than fill the current device with the tiles there are, and of 512
 *     keys or more each (a tile's last one aside); 1 needs no workspace.
 *     pkv_prompt_splits gives a cap that fills num_cus compute units (0 on an
 *     invalid argument).
 *   workspace: pkv_prompt_workspace_bytes device bytes (0 for one split and
 *     where the call would be refused), on the terms of pkv_attend_window's;
 *     one_per_row says that the call passes no tok_offsets.
 * Errors: PKV_EINVAL, PKV_ESHAPE, PKV_EDTYPE, PKV_ENOSPC as above, PKV_ERANGE
 * (more than 2^24 - 1 workgroups (num_tokens * G / 128 + B) * Hkv * max_splits, or
 * more than 65536 tiles of KV heads in splits), PKV_EHIP.
 */
size_t pkv_prompt_workspace_bytes(const pkv_problem* prob, int32_t num_tokens,
                                  int32_t one_per_row, int32_t max_splits);
int32_t pkv_prompt_splits(const pkv_problem* prob, const pkv_view* view, int32_t num_tokens,
                          int32_t one_per_row, int32_t num_cus);
pkv_status pkv_prompt_window(const pkv_problem* prob, const pkv_view* view,
                             const int32_t* tok_offsets, int32_t num_tokens,
                             const int32_t* seq_lens_dev, int32_t max_splits, const void* q,
                             const void* k_pool, const void* v_pool, const int32_t* block_table,
                             void* workspace, size_t workspace_bytes, void* out, float* lse,
                             hipStream_t stream);
pkv_status pkv_prompt_kv4(const pkv_problem* prob, const pkv_view* view,
                          const int32_t* tok_offsets, int32_t num_tokens,
                          const int32_t* seq_lens_dev, int32_t max_splits, const void* q,
                          const void* kv4_pool, const int32_t* block_table, void* workspace,
                          size_t workspace_bytes, void* out, float* lse, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* PKV_CONTEXT_H */
