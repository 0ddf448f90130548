/*
 * draftbranch.h -- C ABI for several branches of one context (drafts, samples,
 * beams) on MI355X (gfx950), in the same library as the draft head
 * (drafthead.h) and the draft layer's attention (draftlayer.h).
 *
 * Branches share the pages of what they have in common.  Between two steps the
 * next batch's page table is made from the present one (draft_branch_fork): a
 * sequence goes on as one branch, as several or as none, full pages are shared,
 * a partly filled one is copied, pages for the coming tokens are taken.  The
 * step's attention reads a shared prefix once for all its branches
 * (draft_branch_attend), and what the head says of their tokens is scored
 * (draft_branch_logprobs).  A pool that has become sparse is drawn together
 * (draft_branch_compact).
 *
 * The conventions are drafthead.h's: DH_OK or a negative DH_E* code, nothing
 * thrown, every argument checked before any HIP call, the caller owns every
 * buffer, device functions enqueue on `stream` and return without waiting,
 * draft_head_last_error() describes the last error of the calling thread.  The
 * cache and a batch are draftlayer.h's.
 *
 * The pages' counts: uses, device int32 [n_pages], says how many table entries
 * name each page (and holds one more for whatever else the caller keeps a page
 * for); a page with none is free, a count below 0 is taken as 0 and left as 0.
 * A table entry outside 0 .. n_pages - 1 names no page.  No input is written
 * except the pages of the pool that are said to be: both functions leave the new
 * table and counts in buffers of their own, so a call can be repeated, and the
 * caller then goes on with the new ones.
 *
 * Workspaces of this header need no initial contents and hold nothing between
 * calls; calls that share one must be ordered (one stream).
 */
#ifndef DRAFTBRANCH_H
#define DRAFTBRANCH_H

#include "draftlayer.h"

#ifdef __cplusplus
extern "C" {
#endif

#define DB_MAX_PAGES (1 << 24)
#define DB_MAX_TOP 64
#define DB_MAX_TOKENS 64
#define DB_MAX_VOCAB (1 << 24)
#define DB_BF16 0
#define DB_FP32 1

/*
 * Bytes of device workspace for draft_branch_fork (to at most n_new rows) and
 * draft_branch_compact over a pool of n_pages: one size serves both, and every
 * smaller pool and batch.
 * Errors: DH_EINVAL (null pointer), DH_ESHAPE.
 */
int draft_branch_pages_workspace_bytes(int n_pages, int n_new, size_t* bytes);

/*
 * DEVICE.  The next batch's page table from the present one.  Row s of the new
 * table goes on from the present sequence p = parents[s] with its len =
 * kv_len[p] tokens (0 .. max_pages*page); a parent outside 0 .. n_seq - 1 is
 * none: the row starts empty (len = 0).  It gets pages for `need[s]` positions
 * (at least len, at most max_pages*page).  With full = len / page and last =
 * ceil(max(need, len) / page), entry j of row s is
 *   j < full           the parent's entry, shared (-1 where that names no page)
 *   full <= j < last   the parent's entry, where it names a page that nothing
 *                      else names (uses = 1) and s is the first row with this
 *                      parent; else a free page
 *   j >= last          -1
 * The free pages are those with uses = 0 before the call (a page that the call
 * frees is free from the next call on); the lowest ids come first, to entries in
 * the order of (s, j).  Where tokens stand in the parent's page j = full (len no
 * multiple of page) and a free page takes its place, codes and scales of the
 * whole page are copied.  The counts give up every entry of the present table
 * and take on every entry of the new one: a present sequence that no row goes on
 * from is freed.
 * If fewer pages are free than asked for, nothing is done: no page is written,
 * uses_out is uses, and table_out is -1 throughout.
 *   k_codes .. v_scale  the pool, whose free pages take the copies
 *   table      int32 [n_seq][max_pages], kv_len int32 [n_seq]
 *   parents, need  int32 [n_new]
 *   uses_out   out, int32 [n_pages];  table_out  out, int32 [n_new][max_pages]
 *   status     out, int32 [2]: free pages after the call; pages that were lacking
 *              (the three, the int32 inputs, the cache and the workspace: none of
 *              these may overlap another, but for inputs among themselves)
 * Limits: 1 <= n_seq, n_new <= DL_MAX_SEQS, n_pages <= DB_MAX_PAGES, D, page,
 * heads and max_pages as in draftlayer.h, n_new * max_pages < 2^31.
 * Errors: DH_EINVAL, DH_ESHAPE, DH_EUNSUP, DH_EHIP.
 */
int draft_branch_fork(uint8_t* k_codes, uint8_t* v_codes, float* k_scale, float* v_scale, int n_pages, int page, int hkv,
                      int D, const int32_t* uses, const int32_t* table, const int32_t* kv_len, int n_seq,
                      const int32_t* parents, const int32_t* need, int n_new, int max_pages, int32_t* uses_out,
                      int32_t* table_out, int32_t* status, void* workspace, size_t workspace_bytes, void* stream);

/*
 * DEVICE.  Moves the pages in use (uses > 0) to the front of the pool: with
 * `used` of them, the k-th page in use at or behind `used` (in ascending order)
 * goes to the k-th free page before it, codes, scales and count.  The places
 * that pages leave keep their codes and have the count 0; pages from `used` on
 * are free then.  Entries of `table` that name a moved page name its new place,
 * all others stay as they are; it has to hold every row that names a page of
 * the pool, n_rows of them with max_pages entries each.
 *   uses_out  out, int32 [n_pages];  table_out  out, int32 [n_rows][max_pages]
 *   status    out, int32 [2]: pages in use; pages moved
 *             (what may not overlap: as in draft_branch_fork)
 * Limits: as draft_branch_fork's, n_rows in 1..DL_MAX_SEQS of any max_pages.
 * Errors: DH_EINVAL, DH_ESHAPE, DH_EUNSUP, DH_EHIP.
 */
int draft_branch_compact(uint8_t* k_codes, uint8_t* v_codes, float* k_scale, float* v_scale, int n_pages, int page,
                         int hkv, int D, const int32_t* uses, const int32_t* table, int n_rows, int max_pages,
                         int32_t* uses_out, int32_t* table_out, int32_t* status, void* workspace,
                         size_t workspace_bytes, void* stream);

/*
 * Bytes of device workspace for draft_branch_attend's calls of up to T rows of
 * up to n_seq sequences with these heads.  It has a place for every row's fp32 sums
 * four times: 40 heads on 8 of 128 ask for 103 MB for few rows, 443 MB for 4,096 and
 * 1,465 MB for 16,384.
 * Errors: DH_EINVAL (null pointer), DH_ESHAPE, DH_EUNSUP.
 */
int draft_branch_attend_workspace_bytes(int T, int n_seq, int hq, int hkv, int D, size_t* bytes);

/*
 * DEVICE.  draft_layer_attend for a batch whose sequences share prefixes.  The
 * sequences group_start[g] .. group_start[g+1] - 1 are a group and have the tokens
 * of the positions 0 .. prefix_len[g] - 1 in common: these are read from the pages
 * that the first sequence's table row names (group members' entries for whole pages
 * of them need not be there), those from prefix_len[g] on from each one's own.  A row
 * sees what it sees in draft_layer_attend, by its position, window and sinks,
 * whichever row the page is taken from; a token at a position that it does not
 * see stays unseen in a prefix too.  Sequences from group_start[n_groups] on have
 * no prefix.  Where the members' table rows name the pages of one prefix, as
 * draft_branch_fork leaves them, the result is draft_layer_attend's of the same
 * batch up to rounding.
 * A prefix is read once for all that share it, with two exceptions, where the
 * caches alone share it:
 *   short contexts  the table's width or the window leaves every row few tokens,
 *             and rows are few: one launch instead of two or three (heads of 128 up
 *             to 2,816 tokens, of 64 4,096, of 256 2,560)
 *   long members    a group whose members have on average 128 rows of query heads
 *             for a kv head (heads of 256: 64): each reads the prefix for itself,
 *             since the products bound such rows.  One long prompt among single
 *             tokens makes its group such a one: 600 rows and 15 of one row over
 *             20,480 tokens, 40 heads on 8 of 128, take 315 us, 278 if shared.
 * Where there is little to share, draft_layer_attend of the same batch is the faster
 * call: 16 prompts of 112 rows over 6,000 tokens 260 us there and 267 here, 204 and 242
 * with 16 heads on 2 of 256, 32 single rows of those under a window of 2,048 19.5 and
 * 26.3, 4 single rows over 1,000 tokens in a table for more than 2,816 11.0 and 15.9.
 *   group_start  device, int32 [n_groups + 1], not decreasing, 0 first, at most n_seq
 *   prefix_len   device, int32 [n_groups], any number of tokens (a negative one is 0)
 *   the other arguments, their limits, what is said of rows without a token to
 *   see, of values that are not finite, and the precision: as draft_layer_attend's;
 *   out, lse and the workspace must not overlap each other or an int32 input
 * Limits: 1 <= n_groups <= n_seq.
 * Errors: DH_EINVAL, DH_ESHAPE, DH_EUNSUP, DH_EHIP.
 */
int draft_branch_attend(const void* q, int64_t ldq, const uint8_t* k_codes, const uint8_t* v_codes,
                        const float* k_scale, const float* v_scale, int n_pages, int page, const int32_t* q_start,
                        const int32_t* kv_len, const int32_t* table, int n_seq, int max_pages,
                        const int32_t* group_start, const int32_t* prefix_len, int n_groups, int T, int hq, int hkv,
                        int D, float scale, int window, int sinks, void* out, float* lse, void* workspace,
                        size_t workspace_bytes, void* stream);

/*
 * Bytes of device workspace for draft_branch_logprobs' calls of up to M rows of
 * up to N logits with up to `top` alternatives.
 * Errors: DH_EINVAL (null pointer), DH_ESHAPE, DH_EUNSUP.
 */
int draft_branch_logprobs_workspace_bytes(int M, int N, int top, size_t* bytes);

/*
 * DEVICE.  Log probabilities under the softmax of rows of logits, such as
 * draft_head_forward_row's bf16 rows or draft_head_coarse's fp32 ones.  With
 * z_j = f x_j, f = scale * (scales ? scales[m] : 1), of row m:
 *   lse         = ln sum_j exp(z_j)
 *   logprob[t]  = z_tok - lse for each of the row's n_tok given tokens; -inf for
 *                 a token outside 0 .. N - 1 (another shard's)
 *   entropy     = sum_j p_j (lse - z_j), p_j = exp(z_j - lse)
 *   top_id, top_logprob  the `top` largest x_j of those above -inf, the larger
 *                 first, of equal ones the lower id first, and their log
 *                 probabilities; id -1 and -inf where the row has no more
 * A row without an element above -inf gets lse, logprob and top_logprob -inf,
 * entropy 0 and ids -1.  A row with a NaN or +inf element, or whose f is not > 0
 * or is too large (f log2(e) has to be below 2^128: f up to 2.35e38), gets NaN in
 * lse, logprob, entropy and top_logprob, and ids -1.
 * The shards of one vocabulary join by their lse: with L = ln sum_r exp(lse_r),
 * log probabilities fall by L - lse_r, and the entropy is
 * L - sum_r exp(lse_r - L) (lse_r - entropy_r).
 * Sums are fp32 under the running maximum; x is taken as it is, differences to
 * the maximum are rounded once, so rows at the type's lowest value are rows too.
 * A difference that is past fp32's largest number is infinite, whatever f: such an
 * element weighs nothing and its log probability is -inf.
 * Rows in which far more elements than `top` are equal to the top-th largest or
 * above it (constant rows) are passed over `top` times more: 72 rows of 124,160
 * equal elements take 66 us with 8 alternatives and 408 with 64, others 17.
 *   logits    device, bf16 (type DB_BF16) or fp32 (DB_FP32), row m at logits +
 *             m*ld elements, ld >= N; aligned to its element alone
 *   scales    device, fp32 [M], or NULL
 *   tokens    device, int32 [M][n_tok]; n_tok = 0: tokens and logprob unused
 *   logprob fp32 [M][n_tok], lse and entropy fp32 [M], top_id int32 [M][top],
 *             top_logprob fp32 [M][top]: out; top = 0: the last two unused
 *   workspace 16-byte aligned; may be NULL where the size asked for is 0
 * Limits: 0 <= M <= DL_MAX_ROWS (M = 0 does nothing), 1 <= N <= DB_MAX_VOCAB,
 * 0 <= top <= DB_MAX_TOP, 0 <= n_tok <= DB_MAX_TOKENS, scale finite and > 0.
 * Errors: DH_EINVAL, DH_ESHAPE, DH_EUNSUP, DH_EHIP.
 */
int draft_branch_logprobs(const void* logits, int type, int64_t ld, int M, int N, float scale, const float* scales,
                          const int32_t* tokens, int n_tok, int top, float* logprob, float* lse, float* entropy,
                          int32_t* top_id, float* top_logprob, void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* DRAFTBRANCH_H */
