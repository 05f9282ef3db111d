/*
 * spec_decode.h -- C ABI of the decode-side operators around the verify step
 * (same library as spec_verify.h, libspecverify.so): attention over a paged
 * key-value cache, the cache's page handling, and sampling from truncated
 * distributions.
 *
 * The conventions of spec_verify.h hold: device pointers of the current CUDA
 * device, buffers owned by the caller, calls asynchronous on `stream`,
 * argument errors returned before any launch, data errors OR-ed into an
 * optional device status word; nothing allocates, traps, prints or waits for
 * the device.
 */
#ifndef SPEC_DECODE_H
#define SPEC_DECODE_H

#include "spec_verify.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Device status bits of these operators (next to those of spec_verify.h). */
#define SPEC_DATA_PAGE_RANGE 64    /* a page table entry in use outside [0, pages): its tokens are skipped */
#define SPEC_DATA_LENGTH_RANGE 128 /* a length, start, parent or kept length out of range (clamped) */
#define SPEC_DATA_CACHE_FULL 256   /* spec_cache_fork: fewer free pages than asked for (-1 entries) */
#define SPEC_DATA_PARAM_RANGE 512  /* a temperature, top-p or min-p that is NaN or out of range (off) */

/*
 * A paged key-value cache: `layers` x `pages` pages of `page_size` tokens.
 * Token t of page p of layer l lies at element l * layer_stride +
 * p * page_stride + t * token_stride of k and of v, and holds
 * [heads, head_dim] values contiguously.  The strides (elements) are free --
 * [layers, pages, page_size, heads, head_dim], a [pages, 2, page_size, ...]
 * interleaving of K and V, one layer of a larger cache -- as long as every
 * token starts on a 16-byte boundary and tokens do not overlap.
 */
typedef struct {
  void* k;
  void* v;
  int64_t layer_stride, page_stride, token_stride;
  int layers, pages, page_size, heads, head_dim;
  int dtype; /* spec_dtype_t */
} spec_cache_t;

/*
 * spec_paged_attention -- attention of the newest Q tokens of B sequences
 * (Q = 1: a decode step; Q = K+1: the target's pass over K drafted tokens and
 * the one before them) over their cached keys and values, the new tokens'
 * own among them (spec_cache_append comes first).
 *
 *   q        [B, Q, Hq, D] with strides in elements (last dimension
 *            contiguous, rows 16-byte aligned), cache's dtype.  Query head h
 *            reads cache head h / (Hq / heads); Hq is a multiple of heads.
 *   cache    one layer (layers == 1), head_dim D 64 or 128.
 *   page_table [B, max_pages] int32, rows table_stride apart (at least
 *            max_pages, or 0: one row holds for every sequence): the page of
 *            token t of sequence b is entry t / page_size of row b.  Entries
 *            past the sequence's length are not read.
 *   lengths  [B] int32: tokens of sequence b, the Q new ones included.
 *   Query i of sequence b stands at position n = lengths[b] - Q + i and sees
 *   tokens 0..n:  out = sum_t softmax_t(scale * q.k_t) v_t,
 *   lse = ln sum_t exp(scale * q.k_t).  A query that sees nothing (n < 0)
 *   gets out = 0, lse = -inf.  Tokens that a query does not see never reach
 *   its result, whatever they hold.
 *   out      [B, Q, Hq, D] contiguous, cache's dtype; lse [B, Q, Hq] fp32 or NULL.
 *   workspace: spec_attention_workspace_size(...) bytes, the first
 *            SPEC_ATTENTION_ZERO_BYTES of them zero-filled once; every call
 *            leaves it fit for the next.  One call at a time.  (30 MB for bf16
 *            heads of 128, 15 for 64, 8 and 4 for fp32, whatever the batch.)
 *
 * Scores, softmax and sums are fp32 (exponentials by ex2.approx, within 2^-22;
 * bf16: products of bf16 pairs summed in fp32; a weight exp(...) multiplies v
 * as the sum of two bf16 values, 2^-17; fp32: operands enter products as two
 * parts of 11 bits, which leaves out 2^-22 of a term), and the output is
 * rounded once.  Sums are divided at the end, of weights of up to 2^8: values
 * from about 2^119 / tokens on may overflow in them.  A value that is not finite in a
 * token that a query sees makes what it reaches not finite (infinite or NaN).
 * The result does not depend on the schedule's timing: partial results are
 * joined in a fixed order.
 */
#define SPEC_ATTENTION_ZERO_BYTES 2048
SPEC_API size_t spec_attention_workspace_size(int B, int Q, int Hq, int heads, int head_dim, int dtype);
SPEC_API spec_status_t spec_paged_attention(
    const void* q, int64_t q_batch_stride, int64_t q_token_stride, int64_t q_head_stride,
    const spec_cache_t* cache, const int32_t* page_table, int64_t table_stride, int max_pages,
    const int32_t* lengths, int B, int Q, int Hq, float scale, void* out, float* lse,
    void* workspace, size_t workspace_bytes, spec_stream_t stream, int32_t* device_status);

/*
 * spec_cache_append -- writes new tokens' keys and values into their pages.
 *
 *   k_new, v_new [T, heads, head_dim] (rows new_stride elements apart, 16-byte
 *            aligned), cache's dtype; one layer.
 *   starts   [B+1] int32: sequence b's new tokens are rows starts[b] ..
 *            starts[b+1]-1; NULL: T / B rows each (T a multiple of B).
 *   lengths  [B]: tokens of sequence b with the new ones; they go to
 *            positions lengths[b] - count .. lengths[b] - 1.
 */
SPEC_API spec_status_t spec_cache_append(
    const void* k_new, const void* v_new, int64_t new_stride, int T, const int32_t* starts,
    const spec_cache_t* cache, const int32_t* page_table, int64_t table_stride, int max_pages,
    const int32_t* lengths, int B, spec_stream_t stream, int32_t* device_status);

/*
 * spec_cache_fork -- the next step's C sequences from the current B: forking,
 * trimming, ending, reordering and reserving in one call.
 *
 *   parents  [C] int32: new sequence c continues sequence parents[c] (-1: a
 *            new, empty one), keeping its first keep[c] tokens.  Current
 *            sequences that nobody names end; their pages become free.
 *   room     tokens to reserve pages for beyond the kept ones.
 *   new_table [C, max_pages]: pages that the kept tokens fill are shared.  A
 *            partly filled last page stays with the first sequence (lowest c)
 *            that ends in it when nobody holds it as a full page; every other
 *            sequence that ends in it gets a page of its own and a copy of
 *            the kept tokens (all layers).  Further pages are reserved up to
 *            keep + room tokens.  New pages are the free pages in ascending
 *            order, given out by sequence, then position.  Unused entries are -1.
 *   new_lengths [C] = keep; ref_counts [pages]: references to each page by
 *            new_table; free_pages [pages]: the pages without, ascending, then
 *            -1; n_free [1].
 *   A parent out of range, or keep outside [0, its length], is
 *   SPEC_DATA_LENGTH_RANGE and keeps nothing; entries for tokens beyond
 *   max_pages * page_size are dropped with the same bit.
 * page_table and lengths are not changed; the outputs must not overlap them.
 * No page that new_table shares is written, and no page is both copied from
 * and written, so the call can be repeated.
 *   workspace: spec_cache_fork_workspace_size(...) bytes, any content.
 */
SPEC_API size_t spec_cache_fork_workspace_size(int pages, int C);
SPEC_API spec_status_t spec_cache_fork(
    const spec_cache_t* cache, const int32_t* page_table, int64_t table_stride, int max_pages,
    const int32_t* lengths, int B, const int32_t* parents, const int32_t* keep, int C, int room,
    int32_t* new_table, int32_t* new_lengths, int32_t* ref_counts, int32_t* free_pages,
    int32_t* n_free, void* workspace, size_t workspace_bytes, spec_stream_t stream,
    int32_t* device_status);

/*
 * spec_cache_compact -- moves the pages in use to the front of the pool: with
 * n pages in use, the i-th used page at or above n moves to the i-th unused
 * page below n (all layers); the others stay.
 *
 *   page_table [B, max_pages]: entries >= 0 are in use (shared ones once).
 *   new_table [B, max_pages], ref_counts [pages] (by the new numbers),
 *   n_live [1] = n.  Pages n.. are free afterwards.
 *   workspace: spec_cache_compact_workspace_size(...) bytes, any content.
 */
SPEC_API size_t spec_cache_compact_workspace_size(int pages);
SPEC_API spec_status_t spec_cache_compact(
    const spec_cache_t* cache, const int32_t* page_table, int64_t table_stride, int max_pages,
    int B, int32_t* new_table, int32_t* ref_counts, int32_t* n_live, void* workspace,
    size_t workspace_bytes, spec_stream_t stream, int32_t* device_status);

/*
 * spec_filtered_sample -- one token per row from its truncated softmax.
 *
 * With M the row's largest logit, a token's weight is the integer
 *   w_j = round(2^40 * 2^t_j),  t_j = max((x_j - M) * (log2(e) / T), -64),
 * each operation rounded to fp32, 2^t by the fixed polynomial of
 * filtered_sample.cu; every sum, cut and draw below is exact integer
 * arithmetic, so results do not depend on the order of summation.
 *   1. the top_k largest logits (ties: lower index first); <= 0 or >= V: all
 *   2. of these, w_j >= round(2^40 * min_p)       (min_p <= 0: all)
 *   3. of these, in order of descending logit (ties: lower index first), the
 *      shortest run whose sum reaches max(1, floor(top_p * total)); >= 1: all
 *   4. the draw: with S the sum of the kept weights, the token with the
 *      lowest index j whose running sum (by index) exceeds floor(u * S).
 * T == 0 (or below 2^-100) keeps the largest logit alone (lowest index among
 * equals).  Tokens of weight 0 are never kept.
 *
 *   logits   [R, V] dtype, rows row_stride elements apart.
 *   uniforms [R] fp32 in [0, 1).
 *   temperatures, top_ks, top_ps, min_ps  [R] or NULL: then the scalar
 *            holds for every row.
 *   tokens   [R] int32; p [R] fp32 = w / S, the token's probability in the
 *            kept distribution (NULL: not wanted); n_kept [R] int32 or NULL.
 *   filtered [R, V] contiguous dtype or NULL: the logits of the kept tokens,
 *            -inf elsewhere -- rows that spec_verify takes as target or draft
 *            logits, so that both sides of the ratio test are truncated.
 *            They may be the logits themselves (row_stride V), and must not
 *            overlap them otherwise.
 *   workspace: spec_filtered_sample_workspace_size(...) bytes (0 for small
 *            calls: NULL), the first SPEC_SAMPLE_ZERO_BYTES of them zero-filled
 *            once; every call leaves it fit for the next.  One call at a time.
 *            (24.6 KB a row, for 4096 rows and more 101 MB.)
 * A row with a NaN or +inf or without a finite logit is
 * SPEC_DATA_NONFINITE_LOGIT: token 0, p 0, n_kept 0, filtered -inf.  A row
 * whose copy into shared memory did not land within the kernel's limit on its
 * waits (SPEC_DEVICE_WAIT_TIMEOUT) gets the same.
 */
#define SPEC_SAMPLE_ZERO_BYTES 64
SPEC_API size_t spec_filtered_sample_workspace_size(int R, int V, int dtype);
SPEC_API spec_status_t spec_filtered_sample(
    const void* logits, int64_t row_stride, const float* uniforms, int R, int V, int dtype,
    float temperature, int top_k, float top_p, float min_p, const float* temperatures,
    const int32_t* top_ks, const float* top_ps, const float* min_ps, int32_t* tokens, float* p,
    int32_t* n_kept, void* filtered, void* workspace, size_t workspace_bytes,
    spec_stream_t stream, int32_t* device_status);

#ifdef __cplusplus
}
#endif

#endif /* SPEC_DECODE_H */
