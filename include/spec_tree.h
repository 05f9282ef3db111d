/*
 * spec_tree.h -- C ABI of speculation over trees of drafted tokens (same
 * library as spec_verify.h and spec_decode.h, libspecverify.so): attention for
 * a tree's nodes over the paged cache, keys rotated on their way into it, the
 * walk that accepts a path, and the move that keeps it.
 *
 * A tree of N nodes is the newest N tokens of its sequence: with n =
 * lengths[b], node i is cache token n - N + i.  parents[i] is the node's parent,
 * a lower index, -1 for a child of the tokens before the tree (the context), or
 * less for no node at all (a batch's smaller trees are padded with them).  A
 * node below one that is none is none.  A parent from the node's own index on is
 * SPEC_DATA_TREE_PARENT, and the node is none.
 *
 * One step of a server: spec_cache_append_rotated and spec_tree_attention per
 * layer, spec_filtered_sample on all nodes' logits, spec_tree_accept,
 * spec_cache_keep, spec_cache_fork with room for the next tree.
 *
 * The conventions of spec_decode.h hold, its page tables, caches and status
 * bits among them.
 */
#ifndef SPEC_TREE_H
#define SPEC_TREE_H

#include "spec_decode.h"

#ifdef __cplusplus
extern "C" {
#endif

#define SPEC_DATA_TREE_PARENT 1024 /* a node's parent at or behind itself: no node */
#define SPEC_DATA_PATH_RANGE 2048  /* spec_cache_keep: a path that does not ascend within the tree (ends there) */

#define SPEC_TREE_MAX_NODES 256

/*
 * spec_tree_attention -- attention of the N nodes of B trees over their
 * sequences' cached keys and values, the nodes' own among them.
 *
 *   q, cache, page_table, lengths, out, lse, scale: as spec_paged_attention's, with
 *            N nodes in the place of Q queries, 1 to SPEC_TREE_MAX_NODES.
 *   parents  [B, N] int32, rows parents_stride apart (at least N, or 0: one
 *            tree holds for every sequence).
 *   out must not overlap q.
 *   Node i sees the tokens before n - N, its ancestors and itself.  No node, or
 *   one before the sequence's first token (n < N), sees nothing: out = 0,
 *   lse = -inf.  Tokens that a node does not see never reach its result,
 *   whatever they hold.
 *   workspace: spec_tree_attention_workspace_size(...) bytes, the first
 *            SPEC_TREE_ATTENTION_ZERO_BYTES of them zero-filled once; every call
 *            leaves it fit for the next.  One call at a time.  (bf16 of more than 24
 *            rows N * Hq / heads: 21 MB for heads of 128, 11 for 64, twice that above 128
 *            rows; 7.6 and 3.9 MB else, whatever the batch.)
 *
 * Arithmetic as spec_paged_attention's; the result does not depend on the
 * schedule's timing.  As there, a value that is not finite in a token that a node
 * sees makes what it reaches not finite: whether infinite or NaN depends on the
 * sizes and on where the token lies, and is not promised.
 */
#define SPEC_TREE_ATTENTION_ZERO_BYTES 2048
SPEC_API size_t spec_tree_attention_workspace_size(int B, int N, int Hq, int heads, int head_dim, int dtype);
SPEC_API spec_status_t spec_tree_attention(
    const void* q, int64_t q_batch_stride, int64_t q_token_stride, int64_t q_head_stride,
    const spec_cache_t* cache, const int32_t* page_table, int64_t table_stride, int max_pages,
    const int32_t* lengths, const int32_t* parents, int64_t parents_stride, int B, int N, int Hq,
    float scale, void* out, float* lse, void* workspace, size_t workspace_bytes,
    spec_stream_t stream, int32_t* device_status);

/*
 * spec_cache_append_rotated -- spec_cache_append with the position rotation
 * applied on the way: new keys are rotated and written into their pages, values
 * are written as they are, and the tokens' queries are rotated too.
 *
 *   k_new, v_new, starts, cache, page_table, lengths: as spec_cache_append's.
 *   q        [T, q_heads, head_dim], rows q_stride elements apart, or NULL (q_heads 0);
 *   q_out    their rotated rows, q_out_stride apart: q itself at its stride, whose
 *            rows share no byte with k_new's and v_new's (of the same stride they may lie
 *            in one another's gaps, as slices of a fused projection do), or memory
 *            that overlaps neither q's, k_new's nor v_new's.
 *   positions [T] int32: the tokens' positions (of a tree's node: the context's
 *            tokens and its depth); NULL: their places in their sequences.
 *   inv_freq [n_freq] fp32, finite: the angle of pair i at position p is
 *            p * inv_freq[i] radians.  Pair i is dimensions i and n_freq + i, or with
 *            `interleaved` 2i and 2i + 1; (x, y) becomes (x cos - y sin, y cos +
 *            x sin).  Dimensions from 2 n_freq on stay.  head_dim a multiple of 8
 *            up to 256, n_freq a multiple of 8 with 2 n_freq <= head_dim.
 * Angles are reduced in fixed point, to 2^-31 of a turn for every position and frequency;
 * sines and cosines are within 2^-23; products and sums are fp32, rounded once.
 * Rows that no sequence claims are SPEC_DATA_LENGTH_RANGE, and zero in q_out
 * unless it is q (then they stay).  A token without a place or page (the bits of
 * spec_cache_append) is not written; its query is rotated all the same.
 */
SPEC_API spec_status_t spec_cache_append_rotated(
    const void* k_new, const void* v_new, int64_t new_stride, int T, const int32_t* starts,
    const void* q, int64_t q_stride, int q_heads, void* q_out, int64_t q_out_stride,
    const int32_t* positions, const float* inv_freq, int n_freq, int interleaved,
    const spec_cache_t* cache, const int32_t* page_table, int64_t table_stride, int max_pages,
    const int32_t* lengths, int B, spec_stream_t stream, int32_t* device_status);

/*
 * spec_tree_accept -- the path that the target's tokens take through each tree.
 *
 *   tokens   [B, N] int32: the nodes' tokens; node 0 (parent -1) is the root, the
 *            token that the step before emitted.  N is 0 to SPEC_TREE_MAX_NODES.
 *   parents  [B, N], rows parents_stride apart (at least N, or 0).
 *   drawn    [B, N] int32: the target's token after each node (sampled or its argmax).
 *   The walk starts at node 0 and goes on to the child whose token is the one drawn
 *   after the node (of equal ones the lowest index) until there is none.
 *   accepted_len [B]: nodes behind the root on the walk.
 *   path     [B, N]: the walk's nodes, the root first, then -1.
 *   out_tokens [B, N]: the tokens drawn after them (accepted_len accepted ones and
 *            the one that ends the walk), then -1.
 *   Where node 0 is no root: accepted_len -1 and nothing but -1.
 *   The outputs overlap nothing, but path and out_tokens may each be one of the
 *   inputs itself (not parents that trees share).
 * With tokens drawn from the target's distribution at each node, what is emitted
 * follows that distribution whatever the tree holds.
 */
SPEC_API spec_status_t spec_tree_accept(const int32_t* tokens, const int32_t* parents, int64_t parents_stride,
                                        const int32_t* drawn, int B, int N, int32_t* accepted_len,
                                        int32_t* out_tokens, int32_t* path, spec_stream_t stream,
                                        int32_t* device_status);

/*
 * spec_cache_keep -- of each sequence's newest N tokens keeps those of a path:
 * token n - N + path[j] moves to n - N + j, all layers, in place.
 *
 *   path     [B, N] int32: ascending indexes below N, ended by -1 (spec_tree_accept's).
 *            An entry that does not ascend, or is not below N, is
 *            SPEC_DATA_PATH_RANGE and ends the path.
 *   new_lengths [B] = lengths - N + entries (not below 0); overlaps neither lengths,
 *            path nor page_table.  A path in a sequence of fewer than N tokens is SPEC_DATA_LENGTH_RANGE:
 *            the sequence stays as it is.
 * The pages that hold the newest N tokens must be the sequence's own (those that
 * spec_cache_fork reserves are).  A token whose page, or the page it goes to,
 * is out of range does not move (SPEC_DATA_PAGE_RANGE).
 */
SPEC_API spec_status_t spec_cache_keep(const spec_cache_t* cache, const int32_t* page_table,
                                       int64_t table_stride, int max_pages, const int32_t* lengths, int B,
                                       const int32_t* path, int N, int32_t* new_lengths,
                                       spec_stream_t stream, int32_t* device_status);

#ifdef __cplusplus
}
#endif

#endif /* SPEC_TREE_H */
