/*
 * pace_draft.h -- C ABI of the operators that serve drafted tokens through a hybrid stack, next
 * to the gated-delta layers of pace.h and the attention layers of pace_cache.h, for AMD Instinct
 * MI355X (gfx950).  One step of a stack that drafts T tokens for each sequence (a chain or a tree):
 *
 *   every gated-delta layer   pace_draft_step: outputs of all drafts, the layer left as it is
 *   every attention layer     pace_cache_write, pace_cache_attention with the tree (pace_cache.h)
 *   once                      pace_draft_verify: which path is accepted, and the token after it
 *   every gated-delta layer   pace_draft_commit: the accepted tokens into its decode buffer
 *   every attention layer     pace_cache_move: the accepted entries to their final positions
 *
 * What is accepted (nodes, counts) stays on the device from one call to the next, so the whole step
 * may be captured in one HIP graph.  pace_cache_move also compacts a cache after entries
 * were dropped and copies sequences into other pages.
 *
 * The conventions are those of pace.h and pace_cache.h: plain C, caller-owned device memory,
 * host-side validation before any launch (PACE_EINVAL / PACE_EUNSUPPORTED, nothing touched),
 * launch errors as PACE_EHIP, no global state, no allocation and no synchronisation.  A call of several launches ends
 * at the first error, and what it writes is then lost: pace_draft_commit may leave a layer's buffer full and not yet
 * folded, which no other call takes for what it is, so the layer's state and buffer have to be set up anew.  Every
 * call only enqueues kernels on `stream` (a hipStream_t, NULL = default stream).  Memory handed to a
 * call, its workspace among it, must not be used by other work until the call's kernels have run:
 * calls that may overlap (other streams, other graphs) need workspaces of their own.
 *
 * Drafts: T nodes a sequence; node 0 is the token that was sampled last (its place is settled, it
 * has not gone through the layers yet), the others hang below it.  parents[i] < i.
 */
#ifndef PACE_DRAFT_H
#define PACE_DRAFT_H

#include "pace.h"
#include "pace_cache.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------ gated-delta layers: outputs of drafts */

/* o of T drafted tokens of every sequence, from the layer's packed state and its decode buffer, which
 * are read and left as they are.  Token i passes through the buffer quantiser (as every decoded
 * token does, pace.h) and sees the state, the buffered tokens, the tokens j < i of its own row
 * of `tree`, and itself:
 *     u_i = beta_i (v_i - a_i S_p^T k_i),   S_i = a_i S_p + k_i u_i^T,   o_i = S_i^T q_i,
 * S_p the state after the last token j of its row (after the buffer where there is none).
 *     tree == NULL:  every j < i (a chain; a single token)
 *     else:          bit j of tree[b * tree_stride + i * ceil(T / 32) + j / 32] (uint32 words on the device,
 *                    as of pace_tree_bits; tree_stride in words, 0: one tree for all sequences).
 * Rows have to be paths: with bit j, row i has the bits of row j.  (Others give numbers, of the sums that the bits say.)
 * No rounding of the state falls between drafts: a path that passes the end of the decode period sees
 * the state as it stands, and is rounded when it is committed.
 * draft_lens int32 [B] (device, NULL = T): sequence b has draft_lens[b] tokens; rows behind them may hold anything (they
 * may be loaded, but no result depends on them), and their o is 0.
 * q, k [B][T][Hk][dk];  v, o [B][T][Hv][dv];  a, beta fp32 [B][T][Hv], contiguous, 16-byte aligned
 * (a, beta: 4-byte).  o must not overlap an input.
 * Every state and buffer kind of pace.h; keys enter as exact codes, products and sums are fp32.
 * As in pace.h, gates lie in 0 < a <= 1, 0 <= beta <= 1, and NaN / Inf inputs are undefined.
 * A result repeats bit for bit and does not depend on the other sequences.
 * Errors: PACE_EINVAL for null pointers, T < 1, a negative tree_stride, misalignment; PACE_EUNSUPPORTED for
 * T > 64 or what pace_decode_step does not take. */
pace_status pace_draft_step(const pace_layer_cfg* cfg, const void* state, const void* buffer,
                            const void* q, const void* k, const void* v, const float* a,
                            const float* beta, int32_t T, const int32_t* draft_lens,
                            const uint32_t* tree, int64_t tree_stride, void* o, void* stream);

/* Takes the accepted tokens nodes[b][0 .. counts[b]) of the drafts into the layer: the state, the buffer's counts and the
 * slots below them end as after pace_decode_step of these tokens one by one, bit for bit; no outputs are formed.
 * (Tokens go to the buffer; where a buffer comes to hold dP tokens the state is rounded.)
 * nodes int32 [B][T] (device, rows of T): indexes into the drafts' tokens in the order in which they are taken; a row
 * ends at its first index outside [0, T).  counts int32 [B] (device): taken as 0 below 0, as `most` above it.
 * most (host, 1 <= most <= T): upper bound of the counts; 1 + 2 ceil(most / dP) launches are made.
 * k, v, a, beta: as of pace_draft_step (T <= 64).
 * workspace: pace_draft_commit_workspace_bytes(cfg, most) bytes, 256-byte aligned.
 * Errors: as pace_draft_step; PACE_EINVAL also for most outside [1, T] and a workspace that is too small. */
pace_status pace_draft_commit(const pace_layer_cfg* cfg, void* state, void* buffer, const void* k,
                              const void* v, const float* a, const float* beta, int32_t T,
                              const int32_t* nodes, const int32_t* counts, int32_t most,
                              void* workspace, size_t workspace_bytes, void* stream);

/* Workspace bytes of pace_draft_commit, written to *bytes_out.  Host only.
 * Errors (nothing is written) as pace_draft_commit. */
pace_status pace_draft_commit_workspace_bytes(const pace_layer_cfg* cfg, int32_t most,
                                              size_t* bytes_out);

/* ------------------------------------------------------------ verification of drafts */

/* 1 <= B <= 65535, 1 <= T <= 1024 nodes, 1 <= V <= 2^24 tokens. */
typedef struct {
  int32_t B, T, V;
  int32_t prob_dtype;    /* pace_io_dtype of target and draft */
} pace_verify_cfg;

/* Which of the drafted tokens are accepted, so that the accepted ones and the token that follows
 * are distributed as the target's, and that following token, from given random numbers.
 *
 * target [B][T][V]: row i holds the probabilities of the token after node i.  draft [B][T][V]: row i
 * the probabilities from which the children of node i were drawn, independently; NULL: the children were not drawn (the
 * likeliest tokens, a lookup).  tokens int32 [B][T]: the nodes' tokens (node 0's may be anything).
 * parents int32: parents[b * parents_stride + i], NULL: a chain (parents_stride in elements, 0: one tree for all sequences); a
 * node whose parent is not in [0, i) is nobody's child.  uniforms fp32 [B][T] in [0, 1): [0] draws the following token,
 * [i] decides on node i.  draft_lens int32 [B] (NULL = T): only nodes below it count; 0: a sequence with nothing to verify.
 *
 * From node x = 0: w = row x of target, W = 1.  For the children c of x in the order of their indexes, t = tokens[c]:
 *   draft given:  accept c if u_c W q(t) < w(t), q = row x of draft; else w = max(w - W q, 0), W = sum of w
 *   draft NULL:   accept c if u_c W < w(t); else W = max(W - w(t), 0), w(t) = 0
 * An accepted child becomes x, and its children follow.  (A child whose token is not in [0, V) is passed over.)  Where no
 * child is left, the following token is the first t with w(0) + .. + w(t) > u_0 sum(w); if sum(w) is 0, that of row x of
 * target; if that is 0 too, -1.
 * Probabilities that are negative, infinite or NaN count as 0, uniforms that are NaN or negative as 0, over 1 as 1 (a sum that none
 * exceeds gives the last token of any weight).
 * Products, differences and sums are fp64.  Rows need not sum to 1 exactly.
 *
 * target_stride, draft_stride: elements from one row to the next (>= V; row b * T + i), so that rows may be padded.
 * Out: nodes int32 [B][T]: the accepted path from node 0, then -1; counts int32 [B]: its length (0 where draft_lens is
 * 0); next int32 [B] (-1 there).
 * workspace: pace_draft_verify_workspace_bytes(cfg) bytes, 256-byte aligned.
 * A result repeats bit for bit and does not depend on the other sequences.
 * Errors: PACE_EINVAL for null pointers, sizes below 1, bad strides, a workspace that is too small, misalignment (elements');
 * PACE_EUNSUPPORTED for sizes over those above, or rows that span more than 2^48 bytes. */
pace_status pace_draft_verify(const pace_verify_cfg* cfg, const void* target, int64_t target_stride,
                              const void* draft, int64_t draft_stride, const int32_t* tokens,
                              const int32_t* parents, int64_t parents_stride,
                              const float* uniforms, const int32_t* draft_lens, int32_t* nodes,
                              int32_t* counts, int32_t* next, void* workspace,
                              size_t workspace_bytes, void* stream);

/* Workspace bytes of pace_draft_verify, written to *bytes_out.  Host only.
 * Errors (nothing is written) as pace_draft_verify. */
pace_status pace_draft_verify_workspace_bytes(const pace_verify_cfg* cfg, size_t* bytes_out);

/* ------------------------------------------------------------ cached entries to other places */

/* Moves cached keys and values, codes and scales as they are (nothing is quantised again): of every sequence b
 * the entry at position start[b] + nodes[b * nodes_stride + i], found through src_table, to position start[b] + i, found through
 * dst_table, for i in [0, counts[b]).
 *   accepted drafts   start = the context's length, nodes, counts of pace_draft_verify, one table
 *   dropped entries   start = 0 (or the length of a prefix that stays), nodes = the entries kept, one table
 *   copies, forks     nodes = NULL (i itself), start = 0, dst_table's pages the new ones.  Rows of src_table may repeat.
 * start, counts int32 [B], nodes int32 (device; nodes_stride in elements, rows of T or more); tables int32 [B][max_pages], as pace_cache.h's.
 * counts are taken as 0 below 0, as T above it.  An entry whose position, here or there, is negative, past the
 * table, or in a page that is not there, is left out: what lies at its destination stays.
 * Within a sequence entries move as if all were read before any is written, provided that a page which both tables hold
 * stands at the same entry of both (one table; a prefix that a fork keeps), and nodes[0] < nodes[1] < ..., with
 * nodes[i] >= i (entries with a negative node are left out); where the two tables share no page, nodes may be any.
 * No page that one sequence's entries are written to may be read or written for another sequence in the same call; pages
 * that are only read may be any number of sequences'.  (Shared pages are copied first.)
 * cfg's Hq and io_dtype have no part in it.  T: upper bound of the counts (host).  T == 0 is allowed and does nothing.
 * Errors: PACE_EINVAL for null pointers, T < 0, nodes_stride < T where nodes is given, misalignment (cache: 256 bytes); PACE_EUNSUPPORTED
 * as pace_cache_write, and for T over 2^30. */
pace_status pace_cache_move(const pace_cache_cfg* cfg, void* cache, const int32_t* src_table,
                            const int32_t* dst_table, const int32_t* start, const int32_t* nodes,
                            int64_t nodes_stride, const int32_t* counts, int32_t T, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* PACE_DRAFT_H */
