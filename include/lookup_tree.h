/*
 * lookup_tree.h -- a verify step over a tree of proposals, on GB300.
 *
 * A request may have several chains of proposals for its next tokens: the lookup's
 * draft, a draft model's, its second choices.  lookup_fuse picks one of them; here all
 * of them are verified in one pass of the target, merged into a tree in which chains
 * share what they begin with.  In the order of a step:
 *   lookup_tree_merge      chains of proposals -> tokens, parents, depths, masks
 *   lookup_norm_append     queries and keys normalised per head (where the model does),
 *                          rotated by the node's depth, keys and values cached
 *   lookup_tree_attention  attention of the nodes over the paged cache: each sees the
 *                          cached tokens and its own ancestors
 *   lookup_verify_tree     the branch that the target agrees with, greedy or sampled
 *   lookup_kv_compact      that branch's cache rows moved to the front of the block
 * They stand beside lookup_fuse, lookup_kv_append, lookup_paged_attention,
 * lookup_verify_logits and lookup_append, and share their conventions
 * (lookup_target.h: the paged cache, kv_len, q_len, streams, workspaces).
 *
 * The tree of request r has n[r] nodes, 1 <= n <= N, in rows 0 .. n - 1 of its block.
 * Node 0 is the last committed token; parent[i] < i is node i's parent (node 0 has
 * none, -1); depth[i] counts the steps to node 0.  Node i is cached at position
 * kv_len[r] + i and rotated as position kv_len[r] + depth[i].  mask int64 [B][N][words],
 * words = ceil(N / 64): bit j % 64 of word j / 64 is set where node i sees node j (its
 * ancestors and itself).  N is at most LOOKUP_TREE_MAX_NODES.
 *
 * All arrays are device memory owned by the caller; every call enqueues its work on
 * `stream` and returns without synchronising.  Return codes are those of
 * lookup_draft.h.  B == 0 enqueues nothing.
 */
#ifndef LOOKUP_TREE_H
#define LOOKUP_TREE_H

#include <stddef.h>
#include <stdint.h>

#include "lookup_target.h"

#ifdef __cplusplus
extern "C" {
#endif

#define LOOKUP_TREE_MAX_NODES 256

/*
 * Chains of proposals merged into a tree.
 *
 * root          int32 [B]: the last committed token of each request
 * chains        int32 [B][C][K], len int32 [B][C]: chain c proposes its first len
 *               tokens (clamped to [0, K]), up to the first negative one
 * tokens        int32 [B][N]: the nodes' tokens; -1 past n
 * parent        int32 [B][N]: -1 for node 0 and past n
 * depth         int32 [B][N]: 0 for node 0 and past n
 * mask          int64 [B][N][words]: 0 past n
 * n             int32 [B]
 *
 * Chain after chain is entered from the root: a token that a child of the node
 * reached so far has leads there, another one becomes a new child while there are
 * fewer than N nodes; where there is no room the rest of the chain is left out.
 * Nodes are numbered as they are made, so chain 0 is nodes 1, 2, 3 ..., and the chains
 * first in line get the room.
 * Errors: LOOKUP_DRAFT_EINVAL for B, C or K < 0, C > 64, C * K > 4096, N outside
 * [1, LOOKUP_TREE_MAX_NODES], a null pointer (chains and len only where C * K > 0) or a
 * misaligned one.
 */
int lookup_tree_merge(const int32_t *root, const int32_t *chains, const int32_t *len, int32_t B, int32_t C, int32_t K,
                      int32_t N, int32_t *tokens, int32_t *parent, int32_t *depth, int64_t *mask, int32_t *n,
                      struct CUstream_st *stream);

/*
 * lookup_kv_append with a norm of every query and key head ahead of the rotation, and
 * positions that may be a tree's.
 *
 * q_weight      type [D] or NULL: q is not normalised; k_weight the same for k
 * eps           >= 0, finite
 * depth         int32 [B][N] or NULL (= the token's index i): token i is rotated as
 *               position kv_len[r] + depth[i], and cached at kv_len[r] + i
 * The rest, N's range included, is lookup_kv_append's.  A head x of D elements becomes
 * x_j * w_j / sqrt(mean(x^2) + eps), then its pairs are rotated; everything in float32
 * (the sum of squares too), rounded once.  v is copied.
 * Made for D a power of two from 16 to 512, a rotated part that is a multiple of 16 elements
 * and addresses and strides that are multiples of 16 bytes; anything else is right, and takes
 * three to four times as long.
 * status        int32 [B] or NULL: 1 when a token of the request has no slot or its
 *               rotated position is negative or past max_pos: that token is not cached
 *               and its row of out_q is zeros
 * Errors: those of lookup_kv_append, and LOOKUP_DRAFT_EINVAL for an eps out of range, a
 * weight that is not aligned to its type or a depth that is not.
 */
int lookup_norm_append(const void *q, const int64_t *q_strides, const void *k, const int64_t *k_strides,
                       const void *v, const int64_t *v_strides, const int32_t *kv_len, const int32_t *q_len,
                       const int32_t *block_table, int32_t B, int32_t N, int32_t Hq, int32_t Hkv, int32_t D,
                       int32_t max_pages, int32_t pages, int32_t page_size, const void *q_weight,
                       const void *k_weight, float eps, const float *rotary, int32_t rot, int32_t max_pos,
                       const int32_t *depth, int32_t interleaved, int32_t type, void *k_cache, void *v_cache,
                       void *out_q, int32_t *status, struct CUstream_st *stream);

/*
 * Attention of a tree's nodes over the paged cache, which already holds the block's own
 * keys and values.  The arguments are those of lookup_paged_attention and
 *
 * mask          int64 [B][N][words], 8-byte aligned: which of the block's tokens each
 *               one sees.  A tree's is lookup_tree_merge's; any other will do (a token
 *               may be left out of its own, and may see later ones).  Bits past
 *               q_len[r] do not count.
 * N             at most LOOKUP_TREE_MAX_NODES
 * window        > 0: of the positions that a token sees, in their order, the last
 *               `window` (for a tree: its ancestors, then the tokens cached before);
 *               0: all of them
 *
 * Token i < q_len[r] sees every cached position j < kv_len[r], and position kv_len[r] + j
 * where bit j of its mask is set.  A token that sees nothing has out = 0 and
 * lse = -infinity.  A value in v_cache that is not finite reaches every token that sees
 * it, however small its weight: that element of out is infinite or NaN.  In a slot of the
 * block it reaches no others, and as the weighted sum has it (an infinity stays one); in a
 * slot before the block that `window` hides from some tokens and not from others it may
 * reach those.
 * The weights are rounded to `type` for their product with v, as lookup_paged_attention's
 * (relative 2^-8 for bfloat16; 2^-11 for float16, where those below 2^-21 of the largest
 * are off by up to 2^-32 of it): the tensor cores take both operands in the cache's type.
 * lse takes them before that; scores, maxima, sums and the weighted sum are float32, and out
 * is rounded once.  A call whose bounded waits run out on the device returns NaN in every
 * element of out and lse.
 * For a given request, N, D and head counts the sums are added in an order that depends
 * on the whole batch's lengths: the same call gives the same bits every time.
 * Blocks of more than 128 rows (N * Hq / Hkv) of D = 64 or 128 go through the cache once
 * for every 256 of them, of D = 256 once for every 128.  The choice goes by N: an N far
 * above the largest count costs time there (30 nodes in blocks of 64, 32 heads on 8: two
 * fifths more).
 */
size_t lookup_tree_attention_workspace_bytes(int32_t B, int32_t N, int32_t Hq, int32_t Hkv, int32_t D);

int lookup_tree_attention(const void *q, const int64_t *q_strides, const void *k_cache, const void *v_cache,
                          const int32_t *block_table, const int32_t *kv_len, const int32_t *q_len,
                          const int64_t *mask, int32_t B, int32_t N, int32_t Hq, int32_t Hkv, int32_t D,
                          int32_t max_pages, int32_t pages, int32_t page_size, float scale, int32_t window,
                          int32_t type, void *out, float *lse, void *workspace, size_t workspace_bytes,
                          struct CUstream_st *stream);

/*
 * Verification of a tree of proposals against the target's logits, greedy or sampled.
 * Every proposal is a choice of the drafter (a point mass), not a draw.
 *
 * tokens        int32 [B][N], parent int32 [B][N], n int32 [B]: the tree.  A node i > 0
 *               whose parent is not in [0, i) is no one's child.  An n outside [1, N]
 *               gives the error row accepted = -1, ncommit = 0, commit and path all -1,
 *               logprobs all 0; so do all requests of a call whose bounded waits run out
 *               on the device (lookup_draft_set_wait_limit_ns).
 * logits        type (f32, f16 or bf16) [B][N][V]: the target's logits after each node;
 *               the last axis dense, the request and node strides in elements.  A NaN
 *               counts as -infinity.
 * noise         float [B][V], exponential draws (> 0), or NULL: every request greedy
 * temperature   float [B] or NULL (= 1): a request whose value is not a positive finite
 *               number is greedy
 * u             float [B][N], uniform [0, 1) draws, one for each node that may be
 *               reached (needed with noise where N > 1)
 * workspace     lookup_verify_tree_workspace_bytes bytes, 16-byte aligned, needs no
 *               initialisation; calls that overlap in time need their own
 * out_accepted  int32 [B]: nodes of the accepted branch, the root not counted
 * out_commit    int32 [B][N]: their tokens, then the target's own token, then -1
 * out_ncommit   int32 [B]
 * out_path      int32 [B][N]: the accepted nodes' indices, rising, then -1
 * out_logprobs  float [B][N] or NULL: log-probability of each committed token, 0 past
 *               ncommit
 *
 * From the root down.  At a node with p = softmax(logits / temperature) (the highest
 * logits share it when they are +infinity; a greedy request's logprobs are at
 * temperature 1), its children are looked at in the order of their indices; one whose
 * token an earlier sibling has, or that is outside [0, V), has no weight.
 * Greedy: the child with the lowest index of the largest logit is next, else that index
 * is committed.
 * Sampled: the first child with u < the sum of p over the children's tokens up to its
 * own (float32, u of the node itself) is next.  If there is none the step commits the
 * token that maximises p(t) / noise[t] over all tokens that are no child's (the lowest
 * index on ties; over all tokens where that leaves nothing above 0).  Either way a
 * node's next token is distributed as p: the tree only decides how many are committed.
 * For a tree of one chain the results are lookup_verify_logits' for point masses.
 * A row with no logit above -infinity has no next node, and its step commits the
 * accepted tokens only (ncommit = accepted).
 * Errors: LOOKUP_DRAFT_EINVAL for B < 0, N outside [1, LOOKUP_TREE_MAX_NODES], V out of
 * range (1 <= V < 2^30), a null required pointer, an unknown type, a misaligned pointer or
 * a workspace that is too small.
 */
size_t lookup_verify_tree_workspace_bytes(int32_t B, int32_t N, int32_t V);

int lookup_verify_tree(const int32_t *tokens, const int32_t *parent, const int32_t *n, const void *logits,
                       const int64_t *logits_strides, int32_t type, int32_t V, const float *noise,
                       const float *temperature, const float *u, int32_t B, int32_t N, int32_t *out_accepted,
                       int32_t *out_commit, int32_t *out_ncommit, int32_t *out_path, float *out_logprobs,
                       void *workspace, size_t workspace_bytes, struct CUstream_st *stream);

/*
 * The accepted branch's rows moved to the front of the block, in every layer's caches.
 *
 * k_caches, v_caches  host arrays of `layers` device pointers, each [pages][Hkv]
 *               [page_size][D] of 16-bit elements, dense; read before the call returns
 * path          int32 [B][N], accepted int32 [B]: lookup_verify_tree's
 * status        int32 [B] or NULL: 0, or 1 for a request that was left as it was: its
 *               accepted is above N, its path does not rise within [1, LOOKUP_TREE_MAX_NODES),
 *               or one of the positions has no slot
 *
 * The row of position kv_len[r] + path[r][j] goes to position kv_len[r] + 1 + j, for j <
 * accepted[r] (0 or less: nothing moves).  Rows behind the branch keep what they hold;
 * the next block overwrites them, as kv_len grows by the committed count.  A page that
 * holds rows of the block belongs to one request alone.
 * Errors: LOOKUP_DRAFT_EINVAL for layers < 0, B or N < 0, N > LOOKUP_TREE_MAX_NODES, sizes
 * below 1, D > 1024, a page_size that is not a power of two, a null pointer (status may
 * be), caches that overlap one another, or a misaligned pointer.
 */
int lookup_kv_compact(void *const *k_caches, void *const *v_caches, int32_t layers, const int32_t *block_table,
                      const int32_t *kv_len, const int32_t *path, const int32_t *accepted, int32_t B, int32_t N,
                      int32_t Hkv, int32_t D, int32_t max_pages, int32_t pages, int32_t page_size, int32_t *status,
                      struct CUstream_st *stream);

#ifdef __cplusplus
}
#endif

#endif /* LOOKUP_TREE_H */
