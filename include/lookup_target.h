/*
 * lookup_target.h -- the target model's side of a verify step, on GB300.
 *
 * A verify step runs the target model once over a block of new tokens per
 * request: the last committed token and the proposals of lookup_draft /
 * lookup_fuse.  Three operators of that pass belong to the drafting loop, because
 * their shapes are the block's (HyperQwen lookup-drafting article,
 * kwkr.cn/news/564408, sections "第2步" and "第3步"):
 *   lookup_kv_append        rotary positions for the block's queries and keys,
 *                           keys and values written to a paged cache
 *   lookup_paged_attention  attention of the block's tokens over that cache (one
 *                           token per request is plain decoding)
 *   lookup_verify_logits    verification of the proposals against the target's
 *                           logits, from given random numbers
 * Proposals that are rejected need no clean-up: the next step's block overwrites
 * their cache slots, since kv_len grows by the committed count only.
 *
 * The paged cache.  k_cache and v_cache are [pages][Hkv][page_size][D], dense, of
 * one 16-bit type.  block_table int32 [B][max_pages] names request r's pages in
 * order: its cached token j is row j % page_size of page block_table[r][j /
 * page_size].  kv_len int32 [B] counts the tokens cached before the block, q_len
 * int32 [B] the block's tokens (NULL = all N); token i of the block has position
 * kv_len[r] + i.  Both calls of a step take the same kv_len and q_len.  A q_len
 * outside [0, N] is clamped to that range, a negative kv_len to 0.
 *
 * All arrays are device memory owned by the caller; every call enqueues its work
 * on `stream` and returns without synchronising.  Return codes are those of
 * lookup_draft.h.  B == 0 or N == 0 enqueues nothing.
 */
#ifndef LOOKUP_TARGET_H
#define LOOKUP_TARGET_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

struct CUstream_st;

/* Element types of the tensors a call takes as void pointers. */
#define LOOKUP_TYPE_F32 0
#define LOOKUP_TYPE_F16 1
#define LOOKUP_TYPE_BF16 2

/*
 * Rotary positions and the append to the paged cache.
 *
 * q, k, v       type [B][N][Hq or Hkv][D], the last axis dense; their request,
 *               token and head strides in elements follow (so they may be parts of
 *               one projection's output).  q may be NULL (nothing is rotated for
 *               it), k and v may both be NULL (nothing is cached).
 * rotary        float [max_pos][rot]: for each position rot/2 cosines, then rot/2
 *               sines; NULL = no rotation (rot is then ignored)
 * rot           leading part of the head that is rotated, even, 2 <= rot <= D
 * interleaved   0: element j pairs with j + rot/2; else 2j pairs with 2j + 1
 * out_q         type [B][N][Hq][D], dense; rows past q_len[r] are zeros
 * status        int32 [B] or NULL: 0, or 1 when a token of the request has no
 *               slot (its position is past the block table or past max_pos, or its
 *               table entry is not in [0, pages)): that token is not cached and
 *               its row of out_q is zeros
 * type          LOOKUP_TYPE_F16 or LOOKUP_TYPE_BF16
 *
 * For a pair (a, b) at position p: a' = a cos - b sin, b' = b cos + a sin, in
 * float32, rounded once; elements rot .. D and v are copied.  Scaling for long
 * contexts is a matter of the table's angles.
 * Errors: LOOKUP_DRAFT_EINVAL for sizes below their ranges, D > 1024, B * N >= 2^31, a
 * page_size that is not a power of two, one of k and v without the other or without a cache,
 * q without out_q, a null kv_len or block_table, or pointers not aligned to
 * their elements.
 */
int lookup_kv_append(const void *q, const int64_t *q_strides, const void *k, const int64_t *k_strides,
                     const void *v, const int64_t *v_strides, const int32_t *kv_len, const int32_t *q_len,
                     const int32_t *block_table, int32_t B, int32_t N, int32_t Hq, int32_t Hkv, int32_t D,
                     int32_t max_pages, int32_t pages, int32_t page_size, const float *rotary, int32_t rot,
                     int32_t max_pos, int32_t interleaved, int32_t type, void *k_cache, void *v_cache,
                     void *out_q, int32_t *status, struct CUstream_st *stream);

/*
 * Attention of the block's tokens over the paged cache, which already holds the
 * block's own keys and values.
 *
 * q             type [B][N][Hq][D], the last axis dense, strides in elements
 * Hq, Hkv       query and key-value heads, Hq a multiple of Hkv; query head h
 *               reads key-value head h / (Hq / Hkv)
 * D             64, 128 or 256
 * page_size     a power of two, 8 .. 1024
 * scale         factor of the products q.k (finite)
 * window        > 0: a token sees itself and the window - 1 tokens before it;
 *               0: everything before it
 * out           type [B][N][Hq][D], dense
 * lse           float [B][N][Hq] or NULL: the logarithm of the softmax's sum
 * workspace     lookup_paged_attention_workspace_bytes bytes, 16-byte aligned;
 *               needs no initialisation; calls that overlap in time need their own
 *
 * Token i < q_len[r], at position p = kv_len[r] + i, sees positions j <= p (and
 * j > p - window).  With s_j = scale * q.k_j in float32: lse = log(sum_j
 * exp(s_j)), out = sum_j exp(s_j - lse) v_j.  The weights are rounded to `type` for
 * their product with v (relative 2^-8 for bfloat16; 2^-11 for float16, where those
 * below 2^-21 of the largest are off by up to 2^-32 of it), and lse takes them before
 * that; everything else is float32.  Rows past q_len[r] have out = 0 and
 * lse = -infinity.  A request's tokens past the block table's end are taken as
 * absent, and a table entry outside [0, pages) as a page of zeros; slots that no
 * token of the request sees are never used, whatever they hold.  A value in v_cache
 * that is not finite, in a slot that some tokens of the block see and others do not
 * (the block's own tokens, a window's edge), may reach the others.
 * A call whose bounded waits run out on the device (lookup_draft_set_wait_limit_ns)
 * returns NaN in every element of out and lse.
 * Made for blocks of N * Hq / Hkv <= 128 rows, a verify block or one token.  A longer
 * block (a prompt) is right, but every 128 rows of it go through all the positions
 * that any of its tokens sees: twice the work where nothing was cached before it, and
 * the whole length where the window is short.
 * Errors: LOOKUP_DRAFT_EINVAL for sizes outside their ranges, a null pointer other than
 * q_len and lse, pointers of q, the caches, out and the workspace or strides of q's axes of two
 * or more that are not multiples of 16 bytes, B * N * Hq above 2^30, a workspace that is too small, or caches (pages * Hkv * page_size) or block tables
 * (max_pages * page_size) of 2^31 - 129 rows or more.
 */
size_t lookup_paged_attention_workspace_bytes(int32_t B, int32_t N, int32_t Hq, int32_t Hkv, int32_t D);

int lookup_paged_attention(const void *q, const int64_t *q_strides, const void *k_cache, const void *v_cache,
                           const int32_t *block_table, const int32_t *kv_len, const int32_t *q_len, int32_t B,
                           int32_t N, int32_t Hq, int32_t Hkv, int32_t D, int32_t max_pages, int32_t pages,
                           int32_t page_size, float scale, int32_t window, int32_t type, void *out, float *lse,
                           void *workspace, size_t workspace_bytes, struct CUstream_st *stream);

/*
 * Verification of a proposal block against the target's logits, greedy or
 * sampled, request by request ("第3步": lossless verification; a lookup-filled
 * position is a point mass on its token).
 *
 * block         int32 [B][P] (0 <= P <= 65536), len int32 [B], as for lookup_verify
 *               (a len outside [0, P] gives the error row accepted = -1,
 *               ncommit = 0, commit all -1, logprobs all 0; so do all requests of a
 *               call whose bounded waits run out on the device,
 *               lookup_draft_set_wait_limit_ns)
 * logits        type (f32, f16 or bf16) [B][P + 1][V]: the target's logits at each
 *               position given the block before it; the last axis dense, the
 *               request and position strides in elements.  A NaN counts as -infinity.
 * noise         float [B][V], exponential draws (> 0), or NULL: every request greedy
 * temperature   float [B] or NULL (= 1): a request whose value is not a positive
 *               finite number is greedy
 * u             float [B][P], uniform [0, 1) draws (needed with noise where P > 0)
 * qprobs        float [B][P][V] or NULL: the proposal distribution at each position,
 *               the last axis dense, strides in elements; NULL = every position is
 *               a point mass
 * point_mass    int32 [B][P] or NULL: positions whose proposal is a point mass
 *               whatever qprobs holds
 * workspace     lookup_verify_logits_workspace_bytes bytes, 16-byte aligned, needs
 *               no initialisation; calls that overlap in time need their own
 * out_accepted  int32 [B], out_commit int32 [B][P + 1], out_ncommit int32 [B]: as
 *               lookup_verify writes them
 * out_logprobs  float [B][P + 1] or NULL: log-probability of each committed token,
 *               0 past ncommit
 *
 * Row i's distribution is p = softmax(logits[i] / temperature) (the highest logits share
 * it when they are +infinity; a greedy request's logprobs are at temperature 1).
 * Greedy: proposal d at i is accepted when it is the lowest index of the row's
 * largest logit; the step then commits that index of row a.
 * Sampled: it is accepted when u[i] * q(d) < p(d) (float32), q(d) = 1 at a point
 * mass; at the first rejection a the step commits the token t that maximises
 * max(p(t) - q(t), 0) / noise[t] in row a, after full acceptance the one that
 * maximises p(t) / noise[t] (the lowest index on ties): a draw from the residual
 * distribution, by the race of exponentials.  Where p - q leaves nothing above 0,
 * p itself is drawn from.
 * A row with no logit above -infinity accepts nothing, and its step commits the
 * a accepted tokens only (ncommit = a, commit[a] = -1).
 * Errors: LOOKUP_DRAFT_EINVAL for B < 0, P or V out of range (1 <= V < 2^30), a null
 * required pointer, an unknown type, a misaligned pointer or a workspace that is
 * too small.
 */
size_t lookup_verify_logits_workspace_bytes(int32_t B, int32_t P, int32_t V);

int lookup_verify_logits(const int32_t *block, const int32_t *len, const void *logits, const int64_t *logits_strides,
                         int32_t type, int32_t V, const float *noise, const float *temperature, const float *u,
                         const float *qprobs, const int64_t *qprobs_strides, const int32_t *point_mass, int32_t B,
                         int32_t P, int32_t *out_accepted, int32_t *out_commit, int32_t *out_ncommit,
                         float *out_logprobs, void *workspace, size_t workspace_bytes, struct CUstream_st *stream);

#ifdef __cplusplus
}
#endif

#endif /* LOOKUP_TARGET_H */
