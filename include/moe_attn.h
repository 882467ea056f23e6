/*
 * moe_attn.h -- C ABI of the attention half of the decoder layer whose MLP
 * half is moe_mlp.h: the operators between the fused query/key/value
 * projection and the output projection, for serving, over a paged key/value
 * cache.  Same library, same conventions as moe_mlp.h:
 *   - every pointer argument except `stream` is a DEVICE pointer; config and
 *     cache structs are HOST memory;
 *   - tensors are row-major and contiguous unless a stride is an argument;
 *     bf16 and fp32 tensors are 16-byte aligned, int32 and int64 arrays have
 *     their type's alignment; bf16 values travel as uint16_t bit patterns;
 *   - the caller owns every buffer, the workspace too, whose contents need no
 *     initialisation and are garbage after a call; the library allocates,
 *     frees and synchronises nothing, and keeps no pointer;
 *   - arguments are validated on the host before anything is enqueued; on an
 *     error nothing is enqueued.  Work goes to `stream` (a hipStream_t, NULL =
 *     the default stream) of the current device and the call returns without
 *     waiting; calls can be captured into a HIP graph;
 *   - results are deterministic: no atomics, fixed summation orders.
 * Status codes are those of moe_mlp.h.
 *
 * The cache.  A page holds page_size tokens of every key/value head:
 *   k [n_pages, n_kv_heads, head_dim / 8, page_size, 8] bf16: dims 8c .. 8c+7
 *     of the page's token t at [page][head][c][t][.];
 *   v [n_pages, n_kv_heads, page_size / 8, head_dim, 8] bf16: tokens
 *     8g .. 8g+7 of the page at dim d at [page][head][g][d][.].
 * Both are the order in which a matrix instruction takes its operand: 16
 * bytes are 8 values along the sum (dims for scores, tokens for the weighted
 * sum of values), and neighbouring rows are 16 bytes apart, so that pages go
 * to registers or to LDS in whole lines with nothing to transpose.
 * Token i of sequence b sits in page page_table[b][i / page_size] at place
 * i % page_size; its slot is page * page_size + place.
 * Page ids, slots and positions are device data that the host cannot check:
 * page ids and positions out of range are clamped into it, tokens with a slot
 * out of range are not stored, and lengths are clamped, so that no access
 * leaves the caller's buffers; the results for such rows are unspecified.
 * What slots hold that no visible key occupies (NaN too), and the page ids of
 * pages without a visible key, do not matter.  A value that one query of a
 * sequence sees should be finite for the others too: those that do not see it
 * give it the weight 0, and 0 * inf is NaN.
 */
#ifndef MOE_ATTN_H
#define MOE_ATTN_H

#include <stddef.h>
#include <stdint.h>

#include "moe_mlp.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MOE_ATTN_MAX_HEADS    1024   /* n_heads */
#define MOE_ATTN_DECODE_MAX_Q 8      /* new tokens per sequence in moe_attn_decode */

#define MOE_ATTN_ROPE_HALF        0  /* rotated pairs are dims (i, i + rotary_dim / 2) */
#define MOE_ATTN_ROPE_INTERLEAVED 1  /* rotated pairs are dims (2i, 2i + 1) */

/* Geometry and constants of one attention layer; no field has a default. */
typedef struct moe_attn_config {
  int32_t n_heads;     /* query heads, a multiple of n_kv_heads, at most MOE_ATTN_MAX_HEADS */
  int32_t n_kv_heads;  /* key/value heads; query head h reads key/value head h / (n_heads / n_kv_heads) */
  int32_t head_dim;    /* 64, 128 or 256 */
  int32_t page_size;   /* tokens per page: 16, 32, 64, 128 or 256 */
  int32_t rotary_dim;  /* rotated dims of each query and key head: 0 (none) or a multiple of 16 up to head_dim */
  int32_t rope_style;  /* MOE_ATTN_ROPE_HALF or _INTERLEAVED */
  int32_t window;      /* a query sees the `window` latest keys, its own among them; 0 = all */
  int32_t n_sinks;     /* and, with a window, the first n_sinks keys of its sequence; >= 0 */
  float   norm_eps;    /* finite, >= 0; added to the mean square */
  float   scale;       /* finite, > 0; multiplies q . k */
} moe_attn_config;

typedef struct moe_attn_cache {
  uint16_t* k;         /* [n_pages, n_kv_heads, head_dim / 8, page_size, 8] bf16 */
  uint16_t* v;         /* [n_pages, n_kv_heads, page_size / 8, head_dim, 8] bf16 */
  int64_t   n_pages;   /* >= 1; n_pages * page_size < 2^31 */
} moe_attn_cache;

/*
 * Queries, keys and values of T new tokens out of the fused projection: RMS
 * norm of every query and key head, rotation by the token's position, and the
 * rows of K and V into the cache, in one pass.
 *   y = x * rsqrt(mean(x^2) + norm_eps) * w        per head, in fp32
 *   (a, b) -> (a cos - b sin, b cos + a sin)       per pair of the first rotary_dim dims, in fp32
 * and one rounding to bf16 (nearest even); V is stored as it is.
 *   qkv       [T, >= (n_heads + 2 n_kv_heads) * head_dim] bf16, rows qkv_stride
 *             elements apart (a multiple of 8): query heads, key heads, value heads.
 *   q_norm_w, k_norm_w [head_dim] fp32; NULL = that side is not normalised.
 *   cos_sin   [n_positions, rotary_dim] fp32: row p holds rotary_dim / 2
 *             cosines, then as many sines; NULL only when rotary_dim is 0.
 *   positions [T] int32 (NULL only when rotary_dim is 0).
 *   slots     [T] int64, distinct; negative (or past the cache) = the token's
 *             K and V are not stored.
 *   q_out     [T, n_heads, head_dim] bf16; does not overlap qkv.
 */
int moe_attn_prepare(const moe_attn_config* cfg, const moe_attn_cache* cache, const uint16_t* qkv,
                     int64_t qkv_stride, int64_t T, const float* q_norm_w, const float* k_norm_w,
                     const float* cos_sin, int64_t n_positions, const int32_t* positions, const int64_t* slots,
                     uint16_t* q_out, void* stream);

/*
 * Workspace bytes of moe_attn_decode (prefill == 0; max_q = its n_q) or
 * moe_attn_prefill (prefill != 0) for T new tokens (decode: B * n_q) of B
 * sequences of at most max_q new tokens and at most max_len tokens in all.
 * `bytes` is a HOST pointer.  Limits (MOE_MLP_ERR_BAD_SHAPE past them, here and
 * in the calls): max_len < 2^30; decode: B * n_q * n_heads < 2^26; prefill:
 * T < 2^26, min(max_q, T) * n_heads < 2^30, and B < 2^16 or
 * B * max_q * n_heads < 2^26; and no launch of 2^32 threads or more (tens of
 * thousands of sequences that may all be very long).
 * The size holds for these arguments alone: a call of fewer or shorter sequences
 * may be cut into more parts, and need more.
 */
int moe_attn_workspace_size(const moe_attn_config* cfg, int64_t T, int64_t B, int64_t max_q, int64_t max_len,
                            int prefill, size_t* bytes);

/*
 * Bytes that are enough for every call of this configuration (and of this form,
 * decode or prefill) with none of T, B, max_q and max_len larger: for a workspace
 * that is allocated once.  Errors as above, for these sizes.
 */
int moe_attn_workspace_bound(const moe_attn_config* cfg, int64_t T, int64_t B, int64_t max_q, int64_t max_len,
                             int prefill, size_t* bytes);

/*
 * Attention of n_q new tokens (1..MOE_ATTN_DECODE_MAX_Q: one, or a verify
 * step) of each of B sequences over the cache, which already holds them
 * (moe_attn_prepare).  Query i of a sequence of length n has position
 * p = n - n_q + i and sees the keys k <= p with p - k < window or k < n_sinks
 * (all k <= p when window is 0):
 *   out = sum_k softmax_k(scale q . k) v_k          over the visible keys
 * in fp32, the softmax weights rounded to bf16 before the sum over v, one
 * rounding of the result.  Scores (scale q . k) up to 2^28 in magnitude.  A
 * query that sees no key (n == 0, p < 0) gives 0.
 *   q         [B, n_q, n_heads, head_dim] bf16;  out the same shape.
 *   seq_lens  [B] int32, the new tokens included, at most max_len.
 *   page_table [B, max_pages] int32.
 *   max_len   0 .. max_pages * page_size; longer sequences are cut to it.
 *             It sets the launch, not the work, and a close bound is faster: 2000
 *             keys of 32/8 heads of 128 dims, bound 131072 or 2000: 20 and 9.9 us
 *             of one sequence, 31 and 26 us of 16, 133 and 82 us of 64.
 */
int moe_attn_decode(const moe_attn_config* cfg, const moe_attn_cache* cache, const uint16_t* q, int64_t B,
                    int64_t n_q, const int32_t* seq_lens, const int32_t* page_table, int64_t max_pages,
                    int64_t max_len, uint16_t* out, void* workspace, size_t ws_bytes, void* stream);

/*
 * The same for prompts, or pieces of prompts behind a cached prefix: sequence
 * b has the new tokens cu_q[b] .. cu_q[b+1]-1 of q, the last ones of its
 * seq_lens[b] tokens, all of them in the cache already.
 *   q         [T, n_heads, head_dim] bf16;  out the same shape (rows outside
 *             cu_q[0] .. cu_q[B] are not written).
 *   cu_q      [B + 1] int32, not decreasing, within 0 .. T.
 *   max_q     the most new tokens of a sequence; further ones are not computed
 *             (their rows of out are not written), and the first max_q keep
 *             their positions, seq_lens[b] - (cu_q[b+1] - cu_q[b]) and on.
 */
int moe_attn_prefill(const moe_attn_config* cfg, const moe_attn_cache* cache, const uint16_t* q, int64_t T,
                     const int32_t* cu_q, int64_t B, int64_t max_q, const int32_t* seq_lens,
                     const int32_t* page_table, int64_t max_pages, int64_t max_len, uint16_t* out, void* workspace,
                     size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_ATTN_H */
