/*
 * ua2a_attn.h -- C ABI of the attention block's operators on the layouts of
 * the Ulysses exchange (ua2a.h): rotary positions joined with the exchange,
 * and attention with a sliding window and sinks, of gathered heads, forward
 * and backward, and of new tokens over the 8-bit cache (ua2a_act.h).
 * Exported by the same library.
 *
 * The conventions of ua2a.h hold: status codes, nothing throws, nothing
 * synchronises or allocates device memory, work is launched only on the given
 * stream, pointers are borrowed device pointers.  A plan (ua2a_plan) gives
 * the shape and the device; its window, path and grid cap play no part here.
 * Its elem_bytes must be the type's (UA2A_TYPE_*).  Layouts, as in ua2a.h:
 *   P  [w][B][S_local][H][D]          (head-complete: all heads of a token)
 *   A  [w][B][S_local*w][H/w][D]      (sequence-gathered)
 */
#ifndef UA2A_ATTN_H
#define UA2A_ATTN_H

#include "ua2a_act.h"

#ifdef __cplusplus
extern "C" {
#endif

#define UA2A_SIDE_P 0
#define UA2A_SIDE_A 1

/*
 * ua2a_rope: rotary positions, one launch, with the exchange where `from` and
 * `to` differ:
 *   out[u] = x[u] cos a - x[z] sin a,  out[z] = x[z] cos a + x[u] sin a
 * for pair i of each head, (u, z) = (2i, 2i + 1) or, with halves, (i, i + pairs);
 * values past 2 * pairs are copied.  The angle of token t is
 *   a = positions[axes[i]][t] * turns[i] / 2^64 turns
 * modulo a turn, exactly up to the rounding of turns[i]; its cosine and sine
 * are good to 32 bits, products are in 32 bits, and results are rounded once.
 * The inverse turns by -a: it is the gradient, with `from` and `to` exchanged.
 *   positions  int32 [naxes][S_local*w], with per_plane [naxes][B][S_local*w]
 *              (gathered order; any values)
 *   turns, axes  device arrays of `pairs` entries; an entry of axes outside
 *              [0, naxes) counts as the nearest
 * out may be x itself where `from` and `to` are equal; no other overlap of
 * out with an input.
 * Errors: INVALID_ARG (NULL, a type that is not the plan's, bad side or flag),
 * SHAPE (pairs < 1 or 2 * pairs > D, naxes < 1, 2^31 tokens, or positions on
 * all axes), ALIGN (x, out by their type, positions and axes by 4,
 * turns by 8), ALIAS, DEVICE (no state change); HIP (the plan becomes
 * disabled); DISABLED.
 */
typedef struct ua2a_rope_s {
    const void* x;
    void* out;
    const int32_t* positions;
    const uint64_t* turns;
    const int32_t* axes;
    int32_t pairs;
    int32_t naxes;
    int32_t halves;
    int32_t inverse;
    int32_t per_plane;
    int32_t from;
    int32_t to;
    int32_t type;
} ua2a_rope_t;

int ua2a_rope(ua2a_plan_t plan, const ua2a_rope_t* args, void* stream);

/*
 * What a query at position p sees, with c(x) = x / chunk: positions j with
 *   c(p) - left <= c(j) <= c(p) + right,  and j < sinks;
 * with right = 0 nothing past p's own chunk, sinks or not.  left, right = -1:
 * no bound on that side.  All of them below 2^31, chunk at least 1.
 */
typedef struct ua2a_window_s {
    int64_t left;
    int64_t right;
    int64_t sinks;
    int64_t chunk;
} ua2a_window_t;

/*
 * ua2a_attention: softmax(scale * q k^T) v of gathered heads (A layout),
 * every sequence (w * B of them) by itself; one launch, or two where parts
 * of the keys goes to workgroups of its own.
 *   q, out     [w][B][S_local*w][H/w][D]
 *   k, v       [w][B][S_local*w][kv_heads/w][D]; query head h of a rank takes
 *              key head h / (H / kv_heads)
 *   counts     optional device array of B int32: tokens of a plane's sequences
 *              (on every rank), clamped to [0, S_local*w]; the others are
 *              padding: no query sees them, whatever they hold, and their own
 *              rows are zeros (lse -infinity)
 *   lse        optional [w][B][H/w][S_local*w]: log of the sum of exp(scale *
 *              scores), natural
 *   workspace  scratch of ua2a_attention_workspace's size, 16-byte aligned
 *              (NULL where that is 0); it belongs to the call until its work
 *              is done
 * Types bf16 and fp16.  Scores, softmax and sums are in 32 bits; the weights
 * exp(s - m) are rounded to the type for the product with v, their sum is
 * not; out is rounded once.  (In fp16 a weight has its 11 digits down to 2^-27
 * of the row's largest, and below that is off by 2^-38 of it at most.  In bf16
 * the sums hold up to 2^8 times v: |v| times the keys stays below 2^119.)  What a row does not see plays no part in it,
 * infinities and NaN included; a row whose weights are all zero is zeros.
 * D must be a multiple of 8 up to 128; all tensors 16-byte aligned; scale > 0
 * and finite, in powers of two too (scale * log2 e), and so must scores be.
 * No output may overlap an input, another output or the workspace.
 * Errors: INVALID_ARG (NULL, type, scale, chunk < 1, a bound < -1), SHAPE (D,
 * kv_heads not a multiple of w or no divisor of H, H/w * D over 2^22, 2^31
 * tokens times heads of a rank or more, 2^38 values of a tensor), ALIGN, ALIAS, CAPACITY (workspace), DEVICE, HIP, DISABLED.
 */
typedef struct ua2a_attention_s {
    const void* q;
    const void* k;
    const void* v;
    void* out;
    float* lse;
    const int32_t* counts;
    void* workspace;
    int64_t workspace_bytes;
    ua2a_window_t window;
    int64_t kv_heads;
    float scale;
    int32_t type;
} ua2a_attention_t;

int ua2a_attention(ua2a_plan_t plan, const ua2a_attention_t* args, void* stream);

/* Bytes of workspace that the call needs (host only; of args only window,
 * kv_heads and type are looked at).  Errors: INVALID_ARG, SHAPE. */
int ua2a_attention_workspace(ua2a_plan_t plan, const ua2a_attention_t* args, int64_t* bytes);

/*
 * ua2a_attention_backward: gradients of ua2a_attention with the same q, k, v,
 * counts, window, kv_heads and scale; two launches, or three.
 *   dout       gradient of out;  out, lse: as the forward call wrote them
 *   dq, dk, dv  all three, in the layouts of q, k, v; rows of padding are zeros
 *   workspace  as above, of ua2a_attention_backward_workspace's size
 * With P = exp(scale * s - lse), delta = sum(dout * out) of a row:
 *   dv = P^T dout,  dS = P * (dout v^T - delta),  dq = scale dS k,  dk = scale dS^T q.
 * Sums are in 32 bits, in a fixed order; P and dS are rounded to the type for
 * the products with dout and q, dS to two values of it (their sum has twice the
 * digits) for the product with k, the gradients once.  In fp16 they go in times
 * a power of two that comes out of the sums again, so that many keys or small
 * gradients leave them their digits: for dq one of each row's own, at which no
 * dS passes the type; for dk and dv one between 1 and 2^15 for 128 keys and the
 * rows that one workgroup walks, as large as their |dout|, |v| and delta allow.
 * There a dS past 65504 is still infinite.  Padding may hold anything;
 * infinities and NaN elsewhere reach the gradients of rows and keys near them too.
 * lse is in 32 bits, so P is off by about 2^-22 of the largest score's size.
 */
typedef struct ua2a_attention_grad_s {
    const void* dout;
    const void* q;
    const void* k;
    const void* v;
    const void* out;
    const float* lse;
    void* dq;
    void* dk;
    void* dv;
    const int32_t* counts;
    void* workspace;
    int64_t workspace_bytes;
    ua2a_window_t window;
    int64_t kv_heads;
    float scale;
    int32_t type;
} ua2a_attention_grad_t;

int ua2a_attention_backward(ua2a_plan_t plan, const ua2a_attention_grad_t* args, void* stream);
int ua2a_attention_backward_workspace(ua2a_plan_t plan, const ua2a_attention_grad_t* args, int64_t* bytes);

/*
 * ua2a_cache_attention: the same attention of n new tokens of every sequence
 * of a cache, over what the cache holds (code * scale, rounded to the type, as
 * ua2a_cache_read gives it).  Up to 16 queries of a key head take their weights
 * as two values of the type into the product with v.
 *   q, out     [w][sequences][n][H/w][D] (the mode-0 exchange of the tokens
 *              that ua2a_cache_write takes has them in this order)
 *   kv_heads   the cache's heads on all ranks (its H in place of the plan's)
 *   starts, counts  device arrays of `sequences` int32, as for
 *              ua2a_cache_write: token t < counts[i] (NULL: n) of sequence i
 *              has position starts[i] + t, where that lies in the cache; the
 *              sequence's positions up to its last such token hold keys
 * Rows without a position are left as they were.  The plan's B and S_local
 * play no part.  Other arguments, types, limits and errors as for
 * ua2a_attention; the codes must be 8-byte aligned.
 */
typedef struct ua2a_cache_attention_s {
    const void* q;
    void* out;
    const int32_t* starts;
    const int32_t* counts;
    void* workspace;
    int64_t workspace_bytes;
    ua2a_window_t window;
    int64_t n;
    int64_t kv_heads;
    float scale;
    int32_t type;
} ua2a_cache_attention_t;

int ua2a_cache_attention(ua2a_plan_t plan, const ua2a_cache_t* cache, const ua2a_cache_attention_t* args, void* stream);

/* Of the cache only sequences, capacity and format, of args only window, n,
 * kv_heads and type are looked at. */
int ua2a_cache_attention_workspace(ua2a_plan_t plan, const ua2a_cache_t* cache, const ua2a_cache_attention_t* args,
                                   int64_t* bytes);

#ifdef __cplusplus
}
#endif

#endif /* UA2A_ATTN_H */
