/*
 * ua2a_act.h -- C ABI of the operators that compute on activations around
 * the Ulysses exchange (ua2a.h): RMS norms joined with it, forward and
 * backward, with 8-bit outputs and 8-bit checkpoints, and an 8-bit key/value
 * cache that the exchange fills.  Exported by the same library.
 *
 * The conventions of ua2a.h hold: status codes, nothing throws, nothing
 * synchronises or allocates device memory, work is launched only on the given
 * stream, pointers are borrowed device pointers.  A plan (ua2a_plan) gives
 * the shape and the device; its window, path and grid cap play no part here.
 * Its elem_bytes must be the type's.  Layouts, as in ua2a.h:
 *   P  [w][B][S_local][H][D]          (head-complete: all heads of a token)
 *   A  [w][B][S_local*w][H/w][D]      (sequence-gathered)
 *
 * 8 bits with scales.  A tensor [..., D] is held as codes [..., D], one byte
 * per value, and scales [..., ceil(D/32)], one byte per block of 32 values
 * along D (the last block of a head may be shorter).  A scale byte s stands
 * for 2^(s - 127), 255 for NaN (e8m0); a code is e4m3 (largest value 448) or e5m2
 * (57344).  Of a block with largest finite magnitude m, the scale is the
 * least power of two, 2^-127 at least, with m <= scale * (largest code): no
 * finite value overflows, and a value's error is at most half a step of its
 * code.  The code is x / scale rounded to nearest even, exactly.  NaN
 * becomes NaN, an infinity NaN in e4m3 and itself in e5m2.  Reading back,
 * code * scale is rounded once to the type; finite values that pass the
 * type's largest stay there.
 */
#ifndef UA2A_ACT_H
#define UA2A_ACT_H

#include "ua2a.h"

#ifdef __cplusplus
extern "C" {
#endif

/* element types */
#define UA2A_TYPE_BF16 0
#define UA2A_TYPE_FP16 1
#define UA2A_TYPE_FP32 2

/* 8-bit formats */
#define UA2A_FORMAT_NONE 0
#define UA2A_FORMAT_E4M3 1
#define UA2A_FORMAT_E5M2 2

#define UA2A_BLOCK 32             /* values that share a scale */

/*
 * ua2a_norm_exchange: RMS norm joined with the exchange, one launch.
 *   mode 0: x in P, out in A:  h = x (+ residual);  out = exchange(norm(h))
 *   mode 1: x in A, out in P:  h = exchange(x) (+ residual);  out = norm(h)
 *   norm(h) = h * rstd * weight,  rstd = 1 / sqrt(mean(h^2) + eps), the mean
 *   over a token's H*D values, or with per_head over each head's D.
 * Sums and products are in 32 bits.  With a residual (P) the sum h, rounded
 * to the type, is written to `sum` (P), and the norm takes that rounded sum.
 *   weight     [H*D], with per_head [D]; NULL: ones; of weight_type, the
 *              plan's type or fp32
 *   out        in the type; with out_format the codes, and out_scales the
 *              scales, in out's layout (quantised from the 32-bit result)
 *   saved, saved_scales   with saved_format: h in 8 bits (P), the checkpoint
 *              that ua2a_norm_exchange_backward takes
 *   rstd       optional: [w][B][S_local], with per_head [w][B][S_local][H]
 * A norm covers at most 65536 values of a 2-byte type or 32768 of fp32, heads
 * counted as whole blocks of 32, where D * elem_bytes is a multiple of 16 and
 * x, residual, out and sum are 16-byte aligned (codes 8-byte); at most 8192
 * otherwise.
 * x, residual and weight may overlap one another; no output may overlap an
 * input or another output.
 * Errors: INVALID_ARG (NULL where needed, a type that is not the plan's, bad
 * mode, format or per_head, eps not finite or not > 0, sum without residual
 * or the reverse), SHAPE (norm too long; 2^31 segments or more), ALIGN,
 * ALIAS, DEVICE (no state change); HIP (the plan becomes disabled); DISABLED.
 */
typedef struct ua2a_norm_s {
    const void* x;
    const void* residual;
    const void* weight;
    void* out;
    void* out_scales;
    void* sum;
    void* saved;
    void* saved_scales;
    float* rstd;
    float eps;
    int32_t type;
    int32_t weight_type;
    int32_t per_head;
    int32_t out_format;
    int32_t saved_format;
} ua2a_norm_t;

int ua2a_norm_exchange(ua2a_plan_t plan, int32_t mode, const ua2a_norm_t* args, void* stream);

/*
 * ua2a_norm_exchange_backward: gradients of ua2a_norm_exchange(mode), one
 * launch, and one more where dweight is asked for.
 *   dy       gradient of out: mode 0 in A, mode 1 in P
 *   dsum     gradient of sum (P), or NULL
 *   saved    h: with saved_format the checkpoint's codes and saved_scales
 *            (P); else the values, in P, or in A with saved_gathered (mode 1
 *            without a residual: x itself)
 *   rstd     as the forward call wrote it
 *   dx       gradient of x, in x's layout.  In mode 0 it is the residual's
 *            gradient too.
 *   dresidual  mode 1: the residual's gradient (P), or NULL
 *   dweight  fp32 [H*D] or [D], or NULL: summed over all tokens in a fixed
 *            order
 *   workspace  scratch of ua2a_norm_workspace's size for the sums of
 *            dweight, 16-byte aligned; NULL without dweight.  It belongs to
 *            the call until its work is done.
 * With g = dy * weight, n = h * rstd:
 *   dh = rstd * (g - n * mean(g * n)) + dsum,  dweight = sum(dy * n).
 * Errors: as above, and CAPACITY for a workspace that is too small.
 */
typedef struct ua2a_norm_grad_s {
    const void* dy;
    const void* dsum;
    const void* saved;
    const void* saved_scales;
    const void* weight;
    const float* rstd;
    void* dx;
    void* dresidual;
    float* dweight;
    void* workspace;
    int64_t workspace_bytes;
    int32_t type;
    int32_t weight_type;
    int32_t per_head;
    int32_t saved_format;
    int32_t saved_gathered;
} ua2a_norm_grad_t;

int ua2a_norm_exchange_backward(ua2a_plan_t plan, int32_t mode, const ua2a_norm_grad_t* args, void* stream);

/* Bytes of workspace that a backward call with dweight needs at most
 * (host only).  Errors: INVALID_ARG, SHAPE. */
int ua2a_norm_workspace(ua2a_plan_t plan, int32_t per_head, int64_t* bytes);

/*
 * An 8-bit key/value cache of sequence-gathered heads, owned by the caller:
 *   codes   [2][w][sequences][capacity][H/w][D]       (keys, then values)
 *   scales  [2][w][sequences][capacity][H/w][ceil(D/32)]
 */
typedef struct ua2a_cache_s {
    void* codes;
    void* scales;
    int64_t sequences;
    int64_t capacity;
    int32_t format;
} ua2a_cache_t;

/*
 * ua2a_cache_write: the mode-0 exchange of new keys and values (P, either may
 * be NULL) straight into the cache, one launch.  The B * S_local*w gathered
 * tokens are taken in order, `sequences` runs of n = B * S_local*w /
 * sequences tokens each (it must divide; one new token for each of many
 * sequences has n = 1).  Token t of sequence i goes to position starts[i] + t
 * where t < counts[i] (NULL: all n) and the position lies in [0, capacity);
 * other tokens are dropped, and every other position is left as it was.
 *   starts, counts  device arrays of `sequences` int32
 * Errors: INVALID_ARG, SHAPE (sequences does not divide; more than 2^31 - 1
 * positions in a sequence; cache over 2^38 values; one of k and v has 2^31 or
 * more pieces of 16 bytes, heads padded to whole blocks -- of one value where
 * D * elem_bytes is no multiple of 16 or k, v are not 16-byte or the codes not
 * 8-byte aligned), ALIGN, ALIAS, DEVICE, HIP, DISABLED.
 */
int ua2a_cache_write(ua2a_plan_t plan, const ua2a_cache_t* cache, int32_t type, const void* k, const void* v,
                     const int32_t* starts, const int32_t* counts, void* stream);

/*
 * ua2a_cache_read: positions starts[i] + t, t < min(n, counts[i]), of every
 * sequence back in the type (either output may be NULL), one launch:
 *   k_out, v_out   [w][sequences][n][H/w][D]
 * Rows without a position are left as they were.  starts NULL: 0; counts
 * NULL: n.  The plan's B and S_local play no part.
 * Errors: as for ua2a_cache_write (SHAPE: n < 1; an output of 2^31 pieces).
 */
int ua2a_cache_read(ua2a_plan_t plan, const ua2a_cache_t* cache, int32_t type, int64_t n, const int32_t* starts,
                    const int32_t* counts, void* k_out, void* v_out, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* UA2A_ACT_H */
