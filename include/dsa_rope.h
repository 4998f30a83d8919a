/*
 * dsa_rope.h -- rotary position embedding with several position axes (part
 * of libdsa.so, CUDA, sm_103a).
 *
 * "Understanding and Exploiting Diagonal Attention Sparsity in
 * Autoregressive Image Generation" (arXiv 2609.19702), section 3, explains
 * the diagonals it exploits by the relative position of tokens in the image
 * grid; models of images and video give a token one position per axis (time,
 * row, column) and let each axis turn its own share of a head's pairs.  The
 * paper has no counterpart of these entry points.
 *
 * With r = pairs[0] + pairs[1] + .. <= head_dim / 2 rotated pairs, pair j
 * (elements j and j + head_dim / 2, the rotate-half form) of a token at
 * position pos[a] on the axis a that owns the pair turns by
 *
 *     angle = pos[a] * base^(-2 j / head_dim)            (restart == 0)
 *     angle = pos[a] * base^(-i / pairs[a])              (restart != 0)
 *
 * where the first pairs[0] pairs belong to axis 0, the next pairs[1] to axis
 * 1 and so on, and i counts the pair within its axis.  (x_j, x_j') becomes
 * (x_j cos - x_j' sin, x_j' cos + x_j sin); pairs j >= r pass unchanged.
 * One axis that owns all pairs is the rotation of dsa_qkv_rope.
 *
 * Arithmetic: base^(..) is a double, 2^-53 of it; its product with a position is
 * held as a 64-bit fraction of a turn, exact modulo a turn to 2^-32 turns at any
 * int32 position.  Sines and cosines are of that fraction in fp32, and they and
 * the rotation are fp32, rounded to the output type once.
 */
#ifndef DSA_ROPE_H
#define DSA_ROPE_H

#include <stddef.h>
#include <stdint.h>

#include "dsa.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct dsa_rope_ctx *dsa_rope; /* opaque; library-owned, host memory only */

/*
 * dsa_rope_create -- the plan of a rotation: head_dim 64 or 128, `axes` in
 * [1, 4], pairs (host, [axes]) each >= 1 with a sum of at most head_dim / 2,
 * base > 1 and finite.  Touches no device.  A plan is never written after
 * its creation: any number of calls, threads and streams may use it at once.
 * Errors: DSA_ERR_ARG, DSA_ERR_OOM.
 */
int dsa_rope_create(int head_dim, int axes, const int *pairs, int restart, double base, dsa_rope *out);

/* Frees the plan (launches that used it keep their own copy).  NULL is accepted. */
int dsa_rope_destroy(dsa_rope r);

/*
 * dsa_rope_apply -- rotates `heads` heads of `tokens` tokens.
 *
 * pos: device, [tokens, axes] int32, any values.
 * x, y: device, head h of token n at x + n * x_stride + h * head_dim
 *     elements of `dtype` (DSA_BF16 or DSA_F32), strides in elements, at
 *     least heads * head_dim and multiples of 16 bytes; 16-byte aligned.  q
 *     and k that lie side by side in a projection's output turn in one call.
 *     y may be x with the same stride (in place); otherwise they must not
 *     overlap.  What lies between the rows of y is left as it was.
 * inverse != 0 turns by the negative angles: the gradient of the rotation
 *     (dL/dx from dL/dy), and its inverse.
 *
 * heads in [1, 65536]; tokens == 0 is allowed.  Asynchronous on `stream`, no workspace; may be
 * captured.  Launched as a programmatic dependent launch: reads nothing
 * before the previous kernel of the stream has completed.
 * Errors: DSA_ERR_STATE (invalid plan), DSA_ERR_ARG, DSA_ERR_CUDA (launch).
 */
int dsa_rope_apply(dsa_rope r, int tokens, int heads, int dtype, const int32_t *pos, const void *x, int64_t x_stride,
                   void *y, int64_t y_stride, int inverse, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* DSA_ROPE_H */
