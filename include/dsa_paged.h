/*
 * dsa_paged.h -- decode attention over a paged KV cache: appending keys and
 * values with the position rotation on the way, and dense causal attention
 * over what the cache holds (part of libdsa.so, CUDA, sm_103a).
 *
 * The streams of a dsa_handle step together and own their rows.  A serving
 * engine has sequences of unequal length that come and go: it keeps one pool
 * of fixed-size pages per layer and a table of each sequence's pages.  This
 * is the dense setting of the method ("Understanding and Exploiting Diagonal
 * Attention Sparsity in Autoregressive Image Generation", arXiv 2609.19702:
 * N_r = N_att = L_dec) over such a pool, with grouped queries and
 * several new tokens per call.  The paper has no counterpart of the pages.
 *
 * The pool (device memory of the caller, e.g. the engine's KV arena):
 *   pages   [num_pages, kv_heads, page_size, 2, head_dim]: per token its K
 *           row, then its V row, in bf16 (DSA_BF16) or E4M3 codes
 *           (DSA_FP8_E4M3)
 *   scales  [num_pages, kv_heads, 2] float (DSA_FP8_E4M3 only): the scale of
 *           the K codes and of the V codes of one page and KV head
 * The batch of a call (device memory; nothing of it is read on the host, so
 * a captured call can be replayed with other contents):
 *   cu      [n_seqs + 1] int32: rows cu[s] .. cu[s + 1] - 1 of the packed
 *           inputs are the new tokens of sequence s (none: it is left out)
 *   lens    [n_seqs] int32: tokens of sequence s, its new ones included; new
 *           token i of n takes position lens[s] - n + i
 *   table   [n_seqs, table_width] int32: page of positions
 *           [page_size * p, page_size * (p + 1)) in entry p; entries beyond
 *           the sequence's last page are not read
 * Rows at and behind cu[n_seqs] (a padded batch) are neither read nor
 * written.
 *
 * What the host cannot check, the kernels do: a sequence whose cu, lens do
 * not fit (cu decreasing or beyond n_tokens, lens negative, shorter than its
 * new tokens or beyond the table) is left out, its rows unwritten; a page
 * number outside the pool holds zeros to the attention and is not appended
 * to.  Both set DSA_ERR_DEVICE_CHECK in the handle's sticky status
 * (dsa_paged_sync_status).
 */
#ifndef DSA_PAGED_H
#define DSA_PAGED_H

#include <stddef.h>
#include <stdint.h>

#include "dsa.h"
#include "dsa_rope.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct dsa_paged_ctx *dsa_paged; /* opaque; library-owned */

/*
 * dsa_paged_create -- binds a pool.
 *
 * q_heads a multiple of kv_heads (query head h reads KV head
 * h / (q_heads / kv_heads)), kv_heads in [1, 1024]; head_dim 64 or 128;
 * page_size 16, 32, 64 or 128; num_pages >= 1 with num_pages * kv_heads *
 * page_size < 2^31; dtype DSA_BF16 or DSA_FP8_E4M3; pages 128-byte aligned,
 * scales 16-byte aligned (NULL for DSA_BF16), both on the current device.  The pool must outlive the
 * handle; its contents are the caller's to copy, share between sequences
 * (pages of a common prefix) or give to another sequence.  Allocates on the
 * current device a workspace for pieces of long sequences (at most 24 MiB)
 * and a status word.  Errors: DSA_ERR_ARG, DSA_ERR_OOM, DSA_ERR_CUDA.
 */
int dsa_paged_create(int q_heads, int kv_heads, int head_dim, int page_size, int num_pages, int dtype, void *pages,
                     float *scales, dsa_paged *out);

/* Frees the handle, not the pool (synchronizes the device first).  NULL is accepted. */
int dsa_paged_destroy(dsa_paged h);

/*
 * dsa_paged_append -- writes the new tokens' keys and values into their
 * pages, with k (and q) rotated on the way.
 *
 * q: device bf16, [n_tokens, q_heads, head_dim], row stride q_stride; its
 *     rotated form goes to q_out ([n_tokens, q_heads, head_dim], contiguous;
 *     may be q itself where q is contiguous).  Both NULL: only k and v.
 * k, v: device bf16, [n_tokens, kv_heads, head_dim], row strides k_stride,
 *     v_stride.  Strides in elements, multiples of 8, at least one row;
 *     16-byte aligned.  They may lie side by side in a projection's output.
 * rope, pos: the rotation plan (its head_dim the handle's) and device int32
 *     positions [n_tokens, axes]; both NULL: no rotation.
 *
 * DSA_BF16 rounds once to bf16.  DSA_FP8_E4M3 stores the E4M3 code nearest
 * to fp32 value / scale (ties to even, magnitudes beyond 448 saturate, NaN
 * stays NaN).  The scale of a page, head and K / V is a power of two, 2^e
 * with e in [-72, 120]: a floating-point code loses nothing to it, and codes
 * move to a larger one by their exponents.  e is the smallest for which the
 * largest finite |v| of the page's new tokens is at most 448 * 2^e; for K the
 * norm of a rotated pair (which the rotation leaves alone; its square rounded to
 * the 24 bits of fp32, of any exponent) takes the place of |v|, so a scale depends on neither position nor rounding.  A
 * token in slot 0 starts the page's scale anew; later tokens keep the larger
 * of the old and the new, and where it grows the codes of the earlier tokens
 * become the codes nearest to code * old / new (exact but for subnormals).
 *
 * Within one call a page may be appended to by one sequence only, and no
 * other call may use that page at the same time.
 * n_tokens == 0 or n_seqs == 0 is allowed.  Asynchronous on `stream`; a
 * programmatic dependent launch that reads nothing before the previous
 * kernel of the stream has completed; may be captured; needs no workspace,
 * so appends through one handle may overlap on other pages.
 * Errors: DSA_ERR_STATE (invalid handle or plan), DSA_ERR_ARG, DSA_ERR_CUDA.
 */
int dsa_paged_append(dsa_paged h, int n_seqs, int n_tokens, const int32_t *cu, const int32_t *lens,
                     const int32_t *table, int table_width, dsa_rope rope, const int32_t *pos, const void *q,
                     int64_t q_stride, const void *k, int64_t k_stride, const void *v, int64_t v_stride, void *q_out,
                     void *stream);

/*
 * dsa_paged_attend -- out = softmax(q K^T / sqrt(head_dim)) V per new token
 * and query head, over the sequence's tokens up to and including the new
 * token itself (lens and cu as for the append that came before).
 *
 * q, out: device bf16, [n_tokens, q_heads, head_dim], contiguous, 16-byte
 *     aligned, n_tokens * q_heads < 2^31; out may be q.
 * max_new >= 1: no sequence has more new tokens than this; a hint that only
 *     chooses the launch.  Any value gives the same result up to the rounding
 *     of the weights (below) and fp32 rounding order; one far too small reads
 *     the cache many times over.
 *
 * Slots behind a sequence's last token may hold anything (NaN included).  A
 * row whose logits hold a NaN is NaN; so are, among the new tokens of the
 * sequence, rows that a NaN or infinity in a later new token's V meets.
 * Products are exact, sums and softmax statistics fp32.  For DSA_FP8_E4M3 an
 * element of q enters the first product to 8 significant bits and 2^-21 of its
 * row's largest.  The weights enter the second product with 16 significant
 * bits (DSA_BF16, max_new x grouped query heads at most 16), 8 (DSA_BF16, more)
 * or 9 (DSA_FP8_E4M3; those under 2^-17 of the row's largest product of a weight
 * and its page's V scale fewer, to 2^-26 of that product), and the result is
 * rounded to bf16 once.
 * Deterministic for given arguments: pieces of one row are joined in the
 * order of their keys.
 * n_tokens == 0 or n_seqs == 0 is allowed.  Asynchronous on `stream`; a
 * programmatic dependent launch that reads nothing before the previous
 * kernel of the stream has completed; may be captured.  Calls of one handle
 * share its workspace: they must not overlap (one stream, or ordered
 * streams; replays of graphs that hold such calls likewise).
 * Errors: DSA_ERR_STATE (invalid handle), DSA_ERR_ARG, DSA_ERR_CUDA;
 * device-side faults via dsa_paged_sync_status.
 */
int dsa_paged_attend(dsa_paged h, int n_seqs, int n_tokens, int max_new, const int32_t *cu, const int32_t *lens,
                     const int32_t *table, int table_width, const void *q, void *out, void *stream);

/*
 * Waits for `stream` and reports the handle's sticky device status:
 * DSA_ERR_TIMEOUT (a bounded wait of the attention gave up; the outputs of
 * that call are undefined) or DSA_ERR_DEVICE_CHECK (a sequence or page that
 * does not fit, see above).  Reading an error resets it; of two the timeout is
 * reported first and the other by the next reading.
 */
int dsa_paged_sync_status(dsa_paged h, void *stream);

/* Test knob: the polls each bounded wait of the attention makes before it
 * gives up (0: at once; default: unbounded polls, one second of wall time). */
int dsa_paged_set_wait_limit(dsa_paged h, uint32_t limit);

#ifdef __cplusplus
}
#endif

#endif /* DSA_PAGED_H */
