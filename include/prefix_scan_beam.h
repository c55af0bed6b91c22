/*
 * prefix_scan_beam.h -- C ABI of beam search's choice: of all tokens that the
 * beams of an item could go on with, the `width` best.
 *
 *     total(beam, token) = score(beam) + logits(beam, token) - log sum exp(logits(beam, .))
 *
 * What it returns is made for what comes after it: `parents` name the rows whose
 * pages ps_pages_fork or ps_pages_reorder (prefix_scan_pages.h) hand on.
 *
 * Order: by total; equal totals by the lower beam, then, within a beam, by the
 * larger logit, then by the lower token.  A beam's own candidates are compared by
 * their logits, exactly.  Totals of different beams are compared in 64 bits, but
 * each row's log sum exp comes from exponentials and sums of 32 bits: it is off by
 * 2^-19 at most, as a rule by 2^-22, so beams whose totals are closer than that may
 * change places.  Equal rows have equal sums, and results do not depend on
 * scheduling.
 *
 * What offers nothing: a token whose logit is -infinity; a beam whose score is not
 * finite; a beam with a NaN or +infinity among its logits.  Where fewer than
 * `width` candidates are left, the rest of the item's results have score
 * -infinity, parent -1 and token -1 (which the page operations take as a row with
 * no parent).  A total below what f32 can hold is chosen in its order like any
 * other; its score is returned as -infinity, with its parent and token.
 *
 * Beams at their end: where `ended` is not NULL and ended[row] != 0, the row's
 * logits are not read; it offers itself once, with its score as it is and
 * `eos_token` as its token.
 *
 * Conventions: device pointers owned by the caller; work is enqueued on
 * `stream` and the call returns without waiting for it; no device memory is
 * allocated and nothing is kept between calls; calls can be captured in CUDA
 * graphs.  Errors found on the host are returned before anything is enqueued:
 * PS_ERR_INVALID_ARG (a bad enum, size, stride or pointer),
 * PS_ERR_WORKSPACE_TOO_SMALL, PS_ERR_OVERLAP (an output that meets an input,
 * another output or the workspace), PS_ERR_CUDA.  The workspace needs no
 * preparation; calls that may run at the same time must not share one.
 */
#ifndef PREFIX_SCAN_BEAM_H
#define PREFIX_SCAN_BEAM_H

#include "prefix_scan_delta.h"

#ifdef __cplusplus
extern "C" {
#endif

#define PS_BEAM_MAX_BEAMS 256
#define PS_BEAM_MAX_WIDTH 64

/*
 * batch         items (0: nothing to do)
 * beams, width  beams of an item, at most 256; candidates to choose, at most 64
 * vocab         tokens
 * item_stride, beam_stride  of the logits, in elements; a row's logits are
 *               contiguous
 * type          of the logits: f32, bf16 or f16
 * eos_token     the token that ends a beam, -1 for none
 * batch * beams and batch * width are at most 2^31 - 1.
 */
typedef struct ps_beam_shape {
    int64_t batch;
    int32_t beams;
    int32_t width;
    int64_t vocab;
    int64_t item_stride;
    int64_t beam_stride;
    ps_real type;
    int32_t eos_token;
} ps_beam_shape;

/* Bytes of workspace of ps_beam_select (0 for shapes that it refuses).  256-byte aligned. */
size_t ps_beam_workspace_size(const ps_beam_shape *shape);

/*
 *   logits       device, of shape->type
 *   scores       device f32 [batch, beams]
 *   ended        device uint8 [batch, beams], or NULL
 *   out_scores   device f32 [batch, width], best first
 *   out_parents  device int32 [batch, width]: item * beams + beam
 *   out_tokens   device int32 [batch, width]
 *   out_ended    device uint8 [batch, width], or NULL: 1 where the parent had ended
 *                or the token is eos_token
 * out_ended may not be `ended`.
 */
ps_status ps_beam_select(const ps_beam_shape *shape, const void *logits, const float *scores, const uint8_t *ended,
                         float *out_scores, int32_t *out_parents, int32_t *out_tokens, uint8_t *out_ended, void *ws,
                         size_t ws_bytes, ps_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* PREFIX_SCAN_BEAM_H */
