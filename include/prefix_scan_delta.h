/*
 * prefix_scan_delta.h -- C ABI of the gated delta rule: the recurrence of
 * matrix-valued states that a linear-attention layer runs over its tokens.
 * It is the scan of affine maps (ps_scan_affine_f32) with K x V matrices in
 * place of numbers:
 *
 *     S <- exp(g) S;   u = beta (v - k^T S);   S <- S + k u^T;   o = scale q^T S
 *
 * for each value head of each sequence, token after token, with a key k and
 * a query q of K numbers, a value v of V numbers, a log decay g and a gate
 * beta.  A key head serves heads_v / heads_k consecutive value heads.
 *
 * Types: q, k, v and o are of one type (f32, bf16 or f16); beta of that type
 * or f32; g, states and gradients of states and of g are f32.  States and all
 * sums are held in 32 bits; over whole sequences matrix products take operands
 * of 16 significant bits (pairs of bf16), f32 q, k and d_o among them, so results
 * carry errors of about 2^-18 relative to the terms that make them up, before
 * their own rounding: chosen for the matrix units' speed, see
 * csrc/delta_common.cuh.  Single steps are f32 throughout.  ps_delta_step takes
 * any number of tokens, so a caller who needs f32's 24 bits of a prompt runs it
 * there, token after token (1111 tokens in three sequences, 3 heads of 80 x 56:
 * off by 1.3e-7 in 492 us, against 5.0e-6 in 88); training has the pairs alone.
 *
 * Extreme inputs: a log decay at or below -87 (-infinity too), where exp(g)
 * leaves the normal range of f32, forgets the state entirely and has gradient
 * 0.  Log decays above 0 make states grow; sums of them over 64 tokens have to
 * stay below 80.  A gate of 0 counts as 2^-60.  NaN and infinities reach the
 * outputs of their own sequence, and of the heads that share the input, and
 * no others (within a chunk of 64 tokens also those before them).
 *
 * A kernel whose bounded waits ran out, which a correct launch never does,
 * finishes instead of hanging, with NaN in the outputs that it is to blame for:
 * a chain's o and state at the end, a step's o (the states in its pages are
 * undefined then).  In training all gradients are NaN from then on, until the
 * next forward call on that workspace.
 *
 * Conventions: device pointers owned by the caller; work is enqueued on
 * `stream` and the call returns without waiting for it; no device memory is
 * allocated and nothing is kept between calls; calls can be captured in CUDA
 * graphs.  Errors found on the host are returned before anything is enqueued:
 * PS_ERR_INVALID_ARG (a bad enum, size, stride or pointer),
 * PS_ERR_WORKSPACE_TOO_SMALL, PS_ERR_OVERLAP (an output that meets an input,
 * another output or the workspace), PS_ERR_CUDA.  The workspace needs no
 * preparation.
 */
#ifndef PREFIX_SCAN_DELTA_H
#define PREFIX_SCAN_DELTA_H

#include "prefix_scan.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum ps_real { PS_REAL_F32 = 0, PS_REAL_BF16 = 1, PS_REAL_F16 = 2 } ps_real;

/*
 * A tensor over (sequence, token, head, innermost): strides in elements; the
 * innermost dimension (K or V numbers; none for g and beta) is contiguous.
 * For packed sequences the token index runs over all of them and seq_stride
 * is not used.  Rows that start on 16-byte boundaries and hold a multiple of
 * eight numbers are read in whole 16-byte pieces, others number by number.
 */
typedef struct ps_delta_tensor {
    const void *data;
    int64_t seq_stride;
    int64_t tok_stride;
    int64_t head_stride;
} ps_delta_tensor;

/* The inputs of a call come as an array of five tensors in this order. */
typedef enum ps_delta_input { PS_DELTA_Q = 0, PS_DELTA_K = 1, PS_DELTA_V = 2, PS_DELTA_G = 3, PS_DELTA_BETA = 4 } ps_delta_input;

/*
 * num_seqs   sequences (0: nothing to do)
 * tokens     tokens of every sequence; with cu_seqlens, of all together
 * cu_seqlens NULL, or a device array of num_seqs + 1 offsets: sequence i has
 *            tokens [cu[i], cu[i+1]).  Offsets are read on the device and
 *            clamped into [0, tokens]; an end before its start is an empty
 *            sequence.  They must not fall: sequences that share tokens then
 *            write the same outputs and the same workspace, so results are
 *            unspecified, and may differ from call to call, for all
 *            sequences; no access leaves the tensors.
 * heads_k, heads_v, dim_k, dim_v  heads_v is a multiple of heads_k; dim_k at
 *            most 128, dim_v at most 1024
 */
typedef struct ps_delta_shape {
    int64_t num_seqs;
    int64_t tokens;
    const int32_t *cu_seqlens;
    int32_t heads_k;
    int32_t heads_v;
    int32_t dim_k;
    int32_t dim_v;
    ps_real type;        /* of q, k, v, o and their gradients */
    ps_real beta_type;   /* PS_REAL_F32, or `type` */
    float scale;
} ps_delta_shape;

/*
 * Bytes of workspace of ps_delta_forward and, with train != 0, of the buffer
 * that a training step's forward call leaves for ps_delta_backward (0 for
 * shapes that the calls refuse).  256-byte aligned.
 */
size_t ps_delta_workspace_size(const ps_delta_shape *shape, int train);

/*
 * Forward over whole sequences, in chunks of 64 tokens.
 *   h0  [num_seqs, heads_v, dim_k, dim_v] f32 states at the start, NULL for 0
 *   ht  the same shape, receives the states at the end; may be NULL or h0
 *   o   contiguous [tokens of all sequences, heads_v, dim_v]; tokens that no
 *       sequence holds are left as they are
 *   train != 0: `ws` keeps what ps_delta_backward reads
 * An empty sequence hands its state on.
 */
ps_status ps_delta_forward(const ps_delta_shape *shape, const ps_delta_tensor inputs[5], const float *h0, float *ht,
                           void *o, int train, void *ws, size_t ws_bytes, ps_stream_t stream);

/*
 * Backward of one ps_delta_forward(train != 0) call with the same shape, q
 * and k; `ws` is that call's workspace, which any number of backward calls may
 * use one after the other but which must not change otherwise.
 *   d_o   gradient of o;  d_ht  gradient of ht or NULL (0)
 *   dq, dk [.., heads_k, dim_k], dv [.., heads_v, dim_v], dbeta, dg
 *         [.., heads_v]: contiguous; dq and dk are summed over the value
 *         heads that share a key head, in a fixed order
 *   dh0   gradient of h0, or NULL
 * Gradients of tokens that no sequence holds are 0.
 * Results are bitwise reproducible from call to call (no atomics) where offsets
 * do not fall.
 */
ps_status ps_delta_backward(const ps_delta_shape *shape, const ps_delta_tensor *q, const ps_delta_tensor *k,
                            const ps_delta_tensor *d_o, const float *d_ht, void *dq, void *dk, void *dv,
                            float *dg, void *dbeta, float *dh0, void *ws, size_t ws_bytes, ps_stream_t stream);

/*
 * The recurrence for the next token or few of many sequences, on states that
 * lie in pages of a pool.
 *   tokens    t >= 0 tokens of each sequence (shape->cu_seqlens must be NULL)
 *   state     contiguous [pages, heads_v, dim_k, dim_v] f32, advanced in place
 *   slots     device [num_seqs]: the page of each sequence's state; pages must
 *             differ.  An index outside [0, pages) (-1, say) is a sequence
 *             that takes no part: its outputs are 0.  NULL: page i for i.
 *   lengths   device [num_seqs]: how many of the t tokens count (clamped to
 *             [0, t]); outputs past them are 0.  NULL: all of them.
 *   o         contiguous [num_seqs, t, heads_v, dim_v]
 * No workspace.
 */
ps_status ps_delta_step(const ps_delta_shape *shape, const ps_delta_tensor inputs[5], float *state, int64_t pages,
                        const int32_t *slots, const int32_t *lengths, void *o, ps_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* PREFIX_SCAN_DELTA_H */
