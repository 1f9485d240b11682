/*
 * gma_block.h -- C ABI of libgma.so, second part: the operators that stand next to the latent-
 * routing mixer in a block.
 *
 *   gma_scan_*  the selective state space scan, the other mixer with a fixed state per sequence;
 *   gma_conv_*  the short causal convolution per channel in front of it;
 *   gma_norm_*  the norms before and after a block, fused with its gate and residual scale.
 *
 * Conventions shared by these entry points
 *   - Everything gma.h says about ownership, streams and errors holds: device memory of the
 *     current CUDA device, caller-owned buffers, no allocation and no synchronisation, all work
 *     on `stream`, argument errors before anything is enqueued, status codes of gma_status_t.  Calls from
 *     several host threads at once are fine.
 *   - Activations are bf16 or fp32 (gma_dtype_t) in token-major rows: gma_rows_t names a tensor
 *     [B][N][width] by its first element and the strides, in elements, between batch rows and
 *     between tokens.  The channels of one token are contiguous; rows may be part of a wider
 *     projection's rows, and any element alignment is taken.  Rows whose addresses and strides are
 *     multiples of 16 bytes take wider accesses.  Output rows must not overlap one another or any
 *     input, unless an entry point says so.  Strides are >= 0.
 *   - Parameters and states are fp32 and contiguous; the scan's a_log, states and checkpoints start on
 *     16-byte boundaries.  Sums, states and statistics are held in fp32.
 *   - `lengths` (NULL, or B int32 in device memory) gives every batch row's number of tokens, taken
 *     as min(max(length, 0), N): the rows behind a sequence's last token are neither read nor
 *     written (with GMA_ROWS_ZERO_TAIL: are written as zeros), and the states that come out are those
 *     after the last token.
 *   - The workspace is 256-byte aligned, needs no initialisation, holds nothing between calls and
 *     has no error word (no kernel behind these entry points waits for another one's signal).
 *     Calls that share one are ordered on the GPU.  Where gma_*_workspace_size gives 0 for valid
 *     arguments, NULL will do.
 *   - Repeated calls on the same inputs give the same bits.
 */
#ifndef GMA_BLOCK_H
#define GMA_BLOCK_H

#include "gma.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Flags of the scan and the convolution: zeros in the output rows (of gradients too) behind a
 * sequence's last token, for buffers that hold anything. */
#define GMA_ROWS_ZERO_TAIL 0x2u

typedef struct {
    void *ptr;             /* first element; NULL: not given */
    int64_t batch, token;  /* strides in elements            */
} gma_rows_t;

/* ------------------------------------------------------------------ selective state space scan
 *
 * Per batch row, channel d (of D) and state n (of S), with group g = d / (D / G):
 *     delta_t = softplus(dt_t[d] + dt_bias[d]),   A[d][n] = -exp(a_log[d][n]),
 *     h_t[d][n] = exp(delta_t A[d][n]) h_{t-1}[d][n] + delta_t b_t[g][n] u_t[d],
 *     p_t[d] = sum_n c_t[g][n] h_t[d][n] + d_skip[d] u_t[d],
 *     y_t[d] = p_t[d] silu(z_t[d])          (y = p without z).
 * S in {8, 16, 32, 64}; 1 <= G, G divides D; 1 <= B <= 65535, 1 <= N <= 2^30, 1 <= D <= 2^24 (the backward
 * pass: N <= 64 * 65535, D * S < 2^30, G <= 65535, B * G * ceil(N * S / 512) < 2^30). */
typedef struct {
    int32_t B, N, D, S, G;
    int32_t dtype;                /* of u, dt, z, b, c, y and their gradients               */
    uint32_t flags;               /* GMA_ROWS_ZERO_TAIL or 0                                 */
    uint32_t reserved;            /* 0                                                       */
    gma_rows_t u, dt, z;          /* [B][N][D]; z may be NULL                                */
    gma_rows_t b, c;              /* [B][N][G][S], a token's G * S values contiguous         */
    const float *a_log;           /* [D][S]                                                  */
    const float *d_skip;          /* [D] or NULL (0)                                         */
    const float *dt_bias;         /* [D] or NULL (0)                                         */
    const float *state_in;        /* [B][D][S] or NULL (zeros): the state before token 0     */
    float *state_out;             /* [B][D][S] or NULL; may be state_in                      */
    const int32_t *lengths;       /* [B] or NULL                                             */
    gma_rows_t y;                 /* [B][N][D] out                                           */
    float *checkpoints;           /* out: the states gma_scan_backward starts from, or NULL  */
} gma_scan_t;

/* `checkpoints` is [B][ceil(N / t)][D][S], the state before every t-th token, with
 * t = gma_scan_checkpoint_tokens (64 or 16, by B, N, D and S, the only fields that these two look at); its
 * bytes.  Both are 0 for sizes that no call takes. */
int gma_scan_checkpoint_tokens(const gma_scan_t *scan);
size_t gma_scan_checkpoint_size(const gma_scan_t *scan);
size_t gma_scan_workspace_size(const gma_scan_t *scan);
gma_status_t gma_scan_forward(const gma_scan_t *scan, void *workspace, size_t workspace_bytes,
                              gma_stream_t stream);

/* One token for every batch row: N is 1, state_in and state_out are required (normally the same
 * buffer), lengths and checkpoints must be NULL; the token strides are ignored. */
gma_status_t gma_scan_step(const gma_scan_t *scan, gma_stream_t stream);

/* The gradients of sum(dy * y) + sum(dstate_out * state_out).  `fwd` holds the forward call's
 * arguments, `checkpoints` as that call wrote them (an input here); its y and state_out are not
 * used.  Parameter gradients are summed over batch and tokens; outputs are written, not
 * accumulated. */
typedef struct {
    gma_scan_t fwd;
    gma_rows_t dy;                /* [B][N][D]                                               */
    const float *dstate_out;      /* [B][D][S] or NULL (zeros)                               */
    gma_rows_t du, ddt, dz;       /* [B][N][D]; dz required with z                           */
    gma_rows_t db, dc;            /* [B][N][G][S]                                            */
    float *da_log;                /* [D][S]                                                  */
    float *dd_skip;               /* [D], required with d_skip                               */
    float *ddt_bias;              /* [D], required with dt_bias                              */
    float *dstate_in;             /* [B][D][S] or NULL                                       */
} gma_scan_grad_t;

/* About B * N * G * 8 S * ceil(D S / (1024 G)) bytes: S^2 / 128 a (token, channel), 2 at 16 states and 32 at 64, and
 * the states of every chunk beside them. */
size_t gma_scan_backward_workspace_size(const gma_scan_grad_t *grad);
gma_status_t gma_scan_backward(const gma_scan_grad_t *grad, void *workspace, size_t workspace_bytes,
                               gma_stream_t stream);

/* ------------------------------------------------------------------ short causal convolution
 *
 * Per batch row and channel, taps k = 0 .. W - 1, with x_{-1}, ..., x_{-(W-1)} the state's rows:
 *     p_t = sum_k weight[d][k] x_{t - W + 1 + k}[d] + bias[d],   y_t = silu(p_t), or p_t.
 * W in {2, 3, 4}; 1 <= B <= 65535, 1 <= N <= 2^30, 1 <= D <= 2^24, B, N and D such that the runs of tokens (at most 256
 * each) of four channels stay below 2^31.  The state is the last W - 1 inputs, oldest first, in dtype. */
#define GMA_CONV_LINEAR 0x1u      /* y_t = p_t */

typedef struct {
    int32_t B, N, D, W;
    int32_t dtype;                /* of x, y, the states and the gradients of x              */
    uint32_t flags;               /* GMA_CONV_LINEAR, GMA_ROWS_ZERO_TAIL                     */
    gma_rows_t x;                 /* [B][N][D]                                               */
    const float *weight;          /* [D][W]                                                  */
    const float *bias;            /* [D] or NULL (0)                                         */
    const void *state_in;         /* [B][W - 1][D] or NULL (zeros)                           */
    void *state_out;              /* [B][W - 1][D] or NULL; may be state_in in gma_conv_step */
    const int32_t *lengths;       /* [B] or NULL                                             */
    gma_rows_t y;                 /* [B][N][D] out                                           */
} gma_conv_t;

gma_status_t gma_conv_forward(const gma_conv_t *conv, gma_stream_t stream);

/* One token for every batch row: N is 1, state_in and state_out are required (normally the same
 * buffer), lengths must be NULL; the token strides are ignored. */
gma_status_t gma_conv_step(const gma_conv_t *conv, gma_stream_t stream);

/* The gradients of sum(dy * y).  `fwd` holds the forward call's arguments; its y and state_out
 * are not used.  The state's rows count as constants. */
typedef struct {
    gma_conv_t fwd;
    gma_rows_t dy, dx;            /* [B][N][D]                                               */
    float *dweight;               /* [D][W]                                                  */
    float *dbias;                 /* [D], required with bias                                 */
} gma_conv_grad_t;

size_t gma_conv_backward_workspace_size(const gma_conv_grad_t *grad);
gma_status_t gma_conv_backward(const gma_conv_grad_t *grad, void *workspace, size_t workspace_bytes,
                               gma_stream_t stream);

/* ------------------------------------------------------------------ norms around a block
 *
 * Per token, over D = H * d channels (channel h * d + j is element j of head h):
 *     a = o silu(gate)                                            (a = o without gate)
 *     v = w_post a / sqrt(mean(a^2) + eps), the mean over groups of `group` channels
 *                                                                 (v = a without w_post)
 *     r' = residual + scale v, stored in residual_dtype           (r' = v in dtype without residual)
 *     h = w_pre r' / sqrt(mean(r'^2) + eps), of r' as stored      (no h without w_pre)
 * o is the mixers' output layout [B][H][N][d], by strides.  1 <= D <= 16384; group is D, or 8, 16, 32,
 * 64, 128 or 256 and divides D; B * N <= 2^30.  A residual is required for scale; w_post or w_pre is
 * required. */
typedef struct {
    int32_t B, N, H, d;
    int32_t group;                /* channels per group of the first norm (D: one group)     */
    int32_t dtype;                /* of o, gate, h and, without a residual, r                */
    int32_t residual_dtype;       /* of residual and r; dtype, or fp32                       */
    float eps;                    /* >= 0                                                    */
    gma_rows_t o;                 /* [B][H][N][d], strides of batch rows and tokens          */
    int64_t o_head;               /* stride between o's heads, in elements                   */
    gma_rows_t gate, residual;    /* [B][N][D] or NULL                                       */
    const float *w_post;          /* [D] or NULL                                             */
    const float *scale;           /* [D] or NULL (1)                                         */
    const float *w_pre;           /* [D] or NULL                                             */
    gma_rows_t r, h;              /* [B][N][D] out; r may be residual (the same strides); h required with w_pre */
} gma_norm_t;

gma_status_t gma_norm_forward(const gma_norm_t *norm, gma_stream_t stream);

/* The gradients of sum(dr * r') + sum(dh * h).  `fwd` holds the forward call's arguments with r as
 * that call wrote it (an input here, needed with w_pre); its residual values and h are not used,
 * but residual.ptr tells whether there was one (it may be r's). */
typedef struct {
    gma_norm_t fwd;
    gma_rows_t dr;                /* [B][N][D] in r's type; may be NULL when dh is given     */
    gma_rows_t dh;                /* [B][N][D] in dtype, or NULL                             */
    gma_rows_t d_o;               /* [B][H][N][d] in dtype, strides of batch rows and tokens */
    int64_t d_o_head;             /* stride between its heads                                */
    gma_rows_t dgate;             /* [B][N][D] in dtype, required with gate                  */
    gma_rows_t dresidual;         /* [B][N][D] in residual_dtype, or NULL; may be dr (the same strides) */
    float *dw_post, *dscale, *dw_pre; /* [D], required with the parameter                    */
} gma_norm_grad_t;

size_t gma_norm_backward_workspace_size(const gma_norm_grad_t *grad);
gma_status_t gma_norm_backward(const gma_norm_grad_t *grad, void *workspace, size_t workspace_bytes,
                               gma_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* GMA_BLOCK_H */
