/*
 * ssm_gated.h -- C ABI of the gated linear recurrence: forward scan, backward, one-token step.
 *
 * A state per channel, decayed by one gate and fed through another; the sibling of the
 * selective scan of ssm_scan.h for models whose recurrence has no B and C.  For every batch
 * row b and channel d (r and i are the gates' pre-activations):
 *   rho_t  = sigmoid(r[b,d,t] + r_bias[d])        recurrence gate
 *   iota_t = sigmoid(i[b,d,t] + i_bias[d])        input gate
 *   v_t    = c * softplus(lam[d]) * rho_t         decay exponent
 *   a_t    = exp(-v_t),   m_t = sqrt(1 - a_t^2)   decay, and the input weight that keeps |h| bounded
 *   h_t    = a_t h_{t-1} + m_t iota_t x[b,d,t]
 *   y_t    = h_t * silu(z[b,d,t])                 (y_t = h_t without z)
 *   h_{-1} = 0 (or a given initial state);  last_state = h_{length-1}
 *
 * Conventions: those of ssm_scan.h (device pointers owned by the caller, no device memory
 * allocated, calls asynchronous on `stream`, status codes), and:
 *   - x, r, i, z, y and their gradients have io_dtype elements (fp32 or bf16), shape (batch, dim,
 *     seqlen) with consecutive steps next to each other; the batch and channel strides are given (in
 *     elements; those of an input may be zero or negative), so that slices of a wider tensor, such
 *     as the three parts of one projection's output, are taken as they are.  Any alignment of the
 *     elements' own size.  What lies between an operand's first and last row has to be readable
 *     memory: a few elements beside a row may be read with it (and are never used).
 *   - lam, r_bias, i_bias, their gradients and every state are fp32 and dense; arithmetic is fp32.
 *   - lengths  NULL, or int32 (batch) on the device: row b has lengths[b] steps (values outside
 *     0 .. seqlen are taken as the nearest of the two).  What lies behind them is not read for any
 *     result, y there is left as it was, and the gradients there are written as zeros.  A row of
 *     length 0 leaves last_state = initial_state.
 *   - reset    NULL, or one byte per (batch, seqlen), dense: where it is not zero a new document of
 *     a packed row begins: a_t = 0 and m_t = 1, so that h_t = iota_t x_t whatever came before
 *     (infinities and NaNs included), and no gradient passes back over the border.
 *   - An output may not be the same buffer as an input, nor may its own rows overlap (both
 *     SSM_ERR_INVALID_ARG); it must not overlap another argument.  Only a state's two ends may be
 *     the same buffer: initial_state and last_state, dlast_state and dinitial_state.
 *   - Every sum is formed in a fixed order: repeated calls give identical results.  (A row is taken in groups that
 *     lie on 16 bytes, so the same row at another offset from them may differ in its last bits.)
 *   - batch * dim < 2^31, seqlen < 2^31 - 65536; a one-token step: batch <= 65535, dim < 2^31 - 65536
 *     (else SSM_ERR_UNSUPPORTED).
 */
#ifndef SSM_GATED_H
#define SSM_GATED_H

#include "ssm_scan.h"

#ifdef __cplusplus
extern "C" {
#endif

/* A (batch, dim, seqlen) operand: address and strides in elements. */
typedef struct {
    const void* data;
    int64_t batch_stride, dim_stride;
} ssm_gated_in_t;
typedef struct {
    void* data;
    int64_t batch_stride, dim_stride;
} ssm_gated_out_t;

/* What forward and backward read alike.  Zero-initialise the whole struct. */
typedef struct {
    ssm_gated_in_t x, r, i;      /* required                                                         */
    ssm_gated_in_t z;            /* data NULL: no output gate                                        */
    const float* lam;            /* (dim), required                                                  */
    const float* r_bias;         /* (dim) or NULL (0)                                                */
    const float* i_bias;         /* (dim) or NULL (0)                                                */
    const float* initial_state;  /* (batch, dim) or NULL (0)                                         */
    const int32_t* lengths;      /* (batch) or NULL (every row has seqlen steps)                     */
    const uint8_t* reset;        /* (batch, seqlen) or NULL (none)                                   */
    int64_t seqlen;
    int32_t batch, dim;
    int32_t io_dtype;            /* ssm_dtype_t of x, r, i, z, y, dy and the gradients of the inputs */
    float c;                     /* decay constant, finite and > 0                                   */
} ssm_gated_args_t;

/*
 * Bytes of the checkpoints of a forward call (a multiple of 16; 0 for invalid sizes): the state
 * before every eighth step, in a layout of the library's own.  Given to the backward of the
 * same inputs they save it a second forward pass.
 */
size_t ssm_gated_checkpoint_size(int batch, int dim, int64_t seqlen);

/*
 * Forward scan.  y is required; last_state (batch, dim) and checkpoints (16-byte aligned, of at least
 * ssm_gated_checkpoint_size() bytes, else SSM_ERR_WORKSPACE) may be NULL.
 */
ssm_status_t ssm_gated_scan_fwd(const ssm_gated_args_t* args, const ssm_gated_out_t* y, float* last_state, void* checkpoints,
                                size_t checkpoint_bytes, ssm_stream_t stream);

/* The gradients of a loss L for the backward.  Zero-initialise the whole struct. */
typedef struct {
    ssm_gated_in_t dy;           /* dL/dy, required                                                  */
    const float* dlast_state;    /* (batch, dim) or NULL (0)                                         */
    ssm_gated_out_t dx, dr, di;  /* required                                                         */
    ssm_gated_out_t dz;          /* required with z, else ignored                                    */
    float* dlam;                 /* (dim) each, summed over batch rows and steps; NULL: not wanted   */
    float* dr_bias;
    float* di_bias;              /* (as if the biases were given, also when they are NULL)           */
    float* dinitial_state;       /* (batch, dim) or NULL                                             */
} ssm_gated_grads_t;

/*
 * Bytes of device workspace of ssm_gated_scan_bwd (a multiple of 256; 0 for invalid sizes);
 * smaller when the forward's checkpoints are given to the backward.
 */
size_t ssm_gated_bwd_workspace_size(int batch, int dim, int64_t seqlen, int have_checkpoints);

/*
 * Backward of ssm_gated_scan_fwd.  With g_t the gradient reaching h_t,
 *   g_t = dy_t silu(z_t) + a_{t+1} g_{t+1}      (dlast_state at the last step)
 *   dz  = dy h silu'(z),  dx = g m iota,  di = g m x iota (1 - iota),
 *   T_t = g a (iota x a v / m - h_{t-1} v)      (dL / d log v; v / m -> 0 with v)
 *   dr  = T (1 - rho),  dlam = sigmoid(lam) / softplus(lam) sum T,  d initial_state = a_0 g_0.
 *   checkpoints  NULL, or those that a forward call with the same args stored; the backward then
 *                skips its own forward pass.
 *   workspace    device buffer of at least ssm_gated_bwd_workspace_size() bytes, 256-byte aligned,
 *                not initialised; not to be used by two calls that can overlap on the GPU.
 */
ssm_status_t ssm_gated_scan_bwd(const ssm_gated_args_t* args, const ssm_gated_grads_t* grads, const void* checkpoints,
                                size_t checkpoint_bytes, void* workspace, size_t workspace_bytes, ssm_stream_t stream);

/* One-token step.  Zero-initialise the whole struct. */
typedef struct {
    float* state;                /* (slots, dim) fp32, read, modified and written in place           */
    int64_t state_stride;        /* elements from slot to slot                                       */
    const int32_t* slots;        /* (batch) on the device: the slot of each row; NULL: row b uses slot b */
    const void *x, *r, *i, *z;   /* io_dtype (batch, dim); z may be NULL                             */
    void* y;
    int64_t x_stride, r_stride, i_stride, z_stride, y_stride; /* elements from row to row            */
    const float *lam, *r_bias, *i_bias;
    int32_t batch, dim, n_slots, io_dtype;
    float c;
} ssm_gated_step_t;

/*
 * One step of the recurrence for every batch row, on the states of a pool.  A row whose slot is
 * outside 0 .. n_slots-1 pads the batch: it is skipped and its row of y left as it was.  Rows that
 * name the same slot are its consecutive tokens: they are applied in batch order.  y may not overlap
 * the inputs.
 */
ssm_status_t ssm_gated_state_update(const ssm_gated_step_t* args, ssm_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* SSM_GATED_H */
