/*
 * m3block.h -- C ABI of libm3scan, operators next to the layer core: the per-channel gated
 * recurrence, the RMS norm of the residual stream with 8-bit rows, and the gradient norm with
 * clipping over all tensors of a training step.
 *
 * The conventions of m3scan.h hold for every entry point here: device pointers owned by the
 * caller, validation on the host, kernels enqueued on `stream` and nothing else (no allocation,
 * no synchronisation; all calls may be captured into a HIP graph), m3_status results with
 * m3_last_error(), a gfx950 GPU as the current device.  Further:
 *  - Alignment.  Every tensor pointer must be aligned to its element size (workspaces: 16 bytes).
 *    Rows that start on 16-byte boundaries (scan: one 4-byte (bf16) or 8-byte (fp32) pair) take
 *    wider loads; nothing else depends on it.
 *  - Pitches.  A pitch is the distance in elements between the first elements of consecutive
 *    rows (tokens); 0 means dense.  Gated scan: rows are at most 2^24 - 1 bytes apart.  Tensors may
 *    be slices of one wider buffer, outputs too, as long as no element is written twice or is both
 *    read and written, except where a call allows it.
 *  - Workspaces are scratch: nothing in them has to survive the call or to be cleared before it.
 *    Two calls that may run at the same time (on two streams, or in two graphs that are replayed at
 *    the same time) need a workspace each; calls that run one after the other may share one.
 */
#ifndef M3BLOCK_H
#define M3BLOCK_H

#include "m3scan.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------------------ gated scan */

typedef struct {
    int64_t batch;       /* b: sequences                                                       */
    int64_t seqlen;      /* L: tokens per sequence; packed: T, the tokens of the whole batch    */
    int64_t width;       /* D: channels                                                        */
    int64_t gate_pitch;  /* pitches of gate, x, y (backward: dy), dgate, dx; 0 = D             */
    int64_t x_pitch;
    int64_t y_pitch;
    int64_t dgate_pitch;
    int64_t dx_pitch;
    int32_t io;          /* m3_dtype of gate, x, y, dy, dgate, dx                               */
    uint32_t flags;      /* 0                                                                   */
} m3_scan_dims;

/*
 * m3_gated_scan -- per-channel gated linear recurrence over whole sequences:
 *
 *   z_t = sigmoid(gate_t + bias),  h_t = (1 - z_t) h_{t-1} + z_t x_t,  y_t = h_t   (h_0 = h_in)
 *
 * the diagonal, convex case of h_t = a_t h_{t-1} + b_t (no page of the reference defines a
 * per-channel gate; z is computed in fp32 from the logit, so neither 1 - z nor z loses digits
 * when the other is near 1, and the state is fp32 throughout).
 *
 * For: the forward pass of training, prefill.  Reads gate and x once and writes y once; the time
 * axis is cut into chunks that run at the same time.
 *
 *   cu_seqlens  [b+1] int32 offsets of a packed batch (sequence s holds tokens cu[s] ..
 *               cu[s+1]-1, cu[0] = 0, nondecreasing, cu[b] <= T), or NULL: dense [b, L, D].  Rows
 *               of y at and past cu[b] are left as they were.  Empty sequences pass h_in through.
 *   gate, x     [b, L, D] or [T, D] io, pitches gate_pitch, x_pitch            required
 *   bias        [D] f32                                                        NULL: 0
 *   h_in        [b, D] f32                                                     NULL: 0
 *   y           like x, pitch y_pitch                                          required
 *   h_out       [b, D] f32, the state after each sequence's last token; may be h_in itself
 *                                                                             required
 *   states      [m3_gated_scan_chunks(dims, packed), D] f32: the state each chunk starts from,
 *               read by m3_gated_scan_backward                                 NULL: not wanted
 *   workspace   m3_gated_scan_workspace_bytes(dims, packed) bytes, 16-byte aligned
 *                                                       required when that is not 0
 * Sizes: fewer than 2^23 blocks of 64 tokens and 128 channels (b ceil(L / 64) ceil(D / 128), packed
 * ceil(T / 64) ceil(D / 128)); more are refused.  The workspace's size is for the current device.
 * Results do not depend on scheduling: equal inputs give equal bits.
 */
int64_t m3_gated_scan_chunks(const m3_scan_dims* dims, int packed);
size_t m3_gated_scan_workspace_bytes(const m3_scan_dims* dims, int packed);
m3_status m3_gated_scan(const m3_scan_dims* dims, const int32_t* cu_seqlens, const void* gate,
                        const void* x, const float* bias, const float* h_in, void* y, float* h_out,
                        float* states, void* workspace, size_t workspace_bytes, hipStream_t stream);

/*
 * m3_gated_scan_step -- one token for b resident states (dims->seqlen must be 1).
 *
 *   gate, x, y  [b, D] io with their pitches;  bias [D] f32 or NULL
 *   h           [b, D] f32 state before the token
 *   h_out       [b, D] f32 state after it; may be h (updated in place)
 * y may be x or gate itself (same pitch).  b * D must be below 2^31.
 */
m3_status m3_gated_scan_step(const m3_scan_dims* dims, const void* gate, const void* x,
                             const float* bias, const float* h, void* y, float* h_out,
                             hipStream_t stream);

/*
 * m3_gated_scan_backward -- gradients of m3_gated_scan.  With the loss's gradients dy of y and
 * dh_out of h_out, backwards over each sequence
 *
 *   l_t = dy_t + (1 - z_{t+1}) l_{t+1}   (after the last token: dh_out)
 *   dx_t = z_t l_t,  dgate_t = z_t (1 - z_t) (x_t - h_{t-1}) l_t
 *   dbias = sum over all tokens of dgate,  dh_in = (1 - z_1) l_1
 *
 * The states h_{t-1} are computed again in fp32 from `states`, not read back from the rounded y.
 *   states      what m3_gated_scan wrote for the same dims, offsets and inputs   required
 *   dy          like y, pitch y_pitch                                            required
 *   dh_out      [b, D] f32                                                       NULL: 0
 *   dgate, dx   like gate, x, pitches dgate_pitch, dx_pitch; rows at and past cu[b] are left as
 *               they were                                                        required
 *   dbias       [D] f32                                                          NULL: not wanted
 *   dh_in       [b, D] f32; an empty sequence passes dh_out through              NULL: not wanted
 *   workspace   m3_gated_scan_backward_workspace_bytes(dims, packed) bytes, 16-byte aligned
 * dbias is summed in a fixed order: equal inputs give equal bits.
 */
size_t m3_gated_scan_backward_workspace_bytes(const m3_scan_dims* dims, int packed);
m3_status m3_gated_scan_backward(const m3_scan_dims* dims, const int32_t* cu_seqlens,
                                 const void* gate, const void* x, const float* bias,
                                 const float* h_in, const float* states, const void* dy,
                                 const float* dh_out, void* dgate, void* dx, float* dbias,
                                 float* dh_in, void* workspace, size_t workspace_bytes,
                                 hipStream_t stream);

/* -------------------------------------------------------------------------------- RMS norm */

typedef struct {
    int64_t rows;
    int64_t width;     /* D <= 16384                                                           */
    int64_t x_pitch;   /* pitches of x, residual, r_out (backward: r, dr_out), y (backward:    */
    int64_t res_pitch; /* dy) and dx; 0 = D.  q is dense.                                       */
    int64_t r_pitch;
    int64_t y_pitch;
    int64_t dx_pitch;
    int64_t group;     /* elements per 8-bit scale: 0 = the whole row, else 32, 64, 128 or 256  */
    int32_t io;        /* m3_dtype of x, residual, r_out, y, r, dy, dr_out, dx                   */
    uint32_t flags;    /* 0                                                                     */
    float eps;         /* added to the mean square                                              */
} m3_norm_dims;

/*
 * m3_rmsnorm -- the residual's addition, the RMS norm and its 8-bit form in one pass:
 *
 *   r = x + residual,  n = r / sqrt(mean(r^2) + eps) * weight      (per row, in fp32)
 *   r_out = round(r), y = round(n)
 *   scale = max |n| / 448 over the row or over each group of `group` consecutive elements (the
 *           last one may be shorter), rounded up below 1e-37, 1 where that maximum is 0;
 *   q = round(n / scale) in e4m3
 *
 * (the RMS norm is the one m3_bcnorm_rope applies to B and C: papernotes.org summary of Mamba-3,
 * key design 4; here over whole rows of the residual stream.)
 *
 *   x, residual  [rows, D] io; residual NULL: r = x
 *   weight       [D] f32                                      NULL: 1
 *   r_out        [rows, D] io; may be x or residual itself (same pitch)   NULL: not wanted
 *   y            [rows, D] io; may be x or residual itself (same pitch)   NULL: not wanted
 *   q, scale     [rows, D] e4m3 (OCP, 8 bits, largest value 448), [rows, ceil(D / group)] f32;
 *                both or neither
 * At least one of y and q is required.  A NaN in a row makes the row's y, q and scales NaN; an infinity
 * makes its own element NaN, and the scale over it, and the row's other elements 0.  The sum of
 * squares is in fp32, as the formula in fp32 has it: rows with magnitudes over about 1e19 overflow it
 * and give y = 0; with eps 0, rows below about 1e-19 lose digits of it, and a row whose squares are
 * all 0 is divided by 0.
 */
m3_status m3_rmsnorm(const m3_norm_dims* dims, const void* x, const void* residual,
                     const float* weight, void* r_out, void* y, void* q, float* scale,
                     hipStream_t stream);

/*
 * m3_rmsnorm_backward -- gradients of n = r / sqrt(mean(r^2) + eps) * weight with respect to r
 * (and with it x and residual, whose gradients are both dx) and weight:
 *
 *   s = 1 / sqrt(mean(r^2) + eps),  u = weight dy
 *   dx = s u - r s^3 mean(u r) + dr_out,  dweight = sum over rows of dy r s
 *
 * in fp32, without the cube: for rows whose squares and products u r sum up within fp32's range.
 *
 *   r          [rows, D] io, m3_rmsnorm's r_out (or x where there was no residual), pitch r_pitch
 *   dy         [rows, D] io, pitch y_pitch
 *   dr_out     [rows, D] io, pitch res_pitch: the gradient of r_out from the residual stream
 *                                                                         NULL: 0
 *   dx         [rows, D] io, pitch dx_pitch; may be dy or dr_out itself (same pitch)
 *   dweight    [D] f32                                                    NULL: not wanted
 *   workspace  m3_rmsnorm_backward_workspace_bytes(dims) bytes, 16-byte aligned; needed for
 *              dweight only
 * dweight is summed in a fixed order: equal inputs give equal bits.
 */
size_t m3_rmsnorm_backward_workspace_bytes(const m3_norm_dims* dims);
m3_status m3_rmsnorm_backward(const m3_norm_dims* dims, const void* r, const float* weight,
                              const void* dy, const void* dr_out, void* dx, float* dweight,
                              void* workspace, size_t workspace_bytes, hipStream_t stream);

/* ------------------------------------------------------------------ gradient norm, clipping */

typedef struct {
    const void* src;  /* gradient, dense                                                        */
    void* dst;        /* m3_grad_clip: where the clipped gradient goes; may be src               */
    int64_t numel;
    int32_t io;       /* m3_dtype of src and dst                                                */
    int32_t pad;
} m3_grad_tensor;

/*
 * m3_grad_norm -- the 2-norm over all elements of `count` tensors, and the factor that brings it
 * to max_norm:
 *
 *   norm = sqrt(sum over all tensors of g^2),  coef = min(1, max_norm / (norm + 1e-6))
 *
 * For: what m3_layer_backward, m3_gated_scan_backward and m3_rmsnorm_backward return.  Squares
 * are summed in fp64 in a fixed order (no overflow, equal inputs give equal bits).
 * A non-finite gradient makes the norm non-finite and follows the formula from there.
 *
 *   tensors    host array (read before the call returns); entries with numel 0 are skipped
 *   stats      [2] f32: norm, coef
 *   workspace  m3_grad_workspace_bytes(tensors, count) bytes, 16-byte aligned; 0 where one
 *              workgroup does it all (and where there is nothing to sum)
 * m3_grad_clip also writes dst = round(coef * src) for every tensor (coef = 1 copies; nothing is
 * written where dst is src and coef is 1).  dst must not overlap another entry's src or dst; a
 * tensor listed twice counts twice in m3_grad_norm and is refused by m3_grad_clip.
 */
size_t m3_grad_workspace_bytes(const m3_grad_tensor* tensors, int64_t count);
m3_status m3_grad_norm(const m3_grad_tensor* tensors, int64_t count, float max_norm, float* stats,
                       void* workspace, size_t workspace_bytes, hipStream_t stream);
m3_status m3_grad_clip(const m3_grad_tensor* tensors, int64_t count, float max_norm, float* stats,
                       void* workspace, size_t workspace_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* M3BLOCK_H */
