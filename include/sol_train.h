/*
 * sol_train.h -- C ABI of libsol's training operators: the gated feed-forward block with
 * its backward pass, and the optimizer step that follows it (global gradient norm, AdamW
 * over many tensors with moments in 32 or 8 bits).
 *
 * The conventions of sol.h hold (layout, pointers, streams, errors, aliasing: only what a
 * function lists; a tensor spans from its first element to its last, and a written tensor's
 * span must not meet another's).  Bounded waits of these kernels that give up are reported by
 * sol_device_errors in bits 16..23.
 */
#ifndef SOL_TRAIN_H
#define SOL_TRAIN_H

#include "sol.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------------------------
 * Gated feed-forward block.
 *
 *     u = [a | b] = x . W_up^T,   act = silu(a) * b,   y = act . W_down^T
 *
 * x, y [n_tokens, d]; W_up [2*inner, d] (gated half in rows [0, inner), as in
 * sol_linear_swiglu); W_down [d, inner]; u [n_tokens, 2*inner].
 * dt must be SOL_DTYPE_BF16.  d and inner are any multiples of 8 (>= 8, below 2^28);
 * n_tokens below 2^30.  Products accumulate in fp32; a and b are not rounded before
 * the activation; act is rounded to bf16 once, as the operand of the second product.
 *
 * Workspace: caller-owned device memory, 256-byte aligned, of at least
 * sol_ffn_workspace_bytes(n_tokens, d, inner) bytes for either call.  It holds nothing
 * between calls; calls that may overlap on the GPU need one each, and a captured graph
 * keeps using the one it was captured with.
 * Results do not depend on timing: work split over the inner dimension is joined in a
 * fixed order, which depends on the sizes and on which gradients are asked for.
 * ------------------------------------------------------------------------------------ */
size_t sol_ffn_workspace_bytes(int64_t n_tokens, int64_t d, int64_t inner);

/* Forward.  u may be NULL (serving: nothing kept for a backward pass). */
typedef struct {
    void* y;
    int64_t ld_y; /* row strides in elements */
    void* u;
    int64_t ld_u;
    const void* x;
    int64_t ld_x;
    const void* w_up;
    int64_t ld_wu;
    const void* w_down;
    int64_t ld_wd;
    void* workspace;
    size_t workspace_bytes;
    int64_t n_tokens, d, inner;
    sol_dtype dt;
} sol_ffn_desc;
sol_status sol_ffn(const sol_ffn_desc* desc, sol_stream_t stream);

/* Backward, from the u that the forward call kept (its bf16 values are the a and b of
 * these formulas):
 *     d_act = dy . W_down,   s = 1 / (1 + exp(-a)),
 *     du = [d_act * b * s * (1 + a * (1 - s)) | d_act * a * s],
 *     dx = du . W_up,   dW_up (+)= du^T . x,   dW_down (+)= dy^T . (silu(a) * b)
 * Each of dx, dw_up, dw_down may be NULL (not computed).  dw_up and dw_down have
 * type grad_dt (SOL_DTYPE_BF16 or SOL_DTYPE_F32); accumulate != 0 adds to what they hold
 * (the sum is formed in fp32 and rounded once).  du and act are rounded to bf16 once, as
 * operands.  n_tokens == 0: the weight gradients are set to zero (accumulate: left as they
 * are), and dy, x, u and dx may be NULL. */
typedef struct {
    void* dx;
    int64_t ld_dx;
    void* dw_up;
    int64_t ld_dwu;
    void* dw_down;
    int64_t ld_dwd;
    const void* dy;
    int64_t ld_dy;
    const void* x;
    int64_t ld_x;
    const void* u;
    int64_t ld_u;
    const void* w_up;
    int64_t ld_wu;
    const void* w_down;
    int64_t ld_wd;
    void* workspace;
    size_t workspace_bytes;
    int64_t n_tokens, d, inner;
    sol_dtype dt, grad_dt;
    int32_t accumulate;
} sol_ffn_backward_desc;
sol_status sol_ffn_backward(const sol_ffn_backward_desc* desc, sol_stream_t stream);

/* ------------------------------------------------------------------------------------
 * AdamW over many tensors at once (decoupled weight decay, Loshchilov and Hutter 2019).
 * For every value of every tensor, with g = grad * factor:
 *     m = beta1 * m + (1 - beta1) * g
 *     v = beta2 * v + (1 - beta2) * g^2
 *     p = p - lr * (weight_decay * p + (m / (1 - beta1^step)) / (sqrt(v / (1 - beta2^step)) + eps))
 * in fp32: v / (1 - beta2^step) above fp32's range (gradients of some 1e19 at the first steps) gives no
 * update, and with eps 0 a value that had no gradient so far moves by 0 / 0.  Parameters are f32; a
 * tensor may have a bf16 copy of them that the step writes too (what the linear layers read).  A
 * parameter kept in bf16 alone is not supported: an update below half a step of its format would be
 * lost.
 *
 * Moments: f32, or 8 bits a value (state_bits 8).  In 8 bits a tensor is cut into blocks
 * of SOL_ADAMW_BLOCK values, each with one f32 scale s, the block's largest magnitude:
 *     m (int8 q in -127..127)  stands for  sign(q) * (q / 127)^2 * s
 *     v (uint8 q in 0..255)    stands for  (q / 255)^4 * s
 * The step computes with the moments in fp32 (the parameters see no rounding of this
 * step's moments) and stores each as one of its two neighbours in the table, the upper one
 * with the probability that makes the expectation the value itself: with beta2 = 0.999 a
 * moment moves by less than half a table step, so rounding to nearest would never let it
 * fall.  A positive v is stored as 1 at least.  The random fractions are a hash of (seed,
 * step, the tensor's place in the plan, the element's index): the same call gives the same
 * result.  A block with a non-finite moment gets a NaN scale: it decodes as NaN.
 * ------------------------------------------------------------------------------------ */
#define SOL_ADAMW_BLOCK 256

typedef struct {
    float* param;       /* [n] */
    void* copy;         /* bf16 [n] or NULL */
    const void* grad;   /* [n] of the plan's grad_dt */
    void* m;            /* [n] f32, or int8 */
    void* v;            /* [n] f32, or uint8 */
    float* m_scale;     /* 8 bits: [ceil(n / 256)]; else NULL */
    float* v_scale;
    int64_t n;          /* >= 0; all other fields may be NULL where it is 0 */
    float weight_decay; /* of this tensor, finite, >= 0 */
} sol_adamw_tensor;

/* The scalars of one step.  lr_device / step_device, where not NULL, are read on the device
 * in place of lr / step when the step runs (for steps captured in a CUDA graph);
 * grad_factor (device, or NULL for 1) multiplies every gradient, such as the second value
 * of sol_adamw_grad_norm. */
typedef struct {
    double lr, beta1, beta2, eps; /* finite; 0 <= beta < 1; eps 0 or >= 2^-126, fp32's least normal number */
    int64_t step;                /* >= 1: the number of this step */
    uint64_t seed;               /* of the 8-bit rounding */
    const float* lr_device;
    const int64_t* step_device;
    const float* grad_factor;
} sol_adamw_scalars;

/* A plan holds the tensors' addresses on the current device (one allocation, made here, not inside a
 * stream capture, and freed by destroy, which may meet a capture that does not use the plan; a captured
 * graph that uses it must not outlive it).  `tensors` is a host array, copied: every buffer, the gradients'
 * too, stays where it is as long as the plan is used, so that gradients are written again at each step, not
 * allocated again (making a plan takes an allocation, two copies and a wait for them, more than a
 * small step).  Every pointer is 16-byte aligned (scales: 4); no written buffer may overlap another
 * buffer of the plan.  grad_dt: SOL_DTYPE_F32 or SOL_DTYPE_BF16, of all gradients. */
typedef struct sol_adamw_plan sol_adamw_plan;
sol_status sol_adamw_plan_create(sol_adamw_plan** plan, const sol_adamw_tensor* tensors, int32_t n_tensors,
                                 sol_dtype grad_dt, int32_t state_bits);
sol_status sol_adamw_plan_destroy(sol_adamw_plan* plan);

/* One step over all tensors of the plan: one kernel, and with step_device and many values a small one
 * ahead of it.  Two steps of one plan must not overlap. */
sol_status sol_adamw_step(const sol_adamw_plan* plan, const sol_adamw_scalars* scalars, sol_stream_t stream);

/* Global norm of the plan's gradients and the factor that clips it:
 *     out[0] = sqrt(sum of g^2 over all tensors),  out[1] = min(1, max_norm / (out[0] + 1e-6))
 * (device f32 [2], 8-byte aligned; a NaN norm gives a NaN factor, and with an infinite max_norm any
 * other norm, an infinite one too, gives 1).  Squares are scaled, so
 * that no gradient of f32's range overflows or vanishes; sums are formed in fp64, in a fixed
 * order.  workspace: SOL_ADAMW_NORM_WORKSPACE bytes, 16-byte aligned, apart from out; calls that may
 * overlap need one each.  max_norm > 0, finite or infinite. */
#define SOL_ADAMW_NORM_WORKSPACE 16384
sol_status sol_adamw_grad_norm(float* out, const sol_adamw_plan* plan, float max_norm, void* workspace,
                               size_t workspace_bytes, sol_stream_t stream);

/* Read 8-bit moments back as values: m_out, v_out [n] of type out_dt (either may be NULL), m, v, m_scale
 * and v_scale as in sol_adamw_tensor (block i of the arrays uses scale i). */
sol_status sol_adamw_state_decode(void* m_out, void* v_out, sol_dtype out_dt, const void* m, const void* v,
                                  const float* m_scale, const float* v_scale, int64_t n, sol_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* SOL_TRAIN_H */
