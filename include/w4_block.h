/*
 * w4_block.h -- C ABI of what stands around a block's 4-bit products (MI355X,
 * gfx950): the norms before and after a block with its gate and residual sum,
 * the tokens sorted by expert for w4_moe_gemm (w4.h) and brought back with
 * weights, and the gradients of these.  Part of the same library as w4.h, with
 * its conventions: the caller owns every buffer, arguments are validated on the
 * host before any HIP call, calls are asynchronous on ``stream``, never
 * allocate, never synchronise and can be captured into a HIP graph; an empty
 * problem is W4_OK, and an array without elements may be NULL; the same call on
 * the same inputs returns the same bits (no floating-point atomics).  Outputs
 * must not overlap an input or each other unless said otherwise.  Rows lie
 * *_stride elements apart (a multiple of 8, at least their length, at most
 * 2^40) and start 16-byte aligned.
 */
#ifndef W4_BLOCK_H
#define W4_BLOCK_H

#include "w4.h"

#ifdef __cplusplus
extern "C" {
#endif

#define W4_NORM_MAX_DIM 16384
#define W4_MOE_MAX_TOP 64
#define W4_MOE_SORT_MAX_EXPERTS 1024

/*
 * w4_block_norm -- a block's output normed, gated and added to the residual
 * stream, and the stream normed for the next block, in one pass.
 *   u  = y / sqrt(mean(y^2) + eps) * (y_weight + weight_add)   (no y_weight: u = y)
 *   h' = residual_scale * h + branch_scale * gate * u          (no gate: 1; no y: h' = h)
 *   z  = h' / sqrt(mean(h'^2) + eps) * (z_weight + weight_add) (no z_weight: z = h')
 * A lane's share of a sum of squares is FP32, or FP64 where FP32 would not hold
 * it; the sum over lanes is FP64, all else FP32.  z is computed from h' before h'
 * is rounded to its type.  Each result is rounded once.
 *   h, h_out     device bf16, or float if h_f32 [T][D].  h_out may be exactly h
 *                (same pointer and stride), or NULL: not stored (then z is given)
 *   y            device bf16 [T][D], or NULL (then h_out must be NULL too)
 *   z            device bf16 [T][D]; may be exactly y; or NULL
 *   y_weight, z_weight  device bf16 [D] or NULL
 *   gate         device bf16 [D] if gate_stride = 0, else [T][D]; or NULL
 *   D            a multiple of 8 in [8, W4_NORM_MAX_DIM]
 *   T            at most 2^21
 * Errors: W4_ERR_NULL, W4_ERR_SHAPE, W4_ERR_ALIGN, W4_ERR_ALIAS, W4_ERR_ARG
 * (strides, scales, eps), W4_ERR_HIP.
 */
typedef struct w4_norm_args {
    const void* h;
    const void* y;
    void* h_out;
    void* z;
    const void* y_weight;
    const void* z_weight;
    const void* gate;
    int64_t h_stride, y_stride, h_out_stride, z_stride, gate_stride; /* elements */
    int T, D, h_f32;
    float residual_scale, branch_scale, eps, weight_add;
} w4_norm_args;
W4_API w4_status w4_block_norm(const w4_norm_args* args, void* stream);

/*
 * w4_block_norm_grad -- the gradients of w4_block_norm's inputs, from those of
 * its outputs.  With n1 = y / rms(y), n2 = h' / rms(h') (rms(x) = sqrt(mean(x^2) + eps)),
 * w1 and w2 the weights with weight_add:
 *   g2  = dz * w2,  dH = dh_out + (g2 - n2 * mean(g2 * n2)) / rms(h')
 *   dh  = residual_scale * dH,  du = branch_scale * gate * dH,  g1 = du * w1
 *   dy  = (g1 - n1 * mean(g1 * n1)) / rms(y)                (no y_weight: dy = du)
 *   d_z_weight = sum_t dz * n2,  d_y_weight = sum_t du * n1
 *   d_gate     = branch_scale * dH * u, summed over t if the gate is shared
 * h' is computed again from h and y, which must hold what they held before the
 * call of w4_block_norm.
 * Means over a row as in w4_block_norm.  A sum over t is FP32 over a run of rows,
 * one after the other, FP64 over the runs: at most ceil(T / 256) rows, so up to
 * 8192 where T is 2^21 (a half, a quarter and an eighth of that for D up to 2048, 1024
 * and 512, whose runs are shared by teams).
 *   args          as for w4_block_norm; h_out and z are not used
 *   dh_out        device, h's type [T][D], or NULL for 0
 *   dz            device bf16 [T][D], or NULL for 0; one of the two is given
 *   dh            device, h's type [T][D], or NULL; may be exactly dh_out
 *   dy            device bf16 [T][D], or NULL; may be exactly dz
 *   d_y_weight, d_z_weight  device float [D], or NULL (without the weight they must be NULL)
 *   d_gate        device float [D] for a shared gate, else bf16 [T][D] with
 *                 stride d_gate_stride; or NULL
 *   dh_out, dz, dh and dy have the strides of their own that follow them
 *   workspace     at least w4_block_norm_grad_workspace_bytes(T, D) bytes,
 *                 16-byte aligned, if d_y_weight, d_z_weight or a shared gate's
 *                 d_gate is given (else it may be NULL): sums over runs of rows.
 *                 Its contents on entry are ignored; calls that share one must
 *                 be ordered
 * T = 0 sets the sums over t to 0.
 * Errors: as w4_block_norm, and W4_ERR_WORKSPACE.
 */
typedef struct w4_norm_grad_args {
    const void* dh_out;
    const void* dz;
    void* dh;
    void* dy;
    int64_t dh_out_stride, dz_stride, dh_stride, dy_stride, d_gate_stride; /* elements */
    float* d_y_weight;
    float* d_z_weight;
    void* d_gate;
} w4_norm_grad_args;
W4_API size_t w4_block_norm_grad_workspace_bytes(int T, int D);
W4_API w4_status w4_block_norm_grad(const w4_norm_args* args, const w4_norm_grad_args* grad, void* workspace,
                                    size_t workspace_bytes, void* stream);

/*
 * w4_moe_sort -- tokens sorted by expert: where every choice goes, and the
 * rows of activations in that order, as w4_moe_gemm takes them.
 * Choice i = t * top + j of token t is experts[t][j].  An expert's choices
 * keep their order; with capacity > 0 only its first ``capacity`` get a row.
 *   row_start[e] = rows of the experts before e,
 *   row_of[i]    = row_start[e] + (choices of e before i)
 *   experts     device int32 [T][top]; an id outside [0, num_experts) gets no row
 *   row_start   device int32 [num_experts + 1], out: w4_moe_gemm's row ranges
 *               with expert_ids = 0 .. num_experts - 1
 *   row_of      device int32 [T][top], out; -1: no row
 *   source      device int32 [T * top], out: the choice i of each row, -1 behind
 *               the last; or NULL
 *   x           device bf16 [T][D], and rows, device bf16 [R][D], out:
 *               rows[row_of[i]] = x[i / top]; rows behind the last are left as
 *               they were, and none at R or beyond is written.  Both NULL: only
 *               the tables
 *   workspace   at least w4_moe_sort_workspace_bytes() bytes, 16-byte aligned
 *               (NULL when that is 0); contents ignored on entry; calls that
 *               share one must be ordered
 *   1 <= top <= W4_MOE_MAX_TOP, 1 <= num_experts <= W4_MOE_SORT_MAX_EXPERTS,
 *   T * top <= 2^23, D a multiple of 8 in [8, 2^20], capacity >= 0.
 * T = 0 writes row_start.
 * Errors: W4_ERR_NULL, W4_ERR_SHAPE, W4_ERR_ALIGN, W4_ERR_WORKSPACE,
 * W4_ERR_ALIAS, W4_ERR_ARG (strides, capacity), W4_ERR_HIP.
 */
typedef struct w4_moe_sort_args {
    const int32_t* experts;
    int32_t* row_start;
    int32_t* row_of;
    int32_t* source;
    const void* x;
    void* rows;
    int64_t x_stride, rows_stride; /* elements */
    int T, top, num_experts, capacity;
    int R, D;
} w4_moe_sort_args;
W4_API size_t w4_moe_sort_workspace_bytes(int T, int top, int num_experts);
W4_API w4_status w4_moe_sort(const w4_moe_sort_args* args, void* workspace, size_t workspace_bytes, void* stream);

/*
 * w4_moe_combine -- the experts' rows back to their tokens, weights applied.
 *   out[t] = add[t] + sum_j weights[t][j] * y[row_of[t][j]]
 * in FP32, j rising, rounded once.  A choice whose row lies outside [0, R)
 * counts for nothing.  Without weights it is the gradient of w4_moe_sort's
 * rows: x's from theirs.
 *   y        device bf16 [R][N]
 *   row_of   device int32 [T][top], or NULL: choice j of token t is row t * top + j
 *            (w4_moe_gemv's outputs)
 *   weights  device float [T][top], or NULL for 1
 *   add      device bf16 [T][N], or NULL for 0 (a shared expert, a residual)
 *   out      device bf16 [T][N]; may be exactly add (same pointer and stride)
 *   N        a multiple of 8 in [8, 2^20];  T * top <= 2^23;  1 <= top <= W4_MOE_MAX_TOP
 * Errors: W4_ERR_NULL, W4_ERR_SHAPE, W4_ERR_ALIGN, W4_ERR_ALIAS, W4_ERR_ARG, W4_ERR_HIP.
 */
typedef struct w4_moe_combine_args {
    const void* y;
    const int32_t* row_of;
    const float* weights;
    const void* add;
    void* out;
    int64_t y_stride, add_stride, out_stride; /* elements */
    int T, top, R, N;
} w4_moe_combine_args;
W4_API w4_status w4_moe_combine(const w4_moe_combine_args* args, void* stream);

/*
 * w4_moe_combine_grad -- the gradients of w4_moe_combine's rows and weights
 * (add's is dout itself).
 *   dy[row_of[t][j]] = weights[t][j] * dout[t],  dweights[t][j] = dout[t] . y[row_of[t][j]]
 * A choice without a row has dweights 0; rows of dy that no choice has are left
 * as they were.  Rows within [0, R) must differ.
 *   dout      device bf16 [T][N]
 *   y         device bf16 [R][N]; NULL if dweights is
 *   row_of, weights  as for w4_moe_combine
 *   dy        device bf16 [R][N], or NULL; may be exactly y
 *   dweights  device float [T][top], or NULL; FP32 sums in a fixed order
 * One of dy and dweights is given.  Sizes as for w4_moe_combine.
 * Errors: as w4_moe_combine.
 */
typedef struct w4_moe_combine_grad_args {
    const void* dout;
    const void* y;
    const int32_t* row_of;
    const float* weights;
    void* dy;
    float* dweights;
    int64_t dout_stride, y_stride, dy_stride; /* elements */
    int T, top, R, N;
} w4_moe_combine_grad_args;
W4_API w4_status w4_moe_combine_grad(const w4_moe_combine_grad_args* args, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* W4_BLOCK_H */
