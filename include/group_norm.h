/*
 * group_norm.h -- the group norm with an activation or gate behind a recurrence, on MI355X
 * (gfx950); part of librwkv7_wkv.so.
 *
 * Each row x [C] (a token, channels last) by itself, in `groups` groups of `size` neighbouring
 * channels (a head's), C = groups * size:
 *
 *     u = (x - mean) / sqrt(var + eps)      mean and var over the group's channels
 *     u = x / sqrt(mean(x^2) + eps)         with `rms`
 *     n = u weight + bias                   per channel
 *     y = n act(gate)  with a gate,  act(n)  without one
 *
 * act is one of none (act(x) = x), silu (x sigmoid(x)) and sigmoid.  It is the norm that
 * rwkv7_wkv_forward has as its epilogue, for any recurrence's readouts, with its gradients.
 *
 * Conventions: those of rwkv7_wkv.h (device pointers, all checks on the host before anything
 * is enqueued, no allocation, no state kept between calls, work enqueued on `stream`, status
 * codes), and
 *  - x, gate, y and their gradients have the element type dt: RWKV7_DT_F32 or RWKV7_DT_BF16
 *    (RWKV7_DT_BF16_W32 returns RWKV7_ERR_UNSUPPORTED); weight, bias and their gradients are
 *    float32 [C].
 *  - size is 1 to 1024.  Tensors need their type's alignment; those that start on 16 bytes,
 *    with groups and strides that are multiples of 16 bytes, are read fastest.
 *  - x and gate may be strided from row to row (slices of a joint projection); the channels of
 *    a row are dense, and so are all other tensors.
 *  - Numerics: float32 throughout, the variance from the differences to the mean; outputs are
 *    rounded once to dt.  The same call gives the same bits.  Sums of squares must be finite
 *    in float32.  With bf16 rows the sigmoid of act is off by up to 2^-22 of itself, and for
 *    a negative argument z by 1.25 |z| 2^-24 more, in the float32 gradients of weight and bias
 *    as well.  Its derivative is off by 2^-22 of 1 (float32 rows too): a sigmoid gate beyond 17
 *    gets the gradient 0.
 *  - Non-finite inputs stay in their row and group (and in the gradients of their channels'
 *    weight and bias).
 */
#ifndef GROUP_NORM_H
#define GROUP_NORM_H

#include "rwkv7_wkv.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    GROUP_NORM_NONE = 0,
    GROUP_NORM_SILU = 1,
    GROUP_NORM_SIGMOID = 2
} group_norm_activation;

typedef struct {
    long long rows;         /* >= 0, at most 2^31 - 1                                    */
    int groups, size;       /* groups * size at most 2^23                                */
    long long x_stride;     /* elements from row to row; 0: C.  At least C, at most 2^23 */
    long long gate_stride;  /* likewise                                                  */
    float eps;
    group_norm_activation activation;
    int rms;
    rwkv7_dtype dt;
} group_norm_problem;

/*
 *   x            : [rows, C] (strided);  gate : likewise, or NULL
 *   weight, bias : [C] float32, or NULL (1 and 0)
 *   y            : [rows, C]; may be x where that is dense
 */
rwkv7_status group_norm_forward(const group_norm_problem *p, const void *x, const void *gate,
                                const float *weight, const float *bias, void *y, void *stream);

/*
 * Gradients of sum <y, dy>, from the forward's inputs alone (it stores nothing).
 *   dy            : [rows, C]
 *   dx            : [rows, C]; may be dy
 *   dgate         : [rows, C]; given exactly where gate is
 *   dweight, dbias : [C] float32 (summed over the rows), or NULL
 *   workspace     : at least group_norm_backward_workspace(p) bytes, aligned to 16; may be NULL
 *                   where neither dweight nor dbias is wanted
 */
rwkv7_status group_norm_backward(const group_norm_problem *p, const void *x, const void *gate,
                                 const float *weight, const float *bias, const void *dy, void *dx,
                                 void *dgate, float *dweight, float *dbias, void *workspace,
                                 size_t workspace_bytes, void *stream);

/* Bytes of device workspace (0 for an invalid problem). */
size_t group_norm_backward_workspace(const group_norm_problem *p);

#ifdef __cplusplus
}
#endif

#endif /* GROUP_NORM_H */
