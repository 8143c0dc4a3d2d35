/*
 * linear_attention.h -- linear attention with a decay for each head on MI355X (gfx950); part
 * of librwkv7_wkv.so.
 *
 * Per sequence and value head h, with a float32 state S [V, K] (row i = value index, column
 * j = key index, as in rwkv7_wkv.h) and the head's log decay g_h, each token t computes
 *
 *     S   = exp(g_h) S + v_t k_t^T
 *     o_t = scale S q_t
 *
 * It is the gated delta rule without the correction by what the key recalls, and with one
 * decay for all tokens of a head.
 *
 * Conventions: those of rwkv7_wkv.h (device pointers, 16-byte alignment, all checks on the
 * host before anything is enqueued, no allocation, no state kept between calls, work enqueued
 * on `stream`, status codes), and of gated_delta.h where both have them:
 *  - q, k, v, o and their gradients have the element type dt: RWKV7_DT_F32 or RWKV7_DT_BF16
 *    (RWKV7_DT_BF16_W32 returns RWKV7_ERR_UNSUPPORTED).  g and its gradient are float32 [Hv]
 *    with their type's alignment.  g is at most 0; -infinity forgets the state at every token.
 *    (A g above 0 grows the state and is computed as it stands while exp(64 g), or exp of the
 *    longest segment's tokens times g, is finite.)
 *  - K is 64 or 128; V a multiple of 64 up to 256; Hv a multiple of Hk: value head h reads
 *    key head h / (Hv / Hk).
 *  - A batch is dense (n_seq sequences of total / n_seq tokens each, rows [n_seq * T]) or
 *    packed (cu_seqlens: n_seq + 1 non-decreasing int32 token offsets on the device; sequence
 *    i has the rows cu_seqlens[i] .. cu_seqlens[i + 1] - 1 of `total`).  Lengths may be 0 and
 *    1.  Rows outside every sequence are neither read nor written.  The kernels clamp the
 *    offsets to [0, total] and to non-negative lengths: wrong ones give wrong results but no
 *    access outside a buffer.
 *  - q, k and v may be strided from token to token (a slice of a joint projection); the
 *    channels of one token are dense [heads, K or V].
 *  - A packed batch is planned by its tokens, its sequences and its heads; the lengths are on the
 *    device.  One sequence that is far longer than the others, such as a prompt among single
 *    tokens, is then a chain of all its chunks: it is several times faster in a call of its own.
 *  - The states of n_seq sequences take less than 2^38 bytes (also where none are given); Hv * V,
 *    and Hv * K times the parts of at most 128 values that V is computed in (192: three of 64), are
 *    at most 2^23.  Larger calls return RWKV7_ERR_SHAPE.
 *  - States s0, s_out are float32 [pool, Hv, V, K].  Without slots, sequence i has state i
 *    (pool = n_seq).  With slots (int32 [n_seq] on the device) sequence i starts from state
 *    slots_in[i] and leaves its final state in slots_out[i].  A slot outside [0, pool) stands
 *    for none: the sequence starts from zeros, or its final state is dropped.  The entries of
 *    slots_out inside the pool must differ from each other, and with s_out == s0 from other
 *    sequences' slots_in; otherwise it is not defined which state remains, or in decode which
 *    mixture of them.
 *  - Numerics: float32 sums and states; what is added to a state keeps 24 bits of significand
 *    from bf16 inputs too.  o and the gradients of bf16 inputs take a state and the decayed
 *    products of the rows of a 64-token chunk with 16 bits (dg with 24), and are rounded once.
 *    The same call gives the same bits.
 *    Long sequences may be computed in segments, whose length depends on the sequences and
 *    heads of the call, so a sequence's last bits may depend on what else the call holds, and on
 *    whether its states are updated in place.
 *  - A workspace serves one call at a time: calls, or captured graphs, that may run at once
 *    need one each.  What it held before does not matter.
 *  - Non-finite inputs propagate within a (sequence, value head) pair, from q and k to all
 *    value heads of their key head, and in the gradients of v's and d_o's to the key head.
 *    In o and dq, tokens of the same 64-token chunk before the non-finite one may become
 *    non-finite too, earlier chunks do not (decode works on single tokens).  dk and dv are
 *    computed from the last token on: likewise, with the order of the tokens turned round and
 *    the chunks counted from the end (of a segment, where the call has some).
 */
#ifndef LINEAR_ATTENTION_H
#define LINEAR_ATTENTION_H

#include "rwkv7_wkv.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct {
    int n_seq;              /* sequences, >= 1                                          */
    int total;              /* rows (tokens) of q, k, v, o; dense: n_seq * T             */
    const int *cu_seqlens;  /* [n_seq + 1] on the device, or NULL: dense                 */
    int Hk, Hv, K, V;
    long long q_stride;     /* elements from one token's q to the next's; 0: Hk * K.     */
    long long k_stride;     /*   A multiple of 16 bytes, at least Hk * K, at most 2^23   */
    long long v_stride;     /* likewise; 0: Hv * V                                       */
    const int *slots_in;    /* [n_seq] on the device, or NULL: state i                   */
    const int *slots_out;   /* likewise                                                  */
    int pool;               /* states in s0 and s_out; n_seq where there are no slots    */
    float scale;            /* factor of the readout, usually K^-0.5                     */
    rwkv7_dtype dt;
} linear_attention_problem;

/*
 * Prefill, and the forward of a training step: all tokens of every sequence.
 *   q, k  : [total, Hk, K] (strided), v : [total, Hv, V] (strided), g : [Hv] float32
 *   s0    : [pool, Hv, V, K] float32, or NULL (zeros)
 *   o     : [total, Hv, V]
 *   s_out : [pool, Hv, V, K] float32, or NULL; may equal s0
 *   workspace : at least linear_attention_forward_workspace(p) bytes
 * q, k, v and o may be NULL when total == 0.
 */
rwkv7_status linear_attention_forward(const linear_attention_problem *p, const void *q,
                                      const void *k, const void *v, const float *g,
                                      const float *s0, void *o, float *s_out, void *workspace,
                                      size_t workspace_bytes, void *stream);

/* Bytes of device workspace (0 for an invalid problem). */
size_t linear_attention_forward_workspace(const linear_attention_problem *p);

/*
 * One token for each of n_seq resident states (total == n_seq, cu_seqlens NULL, slots_in ==
 * slots_out): q, k [n_seq, Hk, K], v, o [n_seq, Hv, V]; state [pool, Hv, V, K] updated in
 * place.  Rows whose slot lies outside the pool are left as they are (o too).
 */
rwkv7_status linear_attention_decode(const linear_attention_problem *p, const void *q,
                                     const void *k, const void *v, const float *g, float *state,
                                     void *o, void *stream);

/*
 * Gradients of sum_t <o_t, d_o_t> + <S_T, ds_T> with respect to q, k, v, g and s0, from the
 * forward's inputs alone (it stores nothing for the backward).  No slots.
 *   d_o    : [total, Hv, V];  s0, ds_T : [n_seq, Hv, V, K] float32 or NULL (zeros)
 *   dq, dk : [total, Hk, K] (summed over the value heads of a key head), dv : [total, Hv, V],
 *            all dense
 *   dg     : [Hv] float32 (summed over the batch), or NULL: a decay that is not learned
 *   ds0    : [n_seq, Hv, V, K] float32 or NULL; may equal ds_T
 *   workspace : at least linear_attention_backward_workspace(p) bytes
 */
rwkv7_status linear_attention_backward(const linear_attention_problem *p, const void *q,
                                       const void *k, const void *v, const float *g,
                                       const void *d_o, const float *s0, const float *ds_T,
                                       void *dq, void *dk, void *dv, float *dg, float *ds0,
                                       void *workspace, size_t workspace_bytes, void *stream);

size_t linear_attention_backward_workspace(const linear_attention_problem *p);

#ifdef __cplusplus
}
#endif

#endif /* LINEAR_ATTENTION_H */
