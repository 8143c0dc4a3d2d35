/*
 * gated_delta.h -- the gated delta rule on MI355X (gfx950), and the moves of
 * recurrent states between the slots of a pool; part of librwkv7_wkv.so.
 *
 * Per sequence and value head h, with a float32 state S [V, K] (row i = value
 * index, column j = key index, as in rwkv7_wkv.h), each token t computes
 *
 *     Sd  = exp(g_t) S                                 (one decay for the whole state)
 *     e   = v_t - Sd k_t                               (what the key does not recall yet)
 *     S   = Sd + beta_t e k_t^T
 *     o_t = scale S q_t
 *
 * It is the WKV7 update with a scalar decay, kappa = k and a = beta, but with
 * one scalar each in place of the vectors w and a, key heads that several value
 * heads share (value head h reads key head h / (Hv / Hk)) and states that need
 * not be square.  With `normalize`, q and k are divided by sqrt(sum of squares
 * + 1e-6) over their K channels first.
 *
 * Conventions: those of rwkv7_wkv.h (device pointers, 16-byte alignment, all
 * checks on the host before anything is enqueued, no allocation, no state kept
 * between calls, work enqueued on `stream`, status codes), and
 *  - q, k, v, g, beta, o and all gradients have the element type dt: RWKV7_DT_F32
 *    or RWKV7_DT_BF16 (RWKV7_DT_BF16_W32 returns RWKV7_ERR_UNSUPPORTED).  The
 *    decay is given as its logarithm: bf16 keeps slow forgetting there (2^-9 of
 *    the logarithm) where it would round a decay near 1 to 1.
 *  - g, beta and their gradients need only their type's alignment, not 16 bytes.
 *  - K is 64 or 128; V a multiple of 64 up to 256; Hv a multiple of Hk.
 *  - A batch is dense (n_seq sequences of total / n_seq tokens each, rows
 *    [n_seq * T]) or packed (cu_seqlens: n_seq + 1 non-decreasing int32 token
 *    offsets on the device; sequence i has the rows cu_seqlens[i] ..
 *    cu_seqlens[i + 1] - 1 of `total`).  Lengths may be 0 and 1.  Rows outside
 *    every sequence are neither read nor written.  The offsets cannot be checked
 *    on the host: the kernels clamp them to [0, total] and to non-negative
 *    lengths, so that wrong ones give wrong results but no access outside a
 *    buffer.
 *  - q, k, v may be strided from token to token (a slice of a joint projection);
 *    the channels of one token are dense [heads, K or V].
 *  - States s0, s_out are float32 [pool, Hv, V, K].  Without slots, sequence i
 *    has state i (pool = n_seq).  With slots (int32 [n_seq] on the device)
 *    sequence i starts from state slots_in[i] and leaves its final state in
 *    slots_out[i].  A slot outside [0, pool) stands for none: the sequence
 *    starts from zeros, or its final state is dropped.  The entries of slots_out
 *    inside the pool must differ from each other, and with s_out == s0 from other
 *    sequences' slots_in; otherwise it is not defined which state remains, or in decode
 *    which mixture of them.
 *  - Numerics: float32 sums, states and norms; exp(g) with g below -200 is 0.
 *    Outputs are rounded once to dt.  The states are float32 results also from
 *    bf16 inputs: what is added to them has 16 bits of significand or more, which leaves
 *    s_out and ds0 2 to 4e-6 of their norm from exact ones (float inputs: 4e-7).  In the
 *    same way bf16 o is 2.2e-3 off, of which its own rounding is 1.7e-3.  The gradients
 *    are formed from states, u and the like that are kept in dt (states with four more
 *    bits for dg): in bf16 2.4 to 3.0e-3, dv 1.7e-3; more where the terms of a sum
 *    cancel.  For more exact results give float32 inputs: bf16 values lose nothing.
 *    The same call gives the same bits.  Few long sequences are computed in
 *    segments, whose length depends on the sequences and heads of the call, so a
 *    long sequence's last bits may depend on what else the call holds.
 *  - A workspace serves one call at a time: calls, or captured graphs, that may run
 *    at once need one each.  What it held before does not matter.
 *  - Non-finite inputs propagate within a (sequence, value head) pair, and from
 *    q and k to all value heads of their key head; tokens of the same 64-token
 *    chunk before the non-finite one may become non-finite too, earlier chunks
 *    do not (decode works on single tokens).  g = -infinity is finite in this
 *    sense: the state is forgotten.
 */
#ifndef GATED_DELTA_H
#define GATED_DELTA_H

#include "rwkv7_wkv.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Tokens of a chunk: stored states are those at multiples of it. */
#define GATED_DELTA_CHUNK 64

/* Elements from one stored state (s_ckpt) to the next: V * K of the state and, in bf16,
 * V * K / 4 for four more bits of each. */
#define GATED_DELTA_CKPT_SIZE(V, K, dt) \
    ((dt) == RWKV7_DT_BF16 ? (V) * (K) + (V) * (K) / 4 : (V) * (K))

typedef struct {
    int n_seq;              /* sequences, >= 1                                          */
    int total;              /* rows (tokens) of q, k, v, g, beta, o; dense: n_seq * T    */
    const int *cu_seqlens;  /* [n_seq + 1] on the device, or NULL: dense                 */
    int Hk, Hv, K, V;
    long long q_stride;     /* elements from one token's q to the next's; 0: Hk * K.     */
    long long k_stride;     /*   A multiple of 16 bytes, at least Hk * K, at most 2^23   */
    long long v_stride;     /* likewise; 0: Hv * V                                       */
    const int *slots_in;    /* [n_seq] on the device, or NULL: state i                   */
    const int *slots_out;   /* likewise                                                  */
    int pool;               /* states in s0 and s_out; n_seq where there are no slots    */
    float scale;            /* factor of the readout, usually K^-0.5                     */
    int normalize;          /* divide q and k by their norms                             */
    rwkv7_dtype dt;
} gated_delta_problem;

/*
 * Prefill: all tokens of every sequence.
 *   q, k    : [total, Hk, K] (strided), v : [total, Hv, V] (strided)
 *   g, beta : [total, Hv]
 *   s0      : [pool, Hv, V, K] float32, or NULL (zeros)
 *   o       : [total, Hv, V]
 *   s_out   : [pool, Hv, V, K] float32, or NULL; may equal s0
 *   workspace : at least gated_delta_forward_workspace(p) bytes
 * q, k, v, g, beta and o may be NULL when total == 0.
 */
rwkv7_status gated_delta_forward(const gated_delta_problem *p, const void *q, const void *k,
                                 const void *v, const void *g, const void *beta,
                                 const float *s0, void *o, float *s_out, void *workspace,
                                 size_t workspace_bytes, void *stream);

/* Bytes of device workspace (0 for an invalid problem). */
size_t gated_delta_forward_workspace(const gated_delta_problem *p);

/*
 * One token for each of n_seq resident states (total == n_seq, cu_seqlens
 * NULL, slots_in == slots_out): q, k [n_seq, Hk, K], v [n_seq, Hv, V], g, beta
 * [n_seq, Hv], o [n_seq, Hv, V]; state [pool, Hv, V, K] updated in place.  Rows
 * whose slot lies outside the pool are left as they are (o too).
 */
rwkv7_status gated_delta_decode(const gated_delta_problem *p, const void *q, const void *k,
                                const void *v, const void *g, const void *beta, float *state,
                                void *o, void *stream);

/*
 * Training forward: gated_delta_forward that also stores, for the backward,
 *   s_ckpt : [chunks, Hv, GATED_DELTA_CKPT_SIZE] in dt, the state at the start of
 *            every chunk: [V, K] and, in bf16, four more bits of each element behind
 *            it (for the gradient of g),
 *            chunks = gated_delta_chunks(p); sequence i's chunks begin at
 *            i * ceil(T / 64) (dense) or cu_seqlens[i] / 64 + i (packed)
 *   u      : [total, Hv, V] in dt, beta_t e_t of every token
 * (rounded to dt: the backward's products take them in that type).  No slots.
 */
rwkv7_status gated_delta_forward_train(const gated_delta_problem *p, const void *q,
                                       const void *k, const void *v, const void *g,
                                       const void *beta, const float *s0, void *o, float *s_out,
                                       void *s_ckpt, void *u, void *workspace,
                                       size_t workspace_bytes, void *stream);

/* Chunks of the problem (0 for an invalid one). */
int gated_delta_chunks(const gated_delta_problem *p);

/*
 * Gradients of sum_t <o_t, d_o_t> + <S_T, ds_T> with respect to q, k, v, g,
 * beta and s0; the inputs, s_ckpt and u are those of gated_delta_forward_train.
 *   d_o   : [total, Hv, V];  ds_T : [n_seq, Hv, V, K] float32 or NULL (zeros)
 *   dq, dk : [total, Hk, K] (summed over the value heads of a key head),
 *   dv     : [total, Hv, V], dg, dbeta : [total, Hv], all dense
 *   ds0    : [n_seq, Hv, V, K] float32 or NULL; may equal ds_T
 *   workspace : at least gated_delta_backward_workspace(p) bytes
 */
rwkv7_status gated_delta_backward(const gated_delta_problem *p, const void *q, const void *k,
                                  const void *v, const void *g, const void *beta,
                                  const void *d_o, const void *s_ckpt, const void *u,
                                  const float *ds_T, void *dq, void *dk, void *dv, void *dg,
                                  void *dbeta, float *ds0, void *workspace,
                                  size_t workspace_bytes, void *stream);

size_t gated_delta_backward_workspace(const gated_delta_problem *p);

/* Moves of one state_move call. */
#define STATE_MOVE_MAX 1024

/*
 * Moves states between the slots of a pool, in every layer at once, as if all
 * sources were read before any target is written: for i = 0 .. n - 1
 *     pool[layer][dst[i]] = old pool[layer][src[i]],  or zeros where src[i] == -1.
 * So one call copies, forks (one source, several targets), reorders (a
 * permutation, as beam search's), compacts and frees, for the states of both
 * recurrences or any other data in slots.
 *   pool : `layers` arrays of `slots` slots of slot_bytes bytes each, layer_bytes
 *          apart (slot_bytes and layer_bytes multiples of 16; layer_bytes >=
 *          slots * slot_bytes, ignored for one layer)
 *   src, dst : int32 [n] on the device, 0 <= n <= STATE_MOVE_MAX.  Pairs with dst
 *          outside [0, slots), or src outside [-1, slots), are left out.  Of
 *          pairs with the same dst the last one counts.
 */
rwkv7_status state_move(void *pool, int layers, size_t layer_bytes, int slots,
                        size_t slot_bytes, const int *src, const int *dst, int n, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* GATED_DELTA_H */
