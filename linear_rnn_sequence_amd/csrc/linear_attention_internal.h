// Internal interface between the host entry points of linear attention
// (linear_attention_api.hip) and its kernel launchers.  Not installed.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "linear_attention.h"

namespace lattn {

// A checked problem.  A value head with more than 128 values is several heads with the same
// decay: `heads` of `V` values (64 or 128) each, `parts` of them to one of the caller's.
struct Problem {
    const int *cu;  // nullptr: dense
    int n_seq, T, total;
    int Hk, heads, parts, K, V;
    int q_stride, k_stride, v_stride;  // elements from token to token, at most 2^23
    const int *slots_in, *slots_out;
    int pool;
    float scale;
    bool bf16;
    int rep() const { return heads / Hk; }  // heads that read the same key head
};

// Sequences in segments of `seg` tokens (0: whole), `units` of them at most; few to each sequence.
struct Segments {
    int seg, units;
    bool few;
};
Segments plan_segments(const Problem &p, bool backward);

struct ForwardArgs {
    Problem p;
    Segments seg;
    const void *q, *k, *v;
    const float *g, *s0;
    void *o;
    float *s_out;
    float *states;  // workspace, segments: [units, heads, V, K]
};

struct BackwardArgs {
    Problem p;
    Segments seg;
    const void *q, *k, *v, *d_o;
    const float *g, *s0, *ds_T;
    void *dq, *dk, *dv;
    float *dg, *ds0;
    float *states, *cotangents;  // workspace, segments: [units, heads, V, K] each
    float *dq_heads, *dk_heads;  // workspace, shared key heads: [total, heads, K] each
    double *dg_units;            // workspace, where dg is wanted: [units, heads]
};

struct DecodeArgs {
    Problem p;  // n_seq rows
    const void *q, *k, *v;
    const float *g;
    float *state;
    void *o;
};

// lets a kernel have `bytes` of shared memory
inline hipError_t allow_lds(const void *kernel, int bytes) {
    return bytes <= 64 * 1024 ? hipSuccess
                              : hipFuncSetAttribute(
                                    kernel, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

hipError_t launch_forward(const ForwardArgs &a, hipStream_t stream);
hipError_t launch_backward(const BackwardArgs &a, hipStream_t stream);
hipError_t launch_decode(const DecodeArgs &a, hipStream_t stream);

}  // namespace lattn
