// Internal interface between the host entry points of the gated delta rule
// (gated_delta_api.hip) and its kernel launchers.  Not installed.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "gated_delta.h"

namespace gdr {

// A checked problem: strides filled in, dense T, number of chunks.
struct Problem {
    const int *cu;  // nullptr: dense
    int n_seq, T, total, slots;
    int Hk, Hv, K, V;
    int q_stride, k_stride, v_stride;  // elements from token to token, at most 2^23
    const int *slots_in, *slots_out;
    int pool;
    float scale;
    bool normalize, bf16;
};

struct ForwardArgs {
    Problem p;
    const void *q, *k, *v, *g, *beta;
    const float *s0;
    void *o;
    float *s_out;
    void *s_ckpt, *u;  // training: nullptr otherwise
    char *records;     // workspace
    char *segments;    // workspace: the segments' states and transitions
};

struct BackwardArgs {
    Problem p;
    const void *q, *k, *v, *g, *beta, *d_o, *s_ckpt, *u;
    const float *ds_T;
    void *dq, *dk, *dv, *dg, *dbeta;
    float *ds0;
    char *records;  // workspace: T^T, P^T and scalars of every chunk and value head
    void *ds;       // workspace: [slots, Hv, GATED_DELTA_CKPT_SIZE], cotangent of each chunk's exit state
    void *dr;       // workspace: [total, Hv, V]
};

struct DecodeArgs {
    Problem p;  // n_seq rows
    const void *q, *k, *v, *g, *beta;
    float *state;
    void *o;
};

// How the forward splits its work: waves of a workgroup, segments of `seg` tokens (0: none), `units`
// of them at most, and the bytes of their states and transitions.
struct Segments {
    int waves, seg, units;
    size_t state_bytes, step_bytes;
};
constexpr int kCus = 256;
Segments plan_segments(const Problem &p);

// lets a kernel have `bytes` of shared memory (it may have 64 KiB with its static arrays,
// none of which come to 16 KiB, anyway)
inline hipError_t allow_lds(const void *kernel, int bytes) {
    return bytes <= 48 * 1024 ? hipSuccess
                              : hipFuncSetAttribute(
                                    kernel, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

size_t forward_record_bytes(bool bf16);
size_t backward_record_bytes(bool bf16);

hipError_t launch_prep(const Problem &p, const void *q, const void *k, const void *g,
                       const void *beta, char *records, bool backward, hipStream_t stream);
hipError_t launch_forward(const ForwardArgs &a, hipStream_t stream);
hipError_t launch_backward_chain(const BackwardArgs &a, hipStream_t stream);
hipError_t launch_gradients(const BackwardArgs &a, hipStream_t stream);
hipError_t launch_backward(const BackwardArgs &a, hipStream_t stream);
hipError_t launch_decode(const DecodeArgs &a, hipStream_t stream);

}  // namespace gdr
