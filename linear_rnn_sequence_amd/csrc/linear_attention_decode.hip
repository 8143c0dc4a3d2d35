// Linear attention: one token for each of a batch of resident states.
//
// With a = exp(g), per value row i:  S_i <- a S_i + v_i k,  o_i = scale S_i . q.
// One pass over the state reads it, updates it, reads it out and writes it back: the traffic
// is the state's bytes twice, and everything else is small.  Rows are independent, so a head's
// rows may go to several workgroups.
//
// Lane (c, r) of a row's K / 4 lanes owns key columns 4c .. 4c + 3 of four value rows: every
// state load instruction of a wave reads whole rows (16 bytes per lane), and the readouts are
// DPP reductions.  State accesses are non-temporal, each state is touched once per call.
//
// What bounds it: memory.  256 sequences of 32 heads of 128 x 128 (1.08 GB) take 176 us, 6.1 TB/s,
// where a large copy reaches 6.6; one sequence 3.1 us, in a call that costs the host 11.
#include "gated_delta_device.h"
#include "linear_attention_internal.h"

namespace lattn {
namespace {

using namespace gdr;

constexpr int kRows = 4;  // value rows per lane
constexpr int kThreads = 256;

struct StepArgs {
    const void *q, *k, *v;
    const float *g;
    float *state;
    void *o;
    const int *slots;
    long long q_stride, k_stride, v_stride;
    int heads, parts, rep, V, pool;
    float scale;
};

__device__ __forceinline__ f32x4 load4(const bf16_t *p) {
    const uint2 u = *reinterpret_cast<const uint2 *>(p);
    return f32x4{wkv7::bf16_lo(u.x), wkv7::bf16_hi(u.x), wkv7::bf16_lo(u.y), wkv7::bf16_hi(u.y)};
}
__device__ __forceinline__ f32x4 load4(const float *p) {
    return *reinterpret_cast<const f32x4 *>(p);
}

template <class E, int K>
__global__ __launch_bounds__(kThreads) void step_kernel(StepArgs p) {
    constexpr int kLanes = K / 4;                            // lanes per row
    constexpr int kWaveRows = 64 / kLanes * kRows;           // 16 or 8
    constexpr int kGroupRows = kWaveRows * (kThreads / 64);  // 64 or 32
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int groups = p.V / kGroupRows;
    const int group = (int)(blockIdx.x % groups);
    const int h = (int)(blockIdx.x / groups % p.heads), b = (int)(blockIdx.x / groups / p.heads);
    const int slot = p.slots ? p.slots[b] : b;
    if (slot < 0 || slot >= p.pool) return;
    const int c = lane % kLanes;
    const int r0 = group * kGroupRows + wave * kWaveRows + lane / kLanes * kRows;

    float *st = p.state + ((size_t)slot * p.heads + h) * p.V * K + (size_t)r0 * K + 4 * c;
    f32x4 S[kRows];
#pragma unroll
    for (int m = 0; m < kRows; ++m)
        S[m] = __builtin_nontemporal_load(reinterpret_cast<const f32x4 *>(st + m * K));
    const f32x4 k = load4(static_cast<const E *>(p.k) + b * p.k_stride + h / p.rep * K + 4 * c);
    const f32x4 q = load4(static_cast<const E *>(p.q) + b * p.q_stride + h / p.rep * K + 4 * c);
    const f32x4 v = load4(static_cast<const E *>(p.v) + b * p.v_stride + (size_t)h * p.V + r0);
    const float a = expf(p.g[h / p.parts]);
    float o[kRows];
#pragma unroll
    for (int m = 0; m < kRows; ++m) {
        f32x4 x;
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            x[e] = a * S[m][e] + v[m] * k[e];
            s += x[e] * q[e];
        }
        __builtin_nontemporal_store(x, reinterpret_cast<f32x4 *>(st + m * K));
        s = wkv7::sum_lanes16(s);
        if constexpr (K == 128) s = wkv7::swap16_add(s, s);
        o[m] = p.scale * s;
    }
    // lane c < 4 of a row group writes row r0 + c
    float mine = o[0];
#pragma unroll
    for (int m = 1; m < kRows; ++m) mine = c == m ? o[m] : mine;
    if (c < kRows)
        static_cast<E *>(p.o)[((size_t)b * p.heads + h) * p.V + r0 + c] = from_float<E>(mine);
}

template <class E, int K>
hipError_t launch_step(const StepArgs &a, int n, hipStream_t stream) {
    constexpr int kGroupRows = 64 / (K / 4) * kRows * (kThreads / 64);
    const size_t blocks = (size_t)n * a.heads * (a.V / kGroupRows);
    hipLaunchKernelGGL((step_kernel<E, K>), dim3((unsigned)blocks), dim3(kThreads), 0, stream, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_decode(const DecodeArgs &d, hipStream_t stream) {
    const Problem &p = d.p;
    StepArgs a{};
    a.q = d.q; a.k = d.k; a.v = d.v; a.g = d.g;
    a.state = d.state; a.o = d.o; a.slots = p.slots_in;
    a.q_stride = p.q_stride; a.k_stride = p.k_stride; a.v_stride = p.v_stride;
    a.heads = p.heads; a.parts = p.parts; a.rep = p.rep(); a.V = p.V; a.pool = p.pool;
    a.scale = p.scale;
    if (p.bf16)
        return p.K == 64 ? launch_step<bf16_t, 64>(a, p.n_seq, stream)
                         : launch_step<bf16_t, 128>(a, p.n_seq, stream);
    return p.K == 64 ? launch_step<float, 64>(a, p.n_seq, stream)
                     : launch_step<float, 128>(a, p.n_seq, stream);
}

}  // namespace lattn
