// Gated delta rule: one token for each of a batch of resident states.
//
// With the old state S and a = exp(g), per value row i (r = S_i . k, m = S_i . q):
//   e = v_i - a r,  S_i <- a S_i + beta e k,  o_i = scale (a m + beta e (k . q)).
// So one pass over the state reads it, forms both row products, and writes it
// back: the traffic is the state's bytes twice, and everything else is small.
// Rows are independent, so a head's rows may go to several workgroups.
//
// Lane (c, r) of a row's K / 4 lanes owns key columns 4c .. 4c + 3 of four value
// rows: every state load instruction of a wave reads whole rows (16 bytes per
// lane), and row sums are DPP reductions.  State accesses are non-temporal,
// each state is touched once per call.  256 sequences of 32 heads of 128 x 128 move
// 1.08 GB in 177 us, 6.1 TB/s, where a large copy reaches 6.6 TB/s; one sequence takes
// 4 us, and the call 11 us of the host.
#include "gated_delta_device.h"
#include "gated_delta_internal.h"

namespace gdr {
namespace {

constexpr int kRows = 4;      // value rows per lane
constexpr int kThreads = 256;

struct StepArgs {
    const void *q, *k, *v, *g, *beta;
    float *state;
    void *o;
    const int *slots;
    long long q_stride, k_stride, v_stride;
    int n_seq, Hk, Hv, V, pool;
    float scale;
    bool normalize;
};

template <int K>
__device__ __forceinline__ float row_sum(float x) {
    x = wkv7::sum_lanes16(x);
    if constexpr (K == 128) x = wkv7::swap16_add(x, x);
    return x;
}
__device__ __forceinline__ f32x4 load4(const bf16_t *p) {
    const uint2 u = *reinterpret_cast<const uint2 *>(p);
    return f32x4{wkv7::bf16_lo(u.x), wkv7::bf16_hi(u.x), wkv7::bf16_lo(u.y), wkv7::bf16_hi(u.y)};
}
__device__ __forceinline__ f32x4 load4(const float *p) {
    return *reinterpret_cast<const f32x4 *>(p);
}
__device__ __forceinline__ float dot4(f32x4 a, f32x4 b) {
    return a[0] * b[0] + a[1] * b[1] + a[2] * b[2] + a[3] * b[3];
}

template <class E, int K>
__global__ __launch_bounds__(kThreads) void step_kernel(StepArgs p) {
    constexpr int kLanes = K / 4;                                 // lanes per row
    constexpr int kWaveRows = 64 / kLanes * kRows;                // 16 or 8
    constexpr int kGroupRows = kWaveRows * (kThreads / 64);       // 64 or 32
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int parts = p.V / kGroupRows;
    const int part = (int)(blockIdx.x % parts);
    const int hv = (int)(blockIdx.x / parts % p.Hv), b = (int)(blockIdx.x / parts / p.Hv);
    const int slot = p.slots ? p.slots[b] : b;
    if (slot < 0 || slot >= p.pool) return;
    const int hk = hv / (p.Hv / p.Hk);
    const int c = lane % kLanes;
    const int r0 = part * kGroupRows + wave * kWaveRows + lane / kLanes * kRows;

    float *st = p.state + ((size_t)slot * p.Hv + hv) * p.V * K + (size_t)r0 * K + 4 * c;
    f32x4 S[kRows];
#pragma unroll
    for (int m = 0; m < kRows; ++m)
        S[m] = __builtin_nontemporal_load(reinterpret_cast<const f32x4 *>(st + m * K));
    f32x4 k = load4(static_cast<const E *>(p.k) + b * p.k_stride + hk * K + 4 * c);
    f32x4 q = load4(static_cast<const E *>(p.q) + b * p.q_stride + hk * K + 4 * c);
    const f32x4 v = load4(static_cast<const E *>(p.v) + b * p.v_stride + (size_t)hv * p.V + r0);
    const size_t at = (size_t)b * p.Hv + hv;
    const float a = __expf(to_float(static_cast<const E *>(p.g)[at]));
    const float beta = to_float(static_cast<const E *>(p.beta)[at]);
    if (p.normalize) {
        k *= 1.f / sqrtf(row_sum<K>(dot4(k, k)) + kNormEps);
        q *= 1.f / sqrtf(row_sum<K>(dot4(q, q)) + kNormEps);
    }
    const float kq = row_sum<K>(dot4(k, q));
    float o[kRows];
#pragma unroll
    for (int m = 0; m < kRows; ++m) {
        const float r = row_sum<K>(dot4(S[m], k)), s = row_sum<K>(dot4(S[m], q));
        const float be = beta * (v[m] - a * r);
        o[m] = p.scale * (a * s + be * kq);
        f32x4 x;
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = a * S[m][e] + be * k[e];
        __builtin_nontemporal_store(x, reinterpret_cast<f32x4 *>(st + m * K));
    }
    // lane c < 4 of a row group writes row r0 + c
    float mine = o[0];
#pragma unroll
    for (int m = 1; m < kRows; ++m) mine = c == m ? o[m] : mine;
    if (c < kRows)
        static_cast<E *>(p.o)[at * p.V + r0 + c] = from_float<E>(mine);
}

template <class E, int K>
hipError_t launch_step(const StepArgs &a, hipStream_t stream) {
    constexpr int kGroupRows = 64 / (K / 4) * kRows * (kThreads / 64);
    const size_t blocks = (size_t)a.n_seq * a.Hv * (a.V / kGroupRows);
    hipLaunchKernelGGL((step_kernel<E, K>), dim3((unsigned)blocks), dim3(kThreads), 0, stream, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_decode(const DecodeArgs &d, hipStream_t stream) {
    const Problem &p = d.p;
    StepArgs a{};
    a.q = d.q; a.k = d.k; a.v = d.v; a.g = d.g; a.beta = d.beta;
    a.state = d.state; a.o = d.o; a.slots = p.slots_in;
    a.q_stride = p.q_stride; a.k_stride = p.k_stride; a.v_stride = p.v_stride;
    a.n_seq = p.n_seq; a.Hk = p.Hk; a.Hv = p.Hv; a.V = p.V; a.pool = p.pool;
    a.scale = p.scale; a.normalize = p.normalize;
    if (p.bf16)
        return p.K == 64 ? launch_step<bf16_t, 64>(a, stream) : launch_step<bf16_t, 128>(a, stream);
    return p.K == 64 ? launch_step<float, 64>(a, stream) : launch_step<float, 128>(a, stream);
}

}  // namespace gdr
