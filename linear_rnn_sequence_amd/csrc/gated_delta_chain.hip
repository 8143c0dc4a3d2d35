// Gated delta rule: the pass over a sequence's chunks that carries the state
// (forward) or its cotangent (backward).
//
// Forward, per chunk with entry state S0 [V, K] and T, P of the preparation
// kernel (c_t = exp(G_t)):
//   R = diag(beta) (V - diag(c) K S0^T),  U = T R,
//   O = diag(scale c) Q S0^T + P U,       S_C = c_C S0 + U^T diag(c_C / c) K.
// Backward, with D the cotangent of the chunk's exit state:
//   dU = P^T dO + diag(c_C / c) K D^T,    dR = T^T dU,    dV = diag(beta) dR,
//   dS0 = c_C D + scale dO^T diag(c) Q - dR^T diag(beta c) K.
//
// A wave owns 16 NT values (rows of the state) over all keys and needs nothing of
// another wave: S^T lies in result tiles [keys, values], which are the right
// operands of K S0^T and Q S0^T as they stand; R, U come out as [tokens,
// values] tiles, the right operands of T R, P U and K^T U.  So a chunk is a
// chain of matrix-core products through registers.  The waves share the
// chunk's k and q (and dO) rows in shared memory, read along the rows for K, Q
// and down the columns for K^T, Q^T; the next chunk's rows are loaded into
// registers meanwhile.
//
// The state is float32 and what is added to it keeps 16 bits of significand or
// more (split operands, gated_delta_device.h), so that s_out and ds0 are
// float32 results; o is rounded to its type and takes S0 and U rounded to it.
#include "gated_delta_device.h"
#include "gated_delta_internal.h"

namespace gdr {
namespace {

struct ChainArgs {
    Layout lay;
    const void *q, *k, *v;  // backward: v is dO
    const char *records;
    const int *slots_in, *slots_out;
    const float *s_in;
    float *s_out;
    void *out;     // o, or dv
    void *states;  // forward: s_ckpt or nullptr; backward: D of every chunk
    void *mid;     // forward: u or nullptr; backward: dR
    long long q_stride, k_stride, v_stride;
    int Hk, Hv, V, pool;
};

template <int K, int NT>
struct State {
    f32x4 t[K / 16][NT];
};

// state of (idx, hv): rows value0 + 16 n + lo, keys in tile_row order
template <int K, int NT>
__device__ __forceinline__ void load_state(State<K, NT> &s, const float *base, int g, int lo) {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int ks = 0; ks < K / 32; ++ks)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                s.t[2 * ks + h][n] = *reinterpret_cast<const f32x4 *>(
                    base + (size_t)(16 * n + lo) * K + 32 * ks + 8 * g + 4 * h);
}
template <int K, int NT>
__device__ __forceinline__ void store_state(const State<K, NT> &s, float *base, int g, int lo) {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int ks = 0; ks < K / 32; ++ks)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                *reinterpret_cast<f32x4 *>(base + (size_t)(16 * n + lo) * K + 32 * ks + 8 * g +
                                           4 * h) = s.t[2 * ks + h][n];
}
// the same rounded to E (the operand of the gradient kernel's products)
template <class E, int K, int NT>
__device__ __forceinline__ void store_rounded(const State<K, NT> &s, E *base, int g, int lo) {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int ks = 0; ks < K / 32; ++ks) {
            const Frag<E> f = to_frag<E>(s.t[2 * ks][n], s.t[2 * ks + 1][n]);
            E *at = base + (size_t)(16 * n + lo) * K + 32 * ks + 8 * g;
            if constexpr (sizeof(E) == 2) {
                *reinterpret_cast<u32x4 *>(at) = f.v;
            } else {
                *reinterpret_cast<f32x4 *>(at) = f.v[0];
                *reinterpret_cast<f32x4 *>(at + 4) = f.v[1];
            }
        }
}

__device__ __forceinline__ f32x4 zero() { return f32x4{0.f, 0.f, 0.f, 0.f}; }

// index of a sequence's state in the pool, or -1
__device__ __forceinline__ int slot_of(const int *slots, int i, int pool) {
    const int s = slots ? slots[i] : i;
    return s >= 0 && s < pool ? s : -1;
}

template <class E, int K, int NT, int W, bool TRAIN>
__global__ __launch_bounds__(64 * W) void forward_chain_kernel(ChainArgs p) {
    using Rec = FwdRecord<E>;
    constexpr int kThreads = 64 * W, kValues = 16 * NT * W, KS = K / 32;
    extern __shared__ __align__(16) char lds[];
    Tile<E, K> tk{reinterpret_cast<E *>(lds)};
    Tile<E, K> tq{reinterpret_cast<E *>(lds + tile_bytes<E, K>(kChunk))};
    __shared__ Scalars sc;

    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), g = lane >> 4, lo = lane & 15;
    const int parts = p.V / kValues;
    const int part = (int)(blockIdx.x % parts);
    const int hv = (int)(blockIdx.x / parts % p.Hv), seq = (int)(blockIdx.x / parts / p.Hv);
    const int hk = hv / (p.Hv / p.Hk);
    const int value0 = part * kValues + wave * 16 * NT;
    const Seq sq = p.lay.seq(seq);
    const size_t state_size = (size_t)p.V * K;

    State<K, NT> S;
    const int in = p.s_in ? slot_of(p.slots_in, seq, p.pool) : -1;
    if (in >= 0) {
        load_state(S, p.s_in + ((size_t)in * p.Hv + hv) * state_size + (size_t)value0 * K, g, lo);
    } else {
#pragma unroll
        for (int m = 0; m < K / 16; ++m)
#pragma unroll
            for (int n = 0; n < NT; ++n) S.t[m][n] = zero();
    }

    const E *kp = static_cast<const E *>(p.k) + (long long)hk * K;
    const E *qp = static_cast<const E *>(p.q) + (long long)hk * K;
    const E *vp = static_cast<const E *>(p.v) + (long long)hv * p.V + value0 + lo;
    const long long row = (long long)p.Hv * p.V;  // dense rows of o and u
    E *op = static_cast<E *>(p.out) + (long long)hv * p.V + value0 + lo;
    E *up = static_cast<E *>(p.mid) + (long long)hv * p.V + value0 + lo;

    Stage<E, K, kChunk, kThreads> gk, gq;
    const int len = sq.end - sq.begin;
    if (len > 0) {
        const int live = len < kChunk ? len : kChunk;
        gk.load(kp + sq.begin * p.k_stride, p.k_stride, live, tid);
        gq.load(qp + sq.begin * p.q_stride, p.q_stride, live, tid);
    }
    for (int c = 0; c * kChunk < len; ++c) {
        const long long first = sq.begin + (long long)c * kChunk;
        const int live = len - c * kChunk < kChunk ? len - c * kChunk : kChunk;
        const size_t chunk_head = (size_t)(sq.slot0 + c) * p.Hv + hv;
        const char *rec = p.records + chunk_head * Rec::kBytes;
        if (c) __syncthreads();  // the last chunk's reads
        gk.store(tk, tid);
        gq.store(tq, tid);
        for (int i = tid; i < (int)sizeof(Scalars) / 16; i += kThreads)
            reinterpret_cast<u32x4 *>(&sc)[i] =
                reinterpret_cast<const u32x4 *>(rec + Rec::kScalars)[i];
        __syncthreads();
        // this chunk's values and matrices, the next chunk's rows
        f32x4 R[4][NT];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int t = tile_row(i, 4 * g + e);
                    R[i][n][e] = t < live ? to_float(vp[(first + t) * p.v_stride + 16 * n]) : 0.f;
                }
        Split<E> T[6];
#pragma unroll
        for (int f = 0; f < 6; ++f) T[f] = get_split<E>(rec + f * Rec::kSplitBytes, lane);
        if ((c + 1) * kChunk < len) {
            const int left = len - (c + 1) * kChunk, l2 = left < kChunk ? left : kChunk;
            gk.load(kp + (first + kChunk) * p.k_stride, p.k_stride, l2, tid);
            gq.load(qp + (first + kChunk) * p.q_stride, p.q_stride, l2, tid);
        }
        if (TRAIN)
            store_rounded<E>(S, static_cast<E *>(p.states) + chunk_head * state_size +
                                    (size_t)value0 * K, g, lo);

        f32x4 O[4][NT];
        {
            f32x4 X[4][NT];
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int n = 0; n < NT; ++n) X[i][n] = O[i][n] = zero();
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                Split<E> b[NT];
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    b[n] = to_split<E>(S.t[2 * ks][n], S.t[2 * ks + 1][n]);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int r = tile_row(i, lo);
                    const Frag<E> fk = tk.rows(r, 32 * ks, g), fq = tq.rows(r, 32 * ks, g);
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        X[i][n] = mma(fk, b[n], X[i][n]);
                        O[i][n] = mma(fq, b[n].hi, O[i][n]);
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int t = tile_row(i, 4 * g + e);
                    const float be = sc.beta[t], ks = sc.kS[t], qs = sc.qS[t];
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        R[i][n][e] = be * R[i][n][e] - ks * X[i][n][e];
                        O[i][n][e] *= qs;
                    }
                }
        }
        f32x4 U[4][NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int i = 0; i < 4; ++i) U[i][n] = zero();
#pragma unroll
            for (int st = 0; st < 2; ++st) {
                const Split<E> b = to_split<E>(R[2 * st][n], R[2 * st + 1][n]);
#pragma unroll
                for (int f = 0; f < 6; ++f)
                    if (kLowStep[f] == st) U[kLowTile[f]][n] = mma(T[f], b, U[kLowTile[f]][n]);
            }
        }
        // the readout
#pragma unroll
        for (int st = 0; st < 2; ++st) {
            Frag<E> b[NT];
#pragma unroll
            for (int n = 0; n < NT; ++n) b[n] = to_frag<E>(U[2 * st][n], U[2 * st + 1][n]);
#pragma unroll
            for (int f = 0; f < 6; ++f)
                if (kLowStep[f] == st) {
                    const Frag<E> a = get_frag<E>(rec + Rec::kP + f * Rec::kFragBytes, lane);
#pragma unroll
                    for (int n = 0; n < NT; ++n)
                        O[kLowTile[f]][n] = mma(a, b[n], O[kLowTile[f]][n]);
                }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int t = tile_row(i, 4 * g + e);
                const float kd = sc.kD[t];
                if (t < live)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
                        op[(first + t) * row + 16 * n] = from_float<E>(O[i][n][e]);
                if (TRAIN && t < live)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
                        up[(first + t) * row + 16 * n] = from_float<E>(U[i][n][e]);
#pragma unroll
                for (int n = 0; n < NT; ++n) U[i][n][e] *= kd;
            }
        // the state
        const float last = sc.last;
#pragma unroll
        for (int m = 0; m < K / 16; ++m)
#pragma unroll
            for (int n = 0; n < NT; ++n) S.t[m][n] *= last;
#pragma unroll
        for (int st = 0; st < 2; ++st) {
            Split<E> b[NT];
#pragma unroll
            for (int n = 0; n < NT; ++n) b[n] = to_split<E>(U[2 * st][n], U[2 * st + 1][n]);
#pragma unroll
            for (int m = 0; m < K / 16; ++m) {
                const Frag<E> a =
                    tk.template cols<8>(32 * st, 32 * (m >> 1) + 4 * (m & 1), lane);
#pragma unroll
                for (int n = 0; n < NT; ++n) S.t[m][n] = mma(a, b[n], S.t[m][n]);
            }
        }
    }
    if (p.s_out) {
        const int out = slot_of(p.slots_out, seq, p.pool);
        if (out >= 0)
            store_state(S, p.s_out + ((size_t)out * p.Hv + hv) * state_size + (size_t)value0 * K,
                        g, lo);
    }
}

template <class E, int K, int NT, int W>
__global__ __launch_bounds__(64 * W) void backward_chain_kernel(ChainArgs p) {
    using Rec = BwdRecord<E>;
    constexpr int kThreads = 64 * W, kValues = 16 * NT * W, KS = K / 32;
    extern __shared__ __align__(16) char lds[];
    Tile<E, K> tk{reinterpret_cast<E *>(lds)};
    Tile<E, K> tq{reinterpret_cast<E *>(lds + tile_bytes<E, K>(kChunk))};
    Tile<E, kValues> to{reinterpret_cast<E *>(lds + 2 * tile_bytes<E, K>(kChunk))};
    __shared__ Scalars sc;

    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), g = lane >> 4, lo = lane & 15;
    const int parts = p.V / kValues;
    const int part = (int)(blockIdx.x % parts);
    const int hv = (int)(blockIdx.x / parts % p.Hv), seq = (int)(blockIdx.x / parts / p.Hv);
    const int hk = hv / (p.Hv / p.Hk);
    const int value0 = part * kValues + wave * 16 * NT;
    const Seq sq = p.lay.seq(seq);
    const size_t state_size = (size_t)p.V * K;

    State<K, NT> D;
    const size_t state_at = ((size_t)seq * p.Hv + hv) * state_size + (size_t)value0 * K;
    if (p.s_in) {
        load_state(D, p.s_in + state_at, g, lo);
    } else {
#pragma unroll
        for (int m = 0; m < K / 16; ++m)
#pragma unroll
            for (int n = 0; n < NT; ++n) D.t[m][n] = zero();
    }

    const long long row = (long long)p.Hv * p.V;
    const E *kp = static_cast<const E *>(p.k) + (long long)hk * K;
    const E *qp = static_cast<const E *>(p.q) + (long long)hk * K;
    const E *dop = static_cast<const E *>(p.v) + (long long)hv * p.V + part * kValues;
    E *dvp = static_cast<E *>(p.out) + (long long)hv * p.V + value0 + lo;
    E *drp = static_cast<E *>(p.mid) + (long long)hv * p.V + value0 + lo;

    const int len = sq.end - sq.begin;
    const int chunks = (len + kChunk - 1) / kChunk;
    Stage<E, K, kChunk, kThreads> gk, gq;
    Stage<E, kValues, kChunk, kThreads> go;
    auto fetch = [&](int c) {
        const long long first = sq.begin + (long long)c * kChunk;
        const int live = len - c * kChunk < kChunk ? len - c * kChunk : kChunk;
        gk.load(kp + first * p.k_stride, p.k_stride, live, tid);
        gq.load(qp + first * p.q_stride, p.q_stride, live, tid);
        go.load(dop + first * row, row, live, tid);
    };
    if (chunks > 0) fetch(chunks - 1);
    for (int c = chunks - 1; c >= 0; --c) {
        const long long first = sq.begin + (long long)c * kChunk;
        const int live = len - c * kChunk < kChunk ? len - c * kChunk : kChunk;
        const size_t chunk_head = (size_t)(sq.slot0 + c) * p.Hv + hv;
        const char *rec = p.records + chunk_head * Rec::kBytes;
        if (c != chunks - 1) __syncthreads();
        gk.store(tk, tid);
        gq.store(tq, tid);
        go.store(to, tid);
        for (int i = tid; i < (int)sizeof(Scalars) / 16; i += kThreads)
            reinterpret_cast<u32x4 *>(&sc)[i] =
                reinterpret_cast<const u32x4 *>(rec + Rec::kScalars)[i];
        __syncthreads();
        if (c > 0) fetch(c - 1);
        store_rounded<E>(D, static_cast<E *>(p.states) + chunk_head * state_size +
                                (size_t)value0 * K, g, lo);

        // dU = diag(c_C / c) K D^T + P^T dO
        f32x4 X[4][NT];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int n = 0; n < NT; ++n) X[i][n] = zero();
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            Split<E> b[NT];
#pragma unroll
            for (int n = 0; n < NT; ++n) b[n] = to_split<E>(D.t[2 * ks][n], D.t[2 * ks + 1][n]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const Frag<E> fk = tk.rows(tile_row(i, lo), 32 * ks, g);
#pragma unroll
                for (int n = 0; n < NT; ++n) X[i][n] = mma(fk, b[n], X[i][n]);
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float kd = sc.kD[tile_row(i, 4 * g + e)];
#pragma unroll
                for (int n = 0; n < NT; ++n) X[i][n][e] *= kd;
            }
        Frag<E> fo[2][NT];
#pragma unroll
        for (int st = 0; st < 2; ++st)
#pragma unroll
            for (int n = 0; n < NT; ++n)
                fo[st][n] = to.template cols<4>(32 * st, wave * 16 * NT + 16 * n, lane);
#pragma unroll
        for (int f = 0; f < 6; ++f) {
            const Split<E> a = get_split<E>(rec + Rec::kP + f * Rec::kSplitBytes, lane);
#pragma unroll
            for (int n = 0; n < NT; ++n)
                X[kUpTile[f]][n] = mma(a, fo[kUpStep[f]][n], X[kUpTile[f]][n]);
        }
        // dR = T^T dU
        f32x4 R[4][NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int i = 0; i < 4; ++i) R[i][n] = zero();
#pragma unroll
            for (int st = 0; st < 2; ++st) {
                const Split<E> b = to_split<E>(X[2 * st][n], X[2 * st + 1][n]);
#pragma unroll
                for (int f = 0; f < 6; ++f)
                    if (kUpStep[f] == st)
                        R[kUpTile[f]][n] =
                            mma(get_split<E>(rec + f * Rec::kSplitBytes, lane), b, R[kUpTile[f]][n]);
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int t = tile_row(i, 4 * g + e);
                const float be = sc.beta[t], ks = -sc.kS[t];
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    if (t < live) {
                        drp[(first + t) * row + 16 * n] = from_float<E>(R[i][n][e]);
                        dvp[(first + t) * row + 16 * n] = from_float<E>(be * R[i][n][e]);
                    }
                    R[i][n][e] *= ks;
                }
            }
        // dS0 = c_C D + dO^T diag(scale c / |q|) Q - dR^T diag(beta c / |k|) K
        const float last = sc.last;
#pragma unroll
        for (int m = 0; m < K / 16; ++m)
#pragma unroll
            for (int n = 0; n < NT; ++n) D.t[m][n] *= last;
#pragma unroll
        for (int st = 0; st < 2; ++st) {
            Split<E> b[NT], bo[NT];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                b[n] = to_split<E>(R[2 * st][n], R[2 * st + 1][n]);
                f32x4 x0, x1;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    x0[e] = fo[st][n].at(e) * sc.qS[32 * st + 8 * g + e];
                    x1[e] = fo[st][n].at(4 + e) * sc.qS[32 * st + 8 * g + 4 + e];
                }
                bo[n] = to_split<E>(x0, x1);
            }
#pragma unroll
            for (int m = 0; m < K / 16; ++m) {
                const int col = 32 * (m >> 1) + 4 * (m & 1);
                const Frag<E> ak = tk.template cols<8>(32 * st, col, lane);
                const Frag<E> aq = tq.template cols<8>(32 * st, col, lane);
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    D.t[m][n] = mma(aq, bo[n], mma(ak, b[n], D.t[m][n]));
            }
        }
    }
    if (p.s_out) store_state(D, p.s_out + state_at, g, lo);
}

template <class E, int K, int NT, int W>
hipError_t launch_forward_t(const ChainArgs &a, bool train, int n_seq, hipStream_t stream) {
    constexpr int kLds = 2 * tile_bytes<E, K>(kChunk);
    const auto fn = train ? forward_chain_kernel<E, K, NT, W, true>
                          : forward_chain_kernel<E, K, NT, W, false>;
    const hipError_t e = hipFuncSetAttribute(
        reinterpret_cast<const void *>(fn), hipFuncAttributeMaxDynamicSharedMemorySize, kLds);
    if (e != hipSuccess) return e;
    const size_t blocks = (size_t)n_seq * a.Hv * (a.V / (16 * NT * W));
    hipLaunchKernelGGL(fn, dim3((unsigned)blocks), dim3(64 * W), kLds, stream, a);
    return hipGetLastError();
}

template <class E, int K, int NT, int W>
hipError_t launch_backward_t(const ChainArgs &a, int n_seq, hipStream_t stream) {
    constexpr int kLds = 2 * tile_bytes<E, K>(kChunk) + tile_bytes<E, 16 * NT * W>(kChunk);
    const auto fn = backward_chain_kernel<E, K, NT, W>;
    const hipError_t e = hipFuncSetAttribute(
        reinterpret_cast<const void *>(fn), hipFuncAttributeMaxDynamicSharedMemorySize, kLds);
    if (e != hipSuccess) return e;
    const size_t blocks = (size_t)n_seq * a.Hv * (a.V / (16 * NT * W));
    hipLaunchKernelGGL(fn, dim3((unsigned)blocks), dim3(64 * W), kLds, stream, a);
    return hipGetLastError();
}

ChainArgs chain_args(const Problem &p) {
    ChainArgs a{};
    a.lay = Layout{p.cu, p.n_seq, p.T, p.total, p.slots};
    a.q_stride = p.q_stride; a.k_stride = p.k_stride; a.v_stride = p.v_stride;
    a.Hk = p.Hk; a.Hv = p.Hv; a.V = p.V; a.pool = p.pool;
    a.slots_in = p.slots_in; a.slots_out = p.slots_out;
    return a;
}

}  // namespace

int chain_values(const Problem &, bool) { return 64; }

hipError_t launch_forward(const ForwardArgs &f, hipStream_t stream) {
    const Problem &p = f.p;
    hipError_t e = launch_prep(p, f.q, f.k, f.g, f.beta, f.records, false, stream);
    if (e != hipSuccess) return e;
    ChainArgs a = chain_args(p);
    a.q = f.q; a.k = f.k; a.v = f.v;
    a.records = f.records;
    a.s_in = f.s0; a.s_out = f.s_out;
    a.out = f.o; a.states = f.s_ckpt; a.mid = f.u;
    const bool train = f.s_ckpt != nullptr;
    if (p.bf16)
        return p.K == 64 ? launch_forward_t<bf16_t, 64, 1, 4>(a, train, p.n_seq, stream)
                         : launch_forward_t<bf16_t, 128, 1, 4>(a, train, p.n_seq, stream);
    return p.K == 64 ? launch_forward_t<float, 64, 1, 4>(a, train, p.n_seq, stream)
                     : launch_forward_t<float, 128, 1, 4>(a, train, p.n_seq, stream);
}

hipError_t launch_backward_chain(const BackwardArgs &b, hipStream_t stream) {
    const Problem &p = b.p;
    hipError_t e = launch_prep(p, b.q, b.k, b.g, b.beta, b.records, true, stream);
    if (e != hipSuccess) return e;
    ChainArgs a = chain_args(p);
    a.q = b.q; a.k = b.k; a.v = b.d_o;
    a.records = b.records;
    a.s_in = b.ds_T; a.s_out = b.ds0;
    a.out = b.dv; a.states = b.ds; a.mid = b.dr;
    if (p.bf16)
        return p.K == 64 ? launch_backward_t<bf16_t, 64, 1, 4>(a, p.n_seq, stream)
                         : launch_backward_t<bf16_t, 128, 1, 4>(a, p.n_seq, stream);
    return p.K == 64 ? launch_backward_t<float, 64, 1, 4>(a, p.n_seq, stream)
                     : launch_backward_t<float, 128, 1, 4>(a, p.n_seq, stream);
}

}  // namespace gdr
