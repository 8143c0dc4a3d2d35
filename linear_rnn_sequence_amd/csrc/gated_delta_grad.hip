// Gated delta rule, backward: the gradients of one chunk from its entry state S0,
// its exit cotangent D, and U, dR of every token (all stored by the two chain
// kernels), every chunk in parallel.
//
// With c_t = exp(G_t), E_ts = exp(G_t - G_s), unit vectors or not as the forward:
//   dP = dO U^T (s <= t),  dA = -dR U^T (s < t),
//   MP = dP * scale E,  MA = dA * beta E  (elementwise, beta of the row),
//   dQ = scale diag(c) dO S0 + MP K,
//   dK = -diag(beta c) dR S0 + diag(c_C / c) U D + MP^T Q + MA K + MA^T K,
//   dbeta_t = dR_t . (v_t - c_t S0 k_t) + sum_s dA_ts E_ts k_t . k_s,
// and, since the decay at t lies on every path from a token before t (or from
// the entry state) to a token at or behind t (or to the exit state),
//   dg_t = sum_{s < t <= t'} (MP * q.k + MA * k.k)_{t's}
//        + sum_{t' >= t} c_t' (scale dO_t' . S0 q_t' - beta dR_t' . S0 k_t')
//        + sum_{s < t} (c_C / c_s) U_s . D k_s + c_C <D, S0>,
// a sum over a rectangle of pairs, in which nothing cancels (differences of row
// and column sums of the same matrices would).
//
// One workgroup of four waves per chunk and key head; it goes through the value
// heads that share the key head and adds their dq and dk up in registers, so no
// atomics are needed and the order of the sums is fixed.  Wave w owns tokens
// 16w .. 16w + 15.  It forms dP and dA in both orientations (rows s for the
// sums over s, rows t for those over t): each then is an operand of the next
// product as it stands, which costs five products of 16 x 16 x V twice instead
// of an exchange between waves.
#include "gated_delta_device.h"
#include "gated_delta_internal.h"

namespace gdr {
namespace {

constexpr int kVt = 32;                // values per step
constexpr int kPitchM = kChunk + 4;

struct GradArgs {
    Layout lay;
    const void *q, *k, *v, *g, *beta, *d_o, *s_ckpt, *u, *ds, *dr;
    void *dq, *dk, *dg, *dbeta;
    long long q_stride, k_stride, v_stride;
    int Hk, Hv, V;
    float scale;
    bool normalize;
};

__device__ __forceinline__ f32x4 zero() { return f32x4{0.f, 0.f, 0.f, 0.f}; }

template <class E, int K>
struct GradLds {
    static constexpr int kQ = tile_bytes<E, K>(kChunk);
    static constexpr int kO = 2 * kQ;
    static constexpr int kOSize = tile_bytes<E, kVt>(kChunk);
    static constexpr int kS = kO + 3 * kOSize;
    static constexpr int kSSize = tile_bytes<E, K>(kVt);
    static constexpr int kBytes = kS + 2 * kSSize;
    // M takes the place of the value steps' tiles
    static_assert(3 * kOSize + 2 * kSSize >= kChunk * kPitchM * 4, "M fits");
};

template <class E, int K>
__global__ __launch_bounds__(256) void gradient_kernel(GradArgs p) {
    using L = GradLds<E, K>;
    constexpr int NK = K / 16;
    extern __shared__ __align__(16) char lds[];
    Tile<E, K> tk{reinterpret_cast<E *>(lds)}, tq{reinterpret_cast<E *>(lds + L::kQ)};
    Tile<E, kVt> to{reinterpret_cast<E *>(lds + L::kO)},
        tr{reinterpret_cast<E *>(lds + L::kO + L::kOSize)},
        tu{reinterpret_cast<E *>(lds + L::kO + 2 * L::kOSize)};
    Tile<E, K> ts{reinterpret_cast<E *>(lds + L::kS)},
        td{reinterpret_cast<E *>(lds + L::kS + L::kSSize)};
    float *sM = reinterpret_cast<float *>(lds + L::kO);
    __shared__ double sG[kChunk];
    __shared__ float sBeta[kChunk], sGrown[kChunk], sRest[kChunk], sRk[kChunk], sRq[kChunk];
    __shared__ float sEntry[kChunk], sLeave[kChunk], sKS[kChunk], sDb[kChunk], sDRV[kChunk],
        sPairs[kChunk], sDS[4];

    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), g = lane >> 4, lo = lane & 15;
    const int half = wave >> 1;
    const int slot = (int)(blockIdx.x / p.Hk), hk = (int)(blockIdx.x % p.Hk);
    Seq sq;
    p.lay.find(slot, sq);
    const int first = sq.begin + (slot - sq.slot0) * kChunk;
    if (slot < sq.slot0 || first >= sq.end) return;  // the whole workgroup
    const int live = sq.end - first < kChunk ? sq.end - first : kChunk;
    const int rep = p.Hv / p.Hk;
    const long long row = (long long)p.Hv * p.V;

    {
        Stage<E, K, kChunk, 256> a, b;
        a.load(static_cast<const E *>(p.k) + first * p.k_stride + (long long)hk * K, p.k_stride,
               live, tid);
        b.load(static_cast<const E *>(p.q) + first * p.q_stride + (long long)hk * K, p.q_stride,
               live, tid);
        a.store(tk, tid);
        b.store(tq, tid);
    }
    __syncthreads();
    {  // reciprocal norms: four lanes per token
        const int t = tid >> 2, part = tid & 3;
        float a = 0.f, b = 0.f;
#pragma unroll 8
        for (int c = part * (K / 4); c < (part + 1) * (K / 4); ++c) {
            const float x = tk.at(t, c), y = tq.at(t, c);
            a += x * x;
            b += y * y;
        }
        a += wkv7::dpp_mov<wkv7::kDppQuadXor1>(a);
        a += wkv7::dpp_mov<wkv7::kDppQuadXor2>(a);
        b += wkv7::dpp_mov<wkv7::kDppQuadXor1>(b);
        b += wkv7::dpp_mov<wkv7::kDppQuadXor2>(b);
        if (part == 0) {
            sRk[t] = p.normalize ? 1.f / sqrtf(a + kNormEps) : 1.f;
            sRq[t] = p.normalize ? 1.f / sqrtf(b + kNormEps) : 1.f;
        }
    }
    // k.k and q.k, rows s in tile_row order, columns t = 16 wave + lo
    f32x4 kk[4], qk[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) kk[i] = qk[i] = zero();
#pragma unroll
    for (int ks = 0; ks < K / 32; ++ks) {
        const Frag<E> bk = tk.rows(16 * wave + lo, 32 * ks, g),
                      bq = tq.rows(16 * wave + lo, 32 * ks, g);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < 2 * half + 2) {
                const Frag<E> a = tk.rows(tile_row(i, lo), 32 * ks, g);
                kk[i] = mma(a, bk, kk[i]);
                qk[i] = mma(a, bq, qk[i]);
            }
    }
    f32x4 dQ[NK], dK[NK];
#pragma unroll
    for (int n = 0; n < NK; ++n) dQ[n] = dK[n] = zero();

    for (int r = 0; r < rep; ++r) {
        const int hv = hk * rep + r;
        const size_t chunk_head = (size_t)slot * p.Hv + hv;
        const E *op = static_cast<const E *>(p.d_o) + first * row + (long long)hv * p.V;
        const E *rp = static_cast<const E *>(p.dr) + first * row + (long long)hv * p.V;
        const E *up = static_cast<const E *>(p.u) + first * row + (long long)hv * p.V;
        const E *sp = static_cast<const E *>(p.s_ckpt) + chunk_head * p.V * K;
        const E *dp = static_cast<const E *>(p.ds) + chunk_head * p.V * K;
        const E *vp = static_cast<const E *>(p.v) + first * p.v_stride + (long long)hv * p.V;

        f32x4 oS[NK], rS[NK], uD[NK], P1[4], A1[4], P2[4], A2[4];
#pragma unroll
        for (int n = 0; n < NK; ++n) oS[n] = rS[n] = uD[n] = zero();
#pragma unroll
        for (int i = 0; i < 4; ++i) P1[i] = A1[i] = P2[i] = A2[i] = zero();
        float ds_sum = 0.f, drv = 0.f;

        for (int v0 = 0; v0 < p.V; v0 += kVt) {
            Stage<E, kVt, kChunk, 256> go, gr, gu;
            Stage<E, K, kVt, 256> gs, gd;
            go.load(op + v0, row, live, tid);
            gr.load(rp + v0, row, live, tid);
            gu.load(up + v0, row, live, tid);
            gs.load(sp + (size_t)v0 * K, K, kVt, tid);
            gd.load(dp + (size_t)v0 * K, K, kVt, tid);
            __syncthreads();  // the last step's reads (and those of the last head's M)
            go.store(to, tid);
            gr.store(tr, tid);
            gu.store(tu, tid);
            gs.store(ts, tid);
            gd.store(td, tid);
            __syncthreads();
            const Frag<E> fo = to.rows(16 * wave + lo, 0, g), fr = tr.rows(16 * wave + lo, 0, g),
                          fu = tu.rows(16 * wave + lo, 0, g);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int t = tile_row(i, lo);
                if (i < 2 * half + 2) {
                    const Frag<E> a = tu.rows(t, 0, g);
                    P1[i] = mma(a, fo, P1[i]);
                    A1[i] = mma(a, fr, A1[i]);
                }
                if (i >= 2 * half) {
                    P2[i] = mma(to.rows(t, 0, g), fu, P2[i]);
                    A2[i] = mma(tr.rows(t, 0, g), fu, A2[i]);
                }
            }
#pragma unroll
            for (int n = 0; n < NK; ++n) {
                const Frag<E> bs = ts.template cols<4>(0, 16 * n, lane),
                              bd = td.template cols<4>(0, 16 * n, lane);
                oS[n] = mma(fo, bs, oS[n]);
                rS[n] = mma(fr, bs, rS[n]);
                uD[n] = mma(fu, bd, uD[n]);
            }
            {  // <D, S0>: 32 K products
                const int x = tid >> 3, y0 = (tid & 7) * (K / 8);
#pragma unroll 8
                for (int y = y0; y < y0 + K / 8; ++y) ds_sum += ts.at(x, y) * td.at(x, y);
            }
            {  // dR . v: four lanes per token
                const int t = tid >> 2, x0 = (tid & 3) * (kVt / 4);
                if (t < live)
#pragma unroll
                    for (int x = x0; x < x0 + kVt / 4; ++x)
                        drv += tr.at(t, x) * to_float(vp[t * p.v_stride + v0 + x]);
            }
        }
        if (wave == 0) {
            const long long at = (long long)(first + lane) * p.Hv + hv;
            const float gt = lane < live ? to_float(static_cast<const E *>(p.g)[at]) : 0.f;
            const float bt = lane < live ? to_float(static_cast<const E *>(p.beta)[at]) : 0.f;
            const double G = scan_decay(gt, lane);
            sG[lane] = G;
            sBeta[lane] = bt;
            sGrown[lane] = decay(G, 0.0);
            sRest[lane] = decay(__shfl(G, 63), G);
        }
        drv += wkv7::dpp_mov<wkv7::kDppQuadXor1>(drv);
        drv += wkv7::dpp_mov<wkv7::kDppQuadXor2>(drv);
        if ((tid & 3) == 0) sDRV[tid >> 2] = drv;
        ds_sum = wkv7::sum_rows4(wkv7::sum_lanes16(ds_sum));
        if (lane == 0) sDS[wave] = ds_sum;
        __syncthreads();

        // what goes through the states
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int t = 16 * wave + 4 * g + e;
            const float grown = sGrown[t], rest = sRest[t], be = sBeta[t], rk = sRk[t],
                        rq = sRq[t];
            float oq = 0.f, rkd = 0.f, ud = 0.f;
#pragma unroll
            for (int n = 0; n < NK; ++n) {
                const float kx = tk.at(t, 16 * n + lo), qx = tq.at(t, 16 * n + lo);
                oq += oS[n][e] * qx;
                rkd += rS[n][e] * kx;
                ud += uD[n][e] * kx;
                dQ[n][e] += p.scale * grown * oS[n][e];
                dK[n][e] += rest * uD[n][e] - be * grown * rS[n][e];
            }
            oq = wkv7::sum_lanes16(oq) * p.scale * grown * rq;
            rkd = wkv7::sum_lanes16(rkd) * grown * rk;
            ud = wkv7::sum_lanes16(ud) * rest * rk;
            if (lo == 0) {
                sEntry[t] = oq - be * rkd;
                sLeave[t] = ud;
                sKS[t] = rkd;
            }
        }
        // pairs, columns t = 16 wave + lo: MP and MA as left operands with rows t
        {
            const int t = 16 * wave + lo;
            const double Gt = sG[t];
            const float be = sBeta[t], rkt = sRk[t], rqt = sRq[t];
            float db = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (i >= 2 * half + 2) break;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int s = tile_row(i, 4 * g + e);
                    const float rks = sRk[s];
                    const float E_ts = s <= t ? decay(Gt, sG[s]) : 0.f;
                    const float mp = s <= t ? p.scale * E_ts * P1[i][e] : 0.f;
                    const float da = s < t ? -E_ts * A1[i][e] : 0.f;
                    const float dak = da * kk[i][e] * rkt * rks;
                    db += dak;
                    if (s < t) sM[t * kPitchM + s] = mp * qk[i][e] * rqt * rks + be * dak;
                    P1[i][e] = mp * rks;
                    A1[i][e] = be * da * rks;
                }
            }
            db = wkv7::sum_rows4(db);
            if (g == 0) sDb[t] = db;
        }
        // and rows t, columns s = 16 wave + lo: the left operands MP^T and MA^T
        {
            const int s = 16 * wave + lo;
            const double Gs = sG[s];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (i < 2 * half) continue;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int t = tile_row(i, 4 * g + e);
                    const float E_ts = s <= t ? decay(sG[t], Gs) : 0.f;
                    P2[i][e] = s <= t ? p.scale * E_ts * P2[i][e] * sRq[t] : 0.f;
                    A2[i][e] = s < t ? -sBeta[t] * E_ts * A2[i][e] * sRk[t] : 0.f;
                }
            }
        }
#pragma unroll
        for (int st = 0; st < 2; ++st) {
            if (st <= half) {
                const Frag<E> fp = to_frag<E>(P1[2 * st], P1[2 * st + 1]),
                              fa = to_frag<E>(A1[2 * st], A1[2 * st + 1]);
#pragma unroll
                for (int n = 0; n < NK; ++n) {
                    const Frag<E> b = tk.template cols<4>(32 * st, 16 * n, lane);
                    dQ[n] = mma(fp, b, dQ[n]);
                    dK[n] = mma(fa, b, dK[n]);
                }
            }
            if (st >= half) {
                const Frag<E> fp = to_frag<E>(P2[2 * st], P2[2 * st + 1]),
                              fa = to_frag<E>(A2[2 * st], A2[2 * st + 1]);
#pragma unroll
                for (int n = 0; n < NK; ++n) {
                    dK[n] = mma(fp, tq.template cols<4>(32 * st, 16 * n, lane), dK[n]);
                    dK[n] = mma(fa, tk.template cols<4>(32 * st, 16 * n, lane), dK[n]);
                }
            }
        }
        __syncthreads();
        // sums over the rectangles s < t <= t': down each quarter of a column first
        {
            float run = 0.f;
            const int s = lane;
#pragma unroll
            for (int i = 15; i >= 0; --i) {
                const int t = 16 * wave + i;
                if (s < t) {
                    run += sM[t * kPitchM + s];
                    sM[t * kPitchM + s] = run;
                }
            }
        }
        __syncthreads();
        {
            const int t = tid >> 2, part = tid & 3, quarter = t >> 4;
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int s = 4 * i + part;
                if (s < t) {
                    sum += sM[t * kPitchM + s];
                    for (int x = quarter + 1; x < 4; ++x) sum += sM[16 * x * kPitchM + s];
                }
            }
            sum += wkv7::dpp_mov<wkv7::kDppQuadXor1>(sum);
            sum += wkv7::dpp_mov<wkv7::kDppQuadXor2>(sum);
            if (part == 0) sPairs[t] = sum;
        }
        __syncthreads();
        if (wave == 0) {
            float entry = sEntry[lane], leave = sLeave[lane];
            const float own = leave;
#pragma unroll
            for (int d = 1; d < 64; d <<= 1) {
                const float a = __shfl_down(entry, d), b = __shfl_up(leave, d);
                if (lane + d < 64) entry += a;
                if (lane >= d) leave += b;
            }
            const float whole = sGrown[63] * (sDS[0] + sDS[1] + sDS[2] + sDS[3]);
            if (lane < live) {
                const long long at = (long long)(first + lane) * p.Hv + hv;
                static_cast<E *>(p.dg)[at] =
                    from_float<E>(sPairs[lane] + entry + (leave - own) + whole);
                static_cast<E *>(p.dbeta)[at] =
                    from_float<E>(sDRV[lane] - sKS[lane] + sDb[lane]);
            }
        }
    }

    // the gradient of x / |x| from that of the unit vector, and out
    E *dqp = static_cast<E *>(p.dq) + (long long)first * p.Hk * K + (long long)hk * K + lo;
    E *dkp = static_cast<E *>(p.dk) + (long long)first * p.Hk * K + (long long)hk * K + lo;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int t = 16 * wave + 4 * g + e;
        if (p.normalize) {
            const float rk = sRk[t], rq = sRq[t];
            float a = 0.f, b = 0.f;
#pragma unroll
            for (int n = 0; n < NK; ++n) {
                a += dQ[n][e] * tq.at(t, 16 * n + lo);
                b += dK[n][e] * tk.at(t, 16 * n + lo);
            }
            a = wkv7::sum_lanes16(a) * rq * rq;
            b = wkv7::sum_lanes16(b) * rk * rk;
#pragma unroll
            for (int n = 0; n < NK; ++n) {
                dQ[n][e] = rq * (dQ[n][e] - tq.at(t, 16 * n + lo) * a);
                dK[n][e] = rk * (dK[n][e] - tk.at(t, 16 * n + lo) * b);
            }
        }
        if (t < live)
#pragma unroll
            for (int n = 0; n < NK; ++n) {
                dqp[(long long)t * p.Hk * K + 16 * n] = from_float<E>(dQ[n][e]);
                dkp[(long long)t * p.Hk * K + 16 * n] = from_float<E>(dK[n][e]);
            }
    }
}

template <class E, int K>
hipError_t launch_gradients_t(const GradArgs &a, int slots, hipStream_t stream) {
    constexpr int kLds = GradLds<E, K>::kBytes;
    const auto fn = gradient_kernel<E, K>;
    const hipError_t e = hipFuncSetAttribute(
        reinterpret_cast<const void *>(fn), hipFuncAttributeMaxDynamicSharedMemorySize, kLds);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(fn, dim3((unsigned)((size_t)slots * a.Hk)), dim3(256), kLds, stream, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_gradients(const BackwardArgs &b, hipStream_t stream) {
    const Problem &p = b.p;
    if (p.slots == 0) return hipSuccess;
    GradArgs a{};
    a.lay = Layout{p.cu, p.n_seq, p.T, p.total, p.slots};
    a.q = b.q; a.k = b.k; a.v = b.v; a.g = b.g; a.beta = b.beta;
    a.d_o = b.d_o; a.s_ckpt = b.s_ckpt; a.u = b.u; a.ds = b.ds; a.dr = b.dr;
    a.dq = b.dq; a.dk = b.dk; a.dg = b.dg; a.dbeta = b.dbeta;
    a.q_stride = p.q_stride; a.k_stride = p.k_stride; a.v_stride = p.v_stride;
    a.Hk = p.Hk; a.Hv = p.Hv; a.V = p.V;
    a.scale = p.scale; a.normalize = p.normalize;
    if (p.bf16)
        return p.K == 64 ? launch_gradients_t<bf16_t, 64>(a, p.slots, stream)
                         : launch_gradients_t<bf16_t, 128>(a, p.slots, stream);
    return p.K == 64 ? launch_gradients_t<float, 64>(a, p.slots, stream)
                     : launch_gradients_t<float, 128>(a, p.slots, stream);
}

hipError_t launch_backward(const BackwardArgs &b, hipStream_t stream) {
    const hipError_t e = launch_backward_chain(b, stream);
    return e != hipSuccess ? e : launch_gradients(b, stream);
}

}  // namespace gdr
