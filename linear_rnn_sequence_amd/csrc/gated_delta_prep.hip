// Gated delta rule: the part of a chunk that does not depend on the state.
//
// For each chunk of 64 tokens and value head, with G the inclusive sums of the
// log decays and E_ts = exp(G_t - G_s):
//   A_ts = beta_t E_ts (k_t . k_s)  (s < t),   T = (I + A)^-1,
//   P_ts = scale E_ts (q_t . k_s)   (s <= t),
// with q and k divided by their norms where that is asked for (the norms enter
// as factors of the products, so the matrix cores see q and k as given).  The
// chain kernels need T and P (forward) or T^T and P^T (backward) as matrix-core
// operands, so they are written in that order, with the chunk's scalars.
//
// One workgroup of four waves per chunk and key head; it forms the products
// k.k and q.k once and then goes through the value heads that share the key
// head.  T by blocks of 16: wave w inverts the diagonal block w (tri_inverse),
// then owns the blocks below it in its block column,
//   T_ij = -T_ii sum_{j <= k < i} A_ik T_kj,
// whose products take T_kj from registers (float32 matrix cores, so T keeps
// float32 accuracy also where keys are alike and A is not small).
#include "gated_delta_device.h"
#include "gated_delta_internal.h"

namespace gdr {
namespace {

constexpr int kPitchA = kChunk + 4;  // floats per row of A and T in shared memory

struct PrepArgs {
    Layout lay;
    const void *q, *k, *g, *beta;
    char *records;
    int q_stride, k_stride;
    int Hk, Hv;
    float scale;
    bool normalize;
};

// D(A B) += for A from shared memory rows (16 x 16 at row0, col0) and B = a result tile
__device__ __forceinline__ f32x4 mul_block(const float *m, int row0, int col0, f32x4 b, f32x4 c,
                                           int g, int lo) {
    const f32x4 a = *reinterpret_cast<const f32x4 *>(m + (row0 + lo) * kPitchA + col0 + 4 * g);
#pragma unroll
    for (int e = 0; e < 4; ++e)
        c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[e], b[e], c, 0, 0, 0);
    return c;
}

template <class E, int K>
constexpr int prep_lds() {
    // A and T take the place of the k and q rows once their products are formed
    constexpr int rows = 2 * tile_bytes<E, K>(kChunk), mats = 2 * kChunk * kPitchA * 4;
    return rows > mats ? rows : mats;
}

template <class E, int K, bool BWD>
__global__ __launch_bounds__(256, 4) void prep_kernel(PrepArgs p) {
    using Rec = typename std::conditional<BWD, BwdRecord<E>, FwdRecord<E>>::type;
    extern __shared__ __align__(16) char lds[];
    Tile<E, K> tk{reinterpret_cast<E *>(lds)};
    Tile<E, K> tq{reinterpret_cast<E *>(lds + tile_bytes<E, K>(kChunk))};
    float *sA = reinterpret_cast<float *>(lds);
    float *sT = sA + kChunk * kPitchA;
    constexpr int kHeads = 4;  // value heads whose decays are summed at a time
    __shared__ Sum2 sG4[kHeads][kChunk];
    __shared__ __align__(16) float sBeta4[kHeads][kChunk];
    __shared__ float sRk[kChunk], sRq[kChunk];

    const int tid = threadIdx.x, lane = tid & 63,
              wave = __builtin_amdgcn_readfirstlane(tid >> 6), g = lane >> 4, lo = lane & 15;
    const int slot = (int)(blockIdx.x / p.Hk), hk = (int)(blockIdx.x % p.Hk);
    Seq sq;
    p.lay.find(slot, kChunk, sq);
    const int first = sq.begin + (slot - sq.slot0) * kChunk;
    if (slot < sq.slot0 || first >= sq.end) return;  // the whole workgroup
    const int live = sq.end - first < kChunk ? sq.end - first : kChunk;
    const int rep = p.Hv / p.Hk;

    // the first four value heads' gates, wave by wave
    float gate = 0.f, strength = 0.f;
    auto load_gates = [&](int r) {
        const size_t at = ((size_t)first + lane) * p.Hv + hk * rep + r;
        const bool in = r < rep && lane < live;
        gate = in ? to_float(static_cast<const E *>(p.g)[at]) : 0.f;
        strength = in ? to_float(static_cast<const E *>(p.beta)[at]) : 0.f;
    };
    load_gates(wave);
    {
        Stage<E, K, kChunk, 256> sk, sqv;
        sk.load(static_cast<const E *>(p.k) + (long long)first * p.k_stride + hk * K, p.k_stride,
                live, tid);
        sqv.load(static_cast<const E *>(p.q) + (long long)first * p.q_stride + hk * K, p.q_stride,
                 live, tid);
        sk.store(tk, tid);
        sqv.store(tq, tid);
    }
    __syncthreads();
    {
        const float a = reciprocal_norm(tk, p.normalize, live, tid);
        const float b = reciprocal_norm(tq, p.normalize, live, tid);
        if ((tid & 3) == 0) {
            sRk[tid >> 2] = a;
            sRq[tid >> 2] = b;
        }
    }
    // k.k: rows 16 wave + 4g + e, columns 16 j + lo, j <= wave (natural order)
    f32x4 kk[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) kk[j] = f32x4{0.f, 0.f, 0.f, 0.f};
    // P: this wave forms the fragments f = wave, wave + 4 of the six.  The fragment's
    // two result tiles are those of P^T (forward: rows s, columns t) or P
    // (backward: rows t, columns s), rows in tile_row order.
    f32x4 qk[2][2];
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int h = 0; h < 2; ++h) qk[n][h] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int ks = 0; ks < K / 32; ++ks) {
        const Frag<E> a = tk.rows(16 * wave + lo, 32 * ks, g);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (j <= wave) kk[j] = mma(a, tk.rows(16 * j + lo, 32 * ks, g), kk[j]);
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            const int f = wave + 4 * n;
            if (f >= 6) break;
            const int tile = BWD ? kUpTile[f] : kLowTile[f], step = BWD ? kUpStep[f] : kLowStep[f];
            const Tile<E, K> ta = BWD ? tq : tk, tb = BWD ? tk : tq;
            const Frag<E> b = tb.rows(tile_row(tile, lo), 32 * ks, g);
#pragma unroll
            for (int h = 0; h < 2; ++h)
                qk[n][h] = mma(ta.rows(tile_row(2 * step + h, lo), 32 * ks, g), b, qk[n][h]);
        }
    }
    __syncthreads();
    // blocks (0, 1) and (2, 3) of T: read as zeros, never written
    if (tid < 128) {
        const int row = 32 * (tid >> 6) + (tid & 15), col = row / 32 * 32 + 16 + 4 * (tid >> 4 & 3);
        *reinterpret_cast<f32x4 *>(sT + row * kPitchA + col) = f32x4{0.f, 0.f, 0.f, 0.f};
    }

    for (int r = 0; r < rep; ++r) {
        const int hv = hk * rep + r;
        char *rec = p.records + ((size_t)slot * p.Hv + hv) * Rec::kBytes;
        if (r % kHeads == 0) {
            if (r) __syncthreads();  // the last heads' reads of sG4, sBeta4
            if (r) load_gates(r + wave);
            if (r + wave < rep) {
                const Sum2 G = scan_decay(gate);
                sG4[wave][lane] = G;
                sBeta4[wave][lane] = strength;
                Scalars *sc = reinterpret_cast<Scalars *>(rec + wave * Rec::kBytes + Rec::kScalars);
                const float from0 = decay(G);
                sc->beta[lane] = strength;
                sc->kS[lane] = -(BWD ? strength : 1.f) * from0 * sRk[lane];
                sc->kD[lane] = decay(last_lane(G), G) * sRk[lane];
                sc->qS[lane] = p.scale * from0 * sRq[lane];
                if (lane == 63) sc->last = from0;
            }
        }
        __syncthreads();  // the above; the last head's reads of sA, sT
        const Sum2 *sG = sG4[r % kHeads];
        const float *sBeta = sBeta4[r % kHeads];
        f32x4 nd{0.f, 0.f, 0.f, 0.f}, ndt{0.f, 0.f, 0.f, 0.f};
        {
            Sum2 Gr[4];
            float rr[4], br[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int row = 16 * wave + 4 * g + e;
                Gr[e] = sG[row];
                rr[e] = sRk[row];
                br[e] = sBeta[row];
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (j > wave) break;
                const int col = 16 * j + lo;
                const Sum2 Gc = sG[col];
                const float rc = sRk[col], bc = sBeta[col];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int row = 16 * wave + 4 * g + e;
                    const float x = kk[j][e] * rr[e] * rc;
                    if (j < wave) {
                        sA[row * kPitchA + col] = br[e] * decay(Gr[e], Gc) * x;
                    } else {  // the diagonal block and its transpose stay in registers
                        const float d = row > col ? decay(Gr[e], Gc) : decay(Gc, Gr[e]);
                        nd[e] = row > col ? br[e] * d * x : 0.f;
                        ndt[e] = row < col ? bc * d * x : 0.f;
                    }
                }
            }
        }
        f32x4 x, xt;
        wkv7::tri_inverse(nd, ndt, lane, x, xt);
#pragma unroll
        for (int e = 0; e < 4; ++e) sT[(16 * wave + 4 * g + e) * kPitchA + 16 * wave + lo] = x[e];
        __syncthreads();
        {  // block column `wave` of T below the diagonal
            f32x4 col[4];
#pragma unroll
            for (int d = 0; d < 4; ++d) col[d] = f32x4{0.f, 0.f, 0.f, 0.f};
            col[0] = x;
#pragma unroll
            for (int d = 1; d < 4; ++d) {
                const int i = wave + d;
                if (i >= 4) break;
                f32x4 acc{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int k = 0; k < d; ++k)
                    acc = mul_block(sA, 16 * i, 16 * (wave + k), col[k], acc, g, lo);
                f32x4 t{0.f, 0.f, 0.f, 0.f};
                t = mul_block(sT, 16 * i, 16 * i, acc, t, g, lo);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    col[d][e] = -t[e];
                    sT[(16 * i + 4 * g + e) * kPitchA + 16 * wave + lo] = -t[e];
                }
            }
        }
        // P needs nothing of T: formed while other waves finish their columns.  The
        // waves with the fewest blocks above take two fragments each.
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            const int f = wave + 4 * n;
            if (f >= 6) break;
            const int tile = BWD ? kUpTile[f] : kLowTile[f], step = BWD ? kUpStep[f] : kLowStep[f];
            const int col = tile_row(tile, lo);
            const Sum2 Gc = sG[col];
            const float rc = p.scale * (BWD ? sRk[col] : sRq[col]);
            f32x4 v[2];
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int row = tile_row(2 * step + h, 4 * g + e);
                    const bool in = BWD ? col <= row : row <= col;  // s <= t
                    const Sum2 Gr = sG[row];
                    const float w = rc * (BWD ? sRq[row] : sRk[row]) *
                                    (BWD ? decay(Gr, Gc) : decay(Gc, Gr));
                    v[h][e] = in ? w * qk[n][h][e] : 0.f;
                }
            if constexpr (BWD)
                put_split<E>(rec + Rec::kP + f * Rec::kSplitBytes, to_split<E>(v[0], v[1]), lane);
            else
                put_frag<E>(rec + Rec::kP + f * FwdRecord<E>::kFragBytes, to_frag<E>(v[0], v[1]),
                            lane);
        }
        __syncthreads();
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            const int f = wave + 4 * n;
            if (f >= 6) break;
            f32x4 v[2];
            if constexpr (BWD) {  // T^T: row s, columns t
                const int s = tile_row(kUpTile[f], lo), t0 = 32 * kUpStep[f] + 8 * g;
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j >> 2][j & 3] = sT[(t0 + j) * kPitchA + s];
            } else {
                const int s0 = 32 * kLowStep[f] + 8 * g;
                const float *src = sT + tile_row(kLowTile[f], lo) * kPitchA + s0;
                v[0] = *reinterpret_cast<const f32x4 *>(src) *
                       *reinterpret_cast<const f32x4 *>(sBeta + s0);
                v[1] = *reinterpret_cast<const f32x4 *>(src + 4) *
                       *reinterpret_cast<const f32x4 *>(sBeta + s0 + 4);
            }
            put_split<E>(rec + f * Rec::kSplitBytes, to_split<E>(v[0], v[1]), lane);
        }
    }
}

template <class E, int K, bool BWD>
hipError_t launch_prep_t(const PrepArgs &a, int slots, hipStream_t stream) {
    constexpr int kLds = prep_lds<E, K>();
    const auto fn = prep_kernel<E, K, BWD>;
    const hipError_t e = hipFuncSetAttribute(
        reinterpret_cast<const void *>(fn), hipFuncAttributeMaxDynamicSharedMemorySize, kLds);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(fn, dim3((unsigned)((size_t)slots * a.Hk)), dim3(256), kLds, stream, a);
    return hipGetLastError();
}

}  // namespace

size_t forward_record_bytes(bool bf16) {
    return bf16 ? FwdRecord<bf16_t>::kBytes : FwdRecord<float>::kBytes;
}
size_t backward_record_bytes(bool bf16) {
    return bf16 ? BwdRecord<bf16_t>::kBytes : BwdRecord<float>::kBytes;
}

hipError_t launch_prep(const Problem &p, const void *q, const void *k, const void *g,
                       const void *beta, char *records, bool backward, hipStream_t stream) {
    PrepArgs a{};
    a.lay = Layout{p.cu, p.n_seq, p.T, p.total};
    a.q = q; a.k = k; a.g = g; a.beta = beta;
    a.records = records;
    a.q_stride = p.q_stride; a.k_stride = p.k_stride;
    a.Hk = p.Hk; a.Hv = p.Hv;
    a.scale = p.scale; a.normalize = p.normalize;
    const int s = p.slots;
    if (s == 0) return hipSuccess;
    if (p.bf16) {
        if (p.K == 64)
            return backward ? launch_prep_t<bf16_t, 64, true>(a, s, stream)
                            : launch_prep_t<bf16_t, 64, false>(a, s, stream);
        return backward ? launch_prep_t<bf16_t, 128, true>(a, s, stream)
                        : launch_prep_t<bf16_t, 128, false>(a, s, stream);
    }
    if (p.K == 64)
        return backward ? launch_prep_t<float, 64, true>(a, s, stream)
                        : launch_prep_t<float, 64, false>(a, s, stream);
    return backward ? launch_prep_t<float, 128, true>(a, s, stream)
                    : launch_prep_t<float, 128, false>(a, s, stream);
}

}  // namespace gdr
