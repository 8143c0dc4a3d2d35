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
// One workgroup of four waves per chunk and key head (for few chunks: value head); it
// forms the products k.k and q.k once and then goes through the value heads that
// share the key head.  Wave w
// has the rows 16w .. of A and the tokens 16 (3 - w) .. of P, so that each has
// five of the lower triangle's tiles.
//
// T by blocks of 16: wave w inverts the diagonal block w (tri_inverse), then owns
// the blocks below it in its block column,
//   T_ij = -T_ii sum_{j <= k < i} A_ik T_kj,
// whose products take T_kj from registers (float32 matrix cores, so T keeps
// float32 accuracy also where keys are alike and A is not small).
//
// What bounds the kernel is the number of vector instructions, most of them for the
// decays.  So outside the diagonal blocks E_ts is a product of two numbers, from s
// to the end of its block of 16 and from there to t (both at most 1), of which
// there are few: a table per value head, with the other factors of t and of s in it
// (32768 tokens, 16 key heads of two value heads, K = 128: 165 us without the tables, 143 us
// with them, 4.3 TB/s of rows and records; 8 x 4096 tokens of 40 heads, K = 64: 200 us).
// Vector units are busy 50 to 60% of the time, the waves wait half of theirs.
// Four workgroups a CU: with the registers for five, 300 us in place of those 200.
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
    int Hk, Hv, heads;  // value heads of a workgroup
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

// Four neighbouring elements of an operand lane (the lower or upper half of its
// eight), rounded to E or split.
template <class E, bool SPLIT>
__device__ __forceinline__ void put_quad(char *frag, int at_lane, int upper, f32x4 v) {
    if constexpr (sizeof(E) == 4) {
        *reinterpret_cast<f32x4 *>(frag + upper * 1024 + at_lane * 16) = v;
    } else {
        char *at = frag + at_lane * 16 + upper * 8;
        const u32x2 hi{cvt_pk(v[0], v[1]), cvt_pk(v[2], v[3])};
        *reinterpret_cast<u32x2 *>(at) = hi;
        if constexpr (SPLIT)
            *reinterpret_cast<u32x2 *>(at + 1024) =
                u32x2{cvt_pk(v[0] - wkv7::bf16_lo(hi[0]), v[1] - wkv7::bf16_hi(hi[0])),
                      cvt_pk(v[2] - wkv7::bf16_lo(hi[1]), v[3] - wkv7::bf16_hi(hi[1]))};
    }
}

// T and A share one array: A's blocks (i, j), i > j, lie in their place, T's diagonal
// blocks on the diagonal, and T_ij, i > j, as it is in the place (j, i).
template <class E, int K>
constexpr int prep_lds() {
    // they take the place of the k and q rows once those products are formed
    constexpr int rows = 2 * tile_bytes<E, K>(kChunk), mats = kChunk * kPitchA * 4;
    return rows > mats ? rows : mats;
}

// of one value head; block x ends at token 16x + 15
struct Decays {
    Sum2 G[kChunk];
    float beta[kChunk];
    float toA[3][kChunk];   // beta_t / |k_t| times the decay from block x's end to t
    float toP[3][kChunk];   // scale / |q_t| times that
    float from[kChunk];     // 1 / |k_s| times the decay from s to its block's end
};

template <class E, int K, bool BWD>
__global__ __launch_bounds__(256, 4) void prep_kernel(PrepArgs p) {
    using Rec = typename std::conditional<BWD, BwdRecord<E>, FwdRecord<E>>::type;
    extern __shared__ __align__(16) char lds[];
    const Tile<E, K> tk{reinterpret_cast<E *>(lds)};
    const Tile<E, K> tq{reinterpret_cast<E *>(lds + tile_bytes<E, K>(kChunk))};
    float *sA = reinterpret_cast<float *>(lds);
    constexpr int kHeads = 2;  // value heads whose tables are made at a time
    __shared__ __align__(16) Decays sD[kHeads];
    __shared__ __align__(16) float sRk[kChunk];
    __shared__ __align__(16) float sRq[kChunk];

    const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, lo = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), pt = 3 - wave;
    const int rep = p.Hv / p.Hk, parts = (rep + p.heads - 1) / p.heads;
    const int slot = (int)(blockIdx.x / (p.Hk * parts)), at = (int)(blockIdx.x % (p.Hk * parts));
    const int hk = at / parts, r0 = at % parts * p.heads;
    const int r1 = r0 + p.heads < rep ? r0 + p.heads : rep;
    Seq sq;
    p.lay.find(slot, kChunk, sq);
    const int first = sq.begin + (slot - sq.slot0) * kChunk;
    if (slot < sq.slot0 || first >= sq.end) return;  // the whole workgroup
    const int live = sq.end - first < kChunk ? sq.end - first : kChunk;

    // two value heads' gates, one for each of the last two waves
    float gate = 0.f, strength = 0.f;
    auto load_gates = [&](int r) {
        const size_t at = ((size_t)first + lane) * p.Hv + hk * rep + r;
        const bool in = r < r1 && lane < live;
        gate = in ? to_float(static_cast<const E *>(p.g)[at]) : 0.f;
        strength = in ? to_float(static_cast<const E *>(p.beta)[at]) : 0.f;
    };
    // a head's table, and the scalars of its record
    auto make_table = [&](int r) {
        Decays &d = sD[(r - r0) % kHeads];
        const Sum2 G = scan_decay(gate);
        const float rk = sRk[lane], rq = p.scale * sRq[lane], from0 = decay(G);
        d.G[lane] = G;
        d.beta[lane] = strength;
        const Sum2 end[4] = {lane_of(G, 15), lane_of(G, 31), lane_of(G, 47), lane_of(G, 63)};
        float c = 0.f;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const float down = decay(end[x], G), on = decay(G, end[x]);
            c = lane / 16 == x ? down : c;
            if (x < 3) {
                d.toA[x][lane] = lane / 16 > x ? strength * rk * on : 0.f;
                d.toP[x][lane] = lane / 16 > x ? rq * on : 0.f;
            }
        }
        d.from[lane] = c * rk;
        Scalars *sc = reinterpret_cast<Scalars *>(
            p.records + ((size_t)slot * p.Hv + hk * rep + r) * Rec::kBytes + Rec::kScalars);
        sc->beta[lane] = strength;
        sc->kS[lane] = -(BWD ? strength : 1.f) * from0 * rk;
        sc->kD[lane] = decay(end[3], G) * rk;
        sc->qS[lane] = from0 * rq;
        if (lane == 63) sc->last = from0;
    };
    if (wave >= 2) load_gates(r0 + wave - 2);
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
    if (p.normalize) {
        const float a = reciprocal_norm(tk, true, live, tid);
        const float b = reciprocal_norm(tq, true, live, tid);
        if ((tid & 3) == 0) {
            sRk[tid >> 2] = a;
            sRq[tid >> 2] = b;
        }
    } else if (tid < kChunk) {
        sRk[tid] = sRq[tid] = tid < live ? 1.f : 0.f;
    }
    // kk: k.k, rows 16 wave + 4g + e, columns 16 j + lo, j <= wave.  qk: q.k with the
    // tokens 16 pt + lo as columns and s = 16 j + 4g + e as rows, j <= pt, or (backward)
    // with s = 16 pt + lo as columns and t = 16 j + 4g + e as rows, j >= pt.
    f32x4 kk[4], qk[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) kk[j] = qk[j] = f32x4{0.f, 0.f, 0.f, 0.f};
    const int pc = BWD ? wave : pt;  // the block of those columns: five tiles with kk's again
    {
        const Tile<E, K> ta = BWD ? tq : tk, tb = BWD ? tk : tq;
#pragma unroll
        for (int ks = 0; ks < K / 32; ++ks) {
            const Frag<E> a = tk.rows(16 * wave + lo, 32 * ks, g),
                          b = tb.rows(16 * pc + lo, 32 * ks, g);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (j <= wave) kk[j] = mma(a, tk.rows(16 * j + lo, 32 * ks, g), kk[j]);
                if (BWD ? j >= pc : j <= pc)
                    qk[j] = mma(ta.rows(16 * j + lo, 32 * ks, g), b, qk[j]);
            }
        }
    }
    __syncthreads();  // the norms; the rows have been read

    for (int r = r0; r < r1; ++r) {
        const int hv = hk * rep + r;
        char *rec = p.records + ((size_t)slot * p.Hv + hv) * Rec::kBytes;
        if (r > r0) __syncthreads();  // the last head's reads of sA and of its table
        if ((r - r0) % kHeads == 0) {
            if (wave >= 2 && r + wave - 2 < r1) {
                if (r > r0) load_gates(r + wave - 2);
                make_table(r + wave - 2);
            }
            __syncthreads();
        }
        const Decays &d = sD[(r - r0) % kHeads];
        f32x4 x, xt;
        {
            const int row0 = 16 * wave + 4 * g;
            f32x4 nd, ndt;
            const Sum2 Gc = d.G[16 * wave + lo];
            const float rc = sRk[16 * wave + lo], bc = d.beta[16 * wave + lo];
            const f32x4 rr = *reinterpret_cast<const f32x4 *>(sRk + row0),
                        br = *reinterpret_cast<const f32x4 *>(d.beta + row0);
            f32x4 diag = kk[0];
#pragma unroll
            for (int j = 1; j < 4; ++j) diag = j == wave ? kk[j] : diag;
#pragma unroll
            for (int e = 0; e < 4; ++e) {  // the diagonal block, and its transpose
                const Sum2 Gr = d.G[row0 + e];
                const int row = 4 * g + e;
                const float y =
                    diag[e] * rr[e] * rc * (row > lo ? decay(Gr, Gc) : decay(Gc, Gr));
                nd[e] = row > lo ? br[e] * y : 0.f;
                ndt[e] = row < lo ? bc * y : 0.f;
            }
#pragma unroll
            for (int j = 0; j < 3; ++j) {
                if (j >= wave) break;
                const f32x4 to = *reinterpret_cast<const f32x4 *>(d.toA[j] + row0);
                const float from = d.from[16 * j + lo];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    sA[(row0 + e) * kPitchA + 16 * j + lo] = kk[j][e] * from * to[e];
            }
            wkv7::tri_inverse(nd, ndt, lane, x, xt);
#pragma unroll
            for (int e = 0; e < 4; ++e) sA[(row0 + e) * kPitchA + 16 * wave + lo] = x[e];
        }
        {  // P: a lane's column, its four neighbouring rows of each tile
            const int col = 16 * pc + lo;
            const Sum2 Gc = d.G[col];
            const float factor = BWD ? sRk[col] : p.scale * sRq[col];
            const float from_col = d.from[col];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                // (a block behind the diagonal that shares a fragment with one before it is
                // written as zeros)
                if (BWD ? j < (pc & ~1) : j > (pc | 1)) continue;
                const int row0 = 16 * j + 4 * g;
                f32x4 v{0.f, 0.f, 0.f, 0.f};
                if (j == pc) {
                    const f32x4 rr = *reinterpret_cast<const f32x4 *>((BWD ? sRq : sRk) + row0) *
                                     (BWD ? p.scale : 1.f) * factor;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const Sum2 Gr = d.G[row0 + e];
                        const bool in = BWD ? lo <= 4 * g + e : 4 * g + e <= lo;  // s <= t
                        const float f = rr[e] * (BWD ? decay(Gr, Gc) : decay(Gc, Gr));
                        v[e] = in ? f * qk[j][e] : 0.f;
                    }
                } else if (BWD ? j > pc : j < pc) {
                    if constexpr (BWD) {  // from column s to rows t
                        const float *to = d.toP[0] + pc * kChunk;
                        v = qk[j] * (from_col * *reinterpret_cast<const f32x4 *>(to + row0));
                    } else {
                        v = qk[j] * (d.toP[j][col] *
                                     *reinterpret_cast<const f32x4 *>(d.from + row0));
                    }
                }
                // in operand order: fragment (tile of the columns, 32 rows), lane of the
                // column and of eight rows
                const int c32 = col & 31;
                const int tile = 2 * (col >> 5) + (c32 >> 2 & 1), step = row0 >> 5;
                const int f = BWD ? (tile < 2 ? 2 * tile + step : tile + 2)
                                  : (tile < 2 ? tile : 2 * tile - 2 + step);
                const int at_lane = 16 * (row0 >> 3 & 3) + 4 * (c32 >> 3) + (c32 & 3);
                put_quad<E, BWD>(rec + Rec::kP + f * (BWD ? Rec::kSplitBytes : FwdRecord<E>::kFragBytes),
                                 at_lane, g & 1, v);
            }
        }
        __syncthreads();
        {  // block column `wave` of T below the diagonal
            f32x4 col[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) col[i] = f32x4{0.f, 0.f, 0.f, 0.f};
            col[0] = x;
#pragma unroll
            for (int n = 1; n < 4; ++n) {
                const int i = wave + n;
                if (i >= 4) break;
                f32x4 acc{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int k = 0; k < n; ++k)
                    acc = mul_block(sA, 16 * i, 16 * (wave + k), col[k], acc, g, lo);
                f32x4 t{0.f, 0.f, 0.f, 0.f};
                t = mul_block(sA, 16 * i, 16 * i, acc, t, g, lo);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    col[n][e] = -t[e];
                    sA[(16 * wave + 4 * g + e) * kPitchA + 16 * i + lo] = -t[e];
                }
            }
        }
        __syncthreads();
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            const int f = wave + 4 * n;
            if (f >= 6) break;
            f32x4 v[2];
            if constexpr (BWD) {  // T^T: row s, columns t
                const int s = tile_row(kUpTile[f], lo), t0 = 32 * kUpStep[f] + 8 * g;
                const float *src = sA + (s & ~15) * kPitchA + (t0 & ~15) + (s & 15);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j >> 2][j & 3] = src[((t0 & 15) + j) * kPitchA];
                if (t0 / 16 < s / 16) v[0] = v[1] = f32x4{0.f, 0.f, 0.f, 0.f};
            } else {
                const int t = tile_row(kLowTile[f], lo), s0 = 32 * kLowStep[f] + 8 * g;
                const float *src = sA + ((s0 & ~15) + (t & 15)) * kPitchA + (t & ~15) + (s0 & 15);
                v[0] = *reinterpret_cast<const f32x4 *>(src) *
                       *reinterpret_cast<const f32x4 *>(d.beta + s0);
                v[1] = *reinterpret_cast<const f32x4 *>(src + 4) *
                       *reinterpret_cast<const f32x4 *>(d.beta + s0 + 4);
                if (s0 / 16 > t / 16) v[0] = v[1] = f32x4{0.f, 0.f, 0.f, 0.f};
            }
            put_split<E>(rec + f * Rec::kSplitBytes, to_split<E>(v[0], v[1]), lane);
        }
    }
}

template <class E, int K, bool BWD>
hipError_t launch_prep_t(const PrepArgs &a, int slots, hipStream_t stream) {
    constexpr int kLds = prep_lds<E, K>();
    const auto fn = prep_kernel<E, K, BWD>;
    const hipError_t e = allow_lds(reinterpret_cast<const void *>(fn), kLds);
    if (e != hipSuccess) return e;
    const int rep = a.Hv / a.Hk;
    const size_t blocks = (size_t)slots * a.Hk * ((rep + a.heads - 1) / a.heads);
    hipLaunchKernelGGL(fn, dim3((unsigned)blocks), dim3(256), kLds, stream, a);
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
    // all value heads of a key head in one workgroup, unless the CUs are not full then:
    // three sequences of up to 63 tokens, two key heads of two: 7.8 us against 10.0 us
    a.heads = (size_t)p.slots * p.Hk <= kCus ? 1 : p.Hv / p.Hk;
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
