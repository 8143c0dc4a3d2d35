// Linear attention with a decay for each head: the pass over a sequence's chunks that
// carries a state, which is the forward and all of the backward.
//
// With a = exp(g) and, in a chunk of C tokens, r = 0 .. C - 1, a pass over rows x, y, z
// (x and y of KD channels, z of VD) with a state S [VD, KD] computes
//   out_r = read a^(r + s) S x_r + intra sum_{j <= r} a^(r - j) (x_r . y_j) z_j
//   S    <- a^C S + write sum_j a^(C - s - j) z_j y_j^T
// The forward is that of (q, k, v) with s = 1, read = intra = scale, write = 1.  The
// gradients are three passes of the same kind:
//   dq: (dO, v, k), s = 1, the state S^T;           read = intra = scale, write = 1
//   dk: (v, dO, q), s = 0, last token first, D^T;   read = 1, intra = write = scale
//   dv: (k, q, dO), s = 0, last token first, D;     likewise
// (D, the cotangent of the state behind a token, is not decayed for that token's gradients,
// as S, the state before it, is for its readout.)  So the backward needs nothing that the
// forward computed: S is carried again, which costs its reads of k and v, where stored
// states would be V K numbers for every 64 (K + V) of those.
//
// dg = sum over all pairs of a token written and a token read of their distance times the
// pair's term.  Within a chunk that is sum (r - j) (x_r . y_j) (z_j . q_r) a^(r - j); across
// chunks the dq pass carries R = dS / dg beside S,
//   R <- a^C (R + C S) + sum_j (C - 1 - j) a^(C - 1 - j) z_j y_j^T,
// reads it out as it does S, and at the end takes its product with the cotangent.  (The usual
// sum of position times q dq - k dk cancels to nothing for long sequences.)
//
// Layout: a wave owns 16 rows of the state over all KD columns, as matrix-core result
// tiles [columns, rows]: S x^T and the products with z^T need nothing of another wave.  The
// chunk's rows of x, y and z lie in shared memory; x y^T, six fragments of the lower
// triangle, is computed by the waves together and passed through it.
#include "gated_delta_device.h"
#include "linear_attention_internal.h"

namespace lattn {
namespace {

using namespace gdr;

enum Mode {
    kOut,   // out and the state
    kGrad,  // the same and dg: the dq pass
    kSum    // the state alone: what a segment adds
};

struct Pass {
    const void *x, *y, *z;
    int x_stride, y_stride, z_stride;  // elements from token to token
    int x_rep, y_rep, z_rep;           // heads that read the same rows
    void *out;                         // [total, heads, VD]
    float read, intra, write;
    int shift;                         // s above; 0: last token first
    bool turned;                       // the states in memory are [KD, VD]
    const float *s_in;                 // whole sequences: the start, or nullptr
    float *s_out;                      // the end, or nullptr
    const int *slots_in, *slots_out;
    int pool;
    float *unit_states;                // segments: their starts (kSum: what they add)
    // kGrad
    const void *e;                     // rows of q
    int e_stride, e_rep;
    const float *cotangent;            // of the sequences' (segments': of the segments') ends, or nullptr
    double *dg;                        // [units, heads]
};

struct PassArgs {
    Layout lay;
    int seg, heads, parts;
    const float *g;
    Pass pass[3];  // by blockIdx.y
};

__device__ __forceinline__ f32x4 zero() { return f32x4{0.f, 0.f, 0.f, 0.f}; }

// A float operand in N bf16 parts, each the rounded rest: 8 bits of significand per part, so
// that three hold a float.
template <class E, int N>
struct Parts {
    Frag<E> p[sizeof(E) == 2 ? N : 1];
    static constexpr int kN = sizeof(E) == 2 ? N : 1;
    __device__ __forceinline__ Parts(f32x4 a, f32x4 b) {
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            p[i] = to_frag<E>(a, b);
            if (i + 1 < kN)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    a[e] -= p[i].at(e);
                    b[e] -= p[i].at(4 + e);
                }
        }
    }
};

// Rows of a chunk on their way from memory to a tile in shared memory; in a reversed pass row
// r is the live - 1 - r-th in memory.  Rows behind `live` are zeros.
template <class E, int C, int THREADS>
struct Rows {
    static constexpr int kRowPieces = Tile<E, C>::kRowPieces, kPiece = Tile<E, C>::kPiece;
    static constexpr int kPer = kChunk * kRowPieces / THREADS;
    static_assert(kChunk * kRowPieces % THREADS == 0, "whole pieces per thread");
    u32x4 d[kPer];
    static __device__ __forceinline__ unsigned offset(int row, int col, int stride, int live,
                                                      bool reverse) {
        // (modulo 2^32: a row before the first one lies behind the buffer's end)
        const unsigned at = reverse ? (unsigned)(live - 1 - row) : (unsigned)row;
        return (at * (unsigned)stride + (unsigned)col) * (unsigned)sizeof(E);
    }
    __device__ __forceinline__ void load(const E *src, int stride, int live, bool reverse, int tid) {
        const Buffer b(src, row_bytes<E>(live, stride));
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int piece = tid + i * THREADS;
            d[i] = b.load16(offset(piece / kRowPieces, piece % kRowPieces * kPiece, stride, live,
                                   reverse));
        }
    }
    __device__ __forceinline__ void put(Tile<E, C> t, int tid) const {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int piece = tid + i * THREADS;
            *reinterpret_cast<u32x4 *>(
                t.p + t.offset(piece / kRowPieces, piece % kRowPieces * kPiece)) = d[i];
        }
    }
    // the way back, from the pieces that put() will write next
    static __device__ __forceinline__ void store(Tile<E, C> t, E *dst, int stride, int live,
                                                 bool reverse, int tid) {
        const Buffer b(dst, row_bytes<E>(live, stride));
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int piece = tid + i * THREADS;
            const int row = piece / kRowPieces, col = piece % kRowPieces * kPiece;
            b.store16(offset(row, col, stride, live, reverse),
                      *reinterpret_cast<const u32x4 *>(t.p + t.offset(row, col)));
        }
    }
};

// The head's log decay to the base 2 (below -200 it is 0 in float32, -infinity with it; a NaN
// stays one) and its powers.  The exponent keeps more than a float's bits: what is off by 2^-24
// of a chunk's exponent would be off by 512 of these after 512 chunks.
struct Decay {
    double g2;
    __device__ __forceinline__ explicit Decay(float g)
        : g2((g < kLowestLogDecay ? kLowestLogDecay : g) * 1.4426950408889634) {}
    __device__ __forceinline__ float power(int n) const {
        const double x = g2 * n;
        const float hi = (float)x;
        return exp2f(hi) * (1.f + 0.6931472f * (float)(x - hi));
    }
    // as the sum of two floats: a chunk's, which is applied once per chunk
    __device__ __forceinline__ Sum2 exact(int n) const {
        const double x = exp2(g2 * n);
        const float hi = (float)x;
        return Sum2{hi, (float)(x - hi)};
    }
};

template <class E, int KD, int VD, Mode MODE>
struct Shared {
    static constexpr int kTileK = tile_bytes<E, KD>(kChunk), kTileV = tile_bytes<E, VD>(kChunk);
    static constexpr int kFrag = 2048;  // bf16: two parts, float: two halves
    static constexpr int kY = 0, kZ = kTileK, kX = kZ + kTileV;
    static constexpr int kP = kX + (MODE == kSum ? 0 : kTileK);
    static constexpr int kE = kP + (MODE == kSum ? 0 : 6 * kFrag);
    static constexpr int kPowers = kE + (MODE == kGrad ? kTileV : 0);
    static constexpr int kBytes = kPowers + 68 * 4;
    // the next chunk's rows are on their way while this one is computed (in float they
    // would take the registers that its products need)
    static constexpr bool kAhead = sizeof(E) == 2 && !(MODE == kGrad && KD > VD);
    // kernels that would need more registers than there are
    static constexpr bool kTight = sizeof(E) == 4 || MODE == kGrad;
    // tiles of columns that the state's products have in registers at a time
    static constexpr int kGroup = sizeof(E) == 4 && MODE == kGrad ? 1 : kTight ? 2 : 4;
};

template <class E, class O, int KD, int VD, Mode MODE>
__global__ __launch_bounds__(VD * 4, sizeof(E) == 2 ? 2 : 1) void pass_kernel(PassArgs a) {
    using L = Shared<E, KD, VD, MODE>;
    constexpr int W = VD / 16, kThreads = 64 * W, KS = KD / 32, M = KD / 16;
    constexpr int kTiles = 12 / W + (12 % W ? 1 : 0);  // of x y^T per wave
    extern __shared__ __align__(16) char lds[];
    const Pass &p = a.pass[blockIdx.y];
    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    int lane = tid & 63, g = lane >> 4, lo = lane & 15;
    const int unit = (int)(blockIdx.x / a.heads), h = (int)(blockIdx.x % a.heads);
    const bool reverse = p.shift == 0;

    // the sequence, or the segment of it
    Seq sq;
    int seq = unit, first = 0;
    if (a.seg) {
        seq = a.lay.find(unit, a.seg, sq);
        const long long ahead = (long long)(unit - sq.slot0) * a.seg;
        if (unit < sq.slot0 || (ahead >= sq.end - sq.begin && ahead > 0)) {
            if (MODE == kGrad && tid == 0) p.dg[(size_t)unit * a.heads + h] = 0.0;
            return;
        }
        first = (int)ahead;
    } else {
        sq = a.lay.seq(unit, kChunk);
    }
    const int rest = sq.end - sq.begin - first, len = a.seg && rest > a.seg ? a.seg : rest;
    const bool ends = reverse ? first == 0 : len == rest;
    if (MODE == kSum && ends) return;  // nothing follows it
    const long long token = (long long)sq.begin + first;
    const int chunks = (len + kChunk - 1) / kChunk;
    const size_t state_size = (size_t)VD * KD;

    const Decay decay(a.g[h / a.parts]);
    float *pw = reinterpret_cast<float *>(lds + L::kPowers);
    if (tid <= kChunk) pw[tid] = decay.power(tid);

    // the wave's rows of a state in memory: row own0 + lo, columns tile_row(m, 4g) ..
    const int own0 = 16 * wave;
    auto load_state = [&](f32x4(&S)[M], const float *base) {
#pragma unroll
        for (int m = 0; m < M; ++m) {
            const int row = own0 + lo, col = tile_row(m, 4 * g);
            if (p.turned)
#pragma unroll
                for (int e = 0; e < 4; ++e) S[m][e] = base[(col + e) * VD + row];
            else
                S[m] = *reinterpret_cast<const f32x4 *>(base + row * KD + col);
        }
    };
    f32x4 S[M], R[MODE == kGrad ? M : 1];
    const float *from = nullptr;
    if (MODE != kSum && a.seg) {
        from = p.unit_states + ((size_t)unit * a.heads + h) * state_size;
    } else if (MODE != kSum && p.s_in) {
        const int slot = p.slots_in ? p.slots_in[seq] : seq;
        if (slot >= 0 && slot < p.pool) from = p.s_in + ((size_t)slot * a.heads + h) * state_size;
    }
    if (from) {
        load_state(S, from);
    } else {
#pragma unroll
        for (int m = 0; m < M; ++m) S[m] = zero();
    }
    if constexpr (MODE == kGrad)
#pragma unroll
        for (int m = 0; m < M; ++m) R[m] = zero();

    const E *xp = static_cast<const E *>(p.x) + token * p.x_stride + h / p.x_rep * KD;
    const E *yp = static_cast<const E *>(p.y) + token * p.y_stride + h / p.y_rep * KD;
    const E *zp = static_cast<const E *>(p.z) + token * p.z_stride + h / p.z_rep * VD;
    const E *ep = MODE == kGrad ? static_cast<const E *>(p.e) + token * p.e_stride + h / p.e_rep * VD
                                : nullptr;
    const int row = a.heads * VD;
    O *op = static_cast<O *>(p.out) + token * row + h * VD;

    const Tile<E, KD> tx{reinterpret_cast<E *>(lds + L::kX)}, ty{reinterpret_cast<E *>(lds + L::kY)};
    const Tile<E, VD> tz{reinterpret_cast<E *>(lds + L::kZ)}, te{reinterpret_cast<E *>(lds + L::kE)};
    char *frags = lds + L::kP;

    auto live_of = [&](int c) {
        const int left = len - c * kChunk;
        return left < kChunk ? left : kChunk;  // none or fewer: nothing is in range
    };
    // the chunk's first token in memory, from the unit's
    auto start_of = [&](int c) {
        const int low = reverse ? len - (c + 1) * kChunk : c * kChunk;
        return (long long)(low > 0 ? low : 0);
    };
    Rows<E, KD, kThreads> gx, gy;
    Rows<E, VD, kThreads> gz, ge;
    auto fetch = [&](int c) {
        const int live = live_of(c);
        const long long at = start_of(c);
        if (MODE != kSum) gx.load(xp + at * p.x_stride, p.x_stride, live, reverse, tid);
        gy.load(yp + at * p.y_stride, p.y_stride, live, reverse, tid);
        gz.load(zp + at * p.z_stride, p.z_stride, live, reverse, tid);
        if constexpr (MODE == kGrad) ge.load(ep + at * p.e_stride, p.e_stride, live, reverse, tid);
    };
    auto put = [&]() {
        if (MODE != kSum) gx.put(tx, tid);
        gy.put(ty, tid);
        gz.put(tz, tid);
        if constexpr (MODE == kGrad) ge.put(te, tid);
    };
    if (chunks > 0) {
        fetch(0);
        put();
    }
    __syncthreads();

    // powers that every whole chunk uses: of the readout of token tile_row(i, lo), of the wave's
    // tiles of x y^T, and of the tokens 32 st + 8 g + j in the state
    float rd[4], pair[kTiles][4], kd[2][8];
#pragma unroll
    for (int i = 0; i < 4; ++i) rd[i] = p.read * pw[tile_row(i, lo) + p.shift];
#pragma unroll
    for (int x = 0; x < kTiles; ++x) {
        const int t = wave + x * W, f = t < 12 ? t >> 1 : 0, i = tile_row(kLowTile[f], lo);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int j = tile_row(2 * kLowStep[f] + (t & 1), 4 * g + e);
            pair[x][e] = j <= i ? p.intra * pw[i - j] : 0.f;
        }
    }
    auto weights = [&](int live) {
#pragma unroll
        for (int st = 0; st < 2; ++st)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int n = live - p.shift - (32 * st + 8 * g + j);
                kd[st][j] = n < 0 ? 0.f : p.write * pw[n];
            }
    };
    weights(kChunk);
    Sum2 whole = decay.exact(kChunk);
    double dg = 0.0;

    for (int c = 0; c < chunks; ++c) {
        const int live = live_of(c);
        if (L::kAhead) fetch(c + 1);
        if constexpr (L::kTight) {  // addresses in shared memory are formed again in every chunk
            asm volatile("" : "+v"(lane));
            g = lane >> 4;
            lo = lane & 15;
        }
        if (live < kChunk) {
            weights(live);
            whole = decay.exact(live);
        }
        f32x4 out[4];
        float dg_chunk = 0.f;
        if constexpr (MODE != kSum) {
            // x y^T, masked and decayed
#pragma unroll
            for (int x = 0; x < kTiles; ++x) {
                const int t = wave + x * W;
                if (t < 12) {
                    const int f = t >> 1, jt = 2 * kLowStep[f] + (t & 1), it = kLowTile[f];
                    f32x4 d = zero();
#pragma unroll
                    for (int ks = 0; ks < KS; ++ks)
                        d = mma(ty.rows(tile_row(jt, lo), 32 * ks, g), tx.rows(tile_row(it, lo), 32 * ks, g), d);
                    const int i = tile_row(it, lo), j0 = tile_row(jt, 4 * g);
                    f32x4 w;
#pragma unroll
                    for (int e = 0; e < 4; ++e) w[e] = j0 + e <= i ? pair[x][e] * d[e] : 0.f;
                    if constexpr (MODE == kGrad) {
                        f32x4 b = zero();
#pragma unroll
                        for (int ks = 0; ks < VD / 32; ++ks)
                            b = mma(tz.rows(tile_row(jt, lo), 32 * ks, g), te.rows(tile_row(it, lo), 32 * ks, g), b);
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (j0 + e < i) dg_chunk += (float)(i - j0 - e) * w[e] * b[e];
                    }
                    char *at = frags + f * L::kFrag;
                    if constexpr (sizeof(E) == 2) {
                        const u32x2 hi = {cvt_pk(w[0], w[1]), cvt_pk(w[2], w[3])};
                        *reinterpret_cast<u32x2 *>(at + lane * 16 + 8 * (t & 1)) = hi;
                        w -= f32x4{wkv7::bf16_lo(hi[0]), wkv7::bf16_hi(hi[0]), wkv7::bf16_lo(hi[1]),
                                   wkv7::bf16_hi(hi[1])};
                        *reinterpret_cast<u32x2 *>(at + 1024 + lane * 16 + 8 * (t & 1)) =
                            u32x2{cvt_pk(w[0], w[1]), cvt_pk(w[2], w[3])};
                    } else {
                        *reinterpret_cast<f32x4 *>(at + lane * 16 + 1024 * (t & 1)) = w;
                    }
                }
            }
            __builtin_amdgcn_sched_barrier(0);
            // S x^T
            constexpr int kRead = MODE == kGrad ? 3 : 2;
            f32x4 moved[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) out[i] = moved[i] = zero();
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                Frag<E> fx[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) fx[i] = tx.rows(tile_row(i, lo), 32 * ks, g);
                const Parts<E, kRead> s(S[2 * ks], S[2 * ks + 1]);
#pragma unroll
                for (int part = s.kN - 1; part >= 0; --part)
#pragma unroll
                    for (int i = 0; i < 4; ++i) out[i] = mma(s.p[part], fx[i], out[i]);
                if constexpr (MODE == kGrad) {
                    const Parts<E, kRead> r(R[2 * ks], R[2 * ks + 1]);
#pragma unroll
                    for (int part = r.kN - 1; part >= 0; --part)
#pragma unroll
                        for (int i = 0; i < 4; ++i) moved[i] = mma(r.p[part], fx[i], moved[i]);
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (MODE == kGrad) {
                    const int t = tile_row(i, lo);
                    const f32x4 m = moved[i] + (float)(t + 1) * out[i];
                    const E *q = te.p + te.offset(t, own0 + 4 * g);
                    float s = 0.f;
#pragma unroll
                    for (int e = 0; e < 4; ++e) s += to_float(q[e]) * m[e];
                    dg_chunk += rd[i] * s;
                }
                out[i] *= rd[i];
            }
            __syncthreads();  // the fragments are whole
        }
#pragma unroll
        for (int m = 0; m < M; ++m) {
            if constexpr (MODE == kGrad) {
                const f32x4 r = R[m] + (float)live * S[m];
                R[m] = r * whole.hi + r * whole.lo;
            }
            S[m] = S[m] * whole.hi + S[m] * whole.lo;
        }
        // z: as it is for the products with the fragments, weighted for the state
#pragma unroll
        for (int st = 0; st < 2; ++st) {
            const Frag<E> z = tz.template cols<4>(32 * st, own0, lane);
            if constexpr (MODE != kSum)
#pragma unroll
                for (int part = kPartsMixed<E> - 1; part >= 0; --part)
#pragma unroll
                    for (int f = 0; f < 6; ++f)
                        if (kLowStep[f] == st)
                            out[kLowTile[f]] =
                                mma(z, get_frag<E>(frags + f * L::kFrag + 1024 * part, lane), out[kLowTile[f]]);
            __builtin_amdgcn_sched_barrier(0);
            f32x4 w[2];
#pragma unroll
            for (int j = 0; j < 8; ++j) w[j >> 2][j & 3] = kd[st][j] * z.at(j);
            const Parts<E, 3> zs(w[0], w[1]);
            if constexpr (MODE == kGrad)
#pragma unroll
                for (int j = 0; j < 8; ++j) w[j >> 2][j & 3] *= (float)(live - p.shift - (32 * st + 8 * g + j));
            const Parts<E, 3> zr(w[0], w[1]);
#pragma unroll
            for (int m0 = 0; m0 < M; m0 += L::kGroup) {
                Frag<E> y[L::kGroup];
#pragma unroll
                for (int m = 0; m < L::kGroup; ++m)
                    y[m] = ty.template cols<8>(32 * st, 32 * ((m0 + m) >> 1) + 4 * ((m0 + m) & 1), lane);
#pragma unroll
                for (int part = zs.kN - 1; part >= 0; --part)
#pragma unroll
                    for (int m = 0; m < L::kGroup; ++m) {
                        S[m0 + m] = mma(y[m], zs.p[part], S[m0 + m]);
                        if constexpr (MODE == kGrad) R[m0 + m] = mma(y[m], zr.p[part], R[m0 + m]);
                    }
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        if constexpr (MODE != kSum) {
            O *to = op + start_of(c) * row;
            if constexpr (sizeof(O) == sizeof(E)) {
                // in the place of the wave's own columns of z
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    E *at = tz.p + tz.offset(tile_row(i, lo), own0 + 4 * g);
                    if constexpr (sizeof(E) == 2)
                        *reinterpret_cast<u32x2 *>(at) =
                            u32x2{cvt_pk(out[i][0], out[i][1]), cvt_pk(out[i][2], out[i][3])};
                    else
                        *reinterpret_cast<f32x4 *>(at) = out[i];
                }
                __syncthreads();  // out is whole, and x and y have been read
                Rows<E, VD, kThreads>::store(tz, to, row, live, reverse, tid);
            } else {
                const Buffer b(to, row_bytes<O>(live, row));
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    b.store4(Rows<O, VD, kThreads>::offset(tile_row(i, lo), own0 + 4 * g, row, live, reverse),
                             out[i], O());
                __syncthreads();
            }
            if constexpr (MODE == kGrad) dg += dg_chunk;
        } else {
            __syncthreads();
        }
        if (!L::kAhead) fetch(c + 1);
        put();
        __syncthreads();
    }

    if constexpr (MODE == kGrad) {
        // <R, cotangent>, and the sum over the workgroup, always in the same order
        if (p.cotangent) {
            load_state(S, p.cotangent + ((size_t)(a.seg ? unit : seq) * a.heads + h) * state_size);
#pragma unroll
            for (int m = 0; m < M; ++m)
#pragma unroll
                for (int e = 0; e < 4; ++e) dg += (double)(R[m][e] * S[m][e]);
        }
#pragma unroll
        for (int x = 32; x; x >>= 1) dg += __shfl_xor(dg, x);
        double *sums = reinterpret_cast<double *>(lds);  // the tiles have been read
        if (lane == 0) sums[wave] = dg;
        __syncthreads();
        if (tid == 0) {
            dg = sums[0];
#pragma unroll
            for (int w = 1; w < W; ++w) dg += sums[w];
            p.dg[(size_t)unit * a.heads + h] = dg;
        }
        return;  // (the dq pass leaves no state)
    }
    float *to = nullptr;
    if (MODE == kSum) {
        to = p.unit_states + ((size_t)unit * a.heads + h) * state_size;
    } else if (p.s_out && ends) {
        const int slot = p.slots_out ? p.slots_out[seq] : seq;
        if (slot >= 0 && slot < p.pool) to = p.s_out + ((size_t)slot * a.heads + h) * state_size;
    }
    if (to)  // (only passes with states [VD, KD] leave one)
#pragma unroll
        for (int m = 0; m < M; ++m)
            *reinterpret_cast<f32x4 *>(to + (own0 + lo) * KD + tile_row(m, 4 * g)) = S[m];
}

// From what the segments add to the states at their starts (in a reversed pass: at their
// ends), in place: start of the next = decay over this one * start of this one + what it adds.
struct CombineArgs {
    Layout lay;
    int seg, heads, parts, state;  // state: its numbers
    const float *g;
    struct Way {
        float *units;
        const float *s_in;
        const int *slots;
        int pool;
        bool reverse;
    } way[2];  // by blockIdx.y
};
__global__ __launch_bounds__(256) void combine_kernel(CombineArgs a) {
    const CombineArgs::Way &p = a.way[blockIdx.y];
    const unsigned parts = (unsigned)a.state / 1024;
    const int seq = (int)(blockIdx.x / parts / a.heads), h = (int)(blockIdx.x / parts % a.heads);
    const Seq sq = a.lay.seq(seq, a.seg);
    const int len = sq.end - sq.begin, n = (len + a.seg - 1) / a.seg;
    const int at = (int)(blockIdx.x % parts * 256 + threadIdx.x) * 4;
    const Decay decay(a.g[h / a.parts]);
    const Sum2 whole = decay.exact(a.seg), last = decay.exact(len - (n - 1) * a.seg);
    f32x4 S = zero();
    if (p.s_in) {
        const int slot = p.slots ? p.slots[seq] : seq;
        if (slot >= 0 && slot < p.pool)
            S = *reinterpret_cast<const f32x4 *>(p.s_in + ((size_t)slot * a.heads + h) * a.state + at);
    }
    const size_t step = (size_t)a.heads * a.state;
    float *u = p.units + ((size_t)sq.slot0 * a.heads + h) * a.state + at;
    // a sequence of no tokens has one segment of none
    const int count = n < 1 ? 1 : n;
    for (int i0 = 0; i0 < count; i0 += 4) {
        f32x4 add[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const int i = i0 + x;
            if (i < count - 1)
                add[x] = *reinterpret_cast<const f32x4 *>(u + (p.reverse ? count - 1 - i : i) * step);
        }
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const int i = i0 + x;
            if (i >= count) break;
            const int unit = p.reverse ? count - 1 - i : i;
            *reinterpret_cast<f32x4 *>(u + unit * step) = S;
            const Sum2 d = p.reverse && i == 0 ? last : whole;
            if (i < count - 1) S = S * d.hi + S * d.lo + add[x];
        }
    }
}

// dg of the caller's heads from the units', in a fixed order
__global__ __launch_bounds__(64) void dg_kernel(const double *units, float *dg, int n, int heads,
                                                int parts) {
    const int h0 = (int)blockIdx.x * parts;
    double s = 0.0;
    for (long long i = threadIdx.x; i < (long long)n * parts; i += 64)
        s += units[i / parts * heads + h0 + i % parts];
    for (int x = 32; x; x >>= 1) s += __shfl_xor(s, x);
    if (threadIdx.x == 0) dg[blockIdx.x] = (float)s;
}

// the gradient of a key head's rows: the sum over the heads that read it.  A workgroup has the
// rows of one chunk (rows outside every sequence are nobody's).
template <class E>
__global__ __launch_bounds__(256) void shared_kernel(Layout lay, const float *dq, const float *dk,
                                                     E *out_q, E *out_k, int rep, int Hk, int K) {
    Seq sq;
    lay.find((int)blockIdx.x, kChunk, sq);
    const long long first = (long long)sq.begin + (long long)((int)blockIdx.x - sq.slot0) * kChunk;
    if ((int)blockIdx.x < sq.slot0 || first >= sq.end) return;
    const int rows = sq.end - first < kChunk ? (int)(sq.end - first) : kChunk, row = Hk * K;
    const float *src = (blockIdx.y ? dk : dq) + first * rep * row;
    E *dst = (blockIdx.y ? out_k : out_q) + first * row;
    for (long long i = threadIdx.x * 4; i < (long long)rows * row; i += 1024) {
        const float *s = src + i / K * rep * K + i % K;
        f32x4 sum = *reinterpret_cast<const f32x4 *>(s);
        for (int r = 1; r < rep; ++r) sum += *reinterpret_cast<const f32x4 *>(s + (size_t)r * K);
        if constexpr (sizeof(E) == 2)
            *reinterpret_cast<u32x2 *>(dst + i) = u32x2{cvt_pk(sum[0], sum[1]), cvt_pk(sum[2], sum[3])};
        else
            *reinterpret_cast<f32x4 *>(dst + i) = sum;
    }
}

template <class E, class O, int KD, int VD, Mode MODE>
hipError_t launch_pass(const PassArgs &a, int units, int passes, hipStream_t stream) {
    using L = Shared<E, KD, VD, MODE>;
    const void *kernel = reinterpret_cast<const void *>(&pass_kernel<E, O, KD, VD, MODE>);
    const hipError_t e = allow_lds(kernel, L::kBytes);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((pass_kernel<E, O, KD, VD, MODE>),
                       dim3((unsigned)((size_t)units * a.heads), (unsigned)passes), dim3(4 * VD), L::kBytes,
                       stream, a);
    return hipGetLastError();
}
template <class E, class O, Mode MODE>
hipError_t launch_pass(const PassArgs &a, int KD, int VD, int units, int passes, hipStream_t stream) {
    if (KD == 64)
        return VD == 64 ? launch_pass<E, O, 64, 64, MODE>(a, units, passes, stream)
                        : launch_pass<E, O, 64, 128, MODE>(a, units, passes, stream);
    return VD == 64 ? launch_pass<E, O, 128, 64, MODE>(a, units, passes, stream)
                    : launch_pass<E, O, 128, 128, MODE>(a, units, passes, stream);
}
// out in the inputs' type, or (wide) in float
template <Mode MODE>
hipError_t launch_pass(const PassArgs &a, bool bf16, bool wide, int KD, int VD, int units, int passes,
                       hipStream_t stream) {
    if (!bf16) return launch_pass<float, float, MODE>(a, KD, VD, units, passes, stream);
    if (MODE != kSum && wide)
        return launch_pass<bf16_t, float, MODE>(a, KD, VD, units, passes, stream);
    return launch_pass<bf16_t, bf16_t, MODE>(a, KD, VD, units, passes, stream);
}

PassArgs common(const Problem &p, const Segments &seg, const float *g) {
    PassArgs a{};
    a.lay = Layout{p.cu, p.n_seq, p.T, p.total};
    a.seg = seg.seg; a.heads = p.heads; a.parts = p.parts;
    a.g = g;
    return a;
}

hipError_t launch_combine(const Problem &p, const Segments &seg, const float *g,
                          const CombineArgs::Way *way, int ways, hipStream_t stream) {
    CombineArgs a{};
    a.lay = Layout{p.cu, p.n_seq, p.T, p.total};
    a.seg = seg.seg; a.heads = p.heads; a.parts = p.parts;
    a.state = p.V * p.K;
    a.g = g;
    for (int i = 0; i < ways; ++i) a.way[i] = way[i];
    hipLaunchKernelGGL(combine_kernel,
                       dim3((unsigned)((size_t)p.n_seq * p.heads * (a.state / 1024)), (unsigned)ways),
                       dim3(256), 0, stream, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_forward(const ForwardArgs &f, hipStream_t stream) {
    const Problem &p = f.p;
    PassArgs a = common(p, f.seg, f.g);
    Pass &w = a.pass[0];
    w.x = f.q; w.y = f.k; w.z = f.v;
    w.x_stride = p.q_stride; w.y_stride = p.k_stride; w.z_stride = p.v_stride;
    w.x_rep = w.y_rep = p.rep(); w.z_rep = 1;
    w.out = f.o;
    w.read = w.intra = p.scale; w.write = 1.f;
    w.shift = 1;
    w.s_in = f.s0; w.s_out = f.s_out;
    w.slots_in = p.slots_in; w.slots_out = p.slots_out; w.pool = p.pool;
    w.unit_states = f.states;
    if (f.seg.seg) {
        hipError_t e = launch_pass<kSum>(a, p.bf16, false, p.K, p.V, f.seg.units, 1, stream);
        if (e != hipSuccess) return e;
        const CombineArgs::Way way{f.states, f.s0, p.slots_in, p.pool, false};
        e = launch_combine(p, f.seg, f.g, &way, 1, stream);
        if (e != hipSuccess) return e;
    }
    return launch_pass<kOut>(a, p.bf16, false, p.K, p.V, f.seg.units, 1, stream);
}

hipError_t launch_backward(const BackwardArgs &b, hipStream_t stream) {
    const Problem &p = b.p;
    const bool wide = p.rep() > 1;
    const int row_v = p.heads * p.V, units = b.seg.units;
    PassArgs a = common(p, b.seg, b.g);
    Pass dq{}, dk{}, dv{};
    dq.x = b.d_o; dq.y = b.v; dq.z = b.k;
    dq.x_stride = row_v; dq.y_stride = p.v_stride; dq.z_stride = p.k_stride;
    dq.x_rep = dq.y_rep = 1; dq.z_rep = p.rep();
    dq.out = wide ? b.dq_heads : b.dq;
    dq.read = dq.intra = p.scale; dq.write = 1.f;
    dq.shift = 1;
    dq.turned = true;
    dq.s_in = b.s0;
    dq.pool = p.n_seq;
    dq.unit_states = b.states;
    dq.e = b.q; dq.e_stride = p.q_stride; dq.e_rep = p.rep();
    dq.cotangent = b.seg.seg ? b.cotangents : b.ds_T;
    dq.dg = b.dg_units;

    dk.x = b.v; dk.y = b.d_o; dk.z = b.q;
    dk.x_stride = p.v_stride; dk.y_stride = row_v; dk.z_stride = p.q_stride;
    dk.x_rep = dk.y_rep = 1; dk.z_rep = p.rep();
    dk.out = wide ? b.dk_heads : b.dk;
    dk.read = 1.f; dk.intra = dk.write = p.scale;
    dk.turned = true;
    dk.s_in = b.ds_T;
    dk.pool = p.n_seq;
    dk.unit_states = b.cotangents;

    dv.x = b.k; dv.y = b.q; dv.z = b.d_o;
    dv.x_stride = p.k_stride; dv.y_stride = p.q_stride; dv.z_stride = row_v;
    dv.x_rep = dv.y_rep = p.rep(); dv.z_rep = 1;
    dv.out = b.dv;
    dv.read = 1.f; dv.intra = dv.write = p.scale;
    dv.s_in = b.ds_T;
    dv.s_out = b.ds0;
    dv.pool = p.n_seq;
    dv.unit_states = b.cotangents;

    hipError_t e;
    if (b.seg.seg) {
        // both states from their own products, [V, K]: k and v, and q and dO last token first
        a.pass[0] = Pass{};
        a.pass[0].y = b.k; a.pass[0].z = b.v;
        a.pass[0].y_stride = p.k_stride; a.pass[0].z_stride = p.v_stride;
        a.pass[0].x_rep = 1; a.pass[0].y_rep = p.rep(); a.pass[0].z_rep = 1;
        a.pass[0].write = 1.f; a.pass[0].shift = 1;
        a.pass[0].unit_states = b.states;
        a.pass[1] = dv;
        e = launch_pass<kSum>(a, p.bf16, false, p.K, p.V, units, 2, stream);
        if (e != hipSuccess) return e;
        const CombineArgs::Way ways[2] = {{b.states, b.s0, nullptr, p.n_seq, false},
                                          {b.cotangents, b.ds_T, nullptr, p.n_seq, true}};
        e = launch_combine(p, b.seg, b.g, ways, 2, stream);
        if (e != hipSuccess) return e;
    }
    // ds_T and ds0 may be the same memory: dv, which writes ds0, is last
    a.pass[0] = dq;
    if (b.dg_units) {
        e = launch_pass<kGrad>(a, p.bf16, wide, p.V, p.K, units, 1, stream);
        a.pass[0] = dk;
        if (e == hipSuccess) e = launch_pass<kOut>(a, p.bf16, wide, p.V, p.K, units, 1, stream);
    } else {
        a.pass[1] = dk;
        e = launch_pass<kOut>(a, p.bf16, wide, p.V, p.K, units, 2, stream);
    }
    if (e != hipSuccess) return e;
    a.pass[0] = dv;
    e = launch_pass<kOut>(a, p.bf16, false, p.K, p.V, units, 1, stream);
    if (e != hipSuccess) return e;
    if (b.dg) {
        hipLaunchKernelGGL(dg_kernel, dim3((unsigned)(p.heads / p.parts)), dim3(64), 0, stream, b.dg_units,
                           b.dg, units, p.heads, p.parts);
        e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (wide && p.total > 0) {
        const unsigned chunks = (unsigned)(p.cu ? p.total / kChunk + p.n_seq
                                                : p.n_seq * ((p.T + kChunk - 1) / kChunk));
        if (p.bf16)
            hipLaunchKernelGGL((shared_kernel<bf16_t>), dim3(chunks, 2), dim3(256), 0, stream, a.lay, b.dq_heads,
                               b.dk_heads, static_cast<bf16_t *>(b.dq), static_cast<bf16_t *>(b.dk), p.rep(), p.Hk, p.K);
        else
            hipLaunchKernelGGL((shared_kernel<float>), dim3(chunks, 2), dim3(256), 0, stream, a.lay, b.dq_heads,
                               b.dk_heads, static_cast<float *>(b.dq), static_cast<float *>(b.dk), p.rep(), p.Hk, p.K);
        e = hipGetLastError();
    }
    return e;
}

// (first form: whole sequences wherever they fill the card)
Segments plan_segments(const Problem &p, bool) {
    Segments s{0, p.n_seq};
    const long long chains = (long long)p.n_seq * p.heads;
    if (chains >= 1024 || p.total <= 256 || p.total <= 128 * p.n_seq) return s;
    long long seg = (long long)p.total * p.heads / 1024;  // about 1024 units
    seg = (seg / 256 + 1) * 256;
    if (!p.cu && seg >= p.T) return s;
    if (seg >= p.total) return s;
    s.seg = (int)seg;
    s.units = p.cu ? p.total / s.seg + p.n_seq : p.n_seq * ((p.T + s.seg - 1) / s.seg);
    return s;
}

}  // namespace lattn
