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
//
// What bounds it: the instructions of a chunk, of which the products of states in two and three
// bf16 parts are the largest share, and what its steps wait for each other.  32768 tokens of 32 heads
// of 128 x 128 take 390 to 410 us (245 the pass, 125 the segments' sums, 12 their combination; 1.1 GB
// at 4.6 TB/s in the pass): matrix cores are busy 46% of the time, vector units 40%, shared memory 51%,
// waves wait 38% of theirs.  A chunk takes 4.2 us of a CU, also where a batch's longest sequence is a
// chain of them (16 ragged sequences of up to 2049 tokens: 152 to 162 us, 33 chunks).  In float a large
// call is at 1.6 to 3 times its operations' floor (8 x 2048 tokens of the same heads: 456 us).
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

// Segments that start as the sequence does, from s_in (or zeros), without a copy of it: none,
// those that are whole sequences (whose state nobody else writes: s_out may be s_in), or every
// sequence's first (in a reversed pass: last) one.  (8 ragged sequences of up to 1024 tokens, 16
// heads of 128, with gradients: 163 us for 168 with copies.)
enum Direct { kNone, kAlone, kStart };

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
    int direct;                        // Direct: which of those are s_in's alone
    // kGrad
    const void *e;                     // rows of q
    int e_stride, e_rep;
    const float *cotangent;            // of the sequences' ends, or nullptr
    const float *unit_cotangents;      // segments': of theirs (not where direct_end, of the last ones')
    bool direct_end;
    double *dg;                        // [units, heads]
};

struct PassArgs {
    Layout lay;
    int seg, heads, parts;
    bool join;  // segments take their starts from the sums of those before them, not from combine_kernel
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
    Parts() = default;
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

// A chunk's 64 rows of C channels in shared memory.  The rows are eight words longer than their
// channels: of all paddings that keep 16 bytes aligned those of 8 more than a multiple of 16
// words are best for every kind of read here (16 bytes along 16 rows: 4.6 cycles a wave, where 12
// words more take 8.1; transposing ones 4.1 for 6.1).  Every address is a lane's own plus a
// number known to the compiler, where a swizzle has to be computed for each (a third of the
// kernel's vector instructions).
//
// Contraction over tokens: element j of lane group g is the token 32 st + 4 g + j, for j >= 4
// 32 st + 16 + 4 g + j - 4, which is how two result tiles of 16 tokens make up an operand.
template <class E, int C>
struct Plane {
    static constexpr int kWords = C * (int)sizeof(E) / 4 + 8, kRow = 4 * kWords;
    static constexpr int kBytes = kChunk * kRow;
    char *p;
    // a lane's place for reads along the rows: row lo, channels 8 g ..
    static __device__ __forceinline__ int along(int g, int lo) {
        return lo * kRow + 8 * g * (int)sizeof(E);
    }
    // channels 32 ks + 8 g .. of row 16 i + lo; `at`: p + along()
    static __device__ __forceinline__ Frag<E> rows(const char *at, int i, int ks) {
        at += 16 * i * kRow + 32 * ks * (int)sizeof(E);
        Frag<E> f;
        if constexpr (sizeof(E) == 2) {
            f.v = *reinterpret_cast<const u32x4 *>(at);
        } else {
            f.v[0] = *reinterpret_cast<const f32x4 *>(at);
            f.v[1] = *reinterpret_cast<const f32x4 *>(at + 16);
        }
        return f;
    }
    // A lane's place for reads down the columns c(lo) = 8 (lo >> 2) + (lo & 3) (STEP 8) or lo
    // (STEP 4).  In bf16 by transposing reads: ds_read_b64_tr_b16 takes from each lane of a
    // group of 16 the address of four elements (lane i: row i >> 2, columns STEP (i & 3) ..)
    // and returns to lane l the four rows' elements of column l.
    template <int STEP>
    static __device__ __forceinline__ int down(int g, int lo) {
        if constexpr (sizeof(E) == 2) return (4 * g + (lo >> 2)) * kRow + STEP * (lo & 3) * 2;
        return 4 * g * kRow + (STEP * (lo >> 2) + (lo & 3)) * 4;
    }
    // the 32 tokens of st of column col + c(lo); `at`: p + down()
    static __device__ __forceinline__ Frag<E> cols(const char *at, int st, int col) {
        at += 32 * st * kRow + col * (int)sizeof(E);
        Frag<E> f;
        if constexpr (sizeof(E) == 2) {
            typedef short s4 __attribute__((ext_vector_type(4)));
            typedef __attribute__((address_space(3))) s4 lds_s4;
            auto read = [](const char *from) {
                return __builtin_bit_cast(
                    u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4 *)from));
            };
            const u32x2 a = read(at), b = read(at + 16 * kRow);
            f.v = u32x4{a[0], a[1], b[0], b[1]};
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                f.v[j >> 2][j & 3] = *reinterpret_cast<const float *>(at + (j < 4 ? j : 12 + j) * kRow);
        }
        return f;
    }
};

// a value that is the same for all lanes, out of the vector registers
__device__ __forceinline__ double uniform(double x) {
    const unsigned long long u = __builtin_bit_cast(unsigned long long, x);
    const unsigned lo = (unsigned)__builtin_amdgcn_readfirstlane((int)u),
                   hi = (unsigned)__builtin_amdgcn_readfirstlane((int)(u >> 32));
    return __builtin_bit_cast(double, (unsigned long long)hi << 32 | lo);
}

// Asks the scheduler for three vector instructions behind each of N matrix products: a product
// keeps the matrix core busy for four of them, and a wave's instructions issue in order.
template <class E, int N>
__device__ __forceinline__ void interleave() {
    if constexpr (sizeof(E) == 2)
#pragma unroll
        for (int i = 0; i < N; ++i) {
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x002, 3, 0);
        }
}

// Rows of a chunk on their way from memory to a plane; in a reversed pass row r is the
// live - 1 - r-th in memory.  Rows behind `live` are zeros.
template <class E, int C, int THREADS>
struct Rows {
    static constexpr int kPiece = 16 / (int)sizeof(E), kRowPieces = C / kPiece;  // elements, per row
    static constexpr int kPer = kChunk * kRowPieces / THREADS, kStep = THREADS / kRowPieces;
    static_assert(THREADS % kRowPieces == 0 && kPer * kStep == kChunk,
                  "a thread's pieces are kStep rows apart");
    u32x4 d[kPer];
    static __device__ __forceinline__ unsigned offset(int row, int col, int stride, int live,
                                                      bool reverse) {
        // (modulo 2^32: a row before the first one lies behind the buffer's end)
        const unsigned at = reverse ? (unsigned)(live - 1 - row) : (unsigned)row;
        return (at * (unsigned)stride + (unsigned)col) * (unsigned)sizeof(E);
    }
    static __device__ __forceinline__ unsigned first(int stride, int live, bool reverse, int tid) {
        return offset(tid / kRowPieces, tid % kRowPieces * kPiece, stride, live, reverse);
    }
    static __device__ __forceinline__ unsigned step(int stride, bool reverse) {
        const unsigned s = (unsigned)(kStep * (int)sizeof(E)) * (unsigned)stride;
        return reverse ? 0u - s : s;
    }
    static __device__ __forceinline__ int place(int tid) {
        return tid / kRowPieces * Plane<E, C>::kRow + tid % kRowPieces * 16;
    }
    __device__ __forceinline__ void load(const E *src, int stride, int live, bool reverse, int tid) {
        const Buffer b(src, row_bytes<E>(live, stride));
        const unsigned from = first(stride, live, reverse, tid), next = step(stride, reverse);
#pragma unroll
        for (int i = 0; i < kPer; ++i) d[i] = b.load16(from + i * next);
    }
    __device__ __forceinline__ void put(char *plane, int tid) const {
        char *at = plane + place(tid);
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            *reinterpret_cast<u32x4 *>(at + i * kStep * Plane<E, C>::kRow) = d[i];
    }
    // the way back, from the pieces that put() will write next
    static __device__ __forceinline__ void store(const char *plane, E *dst, int stride, int live,
                                                 bool reverse, int tid) {
        const Buffer b(dst, row_bytes<E>(live, stride));
        const unsigned from = first(stride, live, reverse, tid), next = step(stride, reverse);
        const char *at = plane + place(tid);
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            b.store16(from + i * next,
                      *reinterpret_cast<const u32x4 *>(at + i * kStep * Plane<E, C>::kRow));
    }
};

// The head's log decay to the base 2 (below -200 it is 0 in float32, -infinity with it; a NaN
// stays one) and its powers, of which the exponents keep more than a float's bits.
struct Decay {
    double g2;
    __device__ __forceinline__ explicit Decay(float g)
        : g2((g < kLowestLogDecay ? kLowestLogDecay : g) * 1.4426950408889634) {}
    __device__ __forceinline__ float power(int n) const {
        const double x = g2 * n;
        const float hi = (float)x;
        return exp2f(hi) * (1.f + 0.6931472f * (float)(x - hi));
    }
    __device__ __forceinline__ double exact(int n) const { return exp2(g2 * n); }
};

template <class E, int KD, int VD, Mode MODE>
struct Shared {
    static constexpr int kWaves = VD / 16, kThreads = 64 * kWaves;
    static constexpr int kTileK = Plane<E, KD>::kBytes, kTileV = Plane<E, VD>::kBytes;
    static constexpr int kFrag = 2048;  // bf16: two parts, float: two halves
    static constexpr int kY = 0, kZ = kTileK, kX = kZ + kTileV;
    static constexpr int kP = kX + (MODE == kSum ? 0 : kTileK);
    static constexpr int kE = kP + (MODE == kSum ? 0 : 6 * kFrag);
    // weights: of the tokens in the state [64], of pairs of tokens by their distance (-64 .. 63;
    // 0 below 0), of the tokens' readouts [64]
    static constexpr int kWrite = kE + (MODE == kGrad ? kTileV : 0), kPair = kWrite + kChunk * 4;
    static constexpr int kReads = kPair + 2 * kChunk * 4;
    static constexpr int kBytes = kReads + kChunk * 4;
    // the next chunk's rows are on their way while this one is computed (in float they
    // would take the registers that its products need)
    static constexpr bool kAhead = sizeof(E) == 2 && !(MODE == kGrad && KD > VD);
    // Waves per SIMD that the registers are shared out to.  Four (128 registers) hide what a wave
    // waits for: 8 x 4096 tokens, 40 heads of 64, took 262 us with two waves of 32 rows of the state
    // each and takes 215; 16 ragged sequences, 32 heads of 128, 158 and 150.
    static constexpr int kPerSimd = sizeof(E) == 4 ? 1 : MODE == kGrad || KD > VD ? 2 : 4;
    // where 128 registers are few, for two operands at a time and the weights of the readout
    static constexpr bool kFew = kPerSimd == 4 && KD == 128 && MODE == kOut;
    static constexpr bool kDouble = !kFew, kWeights = !kFew;
    // tiles of columns that the state's products have in registers at a time
    static constexpr int kGroup = 2;
};

template <class E, class O, int KD, int VD, Mode MODE>
__device__ __forceinline__ void run_pass(const PassArgs &a, const Pass &p) {
    using L = Shared<E, KD, VD, MODE>;
    constexpr int W = L::kWaves, kThreads = L::kThreads, KS = KD / 32, M = KD / 16;
    constexpr int kTiles = (10 + W - 1) / W;  // of x y^T per wave
    extern __shared__ __align__(16) char lds[];
    const int tid = threadIdx.x, lane = tid & 63,
              wave = __builtin_amdgcn_readfirstlane(tid >> 6), g = lane >> 4, lo = lane & 15;
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
    const int tokens = sq.end - sq.begin, rest = tokens - first;
    const int len = a.seg && rest > a.seg ? a.seg : rest;
    const bool ends = reverse ? first == 0 : len == rest;
    const bool starts = reverse ? len == rest : first == 0;
    if (MODE == kSum && ends) return;  // nothing follows it
    const long long token = (long long)sq.begin + first;
    const int chunks = (len + kChunk - 1) / kChunk;
    const size_t state_size = (size_t)VD * KD;

    const Decay decay(a.g[h / a.parts]);
    float *write = reinterpret_cast<float *>(lds + L::kWrite),
          *pairs = reinterpret_cast<float *>(lds + L::kPair),
          *reads = reinterpret_cast<float *>(lds + L::kReads);
    if (tid < kChunk) {
        write[tid] = p.write * decay.power(kChunk - p.shift - tid);
        pairs[tid] = 0.f;
        pairs[kChunk + tid] = p.intra * decay.power(tid);
        reads[tid] = p.read * decay.power(tid + p.shift);
    }

    // the wave's rows of a state in memory: row own0 + lo, columns tile_row(m, 4g) ..
    const int own0 = 16 * wave;
    auto load_state = [&](f32x4(&S)[M], const float *base) {
        if (p.turned) {
#pragma unroll
            for (int m = 0; m < M; ++m)
#pragma unroll
                for (int e = 0; e < 4; ++e) S[m][e] = base[(tile_row(m, 4 * g) + e) * VD + own0 + lo];
        } else {
#pragma unroll
            for (int m = 0; m < M; ++m)
                S[m] = *reinterpret_cast<const f32x4 *>(base + (own0 + lo) * KD + tile_row(m, 4 * g));
        }
    };
    // The state at the segment's start (`back`: the cotangent at its end), where the segments are
    // joined here: the sequence's own, and on top of it what the segments before (behind) add.
    auto joined = [&](f32x4(&S)[M], const float *start, const float *units, bool back) {
#pragma unroll
        for (int m = 0; m < M; ++m) S[m] = zero();
        if (start) load_state(S, start);
        const int all = tokens > a.seg ? (tokens + a.seg - 1) / a.seg : 1, mine = unit - sq.slot0;
        const int before = back ? all - 1 - mine : mine;
#pragma unroll 1
        for (int i = 0; i < before; ++i) {
            const int other = sq.slot0 + (back ? all - 1 - i : i);
            const double d = uniform(decay.exact(back && i == 0 ? tokens - (all - 1) * a.seg : a.seg));
            const float hi = (float)d, lo = (float)(d - hi);
            f32x4 add[M];
            load_state(add, units + ((size_t)other * a.heads + h) * state_size);
#pragma unroll
            for (int m = 0; m < M; ++m) S[m] = S[m] * hi + (S[m] * lo + add[m]);
        }
    };
    f32x4 S[M], R[MODE == kGrad ? M : 1];
    const float *from = nullptr;
    if (MODE != kSum && a.seg && !a.join && !(starts && p.direct >= (ends ? kAlone : kStart))) {
        from = p.unit_states + ((size_t)unit * a.heads + h) * state_size;
    } else if (MODE != kSum && p.s_in) {
        const int slot = p.slots_in ? p.slots_in[seq] : seq;
        if (slot >= 0 && slot < p.pool) from = p.s_in + ((size_t)slot * a.heads + h) * state_size;
    }
    if (MODE != kSum && a.join) {
        joined(S, from, p.unit_states, reverse);
    } else if (from) {
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

    using PK = Plane<E, KD>;
    using PV = Plane<E, VD>;
    char *const px = lds + L::kX, *const py = lds + L::kY;
    char *const pz = lds + L::kZ, *const pe = lds + L::kE;
    const char *const x_rows = px + PK::along(g, lo), *const y_rows = py + PK::along(g, lo),
               *const y_cols = py + PK::template down<8>(g, lo),
               *const z_cols = pz + PV::template down<4>(g, lo) + own0 * (int)sizeof(E),
               *const z_rows = pz + PV::along(g, lo), *const e_rows = pe + PV::along(g, lo);
    // channels own0 + 4 g .. of row lo
    const int own_place = lo * PV::kRow + (own0 + 4 * g) * (int)sizeof(E);
    // channels own0 + 8 (g >> 1) .. of row lo, or of row 16 + lo for odd g
    const int pair_place = (lo + 16 * (g & 1)) * PV::kRow + (own0 + 8 * (g >> 1)) * 2;
    char *const frags = lds + L::kP + lane * 16;

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
        if (MODE != kSum) gx.put(px, tid);
        gy.put(py, tid);
        gz.put(pz, tid);
        if constexpr (MODE == kGrad) ge.put(pe, tid);
    };
    if (chunks > 0) {
        fetch(0);
        put();
    }
    // Fragments 0, 1, 2 .. of x y^T: token tiles 0 and 1 with the tokens 0 .. 31, 2 and 3 with
    // both halves.  Tiles (0, 1) and (2, 3) lie above the diagonal and stay zero.
    if (MODE != kSum && wave == 0)
#pragma unroll
        for (int half = 0; half < 2; ++half)
#pragma unroll
            for (int f = 0; f <= 3; f += 3) {
                if constexpr (sizeof(E) == 2)
                    *reinterpret_cast<u32x2 *>(frags + f * L::kFrag + 1024 * half + 8) = u32x2{0u, 0u};
                else if (half)
                    *reinterpret_cast<f32x4 *>(frags + f * L::kFrag + 1024) = zero();
            }
    __syncthreads();

    float rds[4];  // of the readout of the tokens 16 i + lo
    if constexpr (L::kWeights)
#pragma unroll
        for (int i = 0; i < 4; ++i) rds[i] = p.read * decay.power(16 * i + lo + p.shift);
    // The state's decay over a chunk, as a float: what that is off by goes into the next one,
    // so that after any number of chunks the state has been decayed by the exact power.
    double whole = uniform(decay.exact(kChunk)), owed = 1.0;
    const double rest_of = uniform(decay.exact(live_of(chunks - 1)));  // over the last chunk
    const double back = uniform(whole > 1e-30 ? 1.0 / whole : 0.0);
    double dg = 0.0;

    for (int c = 0; c < chunks; ++c) {
        const int live = live_of(c);
        if (L::kAhead && MODE == kSum) fetch(c + 1);
        if (live < kChunk) {  // the last one (its other weights are read behind the next barrier)
            whole = rest_of;
            if (tid < kChunk) {
                const int n = live - p.shift - tid;
                write[tid] = n < 0 ? 0.f : p.write * decay.power(n);
            }
            if (MODE == kSum) __syncthreads();
        }
        const double want = whole * owed;
        const float fade = (float)want;
        owed = uniform(1.0 + (want - fade) * back);
        f32x4 out[4];
        float dg_chunk = 0.f;
        if constexpr (MODE != kSum) {
            // x y^T, masked and decayed: tiles (it, jt) of the lower triangle, row by row; the waves
            // take turns.  Of eight waves, those without a second tile skip it (390 us against 397,
            // 32768 tokens, 32 heads of 128); of four, those without a third do the last one again,
            // which costs less than the branches (214 us against 218, 8 x 4096, 40 heads of 64).
            auto mine = [&](int n) { return W != 8 || n == 0 || wave + n * W < 10; };
            f32x4 d[kTiles], b[MODE == kGrad ? kTiles : 1];
            int it[kTiles], jt[kTiles];
#pragma unroll
            for (int n = 0; n < kTiles; ++n) {
                const int t = wave + n * W < 10 ? wave + n * W : 9;
                it[n] = 0xffa94 >> 2 * t & 3;
                jt[n] = 0xe4910 >> 2 * t & 3;
                d[n] = zero();
                if constexpr (MODE == kGrad) b[n] = zero();
            }
#pragma unroll
            for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                for (int n = 0; n < kTiles; ++n)
                    if (mine(n))
                        d[n] = mma(PK::rows(y_rows, jt[n], ks), PK::rows(x_rows, it[n], ks), d[n]);
            if constexpr (MODE == kGrad) {
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int ks = 0; ks < VD / 32; ++ks)
#pragma unroll
                    for (int n = 0; n < kTiles; ++n)
                        if (mine(n))
                            b[n] = mma(PV::rows(z_rows, jt[n], ks), PV::rows(e_rows, it[n], ks), b[n]);
            }
#pragma unroll
            for (int n = 0; n < kTiles; ++n) {
                if (!mine(n)) break;
                const int far = 16 * (it[n] - jt[n]) + lo - 4 * g;  // i - j of element 0
                const float *weight = pairs + kChunk + far;
                f32x4 w;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    w[e] = weight[-e] * d[n][e];
                    w[e] = far >= e ? w[e] : 0.f;  // (also where d is not finite)
                    if constexpr (MODE == kGrad) {
                        const float one = (float)(far - e) * w[e] * b[n][e];
                        dg_chunk += far > e && wave + n * W < 10 ? one : 0.f;
                    }
                }
                char *at = frags + (it[n] + (it[n] == 3) + (jt[n] >> 1)) * L::kFrag;
                if constexpr (sizeof(E) == 2) {
                    const u32x2 hi = {cvt_pk(w[0], w[1]), cvt_pk(w[2], w[3])};
                    *reinterpret_cast<u32x2 *>(at + 8 * (jt[n] & 1)) = hi;
                    w -= f32x4{wkv7::bf16_lo(hi[0]), wkv7::bf16_hi(hi[0]), wkv7::bf16_lo(hi[1]),
                               wkv7::bf16_hi(hi[1])};
                    *reinterpret_cast<u32x2 *>(at + 1024 + 8 * (jt[n] & 1)) =
                        u32x2{cvt_pk(w[0], w[1]), cvt_pk(w[2], w[3])};
                } else {
                    *reinterpret_cast<f32x4 *>(at + 1024 * (jt[n] & 1)) = w;
                }
            }
            __builtin_amdgcn_sched_barrier(0);
            // S x^T; the next step's operand is formed beside this one's products.  Two parts of the
            // state, 16 bits, for outputs of 8: against sums in float one output in 430 is rounded the
            // other way (16 ragged sequences of up to 2049 tokens), 1.0e-4 of them in the norm beside the
            // rounding's own 1.7e-3.  Three for dg, whose terms cancel.
            constexpr int kRead = MODE == kGrad ? 3 : 2;
            f32x4 moved[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) out[i] = moved[i] = zero();
            Frag<E> fx[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) fx[i] = PK::rows(x_rows, i, 0);
            Parts<E, kRead> s(S[0], S[1]);
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                Frag<E> fn[4];
                if (L::kDouble && ks + 1 < KS)
#pragma unroll
                    for (int i = 0; i < 4; ++i) fn[i] = PK::rows(x_rows, i, ks + 1);
                if (!L::kDouble && ks > 0)
#pragma unroll
                    for (int i = 0; i < 4; ++i) fx[i] = PK::rows(x_rows, i, ks);
                const Parts<E, kRead> now = s;
                if (ks + 1 < KS) s = Parts<E, kRead>(S[(2 * ks + 2) % M], S[(2 * ks + 3) % M]);
#pragma unroll
                for (int part = now.kN - 1; part >= 0; --part)
#pragma unroll
                    for (int i = 0; i < 4; ++i) out[i] = mma(now.p[part], fx[i], out[i]);
                if constexpr (MODE == kGrad) {
                    const Parts<E, kRead> r(R[2 * ks], R[2 * ks + 1]);
#pragma unroll
                    for (int part = r.kN - 1; part >= 0; --part)
#pragma unroll
                        for (int i = 0; i < 4; ++i) moved[i] = mma(r.p[part], fx[i], moved[i]);
                }
                interleave<E, 4 * Parts<E, kRead>::kN * (MODE == kGrad ? 2 : 1)>();
                __builtin_amdgcn_sched_barrier(0);
                if (L::kDouble)
#pragma unroll
                    for (int i = 0; i < 4; ++i) fx[i] = fn[i];
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float rd = L::kWeights ? rds[i] : reads[16 * i + lo];
                if constexpr (MODE == kGrad) {
                    const f32x4 m = moved[i] + (float)(16 * i + lo + 1) * out[i];
                    const E *q = reinterpret_cast<const E *>(pe + own_place + 16 * i * PV::kRow);
                    float s = 0.f;
#pragma unroll
                    for (int e = 0; e < 4; ++e) s += to_float(q[e]) * m[e];
                    dg_chunk += rd * s;
                }
                out[i] *= rd;
            }
            __syncthreads();  // the fragments are whole
            if (L::kAhead) fetch(c + 1);  // (at the top its registers would be in the way above)
        }
        // z: as it is for the products with the fragments, weighted for the state
        const Frag<E> z[2] = {PV::cols(z_cols, 0, 0), PV::cols(z_cols, 1, 0)};
        Parts<E, 3> zs[2], zr[2];  // (by st)
        auto split = [&](int st) {
            f32x4 w[2];
            const f32x4 kd0 = *reinterpret_cast<const f32x4 *>(write + 32 * st + 4 * g),
                        kd1 = *reinterpret_cast<const f32x4 *>(write + 32 * st + 16 + 4 * g);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                w[0][j] = kd0[j] * z[st].at(j);
                w[1][j] = kd1[j] * z[st].at(4 + j);
            }
            zs[st] = Parts<E, 3>(w[0], w[1]);
            if constexpr (MODE == kGrad) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int token = 32 * st + 4 * g + (j < 4 ? j : 12 + j);
                    w[j >> 2][j & 3] *= (float)(live - p.shift - token);
                }
                zr[st] = Parts<E, 3>(w[0], w[1]);
            }
        };
        auto decayed = [&](int m0) {  // a group of the state's tiles
#pragma unroll
            for (int m = m0; m < m0 + L::kGroup; ++m) {
                if constexpr (MODE == kGrad) R[m] = (R[m] + (float)live * S[m]) * fade;
                S[m] *= fade;
            }
        };
        Frag<E> y[L::kGroup], yn[L::kGroup];
        auto columns = [&](int at, Frag<E>(&y)[L::kGroup]) {
#pragma unroll
            for (int m = 0; m < L::kGroup; ++m) {
                const int col = at % M + m;
                y[m] = PK::cols(y_cols, at / M, 32 * (col >> 1) + 4 * (col & 1));
            }
        };
        if constexpr (MODE != kSum) {
#pragma unroll
            for (int st = 0; st < 2; ++st)
#pragma unroll
                for (int part = kPartsMixed<E> - 1; part >= 0; --part) {
#pragma unroll
                    for (int f = 0; f < 6; ++f)
                        if (kLowStep[f] == st) {
                            const Frag<E> w = get_frag<E>(frags + f * L::kFrag + 1024 * part, 0);
                            out[kLowTile[f]] = mma(z[st], w, out[kLowTile[f]]);
                        }
                    if (sizeof(E) == 4) __builtin_amdgcn_sched_barrier(0);
                }
        }
        split(0);
        decayed(0);
        if (MODE != kSum) interleave<E, 12>();
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (MODE != kSum && sizeof(O) == sizeof(E)) {
            // out in the place of the wave's own columns of z (stores of the lanes' pieces from
            // here, of 64 bytes a row and wave, took 281 us where whole rows take 254: 8 x 4096
            // tokens, 40 heads of 64)
#pragma unroll
            for (int i = 0; i < 4; i += 2) {
                const f32x4 &x = out[i], &y = out[i + 1];
                if constexpr (sizeof(E) == 2) {
                    // Neighbouring lane groups trade the halves of two tiles (v_permlane16_swap:
                    // the odd ones' of its first operand for the even ones' of its second), so
                    // that a lane has eight values of a token: even groups of tile i, odd ones
                    // of i + 1.  (Writes of 8 bytes meet the same banks: 16 cycles for 5.)
                    const auto u = __builtin_amdgcn_permlane16_swap(
                        cvt_pk(x[0], x[1]), cvt_pk(y[0], y[1]), false, false);
                    const auto v = __builtin_amdgcn_permlane16_swap(
                        cvt_pk(x[2], x[3]), cvt_pk(y[2], y[3]), false, false);
                    *reinterpret_cast<u32x4 *>(pz + pair_place + 16 * i * PV::kRow) =
                        u32x4{u[0], v[0], u[1], v[1]};
                } else {
                    char *at = pz + own_place + 16 * i * PV::kRow;
                    *reinterpret_cast<f32x4 *>(at) = x;
                    *reinterpret_cast<f32x4 *>(at + 16 * PV::kRow) = y;
                }
            }
        }
        if constexpr (MODE != kSum && sizeof(O) != sizeof(E)) {
            const Buffer b(op + start_of(c) * row, row_bytes<O>(live, row));
#pragma unroll
            for (int i = 0; i < 4; ++i)
                b.store4(Rows<O, VD, kThreads>::offset(16 * i + lo, own0 + 4 * g, row, live, reverse),
                         out[i], O());
        }
        // the state, kGroup tiles of columns at a time; beside the products the next group's rows of y
        // are on their way, its tiles are decayed, and the second half's z is split
        columns(0, y);
#pragma unroll
        for (int at = 0; at < 2 * M; at += L::kGroup) {
            const int m0 = at % M, st = at / M;
            if (L::kDouble && at + L::kGroup < 2 * M) columns(at + L::kGroup, yn);
            if (!L::kDouble && at) columns(at, y);
            if (at + L::kGroup < M) decayed(at + L::kGroup);
            if (at == (L::kDouble ? 0 : M)) split(1);
#pragma unroll
            for (int part = Parts<E, 3>::kN - 1; part >= 0; --part)
#pragma unroll
                for (int m = 0; m < L::kGroup; ++m) {
                    S[m0 + m] = mma(y[m], zs[st].p[part], S[m0 + m]);
                    if constexpr (MODE == kGrad) R[m0 + m] = mma(y[m], zr[st].p[part], R[m0 + m]);
                }
            if (L::kDouble)
#pragma unroll
                for (int m = 0; m < L::kGroup; ++m) y[m] = yn[m];
            interleave<E, L::kGroup * Parts<E, 3>::kN * (MODE == kGrad ? 2 : 1)>();
            __builtin_amdgcn_sched_barrier(0);
        }
        __syncthreads();  // out is whole, and the planes have been read
        if constexpr (MODE != kSum && sizeof(O) == sizeof(E))
            Rows<E, VD, kThreads>::store(pz, reinterpret_cast<E *>(op + start_of(c) * row), row, live,
                                         reverse, tid);
        if constexpr (MODE == kGrad) dg += dg_chunk;
        if (!L::kAhead) fetch(c + 1);
        put();
        __syncthreads();
    }

    if constexpr (MODE == kGrad) {
        // <R, cotangent>, and the sum over the workgroup, always in the same order
        const bool own = a.seg && !(ends && p.direct_end);
        const float *D = own && !a.join ? p.unit_cotangents : p.cotangent;
        if (D) D += ((size_t)(own && !a.join ? unit : seq) * a.heads + h) * state_size;
        if (D || (own && a.join)) {
            if (a.join)
                joined(S, D, p.unit_cotangents, true);
            else
                load_state(S, D);
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

template <class E, class O, int KD, int VD, Mode MODE>
__global__ __launch_bounds__((Shared<E, KD, VD, MODE>::kThreads),
                             (Shared<E, KD, VD, MODE>::kPerSimd)) void
pass_kernel(PassArgs a) {
    run_pass<E, O, KD, VD, MODE>(a, a.pass[blockIdx.y]);
}
// dq with dg, and the passes behind it, in one launch
template <class E, class O, int KD, int VD>
__global__ __launch_bounds__((Shared<E, KD, VD, kGrad>::kThreads),
                             (Shared<E, KD, VD, kGrad>::kPerSimd)) void
gradient_kernel(PassArgs a) {
    if (blockIdx.y == 0)
        run_pass<E, O, KD, VD, kGrad>(a, a.pass[0]);
    else
        run_pass<E, O, KD, VD, kOut>(a, a.pass[blockIdx.y]);
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
        int direct;
    } way[2];  // by blockIdx.y
};
__global__ __launch_bounds__(256) void combine_kernel(CombineArgs a) {
    const CombineArgs::Way &p = a.way[blockIdx.y];
    const unsigned parts = (unsigned)a.state / 1024;
    const int seq = (int)(blockIdx.x / parts / a.heads), h = (int)(blockIdx.x / parts % a.heads);
    const Seq sq = a.lay.seq(seq, a.seg);
    const int len = sq.end - sq.begin, n = (len + a.seg - 1) / a.seg;
    const int at = (int)(blockIdx.x % parts * 256 + threadIdx.x) * 4;
    if (p.direct != kNone && n < 2) return;
    const Decay decay(a.g[h / a.parts]);
    const double whole = decay.exact(a.seg), last = decay.exact(len - (n - 1) * a.seg);
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
    // eight segments' at a time, the next eight on their way before these are overwritten
    constexpr int kAtOnce = 8;
    f32x4 add[kAtOnce], next[kAtOnce];
    auto fetch = [&](int i0) {
#pragma unroll
        for (int x = 0; x < kAtOnce; ++x)
            if (i0 + x < count - 1)
                next[x] = *reinterpret_cast<const f32x4 *>(
                    u + (p.reverse ? count - 1 - i0 - x : i0 + x) * step);
    };
    fetch(0);
    for (int i0 = 0; i0 < count; i0 += kAtOnce) {
#pragma unroll
        for (int x = 0; x < kAtOnce; ++x) add[x] = next[x];
        fetch(i0 + kAtOnce);
#pragma unroll
        for (int x = 0; x < kAtOnce; ++x) {
            const int i = i0 + x;
            if (i >= count) break;
            const int unit = p.reverse ? count - 1 - i : i;
            if (i > 0 || p.direct != kStart) *reinterpret_cast<f32x4 *>(u + unit * step) = S;
            const double d = p.reverse && i == 0 ? last : whole;
            const float hi = (float)d, lo = (float)(d - hi);  // (as exact as a product of floats is)
            if (i < count - 1) S = S * hi + (S * lo + add[x]);
        }
    }
}

// What is left of the gradients: dg of the caller's heads from the units', in a fixed order
// (blockIdx.y 0), and the gradient of a key head's rows, the sum over the heads that read it (1: of
// q, 2: of k).  There a workgroup has the rows of one chunk; rows outside every sequence are
// nobody's.
struct RestArgs {
    Layout lay;
    const double *units;
    float *dg;
    int n, heads, parts;
    const float *dq, *dk;
    void *out_q, *out_k;
    int rep, Hk, K, chunks;  // 0 chunks: no shared heads
};
template <class E>
__global__ __launch_bounds__(256) void rest_kernel(RestArgs a) {
    if (blockIdx.y == 0) {
        const int head = (int)blockIdx.x * 4 + (int)(threadIdx.x >> 6);  // a wave each
        if (!a.dg || head >= a.heads / a.parts) return;
        double s = 0.0;
        for (long long i = threadIdx.x & 63; i < (long long)a.n * a.parts; i += 64)
            s += a.units[i / a.parts * a.heads + head * a.parts + i % a.parts];
        for (int x = 32; x; x >>= 1) s += __shfl_xor(s, x);
        if ((threadIdx.x & 63) == 0) a.dg[head] = (float)s;
        return;
    }
    if ((int)blockIdx.x >= a.chunks) return;  // many heads, few tokens
    Seq sq;
    a.lay.find((int)blockIdx.x, kChunk, sq);
    const long long first = (long long)sq.begin + (long long)((int)blockIdx.x - sq.slot0) * kChunk;
    if ((int)blockIdx.x < sq.slot0 || first >= sq.end) return;
    const int rows = sq.end - first < kChunk ? (int)(sq.end - first) : kChunk, row = a.Hk * a.K;
    const float *src = (blockIdx.y == 2 ? a.dk : a.dq) + first * a.rep * row;
    E *dst = static_cast<E *>(blockIdx.y == 2 ? a.out_k : a.out_q) + first * row;
    const int shift = a.K == 64 ? 6 : 7;
    for (int i = threadIdx.x * 4; i < rows * row; i += 1024) {  // (below 64 x 2^23)
        const float *s = src + ((size_t)(i >> shift) * a.rep << shift) + (i & (a.K - 1));
        f32x4 sum = *reinterpret_cast<const f32x4 *>(s);
        for (int r = 1; r < a.rep; ++r) sum += *reinterpret_cast<const f32x4 *>(s + (size_t)r * a.K);
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
                       dim3((unsigned)((size_t)units * a.heads), (unsigned)passes),
                       dim3(L::kThreads), L::kBytes, stream, a);
    return hipGetLastError();
}
template <int D>
hipError_t launch_gradients(const PassArgs &a, int units, hipStream_t stream) {
    using L = Shared<float, D, D, kGrad>;
    const hipError_t e =
        allow_lds(reinterpret_cast<const void *>(&gradient_kernel<float, float, D, D>), L::kBytes);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((gradient_kernel<float, float, D, D>),
                       dim3((unsigned)((size_t)units * a.heads), 3), dim3(L::kThreads), L::kBytes,
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
    w.direct = f.s_out && f.s_out == f.s0 ? kAlone : kStart;
    if (f.seg.seg) {
        hipError_t e = launch_pass<kSum>(a, p.bf16, false, p.K, p.V, f.seg.units, 1, stream);
        if (e != hipSuccess) return e;
        a.join = f.seg.few && w.direct == kStart;
        const CombineArgs::Way way{f.states, f.s0, p.slots_in, p.pool, false, w.direct};
        if (!a.join) e = launch_combine(p, f.seg, f.g, &way, 1, stream);
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
    dq.direct = kStart;
    dq.cotangent = b.ds_T;
    dq.unit_cotangents = b.cotangents;
    const bool in_place = b.ds0 && b.ds0 == b.ds_T;  // dk reads what dv writes
    const Direct from_end = in_place ? kNone : kStart;
    dq.direct_end = from_end == kStart;
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
    dk.direct = from_end;

    dv.x = b.k; dv.y = b.q; dv.z = b.d_o;
    dv.x_stride = p.k_stride; dv.y_stride = p.q_stride; dv.z_stride = row_v;
    dv.x_rep = dv.y_rep = p.rep(); dv.z_rep = 1;
    dv.out = b.dv;
    dv.read = 1.f; dv.intra = dv.write = p.scale;
    dv.s_in = b.ds_T;
    dv.s_out = b.ds0;
    dv.pool = p.n_seq;
    dv.unit_states = b.cotangents;
    dv.direct = from_end;

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
        const CombineArgs::Way ways[2] = {{b.states, b.s0, nullptr, p.n_seq, false, kStart},
                                          {b.cotangents, b.ds_T, nullptr, p.n_seq, true, from_end}};
        a.join = b.seg.few && from_end == kStart;
        if (!a.join) e = launch_combine(p, b.seg, b.g, ways, 2, stream);
        if (e != hipSuccess) return e;
    }
    // dq, dk and dv, at once where the shapes and the types of their outputs are alike.  dq with dg
    // is a launch of its own in bf16, where it has half as many waves on a SIMD as the others; in
    // float they are equal.  ds_T and ds0 may be the same memory: then dv, which writes ds0, is
    // launched behind those that read ds_T.
    const bool alike = p.K == p.V && (!wide || !p.bf16) && (b.seg.seg || !in_place);
    int n = 0;
    if (b.dg_units && alike && !p.bf16) {
        a.pass[n++] = dq;
    } else if (b.dg_units) {
        a.pass[0] = dq;
        e = launch_pass<kGrad>(a, p.bf16, wide, p.V, p.K, units, 1, stream);
        if (e != hipSuccess) return e;
    } else {
        a.pass[n++] = dq;
    }
    a.pass[n++] = dk;
    if (alike) a.pass[n++] = dv;
    if (b.dg_units && n == 3)
        e = p.K == 64 ? launch_gradients<64>(a, units, stream) : launch_gradients<128>(a, units, stream);
    else
        e = launch_pass<kOut>(a, p.bf16, wide, p.V, p.K, units, n, stream);
    if (e != hipSuccess) return e;
    if (!alike) {
        a.pass[0] = dv;
        e = launch_pass<kOut>(a, p.bf16, false, p.K, p.V, units, 1, stream);
        if (e != hipSuccess) return e;
    }
    int chunks = 0;
    if (wide && p.total > 0)
        chunks = p.cu ? p.total / kChunk + p.n_seq : p.n_seq * ((p.T + kChunk - 1) / kChunk);
    if (b.dg || chunks) {
        const RestArgs r{a.lay, b.dg_units, b.dg, units, p.heads, p.parts, b.dq_heads, b.dk_heads,
                         b.dq, b.dk, p.rep(), p.Hk, p.K, chunks};
        const int heads = b.dg ? (p.heads / p.parts + 3) / 4 : 0;
        const dim3 grid((unsigned)(chunks > heads ? chunks : heads), chunks ? 3 : 1);
        if (p.bf16)
            hipLaunchKernelGGL((rest_kernel<bf16_t>), grid, dim3(256), 0, stream, r);
        else
            hipLaunchKernelGGL((rest_kernel<float>), grid, dim3(256), 0, stream, r);
        e = hipGetLastError();
    }
    return e;
}

// Dense sequences of at most this many segments are joined by the passes themselves, each reading
// the sums before its own (1.1 us for one), without a combination: 4 x 2048 tokens, 32 heads of 128,
// with gradients, in quarters forward and halves backward, take 398 us for 410; 8 segments of 512
// tokens, 4 heads, would take 31.6 for 23.4.
constexpr int kFewSegments = 4;

// How a call's sequences are cut into segments, which are then done in parallel.  A segment's
// sum and the combination cost about half of the pass again, so whole sequences are taken where
// they fill the card (256 workgroups; 8 x 4096 tokens, 40 heads of 64: 217 us whole, 255 in halves,
// 296 in 256s) or are short (300 tokens, 32 heads of 128: 26 us whole, 31 in 64s, 29 in 128s; 384: 29
// whole and in 128s, 32 in 64s; 448: 33 whole, 28 in 128s; 384 of 4 heads: 28 whole, 27 in 128s).  Else
// about one workgroup per CU (2 x 1000 tokens, 32 heads of 128: 44 us, with two per CU 55; 2 x 4096:
// 109 and 115; with gradients, 4 x 2048: 391 in 1024s, 450 in 512s, 477 whole; 4096 tokens, 16 heads:
// 161 in 256s, 187 in 512s, 203 in 128s).  In the forward two, where one would have more than 2048
// tokens (32768 tokens, 32 heads of 128: 402 us in 2048s, 424 in 4096s and in 1024s, 460 in 512s) or
// has four waves (2 x 4096, 40 heads of 64: 64 us, with one per CU 73).  And not more segments than
// their combination, a step of 0.25 us for each, is worth (6 us for a chunk more in each).  A packed
// batch's longest sequence, which the host does not know, is taken for twice the mean.  Where one is far
// longer this is slow: 32768 tokens beside a single one, 32 heads of 128, take 979 us, beside eight 1946
// (288 chains, all whole), for 408 alone; with gradients 5.3 ms for 1.25 beside eight.
Segments plan_segments(const Problem &p, bool backward) {
    Segments s{0, p.n_seq, false};
    const long long chains = (long long)p.n_seq * p.heads;
    const long long mean = p.total / p.n_seq, longest = p.n_seq > 1 && p.cu ? 2 * mean : mean;
    if (chains >= 256 || longest <= (p.bf16 && !backward ? 384 : 192)) return s;
    const long long share = p.total * (long long)p.heads / 256;
    const bool one = backward || (p.V == 128 && share <= 2048);  // workgroup per CU
    long long chunks = ((one ? share : share / 2) + kChunk - 1) / kChunk;
    if (chunks < 1) chunks = 1;
    while (chunks * chunks * 1600 < longest) ++chunks;
    // (where most sequences are shorter, there are more of them: 16 up to 2049 tokens, 8 heads, take
    // 77 us in 192s, 69 in 512s; 8 up to 1024, 16 heads, with gradients 191 in 192s, 157 in 256s)
    if (p.cu && p.n_seq > 1 && p.bf16 && chunks * kChunk * 3 < 2 * mean)
        chunks = (2 * mean / 3 + kChunk - 1) / kChunk;
    if (!p.cu) {  // equal ones
        const long long all = (p.T + kChunk - 1) / kChunk, n = (all + chunks - 1) / chunks;
        if (n < 2) return s;
        chunks = (all + n - 1) / n;
        s.few = n <= kFewSegments;
    }
    const long long seg = chunks * kChunk;
    if (seg >= p.total) return s;
    s.seg = (int)seg;
    s.units = p.cu ? p.total / s.seg + p.n_seq : p.n_seq * ((p.T + s.seg - 1) / s.seg);
    return s;
}

}  // namespace lattn
