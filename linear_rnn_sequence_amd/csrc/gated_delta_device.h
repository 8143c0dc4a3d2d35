// Device-side helpers of the gated delta rule kernels (gfx950, wave64).
//
// Lane layouts (lane l, g = l >> 4, lo = l & 15, e = 0..3, j = 0..7).  One
// "fragment" is a matrix-core operand that is 32 deep in the contraction index:
//   A operand of P (16 x 32): lane holds P[lo][8g + j]
//   B operand of Q (32 x 16): lane holds Q[8g + j][lo]
//   result D (16 x 16):       lane holds D[4g + e][lo]
// A pair of result tiles of which the rows are the indices 8g + e (first tile)
// and 8g + 4 + e (second) is, element for element, the B operand of those 32
// rows and the A operand of their transpose, so results feed the next product
// from registers.  tile_row gives that order of rows; a matrix whose rows are
// read in it needs no shuffle afterwards.
//
// Element types: bf16 (one v_mfma_f32_16x16x32_bf16 per fragment pair) and float
// (eight v_mfma_f32_16x16x4_f32; the g-th quarter of the lanes gives index 8g + j
// to the j-th).  Where a float32 result has to stay one (the state and what is
// added to it), the bf16 form splits the float operand into hi + lo bf16 parts,
// 16 bits of significand together (relative error at most 2^-17), and adds the
// parts' products: the inputs q, k, v are bf16 and exact.
#pragma once

#include "wkv7_device.h"
#include "wkv7_mfma.h"

namespace gdr {

using wkv7::bf16x8;
using wkv7::bf16x8s;
using wkv7::cvt_pk;
using wkv7::f32x4;
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
typedef unsigned u32x2 __attribute__((ext_vector_type(2)));

constexpr int kChunk = 64;  // tokens per chunk

typedef uint16_t bf16_t;  // storage of a bf16 element

// row of a 16-row tile `tile` that the lane or element index r = 0..15 stands for
__device__ __forceinline__ int tile_row(int tile, int r) {
    return 32 * (tile >> 1) + 8 * (r >> 2) + 4 * (tile & 1) + (r & 3);
}

__device__ __forceinline__ float to_float(bf16_t x) { return __uint_as_float((uint32_t)x << 16); }
__device__ __forceinline__ float to_float(float x) { return x; }
template <class E>
__device__ __forceinline__ E from_float(float x);
template <>
__device__ __forceinline__ bf16_t from_float<bf16_t>(float x) {
    return (bf16_t)wkv7::f32_to_bf16_rne(x);
}
template <>
__device__ __forceinline__ float from_float<float>(float x) {
    return x;
}

// ---------------------------------------------------------------------------
// fragments
// ---------------------------------------------------------------------------
template <class E>
struct Frag;
template <>
struct Frag<bf16_t> {
    u32x4 v;
    static __device__ __forceinline__ Frag zero() { return Frag{u32x4{0u, 0u, 0u, 0u}}; }
    __device__ __forceinline__ float at(int j) const {
        const unsigned u = v[j >> 1];
        return __uint_as_float((j & 1) ? (u & 0xffff0000u) : (u << 16));
    }
};
template <>
struct Frag<float> {
    f32x4 v[2];
    static __device__ __forceinline__ Frag zero() {
        return Frag{{f32x4{0.f, 0.f, 0.f, 0.f}, f32x4{0.f, 0.f, 0.f, 0.f}}};
    }
    __device__ __forceinline__ float at(int j) const { return v[j >> 2][j & 3]; }
};

// a float operand: for bf16 its hi and lo parts, for float itself
template <class E>
struct Split;
template <>
struct Split<bf16_t> {
    Frag<bf16_t> hi, lo;
};
template <>
struct Split<float> {
    Frag<float> hi;
};

__device__ __forceinline__ f32x4 mma(const Frag<bf16_t> &a, const Frag<bf16_t> &b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a.v),
                                                   __builtin_bit_cast(bf16x8, b.v), c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mma(const Frag<float> &a, const Frag<float> &b, f32x4 c) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
        c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.v[j >> 2][j & 3], b.v[j >> 2][j & 3], c, 0, 0,
                                                 0);
    return c;
}
// exact A, float B (and the other way round)
__device__ __forceinline__ f32x4 mma(const Frag<bf16_t> &a, const Split<bf16_t> &b, f32x4 c) {
    return mma(a, b.hi, mma(a, b.lo, c));
}
__device__ __forceinline__ f32x4 mma(const Split<bf16_t> &a, const Frag<bf16_t> &b, f32x4 c) {
    return mma(a.hi, b, mma(a.lo, b, c));
}
// both float: the product of the two lo parts (2^-18 of the whole) is left out
__device__ __forceinline__ f32x4 mma(const Split<bf16_t> &a, const Split<bf16_t> &b, f32x4 c) {
    return mma(a.hi, b.hi, mma(a.hi, b.lo, mma(a.lo, b.hi, c)));
}
__device__ __forceinline__ f32x4 mma(const Frag<float> &a, const Split<float> &b, f32x4 c) {
    return mma(a, b.hi, c);
}
__device__ __forceinline__ f32x4 mma(const Split<float> &a, const Frag<float> &b, f32x4 c) {
    return mma(a.hi, b, c);
}
__device__ __forceinline__ f32x4 mma(const Split<float> &a, const Split<float> &b, f32x4 c) {
    return mma(a.hi, b.hi, c);
}

// one fragment from two result tiles (or eight floats), rounded to E
template <class E>
__device__ __forceinline__ Frag<E> to_frag(f32x4 a, f32x4 b);
template <>
__device__ __forceinline__ Frag<bf16_t> to_frag<bf16_t>(f32x4 a, f32x4 b) {
    return Frag<bf16_t>{
        u32x4{cvt_pk(a[0], a[1]), cvt_pk(a[2], a[3]), cvt_pk(b[0], b[1]), cvt_pk(b[2], b[3])}};
}
template <>
__device__ __forceinline__ Frag<float> to_frag<float>(f32x4 a, f32x4 b) {
    return Frag<float>{{a, b}};
}
template <class E>
__device__ __forceinline__ Split<E> to_split(f32x4 a, f32x4 b);
template <>
__device__ __forceinline__ Split<bf16_t> to_split<bf16_t>(f32x4 a, f32x4 b) {
    Split<bf16_t> s;
    s.hi = to_frag<bf16_t>(a, b);
    f32x4 ra, rb;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        ra[e] = a[e] - s.hi.at(e);
        rb[e] = b[e] - s.hi.at(4 + e);
    }
    s.lo = to_frag<bf16_t>(ra, rb);
    return s;
}
template <>
__device__ __forceinline__ Split<float> to_split<float>(f32x4 a, f32x4 b) {
    return Split<float>{{{a, b}}};
}

// ---------------------------------------------------------------------------
// tiles in shared memory: rows of C elements, 16 bytes of padding behind each
// row so that the 16 rows of a fragment start in different banks
// ---------------------------------------------------------------------------
template <class E, int C>
struct Tile {
    static constexpr int kPitch = C + 16 / (int)sizeof(E);
    static constexpr int kRowPieces = C * (int)sizeof(E) / 16;  // 16-byte pieces of a row
    E *p;
    // fragment along the rows: lane holds M[row][col0 + 8g + j]
    __device__ __forceinline__ Frag<E> rows(int row, int col0, int g) const {
        Frag<E> f;
        const E *s = p + row * kPitch + col0 + 8 * g;
        if constexpr (sizeof(E) == 2) {
            f.v = *reinterpret_cast<const u32x4 *>(s);
        } else {
            f.v[0] = *reinterpret_cast<const f32x4 *>(s);
            f.v[1] = *reinterpret_cast<const f32x4 *>(s + 4);
        }
        return f;
    }
    // fragment down the columns: lane holds M[row0 + 8g + j][c(lo)] for the 16
    // columns c(lo) = col0 + 8 (lo >> 2) + (lo & 3) (STEP 8: the rows of a
    // tile_row tile) or col0 + lo (STEP 4).  In bf16 by two transposing reads:
    // ds_read_b64_tr_b16 takes from each lane of a group of 16 the address of four
    // elements (lane i: row i >> 2, columns 4 (i & 3) ..) and returns to lane l
    // the four rows' elements of column l.
    template <int STEP>
    __device__ __forceinline__ Frag<E> cols(int row0, int col0, int lane) const {
        const int g = lane >> 4, lo = lane & 15;
        Frag<E> f;
        if constexpr (sizeof(E) == 2) {
            typedef short s4 __attribute__((ext_vector_type(4)));
            typedef __attribute__((address_space(3))) s4 lds_s4;
            const E *s = p + (row0 + 8 * g + (lo >> 2)) * kPitch + col0 + STEP * (lo & 3);
            const s4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4 *)s);
            const s4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4 *)(s + 4 * kPitch));
            const u32x2 ua = __builtin_bit_cast(u32x2, a), ub = __builtin_bit_cast(u32x2, b);
            f.v = u32x4{ua[0], ua[1], ub[0], ub[1]};
        } else {
            const E *s = p + (row0 + 8 * g) * kPitch + col0 + STEP * (lo >> 2) + (lo & 3);
#pragma unroll
            for (int j = 0; j < 8; ++j) f.v[j >> 2][j & 3] = s[j * kPitch];
        }
        return f;
    }
    __device__ __forceinline__ float at(int row, int col) const {
        return to_float(p[row * kPitch + col]);
    }
};
template <class E, int C>
constexpr int tile_bytes(int rows) {
    return rows * Tile<E, C>::kPitch * (int)sizeof(E);
}

// Loads of a [ROWS][C] tile with `stride` elements from row to row, held in
// registers until they are written to shared memory; rows at or behind `live`
// are zeros and not read.
template <class E, int C, int ROWS, int THREADS>
struct Stage {
    static constexpr int kPieces = ROWS * Tile<E, C>::kRowPieces;
    static constexpr int kPer = (kPieces + THREADS - 1) / THREADS;
    u32x4 x[kPer];
    __device__ __forceinline__ void load(const E *src, long long stride, int live, int tid) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int piece = tid + i * THREADS;
            const int row = piece / Tile<E, C>::kRowPieces;
            const int col = piece % Tile<E, C>::kRowPieces * (16 / (int)sizeof(E));
            x[i] = u32x4{0u, 0u, 0u, 0u};
            if (row < live && (kPieces % THREADS == 0 || piece < kPieces))
                x[i] = *reinterpret_cast<const u32x4 *>(src + row * stride + col);
        }
    }
    __device__ __forceinline__ void store(Tile<E, C> t, int tid) const {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int piece = tid + i * THREADS;
            if (kPieces % THREADS != 0 && piece >= kPieces) break;
            const int row = piece / Tile<E, C>::kRowPieces;
            const int col = piece % Tile<E, C>::kRowPieces * (16 / (int)sizeof(E));
            *reinterpret_cast<u32x4 *>(t.p + row * Tile<E, C>::kPitch + col) = x[i];
        }
    }
};

// ---------------------------------------------------------------------------
// sequences and chunks
// ---------------------------------------------------------------------------
struct Seq {
    int begin, end;  // tokens
    int slot0;       // its first chunk's number among all chunks
};

// The kernels read cu_seqlens from the device, where the host cannot check it:
// bounds are clamped to [0, total] and to a non-negative length, so that no
// value leads out of a buffer.
__device__ __forceinline__ int clamp_bound(int x, int total) {
    return x < 0 ? 0 : (x > total ? total : x);
}

struct Layout {
    const int *cu;  // [n_seq + 1] or nullptr (every sequence has T tokens)
    int n_seq, T, total, slots;
    __device__ __forceinline__ Seq seq(int i) const {
        Seq s;
        if (!cu) {
            s.begin = i * T;
            s.end = s.begin + T;
            s.slot0 = i * ((T + kChunk - 1) / kChunk);
        } else {
            s.begin = clamp_bound(cu[i], total);
            s.end = clamp_bound(cu[i + 1], total);
            if (s.end < s.begin) s.end = s.begin;
            s.slot0 = s.begin / kChunk + i;
        }
        return s;
    }
    // sequence of a chunk number; the chunk's first token (at or behind the
    // sequence's end for a number that no sequence uses)
    __device__ __forceinline__ int find(int slot, Seq &s) const {
        int i;
        if (!cu) {
            i = slot / ((T + kChunk - 1) / kChunk);
        } else {
            int lo = 0, hi = n_seq - 1;  // the last i with slot0(i) <= slot
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (clamp_bound(cu[mid], total) / kChunk + mid <= slot)
                    lo = mid;
                else
                    hi = mid - 1;
            }
            i = lo;
        }
        s = seq(i);
        return i;
    }
};

// Inclusive sums of the chunk's log decays, lane = token, in float64: the
// decay between two tokens is the exponential of a difference of these sums,
// which in float32 would lose what a strong decay before both of them took.
// exp(-200) is zero in float32, so a log decay below that (-infinity, the
// type's lowest value) is raised to it; a NaN stays one.
constexpr float kLowestLogDecay = -200.f;
__device__ __forceinline__ double scan_decay(float g, int lane) {
    double x = g < kLowestLogDecay ? kLowestLogDecay : g;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const double y = __shfl_up(x, d);
        if (lane >= d) x += y;
    }
    return x;
}
__device__ __forceinline__ float decay(double to, double from) { return __expf((float)(to - from)); }

constexpr float kNormEps = 1e-6f;

// per chunk and value head, written by the preparation kernel
struct Scalars {
    float beta[kChunk];   // write strength
    float kS[kChunk];     // beta exp(G_t) / |k_t|: factor of S0 k_t
    float kD[kChunk];     // exp(G_C - G_t) / |k_t|: factor of k_t in the exit state
    float qS[kChunk];     // scale exp(G_t) / |q_t|: factor of S0 q_t
    float last;           // exp(G_C)
    float pad[3];
};

// Fragments of a chunk's 64 x 64 triangular matrices, (tile of rows, 32 columns),
// that are not all zero: six of the lower triangle, six of an upper one.
__device__ constexpr int kLowTile[6] = {0, 1, 2, 2, 3, 3}, kLowStep[6] = {0, 0, 0, 1, 0, 1};
__device__ constexpr int kUpTile[6] = {0, 0, 1, 1, 2, 3}, kUpStep[6] = {0, 1, 0, 1, 1, 1};

// Record of one chunk and value head.  Each fragment is 64 lanes x 16 bytes per
// part.  Forward: T split, P rounded to E (it only enters o).  Backward: T^T and
// P^T, both split.
template <class E>
struct FwdRecord {
    static constexpr int kSplitBytes = 2048;                       // one split fragment (both types)
    static constexpr int kFragBytes = sizeof(E) == 2 ? 1024 : 2048;
    static constexpr int kP = 6 * kSplitBytes;
    static constexpr int kScalars = kP + 6 * kFragBytes;
    static constexpr int kBytes = kScalars + (int)sizeof(Scalars);
};
template <class E>
struct BwdRecord {
    static constexpr int kSplitBytes = 2048;
    static constexpr int kP = 6 * kSplitBytes;
    static constexpr int kScalars = 12 * kSplitBytes;
    static constexpr int kBytes = kScalars + (int)sizeof(Scalars);
};

template <class E>
__device__ __forceinline__ void put_frag(char *at, const Frag<E> &f, int lane) {
    if constexpr (sizeof(E) == 2) {
        *reinterpret_cast<u32x4 *>(at + lane * 16) = f.v;
    } else {
        *reinterpret_cast<f32x4 *>(at + lane * 16) = f.v[0];
        *reinterpret_cast<f32x4 *>(at + 1024 + lane * 16) = f.v[1];
    }
}
template <class E>
__device__ __forceinline__ Frag<E> get_frag(const char *at, int lane) {
    Frag<E> f;
    if constexpr (sizeof(E) == 2) {
        f.v = *reinterpret_cast<const u32x4 *>(at + lane * 16);
    } else {
        f.v[0] = *reinterpret_cast<const f32x4 *>(at + lane * 16);
        f.v[1] = *reinterpret_cast<const f32x4 *>(at + 1024 + lane * 16);
    }
    return f;
}
template <class E>
__device__ __forceinline__ void put_split(char *at, const Split<E> &s, int lane) {
    put_frag<E>(at, s.hi, lane);
    if constexpr (sizeof(E) == 2) put_frag<E>(at + 1024, s.lo, lane);
}
template <class E>
__device__ __forceinline__ Split<E> get_split(const char *at, int lane) {
    Split<E> s;
    s.hi = get_frag<E>(at, lane);
    if constexpr (sizeof(E) == 2) s.lo = get_frag<E>(at + 1024, lane);
    return s;
}

}  // namespace gdr
