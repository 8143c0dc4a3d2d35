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

#include "gated_delta_kept.h"
#include "wkv7_device.h"
#include "wkv7_mfma.h"

namespace gdr {

using wkv7::bf16x8;
using wkv7::bf16x8s;
using wkv7::cvt_pk;
using wkv7::f32x4;
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
typedef unsigned u32x2 __attribute__((ext_vector_type(2)));

constexpr int kChunk = 64;          // tokens per chunk
constexpr float kNormEps = 1e-6f;

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
    __device__ __forceinline__ float at(int j) const {
        const unsigned u = v[j >> 1];
        return __uint_as_float((j & 1) ? (u & 0xffff0000u) : (u << 16));
    }
};
template <>
struct Frag<float> {
    f32x4 v[2];
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
// Products with a float operand (mixed: the other one is exact) or two (split: the product of
// the two lo parts, 2^-18 of the whole, is left out) in their parts, one at a time,
// smallest first: a kernel that has several results to add to does one part for all of
// them before the next, so that no instruction waits for the one before it.  Float
// operands have one part.
template <class E>
constexpr int kPartsMixed = sizeof(E) == 2 ? 2 : 1;  // one operand split
template <class E>
constexpr int kPartsSplit = sizeof(E) == 2 ? 3 : 1;  // both
__device__ __forceinline__ f32x4 mma_mixed(int part, const Frag<bf16_t> &a,
                                           const Split<bf16_t> &b, f32x4 c) {
    return part == 0 ? mma(a, b.lo, c) : mma(a, b.hi, c);
}
__device__ __forceinline__ f32x4 mma_mixed(int part, const Split<bf16_t> &a,
                                           const Frag<bf16_t> &b, f32x4 c) {
    return part == 0 ? mma(a.lo, b, c) : mma(a.hi, b, c);
}
__device__ __forceinline__ f32x4 mma_mixed(int, const Frag<float> &a, const Split<float> &b,
                                           f32x4 c) {
    return mma(a, b.hi, c);
}
__device__ __forceinline__ f32x4 mma_mixed(int, const Split<float> &a, const Frag<float> &b,
                                           f32x4 c) {
    return mma(a.hi, b, c);
}
__device__ __forceinline__ f32x4 mma_split(int part, const Split<bf16_t> &a,
                                           const Split<bf16_t> &b, f32x4 c) {
    return part == 0 ? mma(a.lo, b.hi, c) : part == 1 ? mma(a.hi, b.lo, c) : mma(a.hi, b.hi, c);
}
__device__ __forceinline__ f32x4 mma_split(int, const Split<float> &a, const Split<float> &b,
                                           f32x4 c) {
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
// buffer accesses: offsets behind `bytes` read zeros and store nothing, so that
// the last chunk of a sequence needs no branches (the compiler counts the loads in
// flight only through straight code)
// ---------------------------------------------------------------------------
struct Buffer {
    __amdgpu_buffer_rsrc_t r;
    // base and bytes are the same for all lanes, which the compiler does not always
    // see (it would then loop over the lanes at every access)
    __device__ __forceinline__ Buffer(const void *base, unsigned bytes)
        : r(__builtin_amdgcn_make_buffer_rsrc(uniform(base), (short)0,
                                              __builtin_amdgcn_readfirstlane((int)bytes),
                                              0x00020000)) {}
    static __device__ __forceinline__ void *uniform(const void *p) {
        const unsigned long long u = reinterpret_cast<unsigned long long>(p);
        const unsigned lo = (unsigned)__builtin_amdgcn_readfirstlane((int)u),
                       hi = (unsigned)__builtin_amdgcn_readfirstlane((int)(u >> 32));
        return reinterpret_cast<void *>((unsigned long long)hi << 32 | lo);
    }
    __device__ __forceinline__ u32x4 load16(unsigned off) const {
        return __builtin_amdgcn_raw_buffer_load_b128(r, (int)off, 0, 0);
    }
    __device__ __forceinline__ float load_float(unsigned off) const {
        return __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(r, (int)off, 0, 0));
    }
    // four elements
    __device__ __forceinline__ void store4(unsigned off, f32x4 x, bf16_t) const {
        __builtin_amdgcn_raw_buffer_store_b64(u32x2{cvt_pk(x[0], x[1]), cvt_pk(x[2], x[3])}, r,
                                              (int)off, 0, 0);
    }
    __device__ __forceinline__ void store4(unsigned off, f32x4 x, float) const {
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, x), r, (int)off, 0, 0);
    }
    __device__ __forceinline__ void store16(unsigned off, u32x4 x) const {
        __builtin_amdgcn_raw_buffer_store_b128(x, r, (int)off, 0, 0);
    }
};

// ---------------------------------------------------------------------------
// tiles in shared memory: rows of C elements in pieces of 16 bytes, piece s of row
// r at place s ^ f(r).  f gives the 16 rows of a tile_row tile different banks
// for reads along the rows, and the 4 rows x 4 pieces of a transposing read as
// different ones as its half pieces allow.
// ---------------------------------------------------------------------------
template <class E, int C>
struct Tile {
    static constexpr int kPiece = 16 / (int)sizeof(E);          // elements
    static constexpr int kRowPieces = C / kPiece;
    E *p;
    static __device__ __forceinline__ int swizzle(int row) {
        if constexpr (kRowPieces >= 16) return (row & 3) << 2 | (row >> 3 & 3);
        if constexpr (kRowPieces == 8) return (row >> 1 & 1) << 2 | (row >> 3 & 3);
        if constexpr (kRowPieces == 4) return row >> 3 & 3;
        return 0;
    }
    static __device__ __forceinline__ int offset(int row, int col) {
        return row * C + ((col / kPiece) ^ swizzle(row)) * kPiece + col % kPiece;
    }
    // fragment along the rows: lane holds M[row][col0 + 8g + j]
    __device__ __forceinline__ Frag<E> rows(int row, int col0, int g) const {
        Frag<E> f;
        if constexpr (sizeof(E) == 2) {
            f.v = *reinterpret_cast<const u32x4 *>(p + offset(row, col0 + 8 * g));
        } else {
            f.v[0] = *reinterpret_cast<const f32x4 *>(p + offset(row, col0 + 8 * g));
            f.v[1] = *reinterpret_cast<const f32x4 *>(p + offset(row, col0 + 8 * g + 4));
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
        const int g = lane >> 4;
        Frag<E> f;
        if constexpr (sizeof(E) == 2) {
            const u32x2 a = quad<STEP>(row0 + 8 * g, col0, lane),
                        b = quad<STEP>(row0 + 8 * g + 4, col0, lane);
            f.v = u32x4{a[0], a[1], b[0], b[1]};
        } else {
            const int lo = lane & 15, col = col0 + STEP * (lo >> 2) + (lo & 3);
#pragma unroll
            for (int j = 0; j < 8; ++j) f.v[j >> 2][j & 3] = p[offset(row0 + 8 * g + j, col)];
        }
        return f;
    }
    // four rows of one column: lane holds M[row0 + e][c(lo)] (row0 may depend on g)
    template <int STEP>
    __device__ __forceinline__ u32x2 quad(int row0, int col0, int lane) const {
        typedef short s4 __attribute__((ext_vector_type(4)));
        typedef __attribute__((address_space(3))) s4 lds_s4;
        const int lo = lane & 15;
        const E *s = p + offset(row0 + (lo >> 2), col0 + STEP * (lo & 3));
        return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4 *)s));
    }
    template <int STEP>
    __device__ __forceinline__ f32x4 column4(int row0, int col0, int lane) const {
        if constexpr (sizeof(E) == 2) {
            const u32x2 u = quad<STEP>(row0, col0, lane);
            return f32x4{wkv7::bf16_lo(u[0]), wkv7::bf16_hi(u[0]), wkv7::bf16_lo(u[1]),
                         wkv7::bf16_hi(u[1])};
        } else {
            const int lo = lane & 15, col = col0 + STEP * (lo >> 2) + (lo & 3);
            return f32x4{p[offset(row0, col)], p[offset(row0 + 1, col)], p[offset(row0 + 2, col)],
                         p[offset(row0 + 3, col)]};
        }
    }
};
template <class E, int C>
constexpr int tile_bytes(int rows) {
    return rows * C * (int)sizeof(E);
}

// extent of `live` rows (none where it is negative): at most 64 of at most 2^23
// elements, which 32 bits hold
template <class E>
__device__ __forceinline__ unsigned row_bytes(int live, int stride) {
    return (unsigned)(live > 0 ? live : 0) * (unsigned)stride * (unsigned)sizeof(E);
}

// Loads of a [ROWS][C] tile with `stride` elements from row to row, held in
// registers until they are written to shared memory; rows at or behind `live`
// are zeros.  The host refuses strides above 2^23 elements: 64 rows of them are
// 2^31 bytes.
template <class E, int C, int ROWS, int THREADS>
struct Stage {
    static constexpr int kRowPieces = Tile<E, C>::kRowPieces, kPiece = Tile<E, C>::kPiece;
    static constexpr int kPieces = ROWS * kRowPieces;
    static constexpr int kPer = kPieces / THREADS;
    static_assert(kPieces % THREADS == 0, "whole pieces per thread");
    u32x4 x[kPer];
    __device__ __forceinline__ void load(const E *src, int stride, int live, int tid) {
        const Buffer b(src, row_bytes<E>(live, stride));
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int piece = tid + i * THREADS;
            const int row = piece / kRowPieces, col = piece % kRowPieces * kPiece;
            x[i] = b.load16((unsigned)(row * stride + col) * (unsigned)sizeof(E));
        }
    }
    __device__ __forceinline__ void store(Tile<E, C> t, int tid) const {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int piece = tid + i * THREADS;
            *reinterpret_cast<u32x4 *>(
                t.p + t.offset(piece / kRowPieces, piece % kRowPieces * kPiece)) = x[i];
        }
    }
    // the way back: `live` rows of the tile to rows `stride` elements apart
    static __device__ __forceinline__ void store_rows(Tile<E, C> t, E *dst, int stride, int live,
                                                      int tid) {
        const Buffer b(dst, row_bytes<E>(live, stride));
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int piece = tid + i * THREADS;
            const int row = piece / kRowPieces, col = piece % kRowPieces * kPiece;
            b.store16((unsigned)(row * stride + col) * (unsigned)sizeof(E),
                      *reinterpret_cast<const u32x4 *>(t.p + t.offset(row, col)));
        }
    }
};

// A stored state: [V, K] and, in bf16, four more bits of each element behind it
// (gated_delta_kept.h).  A word has eight elements', a row K / 8 words, those of the
// columns 32 ks + 8 g + .. at g K / 32 + ks: so a lane of a chain kernel has its words
// side by side.  They are for <S0, D>, a sum of V K products of either sign, of which
// rounded factors would leave 2^-8 of their size, however small the sum.
template <class E, int K>
__device__ __forceinline__ size_t kept_size(int V) {
    return (size_t)V * (sizeof(E) == 2 ? K + K / 4 : K);
}

// Stores a wave's 16 values of 64 tokens, which lie in result tiles [tokens, values],
// by way of 16 columns of shared memory that are its own: pieces of 16 bytes, where
// the lanes' single elements would be four rows of 32 bytes an instruction.
template <class E, int C>
__device__ __forceinline__ void store_values(const f32x4 (&x)[4], Tile<E, C> t, int col0,
                                             const Buffer &b, int stride, int lane) {
    constexpr int kPiece = Tile<E, C>::kPiece, kRowPieces = 16 / kPiece;
    const int g = lane >> 4, lo = lane & 15;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e = 0; e < 4; e += 2) {
            const int row = tile_row(i, 4 * g + e);
            if constexpr (sizeof(E) == 2) {
                const unsigned u = cvt_pk(x[i][e], x[i][e + 1]);
                t.p[t.offset(row, col0 + lo)] = (bf16_t)u;
                t.p[t.offset(row + 1, col0 + lo)] = (bf16_t)(u >> 16);
            } else {
                t.p[t.offset(row, col0 + lo)] = x[i][e];
                t.p[t.offset(row + 1, col0 + lo)] = x[i][e + 1];
            }
        }
#pragma unroll
    for (int j = 0; j < kRowPieces; ++j) {
        const int piece = lane + 64 * j, row = piece / kRowPieces, col = piece % kRowPieces * kPiece;
        b.store16((unsigned)(row * stride + col) * (unsigned)sizeof(E),
                  *reinterpret_cast<const u32x4 *>(t.p + t.offset(row, col0 + col)));
    }
}

// Reciprocal norms of 64 rows, four lanes of 256 threads per row (1 without
// normalisation; 0 for the rows behind the sequence's end).
template <class E, int K>
__device__ __forceinline__ float reciprocal_norm(Tile<E, K> t, bool normalize, int live, int tid) {
    const int row = tid >> 2;
    float a = 0.f;
#pragma unroll
    for (int i = 0; i < K / 32; ++i) {  // pieces of 8 elements, the four lanes side by side
        const Frag<E> f = t.rows(row, 32 * i, tid & 3);
#pragma unroll
        for (int j = 0; j < 8; ++j) a += f.at(j) * f.at(j);
    }
    a += wkv7::dpp_mov<wkv7::kDppQuadXor1>(a);
    a += wkv7::dpp_mov<wkv7::kDppQuadXor2>(a);
    const float r = normalize ? 1.f / sqrtf(a + kNormEps) : 1.f;
    return row < live ? r : 0.f;
}

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
    int n_seq, T, total;
    // Sequence i, its tokens numbered in blocks of `block` tokens (a multiple of
    // 64): the numbers of a sequence's blocks follow each other from slot0 on, and
    // no two sequences share one.
    __device__ __forceinline__ Seq seq(int i, int block) const {
        Seq s;
        if (!cu) {
            s.begin = i * T;
            s.end = s.begin + T;
            s.slot0 = i * ((T + block - 1) / block);
        } else {
            s.begin = clamp_bound(cu[i], total);
            s.end = clamp_bound(cu[i + 1], total);
            if (s.end < s.begin) s.end = s.begin;
            s.slot0 = s.begin / block + i;
        }
        return s;
    }
    // the sequence of a block's number (which may lie behind its last block)
    __device__ __forceinline__ int find(int slot, int block, Seq &s) const {
        int i;
        if (!cu) {
            i = T > 0 ? slot / ((T + block - 1) / block) : slot;
        } else {
            int lo = 0, hi = n_seq - 1;  // the last i with slot0(i) <= slot
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (clamp_bound(cu[mid], total) / block + mid <= slot)
                    lo = mid;
                else
                    hi = mid - 1;
            }
            i = lo;
        }
        s = seq(i, block);
        return i;
    }
};

// Inclusive sums of the chunk's log decays (to the base 2), lane = token, in float64
// and kept as two floats: the decay between two tokens is the power of two of a
// difference of these sums, which in one float would lose what a strong decay
// before both of them took.  exp(-200) is zero in float32, so a log decay below that (-infinity, the
// type's lowest value) is raised to it; a NaN stays one.
constexpr float kLowestLogDecay = -200.f;
template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp_from(double x) {  // 0 where the control has no source
    const unsigned long long u = __builtin_bit_cast(unsigned long long, x);
    const int lo = __builtin_amdgcn_update_dpp(0, (int)u, CTRL, ROWS, 0xF, false);
    const int hi = __builtin_amdgcn_update_dpp(0, (int)(u >> 32), CTRL, ROWS, 0xF, false);
    return __builtin_bit_cast(double, (unsigned long long)(unsigned)lo |
                                          (unsigned long long)(unsigned)hi << 32);
}
struct Sum2 {
    float hi, lo;
};
__device__ __forceinline__ Sum2 scan_decay(float g) {
    double x = g < kLowestLogDecay ? kLowestLogDecay : g;
    x += dpp_from<0x111, 0xF>(x);  // row_shr 1, 2, 4, 8: within 16 lanes
    x += dpp_from<0x112, 0xF>(x);
    x += dpp_from<0x114, 0xF>(x);
    x += dpp_from<0x118, 0xF>(x);
    x += dpp_from<0x142, 0xA>(x);  // lane 15 of rows 0 and 2 to rows 1 and 3
    x += dpp_from<0x143, 0xC>(x);  // lane 31 to rows 2 and 3
    x *= 1.4426950408889634;
    const float hi = (float)x;
    return Sum2{hi, (float)(x - hi)};
}
// value of lane 63 in all lanes
__device__ __forceinline__ float last_lane(float x) {
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(x), 63));
}
__device__ __forceinline__ Sum2 last_lane(Sum2 x) { return Sum2{last_lane(x.hi), last_lane(x.lo)}; }
__device__ __forceinline__ Sum2 lane_of(Sum2 x, int lane) {  // a lane's number for all
    return Sum2{__int_as_float(__builtin_amdgcn_readlane(__float_as_int(x.hi), lane)),
                __int_as_float(__builtin_amdgcn_readlane(__float_as_int(x.lo), lane))};
}
// inclusive sums over the lanes
template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp_from(float x) {
    return __int_as_float(
        __builtin_amdgcn_update_dpp(0, __float_as_int(x), CTRL, ROWS, 0xF, false));
}
__device__ __forceinline__ float scan_lanes(float x) {
    x += dpp_from<0x111, 0xF>(x);
    x += dpp_from<0x112, 0xF>(x);
    x += dpp_from<0x114, 0xF>(x);
    x += dpp_from<0x118, 0xF>(x);
    x += dpp_from<0x142, 0xA>(x);
    x += dpp_from<0x143, 0xC>(x);
    return x;
}
__device__ __forceinline__ float decay(Sum2 to, Sum2 from) {
    return __builtin_amdgcn_exp2f((to.hi - from.hi) + (to.lo - from.lo));
}
__device__ __forceinline__ float decay(Sum2 to) { return __builtin_amdgcn_exp2f(to.hi + to.lo); }

// Value of lane N of each row of 16 lanes, for a product's operand (DPP row_newbcast).
// A wave that keeps a number per token in the lane own_token(lane) has those of the
// four tokens of a result tile i, element e, in lane 4 i + e of its row.
template <int N>
__device__ __forceinline__ float row_bcast(float x) {
    return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(x), 0x150 + N, 0xF, 0xF, true));
}
__device__ __forceinline__ int own_token(int lane) {
    return tile_row((lane & 15) >> 2, 4 * (lane >> 4) + (lane & 3));
}
// the factors of tile I's four tokens
template <int I>
__device__ __forceinline__ f32x4 row_bcast4(float x) {
    return f32x4{row_bcast<4 * I>(x), row_bcast<4 * I + 1>(x), row_bcast<4 * I + 2>(x),
                 row_bcast<4 * I + 3>(x)};
}
__device__ __forceinline__ f32x4 row_bcast4(float x, int i) {  // i known when unrolled
    return i == 0 ? row_bcast4<0>(x) : i == 1 ? row_bcast4<1>(x) : i == 2 ? row_bcast4<2>(x)
                                                                         : row_bcast4<3>(x);
}

// per chunk and value head, written by the preparation kernel
struct Scalars {
    float beta[kChunk];   // write strength (the forward has it in T)
    float kS[kChunk];     // -exp(G_t) / |k_t|, backward: times beta: factor of S0 k_t
    float kD[kChunk];     // exp(G_C - G_t) / |k_t|: factor of k_t in the exit state
    float qS[kChunk];     // scale exp(G_t) / |q_t|: factor of S0 q_t
    float last;           // exp(G_C)
    float pad[3];
};
// in shared memory: the four arrays, a float of each of 256 threads
constexpr int kScalarSpace = 4 * kChunk * 4;

// Fragments of a chunk's 64 x 64 triangular matrices, (tile of rows, 32 columns),
// that are not all zero: six of the lower triangle, six of an upper one.
__device__ constexpr int kLowTile[6] = {0, 1, 2, 2, 3, 3}, kLowStep[6] = {0, 0, 0, 1, 0, 1};
__device__ constexpr int kUpTile[6] = {0, 0, 1, 1, 2, 3}, kUpStep[6] = {0, 1, 0, 1, 1, 1};

// Record of one chunk and value head.  Each fragment is 64 lanes x 16 bytes per
// part.  Forward: T diag(beta) split, P rounded to E (it only enters o).  Backward: T^T and
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
