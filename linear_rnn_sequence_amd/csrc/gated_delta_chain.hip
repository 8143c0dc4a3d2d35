// Gated delta rule: the pass over a sequence's chunks that carries the state
// (forward) or its cotangent (backward).
//
// Forward, per chunk with entry state S0 [V, K] and T, P of the preparation
// kernel (c_t = exp(G_t)):
//   R = V - diag(c) K S0^T,  U = T diag(beta) R,
//   O = diag(scale c) Q S0^T + P U,       S_C = c_C S0 + U^T diag(c_C / c) K.
// Backward, with D the cotangent of the chunk's exit state:
//   dU = P^T dO + diag(c_C / c) K D^T,    dR = T^T dU,    dV = diag(beta) dR,
//   dS0 = c_C D + scale dO^T diag(c) Q - dR^T diag(beta c) K.
//
// A wave owns 16 values (rows of the state) over all keys and needs nothing of
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
// float32 results.  So does what enters o, but for P, which is rounded to o's type (its
// other half would be 6 KB more of a chunk's record): o's error is 1.3 times that of its own
// rounding.  With U rounded as well it was 1.6 times that, and the pass took 1 to 2% less
// (16 ragged sequences 197 us for 202, 32768 tokens 788 for 798).
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
    int q_stride, k_stride, v_stride;
    int Hk, Hv, V, pool;
    // segments: tokens of each (a multiple of 64), and per segment number and value
    // head the state left by the segment, [V, K], and its transition, [parts, K, K]
    int seg;
    float *seg_state;
    void *seg_step;
};

__device__ __forceinline__ f32x4 zero() { return f32x4{0.f, 0.f, 0.f, 0.f}; }

template <int K>
struct State {
    f32x4 t[K / 16];
};

template <int K>
__device__ __forceinline__ void clear(State<K> &s) {
#pragma unroll
    for (int m = 0; m < K / 16; ++m) s.t[m] = zero();
}
// rows lo of the 16 at base, keys in tile_row order
template <int K>
__device__ __forceinline__ void load_state(State<K> &s, const float *base, int g, int lo) {
#pragma unroll
    for (int m = 0; m < K / 16; ++m)
        s.t[m] = *reinterpret_cast<const f32x4 *>(base + lo * K + tile_row(m, 4 * g));
}
template <int K>
__device__ __forceinline__ void store_state(const State<K> &s, float *base, int g, int lo) {
#pragma unroll
    for (int m = 0; m < K / 16; ++m)
        *reinterpret_cast<f32x4 *>(base + lo * K + tile_row(m, 4 * g)) = s.t[m];
}
// the same as a stored state (the gradient kernel's operand)
template <class E, int K>
__device__ __forceinline__ void store_kept(const State<K> &s, E *state, int V, int value0, int g,
                                           int lo) {
    constexpr int KS = K / 32;
    E *row = state + (value0 + lo) * K;
    unsigned word[KS];
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
        const f32x4 a = s.t[2 * ks], b = s.t[2 * ks + 1];
        const Frag<E> f = to_frag<E>(a, b);
        E *at = row + 32 * ks + 8 * g;
        if constexpr (sizeof(E) == 2) {
            *reinterpret_cast<u32x4 *>(at) = f.v;
            word[ks] = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e)
                word[ks] |= kept_code(__float_as_uint(e < 4 ? a[e] : b[e - 4])) << 4 * e;
        } else {
            *reinterpret_cast<f32x4 *>(at) = f.v[0];
            *reinterpret_cast<f32x4 *>(at + 4) = f.v[1];
        }
    }
    if constexpr (sizeof(E) == 2) {
        unsigned *at = reinterpret_cast<unsigned *>(state + V * K) + (value0 + lo) * (K / 8) + g * KS;
        if constexpr (KS == 4)
            *reinterpret_cast<u32x4 *>(at) = u32x4{word[0], word[1], word[2], word[3]};
        else
            *reinterpret_cast<u32x2 *>(at) = u32x2{word[0], word[1]};
    }
}
// the same rounded to E (the operand of the combination's products)
template <class E, int K>
__device__ __forceinline__ void store_rounded(const State<K> &s, E *base, int g, int lo) {
#pragma unroll
    for (int ks = 0; ks < K / 32; ++ks) {
        const Frag<E> f = to_frag<E>(s.t[2 * ks], s.t[2 * ks + 1]);
        E *at = base + lo * K + 32 * ks + 8 * g;
        if constexpr (sizeof(E) == 2) {
            *reinterpret_cast<u32x4 *>(at) = f.v;
        } else {
            *reinterpret_cast<f32x4 *>(at) = f.v[0];
            *reinterpret_cast<f32x4 *>(at + 4) = f.v[1];
        }
    }
}

// index of a sequence's state in the pool, or -1
__device__ __forceinline__ int slot_of(const int *slots, int i, int pool) {
    const int s = slots ? slots[i] : i;
    return s >= 0 && s < pool ? s : -1;
}

// Which (sequence or segment, value head, part of the values) a workgroup has.  Workgroups
// go to the 8 XCDs (each with its own L2) in turn, so those that read the same
// k and q rows, the parts of the value heads of one key head, are given numbers
// that are equal modulo 8.
struct Place {
    int unit, hv, part;
};
__device__ __forceinline__ Place place_of(unsigned block, int Hk, int Hv, int parts) {
    const unsigned members = (unsigned)(Hv / Hk * parts), groups = gridDim.x / members;
    const unsigned whole = groups / 8 * 8 * members;
    unsigned group, member;
    if (block < whole) {
        group = block / (8 * members) * 8 + block % 8;
        member = block / 8 % members;
    } else {
        group = groups / 8 * 8 + (block - whole) / members;
        member = (block - whole) % members;
    }
    Place at;
    at.unit = (int)(group / Hk);
    at.hv = (int)(group % Hk) * (Hv / Hk) + (int)(member / parts);
    at.part = (int)(member % parts);
    return at;
}

enum Mode { kInfer, kTrain, kSummary };

// Shared memory of a forward workgroup of W waves: two buffers with a chunk's k and q
// rows and its record (float with 128 keys has room for the record's scalars only),
// and the values.  kSummary has no use for q and P.  In bf16 with 128 keys and eight waves that
// leaves 80 KB of 128, so that a CU has two workgroups, which take turns at waiting: 448
// of them took 328 us, and 367 us one at a time.
template <class E, int K, int W, Mode MODE>
struct ForwardLds {
    static constexpr int kThreads = 64 * W;
    static constexpr int kTile = tile_bytes<E, K>(kChunk);
    static constexpr bool kRecord = sizeof(E) == 2 || K == 64;
    // a record's bytes behind those left out, and where its parts lie in shared memory
    static constexpr int kPBytes = MODE == kSummary ? FwdRecord<E>::kScalars - FwdRecord<E>::kP : 0;
    static constexpr int kScalarsAt = FwdRecord<E>::kScalars - kPBytes;
    static constexpr int kRecPer =
        (FwdRecord<E>::kBytes - kPBytes + 16 * kThreads - 1) / (16 * kThreads);
    static constexpr int kRows = MODE == kSummary ? kTile : 2 * kTile;
    static constexpr int kRest = kRecord ? kRecPer * 16 * kThreads : kScalarSpace;
    static constexpr int kBuffer = kRows + kRest;
    // Values of a chunk: each wave's own, or the workgroup's rows of them, double-buffered,
    // with o in their place afterwards.  The rows make whole lines of memory where a
    // wave's 16 values are pieces of 32 bytes, but pass through shared memory twice more:
    // with 64 keys, where memory is what a chunk waits for, 320 workgroups took
    // 345 us with them and 375 us without; with 128 keys, where shared memory is the
    // busier, 256 took 307 us with them and 278 us without.  In float a piece has 64 bytes.
    static constexpr bool kShared = sizeof(E) == 2 && MODE != kSummary && K == 64;
    static constexpr int kValueCols = kShared ? 16 * W : 16;
    static constexpr int kValueTile = tile_bytes<E, kValueCols>(kChunk);
    static constexpr int kBytes = 2 * kBuffer + (kShared ? 2 : W) * kValueTile;
    static_assert(kBytes <= 160 * 1024, "fits a CU");
    static_assert(kRecord || kThreads == 256, "a float of each thread");
};

// The chunks' shared rows are double-buffered in shared memory: while the waves work
// on chunk c, the rows of c + 1 go from registers to the other buffer and those
// of c + 2 are on their way to the registers.  The chunk's record (T, P and scalars)
// goes the same way: waves that each loaded T and P for themselves kept the CU's
// vector cache busy longer than its matrix cores (where it does not fit, float with
// 128 keys, they still do).  So a load has about one chunk's time to arrive, and
// a chunk needs one barrier.  Loads of chunks behind the last one are buffer
// accesses out of range.
//
// What bounds it: a chunk of 128 keys and 128 values (eight waves, one workgroup per
// CU) takes about 8200 cycles, of which shared memory is busy 55% (20% bank conflicts),
// a SIMD's matrix core 49% and its vector units 42%; the products depend on each other,
// and two waves per SIMD, of 256 registers each, do not overlap them fully.  16 sequences
// of up to 2049 tokens and 32 heads take 141 us, as long as the longest one's chunks
// one after the other.  With 64 keys and values (8 x 4096 tokens, 40 heads: 318 us)
// it is memory: 1.08 GB with the records, 3.4 TB/s, at most one chunk ahead.
//
// A workgroup takes a whole sequence, or one segment of it (p.seg): kSummary only
// carries the state over a segment, from zeros (from the sequence's state for its
// first one), for p.V / (16 W) parts; the parts behind those start from the
// rows of the unit matrix and see no values, which gives the segment's
// transition S0 -> S0 M.  combine_kernel turns these into the states at the
// segments' starts, from which the segments are then done in parallel (32768 tokens, 32
// heads of 128 x 128, eight segments: 325, 25 and 277 us).
template <class E, int K, int W, Mode MODE>
__global__ __launch_bounds__(64 * W, sizeof(E) == 2 ? 2 : 1) void forward_chain_kernel(
    ChainArgs p) {
    using Rec = FwdRecord<E>;
    using L = ForwardLds<E, K, W, MODE>;
    constexpr int KS = K / 32, kTile = L::kTile, kBuffer = L::kBuffer, kThreads = 64 * W;
    constexpr int kValues = 16 * W;
    // stores of an iteration behind its loads: the state (kTrain), u, and float's o
    constexpr int kStores = (MODE == kTrain ? (K / 32 + 2) * (int)sizeof(E) / 2 + 4 / (int)sizeof(E) - 1
                                            : 0) +
                            (L::kShared || MODE == kSummary ? 0 : 4);
    extern __shared__ __align__(16) char lds[];

    const int tid = threadIdx.x, lane = tid & 63,
              wave = __builtin_amdgcn_readfirstlane(tid >> 6), g = lane >> 4, lo = lane & 15;
    const int v_parts = p.V / kValues;
    const Place at = place_of(blockIdx.x, p.Hk, p.Hv,
                              v_parts + (MODE == kSummary ? (K + kValues - 1) / kValues : 0));
    const int hv = at.hv, hk = hv / (p.Hv / p.Hk);
    const bool step = MODE == kSummary && at.part >= v_parts;  // a part of the transition
    const int value0 = (step ? at.part - v_parts : at.part) * kValues + wave * 16;
    const size_t state_size = (size_t)p.V * K;

    // the sequence, and this workgroup's chunks c0 .. c0 + chunks - 1 of it
    Seq sq;
    int seq = at.unit, first = 0, seg_slot = 0, seg_last = 0;
    bool last_part = true;
    if (p.seg) {
        seq = p.lay.find(at.unit, p.seg, sq);
        seg_slot = at.unit;
        const long long ahead = (long long)(at.unit - sq.slot0) * p.seg;
        if (at.unit < sq.slot0 || (ahead >= sq.end - sq.begin && ahead > 0)) return;
        first = (int)ahead;
        seg_last = sq.slot0 + (sq.end - sq.begin - 1) / p.seg;
        last_part = sq.end - sq.begin - first <= p.seg;
        if (MODE == kSummary && (last_part || (step && first == 0))) return;
    }
    sq = p.lay.seq(seq, kChunk);
    const int c0 = first / kChunk;
    const int rest = sq.end - sq.begin - first, len = p.seg && rest > p.seg ? p.seg : rest;
    const int chunks = (len + kChunk - 1) / kChunk;
    const long long token = (long long)sq.begin + first;

    // The start: of a sequence (kept in the place of its last segment's summary, which
    // nothing needs, since s_out may be s_in: the last segment may be done before
    // the first one starts), of a later segment, or zeros.
    State<K> S;
    const float *from = nullptr;
    if (MODE != kSummary && !last_part && !first)
        from = p.seg_state + ((size_t)seg_last * p.Hv + hv) * state_size;
    else if (MODE != kSummary && first)
        from = p.seg_state + ((size_t)(seg_slot - 1) * p.Hv + hv) * state_size;
    else if (p.s_in && !first && !step) {
        const int in = slot_of(p.slots_in, seq, p.pool);
        if (in >= 0) from = p.s_in + ((size_t)in * p.Hv + hv) * state_size;
    }
    if (from) {
        load_state(S, from + (size_t)value0 * K, g, lo);
    } else {
        clear(S);
        if (step)
#pragma unroll
            for (int m = 0; m < K / 16; ++m)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    S.t[m][e] = tile_row(m, 4 * g + e) == value0 + lo ? 1.f : 0.f;
    }

    if (MODE == kSummary && !first)
        store_state(S, p.seg_state + ((size_t)seg_last * p.Hv + hv) * state_size +
                           (size_t)value0 * K, g, lo);

    const E *kp = static_cast<const E *>(p.k) + token * p.k_stride + hk * K;
    const E *qp = static_cast<const E *>(p.q) + token * p.q_stride + hk * K;
    const int vcol = L::kShared ? wave * 16 : 0;  // this wave's values in the tile of them
    const E *vp = static_cast<const E *>(p.v) + token * p.v_stride + hv * p.V +
                  (step ? 0 : value0 - vcol);
    const int row = p.Hv * p.V;  // dense rows of o and u
    E *op = static_cast<E *>(p.out) + token * row + hv * p.V + value0 - vcol;
    E *up = static_cast<E *>(p.mid) + token * row + hv * p.V + value0;
    const size_t rec_step = (size_t)p.Hv * Rec::kBytes;
    const char *rec = p.records + ((size_t)(sq.slot0 + c0) * p.Hv + hv) * Rec::kBytes;
    const size_t kept = kept_size<E, K>(p.V);
    E *states = static_cast<E *>(p.states) + ((size_t)(sq.slot0 + c0) * p.Hv + hv) * kept;
    using Values = Tile<E, L::kValueCols>;

    auto live_of = [&](int c) {
        const int left = len - c * kChunk;
        return left < kChunk ? left : kChunk;  // none or fewer: nothing is in range
    };
    auto buffer = [&](int c) { return lds + (c & 1) * kBuffer; };
    auto values = [&](int c) {
        return Values{reinterpret_cast<E *>(
            lds + 2 * kBuffer + (L::kShared ? c & 1 : wave) * L::kValueTile)};
    };

    Stage<E, K, kChunk, kThreads> gk, gq;
    Stage<E, L::kValueCols, kChunk, L::kShared ? kThreads : 64> gv;
    const int vtid = L::kShared ? tid : lane;
    u32x4 gr[L::kRecPer];
    float gs = 0.f, last_next = 0.f;
    auto fetch_rows = [&](int c) {
        const int live = live_of(c);
        gk.load(kp + (long long)c * kChunk * p.k_stride, p.k_stride, live, tid);
        if (MODE != kSummary)
            gq.load(qp + (long long)c * kChunk * p.q_stride, p.q_stride, live, tid);
    };
    auto fetch_record = [&](int c) {
        const char *r = rec + c * rec_step;
        if constexpr (L::kRecord) {
            const Buffer b(r, c < chunks ? Rec::kBytes : 0);
#pragma unroll
            for (int i = 0; i < L::kRecPer; ++i) {
                const int at = (tid + i * kThreads) * 16;
                gr[i] = b.load16(at < Rec::kP ? at : at + L::kPBytes);
            }
        } else {
            gs = Buffer(r + Rec::kScalars, c < chunks ? kScalarSpace : 0).load_float(tid * 4);
        }
    };
    auto put_rows = [&](int c) {
        char *b = buffer(c);
        gk.store(Tile<E, K>{reinterpret_cast<E *>(b)}, tid);
        if (MODE != kSummary) gq.store(Tile<E, K>{reinterpret_cast<E *>(b + kTile)}, tid);
        if constexpr (L::kRecord) {
#pragma unroll
            for (int i = 0; i < L::kRecPer; ++i)
                *reinterpret_cast<u32x4 *>(b + L::kRows + (tid + i * kThreads) * 16) = gr[i];
        } else {
            reinterpret_cast<float *>(b + L::kRows)[tid] = gs;
        }
    };
    auto fetch_values = [&](int c) {
        gv.load(vp + (long long)c * kChunk * p.v_stride, p.v_stride, step ? 0 : live_of(c), vtid);
        if constexpr (!L::kRecord)
            last_next = Buffer(rec + c * rec_step + Rec::kScalars + kScalarSpace, c < chunks ? 4 : 0)
                            .load_float(0);
    };
    Split<E> T[6];
    Frag<E> P[6];
    auto fetch_T = [&](int c) {
        const char *src = rec + c * rec_step;
#pragma unroll
        for (int f = 0; f < 6; ++f) T[f] = get_split<E>(src + f * Rec::kSplitBytes, lane);
    };
    auto fetch_P = [&](int c) {
        const char *src = rec + c * rec_step + Rec::kP;
#pragma unroll
        for (int f = 0; f < 6; ++f) P[f] = get_frag<E>(src + f * Rec::kFragBytes, lane);
    };
    if (chunks > 0) {
        fetch_rows(0);
        fetch_record(0);
        if constexpr (L::kShared) {
            fetch_values(0);
            gv.store(values(0), vtid);
        }
        put_rows(0);
        fetch_rows(1);
        fetch_record(1);
        fetch_values(L::kShared ? 1 : 0);
        // as many accesses behind these loads as the loop has, so that it waits for no
        // more than it needs
        const Buffer none(op, 0);
#pragma unroll
        for (int i = 0; i < kStores; ++i) none.store16(0, u32x4{0u, 0u, 0u, 0u});
    }
    // o of chunk c from shared memory, by the threads that put values in its place next
    auto store_o = [&](int c) {
        gv.store_rows(values(c), op + (long long)c * kChunk * row, row, c < 0 ? 0 : live_of(c), vtid);
    };
    for (int c = 0; c < chunks; ++c) {
        const int live = live_of(c);
        __syncthreads();  // buffer c is whole, and the other one has been read
        if constexpr (L::kShared) store_o(c - 1);
        put_rows(c + 1);
        if constexpr (L::kShared) gv.store(values(c + 1), vtid);
        if constexpr (!L::kRecord) fetch_T(c);
        fetch_rows(c + 2);
        if constexpr (!L::kShared) fetch_record(c + 2);
        const char *buf = buffer(c);
        const Tile<E, K> tk{reinterpret_cast<E *>(const_cast<char *>(buf))},
            tq{reinterpret_cast<E *>(const_cast<char *>(buf) + kTile)};
        const char *rc = buf + L::kRows;
        const Scalars &sc = *reinterpret_cast<const Scalars *>(L::kRecord ? rc + L::kScalarsAt : rc);
        const Values tv = values(c);
        if constexpr (!L::kShared) gv.store(tv, vtid);  // read by this wave alone
        const float last = L::kRecord ? sc.last : last_next;
        const float kS = sc.kS[own_token(lane)], kD = sc.kD[own_token(lane)];
        if constexpr (!L::kShared) fetch_values(c + 1);

        // X = K S0^T [tokens, values]; O^T = S0 Q^T [values, tokens], so that a lane
        // ends up with four neighbouring values of a token
        f32x4 X[4], O[4], R[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) X[i] = O[i] = zero();
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            Frag<E> fk[4], fq[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                fk[i] = tk.rows(tile_row(i, lo), 32 * ks, g);
                if (MODE != kSummary) fq[i] = tq.rows(tile_row(i, lo), 32 * ks, g);
            }
            const Split<E> b = to_split<E>(S.t[2 * ks], S.t[2 * ks + 1]);
#pragma unroll
            for (int part = 0; part < kPartsMixed<E>; ++part)
#pragma unroll
                for (int i = 0; i < 4; ++i) X[i] = mma_mixed(part, fk[i], b, X[i]);
            if (MODE != kSummary)
#pragma unroll
                for (int part = 0; part < kPartsMixed<E>; ++part)
#pragma unroll
                    for (int i = 0; i < 4; ++i) O[i] = mma_mixed(part, b, fq[i], O[i]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float qs = sc.qS[tile_row(i, lo)];
            R[i] = tv.template column4<4>(tile_row(i, 4 * g), vcol, lane) + row_bcast4(kS, i) * X[i];
            if (MODE != kSummary) O[i] *= qs;
        }
        if (MODE == kTrain)  // (157 us before these products, 138 us here)
            store_kept<E>(S, states + (size_t)c * p.Hv * kept, p.V, value0, g, lo);
        // (keeps what is read from shared memory for the next products out of the
        // registers that these need)
        if (MODE != kSummary) __builtin_amdgcn_sched_barrier(0);
        if constexpr (L::kShared) {  // not all loads at once: 320 workgroups took 317 us, not 340
            fetch_record(c + 2);
            fetch_values(c + 2);
        }
        if constexpr (!L::kRecord && MODE != kSummary) fetch_P(c);
        f32x4 U[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) U[i] = zero();
#pragma unroll
        for (int st = 0; st < 2; ++st) {
            const Split<E> b = to_split<E>(R[2 * st], R[2 * st + 1]);
            if constexpr (L::kRecord)
#pragma unroll
                for (int f = 0; f < 6; ++f)
                    if (kLowStep[f] == st) T[f] = get_split<E>(rc + f * Rec::kSplitBytes, lane);
#pragma unroll
            for (int part = 0; part < kPartsSplit<E>; ++part)
#pragma unroll
                for (int f = 0; f < 6; ++f)
                    if (kLowStep[f] == st)
                        U[kLowTile[f]] = mma_split(part, T[f], b, U[kLowTile[f]]);
        }
        // the state
#pragma unroll
        for (int m = 0; m < K / 16; ++m) S.t[m] *= last;
#pragma unroll
        for (int st = 0; st < 2; ++st) {
            const Split<E> b = to_split<E>(row_bcast4(kD, 2 * st) * U[2 * st],
                                           row_bcast4(kD, 2 * st + 1) * U[2 * st + 1]);
#pragma unroll
            for (int half = 0; half < K / 64; ++half) {  // four tiles of keys at a time
                Frag<E> a[4];
#pragma unroll
                for (int m = 0; m < 4; ++m)
                    a[m] = tk.template cols<8>(32 * st, 64 * half + 32 * (m >> 1) + 4 * (m & 1), lane);
#pragma unroll
                for (int part = 0; part < kPartsMixed<E>; ++part)
#pragma unroll
                    for (int m = 0; m < 4; ++m)
                        S.t[4 * half + m] = mma_mixed(part, a[m], b, S.t[4 * half + m]);
            }
        }
        if (MODE == kTrain) {
            const Buffer bu(up + (long long)c * kChunk * row, row_bytes<E>(live, row));
            store_values(U, tv, vcol, bu, row, lane);
        }
        if (MODE != kSummary) {
            // the readout: O^T += U^T P^T
#pragma unroll
            for (int st = 0; st < 2; ++st) {
                const Split<E> b = to_split<E>(U[2 * st], U[2 * st + 1]);
                if constexpr (L::kRecord)
#pragma unroll
                    for (int f = 0; f < 6; ++f)
                        if (kLowStep[f] == st)
                            P[f] = get_frag<E>(rc + Rec::kP + f * Rec::kFragBytes, lane);
#pragma unroll
                for (int part = 0; part < kPartsMixed<E>; ++part)
#pragma unroll
                    for (int f = 0; f < 6; ++f)
                        if (kLowStep[f] == st)
                            O[kLowTile[f]] = mma_mixed(part, b, P[f], O[kLowTile[f]]);
            }
            if constexpr (L::kShared) {  // in the place of the values
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    *reinterpret_cast<u32x2 *>(tv.p + tv.offset(tile_row(i, lo), vcol + 4 * g)) =
                        u32x2{cvt_pk(O[i][0], O[i][1]), cvt_pk(O[i][2], O[i][3])};
            } else {
                const Buffer bo(op + (long long)c * kChunk * row, row_bytes<E>(live, row));
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    bo.store4((unsigned)(tile_row(i, lo) * row + 4 * g) * (unsigned)sizeof(E), O[i],
                              E());
            }
        }
    }
    if (L::kShared && chunks > 0) {
        __syncthreads();
        store_o(chunks - 1);
    }
    float *to = nullptr;
    if (MODE == kSummary) {
        if (step) {  // the transition's rows, as the operand planes of combine_kernel
            constexpr int kPlanes = sizeof(E) == 2 ? 2 : 1;
            E *plane = static_cast<E *>(p.seg_step) +
                       ((size_t)seg_slot * p.Hv + hv) * (kPlanes * K * K) + (size_t)value0 * K;
            if (value0 < K) {
                store_rounded<E>(S, plane, g, lo);
                if constexpr (kPlanes == 2) {
                    State<K> low;
#pragma unroll
                    for (int ks = 0; ks < KS; ++ks) {
                        const Frag<E> hi = to_frag<E>(S.t[2 * ks], S.t[2 * ks + 1]);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            low.t[2 * ks][e] = S.t[2 * ks][e] - hi.at(e);
                            low.t[2 * ks + 1][e] = S.t[2 * ks + 1][e] - hi.at(4 + e);
                        }
                    }
                    store_rounded<E>(low, plane + K * K, g, lo);
                }
            }
            return;
        }
        to = p.seg_state + ((size_t)seg_slot * p.Hv + hv) * state_size;
    } else if (p.s_out && last_part) {
        const int out = slot_of(p.slots_out, seq, p.pool);
        if (out >= 0) to = p.s_out + ((size_t)out * p.Hv + hv) * state_size;
    }
    if (to) store_state(S, to + (size_t)value0 * K, g, lo);
}

// From the segments' summaries to the states at their ends, in place: the state
// left by segment j - 1 times the transition of segment j, plus what segment j
// leaves from zeros.  One workgroup per sequence, value head and 64 values, a wave
// per 16 (eight waves, half as many workgroups: 33 us for 25); the next transition is
// loaded while this one is multiplied.  A step of 128 keys takes 4 us, most of them
// for the 64 KB of the transition.
constexpr int kThreads = 256, kValues = 64;  // of the kernels below: four waves of 16 values

template <class E, int K>
__global__ __launch_bounds__(kThreads, 1) void combine_kernel(ChainArgs p) {
    constexpr int kPlanes = sizeof(E) == 2 ? 2 : 1;
    extern __shared__ __align__(16) char lds[];
    const int tid = threadIdx.x, lane = tid & 63,
              wave = __builtin_amdgcn_readfirstlane(tid >> 6), g = lane >> 4, lo = lane & 15;
    const Place at = place_of(blockIdx.x, p.Hk, p.Hv, p.V / kValues);
    const Seq sq = p.lay.seq(at.unit, p.seg);
    const int segments = (sq.end - sq.begin + p.seg - 1) / p.seg;
    if (segments < 3) return;  // the first segment's summary is the second's state already
    const size_t state_size = (size_t)p.V * K;
    float *state = p.seg_state + ((size_t)sq.slot0 * p.Hv + at.hv) * state_size +
                   (size_t)(at.part * kValues + wave * 16) * K;
    const E *step = static_cast<const E *>(p.seg_step) +
                    ((size_t)sq.slot0 * p.Hv + at.hv) * (kPlanes * K * K);
    const Tile<E, K> tm[2] = {Tile<E, K>{reinterpret_cast<E *>(lds)},
                              Tile<E, K>{reinterpret_cast<E *>(lds + tile_bytes<E, K>(K))}};
    // the transitions and states of the next steps, on their way (with 128 keys there are
    // registers for one)
    constexpr int kAhead = K == 64 ? 2 : 1;
    Stage<E, K, K, kThreads> gm[kAhead][kPlanes];
    State<K> S, next[kAhead];
    load_state(S, state, g, lo);
    auto fetch = [&](int set, int j) {
#pragma unroll
        for (int x = 0; x < kPlanes; ++x)
            gm[set][x].load(step + (size_t)j * p.Hv * (kPlanes * K * K) + x * K * K, K,
                            j < segments - 1 ? K : 0, tid);
        if (j < segments - 1) load_state(next[set], state + (size_t)j * p.Hv * state_size, g, lo);
    };
    auto one = [&](int set, int j) {
        __syncthreads();
#pragma unroll
        for (int x = 0; x < kPlanes; ++x) gm[set][x].store(tm[x], tid);
        __syncthreads();
        State<K> R = next[set];
        fetch(set, j + kAhead);
#pragma unroll
        for (int ks = 0; ks < K / 32; ++ks) {
            const Split<E> b = to_split<E>(S.t[2 * ks], S.t[2 * ks + 1]);
#pragma unroll
            for (int half = 0; half < K / 64; ++half) {  // four tiles of keys at a time
                Split<E> a[4];
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    const int col = 64 * half + 32 * (m >> 1) + 4 * (m & 1);
                    a[m].hi = tm[0].template cols<8>(32 * ks, col, lane);
                    if constexpr (kPlanes == 2) a[m].lo = tm[1].template cols<8>(32 * ks, col, lane);
                }
#pragma unroll
                for (int part = 0; part < kPartsSplit<E>; ++part)
#pragma unroll
                    for (int m = 0; m < 4; ++m)
                        R.t[4 * half + m] = mma_split(part, a[m], b, R.t[4 * half + m]);
            }
        }
        S = R;
        store_state(S, state + (size_t)j * p.Hv * state_size, g, lo);
    };
#pragma unroll
    for (int x = 0; x < kAhead; ++x) fetch(x, 1 + x);
    for (int j = 1; j < segments - 1; j += kAhead) {
        one(0, j);
        if (kAhead == 2 && j + 1 < segments - 1) one(kAhead - 1, j + 1);
    }
}

// Shared memory of a backward workgroup: as the forward's (four waves: 256 workgroups for
// four sequences of 32 heads of 128 values).
template <class E, int K>
struct BackwardLds {
    static constexpr int kTile = tile_bytes<E, K>(kChunk);
    static constexpr bool kRecord = sizeof(E) == 2 || K == 64;
    static constexpr int kRecPer = (BwdRecord<E>::kBytes + 16 * kThreads - 1) / (16 * kThreads);
    static constexpr int kRest = kRecord ? kRecPer * 16 * kThreads : kScalarSpace;
    static constexpr int kBuffer = 2 * kTile + kRest;
    static constexpr int kBytes = 2 * kBuffer + tile_bytes<E, kValues>(kChunk);
    static_assert(kBytes <= 160 * 1024, "fits a CU");
};

// The same pipeline backwards: the rows of k and q and the record double-buffered; where
// that does not fit (float, 128 keys) T^T and P^T are loaded again as soon as they have been
// used.  It is bound by the length of the chain of products, one wave per SIMD: 4 x 2048
// tokens, 32 heads of 128 x 128, take 163 us, 5.1 us a chunk, where the matrix cores are
// busy 1 us (26 us more before the parts of split products were interleaved, mma_mixed).
template <class E, int K>
__global__ __launch_bounds__(kThreads, 1) void backward_chain_kernel(ChainArgs p) {
    using Rec = BwdRecord<E>;
    using L = BackwardLds<E, K>;
    constexpr int KS = K / 32, kTile = L::kTile, kBuffer = L::kBuffer;
    extern __shared__ __align__(16) char lds[];

    const int tid = threadIdx.x, lane = tid & 63,
              wave = __builtin_amdgcn_readfirstlane(tid >> 6), g = lane >> 4, lo = lane & 15;
    const Place at = place_of(blockIdx.x, p.Hk, p.Hv, p.V / kValues);
    const int hv = at.hv, hk = hv / (p.Hv / p.Hk);
    const int value0 = at.part * kValues + wave * 16;
    const Seq sq = p.lay.seq(at.unit, kChunk);
    const int len = sq.end - sq.begin, chunks = (len + kChunk - 1) / kChunk;
    const size_t state_size = (size_t)p.V * K;
    const Tile<E, 16> to{reinterpret_cast<E *>(lds + 2 * kBuffer) + wave * kChunk * 16};

    State<K> D;
    const size_t state_at = ((size_t)at.unit * p.Hv + hv) * state_size + (size_t)value0 * K;
    if (p.s_in)
        load_state(D, p.s_in + state_at, g, lo);
    else
        clear(D);

    const int row = p.Hv * p.V;
    const E *kp = static_cast<const E *>(p.k) + (long long)sq.begin * p.k_stride + hk * K;
    const E *qp = static_cast<const E *>(p.q) + (long long)sq.begin * p.q_stride + hk * K;
    const E *dop = static_cast<const E *>(p.v) + (long long)sq.begin * row + hv * p.V + value0;
    E *dvp = static_cast<E *>(p.out) + (long long)sq.begin * row + hv * p.V + value0;
    E *drp = static_cast<E *>(p.mid) + (long long)sq.begin * row + hv * p.V + value0;
    const size_t rec_step = (size_t)p.Hv * Rec::kBytes;
    const char *rec = p.records + ((size_t)sq.slot0 * p.Hv + hv) * Rec::kBytes;
    const size_t kept = kept_size<E, K>(p.V);
    E *states = static_cast<E *>(p.states) + ((size_t)sq.slot0 * p.Hv + hv) * kept;

    auto live_of = [&](int c) {
        const int left = c >= 0 ? len - c * kChunk : 0;
        return left < kChunk ? left : kChunk;
    };
    auto buffer = [&](int c) { return lds + (c & 1) * kBuffer; };

    Stage<E, K, kChunk, kThreads> gk, gq;
    Stage<E, 16, kChunk, 64> go;  // this wave's values
    u32x4 gr[L::kRecPer];
    float gs = 0.f, last_next = 0.f;
    Split<E> T[6], P[6];
    auto record = [&](int c) { return rec + (long long)c * (long long)rec_step; };
    auto fetch_rows = [&](int c) {
        const int live = live_of(c);
        gk.load(kp + (long long)c * kChunk * p.k_stride, p.k_stride, live, tid);
        gq.load(qp + (long long)c * kChunk * p.q_stride, p.q_stride, live, tid);
        if constexpr (L::kRecord) {
            const Buffer b(record(c), live > 0 ? Rec::kBytes : 0);
#pragma unroll
            for (int i = 0; i < L::kRecPer; ++i) gr[i] = b.load16((tid + i * kThreads) * 16);
        } else {
            gs = Buffer(record(c) + Rec::kScalars, live > 0 ? kScalarSpace : 0).load_float(tid * 4);
        }
    };
    auto put_rows = [&](int c) {
        char *b = buffer(c);
        gk.store(Tile<E, K>{reinterpret_cast<E *>(b)}, tid);
        gq.store(Tile<E, K>{reinterpret_cast<E *>(b + kTile)}, tid);
        if constexpr (L::kRecord) {
#pragma unroll
            for (int i = 0; i < L::kRecPer; ++i)
                *reinterpret_cast<u32x4 *>(b + 2 * kTile + (tid + i * kThreads) * 16) = gr[i];
        } else {
            reinterpret_cast<float *>(b + 2 * kTile)[tid] = gs;
        }
    };
    auto fetch_values = [&](int c) {
        go.load(dop + (long long)c * kChunk * row, row, live_of(c), lane);
        if constexpr (!L::kRecord)
            last_next =
                Buffer(record(c) + Rec::kScalars + kScalarSpace, c >= 0 ? 4 : 0).load_float(0);
    };
    auto fetch_T = [&](int c) {
        const char *src = rec + (c > 0 ? c : 0) * rec_step;
#pragma unroll
        for (int f = 0; f < 6; ++f) T[f] = get_split<E>(src + f * Rec::kSplitBytes, lane);
    };
    auto fetch_P = [&](int c) {
        const char *src = rec + (c > 0 ? c : 0) * rec_step + Rec::kP;
#pragma unroll
        for (int f = 0; f < 6; ++f) P[f] = get_split<E>(src + f * Rec::kSplitBytes, lane);
    };
    if (chunks > 0) {
        fetch_rows(chunks - 1);
        if constexpr (!L::kRecord) {
            fetch_P(chunks - 1);
            fetch_T(chunks - 1);
        }
        put_rows(chunks - 1);
        fetch_rows(chunks - 2);
        fetch_values(chunks - 1);
        // as many accesses behind these loads as the loop has
        const Buffer none(dvp, 0);
#pragma unroll
        for (int i = 0; i < (K / 32 + 4) * (int)sizeof(E) / 2 + 4 / (int)sizeof(E) - 1; ++i)
            none.store16(0, u32x4{0u, 0u, 0u, 0u});
    }
    for (int c = chunks - 1; c >= 0; --c) {
        const int live = live_of(c);
        __syncthreads();
        put_rows(c - 1);
        fetch_rows(c - 2);
        char *b0 = buffer(c);
        const Tile<E, K> tk{reinterpret_cast<E *>(b0)}, tq{reinterpret_cast<E *>(b0 + kTile)};
        const char *rc = b0 + 2 * kTile;
        const Scalars &sc = *reinterpret_cast<const Scalars *>(L::kRecord ? rc + Rec::kScalars : rc);
        go.store(to, lane);
        const float last = L::kRecord ? sc.last : last_next;
        const float kS = sc.kS[own_token(lane)], kD = sc.kD[own_token(lane)],
                    beta = sc.beta[own_token(lane)];
        fetch_values(c - 1);

        // dU = diag(c_C / c) K D^T + P^T dO
        f32x4 X[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) X[i] = zero();
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            const Split<E> b = to_split<E>(D.t[2 * ks], D.t[2 * ks + 1]);
            Frag<E> fk[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) fk[i] = tk.rows(tile_row(i, lo), 32 * ks, g);
#pragma unroll
            for (int part = 0; part < kPartsMixed<E>; ++part)
#pragma unroll
                for (int i = 0; i < 4; ++i) X[i] = mma_mixed(part, fk[i], b, X[i]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            X[i] *= row_bcast4(kD, i);
        Frag<E> fo[2];
#pragma unroll
        for (int st = 0; st < 2; ++st) fo[st] = to.template cols<4>(32 * st, 0, lane);
        if constexpr (L::kRecord)
#pragma unroll
            for (int f = 0; f < 6; ++f)
                P[f] = get_split<E>(rc + Rec::kP + f * Rec::kSplitBytes, lane);
#pragma unroll
        for (int part = 0; part < kPartsMixed<E>; ++part)
#pragma unroll
            for (int f = 0; f < 6; ++f)
                X[kUpTile[f]] = mma_mixed(part, P[f], fo[kUpStep[f]], X[kUpTile[f]]);
        if constexpr (!L::kRecord) fetch_P(c - 1);
        store_kept<E>(D, states + (size_t)c * p.Hv * kept, p.V, value0, g, lo);
        __builtin_amdgcn_sched_barrier(0);  // as in the forward
        // dR = T^T dU
        f32x4 R[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) R[i] = zero();
#pragma unroll
        for (int st = 0; st < 2; ++st) {
            const Split<E> b = to_split<E>(X[2 * st], X[2 * st + 1]);
            if constexpr (L::kRecord)
#pragma unroll
                for (int f = 0; f < 6; ++f)
                    if (kUpStep[f] == st) T[f] = get_split<E>(rc + f * Rec::kSplitBytes, lane);
#pragma unroll
            for (int part = 0; part < kPartsSplit<E>; ++part)
#pragma unroll
                for (int f = 0; f < 6; ++f)
                    if (kUpStep[f] == st)
                        R[kUpTile[f]] = mma_split(part, T[f], b, R[kUpTile[f]]);
        }
        if constexpr (!L::kRecord) fetch_T(c - 1);
        {
            const Buffer bv(dvp + (long long)c * kChunk * row, row_bytes<E>(live, row)),
                br(drp + (long long)c * kChunk * row, row_bytes<E>(live, row));
            store_values(R, to, 0, br, row, lane);
            f32x4 dv[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) dv[i] = row_bcast4(beta, i) * R[i];
            store_values(dv, to, 0, bv, row, lane);
#pragma unroll
            for (int i = 0; i < 4; ++i) R[i] *= row_bcast4(kS, i);
        }
        // dS0 = c_C D + dO^T diag(scale c / |q|) Q - dR^T diag(beta c / |k|) K
#pragma unroll
        for (int m = 0; m < K / 16; ++m) D.t[m] *= last;
#pragma unroll
        for (int st = 0; st < 2; ++st) {
            const Split<E> b = to_split<E>(R[2 * st], R[2 * st + 1]);
            f32x4 x0 = *reinterpret_cast<const f32x4 *>(sc.qS + 32 * st + 8 * g),
                  x1 = *reinterpret_cast<const f32x4 *>(sc.qS + 32 * st + 8 * g + 4);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                x0[e] *= fo[st].at(e);
                x1[e] *= fo[st].at(4 + e);
            }
            const Split<E> bo = to_split<E>(x0, x1);
#pragma unroll
            for (int half = 0; half < K / 64; ++half) {  // four tiles of keys at a time
                Frag<E> ak[4], aq[4];
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    const int col = 64 * half + 32 * (m >> 1) + 4 * (m & 1);
                    ak[m] = tk.template cols<8>(32 * st, col, lane);
                    aq[m] = tq.template cols<8>(32 * st, col, lane);
                }
#pragma unroll
                for (int part = 0; part < kPartsMixed<E>; ++part)
#pragma unroll
                    for (int m = 0; m < 4; ++m) {
                        f32x4 &d = D.t[4 * half + m];
                        d = mma_mixed(part, ak[m], b, d);
                    }
#pragma unroll
                for (int part = 0; part < kPartsMixed<E>; ++part)
#pragma unroll
                    for (int m = 0; m < 4; ++m) {
                        f32x4 &d = D.t[4 * half + m];
                        d = mma_mixed(part, aq[m], bo, d);
                    }
            }
        }
    }
    if (p.s_out) store_state(D, p.s_out + state_at, g, lo);
}

template <class F>
hipError_t launch(F fn, size_t blocks, int threads, int lds, const ChainArgs &a,
                  hipStream_t stream) {
    const hipError_t e = allow_lds(reinterpret_cast<const void *>(fn), lds);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(fn, dim3((unsigned)blocks), dim3(threads), lds, stream, a);
    return hipGetLastError();
}

template <class E, int K, int W>
hipError_t launch_forward_t(const ChainArgs &a, bool train, int units, int n_seq,
                            hipStream_t stream) {
    const int parts = a.V / (16 * W), step_parts = (K + 16 * W - 1) / (16 * W);
    if (a.seg) {
        hipError_t e = launch(forward_chain_kernel<E, K, W, kSummary>,
                              (size_t)units * a.Hv * (parts + step_parts), 64 * W,
                              ForwardLds<E, K, W, kSummary>::kBytes, a, stream);
        if (e != hipSuccess) return e;
        e = launch(combine_kernel<E, K>, (size_t)n_seq * a.Hv * (a.V / kValues), kThreads,
                   (sizeof(E) == 2 ? 2 : 1) * tile_bytes<E, K>(K), a, stream);
        if (e != hipSuccess) return e;
    }
    return launch(train ? forward_chain_kernel<E, K, W, kTrain>
                        : forward_chain_kernel<E, K, W, kInfer>,
                  (size_t)units * a.Hv * parts, 64 * W, ForwardLds<E, K, W, kInfer>::kBytes, a,
                  stream);
}

template <class E, int K>
hipError_t launch_backward_t(const ChainArgs &a, int n_seq, hipStream_t stream) {
    return launch(backward_chain_kernel<E, K>, (size_t)n_seq * a.Hv * (a.V / kValues),
                  kThreads, BackwardLds<E, K>::kBytes, a, stream);
}

ChainArgs chain_args(const Problem &p) {
    ChainArgs a{};
    a.lay = Layout{p.cu, p.n_seq, p.T, p.total};
    a.q_stride = p.q_stride; a.k_stride = p.k_stride; a.v_stride = p.v_stride;
    a.Hk = p.Hk; a.Hv = p.Hv; a.V = p.V; a.pool = p.pool;
    a.slots_in = p.slots_in; a.slots_out = p.slots_out;
    return a;
}

}  // namespace

// How the forward pass is split.  A workgroup has eight waves where whole ones of 128
// values come out (two waves per SIMD share one copy of the chunk; float tiles
// leave room for four), unless those would be fewer than the CUs: four sequences of 32
// heads and 2048 tokens (training) took 194 us with 128 workgroups of eight, 139 us with
// 256 of four.  Few long sequences are done in segments: an extra pass for the
// segments' summaries costs about what the pass over them does, so there have to be
// four segments a sequence, long enough for the launches: 8 heads of 128 values,
// two sequences of up to 1001 tokens took 102 us whole and 54 us in segments (float), 34 us
// either way with 128 tokens a segment in bf16, which has shorter chunks.  The rule
// goes by the average length, which the host knows also of a packed batch, and does not
// weigh the combination, whose steps follow each other: a long sequence among many short
// ones is done whole, and the more segments a single one has, the longer is that part (4 us
// a step with 128 keys).
Segments plan_segments(const Problem &p) {
    Segments s{};
    s.units = p.n_seq;
    s.waves = p.bf16 && p.V % 128 == 0 ? 8 : 4;
    const long long chains = (long long)p.n_seq * p.Hv * (p.V / (16 * s.waves));
    const long long average = p.total / p.n_seq;
    const int shortest = p.bf16 ? 256 : 64;  // tokens of a segment
    long long n = kCus / chains;             // segments of an average sequence
    if (n > average / shortest) n = average / shortest;
    if (n < 4) {
        if (chains < kCus) s.waves = 4;
        return s;
    }
    const long long len = (average + n - 1) / n;
    s.seg = (int)((len + kChunk - 1) / kChunk * kChunk);
    s.units = p.cu ? p.total / s.seg + p.n_seq : p.n_seq * ((p.T + s.seg - 1) / s.seg);
    const size_t heads = (size_t)s.units * p.Hv;
    s.state_bytes = heads * p.V * p.K * 4;
    s.step_bytes = heads * p.K * p.K * 4;
    return s;
}

hipError_t launch_forward(const ForwardArgs &f, hipStream_t stream) {
    const Problem &p = f.p;
    hipError_t e = launch_prep(p, f.q, f.k, f.g, f.beta, f.records, false, stream);
    if (e != hipSuccess) return e;
    ChainArgs a = chain_args(p);
    a.q = f.q; a.k = f.k; a.v = f.v;
    a.records = f.records;
    a.s_in = f.s0; a.s_out = f.s_out;
    a.out = f.o; a.states = f.s_ckpt; a.mid = f.u;
    const Segments s = plan_segments(p);
    a.seg = s.seg;
    a.seg_state = reinterpret_cast<float *>(f.segments);
    a.seg_step = f.segments + s.state_bytes;
    const bool train = f.s_ckpt != nullptr;
    const int u = s.units, n = p.n_seq;
    if (!p.bf16)
        return p.K == 64 ? launch_forward_t<float, 64, 4>(a, train, u, n, stream)
                         : launch_forward_t<float, 128, 4>(a, train, u, n, stream);
    if (s.waves == 8)
        return p.K == 64 ? launch_forward_t<bf16_t, 64, 8>(a, train, u, n, stream)
                         : launch_forward_t<bf16_t, 128, 8>(a, train, u, n, stream);
    return p.K == 64 ? launch_forward_t<bf16_t, 64, 4>(a, train, u, n, stream)
                     : launch_forward_t<bf16_t, 128, 4>(a, train, u, n, stream);
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
        return p.K == 64 ? launch_backward_t<bf16_t, 64>(a, p.n_seq, stream)
                         : launch_backward_t<bf16_t, 128>(a, p.n_seq, stream);
    return p.K == 64 ? launch_backward_t<float, 64>(a, p.n_seq, stream)
                     : launch_backward_t<float, 128>(a, p.n_seq, stream);
}

}  // namespace gdr
