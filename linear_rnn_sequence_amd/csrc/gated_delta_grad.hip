// Gated delta rule, backward: the gradients of one chunk from its entry state S0,
// its exit cotangent D, and U, dR of every token (all stored by the two chain
// kernels), every chunk in parallel.
//
// With c_t = exp(G_t), E_ts = exp(G_t - G_s), unit vectors or not as the forward:
//   dP = dO U^T (s <= t),  dA = -dR U^T (s < t),
//   MP = dP * scale E,  MA = dA * beta E  (elementwise, beta of the row),
//   dQ = scale diag(c) dO S0 + MP K,
//   dK = -diag(beta c) dR S0 + diag(c_C / c) U D + MP^T Q + MA K + MA^T K,
//   dbeta_t = dR_t . (v_t - c_t S0 k_t) + sum_s dA_ts E_ts k_t . k_s = dR_t . U_t / beta_t,
// and, since the decay at t lies on every path from a token before t (or from
// the entry state) to a token at or behind t (or to the exit state),
//   dg_t = sum_{s < t <= t'} (MP * q.k + MA * k.k)_{t's}
//        + sum_{t' >= t} c_t' (scale dO_t' . S0 q_t' - beta dR_t' . S0 k_t')
//        + sum_{s < t} (c_C / c_s) U_s . D k_s + c_C <D, S0>,
// a sum over a rectangle of pairs, in which nothing cancels (differences of row
// and column sums of the same matrices would).
//
// The second form of dbeta is the diagonal of the product that dA is.  With e = U_t / beta_t
// = v_t - r the error that the token corrects, r what the state recalls, and dR, U, S0
// rounded (bf16), the first is off by d |dR| sqrt(|e|^2 + |r|^2) or so, the second by
// d |dR| |e| sqrt(2), d = 2^-9.8 being a rounding in the mean.  Where the state recalls v well,
// e is a small difference of v and r, of which the first form would leave little: tokens
// with 2 |e|^2 < |v|^2 take the second one, the others the first, and |r| < 2.5 |e| there
// (the first step's values tell the sizes well enough; all of them cost 9 us of 300).
//
// One workgroup of sixteen waves per chunk and key head; it goes through the value
// heads that share the key head and adds their dq and dk up in registers, so no
// atomics are needed and the order of the sums is fixed.  Wave (w, part) owns
// tokens 16w .. 16w + 15 and a quarter of the keys.  Results over keys are kept as
// [keys, tokens] tiles, so that a lane has one token and four neighbouring keys of
// it: factors of the token are one register, and dq, dk leave in pieces of four.
// Parts 0 and 1 form dP and dA with rows s, parts 2 and 3 with rows t (each
// orientation is the operand of one of the products that follow), and pass them to
// the others as operands through shared memory.  All tiles of the triangles are
// formed, also those that are zero: branches around a few matrix products would
// keep the compiler from having their operands in flight together, which costs more.
//
// What is read once per value head (U, dO, dR, S0, D) goes through two buffers in
// steps of 64 values (float: one buffer, 32 values); the next step's pieces are on
// their way to registers while one is multiplied.
//
// What bounds it: 4 x 2048 tokens, 16 key heads of two value heads, 128 x 128 (2048
// workgroups, one at a time on a CU) take 307 us, about 82000 cycles a workgroup.  Its waves
// wait 53% of them; vector units are busy 46%, shared memory 36% (14% bank conflicts), the
// matrix cores 9%.  1.13 GB are moved, 3.7 TB/s, a third of it registers that did not
// fit (39 of 128, 96 bytes a lane).  Shared memory (150 KB) and registers (128 of
// 16 waves) leave no room for a second workgroup, which would fill the waits, nor for loads one step
// further ahead (more spilled registers: 408 us).
#include "gated_delta_device.h"
#include "gated_delta_internal.h"

namespace gdr {
namespace {

constexpr int kPitchM = kChunk + 4;
constexpr int kThreads = 1024;

struct GradArgs {
    Layout lay;
    const void *q, *k, *v, *g, *beta, *d_o, *s_ckpt, *u, *ds, *dr;
    void *dq, *dk, *dg, *dbeta;
    int q_stride, k_stride, v_stride;
    int Hk, Hv, V;
    float scale;
    bool normalize;
};

__device__ __forceinline__ f32x4 zero() { return f32x4{0.f, 0.f, 0.f, 0.f}; }

template <class E, int K>
struct GradLds {
    static constexpr int kVt = 128 / (int)sizeof(E);  // values per step
    static constexpr int kRows = tile_bytes<E, K>(kChunk);
    static constexpr int kO = tile_bytes<E, kVt>(kChunk), kS = tile_bytes<E, K>(kVt);
    static constexpr int kStep = 3 * kO + 2 * kS;
    static constexpr int kBuffers = sizeof(E) == 2 ? 2 : 1;
    // in the place of a head's last step: M, and the waves' 4 x 2 fragments
    static constexpr int kM = kChunk * kPitchM * 4, kFrag = 512 * (int)sizeof(E);
    static constexpr int kAfter = kM + 4 * 8 * kFrag;
    static constexpr int kSpace = kAfter > kStep ? kAfter : kStep;
    static constexpr int kBytes = 2 * kRows + kBuffers * kSpace;
    static_assert(kBytes <= 153 * 1024, "fits a CU, with the arrays of fixed size (6.3 KiB)");
};

// product of two pieces of 16 bytes, element by element
template <class E>
__device__ __forceinline__ float dot_piece(u32x4 a, u32x4 b, float sum) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(E) == 2)
            sum += wkv7::bf16_lo(a[i]) * wkv7::bf16_lo(b[i]) +
                   wkv7::bf16_hi(a[i]) * wkv7::bf16_hi(b[i]);
        else
            sum += __uint_as_float(a[i]) * __uint_as_float(b[i]);
    }
    return sum;
}

// four neighbouring elements of a row
template <class E, int C>
__device__ __forceinline__ f32x4 row4(Tile<E, C> t, int row, int col) {
    const E *s = t.p + t.offset(row, col);
    if constexpr (sizeof(E) == 2) {
        const u32x2 u = *reinterpret_cast<const u32x2 *>(s);
        return f32x4{wkv7::bf16_lo(u[0]), wkv7::bf16_hi(u[0]), wkv7::bf16_lo(u[1]),
                     wkv7::bf16_hi(u[1])};
    } else {
        return *reinterpret_cast<const f32x4 *>(s);
    }
}
__device__ __forceinline__ float dot4(f32x4 a, f32x4 b) {
    return a[0] * b[0] + a[1] * b[1] + a[2] * b[2] + a[3] * b[3];
}

// The same number, unknown to the compiler: addresses made from it are formed where
// they are used instead of being kept in registers across the loops (there are
// hundreds of them, and they would leave no room for the results).
__device__ __forceinline__ int fresh(int x) {
    asm volatile("" : "+v"(x));
    return x;
}

template <class E, int K>
__global__ __launch_bounds__(kThreads) void gradient_kernel(GradArgs p) {
    using L = GradLds<E, K>;
    constexpr int kVt = L::kVt, NK = K / 64;  // tiles of 16 keys of this wave
    extern __shared__ __align__(16) char lds[];
    const Tile<E, K> tk{reinterpret_cast<E *>(lds)}, tq{reinterpret_cast<E *>(lds + L::kRows)};
    __shared__ Sum2 sG[kChunk];
    __shared__ __align__(16) float sBeta[kChunk], sRk[kChunk], sRq[kChunk];
    __shared__ float sGrown[kChunk], sRest[kChunk];
    __shared__ float sEntry[4][kChunk], sLeave[4][kChunk], sKS[4][kChunk], sDb[kChunk],
        sDRV[kChunk], sOwn[kChunk], sSize[2][kChunk], sPairs[kChunk], sDS[16];

    int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, lo = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int w = wave & 3, part = wave >> 2;  // token tile, quarter of the keys
    const int key0 = part * (K / 4);
    int mine = 16 * w + lo;  // this lane's token
    auto refresh = [&]() {
        tid = fresh(tid);
        lane = tid & 63;
        g = lane >> 4;
        lo = lane & 15;
        mine = 16 * w + lo;
    };
    const int slot = (int)(blockIdx.x / p.Hk), hk = (int)(blockIdx.x % p.Hk);
    Seq sq;
    p.lay.find(slot, kChunk, sq);
    const int first = sq.begin + (slot - sq.slot0) * kChunk;
    if (slot < sq.slot0 || first >= sq.end) return;  // the whole workgroup
    const int live = sq.end - first < kChunk ? sq.end - first : kChunk;
    const int rep = p.Hv / p.Hk, row = p.Hv * p.V;
    const int steps = p.V / kVt;

    // The pieces of a step: half of the threads have dO and U, the others dR and v
    // (for their product only); those of S0 and D go to as many as there are.
    constexpr int kStateThreads = L::kS / 16 < kThreads ? L::kS / 16 : kThreads;
    const bool upper = wave >= 8, with_states = wave < kStateThreads / 64;
    Stage<E, kVt, kChunk, 512> ga, gb;
    Stage<E, K, kVt, kStateThreads> gs, gd;
    unsigned ws[gs.kPer], wd[gs.kPer];  // bf16: the pieces' further bits
    auto fetch = [&](int r, int v0) {
        const int hv = hk * rep + r;
        const int in = r < rep ? live : 0, rows = r < rep && with_states ? kVt : 0;
        const size_t at = (size_t)first * row + hv * p.V + v0;
        const size_t state = ((size_t)slot * p.Hv + hv) * kept_size<E, K>(p.V), st = state + (size_t)v0 * K;
        ga.load(static_cast<const E *>(upper ? p.dr : p.d_o) + at, row, in, tid & 511);
        gb.load(upper ? static_cast<const E *>(p.v) + (size_t)first * p.v_stride + hv * p.V + v0
                      : static_cast<const E *>(p.u) + at,
                upper ? p.v_stride : row, in, tid & 511);
        gs.load(static_cast<const E *>(p.s_ckpt) + st, K, rows, tid);
        gd.load(static_cast<const E *>(p.ds) + st, K, rows, tid);
        if constexpr (sizeof(E) == 2) {
            const size_t at = state + (size_t)p.V * K + (size_t)v0 * (K / 4);
            const Buffer bs(static_cast<const E *>(p.s_ckpt) + at, row_bytes<E>(rows, K / 4)),
                bd(static_cast<const E *>(p.ds) + at, row_bytes<E>(rows, K / 4));
#pragma unroll
            for (int i = 0; i < gs.kPer; ++i) {
                const int piece = tid + i * kStateThreads;
                const int row = piece / (K / 8), col = piece % (K / 8);  // in pieces
                const unsigned word = (unsigned)(row * (K / 8) + (col & 3) * (K / 32) + (col >> 2));
                ws[i] = __float_as_uint(bs.load_float(word * 4u));
                wd[i] = __float_as_uint(bd.load_float(word * 4u));
            }
        }
    };
    {
        constexpr int kRowThreads = L::kRows / 16 < kThreads ? L::kRows / 16 : kThreads;
        Stage<E, K, kChunk, kRowThreads> a, b;
        a.load(static_cast<const E *>(p.k) + (long long)first * p.k_stride + hk * K, p.k_stride,
               live, tid);
        b.load(static_cast<const E *>(p.q) + (long long)first * p.q_stride + hk * K, p.q_stride,
               live, tid);
        if (wave < kRowThreads / 64) {
            a.store(tk, tid);
            b.store(tq, tid);
        }
    }
    fetch(0, 0);
    __syncthreads();
    if (wave < 8) {  // 256 threads do k, 256 do q
        const float a = reciprocal_norm(wave < 4 ? tk : tq, p.normalize, live, tid & 255);
        if ((tid & 3) == 0) (wave < 4 ? sRk : sRq)[(tid & 255) >> 2] = a;
    }
    // q.k (part 0) or k.k, rows s in tile_row order, columns t = 16 w + lo
    f32x4 kq[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) kq[i] = zero();
    if (part < 2)
#pragma unroll
        for (int ks = 0; ks < K / 32; ++ks) {
            const Frag<E> b = (part ? tk : tq).rows(mine, 32 * ks, g);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                kq[i] = mma(tk.rows(tile_row(i, lo), 32 * ks, g), b, kq[i]);
        }
    // [keys key0 + 16 n + 4g + e, token 16 w + lo]
    f32x4 dQ[NK], dK[NK];
#pragma unroll
    for (int n = 0; n < NK; ++n) dQ[n] = dK[n] = zero();

    int buffer = 0;
    for (int r = 0; r < rep; ++r) {
        const int hv = hk * rep + r;
        // parts 0, 1: dP^T, -dA^T, rows s; parts 2, 3: dP, -dA, rows t, columns s
        f32x4 oS[NK], rS[NK], uD[NK], P[4];
#pragma unroll
        for (int n = 0; n < NK; ++n) oS[n] = rS[n] = uD[n] = zero();
#pragma unroll
        for (int i = 0; i < 4; ++i) P[i] = zero();
        float ds_sum = 0.f, drv = 0.f;
        float gt = 0.f, bt = 0.f;
        const long long gate_at = (long long)(first + lane) * p.Hv + hv;
        if (wave == 0 && lane < live) {
            gt = to_float(static_cast<const E *>(p.g)[gate_at]);
            bt = to_float(static_cast<const E *>(p.beta)[gate_at]);
        }
        {  // the sizes of U and v, from the first step's values
            const float size = wkv7::sum_lanes8(dot_piece<E>(gb.x[0], gb.x[0], 0.f));
            if ((tid & 7) == 0) sSize[upper][(tid & 511) >> 3] = size;
        }
        char *b0 = lds;
        for (int j = 0; j < steps; ++j) {
            b0 = lds + 2 * L::kRows + (L::kBuffers == 2 ? buffer * L::kSpace : 0);
            buffer ^= 1;
            const Tile<E, kVt> to{reinterpret_cast<E *>(b0)}, tr{reinterpret_cast<E *>(b0 + L::kO)},
                tu{reinterpret_cast<E *>(b0 + 2 * L::kO)};
            const Tile<E, K> ts{reinterpret_cast<E *>(b0 + 3 * L::kO)},
                td{reinterpret_cast<E *>(b0 + 3 * L::kO + L::kS)};
            if (L::kBuffers == 1) __syncthreads();  // the buffer has been read
            refresh();
            ga.store(upper ? tr : to, tid & 511);
            if (!upper) gb.store(tu, tid & 511);
            if (with_states) {
                gs.store(ts, tid);
                gd.store(td, tid);
            }
            if (upper) drv = dot_piece<E>(ga.x[0], gb.x[0], drv);  // eight lanes per token
            unsigned ms[gs.kPer], md[gs.kPer];
#pragma unroll
            for (int i = 0; i < gs.kPer; ++i) {
                if constexpr (sizeof(E) == 2) {
                    ms[i] = ws[i];
                    md[i] = wd[i];
                } else {
                    ds_sum = dot_piece<E>(gs.x[i], gd.x[i], ds_sum);
                }
            }
            if (j + 1 < steps)
                fetch(r, (j + 1) * kVt);
            else
                fetch(r + 1, 0);
            __syncthreads();
            if constexpr (sizeof(E) == 2) {  // S0 D: its own pieces again, the loads are under way
                if (with_states)
#pragma unroll
                    for (int i = 0; i < gs.kPer; ++i) {
                        const int piece = tid + i * kStateThreads;
                        const int at = ts.offset(piece / (K / 8), piece % (K / 8) * 8);
                        const u32x4 s = *reinterpret_cast<const u32x4 *>(ts.p + at),
                                    d = *reinterpret_cast<const u32x4 *>(td.p + at);
#pragma unroll
                        for (int x = 0; x < 8; ++x) {
                            const unsigned a = s[x >> 1], b = d[x >> 1];
                            const unsigned sb = kept_bits(x & 1 ? a & 0xffff0000u : a << 16, ms[i], x),
                                           db = kept_bits(x & 1 ? b & 0xffff0000u : b << 16, md[i], x);
                            ds_sum += __uint_as_float(sb) * __uint_as_float(db);
                        }
                    }
            }
            const Tile<E, kVt> ta = part < 2 ? tu : part == 2 ? to : tr,
                               tb = part == 0 ? to : part == 1 ? tr : tu;
#pragma unroll
            for (int x = 0; x < kVt; x += 32) {
                // (this and the one below keep the operands of only one group of products in
                // registers: 315 us without them, which spilled others)
                __builtin_amdgcn_sched_barrier(0);
                const Frag<E> fo = to.rows(mine, x, g), fr = tr.rows(mine, x, g),
                              fu = tu.rows(mine, x, g);
                Frag<E> as[NK], ad[NK], a[4];
#pragma unroll
                for (int n = 0; n < NK; ++n) {
                    as[n] = ts.template cols<4>(x, key0 + 16 * n, lane);
                    ad[n] = td.template cols<4>(x, key0 + 16 * n, lane);
                }
#pragma unroll
                for (int n = 0; n < NK; ++n) {
                    oS[n] = mma(as[n], fo, oS[n]);
                    rS[n] = mma(as[n], fr, rS[n]);
                    uD[n] = mma(ad[n], fu, uD[n]);
                }
                __builtin_amdgcn_sched_barrier(0);
                const Frag<E> fb = tb.rows(mine, x, g);
#pragma unroll
                for (int i = 0; i < 4; ++i) a[i] = ta.rows(tile_row(i, lo), x, g);
#pragma unroll
                for (int i = 0; i < 4; ++i) P[i] = mma(a[i], fb, P[i]);
            }
        }
        if (wave == 0) {
            const Sum2 G = scan_decay(gt);
            sG[lane] = G;
            sBeta[lane] = bt;
            sGrown[lane] = decay(G);
            sRest[lane] = decay(last_lane(G), G);
        }
        if (upper) {
            drv = wkv7::sum_lanes8(drv);
            if ((tid & 7) == 0) sDRV[(tid & 511) >> 3] = drv;
        }
        ds_sum = wkv7::sum_rows4(wkv7::sum_lanes16(ds_sum));
        if (lane == 0) sDS[wave] = ds_sum;
        __syncthreads();  // also: the last step has been read
        refresh();
        float *sM = reinterpret_cast<float *>(b0);
        char *frags = b0 + L::kM + w * (8 * L::kFrag);  // P^T, A^T, P, A of this token tile
        const Sum2 Gm = sG[mine];
        const float be = sBeta[mine], rk = sRk[mine], rq = sRq[mine];

        {  // what goes through the states; here the lane's token is t
            const float grown = sGrown[mine], rest = sRest[mine], qf = p.scale * grown,
                        kf = -be * grown;
            float oq = 0.f, rkd = 0.f, ud = 0.f;
#pragma unroll
            for (int n = 0; n < NK; ++n) {
                const f32x4 k4 = row4(tk, mine, key0 + 16 * n + 4 * g),
                            q4 = row4(tq, mine, key0 + 16 * n + 4 * g);
                oq += dot4(oS[n], q4);
                rkd += dot4(rS[n], k4);
                ud += dot4(uD[n], k4);
                dQ[n] += qf * oS[n];
                dK[n] += rest * uD[n] + kf * rS[n];
            }
            oq = wkv7::sum_rows4(oq) * qf * rq;
            rkd = wkv7::sum_rows4(rkd) * grown * rk;
            ud = wkv7::sum_rows4(ud) * rest * rk;
            if (g == 0) {
                sEntry[part][mine] = oq - be * rkd;
                sLeave[part][mine] = ud;
                sKS[part][mine] = rkd;
            }
        }
        // the triangles: P becomes this part's operand, kq the pairs' terms of dg
        f32x4 pairs[4];
        if (part < 2) {  // the lane's token is t, rows are s
            if (part) {  // dR_t . U_t: row t is in one lane of the token's four
                const f32x4 a = w < 2 ? P[0] : P[2], b = w < 2 ? P[1] : P[3], x = lo & 4 ? b : a;
                const float y = lo & 1 ? x[1] : x[0], z = lo & 1 ? x[3] : x[2];
                if (g == (mine >> 3 & 3)) sOwn[mine] = lo & 2 ? z : y;
            }
            float db = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const f32x4 rks = *reinterpret_cast<const f32x4 *>(sRk + tile_row(i, 4 * g));
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int t = mine, s = tile_row(i, 4 * g + e);
                    const float E_ts = decay(Gm, sG[s]);
                    const float m = (part ? s < t : s <= t) ? E_ts * P[i][e] : 0.f;
                    const float x = m * kq[i][e] * rks[e];
                    db += x;
                    pairs[i][e] = x;
                    P[i][e] = m * rks[e];
                }
                const float f = part ? -be : p.scale, fx = f * (part ? rk : rq);
                pairs[i] *= fx;
                P[i] *= f;
            }
            if (part) {
                db = -rk * wkv7::sum_rows4(db);
                if (g == 0) sDb[mine] = db;
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    *reinterpret_cast<f32x4 *>(sM + mine * kPitchM + tile_row(i, 4 * g)) = pairs[i];
            }
        } else {  // the lane's token is s, rows are t
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int t0 = tile_row(i, 4 * g);
                const f32x4 f = part == 2 ? p.scale * *reinterpret_cast<const f32x4 *>(sRq + t0)
                                          : -(*reinterpret_cast<const f32x4 *>(sBeta + t0)) *
                                                *reinterpret_cast<const f32x4 *>(sRk + t0);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int s = mine, t = t0 + e;
                    const float E_ts = decay(sG[t], Gm);
                    P[i][e] = (part == 2 ? s <= t : s < t) ? f[e] * E_ts * P[i][e] : 0.f;
                }
            }
        }
#pragma unroll
        for (int st = 0; st < 2; ++st)
            put_frag<E>(frags + (2 * part + st) * L::kFrag, to_frag<E>(P[2 * st], P[2 * st + 1]),
                        lane);
        __syncthreads();
        refresh();
        if (part == 1)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                f32x4 *at = reinterpret_cast<f32x4 *>(sM + mine * kPitchM + tile_row(i, 4 * g));
                *at += pairs[i];
            }
#pragma unroll
        for (int st = 0; st < 2; ++st) {
            Frag<E> f[4], ak[NK], aq[NK];
#pragma unroll
            for (int x = 0; x < 4; ++x) f[x] = get_frag<E>(frags + (2 * x + st) * L::kFrag, lane);
#pragma unroll
            for (int n = 0; n < NK; ++n) {
                ak[n] = tk.template cols<4>(32 * st, key0 + 16 * n, lane);
                aq[n] = tq.template cols<4>(32 * st, key0 + 16 * n, lane);
            }
#pragma unroll
            for (int n = 0; n < NK; ++n) {
                dQ[n] = mma(ak[n], f[0], dQ[n]);
                dK[n] = mma(ak[n], f[1], dK[n]);
                dK[n] = mma(aq[n], f[2], dK[n]);
                dK[n] = mma(ak[n], f[3], dK[n]);
            }
        }
        __syncthreads();
        // sums over the rectangles s < t <= t': down each sixteenth of a column first
        {
            const int s = lane;
            float x[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = sM[(4 * wave + i) * kPitchM + s];
#pragma unroll
            for (int i = 3; i >= 0; --i) {
                x[i] = s < 4 * wave + i ? x[i] : 0.f;
                if (i < 3) x[i] += x[i + 1];
                sM[(4 * wave + i) * kPitchM + s] = x[i];
            }
        }
        __syncthreads();
        {  // sixteen lanes per token; the sums above start at every fourth token
            const int t = tid >> 4, c = tid & 15;
            f32x4 sum = *reinterpret_cast<const f32x4 *>(sM + t * kPitchM + 4 * c);
#pragma unroll
            for (int x = 1; x < 16; ++x)
                if (4 * x > t)
                    sum += *reinterpret_cast<const f32x4 *>(sM + 4 * x * kPitchM + 4 * c);
            float one = 0.f;
#pragma unroll
            for (int e = 0; e < 4; ++e) one += 4 * c + e < t ? sum[e] : 0.f;
            one = wkv7::sum_lanes16(one);
            if (c == 0) sPairs[t] = one;
        }
        __syncthreads();
        if (wave == 0) {
            float entry = 0.f, own = 0.f, ks = 0.f, whole = 0.f;
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                entry += sEntry[x][63 - lane];  // summed from the chunk's end
                own += sLeave[x][lane];
                ks += sKS[x][lane];
            }
#pragma unroll
            for (int x = 0; x < 16; ++x) whole += sDS[x];
            sEntry[0][63 - lane] = scan_lanes(entry);
            entry = sEntry[0][lane];
            const float leave = scan_lanes(own);
            whole *= sGrown[63];
            if (lane < live) {
                static_cast<E *>(p.dg)[gate_at] =
                    from_float<E>(sPairs[lane] + entry + (leave - own) + whole);
                // (a strength whose square, or U, may have lost bits below the smallest normal
                // number takes the first form)
                const float b = sBeta[lane];
                const bool second = fabsf(b) > 0x1p-40f && 2.f * sSize[0][lane] < b * b * sSize[1][lane];
                static_cast<E *>(p.dbeta)[gate_at] =
                    from_float<E>(second ? sOwn[lane] / b : sDRV[lane] - ks + sDb[lane]);
            }
        }
        __syncthreads();  // before the next head's sums take their places
    }

    // the gradient of x / |x| from that of the unit vector, and out
    if (p.normalize) {
        const float rk = sRk[mine], rq = sRq[mine];
        float a = 0.f, b = 0.f;
#pragma unroll
        for (int n = 0; n < NK; ++n) {
            a += dot4(dQ[n], row4(tq, mine, key0 + 16 * n + 4 * g));
            b += dot4(dK[n], row4(tk, mine, key0 + 16 * n + 4 * g));
        }
        a = wkv7::sum_rows4(a);
        b = wkv7::sum_rows4(b);
        if (g == 0) {
            sEntry[part][mine] = a;
            sLeave[part][mine] = b;
        }
        __syncthreads();
        a = (sEntry[0][mine] + sEntry[1][mine] + sEntry[2][mine] + sEntry[3][mine]) * rq * rq;
        b = (sLeave[0][mine] + sLeave[1][mine] + sLeave[2][mine] + sLeave[3][mine]) * rk * rk;
#pragma unroll
        for (int n = 0; n < NK; ++n) {
            dQ[n] = rq * (dQ[n] - a * row4(tq, mine, key0 + 16 * n + 4 * g));
            dK[n] = rk * (dK[n] - b * row4(tk, mine, key0 + 16 * n + 4 * g));
        }
    }
    const int krow = p.Hk * K;
    const Buffer bq(static_cast<E *>(p.dq) + (size_t)first * krow + hk * K, row_bytes<E>(live, krow)),
        bk(static_cast<E *>(p.dk) + (size_t)first * krow + hk * K, row_bytes<E>(live, krow));
#pragma unroll
    for (int n = 0; n < NK; ++n) {
        const unsigned off = (unsigned)(mine * krow + key0 + 16 * n + 4 * g) * (unsigned)sizeof(E);
        bq.store4(off, dQ[n], E());
        bk.store4(off, dK[n], E());
    }
}

template <class E, int K>
hipError_t launch_gradients_t(const GradArgs &a, int slots, hipStream_t stream) {
    constexpr int kLds = GradLds<E, K>::kBytes;
    const auto fn = gradient_kernel<E, K>;
    const hipError_t e = allow_lds(reinterpret_cast<const void *>(fn), kLds);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(fn, dim3((unsigned)((size_t)slots * a.Hk)), dim3(kThreads), kLds, stream, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_gradients(const BackwardArgs &b, hipStream_t stream) {
    const Problem &p = b.p;
    if (p.slots == 0) return hipSuccess;
    GradArgs a{};
    a.lay = Layout{p.cu, p.n_seq, p.T, p.total};
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
