// Group norm of rows with an activation or gate, forward and backward (include/group_norm.h).
//
// A team of L lanes (a power of two) has one group of one row: each lane NV pieces of VEC
// elements, the lanes' pieces side by side, so that neighbouring teams, which have
// neighbouring groups, read whole lines.  The group lies in registers: mean, then the
// variance from the differences to it, then the output, with one read and one write of
// memory.  Sums over the team are DPP moves and lane swaps.
//
// Forward: y = n act(gate) or act(n), n = u w + b, u = (x - mean) rstd.
// Backward, with the same values formed again from x:
//   dn = dy act(gate) or dy act'(n),  dgate = dy n act'(gate),  du = dn w,
//   dx = rstd (du - mean(du) - u mean(du u)),   dw = sum over rows of dn u,  db = of dn.
// Workgroups keep their groups for many rows, whose sums of dw and db they write as one row of the
// workspace; sum_kernel adds those in a fixed order.
//
// What bounds it: memory.  32768 rows of 32 groups of 128 channels with a gate (bf16, 805 MB) take
// 144 us, 5.6 TB/s, where a large copy reaches 6.6; the gradients of 8191 rows of 40 groups of 64
// (210 MB) 34 us, 6.2 TB/s, and 4 for the sums, with the vector units busy 82% of the time (95% in the
// forward of the same rows).  In float the same rows take 303 us forward, 5.3 TB/s, and 70 for the
// gradients, 6.0.  Groups read by one element or two (16384 rows, bf16, 40 groups of 99, 8 of 513, 80 of
// 50, 32 of 130) run at 3.4 to 3.9 TB/s forward and 2.0 to 3.2 backward: four or eight times the loads.
#include <stdint.h>

#include <initializer_list>
#include <type_traits>

#include "group_norm.h"
#include "wkv7_device.h"
#include "wkv7_mfma.h"

namespace gnorm {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxSize = 1024;

struct Args {
    const void *x, *gate, *dy;
    const float *weight, *bias;
    void *y, *dx, *dgate;
    float *sums;  // [chunks, 2, C]
    long long rows, x_stride, gate_stride;
    int groups, size, act;
    int per_team;  // rows of a team; backward: of a workgroup
    int tile;      // backward: groups of a workgroup
    float eps, inv_size;
    bool rms;
};

// sum over the L lanes of a team, in all of them
template <int L>
__device__ __forceinline__ float team_sum(float x) {
    x = L == 8 ? wkv7::sum_lanes8(x) : wkv7::sum_lanes16(x);
    if constexpr (L >= 32) x = wkv7::swap16_add(x, x);
    if constexpr (L >= 64) x = wkv7::swap32_add(x, x);
    return x;
}

// VEC elements of type E as they lie in memory
template <class E, int VEC>
struct alignas(sizeof(E) * VEC) Raw {
    E e[VEC];
};
__device__ __forceinline__ float widen(uint16_t x) { return __uint_as_float((uint32_t)x << 16); }
__device__ __forceinline__ float widen(float x) { return x; }
template <int VEC>
__device__ __forceinline__ void narrow(Raw<uint16_t, VEC> &r, const float (&x)[VEC]) {
    if constexpr (VEC == 1) {
        r.e[0] = (uint16_t)wkv7::f32_to_bf16_rne(x[0]);
    } else {
        unsigned u[VEC / 2];
#pragma unroll
        for (int i = 0; i < VEC / 2; ++i) u[i] = wkv7::cvt_pk(x[2 * i], x[2 * i + 1]);
        __builtin_memcpy(&r, u, sizeof(r));
    }
}
template <int VEC>
__device__ __forceinline__ void narrow(Raw<float, VEC> &r, const float (&x)[VEC]) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) r.e[i] = x[i];
}

// a store of what nobody reads soon (2% of a large call)
template <class V>
__device__ __forceinline__ void put(V *p, const V &x) {
    typedef unsigned u4 __attribute__((ext_vector_type(4)));
    if constexpr (sizeof(V) == 16)
        __builtin_nontemporal_store(__builtin_bit_cast(u4, x), reinterpret_cast<u4 *>(p));
    else
        *p = x;
}
// the lane's channels of weight or bias (one address for each piece of VEC, as wide loads)
template <int VEC, int NV>
__device__ __forceinline__ void channels(float (&x)[VEC * NV], const float *p, const int (&col)[NV],
                                         float otherwise) {
#pragma unroll
    for (int i = 0; i < VEC * NV; ++i) x[i] = otherwise;
    if (p)
#pragma unroll
        for (int v = 0; v < NV; ++v) __builtin_memcpy(&x[v * VEC], p + col[v], VEC * sizeof(float));
}

// sigmoid.  For rows of 8 bits the hardware's exponential and reciprocal: off by 2^-22 of itself, and
// where x is negative by 1.25 |x| 2^-24 more, since the exponent log2(e) x is a float (2^-19.4 at
// x = -20, 2^-17.4 at -80).  Outputs of bf16 are rounded by up to 2^-8; the float gradients of weight
// and bias, formed from the same rows, take it as it is.
template <class E>
__device__ __forceinline__ float sigmoid(float x) {
    if constexpr (sizeof(E) == 2)
        return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-1.4426950408889634f * x));
    return 1.f / (1.f + expf(-x));
}
// silu and sigmoid, and with them their derivatives; `silu` is the same for all lanes.  (s - s^2 is
// off by a few roundings of s: 2^-22 where s is close to 1, and 0 beyond x = 17.)
template <class E>
__device__ __forceinline__ float activate(float x, bool silu) {
    return sigmoid<E>(x) * (silu ? x : 1.f);
}
template <class E>
__device__ __forceinline__ float activate(float x, bool silu, float &slope) {
    const float s = sigmoid<E>(x), d = s - s * s;
    slope = silu ? s + x * d : d;
    return s * (silu ? x : 1.f);
}
// calls f with whether there is no activation, known to the compiler
template <class F>
__device__ __forceinline__ void by_kind(int act, F f) {
    if (act == GROUP_NORM_NONE)
        f(std::integral_constant<bool, true>());
    else
        f(std::integral_constant<bool, false>());
}

// A lane's channels of its team's group.
template <int VEC, int L, int NV, bool FULL>
struct Lane {
    int col[NV];      // first channels of its pieces (of the group's first one where there is none)
    int lane, pieces;
    __device__ __forceinline__ Lane(int group, int size) {
        lane = (int)(threadIdx.x % L);
        pieces = size / VEC;
#pragma unroll
        for (int v = 0; v < NV; ++v) col[v] = group * size + (has(v * VEC) ? v * L + lane : 0) * VEC;
    }
    // whether there is an element i of the lane's
    __device__ __forceinline__ bool has(int i) const { return FULL || i / VEC * L + lane < pieces; }
};

// the statistics of a row: afterwards x holds u
template <int VEC, int L, int NV, bool FULL>
__device__ __forceinline__ void normalize(float (&x)[VEC * NV], float &rstd,
                                          const Lane<VEC, L, NV, FULL> &at, const Args &a) {
    constexpr int N = VEC * NV;
    float mean = 0.f, var = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) mean += x[i];
    mean = a.rms ? 0.f : team_sum<L>(mean) * a.inv_size;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        x[i] = at.has(i) ? x[i] - mean : 0.f;
        var += x[i] * x[i];
    }
    rstd = rsqrtf(team_sum<L>(var) * a.inv_size + a.eps);
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] *= rstd;
}

// One row after the other, the next one on its way meanwhile.  What a team does once (its place,
// weight and bias) takes as long as three rows: 32768 x 32 groups of 128 took 477 us with a team for
// each row, 278 with two rows to a team, 181 with four.  Two or four rows at once are no faster
// (161 and 160 us for 157).
template <class E, int VEC, int L, int NV, bool GATE, bool FULL>
__global__ __launch_bounds__(kThreads) void forward_kernel(Args a) {
    constexpr int N = VEC * NV;
    using V = Raw<E, VEC>;
    const unsigned team = (blockIdx.x * (unsigned)kThreads + threadIdx.x) / L;
    const long long first = (long long)(team / (unsigned)a.groups) * a.per_team;
    if (first >= a.rows) return;
    const Lane<VEC, L, NV, FULL> at((int)(team % (unsigned)a.groups), a.size);
    const int rows = (int)(a.rows - first < a.per_team ? a.rows - first : a.per_team);
    const long long C = (long long)a.groups * a.size;
    const E *xp = static_cast<const E *>(a.x) + first * a.x_stride,
            *gp = static_cast<const E *>(a.gate) + (GATE ? first * a.gate_stride : 0);
    E *yp = static_cast<E *>(a.y) + first * C;
    V rx[NV], rg[NV];
    auto fetch = [&]() {
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            rx[v] = *reinterpret_cast<const V *>(xp + at.col[v]);
            if constexpr (GATE) rg[v] = *reinterpret_cast<const V *>(gp + at.col[v]);
        }
    };
    fetch();
    float w[N], b[N];
    channels<VEC, NV>(w, a.weight, at.col, 1.f);
    channels<VEC, NV>(b, a.bias, at.col, 0.f);
    const bool silu = a.act == GROUP_NORM_SILU;
    for (int row = 0; row < rows; ++row) {
        float u[N], z[N], rstd;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            u[i] = at.has(i) ? widen(rx[i / VEC].e[i % VEC]) : 0.f;
            if constexpr (GATE) z[i] = widen(rg[i / VEC].e[i % VEC]);
        }
        if (row + 1 < rows) {  // (y may be x: not this row again)
            xp += a.x_stride;
            gp += GATE ? a.gate_stride : 0;
            fetch();
        }
        normalize<VEC, L, NV, FULL>(u, rstd, at, a);
        by_kind(a.act, [&](auto none) {
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                float y[VEC];
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    const int k = v * VEC + i;
                    const float n = u[k] * w[k] + b[k];
                    const float g = GATE ? z[k] : n;
                    const float act = none ? g : activate<E>(g, silu);
                    y[i] = GATE ? n * act : act;
                }
                if (at.has(v * VEC)) {
                    V out;
                    narrow(out, y);
                    put(reinterpret_cast<V *>(yp + at.col[v]), out);
                }
            }
        });
        yp += C;
    }
}

// A workgroup has a tile of neighbouring groups for a chunk of rows; its teams take turns with the
// rows, keep the sums of dw and db in registers, and add them up in shared memory at the end, so that
// a chunk leaves one row of the workspace.
template <class E, int VEC, int L, int NV, bool GATE, bool FULL>
__global__ __launch_bounds__(kThreads, VEC == 8 && NV == 1 ? 4 : 1) void backward_kernel(Args a) {
    constexpr int N = VEC * NV, kTeams = kThreads / L;
    using V = Raw<E, VEC>;
    __shared__ float shared[kThreads * (2 * N + 2)];
    const int tiles = a.groups / a.tile, turns = kTeams / a.tile;
    const int team = (int)threadIdx.x / L, turn = team / a.tile;
    const Lane<VEC, L, NV, FULL> at((int)(blockIdx.x % (unsigned)tiles) * a.tile + team % a.tile, a.size);
    const long long chunk = blockIdx.x / (unsigned)tiles, first = chunk * a.per_team + turn;
    const long long end = (chunk + 1) * a.per_team < a.rows ? (chunk + 1) * a.per_team : a.rows;
    const int rows = first < end ? (int)((end - first + turns - 1) / turns) : 0;
    const long long C = (long long)a.groups * a.size;
    const E *xp = static_cast<const E *>(a.x) + first * a.x_stride,
            *gp = static_cast<const E *>(a.gate) + (GATE ? first * a.gate_stride : 0),
            *dp = static_cast<const E *>(a.dy) + first * C;
    E *dxp = static_cast<E *>(a.dx) + first * C,
      *dzp = static_cast<E *>(a.dgate) + (GATE ? first * C : 0);
    float dw[N], db[N];
#pragma unroll
    for (int i = 0; i < N; ++i) dw[i] = db[i] = 0.f;
    V rx[NV], rg[NV], rd[NV];
    auto fetch = [&]() {
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            rx[v] = *reinterpret_cast<const V *>(xp + at.col[v]);
            rd[v] = *reinterpret_cast<const V *>(dp + at.col[v]);
            if constexpr (GATE) rg[v] = *reinterpret_cast<const V *>(gp + at.col[v]);
        }
    };
    const bool silu = a.act == GROUP_NORM_SILU;
    if (rows > 0) fetch();
    float w[N], b[N];
    channels<VEC, NV>(w, a.weight, at.col, 1.f);
    channels<VEC, NV>(b, a.bias, at.col, 0.f);
    for (int row = 0; row < rows; ++row) {
        float u[N], rstd, gate[N], dy[N], dn[N], dz[N];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            u[i] = at.has(i) ? widen(rx[i / VEC].e[i % VEC]) : 0.f;
            dy[i] = at.has(i) ? widen(rd[i / VEC].e[i % VEC]) : 0.f;
            if constexpr (GATE) gate[i] = widen(rg[i / VEC].e[i % VEC]);
        }
        if (row + 1 < rows) {  // (dx may be dy: not this row's again)
            xp += turns * a.x_stride;
            gp += GATE ? turns * a.gate_stride : 0;
            dp += turns * C;
            fetch();
        }
        normalize<VEC, L, NV, FULL>(u, rstd, at, a);
        float sum = 0.f, along = 0.f;
        by_kind(a.act, [&](auto none) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const float n = u[i] * w[i] + b[i];
                float slope = 1.f, act = GATE ? gate[i] : n;
                if constexpr (!none) act = activate<E>(act, silu, slope);
                dn[i] = dy[i] * (GATE ? act : slope);
                if constexpr (GATE) dz[i] = dy[i] * n * slope;
                dw[i] += dn[i] * u[i];
                db[i] += dn[i];
                dn[i] = at.has(i) ? dn[i] * w[i] : 0.f;
                sum += dn[i];
                along += dn[i] * u[i];
            }
        });
        sum = a.rms ? 0.f : team_sum<L>(sum) * a.inv_size;
        along = team_sum<L>(along) * a.inv_size;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            float d[VEC], z[VEC];
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const int k = v * VEC + i;
                d[i] = rstd * (dn[k] - sum - u[k] * along);
                if constexpr (GATE) z[i] = dz[k];
            }
            if (at.has(v * VEC)) {
                V out;
                narrow(out, d);
                put(reinterpret_cast<V *>(dxp + at.col[v]), out);
                if constexpr (GATE) {
                    narrow(out, z);
                    put(reinterpret_cast<V *>(dzp + at.col[v]), out);
                }
            }
        }
        dxp += turns * C;
        dzp += GATE ? turns * C : 0;
    }
    if (!a.sums) return;
    float *mine = shared + threadIdx.x * 4;  // piece j of a thread: 1024 floats further each
#pragma unroll
    for (int i = 0; i < N; ++i) {
        mine[i / 4 * (4 * kThreads) + i % 4] = dw[i];
        mine[(N + i) / 4 * (4 * kThreads) + (N + i) % 4] = db[i];
    }
    __syncthreads();
    if (turn) return;
    for (int t = 1; t < turns; ++t) {
        const float *other = mine + t * a.tile * L * 4;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            dw[i] += other[i / 4 * (4 * kThreads) + i % 4];
            db[i] += other[(N + i) / 4 * (4 * kThreads) + (N + i) % 4];
        }
    }
    float *s = a.sums + chunk * 2 * C;
#pragma unroll
    for (int v = 0; v < NV; ++v)
        if (at.has(v * VEC)) {
            __builtin_memcpy(s + at.col[v], &dw[v * VEC], VEC * sizeof(float));
            __builtin_memcpy(s + C + at.col[v], &db[v * VEC], VEC * sizeof(float));
        }
}

// out[c] = sum over the chunks' rows of column c (a chunk: [2, C], dweight's and dbias').  A wave adds
// every sixteenth row in turn, eight of them on their way at a time (8191 rows of 40 groups of 64:
// 39.2 us for the gradients, 40.9 with each row waited for).
__global__ __launch_bounds__(1024) void sum_kernel(const float *sums, float *dweight, float *dbias,
                                                   int chunks, int C) {
    __shared__ float part[16][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const long long c = (long long)blockIdx.x * 64 + lane;
    float s = 0.f;
    if (c < 2LL * C)
#pragma unroll 8
        for (int i = wave; i < chunks; i += 16) s += sums[(long long)i * 2 * C + c];
    part[wave][lane] = s;
    __syncthreads();
    if (wave == 0 && c < 2LL * C) {
#pragma unroll
        for (int i = 1; i < 16; ++i) s += part[i][lane];
        if (c < C) {
            if (dweight) dweight[c] = s;
        } else if (dbias) {
            dbias[c - C] = s;
        }
    }
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------
struct Shape {
    int L, nv;  // lanes of a team, 8 to 64, and pieces of a lane, both powers of two
};
Shape shape_of(int size, int vec) {
    const int pieces = size / vec;
    Shape s{8, 1};
    while (s.L < 64 && s.L < pieces) s.L *= 2;
    while (s.L * s.nv < pieces) s.nv *= 2;
    return s;
}

bool aligned(const void *p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

struct Checked {
    Args a;
    int esz;
};
rwkv7_status check_problem(const group_norm_problem *in, Checked &c) {
    if (!in) return RWKV7_ERR_NULL;
    if (in->dt != RWKV7_DT_F32 && in->dt != RWKV7_DT_BF16)
        return in->dt == RWKV7_DT_BF16_W32 ? RWKV7_ERR_UNSUPPORTED : RWKV7_ERR_DTYPE;
    if (in->activation < GROUP_NORM_NONE || in->activation > GROUP_NORM_SIGMOID || in->size > kMaxSize)
        return RWKV7_ERR_UNSUPPORTED;
    if (in->rows < 0 || in->rows > 0x7fffffffLL || in->groups < 1 || in->size < 1) return RWKV7_ERR_SHAPE;
    const long long C = (long long)in->groups * in->size, limit = 1LL << 23;
    const long long xs = in->x_stride ? in->x_stride : C, gs = in->gate_stride ? in->gate_stride : C;
    // (rows and strides below 2^31 and 2^23, so that bytes fit 64 bits by far)
    if (C > limit || xs < C || gs < C || xs > limit || gs > limit) return RWKV7_ERR_SHAPE;
    c.a = Args{};
    c.a.rows = in->rows; c.a.groups = in->groups; c.a.size = in->size;
    c.a.x_stride = xs; c.a.gate_stride = gs;
    c.a.eps = in->eps; c.a.inv_size = 1.f / (float)in->size;
    c.a.act = in->activation;
    c.a.rms = in->rms != 0;
    c.esz = in->dt == RWKV7_DT_BF16 ? 2 : 4;
    return RWKV7_OK;
}

// Rows of a workgroup in the backward: about 1024 workgroups, all that the card holds at once, and
// no fewer than four rows to a team (4096 x 32 groups of 128: 31.0 us, with 2048 workgroups 31.8,
// with 512 39); twice as many where a team would have more than 32 rows, since they do not end
// together (32768 x 32 groups of 128: 262 us for 283).  A team that wrote its own sums made the
// gradients of 8191 x 40 groups of 64 take 58 us for 41.  Whatever the alignment: the workspace's
// size goes by it.
constexpr int kBlocks = 1024, kManyRows = 32;
// groups of a workgroup with teams of L lanes: a power of two that divides their number, a quarter
// of its teams at most, so that at least four take turns with the rows where there are so many
int tile_of(int groups, int L) {
    int tile = 1;
    while (tile * 2 <= kThreads / L / 4 && groups % (tile * 2) == 0) tile *= 2;
    return tile;
}
int backward_rows(const Args &a, int esz) {
    const int L = shape_of(a.size, a.size % (16 / esz) ? 1 : 16 / esz).L, tile = tile_of(a.groups, L);
    const long long turns = kThreads / L / tile, most = (a.rows + 4 * turns - 1) / (4 * turns);
    long long chunks = kBlocks / (a.groups / tile);
    if (a.rows > chunks * turns * kManyRows) chunks *= 2;
    chunks = chunks > most ? most : chunks;
    chunks = chunks < 1 ? 1 : chunks;
    const long long n = (a.rows + chunks - 1) / chunks;
    return (int)(n < 1 ? 1 : n);
}
long long chunks_of(const Args &a, int per_team) { return (a.rows + per_team - 1) / per_team; }

size_t extent(long long rows, long long stride, long long C, int esz) {
    return rows ? (size_t)((rows - 1) * stride + C) * esz : 0;
}

struct Range {
    const void *p;
    size_t bytes;
};
bool overlap(Range a, Range b) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return a.p && b.p && x < y + b.bytes && y < x + a.bytes;
}
bool disjoint(std::initializer_list<Range> outs, std::initializer_list<Range> ins) {
    for (const Range *a = outs.begin(); a != outs.end(); ++a) {
        for (const Range *b = a + 1; b != outs.end(); ++b)
            if (overlap(*a, *b)) return false;
        for (const Range &b : ins)
            if (overlap(*a, b)) return false;
    }
    return true;
}

// Elements of a piece: 16 bytes, or two of 16 bits, or one, as group, strides and addresses allow.
int piece(const Args &a, int esz, std::initializer_list<const void *> ps) {
    auto fits = [&](int vec) {
        if (a.size % vec || a.x_stride % vec || (a.gate && a.gate_stride % vec)) return false;
        for (const void *p : ps)
            if (!aligned(p, (size_t)vec * esz)) return false;
        return true;
    };
    return fits(16 / esz) ? 16 / esz : esz == 2 && fits(2) ? 2 : 1;
}

template <class E, int VEC, int L, int NV, bool FULL>
void (*kernel_of(const Args &a, bool backward))(Args) {
    if (backward)
        return a.gate ? &backward_kernel<E, VEC, L, NV, true, FULL>
                      : &backward_kernel<E, VEC, L, NV, false, FULL>;
    return a.gate ? &forward_kernel<E, VEC, L, NV, true, FULL>
                  : &forward_kernel<E, VEC, L, NV, false, FULL>;
}
template <class E, int VEC, int L, int NV>
hipError_t launch(Args a, bool backward, hipStream_t stream) {
    // teams without idle lanes (the usual sizes) need no masks
    void (*kernel)(Args) = nullptr;
    if constexpr (VEC * sizeof(E) == 16)
        if (a.size == VEC * L * NV) kernel = kernel_of<E, VEC, L, NV, true>(a, backward);
    if (!kernel) kernel = kernel_of<E, VEC, L, NV, false>(a, backward);
    unsigned blocks;
    if (backward) {
        a.per_team = backward_rows(a, (int)sizeof(E));
        a.tile = tile_of(a.groups, L);
        blocks = (unsigned)(chunks_of(a, a.per_team) * (a.groups / a.tile));
    } else {
        // as many rows of a team as leave 32 waves for a SIMD (so that every grid's threads fit 32
        // bits, too): 32768 x 32 groups of 128 took 144 us, with sixteen waves 153, with eight 155
        const long long rows = a.rows * a.groups * L / (64LL * 32768);
        a.per_team = (int)(rows < 1 ? 1 : rows);
        blocks = (unsigned)((chunks_of(a, a.per_team) * a.groups * L + kThreads - 1) / kThreads);
    }
    hipLaunchKernelGGL(kernel, dim3(blocks), dim3(kThreads), 0, stream, a);
    return hipGetLastError();
}
template <class E, int VEC>
hipError_t launch(const Args &a, bool backward, hipStream_t stream) {
    const Shape s = shape_of(a.size, VEC);
    if (s.L == 8) return launch<E, VEC, 8, 1>(a, backward, stream);
    if (s.L == 16) return launch<E, VEC, 16, 1>(a, backward, stream);
    if (s.L == 32) return launch<E, VEC, 32, 1>(a, backward, stream);
    if (s.nv == 1) return launch<E, VEC, 64, 1>(a, backward, stream);
    if (s.nv == 2) return launch<E, VEC, 64, 2>(a, backward, stream);
    if constexpr (VEC <= 4)
        if (s.nv == 4) return launch<E, VEC, 64, 4>(a, backward, stream);
    if constexpr (VEC <= 2)
        if (s.nv == 8) return launch<E, VEC, 64, 8>(a, backward, stream);
    if constexpr (VEC == 1)
        if (s.nv == 16) return launch<E, VEC, 64, 16>(a, backward, stream);
    return hipErrorInvalidValue;
}
hipError_t launch(const Args &a, int esz, int vec, bool backward, hipStream_t stream) {
    if (a.rows == 0) return hipSuccess;
    if (esz == 4)
        return vec == 4 ? launch<float, 4>(a, backward, stream) : launch<float, 1>(a, backward, stream);
    if (vec == 8) return launch<uint16_t, 8>(a, backward, stream);
    return vec == 2 ? launch<uint16_t, 2>(a, backward, stream) : launch<uint16_t, 1>(a, backward, stream);
}

}  // namespace
}  // namespace gnorm

using namespace gnorm;

extern "C" {

size_t group_norm_backward_workspace(const group_norm_problem *in) {
    Checked c;
    if (check_problem(in, c) != RWKV7_OK) return 0;
    return (size_t)chunks_of(c.a, backward_rows(c.a, c.esz)) * 2 * c.a.groups * c.a.size * 4;
}

rwkv7_status group_norm_forward(const group_norm_problem *in, const void *x, const void *gate,
                                const float *weight, const float *bias, void *y, void *stream) {
    Checked c;
    const rwkv7_status st = check_problem(in, c);
    if (st != RWKV7_OK) return st;
    Args &a = c.a;
    if (a.rows > 0 && (!x || !y)) return RWKV7_ERR_NULL;
    const size_t esz = (size_t)c.esz;
    if (!aligned(x, esz) || !aligned(gate, esz) || !aligned(y, esz) || !aligned(weight, 4) ||
        !aligned(bias, 4))
        return RWKV7_ERR_ALIGN;
    const long long C = (long long)a.groups * a.size;
    const size_t params = (size_t)C * 4;
    const bool in_place = y == x && a.x_stride == C;
    if (!disjoint({{y, extent(a.rows, C, C, c.esz)}},
                  {{in_place ? nullptr : x, extent(a.rows, a.x_stride, C, c.esz)},
                   {gate, extent(a.rows, a.gate_stride, C, c.esz)}, {weight, params}, {bias, params}}))
        return RWKV7_ERR_ALIAS;
    a.x = x; a.gate = gate; a.weight = weight; a.bias = bias; a.y = y;
    return launch(a, c.esz, piece(a, c.esz, {x, gate, y}), false,
                  static_cast<hipStream_t>(stream)) == hipSuccess
               ? RWKV7_OK
               : RWKV7_ERR_HIP;
}

rwkv7_status group_norm_backward(const group_norm_problem *in, const void *x, const void *gate,
                                 const float *weight, const float *bias, const void *dy, void *dx,
                                 void *dgate, float *dweight, float *dbias, void *workspace,
                                 size_t workspace_bytes, void *stream) {
    Checked c;
    const rwkv7_status st = check_problem(in, c);
    if (st != RWKV7_OK) return st;
    Args &a = c.a;
    if (a.rows > 0 && (!x || !dy || !dx)) return RWKV7_ERR_NULL;
    if (a.rows > 0 && !gate != !dgate) return RWKV7_ERR_NULL;
    const size_t esz = (size_t)c.esz;
    for (const void *p : {x, gate, dy, (const void *)dx, (const void *)dgate})
        if (!aligned(p, esz)) return RWKV7_ERR_ALIGN;
    for (const float *p : {weight, bias, (const float *)dweight, (const float *)dbias})
        if (!aligned(p, 4)) return RWKV7_ERR_ALIGN;
    const int per_team = backward_rows(a, c.esz);
    const long long chunks = chunks_of(a, per_team), C = (long long)a.groups * a.size;
    const bool sums = dweight || dbias;
    const size_t need = sums ? (size_t)chunks * 2 * C * 4 : 0;
    if (need && (!workspace || workspace_bytes < need)) return RWKV7_ERR_WORKSPACE;
    if (!aligned(workspace, 16)) return RWKV7_ERR_ALIGN;
    const size_t params = (size_t)C * 4, dense = extent(a.rows, C, C, c.esz);
    if (!disjoint({{dx, dense}, {dgate, dense}, {dweight, params}, {dbias, params}, {workspace, need}},
                  {{x, extent(a.rows, a.x_stride, C, c.esz)},
                   {gate, extent(a.rows, a.gate_stride, C, c.esz)}, {weight, params}, {bias, params},
                   {dx == dy ? nullptr : dy, dense}}))
        return RWKV7_ERR_ALIAS;
    a.x = x; a.gate = gate; a.weight = weight; a.bias = bias; a.dy = dy;
    a.dx = dx; a.dgate = dgate;
    a.sums = sums ? static_cast<float *>(workspace) : nullptr;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    if (launch(a, c.esz, piece(a, c.esz, {x, gate, dy, dx, dgate}), true, s) != hipSuccess)
        return RWKV7_ERR_HIP;
    if (sums) {
        hipLaunchKernelGGL(sum_kernel, dim3((unsigned)((2 * C + 63) / 64)), dim3(1024), 0, s,
                           static_cast<const float *>(workspace), dweight, dbias, (int)chunks, (int)C);
        if (hipGetLastError() != hipSuccess) return RWKV7_ERR_HIP;
    }
    return RWKV7_OK;
}

}  // extern "C"
