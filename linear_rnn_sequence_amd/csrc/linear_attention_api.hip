// Host side of linear attention: argument validation and dispatch for the entry points of
// include/linear_attention.h.  Every check runs before anything is enqueued, so a failed call
// launches nothing and writes nothing.
#include <math.h>
#include <stdint.h>

#include <initializer_list>

#include "linear_attention_internal.h"

using namespace lattn;

namespace {

bool aligned(const void *p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
bool aligned16(std::initializer_list<const void *> ps) {
    for (const void *p : ps)
        if (!aligned(p, 16)) return false;
    return true;
}
bool any_null(std::initializer_list<const void *> ps) {
    for (const void *p : ps)
        if (!p) return true;
    return false;
}

// acc *= x, refused where it leaves no room for sums of several
bool mul_ok(size_t &acc, size_t x) {
    if (x != 0 && acc > (SIZE_MAX / 16) / x) return false;
    acc *= x;
    return true;
}

struct Range {
    const void *p;
    size_t bytes;
};
bool overlap(Range a, Range b) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return a.p && b.p && x < y + b.bytes && y < x + a.bytes;
}
// Outputs must not overlap each other or an input.
bool disjoint(std::initializer_list<Range> outs, std::initializer_list<Range> ins) {
    for (const Range *a = outs.begin(); a != outs.end(); ++a) {
        for (const Range *b = a + 1; b != outs.end(); ++b)
            if (overlap(*a, *b)) return false;
        for (const Range &b : ins)
            if (overlap(*a, b)) return false;
    }
    return true;
}

size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

// Sizes in bytes of a problem's tensors.
struct Sizes {
    size_t q, k, v;                     // extent of the strided inputs
    size_t qd, vd;                      // dense [total, Hk, K], [total, Hv, V]
    size_t g;                           // float32 [Hv]
    size_t pool, states;                // float32 [pool, Hv, V, K], [n_seq, Hv, V, K]
    size_t fwd, bwd;                    // workspaces
    size_t b_cot, b_dq, b_dk, b_dg;     // offsets in the backward's
    Segments fseg, bseg;
};

// Checks a problem and fills in what the kernels need.
rwkv7_status check_problem(const linear_attention_problem *in, Problem &p, Sizes &z) {
    if (!in) return RWKV7_ERR_NULL;
    if (in->dt != RWKV7_DT_F32 && in->dt != RWKV7_DT_BF16)
        return in->dt == RWKV7_DT_BF16_W32 ? RWKV7_ERR_UNSUPPORTED : RWKV7_ERR_DTYPE;
    if ((in->K != 64 && in->K != 128) || in->V < 64 || in->V > 256 || in->V % 64)
        return RWKV7_ERR_UNSUPPORTED;
    if (in->n_seq < 1 || in->total < 0 || in->Hk < 1 || in->Hv < 1 || in->Hv % in->Hk ||
        in->pool < 1)
        return RWKV7_ERR_SHAPE;
    if (!in->cu_seqlens && in->total % in->n_seq) return RWKV7_ERR_SHAPE;
    if ((!in->slots_in || !in->slots_out) && in->pool < in->n_seq) return RWKV7_ERR_SHAPE;
    const int esz = in->dt == RWKV7_DT_BF16 ? 2 : 4;
    p = Problem{};
    p.cu = in->cu_seqlens;
    p.n_seq = in->n_seq; p.total = in->total;
    p.T = p.cu ? 0 : p.total / p.n_seq;
    const long long dense_k = (long long)in->Hk * in->K, dense_v = (long long)in->Hv * in->V;
    const long long q_stride = in->q_stride ? in->q_stride : dense_k,
                    k_stride = in->k_stride ? in->k_stride : dense_k,
                    v_stride = in->v_stride ? in->v_stride : dense_v;
    const long long limit = (long long)1 << 23;  // offsets inside a chunk fit 32 bits
    if (q_stride < dense_k || k_stride < dense_k || v_stride < dense_v || q_stride > limit ||
        k_stride > limit || v_stride > limit)
        return RWKV7_ERR_SHAPE;
    if (q_stride * esz % 16 || k_stride * esz % 16 || v_stride * esz % 16)
        return RWKV7_ERR_ALIGN;
    p.Hk = in->Hk; p.K = in->K;
    // Heads of 192 values are three of 64, for every launch has heads of one size.  A prompt is no slower
    // for it by the value, gradients are twice as slow: dq and dk are float rows of each part, to be added
    // up, and have 64 columns of the state (8 x 2048 tokens, 32 heads of 128 keys: 223 us forward and
    // 1564 backward, where 128 values take 158 and 505, 256 in two parts 238 and 1325).
    p.V = in->V % 128 ? 64 : 128;
    p.parts = in->V / p.V;
    p.heads = in->Hv * p.parts;
    if ((long long)p.heads * p.K > limit) return RWKV7_ERR_SHAPE;
    p.q_stride = (int)q_stride; p.k_stride = (int)k_stride; p.v_stride = (int)v_stride;
    p.slots_in = in->slots_in; p.slots_out = in->slots_out;
    p.pool = in->pool;
    p.scale = in->scale;
    p.bf16 = in->dt == RWKV7_DT_BF16;
    if (!aligned(p.cu, 4) || !aligned(p.slots_in, 4) || !aligned(p.slots_out, 4))
        return RWKV7_ERR_ALIGN;

    const size_t total = (size_t)p.total;
    auto extent = [&](long long stride, long long dense, size_t &bytes) {
        bytes = total ? total - 1 : 0;
        if (!mul_ok(bytes, (size_t)stride)) return false;
        bytes += total ? (size_t)dense : 0;
        return mul_ok(bytes, (size_t)esz);
    };
    if (!extent(q_stride, dense_k, z.q) || !extent(k_stride, dense_k, z.k) ||
        !extent(v_stride, dense_v, z.v) || !extent(dense_k, dense_k, z.qd) ||
        !extent(dense_v, dense_v, z.vd))
        return RWKV7_ERR_SHAPE;
    z.g = (size_t)in->Hv * 4;
    size_t state = 4;
    if (!mul_ok(state, (size_t)p.heads) || !mul_ok(state, (size_t)p.V * p.K)) return RWKV7_ERR_SHAPE;
    z.pool = z.states = state;
    if (!mul_ok(z.pool, (size_t)p.pool) || !mul_ok(z.states, (size_t)p.n_seq)) return RWKV7_ERR_SHAPE;
    z.fseg = plan_segments(p, false);
    z.bseg = plan_segments(p, true);
    size_t fwd = z.fseg.seg ? state : 0, bwd = z.bseg.seg ? state : 0;
    size_t rows = p.rep() > 1 ? 4 : 0, dg = 8;
    if (!mul_ok(fwd, (size_t)z.fseg.units) || !mul_ok(bwd, (size_t)z.bseg.units) ||
        !mul_ok(rows, total) || !mul_ok(rows, (size_t)p.heads * p.K) ||
        !mul_ok(dg, (size_t)z.bseg.units) || !mul_ok(dg, (size_t)p.heads))
        return RWKV7_ERR_SHAPE;
    z.fwd = fwd;
    z.b_cot = up256(bwd);
    z.b_dq = 2 * z.b_cot;
    z.b_dk = z.b_dq + up256(rows);
    z.b_dg = z.b_dk + up256(rows);
    z.bwd = z.b_dg + dg;
    // Every grid's extent in threads fits 32 bits: of the passes, 16 rows of a state a wave, and of
    // single tokens, 16 numbers of a state a thread.  (A combination of segments, 4 a thread, is
    // launched for fewer than 256 sequences and heads only.)
    const size_t threads = 4 * (size_t)(p.V > p.K ? p.V : p.K), most = 0xffffffffu;
    if ((size_t)z.fseg.units * p.heads > most / threads ||
        (size_t)z.bseg.units * p.heads > most / threads || z.states / 64 > most)
        return RWKV7_ERR_SHAPE;
    return RWKV7_OK;
}

rwkv7_status done(hipError_t e) { return e == hipSuccess ? RWKV7_OK : RWKV7_ERR_HIP; }

}  // namespace

extern "C" {

size_t linear_attention_forward_workspace(const linear_attention_problem *in) {
    Problem p;
    Sizes z{};
    return check_problem(in, p, z) == RWKV7_OK ? z.fwd : 0;
}

size_t linear_attention_backward_workspace(const linear_attention_problem *in) {
    Problem p;
    Sizes z{};
    return check_problem(in, p, z) == RWKV7_OK ? z.bwd : 0;
}

rwkv7_status linear_attention_forward(const linear_attention_problem *in, const void *q,
                                      const void *k, const void *v, const float *g,
                                      const float *s0, void *o, float *s_out, void *workspace,
                                      size_t workspace_bytes, void *stream) {
    ForwardArgs a{};
    Sizes z{};
    const rwkv7_status st = check_problem(in, a.p, z);
    if (st != RWKV7_OK) return st;
    if (!g || (a.p.total > 0 && any_null({q, k, v, o}))) return RWKV7_ERR_NULL;
    if (!aligned16({q, k, v, s0, o, s_out, workspace}) || !aligned(g, 4)) return RWKV7_ERR_ALIGN;
    if (z.fwd && (!workspace || workspace_bytes < z.fwd)) return RWKV7_ERR_WORKSPACE;
    const size_t n = (size_t)a.p.n_seq * 4;
    if (!disjoint({{o, z.vd}, {s_out, z.pool}, {workspace, z.fwd}},
                  {{q, z.q}, {k, z.k}, {v, z.v}, {g, z.g}, {s0 == s_out ? nullptr : s0, z.pool},
                   {a.p.cu, n + 4}, {a.p.slots_in, n}, {a.p.slots_out, n}}) ||
        // (the states that the call starts from, where it writes them too)
        (s0 == s_out && !disjoint({{o, z.vd}, {workspace, z.fwd}}, {{s0, z.pool}})))
        return RWKV7_ERR_ALIAS;
    a.seg = z.fseg;
    a.q = q; a.k = k; a.v = v; a.g = g;
    a.s0 = s0; a.o = o; a.s_out = s_out;
    a.states = static_cast<float *>(workspace);
    return done(launch_forward(a, static_cast<hipStream_t>(stream)));
}

rwkv7_status linear_attention_decode(const linear_attention_problem *in, const void *q,
                                     const void *k, const void *v, const float *g, float *state,
                                     void *o, void *stream) {
    DecodeArgs a{};
    Sizes z{};
    const rwkv7_status st = check_problem(in, a.p, z);
    if (st != RWKV7_OK) return st;
    if (a.p.cu || a.p.total != a.p.n_seq || a.p.slots_in != a.p.slots_out) return RWKV7_ERR_SHAPE;
    if (any_null({q, k, v, g, state, o})) return RWKV7_ERR_NULL;
    if (!aligned16({q, k, v, state, o}) || !aligned(g, 4)) return RWKV7_ERR_ALIGN;
    if (!disjoint({{o, z.vd}, {state, z.pool}}, {{q, z.q}, {k, z.k}, {v, z.v}, {g, z.g},
                                                 {a.p.slots_in, (size_t)a.p.n_seq * 4}}))
        return RWKV7_ERR_ALIAS;
    a.q = q; a.k = k; a.v = v; a.g = g;
    a.state = state; a.o = o;
    return done(launch_decode(a, static_cast<hipStream_t>(stream)));
}

rwkv7_status linear_attention_backward(const linear_attention_problem *in, const void *q,
                                       const void *k, const void *v, const float *g,
                                       const void *d_o, const float *s0, const float *ds_T,
                                       void *dq, void *dk, void *dv, float *dg, float *ds0,
                                       void *workspace, size_t workspace_bytes, void *stream) {
    BackwardArgs a{};
    Sizes z{};
    const rwkv7_status st = check_problem(in, a.p, z);
    if (st != RWKV7_OK) return st;
    if (a.p.slots_in || a.p.slots_out) return RWKV7_ERR_UNSUPPORTED;
    if (!g || (a.p.total > 0 && any_null({q, k, v, d_o, dq, dk, dv}))) return RWKV7_ERR_NULL;
    if (!aligned16({q, k, v, d_o, s0, ds_T, dq, dk, dv, ds0, workspace}) || !aligned(g, 4) ||
        !aligned(dg, 4))
        return RWKV7_ERR_ALIGN;
    if (!workspace || workspace_bytes < z.bwd) return RWKV7_ERR_WORKSPACE;
    if (!disjoint({{dq, z.qd}, {dk, z.qd}, {dv, z.vd}, {dg, z.g}, {ds0, z.states},
                   {workspace, z.bwd}},
                  {{q, z.q}, {k, z.k}, {v, z.v}, {g, z.g}, {d_o, z.vd}, {s0, z.states},
                   {ds_T == ds0 ? nullptr : ds_T, z.states}, {a.p.cu, (size_t)a.p.n_seq * 4 + 4}}))
        return RWKV7_ERR_ALIAS;
    a.seg = z.bseg;
    a.q = q; a.k = k; a.v = v; a.g = g; a.d_o = d_o; a.s0 = s0; a.ds_T = ds_T;
    a.dq = dq; a.dk = dk; a.dv = dv; a.dg = dg; a.ds0 = ds0;
    char *ws = static_cast<char *>(workspace);
    a.states = reinterpret_cast<float *>(ws);
    a.cotangents = reinterpret_cast<float *>(ws + z.b_cot);
    a.dq_heads = reinterpret_cast<float *>(ws + z.b_dq);
    a.dk_heads = reinterpret_cast<float *>(ws + z.b_dk);
    a.dg_units = dg ? reinterpret_cast<double *>(ws + z.b_dg) : nullptr;
    return done(launch_backward(a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
