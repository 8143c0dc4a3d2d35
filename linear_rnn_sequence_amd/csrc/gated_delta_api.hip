// Host side of the gated delta rule: argument validation and dispatch for the
// entry points of include/gated_delta.h.  Every check runs before anything is
// enqueued, so a failed call launches nothing and writes nothing.
#include <stdint.h>

#include <initializer_list>

#include "gated_delta_internal.h"

using namespace gdr;

namespace {

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned(const void *p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

bool mul_ok(size_t &acc, size_t x) {
    if (x != 0 && acc > (SIZE_MAX / 4) / x) return false;
    acc *= x;
    return true;
}

struct Range {
    uintptr_t lo, hi;
};
Range range(const void *p, size_t bytes) {
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    return p ? Range{lo, lo + bytes} : Range{0, 0};
}
bool overlap(Range a, Range b) { return a.lo < b.hi && b.lo < a.hi; }

// Sizes in bytes of a problem's tensors.
struct Sizes {
    size_t q, k, v;          // extent of the strided inputs
    size_t qd, vd, gate;     // dense [total, Hk, K], [total, Hv, V], [total, Hv]
    size_t pool, states;     // float32 [pool, Hv, V, K], [n_seq, Hv, V, K]
    size_t ckpt;             // dt [slots, Hv, GATED_DELTA_CKPT_SIZE]
    size_t fwd, bwd;         // workspaces
    size_t fwd_seg;          // offset in the forward's
    size_t bwd_ds, bwd_dr;   // offsets in the backward's
};

size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

// Checks a problem and fills in what the kernels need.
rwkv7_status check_problem(const gated_delta_problem *in, Problem &p, Sizes &z) {
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
    p.Hk = in->Hk; p.Hv = in->Hv; p.K = in->K; p.V = in->V;
    p.T = p.cu ? 0 : p.total / p.n_seq;
    const long long slots = p.cu ? (long long)p.total / GATED_DELTA_CHUNK + p.n_seq
                                 : (long long)p.n_seq * ((p.T + GATED_DELTA_CHUNK - 1LL) /
                                                         GATED_DELTA_CHUNK);
    if (slots > 0x7fffffffLL) return RWKV7_ERR_SHAPE;
    p.slots = (int)slots;
    const long long dense_k = (long long)p.Hk * p.K, dense_v = (long long)p.Hv * p.V;
    const long long q_stride = in->q_stride ? in->q_stride : dense_k,
                    k_stride = in->k_stride ? in->k_stride : dense_k,
                    v_stride = in->v_stride ? in->v_stride : dense_v;
    const long long limit = (long long)1 << 23;  // offsets inside a chunk fit 32 bits
    if (q_stride < dense_k || k_stride < dense_k || v_stride < dense_v || q_stride > limit ||
        k_stride > limit || v_stride > limit)
        return RWKV7_ERR_SHAPE;
    if (q_stride * esz % 16 || k_stride * esz % 16 || v_stride * esz % 16)
        return RWKV7_ERR_ALIGN;
    p.q_stride = (int)q_stride; p.k_stride = (int)k_stride; p.v_stride = (int)v_stride;
    p.slots_in = in->slots_in; p.slots_out = in->slots_out;
    p.pool = in->pool;
    p.scale = in->scale;
    p.normalize = in->normalize != 0;
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
    if (!extent(p.q_stride, dense_k, z.q) || !extent(p.k_stride, dense_k, z.k) ||
        !extent(p.v_stride, dense_v, z.v) || !extent(dense_k, dense_k, z.qd) ||
        !extent(dense_v, dense_v, z.vd) || !extent(p.Hv, p.Hv, z.gate))
        return RWKV7_ERR_SHAPE;
    size_t state = 4;
    if (!mul_ok(state, (size_t)p.Hv) || !mul_ok(state, (size_t)p.V * p.K)) return RWKV7_ERR_SHAPE;
    z.pool = z.states = z.ckpt = state;
    if (!mul_ok(z.pool, (size_t)p.pool) || !mul_ok(z.states, (size_t)p.n_seq) ||
        !mul_ok(z.ckpt, (size_t)p.slots))
        return RWKV7_ERR_SHAPE;
    z.ckpt = z.ckpt / 4 / (p.V * p.K) * GATED_DELTA_CKPT_SIZE(p.V, p.K, in->dt) * esz;
    z.fwd = forward_record_bytes(p.bf16);
    size_t rec = backward_record_bytes(p.bf16);
    if (!mul_ok(z.fwd, (size_t)p.Hv) || !mul_ok(z.fwd, (size_t)p.slots) ||
        !mul_ok(rec, (size_t)p.Hv) || !mul_ok(rec, (size_t)p.slots))
        return RWKV7_ERR_SHAPE;
    const Segments seg = plan_segments(p);
    z.fwd_seg = up256(z.fwd);
    if (seg.seg) z.fwd = z.fwd_seg + seg.state_bytes + seg.step_bytes;
    z.bwd_ds = up256(rec);
    z.bwd_dr = z.bwd_ds + up256(z.ckpt);
    z.bwd = z.bwd_dr + z.vd;
    // every grid's extent in threads fits 32 bits
    const size_t chains = (size_t)p.n_seq * p.Hv;
    if (chains > 0xffffffffu / 512 / (p.V / 32) || (size_t)p.slots * p.Hk > 0xffffffffu / 1024)
        return RWKV7_ERR_SHAPE;
    return RWKV7_OK;
}

struct Out {
    const void *p;
    size_t bytes;
};

// Outputs must not overlap each other or an input.
bool disjoint(std::initializer_list<Out> outs, std::initializer_list<Out> ins) {
    for (const Out *a = outs.begin(); a != outs.end(); ++a) {
        const Range ra = range(a->p, a->bytes);
        for (const Out *b = a + 1; b != outs.end(); ++b)
            if (overlap(ra, range(b->p, b->bytes))) return false;
        for (const Out &b : ins)
            if (overlap(ra, range(b.p, b.bytes))) return false;
    }
    return true;
}

bool all_aligned(std::initializer_list<const void *> ps) {
    for (const void *p : ps)
        if (!aligned16(p)) return false;
    return true;
}
// one number per token and head: read and written element by element
bool gates_aligned(const Problem &p, std::initializer_list<const void *> ps) {
    for (const void *x : ps)
        if (!aligned(x, p.bf16 ? 2 : 4)) return false;
    return true;
}
bool any_null(std::initializer_list<const void *> ps) {
    for (const void *p : ps)
        if (!p) return true;
    return false;
}

rwkv7_status forward_impl(const gated_delta_problem *in, const void *q, const void *k,
                          const void *v, const void *g, const void *beta, const float *s0,
                          void *o, float *s_out, void *s_ckpt, void *u, bool train,
                          void *workspace, size_t workspace_bytes, void *stream) {
    ForwardArgs a{};
    Sizes z{};
    const rwkv7_status st = check_problem(in, a.p, z);
    if (st != RWKV7_OK) return st;
    if (train && (a.p.slots_in || a.p.slots_out)) return RWKV7_ERR_UNSUPPORTED;
    if (a.p.total > 0) {
        if (any_null({q, k, v, g, beta, o})) return RWKV7_ERR_NULL;
        if (train && any_null({s_ckpt, u})) return RWKV7_ERR_NULL;
    }
    if (!all_aligned({q, k, v, s0, o, s_out, s_ckpt, u}) || !gates_aligned(a.p, {g, beta}))
        return RWKV7_ERR_ALIGN;
    const size_t need = z.fwd;
    if (need && (!workspace || workspace_bytes < need)) return RWKV7_ERR_WORKSPACE;
    if (!aligned16(workspace)) return RWKV7_ERR_ALIGN;
    const size_t n = (size_t)a.p.n_seq * 4;
    const Out iq{q, z.q}, ik{k, z.k}, iv{v, z.v}, ig{g, z.gate}, ib{beta, z.gate},
        is{s0 == s_out ? nullptr : s0, z.pool}, ic{a.p.cu, n + 4}, i1{a.p.slots_in, n},
        i2{a.p.slots_out, n};
    if (!disjoint({{o, z.vd}, {s_out ? s_out : s0, z.pool}, {workspace, need},
                   {train ? s_ckpt : nullptr, z.ckpt}, {train ? u : nullptr, z.vd}},
                  {iq, ik, iv, ig, ib, s_out ? is : Out{nullptr, 0}, ic, i1, i2}))
        return RWKV7_ERR_ALIAS;
    a.q = q; a.k = k; a.v = v; a.g = g; a.beta = beta;
    a.s0 = s0; a.o = o; a.s_out = s_out;
    a.s_ckpt = train ? s_ckpt : nullptr;
    a.u = train ? u : nullptr;
    a.records = static_cast<char *>(workspace);
    a.segments = a.records ? a.records + z.fwd_seg : nullptr;
    return launch_forward(a, static_cast<hipStream_t>(stream)) == hipSuccess ? RWKV7_OK
                                                                             : RWKV7_ERR_HIP;
}

}  // namespace

extern "C" {

size_t gated_delta_forward_workspace(const gated_delta_problem *in) {
    Problem p;
    Sizes z{};
    return check_problem(in, p, z) == RWKV7_OK ? z.fwd : 0;
}

size_t gated_delta_backward_workspace(const gated_delta_problem *in) {
    Problem p;
    Sizes z{};
    return check_problem(in, p, z) == RWKV7_OK ? z.bwd : 0;
}

int gated_delta_chunks(const gated_delta_problem *in) {
    Problem p;
    Sizes z{};
    return check_problem(in, p, z) == RWKV7_OK ? p.slots : 0;
}

rwkv7_status gated_delta_forward(const gated_delta_problem *p, const void *q, const void *k,
                                 const void *v, const void *g, const void *beta,
                                 const float *s0, void *o, float *s_out, void *workspace,
                                 size_t workspace_bytes, void *stream) {
    return forward_impl(p, q, k, v, g, beta, s0, o, s_out, nullptr, nullptr, false, workspace,
                        workspace_bytes, stream);
}

rwkv7_status gated_delta_forward_train(const gated_delta_problem *p, const void *q,
                                       const void *k, const void *v, const void *g,
                                       const void *beta, const float *s0, void *o, float *s_out,
                                       void *s_ckpt, void *u, void *workspace,
                                       size_t workspace_bytes, void *stream) {
    return forward_impl(p, q, k, v, g, beta, s0, o, s_out, s_ckpt, u, true, workspace,
                        workspace_bytes, stream);
}

rwkv7_status gated_delta_decode(const gated_delta_problem *in, const void *q, const void *k,
                                const void *v, const void *g, const void *beta, float *state,
                                void *o, void *stream) {
    DecodeArgs a{};
    Sizes z{};
    const rwkv7_status st = check_problem(in, a.p, z);
    if (st != RWKV7_OK) return st;
    if (a.p.cu || a.p.total != a.p.n_seq || a.p.slots_in != a.p.slots_out)
        return RWKV7_ERR_SHAPE;
    if (any_null({q, k, v, g, beta, state, o})) return RWKV7_ERR_NULL;
    if (!all_aligned({q, k, v, state, o}) || !gates_aligned(a.p, {g, beta}))
        return RWKV7_ERR_ALIGN;
    if (!disjoint({{o, z.vd}, {state, z.pool}},
                  {{q, z.q}, {k, z.k}, {v, z.v}, {g, z.gate}, {beta, z.gate},
                   {a.p.slots_in, (size_t)a.p.n_seq * 4}}))
        return RWKV7_ERR_ALIAS;
    a.q = q; a.k = k; a.v = v; a.g = g; a.beta = beta;
    a.state = state; a.o = o;
    return launch_decode(a, static_cast<hipStream_t>(stream)) == hipSuccess ? RWKV7_OK
                                                                            : RWKV7_ERR_HIP;
}

rwkv7_status gated_delta_backward(const gated_delta_problem *in, const void *q, const void *k,
                                  const void *v, const void *g, const void *beta,
                                  const void *d_o, const void *s_ckpt, const void *u,
                                  const float *ds_T, void *dq, void *dk, void *dv, void *dg,
                                  void *dbeta, float *ds0, void *workspace,
                                  size_t workspace_bytes, void *stream) {
    BackwardArgs a{};
    Sizes z{};
    const rwkv7_status st = check_problem(in, a.p, z);
    if (st != RWKV7_OK) return st;
    if (a.p.slots_in || a.p.slots_out) return RWKV7_ERR_UNSUPPORTED;
    if (a.p.total > 0 && any_null({q, k, v, g, beta, d_o, s_ckpt, u, dq, dk, dv, dg, dbeta}))
        return RWKV7_ERR_NULL;
    if (!all_aligned({q, k, v, d_o, s_ckpt, u, ds_T, dq, dk, dv, ds0}) ||
        !gates_aligned(a.p, {g, beta, dg, dbeta}))
        return RWKV7_ERR_ALIGN;
    const size_t need = z.bwd;
    if (need && (!workspace || workspace_bytes < need)) return RWKV7_ERR_WORKSPACE;
    if (!aligned16(workspace)) return RWKV7_ERR_ALIGN;
    if (!disjoint({{dq, z.qd}, {dk, z.qd}, {dv, z.vd}, {dg, z.gate}, {dbeta, z.gate},
                   {ds0, z.states}, {workspace, need}},
                  {{q, z.q}, {k, z.k}, {v, z.v}, {g, z.gate}, {beta, z.gate}, {d_o, z.vd},
                   {s_ckpt, z.ckpt}, {u, z.vd}, {ds_T == ds0 ? nullptr : ds_T, z.states},
                   {a.p.cu, (size_t)a.p.n_seq * 4 + 4}}))
        return RWKV7_ERR_ALIAS;
    a.q = q; a.k = k; a.v = v; a.g = g; a.beta = beta;
    a.d_o = d_o; a.s_ckpt = s_ckpt; a.u = u; a.ds_T = ds_T;
    a.dq = dq; a.dk = dk; a.dv = dv; a.dg = dg; a.dbeta = dbeta; a.ds0 = ds0;
    char *ws = static_cast<char *>(workspace);
    a.records = ws;
    a.ds = ws ? ws + z.bwd_ds : nullptr;
    a.dr = ws ? ws + z.bwd_dr : nullptr;
    return launch_backward(a, static_cast<hipStream_t>(stream)) == hipSuccess ? RWKV7_OK
                                                                              : RWKV7_ERR_HIP;
}

}  // extern "C"
