// ssd_linattn_api.cpp -- C entry points of linear attention with a decay for each head and of rotary
// positions.  Host-side validation only; the kernels are in ssd_linattn.hip,
// ssd_linattn_step.hip and ssd_rotary.hip.
#include "../../include/ssd.h"

#include <hip/hip_runtime.h>

#include "ssd_check.h"
#include "ssd_launch.h"

namespace {

using namespace ssd::check;

constexpr int64_t kMaxRow = int64_t(1) << 22;     // elements: 64 rows of fp32 within 2^30 bytes

ssd_status check_linattn(const ssd_linattn_problem *p)
{
    if (p == nullptr) return SSD_ERR_NULL_ARG;
    if (p->batch <= 0 || p->seqlen <= 0 || p->nheads <= 0 || p->ngroups <= 0 || p->key_dim <= 0 ||
        p->value_dim <= 0)
        return SSD_ERR_BAD_SHAPE;
    if (p->nheads % p->ngroups != 0) return SSD_ERR_BAD_SHAPE;
    if (p->key_dim % 8 != 0 || p->key_dim > 256 || p->value_dim % 8 != 0 || p->value_dim > 256)
        return SSD_ERR_UNSUPPORTED;
    if (p->nheads > 65535 || p->batch > 65535 / p->nheads) return SSD_ERR_UNSUPPORTED;
    const int64_t qk = p->ngroups * p->key_dim, vo = p->nheads * p->value_dim;
    if (!pitch_fits(p->q_pitch, qk) || !pitch_fits(p->k_pitch, qk) || !pitch_fits(p->v_pitch, vo) ||
        !pitch_fits(p->do_pitch, vo))
        return SSD_ERR_BAD_SHAPE;
    if (p->decay == SSD_DECAY_TOKEN && !pitch_fits(p->g_pitch, p->nheads)) return SSD_ERR_BAD_SHAPE;
    if (!is_dtype(p->dtype) || !finite(p->scale) || p->decay < SSD_DECAY_NONE ||
        p->decay > SSD_DECAY_TOKEN)
        return SSD_ERR_UNSUPPORTED;
    for (int64_t w : {qk, vo, p->q_pitch, p->k_pitch, p->v_pitch, p->g_pitch, p->do_pitch})
        if (w > kMaxRow) return SSD_ERR_UNSUPPORTED;
    return tokens_fit(p->batch, p->seqlen) ? SSD_OK : SSD_ERR_UNSUPPORTED;
}

// A gradient of shared queries and keys goes through rows of every head's: nheads * key_dim.
ssd_status check_linattn_gradient(const ssd_linattn_problem *p)
{
    const ssd_status st = check_linattn(p);
    if (st != SSD_OK) return st;
    return p->nheads * p->key_dim <= kMaxRow ? SSD_OK : SSD_ERR_UNSUPPORTED;
}

ssd::LinattnShape linattn_shape(const ssd_linattn_problem *p)
{
    ssd::LinattnShape s;
    s.b = p->batch; s.L = p->seqlen; s.H = p->nheads; s.G = p->ngroups;
    s.dk = p->key_dim; s.dv = p->value_dim;
    s.qp = p->q_pitch ? p->q_pitch : s.G * s.dk;
    s.kp = p->k_pitch ? p->k_pitch : s.G * s.dk;
    s.vp = p->v_pitch ? p->v_pitch : s.H * s.dv;
    s.gp = p->g_pitch ? p->g_pitch : s.H;
    s.dop = p->do_pitch ? p->do_pitch : s.H * s.dv;
    s.scale = p->scale;
    s.decay = p->decay;
    s.bf16 = p->dtype == SSD_BF16;
    return s;
}

// Decays and lengths are read element by element.
bool decays_aligned(const ssd_linattn_problem *p, const void *g, const void *dg, const int32_t *lengths)
{
    const bool own = p->decay == SSD_DECAY_NONE ||
                     on_bytes(p->decay == SSD_DECAY_HEAD ? 4 : bytes_of(p->dtype), {g});
    return own && on_bytes(bytes_of(p->dtype), {dg}) && on_bytes(4, {lengths});
}

// Rows are read 16 bytes at a time.
bool rows_aligned(const ssd_linattn_problem *p, std::initializer_list<int64_t> pitches)
{
    for (int64_t w : pitches)
        if (w * bytes_of(p->dtype) % 16 != 0) return false;
    return true;
}

// The inputs' areas (lengths and the first state apart).
struct Inputs {
    Area q, k, v, g;
};
Inputs inputs_of(const ssd_linattn_problem *p, const void *q, const void *k, const void *v,
                 const void *g)
{
    const int64_t e = bytes_of(p->dtype), rows = p->batch * p->seqlen;
    const int64_t qk = p->ngroups * p->key_dim, vo = p->nheads * p->value_dim;
    Inputs in = {rows_of(q, rows, p->q_pitch, qk, e), rows_of(k, rows, p->k_pitch, qk, e),
                 rows_of(v, rows, p->v_pitch, vo, e), dense(nullptr, 0)};
    if (p->decay == SSD_DECAY_HEAD) in.g = dense(g, p->nheads * 4);
    if (p->decay == SSD_DECAY_TOKEN) in.g = rows_of(g, rows, p->g_pitch, p->nheads, e);
    return in;
}

int64_t state_bytes(const ssd_linattn_problem *p)
{
    return p->batch * p->nheads * p->key_dim * p->value_dim * 4;
}

ssd_status check_rotary(const ssd_rotary_problem *p)
{
    if (p == nullptr) return SSD_ERR_NULL_ARG;
    if (p->batch <= 0 || p->seqlen <= 0 || p->q_heads <= 0 || p->k_heads < 0 || p->head_dim <= 0 ||
        p->rotated <= 0 || p->rotated > p->head_dim || p->rotated % 2 != 0)
        return SSD_ERR_BAD_SHAPE;
    if (p->head_dim > 4096 || p->q_heads > kMaxRow / p->head_dim || p->k_heads > kMaxRow / p->head_dim)
        return SSD_ERR_UNSUPPORTED;
    if (!pitch_fits(p->q_pitch, p->q_heads * p->head_dim) ||
        !pitch_fits(p->k_pitch, p->k_heads * p->head_dim))
        return SSD_ERR_BAD_SHAPE;
    if (!is_dtype(p->dtype) || !finite(p->scale) || !is_flag(p->interleaved) || !is_flag(p->inverse) ||
        p->positions < SSD_POSITIONS_START || p->positions > SSD_POSITIONS_EACH)
        return SSD_ERR_UNSUPPORTED;
    if (p->q_pitch > kMaxRow || p->k_pitch > kMaxRow || !tokens_fit(p->batch, p->seqlen) ||
        p->batch * p->seqlen >= int64_t(1) << 24)
        return SSD_ERR_UNSUPPORTED;
    return SSD_OK;
}

}  // namespace

extern "C" {

ssd_status ssd_linattn_validate(const ssd_linattn_problem *problem) { return check_linattn(problem); }

size_t ssd_linattn_workspace_bytes(const ssd_linattn_problem *problem)
{
    return check_linattn(problem) == SSD_OK ? ssd::linattn_workspace_bytes(linattn_shape(problem)) : 0;
}

ssd_status ssd_linattn(const ssd_linattn_problem *problem, const void *q, const void *k,
                       const void *v, const void *g, const float *h0, const int32_t *lengths,
                       void *o, float *hT, void *workspace, size_t workspace_bytes, void *stream)
{
    ssd_status st = check_linattn(problem);
    if (st != SSD_OK) return st;
    if (!q || !k || !v || !o || (!g && problem->decay != SSD_DECAY_NONE)) return SSD_ERR_NULL_ARG;
    const size_t need = ssd_linattn_workspace_bytes(problem);
    const bool work = need > SSD_LINATTN_NO_WORKSPACE;
    if (work && (workspace == nullptr || workspace_bytes < need)) return SSD_ERR_WORKSPACE;
    if (!on_bytes(16, {q, k, v, o, h0, hT, work ? workspace : nullptr}) ||
        !decays_aligned(problem, g, nullptr, lengths) ||
        !rows_aligned(problem, {problem->q_pitch, problem->k_pitch, problem->v_pitch}))
        return SSD_ERR_MISALIGNED;
    const Inputs in = inputs_of(problem, q, k, v, g);
    const int64_t states = state_bytes(problem);
    const Area out = dense(o, problem->batch * problem->seqlen * problem->nheads * problem->value_dim *
                                  bytes_of(problem->dtype));
    const Area last = dense(hT, states), len = dense(lengths, problem->batch * 4);
    const Area ws = dense(work ? workspace : nullptr, (int64_t)need);
    st = check_apart({out, last, ws}, {in.q, in.k, in.v, in.g, len});
    // each element of a state is read before the same thread writes it
    if (st == SSD_OK) st = check_apart({out, ws}, {dense(h0, states)});
    if (st == SSD_OK) st = check_apart({last}, {dense(h0, states, true)});
    if (st != SSD_OK) return st;
    const ssd::LinattnArgs a = {q, k, v, g, h0, lengths, o, hT, workspace};
    return status_of(ssd::launch_linattn(linattn_shape(problem), a, (hipStream_t)stream));
}

size_t ssd_linattn_backward_workspace_bytes(const ssd_linattn_problem *problem)
{
    return check_linattn_gradient(problem) == SSD_OK
               ? ssd::linattn_backward_workspace_bytes(linattn_shape(problem))
               : 0;
}

ssd_status ssd_linattn_backward(const ssd_linattn_problem *problem, const void *dout, const void *q,
                                const void *k, const void *v, const void *g, const float *h0,
                                const float *dhT, const int32_t *lengths, void *dq, void *dk,
                                void *dv, void *dg, float *dh0, void *workspace,
                                size_t workspace_bytes, void *stream)
{
    ssd_status st = check_linattn_gradient(problem);
    if (st != SSD_OK) return st;
    const ssd_linattn_problem &p = *problem;
    if (!dout || !q || !k || !v || !dq || !dk || !dv || (!g && p.decay != SSD_DECAY_NONE))
        return SSD_ERR_NULL_ARG;
    if (dg && p.decay != SSD_DECAY_TOKEN) return SSD_ERR_UNSUPPORTED;
    const size_t need = ssd_linattn_backward_workspace_bytes(problem);
    const bool work = need > SSD_LINATTN_NO_WORKSPACE;
    if (work && (workspace == nullptr || workspace_bytes < need)) return SSD_ERR_WORKSPACE;
    if (!on_bytes(16, {dout, q, k, v, h0, dhT, dq, dk, dv, dh0, work ? workspace : nullptr}) ||
        !decays_aligned(problem, g, dg, lengths) ||
        !rows_aligned(problem, {p.q_pitch, p.k_pitch, p.v_pitch, p.do_pitch}))
        return SSD_ERR_MISALIGNED;
    const int64_t e = bytes_of(p.dtype), rows = p.batch * p.seqlen;
    const int64_t qk = p.ngroups * p.key_dim, vo = p.nheads * p.value_dim;
    const Inputs in = inputs_of(problem, q, k, v, g);
    const int64_t states = state_bytes(problem);
    st = check_apart({dense(dq, rows * qk * e), dense(dk, rows * qk * e), dense(dv, rows * vo * e),
                      dense(dg, rows * p.nheads * e), dense(dh0, states),
                      dense(work ? workspace : nullptr, (int64_t)need)},
                     {in.q, in.k, in.v, in.g, rows_of(dout, rows, p.do_pitch, vo, e), dense(h0, states),
                      dense(dhT, states), dense(lengths, p.batch * 4)});
    if (st != SSD_OK) return st;
    const ssd::LinattnGradArgs a = {dout, q, k, v, g, h0, dhT, lengths, dq, dk, dv, dg, dh0, workspace};
    return status_of(ssd::launch_linattn_backward(linattn_shape(problem), a, (hipStream_t)stream));
}

ssd_status ssd_linattn_step(const ssd_linattn_problem *problem, const void *q, const void *k,
                            const void *v, const void *g, float *h, void *o, void *stream)
{
    ssd_status st = check_linattn(problem);
    if (st != SSD_OK) return st;
    if (problem->seqlen != 1) return SSD_ERR_BAD_SHAPE;
    if (!q || !k || !v || !h || !o || (!g && problem->decay != SSD_DECAY_NONE)) return SSD_ERR_NULL_ARG;
    if (!on_bytes(16, {q, k, v, o, h}) || !decays_aligned(problem, g, nullptr, nullptr) ||
        !rows_aligned(problem, {problem->q_pitch, problem->k_pitch, problem->v_pitch}))
        return SSD_ERR_MISALIGNED;
    Inputs in = inputs_of(problem, q, k, v, g);
    const Area state = dense(h, state_bytes(problem));
    st = check_apart({state}, {in.q, in.k, in.v, in.g});
    if (st != SSD_OK) return st;
    // the team that writes a row of o has read that row of v
    in.v.same = true;
    st = check_apart({dense(o, problem->batch * problem->nheads * problem->value_dim *
                                   bytes_of(problem->dtype))},
                     {in.q, in.k, in.v, in.g, state});
    if (st != SSD_OK) return st;
    const ssd::LinattnArgs a = {q, k, v, g, nullptr, nullptr, o, nullptr, nullptr};
    return status_of(ssd::launch_linattn_step(linattn_shape(problem), a, h, (hipStream_t)stream));
}

ssd_status ssd_rotary_validate(const ssd_rotary_problem *problem) { return check_rotary(problem); }

ssd_status ssd_rotary(const ssd_rotary_problem *problem, const void *q, const void *k,
                      const float *freqs, const int32_t *positions, void *q_out, void *k_out,
                      void *stream)
{
    ssd_status st = check_rotary(problem);
    if (st != SSD_OK) return st;
    const ssd_rotary_problem &p = *problem;
    if (!q || !freqs || !q_out || (p.k_heads > 0 && (!k || !k_out)) ||
        (p.positions != SSD_POSITIONS_START && !positions))
        return SSD_ERR_NULL_ARG;
    if (!on_bytes(bytes_of(p.dtype), {q, k, q_out, k_out}) || !on_bytes(4, {freqs, positions}))
        return SSD_ERR_MISALIGNED;
    const int64_t rows = p.batch * p.seqlen, e = bytes_of(p.dtype);
    const int64_t qw = p.q_heads * p.head_dim, kw = p.k_heads * p.head_dim;
    const bool both = p.k_heads > 0;
    const Area table = dense(freqs, p.rotated / 2 * 4);
    const Area at = dense(p.positions == SSD_POSITIONS_START ? nullptr : positions,
                          (p.positions == SSD_POSITIONS_EACH ? rows : p.batch) * 4);
    const Area yq = dense(q_out, rows * qw * e), yk = dense(both ? k_out : nullptr, rows * kw * e);
    const void *kin = both ? k : nullptr;
    // a thread writes the pairs that it has read, of its own array
    st = check_apart({yq, yk}, {table, at});
    if (st == SSD_OK)
        st = check_apart({yq}, {rows_of(q, rows, p.q_pitch, qw, e, true), rows_of(kin, rows, p.k_pitch, kw, e)});
    if (st == SSD_OK)
        st = check_apart({yk}, {rows_of(q, rows, p.q_pitch, qw, e), rows_of(kin, rows, p.k_pitch, kw, e, true)});
    if (st != SSD_OK) return st;
    ssd::RotaryShape s;
    s.b = p.batch; s.L = p.seqlen; s.Hq = p.q_heads; s.Hk = p.k_heads;
    s.D = p.head_dim; s.rot = p.rotated;
    s.qp = p.q_pitch ? p.q_pitch : qw;
    s.kp = p.k_pitch ? p.k_pitch : kw;
    s.scale = p.scale;
    s.interleaved = p.interleaved != 0; s.inverse = p.inverse != 0; s.bf16 = p.dtype == SSD_BF16;
    s.positions = p.positions;
    return status_of(ssd::launch_rotary(s, q, k, freqs, positions, q_out, k_out, (hipStream_t)stream));
}

}  // extern "C"
