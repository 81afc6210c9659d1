// ssd_block_api.cpp -- C entry points of the operators around the forward: the short causal
// convolution, the selective scan and the block norms.  Host-side validation only; the
// kernels are in ssd_conv.hip, ssd_scan.hip and ssd_norm.hip.
#include "../../include/ssd.h"

#include <hip/hip_runtime.h>

#include <cfloat>
#include <initializer_list>

#include "ssd_launch.h"

namespace {

constexpr int64_t kMaxPitch = int64_t(1) << 24;      // eight rows of fp32 within 2^29 bytes
constexpr int64_t kMaxTokens = int64_t(1) << 30;
constexpr int64_t kMaxRows = int64_t(1) << 31;       // batch * seqlen
constexpr int64_t kMaxChannels = int64_t(1) << 24;
// Workgroups of 256 threads: the dispatch grid counts work-items in 32 bits.
constexpr int64_t kMaxGrid = int64_t(1) << 24;

bool on_bytes(size_t n, std::initializer_list<const void *> ptrs)
{
    for (const void *p : ptrs)
        if ((reinterpret_cast<uintptr_t>(p) & (n - 1)) != 0) return false;
    return true;
}

bool is_dtype(int32_t d) { return d == SSD_F32 || d == SSD_BF16; }
bool is_flag(int32_t f) { return f == 0 || f == 1; }
// 0 (dense) or at least the row's width
bool pitch_fits(int64_t pitch, int64_t width) { return pitch == 0 || pitch >= width; }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
bool finite(float v) { return v - v == 0.0f; }

// batch and seqlen (both positive) within the index limits
bool tokens_fit(int64_t batch, int64_t seqlen)
{
    return seqlen <= kMaxTokens && batch <= kMaxRows / seqlen;
}

ssd_status check_conv(const ssd_conv_problem *p)
{
    if (p == nullptr) return SSD_ERR_NULL_ARG;
    if (p->batch <= 0 || p->seqlen <= 0 || p->channels <= 0) return SSD_ERR_BAD_SHAPE;
    const int64_t *w = p->split;
    if (w[0] <= 0 || w[1] < 0 || w[2] < 0 || (w[1] == 0 && w[2] > 0)) return SSD_ERR_BAD_SHAPE;
    if (w[0] > p->channels || w[1] > p->channels || w[2] > p->channels - w[0] ||
        w[0] + w[1] + w[2] != p->channels)
        return SSD_ERR_BAD_SHAPE;
    if (!pitch_fits(p->x_pitch, p->channels)) return SSD_ERR_BAD_SHAPE;
    if (!is_dtype(p->dtype) || !is_flag(p->silu) || p->width < 2 || p->width > 4)
        return SSD_ERR_UNSUPPORTED;
    if (p->channels > kMaxChannels || p->x_pitch > kMaxPitch || !tokens_fit(p->batch, p->seqlen))
        return SSD_ERR_UNSUPPORTED;
    const int64_t tiles = ceil_div(p->channels, 256) * ceil_div(p->seqlen, 8);
    if (p->batch > (kMaxGrid - 1) / tiles) return SSD_ERR_UNSUPPORTED;
    return SSD_OK;
}

ssd::ConvShape conv_shape(const ssd_conv_problem *p)
{
    ssd::ConvShape s;
    s.b = p->batch; s.L = p->seqlen; s.C = p->channels;
    s.pitch = p->x_pitch ? p->x_pitch : p->channels;
    s.w0 = p->split[0]; s.w1 = p->split[1]; s.w2 = p->split[2];
    s.K = p->width;
    s.silu = p->silu != 0;
    s.bf16 = p->dtype == SSD_BF16;
    return s;
}

ssd_status check_scan(const ssd_scan_problem *p)
{
    if (p == nullptr) return SSD_ERR_NULL_ARG;
    if (p->batch <= 0 || p->seqlen <= 0 || p->channels <= 0 || p->ngroups <= 0 || p->dstate <= 0)
        return SSD_ERR_BAD_SHAPE;
    if (p->channels % p->ngroups != 0) return SSD_ERR_BAD_SHAPE;
    if (p->dstate % 8 != 0 || p->dstate > 64 || p->channels > kMaxChannels)
        return SSD_ERR_UNSUPPORTED;
    const int64_t gn = p->ngroups * p->dstate;   // at most channels * 64
    if (!pitch_fits(p->x_pitch, p->channels) || !pitch_fits(p->dt_pitch, p->channels) ||
        !pitch_fits(p->z_pitch, p->channels) || !pitch_fits(p->B_pitch, gn) ||
        !pitch_fits(p->C_pitch, gn))
        return SSD_ERR_BAD_SHAPE;
    if (!is_dtype(p->dtype) || !is_flag(p->softplus)) return SSD_ERR_UNSUPPORTED;
    for (int64_t pitch : {p->x_pitch, p->dt_pitch, p->z_pitch, p->B_pitch, p->C_pitch, gn})
        if (pitch > kMaxPitch) return SSD_ERR_UNSUPPORTED;
    if (!tokens_fit(p->batch, p->seqlen)) return SSD_ERR_UNSUPPORTED;
    if (p->batch > kMaxRows / p->dstate / p->channels) return SSD_ERR_UNSUPPORTED;
    const int64_t tiles = ceil_div(p->channels / p->ngroups, 64) * p->ngroups;
    if (p->batch > ((int64_t(1) << 20) - 1) / tiles) return SSD_ERR_UNSUPPORTED;
    return SSD_OK;
}

ssd::ScanShape scan_shape(const ssd_scan_problem *p)
{
    ssd::ScanShape s;
    s.b = p->batch; s.L = p->seqlen; s.C = p->channels; s.G = p->ngroups; s.N = p->dstate;
    s.xp = p->x_pitch ? p->x_pitch : p->channels;
    s.dtp = p->dt_pitch ? p->dt_pitch : p->channels;
    s.zp = p->z_pitch ? p->z_pitch : p->channels;
    s.Bp = p->B_pitch ? p->B_pitch : p->ngroups * p->dstate;
    s.Cp = p->C_pitch ? p->C_pitch : p->ngroups * p->dstate;
    s.softplus = p->softplus != 0;
    s.bf16 = p->dtype == SSD_BF16;
    return s;
}

// States and rates are read 16 bytes at a time; B and C four elements at a time, on 4 bytes.
ssd_status check_scan_pointers(const ssd_scan_problem *p, const void *A, const void *B,
                               const void *C, std::initializer_list<const void *> states)
{
    if (!on_bytes(16, {A}) || !on_bytes(16, states) || !on_bytes(4, {B, C}))
        return SSD_ERR_MISALIGNED;
    if (p->dtype == SSD_BF16 && (p->B_pitch % 2 != 0 || p->C_pitch % 2 != 0))
        return SSD_ERR_MISALIGNED;
    return SSD_OK;
}

ssd_status check_norm(const ssd_norm_problem *p)
{
    if (p == nullptr) return SSD_ERR_NULL_ARG;
    if (p->rows <= 0 || p->channels <= 0 || p->ngroups <= 0) return SSD_ERR_BAD_SHAPE;
    if (p->channels % p->ngroups != 0) return SSD_ERR_BAD_SHAPE;
    if (!pitch_fits(p->x_pitch, p->channels) || !pitch_fits(p->z_pitch, p->channels))
        return SSD_ERR_BAD_SHAPE;
    if (!is_dtype(p->dtype) || !is_flag(p->gate_after)) return SSD_ERR_UNSUPPORTED;
    if (p->residual_dtype != SSD_F32 && p->residual_dtype != p->dtype) return SSD_ERR_UNSUPPORTED;
    // the hardware's reciprocal root takes a subnormal number for zero
    if (!finite(p->eps) || !(p->eps >= FLT_MIN) || !finite(p->scale)) return SSD_ERR_UNSUPPORTED;
    if (p->channels > kMaxChannels || p->x_pitch > kMaxPitch || p->z_pitch > kMaxPitch ||
        p->rows > kMaxRows || p->rows > (kMaxGrid - 1) / p->ngroups)
        return SSD_ERR_UNSUPPORTED;
    return SSD_OK;
}

// ---------------------------------------------------------------------------
// Outputs and inputs apart.  The kernels read inputs that other threads' outputs would have
// replaced (a token tile of the convolution reads the rows before it), so memory that an output
// shares with another argument is refused.  `rows` rows of `width` bytes, `pitch` bytes apart;
// `same`: an output with this very layout may be this buffer (each element is read before the
// same thread writes it).
// ---------------------------------------------------------------------------
struct Area {
    const void *p;
    int64_t rows, pitch, width;
    bool same;
};

int64_t bytes_of(int32_t dtype) { return dtype == SSD_BF16 ? 2 : 4; }

Area dense(const void *p, int64_t bytes, bool same = false) { return {p, 1, bytes, bytes, same}; }

// rows of `width` elements at a pitch of `pitch` elements (0: dense)
Area rows_of(const void *p, int64_t rows, int64_t pitch, int64_t width, int64_t bytes,
             bool same = false)
{
    if (pitch == 0 || pitch == width || rows == 1) return dense(p, rows * width * bytes, same);
    return {p, rows, pitch * bytes, width * bytes, same};
}

// Whether a dense output shares memory with `in`.
bool meet(const Area &out, const Area &in)
{
    if (out.p == nullptr || in.p == nullptr) return false;
    // the output's start from the input's, and the input's first row that ends behind it
    const int64_t d = (int64_t)(reinterpret_cast<uintptr_t>(out.p) - reinterpret_cast<uintptr_t>(in.p));
    if (d + out.width <= 0) return false;
    if (d >= in.width) {
        const int64_t row = in.rows == 1 ? 1 : (d - in.width) / in.pitch + 1;
        if (row >= in.rows || row * in.pitch >= d + out.width) return false;
    }
    return !(in.same && d == 0 && in.rows == 1 && in.width == out.width);
}

ssd_status check_apart(std::initializer_list<Area> outs, std::initializer_list<Area> ins)
{
    for (const Area *o = outs.begin(); o != outs.end(); ++o) {
        for (const Area &in : ins)
            if (meet(*o, in)) return SSD_ERR_OVERLAP;
        for (const Area *p = o + 1; p != outs.end(); ++p)
            if (meet(*o, *p)) return SSD_ERR_OVERLAP;
    }
    return SSD_OK;
}

// The convolution's arrays; the final state may be the state's buffer, and a step's only output
// may be x.
ssd_status check_conv_areas(const ssd_conv_problem *p, const void *x, const float *weight,
                            const float *bias, const void *state0, const int32_t *lengths,
                            const void *y0, const void *y1, const void *y2, const void *stateT,
                            bool step)
{
    const int64_t e = bytes_of(p->dtype), rows = p->batch * p->seqlen, C = p->channels;
    const int64_t state = p->batch * (p->width - 1) * C * e;
    const ssd_status st =
        check_apart({dense(y0, rows * p->split[0] * e), dense(y1, rows * p->split[1] * e),
                     dense(y2, rows * p->split[2] * e)},
                    {rows_of(x, rows, p->x_pitch, C, e, step), dense(weight, C * p->width * 4),
                     dense(bias, C * 4), dense(state0, state), dense(lengths, p->batch * 4),
                     dense(stateT, state)});
    if (st != SSD_OK) return st;
    return check_apart({dense(stateT, state)},
                       {rows_of(x, rows, p->x_pitch, C, e), dense(weight, C * p->width * 4),
                        dense(bias, C * 4), dense(state0, state, true),
                        dense(lengths, p->batch * 4)});
}

// The scan's arrays: hT may be h0's buffer, and a step's y the buffer of x, dt or z.
ssd_status check_scan_areas(const ssd_scan_problem *p, const ssd::ScanArgs &a, const void *hT,
                            size_t workspace_bytes, bool step)
{
    const int64_t e = bytes_of(p->dtype), rows = p->batch * p->seqlen, C = p->channels;
    const int64_t gn = p->ngroups * p->dstate, state = p->batch * C * p->dstate * 4;
    const Area y = dense(a.y, rows * C * e), h = dense(hT, state);
    const Area ws = dense(workspace_bytes ? a.ws : nullptr, (int64_t)workspace_bytes);
    const Area A = dense(a.A, C * p->dstate * 4), D = dense(a.D, C * 4),
               bias = dense(a.dt_bias, C * 4), lengths = dense(a.lengths, p->batch * 4),
               B = rows_of(a.B, rows, p->B_pitch, gn, e), Cm = rows_of(a.C, rows, p->C_pitch, gn, e);
    const auto row = [&](const void *q, int64_t pitch, bool same) {
        return rows_of(q, rows, pitch, C, e, same);
    };
    const ssd_status st = check_apart(
        {y}, {row(a.x, p->x_pitch, step), row(a.dt, p->dt_pitch, step), row(a.z, p->z_pitch, step),
              A, B, Cm, D, bias, lengths, dense(a.h0, state), h, ws});
    if (st != SSD_OK) return st;
    return check_apart({h, ws}, {row(a.x, p->x_pitch, false), row(a.dt, p->dt_pitch, false),
                                 row(a.z, p->z_pitch, false), A, B, Cm, D, bias, lengths,
                                 dense(a.h0, state, true)});
}

ssd_status status_of(hipError_t e) { return ssd_status(ssd::hip_status(e)); }

}  // namespace

extern "C" {

ssd_status ssd_conv_validate(const ssd_conv_problem *problem) { return check_conv(problem); }

ssd_status ssd_conv(const ssd_conv_problem *problem, const void *x, const float *weight,
                    const float *bias, const void *state0, const int32_t *lengths, void *y0,
                    void *y1, void *y2, void *stateT, void *stream)
{
    const ssd_status st = check_conv(problem);
    if (st != SSD_OK) return st;
    if (!x || !weight || !y0 || (problem->split[1] > 0 && !y1) || (problem->split[2] > 0 && !y2))
        return SSD_ERR_NULL_ARG;
    if (!on_bytes(16, {weight, bias})) return SSD_ERR_MISALIGNED;
    const ssd_status apart = check_conv_areas(problem, x, weight, bias, state0, lengths, y0,
                                              problem->split[1] ? y1 : nullptr,
                                              problem->split[2] ? y2 : nullptr, stateT, false);
    if (apart != SSD_OK) return apart;
    return status_of(ssd::launch_conv(conv_shape(problem), x, weight, bias, state0, lengths, y0,
                                      y1, y2, stateT, (hipStream_t)stream));
}

ssd_status ssd_conv_step(const ssd_conv_problem *problem, const void *x, const float *weight,
                         const float *bias, void *state, void *y0, void *y1, void *y2,
                         void *stream)
{
    const ssd_status st = check_conv(problem);
    if (st != SSD_OK) return st;
    if (problem->seqlen != 1) return SSD_ERR_BAD_SHAPE;
    if (!x || !weight || !state || !y0 || (problem->split[1] > 0 && !y1) ||
        (problem->split[2] > 0 && !y2))
        return SSD_ERR_NULL_ARG;
    if (!on_bytes(16, {weight, bias})) return SSD_ERR_MISALIGNED;
    const ssd_status apart = check_conv_areas(problem, x, weight, bias, nullptr, nullptr, y0,
                                              problem->split[1] ? y1 : nullptr,
                                              problem->split[2] ? y2 : nullptr, state, true);
    if (apart != SSD_OK) return apart;
    return status_of(ssd::launch_conv_step(conv_shape(problem), x, weight, bias, state, y0, y1,
                                           y2, (hipStream_t)stream));
}

ssd_status ssd_scan_validate(const ssd_scan_problem *problem) { return check_scan(problem); }

size_t ssd_scan_workspace_bytes(const ssd_scan_problem *problem)
{
    return check_scan(problem) == SSD_OK ? ssd::scan_workspace_bytes(scan_shape(problem)) : 0;
}

ssd_status ssd_scan(const ssd_scan_problem *problem, const void *x, const void *dt,
                    const float *A, const void *B, const void *C, const float *D, const void *z,
                    const float *dt_bias, const float *h0, const int32_t *lengths, void *y,
                    float *hT, void *workspace, size_t workspace_bytes, void *stream)
{
    ssd_status st = check_scan(problem);
    if (st != SSD_OK) return st;
    if (!x || !dt || !A || !B || !C || !y) return SSD_ERR_NULL_ARG;
    const ssd::ScanShape s = scan_shape(problem);
    const size_t need = ssd::scan_workspace_bytes(s);
    if (need > SSD_SCAN_NO_WORKSPACE && (workspace == nullptr || workspace_bytes < need))
        return SSD_ERR_WORKSPACE;
    st = check_scan_pointers(problem, A, B, C, {h0, hT, workspace});
    if (st != SSD_OK) return st;
    const ssd::ScanArgs a = {x, dt, A, B, C, D, z, dt_bias, h0, lengths, y, hT, workspace};
    st = check_scan_areas(problem, a, hT, need > SSD_SCAN_NO_WORKSPACE ? need : 0, false);
    if (st != SSD_OK) return st;
    return status_of(ssd::launch_scan(s, a, (hipStream_t)stream));
}

ssd_status ssd_scan_step(const ssd_scan_problem *problem, const void *x, const void *dt,
                         const float *A, const void *B, const void *C, const float *D,
                         const void *z, const float *dt_bias, float *h, void *y, void *stream)
{
    ssd_status st = check_scan(problem);
    if (st != SSD_OK) return st;
    if (problem->seqlen != 1) return SSD_ERR_BAD_SHAPE;
    if (!x || !dt || !A || !B || !C || !h || !y) return SSD_ERR_NULL_ARG;
    st = check_scan_pointers(problem, A, B, C, {h});
    if (st != SSD_OK) return st;
    const ssd::ScanArgs a = {x, dt, A, B, C, D, z, dt_bias, nullptr, nullptr, y, nullptr, nullptr};
    st = check_scan_areas(problem, a, h, 0, true);
    if (st != SSD_OK) return st;
    return status_of(ssd::launch_scan_step(scan_shape(problem), a, h, (hipStream_t)stream));
}

ssd_status ssd_norm_validate(const ssd_norm_problem *problem) { return check_norm(problem); }

ssd_status ssd_norm(const ssd_norm_problem *problem, const void *x, const void *z,
                    const void *residual, const float *weight, void *y, void *residual_out,
                    void *stream)
{
    ssd_status st = check_norm(problem);
    if (st != SSD_OK) return st;
    if (!x || !weight || !y || (residual_out && !residual)) return SSD_ERR_NULL_ARG;
    if (!on_bytes(16, {weight})) return SSD_ERR_MISALIGNED;
    // a lane writes the elements that it has read: outputs may be inputs of their own layout
    const int64_t rows = problem->rows, width = problem->channels, e = bytes_of(problem->dtype);
    const int64_t re = bytes_of(problem->residual_dtype);
    st = check_apart({dense(y, rows * width * e), dense(residual_out, rows * width * re)},
                     {rows_of(x, rows, problem->x_pitch, width, e, true),
                      rows_of(z, rows, problem->z_pitch, width, e, true),
                      dense(residual, rows * width * re, true), dense(weight, width * 4)});
    if (st != SSD_OK) return st;
    ssd::NormShape s;
    s.rows = problem->rows; s.C = problem->channels; s.G = problem->ngroups;
    s.xp = problem->x_pitch ? problem->x_pitch : problem->channels;
    s.zp = problem->z_pitch ? problem->z_pitch : problem->channels;
    s.eps = problem->eps; s.scale = problem->scale;
    s.gate_after = problem->gate_after != 0;
    s.bf16 = problem->dtype == SSD_BF16;
    s.res_bf16 = problem->residual_dtype == SSD_BF16;
    return status_of(ssd::launch_norm(s, x, z, residual, weight, y, residual_out,
                                      (hipStream_t)stream));
}

}  // extern "C"
