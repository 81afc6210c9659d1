// ssd_linattn_step.hip -- linear attention with a decay for each head, one token per sequence:
//
//     h <- a h + v k^T,   o = scale h q,   a = exp(min(g, 0))
//
// in place on the fp32 state [value, key] of every (batch, head).  The step reads and writes the
// state once and does five operations for each of its elements: bound by HBM, or by launch latency at
// small batches.  A team of lanes holds a row, 16 bytes a lane, with its q and k in registers; a
// wave's teams take kRows rows each.
#include <hip/hip_runtime.h>

#include "ssd_device.h"
#include "ssd_launch.h"

namespace ssd {
namespace {

constexpr int kRows = 4;        // rows of a team
constexpr int kStepThreads = 256;

__device__ __forceinline__ f32x4 load4(const float *p) { return *reinterpret_cast<const f32x4 *>(p); }
__device__ __forceinline__ f32x4 load4(const bf16 *p)
{
    const bf16x4 v = *reinterpret_cast<const bf16x4 *>(p);
    return f32x4{(float)v[0], (float)v[1], (float)v[2], (float)v[3]};
}

struct StepDims {
    int64_t qp, kp, vp, gp;
    int H, share, dk, dv, decay;
    int blocks;              // waves of a head
    int64_t waves;
    float scale;
};

template <typename T, int TEAM>
__global__ __launch_bounds__(kStepThreads) void linattn_step_kernel(
    const T *__restrict__ q, const T *__restrict__ k, const T *v, const void *__restrict__ g,
    float *__restrict__ h, T *o, StepDims m)
{
    constexpr int kTeams = 64 / TEAM;
    const int lane = threadIdx.x & 63, team = lane / TEAM, key = lane % TEAM * 4;
    const int64_t wave = (int64_t)blockIdx.x * (kStepThreads / 64) + (threadIdx.x >> 6);
    if (wave >= m.waves) return;
    const int64_t bh = wave / m.blocks, b = bh / m.H;
    const int head = (int)(bh % m.H), row0 = (int)(wave % m.blocks) * kRows * kTeams + team;
    const bool in = key < m.dk;
    const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};

    float *hp = h + (bh * m.dv + row0) * m.dk + key;
    f32x4 s[kRows];
    float x[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        const bool row = row0 + r * kTeams < m.dv;
        s[r] = in && row ? load4(hp + (int64_t)r * kTeams * m.dk) : zero;
        x[r] = row ? (float)v[b * m.vp + (int64_t)head * m.dv + row0 + r * kTeams] : 0.0f;
    }
    const int64_t at = (int64_t)(head / m.share) * m.dk + key;
    const f32x4 kv = in ? load4(k + b * m.kp + at) : zero;
    const f32x4 qv = in ? load4(q + b * m.qp + at) : zero;
    float gv = 0.0f;
    if (m.decay == 1) gv = ((const float *)g)[head];
    if (m.decay == 2) gv = (float)((const T *)g)[b * m.gp + head];
    gv = gv > 0.0f ? 0.0f : gv;
    const float a = fast_exp2(gv * kLog2e);
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        float dot = 0.0f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            s[r][e] = fmaf(x[r], kv[e], a * s[r][e]);
            dot = fmaf(s[r][e], qv[e], dot);
        }
#pragma unroll
        for (int d = 1; d < TEAM; d <<= 1) dot += __shfl_xor(dot, d, 64);
        if (row0 + r * kTeams < m.dv) {
            if (in) *reinterpret_cast<f32x4 *>(hp + (int64_t)r * kTeams * m.dk) = s[r];
            if (key == 0) o[bh * m.dv + row0 + r * kTeams] = Elem<T>::from_f32(dot * m.scale);
        }
    }
}

template <typename T, int TEAM>
hipError_t step_go(const LinattnShape &s, const LinattnArgs &a, float *h, hipStream_t st)
{
    StepDims m;
    m.qp = s.qp; m.kp = s.kp; m.vp = s.vp; m.gp = s.gp;
    m.H = (int)s.H; m.share = (int)(s.H / s.G); m.dk = (int)s.dk; m.dv = (int)s.dv;
    m.decay = s.decay;
    constexpr int rows = kRows * (64 / TEAM);
    m.blocks = (int)((s.dv + rows - 1) / rows);
    m.waves = s.b * s.H * m.blocks;
    m.scale = s.scale;
    const int64_t groups = (m.waves + kStepThreads / 64 - 1) / (kStepThreads / 64);
    hipLaunchKernelGGL((linattn_step_kernel<T, TEAM>), dim3((unsigned)groups), dim3(kStepThreads), 0, st,
                       (const T *)a.q, (const T *)a.k, (const T *)a.v, a.g, h, (T *)a.o, m);
    return hipGetLastError();
}

template <typename T>
hipError_t step_by_key(const LinattnShape &s, const LinattnArgs &a, float *h, hipStream_t st)
{
    if (s.dk <= 8) return step_go<T, 2>(s, a, h, st);
    if (s.dk <= 16) return step_go<T, 4>(s, a, h, st);
    if (s.dk <= 32) return step_go<T, 8>(s, a, h, st);
    if (s.dk <= 64) return step_go<T, 16>(s, a, h, st);
    if (s.dk <= 128) return step_go<T, 32>(s, a, h, st);
    return step_go<T, 64>(s, a, h, st);
}

}  // namespace

hipError_t launch_linattn_step(const LinattnShape &s, const LinattnArgs &a, float *h, hipStream_t st)
{
    return s.bf16 ? step_by_key<bf16>(s, a, h, st) : step_by_key<float>(s, a, h, st);
}

}  // namespace ssd
