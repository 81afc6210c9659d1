// ssd_linattn_step.hip -- linear attention with a decay for each head, one token per sequence:
//
//     h <- a h + v k^T,   o = scale h q,   a = exp(min(g, 0))
//
// in place on the fp32 state [value, key] of every (batch, head).  The step reads and writes the
// state once and does five operations for each of its elements: bound by HBM, or by launch latency at
// small batches.  A team of lanes holds a row, 16 bytes a lane, with its q and k in registers; a
// wave's teams take kRows rows each (of 128 x 16 heads of 128 x 128 two take 50 us, four 49, eight
// 49; of 16 x 16 heads 7.7, 7.8 and 10.3).  A state too large to stay in the caches until the next step goes
// past them: 128 x 16 heads then take 49 us (5.5 TB/s) instead of 60, 16 x 16 7.8 instead of 9.8; 8 x 16,
// which stay in L2 when the same state steps again, 5.8 instead of 5.0.
#include <hip/hip_runtime.h>

#include "ssd_device.h"
#include "ssd_launch.h"

namespace ssd {
namespace {

constexpr int kStepThreads = 256;
constexpr int kRows = 4;        // rows of a team
constexpr int64_t kCached = 10 << 20;

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

// Streams: the state goes past the caches.
template <typename T, int TEAM, bool STREAM>
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
        const float *at = hp + (int64_t)r * kTeams * m.dk;
        s[r] = !(in && row) ? zero
               : STREAM     ? __builtin_nontemporal_load(reinterpret_cast<const f32x4 *>(at))
                            : load4(at);
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
    float dot[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        dot[r] = 0.0f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            s[r][e] = fmaf(x[r], kv[e], a * s[r][e]);
            dot[r] = fmaf(s[r][e], qv[e], dot[r]);
        }
        f32x4 *at = reinterpret_cast<f32x4 *>(hp + (int64_t)r * kTeams * m.dk);
        if (!in || row0 + r * kTeams >= m.dv) continue;
        if (STREAM)
            __builtin_nontemporal_store(s[r], at);
        else
            *at = s[r];
    }
    // Sums over the team: each exchange halves the rows that a lane adds up, then a row's lanes
    // exchange theirs.
    int first = 0;
#pragma unroll
    for (int d = 1, n = kRows; d < TEAM; d <<= 1) {
        if (n > 1) {
            n >>= 1;
            const bool upper = lane & d;
            first += upper ? n : 0;
#pragma unroll
            for (int r = 0; r < n; ++r) {
                const float other = __shfl_xor(upper ? dot[r] : dot[r + n], d, 64);
                dot[r] = (upper ? dot[r + n] : dot[r]) + other;
            }
        } else {
            dot[0] += __shfl_xor(dot[0], d, 64);
        }
    }
    if ((lane % TEAM) >= kRows) return;        // another lane's row
#pragma unroll
    for (int r = 0; r < (TEAM < kRows ? kRows / TEAM : 1); ++r) {
        const int row = row0 + (first + r) * kTeams;
        if (row < m.dv) o[bh * m.dv + row] = Elem<T>::from_f32(dot[r] * m.scale);
    }
}

template <typename T, int TEAM, bool STREAM>
hipError_t step_team(const LinattnShape &s, const LinattnArgs &a, float *h, hipStream_t st)
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
    hipLaunchKernelGGL((linattn_step_kernel<T, TEAM, STREAM>), dim3((unsigned)groups), dim3(kStepThreads), 0, st,
                       (const T *)a.q, (const T *)a.k, (const T *)a.v, a.g, h, (T *)a.o, m);
    return hipGetLastError();
}

template <typename T, int TEAM>
hipError_t step_go(const LinattnShape &s, const LinattnArgs &a, float *h, hipStream_t st)
{
    return s.b * s.H * s.dv * s.dk * 4 <= kCached ? step_team<T, TEAM, false>(s, a, h, st)
                                                  : step_team<T, TEAM, true>(s, a, h, st);
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
