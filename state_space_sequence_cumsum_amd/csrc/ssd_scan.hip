// ssd_scan.hip -- the selective state space scan (a decay rate per channel and state, a step
// size per token and channel), for prompts and for single tokens.
//
//     d_t[c]    = dt_t[c] + dt_bias[c], through softplus where asked
//     h_t[c, n] = exp(d_t[c] A[c, n]) h_{t-1}[c, n] + d_t[c] x_t[c] B_t[g, n]
//     y_t[c]    = (sum_n C_t[g, n] h_t[c, n] + D[c] x_t[c]) silu(z_t[c])
//
// One lane owns a channel and keeps its N states and rates in registers; B_t and C_t are the
// same for all lanes of a wave (one group per wave), so they come through scalar loads and
// enter the products as scalar operands.  Per state and token: a product, an exp2 and three
// more VALU operations, which bound the kernel before HBM does.
#include <hip/hip_runtime.h>

#include "ssd_device.h"
#include "ssd_launch.h"

namespace ssd {
namespace {

__device__ __forceinline__ float silu(float v)
{
    return v * __builtin_amdgcn_rcpf(1.0f + fast_exp2(-kLog2e * v));
}

// log(1 + exp(v)) = max(v, 0) + log1p(e), e = exp(-|v|) in (0, 1], with
// log1p(e) = 2 atanh(s), s = e / (2 + e) in (0, 1/3]; atanh(s) / s is a polynomial in s^2
// (degree 4, interpolated at the Chebyshev points of [0, 1/9]: relative error 4.1e-9), so small
// step sizes keep their relative accuracy (log2(1 + e) would not).
__device__ __forceinline__ float softplus(float v)
{
    const float e = fast_exp2(-kLog2e * fabsf(v));
    const float s = e * __builtin_amdgcn_rcpf(2.0f + e);
    const float q = s * s;
    float p = 0.14078889f;
    p = fmaf(p, q, 0.13982579f);
    p = fmaf(p, q, 0.20012298f);
    p = fmaf(p, q, 0.33333161f);
    p = fmaf(p, q, 1.0f);
    return fmaf(2.0f * s, p, fmaxf(v, 0.0f));
}

struct ScanDims {
    int64_t L, xp, dtp, zp, Bp, Cp;
    int C, Cg, tiles;      // channels, channels per group, 64-channel tiles per group
    int G;
    int sp;                // 1: softplus
};

template <typename T, int N>
__global__ __launch_bounds__(64) void scan_kernel(
    const T *__restrict__ x, const T *__restrict__ dt, const float *__restrict__ A,
    const T *__restrict__ B, const T *__restrict__ Cm, const float *__restrict__ D,
    const T *__restrict__ z, const float *__restrict__ dt_bias, const float *h0,
    const int32_t *__restrict__ lengths, T *__restrict__ y, float *hT, ScanDims m)
{
    const int tile = blockIdx.x % m.tiles;
    const int g = blockIdx.x / m.tiles % m.G;
    const int64_t b = blockIdx.x / m.tiles / m.G;
    const int in_group = tile * 64 + threadIdx.x;
    const bool live = in_group < m.Cg;
    const int c = g * m.Cg + min(in_group, m.Cg - 1);
    int64_t len = m.L;
    if (lengths) len = min((int64_t)max(lengths[b], 0), m.L);

    float a2[N], h[N];
#pragma unroll
    for (int n = 0; n < N; ++n) a2[n] = kLog2e * A[(int64_t)c * N + n];
#pragma unroll
    for (int n = 0; n < N; ++n) h[n] = h0 ? h0[(b * m.C + c) * N + n] : 0.0f;
    const float bias = dt_bias ? dt_bias[c] : 0.0f;
    const float Dv = D ? D[c] : 0.0f;
    const T *xr = x + b * m.L * m.xp, *dr = dt + b * m.L * m.dtp;
    const T *zr = z ? z + b * m.L * m.zp : nullptr;
    const T *Br = B + b * m.L * m.Bp + g * N, *Cr = Cm + b * m.L * m.Cp + g * N;
    T *yr = y + b * m.L * m.C;
    for (int64_t t = 0; t < len; ++t) {
        const float xv = (float)xr[t * m.xp + c];
        float d = (float)dr[t * m.dtp + c] + bias;
        if (m.sp) d = softplus(d);
        const float u = d * xv;
        float acc = Dv * xv;
#pragma unroll
        for (int n = 0; n < N; ++n) {
            h[n] = fmaf(fast_exp2(d * a2[n]), h[n], u * (float)Br[t * m.Bp + n]);
            acc = fmaf((float)Cr[t * m.Cp + n], h[n], acc);
        }
        if (zr) acc *= silu((float)zr[t * m.zp + c]);
        if (live) yr[t * m.C + c] = Elem<T>::from_f32(acc);
    }
    if (hT && live) {
#pragma unroll
        for (int n = 0; n < N; ++n) hT[(b * m.C + c) * N + n] = h[n];
    }
}

// One token: a lane owns a channel.
template <typename T, int N>
__global__ __launch_bounds__(64) void scan_step_kernel(
    const T *__restrict__ x, const T *__restrict__ dt, const float *__restrict__ A,
    const T *__restrict__ B, const T *__restrict__ Cm, const float *__restrict__ D,
    const T *__restrict__ z, const float *__restrict__ dt_bias, float *__restrict__ hp,
    T *__restrict__ y, ScanDims m)
{
    const int tile = blockIdx.x % m.tiles;
    const int g = blockIdx.x / m.tiles % m.G;
    const int64_t b = blockIdx.x / m.tiles / m.G;
    const int in_group = tile * 64 + threadIdx.x;
    if (in_group >= m.Cg) return;
    const int c = g * m.Cg + in_group;
    const float xv = (float)x[b * m.xp + c];
    float d = (float)dt[b * m.dtp + c] + (dt_bias ? dt_bias[c] : 0.0f);
    if (m.sp) d = softplus(d);
    const float u = d * xv;
    float acc = D ? D[c] * xv : 0.0f;
    float *h = hp + (b * m.C + c) * N;
#pragma unroll
    for (int n = 0; n < N; ++n) {
        const float v = fmaf(fast_exp2(d * (kLog2e * A[(int64_t)c * N + n])), h[n],
                             u * (float)B[b * m.Bp + g * N + n]);
        h[n] = v;
        acc = fmaf((float)Cm[b * m.Cp + g * N + n], v, acc);
    }
    if (z) acc *= silu((float)z[b * m.zp + c]);
    y[b * m.C + c] = Elem<T>::from_f32(acc);
}

ScanDims dims_of(const ScanShape &s)
{
    ScanDims m;
    m.L = s.L; m.xp = s.xp; m.dtp = s.dtp; m.zp = s.zp; m.Bp = s.Bp; m.Cp = s.Cp;
    m.C = (int)s.C; m.G = (int)s.G; m.Cg = (int)(s.C / s.G);
    m.tiles = (m.Cg + 63) / 64;
    m.sp = s.softplus;
    return m;
}

template <typename T, int N>
hipError_t scan_go(const ScanShape &s, const ScanArgs &a, float *h, hipStream_t st)
{
    const ScanDims m = dims_of(s);
    const dim3 grid((unsigned)scan_workgroups(s));
    if (h)
        hipLaunchKernelGGL((scan_step_kernel<T, N>), grid, dim3(64), 0, st, (const T *)a.x,
                           (const T *)a.dt, a.A, (const T *)a.B, (const T *)a.C, a.D,
                           (const T *)a.z, a.dt_bias, h, (T *)a.y, m);
    else
        hipLaunchKernelGGL((scan_kernel<T, N>), grid, dim3(64), 0, st, (const T *)a.x,
                           (const T *)a.dt, a.A, (const T *)a.B, (const T *)a.C, a.D,
                           (const T *)a.z, a.dt_bias, a.h0, a.lengths, (T *)a.y, a.hT, m);
    return hipGetLastError();
}

template <typename T>
hipError_t scan_by_state(const ScanShape &s, const ScanArgs &a, float *h, hipStream_t st)
{
    switch (s.N) {
    case 8: return scan_go<T, 8>(s, a, h, st);
    case 16: return scan_go<T, 16>(s, a, h, st);
    case 24: return scan_go<T, 24>(s, a, h, st);
    case 32: return scan_go<T, 32>(s, a, h, st);
    case 40: return scan_go<T, 40>(s, a, h, st);
    case 48: return scan_go<T, 48>(s, a, h, st);
    case 56: return scan_go<T, 56>(s, a, h, st);
    case 64: return scan_go<T, 64>(s, a, h, st);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace

size_t scan_workspace_bytes(const ScanShape &) { return 256; }

int64_t scan_workgroups(const ScanShape &s)
{
    const ScanDims m = dims_of(s);
    return (int64_t)m.tiles * m.G * s.b;
}
int64_t scan_step_workgroups(const ScanShape &s) { return scan_workgroups(s); }

hipError_t launch_scan(const ScanShape &s, const ScanArgs &a, hipStream_t st)
{
    return s.bf16 ? scan_by_state<bf16>(s, a, nullptr, st) : scan_by_state<float>(s, a, nullptr, st);
}

hipError_t launch_scan_step(const ScanShape &s, const ScanArgs &a, float *h, hipStream_t st)
{
    return s.bf16 ? scan_by_state<bf16>(s, a, h, st) : scan_by_state<float>(s, a, h, st);
}

}  // namespace ssd
