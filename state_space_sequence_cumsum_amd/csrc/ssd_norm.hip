// ssd_norm.hip -- the RMS norms before and after a block, fused with the block's gate and
// with the scaled residual addition.
//
//     v = x;  gate first: v *= silu(z);  residual: v = residual + scale v (stored)
//     y = v rsqrt(mean_group(v^2) + eps) weight;  gate after: y *= silu(z)
//
// One pass: a team of lanes -- a power of two up to a wave, or a workgroup -- owns a row's
// group, loads all of it (16 bytes a lane, up to 8 times; single elements where rows do not
// start on 16 bytes) and keeps it in registers from the sum of squares to the scaled output, so
// every element is read and written once: HBM bound.  Teams walk over rows with their weights
// in registers.
//
// Measured (inputs not in the caches): gated norm of 16384 x 2048 bf16, z a slice of rows of
// 4640, 42 us (4.8 TB/s; a copy kernel reaches 6.2; read twice by a workgroup a row: 143 us),
// with a fp32 residual stream 77 us (5.2 TB/s), 3000 x 1001 bf16 in single elements 7.9 us
// (2.3 TB/s), 128 x 1024 with residual 3.9 us, most of it the launch.
#include <hip/hip_runtime.h>

#include "ssd_device.h"
#include "ssd_launch.h"

namespace ssd {
namespace {

constexpr int kNormThreads = 256;

__device__ __forceinline__ float silu(float v)
{
    return v * __builtin_amdgcn_rcpf(1.0f + fast_exp2(-kLog2e * v));
}

// V neighbouring elements as one vector (a plain element for V = 1).
template <typename T, int V> struct Vec {
    typedef T type __attribute__((ext_vector_type(V), aligned(16)));
    type v;
    __device__ __forceinline__ void load(const T *p) { v = *reinterpret_cast<const type *>(p); }
    __device__ __forceinline__ void store(T *p) const { *reinterpret_cast<type *>(p) = v; }
    __device__ __forceinline__ float get(int i) const { return (float)v[i]; }
    __device__ __forceinline__ void set(int i, float f) { v[i] = Elem<T>::from_f32(f); }
};
template <typename T> struct Vec<T, 1> {
    T v;
    __device__ __forceinline__ void load(const T *p) { v = *p; }
    __device__ __forceinline__ void store(T *p) const { *p = v; }
    __device__ __forceinline__ float get(int) const { return (float)v; }
    __device__ __forceinline__ void set(int, float f) { v = Elem<T>::from_f32(f); }
};

template <typename T, typename R> struct NormArgs {
    const T *x, *z;
    const R *residual;
    const float *weight;
    T *y;
    R *residual_out;
    int64_t xp, zp;
    int items, teams;        // (row, group) pairs; teams, a multiple of G, that share them
    int C, Cg, G, log_lanes; // log_lanes: lanes of a team (up to 64; not kWide)
    float eps, scale;
    int gate_after;
};

// The sum over a team's lanes, in all of them.
template <bool kWide> __device__ __forceinline__ float team_sum(float v, int lanes, float *part)
{
    for (int k = (kWide ? 64 : lanes) >> 1; k >= 1; k >>= 1) v += __shfl_xor(v, k, 64);
    if (kWide) {
        __syncthreads();       // the previous row's sums have been read
        if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
        __syncthreads();
        v = (part[0] + part[1]) + (part[2] + part[3]);
    }
    return v;
}

// kRegs vectors of V elements per lane hold a whole row's group.
template <typename T, typename R, int V, int kRegs, bool kWide>
__global__ __launch_bounds__(kNormThreads) void norm_kernel(NormArgs<T, R> a)
{
    __shared__ float part[kNormThreads / 64];
    const int lanes = kWide ? kNormThreads : 1 << a.log_lanes;
    const int lane = threadIdx.x & (lanes - 1);
    const int team = kWide ? blockIdx.x : (blockIdx.x * kNormThreads + threadIdx.x) >> a.log_lanes;
    if (team >= a.teams) return;       // a whole workgroup where there are barriers
    const int g = team % a.G;
    const int64_t row0 = team / a.G, step = a.teams / a.G;
    const int c0 = g * a.Cg + lane * V;
    const int left = a.Cg - lane * V;  // channels from this lane's first vector to the group's end
    const int jump = lanes * V;

    Vec<float, V> w[kRegs];
#pragma unroll
    for (int k = 0; k < kRegs; ++k)
        if (k * jump < left) w[k].load(a.weight + c0 + k * jump);
    const float inv = 1.0f / (float)a.Cg;
    const bool first = a.z && !a.gate_after, after = a.z && a.gate_after;

    const T *x = a.x + row0 * a.xp + c0, *z = a.z + row0 * a.zp + c0;
    const R *res = a.residual + row0 * a.C + c0;
    T *y = a.y + row0 * a.C + c0;
    R *ro = a.residual_out + row0 * a.C + c0;
    for (int item = team; item < a.items; item += a.teams) {
        Vec<T, V> xv[kRegs], zv[kRegs];
        Vec<R, V> rv[kRegs];
#pragma unroll
        for (int k = 0; k < kRegs; ++k)
            if (k * jump < left) {
                xv[k].load(x + k * jump);
                if (a.z) zv[k].load(z + k * jump);
                if (a.residual) rv[k].load(res + k * jump);
            }
        float v[kRegs][V], sum = 0.0f;
#pragma unroll
        for (int k = 0; k < kRegs; ++k) {
            const bool on = k * jump < left;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                float f = xv[k].get(i);
                if (first) f *= silu(zv[k].get(i));
                if (a.residual) f = fmaf(a.scale, f, rv[k].get(i));
                v[k][i] = f;
                if (on) sum = fmaf(f, f, sum);
            }
        }
        const float r = __builtin_amdgcn_rsqf(fmaf(team_sum<kWide>(sum, lanes, part), inv, a.eps));
        // a lane writes the residual elements that it has read: the two may be one buffer
#pragma unroll
        for (int k = 0; k < kRegs; ++k)
            if (k * jump < left) {
                Vec<T, V> o;
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    float f = v[k][i] * r * w[k].get(i);
                    if (after) f *= silu(zv[k].get(i));
                    o.set(i, f);
                }
                o.store(y + k * jump);
                if (a.residual_out) {
                    Vec<R, V> s;
#pragma unroll
                    for (int i = 0; i < V; ++i) s.set(i, v[k][i]);
                    s.store(ro + k * jump);
                }
            }
        x += step * a.xp;
        z += step * a.zp;
        res += step * a.C;
        y += step * a.C;
        ro += step * a.C;
    }
}

// Groups that no team can hold: a workgroup per (row, group) reads them twice.
template <typename T, typename R, int V>
__global__ __launch_bounds__(kNormThreads) void norm_long_kernel(NormArgs<T, R> a)
{
    __shared__ float part[kNormThreads / 64];
    const int64_t row = blockIdx.x / a.G;
    const int c0 = (int)(blockIdx.x % a.G) * a.Cg;
    const bool first = a.z && !a.gate_after, after = a.z && a.gate_after;
    auto values = [&](int c, float *v, Vec<T, V> &zv) {
        Vec<T, V> xv;
        Vec<R, V> rv;
        xv.load(a.x + row * a.xp + c);
        if (a.z) zv.load(a.z + row * a.zp + c);
        if (a.residual) rv.load(a.residual + row * a.C + c);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            v[i] = xv.get(i);
            if (first) v[i] *= silu(zv.get(i));
            if (a.residual) v[i] = fmaf(a.scale, v[i], rv.get(i));
        }
    };
    float sum = 0.0f;
    for (int i = threadIdx.x * V; i < a.Cg; i += kNormThreads * V) {
        float v[V];
        Vec<T, V> zv;
        values(c0 + i, v, zv);
#pragma unroll
        for (int k = 0; k < V; ++k) sum = fmaf(v[k], v[k], sum);
    }
    const float r = __builtin_amdgcn_rsqf(
        fmaf(team_sum<true>(sum, kNormThreads, part), 1.0f / (float)a.Cg, a.eps));
    for (int i = threadIdx.x * V; i < a.Cg; i += kNormThreads * V) {
        const int c = c0 + i;
        float v[V];
        Vec<T, V> zv, o;
        Vec<float, V> w;
        Vec<R, V> s;
        values(c, v, zv);
        w.load(a.weight + c);
#pragma unroll
        for (int k = 0; k < V; ++k) {
            float f = v[k] * r * w.get(k);
            if (after) f *= silu(zv.get(k));
            o.set(k, f);
            s.set(k, v[k]);
        }
        o.store(a.y + row * a.C + c);
        if (a.residual_out) s.store(a.residual_out + row * a.C + c);
    }
}

template <typename T, typename R, int V, int kRegs, bool kWide>
hipError_t norm_go(NormArgs<T, R> a, hipStream_t st)
{
    // 32 waves a CU at most: teams that walk over several rows (200000 rows of 64: 12.5 us, 13.2
    // with a team a row; 16 waves a CU: 13.0)
    const int per_block = kWide ? 1 : kNormThreads >> a.log_lanes;
    const int most = 256 * 8 * per_block;
    a.teams = a.items < most ? a.items : most / a.G * a.G;
    if (a.teams < a.G) a.teams = a.G;
    const unsigned blocks = (unsigned)((a.teams + per_block - 1) / per_block);
    hipLaunchKernelGGL((norm_kernel<T, R, V, kRegs, kWide>), dim3(blocks), dim3(kNormThreads), 0,
                       st, a);
    return hipGetLastError();
}

// The smallest team that holds a group in its registers: part of a wave with one vector a lane,
// a wave with up to 4 (16 single elements), a workgroup with up to 8 (16).  Eight vectors of bf16
// take all 256 registers and up to 45 accumulation registers, one wave a SIMD: gated rows of 16384
// run at 3.6 TB/s, with a fp32 residual at 4.9, where rows of 8192 reach 5.5 and 5.0; rows that are
// read twice (16392 channels) at 3.4 and 3.7.
template <typename T, typename R, int V> hipError_t norm_team(NormArgs<T, R> a, hipStream_t st)
{
    constexpr int kWave = V == 1 ? 16 : 4, kGroup = V == 1 ? 16 : 8;
    const int vectors = a.Cg / V;
    if (vectors <= 64) {
        a.log_lanes = 0;
        while (1 << a.log_lanes < vectors) ++a.log_lanes;
        return norm_go<T, R, V, 1, false>(a, st);
    }
    if (vectors <= 64 * kWave / 2) return norm_go<T, R, V, kWave / 2, false>(a, st);
    if (vectors <= 64 * kWave) return norm_go<T, R, V, kWave, false>(a, st);
    if constexpr (kGroup / 4 * kNormThreads > 64 * kWave)     // (single elements: a wave's reach)
        if (vectors <= kNormThreads * kGroup / 4) return norm_go<T, R, V, kGroup / 4, true>(a, st);
    if (vectors <= kNormThreads * kGroup / 2) return norm_go<T, R, V, kGroup / 2, true>(a, st);
    if (vectors <= kNormThreads * kGroup) return norm_go<T, R, V, kGroup, true>(a, st);
    hipLaunchKernelGGL((norm_long_kernel<T, R, V>), dim3((unsigned)a.items), dim3(kNormThreads), 0,
                       st, a);
    return hipGetLastError();
}

bool on16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

template <typename T, typename R>
hipError_t norm_wide(const NormShape &s, const void *x, const void *z, const void *residual,
                     const float *weight, void *y, void *residual_out, hipStream_t st)
{
    constexpr int V = 16 / sizeof(T);
    NormArgs<T, R> a;
    a.x = (const T *)x; a.z = (const T *)z; a.residual = (const R *)residual;
    a.weight = weight; a.y = (T *)y; a.residual_out = (R *)residual_out;
    a.xp = s.xp; a.zp = s.zp; a.items = (int)(s.rows * s.G); a.teams = a.items;
    a.C = (int)s.C; a.Cg = (int)(s.C / s.G); a.G = (int)s.G; a.log_lanes = 6;
    a.eps = s.eps; a.scale = s.scale; a.gate_after = s.gate_after;
    // every row's group starts on 16 bytes
    if (a.Cg % V == 0 && s.xp % V == 0 && (!z || s.zp % V == 0) && on16(x) && on16(z) &&
        on16(residual) && on16(y) && on16(residual_out))
        return norm_team<T, R, V>(a, st);
    return norm_team<T, R, 1>(a, st);
}

}  // namespace

hipError_t launch_norm(const NormShape &s, const void *x, const void *z, const void *residual,
                       const float *weight, void *y, void *residual_out, hipStream_t st)
{
    if (!s.bf16) return norm_wide<float, float>(s, x, z, residual, weight, y, residual_out, st);
    if (s.res_bf16) return norm_wide<bf16, bf16>(s, x, z, residual, weight, y, residual_out, st);
    return norm_wide<bf16, float>(s, x, z, residual, weight, y, residual_out, st);
}

}  // namespace ssd
