// ssd_norm.hip -- the RMS norms before and after a block, fused with the block's gate and
// with the scaled residual addition.
//
//     v = x;  gate first: v *= silu(z);  residual: v = residual + scale v (stored)
//     y = v rsqrt(mean_group(v^2) + eps) weight;  gate after: y *= silu(z)
//
// Each element is read and written once; HBM bound.
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

template <typename T, typename R>
__global__ __launch_bounds__(kNormThreads) void norm_kernel(
    const T *__restrict__ x, const T *__restrict__ z, const R *residual,
    const float *__restrict__ weight, T *__restrict__ y, R *residual_out, int C, int Cg,
    int64_t xp, int64_t zp, int G, float eps, float scale, bool gate_after)
{
    __shared__ float part[kNormThreads / 64];
    const int64_t row = blockIdx.x / G;
    const int c0 = (int)(blockIdx.x % G) * Cg;
    auto value = [&](int c) {
        float v = (float)x[row * xp + c];
        if (z && !gate_after) v *= silu((float)z[row * zp + c]);
        if (residual) v = fmaf(scale, v, (float)residual[row * C + c]);
        return v;
    };
    float sum = 0.0f;
    for (int i = threadIdx.x; i < Cg; i += kNormThreads) {
        const float v = value(c0 + i);
        sum = fmaf(v, v, sum);
    }
#pragma unroll
    for (int k = 32; k >= 1; k >>= 1) sum += __shfl_xor(sum, k, 64);
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = sum;
    __syncthreads();
    sum = part[0] + part[1] + part[2] + part[3];
    const float r = 1.0f / sqrtf(sum / (float)Cg + eps);
    // each thread reads its own elements of residual before it writes them: residual_out may
    // be the same buffer
    for (int i = threadIdx.x; i < Cg; i += kNormThreads) {
        const int c = c0 + i;
        const float v = value(c);
        float o = v * r * weight[c];
        if (z && gate_after) o *= silu((float)z[row * zp + c]);
        if (residual_out) residual_out[row * C + c] = Elem<R>::from_f32(v);
        y[row * C + c] = Elem<T>::from_f32(o);
    }
}

int64_t norm_workgroups(const NormShape &s) { return s.rows * s.G; }

template <typename T, typename R>
hipError_t norm_go(const NormShape &s, const void *x, const void *z, const void *residual,
                   const float *weight, void *y, void *residual_out, hipStream_t st)
{
    hipLaunchKernelGGL((norm_kernel<T, R>), dim3((unsigned)norm_workgroups(s)),
                       dim3(kNormThreads), 0, st, (const T *)x, (const T *)z, (const R *)residual,
                       weight, (T *)y, (R *)residual_out, (int)s.C, (int)(s.C / s.G), s.xp, s.zp,
                       (int)s.G, s.eps, s.scale, s.gate_after);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_norm(const NormShape &s, const void *x, const void *z, const void *residual,
                       const float *weight, void *y, void *residual_out, hipStream_t st)
{
    if (!s.bf16) return norm_go<float, float>(s, x, z, residual, weight, y, residual_out, st);
    if (s.res_bf16) return norm_go<bf16, bf16>(s, x, z, residual, weight, y, residual_out, st);
    return norm_go<bf16, float>(s, x, z, residual, weight, y, residual_out, st);
}

}  // namespace ssd
