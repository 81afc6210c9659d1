// ssd_conv.hip -- the short causal depthwise convolution in front of the SSD forward, for
// prompts and for single tokens.
//
//     v[b, t, c] = bias[c] + sum_{k < K} w[c, k] u[b, t - K + 1 + k, c]
//     y          = silu(v) or v,          u at t < 0 from the state (K - 1 rows, oldest first)
//
// K is 2 to 4: each input element is read once from HBM and once more for every token tile
// that it is a halo of, and 2 K + 5 flops an element leave the kernel bound by HBM.
#include <hip/hip_runtime.h>

#include "ssd_device.h"
#include "ssd_launch.h"

namespace ssd {
namespace {

constexpr int kConvThreads = 256;   // channels per workgroup
constexpr int kConvTokens = 32;     // tokens per workgroup

__device__ __forceinline__ float silu(float v)
{
    return v * __builtin_amdgcn_rcpf(1.0f + fast_exp2(-kLog2e * v));
}

// Output element (token row `row` of b L rows, channel c): the three outputs are dense and
// stand for the channels [0, w0), [w0, w0 + w1) and [w0 + w1, C).
template <typename T> struct ConvOut {
    T *y0, *y1, *y2;
    int w0, w1, w2;
    __device__ __forceinline__ void put(int64_t row, int c, T v) const
    {
        if (c < w0) y0[row * w0 + c] = v;
        else if (c < w0 + w1) y1[row * w1 + (c - w0)] = v;
        else y2[row * w2 + (c - w0 - w1)] = v;
    }
};

template <typename T, int K>
__global__ __launch_bounds__(kConvThreads) void conv_kernel(
    const T *__restrict__ x, const float *__restrict__ w, const float *__restrict__ bias,
    const T *state0, const int32_t *__restrict__ lengths, ConvOut<T> out, T *stateT, int L, int C,
    int64_t pitch, int nct, int ntt, bool act)
{
    const int ct = blockIdx.x % nct;
    const int tt = blockIdx.x / nct % ntt;
    const int64_t b = blockIdx.x / nct / ntt;
    const int c = ct * kConvThreads + threadIdx.x;
    if (c >= C) return;
    int len = L;
    if (lengths) len = min(max(lengths[b], 0), L);
    const T *xb = x + b * L * pitch + c;
    float wk[K], win[K];
#pragma unroll
    for (int k = 0; k < K; ++k) wk[k] = w[(int64_t)c * K + k];
    const float bv = bias ? bias[c] : 0.0f;

    const int t0 = tt * kConvTokens;
    T first[K - 1];
#pragma unroll
    for (int k = 0; k < K - 1; ++k)
        first[k] = (tt == 0 && state0) ? state0[(b * (K - 1) + k) * C + c] : (T)0.0f;
    // win[k] = u[t - K + 1 + k]
#pragma unroll
    for (int k = 0; k < K - 1; ++k) {
        const int t = t0 - (K - 1) + k;
        win[k + 1] = tt == 0 ? (float)first[k] : (t < len ? (float)xb[t * pitch] : 0.0f);
    }
    const int t1 = min(t0 + kConvTokens, len);
    for (int t = t0; t < t1; ++t) {
#pragma unroll
        for (int k = 0; k + 1 < K; ++k) win[k] = win[k + 1];
        win[K - 1] = (float)xb[t * pitch];
        float v = bv;
#pragma unroll
        for (int k = 0; k < K; ++k) v = fmaf(wk[k], win[k], v);
        out.put(b * L + t, c, Elem<T>::from_f32(act ? silu(v) : v));
    }
    // The first token tile's threads, which alone read state0, write stateT: the two may be
    // one buffer.
    if (tt == 0 && stateT) {
#pragma unroll
        for (int k = 0; k < K - 1; ++k) {
            const int t = len - (K - 1) + k;
            T v = (T)0.0f;
            if (t >= 0) {
                v = xb[t * pitch];
            } else {
#pragma unroll
                for (int j = 0; j < K - 1; ++j)
                    if (j == t + K - 1) v = first[j];
            }
            stateT[(b * (K - 1) + k) * C + c] = v;
        }
    }
}

template <typename T, int K>
__global__ __launch_bounds__(kConvThreads) void conv_step_kernel(
    const T *__restrict__ x, const float *__restrict__ w, const float *__restrict__ bias,
    T *__restrict__ state, ConvOut<T> out, int C, int64_t pitch, int nct, bool act)
{
    const int ct = blockIdx.x % nct;
    const int64_t b = blockIdx.x / nct;
    const int c = ct * kConvThreads + threadIdx.x;
    if (c >= C) return;
    T *sp = state + b * (K - 1) * C + c;
    T u[K];
#pragma unroll
    for (int k = 0; k < K - 1; ++k) u[k] = sp[(int64_t)k * C];
    u[K - 1] = x[b * pitch + c];
    float v = bias ? bias[c] : 0.0f;
#pragma unroll
    for (int k = 0; k < K; ++k) v = fmaf(w[(int64_t)c * K + k], (float)u[k], v);
#pragma unroll
    for (int k = 0; k < K - 1; ++k) sp[(int64_t)k * C] = u[k + 1];
    out.put(b, c, Elem<T>::from_f32(act ? silu(v) : v));
}

template <typename T> ConvOut<T> out_of(const ConvShape &s, void *y0, void *y1, void *y2)
{
    return {(T *)y0, (T *)y1, (T *)y2, (int)s.w0, (int)s.w1, (int)s.w2};
}

int channel_tiles(const ConvShape &s) { return (int)((s.C + kConvThreads - 1) / kConvThreads); }
int token_tiles(const ConvShape &s) { return (int)((s.L + kConvTokens - 1) / kConvTokens); }

int64_t conv_workgroups(const ConvShape &s)
{
    return (int64_t)channel_tiles(s) * token_tiles(s) * s.b;
}

template <typename T, int K>
hipError_t conv_go(const ConvShape &s, const void *x, const float *w, const float *bias,
                   const void *state0, const int32_t *lengths, void *y0, void *y1, void *y2,
                   void *stateT, hipStream_t st)
{
    hipLaunchKernelGGL((conv_kernel<T, K>), dim3((unsigned)conv_workgroups(s)), dim3(kConvThreads),
                       0, st, (const T *)x, w, bias, (const T *)state0, lengths,
                       out_of<T>(s, y0, y1, y2), (T *)stateT, (int)s.L, (int)s.C, s.pitch,
                       channel_tiles(s), token_tiles(s), s.silu);
    return hipGetLastError();
}

template <typename T, int K>
hipError_t step_go(const ConvShape &s, const void *x, const float *w, const float *bias,
                   void *state, void *y0, void *y1, void *y2, hipStream_t st)
{
    hipLaunchKernelGGL((conv_step_kernel<T, K>), dim3((unsigned)conv_workgroups(s)),
                       dim3(kConvThreads), 0, st, (const T *)x, w, bias, (T *)state,
                       out_of<T>(s, y0, y1, y2), (int)s.C, s.pitch, channel_tiles(s), s.silu);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_conv(const ConvShape &s, const void *x, const float *w, const float *bias,
                       const void *state0, const int32_t *lengths, void *y0, void *y1, void *y2,
                       void *stateT, hipStream_t st)
{
#define SSD_CONV(T, K) return conv_go<T, K>(s, x, w, bias, state0, lengths, y0, y1, y2, stateT, st)
    if (s.bf16) {
        if (s.K == 2) SSD_CONV(bf16, 2);
        if (s.K == 3) SSD_CONV(bf16, 3);
        SSD_CONV(bf16, 4);
    }
    if (s.K == 2) SSD_CONV(float, 2);
    if (s.K == 3) SSD_CONV(float, 3);
    SSD_CONV(float, 4);
#undef SSD_CONV
}

hipError_t launch_conv_step(const ConvShape &s, const void *x, const float *w, const float *bias,
                            void *state, void *y0, void *y1, void *y2, hipStream_t st)
{
#define SSD_CONV(T, K) return step_go<T, K>(s, x, w, bias, state, y0, y1, y2, st)
    if (s.bf16) {
        if (s.K == 2) SSD_CONV(bf16, 2);
        if (s.K == 3) SSD_CONV(bf16, 3);
        SSD_CONV(bf16, 4);
    }
    if (s.K == 2) SSD_CONV(float, 2);
    if (s.K == 3) SSD_CONV(float, 3);
    SSD_CONV(float, 4);
#undef SSD_CONV
}

}  // namespace ssd
