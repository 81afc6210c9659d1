// ssd_conv.hip -- the short causal depthwise convolution in front of the SSD forward, for
// prompts and for single tokens.
//
//     v[b, t, c] = bias[c] + sum_{k < K} w[c, k] u[b, t - K + 1 + k, c]
//     y          = silu(v) or v,          u at t < 0 from the state (K - 1 rows, oldest first)
//
// A thread owns 16 bytes of neighbouring channels (one channel where rows do not start on 16
// bytes) and walks a tile of tokens with the K - 1 inputs before the next one in registers, so
// an input is read once, and once more for each later tile it is a halo of (K - 1 rows in 8 to
// 32, from the caches).  2 K + 5 flops an element: HBM bound.  Three outputs, so that the x, B
// and C columns of a block's projection come out as ssd_forward takes them.
//
// Measured (inputs not in the caches): 16384 x 2560 bf16, a slice of rows of 4640, 39 to 41 us
// (4.2 TB/s; a copy kernel reaches 6.2), 262144 x 1536 bf16 299 us (5.4 TB/s), 5 x 2500 x 777
// bf16 one channel a thread 14.0 us (2.8 TB/s); 256 x 384 fp32 4.2 us, most of it the launch.

#include <hip/hip_runtime.h>

#include <type_traits>

#include "ssd_device.h"
#include "ssd_launch.h"

namespace ssd {
namespace {

constexpr int kConvThreads = 256;

__device__ __forceinline__ float silu(float v)
{
    return v * __builtin_amdgcn_rcpf(1.0f + fast_exp2(-kLog2e * v));
}

// V neighbouring channels of one row: 16 bytes where V > 1.
template <typename T, int V> struct Chans {
    typedef T vec __attribute__((ext_vector_type(V)));
    vec v;
    __device__ __forceinline__ void load(const T *p) { v = *reinterpret_cast<const vec *>(p); }
    __device__ __forceinline__ void store(T *p) const { *reinterpret_cast<vec *>(p) = v; }
    __device__ __forceinline__ float get(int i) const { return (float)v[i]; }
    __device__ __forceinline__ void set(int i, float f) { v[i] = Elem<T>::from_f32(f); }
    __device__ __forceinline__ void zero() { v = (T)0.0f; }
};
template <typename T> struct Chans<T, 1> {
    T v;
    __device__ __forceinline__ void load(const T *p) { v = *p; }
    __device__ __forceinline__ void store(T *p) const { *p = v; }
    __device__ __forceinline__ float get(int) const { return (float)v; }
    __device__ __forceinline__ void set(int, float f) { v = Elem<T>::from_f32(f); }
    __device__ __forceinline__ void zero() { v = (T)0.0f; }
};

// The three outputs, dense, stand for the channels [0, w0), [w0, w0 + w1) and [w0 + w1, C).
template <typename T> struct ConvOut {
    T *y0, *y1, *y2;
    int w0, w1, w2;
    // row 0 of channel c's output at that channel, and the output's width
    __device__ __forceinline__ T *at(int c, int &width) const
    {
        width = c < w0 ? w0 : c < w0 + w1 ? w1 : w2;
        return c < w0 ? y0 + c : c < w0 + w1 ? y1 + (c - w0) : y2 + (c - w0 - w1);
    }
};

// The weights and bias of V channels.
template <int K, int V> struct Taps {
    float w[V][K], bias[V];
    __device__ __forceinline__ void load(const float *__restrict__ wp, const float *__restrict__ bp,
                                         int c)
    {
        if constexpr (V % 4 == 0) {          // c is a multiple of 4: whole 16-byte rows
#pragma unroll
            for (int q = 0; q < V * K / 4; ++q) {
                const f32x4 f = *reinterpret_cast<const f32x4 *>(wp + (int64_t)c * K + 4 * q);
#pragma unroll
                for (int i = 0; i < 4; ++i) w[(4 * q + i) / K][(4 * q + i) % K] = f[i];
            }
        } else {
#pragma unroll
            for (int i = 0; i < V * K; ++i) w[i / K][i % K] = wp[(int64_t)c * K + i];
        }
#pragma unroll
        for (int i = 0; i < V; ++i) bias[i] = bp ? bp[c + i] : 0.0f;
    }
};

// A thread owns V channels of `tt` consecutive tokens; neighbouring threads neighbouring
// channels, then token tiles.  The K - 1 inputs before each token stay in registers; kRows rows
// are loaded together (4 instead of 8: 43.5 us against 41.2 for 16384 x 2560 bf16; 16: 42.5).
constexpr int kRows = 8;
template <typename T, int K, int V>
__global__ __launch_bounds__(kConvThreads) void conv_kernel(
    const T *__restrict__ x, const float *__restrict__ w, const float *__restrict__ bias,
    const T *state0, const int32_t *__restrict__ lengths, ConvOut<T> out, T *stateT, int L, int C,
    int64_t pitch, int groups, int tiles, int tt, int64_t threads, bool act)
{
    // Rows off 16 bytes share cache lines with their neighbours: there an XCD (workgroups go to
    // the eight in turn) takes one run of workgroups, so that its L2 completes these lines (5 x
    // 2500 x 777 bf16 15.1 -> 14.0 us, 4000 x 1001 fp32 11.2 -> 10.6; 16384 x 2560 bf16 in whole
    // lines 41.2 -> 42.0).
    const unsigned run = gridDim.x / 8;
    const unsigned block =
        V == 1 && blockIdx.x < run * 8 ? blockIdx.x % 8 * run + blockIdx.x / 8 : blockIdx.x;
    const int64_t id = (int64_t)block * kConvThreads + threadIdx.x;
    if (id >= threads) return;
    const int c = (int)(id % groups) * V;
    const int tile = (int)(id / groups % tiles);
    const int64_t b = id / groups / tiles;
    int len = L;
    if (lengths) len = min(max(lengths[b], 0), L);
    const int t0 = tile * tt, t1 = min(t0 + tt, len);
    if (tile > 0 && t0 >= len) return;
    const T *xb = x + b * L * pitch + c;
    Taps<K, V> taps;
    taps.load(w, bias, c);

    Chans<T, V> first[K - 1];      // the rows before t0
#pragma unroll
    for (int k = 0; k < K - 1; ++k) {
        if (tile > 0) first[k].load(xb + (int64_t)(t0 - (K - 1) + k) * pitch);
        else if (state0) first[k].load(state0 + (b * (K - 1) + k) * C + c);
        else first[k].zero();
    }
    float win[K][V];               // win[k] = u[t - K + 1 + k]
#pragma unroll
    for (int k = 0; k < K - 1; ++k)
#pragma unroll
        for (int i = 0; i < V; ++i) win[k + 1][i] = first[k].get(i);

    int width;
    T *yr = out.at(c, width);
    yr += (b * L + t0) * width;
    const T *xr = xb + (int64_t)t0 * pitch;
    // kRows rows, or (not whole) the n rows that are left: rows past them load the last one
    // again and are not stored.  Whole batches step their pointers by uniform amounts, without
    // a product per row.
    auto rows = [&](int n, auto whole) {
        Chans<T, V> u[kRows];
#pragma unroll
        for (int r = 0; r < kRows; ++r)
            u[r].load(xr + (whole.value ? r : min(r, n - 1)) * pitch);
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            Chans<T, V> o;
#pragma unroll
            for (int i = 0; i < V; ++i) {
#pragma unroll
                for (int k = 0; k + 1 < K; ++k) win[k][i] = win[k + 1][i];
                win[K - 1][i] = u[r].get(i);
                float v = taps.bias[i];
#pragma unroll
                for (int k = 0; k < K; ++k) v = fmaf(taps.w[i][k], win[k][i], v);
                o.set(i, act ? silu(v) : v);
            }
            if (whole.value || r < n) o.store(yr + (int64_t)r * width);
        }
        xr += kRows * pitch;
        yr += (int64_t)kRows * width;
    };
    int t = t0;
    for (; t + kRows <= t1; t += kRows) rows(kRows, std::true_type());
    if (t < t1) rows(t1 - t, std::false_type());
    // The first token tile's threads, which alone read state0, write stateT: the two may be
    // one buffer.
    if (tile == 0 && stateT) {
#pragma unroll
        for (int k = 0; k < K - 1; ++k) {
            const int t = len - (K - 1) + k;
            Chans<T, V> v;
            if (t >= 0) {
                v.load(xb + (int64_t)t * pitch);
            } else {
                v.zero();
#pragma unroll
                for (int j = 0; j < K - 1; ++j)
                    if (j == t + K - 1) v = first[j];
            }
            v.store(stateT + (b * (K - 1) + k) * C + c);
        }
    }
}

template <typename T, int K, int V>
__global__ __launch_bounds__(kConvThreads) void conv_step_kernel(
    const T *__restrict__ x, const float *__restrict__ w, const float *__restrict__ bias,
    T *__restrict__ state, ConvOut<T> out, int C, int64_t pitch, int groups, int64_t threads,
    bool act)
{
    const int64_t id = (int64_t)blockIdx.x * kConvThreads + threadIdx.x;
    if (id >= threads) return;
    const int c = (int)(id % groups) * V;
    const int64_t b = id / groups;
    T *sp = state + b * (K - 1) * C + c;
    Chans<T, V> u[K];
#pragma unroll
    for (int k = 0; k < K - 1; ++k) u[k].load(sp + (int64_t)k * C);
    u[K - 1].load(x + b * pitch + c);
    Taps<K, V> taps;
    taps.load(w, bias, c);
    Chans<T, V> o;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        float v = taps.bias[i];
#pragma unroll
        for (int k = 0; k < K; ++k) v = fmaf(taps.w[i][k], u[k].get(i), v);
        o.set(i, act ? silu(v) : v);
    }
#pragma unroll
    for (int k = 0; k < K - 1; ++k) u[k + 1].store(sp + (int64_t)k * C);
    int width;
    T *yb = out.at(c, width);
    o.store(yb + b * width);
}

template <typename T> ConvOut<T> out_of(const ConvShape &s, void *y0, void *y1, void *y2)
{
    return {(T *)y0, (T *)y1, (T *)y2, (int)s.w0, (int)s.w1, (int)s.w2};
}

bool on16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// Whether every row of every array starts on 16 bytes at each multiple of V channels.
template <typename T>
bool vector_rows(const ConvShape &s, const void *x, const void *state0, const void *y0,
                 const void *y1, const void *y2, const void *stateT)
{
    const int64_t V = 16 / (int64_t)sizeof(T);
    return s.C % V == 0 && s.pitch % V == 0 && s.w0 % V == 0 && s.w1 % V == 0 && on16(x) &&
           on16(state0) && on16(y0) && on16(y1) && on16(y2) && on16(stateT);
}

unsigned blocks_of(int64_t threads) { return (unsigned)((threads + kConvThreads - 1) / kConvThreads); }

template <typename T, int K, int V>
hipError_t conv_go(const ConvShape &s, const void *x, const float *w, const float *bias,
                   const void *state0, const int32_t *lengths, void *y0, void *y1, void *y2,
                   void *stateT, hipStream_t st)
{
    const int groups = (int)(s.C / V);
    // Tokens per thread: 32, fewer where that leaves under 16 waves a CU (for 16 bytes a thread one
    // to two rounds of what is resident: bf16 with four taps takes 171 registers, two waves a SIMD,
    // three taps 139, two 97); below 8 the halo costs what the threads gain (2 x 2048 x 1792: 14.2 us
    // with 4, 11.2 with 8).
    constexpr int64_t kWanted = 256 * 16 * 64;
    int tt = 32;
    while (tt > 8 && groups * ((s.L + tt - 1) / tt) * s.b < kWanted) tt /= 2;
    const int tiles = (int)((s.L + tt - 1) / tt);
    const int64_t threads = (int64_t)groups * tiles * s.b;
    hipLaunchKernelGGL((conv_kernel<T, K, V>), dim3(blocks_of(threads)), dim3(kConvThreads), 0, st,
                       (const T *)x, w, bias, (const T *)state0, lengths,
                       out_of<T>(s, y0, y1, y2), (T *)stateT, (int)s.L, (int)s.C, s.pitch, groups,
                       tiles, tt, threads, s.silu);
    return hipGetLastError();
}

template <typename T, int K, int V>
hipError_t step_go(const ConvShape &s, const void *x, const float *w, const float *bias,
                   void *state, void *y0, void *y1, void *y2, hipStream_t st)
{
    const int groups = (int)(s.C / V);
    const int64_t threads = (int64_t)groups * s.b;
    hipLaunchKernelGGL((conv_step_kernel<T, K, V>), dim3(blocks_of(threads)), dim3(kConvThreads),
                       0, st, (const T *)x, w, bias, (T *)state, out_of<T>(s, y0, y1, y2),
                       (int)s.C, s.pitch, groups, threads, s.silu);
    return hipGetLastError();
}

template <typename T, int K>
hipError_t conv_wide(const ConvShape &s, const void *x, const float *w, const float *bias,
                     const void *state0, const int32_t *lengths, void *y0, void *y1, void *y2,
                     void *stateT, hipStream_t st)
{
    if (vector_rows<T>(s, x, state0, y0, y1, y2, stateT))
        return conv_go<T, K, 16 / sizeof(T)>(s, x, w, bias, state0, lengths, y0, y1, y2, stateT, st);
    return conv_go<T, K, 1>(s, x, w, bias, state0, lengths, y0, y1, y2, stateT, st);
}

template <typename T, int K>
hipError_t step_wide(const ConvShape &s, const void *x, const float *w, const float *bias,
                     void *state, void *y0, void *y1, void *y2, hipStream_t st)
{
    if (vector_rows<T>(s, x, state, y0, y1, y2, nullptr))
        return step_go<T, K, 16 / sizeof(T)>(s, x, w, bias, state, y0, y1, y2, st);
    return step_go<T, K, 1>(s, x, w, bias, state, y0, y1, y2, st);
}

}  // namespace

hipError_t launch_conv(const ConvShape &s, const void *x, const float *w, const float *bias,
                       const void *state0, const int32_t *lengths, void *y0, void *y1, void *y2,
                       void *stateT, hipStream_t st)
{
#define SSD_CONV(T, K) return conv_wide<T, K>(s, x, w, bias, state0, lengths, y0, y1, y2, stateT, st)
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
#define SSD_CONV(T, K) return step_wide<T, K>(s, x, w, bias, state, y0, y1, y2, st)
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
