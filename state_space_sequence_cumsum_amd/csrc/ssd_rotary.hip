// ssd_rotary.hip -- rotary positions: pairs of a head's elements turned by position x frequency,
//
//     (x_a, x_b) <- scale (x_a cos - x_b sin, x_b cos + x_a sin),   angle = position freqs[j]
//
// for j < rot / 2 with (a, b) = (j, j + rot / 2) or, interleaved, (2 j, 2 j + 1); elements from rot on
// go through as they are.  The inverse turns back (the gradient of the forward one).
//
// Angles: position x frequency passes 2^24 radians for far positions, so it is formed in 64 bits as
// quarter turns and reduced there; only the rest, at most an eighth of a turn, is rounded to
// fp32.  A token's sines serve all its heads: a workgroup forms them once for its tokens, into
// LDS, and then streams the heads of both arrays, 16 bytes of each side of the pairs a thread.
// Bound by HBM (each element read and written once), or by launch latency for few tokens: 16384
// tokens of 32 heads of 128 in 43 us (6.2 TB/s, the rate of a copy), one token of 128 sequences 3.3.
// Where a side of the pairs, a head or a row is no whole number of 16 bytes, elements go one by one: the
// same tokens of 32 heads of 80 in 27 us with all of it turned (16 bytes), in 99 with 24 elements in
// halves of 12, in 67 with heads of 84 interleaved (bf16; 1.7 and 2.6 TB/s).
#include <hip/hip_runtime.h>

#include "ssd_device.h"
#include "ssd_launch.h"

namespace ssd {
namespace {

constexpr int kRotThreads = 256;
constexpr int kPairs = 2048;        // pairs of cosine and sine in a workgroup's LDS (16 KB)

struct RotDims {
    int64_t qp, kp, tokens;
    int L, Hq, Hk, D, half;         // half: rot / 2
    int block;                      // tokens of a workgroup
    int positions;
    float scale, sign;
};

// cos and sin of quarters x pi / 2: Taylor polynomials on an eighth of a turn to either side
// (first terms left out: 1.8e-9 for the sine, 4.6e-10 for the cosine)
__device__ __forceinline__ float2 turn_of(double quarters)
{
    const double n = __builtin_rint(quarters);
    const float f = (float)((quarters - n) * 1.5707963267948966);
    const int k = (int)(n - 4.0 * __builtin_floor(n * 0.25));
    const float z = f * f;
    const float s = f + f * z * (-1.0f / 6 + z * (1.0f / 120 + z * (-1.0f / 5040 + z * (1.0f / 362880))));
    const float c = 1.0f + z * (-0.5f + z * (1.0f / 24 + z * (-1.0f / 720 + z * (1.0f / 40320 + z * (-1.0f / 3628800)))));
    const float re = (k & 1) ? s : c, im = (k & 1) ? c : s;
    return {k == 1 || k == 2 ? -re : re, k >= 2 ? -im : im};
}

template <typename T, int V> struct Vec;
template <> struct Vec<bf16, 8> { typedef bf16x8 t; };
template <> struct Vec<float, 4> { typedef f32x4 t; };
template <typename T> struct Vec<T, 1> { typedef T t; };

template <typename V> __device__ __forceinline__ float get(const V &v, int i)
{
    if constexpr (std::is_same<V, float>::value || std::is_same<V, bf16>::value) return (float)v;
    else return (float)v[i];
}
template <typename T, typename V> __device__ __forceinline__ void set(V &v, int i, float x)
{
    if constexpr (std::is_same<V, float>::value || std::is_same<V, bf16>::value) v = (T)x;
    else v[i] = (T)x;
}

// V elements a piece.  In halves a thread takes a piece of both sides; interleaved, one piece of
// V / 2 pairs.  V = 1 (halves) and 1 pair (interleaved) serve rows of any alignment.
template <typename T, int V, bool INTER>
__global__ __launch_bounds__(kRotThreads) void rotary_kernel(const T *q, const T *k,
                                                             const float *__restrict__ freqs,
                                                             const int32_t *__restrict__ positions, T *yq,
                                                             T *yk, RotDims m)
{
    constexpr int PAIRS = INTER ? (V == 1 ? 1 : V / 2) : V;    // pairs of a piece
    constexpr int W = INTER && V == 1 ? 1 : V;                 // elements of a load
    typedef typename Vec<T, W>::t P;
    __shared__ float2 turn[kPairs];
    const int64_t token0 = (int64_t)blockIdx.x * m.block;
    const int count = (int)min((int64_t)m.block, m.tokens - token0);
    for (int p0 = 0; p0 < m.half; p0 += kPairs) {              // one round but for very wide heads
        const int pairs = min(m.half - p0, kPairs);
        if (p0 > 0) __syncthreads();
        for (int i = threadIdx.x; i < count * pairs; i += kRotThreads) {
            const int t = i / pairs, j = i % pairs;
            const int64_t token = token0 + t;
            int64_t pos = token % m.L;
            if (m.positions == 1) pos += positions[token / m.L];
            if (m.positions == 2) pos = positions[token];
            float2 cs = turn_of((double)pos * (double)freqs[p0 + j] * 0.63661977236758134);
            cs.x *= m.scale;
            cs.y *= m.scale * m.sign;
            turn[i] = cs;
        }
        __syncthreads();
        const int units = pairs / PAIRS, heads = m.Hq + m.Hk;
        for (int i = threadIdx.x; i < count * heads * units; i += kRotThreads) {
            const int u = i % units, th = i / units, head = th % heads, t = th / heads;
            const int64_t token = token0 + t;
            const bool second = head >= m.Hq;
            const int h = second ? head - m.Hq : head;
            const T *x = second ? k + token * m.kp : q + token * m.qp;
            x += (int64_t)h * m.D;
            T *y = second ? yk + (token * m.Hk + h) * m.D : yq + (token * m.Hq + h) * m.D;
            const int j = u * PAIRS;
            const int ia = INTER ? 2 * (p0 + j) : p0 + j;
            const int ib = INTER ? ia + 1 : ia + m.half;
            const float2 *cs = turn + t * pairs + j;
            if constexpr (INTER && V > 1) {
                P a = *reinterpret_cast<const P *>(x + ia);
#pragma unroll
                for (int e = 0; e < PAIRS; ++e) {
                    const float re = get(a, 2 * e), im = get(a, 2 * e + 1);
                    set<T>(a, 2 * e, re * cs[e].x - im * cs[e].y);
                    set<T>(a, 2 * e + 1, im * cs[e].x + re * cs[e].y);
                }
                *reinterpret_cast<P *>(y + ia) = a;
            } else {
                P a = *reinterpret_cast<const P *>(x + ia), b = *reinterpret_cast<const P *>(x + ib);
#pragma unroll
                for (int e = 0; e < PAIRS; ++e) {
                    const float re = get(a, e), im = get(b, e);
                    set<T>(a, e, re * cs[e].x - im * cs[e].y);
                    set<T>(b, e, im * cs[e].x + re * cs[e].y);
                }
                *reinterpret_cast<P *>(y + ia) = a;
                *reinterpret_cast<P *>(y + ib) = b;
            }
        }
    }
    // what is not rotated
    const int rest = (m.D - 2 * m.half) / W, heads = m.Hq + m.Hk;
    for (int i = threadIdx.x; i < count * heads * rest; i += kRotThreads) {
        const int u = i % rest, th = i / rest, head = th % heads, t = th / heads;
        const int64_t token = token0 + t;
        const bool second = head >= m.Hq;
        const int h = second ? head - m.Hq : head, at = 2 * m.half + u * W;
        const T *x = second ? k + token * m.kp : q + token * m.qp;
        T *y = second ? yk + (token * m.Hk + h) * m.D : yq + (token * m.Hq + h) * m.D;
        *reinterpret_cast<P *>(y + at) = *reinterpret_cast<const P *>(x + (int64_t)h * m.D + at);
    }
}

template <typename T, int V, bool INTER>
hipError_t rotary_go(const RotDims &m, const void *q, const void *k, const float *freqs,
                     const int32_t *positions, void *yq, void *yk, hipStream_t st)
{
    const int64_t groups = (m.tokens + m.block - 1) / m.block;
    hipLaunchKernelGGL((rotary_kernel<T, V, INTER>), dim3((unsigned)groups), dim3(kRotThreads), 0, st,
                       (const T *)q, (const T *)k, freqs, positions, (T *)yq, (T *)yk, m);
    return hipGetLastError();
}

template <typename T>
hipError_t rotary_by_layout(const RotaryShape &s, const void *q, const void *k, const float *freqs,
                            const int32_t *positions, void *yq, void *yk, hipStream_t st)
{
    constexpr int V = 16 / sizeof(T);
    RotDims m;
    m.qp = s.qp; m.kp = s.kp; m.tokens = s.b * s.L;
    m.L = (int)s.L; m.Hq = (int)s.Hq; m.Hk = (int)s.Hk; m.D = (int)s.D; m.half = (int)(s.rot / 2);
    m.positions = s.positions;
    m.scale = s.scale; m.sign = s.inverse ? -1.0f : 1.0f;
    m.block = 1;
    while (m.block < 16 && 2 * m.block * m.half <= kPairs && m.tokens >= 2048 * m.block) m.block *= 2;
    uintptr_t bits = (uintptr_t)q | (uintptr_t)yq;
    if (s.Hk) bits |= (uintptr_t)k | (uintptr_t)yk;
    bool wide = bits % 16 == 0 && s.D % V == 0 && s.qp % V == 0 && (s.Hk == 0 || s.kp % V == 0);
    wide = wide && (s.interleaved ? s.rot % V == 0 : s.rot / 2 % V == 0);
    if (s.interleaved)
        return wide ? rotary_go<T, V, true>(m, q, k, freqs, positions, yq, yk, st)
                    : rotary_go<T, 1, true>(m, q, k, freqs, positions, yq, yk, st);
    return wide ? rotary_go<T, V, false>(m, q, k, freqs, positions, yq, yk, st)
                : rotary_go<T, 1, false>(m, q, k, freqs, positions, yq, yk, st);
}

}  // namespace

hipError_t launch_rotary(const RotaryShape &s, const void *q, const void *k, const float *freqs,
                         const int32_t *positions, void *yq, void *yk, hipStream_t st)
{
    return s.bf16 ? rotary_by_layout<bf16>(s, q, k, freqs, positions, yq, yk, st)
                  : rotary_by_layout<float>(s, q, k, freqs, positions, yq, yk, st);
}

}  // namespace ssd
