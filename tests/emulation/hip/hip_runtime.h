// hip/hip_runtime.h for a build of the kernels' own sources on the CPU: one workgroup at a time, a
// fiber for every work-item (emulator.cpp).  What crosses lanes (shuffles, lane moves, matrix
// instructions, transposed reads) goes through a slot a lane, with all 64 lanes there.
//
// LDS arrays lie in a section of their own, which every workgroup finds filled with NaN.  Buffer
// accesses that lie in their range in part, or whose offset runs past 32 bits, end the process.
#pragma once

#include <stddef.h>
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include <algorithm>
#include <cfloat>
#include <cmath>
#include <cstdint>
#include <functional>
#include <initializer_list>
#include <type_traits>
#include <utility>

#define __global__
#define __device__
#define __host__
#define __forceinline__ inline
#define __shared__ static __attribute__((section("emulated_lds")))
#define __launch_bounds__(...)
#define __restrict__

struct dim3 {
    unsigned x, y, z;
    dim3(unsigned a = 1, unsigned b = 1, unsigned c = 1) : x(a), y(b), z(c) {}
};
struct Index { unsigned x, y, z; };
extern Index threadIdx, blockIdx, gridDim, blockDim;
typedef int hipError_t;
typedef void *hipStream_t;
constexpr hipError_t hipSuccess = 0, hipErrorInvalidValue = 1;
inline hipError_t hipGetLastError() { return hipSuccess; }
struct float2 { float x, y; };
using std::max;
using std::min;

namespace emulator {
struct Slot { unsigned char b[64]; };
void barrier();          // of the workgroup
void wave_sync();        // all lanes of the wave are here
Slot &slot(int lane);    // of the running wave
int lane_id();
[[noreturn]] void fail(const char *what);
void launch(dim3 grid, dim3 block, const std::function<void()> &body);

// every lane puts a value down and then looks at the others'
template <typename T, typename F> auto exchange(const T &v, F &&look)
{
    static_assert(sizeof(T) <= sizeof(Slot), "");
    memcpy(slot(lane_id()).b, &v, sizeof v);
    wave_sync();
    const auto r = look([](int lane) {
        T t;
        memcpy(&t, slot(lane & 63).b, sizeof t);
        return t;
    });
    wave_sync();
    return r;
}
template <typename T> T from_lane(T v, int lane)
{
    return exchange(v, [&](auto of) { return of(lane); });
}
}  // namespace emulator

#define hipLaunchKernelGGL(kernel, grid, block, lds, stream, ...) \
    emulator::launch(grid, block, [=] { kernel(__VA_ARGS__); })
inline void __syncthreads() { emulator::barrier(); }

inline float __uint_as_float(uint32_t v) { float f; memcpy(&f, &v, 4); return f; }
inline float __shfl_xor(float v, int m, int) { return emulator::from_lane(v, emulator::lane_id() ^ m); }
inline float __shfl_down(float v, int n, int)
{
    const int l = emulator::lane_id();
    return emulator::from_lane(v, l + n < 64 ? l + n : l);
}
// lane moves with bound_ctrl: 0 where no lane is read, or the row is masked out
inline int emulated_dpp(int, int v, int ctrl, int row_mask, int, bool)
{
    const int l = emulator::lane_id();
    int from = -1;
    if (ctrl >= 0x111 && ctrl <= 0x11f) from = (l & 15) >= ctrl - 0x110 ? l - (ctrl - 0x110) : -1;
    else if (ctrl == 0x142) from = l >= 16 ? l / 16 * 16 - 1 : -1;
    else if (ctrl == 0x143) from = l >= 32 ? 31 : -1;
    else if (ctrl == 0x138) from = l - 1;
    else emulator::fail("a lane move that is not known here");
    const int x = emulator::from_lane(v, from < 0 ? l : from);
    return from < 0 || !(row_mask >> (l / 16) & 1) ? 0 : x;
}
#define __builtin_amdgcn_update_dpp emulated_dpp
#define __builtin_amdgcn_readlane(v, lane) emulator::from_lane<int>(v, lane)
#define __builtin_amdgcn_readfirstlane(v) emulator::from_lane<int>(v, 0)
#define __builtin_amdgcn_exp2f exp2f
#define __builtin_amdgcn_sched_barrier(x)
#define __builtin_amdgcn_s_setprio(x)

typedef __bf16 emulated_b8 __attribute__((ext_vector_type(8)));
typedef float emulated_f4 __attribute__((ext_vector_type(4)));
typedef short emulated_s4 __attribute__((ext_vector_type(4)));
typedef unsigned emulated_u2 __attribute__((ext_vector_type(2)));
typedef unsigned emulated_u4 __attribute__((ext_vector_type(4)));

// D[row, col] = C + sum A[row, k] B[k, col]; lane l holds column l % 16 and rows 4 (l / 16) + r of C
template <typename V, typename F> emulated_f4 emulated_mfma(const V &a, const V &b, emulated_f4 c, F &&dot)
{
    struct Both { V a, b; };
    return emulator::exchange(Both{a, b}, [&](auto of) {
        const int l = emulator::lane_id();
        for (int r = 0; r < 4; ++r)
            for (int g = 0; g < 4; ++g)
                c[r] = dot(of(4 * (l / 16) + r + 16 * g).a, of((l & 15) + 16 * g).b, c[r]);
        return c;
    });
}
inline emulated_f4 emulated_mfma_bf16(emulated_b8 a, emulated_b8 b, emulated_f4 c, int, int, int)
{
    return emulated_mfma(a, b, c, [](const emulated_b8 &x, const emulated_b8 &y, float s) {
        for (int e = 0; e < 8; ++e) s += (float)x[e] * (float)y[e];
        return s;
    });
}
inline emulated_f4 emulated_mfma_f32(float a, float b, emulated_f4 c, int, int, int)
{
    return emulated_mfma(a, b, c, [](float x, float y, float s) { return s + x * y; });
}
#define __builtin_amdgcn_mfma_f32_16x16x32_bf16 emulated_mfma_bf16
#define __builtin_amdgcn_mfma_f32_16x16x4f32 emulated_mfma_f32

inline emulated_s4 emulated_transposed_read(const void *p)
{
    emulated_s4 v;
    memcpy(&v, p, sizeof v);
    return emulator::exchange(v, [](auto of) {
        const int l = emulator::lane_id(), i = l & 15;
        emulated_s4 r;
        for (int e = 0; e < 4; ++e) r[e] = of((l & ~15) + 4 * e + i / 4)[i % 4];
        return r;
    });
}
#define __builtin_amdgcn_ds_read_tr16_b64_v4i16(p) emulated_transposed_read((const void *)(p))

// odd rows of 16 of the first value change places with even rows of the second
inline emulated_u2 emulated_swap16(unsigned a, unsigned b, bool, bool)
{
    return emulator::exchange(emulated_u2{a, b}, [](auto of) {
        const int l = emulator::lane_id();
        return l & 16 ? emulated_u2{of(l & ~16)[1], of(l)[1]} : emulated_u2{of(l)[0], of(l | 16)[0]};
    });
}
#define __builtin_amdgcn_permlane16_swap emulated_swap16

struct emulated_buffer { char *base; uint32_t bytes; };
#define __amdgpu_buffer_rsrc_t emulated_buffer
inline emulated_buffer emulated_make_buffer(void *p, short, int bytes, int)
{
    return {(char *)p, (uint32_t)bytes};
}
inline bool emulated_in_range(const emulated_buffer &r, int off, uint32_t size)
{
    const uint64_t at = (uint32_t)off, end = at + size;
    if (end > (uint64_t)1 << 32) emulator::fail("a buffer offset that runs past 32 bits");
    if (at < r.bytes && end > r.bytes) emulator::fail("a buffer access that ends behind its range");
    return end <= r.bytes;
}
template <typename V> V emulated_load(const emulated_buffer &r, int off)
{
    V v;
    memset(&v, 0, sizeof v);
    if (emulated_in_range(r, off, sizeof v)) memcpy(&v, r.base + (uint32_t)off, sizeof v);
    return v;
}
template <typename V> void emulated_store(V v, const emulated_buffer &r, int off)
{
    if (emulated_in_range(r, off, sizeof v)) memcpy(r.base + (uint32_t)off, &v, sizeof v);
}
#define __builtin_amdgcn_make_buffer_rsrc emulated_make_buffer
#define __builtin_amdgcn_raw_buffer_load_b16(r, off, s, p) emulated_load<uint16_t>(r, off)
#define __builtin_amdgcn_raw_buffer_load_b32(r, off, s, p) emulated_load<unsigned>(r, off)
#define __builtin_amdgcn_raw_buffer_load_b64(r, off, s, p) emulated_load<emulated_u2>(r, off)
#define __builtin_amdgcn_raw_buffer_load_b128(r, off, s, p) emulated_load<emulated_u4>(r, off)
#define __builtin_amdgcn_raw_buffer_store_b32(v, r, off, s, p) emulated_store<unsigned>(v, r, off)
#define __builtin_amdgcn_raw_buffer_store_b64(v, r, off, s, p) emulated_store<emulated_u2>(v, r, off)
#define __builtin_amdgcn_raw_buffer_store_b128(v, r, off, s, p) emulated_store<emulated_u4>(v, r, off)

// helpers of ssd_device.h that these kernels do not use
#define __builtin_amdgcn_perm(a, b, sel) (emulator::fail("perm"), 0u)
#define __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, x, y, z) (emulator::fail("32x32"), c)
#define __builtin_amdgcn_mfma_f32_32x32x2f32(a, b, c, x, y, z) (emulator::fail("32x32"), c)

// asm volatile("" : "+v"(x)) only hides a value from the compiler
#define asm
#define volatile(...)
