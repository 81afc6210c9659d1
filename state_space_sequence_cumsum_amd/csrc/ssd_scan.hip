// ssd_scan.hip -- the selective state space scan (a decay rate per channel and state, a step
// size per token and channel), for prompts and for single tokens.
//
//     d_t[c]    = dt_t[c] + dt_bias[c], through softplus where asked
//     h_t[c, n] = exp(d_t[c] A[c, n]) h_{t-1}[c, n] + d_t[c] x_t[c] B_t[g, n]
//     y_t[c]    = (sum_n C_t[g, n] h_t[c, n] + D[c] x_t[c]) silu(z_t[c])
//
// A wave owns 64 channels of one group, a lane one of them, with its N states and rates in
// registers; B_t and C_t, the same for all lanes, are broadcast from LDS.  Per state and token:
// two products, an exp2 and two fused multiply-adds (one without the output), whose issue (four
// cycles each; an exp2 alone takes eight, next to other waves' instructions six or seven) bounds
// the scan before HBM does.  Where the channels give too few waves, the
// tokens are split into segments: one launch scans each segment from zero for its end state, a
// short one chains these into the segments' start states (exp of A times a segment's summed
// steps is its factor), and one scans the segments again from there.  The first scan costs 0.8
// of the second, and the bound is both.  Short prompts do the same within one workgroup and launch.
//
// Measured (bf16, 16384 tokens, 2048 channels, 16 states, gate and softplus): 208 to 214 us (97 to
// 99, 128 to 134 and 17 us for the two scans and the chain, each profiled by itself).  The scans
// issue 44 and 58 thousand VALU instructions a SIMD, 176 and 231 thousand cycles; they take 190 to
// 197 and 247 to 255 thousand, at clocks of 1.74 to 2.26 GHz read within the kernels (85 and 114 us
// at the highest).  HBM's floor is 44 us.  One whole walk per channel: 5.3 ms.

#include <hip/hip_runtime.h>

#include "../../include/ssd.h"
#include "ssd_device.h"
#include "ssd_launch.h"

namespace ssd {
namespace {

__device__ __forceinline__ float silu(float v)
{
    return v * __builtin_amdgcn_rcpf(1.0f + fast_exp2(-kLog2e * v));
}

// log(1 + exp(v)) = max(v, 0) + log1p(e), e = exp(-|v|) in (0, 1], with
// log1p(e) = 2 atanh(s), s = e / (2 + e): 2 s times a polynomial in (2 s)^2 (degree 4,
// interpolated at the Chebyshev points of [0, 4/9]: relative error 4.1e-9), so small step sizes
// keep their relative accuracy (log2(1 + e) would not).
__device__ __forceinline__ float softplus(float v)
{
    const float e = fast_exp2(-kLog2e * fabsf(v));
    const float s = e * __builtin_amdgcn_rcpf(fmaf(0.5f, e, 1.0f));
    const float q = s * s;
    float p = 5.4995661e-4f;
    p = fmaf(p, q, 2.1847779e-3f);
    p = fmaf(p, q, 1.2507686e-2f);
    p = fmaf(p, q, 8.3332902e-2f);
    p = fmaf(p, q, 1.0f);
    float top;   // fmaxf would spend an instruction on a signalling NaN
    asm("v_max_f32 %0, 0, %1" : "=v"(top) : "v"(v));
    return fmaf(s, p, top);
}

// Orders LDS accesses of one wave's lanes for the compiler; the hardware carries a wave's LDS
// accesses out in order, so no instruction is needed.
__device__ __forceinline__ void wave_order()
{
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

struct ScanDims {
    int64_t L, xp, dtp, zp, Bp, Cp;
    int C, Cg, tiles;      // channels, channels per group, 64-channel tiles per group
    int G;
    int sp;                // 1: softplus
    int S, seg;            // segments of the sequence, tokens per segment
};

// ---------------------------------------------------------------------------
// The scan of one segment of tokens.  A wave owns 64 channels of one group; `KIND` says what
// it computes:
//   kWhole  the whole sequence: from h0, writes y and hT
//   kEnds   one segment from a zero state: writes the state at its end and the sum of its steps
//   kOut    one segment from the state at its start (workspace): writes y, the last one hT
// ---------------------------------------------------------------------------
enum Kind { kWhole, kEnds, kOut };

// Four consecutive elements that start on a multiple of four bytes, as fp32.
typedef uint32_t u32x2_a4 __attribute__((ext_vector_type(2), aligned(4)));
typedef uint32_t u32x4_a4 __attribute__((ext_vector_type(4), aligned(4)));
template <typename T> struct Quad;
template <> struct Quad<float> {
    u32x4 v;
    __device__ __forceinline__ void load(const float *p) { v = *reinterpret_cast<const u32x4_a4 *>(p); }
    __device__ __forceinline__ f32x4 get() const { return __builtin_bit_cast(f32x4, v); }
};
template <> struct Quad<bf16> {
    u32x2 v;
    __device__ __forceinline__ void load(const bf16 *p) { v = *reinterpret_cast<const u32x2_a4 *>(p); }
    __device__ __forceinline__ f32x4 get() const
    {
        f32x4 f;
        f[0] = bf_lo(v[0]); f[1] = bf_hi(v[0]); f[2] = bf_lo(v[1]); f[3] = bf_hi(v[1]);
        return f;
    }
};

// One element, as raw bits, at byte offset `off` (per lane) + `row` (uniform) of a raw buffer.
template <typename T>
__device__ __forceinline__ uint32_t buf_load(rsrc_t r, uint32_t off, uint32_t row)
{
    if constexpr (sizeof(T) == 2)
        return (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(r, (int)off, (int)row, 0);
    else
        return (uint32_t)__builtin_amdgcn_raw_buffer_load_b32(r, (int)off, (int)row, 0);
}
template <typename T> __device__ __forceinline__ float bits_to_f32(uint32_t v)
{
    return __uint_as_float(sizeof(T) == 2 ? v << 16 : v);
}
template <typename T>
__device__ __forceinline__ void buf_store(rsrc_t r, uint32_t off, uint32_t row, T v)
{
    if constexpr (sizeof(T) == 2)
        __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(uint16_t, v), r, (int)off, (int)row, 0);
    else
        __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, v), r, (int)off, (int)row, 0);
}

constexpr int kStep = 8;    // segments are multiples of this many tokens

// The workspace of a split scan: per (sequence, segment), the state at the segment's end
// (kEnds) and, after the chain, at its start, as [N][Cw] with Cw = G * tiles * 64, so
// that a wave's lanes stand side by side; and the sum of its step sizes [Cw].
struct ScanWs {
    float *state, *steps;
};

// Tokens of sequence b, and how many of its segments these reach (one at least: an empty
// sequence's first segment hands its initial state on).
__device__ __forceinline__ int64_t tokens_of(const int32_t *lengths, int64_t b, const ScanDims &m)
{
    return lengths ? min((int64_t)max(lengths[b], 0), m.L) : m.L;
}
__device__ __forceinline__ int segments_of(int64_t len, const ScanDims &m)
{
    return max((int)((len + m.seg - 1) / m.seg), 1);
}

template <typename T, int N, int KIND>
__global__ __launch_bounds__(64) __attribute__((amdgpu_waves_per_eu(N <= 16 ? 4 : N <= 32 ? 3 : 2))) void scan_kernel(
    const T *__restrict__ x, const T *__restrict__ dt, const float *__restrict__ A,
    const T *__restrict__ B, const T *__restrict__ Cm, const float *__restrict__ D,
    const T *__restrict__ z, const float *__restrict__ dt_bias, const float *h0,
    const int32_t *__restrict__ lengths, T *__restrict__ y, float *hT, ScanWs ws, ScanDims m)
{
    // tokens whose inputs a lane loads together, one tile ahead (as many as registers allow)
    constexpr int kTile = N <= 16 ? 8 : 4;
    // per token of the tile, B and (except for the end states) C as fp32; read by all lanes of
    // the one wave, so each read is a broadcast
    constexpr int kRow = KIND == kEnds ? N : 2 * N;
    __shared__ __attribute__((aligned(16))) float bc[kTile * kRow];
    const int gt = m.G * m.tiles;
    const int wave = blockIdx.x % gt;
    const int segs = KIND == kEnds ? m.S - 1 : m.S;
    const int seg = blockIdx.x / gt % segs;
    const int64_t b = blockIdx.x / gt / segs;
    const int g = wave / m.tiles;
    const int in_group = (wave % m.tiles) * 64 + threadIdx.x;
    const bool live = in_group < m.Cg;
    const int c = g * m.Cg + min(in_group, m.Cg - 1);
    const int64_t len = tokens_of(lengths, b, m);
    const int last = segments_of(len, m) - 1;
    // segments behind the sequence's last one; nothing continues from the last one's end
    if (KIND == kEnds ? seg >= last : seg > last) return;
    const int64_t t0 = (int64_t)seg * m.seg;
    const int64_t t1 = KIND == kWhole ? len : min(t0 + m.seg, len);
    const int count = (int)max(t1 - t0, (int64_t)0);
    const int Cw = gt * 64;
    const int64_t slot = b * m.S + seg;
    const int cw = wave * 64 + threadIdx.x;

    // A tile's rows are buffers that start at its first token's row; lane offset + row offset
    // stay far below kRange (at most kTile rows of 2^24 elements).  Lanes past the group's end
    // have an offset at its end: they read zeros and store nothing.
    constexpr int kRange = 0x7ffffffe;
    const int64_t row0 = b * m.L + t0;
    const uint32_t lane_off = live ? (uint32_t)(c * sizeof(T)) : (uint32_t)kRange;
    const bool gate = KIND != kEnds && z != nullptr;
    const uint32_t xp = (uint32_t)m.xp * sizeof(T), dp = (uint32_t)m.dtp * sizeof(T),
                   zp = gate ? (uint32_t)m.zp * sizeof(T) : 0;
    const T *xr = x + row0 * m.xp, *dr = dt + row0 * m.dtp;
    // without a gate the buffer is empty: its loads return zero and fetch nothing
    const T *zr = gate ? z + row0 * m.zp : x;
    const int z_range = gate ? kRange : 0;
    T *yr = KIND != kEnds ? y + row0 * m.C : nullptr;

    const T *Br = B + row0 * m.Bp + g * N, *Cr = Cm + row0 * m.Cp + g * N;

    // One tile of all inputs ahead, in registers.  Rows past the last token read that token
    // again and are not used.
    constexpr int kQuads = kTile * kRow / 4;                 // of B and C in a tile
    constexpr int kPer = (kQuads + 63) / 64;                 // per lane
    uint32_t xn[kTile], dn[kTile], zn[kTile];
    Quad<T> bn[kPer];
    auto fetch = [&](int t) {
        const rsrc_t xs = make_rsrc(xr + t * m.xp, kRange);
        const rsrc_t ds = make_rsrc(dr + t * m.dtp, kRange);
        const rsrc_t zs = make_rsrc(zr + (gate ? t * m.zp : 0), z_range);
        const int last = count - 1 - t;
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            const int q = min((int)threadIdx.x + 64 * j, kQuads - 1);
            const int64_t r = t + min(q / (kRow / 4), last);
            const int n = q % (kRow / 4) * 4;
            bn[j].load(KIND == kEnds || n < N ? Br + r * m.Bp + n : Cr + r * m.Cp + (n - N));
        }
#pragma unroll
        for (int i = 0; i < kTile; ++i) {
            const int r = min(i, last);
            xn[i] = buf_load<T>(xs, lane_off, r * xp);
            dn[i] = buf_load<T>(ds, lane_off, r * dp);
            if (KIND != kEnds) zn[i] = buf_load<T>(zs, lane_off, r * zp);
        }
    };
    // the first tile before the rates and states, so that these arrive with it (1024 tokens of
    // 2048 channels 27.6 -> 27.0 us)
    if (count > 0) fetch(0);
    float a2[N], h[N];
#pragma unroll
    for (int n = 0; n < N; n += 4) {
        const f32x4 v = *reinterpret_cast<const f32x4 *>(A + (int64_t)c * N + n);
#pragma unroll
        for (int i = 0; i < 4; ++i) a2[n + i] = kLog2e * v[i];
    }
#pragma unroll
    for (int n = 0; n < N; ++n) h[n] = 0.0f;
    if (KIND == kWhole && h0) {
#pragma unroll
        for (int n = 0; n < N; n += 4) {
            const f32x4 v = *reinterpret_cast<const f32x4 *>(h0 + (b * m.C + c) * N + n);
#pragma unroll
            for (int i = 0; i < 4; ++i) h[n + i] = v[i];
        }
    }
    if (KIND == kOut) {
#pragma unroll
        for (int n = 0; n < N; ++n) h[n] = ws.state[(slot * N + n) * Cw + cw];
    }
    const float bias = dt_bias ? dt_bias[c] : 0.0f;
    const float Dv = KIND != kEnds && D ? D[c] : 0.0f;
    float steps = 0.0f;

    for (int t = 0; t < count; t += kTile) {
        // (one wave: the tile is written over the previous one's reads without a barrier)
        wave_order();
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            const int q = (int)threadIdx.x + 64 * j;
            if (kQuads % 64 == 0 || q < kQuads) *reinterpret_cast<f32x4 *>(bc + 4 * q) = bn[j].get();
        }
        wave_order();
        float xv[kTile], dv[kTile], zv[kTile];
#pragma unroll
        for (int i = 0; i < kTile; ++i) {
            xv[i] = bits_to_f32<T>(xn[i]);
            dv[i] = bits_to_f32<T>(dn[i]) + bias;
            zv[i] = KIND != kEnds ? bits_to_f32<T>(zn[i]) : 0.0f;
        }
        if (m.sp) {
#pragma unroll
            for (int i = 0; i < kTile; ++i) dv[i] = softplus(dv[i]);
        }
        if (t + kTile < count) fetch(t + kTile);
#pragma unroll
        for (int i = 0; i < kTile; ++i) {
            if (t + i >= count) break;
            const float u = dv[i] * xv[i];
            if (KIND == kEnds) steps += dv[i];
            float acc = Dv * xv[i];
#pragma unroll
            for (int n = 0; n < N; n += 4) {
                const f32x4 bv = *reinterpret_cast<const f32x4 *>(bc + i * kRow + n);
                f32x4 cv;
                if (KIND != kEnds) cv = *reinterpret_cast<const f32x4 *>(bc + i * kRow + N + n);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float a = fast_exp2(dv[i] * a2[n + k]);
                    // (the product that replaces h and the sum in its place: no register moves)
                    h[n + k] = fmaf(u, bv[k], a * h[n + k]);
                    if (KIND != kEnds) acc = fmaf(cv[k], h[n + k], acc);
                }
            }
            if (KIND != kEnds) {
                if (gate) acc *= silu(zv[i]);
                buf_store<T>(make_rsrc(yr, kRange), lane_off, 0, Elem<T>::from_f32(acc));
                yr += m.C;
            }
        }
    }
    if (KIND == kEnds) {
#pragma unroll
        for (int n = 0; n < N; ++n) ws.state[(slot * N + n) * Cw + cw] = h[n];
        ws.steps[slot * Cw + cw] = steps;
    } else if (hT && live && seg == last) {
#pragma unroll
        for (int n = 0; n < N; n += 4) {
            f32x4 v;
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = h[n + i];
            *reinterpret_cast<f32x4 *>(hT + (b * m.C + c) * N + n) = v;
        }
    }
}

// The factor 2^v of a whole segment, as f 2^k with f in [0.7, 1.42]: with growing states, or
// quickly shrinking ones, it may leave fp32's range where the states on both sides of it do not,
// and a state that is still zero has to stay zero under it.  Past +-600 every state but zero and
// infinity becomes infinite or zero (2^-149 to 2^128 are 277 apart); a NaN among the steps or
// rates is in the segment's end state too.
struct Factor {
    float f;
    int k;
    __device__ __forceinline__ void set(float v)
    {
        v = __builtin_amdgcn_fmed3f(v, -600.0f, 600.0f);
        const float whole = __builtin_rintf(v);
        f = fast_exp2(v - whole);
        k = (int)whole;
    }
    // 2^v h + end
    __device__ __forceinline__ float apply(float h, float end) const
    {
        return fmaf(f, __builtin_ldexpf(h, k), end);
    }
};

// Turns the segments' end states (each from zero) into their start states, in place: along
// the segments, start[0] = h0 and start[s + 1] = exp(A sum of steps of s) start[s] + end[s].
// A workgroup owns 64 channels and one state; its waves take runs of segments, load them all at
// once, form each run's own decay and end, and after an exchange through LDS walk their runs
// from the true start: two trips to memory whatever the number of segments in a round.
// Wave, segments and their addresses are scalars; a lane adds its channel.
constexpr int kRunWaves = 8, kRun = 16;     // at most: waves of a workgroup, segments of a run
__global__ __launch_bounds__(64 * kRunWaves) void scan_chain_kernel(
    const float *__restrict__ A, const float *h0, const int32_t *__restrict__ lengths, ScanWs ws,
    int N, ScanDims m)
{
    __shared__ Factor run_factor[kRunWaves][64];
    __shared__ float run_end[kRunWaves][64];
    const uint32_t lane = threadIdx.x & 63;
    const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int gt = m.G * m.tiles;
    const int wave = blockIdx.x % gt, n = blockIdx.x / gt % N;
    const int64_t b = blockIdx.x / gt / N;
    const int64_t Cw = (int64_t)gt * 64;
    const int in_group = (wave % m.tiles) * 64 + lane;
    const bool live = in_group < m.Cg;
    const int c = wave / m.tiles * m.Cg + min(in_group, m.Cg - 1);
    // (scaled at its use: the loads below are not to wait for it)
    const float rate = A[(int64_t)c * N + n];
    float h = h0 && live ? h0[(b * m.C + c) * N + n] : 0.0f;
    float *st = ws.state + (b * m.S * N + n) * Cw + wave * 64;
    const float *sm = ws.steps + b * m.S * Cw + wave * 64;
    // segments 0 .. S - 2 have an end state; start states are written for 0 .. S - 1
    const int S = segments_of(tokens_of(lengths, b, m), m);
    const int nw = blockDim.x >> 6;
    for (int s0 = 0; s0 < S; s0 += nw * kRun) {
        const int per = min((S - s0 + nw - 1) / nw, kRun);
        const int first = s0 + wv * per;
        const int starts = min(per, S - first), ends = min(per, S - 1 - first);
        float e[kRun], d[kRun];
        Factor step[kRun];
#pragma unroll
        for (int i = 0; i < kRun; ++i) {
            if (i < ends) {
                e[i] = (st + (int64_t)(first + i) * N * Cw)[lane];
                d[i] = (sm + (first + i) * Cw)[lane];
            }
        }
        // a run's factor by its exponent, the sum of the segments'
        float log_sum = 0.0f, end = 0.0f;
#pragma unroll
        for (int i = 0; i < kRun; ++i) {
            if (i < ends) {
                const float v = rate * (kLog2e * d[i]);
                step[i].set(v);
                end = step[i].apply(end, e[i]);
                log_sum += v;
            }
        }
        run_factor[wv][lane].set(log_sum);
        run_end[wv][lane] = end;
        __syncthreads();
        float mine = h;
        for (int w = 0; w < nw; ++w) {
            if (w == wv) mine = h;
            h = run_factor[w][lane].apply(h, run_end[w][lane]);
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kRun; ++i) {
            if (i < starts) (st + (int64_t)(first + i) * N * Cw)[lane] = mine;
            if (i < ends) mine = step[i].apply(mine, e[i]);
        }
    }
}

// ---------------------------------------------------------------------------
// Short prompts in one launch.  A workgroup owns 64 / kLanes channels of one group, a wave of
// it kShort tokens; within a wave kLanes (4 or 8) lanes share a channel, N / kLanes states each,
// so that few channels still spread over the card.  Inputs and outputs are loaded and stored
// with a lane for one channel of a few tokens, which also forms their softplus and gates, and
// change places with the walk's layout through LDS.  Every wave walks its tokens from zero; the waves then
// share the chain of these ends, each taking some of the states, and walk again from their
// starts with the outputs.
// ---------------------------------------------------------------------------
constexpr int kShort = 16;       // tokens of a wave

template <typename T, int N, int kWaves, int kLanes>
__global__ __launch_bounds__(64 * kWaves) void scan_short_kernel(
    const T *__restrict__ x, const T *__restrict__ dt, const float *__restrict__ A,
    const T *__restrict__ B, const T *__restrict__ Cm, const float *__restrict__ D,
    const T *__restrict__ z, const float *__restrict__ dt_bias, const float *h0,
    const int32_t *__restrict__ lengths, T *__restrict__ y, float *hT, ScanDims m)
{
    constexpr int kCh = 64 / kLanes, kOwn = N / kLanes;  // channels of the workgroup, states of a lane
    constexpr int kSide = 64 / kCh, kPass = kShort / kSide;   // tokens side by side, and passes over them
    constexpr int kRow = 2 * N, kQuads = kShort * kRow / 4, kPer = kQuads / 64;
    __shared__ __attribute__((aligned(16))) float bcs[kWaves][kShort * kRow];
    __shared__ float2 dus[kWaves][kShort][kCh];     // step d, d x
    __shared__ float ys[kWaves][kShort][kCh];
    __shared__ float ends[kWaves][kOwn][64], sums[kWaves][kCh];
    const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lane = threadIdx.x & 63;
    const int tiles = (m.Cg + kCh - 1) / kCh;
    const int tile = blockIdx.x % tiles, g = blockIdx.x / tiles % m.G;
    const int64_t b = blockIdx.x / tiles / m.G;
    const int first = g * m.Cg + tile * kCh, most = g * m.Cg + m.Cg - 1;
    const int64_t len = tokens_of(lengths, b, m);
    const int t0 = wv * kShort;
    const int count = min(max((int)len - t0, 0), kShort);
    const int64_t row0 = b * m.L + t0;

    // the walk's layout: channel lane / kLanes, states part * kOwn ...
    const int ch = lane / kLanes, part = lane % kLanes;
    const int c = min(first + ch, most);
    float a2[kOwn], h[kOwn];
#pragma unroll
    for (int k = 0; k < kOwn; ++k) {
        a2[k] = kLog2e * A[(int64_t)c * N + part * kOwn + k];
        h[k] = 0.0f;
    }
    // the inputs' layout: channel lane % kCh, tokens lane / kCh + kSide j
    const int il = lane % kCh, it = lane / kCh;
    const int ic = min(first + il, most);
    const bool live = first + il <= most;
    float xv[kPass], zv[kPass];
    if (count > 0) {
        Quad<T> q[kPer];
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            const int i = lane + 64 * j;
            const int64_t r = row0 + min(i / (kRow / 4), count - 1);
            const int n = i % (kRow / 4) * 4;
            q[j].load(n < N ? B + r * m.Bp + g * N + n : Cm + r * m.Cp + g * N + (n - N));
        }
        float dv[kPass];
#pragma unroll
        for (int j = 0; j < kPass; ++j) {
            const int64_t r = row0 + min(it + kSide * j, count - 1);
            xv[j] = (float)x[r * m.xp + ic];
            dv[j] = (float)dt[r * m.dtp + ic];
            zv[j] = z ? (float)z[r * m.zp + ic] : 0.0f;
        }
        const float bias = dt_bias ? dt_bias[ic] : 0.0f;
#pragma unroll
        for (int j = 0; j < kPer; ++j)
            *reinterpret_cast<f32x4 *>(&bcs[wv][4 * (lane + 64 * j)]) = q[j].get();
#pragma unroll
        for (int j = 0; j < kPass; ++j) {
            float d = dv[j] + bias;
            if (m.sp) d = softplus(d);
            dus[wv][it + kSide * j][il] = make_float2(d, d * xv[j]);
        }
    }
    wave_order();
    auto states = [&](int i, int at, float *v) {         // kOwn values of B (at 0) or C (at N)
        const float *p = &bcs[wv][i * kRow + at + part * kOwn];
#pragma unroll
        for (int k = 0; k < kOwn; ++k) v[k] = p[k];
    };
    const int nw = blockDim.x >> 6;
    if (nw == 1) {
        // one wave starts from h0 itself
#pragma unroll
        for (int k = 0; k < kOwn; ++k)
            if (h0) h[k] = h0[(b * m.C + c) * N + part * kOwn + k];
    } else {
        float sum = 0.0f;
#pragma unroll 4
        for (int i = 0; i < count; ++i) {
            const float2 du = dus[wv][i][ch];
            float bv[kOwn];
            states(i, 0, bv);
#pragma unroll
            for (int k = 0; k < kOwn; ++k)
                h[k] = fmaf(du.y, bv[k], fast_exp2(du.x * a2[k]) * h[k]);
            sum += du.x;
        }
#pragma unroll
        for (int k = 0; k < kOwn; ++k) ends[wv][k][lane] = h[k];
        if (part == 0) sums[wv][ch] = sum;
        __syncthreads();
        for (int k = wv; k < kOwn; k += nw) {
            const float rate = kLog2e * A[(int64_t)c * N + part * kOwn + k];
            float now = h0 ? h0[(b * m.C + c) * N + part * kOwn + k] : 0.0f;
            float e[kWaves];
            Factor step[kWaves];
#pragma unroll
            for (int w = 0; w < kWaves; ++w) {
                if (w < nw) {
                    e[w] = ends[w][k][lane];
                    step[w].set(rate * sums[w][ch]);
                }
            }
#pragma unroll
            for (int w = 0; w < kWaves; ++w) {
                if (w < nw) {
                    ends[w][k][lane] = now;
                    now = step[w].apply(now, e[w]);
                }
            }
        }
        __syncthreads();               // (h0 has been read: a wave may now write hT over it)
#pragma unroll
        for (int k = 0; k < kOwn; ++k) h[k] = ends[wv][k][lane];
    }
    auto token = [&](int i) {
        const float2 du = dus[wv][i][ch];
        float bv[kOwn], cv[kOwn], acc = 0.0f;
        states(i, 0, bv);
        states(i, N, cv);
#pragma unroll
        for (int k = 0; k < kOwn; ++k) {
            h[k] = fmaf(du.y, bv[k], fast_exp2(du.x * a2[k]) * h[k]);
            acc = fmaf(cv[k], h[k], acc);
        }
        acc += dpp_move<0xb1, 0xf>(acc);     // quad_perm 1 0 3 2
        acc += dpp_move<0x4e, 0xf>(acc);     // quad_perm 2 3 0 1
        if (kLanes == 8) acc += dpp_move<0x141, 0xf>(acc);     // row_half_mirror
        if (part == 0) ys[wv][i][ch] = acc;
    };
    // (four at a time by hand: the lane moves keep the compiler from it)
    int i0 = 0;
    for (; i0 + 4 <= count; i0 += 4) {
        token(i0);
        token(i0 + 1);
        token(i0 + 2);
        token(i0 + 3);
    }
    for (; i0 < count; ++i0) token(i0);
    wave_order();
    const float Dv = D ? D[ic] : 0.0f;
#pragma unroll
    for (int j = 0; j < kPass; ++j) {
        const int i = it + kSide * j;
        if (i < count && live) {
            float v = fmaf(Dv, xv[j], ys[wv][i][il]);
            if (z) v *= silu(zv[j]);
            y[(row0 + i) * m.C + ic] = Elem<T>::from_f32(v);
        }
    }
    // the wave of the sequence's last token (the first wave of an empty sequence)
    if (hT && wv == max((int)((len + kShort - 1) / kShort), 1) - 1 && first + ch <= most) {
#pragma unroll
        for (int k = 0; k < kOwn; ++k) hT[(b * m.C + c) * N + part * kOwn + k] = h[k];
    }
}

// One token.  The state is read and written once, 8 bytes a state element: HBM bound, latency
// bound for few sequences.  kLanes lanes, the largest power of two that divides N / 4, share a
// channel, so that neighbouring lanes hold neighbouring 16 bytes of the state.  128 sequences of
// 2048 channels of 16 states, bf16: 9.5 us with the state out of the caches (3.7 TB/s), 8.4
// where the Infinity Cache holds it (a lane with the 64 bytes of a whole channel: 11.3); one
// sequence: 3.3 us, most of it the launch.
template <typename T, int N>
__global__ __launch_bounds__(256) void scan_step_kernel(
    const T *__restrict__ x, const T *__restrict__ dt, const float *__restrict__ A,
    const T *__restrict__ B, const T *__restrict__ Cm, const float *__restrict__ D,
    const T *__restrict__ z, const float *__restrict__ dt_bias, float *__restrict__ h,
    T *__restrict__ y, ScanDims m, uint32_t threads)
{
    constexpr int kLanes = (N / 4) & -(N / 4), kVecs = N / 4 / kLanes;
    const uint32_t id = blockIdx.x * 256 + threadIdx.x;
    if (id >= threads) return;         // threads is a multiple of kLanes
    const uint32_t bc = id / kLanes, part = id % kLanes;
    const int64_t b = bc / (uint32_t)m.C;
    const int c = (int)(bc % (uint32_t)m.C), g = c / m.Cg;
    float *hp = h + (int64_t)bc * N + part * 4;
    const float *ap = A + (int64_t)c * N + part * 4;
    const T *bp = B + b * m.Bp + g * N + part * 4, *cp = Cm + b * m.Cp + g * N + part * 4;
    f32x4 hv[kVecs], av[kVecs];
    Quad<T> bv[kVecs], cv[kVecs];
#pragma unroll
    for (int k = 0; k < kVecs; ++k) {
        const int n = 4 * kLanes * k;
        hv[k] = *reinterpret_cast<const f32x4 *>(hp + n);
        av[k] = *reinterpret_cast<const f32x4 *>(ap + n);
        bv[k].load(bp + n);
        cv[k].load(cp + n);
    }
    const float xv = (float)x[b * m.xp + c];
    const float zv = z ? (float)z[b * m.zp + c] : 0.0f;
    float d = (float)dt[b * m.dtp + c] + (dt_bias ? dt_bias[c] : 0.0f);
    if (m.sp) d = softplus(d);
    const float u = d * xv, d2 = kLog2e * d;
    float acc = 0.0f;
#pragma unroll
    for (int k = 0; k < kVecs; ++k) {
        const f32x4 bf = bv[k].get(), cf = cv[k].get();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            hv[k][i] = fmaf(u, bf[i], fast_exp2(d2 * av[k][i]) * hv[k][i]);
            acc = fmaf(cf[i], hv[k][i], acc);
        }
        *reinterpret_cast<f32x4 *>(hp + 4 * kLanes * k) = hv[k];
    }
#pragma unroll
    for (int k = 1; k < kLanes; k *= 2) acc += __shfl_xor(acc, k, 64);
    if (D) acc = fmaf(D[c], xv, acc);
    if (z) acc *= silu(zv);
    if (part == 0) y[(int64_t)bc] = Elem<T>::from_f32(acc);
}

// Segments that a sequence is split into, and tokens in each (a multiple of kStep); `waves`
// waves of 64 channels would walk whole sequences.
//   - From 1024 of them (one a SIMD) the sequences stay whole: the end states cost most of a
//     second walk, which more waves then no longer make up for.  2048 tokens of 4096 channels of 16
//     states, whole and split, in us: 8 sequences (512 waves) 696 and 465, 12 (768) 699 and 649, 15
//     (960) 696 and 784, 16 (1024) 692 and 790, 24 (1536) 985 and 1150, 32 (2048) 996 and 1454.  The
//     rule does not know of lengths: ragged batches of those sizes gain from a split up to 2048 waves
//     (686 and 278 at 512, 683 and 486 at 1024, 719 and 670 at 1536, 907 and 792 at 2048), so for
//     them the border lies low, and for dense ones between 768 and 1024 a little high.
//   - So do sequences under 32 tokens, where two more launches cost more than a walk (16 tokens:
//     7.8 us whole, 12.0 split; 32 tokens: 13.0 and 12.1).
//   - Else up to about 16384 waves of at least 64 tokens (30 ragged sequences of 1000 tokens, 2048
//     channels: 220 us, 252 with 8192; dense 380 and 385), or 8192 of at least 32 (one
//     16384-token sequence of 2048 channels: 231 us with 2048 waves, 209 with 4096, 204 with
//     8192, 214 to 219 with 16384; eight ragged ones of 2048 tokens: 204 with 4096, 146 with
//     8192), or 4096 of fewer tokens (four of 2048 tokens, 1024 channels of 32 states: 116 us,
//     125 with 24 tokens), at least 16, or 8 where even these are few (512 tokens, 512 channels: 13.9 us against 17.2).
void split_of(const ScanShape &s, int64_t waves, int &S, int &seg)
{
    int64_t tokens = s.L;
    if (waves < 1024 && s.L >= 32) {
        const int64_t least = waves * s.L <= 8 * 2048 ? 8 : 16;
        const auto share = [&](int64_t n) { return (waves * s.L + n - 1) / n; };
        tokens = share(16384) >= 64 ? share(16384)
                 : share(8192) >= 32 ? (share(8192) < 64 ? share(8192) : 64)
                 : share(4096) < 32  ? share(4096)
                                     : 32;
        if (tokens < least) tokens = least;
    }
    tokens = (tokens + kStep - 1) / kStep * kStep;
    seg = (int)tokens;
    S = (int)((s.L + tokens - 1) / tokens);
}

ScanDims dims_of(const ScanShape &s)
{
    ScanDims m;
    m.L = s.L; m.xp = s.xp; m.dtp = s.dtp; m.zp = s.zp; m.Bp = s.Bp; m.Cp = s.Cp;
    m.C = (int)s.C; m.G = (int)s.G; m.Cg = (int)(s.C / s.G);
    m.tiles = (m.Cg + 63) / 64;
    m.sp = s.softplus;
    split_of(s, (int64_t)m.tiles * m.G * s.b, m.S, m.seg);
    return m;
}

int64_t waves_of(const ScanShape &s, const ScanDims &m) { return (int64_t)m.tiles * m.G * s.b; }

// How a short scan is launched: waves of a workgroup (0: not as one launch), lanes of a channel.
// One launch takes what a workgroup's LDS holds (16 waves of 16 tokens, 8 for more than 32
// states), up to 4096 waves of four lanes a channel; eight lanes up to 2048 of these.  One launch
// with eight lanes, with four, and segments, in us: 64 tokens x 2048 channels x 16 states 6.3,
// 7.5 and 12.4, 256 x 256 8.5, 11.7 and 12.6, 100 x 512 x 64 states 11.2, 17.6 and 24; at 4096
// waves (8 x 64 x 2048) 16.9, 12.5 and 21; at 8192 (4 x 256 x 2048) four lanes take 28.7,
// segments 27.1.  A single token takes 3.3 against 3.7 for whole walks, 16 tokens 4.6 and 8.0.
struct ShortPlan {
    int waves, lanes;
    int64_t groups;
};
ShortPlan short_plan(const ScanShape &s)
{
    constexpr int64_t kMost = 4096, kEight = 2048;
    const int64_t waves = (s.L + kShort - 1) / kShort;
    const auto groups = [&](int64_t lanes) {
        const int64_t ch = 64 / lanes;
        return s.b * s.G * ((s.C / s.G + ch - 1) / ch);
    };
    ShortPlan p = {0, 4, groups(4)};
    if (waves > (s.N <= 32 ? 16 : 8) || waves * p.groups > kMost) return p;
    p.waves = (int)waves;
    if (waves * p.groups <= kEight) p = {(int)waves, 8, groups(8)};
    return p;
}

template <typename T, int N>
hipError_t scan_short(const ShortPlan &p, const ScanDims &m, const ScanArgs &a, hipStream_t st)
{
#define SSD_SHORT(W, LANES)                                                                       \
    hipLaunchKernelGGL((scan_short_kernel<T, N, W, LANES>), dim3((unsigned)p.groups),             \
                       dim3(64 * p.waves), 0, st, (const T *)a.x, (const T *)a.dt, a.A,           \
                       (const T *)a.B, (const T *)a.C, a.D, (const T *)a.z, a.dt_bias, a.h0,      \
                       a.lengths, (T *)a.y, a.hT, m)
    constexpr int kMost = N <= 32 ? 16 : 8;
    if (p.lanes == 4 && p.waves <= 4) SSD_SHORT(4, 4);
    else if (p.lanes == 4) SSD_SHORT(kMost, 4);
    else if (p.waves <= 4) SSD_SHORT(4, 8);
    else SSD_SHORT(kMost, 8);
#undef SSD_SHORT
    return hipGetLastError();
}

template <typename T, int N, int KIND>
hipError_t scan_pass(const ScanShape &s, const ScanDims &m, const ScanWs &ws, const ScanArgs &a,
                     hipStream_t st)
{
    const int64_t waves = waves_of(s, m) * (KIND == kEnds ? m.S - 1 : m.S);
    hipLaunchKernelGGL((scan_kernel<T, N, KIND>), dim3((unsigned)waves), dim3(64), 0, st,
                       (const T *)a.x, (const T *)a.dt, a.A, (const T *)a.B, (const T *)a.C, a.D,
                       (const T *)a.z, a.dt_bias, a.h0, a.lengths, (T *)a.y, a.hT, ws, m);
    return hipGetLastError();
}

template <typename T, int N>
hipError_t scan_go(const ScanShape &s, const ScanArgs &a, float *h, hipStream_t st)
{
    const ScanDims m = dims_of(s);
    if (h) {
        // at most 2^31 / 4 (the limit on batch * channels * dstate)
        const uint32_t threads = (uint32_t)(s.b * s.C * ((N / 4) & -(N / 4)));
        hipLaunchKernelGGL((scan_step_kernel<T, N>), dim3((threads + 255) / 256), dim3(256), 0, st,
                           (const T *)a.x, (const T *)a.dt, a.A, (const T *)a.B, (const T *)a.C,
                           a.D, (const T *)a.z, a.dt_bias, h, (T *)a.y, m, threads);
        return hipGetLastError();
    }
    const ShortPlan p = short_plan(s);
    if (p.waves > 0) return scan_short<T, N>(p, m, a, st);
    const int64_t Cw = (int64_t)m.G * m.tiles * 64;
    ScanWs ws;
    ws.state = (float *)a.ws;
    ws.steps = ws.state + s.b * m.S * N * Cw;
    if (m.S == 1) return scan_pass<T, N, kWhole>(s, m, ws, a, st);
    hipError_t e = scan_pass<T, N, kEnds>(s, m, ws, a, st);
    if (e != hipSuccess) return e;
    // Waves of a chain workgroup: runs of eight segments where there are few workgroups (32768
    // tokens of 512 channels: 130 us, 141 with runs of sixteen), else of sixteen (four sequences
    // of 2048 tokens, 2048 channels: 115 us against 121)
    const int64_t chains = (int64_t)m.G * m.tiles * N * s.b;
    const int least = chains < 1024 ? 8 : 16;
    const int run_waves = m.S >= least * kRunWaves ? kRunWaves : (m.S + least - 1) / least;
    hipLaunchKernelGGL(scan_chain_kernel, dim3((unsigned)chains), dim3(64 * run_waves), 0, st, a.A,
                       a.h0, a.lengths, ws, N, m);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    return scan_pass<T, N, kOut>(s, m, ws, a, st);
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

size_t scan_workspace_bytes(const ScanShape &s)
{
    const ScanDims m = dims_of(s);
    if (m.S == 1 || short_plan(s).waves > 0) return SSD_SCAN_NO_WORKSPACE;
    return (size_t)s.b * m.S * (s.N + 1) * m.G * m.tiles * 64 * sizeof(float);
}

hipError_t launch_scan(const ScanShape &s, const ScanArgs &a, hipStream_t st)
{
    return s.bf16 ? scan_by_state<bf16>(s, a, nullptr, st) : scan_by_state<float>(s, a, nullptr, st);
}

hipError_t launch_scan_step(const ScanShape &s, const ScanArgs &a, float *h, hipStream_t st)
{
    return s.bf16 ? scan_by_state<bf16>(s, a, h, st) : scan_by_state<float>(s, a, h, st);
}

}  // namespace ssd
