// ssd_linattn.hip -- linear attention with a decay for each head: prompts, their gradients.
//
// With a_t = exp(min(g_t, 0)) and the state S [value, key] of a head,
//     S_t = a_t S_(t-1) + v_t k_t^T,      o_t = scale S_t q_t
// is evaluated 64 tokens (a chunk) at a time.  With G_t the sum of the log decays from the
// chunk's first token through t, E its last,
//     o_t = scale (exp(G_t) S q_t + sum_(s <= t) exp(G_t - G_s) (k_s . q_t) v_s)
//     S  <- exp(G_E) S + sum_s exp(G_E - G_s) v_s k_s^T
// so that a chunk is four matrix products.  A "walk" does that for one head and 64 of its
// values, chunk by chunk, the state in registers.
//
// The gradients are walks too, in other roles (dS the gradient of the state):
//     dq_t = scale S_t^T do_t                        forward in time:  q <- do, k <- v, v <- k
//     dk_t = dS_t^T v_t                              back in time:     q <- v, k <- do, v <- q
//     dv_t = dS_t k_t                                back in time:     q <- k, k <- q, v <- do
//     dS_(t-1) = a_t (dS_t), dS_t += scale do_t q_t^T
// Back in time a token's own decay lies behind it: the factors of a chunk swap their ends.
//
// Exponents.  Every log decay goes through min(g, 0) (a decay never grows) and max(.., -1000)
// in base 2 (a factor of 2^-150 is zero in fp32), so sums of 64 stay below 2^16.  Each is
// split into a multiple of 2^-8 and a rest: sums and differences of the first parts are exact
// in fp32, those of the rest err by less than 2^-27, however far G has fallen.
//
// Rounding.  States and all sums are fp32.  For bf16 the matrix operands are bf16: inputs as
// they are, the decayed scores and the state that a chunk reads each rounded once; but what
// is added to the state, w_s v_s, goes in as three bf16 parts (8 + 8 + 8 bits, fp32's 24), so
// that states, which leave the kernel in fp32, hold fp32's precision.
#include <hip/hip_runtime.h>

#include "../../include/ssd.h"
#include "ssd_device.h"
#include "ssd_launch.h"

namespace ssd {
namespace {

constexpr int kChunk = 64;       // tokens of a chunk
constexpr int kBlock = 64;       // values of a walk
constexpr int kThreads = 256;    // four waves

// What a walk is run for: the state that a segment of chunks leaves, from zero; an output (of the
// forward, or the gradient of v); the gradient of q or k with its part of the decays' gradient.
enum Kind { kEnds, kOut, kDq, kDk };

// A walk's arrays, in the roles of the forward.
struct Walk {
    const void *q, *k, *v;
    int64_t qp, kp, vp;         // elements from token to token
    int qdiv, kdiv, vdiv;       // heads that share one of q, k, v
    const void *g;
    int64_t gp;
    int decay;
    const int32_t *lengths;
    void *o;                    // [b, L, H, vd]
    bool o32;                   // in fp32 (else in the inputs' type)
    const float *init;          // value v, key k of a head at v sv + k sk; may be NULL
    int64_t sv, sk;
    float *last;                // [b, H, vd, kd]; may be NULL
    // Segments: `seg` chunks each, nseg of them, in the walk's order.  With more than one, kEnds
    // leaves their ends (from zero) and decays, a chain over those their starts, for the others.
    int seg, nseg;
    float *ends;                // [b H, nseg, vd kd] in init's layout: segment s's end at s + 1, then
                                // its start at s
    float *decays;              // [b H, nseg]: over segment s
    float inter, intra;         // factors of an output's two parts
    float weight;               // factor of what is added to the state
    int L, H, kd, vd, nvb;
    int64_t groups;             // heads x segments
    // kDq, kDk: the array whose product with the output the decays' gradient takes (q, k), this
    // walk's part of it, and the states before each chunk, [b H, chunks, vd, kd]
    const void *x;
    int64_t xp;
    int xdiv;
    float *part;                // [b H, nvb, L]
    void *states;
    float *cross;               // [b H, nvb, chunks]
    int nchunks;
};

struct DecayGradient {
    const void *g;
    int64_t gp;
    const int32_t *lengths;
    const float *read, *written, *cross;
    void *dg;
    int64_t bh;
    int L, H, nvb, nchunks;
};

// ---------------------------------------------------------------------------
// Tiles of 16 x 16.  An accumulator's lane l holds column l % 16, rows 4 (l / 16) + r.
// A key fragment is 16 bytes of a row (row l % 16): bf16 keys 8 (l / 16) + e of 32, one
// instruction; fp32 keys 4 (l / 16) + e of 16, one instruction for each e.  A source fragment
// is eight tokens of one column (column l % 16), in the order in which two accumulators
// hold their rows: tokens 4 (l / 16) + e of the first 16 and of the second.
// ---------------------------------------------------------------------------
template <typename T> struct Tile;
template <> struct Tile<bf16> {
    typedef bf16x8 key;
    typedef bf16x8 src;
    static constexpr int kKeys = 32;
    static constexpr int kStepKeys = 8;
    // 32 bytes off a multiple of 128: the transpose reads' four rows in different banks
    static constexpr int pitch(int n) { return n + 16; }
    static constexpr int state_pitch(int n) { return n + 8; }
};
template <> struct Tile<float> {
    typedef f32x4 key;
    typedef f32x8 src;
    static constexpr int kKeys = 16;
    static constexpr int kStepKeys = 4;
    static constexpr int pitch(int n) { return n + 4; }
    static constexpr int state_pitch(int n) { return n + 4; }
};

__device__ __forceinline__ f32x4 mma16(const bf16x8 &a, const bf16x8 &b, f32x4 c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mma16(const f32x4 &a, const f32x4 &b, f32x4 c)
{
#pragma unroll
    for (int e = 0; e < 4; ++e) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[e], b[e], c, 0, 0, 0);
    return c;
}
__device__ __forceinline__ f32x4 mma16(const f32x8 &a, const f32x8 &b, f32x4 c)
{
#pragma unroll
    for (int e = 0; e < 8; ++e) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[e], b[e], c, 0, 0, 0);
    return c;
}

// The source fragment of tokens `row` .. `row` + 31 and columns `col` .. `col` + 15 of a tile
// stored token by token.
__device__ __forceinline__ bf16x8 load_src(const bf16 *s, int pitch, int row, int col, int lane)
{
    const bf16 *p = s + (row + 4 * (lane >> 4) + ((lane & 15) >> 2)) * pitch + col + 4 * (lane & 3);
    return cat8(tr_read4(p), tr_read4(p + 16 * pitch));
}
__device__ __forceinline__ f32x8 load_src(const float *s, int pitch, int row, int col, int lane)
{
    const float *p = s + (row + 4 * (lane >> 4)) * pitch + col + (lane & 15);
    f32x8 f;
#pragma unroll
    for (int e = 0; e < 4; ++e) { f[e] = p[e * pitch]; f[4 + e] = p[(16 + e) * pitch]; }
    return f;
}

// acc += a (w x)^T for the source fragments a and x: three bf16 parts of each product w x
// hold its 24 bits.
__device__ __forceinline__ void split3(const bf16x8 &x, const f32x8 &w, bf16x8 (&p)[3])
{
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        float v = (float)x[e] * w[e];
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            p[i][e] = (bf16)v;
            v -= (float)p[i][e];
        }
    }
}

template <typename T> __device__ __forceinline__ typename Tile<T>::src pack_src(const f32x4 &a,
                                                                                 const f32x4 &b);
template <> __device__ __forceinline__ bf16x8 pack_src<bf16>(const f32x4 &a, const f32x4 &b)
{
    bf16x8 r;
#pragma unroll
    for (int e = 0; e < 4; ++e) { r[e] = (bf16)a[e]; r[4 + e] = (bf16)b[e]; }
    return r;
}
template <> __device__ __forceinline__ f32x8 pack_src<float>(const f32x4 &a, const f32x4 &b)
{
    f32x8 r;
#pragma unroll
    for (int e = 0; e < 4; ++e) { r[e] = a[e]; r[4 + e] = b[e]; }
    return r;
}

// Four elements as T, in LDS or memory.
__device__ __forceinline__ void store4(bf16 *p, const f32x4 &v)
{
    bf16x4 r;
#pragma unroll
    for (int e = 0; e < 4; ++e) r[e] = (bf16)v[e];
    *reinterpret_cast<bf16x4 *>(p) = r;
}
__device__ __forceinline__ void store4(float *p, const f32x4 &v) { *reinterpret_cast<f32x4 *>(p) = v; }
__device__ __forceinline__ f32x4 load4(const bf16 *p)
{
    const bf16x4 v = *reinterpret_cast<const bf16x4 *>(p);
    f32x4 r;
#pragma unroll
    for (int e = 0; e < 4; ++e) r[e] = (float)v[e];
    return r;
}
__device__ __forceinline__ f32x4 load4(const float *p) { return *reinterpret_cast<const f32x4 *>(p); }

// The same through a buffer, past whose end nothing is written.
__device__ __forceinline__ void buf_store4(rsrc_t r, uint32_t off, const f32x4 &v, bf16 *)
{
    u32x2 w;
    w[0] = pack_bf16(v[0], v[1]);
    w[1] = pack_bf16(v[2], v[3]);
    __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(__attribute__((ext_vector_type(2))) unsigned int, w), r,
                                          (int)off, 0, 0);
}
__device__ __forceinline__ void buf_store4(rsrc_t r, uint32_t off, const f32x4 &v, float *)
{
    buf_store_b128(r, off, __builtin_bit_cast(u32x4, v));
}

// A token's log decay in base 2, between -1000 and 0; a NaN stays one.
__device__ __forceinline__ float decay2(float g)
{
    g *= kLog2e;
    g = g > 0.0f ? 0.0f : g;
    return g < -1000.0f ? -1000.0f : g;
}

__device__ __forceinline__ float rows_sum(float v)      // over the four rows of 16 lanes
{
    v += __shfl_xor(v, 16, 64);
    return v + __shfl_xor(v, 32, 64);
}
__device__ __forceinline__ float columns_sum(float v)   // over the 16 lanes of a row, in lane 15
{
    v += dpp_move<0x111, 0xf>(v);
    v += dpp_move<0x112, 0xf>(v);
    v += dpp_move<0x114, 0xf>(v);
    return v + dpp_move<0x118, 0xf>(v);
}

// ---------------------------------------------------------------------------
// A walk: one (batch, head) and 64 of its values, all chunks.
//
// Products per chunk and wave (w the wave, i its 16 targets, all transposed so that an
// accumulator is the next product's operand as it stands):
//   scores [source, i] = K q_i          keys contracted, K from LDS, q from memory
//   o [value, i] = S q_i                S [value, key] rounded into LDS by the last chunk
//   o += V^T scores                     tokens contracted, V read transposed
//   S [key, value w] += K^T (w V)       tokens contracted, K read transposed
// The next chunk's K, V and q are on their way while these run.
// ---------------------------------------------------------------------------
template <typename T, int DK, bool REV, Kind KIND>
__global__ __launch_bounds__(kThreads, DK * sizeof(T) <= 256 ? 2 : 1) void walk_kernel(Walk a)
{
    typedef typename Tile<T>::key Key;
    typedef typename Tile<T>::src Src;
    constexpr int KP = Tile<T>::pitch(DK), VP = Tile<T>::pitch(kBlock), SP = Tile<T>::state_pitch(DK);
    constexpr int KK = DK / Tile<T>::kKeys, KT = DK / 16;
    constexpr int kVec = 16 / (int)sizeof(T);                        // elements of 16 bytes
    constexpr int KI = kChunk * DK / kVec / kThreads;                // 16-byte pieces a thread
    constexpr int VI = kChunk * kBlock / kVec / kThreads;
    constexpr int BK = kBlock / Tile<T>::kKeys;                      // fragments of 64 values
    __shared__ __attribute__((aligned(16))) T sK[kChunk * KP];
    __shared__ __attribute__((aligned(16))) T sV[kChunk * VP];
    __shared__ __attribute__((aligned(16))) T sS[kBlock * SP];
    __shared__ __attribute__((aligned(16))) float sHi[kChunk], sLo[kChunk], sIn[kChunk], sW[kChunk];
    __shared__ float sZ[kChunk], sC[4][kChunk], sX[4];

    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int c16 = lane & 15, g4 = lane >> 4;
    // workgroups are dealt to the 8 XCDs in turn: the blocks of values of one segment go to the same
    // one, whose L2 then holds the q and k that they share
    const int64_t group = (int64_t)(blockIdx.x / (8 * a.nvb)) * 8 + blockIdx.x % 8;
    const int vb = blockIdx.x / 8 % a.nvb;
    const int walks = KIND == kEnds ? a.nseg - 1 : a.nseg;
    if (group >= a.groups) return;
    const int64_t bh = group / walks;
    const int s = (int)(group % walks);
    const int64_t b = bh / a.H;
    const int h = (int)(bh % a.H);
    const int v0 = vb * kBlock;
    int n = a.L;
    if (a.lengths) n = min(max(a.lengths[b], 0), a.L);
    const int nc = (n + kChunk - 1) / kChunk;
    const int it0 = min(s * a.seg, nc), it1 = min(it0 + a.seg, nc);     // in the walk's order

    const int64_t row0 = b * a.L;
    const T *qb = (const T *)a.q + row0 * a.qp + (int64_t)(h / a.qdiv) * a.kd;
    const T *kb = (const T *)a.k + row0 * a.kp + (int64_t)(h / a.kdiv) * a.kd;
    const T *vbp = (const T *)a.v + row0 * a.vp + (int64_t)(h / a.vdiv) * a.vd + v0;
    const T *xb = KIND == kDq || KIND == kDk
                      ? (const T *)a.x + row0 * a.xp + (int64_t)(h / a.xdiv) * a.vd + v0
                      : nullptr;
    const int vw = min(a.vd - v0, kBlock);

    // the state's accumulators: column the wave's value, rows 16 keys each
    const int val = 16 * wave + c16;
    const bool has_val = val < vw;
    const int64_t size = (int64_t)a.kd * a.vd;
    f32x4 S[KT];
#pragma unroll
    for (int kt = 0; kt < KT; ++kt) {
        S[kt] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        const int key = 16 * kt + 4 * g4;
        if (!has_val || key >= a.kd) continue;
        const int64_t at = (int64_t)(v0 + val) * a.sv + (int64_t)key * a.sk;
        const float *p = KIND == kEnds   ? nullptr
                         : a.nseg > 1    ? a.ends + (bh * a.nseg + s) * size + at
                         : a.init        ? a.init + bh * size + at
                                         : nullptr;
        if (p)
#pragma unroll
            for (int r = 0; r < 4; ++r) S[kt][r] = p[r * a.sk];
    }

    u32x4 kr[KI], vr[VI];
    Key qn[KIND == kEnds ? 1 : KK];
    float gn = 0.0f;
    const auto fetch = [&](int c) {
        const int t0 = c * kChunk, rows = min(kChunk, n - t0);
        const rsrc_t rk = make_rsrc(kb + (int64_t)t0 * a.kp, (int)(((rows - 1) * a.kp + a.kd) * sizeof(T)));
        const rsrc_t rv = make_rsrc(vbp + (int64_t)t0 * a.vp, (int)(((rows - 1) * a.vp + vw) * sizeof(T)));
        const rsrc_t rq = make_rsrc(qb + (int64_t)t0 * a.qp, (int)(((rows - 1) * a.qp + a.kd) * sizeof(T)));
#pragma unroll
        for (int i = 0; i < KI; ++i) {
            const int p = tid + i * kThreads, row = p / (DK / kVec), col = p % (DK / kVec) * kVec;
            kr[i] = buf_load_b128(rk, col < a.kd ? (uint32_t)((row * (int)a.kp + col) * (int)sizeof(T)) : ~0u);
        }
#pragma unroll
        for (int i = 0; i < VI; ++i) {
            const int p = tid + i * kThreads, row = p / (kBlock / kVec), col = p % (kBlock / kVec) * kVec;
            vr[i] = buf_load_b128(rv, col < vw ? (uint32_t)((row * (int)a.vp + col) * (int)sizeof(T)) : ~0u);
        }
        if constexpr (KIND != kEnds) {
#pragma unroll
            for (int kk = 0; kk < KK; ++kk) {
                const int col = Tile<T>::kKeys * kk + Tile<T>::kStepKeys * g4;
                qn[kk] = __builtin_bit_cast(Key, buf_load_b128(rq, col < a.kd
                    ? (uint32_t)(((16 * wave + c16) * (int)a.qp + col) * (int)sizeof(T)) : ~0u));
            }
        }
        gn = 0.0f;
        if (a.decay != 0 && lane < rows)
            gn = a.decay == 1 ? ((const float *)a.g)[h]
                              : (float)((const T *)a.g)[(row0 + t0 + lane) * a.gp + h];
    };
    // rows of the outputs (those behind the sequence and values behind the block dropped)
    const auto store_out = [&](auto *base, int t0, int rows, int i, const f32x4 (&o)[4]) {
        typedef std::remove_pointer_t<decltype(base)> O;
        const int pitch = a.H * a.vd;
        const rsrc_t ro = make_rsrc(base + ((row0 + t0) * a.H + h) * a.vd + v0,
                                    ((rows - 1) * pitch + vw) * (int)sizeof(O));
#pragma unroll
        for (int vt = 0; vt < 4; ++vt) {
            const int v = 16 * vt + 4 * g4;
            buf_store4(ro, v < vw ? (uint32_t)((i * pitch + v) * (int)sizeof(O)) : ~0u, o[vt], (O *)nullptr);
        }
    };
    if (it0 < it1) fetch(REV ? nc - 1 - it0 : it0);

    float passed = 1.0f;      // the decay over the segment
    for (int it = it0; it < it1; ++it) {
        const int c = REV ? nc - 1 - it : it;
        const int t0 = c * kChunk, rows = min(kChunk, n - t0);
        // the chunk into LDS: K, V, the state as the products read it, and the factors
#pragma unroll
        for (int i = 0; i < KI; ++i) {
            const int p = tid + i * kThreads, row = p / (DK / kVec), col = p % (DK / kVec) * kVec;
            *reinterpret_cast<u32x4 *>(sK + row * KP + col) = kr[i];
        }
#pragma unroll
        for (int i = 0; i < VI; ++i) {
            const int p = tid + i * kThreads, row = p / (kBlock / kVec), col = p % (kBlock / kVec) * kVec;
            *reinterpret_cast<u32x4 *>(sV + row * VP + col) = vr[i];
        }
        Key q[KIND == kEnds ? 1 : KK];
        if constexpr (KIND != kEnds) {
#pragma unroll
            for (int kt = 0; kt < KT; ++kt) store4(sS + val * SP + 16 * kt + 4 * g4, S[kt]);
#pragma unroll
            for (int kk = 0; kk < KK; ++kk) q[kk] = qn[kk];
        }
        const float g2 = decay2(gn);
        const float ghi = __builtin_rintf(g2 * 256.0f) * (1.0f / 256.0f);
        const float hi = wave_inclusive_sum(ghi), lo = wave_inclusive_sum(g2 - ghi);
        const float hE = wave_read(hi, 63), lE = wave_read(lo, 63);
        const float from_start = fast_exp2(hi + lo), to_end = fast_exp2((hE - hi) + (lE - lo));
        const float whole = fast_exp2(hE + lE);
        if (KIND == kEnds) passed *= whole;
        if (wave == 0) {
            sHi[lane] = hi;
            sLo[lane] = lo;
            sIn[lane] = (REV ? to_end : from_start) * a.inter;
            sW[lane] = (REV ? from_start : to_end) * a.weight;
        }
        __syncthreads();
        if (it + 1 < it1) fetch(REV ? c - 1 : c + 1);

        if constexpr (KIND != kEnds) {
            // what the state before the chunk gives
            const int i = 16 * wave + c16;                     // this lane's target
            f32x4 o[4] = {};
#pragma unroll
            for (int kk = 0; kk < KK; ++kk)
#pragma unroll
                for (int vt = 0; vt < 4; ++vt) {
                    const Key s = *reinterpret_cast<const Key *>(
                        sS + (16 * vt + c16) * SP + Tile<T>::kKeys * kk + Tile<T>::kStepKeys * g4);
                    o[vt] = mma16(s, q[kk], o[vt]);
                }
            const float in = sIn[i];
#pragma unroll
            for (int vt = 0; vt < 4; ++vt) o[vt] *= in;

            // partner rows of the gradient of the decays
            float part = 0.0f;
            Key xf[KIND == kDq ? BK : 1];
            if constexpr (KIND == kDq || KIND == kDk) {
                const rsrc_t rx = make_rsrc(xb + (int64_t)t0 * a.xp, (int)(((rows - 1) * a.xp + vw) * sizeof(T)));
                if (i < rows) {
                    const T *p = xb + (int64_t)(t0 + i) * a.xp;
#pragma unroll
                    for (int vt = 0; vt < 4; ++vt)
                        if (16 * vt + 4 * g4 < vw) {
                            const f32x4 x = load4(p + 16 * vt + 4 * g4);
#pragma unroll
                            for (int r = 0; r < 4; ++r) part += o[vt][r] * x[r];
                        }
                }
                if constexpr (KIND == kDq)
#pragma unroll
                    for (int kk = 0; kk < BK; ++kk) {
                        const int col = Tile<T>::kKeys * kk + Tile<T>::kStepKeys * g4;
                        xf[kk] = __builtin_bit_cast(Key, buf_load_b128(rx, col < vw
                            ? (uint32_t)((i * (int)a.xp + col) * (int)sizeof(T)) : ~0u));
                    }
            }

            // scores, two tiles of 16 sources at a time, and what the chunk's own tokens give
            const float hi_i = sHi[i], lo_i = sLo[i];
#pragma unroll
            for (int pr = 0; pr < 2; ++pr) {
                if (REV ? 2 * pr + 1 < wave : 2 * pr > wave) {
                    if constexpr (KIND == kDq)
                        if (c16 == 15)
#pragma unroll
                            for (int r = 0; r < 8; ++r) sC[wave][32 * pr + 16 * (r >> 2) + 4 * g4 + (r & 3)] = 0.0f;
                    continue;
                }
                f32x4 p[2];
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int s0 = 32 * pr + 16 * u;
                    p[u] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int kk = 0; kk < KK; ++kk) {
                        const Key k = *reinterpret_cast<const Key *>(
                            sK + (s0 + c16) * KP + Tile<T>::kKeys * kk + Tile<T>::kStepKeys * g4);
                        p[u] = mma16(k, q[kk], p[u]);
                    }
                    const f32x4 hs = load4(sHi + s0 + 4 * g4), ls = load4(sLo + s0 + 4 * g4);
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        // selections before the exponential, which is formed for every pair: no
                        // branches, and nothing not finite from a pair that does not count
                        const int t = s0 + 4 * g4 + r;
                        const bool keep = REV ? t >= i : t <= i;
                        float e = REV ? (hs[r] - hi_i) + (ls[r] - lo_i) : (hi_i - hs[r]) + (lo_i - ls[r]);
                        e = keep ? e : 0.0f;
                        const float x = keep ? p[u][r] : 0.0f;
                        p[u][r] = x * a.intra * fast_exp2(e);
                    }
                    if constexpr (KIND == kDq) {
                        // scores of the other pair: their products' sums by target and by source
                        f32x4 m = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                        for (int kk = 0; kk < BK; ++kk) {
                            const Key v = *reinterpret_cast<const Key *>(
                                sV + (s0 + c16) * VP + Tile<T>::kKeys * kk + Tile<T>::kStepKeys * g4);
                            m = mma16(v, xf[kk], m);
                        }
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            const float prod = p[u][r] != 0.0f ? m[r] * p[u][r] : 0.0f;
                            part += prod;
                            const float col = columns_sum(prod);
                            if (c16 == 15) sC[wave][s0 + 4 * g4 + r] = col;
                        }
                    }
                }
                const Src ps = pack_src<T>(p[0], p[1]);
#pragma unroll
                for (int vt = 0; vt < 4; ++vt)
                    o[vt] = mma16(load_src(sV, VP, 32 * pr, 16 * vt, lane), ps, o[vt]);
            }
            if constexpr (KIND == kDq || KIND == kDk) {
                part = rows_sum(part);
                if (KIND == kDq && g4 == 0) sZ[i] = part;
                if (KIND == kDk && g4 == 0 && i < rows) a.part[(bh * a.nvb + vb) * a.L + t0 + i] = part;
            }
            if (a.o32) store_out((float *)a.o, t0, rows, i, o);
            else store_out((T *)a.o, t0, rows, i, o);

            if constexpr (KIND == kDq || KIND == kDk) {
                // states before the chunk out of the forward walk; their products with the gradients
                // of the states behind it in the backward one
                float x = 0.0f;
                T *sc = (T *)a.states + ((bh * a.nchunks + c) * a.vd + v0 + val) * a.kd;
#pragma unroll
                for (int kt = 0; kt < KT; ++kt) {
                    const int key = 16 * kt + 4 * g4;
                    if (has_val && key < a.kd) {
                        if (KIND == kDq) {
                            store4(sc + key, S[kt]);
                        } else {
                            const f32x4 s = load4(sc + key);
#pragma unroll
                            for (int r = 0; r < 4; ++r) x += s[r] * S[kt][r];
                        }
                    }
                }
                if constexpr (KIND == kDk) {
                    x = rows_sum(columns_sum(x)) * whole;
                    if (lane == 15) sX[wave] = x;
                }
            }
        }

        // the state behind the chunk
#pragma unroll
        for (int kt = 0; kt < KT; ++kt) S[kt] *= whole;
#pragma unroll
        for (int pr = 0; pr < 2; ++pr) {
            const Src v = load_src(sV, VP, 32 * pr, 16 * wave, lane);
            const f32x4 w0 = load4(sW + 32 * pr + 4 * g4), w1 = load4(sW + 32 * pr + 16 + 4 * g4);
            f32x8 w;
#pragma unroll
            for (int e = 0; e < 4; ++e) { w[e] = w0[e]; w[4 + e] = w1[e]; }
            if constexpr (sizeof(T) == 4) {
                const Src wv = v * w;
#pragma unroll
                for (int kt = 0; kt < KT; ++kt)
                    S[kt] = mma16(load_src(sK, KP, 32 * pr, 16 * kt, lane), wv, S[kt]);
            } else {
                bf16x8 wv[3];
                split3(v, w, wv);
                // four tiles side by side: a product's three parts wait for each other
#pragma unroll
                for (int kt = 0; kt < KT; kt += 4) {
                    Src k[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) k[i] = load_src(sK, KP, 32 * pr, 16 * (kt + i), lane);
#pragma unroll
                    for (int e = 0; e < 3; ++e)
#pragma unroll
                        for (int i = 0; i < 4; ++i) S[kt + i] = mma16(k[i], wv[e], S[kt + i]);
                }
            }
        }
        __syncthreads();
        if (KIND == kDq && wave == 0 && lane < rows)
            a.part[(bh * a.nvb + vb) * a.L + t0 + lane] =
                sZ[lane] - (((sC[0][lane] + sC[1][lane]) + sC[2][lane]) + sC[3][lane]);
        if (KIND == kDk && tid == 0)
            a.cross[(bh * a.nvb + vb) * a.nchunks + c] = ((sX[0] + sX[1]) + sX[2]) + sX[3];
    }

    if constexpr (KIND == kEnds) {
        if (tid == 0 && vb == 0) a.decays[bh * a.nseg + s] = passed;
        if (has_val) {
            float *p = a.ends + (bh * a.nseg + s + 1) * size + (int64_t)(v0 + val) * a.sv;
#pragma unroll
            for (int kt = 0; kt < KT; ++kt)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int key = 16 * kt + 4 * g4 + r;
                    if (key < a.kd) p[key * a.sk] = S[kt][r];
                }
        }
    } else if (a.last && has_val && s == a.nseg - 1) {
        float *p = a.last + bh * size + (int64_t)(v0 + val) * a.kd;
#pragma unroll
        for (int kt = 0; kt < KT; ++kt)
            if (16 * kt + 4 * g4 < a.kd)
                store4(p + 16 * kt + 4 * g4, S[kt]);
    }
}

// ---------------------------------------------------------------------------
// Starts of the segments of every head out of their ends, in place: a thread for four elements of a
// head's state, eight segments' ends on their way at a time.
// ---------------------------------------------------------------------------
__global__ __launch_bounds__(kThreads) void chain_kernel(float *ends, const float *__restrict__ decays,
                                                         const float *__restrict__ init, int64_t quads,
                                                         int size4, int nseg)
{
    constexpr int kAhead = 8;
    const int64_t id = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (id >= quads) return;
    const int64_t bh = id / size4;
    f32x4 *p = reinterpret_cast<f32x4 *>(ends) + bh * nseg * size4 + id % size4;
    f32x4 S = init ? reinterpret_cast<const f32x4 *>(init)[id] : f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    for (int s0 = 0; s0 < nseg; s0 += kAhead) {
        f32x4 end[kAhead];
        float d[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int s = min(s0 + i, nseg - 2);
            end[i] = p[(int64_t)(s + 1) * size4];
            d[i] = decays[bh * nseg + s];
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            if (s0 + i >= nseg) break;
            p[(int64_t)(s0 + i) * size4] = S;
            S = S * d[i] + end[i];
        }
    }
}

// ---------------------------------------------------------------------------
// Gradient of the log decays, a wave for a chunk of a head, a lane for a token.  g_t scales all
// that passes token t: read behind it or in it (u: reads of the chunk's start state, and pairs
// within the chunk by their targets less by their sources, `read`), written before it and read
// behind the chunk (`written`), and what passes the whole chunk (`cross`).
// ---------------------------------------------------------------------------
template <typename T>
__global__ __launch_bounds__(kThreads) void decay_gradient_kernel(DecayGradient a)
{
    const int lane = threadIdx.x & 63;
    for (int64_t id = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); id < a.bh * a.nchunks;
         id += (int64_t)gridDim.x * 4) {
        const int64_t bh = id / a.nchunks;
        const int c = (int)(id % a.nchunks);
        const int64_t b = bh / a.H;
        const int h = (int)(bh % a.H);
        int n = a.L;
        if (a.lengths) n = min(max(a.lengths[b], 0), a.L);
        const int t = c * kChunk + lane;
        if (c * kChunk >= n) continue;
        float read = 0.0f, written = 0.0f, cross = 0.0f;
        for (int i = 0; i < a.nvb; ++i) {
            if (t < n) {
                read += a.read[(bh * a.nvb + i) * a.L + t];
                written += a.written[(bh * a.nvb + i) * a.L + t];
            }
            cross += a.cross[(bh * a.nvb + i) * a.nchunks + c];
        }
        const float before = wave_shift_up1(wave_inclusive_sum(written));
        float behind = read;                  // of this lane and those behind it
#pragma unroll
        for (int s = 1; s < 64; s <<= 1) {
            const float up = __shfl_down(behind, s, 64);
            behind += lane + s < 64 ? up : 0.0f;
        }
        if (t >= n) continue;
        const float g = (float)((const T *)a.g)[(b * a.L + t) * a.gp + h];
        float d = behind + before + cross;
        if (g > 0.0f || g * kLog2e < -1000.0f) d = 0.0f;
        ((T *)a.dg)[(b * a.L + t) * a.H + h] = Elem<T>::from_f32(d);
    }
}

// Gradients of shared queries or keys: the sum of their heads', in the heads' order.
template <typename T>
__global__ __launch_bounds__(kThreads) void shared_sum_kernel(const float *__restrict__ per_head,
                                                              T *__restrict__ out,
                                                              const int32_t *__restrict__ lengths,
                                                              int64_t quads, int L, int G, int share, int kd)
{
    const int kq = kd / 4;
    for (int64_t id = (int64_t)blockIdx.x * kThreads + threadIdx.x; id < quads;
         id += (int64_t)gridDim.x * kThreads) {
        const int64_t row = id / kq;              // token and group
        const int64_t token = row / G;
        if (lengths && (int)(token % L) >= lengths[token / L]) continue;
        const float *p = per_head + row * share * kd + id % kq * 4;
        f32x4 s = load4(p);
        for (int i = 1; i < share; ++i) s += load4(p + (int64_t)i * kd);
        store4(out + row * kd + id % kq * 4, s);
    }
}

// Workgroups for `work` items, `each` a workgroup: the last kernels' loops take what is beyond.
unsigned groups_for(int64_t work, int each)
{
    const int64_t n = (work + each - 1) / each;
    return (unsigned)(n < (1 << 20) ? n : (1 << 20));
}

template <typename T, int DK, bool REV, Kind KIND>
hipError_t walk_go(Walk a, int64_t bh, hipStream_t st)
{
    a.groups = bh * (KIND == kEnds ? a.nseg - 1 : a.nseg);
    const int64_t blocks = (a.groups + 7) / 8 * 8 * a.nvb;
    hipLaunchKernelGGL((walk_kernel<T, DK, REV, KIND>), dim3((unsigned)blocks), dim3(kThreads), 0, st, a);
    return hipGetLastError();
}

template <typename T, bool REV, Kind KIND>
hipError_t walk_by_key(const Walk &a, int64_t bh, hipStream_t st)
{
    if (a.kd <= 64) return walk_go<T, 64, REV, KIND>(a, bh, st);
    if (a.kd <= 128) return walk_go<T, 128, REV, KIND>(a, bh, st);
    return walk_go<T, 256, REV, KIND>(a, bh, st);
}

// The ends of a walk's segments, and their starts.
template <typename T, bool REV> hipError_t starts_go(const Walk &a, int64_t bh, hipStream_t st)
{
    const hipError_t e = walk_by_key<T, REV, kEnds>(a, bh, st);
    if (e != hipSuccess) return e;
    const int size4 = a.kd * a.vd / 4;
    const int64_t quads = bh * size4;
    hipLaunchKernelGGL(chain_kernel, dim3((unsigned)((quads + kThreads - 1) / kThreads)), dim3(kThreads), 0,
                       st, a.ends, a.decays, a.init, quads, size4, a.nseg);
    return hipGetLastError();
}

int blocks_of(int64_t values) { return (int)((values + kBlock - 1) / kBlock); }

// How the chunks of a walk are split into segments, whose ends a first walk leaves.
struct Split {
    int seg, nseg;
};
Split split_of(int64_t walks, int chunks)
{
    constexpr int kWant = 512, kLeast = 4;
    const int64_t n = (kWant + walks - 1) / walks;
    int seg = (int)((chunks + n - 1) / n);
    if (seg < kLeast) seg = kLeast;
    return {seg, (chunks + seg - 1) / seg};
}

int chunks_of(const LinattnShape &s) { return (int)((s.L + kChunk - 1) / kChunk); }

// Workspace of one split: ends and decays (byte offsets).
int64_t ends_bytes(const LinattnShape &s, int nseg)
{
    return nseg > 1 ? s.b * s.H * nseg * s.dk * s.dv * 4 : 0;
}
int64_t decays_bytes(const LinattnShape &s, int nseg)
{
    return nseg > 1 ? (s.b * s.H * nseg * 4 + 255) / 256 * 256 : 0;
}
Split forward_split(const LinattnShape &s)
{
    return split_of(s.b * s.H * blocks_of(s.dv), chunks_of(s));
}

Split grad_split(const LinattnShape &s)
{
    const int64_t least = blocks_of(s.dk) < blocks_of(s.dv) ? blocks_of(s.dk) : blocks_of(s.dv);
    return split_of(s.b * s.H * least, chunks_of(s));
}

// Workspace of the gradients (byte offsets, on 256 bytes): with a decays' gradient the states
// before each chunk and the parts that its kernel adds up; with shared heads every head's dq and dk.
struct GradLayout {
    int64_t states, read, written, cross, dq, dk, ends, decays, back_ends, back_decays, bytes;
    Split split;
};
GradLayout grad_layout(const LinattnShape &s, bool gates)
{
    GradLayout y;
    int64_t at = 0;
    const auto take = [&](bool wanted, int64_t bytes) {
        const int64_t off = at;
        if (wanted) at += (bytes + 255) / 256 * 256;
        return off;
    };
    const int64_t bh = s.b * s.H, nvb = blocks_of(s.dk), nc = chunks_of(s);
    y.states = take(gates, bh * nc * s.dk * s.dv * (s.bf16 ? 2 : 4));
    y.read = take(gates, bh * nvb * s.L * 4);
    y.written = take(gates, bh * nvb * s.L * 4);
    y.cross = take(gates, bh * nvb * nc * 4);
    const int64_t heads = s.b * s.L * s.H * s.dk * 4;
    y.dq = take(s.H > s.G, heads);
    y.dk = take(s.H > s.G, heads);
    y.split = grad_split(s);
    const int nseg = y.split.nseg;
    y.ends = take(nseg > 1, ends_bytes(s, nseg));
    y.decays = take(nseg > 1, decays_bytes(s, nseg));
    y.back_ends = take(nseg > 1, ends_bytes(s, nseg));
    y.back_decays = take(nseg > 1, decays_bytes(s, nseg));
    y.bytes = at;
    return y;
}

template <typename T> hipError_t forward_go(const LinattnShape &s, const LinattnArgs &a, hipStream_t st)
{
    Walk w = {};
    w.q = a.q; w.k = a.k; w.v = a.v;
    w.qp = s.qp; w.kp = s.kp; w.vp = s.vp;
    w.qdiv = w.kdiv = (int)(s.H / s.G); w.vdiv = 1;
    w.g = a.g; w.gp = s.gp; w.decay = s.decay; w.lengths = a.lengths;
    w.o = a.o; w.init = a.h0; w.last = a.hT;
    w.sv = s.dk; w.sk = 1;
    w.weight = 1.0f;
    w.inter = w.intra = s.scale;
    w.L = (int)s.L; w.H = (int)s.H; w.kd = (int)s.dk; w.vd = (int)s.dv;
    w.nvb = blocks_of(s.dv);
    const Split y = forward_split(s);
    w.seg = y.seg; w.nseg = y.nseg;
    w.ends = (float *)a.ws;
    w.decays = (float *)((char *)a.ws + ends_bytes(s, y.nseg));
    if (y.nseg > 1) {
        const hipError_t e = starts_go<T, false>(w, s.b * s.H, st);
        if (e != hipSuccess) return e;
    }
    return walk_by_key<T, false, kOut>(w, s.b * s.H, st);
}

// Gradients: three walks (q's forward in time, then k's and v's back), the decays' from the parts
// that the first two leave, shared heads' sums.
template <typename T>
hipError_t backward_go(const LinattnShape &s, const LinattnGradArgs &a, hipStream_t st)
{
    const GradLayout y = grad_layout(s, a.dg != nullptr);
    char *ws = (char *)a.ws;
    const auto at = [&](int64_t off) { return ws ? ws + off : nullptr; };
    const int share = (int)(s.H / s.G);
    const int64_t bh = s.b * s.H;
    const bool gates = a.dg != nullptr;
    hipError_t e;

    Walk w = {};
    w.g = a.g; w.gp = s.gp; w.decay = s.decay; w.lengths = a.lengths;
    w.L = (int)s.L; w.H = (int)s.H;
    w.nchunks = chunks_of(s);
    w.states = at(y.states);
    w.cross = (float *)at(y.cross);

    w.seg = y.split.seg; w.nseg = y.split.nseg;
    Walk back = w;       // states' gradients, back in time
    w.ends = (float *)at(y.ends); w.decays = (float *)at(y.decays);
    back.ends = (float *)at(y.back_ends); back.decays = (float *)at(y.back_decays);
    if (w.nseg > 1) {
        Walk f = w, r = back;
        f.k = a.k; f.kp = s.kp; f.kdiv = share;
        f.v = a.v; f.vp = s.vp; f.vdiv = 1;
        f.init = a.h0; f.weight = 1.0f;
        r.k = a.q; r.kp = s.qp; r.kdiv = share;
        r.v = a.dout; r.vp = s.dop; r.vdiv = 1;
        r.init = a.dhT; r.weight = s.scale;
        for (Walk *x : {&f, &r}) {
            x->qdiv = 1;
            x->sv = s.dk; x->sk = 1;
            x->kd = (int)s.dk; x->vd = (int)s.dv; x->nvb = blocks_of(s.dv);
        }
        e = starts_go<T, false>(f, bh, st);
        if (e == hipSuccess) e = starts_go<T, true>(r, bh, st);
        if (e != hipSuccess) return e;
    }

    Walk q = w;          // dq = scale S^T do
    q.q = a.dout; q.qp = s.dop; q.qdiv = 1;
    q.k = a.v; q.kp = s.vp; q.kdiv = 1;
    q.v = a.k; q.vp = s.kp; q.vdiv = share;
    q.o = share > 1 ? at(y.dq) : a.dq; q.o32 = share > 1;
    q.init = a.h0; q.sv = 1; q.sk = s.dk;
    q.inter = q.intra = s.scale; q.weight = 1.0f;
    q.kd = (int)s.dv; q.vd = (int)s.dk; q.nvb = blocks_of(s.dk);
    q.x = a.q; q.xp = s.qp; q.xdiv = share;
    q.part = (float *)at(y.read);
    e = gates ? walk_by_key<T, false, kDq>(q, bh, st) : walk_by_key<T, false, kOut>(q, bh, st);
    if (e != hipSuccess) return e;

    Walk k = back;       // dk = dS^T v, scale in dS
    k.q = a.v; k.qp = s.vp; k.qdiv = 1;
    k.k = a.dout; k.kp = s.dop; k.kdiv = 1;
    k.v = a.q; k.vp = s.qp; k.vdiv = share;
    k.o = share > 1 ? at(y.dk) : a.dk; k.o32 = share > 1;
    k.init = a.dhT; k.sv = 1; k.sk = s.dk;
    k.inter = 1.0f; k.intra = k.weight = s.scale;
    k.kd = (int)s.dv; k.vd = (int)s.dk; k.nvb = blocks_of(s.dk);
    k.x = a.k; k.xp = s.kp; k.xdiv = share;
    k.part = (float *)at(y.written);
    e = gates ? walk_by_key<T, true, kDk>(k, bh, st) : walk_by_key<T, true, kOut>(k, bh, st);
    if (e != hipSuccess) return e;

    Walk v = back;       // dv = dS k
    v.q = a.k; v.qp = s.kp; v.qdiv = share;
    v.k = a.q; v.kp = s.qp; v.kdiv = share;
    v.v = a.dout; v.vp = s.dop; v.vdiv = 1;
    v.o = a.dv;
    v.init = a.dhT; v.sv = s.dk; v.sk = 1;
    v.last = a.dh0;
    v.inter = 1.0f; v.intra = v.weight = s.scale;
    v.kd = (int)s.dk; v.vd = (int)s.dv; v.nvb = blocks_of(s.dv);
    e = walk_by_key<T, true, kOut>(v, bh, st);
    if (e != hipSuccess) return e;

    if (gates) {
        DecayGradient d = {};
        d.g = a.g; d.gp = s.gp; d.lengths = a.lengths;
        d.read = q.part; d.written = k.part; d.cross = w.cross;
        d.dg = a.dg;
        d.bh = bh; d.L = (int)s.L; d.H = (int)s.H; d.nvb = q.nvb; d.nchunks = w.nchunks;
        hipLaunchKernelGGL((decay_gradient_kernel<T>), dim3(groups_for(bh * w.nchunks, 4)), dim3(kThreads),
                           0, st, d);
        e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (share > 1) {
        const int64_t quads = s.b * s.L * s.G * (s.dk / 4);
        for (int i = 0; i < 2; ++i) {
            hipLaunchKernelGGL((shared_sum_kernel<T>), dim3(groups_for(quads, kThreads)), dim3(kThreads),
                               0, st, (const float *)at(i ? y.dk : y.dq), (T *)(i ? a.dk : a.dq), a.lengths, quads, (int)s.L, (int)s.G, share, (int)s.dk);
            e = hipGetLastError();
            if (e != hipSuccess) return e;
        }
    }
    return hipSuccess;
}

}  // namespace

hipError_t launch_linattn(const LinattnShape &s, const LinattnArgs &a, hipStream_t st)
{
    return s.bf16 ? forward_go<bf16>(s, a, st) : forward_go<float>(s, a, st);
}

size_t linattn_workspace_bytes(const LinattnShape &s)
{
    const int n = forward_split(s).nseg;
    return n > 1 ? (size_t)(ends_bytes(s, n) + decays_bytes(s, n)) : SSD_LINATTN_NO_WORKSPACE;
}

size_t linattn_backward_workspace_bytes(const LinattnShape &s)
{
    const int64_t n = grad_layout(s, s.decay == SSD_DECAY_TOKEN).bytes;
    return n ? (size_t)n : SSD_LINATTN_NO_WORKSPACE;
}

hipError_t launch_linattn_backward(const LinattnShape &s, const LinattnGradArgs &a, hipStream_t st)
{
    return s.bf16 ? backward_go<bf16>(s, a, st) : backward_go<float>(s, a, st);
}

}  // namespace ssd
