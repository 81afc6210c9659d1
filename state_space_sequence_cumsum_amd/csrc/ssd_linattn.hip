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
// they are, the decayed scores and the state that a chunk reads each rounded once (twice the half
// step of an output's own rounding at most; two parts of each with a gradient of the decays); but
// what is added to the state, w_s v_s, goes in as three bf16 parts (8 + 8 + 8 bits, fp32's 24)
// where the state leaves the kernel in fp32 or starts a segment, and as two where it only makes the
// outputs of its own segment, an error of 2^-17.
//
// Segments.  A walk is serial, 4 us a chunk of 64 tokens, and a chip full of walks takes 512
// workgroups.  Where heads and blocks of values give fewer, a first walk without outputs leaves the
// ends of segments of the prompt, from zero, a chain turns them into starts, and the outputs' walk
// takes all segments at once: 16384 tokens of 16 heads of 128 x 128 take 125 us in 512 workgroups
// (ends 38, chain 16, outputs 66; the 271 MB of inputs and outputs at a copy's rate would take 44, the
// 17 GFLOP of a token's 4 x 128 x 128 at a large product's 15), and 1 ms in 16 walks of 256 chunks each.
//
// What bounds it: a chunk is a chain of short phases between two barriers (rows to LDS, scores,
// state read, state update, outputs), 9000 to 12000 cycles with two workgroups a CU, of which the
// matrix instructions take a fifth, and HBM is busy less than half of the time (2.7 TB/s in the
// outputs' walk); asking for the next chunk's rows is the longest (its loads wait for room), then
// the state update.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "../../include/ssd.h"
#include "ssd_device.h"
#include "ssd_launch.h"

namespace ssd {
namespace {

// Tokens of a chunk: 64, or 32 of the widest fp32 heads, whose rows would not fit into LDS and
// registers otherwise.
template <typename T, int DK> constexpr int chunk_tokens() { return DK * sizeof(T) <= 512 ? 64 : 32; }
int chunk_tokens(bool bf16, int64_t keys) { return bf16 || keys <= 128 ? 64 : 32; }
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
    float *last;                // [b, H, vd, kd], of a walk of one segment; may be NULL
    // Segments: `seg` tokens each (a multiple of 64), nseg of them, in the walk's order.  With more than one, kEnds
    // leaves their ends (from zero) and decays, a chain over those their starts, for the others.
    int seg, nseg;
    float *ends;                // [b H, nseg, vd kd], in init's layout: ends, then starts
    float *decays;              // [b H, nseg]: over segment s
    float inter, intra;         // factors of an output's two parts
    float weight;               // factor of what is added to the state
    int L, H, kd, vd, nvb;
    int64_t groups;             // heads x segments
    // kDq, kDk: the array whose products with the outputs the decays' gradient takes (q, k): those
    // (kDk: of what the chunk's own tokens give, and of what the state behind it gives), and the states
    // before each chunk, [b H, chunks, nvb] of them as a workgroup's lanes hold them (both walks have
    // the same roles of values and keys): whole 16-byte accesses, lane beside lane, with their
    // products with the gradients behind it
    const void *x;
    int64_t xp;
    int xdiv;
    float *part, *written;      // [b H, nvb, L]
    void *states;
    float *cross;               // [b H, nvb, chunks]
    int nchunks;
};

struct DecayGradient {
    const void *g;
    int64_t gp;
    const int32_t *lengths;
    const float *read, *own, *written, *cross;
    void *dg;
    int64_t bh;
    int L, H, nvb, nchunks, chunk;
};

// ---------------------------------------------------------------------------
// Tiles of 16 x 16.  An accumulator's lane l holds column l % 16, rows 4 (l / 16) + r.  An operand's
// fragment holds 16 bytes of one row (A) or column (B), l % 16, along the contracted index: a step
// of it, 32 for bf16 (one instruction) or 16 for fp32 (one for each of the four).  There are two
// orders, the same for both operands of a product:
//   straight  bf16 8 (l / 16) + e, fp32 4 (l / 16) + e: what a 16-byte read of a row gives
//   paired    bf16 4 (l / 16) + e and 16 + 4 (l / 16) + e, fp32 as straight: what two accumulators
//             (fp32: one), one behind the other along the rows, hold as they stand
// ---------------------------------------------------------------------------
template <typename T> struct Tile;
template <> struct Tile<bf16> {
    typedef bf16x8 frag;
    static constexpr int kStep = 32, kPart = 8;
    static constexpr int row_pitch(int n) { return n + 8; }
};
template <> struct Tile<float> {
    typedef f32x4 frag;
    static constexpr int kStep = 16, kPart = 4;
    static constexpr int row_pitch(int n) { return n + 4; }
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

// ---------------------------------------------------------------------------
// Rows of queries and keys in LDS, N elements each.  For bf16 a row's pieces of 16 bytes change
// places by the row (exclusive or with bits of it): the 16 rows of a fragment's straight read, the
// 8 rows of half a transpose read (two pieces of each) and the rows of a paired read then all lie
// in different banks, which no padding gives (at 288 bytes a row straight reads of 16 rows
// conflicted, at 272 transpose reads of 8).  fp32 rows are padded by 16 bytes.
// ---------------------------------------------------------------------------
// A lane's place is one offset; what a fragment's step and tile add to it is a constant, `on` (an
// exclusive or of bits that the lane's own columns leave free, or a sum).
template <typename T, int N> struct Rows;
template <int N> struct Rows<bf16, N> {
    // 16 rows and 16 bytes: halves of two tiles' fragments that lie a multiple of 512 bytes apart
    // would be read by one instruction, and then moved (57 moves a chunk of 128 values)
    static constexpr int kTile = 16 * N + 8;
    // elements from the start of the rows to row r's piece of column c (a multiple of 8)
    static __device__ __forceinline__ int at(int r, int c)
    {
        const int turn = N == 64 ? (r >> 1 & 3) << 1 | (r >> 3 & 1) : (r & 7) << 1 | (r >> 3 & 1);
        return r * N + (r >> 4) * 8 + ((c >> 3) ^ turn) * 8;
    }
    static __device__ __forceinline__ int on(int off, int columns) { return off ^ columns; }
    // places of a lane in row l % 16 of straight and paired fragments, and down 16 columns
    static __device__ __forceinline__ int straight(int lane) { return at(lane & 15, 8 * (lane >> 4)); }
    static __device__ __forceinline__ int paired(int lane)
    {
        return at(lane & 15, 8 * (lane >> 5)) + 4 * (lane >> 4 & 1);
    }
    static __device__ __forceinline__ int down(int lane)
    {
        return at(4 * (lane >> 4) + ((lane & 15) >> 2), 8 * (lane >> 1 & 1)) + 4 * (lane & 1);
    }
};
template <int N> struct Rows<float, N> {
    static constexpr int kPitch = N + 4, kTile = 16 * kPitch;
    static __device__ __forceinline__ int at(int r, int c) { return r * kPitch + c; }
    static __device__ __forceinline__ int on(int off, int columns) { return off + columns; }
    static __device__ __forceinline__ int straight(int lane) { return at(lane & 15, 4 * (lane >> 4)); }
    static __device__ __forceinline__ int paired(int lane) { return straight(lane); }
    static __device__ __forceinline__ int down(int lane) { return at(4 * (lane >> 4), lane & 15); }
};

// A straight or paired fragment of step m of row 16 i + l % 16.
template <int N, typename T>
__device__ __forceinline__ typename Tile<T>::frag load_straight(const T *s, int place, int i, int m)
{
    typedef Rows<T, N> R;
    return *reinterpret_cast<const typename Tile<T>::frag *>(s + i * R::kTile +
                                                             R::on(place, Tile<T>::kStep * m));
}
template <int N> __device__ __forceinline__ bf16x8 load_paired(const bf16 *s, int place, int i, int m)
{
    const bf16 *p = s + i * Rows<bf16, N>::kTile;
    return cat8(*reinterpret_cast<const bf16x4 *>(p + (place ^ 32 * m)),
                *reinterpret_cast<const bf16x4 *>(p + (place ^ (32 * m + 16))));
}
template <int N> __device__ __forceinline__ f32x4 load_paired(const float *s, int place, int i, int m)
{
    return load_straight<N>(s, place, i, m);
}
// A paired fragment of step m of rows, down columns 16 j + l % 16.
template <int N> __device__ __forceinline__ bf16x8 load_down(const bf16 *s, int place, int m, int j)
{
    constexpr int tile = Rows<bf16, N>::kTile;
    const bf16 *p = s + 2 * m * tile + (place ^ 16 * j);
    return cat8(tr_read4(p), tr_read4(p + tile));
}
template <int N> __device__ __forceinline__ f32x4 load_down(const float *s, int place, int m, int j)
{
    constexpr int pitch = Rows<float, N>::kPitch;
    const float *p = s + 16 * m * pitch + place + 16 * j;
    return f32x4{p[0], p[pitch], p[2 * pitch], p[3 * pitch]};
}
// A paired fragment of step m out of accumulators.
template <typename T, int N>
__device__ __forceinline__ typename Tile<T>::frag of_accumulators(const f32x4 (&acc)[N], int m)
{
    if constexpr (sizeof(T) == 4) {
        return acc[m];
    } else {
        u32x4 r;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            r[2 * i] = pack_bf16(acc[2 * m + i][0], acc[2 * m + i][1]);
            r[2 * i + 1] = pack_bf16(acc[2 * m + i][2], acc[2 * m + i][3]);
        }
        return __builtin_bit_cast(bf16x8, r);
    }
}
// What bf16 leaves of those accumulators, as an operand.
template <int N> __device__ __forceinline__ bf16x8 rest_of_accumulators(const f32x4 (&acc)[N], int m, const bf16x8 &part)
{
    const u32x4 w = __builtin_bit_cast(u32x4, part);
    u32x4 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const f32x4 &x = acc[2 * m + (i >> 1)];
        r[i] = pack_bf16(x[2 * (i & 1)] - bf_lo(w[i]), x[2 * (i & 1) + 1] - bf_hi(w[i]));
    }
    return __builtin_bit_cast(bf16x8, r);
}
// Where source `s` of a target's scores is kept, for a paired read of 16 bytes.
template <typename T> __device__ __forceinline__ int paired_place(int tile, int g4)
{
    if constexpr (sizeof(T) == 4) return 16 * tile + 4 * g4;
    else return 32 * (tile >> 1) + 8 * g4 + 4 * (tile & 1);
}

// The products w x of a fragment and its tokens' weights as operands: three bf16 parts hold a
// product's 24 bits (two 16 of them), fp32 is one.
template <int PARTS>
__device__ __forceinline__ void weigh(const bf16x8 &x, const float *w, int m, int g4, bf16x8 (&p)[PARTS])
{
    const f32x4 w0 = *reinterpret_cast<const f32x4 *>(w + 32 * m + 4 * g4);
    const f32x4 w1 = *reinterpret_cast<const f32x4 *>(w + 32 * m + 16 + 4 * g4);
    f32x8 v;
#pragma unroll
    for (int e = 0; e < 4; ++e) { v[e] = (float)x[e] * w0[e]; v[4 + e] = (float)x[4 + e] * w1[e]; }
#pragma unroll
    for (int i = 0; i < PARTS; ++i) {
        u32x4 r;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            r[e] = pack_bf16(v[2 * e], v[2 * e + 1]);
            v[2 * e] -= bf_lo(r[e]);
            v[2 * e + 1] -= bf_hi(r[e]);
        }
        p[i] = __builtin_bit_cast(bf16x8, r);
    }
}
template <int PARTS>
__device__ __forceinline__ void weigh(const f32x4 &x, const float *w, int m, int g4, f32x4 (&p)[PARTS])
{
    p[0] = x * *reinterpret_cast<const f32x4 *>(w + 16 * m + 4 * g4);
}

// Four elements as T, in LDS or memory.
__device__ __forceinline__ void store4(bf16 *p, const f32x4 &v)
{
    u32x2 r;
    r[0] = pack_bf16(v[0], v[1]);
    r[1] = pack_bf16(v[2], v[3]);
    *reinterpret_cast<u32x2 *>(p) = r;
}
__device__ __forceinline__ void store4(float *p, const f32x4 &v) { *reinterpret_cast<f32x4 *>(p) = v; }
__device__ __forceinline__ f32x4 load4(const float *p) { return *reinterpret_cast<const f32x4 *>(p); }

// The same through a buffer: past its end nothing is written, and zeros are read.
typedef unsigned int u2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ void buf_store4(rsrc_t r, uint32_t off, const f32x4 &v, bf16 *)
{
    u2 w;
    w[0] = pack_bf16(v[0], v[1]);
    w[1] = pack_bf16(v[2], v[3]);
    __builtin_amdgcn_raw_buffer_store_b64(w, r, (int)off, 0, 0);
}
__device__ __forceinline__ void buf_store4(rsrc_t r, uint32_t off, const f32x4 &v, float *)
{
    buf_store_b128(r, off, __builtin_bit_cast(u32x4, v));
}
// One element as it comes, and as fp32; four.
__device__ __forceinline__ uint32_t buf_load1(rsrc_t r, uint32_t off, bf16 *)
{
    return (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(r, (int)off, 0, 0);
}
__device__ __forceinline__ uint32_t buf_load1(rsrc_t r, uint32_t off, float *) { return buf_load_b32(r, off); }
template <typename T> __device__ __forceinline__ float as_float(uint32_t v)
{
    return __uint_as_float(sizeof(T) == 2 ? v << 16 : v);
}
template <typename T> struct Raw4;
template <> struct Raw4<bf16> { typedef u2 t; };
template <> struct Raw4<float> { typedef u32x4 t; };
__device__ __forceinline__ u2 buf_load4(rsrc_t r, uint32_t off, bf16 *)
{
    return __builtin_amdgcn_raw_buffer_load_b64(r, (int)off, 0, 0);
}
__device__ __forceinline__ u32x4 buf_load4(rsrc_t r, uint32_t off, float *) { return buf_load_b128(r, off); }
__device__ __forceinline__ f32x4 as_floats(const u2 &v)
{
    return f32x4{bf_lo(v[0]), bf_hi(v[0]), bf_lo(v[1]), bf_hi(v[1])};
}
__device__ __forceinline__ f32x4 as_floats(const u32x4 &v) { return __builtin_bit_cast(f32x4, v); }
__device__ __forceinline__ float dot4(const f32x4 &a, const f32x4 &b)
{
    return fmaf(a[3], b[3], fmaf(a[2], b[2], fmaf(a[1], b[1], a[0] * b[0])));
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
// A walk: one (batch, head) and a block of 64 NV of its values, chunk by chunk.  Each of the four
// waves has 16 NV values: their state [key, value], whose accumulators are an operand as they stand,
// and their outputs [value, target].  A chunk's products, a wave's share:
//   scores [source, target]   of the ten 16 x 16 tiles on this side of the diagonal, two or three;
//                             decayed and rounded, they go to the other waves through LDS
//   o = S q                   keys contracted, all targets
//   S += K^T (w V)            tokens contracted, K and V read transposed
//   o += V^T scores           tokens contracted, behind the second of the two barriers of a chunk
// The next chunk's rows are on their way meanwhile, in registers.
// ---------------------------------------------------------------------------
// Waves of a SIMD that the registers leave room for: those of the workgroups that LDS holds.
template <typename T, int DK, int NV> constexpr int waves_for()
{
    if (sizeof(T) == 2) return DK > 128 ? 1 : DK == 128 || NV == 2 ? 2 : 3;
    return DK == 128 ? 1 : 2;
}

// PARTS: bf16 parts of what is added to the state, 3, or 2 where the state only makes outputs.  With
// 3, 128 keys and 128 values one or two registers a lane are in scratch (none with 2); bf16 keys past 128
// take more than 256 registers, accumulator registers among them, but for walks of 64 values
// without a part in the decays' gradient.
template <typename T, int DK, int NV, bool REV, Kind KIND, int PARTS>
__global__ __launch_bounds__(kThreads, (waves_for<T, DK, NV>())) void walk_kernel(Walk a)
{
    typedef typename Tile<T>::frag Frag;
    typedef typename Raw4<T>::t Raw;
    constexpr bool kOuts = KIND != kEnds, kParts = KIND == kDq || KIND == kDk;
    // Scores and the state that is read in two bf16 parts: the decays' gradient adds up their
    // products with both sides' rows, and with one part its error, 2.6e-3 of its size, was half as
    // large again as that of its own rounding (1.7e-3; now 2.0e-3 to 2.5e-3, what is left being the
    // states between the two walks, in one part).  dq and dk err by their own rounding alone, 1.7e-3;
    // by 2.4e-3, with other bits, where no decays' gradient is wanted.  2 % of the gradients' time.
    constexpr bool kFine = kParts && sizeof(T) == 2;
    constexpr int CH = chunk_tokens<T, DK>(), NI = CH / 16, kTiles = NI * (NI + 1) / 2;
    constexpr int BV = 64 * NV;                                      // values
    typedef Rows<T, DK> KeyRows;
    typedef Rows<T, BV> ValRows;
    constexpr int PP = Tile<T>::row_pitch(CH);                       // a target's scores
    constexpr int KK = DK / Tile<T>::kStep, KT = DK / 16, MM = CH / Tile<T>::kStep;
    constexpr int kVec = 16 / (int)sizeof(T);                        // elements of 16 bytes
    constexpr int KI = CH * DK / kVec / kThreads;                // 16-byte pieces a thread
    constexpr int VI = CH * BV / kVec / kThreads;
    constexpr int QI = kOuts ? KI : 1, kSide = 2;
    constexpr int KR = kThreads / (DK / kVec), VR = kThreads / (BV / kVec);  // rows of a round of pieces
    static_assert(KI * KR == CH && VI * VR == CH, "pieces of whole rows");
    __shared__ __attribute__((aligned(16))) T sK[NI * KeyRows::kTile];
    __shared__ __attribute__((aligned(16))) T sV[NI * ValRows::kTile];
    __shared__ __attribute__((aligned(16))) T sQ[NI * KeyRows::kTile];
    __shared__ __attribute__((aligned(16))) T sP[kFine ? 2 * CH * PP : CH * PP];
    __shared__ __attribute__((aligned(16))) float sHi[CH], sLo[CH], sIn[CH], sW[CH];
    __shared__ float sPart[4][CH], sWritten[4][CH], sX[4];

    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int c16 = lane & 15, g4 = lane >> 4;
    // workgroups are dealt to the 8 XCDs in turn: the blocks of values of one segment go to the same
    // one, whose L2 then holds the q and k that they share
    const int64_t group = (int64_t)(blockIdx.x / (8 * a.nvb)) * 8 + blockIdx.x % 8;
    const int vb = blockIdx.x / 8 % a.nvb;
    if (group >= a.groups) return;
    const int64_t bh = group / a.nseg;
    const int s = (int)(group % a.nseg);
    const int64_t b = bh / a.H;
    const int h = (int)(bh % a.H);
    const int v0 = vb * BV;
    int n = a.L;
    if (a.lengths) n = min(max(a.lengths[b], 0), a.L);
    // segment s in the walk's order: the s-th, or back in time the s-th from the sequence's end
    const int nc = (n + CH - 1) / CH, seg = a.seg / CH;
    const int at = REV ? (nc + seg - 1) / seg - 1 - s : s;
    const int c0 = at < 0 ? 0 : min(at * seg, nc), count = at < 0 ? 0 : min(seg, nc - c0);

    const int64_t row0 = b * a.L;
    const T *qb = (const T *)a.q + row0 * a.qp + (int64_t)(h / a.qdiv) * a.kd;
    const T *kb = (const T *)a.k + row0 * a.kp + (int64_t)(h / a.kdiv) * a.kd;
    const T *vbp = (const T *)a.v + row0 * a.vp + (int64_t)(h / a.vdiv) * a.vd + v0;
    const T *xb = kParts ? (const T *)a.x + row0 * a.xp + (int64_t)(h / a.xdiv) * a.vd + v0 : nullptr;
    const int vw = min(a.vd - v0, BV);

    // the state's accumulators: column a value, rows 16 keys each
    const int val0 = 16 * NV * wave + c16, val4 = 16 * NV * wave + 4 * g4;   // and a target's four
    const int64_t size = (int64_t)a.kd * a.vd;
    f32x4 S[NV][KT];
    const float *start = KIND == kEnds ? nullptr
                         : a.nseg > 1  ? a.ends + (bh * a.nseg + s) * size
                         : a.init      ? a.init + bh * size
                                       : nullptr;
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int kt = 0; kt < KT; ++kt) {
            S[v][kt] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
            const int key = 16 * kt + 4 * g4, val = val0 + 16 * v;
            if (start && val < vw && key < a.kd)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    S[v][kt][r] = start[(int64_t)(v0 + val) * a.sv + (int64_t)(key + r) * a.sk];
        }

    // Rows of the chunk ahead: a thread's pieces lie KR (VR) rows apart.  Offsets are bytes from the
    // chunk's first row, below 2^30; kNowhere and what is added to it lies past every buffer's end.
    constexpr uint32_t kNowhere = 1u << 31;
    u32x4 kr[KI], vr[VI], qr[QI];
    uint32_t gn = 0;
    const float ghead = a.decay == SSD_DECAY_HEAD ? ((const float *)a.g)[h] : 0.0f;
    const int krow = tid / (DK / kVec), kcol = tid % (DK / kVec) * kVec;
    const int vrow = tid / (BV / kVec), vcol = tid % (BV / kVec) * kVec;
    const auto rows_at = [&](const T *base, int64_t pitch, int t, int rows, int width) {
        return make_rsrc(base + t * pitch, ((rows - 1) * (int)pitch + width) * (int)sizeof(T));
    };
    const auto bytes = [](int row, int64_t pitch, int col) {
        return (uint32_t)((row * (int)pitch + col) * (int)sizeof(T));
    };
    uint32_t koff = kcol < a.kd ? bytes(krow, a.kp, kcol) : kNowhere;
    uint32_t qoff = kcol < a.kd ? bytes(krow, a.qp, kcol) : kNowhere;
    uint32_t voff = vcol < vw ? bytes(vrow, a.vp, vcol) : kNowhere;
    const uint32_t goff = bytes(lane, a.gp, h);
    // A chunk's rows are asked for in three goes between products: a load waits for room among those
    // on their way, and one after the other the twelve of a chunk held their wave up for 4000
    // to 5500 cycles with the chip full.
    const auto fetch_k = [&](int c) {
        const int t0 = c * CH;
        const rsrc_t rk = rows_at(kb, a.kp, t0, min(CH, n - t0), a.kd);
        asm volatile("" : "+v"(koff), "+v"(voff), "+v"(qoff));      // (as the places in LDS below)
#pragma unroll
        for (int i = 0; i < KI; ++i) kr[i] = buf_load_b128(rk, koff + bytes(i * KR, a.kp, 0));
    };
    const auto fetch_v = [&](int c) {
        const int t0 = c * CH;
        const rsrc_t rv = rows_at(vbp, a.vp, t0, min(CH, n - t0), vw);
        asm volatile("" : "+v"(koff), "+v"(voff), "+v"(qoff));
#pragma unroll
        for (int i = 0; i < VI; ++i) vr[i] = buf_load_b128(rv, voff + bytes(i * VR, a.vp, 0));
    };
    const auto fetch_q = [&](int c) {
        const int t0 = c * CH, rows = min(CH, n - t0);
        asm volatile("" : "+v"(koff), "+v"(voff), "+v"(qoff));
        if constexpr (kOuts) {
            const rsrc_t rq = rows_at(qb, a.qp, t0, rows, a.kd);
#pragma unroll
            for (int i = 0; i < KI; ++i) qr[i] = buf_load_b128(rq, qoff + bytes(i * KR, a.qp, 0));
        }
        // as it comes: a conversion here would wait for all of these loads
        if (a.decay == SSD_DECAY_TOKEN)
            gn = buf_load1(rows_at((const T *)a.g + row0 * a.gp, a.gp, t0, rows, a.H), goff, (T *)nullptr);
    };
    // The decays' gradient: a chunk's parts of the waves, added up by the first one.  What the waves put
    // down between the chunk's two barriers is gathered behind the second one, into the first
    // wave's own place, as they put down the next chunk's behind the next barrier; what they put
    // down behind the second one is added up, and all of it stored, behind the next barrier.
    const auto gather_parts = [&] {
        if (wave != 0 || lane >= CH) return;
        float written = 0.0f, cross = 0.0f;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            written += sWritten[w][lane];
            cross += sX[w];
        }
        sWritten[0][lane] = written;
        if (lane == 0) sX[0] = cross;
    };
    const auto store_parts = [&](int c) {
        const int t = c * CH + lane;
        if (wave != 0 || lane >= CH || t >= n) return;
        const int64_t at = (bh * a.nvb + vb) * a.L + t;
        float part = 0.0f;
#pragma unroll
        for (int w = 0; w < 4; ++w) part += sPart[w][lane];
        if constexpr (KIND == kDq) {
            a.part[at] = part;
        } else {
            const float written = sWritten[0][lane];
            a.part[at] = part - written;
            a.written[at] = written;
            if (lane == 0) a.cross[(bh * a.nvb + vb) * a.nchunks + c] = sX[0];
        }
    };

    if constexpr (kOuts)      // scores across the diagonal stay zero
        for (int i = tid; i < (int)(sizeof(sP) / sizeof(T)); i += kThreads) sP[i] = (T)0.0f;
    if (count > 0) {
        const int first = REV ? c0 + count - 1 : c0;
        fetch_k(first);
        fetch_v(first);
        fetch_q(first);
    }

    // Of two workgroups on a compute unit (256 apart) one goes first: in step they would both be in
    // products, or both in what lies between (out: 77 us against 81 with 16384 tokens of 16 heads
    // of 128 x 128; the ends' walk gains from priority for the products instead, 48 against 51)
    if (kOuts && (blockIdx.x >> 8 & 1)) __builtin_amdgcn_s_setprio(2);
    int straight = KeyRows::straight(lane), paired = KeyRows::paired(lane), down = KeyRows::down(lane);
    int vdown = ValRows::on(ValRows::down(lane), 16 * NV * wave);
    float passed = 1.0f;      // the decay over the segment
    int c = 0;
    for (int it = 0; it < count; ++it) {
        const int last_c = c;
        c = REV ? c0 + count - 1 - it : c0 + it;
        const int t0 = c * CH, rows = min(CH, n - t0);
        // the chunk into LDS, and its factors
#pragma unroll
        for (int i = 0; i < KI; ++i) {
            *reinterpret_cast<u32x4 *>(sK + KeyRows::at(krow + i * KR, kcol)) = kr[i];
            if constexpr (kOuts) *reinterpret_cast<u32x4 *>(sQ + KeyRows::at(krow + i * KR, kcol)) = qr[i];
        }
#pragma unroll
        for (int i = 0; i < VI; ++i)
            *reinterpret_cast<u32x4 *>(sV + ValRows::at(vrow + i * VR, vcol)) = vr[i];
        const float g2 = decay2(a.decay == SSD_DECAY_TOKEN ? as_float<T>(gn) : lane < rows ? ghead : 0.0f);
        const float ghi = __builtin_rintf(g2 * 256.0f) * (1.0f / 256.0f);
        const float hi = wave_inclusive_sum(ghi), lo = wave_inclusive_sum(g2 - ghi);
        const float hE = wave_read(hi, 63), lE = wave_read(lo, 63);
        const float whole = fast_exp2(hE + lE);
        if (KIND == kEnds) passed *= whole;
        if (wave == 0 && lane < CH) {
            const float from_start = fast_exp2(hi + lo), to_end = fast_exp2((hE - hi) + (lE - lo));
            sHi[lane] = hi;
            sLo[lane] = lo;
            sIn[lane] = (REV ? to_end : from_start) * a.inter;
            sW[lane] = (REV ? from_start : to_end) * a.weight;
        }
        __syncthreads();
        if (kParts && it > 0) store_parts(last_c);
        // hidden from the compiler, which would hold every address that follows from them in a
        // register for all chunks
        asm volatile("" : "+v"(straight), "+v"(paired), "+v"(down), "+v"(vdown));

        f32x4 o[NV][NI] = {};
        Raw xr[kParts ? NV : 1][NI];
        // the states before the chunk, out of the forward walk for the backward one, which asks for
        // them early where registers allow
        constexpr bool kAhead = KIND == kDk && sizeof(T) == 2;
        constexpr int KP = KT * (int)sizeof(T) / 4;        // 16-byte pieces of a lane's keys
        u32x4 before[kAhead ? NV : 1][kAhead ? KP : 1];
        const rsrc_t rs = make_rsrc(
            kParts ? (T *)a.states + ((bh * a.nchunks + c) * a.nvb + vb) * (BV * DK) : nullptr,
            BV * DK * (int)sizeof(T));
        const auto piece = [&](int v, int kp) { return (uint32_t)(((wave * NV + v) * KP + kp) * 64 + lane) * 16; };
        if constexpr (kAhead)
#pragma unroll
            for (int v = 0; v < NV; ++v)
#pragma unroll
                for (int kp = 0; kp < KP; ++kp) before[v][kp] = buf_load_b128(rs, piece(v, kp));
        if constexpr (kOuts) {
            if constexpr (kParts) {
                // rows whose products with the outputs the decays' gradient takes
                const rsrc_t rx = rows_at(xb, a.xp, t0, rows, vw);
#pragma unroll
                for (int v = 0; v < NV; ++v) {
                    const uint32_t off = val4 + 16 * v < vw ? bytes(c16, a.xp, val4 + 16 * v) : kNowhere;
#pragma unroll
                    for (int i = 0; i < NI; ++i)
                        xr[v][i] = buf_load4(rx, off + bytes(16 * i, a.xp, 0), (T *)nullptr);
                }
            }
            // Scores: tile j of them is that of targets i and sources u, u <= i (back in time the
            // other way round).  The tile's place is hidden from the compiler, which would hold
            // every address that follows from it in a register for all chunks.
            int first = wave;
            asm volatile("" : "+s"(first));
#pragma unroll
            for (int j0 = 0; j0 < kTiles; j0 += 4) {
                const int j = j0 + first;
                if (j >= kTiles) break;
                const int row = j < 1 ? 0 : j < 3 ? 1 : j < 6 ? 2 : 3, col = j - row * (row + 1) / 2;
                const int i = REV ? NI - 1 - row : row, u = REV ? NI - 1 - col : col;
                f32x4 p = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int kk = 0; kk < KK; ++kk)
                    p = mma16(load_straight<DK>(sK, straight, u, kk), load_straight<DK>(sQ, straight, i, kk), p);
                const float hi_t = sHi[16 * i + c16], lo_t = sLo[16 * i + c16];
                const f32x4 hs = load4(sHi + 16 * u + 4 * g4), ls = load4(sLo + 16 * u + 4 * g4);
                float e[4];
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    e[r] = REV ? (hs[r] - hi_t) + (ls[r] - lo_t) : (hi_t - hs[r]) + (lo_t - ls[r]);
                if (i == u)
                    // on the diagonal; before the exponential, which is formed for every pair: nothing
                    // not finite from a pair that does not count
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int d = c16 - (4 * g4 + r);
                        const bool keep = REV ? d <= 0 : d >= 0;
                        e[r] = keep ? e[r] : 0.0f;
                        p[r] = keep ? p[r] : 0.0f;
                    }
#pragma unroll
                for (int r = 0; r < 4; ++r) p[r] *= a.intra * fast_exp2(e[r]);
                T *at = sP + (16 * i + c16) * PP + paired_place<T>(u, g4);
                store4(at, p);
                if constexpr (kFine) {
#pragma unroll
                    for (int r = 0; r < 4; ++r) p[r] -= (float)(T)p[r];
                    store4(at + CH * PP, p);
                }
            }

            // what the state before the chunk gives
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int kk = 0; kk < KK; ++kk) {
                Frag q[NI];
#pragma unroll
                for (int i = 0; i < NI; ++i) q[i] = load_paired<DK>(sQ, paired, i, kk);
#pragma unroll
                for (int v = 0; v < NV; ++v) {
                    const Frag f = of_accumulators<T>(S[v], kk);
#pragma unroll
                    for (int i = 0; i < NI; ++i) o[v][i] = mma16(f, q[i], o[v][i]);
                    if constexpr (kFine) {
                        const Frag r = rest_of_accumulators(S[v], kk, f);
#pragma unroll
                        for (int i = 0; i < NI; ++i) o[v][i] = mma16(r, q[i], o[v][i]);
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                const float in = sIn[16 * i + c16];
#pragma unroll
                for (int v = 0; v < NV; ++v) o[v][i] *= in;
                if constexpr (KIND == kDk) {
                    float dot = 0.0f;
#pragma unroll
                    for (int v = 0; v < NV; ++v) dot += dot4(o[v][i], as_floats(xr[v][i]));
                    dot = rows_sum(dot);
                    if (g4 == 0) sWritten[wave][16 * i + c16] = dot;
                }
            }
        }

        if constexpr (kParts) {
            // the states before the chunk out of the forward walk; their products with the
            // gradients of the states behind it in the backward one
            float x = 0.0f;
#pragma unroll
            for (int v = 0; v < NV; ++v)
#pragma unroll
                for (int kp = 0; kp < KP; ++kp) {
                    if constexpr (KIND == kDq) {
                        buf_store_b128(rs, piece(v, kp), __builtin_bit_cast(u32x4, of_accumulators<T>(S[v], kp)));
                    } else {
                        u32x4 w;
                        if constexpr (kAhead) w = before[v][kp];
                        else w = buf_load_b128(rs, piece(v, kp));
                        if constexpr (sizeof(T) == 4) {
                            x += dot4(as_floats(w), S[v][kp]);
                        } else {
                            x += dot4(as_floats(u2{w[0], w[1]}), S[v][2 * kp]);
                            x += dot4(as_floats(u2{w[2], w[3]}), S[v][2 * kp + 1]);
                        }
                    }
                }
            if constexpr (KIND == kDk) {
                x = rows_sum(columns_sum(x)) * whole;
                if (lane == 15) sX[wave] = x;
            }
        }

        // the chunk ahead is asked for from here on, so that its rows hold no registers while the
        // products above need them
        const bool more = it + 1 < count;
        const int ahead = REV ? c - 1 : c + 1;
        __builtin_amdgcn_sched_barrier(0);
        if (more) fetch_k(ahead);

        // the state behind the chunk
        Frag vf[MM][NV];
#pragma unroll
        for (int m = 0; m < MM; ++m)
#pragma unroll
            for (int v = 0; v < NV; ++v) vf[m][v] = load_down<BV>(sV, vdown, m, v);
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int kt = 0; kt < KT; ++kt) S[v][kt] *= whole;
        if (!kOuts) __builtin_amdgcn_s_setprio(1);
#pragma unroll
        for (int m = 0; m < MM; ++m) {
            Frag w[NV][PARTS];
#pragma unroll
            for (int v = 0; v < NV; ++v) weigh(vf[m][v], sW, m, g4, w[v]);
            asm volatile("" : "+v"(down));
            __builtin_amdgcn_sched_barrier(0);
            // tiles of keys side by side: a product's parts wait for each other
#pragma unroll
            for (int kt = 0; kt < KT; kt += kSide) {
                Frag k[kSide];
#pragma unroll
                for (int i = 0; i < kSide; ++i) k[i] = load_down<DK>(sK, down, m, kt + i);
#pragma unroll
                for (int e = 0; e < PARTS; ++e)
#pragma unroll
                    for (int i = 0; i < kSide; ++i)
#pragma unroll
                        for (int v = 0; v < NV; ++v) S[v][kt + i] = mma16(k[i], w[v][e], S[v][kt + i]);
            }
            static_assert(MM > 1, "");
            __builtin_amdgcn_sched_barrier(0);
            if (more && m == 0) fetch_v(ahead);
            if (more && m == 1) fetch_q(ahead);
            __builtin_amdgcn_sched_barrier(0);
        }
        if (!kOuts) __builtin_amdgcn_s_setprio(0);
        __syncthreads();
        if constexpr (KIND == kDk) gather_parts();

        if constexpr (kOuts) {
            // what the chunk's own tokens give: steps of sources that reach these targets
#pragma unroll
            for (int i = 0; i < NI; ++i)
#pragma unroll
                for (int m = 0; m < MM; ++m) {
                    if (REV ? Tile<T>::kStep * (m + 1) <= 16 * i : Tile<T>::kStep * m > 16 * i) continue;
                    const T *at = sP + (16 * i + c16) * PP + Tile<T>::kStep * m + Tile<T>::kPart * g4;
#pragma unroll
                    for (int e = 0; e < (kFine ? 2 : 1); ++e) {
                        const Frag p = *reinterpret_cast<const Frag *>(at + e * CH * PP);
#pragma unroll
                        for (int v = 0; v < NV; ++v) o[v][i] = mma16(vf[m][v], p, o[v][i]);
                    }
                }
            if constexpr (kParts) {
#pragma unroll
                for (int i = 0; i < NI; ++i) {
                    float dot = 0.0f;
#pragma unroll
                    for (int v = 0; v < NV; ++v) dot += dot4(o[v][i], as_floats(xr[v][i]));
                    dot = rows_sum(dot);
                    if (g4 == 0) sPart[wave][16 * i + c16] = dot;
                }
            }
            // rows behind the sequence and values behind the block are dropped
            const int pitch = a.H * a.vd;
            const auto store = [&](auto *base) {
                typedef std::remove_pointer_t<decltype(base)> O;
                const rsrc_t ro = make_rsrc(base + ((row0 + t0) * a.H + h) * a.vd + v0,
                                            ((rows - 1) * pitch + vw) * (int)sizeof(O));
                const auto place = [&](int row, int val) {
                    return val < vw ? (uint32_t)((row * pitch + val) * (int)sizeof(O)) : kNowhere;
                };
                if constexpr (sizeof(O) == 2 && NV == 2) {
                    // Two tiles of values side by side: lanes of odd rows of 16 give their first tile's
                    // four to the row before them and take its second tile's, so that each holds
                    // eight values of one tile, 16 bytes, and four lanes 64 bytes of a row.
                    uint32_t off = place(c16, 16 * NV * wave + 16 * (g4 & 1) + 8 * (g4 >> 1));
#pragma unroll
                    for (int i = 0; i < NI; ++i) {
                        u32x4 w;
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const auto x = __builtin_amdgcn_permlane16_swap(
                                pack_bf16(o[0][i][2 * j], o[0][i][2 * j + 1]),
                                pack_bf16(o[1][i][2 * j], o[1][i][2 * j + 1]), false, false);
                            w[j] = x[0];
                            w[2 + j] = x[1];
                        }
                        buf_store_b128(ro, off, w);
                        off += (uint32_t)(16 * pitch * (int)sizeof(O));
                    }
                } else {
#pragma unroll
                    for (int v = 0; v < NV; ++v) {
                        uint32_t off = place(c16, val4 + 16 * v);
#pragma unroll
                        for (int i = 0; i < NI; ++i) {
                            buf_store4(ro, off, o[v][i], (O *)nullptr);
                            off += (uint32_t)(16 * pitch * (int)sizeof(O));
                        }
                    }
                }
            };
            if (a.o32) store((float *)a.o);
            else store((T *)a.o);
        }
    }
    if (kParts && count > 0) {
        __syncthreads();
        store_parts(c);
    }

    if constexpr (KIND == kEnds)
        if (tid == 0 && vb == 0) a.decays[bh * a.nseg + s] = passed;
    float *p = KIND == kEnds ? a.ends + (bh * a.nseg + s) * size
               : a.last      ? a.last + bh * size
                             : nullptr;
    if (p)
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int kt = 0; kt < KT; ++kt) {
                const int key = 16 * kt + 4 * g4, val = val0 + 16 * v;
                if (val < vw && key < a.kd) store4(p + (int64_t)(v0 + val) * a.kd + key, S[v][kt]);
            }
}

// ---------------------------------------------------------------------------
// Starts of the segments of every head out of their ends, in place, and the last state: a thread
// for four elements of a head's state, the next kAhead segments' ends on their way while those
// before them are chained.  One wave a workgroup, as a single head has no more than 64 to spread.
// ---------------------------------------------------------------------------
constexpr int kChainThreads = 64;
__global__ __launch_bounds__(kChainThreads) void chain_kernel(float *ends, const float *__restrict__ decays,
                                                              const float *init, float *last, int64_t quads,
                                                              int size4, int nseg)
{
    constexpr int kAhead = 8;
    const int64_t id = (int64_t)blockIdx.x * kChainThreads + threadIdx.x;
    if (id >= quads) return;
    const int64_t bh = id / size4;
    f32x4 *p = reinterpret_cast<f32x4 *>(ends) + bh * nseg * size4 + id % size4;
    f32x4 S = init ? reinterpret_cast<const f32x4 *>(init)[id] : f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    f32x4 end[kAhead], next[kAhead];
    float d[kAhead], dnext[kAhead];
    const auto fetch = [&](int s0) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int s = min(s0 + i, nseg - 1);
            next[i] = p[(int64_t)s * size4];
            dnext[i] = decays[bh * nseg + s];
        }
    };
    fetch(0);
    for (int s0 = 0; s0 < nseg; s0 += kAhead) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            end[i] = next[i];
            d[i] = dnext[i];
        }
        if (s0 + kAhead < nseg) fetch(s0 + kAhead);
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            if (s0 + i >= nseg) break;
            p[(int64_t)(s0 + i) * size4] = S;
            S = S * d[i] + end[i];
        }
    }
    if (last) reinterpret_cast<f32x4 *>(last)[id] = S;
}

// ---------------------------------------------------------------------------
// Gradient of the log decays, a wave for a chunk of a head, a lane for a token.  g_t scales every
// product of a read in or behind token t with a write before it.  In t's chunk:
//   read     all that is read by its tokens from t on, q . dq
//   own      less what these tokens write themselves and the chunk reads, the part of k . dk from
//            within the chunk (its pairs are the same rounded scores as in q . dq: what is on one
//            side of t cancels but for fp32's sums, however small the rest)
//   written  what its tokens before t write and is read behind the chunk, the other part of k . dk
//   cross    and what passes the whole chunk, <S, dS>
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
        const int t = lane < a.chunk ? c * a.chunk + lane : n;
        if (c * a.chunk >= n) continue;
        float read = 0.0f, written = 0.0f, cross = 0.0f;
        for (int i = 0; i < a.nvb; ++i) {
            if (t < n) {
                read += a.read[(bh * a.nvb + i) * a.L + t] - a.own[(bh * a.nvb + i) * a.L + t];
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

template <typename T, int NV, bool REV, Kind KIND, int PARTS>
hipError_t walk_by_key(const Walk &a, hipStream_t st)
{
    const dim3 blocks((unsigned)((a.groups + 7) / 8 * 8 * a.nvb)), threads(kThreads);
    if (a.kd <= 64)
        hipLaunchKernelGGL((walk_kernel<T, 64, NV, REV, KIND, PARTS>), blocks, threads, 0, st, a);
    else if (a.kd <= 128)
        hipLaunchKernelGGL((walk_kernel<T, 128, NV, REV, KIND, PARTS>), blocks, threads, 0, st, a);
    else
        hipLaunchKernelGGL((walk_kernel<T, 256, NV, REV, KIND, PARTS>), blocks, threads, 0, st, a);
    return hipGetLastError();
}

// Values of a walk: 64, or 128 (bf16, without a part in the decays' gradient) where there are more.
int block_of(bool bf16, Kind kind, int64_t values)
{
    return bf16 && (kind == kEnds || kind == kOut) && values > 64 ? 128 : 64;
}
int blocks_of(bool bf16, Kind kind, int64_t values)
{
    const int block = block_of(bf16, kind, values);
    return (int)((values + block - 1) / block);
}

template <typename T, bool REV, Kind KIND> hipError_t walk_launch(Walk a, int64_t bh, hipStream_t st)
{
    a.groups = bh * a.nseg;
    a.nvb = blocks_of(sizeof(T) == 2, KIND, a.vd);
    if constexpr (sizeof(T) == 4) {
        return walk_by_key<T, 1, REV, KIND, 1>(a, st);
    } else if constexpr (KIND == kDq || KIND == kDk) {
        return walk_by_key<T, 1, REV, KIND, 2>(a, st);
    } else {
        const bool wide = block_of(true, KIND, a.vd) == 128;
        if (KIND == kEnds || a.last)
            return wide ? walk_by_key<T, 2, REV, KIND, 3>(a, st) : walk_by_key<T, 1, REV, KIND, 3>(a, st);
        if constexpr (KIND == kOut)
            return wide ? walk_by_key<T, 2, REV, KIND, 2>(a, st) : walk_by_key<T, 1, REV, KIND, 2>(a, st);
        return hipErrorInvalidValue;
    }
}

// The ends of a walk's segments, then their starts and the last state.
template <typename T, bool REV> hipError_t starts_go(const Walk &a, float *last, int64_t bh, hipStream_t st)
{
    const hipError_t e = walk_launch<T, REV, kEnds>(a, bh, st);
    if (e != hipSuccess) return e;
    const int size4 = a.kd * a.vd / 4;
    const int64_t quads = bh * size4;
    hipLaunchKernelGGL(chain_kernel, dim3((unsigned)((quads + kChainThreads - 1) / kChainThreads)),
                       dim3(kChainThreads), 0, st, a.ends, a.decays, a.init, last, quads, size4, a.nseg);
    return hipGetLastError();
}


// How the chunks of a walk are split into segments, whose ends a first walk leaves.  `keys`: of the
// widest state.  As many as give each CU two workgroups, 512, or one where a walk leaves no room for
// two (256).  More do not pay, though walks of 64 values fit three a CU: 24 heads of 2 x 2048 tokens
// of 128 x 64 take 43 us in 384, 50 in 528 and 45 in 768, 16384 tokens of 16 heads of 128 x 128 113
// in 512, 153 in 688 and 155 in 1024 (123 in 256; the same inputs again).  fp32 keys past 128 count as
// one a CU; by their LDS two fit, and 8192 tokens of 8 heads of 256 x 256 take 329 us in 256, 289 in 512.
// While each has a CU to itself a segment may be one chunk; else it is two or more, as the chain over the
// segments is then the longer part (4 x 1024 tokens of 8 heads of 128 x 128: 37 us with two, 46 with one).
// Segments are walked twice, and their ends and the chain are launches that take about the time of
// two chunks (fp32: one), so there are none unless that is less than one walk over all: 256
// tokens of 8 bf16 heads of 128 x 128 take 21 us in one walk and 24 in four segments, the gradients of 256
// of 4 fp32 heads of 64 x 64 87 and 50.
struct Split {
    int seg, nseg;
};
Split split_of(bool is_bf16, int64_t keys, int64_t walks, int64_t tokens)
{
    const int64_t fit = (is_bf16 ? keys <= 128 : keys <= 64) ? 512 : 256;
    const int64_t chunks = (tokens + 63) / 64, n = std::max<int64_t>(fit / walks, 1);
    int64_t seg = (chunks + n - 1) / n;
    if (seg == 1 && walks * chunks > 256) seg = 2;
    if (2 * seg + (is_bf16 ? 2 : 1) >= chunks) seg = chunks;
    return {(int)seg * 64, (int)((chunks + seg - 1) / seg)};
}

// Chunks of the walks that leave parts of the decays' gradient (their keys are the values).
int part_chunks(const LinattnShape &s)
{
    const int n = chunk_tokens(s.bf16, s.dv);
    return (int)((s.L + n - 1) / n);
}

// Keys that a walk's state has room for.
int64_t padded_keys(int64_t keys) { return keys <= 64 ? 64 : keys <= 128 ? 128 : 256; }

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
    return split_of(s.bf16, s.dk, s.b * s.H * blocks_of(s.bf16, kOut, s.dv), s.L);
}

Split grad_split(const LinattnShape &s)
{
    return split_of(s.bf16, std::max(s.dk, s.dv),
                    s.b * s.H * std::min(blocks_of(s.bf16, kOut, s.dk), blocks_of(s.bf16, kOut, s.dv)), s.L);
}

// Workspace of the gradients (byte offsets, on 256 bytes): with a decays' gradient the states
// before each chunk and the parts that its kernel adds up; with shared heads every head's dq and dk.
struct GradLayout {
    int64_t states, read, own, written, cross, dq, dk, ends, decays, back_ends, back_decays, bytes;
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
    const int64_t bh = s.b * s.H, nvb = blocks_of(s.bf16, kDq, s.dk), nc = part_chunks(s);
    y.states = take(gates, bh * nc * nvb * 64 * padded_keys(s.dv) * (s.bf16 ? 2 : 4));
    y.read = take(gates, bh * nvb * s.L * 4);
    y.own = take(gates, bh * nvb * s.L * 4);
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
    const Split y = forward_split(s);
    w.seg = y.seg; w.nseg = y.nseg;
    w.ends = (float *)a.ws;
    w.decays = (float *)((char *)a.ws + ends_bytes(s, y.nseg));
    if (y.nseg > 1) {
        const hipError_t e = starts_go<T, false>(w, w.last, s.b * s.H, st);
        if (e != hipSuccess) return e;
        w.last = nullptr;
    }
    return walk_launch<T, false, kOut>(w, s.b * s.H, st);
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
    w.nchunks = part_chunks(s);
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
            x->kd = (int)s.dk; x->vd = (int)s.dv;
        }
        e = starts_go<T, false>(f, nullptr, bh, st);
        if (e == hipSuccess) e = starts_go<T, true>(r, a.dh0, bh, st);
        if (e != hipSuccess) return e;
    }

    Walk q = w;          // dq = scale S^T do
    q.q = a.dout; q.qp = s.dop; q.qdiv = 1;
    q.k = a.v; q.kp = s.vp; q.kdiv = 1;
    q.v = a.k; q.vp = s.kp; q.vdiv = share;
    q.o = share > 1 ? at(y.dq) : a.dq; q.o32 = share > 1;
    q.init = a.h0; q.sv = 1; q.sk = s.dk;
    q.inter = q.intra = s.scale; q.weight = 1.0f;
    q.kd = (int)s.dv; q.vd = (int)s.dk;
    q.x = a.q; q.xp = s.qp; q.xdiv = share;
    q.part = (float *)at(y.read);
    e = gates ? walk_launch<T, false, kDq>(q, bh, st) : walk_launch<T, false, kOut>(q, bh, st);
    if (e != hipSuccess) return e;

    Walk k = back;       // dk = dS^T v, scale in dS
    k.q = a.v; k.qp = s.vp; k.qdiv = 1;
    k.k = a.dout; k.kp = s.dop; k.kdiv = 1;
    k.v = a.q; k.vp = s.qp; k.vdiv = share;
    k.o = share > 1 ? at(y.dk) : a.dk; k.o32 = share > 1;
    k.init = a.dhT; k.sv = 1; k.sk = s.dk;
    k.inter = 1.0f; k.intra = k.weight = s.scale;
    k.kd = (int)s.dv; k.vd = (int)s.dk;
    k.x = a.k; k.xp = s.kp; k.xdiv = share;
    k.part = (float *)at(y.own); k.written = (float *)at(y.written);
    e = gates ? walk_launch<T, true, kDk>(k, bh, st) : walk_launch<T, true, kOut>(k, bh, st);
    if (e != hipSuccess) return e;

    Walk v = back;       // dv = dS k
    v.q = a.k; v.qp = s.kp; v.qdiv = share;
    v.k = a.q; v.kp = s.qp; v.kdiv = share;
    v.v = a.dout; v.vp = s.dop; v.vdiv = 1;
    v.o = a.dv;
    v.init = a.dhT; v.sv = s.dk; v.sk = 1;
    v.last = v.nseg > 1 ? nullptr : a.dh0;
    v.inter = 1.0f; v.intra = v.weight = s.scale;
    v.kd = (int)s.dk; v.vd = (int)s.dv;
    e = walk_launch<T, true, kOut>(v, bh, st);
    if (e != hipSuccess) return e;

    if (gates) {
        DecayGradient d = {};
        d.g = a.g; d.gp = s.gp; d.lengths = a.lengths;
        d.read = q.part; d.own = k.part; d.written = k.written; d.cross = w.cross;
        d.dg = a.dg;
        d.bh = bh; d.L = (int)s.L; d.H = (int)s.H; d.nvb = blocks_of(s.bf16, kDq, s.dk);
        d.nchunks = w.nchunks; d.chunk = chunk_tokens(s.bf16, s.dv);
        hipLaunchKernelGGL((decay_gradient_kernel<T>), dim3(groups_for(bh * w.nchunks, 4)), dim3(kThreads),
                           0, st, d);
        e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (share > 1) {
        const int64_t quads = s.b * s.L * s.G * (s.dk / 4);
        for (int i = 0; i < 2; ++i) {
            hipLaunchKernelGGL((shared_sum_kernel<T>), dim3(groups_for(quads, kThreads)), dim3(kThreads),
                               0, st, (const float *)at(i ? y.dk : y.dq), (T *)(i ? a.dk : a.dq),
                               a.lengths, quads, (int)s.L, (int)s.G, share, (int)s.dk);
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
