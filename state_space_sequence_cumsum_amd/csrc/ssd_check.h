// ssd_check.h -- host-side argument checks shared by the entry points of the operators around the
// forward and of linear attention.
#pragma once

#include "../../include/ssd.h"

#include <cstdint>
#include <initializer_list>

#include "ssd_launch.h"

namespace ssd {
namespace check {

constexpr int64_t kMaxTokens = int64_t(1) << 30;
constexpr int64_t kMaxRows = int64_t(1) << 31;       // batch * seqlen

inline bool on_bytes(size_t n, std::initializer_list<const void *> ptrs)
{
    for (const void *p : ptrs)
        if ((reinterpret_cast<uintptr_t>(p) & (n - 1)) != 0) return false;
    return true;
}

inline bool is_dtype(int32_t d) { return d == SSD_F32 || d == SSD_BF16; }
inline bool is_flag(int32_t f) { return f == 0 || f == 1; }
// 0 (dense) or at least the row's width
inline bool pitch_fits(int64_t pitch, int64_t width) { return pitch == 0 || pitch >= width; }
inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline bool finite(float v) { return v - v == 0.0f; }

// batch and seqlen (both positive) within the index limits
inline bool tokens_fit(int64_t batch, int64_t seqlen)
{
    return seqlen <= kMaxTokens && batch <= kMaxRows / seqlen;
}

// ---------------------------------------------------------------------------
// Outputs and inputs apart.  The kernels read inputs that other threads' outputs would have
// replaced (a token tile of the convolution reads the rows before it), so memory that an output
// shares with another argument is refused.  `rows` rows of `width` bytes, `pitch` bytes apart;
// `same`: an output with this very layout may be this buffer (each element is read before the
// same thread writes it).
// ---------------------------------------------------------------------------
struct Area {
    const void *p;
    int64_t rows, pitch, width;
    bool same;
};

inline int64_t bytes_of(int32_t dtype) { return dtype == SSD_BF16 ? 2 : 4; }

inline Area dense(const void *p, int64_t bytes, bool same = false) { return {p, 1, bytes, bytes, same}; }

// rows of `width` elements at a pitch of `pitch` elements (0: dense)
inline Area rows_of(const void *p, int64_t rows, int64_t pitch, int64_t width, int64_t bytes,
             bool same = false)
{
    if (pitch == 0 || pitch == width || rows == 1) return dense(p, rows * width * bytes, same);
    return {p, rows, pitch * bytes, width * bytes, same};
}

// Whether a dense output shares memory with `in`.
inline bool meet(const Area &out, const Area &in)
{
    if (out.p == nullptr || in.p == nullptr) return false;
    // the output's start from the input's, and the input's first row that ends behind it
    const int64_t d = (int64_t)(reinterpret_cast<uintptr_t>(out.p) - reinterpret_cast<uintptr_t>(in.p));
    if (d + out.width <= 0) return false;
    if (d >= in.width) {
        const int64_t row = in.rows == 1 ? 1 : (d - in.width) / in.pitch + 1;
        if (row >= in.rows || row * in.pitch >= d + out.width) return false;
    }
    return !(in.same && d == 0 && in.rows == 1 && in.width == out.width);
}

inline ssd_status check_apart(std::initializer_list<Area> outs, std::initializer_list<Area> ins)
{
    for (const Area *o = outs.begin(); o != outs.end(); ++o) {
        for (const Area &in : ins)
            if (meet(*o, in)) return SSD_ERR_OVERLAP;
        for (const Area *p = o + 1; p != outs.end(); ++p)
            if (meet(*o, *p)) return SSD_ERR_OVERLAP;
    }
    return SSD_OK;
}

inline ssd_status status_of(hipError_t e) { return ssd_status(ssd::hip_status(e)); }

}  // namespace check
}  // namespace ssd
