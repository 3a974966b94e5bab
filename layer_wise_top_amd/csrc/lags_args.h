// Checks of arguments that the operators' entry points share (host side).
#pragma once

#include "lags.h"
#include "lags_act.h"

namespace lags {

typedef unsigned __int128 u128;
constexpr int64_t kMaxDim = 0x7fffffff;
constexpr u128 kMaxBytes = (u128)1 << 62;

inline bool aligned(const void *p, size_t a) { return ((uintptr_t)p & (a - 1)) == 0; }
inline bool known_dtype(int32_t d) { return d == LAGS_F32 || d == LAGS_BF16 || d == LAGS_F16; }

// A strided region of device memory: `rows` runs of `width` bytes, `pitch` bytes apart.
struct Region {
    const void *p;
    u128 rows, width, pitch;
    u128 bytes() const { return rows ? (rows - 1) * pitch + width : 0; }
};

inline Region flat(const void *p, size_t bytes) { return {p, 1, bytes, bytes}; }

// Columns of one buffer taken at the same pitch do not overlap where their
// columns do not; regions of unlike pitch count as overlapping where their
// address ranges meet.
inline bool overlap(const Region &a, const Region &b)
{
    if (!a.p || !b.p || !a.bytes() || !b.bytes()) return false;
    const u128 x = (uintptr_t)a.p, y = (uintptr_t)b.p;
    if (x + a.bytes() <= y || y + b.bytes() <= x) return false;
    if (a.pitch != b.pitch || a.rows < 2 || b.rows < 2) return true;
    // the later column's distance past the earlier one, within a row
    const u128 d = x <= y ? (y - x) % a.pitch : (a.pitch - (x - y) % a.pitch) % a.pitch;
    return d < a.width || d + b.width > a.pitch;
}

// A [rows, cols] matrix argument: its region, or a status.
inline int matrix(const void *p, int64_t rows, int64_t cols, int64_t ld, int32_t dtype, Region &r)
{
    const uint32_t e = elem_bytes(dtype);
    if (!p || !aligned(p, e) || ld < cols) return LAGS_EINVAL;
    if (ld > kMaxDim || (u128)rows * (u128)ld * e > kMaxBytes) return LAGS_ERANGE;
    r = {p, (u128)rows, (u128)cols * e, (u128)ld * e};
    return LAGS_OK;
}

inline bool ckpt_dims(int64_t rows, int64_t cols)
{
    return rows >= 0 && cols >= 1 && cols <= kMaxDim && (u128)rows * (u128)(cols + 64) * 2 <= kMaxBytes;
}

inline int hip(hipError_t e) { return e == hipSuccess ? LAGS_OK : LAGS_EHIP; }

// `out` must not overlap any of the n regions of `all` but itself.
inline bool clear_of(const Region *all, int n, int out)
{
    for (int i = 0; i < n; ++i)
        if (i != out && overlap(all[i], all[out])) return false;
    return true;
}

inline bool same(const Region &a, const Region &b) { return a.p == b.p && a.pitch == b.pitch; }

}  // namespace lags
