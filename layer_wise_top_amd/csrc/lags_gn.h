// Device side shared by the group normalisation kernels: a workgroup's
// geometry, sums over it, and per-channel parameters.
#pragma once

#include "lags_act.h"

#include <type_traits>

namespace lags {

constexpr uint32_t kResident = 1024;  // threads of a resident workgroup, at most (forward)
constexpr uint32_t kResidentBwd = 512;   // backward; 1024 of up to kWideRows rows where a slab has so many lanes
constexpr uint32_t kWideRows = 4;
constexpr uint32_t kMostRows = 13;   // register rows a thread, at most

// A workgroup takes `w` channels (whole groups, whole runs) of one sample:
// 2^tcl lanes span them in 16-byte vectors, the other lane bits and the waves
// take positions.
struct Geo {
    uint32_t tcl, col, row, tr, parts;   // column vector, first position, positions a sweep, sums a channel
    uint32_t n, chunk, c0, wc, ng, c;
    int nv;                              // channels of the thread's vector (<= 0: idle)
};
// Slabs of one sample run side by side on one XCD (workgroups are dealt to
// the 8 XCDs in turn): they share cache lines at their edges.
__device__ inline Geo geometry(const GnArgs &a, uint32_t V, uint32_t nchunk)
{
    const uint32_t per = gridDim.x / 8, main = per * 8, id = blockIdx.x;
    const uint32_t b = id < main ? (id & 7) * per + (id >> 3) : id;
    Geo g;
    const uint32_t s = b / a.nslab, slab = b - s * a.nslab;
    g.n = nchunk == 1 ? s : s / nchunk;
    g.chunk = s - g.n * nchunk;
    g.tcl = a.tcl;
    g.col = threadIdx.x & ((1u << a.tcl) - 1);
    g.row = threadIdx.x >> a.tcl;
    g.tr = blockDim.x >> a.tcl;
    g.parts = a.tcl >= 6 ? g.tr : blockDim.x >> 6;
    g.c0 = slab * a.w;
    g.wc = min(a.w, a.C - g.c0);
    g.ng = (uint32_t)(((float)g.wc + 0.5f) * a.inv_cg);
    g.c = g.c0 + g.col * V;
    g.nv = (int)g.wc - (int)(g.col * V);
    return g;
}
// c / cg for c up to a slab's channels times its parts (65536): the product is
// off by less than 2^-6 / cg, the quotient's distance from an integer at least
// half of 1 / cg.
__device__ inline uint32_t over_cg(uint32_t c, float inv_cg) { return (uint32_t)(((float)c + 0.5f) * inv_cg); }

// ---- sums over a workgroup -------------------------------------------------

// The lane 8, 4, 2 or 1 away.
template <int O> __device__ inline float lane_xor(float x)
{
    const int v = __builtin_bit_cast(int, x);
    if constexpr (O == 8) return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, v, 0x128, 0xf, 0xf, false));
    if constexpr (O == 4) {              // 7 - lane, then 3 - lane
        const int m = __builtin_amdgcn_update_dpp(0, v, 0x141, 0xf, 0xf, false);
        return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, m, 0x1b, 0xf, 0xf, false));
    }
    if constexpr (O == 2) return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, v, 0x4e, 0xf, 0xf, false));
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, v, 0xb1, 0xf, 0xf, false));
}
// x of both halves (O = 32) or of both rows of a pair (16) in the lower one, y
// of both in the upper one: their sums.
template <int O> __device__ inline float swap_sum(float x, float y)
{
    const uint32_t a = asu(x), b = asu(y);
    if constexpr (O == 32) {
        const auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
        return asf(r[0]) + asf(r[1]);
    } else {
        const auto r = __builtin_amdgcn_permlane16_swap(a, b, false, false);
        return asf(r[0]) + asf(r[1]);
    }
}

// Sums over the lane bits 32 .. tc (the rows of a wave).  Each step halves the
// values a lane holds, the upper half of them going to the lanes with the bit
// set, so log2(V) steps cost V - 1 exchanges and leave each lane one column's
// sum; `base` is the first column it holds, `cur` how many.
template <int V, int CUR, int O>
__device__ inline void row_reduce(float (&v)[V], uint32_t tc, uint32_t lane, uint32_t &base, uint32_t &cur)
{
    if constexpr (O >= 1) {
        if (O >= (int)tc) {
            if constexpr (CUR > 1) {
                const bool up = lane & O;
#pragma unroll
                for (int j = 0; j < CUR / 2; ++j) {
                    if constexpr (O >= 16) {
                        v[j] = swap_sum<O>(v[j], v[j + CUR / 2]);
                    } else {
                        const float send = up ? v[j] : v[j + CUR / 2];
                        const float keep = up ? v[j + CUR / 2] : v[j];
                        v[j] = keep + lane_xor<O>(send);
                    }
                }
                if (up) base += CUR / 2;
                cur = CUR / 2;
                row_reduce<V, CUR / 2, O / 2>(v, tc, lane, base, cur);
            } else {
                if constexpr (O >= 16)
                    v[0] = swap_sum<O>(v[0], v[0]);
                else
                    v[0] += lane_xor<O>(v[0]);
                row_reduce<V, 1, O / 2>(v, tc, lane, base, cur);
            }
        }
    }
}

// Per-channel sums of the workgroup's waves, left as sh[part][channel of the
// slab, padded to 2^tcl vectors].
template <int V> __device__ inline void to_parts(float (&v)[V], const Geo &g, float *sh)
{
    const uint32_t lane = threadIdx.x & 63, tc = 1u << g.tcl;
    uint32_t base = 0, cur = V;
    row_reduce<V, V, 32>(v, tc, lane, base, cur);
    const uint32_t part = g.tcl >= 6 ? g.row : threadIdx.x >> 6;
    float *p = sh + part * (tc * V) + g.col * V + base;
    // lanes that hold the same columns hold the same sums
#pragma unroll
    for (int j = 0; j < V; ++j)
        if (j < (int)cur) p[j] = v[j];
}

// Group sums from the parts, 2^k lanes a group, each channel's times its
// weight if there are any; done(group of the slab, sum) runs on one lane of each.
template <int V, typename F>
__device__ inline void to_groups(const Geo &g, const float *sh, uint32_t cg, float inv_cg, F done,
                                 const float *weight = nullptr)
{
    const uint32_t wp = V << g.tcl, items = cg * g.parts;
    uint32_t lg = 1;
    while (lg < 64 && lg < items) lg <<= 1;
    const uint32_t sub = threadIdx.x & (lg - 1), lgl = __builtin_ctz(lg), per = blockDim.x >> lgl;
    // every lane of a wave runs every iteration: the exchanges need them
    for (uint32_t g0 = 0; g0 < g.ng; g0 += per) {
        const uint32_t gi = g0 + (threadIdx.x >> lgl);
        float s = 0;
        if (gi < g.ng)
#pragma unroll 4
            for (uint32_t i = sub; i < items; i += lg) {
                const uint32_t p = over_cg(i, inv_cg), c = gi * cg + i - p * cg;
                s += weight ? sh[p * wp + c] * weight[c] : sh[p * wp + c];
            }
        if (lg > 1) s += lane_xor<1>(s);
        if (lg > 2) s += lane_xor<2>(s);
        if (lg > 4) s += lane_xor<4>(s);
        if (lg > 8) s += lane_xor<8>(s);
        if (lg > 16) s = swap_sum<16>(s, s);
        if (lg > 32) s = swap_sum<32>(s, s);
        if (gi < g.ng && sub == 0) done(gi, s);
    }
}

// Sums of a thread's channels for their groups.  UNI: the thread's vector lies
// in one group, so its channels are added up first and a lane carries one
// value; else one a channel.
template <int V, bool UNI> struct GroupSum {
    static constexpr int N = UNI ? 1 : V;
    float v[N];
    __device__ GroupSum(const float (&s)[V])
    {
        if constexpr (UNI) {
            float t[V];
            for (int j = 0; j < V; ++j) t[j] = s[j];
#pragma unroll
            for (int h = V / 2; h; h >>= 1)
                for (int j = 0; j < h; ++j) t[j] += t[j + h];
            v[0] = t[0];
        } else {
            for (int j = 0; j < V; ++j) v[j] = s[j];
        }
    }
    __device__ void parts(const Geo &g, float *sh) { to_parts<N>(v, g, sh); }
    template <typename F> __device__ static void groups(const Geo &g, const float *sh, const GnArgs &a, F done)
    {
        if constexpr (UNI)
            to_groups<1>(g, sh, a.cg / V, a.inv_cg * V, done);
        else
            to_groups<V>(g, sh, a.cg, a.inv_cg, done);
    }
};

// The sum over a wave, on every lane.
__device__ inline float wave_sum(float s)
{
    s += lane_xor<1>(s);
    s += lane_xor<2>(s);
    s += lane_xor<4>(s);
    s += lane_xor<8>(s);
    s = swap_sum<16>(s, s);
    return swap_sum<32>(s, s);
}

// ---- per-channel values ----------------------------------------------------
// UNI: a thread's vector lies in one group (cg is a multiple of it), so what a
// group has is one value; else one a channel.
template <int V, bool UNI> struct PerGroup {
    float v[UNI ? 1 : V];
    __device__ float operator[](int j) const { return v[UNI ? 0 : j]; }
    // f(group of the slab) of each channel's group
    template <typename F> __device__ void set(const Geo &g, uint32_t cg, float inv_cg, F f)
    {
        const uint32_t c = g.nv > 0 ? g.col * V : 0;
        uint32_t q = over_cg(c, inv_cg), r = c - q * cg;
#pragma unroll
        for (int j = 0; j < (UNI ? 1 : V); ++j) {
            v[j] = f(min(q, g.ng - 1));
            if (!UNI && ++r == cg) r = 0, ++q;
        }
    }
};

// A parameter's values at the thread's channels; `other` where there is none.
template <int V> __device__ inline void load_param(const float *p, const Geo &g, float other, float (&f)[V])
{
    const auto r = window(p ? p + g.c0 : p, p ? (int64_t)g.wc * 4 : 0);
    const uint32_t at = g.nv > 0 ? g.col * V * 4 : 0x80000000u;
#pragma unroll
    for (int i = 0; i < V / 4; ++i) {
        const u32x4 v = __builtin_amdgcn_raw_buffer_load_b128(r, at + 16 * i, 0, 0);
        for (int j = 0; j < 4; ++j) f[4 * i + j] = p ? asf(v[j]) : other;
    }
}

// The vector, which the compiler takes to be made anew here, once `t` is
// known.  Between two passes over the vectors this keeps them as they were
// loaded, not unpacked in twice the registers; within a pass it keeps the
// compiler from unpacking all of them at its start.
__device__ inline void keep(u32x4 &v, float t) { asm volatile("" : "+v"(v) : "v"(t)); }

// The sums are up to date here: without this the compiler puts them off and
// keeps what they add, for every vector.
template <int V> __device__ inline void settle(float (&s)[V])
{
#pragma unroll
    for (int j = 0; j < V; ++j) asm volatile("" : "+v"(s[j]));
}

// max(x, 0) that keeps a NaN.
__device__ inline float above_zero(float x) { return x < 0 ? 0.0f : x; }

template <typename F> hipError_t by_bool(bool b, F f)
{
    return b ? f(std::true_type()) : f(std::false_type());
}
template <typename F> hipError_t by_act(int act, F f)
{
    if (act == kActRelu) return f(std::integral_constant<int, kActRelu>());
    if (act == kActSilu) return f(std::integral_constant<int, kActSilu>());
    return f(std::integral_constant<int, kActNone>());
}
// The kernel for at least `rows` register rows of those for 2, 4, 8 and 13:
// rows are cheapest where all are used (absent ones read zeros), and 13 rows of
// two vectors are what a backward thread holds at three waves a SIMD.
template <typename F> hipError_t by_rows(uint32_t rows, F f)
{
    if (rows <= 2) return f(std::integral_constant<int, 2>());
    if (rows <= 4) return f(std::integral_constant<int, 4>());
    if (rows <= 8) return f(std::integral_constant<int, 8>());
    return f(std::integral_constant<int, kMostRows>());
}
// Whether rows of 16-bit values may start inside a word; fp32 rows never do.
template <int D> bool odd_rows(const void *p, int64_t ld)
{
    return D != kF32 && p && (((uintptr_t)p | (uint64_t)ld * 2) & 3);
}
template <int D, typename F> hipError_t by_odd(bool odd, F f)
{
    if constexpr (D != kF32)
        if (odd) return f(std::true_type());
    return f(std::false_type());
}
// LDS of the sums: `arrays` of per-wave channel sums, and `per_group` floats a group.
inline size_t lds_bytes(const GnPlan &p, uint32_t V, uint32_t cg, uint32_t arrays, uint32_t per_group,
                        uint32_t per_channel = 0)
{
    const uint32_t parts = p.tcl >= 6 ? p.threads >> p.tcl : p.threads >> 6;
    return ((size_t)arrays * parts * (V << p.tcl) + (size_t)per_group * (p.w / cg) + (size_t)per_channel * p.w) * 4;
}

}  // namespace lags
