// Kernels of a linear layer: z = x W^T + bias, y = act(z) + res, and the product
// dx = dz W of its backward.
//
// Both are C[m][n] = sum over k of A[m][k] B'[k][n]; A's rows (x, dz) run along k.
// Forward B is W [n][k], whose rows run along k too, so that a matrix
// instruction's operands are 16 consecutive bytes of LDS each.  Backward B is W
// [k][n], staged as it comes and transposed by the LDS transpose reads (fp32: by
// reading a value a lane).  fp32 runs on the fp32 matrix instructions; all sums are
// held in fp32.
#pragma once

#include "lags_gn.h"
#include "lags_layer.h"

#include <algorithm>
#include <type_traits>

namespace lags {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

// ---- activations -----------------------------------------------------------
// s = 1 / (1 + exp(-u)) and 1 - s.  16-bit types: the hardware's exponential and
// reciprocal, good to a few units of 2^-23 and, since u / ln 2 is rounded first, |u| 2^-24 of the
// result (5e-6 where |u| is 87).  That is far below dz's rounding; the fp32 sums of dbias take it as it is.
template <int D> __device__ inline float sigmoid(float u, float &rest)
{
    if constexpr (D == kF32) {
        const float q = expf(-u), s = 1.0f / (1.0f + q);
        rest = q * s;
        return s;
    }
    const float q = __expf(-u), s = __builtin_amdgcn_rcpf(1.0f + q);
    rest = q * s;
    return s;
}
constexpr float kGelu = 1.5957691216057308f;      // 2 sqrt(2 / pi)
// Past these magnitudes of z, where exp(-u) is about to leave fp32's range and the sigmoid is 0 or 1
// but for less than 2^-124, z is taken as this (a NaN stays), so that no infinity meets a zero.
constexpr float kFarSilu = 87, kFarGelu = 10;
__device__ inline float within(float z, float top) { return z < -top ? -top : z > top ? top : z; }

template <int D> __device__ inline float act_value(float z, int act)
{
    float rest;
    if (act == kActRelu) return above_zero(z);
    if (act == kActSilu) return (z < -kFarSilu ? -kFarSilu : z) * sigmoid<D>(within(z, kFarSilu), rest);
    if (act == kActGelu) {
        const float c = within(z, kFarGelu);
        return (z < -kFarGelu ? -kFarGelu : z) * sigmoid<D>(kGelu * c * __builtin_fmaf(0.044715f * c, c, 1.0f), rest);
    }
    return z;
}
template <int D> __device__ inline float act_slope(float z, int act)
{
    float rest;
    if (act == kActRelu) return z > 0 ? 1.0f : z != z ? z : 0.0f;
    if (act == kActSilu) {
        const float c = within(z, kFarSilu), s = sigmoid<D>(c, rest);
        return s * __builtin_fmaf(c, rest, 1.0f);
    }
    if (act == kActGelu) {
        const float c = within(z, kFarGelu), q = c * c;
        const float s = sigmoid<D>(kGelu * c * __builtin_fmaf(0.044715f, q, 1.0f), rest);
        return s * __builtin_fmaf(c * rest * kGelu, __builtin_fmaf(0.134145f, q, 1.0f), 1.0f);
    }
    return 1.0f;
}

// ---- what becomes of a sum -------------------------------------------------
// V consecutive sums of row m from column n on, nv of them within the matrix.
template <int D> __device__ inline void finish(const LinArgs &a, int64_t m, uint32_t n, int nv, float (&f)[Elem<D>::V])
{
    constexpr int V = Elem<D>::V, E = Elem<D>::E;
    if (a.bias) {
        for (int i = 0; i < V; i += 4) {
            if (i + 4 <= nv) {
                const f32x4_u4 b = *(const f32x4_u4 *)(a.bias + n + i);
                for (int j = 0; j < 4; ++j) f[i + j] += b[j];
            } else {
                for (int j = i; j < i + 4; ++j)
                    if (j < nv) f[j] += a.bias[n + j];
            }
        }
    }
    if (a.z) store_vec<D>((char *)a.z + (m * a.ldz + n) * E, Elem<D>::pack(f), nv);
    if (a.act != kActNone)
        for (int j = 0; j < V; ++j) f[j] = act_value<D>(f[j], a.act);
    if (a.res) {
        float r[V];
        Elem<D>::unpack(load_vec<D>((const char *)a.res + (m * a.ldr + n) * E, nv), r);
        for (int j = 0; j < V; ++j) f[j] += r[j];
    }
    store_vec<D>((char *)a.y + (m * a.ldy + n) * E, Elem<D>::pack(f), nv);
}

// 16 bytes to a row; `past`: past the caches.
__device__ inline void put_row(u32x4 v, __amdgpu_buffer_rsrc_t r, uint32_t at, uint32_t past)
{
    if (past)
        __builtin_amdgcn_raw_buffer_store_b128(v, r, at, 0, 2);
    else
        __builtin_amdgcn_raw_buffer_store_b128(v, r, at, 0, 0);
}

// ---- the product -----------------------------------------------------------
constexpr int kStep = 128;                        // bytes of k staged at a time
#define LAGS_INLINE __attribute__((always_inline))    // lambdas that take arrays of registers
enum : int { kDirect = 0, kWords = 1, kHalves = 2 };   // see stage below

// Byte offset of 16-byte vector v of row r in a tile of 128-byte rows: a read of
// one vector column over 16 rows then takes all banks once.
__device__ inline int at_rows(int r, int v) { return r * kStep + ((v ^ (r & 7) ^ (r >> 3 & 3)) << 4); }
// Byte offset of 16-byte vector v of row k in a tile of BN 16-bit columns, for
// transpose reads: 16 lanes take 32 bytes from each of four consecutive rows.
template <int BN> __device__ inline int at_columns(int k, int v)
{
    const int x = BN % 128 == 0 ? k & 3 : k >> 1 & 1;
    return k * BN * 2 + ((v >> 2 ^ x) << 6) + ((v & 3) << 4);
}
// Eight consecutive rows of one column for each lane: lane l holds column cb +
// l % 32, rows kb + 8 (l / 32) + 0..7.
template <int BN> __device__ inline u32x4 transposed(const char *tile, int kb, int cb)
{
    const int l = threadIdx.x & 63, i = l & 15;
    const int k = kb + 8 * (l >> 5) + (i >> 2), c = cb + (l & 16) + (i & 3) * 4;
    typedef __attribute__((address_space(3))) s16x4 lds4;
    const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4 *)(tile + at_columns<BN>(k, c >> 3) + (c & 4) * 2));
    const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4 *)(tile + at_columns<BN>(k + 4, c >> 3) + (c & 4) * 2));
    return __builtin_bit_cast(u32x4, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
}

template <int D> __device__ inline f32x16 multiply(u32x4 w, u32x4 x, f32x16 acc)
{
    if constexpr (D == kBF16)
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, w), __builtin_bit_cast(bf16x8, x), acc, 0, 0, 0);
    else if constexpr (D == kF16)
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, w), __builtin_bit_cast(f16x8, x), acc, 0, 0, 0);
    else {
        for (int t = 0; t < 4; ++t) acc = __builtin_amdgcn_mfma_f32_32x32x2f32(asf(w[t]), asf(x[t]), acc, 0, 0, 0);
        return acc;
    }
}

// 16 bytes of a buffer into LDS at `to`, which the wave shares, lane after lane.
__device__ inline void load_to_lds(__amdgpu_buffer_rsrc_t r, char *to, uint32_t at)
{
#if defined(__HIP_DEVICE_COMPILE__)      // the host pass does not know this size
    typedef __attribute__((address_space(3))) void lds_void;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void *)to, 16, at, 0, 0, 0);
#endif
}
// What the lanes of a wave wrote to LDS before is read by any of them after.
__device__ inline void wave_sync()
{
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

__device__ inline uint32_t deal(uint32_t b, uint32_t n)
{
    const uint32_t per = n / 8, main = per * 8;
    return b < main ? (b & 7) * per + (b >> 3) : b;
}

// A workgroup: a BM x BN tile of the product over one slice of k; WM x WN waves.
// The loop (direct loads): a step is 128 bytes of k, in quarters; a quarter's operands are read
// from LDS between the products of the quarter before, and the loads of steps to come are issued
// between products too, a few at a time, since a burst of them keeps the waves from issuing anything
// else for half a step.  Loads need most of a step to arrive: A has three places in LDS and B two (160 KB
// with 256 x 256), so that B's for the next step but one follow the barrier that frees their place, and A's
// come after them, a step ahead of need.  One barrier a step, before its last quarter.
//   8192 x 8192 x 8192 bf16     772 us, 1.42 PFLOP/s (the library's product 674 to 714; operands of zeros, which
//                               hold the clock up, 550)
//   16384 x 2048 to 8192 bf16   416 to 422 us, 1.3 (373 to 392); with gelu and z 482 to 518: the results of a compute
//                               unit's one workgroup are written between its products, not beside them.  The
//                               matrix units are busy 62 % of that, 78 to 80 % of 16384 x 8192 to 2048
//   8192 x 8192 x 8192 fp32     7310 us, 150 TFLOP/s (7160)
// Products that do not fill whole rounds of 256 tiles, or whose operands are staged through registers, take 1.5 to
// 2.4 times what their operations need: 3230 x 6224 to 5400 bf16 279 us (136 at 1.6 PFLOP/s; the library's 219);
// 16384 x 2048 to 8192 with W one word off a vector 497, one value off 622, of 2049 columns 641.
// NN: B is [k][n].  HOW a tile gets into LDS: kDirect, loads that write it themselves
// (operands of whole, aligned 16-byte vectors); kWords and kHalves, through
// registers, rows that start on any word, or on any half of one (five words are
// read for each vector's four and shifted into place).
template <int D, int BM, int BN, int WM, int WN, bool NN, int HOW>
__global__ __launch_bounds__(64 * WM * WN) void k_linear(LinArgs a)
{
    constexpr int kThreads = 64 * WM * WN;
    constexpr int V = Elem<D>::V, E = Elem<D>::E, KS = kStep / E;
    constexpr int NX = BM / WM / 32, NW = BN / WN / 32;
    constexpr int PA = BM * 8 / kThreads, PB = BN * 8 / kThreads;     // vectors a thread
    constexpr int RV = NN ? BN * E / 16 : 8;                          // vectors a row of B's tile
    constexpr int TA = BM * kStep, BUF = TA + BN * kStep;
    static_assert(BM * 8 % kThreads == 0 && BN * 8 % kThreads == 0, "whole passes");
    extern __shared__ __attribute__((aligned(1024))) char lds[];

    // tiles in bands of eight rows of them, so that those in flight on an XCD share operands in its L2
    const uint32_t b = deal(blockIdx.x, gridDim.x), tiles = a.tm * a.tn, slice = b / tiles, tile = b - slice * tiles;
    const uint32_t band = tile / (8 * a.tn), in = tile - band * 8 * a.tn, high = min(8u, a.tm - band * 8);
    const int64_t m0 = (int64_t)(band * 8 + in % high) * BM;
    const uint32_t n0 = in / high * BN;
    const uint32_t k0 = slice * a.k_per, k1 = min(a.K, k0 + a.k_per);
    const int t = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(t >> 6), lane = t & 63;

    // windows of the operands from this slice's k on; they end with the last valid value
    const int64_t rows = min((int64_t)BM, a.M - m0);
    const char *pa = (const char *)a.a + (m0 * a.lda + k0) * E;
    int64_t la = ((rows - 1) * a.lda + (a.K - k0)) * E;
    const char *pb;
    int64_t lb, step_b;
    if constexpr (NN) {
        pb = (const char *)a.b + ((int64_t)k0 * a.ldb + n0) * E;
        lb = ((int64_t)(k1 - k0 - 1) * a.ldb + (a.N - n0)) * E;
        step_b = KS * a.ldb * E;
    } else {
        pb = (const char *)a.b + ((int64_t)n0 * a.ldb + k0) * E;
        lb = ((int64_t)(min((uint32_t)BN, a.N - n0) - 1) * a.ldb + (a.K - k0)) * E;
        step_b = kStep;
    }
    const int ia = HOW == kHalves ? (int)((uintptr_t)pa & 3) : 0, ib = HOW == kHalves ? (int)((uintptr_t)pb & 3) : 0;
    pa -= ia, pb -= ib;
    if constexpr (HOW == kHalves) la = (la + ia + 3) & ~(int64_t)3, lb = (lb + ib + 3) & ~(int64_t)3;

    // Vector `id` of a tile: the row and vector it holds.  Direct loads write LDS in the order of the
    // lanes, so there the exchange of vectors is applied to what is loaded.
    uint32_t oa[PA], ob[PB];
    auto vec_a = [&](int id) { return HOW == kDirect ? (id & 7) ^ (id >> 3 & 7) ^ (id >> 6 & 3) : id & 7; };
    auto vec_b = [&](int id) {
        if constexpr (!NN) return vec_a(id);
        const int k = id / RV, v = id % RV;
        if constexpr (HOW != kDirect || E == 4) return v;
        return ((v >> 2 ^ (BN % 128 == 0 ? k & 3 : k >> 1 & 1)) << 2) | (v & 3);
    };
#pragma unroll
    for (int p = 0; p < PA; ++p) oa[p] = ia + (uint32_t)((t + p * kThreads) / 8 * a.lda * E) + vec_a(t + p * kThreads) * 16;
#pragma unroll
    for (int p = 0; p < PB; ++p) ob[p] = ib + (uint32_t)((t + p * kThreads) / RV * a.ldb * E) + vec_b(t + p * kThreads) * 16;

    uint32_t k = k0;                                   // what is loaded next
    auto move = [&] { k += KS, pa += kStep, la -= kStep, pb += step_b, lb -= step_b; };
    u32x4 va[HOW == kDirect ? 1 : PA], vb[HOW == kDirect ? 1 : PB];
    uint32_t xa[HOW == kHalves ? PA : 1], xb[HOW == kHalves ? PB : 1];
    int held = 0;                                      // how much of k the registers hold
    auto load = [&] {
        const auto ra = window(pa, la), rb = window(pb, lb);
#pragma unroll
        for (int p = 0; p < PA; ++p) {
            va[p] = __builtin_amdgcn_raw_buffer_load_b128(ra, oa[p] & ~3u, 0, 0);
            if constexpr (HOW == kHalves) xa[p] = __builtin_amdgcn_raw_buffer_load_b32(ra, (oa[p] & ~3u) + 16, 0, 0);
        }
#pragma unroll
        for (int p = 0; p < PB; ++p) {
            vb[p] = __builtin_amdgcn_raw_buffer_load_b128(rb, ob[p] & ~3u, 0, 0);
            if constexpr (HOW == kHalves) xb[p] = __builtin_amdgcn_raw_buffer_load_b32(rb, (ob[p] & ~3u) + 16, 0, 0);
        }
        held = (int)(a.K - k);
        move();
    };
    auto whole = [&](u32x4 &v, uint32_t x, uint32_t o) {
        const uint32_t sh = (o & 2) * 8;
        for (int i = 0; i < 3; ++i) v[i] = __builtin_amdgcn_alignbit(v[i + 1], v[i], sh);
        v[3] = __builtin_amdgcn_alignbit(x, v[3], sh);
    };
    auto cut = [&](u32x4 &v, int n) {                  // all but the first n values
        for (int i = 0; i < 4; ++i) {
            if constexpr (E == 4)
                v[i] = i < n ? v[i] : 0;
            else
                v[i] = 2 * i + 1 < n ? v[i] : 2 * i < n ? v[i] & 0xffffu : 0;
        }
    };
    auto stage = [&](char *buf) {
#pragma unroll
        for (int p = 0; p < PA; ++p) {
            const int id = t + p * kThreads;
            if constexpr (HOW == kHalves) whole(va[p], xa[p], oa[p]);
            if (held < KS) cut(va[p], held - (id & 7) * V);
            *(u32x4 *)(buf + at_rows(id >> 3, id & 7)) = va[p];
        }
#pragma unroll
        for (int p = 0; p < PB; ++p) {
            const int id = t + p * kThreads;
            if constexpr (HOW == kHalves) whole(vb[p], xb[p], ob[p]);
            if constexpr (NN) {
                if (id / RV >= held) vb[p] = u32x4{0, 0, 0, 0};
                *(u32x4 *)(buf + TA + (E == 2 ? at_columns<BN>(id / RV, id % RV) : id * 16)) = vb[p];
            } else {
                if (held < KS) cut(vb[p], held - (id & 7) * V);
                *(u32x4 *)(buf + TA + at_rows(id >> 3, id & 7)) = vb[p];
            }
        }
    };

    const int mw = wave / WN * (BM / WM), nw = wave % WN * (BN / WN);
    f32x16 acc[NW][NX] = {};
    // Operand f of a quarter's products (32 bytes of k; W's first, x's, W's others), and product p.
    auto fetch = [&](const char *ta, const char *tb, int q, int f, u32x4 (&x)[NX], u32x4 (&w)[NW]) LAGS_INLINE {
        const int j = f - 1, i = f == 0 ? 0 : f - NX;
        if (j >= 0 && j < NX) {
            x[j] = *(const u32x4 *)(ta + at_rows(mw + 32 * j + (lane & 31), 2 * q + (lane >> 5)));
            return;
        }
        const int n = nw + 32 * i;
        if constexpr (!NN)
            w[i] = *(const u32x4 *)(tb + at_rows(n + (lane & 31), 2 * q + (lane >> 5)));
        else if constexpr (E == 2)
            w[i] = transposed<BN>(tb, 16 * q, n);
        else
            for (int e = 0; e < 4; ++e)
                w[i][e] = *(const uint32_t *)(tb + ((8 * q + 4 * (lane >> 5) + e) * BN + n + (lane & 31)) * 4);
    };
    constexpr int P = NX * NW, F = NX + NW;
    auto product = [&](int p, u32x4 (&x)[NX], u32x4 (&w)[NW]) LAGS_INLINE {
        acc[p / NX][p % NX] = multiply<D>(w[p / NX], x[p % NX], acc[p / NX][p % NX]);
    };
    if constexpr (HOW == kDirect) {
        const int steps = (int)((k1 - k0 + KS - 1) / KS);
        const auto ra = window(pa, la), rb0 = window(pb, lb);
        const int vec = vec_a(t) * V;
        char *const wa = lds + wave * 1024, *const wb = wa + 3 * TA;
        // loads l0 .. l1 - 1 of step i's rows of A to `to`, or of B
        auto load_a = [&](char *to, int i, int l0, int l1) LAGS_INLINE {
            const uint32_t kv = vec < (int)(k1 - k0) - i * KS ? i * kStep : 0x80000000u;
#pragma unroll
            for (int p = 0; p < PA; ++p)
                if (p >= l0 && p < l1) load_to_lds(ra, to + p * kThreads * 16, oa[p] + kv);
        };
        auto load_b = [&](char *to, int i, int l0, int l1) LAGS_INLINE {
            if constexpr (NN) {
                const auto rb = window(pb + i * step_b, lb - i * step_b);
#pragma unroll
                for (int p = 0; p < PB; ++p)
                    if (p >= l0 && p < l1) load_to_lds(rb, to + p * kThreads * 16, ob[p]);
            } else {
                const uint32_t kv = vec < (int)(k1 - k0) - i * KS ? i * kStep : 0x80000000u;
#pragma unroll
                for (int p = 0; p < PB; ++p)
                    if (p >= l0 && p < l1) load_to_lds(rb0, to + p * kThreads * 16, ob[p] + kv);
            }
        };
        // this wave's loads but the last `left`, its reads of LDS, and everybody else's
        auto arrived = [&](auto left) LAGS_INLINE {
            asm volatile("" ::: "memory");
            __builtin_amdgcn_s_waitcnt(0x0070 | (left & 15) | (left >> 4) << 14);
            __builtin_amdgcn_s_barrier();
            asm volatile("" ::: "memory");
        };
        u32x4 x0[NX], w0[NW], x1[NX], w1[NW];
        // a quarter's products, between them the reads of the next quarter's operands and n loads
        auto quarter = [&](u32x4 (&x)[NX], u32x4 (&w)[NW], const char *ta, const char *tb, int q, u32x4 (&xn)[NX], u32x4 (&wn)[NW],
                           int n, auto ld) LAGS_INLINE {
#pragma unroll
            for (int p = 0; p < P; ++p) {
                product(p, x, w);
#pragma unroll
                for (int f = (p * F + P - 1) / P; f < ((p + 1) * F + P - 1) / P; ++f) fetch(ta, tb, q, f, xn, wn);
                const int l0 = (p * n + P - 1) / P, l1 = ((p + 1) * n + P - 1) / P;
                if (l1 > l0) ld(l0, l1);
            }
            __builtin_amdgcn_sched_barrier(0);
        };
        // steps past the last read as zeros: nobody looks at them
        load_a(wa, 0, 0, PA);
        load_b(wb, 0, 0, PB);
        load_a(wa + TA, 1, 0, PA);
        load_b(wb + BN * kStep, 1, 0, PB);
        arrived(std::integral_constant<int, PA + PB>());
#pragma unroll
        for (int f = 0; f < F; ++f) fetch(lds, lds + 3 * TA, 0, f, x0, w0);
        int ca = 0;                                    // A's place in its ring
        constexpr int H = (PA + 1) / 2;
        for (int s = 0; s < steps; ++s) {
            const int cb = s & 1, na = ca == 2 ? 0 : ca + 1, fa = na == 2 ? 0 : na + 1;
            const char *ta = lds + ca * TA, *tb = lds + 3 * TA + cb * (BN * kStep);
            const char *ta1 = lds + na * TA, *tb1 = lds + 3 * TA + (cb ^ 1) * (BN * kStep);
            char *la2 = wa + fa * TA, *lb2 = wb + cb * (BN * kStep);
            quarter(x0, w0, ta, tb, 1, x1, w1, H, [&](int l0, int l1) LAGS_INLINE { load_a(la2, s + 2, l0, l1); });
            quarter(x1, w1, ta, tb, 2, x0, w0, PA - H, [&](int l0, int l1) LAGS_INLINE { load_a(la2, s + 2, H + l0, H + l1); });
            quarter(x0, w0, ta, tb, 3, x1, w1, 0, [&](int, int) {});
            // all but the loads of A just issued have arrived, everybody has read this step's last operands
            arrived(std::integral_constant<int, PA>());
            quarter(x1, w1, ta1, tb1, 0, x0, w0, PB, [&](int l0, int l1) LAGS_INLINE { load_b(lb2, s + 2, l0, l1); });
            ca = na;
        }
        arrived(std::integral_constant<int, 0>());     // the loads past the last step, before LDS is used again
    } else {
        load();
        stage(lds);
        load();
        int cur = 0;
        for (uint32_t s = k0; s < k1; s += KS) {
            __syncthreads();
            const char *buf = lds + cur * BUF;
            cur ^= 1;
            u32x4 x[NX], w[NW];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                if (q == 2) {
                    stage(lds + cur * BUF);
                    load();
                }
#pragma unroll
                for (int f = 0; f < F; ++f) fetch(buf, buf + TA, q, f, x, w);
#pragma unroll
                for (int p = 0; p < P; ++p) product(p, x, w);
            }
        }
        __syncthreads();
    }

    // Each wave turns 32 rows of 64 (or 32) sums round in LDS of its own, so that a lane has
    // consecutive columns of a row.
    constexpr int CW = NW >= 2 ? 64 : 32, PITCH = CW + 4, QW = CW / 32;
    float *own = (float *)lds + wave * 32 * PITCH;
    constexpr int LR = CW / V, RP = 64 / LR;           // lanes a row, rows at a time
    auto turn = [&](int i0, int j) LAGS_INLINE {
        wave_sync();
#pragma unroll
        for (int i = 0; i < QW; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                *(f32x4 *)(own + (lane & 31) * PITCH + 32 * i + 8 * r + 4 * (lane >> 5)) =
                    f32x4{acc[i0 + i][j][4 * r], acc[i0 + i][j][4 * r + 1], acc[i0 + i][j][4 * r + 2], acc[i0 + i][j][4 * r + 3]};
        wave_sync();
    };
    auto row = [&](int r, float (&f)[V]) LAGS_INLINE {
        for (int e = 0; e < V; e += 4) *(f32x4 *)(f + e) = *(const f32x4 *)(own + r * PITCH + lane % LR * V + e);
    };
    // Rows of whole vectors from whole words go through windows that end with the last row, so that no
    // store stands behind a branch.
    auto rows_at = [&](const void *p, int64_t ld, int e) LAGS_INLINE {
        return window((const char *)p + (m0 * ld + n0) * e, p ? ((rows - 1) * ld + (a.N - n0)) * e : 0);
    };
    auto whole_rows = [&](auto act) LAGS_INLINE {
        const auto ry = rows_at(a.y, a.ldy, E), rz = rows_at(a.z, a.ldz, E), rr = rows_at(a.res, a.ldr, E);
        const auto rb = window(a.bias + n0, a.bias ? (int64_t)(a.N - n0) * 4 : 0);
#pragma unroll
        for (int i0 = 0; i0 < NW; i0 += QW) {
            const uint32_t c = nw + 32 * i0 + lane % LR * V;
            const bool on = n0 + c < a.N;
            float b[V];
            for (int e = 0; e < V; e += 4)
                *(u32x4 *)(b + e) = __builtin_amdgcn_raw_buffer_load_b128(rb, on ? (c + e) * 4 : 0x80000000u, 0, 0);
#pragma unroll
            for (int j = 0; j < NX; ++j) {
                turn(i0, j);
                const uint32_t r1 = mw + 32 * j + lane / LR;
                uint32_t oy = on ? (r1 * (uint32_t)a.ldy + c) * E : 0x80000000u, oz = on ? (r1 * (uint32_t)a.ldz + c) * E : 0x80000000u;
                uint32_t orr = on ? (r1 * (uint32_t)a.ldr + c) * E : 0x80000000u;
#pragma unroll
                for (int r0 = 0; r0 < 32; r0 += RP) {
                    float f[V];
                    row(r0 + lane / LR, f);
                    if (a.bias)
                        for (int e = 0; e < V; ++e) f[e] += b[e];
                    if (a.z) put_row(Elem<D>::pack(f), rz, oz, a.past);
                    if constexpr (act != kActNone)
                        for (int e = 0; e < V; ++e) f[e] = act_value<D>(f[e], act);
                    if (a.res) {
                        float g[V];
                        Elem<D>::unpack(__builtin_amdgcn_raw_buffer_load_b128(rr, orr, 0, 0), g);
                        for (int e = 0; e < V; ++e) f[e] += g[e];
                    }
                    put_row(Elem<D>::pack(f), ry, oy, a.past);
                    oy += RP * (uint32_t)a.ldy * E, oz += RP * (uint32_t)a.ldz * E, orr += RP * (uint32_t)a.ldr * E;
                }
            }
        }
    };
    if (a.whole && a.split == 1) {
        if (a.act == kActRelu)
            whole_rows(std::integral_constant<int, kActRelu>());
        else if (a.act == kActSilu)
            whole_rows(std::integral_constant<int, kActSilu>());
        else if (a.act == kActGelu)
            whole_rows(std::integral_constant<int, kActGelu>());
        else
            whole_rows(std::integral_constant<int, kActNone>());
        return;
    }
#pragma unroll
    for (int j = 0; j < NX; ++j)
#pragma unroll
        for (int i0 = 0; i0 < NW; i0 += QW) {
            turn(i0, j);
            const uint32_t n = n0 + nw + 32 * i0 + lane % LR * V;
            const int nv = (int)a.N - (int)n;
#pragma unroll 1
            for (int r = lane / LR; r < 32; r += RP) {
                const int64_t m = m0 + mw + 32 * j + r;
                float f[V];
                row(r, f);
                if (m >= a.M || nv <= 0) continue;
                if (a.split > 1) {
                    float *out = a.part + ((size_t)slice * a.M + m) * a.N + n;
                    for (int e = 0; e < V; e += 4) store_vec<kF32>(out + e, u32x4{asu(f[e]), asu(f[e + 1]), asu(f[e + 2]), asu(f[e + 3])}, nv - e);
                } else {
                    finish<D>(a, m, n, nv, f);
                }
            }
        }
}

// The slices' sums, in a fixed order, and what becomes of them.
template <int D> __global__ __launch_bounds__(256) void k_linear_join(LinArgs a)
{
    constexpr int V = Elem<D>::V;
    const uint32_t nv = (a.N + V - 1) / V;
    const size_t i = (size_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t m = i / nv;
    const uint32_t n = (uint32_t)(i - (size_t)m * nv) * V;
    if (m >= a.M) return;
    const int left = (int)(a.N - n);
    float f[V] = {};
#pragma unroll 8
    for (uint32_t s = 0; s < a.split; ++s) {
        const float *p = a.part + ((size_t)s * a.M + m) * a.N + n;
        for (int e = 0; e < V; e += 4) {
            const u32x4 v = load_vec<kF32>(p + e, left - e);
            for (int j = 0; j < 4; ++j) f[e + j] += asf(v[j]);
        }
    }
    finish<D>(a, m, n, left, f);
}

// dz = dy act'(z), and its column sums before rounding: part[workgroup row][N].
// 2^tl lanes span a slab of a row; the other lanes and the waves take rows.
template <int D> __global__ __launch_bounds__(256) void k_linear_dz(LinArgs a)
{
    constexpr int V = Elem<D>::V, E = Elem<D>::E;
    __shared__ float sh[4][V][64];
    const uint32_t T = 1u << a.tl, col = threadIdx.x & (T - 1), R = 256 >> a.tl;
    const uint32_t slab = blockIdx.x % a.nslab, chunk = blockIdx.x / a.nslab;
    const uint32_t n = (slab * T + col) * V;
    const int nv = (int)a.N - (int)n;
    const int64_t lo = (int64_t)chunk * a.rows_per, hi = min(a.M, lo + a.rows_per);
    float sum[V] = {};
    // whole: every lane of the wave has a whole vector, so that no load stands behind a branch
    auto pass = [&](auto whole, auto act) {
        constexpr int U = 4;
        const int n_of = whole ? V : nv;
        // dy and z are read once: 189 -> 173 us, 16384 x 8192 bf16 with gelu
        auto once = [&](const char *p) {
            if constexpr (whole) return __builtin_nontemporal_load((const u32x4_u2 *)p);
            return load_vec<D>(p, n_of);
        };
        for (int64_t m = lo + (threadIdx.x >> a.tl); m < hi; m += R * U) {
            u32x4 d[U], z[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t r = min(m + u * R, hi - 1);
                d[u] = once((const char *)a.dy + (r * a.lddy + n) * E);
                if (act) z[u] = once((const char *)a.zin + (r * a.ldz + n) * E);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (m + u * R >= hi) break;
                float f[V];
                Elem<D>::unpack(d[u], f);
                if (act) {
                    float g[V];
                    Elem<D>::unpack(z[u], g);
                    for (int j = 0; j < V; ++j) f[j] *= act_slope<D>(g[j], act);
                    store_vec<D>((char *)a.dz + ((m + u * R) * a.lddz + n) * E, Elem<D>::pack(f), n_of);
                }
                for (int j = 0; j < V; ++j) sum[j] += f[j];
            }
        }
    };
    auto with = [&](auto act) {
        if (__all(nv >= V))
            pass(std::true_type(), act);
        else if (nv > 0)
            pass(std::false_type(), act);
    };
    if (a.act == kActRelu)
        with(std::integral_constant<int, kActRelu>());
    else if (a.act == kActSilu)
        with(std::integral_constant<int, kActSilu>());
    else if (a.act == kActGelu)
        with(std::integral_constant<int, kActGelu>());
    else
        with(std::integral_constant<int, kActNone>());
    if (!a.part && !a.dbias) return;
    for (int j = 0; j < V; ++j) {
        float v = sum[j];
        if (a.tl < 1) v += lane_xor<1>(v);
        if (a.tl < 2) v += lane_xor<2>(v);
        if (a.tl < 3) v += lane_xor<4>(v);
        if (a.tl < 4) v += lane_xor<8>(v);
        if (a.tl < 5) v = swap_sum<16>(v, v);
        if (a.tl < 6) v = swap_sum<32>(v, v);
        sh[threadIdx.x >> 6][j][threadIdx.x & 63] = v;
    }
    __syncthreads();
    if (threadIdx.x < T && nv > 0)
        for (int j = 0; j < V; ++j)
            if (j < nv) {
                const float v = (sh[0][j][col] + sh[1][j][col]) + (sh[2][j][col] + sh[3][j][col]);
                if (a.dbias)
                    a.dbias[n + j] = a.add ? a.dbias[n + j] + v : v;
                else
                    a.part[(size_t)chunk * a.N + n + j] = v;
            }
}

// W [N][K] (a.b, a.ldb) turned round: out [K][N].  A workgroup turns 64 x 64
// values in LDS.  8192 x 2048 bf16 17 us, 3.9 TB/s.
template <int D> __global__ __launch_bounds__(256) void k_linear_turn(LinArgs a, void *out)
{
    static_assert(Elem<D>::E == 2, "");
    __shared__ uint16_t sh[64][66];
    const uint32_t tk = (a.N + 63) / 64, n0 = blockIdx.x / tk * 64, k0 = blockIdx.x % tk * 64;   // a.N: W's columns
    const uint32_t r = threadIdx.x >> 3, v = (threadIdx.x & 7) * 8;
    u32x4 x[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t n = n0 + r + 32 * i;
        x[i] = n < a.K ? load_vec<D>((const uint16_t *)a.b + (int64_t)n * a.ldb + k0 + v, (int)a.N - (int)(k0 + v)) : u32x4{0, 0, 0, 0};
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
        for (int j = 0; j < 4; ++j) *(uint32_t *)&sh[r + 32 * i][v + 2 * j] = x[i][j];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t k = k0 + r + 32 * i;
        u32x4 y;
        for (int j = 0; j < 4; ++j)
            y[j] = (uint32_t)sh[v + 2 * j][r + 32 * i] | (uint32_t)sh[v + 2 * j + 1][r + 32 * i] << 16;
        if (k < a.N) store_vec<D>((uint16_t *)out + (size_t)k * a.K + n0 + v, y, (int)a.K - (int)(n0 + v));
    }
}

// ---- launches --------------------------------------------------------------
template <int D, int BM, int BN, int WM, int WN, bool NN> hipError_t run_linear(const LinArgs &a, int how, hipStream_t s)
{
    constexpr int turn = WM * WN * 32 * (BN / WN >= 64 ? 68 : 36) * 4, ring = (3 * BM + 2 * BN) * kStep;
    constexpr int two = 2 * (BM + BN) * kStep;
    static_assert(two >= turn, "the results' turn fits");
    const int lds = how == kDirect ? ring : two;
    auto k = k_linear<D, BM, BN, WM, WN, NN, kDirect>;
    if (how == kWords) k = k_linear<D, BM, BN, WM, WN, NN, kWords>;
    if constexpr (D != kF32)
        if (how == kHalves) k = k_linear<D, BM, BN, WM, WN, NN, kHalves>;
    if (hipError_t e = allow_lds((const void *)k, lds); e != hipSuccess) return e;
    k<<<a.tm * a.tn * a.split, 64 * WM * WN, lds, s>>>(a);
    return hipGetLastError();
}
template <int D, bool NN> hipError_t run_tile(uint32_t tile, const LinArgs &a, int how, hipStream_t s)
{
    constexpr LinTile t0 = kLinTiles[0], t1 = kLinTiles[1], t2 = kLinTiles[2], t3 = kLinTiles[3];
    switch (tile) {
    case 0: return run_linear<D, t0.bm, t0.bn, t0.wm, t0.wn, NN>(a, how, s);
    case 1: return run_linear<D, t1.bm, t1.bn, t1.wm, t1.wn, NN>(a, how, s);
    case 2: return run_linear<D, t2.bm, t2.bn, t2.wm, t2.wn, NN>(a, how, s);
    case 3: return run_linear<D, t3.bm, t3.bn, t3.wm, t3.wn, NN>(a, how, s);
    }
    return hipErrorInvalidValue;
}

template <int D> hipError_t product(const LinPlan &p, LinArgs a, bool nn, int how, hipStream_t s)
{
    if constexpr (D != kF32)
        if (nn && p.turn && how == kDirect) {
            // a.N columns of W, a.K rows
            k_linear_turn<D><<<((a.K + 63) / 64) * ((a.N + 63) / 64), 256, 0, s>>>(a, a.turned);
            if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
            a.b = a.turned, a.ldb = a.K, nn = false;
        }
    a.tn = p.tn, a.split = p.split, a.k_per = p.k_per;
    constexpr int64_t V = Elem<D>::V, E = Elem<D>::E;
    const LinTile &t = kLinTiles[p.tile];
    const uint64_t vecs = (a.N + V - 1) / V;
    // A launch takes so many rows at most: tiles, and threads that join their slices.  Rows beyond are launches
    // of their own, which take the workspace one after the other; an output's sums do not depend on the cut.
    int64_t most = (int64_t)(kMostThreads / ((uint64_t)64 * t.wm * t.wn * p.tn * p.split)) * t.bm;
    if (a.split > 1) most = std::min(most, (int64_t)((kMostThreads - 255) / vecs));
    for (int64_t left = a.M;;) {
        a.M = std::min(left, most);
        a.tm = (uint32_t)((a.M + t.bm - 1) / t.bm);
        hipError_t e = nn ? run_tile<D, true>(p.tile, a, how, s) : run_tile<D, false>(p.tile, a, how, s);
        if (e == hipSuccess && a.split > 1) {
            k_linear_join<D><<<(uint32_t)(((uint64_t)a.M * vecs + 255) / 256), 256, 0, s>>>(a);
            e = hipGetLastError();
        }
        left -= a.M;
        if (e != hipSuccess || !left) return e;
        a.a = (const char *)a.a + a.M * a.lda * E, a.y = (char *)a.y + a.M * a.ldy * E;
        if (a.z) a.z = (char *)a.z + a.M * a.ldz * E;
        if (a.res) a.res = (const char *)a.res + a.M * a.ldr * E;
    }
}
template <int D> hipError_t slopes(const DzPlan &p, LinArgs a, hipStream_t s)
{
    a.tl = p.tl, a.nslab = p.nslab, a.rows_per = p.rows_per;
    k_linear_dz<D><<<p.nslab * p.chunks, 256, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace lags
