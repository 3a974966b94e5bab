// Weight gradient of a linear layer (or 1x1 convolution) whose input was kept
// as an 8-bit checkpoint: dW[o][c] = sum over rows m of dY[m][o] X[m][c].
//
// A value of the checkpoint, q 2^k with |q| <= 127, has seven significant
// bits and is exact in bf16 (2^128 apart, see below), so the product runs on
// the bf16 matrix instructions with fp32 sums and no rounding of X.  dY is cut
// into bf16 terms that add up to it: one for bf16, two for fp16 (11 bits), three
// for fp32 (24 bits, of which bf16 holds those from 2^-133 up: all of them
// where |dY| >= 2^-110); every product of two terms is exact in fp32, so what
// is rounded is the summation alone.
// Both operands lie with the summed index (rows) slow, so a tile is staged in
// LDS as it comes, X being expanded to bf16 on the way, and is transposed by
// the LDS transpose reads that feed the matrix instructions.
#include "lags_act.h"

#include <cmath>
#include <type_traits>

namespace lags {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

template <int D> constexpr int kTerms = D == kBF16 ? 1 : D == kF16 ? 2 : 3;

// Byte offset in a staged [32][B] bf16 tile.  A transpose read of 16 lanes
// takes 32 bytes from each of four consecutive rows: the 64-byte blocks of a
// row are exchanged by its number so that those rows fall into different banks.
template <int B> __device__ inline int tile_at(int k, int c)
{
    const int x = B % 128 == 0 ? k & 3 : (k >> 1) & 1;
    return k * B * 2 + (((c >> 5) ^ x) << 6) + (c & 31) * 2;
}

// Eight consecutive rows of one column for each lane of a 32-column fragment:
// lane l holds column cb + l % 32, rows kb + 8 (l / 32) + 0..7.
template <int B> __device__ inline bf16x8 fragment(const char *tile, int kb, int cb)
{
    const int l = threadIdx.x & 63, i = l & 15;
    const int k = kb + 8 * (l >> 5) + (i >> 2), c = cb + (l & 16) + (i & 3) * 4;
    typedef __attribute__((address_space(3))) s16x4 lds4;
    const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4 *)(tile + tile_at<B>(k, c)));
    const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4 *)(tile + tile_at<B>(k + 4, c)));
    return __builtin_bit_cast(bf16x8, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
}

// The bf16 terms of a vector of dY, eight (or four) columns, two to a word.
// A term is cut, not rounded, so it cannot overflow; what is left is exact.  An infinity or NaN is its own leading term with nothing left.
template <int D, int T> __device__ inline void terms(u32x4 v, uint32_t (&t)[T][Elem<D>::V / 2])
{
    constexpr int V = Elem<D>::V;
    if constexpr (D == kBF16) {
        for (int i = 0; i < 4; ++i) t[0][i] = v[i];
    } else {
        float f[V];
        Elem<D>::unpack(v, f);
        uint32_t h[T][V];
        for (int j = 0; j < V; ++j) {
            const bool finite = __builtin_fabsf(f[j]) < __builtin_inff();
            float r = f[j];
            for (int k = 0; k < T; ++k) {
                h[k][j] = asu(r) & 0xffff0000u;
                r = finite ? r - asf(h[k][j]) : 0.0f;
            }
            if (f[j] != f[j]) h[0][j] = 0x7fc00000u;     // a NaN whose upper payload is zero
        }
        for (int k = 0; k < T; ++k)
            for (int i = 0; i < V / 2; ++i)
                t[k][i] = __builtin_amdgcn_perm(h[k][2 * i + 1], h[k][2 * i], 0x07060302u);
    }
}

// Rounding of fp32 vector operations from here on (the compiler moves nothing
// across): two bits of the mode register, from bit 0.
enum : int { kNearest = 0, kTowardZero = 3 };
template <int MODE> __device__ inline void rounding() { __builtin_amdgcn_s_setreg(1 | (2 - 1) << 11, MODE); }

__device__ inline uint32_t deal(uint32_t b, uint32_t n)
{
    const uint32_t per = n / 8, main = per * 8;
    return b < main ? (b & 7) * per + (b >> 3) : b;
}

// A workgroup: a BO x BC tile of dW over one slice of the rows; WR x WC waves,
// K rows staged at a time.  ODD: rows of 16-bit values that may start inside a
// word (odd pitch, odd slice): five words are read for each vector's four and
// shifted into place.
// The next step's vectors are loaded a step ahead and written to the other half
// of LDS between this step's products.  Few rows and outputs are bound by
// latency, many rows by memory, large products by the LDS reads that feed the
// matrix instructions and the clock that the card holds under them:
//   16384 x 8192 x 2048 bf16   460-490 us, 1.12 to 1.19 PFLOP/s (256 x 256, 64 rows
//                              staged; matrix instructions in 52 % of the cycles);
//                              560 us in the first launches after an idle second
//   8192 x 8192 x 2048 fp16    470-485 us, 1.14 to 1.17 PFLOP/s in two terms (the
//                              256 x 256 kernel spills 5 registers)
//   700 x 6000 x 1500 fp32     50 us, 0.75 PFLOP/s in three terms (192 x 256 on
//                              192 of 256 compute units; 256 x 256 leaves 112 idle)
//   200704 x 256 x 64 bf16     24-27 us, 4.6 to 5.1 TB/s (64 x 64, 126 slices)
//   2048 x 64 x 32 fp32        5.5 us
template <int D, int BO, int BC, int WR, int WC, int K, bool ODD>
__global__ __launch_bounds__(64 * WR * WC) void k_wgrad(WgradArgs a)
{
    constexpr int kThreads = 64 * WR * WC;
    constexpr int V = Elem<D>::V, E = Elem<D>::E, T = kTerms<D>;
    constexpr int VO = BO / V, NA = VO * K, PA = (NA + kThreads - 1) / kThreads;   // dY: vectors a row, in all, passes
    constexpr int VC = BC / 16, RX = kThreads / VC, PX = RX >= K ? 1 : K / RX;
    constexpr int NI = BO / WR / 32, NJ = BC / WC / 32;
    constexpr int TA = K * BO * 2, TX = K * BC * 2, BUF = T * TA + TX;
    extern __shared__ __attribute__((aligned(128))) char lds[];

    uint32_t b = deal(blockIdx.x, gridDim.x);
    const uint32_t tile = b % (a.to * a.tc), slice = b / (a.to * a.tc);
    const uint32_t o0 = tile / a.tc * BO, c0 = tile % a.tc * BC;
    const int64_t lo = slice * a.rows_per, hi = min(a.M, lo + a.rows_per);
    const int t = threadIdx.x, wave = t >> 6, lane = t & 63;
    const int xr = t / VC, xc = t % VC * 16;

    // What is staged next; the windows move with it and end with the slice's last value, so rows
    // past it read as zeros.  dY's window starts and ends on whole words: what else those hold is
    // shifted out, lies in columns past O, which are not stored, or (ODD) in the row after the
    // slice, which stage() clears.
    const char *pa = (const char *)a.dy + (lo * a.lddy + o0) * E;
    const uint8_t *px = a.codes + lo * a.pitch + c0, *ps = a.scales + lo * a.nrun + c0 / kRun;
    int64_t la = hi > lo ? ((hi - lo - 1) * a.lddy + (a.O - o0)) * E : 0;
    int64_t lx = (hi - lo) * a.pitch - c0, ls = (hi - lo) * a.nrun - c0 / kRun;
    const int into = (int)((uintptr_t)pa & 3);
    pa -= into;
    la = (la + into + 3) & ~(int64_t)3;
    // dY's vectors go to the threads in turn (the last pass may not need all); a thread's place in a
    // word is the same every step, K being even
    int vx_at[PX], vs_at[PX];
    uint32_t va_at[PA];
    static_assert(K % 2 == 0, "");
    for (int p = 0; p < PA; ++p) {
        const int id = t + p * kThreads;
        va_at[p] = into + (uint32_t)((id / VO * a.lddy + id % VO * V) * E);
    }
    for (int p = 0; p < PX; ++p) {
        vx_at[p] = (xr + p * RX) * (int)a.pitch + xc;
        vs_at[p] = (xr + p * RX) * (int)a.nrun + xc / (int)kRun;
    }
    u32x4 va[PA], vx[PX];
    uint32_t ve[PA], sx[PX];
    int64_t m = lo - K;                  // the row that the registers start with
    auto load = [&] {
        m += K;
        const auto ra = window(pa, la), rx = window(px, lx), rs = window(ps, ls);
#pragma unroll
        for (int p = 0; p < PA; ++p) {
            va[p] = __builtin_amdgcn_raw_buffer_load_b128(ra, va_at[p] & ~3u, 0, 0);
            if constexpr (ODD) ve[p] = __builtin_amdgcn_raw_buffer_load_b32(ra, (va_at[p] & ~3u) + 16, 0, 0);
        }
#pragma unroll
        for (int p = 0; p < PX; ++p) {
            vx[p] = __builtin_amdgcn_raw_buffer_load_b128(rx, vx_at[p], 0, 0);
            sx[p] = __builtin_amdgcn_raw_buffer_load_b8(rs, vs_at[p], 0, 0);
        }
        pa += K * a.lddy * E, la -= K * a.lddy * E;
        px += (int64_t)K * a.pitch, lx -= (int64_t)K * a.pitch;
        ps += (int64_t)K * a.nrun, ls -= (int64_t)K * a.nrun;
    };
    auto stage_dy = [&](char *buf) {
#pragma unroll
        for (int p = 0; p < PA; ++p) {
            const int id = t + p * kThreads;
            if (NA % kThreads && id >= NA) break;
            uint32_t w[T][V / 2];
            if constexpr (ODD) {
                const uint32_t shift = (va_at[p] & 2) * 8;
                for (int i = 0; i < 3; ++i) va[p][i] = __builtin_amdgcn_alignbit(va[p][i + 1], va[p][i], shift);
                va[p][3] = __builtin_amdgcn_alignbit(ve[p], va[p][3], shift);
                if (m + id / VO >= hi) va[p] = u32x4{0, 0, 0, 0};
            }
            terms<D, T>(va[p], w);
            for (int k = 0; k < T; ++k) {
                char *q = buf + k * TA + tile_at<BO>(id / VO, id % VO * V);
                if constexpr (V == 8)
                    *(u32x4 *)q = u32x4{w[k][0], w[k][1], w[k][V / 2 - 2], w[k][V / 2 - 1]};
                else
                    *(u32x2 *)q = u32x2{w[k][0], w[k][1]};
            }
        }
    };
    auto stage_x = [&](char *buf) {
        if (RX <= K || xr < K) {
#pragma unroll
            for (int p = 0; p < PX; ++p) {
                uint32_t w[8];
                const float step = run_step(sx[p]);
                for (int i = 0; i < 4; ++i) {
                    float f[4];
                    run_values(vx[p][i], step, f);
                    w[2 * i] = __builtin_amdgcn_perm(asu(f[1]), asu(f[0]), 0x07060302u);
                    w[2 * i + 1] = __builtin_amdgcn_perm(asu(f[3]), asu(f[2]), 0x07060302u);
                }
                char *q = buf + T * TA + tile_at<BC>(xr + p * RX, xc);
                *(u32x4 *)q = u32x4{w[0], w[1], w[2], w[3]};
                *(u32x4 *)(q + 16) = u32x4{w[4], w[5], w[6], w[7]};
            }
        }
    };

    const int oi = wave / WC * (BO / WR), cj = wave % WC * (BC / WC);
    f32x16 acc[NI][NJ] = {};
    auto multiply = [&](const char *buf, int k) {
        bf16x8 fx[NJ];
#pragma unroll
        for (int j = 0; j < NJ; ++j) fx[j] = fragment<BC>(buf + T * TA, k, cj + 32 * j);
        // the smallest terms first
#pragma unroll
        for (int q = T - 1; q >= 0; --q)
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                const bf16x8 fa = fragment<BO>(buf + q * TA, k, oi + 32 * i);
#pragma unroll
                for (int j = 0; j < NJ; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fa, fx[j], acc[i][j], 0, 0, 0);
            }
    };
    int cur = 0;
    // What staging computes is exact but for one value, 64 steps of 2^122 (which finite magnitudes from
    // 127.5/128 2^128 up round to): cut, it is the largest bf16 value; rounded, it would be an infinity,
    // and NaN where dY is zero.  The matrix instructions have a rounding of their own.
    rounding<kTowardZero>();
    load();
    stage_dy(lds);
    stage_x(lds);
    load();
    for (int64_t step = lo; step < hi; step += K) {
        __syncthreads();
        const char *buf = lds + cur * BUF;
        cur ^= 1;
        // The next step's tiles, loaded while the last step ran, are staged between this one's products.
        // The fences keep the pieces apart: left alone the compiler gathers the LDS reads and the loads
        // at the end, where the matrix unit waits for them (8192 x 2048 over 16384 rows: 505 us; so 490).
        multiply(buf, 0);
        stage_dy(lds + cur * BUF);
        if constexpr (K >= 64) {
            __builtin_amdgcn_sched_barrier(0);
            multiply(buf, 16);
        }
        stage_x(lds + cur * BUF);
        load();
#pragma unroll
        for (int k = K >= 64 ? 32 : 16; k < K; k += 16) {
            __builtin_amdgcn_sched_barrier(0);
            multiply(buf, k);
        }
    }

    rounding<kNearest>();
    float *out = a.split > 1 ? a.part + (size_t)slice * a.O * a.C : a.dw;
    const bool add = a.split == 1 && a.add;
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            const uint32_t c = c0 + cj + 32 * j + (lane & 31);
            if (c >= a.C) continue;
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const uint32_t o = o0 + oi + 32 * i + (r >> 2) * 8 + (lane >> 5) * 4 + (r & 3);
                if (o >= a.O) continue;
                float *p = out + (size_t)o * a.C + c;
                *p = add ? *p + acc[i][j][r] : acc[i][j][r];
            }
        }
}

// Sum of the slices, in a fixed order: a workgroup takes 256 values of dW, its
// W waves each a run of the slices.  Bound by a launch and a trip to memory:
// 4.7 us for 126 slices of 256 x 64.
template <int W> __global__ __launch_bounds__(64 * W) void k_wgrad_sum(WgradArgs a)
{
    __shared__ f32x4 sh[W][64];
    const size_t n = (size_t)a.O * a.C, i = ((size_t)blockIdx.x * 64 + (threadIdx.x & 63)) * 4;
    const uint32_t w = threadIdx.x >> 6;
    const uint32_t k0 = w * a.split / W, k1 = (w + 1) * a.split / W;
    f32x4 s = {0, 0, 0, 0};
    if (i + 4 <= n) {
#pragma unroll 8
        for (uint32_t k = k0; k < k1; ++k) s += *(const f32x4_u4 *)(a.part + k * n + i);
    } else {
        for (uint32_t k = k0; k < k1; ++k)
            for (int j = 0; j < 3; ++j)
                if (i + j < n) s[j] += a.part[k * n + i + j];
    }
    sh[w][threadIdx.x & 63] = s;
    __syncthreads();
    if (w) return;
    for (int k = 1; k < W; ++k) s += sh[k][threadIdx.x];
    if (i + 4 <= n) {
        f32x4_u4 *p = (f32x4_u4 *)(a.dw + i);
        *p = a.add ? *p + s : s;
    } else {
        for (int j = 0; j < 3; ++j)
            if (i + j < n) a.dw[i + j] = a.add ? a.dw[i + j] + s[j] : s[j];
    }
}

template <int D, int BO, int BC, int WR, int WC, int K> hipError_t run(const WgradArgs &a, hipStream_t s)
{
    constexpr int T = kTerms<D>;
    constexpr int lds = 2 * (T * K * BO * 2 + K * BC * 2);
    bool odd = false;
    if constexpr (D != kF32) odd = (((uintptr_t)a.dy | (uint64_t)a.lddy * Elem<D>::E) & 3) != 0;
    auto k = k_wgrad<D, BO, BC, WR, WC, K, false>;
    if constexpr (D != kF32)
        if (odd) k = k_wgrad<D, BO, BC, WR, WC, K, true>;
    if (hipError_t e = allow_lds((const void *)k, lds); e != hipSuccess) return e;
    k<<<a.to * a.tc * a.split, 64 * WR * WC, lds, s>>>(a);
    return hipGetLastError();
}

// The tiles, and the time (ns) that one takes a row on a compute unit that is
// full of them, for one, two and three terms; `alone`: when it is the only one.
// Measured with 8192 x 2048 outputs over 4096 to 16384 rows, and with one
// workgroup a unit over 200704 rows.  No time: not built (256 x 64 in three
// terms took 57 ns, four of 64 x 64 take 44).
struct Tile {
    int bo, bc;
    float full[3], alone[3];
};
constexpr Tile kTiles[] = {
    {256, 256, {32.0f, 58.0f, 91.0f}, {31.0f, 50.0f, 80.0f}},
    {192, 256, {25.0f, 45.0f, 70.0f}, {25.0f, 40.0f, 62.0f}},
    {128, 128, {10.4f, 20.0f, 27.5f}, {20.0f, 25.0f, 35.0f}},
    {256, 64, {11.0f, 27.0f, 0}, {20.0f, 40.0f, 0}},
    {64, 256, {11.5f, 20.0f, 26.0f}, {20.0f, 25.0f, 31.0f}},
    {64, 64, {4.3f, 7.4f, 11.0f}, {8.5f, 12.0f, 17.0f}},
};
template <int D> hipError_t run_tile(uint32_t tile, const WgradArgs &a, hipStream_t s)
{
    constexpr int K = D == kBF16 ? 64 : 32;
    switch (tile) {
    case 0: return run<D, 256, 256, 2, 4, K>(a, s);
    case 1: return run<D, 192, 256, 2, 4, K>(a, s);
    case 2: return run<D, 128, 128, 2, 2, K>(a, s);
    case 3:
        if constexpr (D != kF32) return run<D, 256, 64, 4, 1, K>(a, s);
        break;
    case 4: return run<D, 64, 256, 1, 4, K>(a, s);
    case 5: return run<D, 64, 64, 2, 2, 64>(a, s);
    }
    return hipErrorInvalidValue;
}

}  // namespace

// The tile and the number of row slices with the least time by a model of it:
// the rounds of workgroups on 256 compute units, or the bytes of the operands,
// then dW once, or the slices' sums written and read again.
WgradPlan wgrad_plan(int dtype, int64_t M, int64_t O, int64_t C)
{
    const int terms = dtype == kBF16 ? 0 : dtype == kF16 ? 1 : 2;
    const double in = (double)M * (O * elem_bytes(dtype) + C * 1.04) / 4800, out = (double)O * C * 4;
    WgradPlan best = {};
    double least = 0;
    for (uint32_t t = 0; t < sizeof(kTiles) / sizeof(kTiles[0]); ++t) {
        if (!kTiles[t].full[terms]) continue;
        WgradPlan p = {};
        p.tile = t;
        p.to = (uint32_t)((O + kTiles[t].bo - 1) / kTiles[t].bo);
        p.tc = (uint32_t)((C + kTiles[t].bc - 1) / kTiles[t].bc);
        const double tiles = (double)p.to * p.tc;
        // a dW above 2^32 values is not sliced: its sum would be more threads than a launch has
        const int64_t slices = O * C > (int64_t)1 << 32 ? 1 : 512;
        for (int64_t want = 1; want <= slices; want = want < 4 ? want + 1 : want % 3 ? want + want / 2 : want / 3 * 4) {
            int64_t per = ((M + want - 1) / want + 63) / 64 * 64;
            if (per < 64) per = 64;
            p.rows_per = per;
            p.split = (uint32_t)((M + per - 1) / per);
            if (p.split < 1) p.split = 1;
            const double n = std::ceil(tiles * p.split / 256);
            const double rows = (double)(p.split > 1 ? per : M);
            const double uneven = tiles * p.split > 256 ? n * 256 / (tiles * p.split) : 1;
            double ns = std::fmax(rows * std::fmax(n * kTiles[t].full[terms], kTiles[t].alone[terms]), in * uneven);
            ns += p.split > 1 ? 3500 + out * (2 * p.split + 1) / 7500 : out / 5000;
            if (!least || ns < least) least = ns, best = p;
            if (want > 1 && (per == 64 || tiles * want > 4096)) break;
        }
    }
    return best;
}

hipError_t launch_wgrad(const WgradPlan &p, WgradArgs a, int dtype, hipStream_t s)
{
    a.to = p.to, a.tc = p.tc, a.split = p.split, a.rows_per = p.rows_per;
    hipError_t e = dtype == kF32    ? run_tile<kF32>(p.tile, a, s)
                   : dtype == kBF16 ? run_tile<kBF16>(p.tile, a, s)
                                    : run_tile<kF16>(p.tile, a, s);
    if (e != hipSuccess || p.split == 1) return e;
    const uint32_t g = (uint32_t)(((size_t)a.O * a.C + 255) / 256);
    if (p.split >= 32)
        k_wgrad_sum<16><<<g, 1024, 0, s>>>(a);
    else if (p.split >= 4)
        k_wgrad_sum<4><<<g, 256, 0, s>>>(a);
    else
        k_wgrad_sum<2><<<g, 128, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace lags
