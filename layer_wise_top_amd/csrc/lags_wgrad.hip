// Weight gradient of a linear layer (or 1x1 convolution) whose input was kept
// as an 8-bit checkpoint: dW[o][c] = sum over rows m of dY[m][o] X[m][c].
//
// A value of the checkpoint, q 2^k with |q| <= 127, has seven significant
// bits and is exact in bf16, so the product runs on the bf16 matrix
// instructions with fp32 sums and no rounding of X.  dY is cut into bf16 terms
// that add up to it exactly: one for bf16, two for fp16 (11 bits), three for
// fp32 (24 bits); every product of two terms is exact in fp32, so what is
// rounded is the summation alone.
// Both operands lie with the summed index (rows) slow, so a tile is staged in
// LDS as it comes, X being expanded to bf16 on the way, and is transposed by
// the LDS transpose reads that feed the matrix instructions.
#include "lags_act.h"

#include <type_traits>

namespace lags {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int kThreads = 256;
constexpr int kStep = 32;            // rows staged at a time

template <int D> constexpr int kTerms = D == kBF16 ? 1 : D == kF16 ? 2 : 3;

// Byte offset in a staged [kStep][B] bf16 tile.  A transpose read of 16 lanes
// takes 32 bytes from each of four consecutive rows: the 64-byte blocks of a
// row are exchanged by its number so that those rows fall into different banks.
template <int B> __device__ inline int tile_at(int k, int c)
{
    const int x = B >= 128 ? k & 3 : (k >> 1) & 1;
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
// The leading term is cut, not rounded, so it cannot overflow; what is left
// is exact.  An infinity or NaN is its own leading term with nothing left.
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

__device__ inline uint32_t deal(uint32_t b, uint32_t n)
{
    const uint32_t per = n / 8, main = per * 8;
    return b < main ? (b & 7) * per + (b >> 3) : b;
}

// A workgroup: a BO x BC tile of dW over one slice of the rows; WR x WC waves.
template <int D, int BO, int BC, int WR, int WC>
__global__ __launch_bounds__(kThreads) void k_wgrad(WgradArgs a)
{
    constexpr int V = Elem<D>::V, E = Elem<D>::E, T = kTerms<D>;
    constexpr int VO = BO / V, RA = kThreads / VO, PA = kStep / RA;      // dY: vectors a row, rows a pass, passes
    constexpr int VC = BC / 16, RX = kThreads / VC, PX = RX >= kStep ? 1 : kStep / RX;
    constexpr int NI = BO / WR / 32, NJ = BC / WC / 32;
    constexpr int TA = kStep * BO * 2, TX = kStep * BC * 2, BUF = T * TA + TX;
    extern __shared__ __attribute__((aligned(128))) char lds[];

    uint32_t b = deal(blockIdx.x, gridDim.x);
    const uint32_t tile = b % (a.to * a.tc), slice = b / (a.to * a.tc);
    const uint32_t o0 = tile / a.tc * BO, c0 = tile % a.tc * BC;
    const int64_t lo = slice * a.rows_per, hi = min(a.M, lo + a.rows_per);
    const int t = threadIdx.x, wave = t >> 6, lane = t & 63;
    const int ar = t / VO, ac = t % VO * V, xr = t / VC, xc = t % VC * 16;
    const int an = (int)a.O - (int)(o0 + ac);
    const bool xin = c0 + xc < a.pitch && xr < kStep;
    const char *pa = (const char *)a.dy + ((lo + ar) * a.lddy + o0 + ac) * E;
    const uint8_t *px = a.codes + (lo + xr) * a.pitch + c0 + xc;
    const uint8_t *ps = a.scales + (lo + xr) * a.nrun + (c0 + xc) / kRun;

    u32x4 va[PA], vx[PX];
    uint32_t sx[PX];
    auto load = [&](int64_t m) {
#pragma unroll
        for (int p = 0; p < PA; ++p)
            va[p] = load_vec<D>(pa + p * RA * a.lddy * E, m + ar + p * RA < hi ? an : 0);
#pragma unroll
        for (int p = 0; p < PX; ++p) {
            vx[p] = u32x4{0, 0, 0, 0};
            sx[p] = 0;
            if (xin && m + xr + p * RX < hi) {
                vx[p] = *(const u32x4 *)(px + (int64_t)p * RX * a.pitch);
                sx[p] = ps[(int64_t)p * RX * a.nrun];
            }
        }
        pa += kStep * a.lddy * E;
        px += (int64_t)kStep * a.pitch;
        ps += (int64_t)kStep * a.nrun;
    };
    auto stage = [&](char *buf) {
#pragma unroll
        for (int p = 0; p < PA; ++p) {
            uint32_t w[T][V / 2];
            terms<D, T>(va[p], w);
            for (int k = 0; k < T; ++k) {
                char *q = buf + k * TA + tile_at<BO>(ar + p * RA, ac);
                if constexpr (V == 8)
                    *(u32x4 *)q = u32x4{w[k][0], w[k][1], w[k][V / 2 - 2], w[k][V / 2 - 1]};
                else
                    *(u32x2 *)q = u32x2{w[k][0], w[k][1]};
            }
        }
        if (xr < kStep) {
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
    int cur = 0;
    if (lo < hi) {
        load(lo);
        stage(lds);
    }
    for (int64_t m = lo; m < hi; m += kStep) {
        __syncthreads();
        const bool more = m + kStep < hi;
        if (more) load(m + kStep);
        const char *buf = lds + cur * BUF;
#pragma unroll
        for (int k = 0; k < kStep; k += 16) {
            bf16x8 fx[NJ];
            for (int j = 0; j < NJ; ++j) fx[j] = fragment<BC>(buf + T * TA, k, cj + 32 * j);
            // the smallest terms first
            for (int q = T - 1; q >= 0; --q)
                for (int i = 0; i < NI; ++i) {
                    const bf16x8 fa = fragment<BO>(buf + q * TA, k, oi + 32 * i);
                    for (int j = 0; j < NJ; ++j)
                        acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fa, fx[j], acc[i][j], 0, 0, 0);
                }
        }
        cur ^= 1;
        if (more) stage(lds + cur * BUF);
    }

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

// Sum of the slices, in order.
__global__ __launch_bounds__(256) void k_wgrad_sum(WgradArgs a)
{
    const size_t n = (size_t)a.O * a.C;
    for (size_t i = (size_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (size_t)gridDim.x * 256) {
        float s = 0;
#pragma unroll 8
        for (uint32_t k = 0; k < a.split; ++k) s += a.part[k * n + i];
        a.dw[i] = a.add ? a.dw[i] + s : s;
    }
}

template <int D, int BO, int BC, int WR, int WC> hipError_t run(const WgradArgs &a, hipStream_t s)
{
    constexpr int T = kTerms<D>;
    constexpr int lds = 2 * (T * kStep * BO * 2 + kStep * BC * 2);
    const auto k = k_wgrad<D, BO, BC, WR, WC>;
    if (lds > 65536)
        if (hipError_t e = hipFuncSetAttribute((const void *)k, hipFuncAttributeMaxDynamicSharedMemorySize, lds);
            e != hipSuccess)
            return e;
    k<<<a.to * a.tc * a.split, kThreads, lds, s>>>(a);
    return hipGetLastError();
}

template <int D> hipError_t run_tile(uint32_t tile, const WgradArgs &a, hipStream_t s)
{
    if (tile == 128) return run<D, 128, 128, 2, 2>(a, s);
    return run<D, 64, 64, 2, 2>(a, s);
}

}  // namespace

WgradPlan wgrad_plan(int dtype, int64_t M, int64_t O, int64_t C)
{
    WgradPlan p = {};
    p.tile = O <= 64 || C <= 64 ? 64 : 128;
    p.to = (uint32_t)((O + p.tile - 1) / p.tile);
    p.tc = (uint32_t)((C + p.tile - 1) / p.tile);
    int64_t split = 512 / ((int64_t)p.to * p.tc);
    const int64_t most = (M + 255) / 256;
    if (split > most) split = most;
    if (split < 1) split = 1;
    int64_t per = (M + split - 1) / split;
    per = (per + kStep - 1) / kStep * kStep;
    if (per < kStep) per = kStep;
    p.rows_per = per;
    p.split = (uint32_t)((M + per - 1) / per);
    if (p.split < 1) p.split = 1;
    return p;
}

hipError_t launch_wgrad(const WgradPlan &p, WgradArgs a, int dtype, hipStream_t s)
{
    a.to = p.to, a.tc = p.tc, a.split = p.split, a.rows_per = p.rows_per;
    hipError_t e = dtype == kF32    ? run_tile<kF32>(p.tile, a, s)
                   : dtype == kBF16 ? run_tile<kBF16>(p.tile, a, s)
                                    : run_tile<kF16>(p.tile, a, s);
    if (e != hipSuccess || p.split == 1) return e;
    const size_t n = (size_t)a.O * a.C, g = (n + 255) / 256;
    k_wgrad_sum<<<(uint32_t)(g < 65536 ? g : 65536), 256, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace lags
