// Layer normalisation, both directions: s = x + res (rounded to the type), y =
// (s - mean) rstd gamma + beta over the channels of each row;  backward: with
// g = gamma dy and xh = (s - mean) rstd, dx = rstd (g - <g> - xh <g xh>) + dsum,
// < > the mean over the row, dgamma = sum dy xh and dbeta = sum dy over the rows.
//
// Bound by memory: a row is read once and held in registers, 32 values a lane
// at most.  Up to 2048 channels are a wave's or less (several rows a wave up to
// 32 lanes' worth), so that its sums are lane exchanges without a barrier; wider
// rows are a workgroup's.  Workgroups walk the rows with gamma and beta, and
// backward the channel sums, in registers; the next rows are requested before
// this one's sums.
//   16384 x 2048 bf16, forward with a residual   50 us, 5.3 TB/s (a large copy reaches 5.1)
//   the same, backward from a checkpoint         54 us, 4.4 TB/s, 5 of it the parameters' last sum
//   16384 x 2048 fp32                            forward 101 us, backward 106, 5.2 TB/s
//   700 x 1500 fp32, backward                    12 us: 10 for 175 workgroups, a row a wave and less than a
//                                                wave a SIMD, then the parameters' last sum
//   4000 x 8190 bf16                             forward 46 us, backward 53 (45 from a checkpoint at a copy's rate)
//   2000 x 16384 bf16                            forward 47 us, backward 119 (45)
//   2000 x 16384 fp32                            forward 114 us, backward 215 (102 each)
// 8193 channels and more: 1024 threads have 128 registers, and the fp32 forward spills 19 of them, the
// backward 23 to 44 (16 bits) and 81 to 86 (fp32).
#include "lags_layer.h"
#include "lags_gn.h"

#include <algorithm>

namespace lags {
namespace {

template <int D, int NV, bool WIDE, int EDGE> struct Row {
    static constexpr int V = Elem<D>::V, E = Elem<D>::E;
    uint32_t T, col, sub, R;             // lanes a row, this one's place, its row of the R at a time
    uint32_t C;
    int nv[NV];                          // channels of each vector (<= 0: idle)
    __device__ explicit Row(const LnArgs &a)
    {
        T = 1u << a.tl, C = a.C;
        col = threadIdx.x & (T - 1);
        sub = WIDE ? 0 : (threadIdx.x & 63) >> a.tl;
        R = WIDE ? 1 : 64 >> a.tl;
        for (int k = 0; k < NV; ++k) nv[k] = (int)C - (int)((col + k * T) * V);
    }
    __device__ uint32_t chan(int k) const { return (col + k * T) * V; }
    // this lane's vectors of rows row0 .. row0 + n - 1 (row0 + sub of them)
    __device__ void load(const void *base, int64_t row0, uint32_t n, int64_t ld, u32x4 (&v)[NV]) const
    {
        const char *p = (const char *)base + row0 * ld * E;
        const uint32_t into = EDGE == kShifted ? (uint32_t)((uintptr_t)p & 3) : 0;
        const auto r = window(p - into, n ? (((int64_t)(n - 1) * ld + C) * E + into + 3) & ~(int64_t)3 : 0);
        const uint32_t o = into + sub * (uint32_t)(ld * E);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const uint32_t at = nv[k] > 0 ? o + chan(k) * E : 0x80000000u;
            if constexpr (EDGE == kShifted) {
                v[k] = __builtin_amdgcn_raw_buffer_load_b128(r, at & ~3u, 0, 0);
                const uint32_t e = __builtin_amdgcn_raw_buffer_load_b32(r, (at & ~3u) + 16, 0, 0), sh = (at & 2) * 8;
                for (int i = 0; i < 3; ++i) v[k][i] = __builtin_amdgcn_alignbit(v[k][i + 1], v[k][i], sh);
                v[k][3] = __builtin_amdgcn_alignbit(e, v[k][3], sh);
                if (sub >= n) v[k] = u32x4{0, 0, 0, 0};   // the word that ends the last row may start another
            } else {
                v[k] = __builtin_amdgcn_raw_buffer_load_b128(r, at, 0, 0);
            }
        }
    }
    // the values of a vector; those past the last channel are `past`
    __device__ void values(u32x4 v, int k, float (&f)[V], float past = 0.0f) const
    {
        Elem<D>::unpack(v, f);
        if constexpr (EDGE != kWhole)
            for (int j = 0; j < V; ++j) f[j] = j < nv[k] ? f[j] : past;
    }
    __device__ void store(void *base, int64_t row, int64_t ld, int k, u32x4 v) const
    {
        char *p = (char *)base + (row * ld + chan(k)) * E;
        if constexpr (EDGE != kWhole)
            store_vec<D>(p, v, nv[k]);
        else if (nv[k] > 0)
            *(u32x4_u2 *)p = v;
    }
    __device__ void param(const float *p, float other, float (&f)[NV][V]) const
    {
        const auto r = window(p, p ? (int64_t)C * 4 : 0);
#pragma unroll
        for (int k = 0; k < NV; ++k)
            for (int i = 0; i < V / 4; ++i) {
                const u32x4 v = __builtin_amdgcn_raw_buffer_load_b128(r, nv[k] > 0 ? chan(k) * 4 + 16 * i : 0x80000000u, 0, 0);
                for (int j = 0; j < 4; ++j) f[k][4 * i + j] = p ? asf(v[j]) : other;
            }
    }
};

// Sums over a row's lanes, on each of them.  Wide rows join their waves'
// through sh[slot]; two sums of one row, and the last of one row and the first
// of the next, take different slots, so one barrier each is enough.
template <bool WIDE> __device__ inline void row_sums(float &a, float &b, uint32_t tl, float2 (*sh)[16], int slot)
{
    auto lanes = [&](float s) {
        s += lane_xor<1>(s);
        s += lane_xor<2>(s);
        s += lane_xor<4>(s);
        if (WIDE || tl > 3) s += lane_xor<8>(s);
        if (WIDE || tl > 4) s = swap_sum<16>(s, s);
        if (WIDE || tl > 5) s = swap_sum<32>(s, s);
        return s;
    };
    a = lanes(a), b = lanes(b);
    if constexpr (WIDE) {
        const uint32_t lane = threadIdx.x & 63, waves = blockDim.x >> 6;
        if (lane == 0) sh[slot][threadIdx.x >> 6] = make_float2(a, b);
        __syncthreads();
        const float2 p = sh[slot][lane & 15];
        a = wave_sum(lane < waves ? p.x : 0.0f), b = wave_sum(lane < waves ? p.y : 0.0f);
    }
}

// A vector's codes, and its run's scale byte from the run's first lane.
template <int D> __device__ inline void write_codes(uint8_t *codes, uint8_t *scales, uint32_t c, uint32_t C,
                                                    uint32_t pitch, bool row, u32x4 raw)
{
    constexpr int V = Elem<D>::V;
    float f[V];
    Elem<D>::unpack(raw, f);
    const uint32_t s = run_scale(run_top<V>(Elem<D>::top(raw)));
    uint32_t q[V / 4];
    run_codes<V>(f, s, q);
    if (!row) return;
    if (c < pitch) {
        if constexpr (V == 8)
            *(u32x2 *)(codes + c) = u32x2{q[0], q[V / 4 - 1]};
        else
            *(uint32_t *)(codes + c) = q[0];
    }
    if (c % kRun == 0 && c < C) scales[c / kRun] = (uint8_t)s;
}

template <int D, int NV, int MOST, int EDGE> __global__ __launch_bounds__(MOST ? MOST : 256) void k_ln_forward(LnArgs a)
{
    constexpr bool WIDE = MOST != 0;
    constexpr int V = Elem<D>::V;
    __shared__ float2 sh[2][16];
    const Row<D, NV, WIDE, EDGE> row(a);
    float gamma[NV][V], beta[NV][V];
    row.param(a.gamma, 1.0f, gamma);
    row.param(a.beta, 0.0f, beta);
    const int64_t per = WIDE ? 1 : 4 * row.R, step = per * gridDim.x;
    int64_t r0 = per * blockIdx.x + (WIDE ? 0 : row.R * __builtin_amdgcn_readfirstlane(threadIdx.x >> 6));
    u32x4 x[NV], res[NV];
    auto load = [&](int64_t r) {
        const uint32_t n = r < a.rows ? (uint32_t)min((int64_t)row.R, a.rows - r) : 0;
        const int64_t at = n ? r : 0;
        row.load(a.x, at, n, a.ldx, x);
        if (a.res) row.load(a.res, at, n, a.ldr, res);
    };
    load(r0);
    for (; r0 < a.rows; r0 += step) {
        const int64_t r = r0 + row.sub;
        const bool on = r < a.rows;
        float f[NV][V];
#pragma unroll
        for (int k = 0; k < NV; ++k) row.values(x[k], k, f[k]);
        if (a.res) {
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                float b[V];
                row.values(res[k], k, b);
                for (int j = 0; j < V; ++j) f[k][j] += b[j];
                const u32x4 s = Elem<D>::pack(f[k]);
                Elem<D>::unpack(s, f[k]);              // the norm is that of the sum as it is held
                if (a.sum && on) row.store(a.sum, r, a.lds, k, s);
            }
        }
        load(r0 + step);
        // Sums of values by 2^-14 cannot overflow (the factor is exact, and a row has 2^14 values at
        // most).  What the first mean is off by, e, is taken out of the variance, and where the mean
        // exceeds the spread also out of the mean, so a large common offset costs no digits; below that e
        // is as uncertain as the mean itself.
        float m = 0, none = 0;
#pragma unroll
        for (int k = 0; k < NV; ++k)
            for (int j = 0; j < V; ++j) m = __builtin_fmaf(f[k][j], 0x1p-14f, m);
        row_sums<WIDE>(m, none, a.tl, sh, 0);
        const float count = (float)a.C;
        m = m / (count * 0x1p-14f);
        float e = 0, q = 0;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            float ek = 0, qk = 0;
            for (int j = 0; j < V; ++j) {
                const float d = EDGE == kWhole || j < row.nv[k] ? f[k][j] - m : 0.0f;
                ek = __builtin_fmaf(d, 0x1p-14f, ek), qk = __builtin_fmaf(d, d, qk);
            }
            e += row.nv[k] > 0 ? ek : 0.0f, q += row.nv[k] > 0 ? qk : 0.0f;
        }
        row_sums<WIDE>(e, q, a.tl, sh, 1);
        e = e / (count * 0x1p-14f), q = q / count;
        const float v = __builtin_fmaf(-e, e, q);
        const float mean = m * m > v ? m + e : m;
        const float rstd = 1.0f / __builtin_sqrtf((v < 0 ? 0.0f : v) + a.eps);
        if (row.col == 0 && on) {
            if (a.mean) a.mean[r] = mean;
            if (a.rstd) a.rstd[r] = rstd;
        }
        if (a.wcodes)
#pragma unroll
            for (int k = 0; k < NV; ++k)
                write_codes<D>(a.wcodes + r * a.pitch, a.wscales + r * a.nrun, row.chan(k), a.C, a.pitch, on,
                               Elem<D>::pack(f[k]));
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            for (int j = 0; j < V; ++j)
                f[k][j] = __builtin_fmaf((f[k][j] - mean) * rstd, gamma[k][j], beta[k][j]);
            const u32x4 y = Elem<D>::pack(f[k]);
            if (on) row.store(a.y, r, a.ldy, k, y);
            if (a.ycodes) {
                float h[V];
                row.values(y, k, h);
                const u32x4 held = row.nv[k] > 0 ? Elem<D>::pack(h) : u32x4{0, 0, 0, 0};
                write_codes<D>(a.ycodes + r * a.pitch, a.yscales + r * a.nrun, row.chan(k), a.C, a.pitch, on, held);
            }
        }
    }
}

// CK: s comes as its checkpoint.
template <int D, int NV, int MOST, int EDGE, bool CK>
__global__ __launch_bounds__(MOST ? MOST : 256) void k_ln_backward(LnArgs a)
{
    constexpr bool WIDE = MOST != 0;
    constexpr int V = Elem<D>::V;
    __shared__ float2 sh[2][16];
    const Row<D, NV, WIDE, EDGE> row(a);
    float gamma[NV][V], dg[NV][V] = {}, db[NV][V] = {};
    row.param(a.gamma, 1.0f, gamma);
    const int64_t per = WIDE ? 1 : 4 * row.R, step = per * gridDim.x;
    int64_t r0 = per * blockIdx.x + (WIDE ? 0 : row.R * __builtin_amdgcn_readfirstlane(threadIdx.x >> 6));
    u32x4 dy[NV], ds[NV], x[CK ? 1 : NV];
    u32x2 q[CK ? NV : 1];
    uint32_t sc[CK ? NV : 1];
    float mean, rstd;
    auto load = [&](int64_t r) {
        const uint32_t n = r < a.rows ? (uint32_t)min((int64_t)row.R, a.rows - r) : 0;
        const int64_t at = n ? r : 0;
        row.load(a.dy, at, n, a.lddy, dy);
        if (a.dsum) row.load(a.dsum, at, n, a.ldds, ds);
        if constexpr (CK) {
            const auto rc = window(a.rcodes + at * a.pitch, (int64_t)n * a.pitch);
            const auto rs = window(a.rscales + at * a.nrun, (int64_t)n * a.nrun);
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const uint32_t c = row.chan(k);
                const uint32_t o = row.nv[k] > 0 ? row.sub * a.pitch + c : 0x80000000u;
                if constexpr (V == 8)
                    q[k] = __builtin_amdgcn_raw_buffer_load_b64(rc, o, 0, 0);
                else
                    q[k][0] = __builtin_amdgcn_raw_buffer_load_b32(rc, o, 0, 0);
                sc[k] = __builtin_amdgcn_raw_buffer_load_b8(
                    rs, row.nv[k] > 0 ? row.sub * a.nrun + c / kRun : 0x80000000u, 0, 0);
            }
        } else {
            row.load(a.x, at, n, a.ldx, x);
        }
        const auto rm = window(a.mean + at, (int64_t)n * 4), rr = window(a.rstd + at, (int64_t)n * 4);
        mean = asf(__builtin_amdgcn_raw_buffer_load_b32(rm, row.sub * 4, 0, 0));
        rstd = asf(__builtin_amdgcn_raw_buffer_load_b32(rr, row.sub * 4, 0, 0));
    };
    load(r0);
    for (int slot = 0; r0 < a.rows; r0 += step, slot ^= 1) {
        const int64_t r = r0 + row.sub;
        float g[NV][V], xh[NV][V], s1 = 0, s2 = 0;
        u32x4 add[NV];
        const float rs = rstd;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            float d[V];
            row.values(dy[k], k, d);
            // Columns past the last channel have s = mean and xh = 0: with s = 0, as loaded, -mean * rstd may be
            // infinite (a constant row far from zero) and would make the row's second sum 0 * inf.
            if constexpr (CK) {
                for (int i = 0; i < V / 4; ++i) run_values(q[k][i], run_step(sc[k]), xh[k] + 4 * i);
                if constexpr (EDGE != kWhole)
                    for (int j = 0; j < V; ++j) xh[k][j] = j < row.nv[k] ? xh[k][j] : mean;
            } else {
                row.values(x[k], k, xh[k], mean);
            }
            const float mu = EDGE == kWhole && row.nv[k] <= 0 ? 0.0f : mean;
            for (int j = 0; j < V; ++j) {
                xh[k][j] = (xh[k][j] - mu) * rs;
                db[k][j] += d[j];
                dg[k][j] = __builtin_fmaf(d[j], xh[k][j], dg[k][j]);
                g[k][j] = d[j] * gamma[k][j];
                s1 += g[k][j];
                s2 = __builtin_fmaf(g[k][j], xh[k][j], s2);
            }
            add[k] = ds[k];
        }
        load(r0 + step);
        row_sums<WIDE>(s1, s2, a.tl, sh, slot);
        s1 *= a.inv_c, s2 *= a.inv_c;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            for (int j = 0; j < V; ++j) g[k][j] = rs * (g[k][j] - s1 - xh[k][j] * s2);
            if (a.dsum) {
                float b[V];
                Elem<D>::unpack(add[k], b);
                for (int j = 0; j < V; ++j) g[k][j] += b[j];
            }
            if (r < a.rows) row.store(a.dx, r, a.lddx, k, Elem<D>::pack(g[k]));
        }
    }
    if (!a.part) return;
    // a workgroup's sums go to its place, or, where it is the only one, to the gradients
    float *out = a.part + (size_t)blockIdx.x * 2 * a.C;
    auto put = [&](int which, uint32_t c, float v) {
        if (gridDim.x > 1) {
            out[which * a.C + c] = v;
        } else if (float *g = which ? a.dgamma : a.dbeta) {
            g[c] = a.add ? g[c] + v : v;
        }
    };
    if constexpr (WIDE) {
#pragma unroll
        for (int k = 0; k < NV; ++k)
            for (int j = 0; j < V; ++j)
                if (j < row.nv[k]) {
                    put(0, row.chan(k) + j, db[k][j]);
                    put(1, row.chan(k) + j, dg[k][j]);
                }
    } else {
        // the rows side by side in a wave, then the four waves
        __shared__ float join[4][NV * V][64];
        for (int which = 0; which < 2; ++which) {
#pragma unroll
            for (int k = 0; k < NV; ++k)
                for (int j = 0; j < V; ++j) {
                    float v = which ? dg[k][j] : db[k][j];
                    if (a.tl < 4) v += lane_xor<8>(v);
                    if (a.tl < 5) v = swap_sum<16>(v, v);
                    if (a.tl < 6) v = swap_sum<32>(v, v);
                    join[threadIdx.x >> 6][k * V + j][threadIdx.x & 63] = v;
                }
            __syncthreads();
            for (uint32_t c = threadIdx.x; c < a.C; c += 256) {
                const uint32_t v = c / V, l = v & (row.T - 1), i = (v >> a.tl) * V + c % V;
                put(which, c, (join[0][i][l] + join[1][i][l]) + (join[2][i][l] + join[3][i][l]));
            }
            __syncthreads();
        }
    }
}

// The kernel of a plan: vectors a lane, threads of a row's workgroup at most (0: a
// wave takes whole rows), and what the edges ask for.
template <int D, typename F> hipError_t by_plan(const LnPlan &p, int edge, F f)
{
    auto with = [&](auto nv, auto most) {
        if constexpr (D != kF32)
            if (edge == kShifted) return f(nv, most, std::integral_constant<int, kShifted>());
        if (edge != kWhole) return f(nv, most, std::integral_constant<int, kRagged>());
        return f(nv, most, std::integral_constant<int, kWhole>());
    };
    auto wide = [&](auto most) {
        if (D == kF32 && p.nv > 2) return with(std::integral_constant<int, D == kF32 ? 4 : 2>(), most);
        if (p.nv > 1) return with(std::integral_constant<int, 2>(), most);
        return with(std::integral_constant<int, 1>(), most);
    };
    if (p.tl > 9) return wide(std::integral_constant<int, 1024>());
    if (p.tl > 8) return wide(std::integral_constant<int, 512>());
    if (p.tl > 6) return wide(std::integral_constant<int, 256>());
    const std::integral_constant<int, 0> most;
    if (p.nv <= 1) return with(std::integral_constant<int, 1>(), most);
    if (p.nv <= 2) return with(std::integral_constant<int, 2>(), most);
    if constexpr (D == kF32)
        if (p.nv > 4) return with(std::integral_constant<int, 8>(), most);
    return with(std::integral_constant<int, 4>(), most);
}

template <int D> hipError_t forward(const LnPlan &p, const LnArgs &a, int edge, hipStream_t s)
{
    return by_plan<D>(p, edge, [&](auto nv, auto most, auto e) {
        k_ln_forward<D, nv, most, e><<<p.groups, p.threads, 0, s>>>(a);
        return hipGetLastError();
    });
}
template <int D> hipError_t backward(const LnPlan &p, const LnArgs &a, int edge, hipStream_t s)
{
    return by_plan<D>(p, edge, [&](auto nv, auto most, auto e) {
        return by_bool(a.rcodes != nullptr, [&](auto ck) {
            k_ln_backward<D, nv, most, e, ck><<<p.groups, p.threads, 0, s>>>(a);
            return hipGetLastError();
        });
    });
}

}  // namespace

// Lanes a row: a power of two, 8 at least (a run of a checkpoint is 8 lanes of
// fp32).  Up to a wave's vectors one a lane; up to 2048 channels a wave with 32
// values a lane; beyond, or backward with rows shifted into place (whose further
// registers would spill), a workgroup of 16 a lane.  us for 16384 rows backward
// from a checkpoint, bf16, a wave and a workgroup: 2048 channels 55 and 61, 1500 52 and
// 50, 1501 (shifted) 82 and 60.
LnPlan ln_plan(int dtype, bool backward, int edge, int64_t rows, uint32_t C)
{
    LnPlan p = {};
    const uint32_t V = 16 / elem_bytes(dtype), most = 16 / V, vecs = (C + V - 1) / V;
    p.tl = 3;
    while (p.tl < 6 && (1u << p.tl) < vecs) ++p.tl;
    if ((backward && edge == kShifted ? most : 2 * most) << 6 < vecs)
        while (most << p.tl < vecs) ++p.tl;
    p.nv = (vecs + (1u << p.tl) - 1) >> p.tl;
    const bool wide = p.tl > 6;
    p.threads = wide ? 1u << p.tl : 256;
    const int64_t per = wide ? 1 : 4 * (64 >> p.tl);
    // Workgroups: as many as run at a time, so that each loads gamma and beta once; backward each
    // leaves eight bytes a channel, and one a compute unit is enough where it holds much.  us for 16384
    // rows, 256, 512 and 1024 workgroups: forward 2048 channels bf16 with a residual 49.2, 49.4, 49.2; 1500:
    // 55, 43, 44; backward 2048 from a checkpoint 55, 61, 75; 65536 rows of 512: 70, 53, 54; 6000 of 4096: 43,
    // 49, 63.
    int64_t groups = 512;
    if (backward && p.nv == 2 * most) groups = 256;
    if (wide) groups = p.threads == 128 ? 1024 : backward || p.threads > 256 ? 256 : 512;
    const int64_t want = (rows + per - 1) / per;
    // backward: a single workgroup of up to four rounds needs no second launch for its sums
    p.groups = (uint32_t)(backward && want <= 4 ? 1 : std::max<int64_t>(1, std::min(groups, want)));
    return p;
}

hipError_t launch_ln_forward(const LnPlan &p, LnArgs a, int dtype, int edge, hipStream_t s)
{
    a.tl = p.tl;
    return dtype == kF32 ? forward<kF32>(p, a, edge, s)
           : dtype == kBF16 ? forward<kBF16>(p, a, edge, s)
                            : forward<kF16>(p, a, edge, s);
}

hipError_t launch_ln_backward(const LnPlan &p, LnArgs a, int dtype, int edge, hipStream_t s)
{
    a.tl = p.tl;
    if (a.rows) {
        const hipError_t e = dtype == kF32 ? backward<kF32>(p, a, edge, s)
                             : dtype == kBF16 ? backward<kBF16>(p, a, edge, s)
                                              : backward<kF16>(p, a, edge, s);
        if (e != hipSuccess) return e;
    }
    if (!a.part || (a.rows && p.groups == 1)) return hipSuccess;
    return launch_params(a.part, a.rows ? p.groups : 0, a.C, a.dgamma, a.dbeta, a.add, s);
}

}  // namespace lags
