// Group normalisation with an activation, channels last: the backward pass,
// from the forward's input or from its 8-bit checkpoint.
//
//   dz = dy * act'(z);  dbeta = sum dz;  dgamma = sum dz xh
//   dx = rstd * (gamma dz - <gamma dz> - xh <gamma dz xh>)   (< > over a group)
//
// All four sums come from two a channel, sum dz and sum dz xh.
//   resident: a sample's slab of dy and of the stored input fits the registers
//             of a workgroup: both are read once; a workgroup takes `nper`
//             samples in turn and leaves their channel sums in the workspace.
//   split:    a first launch leaves the channel sums of chunks of positions in
//             the workspace; a second one joins them and reads the data again.
// A last launch adds the workspace's rows up to dgamma and dbeta.  Sums run in
// a fixed order (no atomics).
// Bound by memory where the data is large, silu's backward (an exponential and
// a reciprocal a value, twice) by arithmetic as well; small ones by the
// launches and a chain of two trips to memory and three barriers:
//   resident  64 x 784 x 512 bf16 from the checkpoint: silu 48 us (3.1 TB/s),
//             relu 41 us; 32 x 256 x 32 fp32: 7.0 us
//   split     64 x 3136 x 256 bf16 from the checkpoint, relu: 43 us for the
//             sums (without their arithmetic too: the reads share the memory
//             with the 103 MB that the call before left to be written back) and
//             46 us for dx (5.7 TB/s)
#pragma once

#include "lags_gn.h"

namespace lags {
namespace {

// A vector of the stored input: as it was, or 8-bit codes with their scale.
// `kUnit` is what x and its mean are multiplied by before they are subtracted.
template <int D, bool CK> struct Stored {
    static constexpr float kUnit = 1;
    u32x4 v;
    // x - mu, rounded once
    template <bool U> __device__ void centred(const PerGroup<Elem<D>::V, U> &mu, float (&f)[Elem<D>::V]) const
    {
        Elem<D>::unpack(v, f);
        for (int j = 0; j < Elem<D>::V; ++j) f[j] -= mu[j];
    }
    __device__ void hold(float t) { keep(v, t); }
};
template <int D> struct Stored<D, true> {
    // half: 64 steps of 2^122, which the largest finite values round to, are past fp32
    static constexpr float kUnit = 0.5f;
    uint32_t q[Elem<D>::V / 4], s;
    // a value is code times step exactly, so this too is rounded once
    template <bool U> __device__ void centred(const PerGroup<Elem<D>::V, U> &mu, float (&f)[Elem<D>::V]) const
    {
        const float step = kUnit * run_step(s);
        for (int i = 0; i < Elem<D>::V / 4; ++i) code_values(q[i], f + 4 * i);
        for (int j = 0; j < Elem<D>::V; ++j) f[j] = __builtin_fmaf(f[j], step, -mu[j]);
    }
    __device__ void hold(float t)
    {
        for (int i = 0; i < Elem<D>::V / 4; ++i) asm volatile("" : "+v"(q[i]) : "v"(t));
        asm volatile("" : "+v"(s) : "v"(t));
    }
};
template <int D, bool CK, bool ODD> struct Source;
template <int D, bool ODD> struct Source<D, false, ODD> {
    Reader<D, ODD> r;
    __device__ Source(const GnArgs &a, int64_t row0, uint32_t n, const Geo &g)
        : r(a.x, row0, n, a.ldx, g.c0, g.wc, g.col)
    {
    }
    __device__ Stored<D, false> load(uint32_t row) const { return {r.load(row)}; }
};
template <int D, bool ODD> struct Source<D, true, ODD> {
    __amdgpu_buffer_rsrc_t rq, rs;
    uint32_t q_at, s_at, pitch, nrun;
    __device__ Source(const GnArgs &a, int64_t row0, uint32_t n, const Geo &g)
    {
        constexpr uint32_t V = Elem<D>::V;
        rq = window(a.rcodes + row0 * a.pitch + g.c0, (int64_t)n * a.pitch - g.c0);
        rs = window(a.rscales + row0 * a.nrun + g.c0 / kRun, (int64_t)n * a.nrun - g.c0 / kRun);
        const bool in = g.nv > 0;
        q_at = in ? g.col * V : 0x80000000u, s_at = in ? g.col * V / kRun : 0x80000000u;
        pitch = a.pitch, nrun = a.nrun;
    }
    __device__ Stored<D, true> load(uint32_t row) const
    {
        Stored<D, true> x;
        if constexpr (Elem<D>::V == 8) {
            const u32x2 w = __builtin_amdgcn_raw_buffer_load_b64(rq, q_at + row * pitch, 0, 0);
            x.q[0] = w[0], x.q[Elem<D>::V / 4 - 1] = w[1];
        } else {
            x.q[0] = __builtin_amdgcn_raw_buffer_load_b32(rq, q_at + row * pitch, 0, 0);
        }
        x.s = __builtin_amdgcn_raw_buffer_load_b8(rs, s_at + row * nrun, 0, 0);
        return x;
    }
};

// dy act'(z) for z = xh ga + be, both operations rounded.  relu asks only
// whether z > 0: a rounded sum has the sign of the exact one, so that is
// whether the rounded product exceeds -be.
template <int ACT, int V> __device__ inline void act_grad(const float (&xh)[V], const float (&ga)[V],
                                                 const float (&be)[V], float (&d)[V])
{
    if constexpr (ACT == kActRelu) {
#pragma unroll
        for (int j = 0; j < V; ++j) d[j] = xh[j] * ga[j] > -be[j] ? d[j] : 0.0f;
    } else if constexpr (ACT == kActSilu) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const float z = xh[j] * ga[j] + be[j];
            const float sg = __builtin_amdgcn_rcpf(1.0f + __expf(-z));
            d[j] *= sg * __builtin_fmaf(z, 1.0f - sg, 1.0f);
        }
    }
}

template <int V, bool UNI> struct Chan {     // a thread's channels
    PerGroup<V, UNI> mu, rs;
    float ga[V], be[V];
    // `unit` times the means, rstd over it
    __device__ void load(const GnArgs &a, const Geo &g, float unit)
    {
        const float *m = a.mean + (size_t)g.n * a.G + over_cg(g.c0, a.inv_cg);
        const float *r = a.rstd + (size_t)g.n * a.G + over_cg(g.c0, a.inv_cg);
        mu.set(g, a.cg, a.inv_cg, [&](uint32_t i) { return unit * m[i]; });
        rs.set(g, a.cg, a.inv_cg, [&](uint32_t i) { return r[i] / unit; });
    }
};

template <int D, int ACT, bool CK, bool UNI>
__device__ inline void bwd_sums(const Stored<D, CK> &x, u32x4 dy, const Chan<Elem<D>::V, UNI> &ch,
                                float (&sa)[Elem<D>::V], float (&sb)[Elem<D>::V])
{
    constexpr int V = Elem<D>::V;
    float xh[V], d[V];
    x.centred(ch.mu, xh);
    Elem<D>::unpack(dy, d);
#pragma unroll
    for (int j = 0; j < V; ++j) xh[j] *= ch.rs[j];
    act_grad<ACT, V>(xh, ch.ga, ch.be, d);
#pragma unroll
    for (int j = 0; j < V; ++j) {
        sa[j] += d[j];
        sb[j] = __builtin_fmaf(d[j], xh[j], sb[j]);
    }
    settle<V>(sa);
    settle<V>(sb);
}

// One vector of dx from rstd times the means (s1, s2); a value of it.
template <int D, int ACT, bool CK, bool ODD, bool UNI>
__device__ inline float bwd_emit(const Writer<D, ODD> &w, const Stored<D, CK> &x, u32x4 dy,
                                const Chan<Elem<D>::V, UNI> &ch, const PerGroup<Elem<D>::V, UNI> &s1,
                                const PerGroup<Elem<D>::V, UNI> &s2, uint32_t row)
{
    constexpr int V = Elem<D>::V;
    float xh[V], d[V];
    x.centred(ch.mu, xh);
    Elem<D>::unpack(dy, d);
#pragma unroll
    for (int j = 0; j < V; ++j) xh[j] *= ch.rs[j];
    act_grad<ACT, V>(xh, ch.ga, ch.be, d);
#pragma unroll
    for (int j = 0; j < V; ++j)
        d[j] = __builtin_fmaf(ch.ga[j] * (ch.rs[j] * Stored<D, CK>::kUnit), d[j], -__builtin_fmaf(xh[j], s2[j], s1[j]));
    w.store(row, Elem<D>::pack(d));
    return d[0];
}

// LDS of the joins: two arrays of parts of the channel sums and two of the
// group sums, the group means, and (resident) gamma and the channel sums of
// the samples so far.
struct Joins {
    float *a, *b, *ga, *gb, *mean, *gamma, *total;
    __device__ Joins(float *sh, const Geo &g, uint32_t V)
    {
        const uint32_t nl = g.parts << g.tcl;
        a = sh, b = a + nl * V, ga = b + nl * V, gb = ga + nl, mean = gb + nl;
        gamma = mean + 2 * g.ng, total = gamma + g.wc;
    }
};

// rstd times the means of gamma dz and gamma dz xh over each channel's group,
// from every thread's per-channel sums, which are used up; TOTAL: and their
// sums over the samples.  ONE (with UNI): the group sums are made of one value
// a thread, not of the channels' sums.  That is less to add up where a group is
// wide (8192 x 1 x 2048, one group: 92 us, else 161), but takes registers that
// only the shortest samples leave (64 x 784 x 512 in 8 rows: 43 us, else 41).
template <int V, bool UNI, bool TOTAL, bool ONE>
__device__ inline void group_means(const GnArgs &a, const Geo &g, const Joins &m, const Chan<V, UNI> &ch, float unit,
                                   float (&sa)[V], float (&sb)[V], PerGroup<V, UNI> &s1, PerGroup<V, UNI> &s2)
{
    const float cnt = (float)((uint64_t)a.S * a.cg);
    auto mean_a = [&](uint32_t i, float s) { m.mean[i] = s / cnt; };
    auto mean_b = [&](uint32_t i, float s) { m.mean[g.ng + i] = s / cnt; };
    if constexpr (TOTAL) {
        if constexpr (ONE) {
            float ta[V], tb[V];
            for (int j = 0; j < V; ++j) ta[j] = sa[j] * ch.ga[j], tb[j] = sb[j] * ch.ga[j];
            GroupSum<V, true>(ta).parts(g, m.ga);
            GroupSum<V, true>(tb).parts(g, m.gb);
        }
        to_parts<V>(sa, g, m.a);
        to_parts<V>(sb, g, m.b);
        __syncthreads();
        if constexpr (ONE) {
            GroupSum<V, true>::groups(g, m.ga, a, mean_a);
            GroupSum<V, true>::groups(g, m.gb, a, mean_b);
        } else {
            to_groups<V>(g, m.a, a.cg, a.inv_cg, mean_a, m.gamma);
            to_groups<V>(g, m.b, a.cg, a.inv_cg, mean_b, m.gamma);
        }
    } else {
        for (int j = 0; j < V; ++j) sa[j] *= ch.ga[j], sb[j] *= ch.ga[j];
        GroupSum<V, UNI> ua(sa), ub(sb);
        ua.parts(g, m.a);
        ub.parts(g, m.b);
        __syncthreads();
        ua.groups(g, m.a, a, mean_a);
        ub.groups(g, m.b, a, mean_b);
    }
    if constexpr (TOTAL)
        for (uint32_t i = threadIdx.x; i < g.wc; i += blockDim.x) {
            float u = 0, v = 0;
            for (uint32_t k = 0; k < g.parts; ++k) u += m.a[k * (V << g.tcl) + i], v += m.b[k * (V << g.tcl) + i];
            m.total[i] += u, m.total[g.wc + i] += v;
        }
    __syncthreads();
    s1.set(g, a.cg, a.inv_cg, [&](uint32_t i) { return m.mean[i]; });
    s2.set(g, a.cg, a.inv_cg, [&](uint32_t i) { return m.mean[g.ng + i]; });
    for (int j = 0; j < (UNI ? 1 : V); ++j) s1.v[j] *= ch.rs[j] * unit, s2.v[j] *= ch.rs[j] * unit;
}

// The workgroup's per-channel sums, to p[0..C) (sum dz) and p[C..2C) (sum dz xh).
template <int V>
__device__ inline void put_channel_sums(const Geo &g, float *sh, uint32_t C, float *p, float (&sa)[V], float (&sb)[V])
{
    const uint32_t wp = V << g.tcl, np = g.parts * wp;
    to_parts<V>(sa, g, sh);
    to_parts<V>(sb, g, sh + np);
    __syncthreads();
    for (uint32_t i = threadIdx.x; i < g.wc; i += blockDim.x) {
        float a = 0, b = 0;
        for (uint32_t k = 0; k < g.parts; ++k) a += sh[k * wp + i], b += sh[np + k * wp + i];
        p[g.c0 + i] = a, p[C + g.c0 + i] = b;
    }
}

// Threads at most: a slab of 2049 to 4096 fp32 channels has 1024 lanes of columns.
constexpr int bwd_threads(int dtype, int rows)
{
    return dtype == kF32 && rows <= (int)kWideRows ? 1024 : (int)kResidentBwd;
}
// Waves a SIMD, at least: two workgroups a compute unit, so that one loads
// while another sums or stores, at the price of registers spilled by kernels of
// 16-bit values: from the checkpoint 1 (relu) to 9 (silu), from x 8 to 18, up to
// 42 in rows that start inside a word.  One wave less spills none, but takes
// longer (64 x 784 x 512 bf16 relu from the checkpoint 55 us, else 41; from x 56,
// else 50), except with silu from x (52, else 59).
constexpr int bwd_waves(int threads, int rows, bool uni) { return threads == 1024 || (uni && rows <= 8) ? 4 : uni ? 3 : 2; }

// Resident: R vectors a thread of dy and of the stored input.
template <int D, int ACT, bool CK, int R, bool ODD, bool UNI>
__global__ __launch_bounds__(bwd_threads(D, R), bwd_waves(bwd_threads(D, R), R, UNI)) void k_gn_bwd(GnArgs a)
{
    constexpr int V = Elem<D>::V;
    extern __shared__ float sh[];
    Geo g = geometry(a, V, 1);
    const uint32_t p = g.n, n_hi = min(a.N, (p + 1) * a.nper);
    Chan<V, UNI> ch;
    load_param<V>(a.gamma, g, 1.0f, ch.ga);
    load_param<V>(a.beta, g, 0.0f, ch.be);
    const Joins joins(sh, g, V);
    for (uint32_t i = threadIdx.x; i < g.wc; i += blockDim.x) {
        joins.total[i] = joins.total[g.wc + i] = 0;
        joins.gamma[i] = a.gamma ? a.gamma[g.c0 + i] : 1.0f;    // read after the sums' barrier
    }
    for (g.n = p * a.nper; g.n < n_hi; ++g.n) {
        const int64_t row0 = (int64_t)g.n * a.S;
        uint32_t first = g.row;          // made anew, or every vector's offsets are kept from sample to sample
        asm volatile("" : "+v"(first));
        const Source<D, CK, ODD> xs(a, row0, a.S, g);
        const Reader<D, ODD> ds(a.dy, row0, a.S, a.lddy, g.c0, g.wc, g.col);
        Stored<D, CK> x[R];
        u32x4 dy[R];
#pragma unroll
        for (int k = 0; k < R; ++k) {
            x[k] = xs.load(first + k * g.tr);
            dy[k] = ds.load(first + k * g.tr);
        }
        ch.load(a, g, Stored<D, CK>::kUnit);
        float sa[V], sb[V];
        for (int j = 0; j < V; ++j) sa[j] = sb[j] = 0;
#pragma unroll
        for (int k = 0; k < R; ++k) {              // absent positions: dy = 0
            x[k].hold(sa[0]);
            keep(dy[k], sa[0]);
            bwd_sums<D, ACT, CK, UNI>(x[k], dy[k], ch, sa, sb);
        }
        PerGroup<V, UNI> s1, s2;
        group_means<V, UNI, true, UNI && R == 2>(a, g, joins, ch, Stored<D, CK>::kUnit, sa, sb, s1, s2);
        const Writer<D, ODD> w(a.dx, row0, a.S, a.lddx, g.c0, g.wc, g.col);
        float last = s1[0];
#pragma unroll
        for (int k = 0; k < R; ++k) {
            x[k].hold(last);
            keep(dy[k], last);
            last = bwd_emit<D, ACT, CK, ODD, UNI>(w, x[k], dy[k], ch, s1, s2, first + k * g.tr);
        }
    }
    float *out = a.part + (size_t)p * 2 * a.C + g.c0;
    for (uint32_t i = threadIdx.x; i < g.wc; i += blockDim.x)
        out[i] = joins.total[i], out[a.C + i] = joins.total[g.wc + i];
}

// Split form, first launch: per-channel sums of a chunk, part[sample][chunk][2][C].
template <int D, int ACT, bool CK, bool ODD, bool UNI>
__global__ __launch_bounds__(1024) void k_gn_bwd_sums(GnArgs a)
{
    constexpr int V = Elem<D>::V, U = kSweep;
    extern __shared__ float sh[];
    const Geo g = geometry(a, V, a.nchunk);
    Chan<V, UNI> ch;
    load_param<V>(a.gamma, g, 1.0f, ch.ga);
    load_param<V>(a.beta, g, 0.0f, ch.be);
    ch.load(a, g, Stored<D, CK>::kUnit);
    float sa[V], sb[V];
    for (int j = 0; j < V; ++j) sa[j] = sb[j] = 0;
    const uint32_t lo = g.chunk * a.chunk, rows = min(a.S - lo, a.chunk);
    for (uint32_t s0 = 0; s0 < rows; s0 += U * g.tr) {
        const int64_t r0 = (int64_t)g.n * a.S + lo + s0;
        const Source<D, CK, ODD> xs(a, r0, rows - s0, g);
        const Reader<D, ODD> ds(a.dy, r0, rows - s0, a.lddy, g.c0, g.wc, g.col);
        Stored<D, CK> x[U];
        u32x4 dy[U];
#pragma unroll
        for (int k = 0; k < U; ++k) {
            x[k] = xs.load(g.row + k * g.tr);
            dy[k] = ds.load(g.row + k * g.tr);
        }
#pragma unroll
        for (int k = 0; k < U; ++k) {              // absent positions: dy = 0
            x[k].hold(sa[0]);
            keep(dy[k], sa[0]);
            bwd_sums<D, ACT, CK, UNI>(x[k], dy[k], ch, sa, sb);
        }
    }
    put_channel_sums<V>(g, sh, a.C, a.part + ((size_t)g.n * a.nchunk + g.chunk) * 2 * a.C, sa, sb);
}

// Split form, second launch: joins the chunks' sums, then streams.
template <int D, int ACT, bool CK, bool ODD, bool UNI>
__global__ __launch_bounds__(1024) void k_gn_bwd_apply(GnArgs a)
{
    constexpr int V = Elem<D>::V, U = kSweep;
    extern __shared__ float sh[];
    const Geo g = geometry(a, V, a.nchunk);
    Chan<V, UNI> ch;
    load_param<V>(a.gamma, g, 1.0f, ch.ga);
    load_param<V>(a.beta, g, 0.0f, ch.be);
    ch.load(a, g, Stored<D, CK>::kUnit);
    float sa[V], sb[V];
    for (int j = 0; j < V; ++j) sa[j] = sb[j] = 0;
    const Joins joins(sh, g, V);
    for (uint32_t k = g.row; k < a.nchunk; k += g.tr) {
        const float *p = a.part + ((size_t)g.n * a.nchunk + k) * 2 * a.C;
        float u[V], v[V];
        load_param<V>(p, g, 0.0f, u);
        load_param<V>(p + a.C, g, 0.0f, v);
        for (int j = 0; j < V; ++j) sa[j] += u[j], sb[j] += v[j];
    }
    PerGroup<V, UNI> s1, s2;
    group_means<V, UNI, false, false>(a, g, joins, ch, Stored<D, CK>::kUnit, sa, sb, s1, s2);
    float last = s1[0];
    const uint32_t lo = g.chunk * a.chunk, rows = min(a.S - lo, a.chunk);
    for (uint32_t s0 = 0; s0 < rows; s0 += U * g.tr) {
        const int64_t r0 = (int64_t)g.n * a.S + lo + s0;
        const Source<D, CK, ODD> xs(a, r0, rows - s0, g);
        const Reader<D, ODD> ds(a.dy, r0, rows - s0, a.lddy, g.c0, g.wc, g.col);
        const Writer<D, ODD> w(a.dx, r0, rows - s0, a.lddx, g.c0, g.wc, g.col);
        Stored<D, CK> x[U];
        u32x4 dy[U];
#pragma unroll
        for (int k = 0; k < U; ++k) {
            x[k] = xs.load(g.row + k * g.tr);
            dy[k] = ds.load(g.row + k * g.tr);
        }
#pragma unroll
        for (int k = 0; k < U; ++k) {
            x[k].hold(last);
            keep(dy[k], last);
            last = bwd_emit<D, ACT, CK, ODD, UNI>(w, x[k], dy[k], ch, s1, s2, g.row + k * g.tr);
        }
    }
}

}  // namespace

template <int D> hipError_t launch_gn_backward(const GnPlan &p, const GnArgs &a, hipStream_t s)
{
    constexpr uint32_t V = Elem<D>::V;
    const size_t lds = p.resident ? lds_bytes(p, V, a.cg, 3, 2, 3) : lds_bytes(p, V, a.cg, 3, 2);
    const bool odd = odd_rows<D>(a.x, a.ldx) || odd_rows<D>(a.dy, a.lddy) || odd_rows<D>(a.dx, a.lddx);
    return by_act(a.act, [&](auto A) {
        return by_bool(a.rcodes != nullptr, [&](auto K) {
            auto run = [&](auto O, auto U) {
                if (p.resident)
                    return by_rows(p.rows, [&](auto R) {
                        const auto k = k_gn_bwd<D, A(), K(), R(), O(), U()>;
                        if (hipError_t e = allow_lds((const void *)k, lds); e != hipSuccess) return e;
                        k<<<p.nparts * p.nslab, p.threads, lds, s>>>(a);
                        return hipGetLastError();
                    });
                const uint32_t grid = a.N * p.nchunk * p.nslab;
                k_gn_bwd_sums<D, A(), K(), O(), U()><<<grid, p.threads, lds, s>>>(a);
                if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
                k_gn_bwd_apply<D, A(), K(), O(), U()><<<grid, p.threads, lds, s>>>(a);
                return hipGetLastError();
            };
            return by_odd<D>(odd, [&](auto O) { return by_bool(a.cg % V == 0, [&](auto U) { return run(O, U); }); });
        });
    });
}

}  // namespace lags
