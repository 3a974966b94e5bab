// Group normalisation with an activation, channels last: the forward pass,
// optionally writing the input's 8-bit checkpoint on the way.
//
//   xh = (x - mean) * rstd;  z = xh * gamma + beta;  y = act(z)
//
// with each operation of xh and z rounded by itself in fp32, so the backward's
// z, and with it relu's mask, has one value wherever it is computed.
//   resident: a sample's slab of channels fits the registers of a workgroup:
//             read once, mean first, then squared distances from it.
//   split:    it does not, or there are too few slabs to fill the GPU: the
//             positions are cut into chunks, a first launch leaves each chunk's
//             mean and squared distances in the workspace, a second one reads
//             the data again (from the 256 MB cache, if it fits) and joins them.
// Chunks are joined by means and squared distances, so a large common offset
// costs no digits.  Sums run in a fixed order (no atomics).
// Bound by memory where the data is large, by a launch and two trips to memory
// where it is small:
//   resident  64 x 784 x 512 bf16, silu and checkpoint: 39 us, 131 MB (3.4 TB/s;
//             silu costs an exponential and a reciprocal a value); 32 x 64 x 64
//             fp32: 4.7 us
//   split     64 x 12544 x 64 bf16: 20 + 37 us, 5.1 and 5.6 TB/s, but the data
//             is read twice
#pragma once

#include "lags_gn.h"

namespace lags {
namespace {

template <int ACT> __device__ inline float activate(float z)
{
    if constexpr (ACT == kActRelu) return z > 0 ? z : (z != z ? z : 0.0f);
    if constexpr (ACT == kActSilu) return z * __builtin_amdgcn_rcpf(1.0f + __expf(-z));
    return z;
}

template <int V, bool UNI> struct Norm {
    PerGroup<V, UNI> mu, rs;
    float ga[V], be[V];
};

// One vector of y, and of the checkpoint; a value of it.
template <int D, int ACT, bool CK, bool ODD, bool UNI>
__device__ inline float emit(const Geo &g, const Writer<D, ODD> &wy, const CodeWriter<D> &wq,
                            const Norm<Elem<D>::V, UNI> &nm, u32x4 raw, uint32_t row)
{
    constexpr int V = Elem<D>::V;
    float f[V], y[V];
    Elem<D>::unpack(raw, f);
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const float xh = (f[j] - nm.mu[j]) * nm.rs[j];
        y[j] = activate<ACT>(xh * nm.ga[j] + nm.be[j]);
    }
    wy.store(row, Elem<D>::pack(y));
    if constexpr (CK) wq.store(row, raw, f, g.nv);
    return y[0];
}

// Resident: R vectors a thread, all requested at once; the second pass runs on
// the registers.
template <int D, int ACT, bool CK, int R, bool ODD, bool UNI>
__global__ __launch_bounds__(kResident) void k_gn_fwd(GnArgs a)
{
    constexpr int V = Elem<D>::V;
    extern __shared__ float sh[];
    const Geo g = geometry(a, V, 1);
    float *gs = sh + g.parts * (V << a.tcl);        // [2][ng]: mean, rstd
    const int64_t row0 = (int64_t)g.n * a.S;
    const Reader<D, ODD> rx(a.x, row0, a.S, a.ldx, g.c0, g.wc, g.col);
    u32x4 raw[R];
#pragma unroll
    for (int k = 0; k < R; ++k) raw[k] = rx.load(g.row + k * g.tr);
    Norm<V, UNI> nm;
    load_param<V>(a.gamma, g, 1.0f, nm.ga);
    load_param<V>(a.beta, g, 0.0f, nm.be);
    float acc[V];
#pragma unroll
    for (int j = 0; j < V; ++j) acc[j] = 0;
#pragma unroll
    for (int k = 0; k < R; ++k) {                  // absent positions hold zeros
        keep(raw[k], acc[0]);
        float f[V];
        Elem<D>::unpack(raw[k], f);
        for (int j = 0; j < V; ++j) acc[j] += f[j];
    }
    const float cnt = (float)((uint64_t)a.S * a.cg);
    GroupSum<V, UNI> sum(acc);
    sum.parts(g, sh);
    __syncthreads();
    sum.groups(g, sh, a, [&](uint32_t i, float s) { gs[i] = s / cnt; });
    __syncthreads();
    nm.mu.set(g, a.cg, a.inv_cg, [&](uint32_t i) { return gs[i]; });
#pragma unroll
    for (int j = 0; j < V; ++j) acc[j] = 0;
#pragma unroll
    for (int k = 0; k < R; ++k) {
        keep(raw[k], acc[0]);
        if (g.row + k * g.tr < a.S) {
            float f[V];
            Elem<D>::unpack(raw[k], f);
            for (int j = 0; j < V; ++j) {
                const float d = f[j] - nm.mu[j];
                acc[j] = __builtin_fmaf(d, d, acc[j]);
            }
        }
    }
    GroupSum<V, UNI> squares(acc);
    squares.parts(g, sh);
    __syncthreads();
    squares.groups(g, sh, a, [&](uint32_t i, float s) {
        const float r = 1.0f / sqrtf(s / cnt + a.eps);
        gs[g.ng + i] = r;
        const int64_t at = (int64_t)g.n * a.G + over_cg(g.c0, a.inv_cg) + i;
        if (a.mean) a.mean[at] = gs[i];
        if (a.rstd) a.rstd[at] = r;
    });
    __syncthreads();
    nm.rs.set(g, a.cg, a.inv_cg, [&](uint32_t i) { return gs[g.ng + i]; });
    const Writer<D, ODD> wy(a.y, row0, a.S, a.ldy, g.c0, g.wc, g.col, a.past);
    const CodeWriter<D> wq(a.wcodes, a.wscales, row0, a.S, a.pitch, a.nrun, a.C, g.c0, g.wc, g.col);
    float last = nm.rs[0];
#pragma unroll
    for (int k = 0; k < R; ++k) {
        keep(raw[k], last);
        last = emit<D, ACT, CK, ODD, UNI>(g, wy, wq, nm, raw[k], g.row + k * g.tr);
    }
}

// Split form, first launch: mean and squared distances of a chunk's groups,
// part[sample][group][chunk][2].  A thread sums, in one pass over its
// positions, each channel's distances from its first value there and their
// squares.  That value being one of the data, what its distance from the mean
// costs in digits is bounded: a relative error of the thread's count of
// positions times fp32's rounding.  Zero stands for a first value of 2^96 or
// more (a type's lowest value as a mask), distances from which would add up
// past fp32; squares that do leave a variance of infinity, as in the resident
// form, not infinity less infinity.
template <int D, bool ODD, bool UNI> __global__ __launch_bounds__(1024) void k_gn_stats(GnArgs a)
{
    constexpr int V = Elem<D>::V, U = kSweep;
    extern __shared__ float sh[];
    const Geo g = geometry(a, V, a.nchunk);
    float *gs = sh + g.parts * (V << a.tcl);       // [ng]
    const uint32_t lo = g.chunk * a.chunk, rows = min(a.S - lo, a.chunk);
    float first[V], s1[V], s2[V];
    for (int j = 0; j < V; ++j) first[j] = s1[j] = s2[j] = 0;
    for (uint32_t s0 = 0; s0 < rows; s0 += U * g.tr) {
        const Reader<D, ODD> rx(a.x, (int64_t)g.n * a.S + lo + s0, rows - s0, a.ldx, g.c0, g.wc, g.col);
        u32x4 raw[U];
#pragma unroll
        for (int k = 0; k < U; ++k) raw[k] = rx.load(g.row + k * g.tr);
        if (s0 == 0) {
            Elem<D>::unpack(raw[0], first);
            for (int j = 0; j < V; ++j) first[j] = __builtin_fabsf(first[j]) < 0x1p96f ? first[j] : 0.0f;
        }
#pragma unroll
        for (int k = 0; k < U; ++k)
            if (s0 + g.row + k * g.tr < rows) {
                keep(raw[k], s1[0]);
                float f[V];
                Elem<D>::unpack(raw[k], f);
                for (int j = 0; j < V; ++j) {
                    const float d = f[j] - first[j];
                    s1[j] += d;
                    s2[j] = __builtin_fmaf(d, d, s2[j]);
                }
            }
    }
    // the thread's own mean and squared distances from it
    const uint32_t mine = g.row < rows ? (rows - g.row - 1) / g.tr + 1 : 0;
    const float cm = (float)mine, inv = mine ? 1.0f / cm : 0.0f;
    float mean[V], t[V];
    for (int j = 0; j < V; ++j) {
        const float d = s1[j] * inv;
        const float q = s1[j] * d;
        if (q < __builtin_inff()) s2[j] = above_zero(s2[j] - q);     // else s2 is infinite or NaN
        mean[j] = first[j] + d;
        t[j] = cm * mean[j];
    }
    const float cnt = (float)((uint64_t)rows * a.cg);
    GroupSum<V, UNI> sum(t);
    sum.parts(g, sh);
    __syncthreads();
    sum.groups(g, sh, a, [&](uint32_t i, float s) { gs[i] = s / cnt; });
    __syncthreads();
    PerGroup<V, UNI> mu;
    mu.set(g, a.cg, a.inv_cg, [&](uint32_t i) { return gs[i]; });
    for (int j = 0; j < V; ++j) {
        const float d = mean[j] - mu[j];
        s2[j] = mine ? __builtin_fmaf(cm * d, d, s2[j]) : 0.0f;
    }
    GroupSum<V, UNI> squares(s2);
    squares.parts(g, sh);
    __syncthreads();
    squares.groups(g, sh, a, [&](uint32_t i, float s) {
        float *p = a.part + 2 * (((size_t)g.n * a.G + over_cg(g.c0, a.inv_cg) + i) * a.nchunk + g.chunk);
        p[0] = gs[i], p[1] = s;
    });
}

// Split form, second launch: joins the chunks' statistics, then streams.
template <int D, int ACT, bool CK, bool ODD, bool UNI>
__global__ __launch_bounds__(1024) void k_gn_apply(GnArgs a)
{
    constexpr int V = Elem<D>::V, U = kSweep;
    extern __shared__ float sh[];
    const Geo g = geometry(a, V, a.nchunk);
    Norm<V, UNI> nm;
    load_param<V>(a.gamma, g, 1.0f, nm.ga);
    load_param<V>(a.beta, g, 0.0f, nm.be);
    // a wave joins a group: its lanes take the chunks
    const uint32_t lane = threadIdx.x & 63, g0 = over_cg(g.c0, a.inv_cg);
    const float total = (float)((uint64_t)a.S * a.cg);
    for (uint32_t i = threadIdx.x >> 6; i < g.ng; i += blockDim.x >> 6) {
        const float *p = a.part + 2 * ((size_t)g.n * a.G + g0 + i) * a.nchunk;
        float s = 0, m2 = 0;
        for (uint32_t k = lane; k < a.nchunk; k += 64)
            s = __builtin_fmaf(p[2 * k], (float)((uint64_t)min(a.chunk, a.S - k * a.chunk) * a.cg), s);
        const float m = wave_sum(s) / total;
        for (uint32_t k = lane; k < a.nchunk; k += 64) {
            const float d = p[2 * k] - m;
            m2 += __builtin_fmaf(d * d, (float)((uint64_t)min(a.chunk, a.S - k * a.chunk) * a.cg), p[2 * k + 1]);
        }
        const float r = 1.0f / sqrtf(wave_sum(m2) / total + a.eps);
        if (lane == 0) {
            sh[i] = m, sh[g.ng + i] = r;
            const int64_t at = (int64_t)g.n * a.G + g0 + i;
            if (g.chunk == 0 && a.mean) a.mean[at] = m;
            if (g.chunk == 0 && a.rstd) a.rstd[at] = r;
        }
    }
    __syncthreads();
    nm.mu.set(g, a.cg, a.inv_cg, [&](uint32_t i) { return sh[i]; });
    nm.rs.set(g, a.cg, a.inv_cg, [&](uint32_t i) { return sh[g.ng + i]; });
    const uint32_t lo = g.chunk * a.chunk, rows = min(a.S - lo, a.chunk);
    float last = nm.rs[0];
    for (uint32_t s0 = 0; s0 < rows; s0 += U * g.tr) {
        const int64_t r0 = (int64_t)g.n * a.S + lo + s0;
        const Reader<D, ODD> rx(a.x, r0, rows - s0, a.ldx, g.c0, g.wc, g.col);
        const Writer<D, ODD> wy(a.y, r0, rows - s0, a.ldy, g.c0, g.wc, g.col, a.past);
        const CodeWriter<D> wq(a.wcodes, a.wscales, r0, rows - s0, a.pitch, a.nrun, a.C, g.c0, g.wc, g.col);
        u32x4 raw[U];
#pragma unroll
        for (int k = 0; k < U; ++k) raw[k] = rx.load(g.row + k * g.tr);
#pragma unroll
        for (int k = 0; k < U; ++k) {
            keep(raw[k], last);
            last = emit<D, ACT, CK, ODD, UNI>(g, wy, wq, nm, raw[k], g.row + k * g.tr);
        }
    }
}

}  // namespace

template <int D> hipError_t launch_gn_forward(const GnPlan &p, const GnArgs &a, hipStream_t s)
{
    constexpr uint32_t V = Elem<D>::V;
    const bool odd = odd_rows<D>(a.x, a.ldx) || odd_rows<D>(a.y, a.ldy);
    const uint32_t grid = a.N * p.nchunk * p.nslab;
    if (!p.resident) {
        const hipError_t e = by_odd<D>(odd, [&](auto O) {
            return by_bool(a.cg % V == 0, [&](auto U) {
                k_gn_stats<D, O(), U()><<<grid, p.threads, lds_bytes(p, V, a.cg, 1, 1), s>>>(a);
                return hipGetLastError();
            });
        });
        if (e != hipSuccess) return e;
    }
    return by_act(a.act, [&](auto A) {
        return by_bool(a.wcodes != nullptr, [&](auto K) {
            auto run = [&](auto O, auto U) {
                if (p.resident)
                    return by_rows(p.rows, [&](auto R) {
                        k_gn_fwd<D, A(), K(), R(), O(), U()>
                            <<<a.N * p.nslab, p.threads, lds_bytes(p, V, a.cg, 1, 2), s>>>(a);
                        return hipGetLastError();
                    });
                k_gn_apply<D, A(), K(), O(), U()><<<grid, p.threads, lds_bytes(p, V, a.cg, 0, 2), s>>>(a);
                return hipGetLastError();
            };
            return by_odd<D>(odd, [&](auto O) { return by_bool(a.cg % V == 0, [&](auto U) { return run(O, U); }); });
        });
    });
}

}  // namespace lags
