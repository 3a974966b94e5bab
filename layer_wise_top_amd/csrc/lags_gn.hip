// Group normalisation with an activation, channels last: forward (optionally
// writing the input's 8-bit checkpoint) and backward (from the input or from
// its checkpoint).
//
//   xh = (x - mean) * rstd;  z = xh * gamma + beta;  y = act(z)
//   dz = dy * act'(z);  dbeta = sum dz;  dgamma = sum dz xh
//   dx = rstd * (gamma dz - <gamma dz> - xh <gamma dz xh>)   (< > over a group)
//
// with each operation of xh and z rounded by itself in fp32, so the backward's
// z, and with it relu's mask, has one value wherever it is computed.
// Everything is bound by memory, so what matters is how often a sample is
// read.  A workgroup takes one sample's slab of whole groups (and whole runs
// of 32 channels): 2^tcl lanes span the slab's channels in 16-byte vectors,
// the other lane bits and the waves take positions.
//   resident: the slab fits the registers of a workgroup; it is read once.
//   split:    it does not, or there are too few slabs to fill the GPU; the
//             positions are cut into chunks, a first launch leaves each
//             chunk's sums in the workspace, a second one reads the data again
//             and joins them.
// Sums run in a fixed order (no atomics): results repeat bit for bit.
// Statistics are two-pass, mean first, then squared distances from it; chunks
// are joined by their means and squared distances, so a large common offset
// costs no digits.
#include "lags_act.h"

#include <type_traits>

namespace lags {
namespace {

constexpr uint32_t kFwdThreads = 1024, kBwdThreads = 512;   // a resident workgroup, at most
constexpr uint32_t kMostRows = 16;                           // register rows a thread, at most
constexpr uint32_t kStatRows = 8;                            // rows a thread of a statistics sub-chunk

// ---- sums over a workgroup -------------------------------------------------

// One step of a halving exchange: of the CUR values each lane still holds,
// the upper half goes to (or comes from) the lane `o` away, so log2(V) steps
// cost V - 1 exchanges and leave each lane one column's sum over those lanes.
template <int V, int CUR, int O>
__device__ inline void row_reduce(float (&v)[V], uint32_t tc, uint32_t lane, uint32_t &base, uint32_t &cur)
{
    if constexpr (O >= 1) {
        if (O >= (int)tc) {              // lane bit O tells rows apart
            if constexpr (CUR > 1) {
                const bool up = lane & O;
#pragma unroll
                for (int j = 0; j < CUR / 2; ++j) {
                    const float send = up ? v[j] : v[j + CUR / 2];
                    const float keep = up ? v[j + CUR / 2] : v[j];
                    v[j] = keep + __shfl_xor(send, O);
                }
                if (up) base += CUR / 2;
                cur = CUR / 2;
                row_reduce<V, CUR / 2, O / 2>(v, tc, lane, base, cur);
            } else {
                v[0] += __shfl_xor(v[0], O);
                row_reduce<V, 1, O / 2>(v, tc, lane, base, cur);
            }
        }
    }
}

struct Geo {
    uint32_t tcl, col, row, tr, parts;   // column vector, first position, positions a sweep
};
__device__ inline Geo geometry(uint32_t tcl)
{
    Geo g;
    g.tcl = tcl;
    g.col = threadIdx.x & ((1u << tcl) - 1);
    g.row = threadIdx.x >> tcl;
    g.tr = blockDim.x >> tcl;
    g.parts = tcl >= 6 ? g.tr : blockDim.x >> 6;
    return g;
}

// Per-channel sums of the workgroup's waves, left as sh[part][channel of the
// slab, padded to 2^tcl vectors].
template <int V> __device__ inline void to_parts(float (&v)[V], const Geo &g, float *sh)
{
    const uint32_t lane = threadIdx.x & 63, tc = 1u << g.tcl;
    uint32_t base = 0, cur = V;
    row_reduce<V, V, 32>(v, tc, lane, base, cur);
    const uint32_t part = g.tcl >= 6 ? g.row : threadIdx.x >> 6;
    float *p = sh + (size_t)part * (tc * V) + g.col * V + base;
    // after the halving steps, lanes that hold the same columns hold the same sums
#pragma unroll
    for (int j = 0; j < V; ++j)
        if (j < (int)cur) p[j] = v[j];
}

// Group sums from the parts: gs[g], 2^k lanes a group.
template <int V> __device__ inline void to_groups(const Geo &g, const float *sh, uint32_t ng, uint32_t cg, float *gs)
{
    const uint32_t wp = V << g.tcl, items = cg * g.parts;
    uint32_t lg = 1;
    while (lg < 64 && lg < items) lg <<= 1;
    const uint32_t sub = threadIdx.x & (lg - 1), per = blockDim.x / lg;
    // every lane of a wave runs every iteration: the exchanges need them
    for (uint32_t g0 = 0; g0 < ng; g0 += per) {
        const uint32_t gi = g0 + threadIdx.x / lg;
        float s = 0;
        if (gi < ng) {
            for (uint32_t i = sub; i < items; i += lg) {
                const uint32_t p = i / cg;
                s += sh[p * wp + gi * cg + i - p * cg];
            }
        }
        for (uint32_t o = lg >> 1; o; o >>= 1) s += __shfl_xor(s, o);
        if (gi < ng && sub == 0) gs[gi] = s;
    }
}

// Which group each channel of a thread's vector belongs to.
template <int V> __device__ inline void group_of(uint32_t c, uint32_t cg, uint32_t (&gi)[V])
{
    uint32_t q = c / cg, r = c - q * cg;
#pragma unroll
    for (int j = 0; j < V; ++j) {
        gi[j] = q;
        if (++r == cg) r = 0, ++q;
    }
}

template <int V> __device__ inline void load_param(const float *p, uint32_t c, int n, float other, float (&f)[V])
{
    for (int j = 0; j < V; ++j) f[j] = p && j < n ? p[c + j] : other;
}

// Slabs of one sample run side by side on one XCD (workgroups are dealt to
// the 8 XCDs in turn): they share cache lines at their edges.
__device__ inline uint32_t deal(uint32_t b, uint32_t n)
{
    const uint32_t per = n / 8, main = per * 8;
    return b < main ? (b & 7) * per + (b >> 3) : b;
}

template <int ACT> __device__ inline float act(float z)
{
    if constexpr (ACT == kActRelu) return z > 0 ? z : (z != z ? z : 0.0f);
    if constexpr (ACT == kActSilu) return z * __builtin_amdgcn_rcpf(1.0f + __expf(-z));
    return z;
}
template <int ACT> __device__ inline float act_grad(float z, float dy)
{
    if constexpr (ACT == kActRelu) return z > 0 ? dy : 0.0f;
    if constexpr (ACT == kActSilu) {
        const float sg = __builtin_amdgcn_rcpf(1.0f + __expf(-z));
        return dy * (sg * (1.0f + z * (1.0f - sg)));
    }
    return dy;
}

// ---- forward ---------------------------------------------------------------

// One vector of y, and of the checkpoint.
template <int D, int ACT, bool CK>
__device__ inline void emit(const GnArgs &a, u32x4 raw, int64_t r, uint32_t c, int nv,
                            const float (&mu)[Elem<D>::V], const float (&rs)[Elem<D>::V],
                            const float (&ga)[Elem<D>::V], const float (&be)[Elem<D>::V])
{
    constexpr int V = Elem<D>::V, E = Elem<D>::E;
    float f[V], y[V];
    Elem<D>::unpack(raw, f);
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const float xh = (f[j] - mu[j]) * rs[j];
        const float z = xh * ga[j] + be[j];
        y[j] = act<ACT>(z);
    }
    if (nv > 0) store_vec<D>((char *)a.y + (r * a.ldy + c) * E, Elem<D>::pack(y), nv);
    if constexpr (CK) {
        const uint32_t s = run_scale(run_top<V>(Elem<D>::top(raw)));
        uint32_t q[V / 4];
        run_codes<V>(f, s, q);
        if (c < a.pitch && (nv > 0 || c >= a.C)) {       // the row's pad gets zeros; lanes past the slab write nothing
            uint8_t *p = a.wcodes + r * a.pitch + c;
            if constexpr (V == 8)
                *(u32x2 *)p = u32x2{q[0], q[1]};
            else
                *(uint32_t *)p = q[0];
        }
        if (nv > 0 && c % kRun == 0) a.wscales[r * a.nrun + c / kRun] = (uint8_t)s;
    }
}

template <int D, int ACT, bool CK, int R>
__global__ __launch_bounds__(1024) void k_gn_fwd(GnArgs a)
{
    constexpr int V = Elem<D>::V, E = Elem<D>::E;
    extern __shared__ float sh[];
    const Geo g = geometry(a.tcl);
    const uint32_t b = deal(blockIdx.x, gridDim.x);
    const uint32_t n = b / a.nslab, slab = b - n * a.nslab;
    const uint32_t c0 = slab * a.w, wc = min(a.w, a.C - c0), ng = wc / a.cg;
    const uint32_t c = c0 + g.col * V;
    const int nv = (int)wc - (int)(g.col * V);
    float *gs = sh + g.parts * (V << a.tcl);        // [2][ng]
    const int64_t r0 = (int64_t)n * a.S + g.row;
    u32x4 raw[R];
#pragma unroll
    for (int k = 0; k < R; ++k) {
        const uint32_t r = g.row + k * g.tr;
        raw[k] = load_vec<D>((const char *)a.x + ((r0 + k * g.tr) * a.ldx + c) * E, r < a.S ? nv : 0);
    }
    float acc[V], mu[V], rs[V];
#pragma unroll
    for (int j = 0; j < V; ++j) acc[j] = 0;
#pragma unroll
    for (int k = 0; k < R; ++k) {                  // absent positions hold zeros
        float f[V];
        Elem<D>::unpack(raw[k], f);
        for (int j = 0; j < V; ++j) acc[j] += f[j];
    }
    to_parts<V>(acc, g, sh);
    __syncthreads();
    to_groups<V>(g, sh, ng, a.cg, gs);
    __syncthreads();
    const float cnt = (float)((uint64_t)a.S * a.cg);
    uint32_t gi[V];
    group_of<V>(nv > 0 ? g.col * V : 0, a.cg, gi);
#pragma unroll
    for (int j = 0; j < V; ++j) {
        mu[j] = gs[j < nv ? gi[j] : 0] / cnt;
        acc[j] = 0;
    }
#pragma unroll
    for (int k = 0; k < R; ++k)
        if (g.row + k * g.tr < a.S) {
            float f[V];
            Elem<D>::unpack(raw[k], f);
            for (int j = 0; j < V; ++j) {
                const float d = f[j] - mu[j];
                acc[j] = __builtin_fmaf(d, d, acc[j]);
            }
        }
    to_parts<V>(acc, g, sh);
    __syncthreads();
    to_groups<V>(g, sh, ng, a.cg, gs + ng);
    __syncthreads();
#pragma unroll
    for (int j = 0; j < V; ++j) rs[j] = 1.0f / sqrtf(gs[ng + (j < nv ? gi[j] : 0)] / cnt + a.eps);
    for (uint32_t i = threadIdx.x; i < ng; i += blockDim.x) {
        const int64_t at = (int64_t)n * a.G + c0 / a.cg + i;
        if (a.mean) a.mean[at] = gs[i] / cnt;
        if (a.rstd) a.rstd[at] = 1.0f / sqrtf(gs[ng + i] / cnt + a.eps);
    }
    float ga[V], be[V];
    load_param<V>(a.gamma, c, nv, 1.0f, ga);
    load_param<V>(a.beta, c, nv, 0.0f, be);
#pragma unroll
    for (int k = 0; k < R; ++k)
        if (g.row + k * g.tr < a.S)
            emit<D, ACT, CK>(a, raw[k], r0 + k * g.tr, c, nv, mu, rs, ga, be);
}

// Split form, first launch: mean and squared distances of a chunk's groups,
// part[sample][group][chunk][2].  Sub-chunks of R register rows a thread are
// joined as they come.
template <int D, int R> __global__ __launch_bounds__(1024) void k_gn_stats(GnArgs a)
{
    constexpr int V = Elem<D>::V, E = Elem<D>::E;
    extern __shared__ float sh[];
    const Geo g = geometry(a.tcl);
    const uint32_t per = a.nchunk * a.nslab;
    const uint32_t b = deal(blockIdx.x, gridDim.x);
    const uint32_t n = b / per, rest = b - n * per, chunk = rest / a.nslab, slab = rest - chunk * a.nslab;
    const uint32_t c0 = slab * a.w, wc = min(a.w, a.C - c0), ng = wc / a.cg;
    const uint32_t c = c0 + g.col * V;
    const int nv = (int)wc - (int)(g.col * V);
    float *gs = sh + g.parts * (V << a.tcl);       // [2][ng] of a sub-chunk, then [2][ng] joined
    float *jo = gs + 2 * ng;
    const uint32_t lo = chunk * a.chunk, hi = min(a.S, lo + a.chunk);
    uint32_t gi[V];
    group_of<V>(nv > 0 ? g.col * V : 0, a.cg, gi);
    for (uint32_t s0 = lo; s0 < hi; s0 += R * g.tr) {
        const uint32_t rows = min(hi - s0, R * g.tr);
        const int64_t r0 = (int64_t)n * a.S + s0 + g.row;
        u32x4 raw[R];
        float acc[V], mu[V];
#pragma unroll
        for (int k = 0; k < R; ++k)
            raw[k] = load_vec<D>((const char *)a.x + ((r0 + k * g.tr) * a.ldx + c) * E,
                                 g.row + k * g.tr < rows ? nv : 0);
#pragma unroll
        for (int j = 0; j < V; ++j) acc[j] = 0;
#pragma unroll
        for (int k = 0; k < R; ++k) {
            float f[V];
            Elem<D>::unpack(raw[k], f);
            for (int j = 0; j < V; ++j) acc[j] += f[j];
        }
        to_parts<V>(acc, g, sh);
        __syncthreads();
        to_groups<V>(g, sh, ng, a.cg, gs);
        __syncthreads();
        const float cnt = (float)((uint64_t)rows * a.cg);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            mu[j] = gs[j < nv ? gi[j] : 0] / cnt;
            acc[j] = 0;
        }
#pragma unroll
        for (int k = 0; k < R; ++k)
            if (g.row + k * g.tr < rows) {
                float f[V];
                Elem<D>::unpack(raw[k], f);
                for (int j = 0; j < V; ++j) {
                    const float d = f[j] - mu[j];
                    acc[j] = __builtin_fmaf(d, d, acc[j]);
                }
            }
        to_parts<V>(acc, g, sh);
        __syncthreads();
        to_groups<V>(g, sh, ng, a.cg, gs + ng);
        __syncthreads();
        const float before = (float)((uint64_t)(s0 - lo) * a.cg);
        for (uint32_t i = threadIdx.x; i < ng; i += blockDim.x) {
            const float m = gs[i] / cnt, m2 = gs[ng + i];
            if (s0 == lo) {
                jo[i] = m, jo[ng + i] = m2;
            } else {
                const float d = m - jo[i], f = cnt / (before + cnt);
                jo[i] += d * f;
                jo[ng + i] += m2 + d * d * (before * f);
            }
        }
        __syncthreads();                           // gs is written again
    }
    for (uint32_t i = threadIdx.x; i < ng; i += blockDim.x) {
        float *p = a.part + 2 * (((size_t)n * a.G + c0 / a.cg + i) * a.nchunk + chunk);
        p[0] = jo[i], p[1] = jo[ng + i];
    }
}

// Split form, second launch: joins the chunks' statistics, then streams.
template <int D, int ACT, bool CK> __global__ __launch_bounds__(1024) void k_gn_apply(GnArgs a)
{
    constexpr int V = Elem<D>::V, E = Elem<D>::E, U = 4;
    extern __shared__ float sh[];
    const Geo g = geometry(a.tcl);
    const uint32_t per = a.nchunk * a.nslab;
    const uint32_t b = deal(blockIdx.x, gridDim.x);
    const uint32_t n = b / per, rest = b - n * per, chunk = rest / a.nslab, slab = rest - chunk * a.nslab;
    const uint32_t c0 = slab * a.w, wc = min(a.w, a.C - c0), ng = wc / a.cg;
    const uint32_t c = c0 + g.col * V;
    const int nv = (int)wc - (int)(g.col * V);
    // a wave joins a group: its lanes take the chunks
    const uint32_t lane = threadIdx.x & 63;
    const float total = (float)((uint64_t)a.S * a.cg);
    for (uint32_t i = threadIdx.x >> 6; i < ng; i += blockDim.x >> 6) {
        const float *p = a.part + 2 * ((size_t)n * a.G + c0 / a.cg + i) * a.nchunk;
        float s = 0, m2 = 0;
        for (uint32_t k = lane; k < a.nchunk; k += 64)
            s = __builtin_fmaf(p[2 * k], (float)((uint64_t)min(a.chunk, a.S - k * a.chunk) * a.cg), s);
        for (uint32_t o = 32; o; o >>= 1) s += __shfl_xor(s, o);
        const float m = s / total;
        for (uint32_t k = lane; k < a.nchunk; k += 64) {
            const float d = p[2 * k] - m;
            m2 += __builtin_fmaf(d * d, (float)((uint64_t)min(a.chunk, a.S - k * a.chunk) * a.cg), p[2 * k + 1]);
        }
        for (uint32_t o = 32; o; o >>= 1) m2 += __shfl_xor(m2, o);
        const float r = 1.0f / sqrtf(m2 / total + a.eps);
        if (lane == 0) {
            sh[i] = m, sh[ng + i] = r;
            const int64_t at = (int64_t)n * a.G + c0 / a.cg + i;
            if (chunk == 0 && a.mean) a.mean[at] = m;
            if (chunk == 0 && a.rstd) a.rstd[at] = r;
        }
    }
    __syncthreads();
    float mu[V], rs[V], ga[V], be[V];
    uint32_t gi[V];
    group_of<V>(nv > 0 ? g.col * V : 0, a.cg, gi);
    for (int j = 0; j < V; ++j) {
        const uint32_t i = j < nv ? gi[j] : 0;
        mu[j] = sh[i], rs[j] = sh[ng + i];
    }
    load_param<V>(a.gamma, c, nv, 1.0f, ga);
    load_param<V>(a.beta, c, nv, 0.0f, be);
    const uint32_t lo = chunk * a.chunk, hi = min(a.S, lo + a.chunk);
    for (uint32_t s0 = lo + g.row; s0 < hi; s0 += U * g.tr) {
        u32x4 raw[U];
        const int64_t r0 = (int64_t)n * a.S + s0;
#pragma unroll
        for (int k = 0; k < U; ++k)
            raw[k] = load_vec<D>((const char *)a.x + ((r0 + k * g.tr) * a.ldx + c) * E,
                                 s0 + k * g.tr < hi ? nv : 0);
#pragma unroll
        for (int k = 0; k < U; ++k)
            if (s0 + k * g.tr < hi) emit<D, ACT, CK>(a, raw[k], r0 + k * g.tr, c, nv, mu, rs, ga, be);
    }
}

// ---- backward --------------------------------------------------------------

// A vector of the stored input: as it was, or 8-bit codes with their step.
template <int D, bool CK> struct Src;
template <int D> struct Src<D, false> {
    u32x4 v;
    __device__ void load(const GnArgs &a, int64_t r, uint32_t c, int nv)
    {
        v = load_vec<D>((const char *)a.x + (r * a.ldx + c) * Elem<D>::E, nv);
    }
    __device__ void values(float (&f)[Elem<D>::V]) const { Elem<D>::unpack(v, f); }
};
template <int D> struct Src<D, true> {
    uint32_t q[Elem<D>::V / 4], s;
    __device__ void load(const GnArgs &a, int64_t r, uint32_t c, int nv)
    {
        s = 0;
        for (int i = 0; i < Elem<D>::V / 4; ++i) q[i] = 0;
        if (nv > 0) {                    // the pad up to the pitch may be read
            const uint8_t *p = a.rcodes + r * a.pitch + c;
            if constexpr (Elem<D>::V == 8) {
                const u32x2 w = *(const u32x2 *)p;
                q[0] = w[0], q[Elem<D>::V / 4 - 1] = w[1];
            } else {
                q[0] = *(const uint32_t *)p;
            }
            s = a.rscales[r * a.nrun + c / kRun];
        }
    }
    __device__ void values(float (&f)[Elem<D>::V]) const
    {
        for (int i = 0; i < Elem<D>::V / 4; ++i) run_values(q[i], run_step(s), f + 4 * i);
    }
};

template <int V> struct Chan {               // a thread's channels
    float mu[V], rs[V], ga[V], be[V];
};

template <int D, int ACT, bool CK>
__device__ inline void bwd_sums(const Src<D, CK> &x, u32x4 dy, const Chan<Elem<D>::V> &ch,
                                float (&sa)[Elem<D>::V], float (&sb)[Elem<D>::V])
{
    constexpr int V = Elem<D>::V;
    float f[V], d[V];
    x.values(f);
    Elem<D>::unpack(dy, d);
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const float xh = (f[j] - ch.mu[j]) * ch.rs[j];
        const float z = xh * ch.ga[j] + ch.be[j];
        const float dz = act_grad<ACT>(z, d[j]);
        sa[j] += dz;
        sb[j] = __builtin_fmaf(dz, xh, sb[j]);
    }
}

template <int D, int ACT, bool CK>
__device__ inline void bwd_emit(const GnArgs &a, const Src<D, CK> &x, u32x4 dy, int64_t r, uint32_t c, int nv,
                                const Chan<Elem<D>::V> &ch, const float (&s1)[Elem<D>::V],
                                const float (&s2)[Elem<D>::V])
{
    constexpr int V = Elem<D>::V;
    float f[V], d[V];
    x.values(f);
    Elem<D>::unpack(dy, d);
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const float xh = (f[j] - ch.mu[j]) * ch.rs[j];
        const float z = xh * ch.ga[j] + ch.be[j];
        const float dz = act_grad<ACT>(z, d[j]);
        d[j] = ch.rs[j] * (ch.ga[j] * dz - s1[j] - xh * s2[j]);
    }
    if (nv > 0) store_vec<D>((char *)a.dx + (r * a.lddx + c) * Elem<D>::E, Elem<D>::pack(d), nv);
}

// Means of gamma dz and gamma dz xh over each channel's group, from every
// thread's per-channel sums.
template <int V>
__device__ inline void group_means(const Geo &g, float *sh, uint32_t ng, uint32_t cg, uint32_t S, int nv,
                                   const float (&ga)[V], const float (&sa)[V], const float (&sb)[V],
                                   float (&s1)[V], float (&s2)[V])
{
    const uint32_t np = g.parts * (V << g.tcl);
    float *sh2 = sh + np, *gs = sh2 + np;
    for (int j = 0; j < V; ++j) s1[j] = ga[j] * sa[j], s2[j] = ga[j] * sb[j];
    to_parts<V>(s1, g, sh);
    to_parts<V>(s2, g, sh2);
    __syncthreads();
    to_groups<V>(g, sh, ng, cg, gs);
    to_groups<V>(g, sh2, ng, cg, gs + ng);
    __syncthreads();
    const float cnt = (float)((uint64_t)S * cg);
    uint32_t gi[V];
    group_of<V>(nv > 0 ? g.col * V : 0, cg, gi);
    for (int j = 0; j < V; ++j) {
        const uint32_t i = j < nv ? gi[j] : 0;
        s1[j] = gs[i] / cnt, s2[j] = gs[ng + i] / cnt;
    }
}

// The workgroup's per-channel sums, to p[0..C) (sum dz) and p[C..2C) (sum dz xh).
template <int V>
__device__ inline void put_channel_sums(const Geo &g, float *sh, uint32_t c0, uint32_t wc, uint32_t C, float *p,
                                        float (&sa)[V], float (&sb)[V])
{
    const uint32_t wp = V << g.tcl, np = g.parts * wp;
    __syncthreads();
    to_parts<V>(sa, g, sh);
    to_parts<V>(sb, g, sh + np);
    __syncthreads();
    for (uint32_t i = threadIdx.x; i < wc; i += blockDim.x) {
        float a = 0, b = 0;
        for (uint32_t k = 0; k < g.parts; ++k) a += sh[k * wp + i], b += sh[np + k * wp + i];
        p[c0 + i] = a, p[C + c0 + i] = b;
    }
}

template <int V>
__device__ inline void load_stats(const GnArgs &a, uint32_t n, uint32_t c, int nv, Chan<V> &ch)
{
    uint32_t gi[V];
    group_of<V>(nv > 0 ? c : 0, a.cg, gi);
    for (int j = 0; j < V; ++j) {
        const size_t at = (size_t)n * a.G + gi[j];
        ch.mu[j] = j < nv ? a.mean[at] : 0.0f;
        ch.rs[j] = j < nv ? a.rstd[at] : 0.0f;
    }
}

// Resident: nper samples in turn, each read once; per-channel sums over them
// go to one row of the workspace.
template <int D, int ACT, bool CK, int R>
__global__ __launch_bounds__(kBwdThreads) void k_gn_bwd(GnArgs a)
{
    constexpr int V = Elem<D>::V, E = Elem<D>::E;
    extern __shared__ float sh[];
    const Geo g = geometry(a.tcl);
    const uint32_t b = deal(blockIdx.x, gridDim.x);
    const uint32_t p = b / a.nslab, slab = b - p * a.nslab;
    const uint32_t c0 = slab * a.w, wc = min(a.w, a.C - c0), ng = wc / a.cg;
    const uint32_t c = c0 + g.col * V;
    const int nv = (int)wc - (int)(g.col * V);
    const uint32_t n_hi = min(a.N, (p + 1) * a.nper);
    Chan<V> ch;
    load_param<V>(a.gamma, c, nv, 1.0f, ch.ga);
    load_param<V>(a.beta, c, nv, 0.0f, ch.be);
    float ta[V], tb[V];
    for (int j = 0; j < V; ++j) ta[j] = tb[j] = 0;
    for (uint32_t n = p * a.nper; n < n_hi; ++n) {
        const int64_t r0 = (int64_t)n * a.S + g.row;
        Src<D, CK> x[R];
        u32x4 dy[R];
#pragma unroll
        for (int k = 0; k < R; ++k) {
            const int m = g.row + k * g.tr < a.S ? nv : 0;
            const int64_t r = r0 + k * g.tr;
            x[k].load(a, r, c, m);
            dy[k] = load_vec<D>((const char *)a.dy + (r * a.lddy + c) * E, m);
        }
        load_stats<V>(a, n, c, nv, ch);
        float sa[V], sb[V], s1[V], s2[V];
        for (int j = 0; j < V; ++j) sa[j] = sb[j] = 0;
#pragma unroll
        for (int k = 0; k < R; ++k)
            if (g.row + k * g.tr < a.S) bwd_sums<D, ACT, CK>(x[k], dy[k], ch, sa, sb);
        for (int j = 0; j < V; ++j) ta[j] += sa[j], tb[j] += sb[j];
        group_means<V>(g, sh, ng, a.cg, a.S, nv, ch.ga, sa, sb, s1, s2);
#pragma unroll
        for (int k = 0; k < R; ++k)
            if (g.row + k * g.tr < a.S) bwd_emit<D, ACT, CK>(a, x[k], dy[k], r0 + k * g.tr, c, nv, ch, s1, s2);
    }
    if (a.dgamma || a.dbeta) put_channel_sums<V>(g, sh, c0, wc, a.C, a.part + (size_t)p * 2 * a.C, ta, tb);
}

// Split form, first launch: per-channel sums of a chunk, part[sample][chunk][2][C].
template <int D, int ACT, bool CK> __global__ __launch_bounds__(1024) void k_gn_bwd_sums(GnArgs a)
{
    constexpr int V = Elem<D>::V, E = Elem<D>::E, U = 4;
    extern __shared__ float sh[];
    const Geo g = geometry(a.tcl);
    const uint32_t per = a.nchunk * a.nslab;
    const uint32_t b = deal(blockIdx.x, gridDim.x);
    const uint32_t n = b / per, rest = b - n * per, chunk = rest / a.nslab, slab = rest - chunk * a.nslab;
    const uint32_t c0 = slab * a.w, wc = min(a.w, a.C - c0);
    const uint32_t c = c0 + g.col * V;
    const int nv = (int)wc - (int)(g.col * V);
    Chan<V> ch;
    load_param<V>(a.gamma, c, nv, 1.0f, ch.ga);
    load_param<V>(a.beta, c, nv, 0.0f, ch.be);
    load_stats<V>(a, n, c, nv, ch);
    float sa[V], sb[V];
    for (int j = 0; j < V; ++j) sa[j] = sb[j] = 0;
    const uint32_t lo = chunk * a.chunk, hi = min(a.S, lo + a.chunk);
    for (uint32_t s0 = lo + g.row; s0 < hi; s0 += U * g.tr) {
        const int64_t r0 = (int64_t)n * a.S + s0;
        Src<D, CK> x[U];
        u32x4 dy[U];
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int m = s0 + k * g.tr < hi ? nv : 0;
            x[k].load(a, r0 + k * g.tr, c, m);
            dy[k] = load_vec<D>((const char *)a.dy + ((r0 + k * g.tr) * a.lddy + c) * E, m);
        }
#pragma unroll
        for (int k = 0; k < U; ++k)
            if (s0 + k * g.tr < hi) bwd_sums<D, ACT, CK>(x[k], dy[k], ch, sa, sb);
    }
    put_channel_sums<V>(g, sh, c0, wc, a.C, a.part + ((size_t)n * a.nchunk + chunk) * 2 * a.C, sa, sb);
}

// Split form, second launch: joins the chunks' sums, then streams.
template <int D, int ACT, bool CK> __global__ __launch_bounds__(1024) void k_gn_bwd_apply(GnArgs a)
{
    constexpr int V = Elem<D>::V, E = Elem<D>::E, U = 4;
    extern __shared__ float sh[];
    const Geo g = geometry(a.tcl);
    const uint32_t per = a.nchunk * a.nslab;
    const uint32_t b = deal(blockIdx.x, gridDim.x);
    const uint32_t n = b / per, rest = b - n * per, chunk = rest / a.nslab, slab = rest - chunk * a.nslab;
    const uint32_t c0 = slab * a.w, wc = min(a.w, a.C - c0), ng = wc / a.cg;
    const uint32_t c = c0 + g.col * V;
    const int nv = (int)wc - (int)(g.col * V);
    Chan<V> ch;
    load_param<V>(a.gamma, c, nv, 1.0f, ch.ga);
    load_param<V>(a.beta, c, nv, 0.0f, ch.be);
    load_stats<V>(a, n, c, nv, ch);
    float sa[V], sb[V], s1[V], s2[V];
    for (int j = 0; j < V; ++j) sa[j] = sb[j] = 0;
    for (uint32_t k = g.row; k < a.nchunk; k += g.tr) {
        const float *p = a.part + ((size_t)n * a.nchunk + k) * 2 * a.C + c;
        for (int j = 0; j < V; ++j)
            if (j < nv) sa[j] += p[j], sb[j] += p[a.C + j];
    }
    group_means<V>(g, sh, ng, a.cg, a.S, nv, ch.ga, sa, sb, s1, s2);
    const uint32_t lo = chunk * a.chunk, hi = min(a.S, lo + a.chunk);
    for (uint32_t s0 = lo + g.row; s0 < hi; s0 += U * g.tr) {
        const int64_t r0 = (int64_t)n * a.S + s0;
        Src<D, CK> x[U];
        u32x4 dy[U];
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int m = s0 + k * g.tr < hi ? nv : 0;
            x[k].load(a, r0 + k * g.tr, c, m);
            dy[k] = load_vec<D>((const char *)a.dy + ((r0 + k * g.tr) * a.lddy + c) * E, m);
        }
#pragma unroll
        for (int k = 0; k < U; ++k)
            if (s0 + k * g.tr < hi) bwd_emit<D, ACT, CK>(a, x[k], dy[k], r0 + k * g.tr, c, nv, ch, s1, s2);
    }
}

// dgamma, dbeta: the sum over the workspace's rows, in a fixed order.
constexpr uint32_t kParChan = 16, kParRows = 64;
__global__ __launch_bounds__(kParChan * kParRows) void k_gn_params(GnArgs a, uint32_t rows)
{
    __shared__ float sh[2][kParRows][kParChan + 1];
    const uint32_t ci = threadIdx.x % kParChan, ri = threadIdx.x / kParChan;
    const uint32_t c = blockIdx.x * kParChan + ci;
    float s = 0, t = 0;
    if (c < a.C) {
#pragma unroll 4
        for (uint32_t r = ri; r < rows; r += kParRows) {
            const float *p = a.part + (size_t)r * 2 * a.C + c;
            s += p[0], t += p[a.C];
        }
    }
    sh[0][ri][ci] = s, sh[1][ri][ci] = t;
    for (uint32_t h = kParRows / 2; h; h >>= 1) {
        __syncthreads();
        if (ri < h) {
            sh[0][ri][ci] += sh[0][ri + h][ci];
            sh[1][ri][ci] += sh[1][ri + h][ci];
        }
    }
    if (ri == 0 && c < a.C) {
        if (a.dbeta) a.dbeta[c] = a.add ? a.dbeta[c] + sh[0][0][ci] : sh[0][0][ci];
        if (a.dgamma) a.dgamma[c] = a.add ? a.dgamma[c] + sh[1][0][ci] : sh[1][0][ci];
    }
}

uint32_t gcd(uint32_t a, uint32_t b) { return b ? gcd(b, a % b) : a; }

template <typename F> hipError_t by_rows(uint32_t rows, F f)
{
    if (rows <= 1) return f(std::integral_constant<int, 1>());
    if (rows <= 2) return f(std::integral_constant<int, 2>());
    if (rows <= 4) return f(std::integral_constant<int, 4>());
    if (rows <= 8) return f(std::integral_constant<int, 8>());
    return f(std::integral_constant<int, 16>());
}
template <typename F> hipError_t by_type(int dtype, F f)
{
    if (dtype == kF32) return f(std::integral_constant<int, kF32>());
    if (dtype == kBF16) return f(std::integral_constant<int, kBF16>());
    return f(std::integral_constant<int, kF16>());
}
template <typename F> hipError_t by_act(int act, F f)
{
    if (act == kActRelu) return f(std::integral_constant<int, kActRelu>());
    if (act == kActSilu) return f(std::integral_constant<int, kActSilu>());
    return f(std::integral_constant<int, kActNone>());
}
template <typename F> hipError_t by_bool(bool b, F f)
{
    return b ? f(std::true_type()) : f(std::false_type());
}

// LDS of the sums: `arrays` of per-wave channel sums, and `per_group` floats a group.
size_t lds_bytes(const GnPlan &p, uint32_t V, uint32_t cg, uint32_t arrays, uint32_t per_group)
{
    const uint32_t parts = p.tcl >= 6 ? p.threads >> p.tcl : p.threads >> 6;
    return ((size_t)arrays * parts * (V << p.tcl) + (size_t)per_group * (p.w / cg)) * 4;
}

void set_plan(GnArgs &a, const GnPlan &p)
{
    a.w = p.w, a.nslab = p.nslab, a.tcl = p.tcl, a.nchunk = p.nchunk, a.chunk = p.chunk;
    a.nper = p.nper, a.nparts = p.nparts;
}

}  // namespace

// ---- planning --------------------------------------------------------------

GnPlan gn_plan(int dtype, bool backward, uint64_t N, uint64_t S, uint32_t C, uint32_t G)
{
    GnPlan p = {};
    const uint32_t E = elem_bytes(dtype), V = 16 / E, cg = C / G;
    // slabs: whole groups and whole runs, 64 bytes of a row if a few groups give that
    const uint64_t whole = (uint64_t)(cg / gcd(cg, kRun)) * kRun;
    const uint32_t unit = whole < C ? (uint32_t)whole : C;
    if (unit > kSlabMax) return p;
    uint32_t w = unit;
    while (w < C && w * E < 64) w += unit;
    // wider while a 256-thread workgroup would have idle lanes
    while (w < C && (uint64_t)(w + unit) * S <= 256 * V && w + unit <= kSlabMax) w += unit;
    if (w > C) w = C;
    while ((V << p.tcl) < w || (V << p.tcl) < kRun) ++p.tcl;
    p.w = w;
    p.nslab = (C + w - 1) / w;
    const uint64_t vecs = S << p.tcl;              // lanes' vectors of a slab
    const uint32_t most = backward ? kBwdThreads : kFwdThreads;
    p.resident = (1u << p.tcl) <= most &&
                 (vecs <= 256 * 8 || (vecs <= (uint64_t)most * kMostRows && N * p.nslab >= 128));
    if (p.resident) {
        p.threads = 1u << p.tcl;
        if (p.threads < 64) p.threads = 64;
        while (p.threads < most && (uint64_t)p.threads * (backward ? 4 : 8) < vecs) p.threads *= 2;
        p.rows = (uint32_t)((vecs + p.threads - 1) / p.threads);
        // backward: several samples a workgroup where there are far more than fill the GPU
        uint64_t nper = 1;
        while (N * p.nslab / nper > 4096 && nper < N) nper *= 2;
        p.nper = (uint32_t)nper;
        p.nparts = (uint32_t)((N + nper - 1) / nper);
    } else {
        p.threads = 1u << p.tcl;
        if (p.threads < 256) p.threads = 256;
        p.rows = kStatRows;
        // chunks: about 2048 workgroups, whole sub-chunks each
        const uint64_t sweep = (uint64_t)(p.threads >> p.tcl) * kStatRows;
        uint64_t want = 2048 / (N * p.nslab);
        if (want < 1) want = 1;
        uint64_t chunk = (S + want - 1) / want;
        chunk = (chunk + sweep - 1) / sweep * sweep;
        if (chunk > S) chunk = S;
        p.chunk = (uint32_t)chunk;
        p.nchunk = (uint32_t)((S + chunk - 1) / chunk);
        if (N * p.nchunk > 0x7fffffffull) return GnPlan{};
        p.nparts = (uint32_t)(N * p.nchunk);
    }
    const uint64_t grid = (p.resident ? N : N * p.nchunk) * p.nslab;
    return grid <= 0x7fffffffull ? p : GnPlan{};
}

size_t gn_part_floats(const GnPlan &p, bool backward, uint64_t N, uint32_t C, uint32_t G)
{
    if (backward) return (size_t)p.nparts * 2 * C;
    return p.resident ? 0 : (size_t)N * G * p.nchunk * 2;
}

hipError_t launch_gn_forward(const GnPlan &p, GnArgs a, int dtype, int act, hipStream_t s)
{
    set_plan(a, p);
    const uint32_t V = 16 / elem_bytes(dtype);
    return by_type(dtype, [&](auto D) {
        if (!p.resident) {
            const uint32_t grid = a.N * p.nchunk * p.nslab;
            k_gn_stats<D(), kStatRows><<<grid, p.threads, lds_bytes(p, V, a.cg, 1, 4), s>>>(a);
            if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
            return by_act(act, [&](auto A) {
                return by_bool(a.wcodes != nullptr, [&](auto K) {
                    k_gn_apply<D(), A(), K()><<<grid, p.threads, lds_bytes(p, V, a.cg, 0, 2), s>>>(a);
                    return hipGetLastError();
                });
            });
        }
        return by_act(act, [&](auto A) {
            return by_bool(a.wcodes != nullptr, [&](auto K) {
                return by_rows(p.rows, [&](auto R) {
                    k_gn_fwd<D(), A(), K(), R()>
                        <<<a.N * p.nslab, p.threads, lds_bytes(p, V, a.cg, 1, 2), s>>>(a);
                    return hipGetLastError();
                });
            });
        });
    });
}

hipError_t launch_gn_backward(const GnPlan &p, GnArgs a, int dtype, int act, hipStream_t s)
{
    set_plan(a, p);
    const uint32_t V = 16 / elem_bytes(dtype);
    if (a.N && a.S) {
        const size_t lds = lds_bytes(p, V, a.cg, 2, 2);
        const hipError_t e = by_type(dtype, [&](auto D) {
            return by_act(act, [&](auto A) {
                return by_bool(a.rcodes != nullptr, [&](auto K) {
                    if (!p.resident) {
                        const uint32_t grid = a.N * p.nchunk * p.nslab;
                        k_gn_bwd_sums<D(), A(), K()><<<grid, p.threads, lds, s>>>(a);
                        if (hipError_t f = hipGetLastError(); f != hipSuccess) return f;
                        k_gn_bwd_apply<D(), A(), K()><<<grid, p.threads, lds, s>>>(a);
                        return hipGetLastError();
                    }
                    return by_rows(p.rows, [&](auto R) {
                        k_gn_bwd<D(), A(), K(), R()><<<p.nparts * p.nslab, p.threads, lds, s>>>(a);
                        return hipGetLastError();
                    });
                });
            });
        });
        if (e != hipSuccess) return e;
    }
    if (!a.dgamma && !a.dbeta) return hipSuccess;
    k_gn_params<<<(a.C + kParChan - 1) / kParChan, kParChan * kParRows, 0, s>>>(a, a.N && a.S ? p.nparts : 0);
    return hipGetLastError();
}

}  // namespace lags
