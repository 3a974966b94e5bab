// 8-bit activation checkpoints: pack and unpack.
//
// A run of 32 consecutive columns of a row is held as 32 signed bytes and one
// power-of-two step (lags_act.h).  Both directions are one pass over the data
// and bound by memory: a lane takes one 16-byte vector of the matrix (four or
// eight lanes a run, the largest magnitude found by lane exchanges), so a
// wave's accesses to the matrix are 1 KiB without gaps.
// 16384 x 8192 bf16: pack 87 us (4.7 TB/s; a large copy reaches 5.0), unpack
// 63 us (6.5 TB/s: the checkpoint is still in the 256 MB cache).  2048 x 64
// fp32: 3 us each, a launch.
#include "lags_act.h"

namespace lags {
namespace {

constexpr int kThreads = 256;
constexpr int kVecs = 4;          // vectors a thread, all requested before the first is used

struct Slot {
    int64_t row;
    uint32_t vec;
};

// Vector `i` past the workgroup's first one: the division of the first slot
// by the vectors of a row is scalar work, the rest a multiply.
__device__ inline Slot slot_at(const PackArgs &a, int64_t row0, uint32_t rem0, uint32_t i)
{
    const uint32_t t = rem0 + i;
    const uint32_t q = (uint32_t)(((uint64_t)t * a.magic) >> 32) >> a.shift;
    return {row0 + q, t - q * a.nvp};
}

template <int D> __global__ __launch_bounds__(kThreads) void k_pack(PackArgs a)
{
    constexpr int V = Elem<D>::V, E = Elem<D>::E;
    const int64_t first = (int64_t)blockIdx.x * (kThreads * kVecs);
    const int64_t row0 = first / a.nvp;
    const uint32_t rem0 = (uint32_t)(first - row0 * a.nvp);
    Slot sl[kVecs];
    u32x4 v[kVecs];
    int n[kVecs];
#pragma unroll
    for (int u = 0; u < kVecs; ++u) {
        sl[u] = slot_at(a, row0, rem0, u * kThreads + threadIdx.x);
        n[u] = sl[u].row < a.s.rows ? (int)a.s.cols - (int)(sl[u].vec * V) : 0;
        v[u] = load_vec<D>((const char *)a.src + (sl[u].row * a.ld + sl[u].vec * V) * E, n[u]);
    }
#pragma unroll
    for (int u = 0; u < kVecs; ++u) {
        const uint32_t s = run_scale(run_top<V>(Elem<D>::top(v[u])));
        float f[V];
        uint32_t q[V / 4];
        Elem<D>::unpack(v[u], f);
        run_codes<V>(f, s, q);
        const uint32_t c = sl[u].vec * V;
        if (sl[u].row >= a.s.rows) continue;
        if (c < a.s.pitch) {             // the pad up to the pitch gets zeros
            uint8_t *p = (uint8_t *)a.dst + sl[u].row * a.s.pitch + c;
            if constexpr (V == 8)
                *(u32x2 *)p = u32x2{q[0], q[1]};
            else
                *(uint32_t *)p = q[0];
        }
        if (c % kRun == 0) a.wscale[sl[u].row * a.s.nrun + c / kRun] = (uint8_t)s;
    }
}

template <int D> __global__ __launch_bounds__(kThreads) void k_unpack(PackArgs a)
{
    constexpr int V = Elem<D>::V, E = Elem<D>::E;
    const int64_t first = (int64_t)blockIdx.x * (kThreads * kVecs);
    const int64_t row0 = first / a.nvp;
    const uint32_t rem0 = (uint32_t)(first - row0 * a.nvp);
    Slot sl[kVecs];
    uint32_t q[kVecs][V / 4], s[kVecs];
    int n[kVecs];
#pragma unroll
    for (int u = 0; u < kVecs; ++u) {
        sl[u] = slot_at(a, row0, rem0, u * kThreads + threadIdx.x);
        const uint32_t c = sl[u].vec * V;
        n[u] = sl[u].row < a.s.rows ? (int)a.s.cols - (int)c : 0;
        if (n[u] > 0) {
            const uint8_t *p = (const uint8_t *)a.src + sl[u].row * a.s.pitch + c;
            if constexpr (V == 8) {
                const u32x2 w = *(const u32x2 *)p;
                q[u][0] = w[0], q[u][V / 4 - 1] = w[1];
            } else {
                q[u][0] = *(const uint32_t *)p;
            }
            s[u] = a.rscale[sl[u].row * a.s.nrun + c / kRun];
        }
    }
#pragma unroll
    for (int u = 0; u < kVecs; ++u) {
        if (n[u] <= 0) continue;
        float f[V];
        for (int i = 0; i < V / 4; ++i) run_values(q[u][i], run_step(s[u]), f + 4 * i);
        store_vec<D>((char *)a.dst + (sl[u].row * a.ld + sl[u].vec * V) * E, Elem<D>::pack(f), n[u]);
    }
}

uint32_t vectors_a_row(const CkptShape &s, int dtype) { return s.nrun * (kRun * elem_bytes(dtype) / 16); }

// nvp, and the multiply-shift that divides by it exactly for every value
// below 2^31 (a workgroup's slots stay below nvp + kThreads * kVecs).  Returns the workgroups.
uint32_t plan(PackArgs &a, int dtype)
{
    a.nvp = vectors_a_row(a.s, dtype);
    uint32_t l = 0;
    while ((uint64_t)1 << l < a.nvp) ++l;
    // ceil(2^(32+l-1) / nvp) for l >= 1 stays below 2^32 and is exact below 2^31
    if (l == 0) {
        a.magic = 0x80000000u, a.shift = 0;      // nvp = 1 does not occur: a run has 4 vectors at least
    } else {
        a.magic = (uint32_t)((((uint64_t)1 << (31 + l)) + a.nvp - 1) / a.nvp);
        a.shift = l - 1;
    }
    const uint64_t slots = (uint64_t)a.s.rows * a.nvp, per = kThreads * kVecs;
    return (uint32_t)((slots + per - 1) / per);
}

}  // namespace

int64_t pack_rows(const CkptShape &s, int dtype)
{
    constexpr uint64_t per = kThreads * kVecs;
    return (int64_t)(kMostThreads / kThreads * per / vectors_a_row(s, dtype));
}

hipError_t launch_pack(const PackArgs &a0, int dtype, hipStream_t s)
{
    PackArgs a = a0;
    const uint32_t g = plan(a, dtype);
    switch (dtype) {
    case kF32: k_pack<kF32><<<g, kThreads, 0, s>>>(a); break;
    case kBF16: k_pack<kBF16><<<g, kThreads, 0, s>>>(a); break;
    default: k_pack<kF16><<<g, kThreads, 0, s>>>(a); break;
    }
    return hipGetLastError();
}

hipError_t launch_unpack(const PackArgs &a0, int dtype, hipStream_t s)
{
    PackArgs a = a0;
    const uint32_t g = plan(a, dtype);
    switch (dtype) {
    case kF32: k_unpack<kF32><<<g, kThreads, 0, s>>>(a); break;
    case kBF16: k_unpack<kBF16><<<g, kThreads, 0, s>>>(a); break;
    default: k_unpack<kF16><<<g, kThreads, 0, s>>>(a); break;
    }
    return hipGetLastError();
}

}  // namespace lags
