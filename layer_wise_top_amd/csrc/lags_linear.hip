// Linear layers: plans, and the choice of the element type.
#include "lags_gn.h"
#include "lags_layer.h"

#include <algorithm>
#include <cmath>

namespace lags {
namespace {

// dbias: sums over part's rows, in a fixed order; 64 columns a workgroup, a wave each
// sixteenth of the rows.
constexpr uint32_t kBiasWaves = 16;
__global__ __launch_bounds__(64 * kBiasWaves) void k_linear_dbias(const float *part, uint32_t rows, uint32_t N,
                                                                  float *dbias, uint32_t add)
{
    __shared__ float sh[kBiasWaves][64];
    const uint32_t w = threadIdx.x >> 6, l = threadIdx.x & 63, n = blockIdx.x * 64 + l;
    float s = 0;
    if (n < N) {
#pragma unroll 4
        for (uint32_t r = w; r < rows; r += kBiasWaves) s += part[(size_t)r * N + n];
    }
    sh[w][l] = s;
    __syncthreads();
    if (w || n >= N) return;
    for (uint32_t k = 1; k < kBiasWaves; ++k) s += sh[k][l];
    dbias[n] = add ? dbias[n] + s : s;
}

}  // namespace

namespace {
// Microseconds that a tile takes a step of 128 bytes of k on a compute unit that is full of them
// (`alone`: when it is the only one on an idle card), and for its results, and how many a compute unit
// holds: 16-bit values, the same with W as it comes (backward), and fp32, whose steps are half as long.
// Fitted to 620 products of 16 to 16384 rows and 64 to 8192 columns and outputs, each in every tile and up to 27
// slices: the plan's time is 1.015, 1.03 and 1.016 of the best measured one, geometric mean.  Up to 64 rows of 16
// bits take W from memory, not from a cache that others' reads have filled, and `alone` is 2 (backward 1.5)
// times that: over 107 products of 1 to 64 rows with W not in any cache 1.05 and 1.07 of the best of these tiles,
// without it 1.15 and 1.10.  Their tiles are mostly empty there, and reading W once would take 1.2 to 2.9 times less.
// Operands staged through registers take the same plan, so that sums have the same order, though not the same times.
struct Cost {
    float full, alone, out;
    int held;
};
constexpr Cost kCost[3][4] = {
    {{1.60f, 0.94f, 3.4f, 1}, {0.46f, 0.67f, 1.2f, 2}, {0.246f, 0.342f, 0.31f, 4}, {0.56f, 0.37f, 0.25f, 3}},
    {{2.00f, 0.95f, 3.5f, 1}, {0.54f, 0.92f, 1.2f, 2}, {0.232f, 0.593f, 0.26f, 5}, {0.23f, 0.60f, 0.29f, 4}},
    {{7.7f, 7.2f, 10.9f, 1}, {1.98f, 2.15f, 2.0f, 2}, {0.556f, 0.736f, 0.20f, 4}, {0.577f, 0.727f, 0.34f, 3}}};
}  // namespace

// The tile and the slices of k with the least time by a model of it (`least`): the rounds of workgroups on 256
// compute units, or the bytes of the operands; then the slices' sums, written and read again.
//   700 x 6000 to 1500 fp32   114 to 119 us (128 x 128, 7 slices; 64 x 64 in 6: 121, whole 193), the library's
//                             product 113
//   1 x 2048 to 8192 bf16     9.5 us with W in the caches, 13.6 with W from memory (32 x 128, 4 slices; W's bytes at
//                             the rate of a copy 6.5; the library's product 17 and 13)
static LinPlan plan_of(int dtype, bool backward, int64_t M, int64_t N, int64_t K, double &least)
{
    const int64_t e = elem_bytes(dtype), ks = 128 / e, steps = (K + ks - 1) / ks;
    const double in = (double)(M * K + N * K) * e / 5e6, sums = (double)M * N * 4 / 5e6;
    const double far = dtype == kF32 || M > 64 ? 1 : backward ? 1.5 : 2;
    LinPlan best = {};
    least = 0;
    for (uint32_t t = 0; t < 4; ++t) {
        const Cost &c = kCost[dtype == kF32 ? 2 : backward][t];
        LinPlan p = {};
        p.tile = t;
        p.tm = (uint32_t)((M + kLinTiles[t].bm - 1) / kLinTiles[t].bm);
        p.tn = (uint32_t)((N + kLinTiles[t].bn - 1) / kLinTiles[t].bn);
        const double tiles = (double)p.tm * p.tn;
        int64_t last = 0;
        for (int64_t want = 1; want <= 32 && want <= steps; want += want < 4 ? 1 : want / 4) {
            const int64_t per = (steps + want - 1) / want;
            if (per == last) continue;
            last = per;
            p.k_per = (uint32_t)std::min(per * ks, K);
            p.split = (uint32_t)((steps + per - 1) / per);
            // whole rounds of all the card holds, and the rest; a card that is part idle runs faster
            const double units = tiles * p.split / 256, whole = std::floor(units / c.held) * c.held;
            const double rest = units - whole, some = rest > 1 ? 1 : rest * rest;
            const double alone = c.alone * far;
            const double step = whole * c.full + (rest ? std::fmax(std::ceil(rest) * c.full, alone) * some +
                                                             alone * (1 - some) : 0);
            double us = std::fmax(per * step, in) + std::ceil(units) * c.out;
            if (p.split > 1) us += 4.5 + 0.22 * p.split + sums * (p.split + 1);     // another launch, loads in turn
            if (!least || us < least) least = us, best = p;
        }
    }
    return best;
}

LinPlan linear_plan(int dtype, bool backward, int64_t M, int64_t N, int64_t K)
{
    double as_is, turned;
    LinPlan p = plan_of(dtype, backward, M, N, K, as_is);
    // A large backward product of 16-bit values takes W turned round, in the workspace, rather than
    // staged as it comes and transposed on the way to the registers; the plan is then the same for
    // operands that cannot use it, whose sums have the same order.
    if (!backward || dtype == kF32 || K % 8 || N * K > (int64_t)1 << 35) return p;      // more would be more threads than a launch has
    LinPlan q = plan_of(dtype, false, M, N, K, turned);
    if (turned + 4.5 + (double)N * K * 4 / 3.5e6 >= as_is) return p;
    q.turn = true;
    return q;
}

// 2^tl lanes of 16-byte vectors a slab, rows in chunks of about 2048 workgroups; up to 256 rows one chunk
// and narrow slabs, so that the column sums are whole in one launch (whole backward of 128 x 512 x 512 fp16 13.4
// -> 11.8 us; of 1000 x 300 x 2000 bf16 23 -> 40, too few workgroups).
DzPlan dz_plan(int dtype, int64_t M, int64_t N)
{
    DzPlan p = {};
    const bool one = M <= 256;
    const uint32_t V = 16 / elem_bytes(dtype);
    const uint64_t vecs = (N + V - 1) / V;
    while (p.tl < (one ? 3 : 6) && (1u << p.tl) < vecs) ++p.tl;
    p.nslab = (uint32_t)((vecs + (1u << p.tl) - 1) >> p.tl);
    const int64_t rows = (int64_t)(256 >> p.tl) * 4;         // a workgroup's in one round
    const int64_t chunks = one ? 1 : std::max<int64_t>(1, 2048 / p.nslab);
    p.rows_per = std::max<int64_t>(1, (M + chunks - 1) / chunks);
    p.rows_per = (p.rows_per + rows - 1) / rows * rows;
    p.chunks = (uint32_t)((M + p.rows_per - 1) / p.rows_per);
    return p;
}

hipError_t launch_linear(const LinPlan &p, const LinArgs &a, bool nn, int how, int dtype, hipStream_t s)
{
    return dtype == kF32 ? product<kF32>(p, a, nn, how, s)
           : dtype == kBF16 ? product<kBF16>(p, a, nn, how, s)
                            : product<kF16>(p, a, nn, how, s);
}
hipError_t launch_slopes(const DzPlan &p, const LinArgs &a, int dtype, hipStream_t s)
{
    return dtype == kF32 ? slopes<kF32>(p, a, s) : dtype == kBF16 ? slopes<kBF16>(p, a, s) : slopes<kF16>(p, a, s);
}
hipError_t launch_dbias(const float *part, uint32_t rows, uint32_t N, float *dbias, uint32_t add, hipStream_t s)
{
    k_linear_dbias<<<(N + 63) / 64, 64 * kBiasWaves, 0, s>>>(part, rows, N, dbias, add);
    return hipGetLastError();
}

}  // namespace lags
