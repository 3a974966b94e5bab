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

struct Tile {
    int bm, bn;
};
constexpr Tile kTiles[] = {{256, 256}, {128, 128}, {64, 64}, {32, 128}};

}  // namespace

LinPlan linear_plan(int dtype, int64_t M, int64_t N, int64_t K)
{
    LinPlan p = {};
    const int64_t ks = 128 / elem_bytes(dtype), steps = (K + ks - 1) / ks;
    // large tiles where there are enough of them; slices of k where there are few
    p.tile = M <= 32 ? 3 : 2;
    if (M * N >= (int64_t)128 * 128 * 200) p.tile = 1;
    if (M * N >= (int64_t)256 * 256 * 200) p.tile = 0;
    p.tm = (uint32_t)((M + kTiles[p.tile].bm - 1) / kTiles[p.tile].bm);
    p.tn = (uint32_t)((N + kTiles[p.tile].bn - 1) / kTiles[p.tile].bn);
    int64_t want = std::max<int64_t>(1, std::min<int64_t>(512 / ((int64_t)p.tm * p.tn), steps / 4));
    p.steps_per = (uint32_t)((steps + want - 1) / want);
    p.split = (uint32_t)((steps + p.steps_per - 1) / p.steps_per);
    return p;
}

// 2^tl lanes of 16-byte vectors a slab, rows in chunks of about 2048 workgroups.
DzPlan dz_plan(int dtype, int64_t M, int64_t N)
{
    DzPlan p = {};
    const uint32_t V = 16 / elem_bytes(dtype);
    const uint64_t vecs = (N + V - 1) / V;
    while (p.tl < 6 && (1u << p.tl) < vecs) ++p.tl;
    p.nslab = (uint32_t)((vecs + (1u << p.tl) - 1) >> p.tl);
    const int64_t rows = (int64_t)(256 >> p.tl) * 4;         // a workgroup's in one round
    int64_t chunks = std::max<int64_t>(1, 2048 / p.nslab);
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
