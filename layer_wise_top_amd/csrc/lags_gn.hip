// Group normalisation: the choice of the element type, and the parameters'
// gradients, whose last sum does not depend on it.
#include "lags_gn.h"
#include "lags_layer.h"

namespace lags {
namespace {

// dgamma, dbeta: the sum over the workspace's rows, in a fixed order.  A wave
// takes 16 channels by 4 rows, its 15 fellows the next rows.  Bound by the
// latency of a launch and a load: 4.6 us for 64 rows of 512 channels, 2.4 us
// for 32 of 32.
constexpr uint32_t kParChan = 16, kParRows = 64;
__global__ __launch_bounds__(kParChan * kParRows) void k_gn_params(const float *part, uint32_t rows, uint32_t C,
                                                                   float *dgamma, float *dbeta, uint32_t add)
{
    __shared__ float sh[2][kParRows / 4][kParChan];
    const uint32_t ci = threadIdx.x % kParChan, ri = threadIdx.x / kParChan;
    const uint32_t c = blockIdx.x * kParChan + ci;
    float s = 0, t = 0;
    if (c < C) {
#pragma unroll 4
        for (uint32_t r = ri; r < rows; r += kParRows) {
            const float *p = part + (size_t)r * 2 * C + c;
            s += p[0], t += p[C];
        }
    }
    s = swap_sum<32>(swap_sum<16>(s, s), swap_sum<16>(s, s));
    t = swap_sum<32>(swap_sum<16>(t, t), swap_sum<16>(t, t));
    if (ri % 4 == 0) sh[0][ri / 4][ci] = s, sh[1][ri / 4][ci] = t;
    __syncthreads();
    if (threadIdx.x >= 2 * kParChan || c >= C) return;
    const uint32_t which = threadIdx.x / kParChan;         // 0: dbeta, 1: dgamma
    float *out = which ? dgamma : dbeta;
    if (!out) return;
    float u = 0;
    for (uint32_t k = 0; k < kParRows / 4; ++k) u += sh[which][k][ci];
    out[c] = add ? out[c] + u : u;
}

}  // namespace

hipError_t launch_params(const float *part, uint32_t rows, uint32_t C, float *dgamma, float *dbeta, uint32_t add,
                         hipStream_t s)
{
    if (!dgamma && !dbeta) return hipSuccess;
    k_gn_params<<<(C + kParChan - 1) / kParChan, kParChan * kParRows, 0, s>>>(part, rows, C, dgamma, dbeta, add);
    return hipGetLastError();
}

hipError_t launch_gn_forward(const GnPlan &p, const GnArgs &all, int dtype, hipStream_t s)
{
    const uint32_t E = elem_bytes(dtype);
    // samples of one launch (split: all of them, the plan sees to that)
    const uint32_t most = p.resident ? (uint32_t)(kMostThreads / p.threads / p.nslab) : all.N;
    for (uint32_t n = 0; n < all.N;) {
        GnArgs a = all;
        a.N = all.N - n < most ? all.N - n : most;
        const int64_t row = (int64_t)n * a.S, group = (int64_t)n * a.G;
        a.x = (const char *)a.x + row * a.ldx * E, a.y = (char *)a.y + row * a.ldy * E;
        if (a.mean) a.mean += group;
        if (a.rstd) a.rstd += group;
        if (a.wcodes) a.wcodes += row * a.pitch, a.wscales += row * a.nrun;
        const hipError_t e = dtype == kF32    ? launch_gn_forward<kF32>(p, a, s)
                             : dtype == kBF16 ? launch_gn_forward<kBF16>(p, a, s)
                                              : launch_gn_forward<kF16>(p, a, s);
        if (e != hipSuccess) return e;
        n += a.N;
    }
    return hipSuccess;
}

hipError_t launch_gn_backward(const GnPlan &p, const GnArgs &a, int dtype, hipStream_t s)
{
    const bool any = a.N && a.S;
    if (any) {
        const hipError_t e = dtype == kF32    ? launch_gn_backward<kF32>(p, a, s)
                             : dtype == kBF16 ? launch_gn_backward<kBF16>(p, a, s)
                                              : launch_gn_backward<kF16>(p, a, s);
        if (e != hipSuccess) return e;
    }
    return launch_params(a.part, any ? p.nparts : 0, a.C, a.dgamma, a.dbeta, a.add, s);
}

}  // namespace lags
