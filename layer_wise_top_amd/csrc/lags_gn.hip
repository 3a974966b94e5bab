// Group normalisation: the choice of the element type, and the parameters'
// gradients, whose last sum does not depend on it.
#include "lags_act.h"

namespace lags {
namespace {

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

}  // namespace

hipError_t launch_gn_forward(const GnPlan &p, const GnArgs &a, int dtype, hipStream_t s)
{
    switch (dtype) {
    case kF32: return launch_gn_forward<kF32>(p, a, s);
    case kBF16: return launch_gn_forward<kBF16>(p, a, s);
    default: return launch_gn_forward<kF16>(p, a, s);
    }
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
    if (!a.dgamma && !a.dbeta) return hipSuccess;
    k_gn_params<<<(a.C + kParChan - 1) / kParChan, kParChan * kParRows, 0, s>>>(a, any ? p.nparts : 0);
    return hipGetLastError();
}

}  // namespace lags
