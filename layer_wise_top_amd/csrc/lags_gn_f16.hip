// Group normalisation kernels of one element type.
#include "lags_gn_bwd.h"
#include "lags_gn_fwd.h"

namespace lags {
template hipError_t launch_gn_forward<kF16>(const GnPlan &, const GnArgs &, hipStream_t);
template hipError_t launch_gn_backward<kF16>(const GnPlan &, const GnArgs &, hipStream_t);
}  // namespace lags
