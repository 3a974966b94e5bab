// The linear layer's kernels for one element type.
#include "lags_linear.h"

namespace lags {
template hipError_t product<kF16>(const LinPlan &, LinArgs, bool, int, hipStream_t);
template hipError_t slopes<kF16>(const DzPlan &, LinArgs, hipStream_t);
}  // namespace lags
