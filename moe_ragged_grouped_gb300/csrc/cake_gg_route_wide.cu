// cake_gg_route_wide.cu -- routing kernels for up to 512 experts.
#include "cake_gg_route.cuh"

namespace cakegg {

template cudaError_t launch_route<16>(const RouteParams &, int, bool, size_t, cudaStream_t);
template cudaError_t launch_route_grad_whole<16>(const RouteGradParams &, cudaStream_t);

}  // namespace cakegg
