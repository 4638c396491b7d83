// cake_gg_route_widest.cu -- routing kernels for up to 1024 experts.
#include "cake_gg_route.cuh"

namespace cakegg {

template cudaError_t launch_route<32>(const RouteParams &, int, bool, size_t, cudaStream_t);
template cudaError_t launch_route_grad_whole<32>(const RouteGradParams &, cudaStream_t);

}  // namespace cakegg
