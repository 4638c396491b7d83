// cake_gg_route_narrow.cu -- routing kernels for up to 256 experts.
#include "cake_gg_route.cuh"

namespace cakegg {

template cudaError_t launch_route<1>(const RouteParams &, int, bool, size_t, cudaStream_t);
template cudaError_t launch_route_grad_whole<1>(const RouteGradParams &, cudaStream_t);
template cudaError_t launch_route<2>(const RouteParams &, int, bool, size_t, cudaStream_t);
template cudaError_t launch_route_grad_whole<2>(const RouteGradParams &, cudaStream_t);
template cudaError_t launch_route<4>(const RouteParams &, int, bool, size_t, cudaStream_t);
template cudaError_t launch_route_grad_whole<4>(const RouteGradParams &, cudaStream_t);
template cudaError_t launch_route<8>(const RouteParams &, int, bool, size_t, cudaStream_t);
template cudaError_t launch_route_grad_whole<8>(const RouteGradParams &, cudaStream_t);

cudaError_t launch_route_grad(const RouteGradParams &p, cudaStream_t stream)
{
    int lanes = 1;
    while (lanes < p.top_k) lanes *= 2;
    const int64_t blocks = (p.T + 256 / lanes - 1) / (256 / lanes);
    return p.bf16 ? route_launch(route_grad_kernel<uint16_t>, p, blocks, 256, 0, 1, stream)
                  : route_launch(route_grad_kernel<float>, p, blocks, 256, 0, 1, stream);
}

}  // namespace cakegg
