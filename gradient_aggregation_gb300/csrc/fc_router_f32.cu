#include "fc_router.cuh"

namespace fc {

template cudaError_t router_forward<float>(const RouterForward &, int, cudaStream_t);
template cudaError_t router_backward<float>(const RouterBackward &, int, cudaStream_t);

}  // namespace fc
