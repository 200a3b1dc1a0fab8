#include "fc_router.cuh"

namespace fc {

template cudaError_t router_forward<float>(const RouterForward &, const RouterCut &, cudaStream_t);
template cudaError_t router_backward<float>(const RouterBackward &, const RouterCut &, cudaStream_t);

}  // namespace fc
