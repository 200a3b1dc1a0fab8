#include "fc_router.cuh"

namespace fc {

template cudaError_t router_forward<__nv_bfloat16>(const RouterForward &, const RouterCut &, cudaStream_t);
template cudaError_t router_backward<__nv_bfloat16>(const RouterBackward &, const RouterCut &, cudaStream_t);

}  // namespace fc
