#include "fc_router.cuh"

namespace fc {

template cudaError_t router_forward<__nv_bfloat16>(const RouterForward &, bool *, int *, cudaStream_t);
template cudaError_t router_backward<__nv_bfloat16>(const RouterBackward &, cudaStream_t);

}  // namespace fc
