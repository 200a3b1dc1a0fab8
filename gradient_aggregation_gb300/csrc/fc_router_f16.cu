#include "fc_router.cuh"

namespace fc {

template cudaError_t router_forward<__half>(const RouterForward &, bool *, int *, cudaStream_t);
template cudaError_t router_backward<__half>(const RouterBackward &, cudaStream_t);

}  // namespace fc
