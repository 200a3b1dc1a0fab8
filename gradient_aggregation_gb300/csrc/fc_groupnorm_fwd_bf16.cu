#include "fc_groupnorm_fwd.cuh"

namespace fc {

template cudaError_t gn_forward<__nv_bfloat16>(const GnForward &, int, cudaStream_t);

}  // namespace fc
