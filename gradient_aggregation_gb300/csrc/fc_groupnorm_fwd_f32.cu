#include "fc_groupnorm_fwd.cuh"

namespace fc {

template cudaError_t gn_forward<float>(const GnForward &, int, cudaStream_t);

}  // namespace fc
