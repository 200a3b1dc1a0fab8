#include "fc_groupnorm_bwd.cuh"

namespace fc {

template cudaError_t gn_backward<__half>(const GnBackward &, int, cudaStream_t);

}  // namespace fc
