#include "fc_groupnorm_fwd.cuh"

namespace fc {

template cudaError_t gn_forward<__half>(const GnForward &, int, cudaStream_t);

}  // namespace fc
