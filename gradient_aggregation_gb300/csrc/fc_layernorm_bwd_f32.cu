#include "fc_layernorm_bwd.cuh"

namespace fc {

template cudaError_t ln_backward<float>(const LnBackward &, cudaStream_t);

}  // namespace fc
