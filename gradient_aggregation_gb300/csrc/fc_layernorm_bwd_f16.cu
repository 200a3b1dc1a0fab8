#include "fc_layernorm_bwd.cuh"

namespace fc {

template cudaError_t ln_backward<__half>(const LnBackward &, cudaStream_t);

}  // namespace fc
