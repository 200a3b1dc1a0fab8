#include "fc_layernorm_fwd.cuh"

namespace fc {

template cudaError_t ln_forward<__half>(const LnForward &, cudaStream_t);

}  // namespace fc
