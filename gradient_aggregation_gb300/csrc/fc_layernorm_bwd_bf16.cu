#include "fc_layernorm_bwd.cuh"

namespace fc {

template cudaError_t ln_backward<__nv_bfloat16>(const LnBackward &, cudaStream_t);

}  // namespace fc
