// Layer norm, forward: the choice of the element type.  The kernels are in
// fc_layernorm_fwd.cuh; each element type is compiled in a file of its own, so
// that they build side by side.
#include "fc_layernorm_fwd.cuh"

namespace fc {

extern template cudaError_t ln_forward<float>(const LnForward &, cudaStream_t);
extern template cudaError_t ln_forward<__half>(const LnForward &, cudaStream_t);
extern template cudaError_t ln_forward<__nv_bfloat16>(const LnForward &, cudaStream_t);

cudaError_t launch_ln_forward(const LnForward &a, int type, cudaStream_t s)
{
    if (type == FC_TYPE_F32) return ln_forward<float>(a, s);
    if (type == FC_TYPE_F16) return ln_forward<__half>(a, s);
    return ln_forward<__nv_bfloat16>(a, s);
}

}  // namespace fc
