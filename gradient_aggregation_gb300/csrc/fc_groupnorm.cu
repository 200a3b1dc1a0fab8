// Group norm: the workspace's layout and the choice of the element type.  The
// kernels are in fc_groupnorm.cuh; each element type and direction is compiled
// in a file of its own, so that they build side by side.
#include <algorithm>

#include "fc_groupnorm_bwd.cuh"
#include "fc_groupnorm_fwd.cuh"

namespace fc {

extern template cudaError_t gn_forward<float>(const GnForward &, int, cudaStream_t);
extern template cudaError_t gn_forward<__half>(const GnForward &, int, cudaStream_t);
extern template cudaError_t gn_forward<__nv_bfloat16>(const GnForward &, int, cudaStream_t);
extern template cudaError_t gn_backward<float>(const GnBackward &, int, cudaStream_t);
extern template cudaError_t gn_backward<__half>(const GnBackward &, int, cudaStream_t);
extern template cudaError_t gn_backward<__nv_bfloat16>(const GnBackward &, int, cudaStream_t);

// Parts of 64 positions or more, as many as make 1024 blocks over the samples;
// none is empty.
int64_t gn_parts(const GnShape &n)
{
    const int64_t most = std::max<int64_t>(1, 1024 / std::max<int64_t>(1, n.samples));
    const int64_t want = std::min(most, (n.positions + 63) / 64);
    const int64_t rows = (n.positions + want - 1) / want;
    return (n.positions + rows - 1) / rows;
}

int64_t gn_sets(const GnShape &n) { return n.samples * gn_parts(n); }

cudaError_t launch_gn_forward(const GnForward &a, int type, int act, cudaStream_t s)
{
    if (type == FC_TYPE_F32) return gn_forward<float>(a, act, s);
    if (type == FC_TYPE_F16) return gn_forward<__half>(a, act, s);
    return gn_forward<__nv_bfloat16>(a, act, s);
}

cudaError_t launch_gn_backward(const GnBackward &a, int type, int act, cudaStream_t s)
{
    if (a.n.samples == 0) return gn_join(a, 0, s);
    if (type == FC_TYPE_F32) return gn_backward<float>(a, act, s);
    if (type == FC_TYPE_F16) return gn_backward<__half>(a, act, s);
    return gn_backward<__nv_bfloat16>(a, act, s);
}

}  // namespace fc
