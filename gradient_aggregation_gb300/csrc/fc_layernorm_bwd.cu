// Layer norm, backward: the joining of the blocks' column sums, and the choice
// of the element type.  The kernels are in fc_layernorm_bwd.cuh; each element
// type is compiled in a file of its own, so that they build side by side.
#include "fc_layernorm_bwd.cuh"

namespace fc {

extern template cudaError_t ln_backward<float>(const LnBackward &, cudaStream_t);
extern template cudaError_t ln_backward<__half>(const LnBackward &, cudaStream_t);
extern template cudaError_t ln_backward<__nv_bfloat16>(const LnBackward &, cudaStream_t);

// Adds `parts` sets of column sums; blockIdx.y: 0 for dweight, 1 for dbias.
// 32 columns a block, each by 32 threads that take every 32nd set, all their
// loads in flight.
#define FC_LN_JOIN 32

__global__ void __launch_bounds__(32 * FC_LN_JOIN)
    k_ln_join(const float *__restrict__ partials, const int parts, const int64_t cols,
              const int64_t padded, void *dweight, void *dbias, const int gtype)
{
    __shared__ float sm[FC_LN_JOIN][33];
    wait_for_prior_grid();
    allow_dependent_launch();
    void *out = blockIdx.y ? dbias : dweight;
    if (!out) return;
    const int lane = threadIdx.x & 31, q = threadIdx.x >> 5;
    const int64_t c = (int64_t)blockIdx.x * 32 + lane;
    const float *p = partials + (int64_t)blockIdx.y * parts * padded + c;
    float s = 0.f;
    if (c < cols) {
#pragma unroll 10
        for (int i = q; i < parts; i += FC_LN_JOIN) s += __ldcg(p + i * padded);
    }
    sm[q][lane] = s;
    __syncthreads();
    if (q == 0 && c < cols) {
        s = 0.f;
#pragma unroll
        for (int i = 0; i < FC_LN_JOIN; ++i) s += sm[i][lane];
        store_sum(out, gtype, c, s);
    }
}

// As many sets as blocks leave, and no more than rows.  Several blocks an SM up to
// 256 columns; one above (a GB300 has 152 to 160 SMs), and two to a row where rows
// go in halves whatever their type; beyond 16384 columns as many as make 4096 blocks
// of 128 columns.
int64_t ln_max_parts(int64_t rows, int64_t cols)
{
    const int64_t strips = (cols + 127) / 128;
    const int64_t most = cols <= 256     ? 1024
                         : cols <= 12288 ? 160
                         : cols <= 16384 ? 80
                                         : std::max<int64_t>(1, 4096 / strips);
    return std::min(rows, most);
}

cudaError_t ln_join(const LnBackward &a, int parts, cudaStream_t s)
{
    if (!a.partials) return cudaSuccess;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((a.cols + 31) / 32), 2);
    cfg.blockDim = dim3(32 * FC_LN_JOIN);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k_ln_join, (const float *)a.partials, parts, a.cols,
                              ln_padded(a.cols), a.dweight, a.dbias, a.gtype);
}

cudaError_t launch_ln_backward(const LnBackward &a, int type, cudaStream_t s)
{
    if (a.rows == 0) return ln_join(a, 0, s);
    if (type == FC_TYPE_F32) return ln_backward<float>(a, s);
    if (type == FC_TYPE_F16) return ln_backward<__half>(a, s);
    return ln_backward<__nv_bfloat16>(a, s);
}

}  // namespace fc
