// The router: the joining of what the blocks leave, the workspace's layout and the
// choice of the element type.  The kernels over the rows are in fc_router.cuh; each
// element type is compiled in a file of its own, so that they build side by side.
#include <algorithm>
#include <mutex>
#include <new>
#include <set>
#include <utility>

#include "fc_router.cuh"

namespace fc {

extern template cudaError_t router_forward<float>(const RouterForward &, const RouterCut &, cudaStream_t);
extern template cudaError_t router_forward<__half>(const RouterForward &, const RouterCut &,
                                                  cudaStream_t);
extern template cudaError_t router_forward<__nv_bfloat16>(const RouterForward &, const RouterCut &,
                                                  cudaStream_t);
extern template cudaError_t router_backward<float>(const RouterBackward &, const RouterCut &,
                                                  cudaStream_t);
extern template cudaError_t router_backward<__half>(const RouterBackward &, const RouterCut &,
                                                  cudaStream_t);
extern template cudaError_t router_backward<__nv_bfloat16>(const RouterBackward &, const RouterCut &,
                                                  cudaStream_t);

// Adds the parts of 32 experts of one group, 32 threads to an expert, and leaves
// their share of the balance loss; the last block adds the shares, in their order.
__global__ void __launch_bounds__(1024)
    k_router_join(const RouterForward a, const int parts)
{
    __shared__ float s_p[32][33];
    __shared__ int s_c[32][33];
    __shared__ float s_w[32];
    __shared__ int s_n, s_last;
    __shared__ float s_b[32], s_z[32];
    wait_for_prior_grid();
    allow_dependent_launch();
    const int E = a.n.experts, tiles = (E + 31) / 32;
    const int64_t group = blockIdx.x / tiles;
    const int tile = (int)(blockIdx.x - group * tiles);
    const RouterWs ws = router_ws(a.ws, a.n.groups, parts, E);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int e = tile * 32 + lane;
    float p = 0.f;
    int c = 0;
    if (e < E) {
#pragma unroll 4
        for (int i = warp; i < parts; i += 32) {
            p += __ldcg(ws.probs + (group * parts + i) * E + e);
            c += __ldcg(ws.counts + (group * parts + i) * E + e);
        }
    }
    s_p[warp][lane] = p;
    s_c[warp][lane] = c;
    if (warp == 0) {
        int n = 0;
        float z = 0.f;
        for (int i = lane; i < parts; i += 32) {
            n += __ldcg(ws.routed + group * parts + i);
            z += __ldcg(ws.z + group * parts + i);
        }
        n = __reduce_add_sync(0xffffffffu, n);
        z = warp_sum_f32(z);
        if (lane == 0) {
            s_n = n;
            s_w[0] = z;
        }
    }
    __syncthreads();
    const int n = s_n;
    const float each = 1.f / (float)max(n, 1);
    if (warp == 0) {
        p = 0.f;
        c = 0;
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            p += s_p[i][lane];
            c += s_c[i][lane];
        }
        p *= each;
        if (e < E) {
            a.probs[group * E + e] = p;
            a.counts[group * E + e] = c;
        }
        const float b = warp_sum_f32(e < E ? (float)c * p : 0.f);
        if (lane == 0) {
            if (tile == 0) a.routed[group] = n;
            float *const share = ws.share + 2 * (group * tiles + tile);
            share[0] = b * each * ((float)E / (float)a.n.k);
            share[1] = tile == 0 ? s_w[0] * each : 0.f;
            __threadfence();
            s_last = atomicAdd(ws.done, 1u) + 1 == gridDim.x;
        }
    }
    __syncthreads();
    if (!s_last) return;
    __threadfence();
    float b = 0.f, z = 0.f;
    for (int64_t i = threadIdx.x; i < (int64_t)gridDim.x; i += 1024) {
        b += __ldcg(ws.share + 2 * i);
        z += __ldcg(ws.share + 2 * i + 1);
    }
    b = warp_sum_f32(b);
    z = warp_sum_f32(z);
    if (lane == 0) {
        s_b[warp] = b;
        s_z[warp] = z;
    }
    __syncthreads();
    if (warp == 0) {
        b = warp_sum_f32(s_b[lane]);
        z = warp_sum_f32(s_z[lane]);
        if (lane == 0) {
            a.loss[0] = b / (float)a.n.groups;
            a.loss[1] = z / (float)a.n.groups;
        }
    }
}

cudaError_t router_allow(const void *kernel)
{
    static std::mutex mu;
    // never destroyed: calls may come from threads that outlive the statics
    static auto *const done = new (std::nothrow) std::set<std::pair<const void *, int>>;
    int dev = 0;
    cudaGetDevice(&dev);
    std::lock_guard<std::mutex> lock(mu);
    if (done && done->count({kernel, dev})) return cudaSuccess;
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 200 * 1024);
    if (e != cudaSuccess) return e;
    try {
        if (done) done->insert({kernel, dev});
    } catch (const std::bad_alloc &) {  // set again next time
    }
    return cudaSuccess;
}

int64_t router_parts(int64_t sequences, int64_t tokens, int64_t groups)
{
    if (sequences * tokens == 0) return 1;
    return std::min<int64_t>(sequences * tokens / groups, std::max<int64_t>(1, 1216 / groups));
}

size_t router_workspace(int64_t sequences, int64_t tokens, int64_t experts, int64_t groups)
{
    const int64_t parts = router_parts(sequences, tokens, groups);
    const int64_t words = groups * parts * (2 * experts + 2) + 2 * groups * ((experts + 31) / 32) + 1;
    return (size_t)((words * 4 + 255) / 256 * 256);
}

// Rows of a warp at a time: 32, so that every lane has one where lanes take rows, but
// fewer where that would leave warps of the GPU without any; at least as many as lie
// side by side.
static RouterCut router_cut(const RouterShape &n)
{
    const int64_t rows = n.sequences * n.tokens, per = rows / n.groups;
    int beside = 32;
    while (beside > 1 && 256 / beside < n.experts) beside /= 2;
    RouterCut c = {};
    c.rows = 32;
    while (c.rows > beside && rows / c.rows < 2432) c.rows /= 2;
    c.warps = FC_ROUTER_WARPS;
    while (c.warps > 1 && per <= (int64_t)c.rows * (c.warps / 2)) c.warps /= 2;
    const int64_t most = router_parts(n.sequences, n.tokens, n.groups);
    c.parts = (int)std::max<int64_t>(1, std::min(most, (per + c.rows * c.warps - 1) / (c.rows * c.warps)));
    c.joins = n.groups * c.parts <= FC_ROUTER_JOIN;
    return c;
}

cudaError_t launch_router_forward(const RouterForward &a, int type, cudaStream_t s)
{
    const RouterCut cut = router_cut(a.n);
    cudaError_t e;
    if (type == FC_TYPE_F32)
        e = router_forward<float>(a, cut, s);
    else if (type == FC_TYPE_F16)
        e = router_forward<__half>(a, cut, s);
    else
        e = router_forward<__nv_bfloat16>(a, cut, s);
    if (e != cudaSuccess || cut.joins) return e;
    const unsigned tiles = (unsigned)((a.n.experts + 31) / 32);
    return launch_after_prior(k_router_join, (unsigned)(a.n.groups * tiles), 1024, 0, s, a, cut.parts);
}

cudaError_t launch_router_backward(const RouterBackward &a, int type, cudaStream_t s)
{
    const RouterCut cut = router_cut(a.n);
    if (type == FC_TYPE_F32) return router_backward<float>(a, cut, s);
    if (type == FC_TYPE_F16) return router_backward<__half>(a, cut, s);
    return router_backward<__nv_bfloat16>(a, cut, s);
}

}  // namespace fc
