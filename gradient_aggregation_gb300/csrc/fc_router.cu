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

extern template cudaError_t router_forward<float>(const RouterForward &, bool *, int *, cudaStream_t);
extern template cudaError_t router_forward<__half>(const RouterForward &, bool *, int *, cudaStream_t);
extern template cudaError_t router_forward<__nv_bfloat16>(const RouterForward &, bool *, int *, cudaStream_t);
extern template cudaError_t router_backward<float>(const RouterBackward &, cudaStream_t);
extern template cudaError_t router_backward<__half>(const RouterBackward &, cudaStream_t);
extern template cudaError_t router_backward<__nv_bfloat16>(const RouterBackward &, cudaStream_t);

// Adds the parts of 8 experts of one group, ADD / 8 threads to an expert, eight of their
// loads in flight, and leaves their share of the balance loss; the last block adds the
// shares, in their order.
template <int ADD>
__global__ void __launch_bounds__(ADD) k_router_join(const RouterForward a, const int parts)
{
    constexpr int kTeam = ADD / 8, kWarps = ADD / 32;
    __shared__ float s_p[kTeam][9];
    __shared__ int s_c[kTeam][9];
    __shared__ float s_w[kWarps], s_z[kWarps];
    __shared__ int s_n[kWarps], s_last;
    wait_for_prior_grid();
    allow_dependent_launch();
    const int E = a.n.experts, tiles = (E + 7) / 8;
    const int64_t group = blockIdx.x / (unsigned)tiles;
    const int tile = (int)(blockIdx.x - group * tiles);
    const RouterWs ws = router_ws(a.ws, a.n.groups, parts, E);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int q = threadIdx.x >> 3, e = tile * 8 + (threadIdx.x & 7);
    float p = 0.f;
    int c = 0;
    if (e < E) {
        const int64_t at = group * parts * E + e;
#pragma unroll 8
        for (int i = q; i < parts; i += kTeam) {
            p += __ldcg(ws.probs + at + (int64_t)i * E);
            c += __ldcg(ws.counts + at + (int64_t)i * E);
        }
    }
    s_p[q][threadIdx.x & 7] = p;
    s_c[q][threadIdx.x & 7] = c;
    int n = 0;
    float z = 0.f;
    for (int i = threadIdx.x; i < parts; i += ADD) {
        n += __ldcg(ws.routed + group * parts + i);
        z += __ldcg(ws.z + group * parts + i);
    }
    n = __reduce_add_sync(0xffffffffu, n);
    z = warp_sum_f32(z);
    if (lane == 0) {
        s_n[warp] = n;
        s_z[warp] = z;
    }
    __syncthreads();
    n = __reduce_add_sync(0xffffffffu, lane < kWarps ? s_n[lane] : 0);
    z = warp_sum_f32(lane < kWarps ? s_z[lane] : 0.f);
    const float each = 1.f / (float)max(n, 1);
    if (warp < 8) {  // an expert each
        p = 0.f;
        c = 0;
#pragma unroll
        for (int i = 0; i < kTeam; i += 32) {
            p += s_p[i + lane][warp];
            c += s_c[i + lane][warp];
        }
        p = warp_sum_f32(p) * each;
        c = __reduce_add_sync(0xffffffffu, c);
        if (lane == 0) {
            const int w = tile * 8 + warp;
            if (w < E) {
                a.probs[group * E + w] = p;
                a.counts[group * E + w] = c;
            }
            s_w[warp] = w < E ? (float)c * p : 0.f;
        }
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        float b = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) b += s_w[i];
        if (tile == 0) a.routed[group] = n;
        float *const share = ws.share + 2 * (group * tiles + tile);
        share[0] = b * each * ((float)E / (float)a.n.k);
        share[1] = tile == 0 ? z * each : 0.f;
        __threadfence();
        s_last = atomicAdd(ws.done, 1u) + 1 == gridDim.x;
        __threadfence();
    }
    __syncthreads();
    if (!s_last) return;
    float b = 0.f;
    z = 0.f;
    for (int64_t i = threadIdx.x; i < (int64_t)gridDim.x; i += ADD) {
        b += __ldcg(ws.share + 2 * i);
        z += __ldcg(ws.share + 2 * i + 1);
    }
    b = warp_sum_f32(b);
    z = warp_sum_f32(z);
    if (lane == 0) {
        s_w[warp] = b;
        s_z[warp] = z;
    }
    __syncthreads();
    if (warp == 0) {
        b = warp_sum_f32(lane < kWarps ? s_w[lane] : 0.f);
        z = warp_sum_f32(lane < kWarps ? s_z[lane] : 0.f);
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

size_t router_workspace(int64_t sequences, int64_t tokens, int64_t experts, int64_t groups)
{
    const int64_t parts = router_parts(sequences, tokens, groups);
    const int64_t words = groups * parts * (2 * experts + 2) + 2 * groups * ((experts + 7) / 8) + 1;
    return (size_t)((words * 4 + 255) / 256 * 256);
}

cudaError_t launch_router_forward(const RouterForward &a, int type, cudaStream_t s)
{
    bool joins = false;
    int parts = 1;
    cudaError_t e;
    if (type == FC_TYPE_F32)
        e = router_forward<float>(a, &joins, &parts, s);
    else if (type == FC_TYPE_F16)
        e = router_forward<__half>(a, &joins, &parts, s);
    else
        e = router_forward<__nv_bfloat16>(a, &joins, &parts, s);
    if (e != cudaSuccess || joins) return e;
    const unsigned tiles = (unsigned)((a.n.experts + 7) / 8);
    const unsigned grid = (unsigned)(a.n.groups * tiles);
    // one round of loads either way (131072 x 8 bf16: 12.8 us with small blocks, 10.6 with
    // large ones; 16 groups of 2048 x 60 fp32: 11.1 and 12.9)
    if (parts <= 256) return launch_after_prior(k_router_join<256>, grid, 256, 0, s, a, parts);
    return launch_after_prior(k_router_join<1024>, grid, 1024, 0, s, a, parts);
}

cudaError_t launch_router_backward(const RouterBackward &a, int type, cudaStream_t s)
{
    if (type == FC_TYPE_F32) return router_backward<float>(a, s);
    if (type == FC_TYPE_F16) return router_backward<__half>(a, s);
    return router_backward<__nv_bfloat16>(a, s);
}

}  // namespace fc
