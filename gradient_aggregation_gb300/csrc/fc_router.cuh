// The router of a mixture of experts, for one element type T: softmax over the
// experts, the k largest, and what the balance loss needs; and its gradient.
//
// A warp holds a row, lane l the experts l, l + 32, ...: a lane's experts stay the
// same from row to row, so the sums of the probabilities stay in its registers.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fc.h"
#include "fc_cluster.cuh"
#include "fc_internal.h"
#include "fc_router.h"

namespace fc {

#define FC_ROUTER_BLOCK 256
#define FC_ROUTER_FAR 16.f
#define FC_ROUTER_WARPS (FC_ROUTER_BLOCK / 32)

__device__ __forceinline__ float rt_f32(float x) { return x; }
__device__ __forceinline__ float rt_f32(__half x) { return __half2float(x); }
__device__ __forceinline__ float rt_f32(__nv_bfloat16 x) { return __bfloat162float(x); }

template <class T>
__device__ __forceinline__ T rt_round(float x)
{
    if constexpr (sizeof(T) == 4)
        return x;
    else if constexpr (__is_same(T, __half))
        return __float2half_rn(x);
    else
        return __float2bfloat16_rn(x);
}

// Ordered like the number it stands for: -0 like 0, NaN below everything, and
// above 0 for whatever is more than -infinity.
__device__ __forceinline__ uint32_t rt_key(float x)
{
    const uint32_t u = __float_as_uint(x + 0.f);
    const uint32_t key = u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
    return x > -INFINITY ? key : 0u;
}

// What the blocks leave, and where.
struct RouterWs {
    float *probs;     // [groups][parts][experts]
    int32_t *counts;  // [groups][parts][experts]
    float *z;         // [groups][parts]
    int32_t *routed;  // [groups][parts]
    float *share;     // [groups][tiles][2]
    unsigned *done;
};

__host__ __device__ inline RouterWs router_ws(void *ws, int64_t groups, int64_t parts, int64_t e)
{
    RouterWs w;
    w.probs = static_cast<float *>(ws);
    w.counts = reinterpret_cast<int32_t *>(w.probs + groups * parts * e);
    w.z = reinterpret_cast<float *>(w.counts + groups * parts * e);
    w.routed = reinterpret_cast<int32_t *>(w.z + groups * parts);
    w.share = reinterpret_cast<float *>(w.routed + groups * parts);
    w.done = reinterpret_cast<unsigned *>(w.share + 2 * groups * ((e + 31) / 32));
    return w;
}

template <class T, int EPL>
__global__ void __launch_bounds__(FC_ROUTER_BLOCK)
    k_router_fwd(const RouterForward a, const int parts)
{
    __shared__ int s_counts[32 * EPL];
    __shared__ float s_probs[FC_ROUTER_WARPS][32 * EPL];
    __shared__ float s_z[FC_ROUTER_WARPS];
    __shared__ int s_n[FC_ROUTER_WARPS];
    wait_for_prior_grid();
    allow_dependent_launch();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int E = a.n.experts, k = a.n.k;
    const int64_t group = blockIdx.x / parts;
    const int part = (int)(blockIdx.x - group * parts);
    const int64_t per = a.n.sequences * a.n.tokens / a.n.groups;  // rows of a group
    const RouterWs ws = router_ws(a.ws, a.n.groups, parts, E);
    if (blockIdx.x == 0 && threadIdx.x == 0) *ws.done = 0;
    for (int e = threadIdx.x; e < 32 * EPL; e += FC_ROUTER_BLOCK) s_counts[e] = 0;
    __syncthreads();
    float sum[EPL], zsum = 0.f;
    int routed = 0;
#pragma unroll
    for (int i = 0; i < EPL; ++i) sum[i] = 0.f;
    for (int64_t at = (int64_t)part * FC_ROUTER_WARPS + warp; at < per;
         at += (int64_t)parts * FC_ROUTER_WARPS) {
        const int64_t row = group * per + at;
        bool live = true;
        if (a.lengths) {
            const int64_t seq = row / a.n.tokens;
            live = row - seq * a.n.tokens < __ldg(a.lengths + seq);
        }
        float x[EPL], top = -INFINITY;
        bool any = false;
        if (live) {
            const T *p = static_cast<const T *>(a.logits) + row * a.ld;
#pragma unroll
            for (int i = 0; i < EPL; ++i) {
                const int e = lane + 32 * i;
                x[i] = e < E ? rt_f32(__ldcs(p + e)) : -INFINITY;
                top = fmaxf(top, x[i]);
                any |= !(x[i] == -INFINITY);
            }
            live = __any_sync(0xffffffffu, any);
        }
        if (!live) {  // behind the end, or no expert is open to it
            if (lane < k) {
                a.chosen[row * k + lane] = -1;
                a.weights[row * k + lane] = 0.f;
            }
            if (lane == 0) a.lse[row] = -INFINITY;
            continue;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        float total = 0.f, p[EPL];
        uint32_t key[EPL];
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            p[i] = expf(x[i] - top);
            total += p[i];
            key[i] = rt_key(x[i]);
        }
        total = warp_sum_f32(total);
        const float inv = 1.f / total, lse = top + logf(total);
#pragma unroll
        for (int i = 0; i < EPL; ++i) sum[i] = fmaf(p[i], inv, sum[i]);
        zsum = fmaf(lse, lse, zsum);
        ++routed;
        // the k largest, one after another; of equal ones the lowest
        int mine = -1;
        float value = -INFINITY;
        for (int j = 0; j < k; ++j) {
            uint32_t best = 0;
            int at_i = 0;
#pragma unroll
            for (int i = 0; i < EPL; ++i)
                if (key[i] > best) {
                    best = key[i];
                    at_i = i;
                }
            const uint32_t most = __reduce_max_sync(0xffffffffu, best);
            if (most == 0) break;
            const int e = (int)__reduce_min_sync(0xffffffffu,
                                                 best == most ? (unsigned)(lane + 32 * at_i) : ~0u);
            const bool owner = best == most && lane + 32 * at_i == e;
#pragma unroll
            for (int i = 0; i < EPL; ++i)
                if (owner && i == at_i) key[i] = 0;
            if (lane == j) {
                mine = e;
                const uint32_t u = most & 0x80000000u ? most ^ 0x80000000u : ~most;
                value = __uint_as_float(u);
            }
        }
        float w = mine >= 0 ? expf(value - top) : 0.f;
        // a row with a NaN has a total of NaN, and so weights of NaN
        const float chosen = a.n.normalise ? fmaf(0.f, total, warp_sum_f32(w)) : total;
        if (lane < k) {
            a.chosen[row * k + lane] = mine;
            a.weights[row * k + lane] = mine >= 0 ? w / chosen : 0.f;
            if (mine >= 0) atomicAdd(&s_counts[mine], 1);
        }
        if (lane == 0) a.lse[row] = lse;
    }
#pragma unroll
    for (int i = 0; i < EPL; ++i) s_probs[warp][lane + 32 * i] = sum[i];
    if (lane == 0) {
        s_z[warp] = zsum;
        s_n[warp] = routed;
    }
    __syncthreads();
    const int64_t out = (group * parts + part) * E;
    for (int e = threadIdx.x; e < E; e += FC_ROUTER_BLOCK) {
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < FC_ROUTER_WARPS; ++w) v += s_probs[w][e];
        ws.probs[out + e] = v;
        ws.counts[out + e] = s_counts[e];
    }
    if (threadIdx.x == 0) {
        float v = 0.f;
        int n = 0;
#pragma unroll
        for (int w = 0; w < FC_ROUTER_WARPS; ++w) {
            v += s_z[w];
            n += s_n[w];
        }
        ws.z[group * parts + part] = v;
        ws.routed[group * parts + part] = n;
    }
}

// Backward: with c_e the derivative of the balance loss by every probability of
// expert e in the row's group,
//   dlogits_e = p_e (c_e - sum_j p_j c_j + 2 dz lse / (groups n)) + the weights' part
template <class T, int EPL>
__global__ void __launch_bounds__(FC_ROUTER_BLOCK)
    k_router_bwd(const RouterBackward a, const int parts)
{
    __shared__ float s_add[FC_ROUTER_WARPS][32 * EPL];
    wait_for_prior_grid();
    allow_dependent_launch();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int E = a.n.experts, k = a.n.k;
    const int64_t group = blockIdx.x / parts;
    const int part = (int)(blockIdx.x - group * parts);
    const int64_t per = a.n.sequences * a.n.tokens / a.n.groups;
    float *const add = s_add[warp];
#pragma unroll
    for (int i = 0; i < EPL; ++i) add[lane + 32 * i] = 0.f;
    const float n = a.dloss ? (float)max(__ldg(a.routed + group), 1) : 1.f;
    const float each = 1.f / (n * (float)a.n.groups);
    const float d0 = a.dloss ? __ldg(a.dloss) : 0.f, d1 = a.dloss ? __ldg(a.dloss + 1) : 0.f;
    const float scale = d0 * ((float)E / (float)k) * each / n;
    float c[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        const int e = lane + 32 * i;
        c[i] = a.dloss && e < E ? scale * (float)__ldg(a.counts + group * E + e) : 0.f;
    }
    __syncwarp();
    for (int64_t at = (int64_t)part * FC_ROUTER_WARPS + warp; at < per;
         at += (int64_t)parts * FC_ROUTER_WARPS) {
        const int64_t row = group * per + at;
        const float lse = __ldg(a.lse + row);
        T *const out = static_cast<T *>(a.dlogits) + row * a.lddl;
        if (lse == -INFINITY) {
#pragma unroll
            for (int i = 0; i < EPL; ++i)
                if (lane + 32 * i < E) __stcs(out + lane + 32 * i, rt_round<T>(0.f));
            continue;
        }
        const T *x = static_cast<const T *>(a.logits) + row * a.ld;
        float p[EPL], inner = 0.f;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            const int e = lane + 32 * i;
            p[i] = e < E ? expf(rt_f32(__ldcs(x + e)) - lse) : 0.f;
            inner = fmaf(p[i], c[i], inner);
        }
        if (fabsf(lse) > FC_ROUTER_FAR) {
            // lse's own rounding is |lse| units of a probability: added up again
            float total = 0.f;
#pragma unroll
            for (int i = 0; i < EPL; ++i) total += p[i];
            const float inv = 1.f / warp_sum_f32(total);
            inner *= inv;
#pragma unroll
            for (int i = 0; i < EPL; ++i) p[i] *= inv;
        }
        float part2 = 0.f;
        int e = -1;
        float w = 0.f, dw = 0.f;
        if (a.dweights) {
            if (lane < k) {
                e = __ldg(a.chosen + row * k + lane);
                if ((unsigned)e < (unsigned)E) {
                    w = __ldg(a.weights + row * k + lane);
                    dw = __ldg(a.dweights + row * k + lane);
                } else {
                    e = -1;
                }
            }
            part2 = warp_sum_f32(w * dw);
            if (e >= 0) add[e] = a.n.normalise ? w * (dw - part2) : w * dw;
            if (a.n.normalise) part2 = 0.f;
            __syncwarp();
        }
        inner = warp_sum_f32(inner);
        const float sub = 2.f * d1 * lse * each - inner - part2;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            const int q = lane + 32 * i;
            if (q < E) __stcs(out + q, rt_round<T>(fmaf(p[i], c[i] + sub, add[q])));
        }
        if (a.dweights) {
            __syncwarp();
            if (e >= 0) add[e] = 0.f;
            __syncwarp();
        }
    }
}

template <class T, int EPL>
cudaError_t router_forward_width(const RouterForward &a, int parts, cudaStream_t s)
{
    return launch_after_prior(k_router_fwd<T, EPL>, (unsigned)(a.n.groups * parts), FC_ROUTER_BLOCK, 0,
                              s, a, parts);
}

template <class T, int EPL>
cudaError_t router_backward_width(const RouterBackward &a, int parts, cudaStream_t s)
{
    return launch_after_prior(k_router_bwd<T, EPL>, (unsigned)(a.n.groups * parts), FC_ROUTER_BLOCK, 0,
                              s, a, parts);
}

template <class T>
cudaError_t router_forward(const RouterForward &a, int parts, cudaStream_t s)
{
    const int e = a.n.experts;
    if (e <= 32) return router_forward_width<T, 1>(a, parts, s);
    if (e <= 64) return router_forward_width<T, 2>(a, parts, s);
    if (e <= 128) return router_forward_width<T, 4>(a, parts, s);
    if (e <= 256) return router_forward_width<T, 8>(a, parts, s);
    if (e <= 512) return router_forward_width<T, 16>(a, parts, s);
    return router_forward_width<T, 32>(a, parts, s);
}

template <class T>
cudaError_t router_backward(const RouterBackward &a, int parts, cudaStream_t s)
{
    const int e = a.n.experts;
    if (e <= 32) return router_backward_width<T, 1>(a, parts, s);
    if (e <= 64) return router_backward_width<T, 2>(a, parts, s);
    if (e <= 128) return router_backward_width<T, 4>(a, parts, s);
    if (e <= 256) return router_backward_width<T, 8>(a, parts, s);
    if (e <= 512) return router_backward_width<T, 16>(a, parts, s);
    return router_backward_width<T, 32>(a, parts, s);
}

}  // namespace fc
