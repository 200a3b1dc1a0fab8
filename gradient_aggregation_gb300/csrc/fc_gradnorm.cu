// Global L2 norm of many gradient tensors, and the factor for the step.
//
// norm = sqrt(sum g^2) / S; the factor is (1/S) * min(1, max_norm / norm),
// or NaN where the norm is not finite.  One read of the gradient and two
// words out, so it is bound by HBM, and by latency below a few megabytes.
//
// A tile is 8 KB of one segment, cut at 16-byte boundaries of the segment's own
// address: every load is a full aligned vector but for a segment's first and
// last granule, and no load touches a byte outside the segment.  Each thread has
// its two 16-byte loads of a tile in flight at once, and eight CTAs share an SM.
// The squares of one tile are summed per thread in fp32 (at most 16 terms),
// tiles and threads in float-float; CTAs take tiles in a fixed round, and the
// last CTA to finish adds the CTAs' sums in their order, so the result depends
// on the data and on the grid only.
//
// Measured on 62.4M fp32 elements (250 MB): 42.7 us, 5.8 TB/s (46.7 with the
// loads allocating in L1 too); 133k fp16 elements: 3.5 us, all of it latency
// (two trips to memory, the arrival of the CTAs and the last one's sum).  Tiles
// of 32 KB and blocks of 512 threads: 42.9 and 4.0 us.
#include "fc_opt.h"

namespace fc {


__device__ __forceinline__ float sumsq16(const uint4 &q, float)
{
    const float a = __uint_as_float(q.x), b = __uint_as_float(q.y);
    const float c = __uint_as_float(q.z), d = __uint_as_float(q.w);
    return (a * a + b * b) + (c * c + d * d);
}

__device__ __forceinline__ float sumsq16(const uint4 &q, __half)
{
    float x[8];
    unpack8(q, x);
    return group_sumsq(x);
}

__device__ __forceinline__ float sumsq16(const uint4 &q, __nv_bfloat16)
{
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
    float x[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
    return group_sumsq(x);
}

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }

__device__ __forceinline__ uint4 ld_once16(const void *p)
{
    uint4 v;
    asm("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
        : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
        : "l"(p));
    return v;
}

// Block sum of one float-float per thread; thread 0's result is the defined one.
template <int BLOCK>
__device__ __forceinline__ FF block_sum_ff(FF x, FF *sm)
{
    x = warp_sum_ff(x);
    if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = x;
    __syncthreads();
    FF t = {0.f, 0.f};
    if (threadIdx.x < 32) {
        if (threadIdx.x < BLOCK / 32) t = sm[threadIdx.x];
        t = warp_sum_ff(t);
    }
    return t;
}

#define FC_NORM_BLOCK 256

template <class GT, class Tab>
__global__ void __launch_bounds__(FC_NORM_BLOCK)
    k_grad_norm(const __grid_constant__ Tab tab, const float loss_scale, const float max_norm,
                FF *__restrict__ partials, unsigned *__restrict__ done,
                float *__restrict__ norm, float *__restrict__ scale)
{
    __shared__ FF sm[FC_NORM_BLOCK / 32];
    __shared__ bool last;
    constexpr int BLOCK = FC_NORM_BLOCK, TILE = FC_NORM_TILE, U = TILE / (16 * BLOCK);
    constexpr int E = 16 / (int)sizeof(GT);
    wait_for_prior_grid();
    allow_dependent_launch();
    const int tiles = tab.tile0[tab.L];
    FF acc = {0.f, 0.f};
    for (int t = blockIdx.x; t < tiles; t += gridDim.x) {
        int lo = 0, hi = tab.L - 1;  // the segment whose tiles hold t
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (tab.tile0[mid + 1] > t)
                hi = mid;
            else
                lo = mid + 1;
        }
        const GT *p = static_cast<const GT *>(tab.ptr[lo]);
        const GT *end = p + tab.n[lo];
        const GT *base = reinterpret_cast<const GT *>(
            ((uintptr_t)p & ~(uintptr_t)15) + (uintptr_t)(t - tab.tile0[lo]) * TILE);
        float ss = 0.f;
        if (base >= p && base + TILE / sizeof(GT) <= end) {
            uint4 q[U];
#pragma unroll
            for (int i = 0; i < U; ++i)
                q[i] = ld_once16(reinterpret_cast<const uint4 *>(base) + threadIdx.x + i * BLOCK);
#pragma unroll
            for (int i = 0; i < U; i += 2) ss += sumsq16(q[i], GT()) + sumsq16(q[i + 1], GT());
        } else {
            float part[U];
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const GT *g = base + (threadIdx.x + i * BLOCK) * E;
                part[i] = 0.f;
                if (g >= p && g + E <= end) {
                    part[i] = sumsq16(ld_once16(g), GT());
                } else {
                    for (int e = 0; e < E; ++e)
                        if (g + e >= p && g + e < end) {
                            const float x = to_f32(g[e]);
                            part[i] += x * x;
                        }
                }
            }
#pragma unroll
            for (int i = 0; i < U; i += 2) ss += part[i] + part[i + 1];
        }
        acc = ff_add(acc, ss);
    }
    const FF sum = block_sum_ff<BLOCK>(acc, sm);
    if (threadIdx.x == 0) {
        // an infinite or NaN sum leaves NaN as its rounding error: hi says it
        __stcg(reinterpret_cast<float2 *>(partials + blockIdx.x), make_float2(sum.hi, sum.lo));
        __threadfence();
        last = atomicAdd(done, 1u) == gridDim.x - 1;
    }
    __syncthreads();
    if (!last) return;
    __threadfence();
    FF all = {0.f, 0.f};
    for (int i = threadIdx.x; i < gridDim.x; i += BLOCK) {
        const float2 x = __ldcg(reinterpret_cast<const float2 *>(partials + i));
        all = ff_add(all, FF{x.x, x.y});
    }
    const FF total = block_sum_ff<BLOCK>(all, sm);
    if (threadIdx.x == 0) {
        const float ss = isfinite(total.hi) ? total.hi + total.lo : total.hi;
        const float n = __fdiv_rn(__fsqrt_rn(ss), loss_scale);
        float f = 1.f;
        if (max_norm > 0.f && n > max_norm) f = __fdiv_rn(max_norm, n);
        norm[0] = n;
        scale[0] = isfinite(n) ? __fdiv_rn(f, loss_scale) : __int_as_float(0x7fffffff);
        *done = 0u;
    }
}

template <class GT, class Tab>
static cudaError_t launch_typed(const Tab &tab, float loss_scale, float max_norm, FF *partials,
                                unsigned *done, float *norm, float *scale, cudaStream_t s)
{
    const auto kernel = k_grad_norm<GT, Tab>;
    int grid = grid_for((const void *)kernel, FC_NORM_BLOCK, 0, tab.tile0[tab.L]);
    if (grid > FC_NORM_MAX_GRID) grid = FC_NORM_MAX_GRID;
    return launch_after_prior(kernel, (unsigned)grid, FC_NORM_BLOCK, 0, s, tab, loss_scale,
                              max_norm, partials, done, norm, scale);
}

template <class Tab>
cudaError_t launch_grad_norm(const Tab &tab, int gtype, float loss_scale, float max_norm,
                             FF *partials, unsigned *done, float *norm, float *scale,
                             cudaStream_t s)
{
    if (gtype == FC_TYPE_F32)
        return launch_typed<float>(tab, loss_scale, max_norm, partials, done, norm, scale, s);
    if (gtype == FC_TYPE_F16)
        return launch_typed<__half>(tab, loss_scale, max_norm, partials, done, norm, scale, s);
    return launch_typed<__nv_bfloat16>(tab, loss_scale, max_norm, partials, done, norm, scale, s);
}

#define FC_INST(Tab)                                                                              \
    template cudaError_t launch_grad_norm<Tab>(const Tab &, int, float, float, FF *, unsigned *,   \
                                               float *, float *, cudaStream_t);
FC_INST(NormTableS)
FC_INST(NormTableL)

}  // namespace fc
