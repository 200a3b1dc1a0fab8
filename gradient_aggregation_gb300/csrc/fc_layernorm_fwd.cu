// Layer norm, forward.
//
//   mean = sum x / n;  rstd = 1 / sqrt(sum (x - mean)^2 / n + eps)
//   y = (x - mean) * rstd * w + b
//
// Bound by HBM: x is read once and y written once.  The row stays in
// registers, so the variance is the sum of squared differences and costs no
// second read.  Where a row spans several warps, each warp takes the mean
// and the squared differences of its own part (two shuffle reductions), and
// the parts are joined by
//   M2 = sum_w [ M2_w + n_w (mean_w - mean)^2 ]
// which needs one exchange through shared memory and one barrier a row.
#include "fc_layernorm.cuh"

namespace fc {

template <class T, int VEC, int K, int TPR, int BLOCK>
__global__ void __launch_bounds__(BLOCK)
    k_ln_fwd(const LnForward a, const bool pvec)
{
    constexpr int G = BLOCK / TPR;
    constexpr int WARPS = TPR > 32 ? TPR / 32 : 1;
    constexpr bool HOLD = K * VEC <= 8;  // the parameters stay in registers
    __shared__ float2 part[2][G][WARPS];
    wait_for_prior_grid();
    allow_dependent_launch();
    const int t = threadIdx.x % TPR, g = threadIdx.x / TPR;
    const int cols = (int)a.cols;
    const int nvec = cols / VEC;
    const float inv_n = 1.f / (float)cols;
    const T *x = static_cast<const T *>(a.x);
    T *y = static_cast<T *>(a.y);
    const int64_t stride = (int64_t)gridDim.x * G;
    int64_t row = (int64_t)blockIdx.x * G + g;

    // elements of the row that this thread's warp holds, and those of the
    // warp whose part this lane joins
    float n_own = 0.f, n_join = 0.f;
    const int lw = threadIdx.x & (WARPS - 1);
    if constexpr (WARPS > 1) {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            n_own += (float)(VEC * min(max(nvec - (t & ~31) - k * TPR, 0), 32));
            n_join += (float)(VEC * min(max(nvec - 32 * lw - k * TPR, 0), 32));
        }
    }
    const float r_own = n_own > 0.f ? 1.f / n_own : 0.f;
    const float r_join = n_join > 0.f ? 1.f / n_join : 0.f;
    float pw[HOLD ? K : 1][VEC], pb[HOLD ? K : 1][VEC];
    if constexpr (HOLD) {
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (t + k * TPR < nvec) {
                load_params<T, VEC>(a.weight, a.ptype, pvec, (t + k * TPR) * VEC, 1.f, pw[k]);
                load_params<T, VEC>(a.bias, a.ptype, pvec, (t + k * TPR) * VEC, 0.f, pb[k]);
            }
    }

    Vec<T, VEC> next[K];
    auto load = [&](int64_t r) {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            if (r < a.rows && t + k * TPR < nvec)
                next[k].load(x + r * a.ldx + (int64_t)(t + k * TPR) * VEC);
            else
                next[k].clear();
        }
    };
    load(row);
    // every thread of the block runs the same number of rounds (a warp may
    // hold several rows, and its shuffles name all lanes)
    const int64_t rounds = (a.rows + stride - 1) / stride;
    int buf = 0;
    for (int64_t it = 0; it < rounds; ++it, row += stride, buf ^= 1) {
        Vec<T, VEC> v[K];
#pragma unroll
        for (int k = 0; k < K; ++k) v[k] = next[k];
        if (it + 1 < rounds) load(row + stride);
        const bool live = row < a.rows;
        float s = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            float f[VEC];
            v[k].get(f);
#pragma unroll
            for (int e = 0; e < VEC; ++e) s += f[e];
        }
        s = lanes_sum<TPR>(s);
        float mean = s * (WARPS > 1 ? r_own : inv_n);
        float m2 = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            if (t + k * TPR < nvec) {
                float f[VEC];
                v[k].get(f);
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const float d = f[e] - mean;
                    m2 = fmaf(d, d, m2);
                }
            }
        }
        m2 = lanes_sum<TPR>(m2);
        if constexpr (WARPS > 1) {
            if ((t & 31) == 0) part[buf][g][t >> 5] = make_float2(s, m2);
            group_sync<TPR, BLOCK>(g);
            const float2 p = part[buf][g][lw];
            mean = lanes_sum<WARPS>(p.x) * inv_n;
            const float d = p.x * r_join - mean;
            m2 = lanes_sum<WARPS>(fmaf(n_join * d, d, p.y));
        }
        const float rstd = rsqrtf(m2 * inv_n + a.eps);
        if (live) {
            if (a.mean && t == 0) {
                a.mean[row] = mean;
                a.rstd[row] = rstd;
            }
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const int c = (t + k * TPR) * VEC;
                if (t + k * TPR < nvec) {
                    float f[VEC], w[VEC], b[VEC];
                    v[k].get(f);
                    if constexpr (HOLD) {
#pragma unroll
                        for (int e = 0; e < VEC; ++e) {
                            w[e] = pw[k][e];
                            b[e] = pb[k][e];
                        }
                    } else {
                        load_params<T, VEC>(a.weight, a.ptype, pvec, c, 1.f, w);
                        load_params<T, VEC>(a.bias, a.ptype, pvec, c, 0.f, b);
                    }
#pragma unroll
                    for (int e = 0; e < VEC; ++e) f[e] = fmaf((f[e] - mean) * rstd, w[e], b[e]);
                    Vec<T, VEC>::store(y + row * a.ldy + c, f);
                }
            }
        }
    }
}

// Rows wider than the registers hold: one block a row, three passes over it
// (the second and third from L2 where the row fits).
#define FC_LN_WIDE_BLOCK 512

__device__ __forceinline__ float ln_block_sum(float x, float *sm)
{
    x = lanes_sum<32>(x);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = x;
    __syncthreads();
    float s = 0.f;
    for (int w = 0; w < FC_LN_WIDE_BLOCK / 32; ++w) s += sm[w];
    return s;
}

template <class T>
__global__ void __launch_bounds__(FC_LN_WIDE_BLOCK) k_ln_fwd_wide(const LnForward a)
{
    __shared__ float sm[FC_LN_WIDE_BLOCK / 32];
    wait_for_prior_grid();
    allow_dependent_launch();
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const T *x = static_cast<const T *>(a.x) + row * a.ldx;
        T *y = static_cast<T *>(a.y) + row * a.ldy;
        // sums of a thread in float-float: a row may have millions of columns
        FF s = {0.f, 0.f};
        for (int64_t c = threadIdx.x; c < a.cols; c += FC_LN_WIDE_BLOCK)
            s = ff_add(s, ln_f32(x[c]));
        const float mean = ln_block_sum(s.hi + s.lo, sm) / (float)a.cols;
        FF q = {0.f, 0.f};
        for (int64_t c = threadIdx.x; c < a.cols; c += FC_LN_WIDE_BLOCK) {
            const float d = ln_f32(x[c]) - mean;
            q = ff_add(q, d * d);
        }
        const float rstd = rsqrtf(ln_block_sum(q.hi + q.lo, sm) / (float)a.cols + a.eps);
        if (a.mean && threadIdx.x == 0) {
            a.mean[row] = mean;
            a.rstd[row] = rstd;
        }
        for (int64_t c = threadIdx.x; c < a.cols; c += FC_LN_WIDE_BLOCK) {
            float w[1], b[1];
            load_params<T, 1>(a.weight, a.ptype, false, c, 1.f, w);
            load_params<T, 1>(a.bias, a.ptype, false, c, 0.f, b);
            y[c] = ln_round<T>(fmaf((ln_f32(x[c]) - mean) * rstd, w[0], b[0]));
        }
    }
}

template <class T, int VEC, int K, int TPR, int BLOCK>
static cudaError_t go(const LnForward &a, bool pvec, cudaStream_t s)
{
    const auto kernel = k_ln_fwd<T, VEC, K, TPR, BLOCK>;
    const int64_t ctas = (a.rows + BLOCK / TPR - 1) / (BLOCK / TPR);
    const int grid = grid_for((const void *)kernel, BLOCK, 0, ctas);
    return launch_after_prior(kernel, (unsigned)grid, BLOCK, 0, s, a, pvec);
}

template <class T>
static cudaError_t forward(const LnForward &a, cudaStream_t s)
{
    constexpr int V = 16 / (int)sizeof(T);
    auto on16 = [](const void *p, int64_t ld) {
        return ((uintptr_t)p & 15) == 0 && (ld * (int64_t)sizeof(T)) % 16 == 0;
    };
    const bool pvec = ((uintptr_t)a.weight & 15) == 0 && ((uintptr_t)a.bias & 15) == 0;
    const int64_t c = a.cols;
    if (c % V == 0 && on16(a.x, a.ldx) && on16(a.y, a.ldy)) {
        const int64_t n = c / V;
        if (n <= 8) return go<T, V, 1, 8, 128>(a, pvec, s);
        if (n <= 16) return go<T, V, 1, 16, 128>(a, pvec, s);
        if (n <= 32) return go<T, V, 1, 32, 128>(a, pvec, s);
        if (n <= 64) return go<T, V, 2, 32, 128>(a, pvec, s);
        if (n <= 128) return go<T, V, 1, 128, 256>(a, pvec, s);
        if (n <= 256) return go<T, V, 1, 256, 256>(a, pvec, s);
        if (n <= 512) return go<T, V, 1, 512, 512>(a, pvec, s);
        if (n <= 1024) return go<T, V, 1, 1024, 1024>(a, pvec, s);
        if (n <= 2048) return go<T, V, 2, 1024, 1024>(a, pvec, s);
    } else {
        if (c <= 32) return go<T, 1, 1, 32, 128>(a, pvec, s);
        if (c <= 128) return go<T, 1, 4, 32, 128>(a, pvec, s);
        if (c <= 512) return go<T, 1, 4, 128, 256>(a, pvec, s);
        if (c <= 1024) return go<T, 1, 8, 128, 256>(a, pvec, s);
        if (c <= 2048) return go<T, 1, 8, 256, 256>(a, pvec, s);
        if (c <= 4096) return go<T, 1, 8, 512, 512>(a, pvec, s);
        if (c <= 8192) return go<T, 1, 8, 1024, 1024>(a, pvec, s);
        if (c <= 16384) return go<T, 1, 16, 1024, 1024>(a, pvec, s);
    }
    const auto wide = k_ln_fwd_wide<T>;
    const int grid = grid_for((const void *)wide, FC_LN_WIDE_BLOCK, 0, a.rows);
    return launch_after_prior(wide, (unsigned)grid, FC_LN_WIDE_BLOCK, 0, s, a);
}

cudaError_t launch_ln_forward(const LnForward &a, int type, cudaStream_t s)
{
    if (type == FC_TYPE_F32) return forward<float>(a, s);
    if (type == FC_TYPE_F16) return forward<__half>(a, s);
    return forward<__nv_bfloat16>(a, s);
}

}  // namespace fc
