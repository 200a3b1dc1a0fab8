// Layer norm, backward.
//
//   h = (x - mean) * rstd;  q = dy * w
//   dx = rstd * (q - sum(q) / n - h * sum(q h) / n)
//   dweight = sum over rows of dy * h;  dbias = sum over rows of dy
//
// Bound by HBM: dy and x are read once and dx written once.  A block takes
// rows in rounds; the two row sums cost one shuffle reduction and, where a
// row spans several warps, one exchange and one barrier.  A thread owns the
// same columns in every row, so the column sums stay in its registers until
// the block has no more rows; each block then leaves one set of sums, and a
// second kernel adds the sets in their order (no atomics: the same inputs
// give the same bits).
#include "fc_layernorm.cuh"

namespace fc {

template <class T, int VEC, int K, int TPR, int BLOCK>
__global__ void __launch_bounds__(BLOCK) k_ln_bwd(const LnBackward a, const bool pvec)
{
    constexpr int G = BLOCK / TPR;
    constexpr int WARPS = TPR > 32 ? TPR / 32 : 1;
    constexpr bool HOLD = K * VEC <= 8;
    __shared__ float2 part[2][G][WARPS];
    wait_for_prior_grid();
    allow_dependent_launch();
    const int t = threadIdx.x % TPR, g = threadIdx.x / TPR;
    const int cols = (int)a.cols;
    const int nvec = cols / VEC;
    const float inv_n = 1.f / (float)cols;
    const T *x = static_cast<const T *>(a.x);
    const T *dy = static_cast<const T *>(a.dy);
    T *dx = static_cast<T *>(a.dx);
    const int64_t stride = (int64_t)gridDim.x * G;
    int64_t row = (int64_t)blockIdx.x * G + g;

    float pw[HOLD ? K : 1][VEC];
    if constexpr (HOLD) {
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (t + k * TPR < nvec)
                load_params<T, VEC>(a.weight, a.ptype, pvec, (t + k * TPR) * VEC, 1.f, pw[k]);
    }
    float dw[K][VEC], db[K][VEC];
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int e = 0; e < VEC; ++e) dw[k][e] = db[k][e] = 0.f;

    Vec<T, VEC> nx[K], ny[K];
    float nmean = 0.f, nrstd = 0.f;
    auto load = [&](int64_t r) {
        const bool in = r < a.rows;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            if (in && t + k * TPR < nvec) {
                nx[k].load(x + r * a.ldx + (int64_t)(t + k * TPR) * VEC);
                ny[k].load(dy + r * a.lddy + (int64_t)(t + k * TPR) * VEC);
            } else {
                nx[k].clear();
                ny[k].clear();
            }
        }
        // a row that is not there has h = 0 and dy = 0: it adds nothing
        nmean = in ? __ldg(a.mean + r) : 0.f;
        nrstd = in ? __ldg(a.rstd + r) : 0.f;
    };
    load(row);
    const int64_t rounds = (a.rows + stride - 1) / stride;
    int buf = 0;
    for (int64_t it = 0; it < rounds; ++it, row += stride, buf ^= 1) {
        Vec<T, VEC> vx[K], vy[K];
        const float mean = nmean, rstd = nrstd;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            vx[k] = nx[k];
            vy[k] = ny[k];
        }
        if (it + 1 < rounds) load(row + stride);
        float s1 = 0.f, s2 = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            if (t + k * TPR < nvec) {
                float fx[VEC], fy[VEC], w[VEC];
                vx[k].get(fx);
                vy[k].get(fy);
                if constexpr (HOLD) {
#pragma unroll
                    for (int e = 0; e < VEC; ++e) w[e] = pw[k][e];
                } else {
                    load_params<T, VEC>(a.weight, a.ptype, pvec, (t + k * TPR) * VEC, 1.f, w);
                }
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const float h = (fx[e] - mean) * rstd;
                    const float q = fy[e] * w[e];
                    s1 += q;
                    s2 = fmaf(q, h, s2);
                    dw[k][e] = fmaf(fy[e], h, dw[k][e]);
                    db[k][e] += fy[e];
                }
            }
        }
        s1 = lanes_sum<TPR>(s1);
        s2 = lanes_sum<TPR>(s2);
        if constexpr (WARPS > 1) {
            if ((t & 31) == 0) part[buf][g][t >> 5] = make_float2(s1, s2);
            group_sync<TPR, BLOCK>(g);
            const float2 p = part[buf][g][threadIdx.x & (WARPS - 1)];
            s1 = lanes_sum<WARPS>(p.x);
            s2 = lanes_sum<WARPS>(p.y);
        }
        s1 *= inv_n;
        s2 *= inv_n;
        if (row < a.rows) {
#pragma unroll
            for (int k = 0; k < K; ++k) {
                if (t + k * TPR < nvec) {
                    const int c = (t + k * TPR) * VEC;
                    float fx[VEC], fy[VEC], w[VEC];
                    vx[k].get(fx);
                    vy[k].get(fy);
                    if constexpr (HOLD) {
#pragma unroll
                        for (int e = 0; e < VEC; ++e) w[e] = pw[k][e];
                    } else {
                        load_params<T, VEC>(a.weight, a.ptype, pvec, c, 1.f, w);
                    }
#pragma unroll
                    for (int e = 0; e < VEC; ++e) {
                        const float h = (fx[e] - mean) * rstd;
                        fx[e] = rstd * (fmaf(fy[e], w[e], -s1) - h * s2);
                    }
                    Vec<T, VEC>::store(dx + row * a.lddx + c, fx);
                }
            }
        }
    }
    if (!a.partials) return;
    float *pdw = a.partials + (int64_t)blockIdx.x * cols;
    float *pdb = a.partials + ((int64_t)gridDim.x + blockIdx.x) * cols;
    if constexpr (G == 1) {
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (t + k * TPR < nvec)
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    pdw[(t + k * TPR) * VEC + e] = dw[k][e];
                    pdb[(t + k * TPR) * VEC + e] = db[k][e];
                }
    } else {
        // the row groups of the block are added in their order
        __shared__ float sw[TPR * K * VEC], sb[TPR * K * VEC];
        for (int r = 0; r < G; ++r) {
            __syncthreads();
            if (g == r) {
#pragma unroll
                for (int k = 0; k < K; ++k)
#pragma unroll
                    for (int e = 0; e < VEC; ++e) {
                        const int c = (t + k * TPR) * VEC + e;
                        sw[c] = r ? sw[c] + dw[k][e] : dw[k][e];
                        sb[c] = r ? sb[c] + db[k][e] : db[k][e];
                    }
            }
        }
        __syncthreads();
        for (int c = threadIdx.x; c < cols; c += BLOCK) {
            pdw[c] = sw[c];
            pdb[c] = sb[c];
        }
    }
}

// Rows wider than the registers hold: one block a row, two passes over it.
#define FC_LN_WIDE_BLOCK 512

template <class T>
__global__ void __launch_bounds__(FC_LN_WIDE_BLOCK) k_ln_bwd_wide(const LnBackward a)
{
    __shared__ float2 sm[FC_LN_WIDE_BLOCK / 32];
    wait_for_prior_grid();
    allow_dependent_launch();
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const T *x = static_cast<const T *>(a.x) + row * a.ldx;
        const T *dy = static_cast<const T *>(a.dy) + row * a.lddy;
        T *dx = static_cast<T *>(a.dx) + row * a.lddx;
        const float mean = a.mean[row], rstd = a.rstd[row];
        FF f1 = {0.f, 0.f}, f2 = {0.f, 0.f};
        for (int64_t c = threadIdx.x; c < a.cols; c += FC_LN_WIDE_BLOCK) {
            float w[1];
            load_params<T, 1>(a.weight, a.ptype, false, c, 1.f, w);
            const float q = ln_f32(dy[c]) * w[0];
            f1 = ff_add(f1, q);
            f2 = ff_add(f2, q * ((ln_f32(x[c]) - mean) * rstd));
        }
        float s1 = lanes_sum<32>(f1.hi + f1.lo), s2 = lanes_sum<32>(f2.hi + f2.lo);
        __syncthreads();
        if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = make_float2(s1, s2);
        __syncthreads();
        s1 = s2 = 0.f;
        for (int w = 0; w < FC_LN_WIDE_BLOCK / 32; ++w) {
            s1 += sm[w].x;
            s2 += sm[w].y;
        }
        s1 /= (float)a.cols;
        s2 /= (float)a.cols;
        for (int64_t c = threadIdx.x; c < a.cols; c += FC_LN_WIDE_BLOCK) {
            float w[1];
            load_params<T, 1>(a.weight, a.ptype, false, c, 1.f, w);
            const float h = (ln_f32(x[c]) - mean) * rstd;
            dx[c] = ln_round<T>(rstd * (fmaf(ln_f32(dy[c]), w[0], -s1) - h * s2));
        }
    }
}

// Column sums of wide rows: block (i, p) adds rows p, p + parts, ... of 128
// columns.
template <class T>
__global__ void __launch_bounds__(128) k_ln_colsum_wide(const LnBackward a)
{
    wait_for_prior_grid();
    allow_dependent_launch();
    const int64_t c = (int64_t)blockIdx.x * 128 + threadIdx.x;
    if (c >= a.cols) return;
    float dw = 0.f, db = 0.f;
    for (int64_t r = blockIdx.y; r < a.rows; r += gridDim.y) {
        const float y = ln_f32(static_cast<const T *>(a.dy)[r * a.lddy + c]);
        const float h = (ln_f32(static_cast<const T *>(a.x)[r * a.ldx + c]) - a.mean[r]) * a.rstd[r];
        dw = fmaf(y, h, dw);
        db += y;
    }
    a.partials[(int64_t)blockIdx.y * a.cols + c] = dw;
    a.partials[((int64_t)gridDim.y + blockIdx.y) * a.cols + c] = db;
}

// Adds `parts` sets of column sums; blockIdx.y: 0 for dweight, 1 for dbias.
// 32 columns a block, each by 16 threads that take every 16th set, four
// loads in flight.
#define FC_LN_JOIN 16

__global__ void __launch_bounds__(32 * FC_LN_JOIN)
    k_ln_join(const float *__restrict__ partials, const int parts, const int64_t cols,
              void *dweight, void *dbias, const int gtype)
{
    __shared__ float sm[FC_LN_JOIN][33];
    wait_for_prior_grid();
    allow_dependent_launch();
    void *out = blockIdx.y ? dbias : dweight;
    if (!out) return;
    const int lane = threadIdx.x & 31, q = threadIdx.x >> 5;
    const int64_t c = (int64_t)blockIdx.x * 32 + lane;
    const float *p = partials + (int64_t)blockIdx.y * parts * cols + c;
    float s = 0.f;
    if (c < cols) {
#pragma unroll 4
        for (int i = q; i < parts; i += FC_LN_JOIN) s += __ldcg(p + (int64_t)i * cols);
    }
    sm[q][lane] = s;
    __syncthreads();
    if (q == 0 && c < cols) {
        s = 0.f;
#pragma unroll
        for (int i = 0; i < FC_LN_JOIN; ++i) s += sm[i][lane];
        if (gtype == FC_TYPE_F32)
            static_cast<float *>(out)[c] = s;
        else if (gtype == FC_TYPE_F16)
            static_cast<__half *>(out)[c] = __float2half_rn(s);
        else
            static_cast<__nv_bfloat16 *>(out)[c] = __float2bfloat16_rn(s);
    }
}

// At most 1024 blocks, and no more than rows.
int64_t ln_max_parts(int64_t rows, int64_t cols)
{
    (void)cols;
    return rows < 1024 ? rows : 1024;
}

static cudaError_t join(const LnBackward &a, int parts, cudaStream_t s)
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
    return cudaLaunchKernelEx(&cfg, k_ln_join, (const float *)a.partials, parts, a.cols, a.dweight,
                              a.dbias, a.gtype);
}

template <class T, int VEC, int K, int TPR, int BLOCK>
static cudaError_t go(const LnBackward &a, bool pvec, cudaStream_t s)
{
    const auto kernel = k_ln_bwd<T, VEC, K, TPR, BLOCK>;
    const int64_t ctas = (a.rows + BLOCK / TPR - 1) / (BLOCK / TPR);
    int grid = grid_for((const void *)kernel, BLOCK, 0, ctas);
    const int64_t most = ln_max_parts(a.rows, a.cols);
    if (grid > most) grid = (int)most;
    cudaError_t e = launch_after_prior(kernel, (unsigned)grid, BLOCK, 0, s, a, pvec);
    return e != cudaSuccess ? e : join(a, grid, s);
}

template <class T>
static cudaError_t backward(const LnBackward &a, cudaStream_t s)
{
    if (a.rows == 0) return join(a, 0, s);
    constexpr int V = 16 / (int)sizeof(T);
    auto on16 = [](const void *p, int64_t ld) {
        return ((uintptr_t)p & 15) == 0 && (ld * (int64_t)sizeof(T)) % 16 == 0;
    };
    const bool pvec = ((uintptr_t)a.weight & 15) == 0;
    const int64_t c = a.cols;
    if (c % V == 0 && on16(a.x, a.ldx) && on16(a.dy, a.lddy) && on16(a.dx, a.lddx)) {
        const int64_t n = c / V;
        if (n <= 8) return go<T, V, 1, 8, 128>(a, pvec, s);
        if (n <= 16) return go<T, V, 1, 16, 128>(a, pvec, s);
        if (n <= 32) return go<T, V, 1, 32, 128>(a, pvec, s);
        if (n <= 64) return go<T, V, 1, 64, 256>(a, pvec, s);
        if (n <= 128) return go<T, V, 1, 128, 256>(a, pvec, s);
        if (n <= 256) return go<T, V, 1, 256, 256>(a, pvec, s);
        if (n <= 512) return go<T, V, 1, 512, 512>(a, pvec, s);
        if (n <= 1024) return go<T, V, 1, 1024, 1024>(a, pvec, s);
        if (n <= 2048) return go<T, V, 2, 1024, 1024>(a, pvec, s);
    } else {
        if (c <= 32) return go<T, 1, 1, 32, 128>(a, pvec, s);
        if (c <= 128) return go<T, 1, 4, 32, 128>(a, pvec, s);
        if (c <= 512) return go<T, 1, 4, 128, 256>(a, pvec, s);
        if (c <= 1024) return go<T, 1, 4, 256, 256>(a, pvec, s);
        if (c <= 2048) return go<T, 1, 8, 256, 256>(a, pvec, s);
        if (c <= 4096) return go<T, 1, 8, 512, 512>(a, pvec, s);
        if (c <= 8192) return go<T, 1, 8, 1024, 1024>(a, pvec, s);
    }
    const auto wide = k_ln_bwd_wide<T>;
    const int grid = grid_for((const void *)wide, FC_LN_WIDE_BLOCK, 0, a.rows);
    cudaError_t e = launch_after_prior(wide, (unsigned)grid, FC_LN_WIDE_BLOCK, 0, s, a);
    if (e != cudaSuccess || !a.partials) return e;
    const int64_t strips = (c + 127) / 128;
    int64_t parts = ln_max_parts(a.rows, c);
    if (strips * parts > 4096) parts = 4096 / strips < 1 ? 1 : 4096 / strips;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)strips, (unsigned)parts);
    cfg.blockDim = dim3(128);
    cfg.stream = s;
    e = cudaLaunchKernelEx(&cfg, k_ln_colsum_wide<T>, a);
    return e != cudaSuccess ? e : join(a, (int)parts, s);
}

cudaError_t launch_ln_backward(const LnBackward &a, int type, cudaStream_t s)
{
    if (type == FC_TYPE_F32) return backward<float>(a, s);
    if (type == FC_TYPE_F16) return backward<__half>(a, s);
    return backward<__nv_bfloat16>(a, s);
}

}  // namespace fc
