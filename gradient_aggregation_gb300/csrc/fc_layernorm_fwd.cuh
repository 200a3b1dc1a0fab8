// Layer norm, forward: the kernels, for one element type T.
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
//
// Kernels: k_ln_fwd_rows and k_ln_fwd_any for many rows, and k_ln_fwd, which
// spreads each row over as many threads as it has vectors, for few rows and
// for narrow ones.
#pragma once

#include <algorithm>

#include "fc_layernorm.cuh"
#include "fc_pairs.cuh"

namespace fc {

// ---- many rows --------------------------------------------------------------------------------
//
// A row is held by TPR threads (one warp up to 2048 columns of a 16-bit type),
// as pairs of fp32 that one instruction works on; short rows go RW at a time, so
// that their reductions overlap.  The parameters are in shared memory as fp32.
//
// k_ln_fwd_rows: every row starts on a 16-byte boundary and is whole vectors of
// 16 bytes; a lane holds K of them, and the parameters lie in planes of 4
// columns that a warp reads without conflicts.  Measured at 134M elements of
// bf16 (537 MB), 768 / 2048 / 4096 columns: 89 / 84 / 88 us, 0.95 of the copy
// rate at 2048.
// k_ln_fwd_any: rows that start at any element and have any width, word by word
// (see fc_pairs.cuh).

// Mean and 1/sqrt of the variance of RW rows in pairs; `held` columns a warp.
template <int NP, int TPR, int RW, int BLOCK>
struct PairStats {
    static constexpr int WARPS = TPR / 32;
    float inv_n, eps, r_own, n_join, r_join;

    __device__ __forceinline__ PairStats(int cols, int held, float eps_, int t)
        : inv_n(1.f / (float)cols), eps(eps_), r_own(inv_n), n_join(0.f), r_join(0.f)
    {
        if constexpr (WARPS > 1) {
            // elements that this thread's warp holds, and the warp whose part
            // this lane joins
            const int join = (int)threadIdx.x & (WARPS - 1);
            const float n_own = (float)min(max(cols - (t >> 5) * held, 0), held);
            n_join = (float)min(max(cols - join * held, 0), held);
            r_own = n_own > 0.f ? 1.f / n_own : 0.f;
            r_join = n_join > 0.f ? 1.f / n_join : 0.f;
        }
    }

    // get(r, p): pair p of row r, zero past the row.  Blocks of B pairs lie inside
    // the row (inside(b) = 1), past it (0) or both (2): there centre(r, m, p) gives
    // the pair with m in place of what lies past the row.
    template <int B, class Get, class Inside, class Centre>
    __device__ __forceinline__ void run(Get &&get, Inside &&inside, Centre &&centre, int t, int g,
                                               float2 *part, float (&mean)[RW],
                                               float (&rstd)[RW]) const
    {
        float m2[RW];
#pragma unroll
        for (int r = 0; r < RW; ++r) {
            F2 s = get(r, 0);
#pragma unroll
            for (int p = 1; p < NP; ++p) s = add2(s, get(r, p));
            const float2 u = un2(s);
            mean[r] = u.x + u.y;
        }
#pragma unroll
        for (int r = 0; r < RW; ++r) mean[r] = lanes_sum<32>(mean[r]);
        const float s0 = mean[0];
#pragma unroll
        for (int r = 0; r < RW; ++r) {
            mean[r] *= r_own;
            const F2 mm = f2(-mean[r], -mean[r]), one = f2(1.f, 1.f);
            F2 q = f2(0.f, 0.f);
#pragma unroll
            for (int b = 0; b < NP / B; ++b) {
                const int in = inside(b);
                if (in == 1) {
#pragma unroll
                    for (int p = b * B; p < (b + 1) * B; ++p) {
                        const F2 d = fma2(get(r, p), one, mm);
                        q = fma2(d, d, q);
                    }
                } else if (in == 2) {
#pragma unroll
                    for (int p = b * B; p < (b + 1) * B; ++p) {
                        const F2 d = fma2(centre(r, mean[r], p), one, mm);
                        q = fma2(d, d, q);
                    }
                }
            }
            const float2 u = un2(q);
            m2[r] = u.x + u.y;
        }
#pragma unroll
        for (int r = 0; r < RW; ++r) m2[r] = lanes_sum<32>(m2[r]);
        if constexpr (WARPS > 1) {
            if ((threadIdx.x & 31) == 0) part[t >> 5] = make_float2(s0, m2[0]);
            group_sync<TPR, BLOCK>(g);
            const float2 p = part[threadIdx.x & (WARPS - 1)];
            mean[0] = lanes_sum<WARPS>(p.x) * inv_n;
            const float d = p.x * r_join - mean[0];
            m2[0] = lanes_sum<WARPS>(fmaf(n_join * d, d, p.y));
        }
#pragma unroll
        for (int r = 0; r < RW; ++r) rstd[r] = rsqrtf(m2[r] * inv_n + eps);
    }
};

__device__ __forceinline__ F2 normalised(F2 x, F2 minus_mean, F2 rstd, F2 w, F2 b)
{
    return fma2(mul2(fma2(x, f2(1.f, 1.f), minus_mean), rstd), w, b);
}

template <class T, int K, int TPR, int RW, int BLOCK>
__global__ void __launch_bounds__(BLOCK, 512 / BLOCK) k_ln_fwd_rows(const LnForward a)
{
    constexpr int VEC = 16 / (int)sizeof(T), P = VEC / 2;
    constexpr int G = BLOCK / TPR, WARPS = TPR / 32;
    static_assert(RW == 1 || TPR == 32, "several rows at a time belong to one warp");
    extern __shared__ __align__(16) float4 planes[];  // [2][VEC / 4][nvec]: weight, bias
    __shared__ float2 part[2][G][WARPS];
    wait_for_prior_grid();
    allow_dependent_launch();
    const int t = threadIdx.x % TPR, g = threadIdx.x / TPR, lane = threadIdx.x & 31;
    const int cols = (int)a.cols, nvec = cols / VEC;
    {
        float *const p = reinterpret_cast<float *>(planes);
        for (int c = threadIdx.x; c < cols; c += BLOCK) {
            float w[1], b[1];
            load_params<T, 1>(a.weight, a.ptype, false, c, 1.f, w);
            load_params<T, 1>(a.bias, a.ptype, false, c, 0.f, b);
            const int at = ((c % VEC / 4) * nvec + c / VEC) * 4 + (c & 3);
            p[at] = w[0];
            p[cols + at] = b[0];
        }
    }
    __syncthreads();
    const T *const x = static_cast<const T *>(a.x);
    T *const y = static_cast<T *>(a.y);
    const PairStats<K * P, TPR, RW, BLOCK> stats(cols, 32 * K * VEC, a.eps, t);
    const int first = (t >> 5) * (32 * K) + lane;  // this lane's first vector
    int buf = 0;
    const int64_t stride = (int64_t)gridDim.x * G * RW;
    int64_t row0 = ((int64_t)blockIdx.x * G + g) * RW;
    auto load = [&](int64_t r0, uint32_t (&v)[RW][4 * K]) {
#pragma unroll
        for (int r = 0; r < RW; ++r)
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const int j = first + 32 * k;
                const uint4 q =
                    j < nvec && r0 + r < a.rows
                        ? __ldcs(reinterpret_cast<const uint4 *>(x + (r0 + r) * a.ldx) + j)
                        : make_uint4(0, 0, 0, 0);
                v[r][4 * k] = q.x;
                v[r][4 * k + 1] = q.y;
                v[r][4 * k + 2] = q.z;
                v[r][4 * k + 3] = q.w;
            }
    };
    // a block that works on one row alone loads the next meanwhile (16384 fp32
    // columns 121 us without, 95 with; where other blocks share the SM it gains
    // nothing: 4096 bf16 columns 87 and 98)
    constexpr bool AHEAD = TPR == 512;
    uint32_t v[RW][4 * K], next[AHEAD ? RW : 1][4 * K];
    if constexpr (AHEAD) load(row0, next);
    for (; row0 < a.rows; row0 += stride) {
        if constexpr (AHEAD) {
#pragma unroll
            for (int r = 0; r < RW; ++r)
#pragma unroll
                for (int i = 0; i < 4 * K; ++i) v[r][i] = next[r][i];
            load(row0 + stride, next);
        } else {
            load(row0, v);
        }
        auto get = [&](int r, int p) { return pair_of<T>(v[r], p); };
        auto inside = [&](int k) { return first + 32 * k < nvec ? 1 : 0; };
        float mean[RW], rstd[RW];
        auto never = [&](int r, float, int p) { return get(r, p); };
        stats.template run<P>(get, inside, never, t, g, part[buf][g], mean, rstd);
        buf ^= 1;
#pragma unroll
        for (int r = 0; r < RW; ++r) {
            if (row0 + r >= a.rows) continue;
            if (a.mean && t == 0) {
                a.mean[row0 + r] = mean[r];
                a.rstd[row0 + r] = rstd[r];
            }
            const F2 mm = f2(-mean[r], -mean[r]), rr = f2(rstd[r], rstd[r]);
            uint4 *const out = reinterpret_cast<uint4 *>(y + (row0 + r) * a.ldy);
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const int j = first + 32 * k;
                if (j >= nvec) continue;
                F2 f[P];
#pragma unroll
                for (int p = 0; p < P; p += 2) {
                    const float4 w4 = planes[(p / 2) * nvec + j];
                    const float4 b4 = planes[(VEC / 4 + p / 2) * nvec + j];
                    f[p] = normalised(get(r, k * P + p), mm, rr, f2(w4.x, w4.y), f2(b4.x, b4.y));
                    f[p + 1] = normalised(get(r, k * P + p + 1), mm, rr, f2(w4.z, w4.w),
                                          f2(b4.z, b4.w));
                }
                __stcs(out + j, from_pairs<T>(f));
            }
        }
    }
}

// Blocks of 256 on an SM: three where a lane holds two vectors (67M elements of
// bf16 in rows of 333: 87 us, with two 98), else two (rows of 129: 135 us with two,
// three or four; rows of 1001 and four vectors a lane: 59 us, with three 61).
template <class T, int K, int TPR, int BLOCK, int D>
__global__ void __launch_bounds__(BLOCK, BLOCK == 512 ? 1 : K == 2 ? 3 : 2)
    k_ln_fwd_any(const LnForward a)
{
    constexpr int VEC = 16 / (int)sizeof(T), NP = K * VEC / 2;
    constexpr int G = BLOCK / TPR, WARPS = TPR / 32, STEP = pair_step<T>();
    constexpr int SLOTS = warp_slots<K, true>(), ROW = BLOCK / 32 * SLOTS;
    extern __shared__ __align__(16) uint4 ring[];  // [D][warps][SLOTS], then the parameters
    __shared__ float2 part[2][G][WARPS];
    wait_for_prior_grid();
    allow_dependent_launch();
    const int t = threadIdx.x % TPR, g = threadIdx.x / TPR, lane = threadIdx.x & 31;
    constexpr int B = NP % 4 ? 2 : 4;  // pairs a block
    const int cols = (int)a.cols, room = (cols + 64 * B - 1) / (64 * B) * (64 * B);
    const int base = (t >> 5) * (64 * NP);
    const uint4 *const mine = ring + (threadIdx.x >> 5) * SLOTS;
    const uint32_t slot = (uint32_t)__cvta_generic_to_shared(mine + lane);
    const T *const x = static_cast<const T *>(a.x);
    T *const y = static_cast<T *>(a.y);
    const int64_t stride = (int64_t)gridDim.x * G;
    int64_t row = (int64_t)blockIdx.x * G + g;
    auto issue = [&](int64_t r, int d) {
        if (r < a.rows)
            copy_row<T, K, true>(x, a.ldx, r, cols, base, slot + (uint32_t)(d * ROW) * 16);
        cp_async_commit();
    };
    for (int i = threadIdx.x; i < D * ROW; i += BLOCK) ring[i] = make_uint4(0, 0, 0, 0);
    __syncthreads();
#pragma unroll
    for (int d = 0; d < D - 1; ++d) issue(row + d * stride, d);
    float *const params = reinterpret_cast<float *>(ring + D * ROW);
    for (int c = threadIdx.x; c < room; c += BLOCK) {
        float w[1] = {0.f}, b[1] = {0.f};
        if (c < cols) {
            load_params<T, 1>(a.weight, a.ptype, false, c, 1.f, w);
            load_params<T, 1>(a.bias, a.ptype, false, c, 0.f, b);
        }
        params[c] = w[0];
        params[room + c] = b[0];
    }
    __syncthreads();
    const PairStats<NP, TPR, 1, BLOCK> stats(cols, 64 * NP, a.eps, t);
    int buf = 0, d = 0;
    for (; row < a.rows; row += stride) {
        issue(row + (D - 1) * stride, d == 0 ? D - 1 : d - 1);
        cp_async_wait<D - 1>();
        __syncwarp();
        uint32_t v[4 * K];
        take_row<T, K, true>(mine + d * ROW, past16(x + row * a.ldx), cols, base, v);
        if (++d == D) d = 0;
        auto get = [&](int, int p) { return pair_of<T>(v, p); };
        auto inside = [&](int b) {
            return cols - base >= 64 * B * (b + 1) ? 1 : cols - base > 64 * B * b ? 2 : 0;
        };
        auto centre = [&](int, float m, int p) {
            const int c = pair_column<T>(base, lane, p);
            const float2 u = un2(pair_of<T>(v, p));
            return f2(c < cols ? u.x : m, c + STEP < cols ? u.y : m);
        };
        float mean[1], rstd[1];
        stats.template run<B>(get, inside, centre, t, g, part[buf][g], mean, rstd);
        buf ^= 1;
        if (a.mean && t == 0) {
            a.mean[row] = mean[0];
            a.rstd[row] = rstd[0];
        }
        const F2 mm = f2(-mean[0], -mean[0]), rr = f2(rstd[0], rstd[0]);
        F2 f[NP];
#pragma unroll
        for (int b = 0; b < NP / B; ++b) {
            // the parameters reach to the end of the last block
            if (inside(b) == 0) continue;
#pragma unroll
            for (int p = b * B; p < (b + 1) * B; ++p) {
                const int c = pair_column<T>(base, lane, p);
                if constexpr (sizeof(T) == 2) {
                    const float2 w = *reinterpret_cast<const float2 *>(params + c);
                    const float2 z = *reinterpret_cast<const float2 *>(params + room + c);
                    f[p] = normalised(pair_of<T>(v, p), mm, rr, f2(w.x, w.y), f2(z.x, z.y));
                } else {
                    f[p] = normalised(pair_of<T>(v, p), mm, rr, f2(params[c], params[c + 32]),
                                      f2(params[room + c], params[room + c + 32]));
                }
            }
        }
        store_pairs<T, NP>(y + row * a.ldy, cols, base, f);
    }
    cp_async_wait<0>();
}

// ---- few rows, narrow rows ------------------------------------------------------------------

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

// ---- launches -------------------------------------------------------------------------------

template <class T, int VEC, int K, int TPR, int BLOCK>
static cudaError_t go(const LnForward &a, bool pvec, cudaStream_t s)
{
    const auto kernel = k_ln_fwd<T, VEC, K, TPR, BLOCK>;
    const int64_t ctas = (a.rows + BLOCK / TPR - 1) / (BLOCK / TPR);
    const int grid = grid_for((const void *)kernel, BLOCK, 0, ctas);
    return launch_after_prior(kernel, (unsigned)grid, BLOCK, 0, s, a, pvec);
}

template <class T, int K, int TPR, int RW>
static cudaError_t go_rows(const LnForward &a, cudaStream_t s)
{
    // one block an SM where the parameters of a row take much of its memory
    constexpr int BLOCK = TPR >= 256 ? 512 : 256;
    const auto kernel = k_ln_fwd_rows<T, K, TPR, RW, BLOCK>;
    const size_t smem = 2 * sizeof(float) * (size_t)a.cols;
    // what the widest row of the class needs: the limit belongs to the kernel, and
    // calls of other widths on other host threads must not lower it before this launch
    constexpr size_t most = 2 * sizeof(float) * (size_t)(K * TPR * (16 / (int)sizeof(T)));
    if (most > 40 * 1024) {
        cudaError_t e = cudaFuncSetAttribute(
            (const void *)kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
        if (e != cudaSuccess) return e;
    }
    const int64_t per = BLOCK / TPR * RW;
    // All of the shared memory only where the parameters need it: at 2048
    // columns it took 97 us in place of 84.  The choice is the kernel's, not the
    // width's, or it would depend on the widths called before.
    const int grid = grid_for((const void *)kernel, BLOCK, most, (a.rows + per - 1) / per,
                              most > 50 * 1024 ? cudaSharedmemCarveoutMaxShared : FC_CARVEOUT);
    return launch_after_prior(kernel, (unsigned)grid, BLOCK, smem, s, a);
}

template <class T, int K, int TPR>
static cudaError_t go_any(const LnForward &a, cudaStream_t s)
{
    constexpr int BLOCK = TPR >= 256 ? 512 : 256, D = 3;
    const auto kernel = k_ln_fwd_any<T, K, TPR, BLOCK, D>;
    constexpr size_t slots = (size_t)D * (BLOCK / 32) * warp_slots<K, true>() * 16;
    const size_t smem =
        slots + 2 * sizeof(float) * (size_t)((a.cols + 255) & ~(int64_t)255);
    // as in go_rows: the widest row's
    constexpr size_t most =
        slots + 2 * sizeof(float) * (size_t)((K * TPR * (16 / (int)sizeof(T)) + 255) & ~255);
    static_assert(most + 256 <= 227 * 1024, "a block's shared memory");
    cudaError_t e = cudaFuncSetAttribute((const void *)kernel,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
    if (e != cudaSuccess) return e;
    const int64_t ctas = (a.rows + BLOCK / TPR - 1) / (BLOCK / TPR);
    const int grid =
        grid_for((const void *)kernel, BLOCK, most, ctas, cudaSharedmemCarveoutMaxShared);
    return launch_after_prior(kernel, (unsigned)grid, BLOCK, smem, s, a);
}

// The smallest TPR * K that holds a row of n vectors.
template <class T>
static cudaError_t many_rows(const LnForward &a, int64_t n, cudaStream_t s)
{
    if (n <= 32) return go_rows<T, 1, 32, 4>(a, s);
    if (n <= 64) return go_rows<T, 2, 32, 4>(a, s);
    if (n <= 96) return go_rows<T, 3, 32, 2>(a, s);
    if (n <= 128) return go_rows<T, 4, 32, 2>(a, s);
    if (n <= 192) return go_rows<T, 6, 32, 1>(a, s);
    if (n <= 256) return go_rows<T, 8, 32, 1>(a, s);
    if (n <= 384) return go_rows<T, 6, 64, 1>(a, s);
    if (n <= 512) return go_rows<T, 8, 64, 1>(a, s);
    if (n <= 768) return go_rows<T, 6, 128, 1>(a, s);
    if (n <= 1024) return go_rows<T, 8, 128, 1>(a, s);
    if (n <= 1536) return go_rows<T, 6, 256, 1>(a, s);
    if constexpr (sizeof(T) == 4) {
        if (n > 3072) return go_rows<T, 8, 512, 1>(a, s);
        if (n > 2048) return go_rows<T, 6, 512, 1>(a, s);
    }
    return go_rows<T, 8, 256, 1>(a, s);
}

// Classes half as wide again as the last (K = 3) and twice as wide: 67M elements
// of bf16 in rows of 517 / 1101 / 2051 / 4101 columns took 96 / 99 / 108 / 104 us
// in classes of twice the width alone, 82 / 86 / 93 / 94 with both.
template <class T>
static cudaError_t many_rows_any(const LnForward &a, int64_t n, cudaStream_t s)
{
    if (n <= 32) return go_any<T, 1, 32>(a, s);
    if (n <= 64) return go_any<T, 2, 32>(a, s);
    if (n <= 96) return go_any<T, 3, 32>(a, s);
    if (n <= 128) return go_any<T, 4, 32>(a, s);
    if (n <= 192) return go_any<T, 3, 64>(a, s);
    if (n <= 256) return go_any<T, 4, 64>(a, s);
    if (n <= 384) return go_any<T, 3, 128>(a, s);
    if (n <= 512) return go_any<T, 4, 128>(a, s);
    if (n <= 768) return go_any<T, 3, 256>(a, s);
    if (n <= 1024) return go_any<T, 4, 256>(a, s);
    if (n <= 1536) return go_any<T, 3, 512>(a, s);
    return go_any<T, 4, 512>(a, s);
}

// Few rows: what counts is the latency of a row, so a row is spread over as many
// threads as it has vectors, to 1024 (or four elements a thread, more above 4096
// columns), and no ring and no copy of the parameters is set up first.  Where that
// ends is measured, few
// against many in us: rows of vectors, 1 MB of 256 columns 1.85 and 2.44
// (bf16), 2.50 and 2.47 (fp32), and 2 MB 3.02 and 2.49, 3.12 and 2.48; of 1024
// columns 2 MB 2.93 and 3.49 (bf16), 3.04 and 2.51 (fp32), 4 MB 3.65 and 3.58
// (bf16); of 2048 columns 2 MB 2.49 and 2.89 and 4 MB 3.75 and 2.99 (fp32), 4
// MB 4.29 and 4.40 (bf16).  Rows word by word, 523 of 1001 columns 3.91 and 3.78
// (bf16), 3.48 and 3.35 (fp32); 1047 rows 4.93 and 3.84, 4.45 and 4.01; 524 of
// 2001 columns 4.79 and 4.91, 4.37 and 4.80; bf16, 512 of 8001 columns 8.1 and
// 9.9, but of 12001 columns, whose rows take an SM each, 20.3 and 15.3 (128 rows:
// 6.7 and 9.1).  fp32 rows of 8193 to 16384 columns have only the three passes
// beside it: 512 of 12001 columns 22 and 29.
template <class T>
static bool few_rows(int64_t rows, int64_t n, bool vectors)
{
    if (!vectors) return rows <= (sizeof(T) == 2 && n > 1024 ? 152 : 512);
    const int shift = sizeof(T) == 2 ? (n > 64 ? 18 : 16) : (n > 256 ? 17 : 16);
    return rows * n <= (int64_t)1 << shift;
}

template <class T>
cudaError_t ln_forward(const LnForward &a, cudaStream_t s)
{
    constexpr int V = 16 / (int)sizeof(T);
    auto on16 = [](const void *p, int64_t ld) {
        return ((uintptr_t)p & 15) == 0 && (ld * (int64_t)sizeof(T)) % 16 == 0;
    };
    const bool pvec = ((uintptr_t)a.weight & 15) == 0 && ((uintptr_t)a.bias & 15) == 0;
    const int64_t c = a.cols, n = (c + V - 1) / V;
    const bool vectors = c % V == 0 && on16(a.x, a.ldx) && on16(a.y, a.ldy);
    const bool few = few_rows<T>(a.rows, n, vectors);
    const bool one_pass = vectors ? n <= (sizeof(T) == 4 ? 4096 : 2048)
                                  : n <= 2048 || (few && c <= 16384);
    if (!one_pass) {
        const auto wide = k_ln_fwd_wide<T>;
        const int grid = grid_for((const void *)wide, FC_LN_WIDE_BLOCK, 0, a.rows);
        return launch_after_prior(wide, (unsigned)grid, FC_LN_WIDE_BLOCK, 0, s, a);
    }
    if (vectors) {
        if (n <= 8) return go<T, V, 1, 8, 128>(a, pvec, s);
        if (n <= 16) return go<T, V, 1, 16, 128>(a, pvec, s);
        if (!few) return many_rows<T>(a, n, s);
        if (n <= 32) return go<T, V, 1, 32, 128>(a, pvec, s);
        if (n <= 128) return go<T, V, 1, 128, 256>(a, pvec, s);
        if (n <= 256) return go<T, V, 1, 256, 256>(a, pvec, s);
        if (n <= 512) return go<T, V, 1, 512, 512>(a, pvec, s);
        if (n <= 1024) return go<T, V, 1, 1024, 1024>(a, pvec, s);
        if (n <= 2048) return go<T, V, 2, 1024, 1024>(a, pvec, s);
        return many_rows<T>(a, n, s);
    }
    if (c <= 32) return go<T, 1, 1, 32, 128>(a, pvec, s);
    if (c <= 128) return go<T, 1, 4, 32, 128>(a, pvec, s);
    if (!few) return many_rows_any<T>(a, n, s);
    if (c <= 512) return go<T, 1, 4, 128, 256>(a, pvec, s);
    if (c <= 1024) return go<T, 1, 4, 256, 256>(a, pvec, s);
    if (c <= 2048) return go<T, 1, 4, 512, 512>(a, pvec, s);
    if (c <= 4096) return go<T, 1, 4, 1024, 1024>(a, pvec, s);
    if (c <= 8192) return go<T, 1, 8, 1024, 1024>(a, pvec, s);
    return go<T, 1, 16, 1024, 1024>(a, pvec, s);
}

}  // namespace fc
