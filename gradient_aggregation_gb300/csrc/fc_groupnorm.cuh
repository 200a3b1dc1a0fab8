// Pieces that the group norm kernels share.
//
// A block of T threads works on a slab of channels, cut into vectors of AB bytes
// (16 where every row starts on a 16-byte boundary, else 4 or one element):
// thread t holds vector t % V of rows t / V, t / V + T / V, ..., so its channels
// stay the same and what belongs to a channel stays in its registers.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fc.h"
#include "fc_cluster.cuh"
#include "fc_groupnorm.h"
#include "fc_internal.h"
#include "fc_pairs.cuh"

namespace fc {

template <int AB>
struct GnRaw;
template <>
struct GnRaw<16> {
    using type = uint4;
};
template <>
struct GnRaw<4> {
    using type = uint32_t;
};
template <>
struct GnRaw<2> {
    using type = unsigned short;
};

// AB bytes of T as pairs of fp32; a single element is paired with 0.
template <class T, int AB>
struct Gv {
    static constexpr int NE = AB / (int)sizeof(T);
    static constexpr int NP = (NE + 1) / 2;
    using Raw = typename GnRaw<AB>::type;

    static __device__ __forceinline__ void get(const Raw &r, F2 (&f)[NP])
    {
        if constexpr (AB == 16) {
            const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
            for (int p = 0; p < NP; ++p) {
                if constexpr (sizeof(T) == 4)
                    f[p] = f2(__uint_as_float(w[2 * p]), __uint_as_float(w[2 * p + 1]));
                else
                    f[p] = pair_of_word<T>(w[p]);
            }
        } else if constexpr (sizeof(T) == 4) {
            f[0] = f2(__uint_as_float(r), 0.f);
        } else {
            f[0] = pair_of_word<T>((uint32_t)r);
        }
    }

    static __device__ __forceinline__ Raw put(const F2 (&f)[NP])
    {
        if constexpr (AB == 16)
            return from_pairs<T>(f);
        else if constexpr (sizeof(T) == 4)
            return __float_as_uint(un2(f[0]).x);
        else
            return (Raw)word_of_pair<T>(f[0]);
    }
};

__device__ __forceinline__ float gn_param(const void *p, int ptype, int type16, int64_t c, float none)
{
    if (!p) return none;
    if (ptype == FC_TYPE_F32) return __ldg(static_cast<const float *>(p) + c);
    if (type16 == FC_TYPE_F16) return __half2float(static_cast<const __half *>(p)[c]);
    return __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[c]);
}

template <class T>
constexpr int gn_type()
{
    return sizeof(T) == 4 ? FC_TYPE_F32 : __is_same(T, __half) ? FC_TYPE_F16 : FC_TYPE_BF16;
}

// Channels c0.. of a parameter as pairs; those past `end` are 0.
template <class T, int NE>
__device__ __forceinline__ void gn_params(const void *p, int ptype, int64_t c0, float none,
                                          F2 (&f)[(NE + 1) / 2])
{
    float v[NE + 1];
    v[NE] = 0.f;
#pragma unroll
    for (int e = 0; e < NE; ++e) v[e] = gn_param(p, ptype, gn_type<T>(), c0 + e, none);
#pragma unroll
    for (int q = 0; q < (NE + 1) / 2; ++q) f[q] = f2(v[2 * q], v[2 * q + 1]);
}

// x / (1 + e^-x): the exponential and the quotient are within 2 ulp each, and the
// exponent's own rounding adds |x| ulp.
__device__ __forceinline__ float gn_silu(float z) { return __fdividef(z, 1.f + __expf(-z)); }

template <int ACT>
__device__ __forceinline__ float gn_act(float z)
{
    if (ACT == FC_ACT_RELU) return z < 0.f ? 0.f : z;  // keeps NaN
    if (ACT == FC_ACT_SILU) return gn_silu(z);
    return z;
}

// Which side of 0 a value lies on that fp32 cannot tell: an error of z's size would be
// one of the gradient's.  Reached by about one value in a million.
static __device__ __noinline__ bool gn_positive(float x, float mean, float rstd, float w, float b)
{
    return ((double)x - (double)mean) * (double)rstd * (double)w + (double)b > 0.0;
}

// dy * act'(z), z = h w + b, h = (x - mean) rstd.
template <int ACT>
__device__ __forceinline__ float gn_dz(float dy, float x, float mean, float rstd, float h, float w,
                                       float b)
{
    if (ACT == FC_ACT_NONE) return dy;
    const float z = fmaf(h, w, b);
    if (ACT == FC_ACT_RELU) {
        bool on = z > 0.f;
        // z's error is below 5 roundings of b, where h w nearly cancels it; without b
        // the sign is exact
        if (fabsf(z) < fabsf(b) * 0x1p-20f) on = gn_positive(x, mean, rstd, w, b);
        return on ? dy : 0.f;
    }
    // s (1 + z (1 - s))
    const float s = __fdividef(1.f, 1.f + __expf(-z));
    return dy * (s * fmaf(z, 1.f - s, 1.f));
}

template <int ACT, int NP>
__device__ __forceinline__ void gn_dz_pairs(const F2 (&dy)[NP], const F2 (&x)[NP], const F2 (&mean)[NP],
                                            const F2 (&rstd)[NP], const F2 (&h)[NP],
                                            const F2 (&w)[NP], const F2 (&b)[NP], F2 (&dz)[NP])
{
#pragma unroll
    for (int p = 0; p < NP; ++p) {
        if (ACT == FC_ACT_NONE) {
            dz[p] = dy[p];
        } else {
            const float2 y = un2(dy[p]), u = un2(x[p]), m = un2(mean[p]), r = un2(rstd[p]),
                         g = un2(h[p]), v = un2(w[p]), c = un2(b[p]);
            dz[p] = f2(gn_dz<ACT>(y.x, u.x, m.x, r.x, g.x, v.x, c.x),
                       gn_dz<ACT>(y.y, u.y, m.y, r.y, g.y, v.y, c.y));
        }
    }
}

__device__ __forceinline__ F2 neg2(F2 a)
{
    const float2 v = un2(a);
    return f2(-v.x, -v.y);
}

// ---- streaming: any alignment, groups of any size -----------------------------------------
//
// The samples' statistics are formed first (a pass over the positions, cut into
// parts, and one over what the parts leave), and a second pass over the positions
// writes the result.

struct GnTile {
    int vecs;      // vectors of a row: channels * sizeof(T) / AB
    int tiles, vt; // tiles of vt vectors (the last may be narrower)
    int parts;     // parts of the positions
    int64_t rows;  // positions of a part
};

#define FC_GN_BLOCK 256
#define FC_GN_RUN 64  // rows between two fresh pivots

struct GnPlace {
    int64_t n, first, end;  // sample, this block's positions
    int part, v, r, R, c0;  // part, vector of the tile, row, rows at a time, first channel
    bool on;
};

template <int NE>
__device__ __forceinline__ GnPlace gn_place(const GnTile &t, int64_t positions)
{
    GnPlace q;
    const int64_t b = blockIdx.x;
    const int tile = (int)(b % t.tiles);
    const int64_t np = b / t.tiles;
    q.part = (int)(np % t.parts);
    q.n = np / t.parts;
    q.first = q.part * t.rows;
    q.end = q.first + t.rows < positions ? q.first + t.rows : positions;
    const int vt = min(t.vt, t.vecs - tile * t.vt);
    q.R = FC_GN_BLOCK / vt;
    q.v = threadIdx.x % vt;
    q.r = threadIdx.x / vt;
    q.on = q.r < q.R;
    q.c0 = (tile * t.vt + q.v) * NE;
    return q;
}

// Per channel of a part: mean and sum of squared differences from it.
//
// A thread sums x - p and (x - p)^2 for a p among its own values, over at most
// FC_GN_RUN rows, and joins such runs by their means: the error is FC_GN_RUN
// roundings of the sum of squares even if p lies far from all the other values,
// as p itself adds as much to the sum.
template <class T, int AB>
__global__ void __launch_bounds__(FC_GN_BLOCK)
    k_gn_stats(const GnImages x, const GnShape n, const GnTile tile, float *__restrict__ out,
               const int64_t sets)
{
    using V = Gv<T, AB>;
    constexpr int NE = V::NE, NP = V::NP;
    __shared__ float sm[2][FC_GN_BLOCK * NE];
    wait_for_prior_grid();
    allow_dependent_launch();
    const GnPlace q = gn_place<NE>(tile, n.positions);
    const T *base = static_cast<const T *>(x.p) + q.n * x.ss + q.c0;
    F2 mean[NP], m2[NP];
#pragma unroll
    for (int p = 0; p < NP; ++p) mean[p] = m2[p] = f2(0.f, 0.f);
    float count = 0.f;
    if (q.on) {
        for (int64_t run = q.first + q.r; run < q.end; run += (int64_t)FC_GN_RUN * q.R) {
            F2 neg[NP], s[NP], ss[NP];
            float k = 0.f;
#pragma unroll 4
            for (int i = 0; i < FC_GN_RUN; ++i) {
                const int64_t row = run + (int64_t)i * q.R;
                if (row >= q.end) break;
                F2 f[NP];
                V::get(*reinterpret_cast<const typename V::Raw *>(base + row * x.ld), f);
#pragma unroll
                for (int p = 0; p < NP; ++p) {
                    if (i == 0) {
                        neg[p] = neg2(f[p]);
                        s[p] = ss[p] = f2(0.f, 0.f);
                    } else {
                        const F2 d = add2(f[p], neg[p]);
                        s[p] = add2(s[p], d);
                        ss[p] = fma2(d, d, ss[p]);
                    }
                }
                k += 1.f;
            }
            const float inv = 1.f / k, total = count + k, part = k / total;
#pragma unroll
            for (int p = 0; p < NP; ++p) {
                const F2 ms = mul2(s[p], f2(inv, inv));
                // sum of squares about the run's mean, and the run's mean
                const F2 r2 = fma2(neg2(ms), s[p], ss[p]);
                const F2 rm = add2(ms, neg2(neg[p]));
                const F2 d = add2(rm, neg2(mean[p]));
                mean[p] = fma2(d, f2(part, part), mean[p]);
                m2[p] = add2(m2[p], fma2(mul2(d, d), f2(count * part, count * part), r2));
            }
            count = total;
        }
    }
    if (q.on) {
#pragma unroll
        for (int e = 0; e < NE; ++e) {
            const float2 a = un2(mean[e / 2]), b = un2(m2[e / 2]);
            sm[0][threadIdx.x * NE + e] = e & 1 ? a.y : a.x;
            sm[1][threadIdx.x * NE + e] = e & 1 ? b.y : b.x;
        }
    }
    __syncthreads();
    // one thread a channel joins the R rows of threads
    const int vt = min(tile.vt, tile.vecs - (int)(blockIdx.x % tile.tiles) * tile.vt);
    const int64_t rows = q.end - q.first;
    const int64_t set = q.n * tile.parts + q.part, padded = (n.channels + 7) & ~7;
    const int first = (int)(blockIdx.x % tile.tiles) * tile.vt * NE;
    for (int c = threadIdx.x; c < vt * NE; c += FC_GN_BLOCK) {
        float sum = 0.f;
        for (int r = 0; r < q.R; ++r) {
            const int64_t have = rows > r ? (rows - r + q.R - 1) / q.R : 0;
            sum = fmaf((float)have, sm[0][r * vt * NE + c], sum);
        }
        const float m = rows > 0 ? sum / (float)rows : 0.f;
        float sq = 0.f;
        for (int r = 0; r < q.R; ++r) {
            const int64_t have = rows > r ? (rows - r + q.R - 1) / q.R : 0;
            const float d = sm[0][r * vt * NE + c] - m;
            sq += have ? fmaf((float)have * d, d, sm[1][r * vt * NE + c]) : 0.f;
        }
        out[set * padded + first + c] = m;
        out[(sets + set) * padded + first + c] = sq;
    }
}

template <int TPG>
__device__ __forceinline__ float gn_team_sum(float v, float *sm)
{
    v = warp_sum_f32(v);
    if constexpr (TPG > 32) {
        __syncthreads();
        if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = v;
        __syncthreads();
        v = 0.f;
#pragma unroll
        for (int i = 0; i < TPG / 32; ++i) v += sm[i];
    }
    return v;
}

// Joins the parts and channels of every group: TPG threads a group and sample.
template <int TPG>
__global__ void __launch_bounds__(256)
    k_gn_finish(const GnShape n, const int parts, const int64_t part_rows,
                const float *__restrict__ in, const int64_t sets, const float eps,
                float *__restrict__ stat, float *mean_out, float *rstd_out)
{
    __shared__ float sm[8];
    wait_for_prior_grid();
    allow_dependent_launch();
    const int64_t at = (int64_t)blockIdx.x * (256 / TPG) + threadIdx.x / TPG;
    if (at >= n.samples * n.groups) return;  // whole warps, or whole blocks
    const int lane = threadIdx.x % TPG, cpg = n.channels / n.groups;
    const int64_t sample = at / n.groups, padded = (n.channels + 7) & ~7;
    const int c0 = (int)(at - sample * n.groups) * cpg;
    const int64_t entries = (int64_t)parts * cpg;
    const float total = (float)n.positions * (float)cpg;
    float s = 0.f;
    for (int64_t i = lane; i < entries; i += TPG) {
        const int64_t p = i / cpg;
        const int64_t set = sample * parts + p;
        const int64_t left = n.positions - p * part_rows;
        const float have = (float)(left < part_rows ? left : part_rows);
        s = fmaf(have, __ldcg(in + set * padded + c0 + (i - p * cpg)), s);
    }
    const float m = gn_team_sum<TPG>(s, sm) / total;
    float q = 0.f;
    for (int64_t i = lane; i < entries; i += TPG) {
        const int64_t p = i / cpg;
        const int64_t set = sample * parts + p;
        const int64_t left = n.positions - p * part_rows;
        const float have = (float)(left < part_rows ? left : part_rows);
        const int64_t j = set * padded + c0 + (i - p * cpg);
        const float d = __ldcg(in + j) - m;
        q += fmaf(have * d, d, __ldcg(in + sets * padded + j));
    }
    q = gn_team_sum<TPG>(q, sm);
    if (lane == 0) {
        const float r = 1.f / sqrtf(q / total + eps);
        stat[2 * at] = m;
        stat[2 * at + 1] = r;
        if (mean_out) {
            mean_out[at] = m;
            rstd_out[at] = r;
        }
    }
}

// y from the statistics.
template <class T, int AB, int ACT>
__global__ void __launch_bounds__(FC_GN_BLOCK)
    k_gn_apply(const GnForward a, const GnTile tile, const float *__restrict__ stat)
{
    using V = Gv<T, AB>;
    constexpr int NE = V::NE, NP = V::NP;
    const GnPlace q = gn_place<NE>(tile, a.n.positions);
    const int cpg = a.n.channels / a.n.groups;
    F2 w[NP], b[NP], m[NP];
    if (q.on) {
        gn_params<T, NE>(a.weight, a.ptype, q.c0, 1.f, w);
        gn_params<T, NE>(a.bias, a.ptype, q.c0, 0.f, b);
    }
    wait_for_prior_grid();
    allow_dependent_launch();
    if (!q.on) return;
    const float *st = stat + 2 * q.n * a.n.groups;
#pragma unroll
    for (int p = 0; p < NP; ++p) {
        const int g0 = (q.c0 + 2 * p) / cpg, g1 = NE > 1 ? (q.c0 + 2 * p + 1) / cpg : g0;
        m[p] = f2(-__ldcg(st + 2 * g0), -__ldcg(st + 2 * g1));
        w[p] = mul2(w[p], f2(__ldcg(st + 2 * g0 + 1), __ldcg(st + 2 * g1 + 1)));
    }
    const T *x = static_cast<const T *>(a.x.p) + q.n * a.x.ss + q.c0;
    T *y = static_cast<T *>(const_cast<void *>(a.y.p)) + q.n * a.y.ss + q.c0;
#pragma unroll 4
    for (int64_t row = q.first + q.r; row < q.end; row += q.R) {
        F2 f[NP];
        V::get(__ldcs(reinterpret_cast<const typename V::Raw *>(x + row * a.x.ld)), f);
#pragma unroll
        for (int p = 0; p < NP; ++p) {
            f[p] = fma2(add2(f[p], m[p]), w[p], b[p]);
            if (ACT != FC_ACT_NONE) {
                const float2 z = un2(f[p]);
                f[p] = f2(gn_act<ACT>(z.x), gn_act<ACT>(z.y));
            }
        }
        __stcs(reinterpret_cast<typename V::Raw *>(y + row * a.y.ld), V::put(f));
    }
}

// What a thread of the backward pass holds of its channels.
template <class T, int NE>
struct GnChannels {
    static constexpr int NP = (NE + 1) / 2;
    F2 neg[NP], mean[NP], rstd[NP], w[NP], b[NP];

    __device__ __forceinline__ void params(const GnBackward &a, int64_t c)
    {
        gn_params<T, NE>(a.weight, a.ptype, c, 1.f, w);
        gn_params<T, NE>(a.bias, a.ptype, c, 0.f, b);
    }
    // mean and rstd of the groups that channels c.. of sample n belong to
    __device__ __forceinline__ void stats(const GnBackward &a, int64_t n, int c, int cpg)
    {
        const float *m = a.mean + n * a.n.groups, *r = a.rstd + n * a.n.groups;
#pragma unroll
        for (int p = 0; p < NP; ++p) {
            const int g0 = (c + 2 * p) / cpg, g1 = NE > 1 ? (c + 2 * p + 1) / cpg : g0;
            mean[p] = f2(__ldg(m + g0), __ldg(m + g1));
            rstd[p] = f2(__ldg(r + g0), __ldg(r + g1));
            neg[p] = neg2(mean[p]);
        }
    }
    // h and dz of a vector
    template <int ACT>
    __device__ __forceinline__ void at(const F2 (&x)[NP], const F2 (&dy)[NP], F2 (&h)[NP],
                                       F2 (&dz)[NP]) const
    {
#pragma unroll
        for (int p = 0; p < NP; ++p) h[p] = mul2(add2(x[p], neg[p]), rstd[p]);
        gn_dz_pairs<ACT, NP>(dy, x, mean, rstd, h, w, b, dz);
    }
};

// Per channel of a part: the sums of dz h and of dz.
template <class T, int AB, int ACT>
__global__ void __launch_bounds__(FC_GN_BLOCK)
    k_gn_sums(const GnBackward a, const GnTile tile, float *__restrict__ out, const int64_t sets)
{
    using V = Gv<T, AB>;
    constexpr int NE = V::NE, NP = V::NP;
    __shared__ float sm[2][FC_GN_BLOCK * NE];
    wait_for_prior_grid();
    allow_dependent_launch();
    const GnPlace q = gn_place<NE>(tile, a.n.positions);
    F2 sh[NP], s[NP];
#pragma unroll
    for (int p = 0; p < NP; ++p) sh[p] = s[p] = f2(0.f, 0.f);
    if (q.on) {
        GnChannels<T, NE> ch;
        ch.params(a, q.c0);
        ch.stats(a, q.n, q.c0, a.n.channels / a.n.groups);
        const T *x = static_cast<const T *>(a.x.p) + q.n * a.x.ss + q.c0;
        const T *dy = static_cast<const T *>(a.dy.p) + q.n * a.dy.ss + q.c0;
#pragma unroll 2
        for (int64_t row = q.first + q.r; row < q.end; row += q.R) {
            F2 f[NP], g[NP], h[NP], dz[NP];
            V::get(*reinterpret_cast<const typename V::Raw *>(x + row * a.x.ld), f);
            V::get(*reinterpret_cast<const typename V::Raw *>(dy + row * a.dy.ld), g);
            ch.template at<ACT>(f, g, h, dz);
#pragma unroll
            for (int p = 0; p < NP; ++p) {
                sh[p] = fma2(dz[p], h[p], sh[p]);
                s[p] = add2(s[p], dz[p]);
            }
        }
#pragma unroll
        for (int e = 0; e < NE; ++e) {
            const float2 u = un2(sh[e / 2]), v = un2(s[e / 2]);
            sm[0][threadIdx.x * NE + e] = e & 1 ? u.y : u.x;
            sm[1][threadIdx.x * NE + e] = e & 1 ? v.y : v.x;
        }
    }
    __syncthreads();
    const int vt = min(tile.vt, tile.vecs - (int)(blockIdx.x % tile.tiles) * tile.vt);
    const int64_t set = q.n * tile.parts + q.part, padded = (a.n.channels + 7) & ~7;
    const int first = (int)(blockIdx.x % tile.tiles) * tile.vt * NE;
    for (int c = threadIdx.x; c < vt * NE; c += FC_GN_BLOCK) {
        float u = 0.f, v = 0.f;
        for (int r = 0; r < q.R; ++r) {
            u += sm[0][r * vt * NE + c];
            v += sm[1][r * vt * NE + c];
        }
        out[set * padded + first + c] = u;
        out[(sets + set) * padded + first + c] = v;
    }
}

// sum q / M and sum q h / M of every group and sample, from the parts' sums.
template <class T, int TPG>
__global__ void __launch_bounds__(256)
    k_gn_finish_sums(const GnBackward a, const int parts, const float *__restrict__ in,
                     const int64_t sets, float *__restrict__ stat)
{
    __shared__ float sm[8];
    wait_for_prior_grid();
    allow_dependent_launch();
    const GnShape &n = a.n;
    const int64_t at = (int64_t)blockIdx.x * (256 / TPG) + threadIdx.x / TPG;
    if (at >= n.samples * n.groups) return;
    const int lane = threadIdx.x % TPG, cpg = n.channels / n.groups;
    const int64_t sample = at / n.groups, padded = (n.channels + 7) & ~7;
    const int c0 = (int)(at - sample * n.groups) * cpg;
    const int64_t entries = (int64_t)parts * cpg;
    const float inv = 1.f / ((float)n.positions * (float)cpg);
    float s1 = 0.f, s2 = 0.f;
    for (int64_t i = lane; i < entries; i += TPG) {
        const int64_t p = i / cpg;
        const int c = c0 + (int)(i - p * cpg);
        const float w = gn_param(a.weight, a.ptype, gn_type<T>(), c, 1.f);
        const int64_t j = (sample * parts + p) * padded + c;
        s2 = fmaf(w, __ldcg(in + j), s2);
        s1 = fmaf(w, __ldcg(in + sets * padded + j), s1);
    }
    s1 = gn_team_sum<TPG>(s1, sm);
    s2 = gn_team_sum<TPG>(s2, sm);
    if (lane == 0) {
        stat[2 * at] = s1 * inv;
        stat[2 * at + 1] = s2 * inv;
    }
}

// dx of a vector: rstd (dz w - c1 - h c2).
template <int NP>
__device__ __forceinline__ void gn_dx(const F2 (&dz)[NP], const F2 (&h)[NP], const F2 (&w)[NP],
                                      const F2 (&rstd)[NP], const F2 (&n1)[NP], const F2 (&n2)[NP],
                                      F2 (&dx)[NP])
{
#pragma unroll
    for (int p = 0; p < NP; ++p)
        dx[p] = mul2(fma2(h[p], n2[p], fma2(dz[p], w[p], n1[p])), rstd[p]);
}

template <class T, int AB, int ACT>
__global__ void __launch_bounds__(FC_GN_BLOCK)
    k_gn_apply_bwd(const GnBackward a, const GnTile tile, const float *__restrict__ stat)
{
    using V = Gv<T, AB>;
    constexpr int NE = V::NE, NP = V::NP;
    wait_for_prior_grid();
    allow_dependent_launch();
    const GnPlace q = gn_place<NE>(tile, a.n.positions);
    if (!q.on) return;
    const int cpg = a.n.channels / a.n.groups;
    GnChannels<T, NE> ch;
    ch.params(a, q.c0);
    ch.stats(a, q.n, q.c0, cpg);
    F2 n1[NP], n2[NP];
    const float *st = stat + 2 * q.n * a.n.groups;
#pragma unroll
    for (int p = 0; p < NP; ++p) {
        const int g0 = (q.c0 + 2 * p) / cpg, g1 = NE > 1 ? (q.c0 + 2 * p + 1) / cpg : g0;
        n1[p] = f2(-__ldcg(st + 2 * g0), -__ldcg(st + 2 * g1));
        n2[p] = f2(-__ldcg(st + 2 * g0 + 1), -__ldcg(st + 2 * g1 + 1));
    }
    const T *x = static_cast<const T *>(a.x.p) + q.n * a.x.ss + q.c0;
    const T *dy = static_cast<const T *>(a.dy.p) + q.n * a.dy.ss + q.c0;
    T *dx = static_cast<T *>(const_cast<void *>(a.dx.p)) + q.n * a.dx.ss + q.c0;
#pragma unroll 2
    for (int64_t row = q.first + q.r; row < q.end; row += q.R) {
        F2 f[NP], g[NP], h[NP], dz[NP];
        V::get(__ldcs(reinterpret_cast<const typename V::Raw *>(x + row * a.x.ld)), f);
        V::get(__ldcs(reinterpret_cast<const typename V::Raw *>(dy + row * a.dy.ld)), g);
        ch.template at<ACT>(f, g, h, dz);
        F2 o[NP];
        gn_dx<NP>(dz, h, ch.w, ch.rstd, n1, n2, o);
        __stcs(reinterpret_cast<typename V::Raw *>(dx + row * a.dx.ld), V::put(o));
    }
}

// ---- host ------------------------------------------------------------------------------------

// Widest access that every row of the images allows: 16, 4 or sizeof(T) bytes.
template <class T>
int gn_access(const GnShape &n, std::initializer_list<const GnImages *> images)
{
    uintptr_t bits = (uintptr_t)n.channels * sizeof(T);
    for (const GnImages *i : images) {
        bits |= (uintptr_t)i->p;
        if (n.positions > 1) bits |= (uintptr_t)i->ld * sizeof(T);
        if (n.samples > 1) bits |= (uintptr_t)i->ss * sizeof(T);
    }
    return bits % 16 == 0 ? 16 : bits % 4 == 0 ? 4 : (int)sizeof(T);
}

inline GnTile gn_tile(const GnShape &n, int ne)
{
    GnTile t;
    t.vecs = n.channels / ne;
    t.tiles = (t.vecs + FC_GN_BLOCK - 1) / FC_GN_BLOCK;
    t.vt = (t.vecs + t.tiles - 1) / t.tiles;
    t.parts = (int)gn_parts(n);
    t.rows = (n.positions + t.parts - 1) / t.parts;
    return t;
}

inline unsigned gn_grid(const GnShape &n, const GnTile &t)
{
    return (unsigned)(n.samples * t.parts * t.tiles);
}

}  // namespace fc
