// Pieces that the group norm kernels share.
//
// A block of T threads works on a slab of channels, cut into vectors of AB bytes
// (16 where every row starts on a 16-byte boundary, else 4 or one element):
// thread t holds vector t % V of rows t / V, t / V + T / V, ..., so its channels
// stay the same and what belongs to a channel stays in its registers.
#pragma once

#include <algorithm>

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
struct GnRaw<8> {
    using type = uint2;
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
        } else if constexpr (AB == 8) {
            if constexpr (sizeof(T) == 4) {
                f[0] = f2(__uint_as_float(r.x), __uint_as_float(r.y));
            } else {
                f[0] = pair_of_word<T>(r.x);
                f[1] = pair_of_word<T>(r.y);
            }
        } else if constexpr (sizeof(T) == 4) {
            f[0] = f2(__uint_as_float(r), 0.f);
        } else {
            f[0] = pair_of_word<T>((uint32_t)r);
        }
    }

    static __device__ __forceinline__ Raw put(const F2 (&f)[NP])
    {
        if constexpr (AB == 16) {
            return from_pairs<T>(f);
        } else if constexpr (AB == 8) {
            if constexpr (sizeof(T) == 4) {
                const float2 a = un2(f[0]);
                return make_uint2(__float_as_uint(a.x), __float_as_uint(a.y));
            } else {
                return make_uint2(word_of_pair<T>(f[0]), word_of_pair<T>(f[1]));
            }
        } else if constexpr (sizeof(T) == 4)
            return __float_as_uint(un2(f[0]).x);
        else
            return (Raw)word_of_pair<T>(f[0]);
    }
};

template <class T>
__device__ __forceinline__ float gn_param(const void *p, int ptype, int64_t c, float none)
{
    if (!p) return none;
    if (sizeof(T) == 4 || ptype == FC_TYPE_F32) return __ldg(static_cast<const float *>(p) + c);
    if constexpr (__is_same(T, __half))
        return __half2float(static_cast<const __half *>(p)[c]);
    else if constexpr (sizeof(T) == 2)
        return __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[c]);
    return none;
}

// Channels c0 (a multiple of NE) and the next of a parameter, as pairs.
template <class T, int NE>
__device__ __forceinline__ void gn_params(const void *p, int ptype, int64_t c0, float none,
                                          F2 (&f)[(NE + 1) / 2])
{
    constexpr int NP = (NE + 1) / 2;
    if (!p) {
#pragma unroll
        for (int q = 0; q < NP; ++q) f[q] = f2(none, NE > 1 ? none : 0.f);
        return;
    }
    const bool whole = ((uintptr_t)p & 15) == 0;
    if (NE >= 4 && whole && (sizeof(T) == 4 || ptype == FC_TYPE_F32)) {
        const float4 *q = reinterpret_cast<const float4 *>(static_cast<const float *>(p) + c0);
#pragma unroll
        for (int i = 0; i < NE / 4; ++i) {
            const float4 v = __ldg(q + i);
            f[2 * i] = f2(v.x, v.y);
            f[2 * i + 1] = f2(v.z, v.w);
        }
        return;
    }
    if constexpr (NE == 8 && sizeof(T) == 2) {
        if (whole) {
            Gv<T, 16>::get(__ldg(reinterpret_cast<const uint4 *>(static_cast<const T *>(p) + c0)), f);
            return;
        }
    }
    float v[NE + 1];
    v[NE] = 0.f;
#pragma unroll
    for (int e = 0; e < NE; ++e) v[e] = gn_param<T>(p, ptype, c0 + e, none);
#pragma unroll
    for (int q = 0; q < NP; ++q) f[q] = f2(v[2 * q], v[2 * q + 1]);
}

__device__ __forceinline__ F2 neg2(F2 a)
{
    const float2 v = un2(a);
    return f2(-v.x, -v.y);
}

// 1 / (1 + e^-z) of a vector, off by 10 + 1.5 |z| roundings at most (what is below
// 2^-126 is flushed).  Two special-function instructions a value; a reciprocal shared
// by two values spares a quarter of them and costs more issue slots than it gives.
template <int NP>
__device__ __forceinline__ void gn_sigmoid(const F2 (&z)[NP], F2 (&s)[NP])
{
    constexpr float kL = -1.44269504f;
#pragma unroll
    for (int p = 0; p < NP; ++p) {
        const float2 t = un2(mul2(z[p], f2(kL, kL)));
        const float2 a = un2(add2(f2(ex2_ftz(t.x), ex2_ftz(t.y)), f2(1.f, 1.f)));
        s[p] = f2(rcp_ftz(a.x), rcp_ftz(a.y));
    }
}

template <int ACT, int NP>
__device__ __forceinline__ void gn_act(F2 (&z)[NP])
{
    if constexpr (ACT == FC_ACT_RELU) {
#pragma unroll
        for (int p = 0; p < NP; ++p) {
            const float2 v = un2(z[p]);
            z[p] = f2(v.x < 0.f ? 0.f : v.x, v.y < 0.f ? 0.f : v.y);  // keeps NaN
        }
    } else if constexpr (ACT == FC_ACT_SILU) {
        F2 s[NP];
        gn_sigmoid<NP>(z, s);
#pragma unroll
        for (int p = 0; p < NP; ++p) z[p] = mul2(z[p], s[p]);
    }
}

// (x - mean) rstd w + b > 0 where fp32 cannot tell (an error of z's size would be one of
// the gradient's): every step with its rounding error, good to 2^-44 of b.
__device__ __forceinline__ bool gn_positive(float x, float mean, float rstd, float w, float b)
{
    const float d = __fsub_rn(x, mean), t = __fsub_rn(d, x);
    const float dl = __fadd_rn(__fsub_rn(x, __fsub_rn(d, t)), __fsub_rn(-mean, t));
    const float k = __fmul_rn(rstd, w), kl = __fmaf_rn(rstd, w, -k);
    const float p = __fmul_rn(d, k);
    const float pl = __fadd_rn(__fmaf_rn(d, k, -p), __fmaf_rn(d, kl, __fmul_rn(dl, k)));
    const float s = __fadd_rn(p, b), u = __fsub_rn(s, p);
    const float sl = __fadd_rn(__fsub_rn(p, __fsub_rn(s, u)), __fsub_rn(b, u));
    return __fadd_rn(s, __fadd_rn(sl, pl)) > 0.f;
}

// Where a vector's values come from, for a second look at them.
struct GnSource {
    const void *x;              // the vector
    const float *mean, *rstd;   // of its first group, those of the next `stride` further
    int stride, off, cpg;       // off: of its first channel in the group
    const void *weight, *bias;
    int ptype, c;               // c: its first channel
};

// A bit for each element of a vector: z > 0 as in exact arithmetic.  Out of line: about
// one vector in 100,000 is looked at again.
template <class T, int NE>
static __device__ __noinline__ uint32_t gn_positive_bits(const GnSource s)
{
    uint32_t bits = 0;
#pragma unroll 1
    for (int e = 0; e < NE; ++e) {
        const int g = (s.off + e) / s.cpg * s.stride;
        float x;
        if constexpr (sizeof(T) == 4)
            x = static_cast<const float *>(s.x)[e];
        else if constexpr (__is_same(T, __half))
            x = __half2float(static_cast<const __half *>(s.x)[e]);
        else
            x = __bfloat162float(static_cast<const __nv_bfloat16 *>(s.x)[e]);
        bits |= (uint32_t)gn_positive(x, s.mean[g], s.rstd[g],
                                      gn_param<T>(s.weight, s.ptype, s.c + e, 1.f),
                                      gn_param<T>(s.bias, s.ptype, s.c + e, 0.f)) << e;
    }
    return bits;
}

// dy * act'(z), z = d rw + b with d = x - mean and rw = rstd w; source() says where the
// vector came from.
template <class T, int ACT, int NE, class Source>
__device__ __forceinline__ void gn_dz(const F2 (&dy)[(NE + 1) / 2], const F2 (&d)[(NE + 1) / 2],
                                      const F2 (&rw)[(NE + 1) / 2], const F2 (&b)[(NE + 1) / 2],
                                      F2 (&dz)[(NE + 1) / 2], Source source)
{
    constexpr int NP = (NE + 1) / 2;
    if constexpr (ACT == FC_ACT_NONE) {
#pragma unroll
        for (int p = 0; p < NP; ++p) dz[p] = dy[p];
    } else if constexpr (ACT == FC_ACT_RELU) {
        // z's error is below 5 roundings of b where d rw nearly cancels it; without b the
        // sign is exact
        float near = INFINITY;
        uint32_t bits = 0;
#pragma unroll
        for (int p = 0; p < NP; ++p) {
            const float2 z = un2(fma2(d[p], rw[p], b[p])), c = un2(b[p]);
            near = fminf(near, fminf(fmaf(fabsf(c.x), -0x1p-20f, fabsf(z.x)),
                                     fmaf(fabsf(c.y), -0x1p-20f, fabsf(z.y))));
            bits |= (z.x > 0.f ? 1u << 2 * p : 0u) | (z.y > 0.f ? 2u << 2 * p : 0u);
        }
        if (near < 0.f) bits = gn_positive_bits<T, NE>(source());
#pragma unroll
        for (int p = 0; p < NP; ++p) {
            const float2 y = un2(dy[p]);
            dz[p] = f2(bits & 1u << 2 * p ? y.x : 0.f, bits & 2u << 2 * p ? y.y : 0.f);
        }
    } else {
        F2 z[NP], s[NP];
#pragma unroll
        for (int p = 0; p < NP; ++p) z[p] = fma2(d[p], rw[p], b[p]);
        gn_sigmoid<NP>(z, s);
        // s (1 + z (1 - s))
#pragma unroll
        for (int p = 0; p < NP; ++p)
            dz[p] = mul2(mul2(dy[p], s[p]),
                         fma2(z[p], fma2(s[p], f2(-1.f, -1.f), f2(1.f, 1.f)), f2(1.f, 1.f)));
    }
}

// ---- a vector's groups --------------------------------------------------------------------
//
// ONE: every vector lies in one group.

// Calls f(j, first, last) for every group j that the vector touches, of which it has the
// elements [first, last); `off`: its first element's place in its group.
template <int NE, bool ONE, class F>
__device__ __forceinline__ void gn_pieces(int off, int cpg, F f)
{
    if constexpr (ONE) {
        f(0, 0, NE);
    } else {
        int first = 0, last = min(NE, cpg - off);
        for (int j = 0; first < NE; ++j) {
            f(j, first, last);
            first = last;
            last = min(NE, last + cpg);
        }
    }
}

template <int NE>
__device__ __forceinline__ float gn_element(const F2 (&f)[(NE + 1) / 2], int e)
{
    const float2 a = un2(f[e / 2]);
    return e & 1 ? a.y : a.x;
}

// Adds up elements [first, last) of a vector of values.
template <int NE, bool ONE>
__device__ __forceinline__ float gn_add(const F2 (&f)[(NE + 1) / 2], int first, int last)
{
    float x = 0.f;
#pragma unroll
    for (int e = 0; e < NE; ++e)
        if (ONE || (e >= first && e < last)) x += gn_element<NE>(f, e);
    return x;
}

// A group's value for each pair of the vector (ONE: the same for all).
template <int NE, bool ONE>
struct GnOf {
    static constexpr int NP = (NE + 1) / 2;
    F2 f[ONE ? 1 : NP];

    __device__ __forceinline__ F2 operator[](int p) const { return f[ONE ? 0 : p]; }
    template <class L>
    __device__ __forceinline__ void load(int g0, int off, int cpg, L value)
    {
        if constexpr (ONE) {
            const float v = value(g0);
            f[0] = f2(v, v);
        } else {
            float v[2 * NP] = {};
            int left = cpg - off, g = g0;
#pragma unroll
            for (int e = 0; e < NE; ++e) {
                v[e] = value(g);
                if (--left == 0 && e < NE - 1) {
                    ++g;
                    left = cpg;
                }
            }
#pragma unroll
            for (int p = 0; p < NP; ++p) f[p] = f2(v[2 * p], v[2 * p + 1]);
        }
    }
};

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
#define FC_GN_RUN 64  // rows between two fresh pivots, a multiple of any batch

// Rows whose loads a thread has in flight at a time: up to 64 bytes, of two tensors 32
// each.  A store of the row before, which may be to where the next is read from, holds a
// load up otherwise (4 x 45956 x 182 fp32 in 2 groups, backward: 339 us row by row, 147 now).
template <int AB, int TENSORS>
constexpr int gn_batch()
{
    return AB == 16 ? 4 / TENSORS : AB == 8 ? 8 / TENSORS : 8;
}

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
    constexpr int NE = V::NE, NP = V::NP, U = gn_batch<AB, 1>();
    __shared__ float sm[2][FC_GN_BLOCK * NE];
    wait_for_prior_grid();
    allow_dependent_launch();
    const GnPlace q = gn_place<NE>(tile, n.positions);
    const T *base = static_cast<const T *>(x.p) + q.n * x.ss + q.c0;
    const int64_t step = q.R * x.ld;
    F2 mean[NP], m2[NP];
#pragma unroll
    for (int p = 0; p < NP; ++p) mean[p] = m2[p] = f2(0.f, 0.f);
    float count = 0.f;
    if (q.on) {
        for (int64_t run = q.first + q.r; run < q.end; run += (int64_t)FC_GN_RUN * q.R) {
            F2 neg[NP], s[NP], ss[NP];
            float k = 0.f;
            const T *at = base + run * x.ld;
            int left = (int)min((int64_t)FC_GN_RUN, (q.end - run + q.R - 1) / q.R);
#pragma unroll
            for (int p = 0; p < NP; ++p) s[p] = ss[p] = f2(0.f, 0.f);
            V::get(*reinterpret_cast<const typename V::Raw *>(at), neg);
#pragma unroll
            for (int p = 0; p < NP; ++p) neg[p] = neg2(neg[p]);
            k = (float)left;
            for (; left > 0; left -= U, at += U * step) {
                typename V::Raw raw[U];
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (u < left)
                        raw[u] = *reinterpret_cast<const typename V::Raw *>(at + u * step);
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    if (u >= left) break;
                    F2 f[NP];
                    V::get(raw[u], f);
#pragma unroll
                    for (int p = 0; p < NP; ++p) {
                        const F2 d = add2(f[p], neg[p]);
                        s[p] = add2(s[p], d);
                        ss[p] = fma2(d, d, ss[p]);
                    }
                }
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

// Where the parts of a group are many, a first step joins them channel by channel into
// one set a sample, 8 threads a channel: a group's own threads alone took 40 us for 318
// parts of 268 channels.
#define FC_GN_ENTRIES 4096  // parts times channels of a group that its threads join alone

// Over the block's 8 warps, lane by lane.
static __device__ __forceinline__ float gn_sum_warps(float (&sm)[8][32], float v)
{
    const int c = threadIdx.x & 31;
    __syncthreads();
    sm[threadIdx.x >> 5][c] = v;
    __syncthreads();
    v = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) v += sm[k][c];
    return v;
}

// SQUARES: of means and sums of squares about them, else of two sums.  Sets of both values
// are `sets` apart in `in`, `samples` in `out`.
template <bool SQUARES>
__global__ void __launch_bounds__(256)
    k_gn_join_parts(const GnShape n, const int parts, const int64_t part_rows,
                    const float *__restrict__ in, const int64_t sets, float *__restrict__ out)
{
    __shared__ float sm[8][32];
    wait_for_prior_grid();
    allow_dependent_launch();
    const int64_t padded = (n.channels + 7) & ~7;
    const int strips = (n.channels + 31) / 32, r = threadIdx.x >> 5;
    const int64_t sample = blockIdx.x / strips;
    const int c = (int)(blockIdx.x - sample * strips) * 32 + (threadIdx.x & 31);
    const bool on = c < n.channels;
    const float *const from = in + sample * parts * padded + c;
    const float last = (float)(n.positions - (parts - 1) * part_rows);
    float u = 0.f, v = 0.f;
    if (on) {
#pragma unroll 4
        for (int p = r; p < parts; p += 8) {
            const float *const at = from + p * padded;
            if (SQUARES) {
                u = fmaf(p < parts - 1 ? (float)part_rows : last, __ldcg(at), u);
            } else {
                u += __ldcg(at);
                v += __ldcg(at + sets * padded);
            }
        }
    }
    u = gn_sum_warps(sm, u);
    if (SQUARES) {
        u /= (float)n.positions;
        if (on) {
#pragma unroll 4
            for (int p = r; p < parts; p += 8) {
                const float *const at = from + p * padded;
                const float d = __ldcg(at) - u;
                v += fmaf((p < parts - 1 ? (float)part_rows : last) * d, d,
                          __ldcg(at + sets * padded));
            }
        }
    }
    v = gn_sum_warps(sm, v);
    if (on && r == 0) {
        out[sample * padded + c] = u;
        out[(n.samples + sample) * padded + c] = v;
    }
}

inline cudaError_t gn_join_parts(bool squares, const GnShape &n, const GnTile &t, const float *in,
                                 int64_t sets, float *out, cudaStream_t s)
{
    const unsigned grid = (unsigned)(n.samples * ((n.channels + 31) / 32));
    return launch_after_prior(squares ? k_gn_join_parts<true> : k_gn_join_parts<false>, grid, 256, 0,
                              s, n, t.parts, t.rows, in, sets, out);
}

// Calls f(part, channel) for a thread's share of a group's parts and channels, TPG side by
// side.
template <int TPG, class F>
__device__ __forceinline__ void gn_entries(int lane, int parts, int cpg, F f)
{
    int p = lane / cpg, c = lane - p * cpg;
    const int dp = TPG / cpg, dc = TPG - dp * cpg;
#pragma unroll 4
    while (p < parts) {
        f(p, c);
        p += dp;
        c += dc;
        if (c >= cpg) {
            c -= cpg;
            ++p;
        }
    }
}

// Joins the parts and channels of every group: TPG threads a group and sample.
template <int TPG>
__global__ void __launch_bounds__(TPG > 256 ? TPG : 256)
    k_gn_finish(const GnShape n, const int parts, const int64_t part_rows,
                const float *__restrict__ in, const int64_t sets, const float eps,
                float *__restrict__ stat, float *mean_out, float *rstd_out)
{
    __shared__ float sm[TPG > 32 ? TPG / 32 : 1];
    wait_for_prior_grid();
    allow_dependent_launch();
    const int64_t at = (int64_t)blockIdx.x * (TPG < 256 ? 256 / TPG : 1) + threadIdx.x / TPG;
    if (at >= n.samples * n.groups) return;  // whole warps, or whole blocks
    const int lane = threadIdx.x % TPG, cpg = n.channels / n.groups;
    const int64_t sample = at / n.groups, padded = (n.channels + 7) & ~7;
    const int c0 = (int)(at - sample * n.groups) * cpg;
    const float total = (float)n.positions * (float)cpg;
    const float *const from = in + sample * parts * padded + c0;
    const float last = (float)(n.positions - (parts - 1) * part_rows);
    float s = 0.f;
    gn_entries<TPG>(lane, parts, cpg, [&](int p, int c) {
        s = fmaf(p < parts - 1 ? (float)part_rows : last, __ldcg(from + p * padded + c), s);
    });
    const float m = gn_team_sum<TPG>(s, sm) / total;
    float q = 0.f;
    gn_entries<TPG>(lane, parts, cpg, [&](int p, int c) {
        const float *const at = from + p * padded + c;
        const float d = __ldcg(at) - m;
        q += fmaf((p < parts - 1 ? (float)part_rows : last) * d, d, __ldcg(at + sets * padded));
    });
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
    constexpr int NE = V::NE, NP = V::NP, U = gn_batch<AB, 1>();
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
    const int64_t row = q.first + q.r, sx = q.R * a.x.ld, sy = q.R * a.y.ld;
    const T *x = static_cast<const T *>(a.x.p) + q.n * a.x.ss + row * a.x.ld + q.c0;
    T *y = static_cast<T *>(const_cast<void *>(a.y.p)) + q.n * a.y.ss + row * a.y.ld + q.c0;
    for (int64_t left = row < q.end ? (q.end - row + q.R - 1) / q.R : 0; left > 0;
         left -= U, x += U * sx, y += U * sy) {
        typename V::Raw raw[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (u < left) raw[u] = __ldcs(reinterpret_cast<const typename V::Raw *>(x + u * sx));
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (u >= left) break;
            F2 f[NP];
            V::get(raw[u], f);
#pragma unroll
            for (int p = 0; p < NP; ++p) f[p] = fma2(add2(f[p], m[p]), w[p], b[p]);
            gn_act<ACT, NP>(f);
            __stcs(reinterpret_cast<typename V::Raw *>(y + u * sy), V::put(f));
        }
    }
}

// What a thread of the backward pass holds of its vector's channels.  With d = x - mean,
// z = d (rstd w) + bias; sums of dz h are sums of dz d times rstd.
template <class T, int NE, bool ONE>
struct GnChannels {
    static constexpr int NP = (NE + 1) / 2;
    F2 b[NP], rw[NP];  // bias, rstd * weight
    GnOf<NE, ONE> mean, rstd;

    __device__ __forceinline__ void scale(const F2 (&w)[NP])
    {
#pragma unroll
        for (int p = 0; p < NP; ++p) rw[p] = mul2(rstd[p], w[p]);
    }
    // d and dz of a vector
    template <int ACT, class Source>
    __device__ __forceinline__ void at(const F2 (&x)[NP], const F2 (&dy)[NP], F2 (&d)[NP],
                                       F2 (&dz)[NP], Source source) const
    {
#pragma unroll
        for (int p = 0; p < NP; ++p) d[p] = add2(x[p], neg2(mean[p]));
        gn_dz<T, ACT, NE>(dy, d, rw, b, dz, source);
    }
};

// Blocks of an SM that the streaming backward pass's registers are held to.  A fourth is
// worth more than registers beyond 64 (190 x 1092 x 167 bf16: 163 us without it, 134 with;
// 10 x 11404 x 480: 151 and 137; against that 8 x 10830 x 304 fp32: 117 and 121), but not
// with the ReLU's call out of line (8 x 16427 x 384 bf16 at an odd pitch: three 233, four 274).
template <int AB, int ACT>
__host__ __device__ constexpr int gn_blocks_bwd()
{
    return AB == 16 ? 2 : ACT == FC_ACT_RELU ? 3 : 4;
}

// Per channel of a part: the sums of dz h and of dz.
template <class T, int AB, int ACT>
__global__ void __launch_bounds__(FC_GN_BLOCK, gn_blocks_bwd<AB, ACT>())
    k_gn_sums(const GnBackward a, const GnTile tile, float *__restrict__ out, const int64_t sets)
{
    using V = Gv<T, AB>;
    constexpr int NE = V::NE, NP = V::NP, U = gn_batch<AB, 2>();
    __shared__ float sm[2][FC_GN_BLOCK * NE];
    wait_for_prior_grid();
    allow_dependent_launch();
    const GnPlace q = gn_place<NE>(tile, a.n.positions);
    F2 sh[NP], s[NP];
#pragma unroll
    for (int p = 0; p < NP; ++p) sh[p] = s[p] = f2(0.f, 0.f);
    if (q.on) {
        GnChannels<T, NE, false> ch;
        const int cpg = a.n.channels / a.n.groups, g0 = q.c0 / cpg;
        const int64_t at = q.n * a.n.groups;
        F2 w[NP];
        gn_params<T, NE>(a.weight, a.ptype, q.c0, 1.f, w);
        gn_params<T, NE>(a.bias, a.ptype, q.c0, 0.f, ch.b);
        ch.mean.load(g0, q.c0 - g0 * cpg, cpg, [&](int g) { return __ldg(a.mean + at + g); });
        ch.rstd.load(g0, q.c0 - g0 * cpg, cpg, [&](int g) { return __ldg(a.rstd + at + g); });
        ch.scale(w);
        const int64_t row = q.first + q.r, sx = q.R * a.x.ld, sy = q.R * a.dy.ld;
        const T *x = static_cast<const T *>(a.x.p) + q.n * a.x.ss + row * a.x.ld + q.c0;
        const T *dy = static_cast<const T *>(a.dy.p) + q.n * a.dy.ss + row * a.dy.ld + q.c0;
        for (int64_t left = row < q.end ? (q.end - row + q.R - 1) / q.R : 0; left > 0;
             left -= U, x += U * sx, dy += U * sy) {
            typename V::Raw rx[U], ry[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (u < left) {
                    rx[u] = *reinterpret_cast<const typename V::Raw *>(x + u * sx);
                    ry[u] = *reinterpret_cast<const typename V::Raw *>(dy + u * sy);
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (u >= left) break;
                F2 f[NP], g[NP], h[NP], dz[NP];
                V::get(rx[u], f);
                V::get(ry[u], g);
                ch.template at<ACT>(f, g, h, dz, [&] {
                    return GnSource{x + u * sx, a.mean + at + g0, a.rstd + at + g0, 1,
                                    q.c0 - g0 * cpg, cpg, a.weight, a.bias, a.ptype, q.c0};
                });
#pragma unroll
                for (int p = 0; p < NP; ++p) {
                    sh[p] = fma2(dz[p], h[p], sh[p]);
                    s[p] = add2(s[p], dz[p]);
                }
            }
        }
#pragma unroll
        for (int p = 0; p < NP; ++p) sh[p] = mul2(sh[p], ch.rstd[p]);
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
__global__ void __launch_bounds__(TPG > 256 ? TPG : 256)
    k_gn_finish_sums(const GnBackward a, const int parts, const float *__restrict__ in,
                     const int64_t sets, float *__restrict__ stat)
{
    __shared__ float sm[TPG > 32 ? TPG / 32 : 1];
    wait_for_prior_grid();
    allow_dependent_launch();
    const GnShape &n = a.n;
    const int64_t at = (int64_t)blockIdx.x * (TPG < 256 ? 256 / TPG : 1) + threadIdx.x / TPG;
    if (at >= n.samples * n.groups) return;
    const int lane = threadIdx.x % TPG, cpg = n.channels / n.groups;
    const int64_t sample = at / n.groups, padded = (n.channels + 7) & ~7;
    const int c0 = (int)(at - sample * n.groups) * cpg;
    const float inv = 1.f / ((float)n.positions * (float)cpg);
    const float *const from = in + sample * parts * padded + c0;
    float s1 = 0.f, s2 = 0.f;
    gn_entries<TPG>(lane, parts, cpg, [&](int p, int c) {
        const float w = gn_param<T>(a.weight, a.ptype, c0 + c, 1.f);
        const float *const at = from + p * padded + c;
        s2 = fmaf(w, __ldcg(at), s2);
        s1 = fmaf(w, __ldcg(at + sets * padded), s1);
    });
    s1 = gn_team_sum<TPG>(s1, sm);
    s2 = gn_team_sum<TPG>(s2, sm);
    if (lane == 0) {
        stat[2 * at] = s1 * inv;
        stat[2 * at + 1] = s2 * inv;
    }
}

// dx = rstd w dz - rstd c1 - rstd^2 c2 d, c1 and c2 the means of q and of q h.
template <int NE, bool ONE>
struct GnSlope {
    GnOf<NE, ONE> k1, k2;  // -rstd c1, -rstd^2 c2
    static constexpr int NP = (NE + 1) / 2;

    __device__ __forceinline__ void scale(const GnOf<NE, ONE> &rstd)
    {
#pragma unroll
        for (int p = 0; p < (ONE ? 1 : NP); ++p) {
            k1.f[p] = mul2(k1.f[p], rstd.f[p]);
            k2.f[p] = mul2(k2.f[p], mul2(rstd.f[p], rstd.f[p]));
        }
    }
    __device__ __forceinline__ void dx(const F2 (&d)[NP], const F2 (&rw)[NP], F2 (&dz)[NP]) const
    {
#pragma unroll
        for (int p = 0; p < NP; ++p) dz[p] = fma2(dz[p], rw[p], fma2(d[p], k2[p], k1[p]));
    }
};

template <class T, int AB, int ACT>
__global__ void __launch_bounds__(FC_GN_BLOCK, gn_blocks_bwd<AB, ACT>())
    k_gn_apply_bwd(const GnBackward a, const GnTile tile, const float *__restrict__ stat)
{
    using V = Gv<T, AB>;
    constexpr int NE = V::NE, NP = V::NP, U = gn_batch<AB, 2>();
    wait_for_prior_grid();
    allow_dependent_launch();
    const GnPlace q = gn_place<NE>(tile, a.n.positions);
    if (!q.on) return;
    const int cpg = a.n.channels / a.n.groups, g0 = q.c0 / cpg, off = q.c0 - g0 * cpg;
    const int64_t at = q.n * a.n.groups;
    const float *st = stat + 2 * at;
    GnChannels<T, NE, false> ch;
    F2 w[NP];
    gn_params<T, NE>(a.weight, a.ptype, q.c0, 1.f, w);
    gn_params<T, NE>(a.bias, a.ptype, q.c0, 0.f, ch.b);
    ch.mean.load(g0, off, cpg, [&](int g) { return __ldg(a.mean + at + g); });
    ch.rstd.load(g0, off, cpg, [&](int g) { return __ldg(a.rstd + at + g); });
    ch.scale(w);
    GnSlope<NE, false> to;
    to.k1.load(g0, off, cpg, [&](int g) { return -__ldcg(st + 2 * g); });
    to.k2.load(g0, off, cpg, [&](int g) { return -__ldcg(st + 2 * g + 1); });
    to.scale(ch.rstd);
    const int64_t row = q.first + q.r, sx = q.R * a.x.ld, sy = q.R * a.dy.ld, sd = q.R * a.dx.ld;
    const T *x = static_cast<const T *>(a.x.p) + q.n * a.x.ss + row * a.x.ld + q.c0;
    const T *dy = static_cast<const T *>(a.dy.p) + q.n * a.dy.ss + row * a.dy.ld + q.c0;
    T *dx = static_cast<T *>(const_cast<void *>(a.dx.p)) + q.n * a.dx.ss + row * a.dx.ld + q.c0;
    for (int64_t left = row < q.end ? (q.end - row + q.R - 1) / q.R : 0; left > 0;
         left -= U, x += U * sx, dy += U * sy, dx += U * sd) {
        typename V::Raw rx[U], ry[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (u < left) {
                rx[u] = __ldcs(reinterpret_cast<const typename V::Raw *>(x + u * sx));
                ry[u] = __ldcs(reinterpret_cast<const typename V::Raw *>(dy + u * sy));
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (u >= left) break;
            F2 f[NP], g[NP], h[NP], dz[NP];
            V::get(rx[u], f);
            V::get(ry[u], g);
            ch.template at<ACT>(f, g, h, dz, [&] {
                return GnSource{x + u * sx, a.mean + at + g0, a.rstd + at + g0, 1, off, cpg,
                                a.weight, a.bias, a.ptype, q.c0};
            });
            to.dx(h, ch.rw, dz);
            __stcs(reinterpret_cast<typename V::Raw *>(dx + u * sd), V::put(dz));
        }
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

// The images from sample `first` on.
template <class T>
GnImages gn_from(const GnImages &i, int64_t first)
{
    return {static_cast<const T *>(i.p) + first * i.ss, i.ld, i.ss};
}

inline unsigned gn_grid(const GnShape &n, const GnTile &t)
{
    return (unsigned)(n.samples * t.parts * t.tiles);
}

}  // namespace fc
