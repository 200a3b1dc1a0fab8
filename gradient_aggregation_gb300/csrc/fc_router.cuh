// The router of a mixture of experts, for one element type T: softmax over the
// experts, the k largest, and what the balance loss needs; and its gradient.
//
// Experts are cut into groups of eight, a vector load or two.  LPR lanes of a warp
// share a row, each with one group (VPL groups where there are more than 256 experts),
// 32 / LPR rows side by side, so that a lane's experts stay the same from row to row
// and the sums of their probabilities stay in its registers.
//
// Choosing the k largest with the lanes of a row side by side would cost a reduction
// over the warp for each of them.  Instead the lanes leave the largest of every group in
// shared memory, and then each lane chooses for a row of its own: the largest of the
// groups' largest, that group's elements once more (from L1 or L2), the largest that is
// left of them; 32 rows at a time.  A row of 256 experts takes 147 instructions of a warp
// with k = 8 and 115 with k = 1.
//
// 131072 x 256 bf16, k = 8: 40 us forward, 36 backward (by warp reductions 148 and 68); the
// bytes alone take 11 and 22.  Bound by instructions and the wait for loads: they issue in
// 0.55 to 0.6 of the cycles.  64 x 256: 9 us, three trips to memory and a cluster's start.
#pragma once

#include <algorithm>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fc.h"
#include "fc_cluster.cuh"
#include "fc_internal.h"
#include "fc_pairs.cuh"
#include "fc_router.h"

namespace fc {

#define FC_ROUTER_FAR 16.f  // |lse| from which on the backward pass takes differences first
#define FC_ROUTER_APART 65536.f  // the largest logit's size from which on the forward pass does

constexpr float kRtLog2e = 1.44269504f;

// Eight elements of a row, loaded ahead of their use.  ALIGNED: E is whole 16-byte
// vectors and so is every row's start; what lies past E, or is not there, is -infinity.
template <class T, bool ALIGNED>
struct Rt8 {
    static constexpr bool kWord = ALIGNED && sizeof(T) == 2;
    uint4 q;
    F2 f[kWord ? 1 : 4];

    __device__ __forceinline__ void load(const T *row, int e0, int E, bool here)
    {
        if constexpr (kWord) {
            constexpr uint32_t none = __is_same(T, __half) ? 0xfc00fc00u : 0xff80ff80u;
            q = make_uint4(none, none, none, none);
            if (here && e0 < E) q = *reinterpret_cast<const uint4 *>(row + e0);
        } else if constexpr (ALIGNED) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float4 v = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
                if (here && e0 + 4 * h < E) v = *reinterpret_cast<const float4 *>(row + e0 + 4 * h);
                f[2 * h] = f2(v.x, v.y);
                f[2 * h + 1] = f2(v.z, v.w);
            }
        } else {
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                v[i] = -INFINITY;
                if (here && e0 + i < E) {
                    if constexpr (sizeof(T) == 4)
                        v[i] = row[e0 + i];
                    else if constexpr (__is_same(T, __half))
                        v[i] = __half2float(row[e0 + i]);
                    else
                        v[i] = __bfloat162float(row[e0 + i]);
                }
            }
#pragma unroll
            for (int p = 0; p < 4; ++p) f[p] = f2(v[2 * p], v[2 * p + 1]);
        }
    }
    __device__ __forceinline__ void get(F2 (&x)[4]) const
    {
        if constexpr (kWord) {
            x[0] = pair_of_word<T>(q.x);
            x[1] = pair_of_word<T>(q.y);
            x[2] = pair_of_word<T>(q.z);
            x[3] = pair_of_word<T>(q.w);
        } else {
#pragma unroll
            for (int p = 0; p < 4; ++p) x[p] = f[p];
        }
    }
};

template <class T, bool ALIGNED>
__device__ __forceinline__ void rt_store(T *row, int e0, int E, const F2 (&f)[4])
{
    if constexpr (ALIGNED && sizeof(T) == 2) {
        if (e0 < E) __stcs(reinterpret_cast<uint4 *>(row + e0), from_pairs<T>(f));
    } else if constexpr (ALIGNED) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float2 a = un2(f[2 * h]), b = un2(f[2 * h + 1]);
            if (e0 + 4 * h < E)
                __stcs(reinterpret_cast<float4 *>(row + e0 + 4 * h), make_float4(a.x, a.y, b.x, b.y));
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float2 a = un2(f[i / 2]);
            const float v = i & 1 ? a.y : a.x;
            if (e0 + i < E) {
                if constexpr (sizeof(T) == 4)
                    row[e0 + i] = v;
                else if constexpr (__is_same(T, __half))
                    row[e0 + i] = __float2half_rn(v);
                else
                    row[e0 + i] = __float2bfloat16_rn(v);
            }
        }
    }
}

// What a group leaves of its largest element: a word that is ordered by the element,
// then from the lowest group up, and that also says which of the eight are chosen
// already.  0: none is left that is more than -infinity (NaN counts as less).
template <class T>
struct RtWord {
    using type = uint32_t;
    // 16-bit values are the upper halves of words of fp32 (bf16), or as many of their bits
    static __device__ __forceinline__ uint32_t make(float x, int group, uint32_t taken)
    {
        if (!(x > -INFINITY)) return 0;
        uint32_t h;
        if constexpr (__is_same(T, __half))
            h = __half_as_ushort(__float2half_rn(x + 0.f));
        else
            h = __float_as_uint(x + 0.f) >> 16;
        h ^= h & 0x8000u ? 0xffffu : 0x8000u;
        return h << 16 | (uint32_t)(127 - group) << 8 | taken;
    }
    static __device__ __forceinline__ float value(uint32_t w)
    {
        uint32_t h = w >> 16;
        h ^= h & 0x8000u ? 0x8000u : 0xffffu;
        if constexpr (__is_same(T, __half))
            return __half2float(__ushort_as_half((unsigned short)h));
        else
            return __uint_as_float(h << 16);
    }
    static __device__ __forceinline__ int group(uint32_t w) { return 127 - (int)(w >> 8 & 127); }
    static __device__ __forceinline__ uint32_t taken(uint32_t w) { return w & 255; }
};

template <>
struct RtWord<float> {
    using type = unsigned long long;
    static __device__ __forceinline__ type make(float x, int group, uint32_t taken)
    {
        if (!(x > -INFINITY)) return 0;
        const uint32_t u = __float_as_uint(x + 0.f);
        const uint32_t key = u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
        return (type)key << 32 | (uint32_t)(127 - group) << 8 | taken;
    }
    static __device__ __forceinline__ float value(type w)
    {
        const uint32_t key = (uint32_t)(w >> 32);
        return __uint_as_float(key & 0x80000000u ? key ^ 0x80000000u : ~key);
    }
    static __device__ __forceinline__ int group(type w) { return 127 - (int)((uint32_t)w >> 8 & 127); }
    static __device__ __forceinline__ uint32_t taken(type w) { return (uint32_t)w & 255; }
};

// Words of a row in shared memory: whole 16-byte vectors, an odd number of them, so that
// 32 lanes with a row each read theirs without a conflict.
template <class T>
__host__ __device__ constexpr int rt_stride(int groups)
{
    constexpr int per = 16 / (int)sizeof(typename RtWord<T>::type);
    const int vecs = (groups + per - 1) / per;
    return (vecs | 1) * per;
}

// A warp's shared memory: the words of `rows` rows, two numbers a row, and the chosen
// experts and their weights.
template <class T>
__host__ __device__ constexpr int rt_warp_bytes(int groups, int rows, int k)
{
    return (rt_stride<T>(groups) * (int)sizeof(typename RtWord<T>::type) * rows + 8 * rows +
            8 * rows * k + 15) / 16 * 16;
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
    w.done = reinterpret_cast<unsigned *>(w.share + 2 * groups * ((e + 7) / 8));
    return w;
}

// Sum over the LPR lanes of a row.
template <int LPR>
__device__ __forceinline__ float rt_row_sum(float x)
{
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// The sums of U values, each over the LPR lanes of its rows.  Two sums take a shuffle
// for each step of one, and one more.
template <int LPR, int U>
__device__ __forceinline__ void rt_row_sums(float (&x)[U])
{
    if constexpr (LPR >= 4 && U == 2) {
        const bool high = threadIdx.x & (LPR / 2);
        float a = high ? x[1] : x[0];
        a += __shfl_xor_sync(0xffffffffu, high ? x[0] : x[1], LPR / 2);
        a = rt_row_sum<LPR / 2>(a);
        const float b = __shfl_xor_sync(0xffffffffu, a, LPR / 2);
        x[0] = high ? b : a;
        x[1] = high ? a : b;
    } else {
#pragma unroll
        for (int u = 0; u < U; ++u) x[u] = rt_row_sum<LPR>(x[u]);
    }
}

template <int LPR>
__device__ __forceinline__ float rt_row_max(float x)
{
    if constexpr (LPR == 32) {
        float y;
        asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
        return y;
    }
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
    return x;
}

// Rows of a lane at a time.
template <int LPR, int VPL>
__host__ __device__ constexpr int rt_rows()
{
    return LPR < 8 ? 1 : VPL <= 2 ? 2 : 1;
}

// Blocks of an SM that the registers leave room for: loads in flight matter more than
// their number in one warp (256 bf16 experts: 64 registers and two rows of a lane at a
// time 39 us, 124 and four 45).
template <class T, int VPL>
__host__ __device__ constexpr int rt_blocks()
{
    return VPL > 1 ? 4 : sizeof(T) == 2 ? 7 : 5;
}

template <class T, int LPR, int VPL, bool ALIGNED>
__global__ void __launch_bounds__(32 * FC_ROUTER_WARPS, rt_blocks<T, VPL>())
    k_router_fwd(const __grid_constant__ RouterForward a, const __grid_constant__ RouterCut cut)
{
    using Word = typename RtWord<T>::type;
    constexpr int RPI = 32 / LPR;  // rows side by side
    constexpr int U = rt_rows<LPR, VPL>();
    extern __shared__ uint4 dyn[];
    __shared__ float s_z[FC_ROUTER_WARPS];
    __shared__ int s_n[FC_ROUTER_WARPS];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = cut.warps;
    const int E = a.n.experts, k = a.n.k, G = (E + 7) / 8;
    constexpr int NG = LPR * VPL, stride = rt_stride<T>(NG);  // groups, with those past E
    // the block's counts and, at the end, its sums; then each warp's own
    int *const s_counts = reinterpret_cast<int *>(dyn);
    char *const own = reinterpret_cast<char *>(s_counts + (E + 3) / 4 * 4) +
                      (size_t)warp * rt_warp_bytes<T>(NG, cut.rows, k);
    Word *const words = reinterpret_cast<Word *>(own);
    float2 *const stats = reinterpret_cast<float2 *>(words + stride * cut.rows);
    int *const chosen = reinterpret_cast<int *>(stats + cut.rows);
    float *const weights = reinterpret_cast<float *>(chosen + cut.rows * k);
    const int64_t group = blockIdx.x / (unsigned)cut.parts;
    const int part = (int)(blockIdx.x - group * cut.parts);
    const int64_t per = a.n.sequences * a.n.tokens / a.n.groups;  // rows of a group
    const RouterWs ws = router_ws(a.ws, a.n.groups, cut.parts, E);
    for (int e = threadIdx.x; e < E; e += 32 * warps) s_counts[e] = 0;
    if (NG % 4)  // the vectors that end behind a row's words
        for (int i = lane; i < stride * cut.rows; i += 32) words[i] = 0;
    const int q = lane % LPR, sub = lane / LPR;  // of the row, of the rows side by side
    F2 sum[VPL][4];
#pragma unroll
    for (int v = 0; v < VPL; ++v)
#pragma unroll
        for (int p = 0; p < 4; ++p) sum[v][p] = f2(0.f, 0.f);
    float zsum = 0.f;
    int routed = 0;
    wait_for_prior_grid();
    allow_dependent_launch();
    if (blockIdx.x == 0 && threadIdx.x == 0) *ws.done = 0;
    __syncthreads();
    const T *const logits = static_cast<const T *>(a.logits);
    const int64_t tile0 = ((int64_t)part * warps + warp) * cut.rows;
    for (int64_t at = tile0; at < per; at += (int64_t)cut.parts * warps * cut.rows) {
        const int64_t row0 = group * per + at;
        const int rows = (int)(per - at < cut.rows ? per - at : cut.rows);
        // which of the tile's rows are there
        bool there = lane < rows;
        if (there && a.lengths) {
            const int64_t row = row0 + lane, seq = row / a.n.tokens;
            there = row - seq * a.n.tokens < __ldg(a.lengths + seq);
        }
        const unsigned present = __ballot_sync(0xffffffffu, there);
        // the softmax, U rows of a lane at a time.  WHOLE: all of them are there
        auto softmax = [&](int r0, auto whole) {
            constexpr bool WHOLE = decltype(whole)::value;
            Rt8<T, ALIGNED> raw[U][VPL];
            const T *from = logits + (row0 + r0 + sub) * a.ld;
#pragma unroll
            for (int u = 0; u < U; ++u, from += RPI * a.ld)
#pragma unroll
                for (int v = 0; v < VPL; ++v) {
                    const int r = r0 + u * RPI + sub;
                    raw[u][v].load(from, 8 * (q + LPR * v), E,
                                   WHOLE || (r < rows && present >> r & 1));
                }
            F2 x[U][VPL][4];
            float top[U], total[U];
            bool odd = false;
            Word *to = words + (r0 + sub) * stride + q;
#pragma unroll
            for (int u = 0; u < U; ++u, to += RPI * stride) {
                const int r = r0 + u * RPI + sub;
                top[u] = -INFINITY;
#pragma unroll
                for (int v = 0; v < VPL; ++v) {
                    raw[u][v].get(x[u][v]);
                    float most = -INFINITY;
#pragma unroll
                    for (int p = 0; p < 4; ++p) {
                        const float2 e = un2(x[u][v][p]);
                        most = fmaxf(most, fmaxf(e.x, e.y));
                    }
                    top[u] = fmaxf(top[u], most);
                    if (WHOLE || r < rows)
                        to[LPR * v] = RtWord<T>::make(most, q + LPR * v, 0);
                }
                top[u] = rt_row_max<LPR>(top[u]);
                odd |= !(fabsf(top[u]) < FC_ROUTER_APART);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                // one shift for all of a row: its rounding, of 2^-8 at most here, is a factor of all
                // terms and leaves their quotients (the chosen ones' terms are formed with it
                // as well, below), and of the lse it is a rounding
                const float shift = -top[u] * kRtLog2e;
                F2 acc = f2(0.f, 0.f);
#pragma unroll
                for (int v = 0; v < VPL; ++v)
#pragma unroll
                    for (int p = 0; p < 4; ++p) {
                        const float2 e = un2(fma2(x[u][v][p], f2(kRtLog2e, kRtLog2e),
                                                  f2(shift, shift)));
                        x[u][v][p] = f2(ex2_ftz(e.x), ex2_ftz(e.y));
                        acc = add2(acc, x[u][v][p]);
                    }
                const float2 both = un2(acc);
                total[u] = both.x + both.y;
            }
            unsigned routes = WHOLE ? ~0u : 0u;  // a bit for each u
            if (!WHOLE) {
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int r = r0 + u * RPI + sub;
                    routes |= (unsigned)(r < rows && present >> r & 1) << u;
                }
            }
            if (__any_sync(0xffffffffu, odd)) {
                // rows closed to all experts, or with numbers whose shift would be rounded by
                // more (a factor that fp32 may not hold): those once more, the difference first
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const bool live = routes >> u & 1, closed = !(top[u] > -INFINITY);
                    const bool again = !(fabsf(top[u]) < FC_ROUTER_APART);  // the others keep their bits
                    bool nan = false;
                    F2 acc = f2(0.f, 0.f);
#pragma unroll
                    for (int v = 0; v < VPL; ++v) {
                        F2 y[4];
                        raw[u][v].get(y);
#pragma unroll
                        for (int p = 0; p < 4; ++p) {
                            const F2 d = add2(y[p], f2(-top[u], -top[u]));
                            const float2 e = un2(mul2(d, f2(kRtLog2e, kRtLog2e)));
                            const float2 w = un2(y[p]);
                            nan |= w.x != w.x || w.y != w.y;
                            const F2 o = f2(ex2_ftz(e.x), ex2_ftz(e.y));
                            if (again) x[u][v][p] = o;
                            acc = add2(acc, o);
                        }
                    }
                    const float2 both = un2(acc);
                    if (again) total[u] = both.x + both.y;
                    // of the row's own lanes: nothing but NaN makes no closed row
                    const unsigned votes = __ballot_sync(0xffffffffu, nan);
                    const unsigned own_lanes = (LPR == 32 ? ~0u : (1u << (LPR & 31)) - 1u) << (sub * LPR);
                    if (!live || (closed && !(votes & own_lanes))) routes &= ~(1u << u);
                }
            }
            rt_row_sums<LPR, U>(total);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int r = r0 + u * RPI + sub;
                const float inv = rcp_ftz(total[u]);
                const bool on = routes >> u & 1;
                if (on) {
#pragma unroll
                    for (int v = 0; v < VPL; ++v)
#pragma unroll
                        for (int p = 0; p < 4; ++p)
                            sum[v][p] = fma2(x[u][v][p], f2(inv, inv), sum[v][p]);
                }
                if (q == 0 && (WHOLE || r < rows)) stats[r] = make_float2(top[u], on ? total[u] : -1.f);
            }
        };
        if (rows % (RPI * U) == 0 && present == (rows == 32 ? ~0u : (1u << rows) - 1u)) {
            for (int r0 = 0; r0 < rows; r0 += RPI * U) softmax(r0, Yes<true>());
        } else {
            for (int r0 = 0; r0 < rows; r0 += RPI * U) softmax(r0, Yes<false>());
        }
        __syncwarp();
        // the choice, a lane a row
        if (lane < rows) {
            const float2 st = stats[lane];
            const T *const row = logits + (row0 + lane) * a.ld;
            Word *const mine = words + lane * stride;
            const bool routes = !(st.y < 0.f);
            const float scale = 1.f / st.y;
            // a term as the row's total has it, bit for bit: ex2(x log2e + shift), or from the
            // difference (value - 0 and + 0 round nothing)
            const bool apart = !(fabsf(st.x) < FC_ROUTER_APART);
            const float less = apart ? st.x : 0.f, shift = apart ? 0.f : -st.x * kRtLog2e;
            float chosen_sum = 0.f;
            int j = 0;
            if (routes) {
                for (; j < k; ++j) {
                    Word most = 0;
                    if constexpr (sizeof(Word) == 4) {
                        const uint4 *const w4 = reinterpret_cast<const uint4 *>(mine);
                        uint4 m = w4[0];
#pragma unroll
                        for (int g = 1; g < (NG + 3) / 4; ++g) {
                            const uint4 w = w4[g];
                            m.x = max(m.x, w.x);
                            m.y = max(m.y, w.y);
                            m.z = max(m.z, w.z);
                            m.w = max(m.w, w.w);
                        }
                        most = max(max(m.x, m.y), max(m.z, m.w));
                    } else {
                        const ulonglong2 *const w2 = reinterpret_cast<const ulonglong2 *>(mine);
                        ulonglong2 m = w2[0];
#pragma unroll
                        for (int g = 1; g < (NG + 1) / 2; ++g) {
                            const ulonglong2 w = w2[g];
                            m.x = max(m.x, w.x);
                            m.y = max(m.y, w.y);
                        }
                        most = max(m.x, m.y);
                    }
                    if (most == 0) break;
                    const int g = RtWord<T>::group(most);
                    const uint32_t taken = RtWord<T>::taken(most);
                    const float value = RtWord<T>::value(most);
                    Rt8<T, ALIGNED> raw;
                    F2 f[4];
                    raw.load(row, 8 * g, E, true);
                    raw.get(f);
                    // the first of its equals that is not chosen yet, and what then is the
                    // group's largest: an equal, or the largest below
                    uint32_t same = 0;
                    float below[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float2 e = un2(f[i / 2]);
                        const float x = i & 1 ? e.y : e.x;
                        if (x == value) same |= 1u << i;
                        below[i] = x < value ? x : -INFINITY;
                    }
#pragma unroll
                    for (int o = 4; o > 0; o >>= 1)
#pragma unroll
                        for (int i = 0; i < o; ++i) below[i] = fmaxf(below[i], below[i + o]);
                    const float left = below[0];
                    same &= ~taken;
                    const int at_e = __ffs(same) - 1;
                    const bool again = same & (same - 1);
                    mine[g] = RtWord<T>::make(again ? value : left, g,
                                              again ? taken | 1u << at_e : 0);
                    const float p = ex2_ftz(fmaf(value - less, kRtLog2e, shift));
                    chosen_sum += p;
                    chosen[lane * k + j] = 8 * g + at_e;
                    weights[lane * k + j] = p;
                    atomicAdd(&s_counts[8 * g + at_e], 1);
                }
                const float lse = st.x + logf(st.y);
                zsum = fmaf(lse, lse, zsum);
                ++routed;
                a.lse[row0 + lane] = lse;
                // a row with a NaN has a total of NaN, and so weights of NaN
                const float by = a.n.normalise ? 1.f / fmaf(0.f, st.y, chosen_sum) : scale;
                for (int i = 0; i < j; ++i) weights[lane * k + i] *= by;
            } else {
                a.lse[row0 + lane] = -INFINITY;
            }
            for (; j < k; ++j) {
                chosen[lane * k + j] = -1;
                weights[lane * k + j] = 0.f;
            }
        }
        __syncwarp();
        for (int i = lane; i < rows * k; i += 32) {
            __stcs(a.chosen + row0 * k + i, chosen[i]);
            __stcs(a.weights + row0 * k + i, weights[i]);
        }
        __syncwarp();
    }
    // over the rows side by side, then over the warps
#pragma unroll
    for (int o = LPR; o < 32; o <<= 1)
#pragma unroll
        for (int v = 0; v < VPL; ++v)
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                const float2 e = un2(sum[v][p]);
                sum[v][p] = add2(sum[v][p], f2(__shfl_xor_sync(0xffffffffu, e.x, o),
                                               __shfl_xor_sync(0xffffffffu, e.y, o)));
            }
    zsum = warp_sum_f32(zsum);
    routed = __reduce_add_sync(0xffffffffu, routed);
    __syncthreads();
    float *const s_probs = reinterpret_cast<float *>(s_counts + (E + 3) / 4 * 4);
    const int width = G * 8;
    if (sub == 0) {
#pragma unroll
        for (int v = 0; v < VPL; ++v) {
            const int g = q + LPR * v;
            if (g < G) {
#pragma unroll
                for (int p = 0; p < 4; ++p) {
                    const float2 e = un2(sum[v][p]);
                    s_probs[warp * width + 8 * g + 2 * p] = e.x;
                    s_probs[warp * width + 8 * g + 2 * p + 1] = e.y;
                }
            }
        }
    }
    if (lane == 0) {
        s_z[warp] = zsum;
        s_n[warp] = routed;
    }
    __syncthreads();
    float z = 0.f;
    int n = 0;
    for (int w = 0; w < warps; ++w) {
        z += s_z[w];
        n += s_n[w];
    }
    // the block's sums by expert, in place of the first warp's
    for (int e = threadIdx.x; e < E; e += 32 * warps) {
        float v = 0.f;
        for (int w = 0; w < warps; ++w) v += s_probs[w * width + e];
        s_probs[e] = v;
    }
    if (cut.joins) {
        // few blocks: one cluster, which holds all there is
        __shared__ float s_b[FC_ROUTER_WARPS];
        __shared__ float2 s_all;
        if (threadIdx.x == 0) s_all = make_float2(z, (float)n);
        if (gridDim.x > 1)
            cluster_sync();
        else
            __syncthreads();
        // the blocks share the experts; the first adds the losses
        __shared__ float2 s_share;
        float b = 0.f, zs = 0.f;
        for (int64_t g = 0; g < a.n.groups; ++g) {
            int gn = 0;
            float gz = 0.f;
            for (int i = 0; i < cut.parts; ++i) {
                const uint32_t from = (uint32_t)(g * cut.parts + i);
                gz += ld_cluster_f32(&s_all.x, from);
                gn += (int)ld_cluster_f32(&s_all.y, from);
            }
            const float each = 1.f / (float)max(gn, 1);
            for (int e = blockIdx.x * 32 * warps + threadIdx.x; e < E; e += gridDim.x * 32 * warps) {
                float p = 0.f;
                int c = 0;
#pragma unroll 4
                for (int i = 0; i < cut.parts; ++i) {
                    const uint32_t from = (uint32_t)(g * cut.parts + i);
                    p += ld_cluster_f32(s_probs + e, from);
                    c += __float_as_int(ld_cluster_f32(reinterpret_cast<float *>(s_counts) + e, from));
                }
                p *= each;
                a.probs[g * E + e] = p;
                a.counts[g * E + e] = c;
                b = fmaf((float)c * p, each, b);
            }
            zs += gz * each;
            if (blockIdx.x == 0 && threadIdx.x == 0) a.routed[g] = gn;
        }
        b = warp_sum_f32(b);
        if (lane == 0) s_b[warp] = b;
        __syncthreads();
        if (threadIdx.x == 0) {
            b = 0.f;
            for (int w = 0; w < warps; ++w) b += s_b[w];
            s_share = make_float2(b, zs);
        }
        if (gridDim.x > 1)
            cluster_sync();
        else
            __syncthreads();
        if (blockIdx.x == 0 && threadIdx.x == 0) {
            b = 0.f;
            for (uint32_t i = 0; i < gridDim.x; ++i) b += ld_cluster_f32(&s_share.x, i);
            a.loss[0] = b * ((float)E / (float)k) / (float)a.n.groups;
            a.loss[1] = zs / (float)a.n.groups;
        }
        if (gridDim.x > 1) cluster_sync();  // no block leaves while another reads its sums
        return;
    }
    const int64_t out = (group * cut.parts + part) * E;
    for (int e = threadIdx.x; e < E; e += 32 * warps) {
        ws.probs[out + e] = s_probs[e];
        ws.counts[out + e] = s_counts[e];
    }
    if (threadIdx.x == 0) {
        ws.z[group * cut.parts + part] = z;
        ws.routed[group * cut.parts + part] = n;
    }
}

// A warp's shared memory in the backward pass: lse and the weights' common part of each
// row, the chosen experts and what their weights add, and U * 256 * VPL sums by expert.
__host__ __device__ constexpr int rt_warp_bytes_bwd(int rows, int k, int adds)
{
    return (8 * rows + 8 * rows * k + 15) / 16 * 16 + 4 * adds;
}

// Backward: with c_e the derivative of the balance loss by every probability of
// expert e in the row's group,
//   dlogits_e = p_e (c_e - sum_j p_j c_j + 2 dz lse / (groups n)) + the weights' part
template <class T, int LPR, int VPL, bool ALIGNED>
__global__ void __launch_bounds__(32 * FC_ROUTER_WARPS, rt_blocks<T, VPL>())
    k_router_bwd(const __grid_constant__ RouterBackward a, const __grid_constant__ RouterCut cut)
{
    constexpr int RPI = 32 / LPR;
    constexpr int U = rt_rows<LPR, VPL>();
    extern __shared__ uint4 dyn[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = cut.warps;
    const int E = a.n.experts, k = a.n.k;
    const int q = lane % LPR, sub = lane / LPR;
    char *const own = reinterpret_cast<char *>(dyn) +
                      (size_t)warp * rt_warp_bytes_bwd(cut.rows, k, U * 256 * VPL);
    // what the weights add to the experts of the U * RPI rows at hand
    float *const add = reinterpret_cast<float *>(own);
    float2 *const stats = reinterpret_cast<float2 *>(add + U * 256 * VPL);
    int *const chosen = reinterpret_cast<int *>(stats + cut.rows);
    float *const value = reinterpret_cast<float *>(chosen + cut.rows * k);
    for (int i = lane; i < U * 256 * VPL; i += 32) add[i] = 0.f;
    const int64_t group = blockIdx.x / (unsigned)cut.parts;
    const int part = (int)(blockIdx.x - group * cut.parts);
    const int64_t per = a.n.sequences * a.n.tokens / a.n.groups;
    wait_for_prior_grid();
    allow_dependent_launch();
    const float n = a.dloss ? (float)max(__ldg(a.routed + group), 1) : 1.f;
    const float each = 1.f / (n * (float)a.n.groups);
    const float d0 = a.dloss ? __ldg(a.dloss) : 0.f, d1 = a.dloss ? __ldg(a.dloss + 1) : 0.f;
    const float scale = d0 * ((float)E / (float)k) * each / n;
    const int logk = 31 - __clz(k);
    F2 c[VPL][4];
#pragma unroll
    for (int v = 0; v < VPL; ++v)
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            const int e = 8 * (q + LPR * v) + 2 * p;
            c[v][p] = f2(a.dloss && e < E ? scale * (float)__ldg(a.counts + group * E + e) : 0.f,
                         a.dloss && e + 1 < E ? scale * (float)__ldg(a.counts + group * E + e + 1) : 0.f);
        }
    const T *const logits = static_cast<const T *>(a.logits);
    T *const dlogits = static_cast<T *>(a.dlogits);
    const int64_t tile0 = ((int64_t)part * warps + warp) * cut.rows;
    for (int64_t at = tile0; at < per; at += (int64_t)cut.parts * warps * cut.rows) {
        const int64_t row0 = group * per + at;
        const int rows = (int)(per - at < cut.rows ? per - at : cut.rows);
        // a lane a row: its lse, and what the weights' gradients come to
        const float my_lse = lane < rows ? __ldg(a.lse + row0 + lane) : -INFINITY;
        const unsigned live_rows = __ballot_sync(0xffffffffu, my_lse != -INFINITY);
        if (lane < rows)
            stats[lane] = make_float2(my_lse, my_lse != -INFINITY ? 2.f * d1 * my_lse * each : 0.f);
        __syncwarp();
        if (a.dweights) {
            const int all = rows * k;
            if (!(k & (k - 1))) {
                // k lanes side by side have a row's entries
                for (int i0 = 0; i0 < all; i0 += 32) {
                    const int i = i0 + lane;
                    int e = -1;
                    float w = 0.f, dw = 0.f;
                    if (i < all) {
                        e = __ldg(a.chosen + row0 * k + i);
                        w = __ldg(a.weights + row0 * k + i);
                        dw = __ldg(a.dweights + row0 * k + i);
                        if ((unsigned)e >= (unsigned)E || !(live_rows >> (i >> logk) & 1)) {
                            e = -1;
                            w = dw = 0.f;
                        }
                    }
                    float inner = w * dw;
                    for (int o = k >> 1; o > 0; o >>= 1)
                        inner += __shfl_xor_sync(0xffffffffu, inner, o);
                    if (i < all) {
                        chosen[i] = e;
                        value[i] = w * (a.n.normalise ? dw - inner : dw);
                        if (!a.n.normalise && !(i & (k - 1))) stats[i >> logk].y -= inner;
                    }
                }
            } else {
                for (int i = lane; i < all; i += 32) {
                    const int e = __ldg(a.chosen + row0 * k + i);
                    const bool ok = (unsigned)e < (unsigned)E;
                    chosen[i] = ok ? e : -1;
                    value[i] = ok ? __ldg(a.weights + row0 * k + i) : 0.f;
                }
                __syncwarp();
                if (lane < rows && my_lse != -INFINITY) {
                    const float *const dw = a.dweights + (row0 + lane) * k;
                    float inner = 0.f;
                    for (int j = 0; j < k; ++j)
                        if (chosen[lane * k + j] >= 0)
                            inner = fmaf(value[lane * k + j], __ldg(dw + j), inner);
                    for (int j = 0; j < k; ++j)
                        if (chosen[lane * k + j] >= 0)
                            value[lane * k + j] *= a.n.normalise ? __ldg(dw + j) - inner : __ldg(dw + j);
                    if (!a.n.normalise) stats[lane].y -= inner;
                }
            }
            __syncwarp();
        }
        // U rows of a lane at a time.  WHOLE: all of them are there
        auto gradient = [&](int r0, auto whole) {
            constexpr bool WHOLE = decltype(whole)::value;
            Rt8<T, ALIGNED> raw[U][VPL];
            const T *from = logits + (row0 + r0 + sub) * a.ld;
            T *to = dlogits + (row0 + r0 + sub) * a.lddl;
#pragma unroll
            for (int u = 0; u < U; ++u, from += RPI * a.ld)
#pragma unroll
                for (int v = 0; v < VPL; ++v) {
                    const int r = r0 + u * RPI + sub;
                    raw[u][v].load(from, 8 * (q + LPR * v), E,
                                   WHOLE || (r < rows && live_rows >> r & 1));
                }
            // the entries of rows r0 .. are next to one another, as are the rows' sums
            const int entries = min(RPI * U, rows - r0) * k;
            auto scatter = [&](bool clear) {
                for (int i = lane; i < entries; i += 32) {
                    const int e = chosen[r0 * k + i];
                    const int r = k & (k - 1) ? i / k : i >> logk;
                    if (e >= 0)
                        add[r * (LPR * VPL * 8) + (e >> 2 & 1) * (LPR * VPL * 4) + (e >> 3) * 4 +
                            (e & 3)] = clear ? 0.f : value[r0 * k + i];
                }
                __syncwarp();
            };
            if (a.dweights) scatter(false);
            F2 x[U][VPL][4];
            float inner[U];
            float2 st[U];
            bool far = false;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int r = r0 + u * RPI + sub;
                st[u] = make_float2(0.f, 0.f);
                if (WHOLE || (r < rows && live_rows >> r & 1)) st[u] = stats[r];
                far |= fabsf(st[u].x) > FC_ROUTER_FAR;
                const float shift = -st[u].x * kRtLog2e;
                F2 acc = f2(0.f, 0.f);
#pragma unroll
                for (int v = 0; v < VPL; ++v) {
                    raw[u][v].get(x[u][v]);
#pragma unroll
                    for (int p = 0; p < 4; ++p) {
                        const float2 e = un2(fma2(x[u][v][p], f2(kRtLog2e, kRtLog2e),
                                                  f2(shift, shift)));
                        x[u][v][p] = f2(ex2_ftz(e.x), ex2_ftz(e.y));
                        acc = fma2(x[u][v][p], c[v][p], acc);
                    }
                }
                const float2 both = un2(acc);
                inner[u] = both.x + both.y;
            }
            if (__any_sync(0xffffffffu, far)) {
                // lse's own rounding is |lse| units of a probability: the differences first,
                // and added up again
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const bool again = fabsf(st[u].x) > FC_ROUTER_FAR;  // the others keep their bits
                    F2 all = f2(0.f, 0.f), acc = f2(0.f, 0.f), y[VPL][4];
#pragma unroll
                    for (int v = 0; v < VPL; ++v) {
                        raw[u][v].get(y[v]);
#pragma unroll
                        for (int p = 0; p < 4; ++p) {
                            const F2 d = add2(y[v][p], f2(-st[u].x, -st[u].x));
                            const float2 e = un2(mul2(d, f2(kRtLog2e, kRtLog2e)));
                            y[v][p] = f2(ex2_ftz(e.x), ex2_ftz(e.y));
                            all = add2(all, y[v][p]);
                            acc = fma2(y[v][p], c[v][p], acc);
                        }
                    }
                    const float2 t = un2(all), both = un2(acc);
                    const float inv = 1.f / rt_row_sum<LPR>(t.x + t.y);
                    if (again) {
                        inner[u] = (both.x + both.y) * inv;
#pragma unroll
                        for (int v = 0; v < VPL; ++v)
#pragma unroll
                            for (int p = 0; p < 4; ++p) x[u][v][p] = mul2(y[v][p], f2(inv, inv));
                    }
                }
            }
            rt_row_sums<LPR, U>(inner);
            // a row's sums: the first halves of all groups, then the second ones
            const float *plus = add + sub * (LPR * VPL * 8) + 4 * q;
#pragma unroll
            for (int u = 0; u < U; ++u, to += RPI * a.lddl, plus += RPI * LPR * VPL * 8) {
                const int r = r0 + u * RPI + sub;
                const bool here = WHOLE || r < rows, live = WHOLE || (here && live_rows >> r & 1);
                const float less = st[u].y - inner[u];
#pragma unroll
                for (int v = 0; v < VPL; ++v) {
                    const float4 u0 = *reinterpret_cast<const float4 *>(plus + 4 * LPR * v);
                    const float4 u1 = *reinterpret_cast<const float4 *>(plus + 4 * LPR * (v + VPL));
                    const F2 w[4] = {f2(u0.x, u0.y), f2(u0.z, u0.w), f2(u1.x, u1.y), f2(u1.z, u1.w)};
#pragma unroll
                    for (int p = 0; p < 4; ++p) {
                        x[u][v][p] = fma2(x[u][v][p], add2(c[v][p], f2(less, less)), w[p]);
                        if (!live) x[u][v][p] = f2(0.f, 0.f);
                    }
                    if (here) rt_store<T, ALIGNED>(to, 8 * (q + LPR * v), E, x[u][v]);
                }
            }
            if (a.dweights) {
                __syncwarp();
                scatter(true);
            }
        };
        if (rows % (RPI * U) == 0 && live_rows == (rows == 32 ? ~0u : (1u << rows) - 1u)) {
            for (int r0 = 0; r0 < rows; r0 += RPI * U) gradient(r0, Yes<true>());
        } else {
            for (int r0 = 0; r0 < rows; r0 += RPI * U) gradient(r0, Yes<false>());
        }
        __syncwarp();
    }
}

// ---- host ------------------------------------------------------------------------------------

// Raises the kernel's limit of shared memory, once a kernel and device.
cudaError_t router_allow(const void *kernel);

template <class T, int LPR, int VPL, bool ALIGNED>
cudaError_t router_forward_one(const RouterForward &a, bool *joins, int *parts, cudaStream_t s)
{
    auto *const kernel = k_router_fwd<T, LPR, VPL, ALIGNED>;
    const int E = a.n.experts, G = (E + 7) / 8;
    auto bytes = [&](int warps, int rows) {
        const size_t own = (size_t)warps * rt_warp_bytes<T>(LPR * VPL, rows, a.n.k);
        const size_t sums = (size_t)warps * G * 8 * sizeof(float);
        return (size_t)(E + 3) / 4 * 16 + (own > sums ? own : sums);
    };
    const int choose = a.n.k * (100 + (int)sizeof(T) / 2 * LPR * VPL) + 200;
    const RouterCut cut = router_cut(a.n, 32 / LPR, rt_blocks<T, VPL>(),
                                     32 / LPR * rt_rows<LPR, VPL>(), 30 + 60 * VPL, choose,
                                     bytes);
    *joins = cut.joins;
    *parts = cut.parts;
    const size_t smem = bytes(cut.warps, cut.rows);
    if (smem > 40 * 1024) {
        const cudaError_t e = router_allow((const void *)kernel);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.n.groups * cut.parts));
    cfg.blockDim = dim3(32 * cut.warps);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cfg.gridDim.x;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cut.joins && cfg.gridDim.x > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, a, cut);
}

template <class T, int LPR, int VPL, bool ALIGNED>
cudaError_t router_backward_one(const RouterBackward &a, cudaStream_t s)
{
    auto *const kernel = k_router_bwd<T, LPR, VPL, ALIGNED>;
    auto bytes = [&](int warps, int rows) {
        return (size_t)warps * rt_warp_bytes_bwd(rows, a.n.k, rt_rows<LPR, VPL>() * 256 * VPL);
    };
    const RouterCut cut = router_cut(a.n, 32 / LPR, rt_blocks<T, VPL>(),
                                     32 / LPR * rt_rows<LPR, VPL>(), 40 + 60 * VPL,
                                     100 + 20 * a.n.k, bytes);
    const size_t smem = bytes(cut.warps, cut.rows);
    if (smem > 40 * 1024) {
        const cudaError_t e = router_allow((const void *)kernel);
        if (e != cudaSuccess) return e;
    }
    return launch_after_prior(kernel, (unsigned)(a.n.groups * cut.parts), 32 * cut.warps, smem, s, a, cut);
}

// Calls f.template run<LPR, VPL>() for the lanes and groups that a row of E experts takes.
template <class F>
cudaError_t router_width(int E, F f)
{
    if (E <= 8) return f.template run<1, 1>();
    if (E <= 16) return f.template run<2, 1>();
    if (E <= 32) return f.template run<4, 1>();
    if (E <= 64) return f.template run<8, 1>();
    if (E <= 128) return f.template run<16, 1>();
    if (E <= 256) return f.template run<32, 1>();
    if (E <= 512) return f.template run<32, 2>();
    return f.template run<32, 4>();
}

template <class T>
bool router_aligned(int E, const void *p, int64_t ld, int64_t rows)
{
    uintptr_t bits = (uintptr_t)p | (uintptr_t)E * sizeof(T);
    if (rows > 1) bits |= (uintptr_t)ld * sizeof(T);
    return bits % 16 == 0;
}

template <class T>
struct RouterForwardRun {
    const RouterForward &a;
    bool *joins;
    int *parts;
    cudaStream_t s;
    bool aligned;
    template <int LPR, int VPL>
    cudaError_t run() const
    {
        return aligned ? router_forward_one<T, LPR, VPL, true>(a, joins, parts, s)
                       : router_forward_one<T, LPR, VPL, false>(a, joins, parts, s);
    }
};

// *joins: the launch has joined what its blocks left, `parts` of a group.
template <class T>
cudaError_t router_forward(const RouterForward &a, bool *joins, int *parts, cudaStream_t s)
{
    const bool aligned = router_aligned<T>(a.n.experts, a.logits, a.ld, a.n.sequences * a.n.tokens);
    return router_width(a.n.experts, RouterForwardRun<T>{a, joins, parts, s, aligned});
}

template <class T>
struct RouterBackwardRun {
    const RouterBackward &a;
    cudaStream_t s;
    bool aligned;
    template <int LPR, int VPL>
    cudaError_t run() const
    {
        return aligned ? router_backward_one<T, LPR, VPL, true>(a, s)
                       : router_backward_one<T, LPR, VPL, false>(a, s);
    }
};

template <class T>
cudaError_t router_backward(const RouterBackward &a, cudaStream_t s)
{
    const int64_t rows = a.n.sequences * a.n.tokens;
    const bool aligned = router_aligned<T>(a.n.experts, a.logits, a.ld, rows) &&
                         router_aligned<T>(a.n.experts, a.dlogits, a.lddl, rows);
    return router_width(a.n.experts, RouterBackwardRun<T>{a, s, aligned});
}

}  // namespace fc
