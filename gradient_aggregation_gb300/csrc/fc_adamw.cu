// AdamW over many tensors at once, moments in fp32 or in 8 bits.
//
//   g = s * grad;  m = b1 m + (1-b1) g;  v = b2 v + (1-b2) g^2
//   w = w - lr wd d w - (lr / c1) m / (sqrt(v) / sqrt(c2) + eps)
//
// with c = 1 - b^t = -expm1(t ln b), which keeps its relative accuracy for
// small t where 1 - b^t in fp32 would cancel.
//
// Bound by HBM: with fp32 moments each element moves 24 bytes of state and
// weights, the gradient and the low-precision copy; with 8-bit moments 12.
//
// Layout: one warp takes one unit of 256 elements of the fused vector, which
// is also the block of an 8-bit state.  Lane l holds elements 4l..4l+3 and
// 128+4l..128+4l+3, so that every access of the state is one full 16-byte
// vector a lane for fp32 (8 bytes for 16-bit types, 4 for 8-bit ones),
// contiguous over the warp.  The state is always aligned; a gradient tensor
// sits at its own address, so its groups of 4 may be shifted against the
// fused index by 1 to 3 elements, the same shift for a whole layer: then a
// lane loads the two aligned groups around its own and selects, which keeps
// wide loads for layers of any size.  A unit that holds a layer boundary or
// the end of the vector goes element by element (at most two units a layer).
//
// Warps of a persistent grid take units in rounds.  The first unit's loads
// are issued before the step's scalars (count, factor) are awaited.
#include <cuda_fp8.h>

#include "fc_opt.h"

namespace fc {

#define FC_ADAM_BLOCK 256

struct StepScalars {
    float s;    // factor on the gradient
    float lrc;  // lr / c1
    float rc2;  // 1 / sqrt(c2)
    unsigned key;
    int skip;
};

// 32-bit mixing by multiplications and xor-shifts (a bijection of 32 bits).
__device__ __forceinline__ unsigned mix32(unsigned x)
{
    x ^= x >> 16;
    x *= 0x7feb352du;
    x ^= x >> 15;
    x *= 0x846ca68bu;
    x ^= x >> 16;
    return x;
}

// Read by one thread of each CTA.  A CTA arrives at steps[1] once it has read
// steps[0]; the last one to arrive counts the step, so no CTA can read the
// new count.
__device__ __forceinline__ void load_scalars(StepScalars &sc, const AdamHyper &h,
                                             const float *scale, int32_t *steps,
                                             uint64_t seed)
{
    const float s = scale ? __ldcg(scale) : 1.f;
    const int32_t done = __ldcg(steps);
    const float t = (float)(done + 1);
    const float c1 = -expm1f(t * h.lnb1);
    const float c2 = -expm1f(t * h.lnb2);
    sc.s = s;
    sc.lrc = __fdiv_rn(h.lr, c1);
    sc.rc2 = __fdiv_rn(1.f, __fsqrt_rn(c2));
    sc.skip = !isfinite(s);
    sc.key = mix32((unsigned)seed ^ mix32((unsigned)(seed >> 32) ^ mix32((unsigned)(done + 1))));
    if (!sc.skip) {
        __threadfence();
        if (atomicAdd(reinterpret_cast<unsigned *>(steps) + 1, 1u) == gridDim.x - 1) {
            steps[0] = done + 1;
            steps[1] = 0;
        }
    }
}

__device__ __forceinline__ float as_f32(float x) { return x; }
__device__ __forceinline__ float as_f32(__half x) { return __half2float(x); }
__device__ __forceinline__ float as_f32(__nv_bfloat16 x) { return __bfloat162float(x); }

// A lane's four gradient elements as they are loaded.
template <class GT>
struct Raw4 {
    uint2 q;
};
template <>
struct Raw4<float> {
    uint4 q;
};

__device__ __forceinline__ void unpack4(const Raw4<float> &r, float *g)
{
    g[0] = __uint_as_float(r.q.x);
    g[1] = __uint_as_float(r.q.y);
    g[2] = __uint_as_float(r.q.z);
    g[3] = __uint_as_float(r.q.w);
}

__device__ __forceinline__ void unpack4(const Raw4<__half> &r, float *g)
{
    const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&r.q.x));
    const float2 b = __half22float2(*reinterpret_cast<const __half2 *>(&r.q.y));
    g[0] = a.x;
    g[1] = a.y;
    g[2] = b.x;
    g[3] = b.y;
}

__device__ __forceinline__ void unpack4(const Raw4<__nv_bfloat16> &r, float *g)
{
    g[0] = __uint_as_float(r.q.x << 16);
    g[1] = __uint_as_float(r.q.x & 0xffff0000u);
    g[2] = __uint_as_float(r.q.y << 16);
    g[3] = __uint_as_float(r.q.y & 0xffff0000u);
}

// Elements d..d+3 (d = 1, 2, 3) of the eight in a:b.
__device__ __forceinline__ uint4 select4(const uint4 &a, const uint4 &b, int d)
{
    uint32_t w0 = a.x, w1 = a.y, w2 = a.z, w3 = a.w, w4 = b.x, w5 = b.y;
    if (d & 2) { w0 = w2; w1 = w3; w2 = w4; w3 = w5; w4 = b.z; }
    if (d & 1) { w0 = w1; w1 = w2; w2 = w3; w3 = w4; }
    return make_uint4(w0, w1, w2, w3);
}

__device__ __forceinline__ uint2 select4(const uint2 &a, const uint2 &b, int d)
{
    uint32_t w0 = a.x, w1 = a.y, w2 = b.x;
    if (d & 2) { w0 = w1; w1 = w2; w2 = b.y; }
    if (d & 1) {
        w0 = __funnelshift_r(w0, w1, 16);
        w1 = __funnelshift_r(w1, w2, 16);
    }
    return make_uint2(w0, w1);
}

template <class GT>
__device__ __forceinline__ Raw4<GT> gather4(const GT *p)
{
    Raw4<GT> r;
    if constexpr (sizeof(GT) == 4) {
        const unsigned *u = reinterpret_cast<const unsigned *>(p);
        r.q = make_uint4(__ldg(u), __ldg(u + 1), __ldg(u + 2), __ldg(u + 3));
    } else {
        const unsigned short *u = reinterpret_cast<const unsigned short *>(p);
        const unsigned a = __ldg(u), b = __ldg(u + 1), c = __ldg(u + 2), d = __ldg(u + 3);
        r.q = make_uint2(a | b << 16, c | d << 16);
    }
    return r;
}

// Four elements at p inside the segment [first, end), p `d` elements past a
// boundary of 4.
template <class GT>
__device__ __forceinline__ Raw4<GT> load4(const GT *p, const GT *first, const GT *end, int d)
{
    using Q = decltype(Raw4<GT>::q);
    Raw4<GT> r;
    if (d == 0) {
        r.q = __ldcs(reinterpret_cast<const Q *>(p));
        return r;
    }
    const GT *a = p - d;
    if (a >= first && a + 8 <= end) {
        const Q *q = reinterpret_cast<const Q *>(a);
        r.q = select4(__ldg(q), __ldg(q + 1), d);
        return r;
    }
    return gather4(p);
}

template <class Tab>
__device__ __forceinline__ int find_segment(const Tab &t, int64_t f)
{
    int lo = 0, hi = t.L - 1;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (t.off[mid + 1] > f)
            hi = mid;
        else
            lo = mid + 1;
    }
    return lo;
}

__device__ __forceinline__ void store_low4(void *low, int ltype, int64_t i, const float *w)
{
    uint2 q;
    if (ltype == FC_TYPE_F16) {
        const __half2 a = __floats2half2_rn(w[0], w[1]), b = __floats2half2_rn(w[2], w[3]);
        q.x = *reinterpret_cast<const uint32_t *>(&a);
        q.y = *reinterpret_cast<const uint32_t *>(&b);
    } else {
        const __nv_bfloat162 a = __floats2bfloat162_rn(w[0], w[1]);
        const __nv_bfloat162 b = __floats2bfloat162_rn(w[2], w[3]);
        q.x = *reinterpret_cast<const uint32_t *>(&a);
        q.y = *reinterpret_cast<const uint32_t *>(&b);
    }
    __stcs(reinterpret_cast<uint2 *>(static_cast<uint16_t *>(low) + i), q);
}

__device__ __forceinline__ void store_low1(void *low, int ltype, int64_t i, float w)
{
    if (ltype == FC_TYPE_F16)
        static_cast<__half *>(low)[i] = __float2half_rn(w);
    else
        static_cast<__nv_bfloat16 *>(low)[i] = __float2bfloat16_rn(w);
}

__device__ __forceinline__ float fast_sqrt(float x)
{
    float y;  // at most one unit in the last place off
    asm("sqrt.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// One element; returns sqrt(v).  The quotient is the fast division (2 units
// in the last place): it enters w scaled by lr, far below w's own rounding.
__device__ __forceinline__ float adam1(float graw, float decay, const AdamHyper &h,
                                       const StepScalars &sc, float &m, float &v, float &w)
{
    const float g = graw * sc.s;
    m = fmaf(h.b1, m, h.omb1 * g);
    v = fmaf(h.b2, v, h.omb2 * g * g);
    const float r = fast_sqrt(v);
    const float step = __fdividef(sc.lrc * m, fmaf(r, sc.rc2, h.eps));
    w = fmaf(-h.lrwd * decay, w, w) - step;
    return r;
}

// The part of a unit that both state formats share.
template <class GT>
struct UnitGrad {
    Raw4<GT> g[2];
    float decay;
};

// True if the unit at `lo` is whole and inside segment `sg` (moved on to the
// unit's first segment); then its gradient loads are issued.
template <class GT, class Tab>
__device__ __forceinline__ bool load_unit_grad(const Tab &tab, int64_t lo, int64_t N, int lane,
                                               int &sg, UnitGrad<GT> &u)
{
    if (!(tab.off[sg] <= lo && lo < tab.off[sg + 1])) sg = find_segment(tab, lo);
    const int64_t off = tab.off[sg], oend = tab.off[sg + 1];
    if (lo + FC_STATE_BLOCK > oend) return false;
    const GT *first = static_cast<const GT *>(tab.ptr[sg]);
    const GT *p = first + (lo - off) + 4 * lane;
    const GT *end = first + (oend - off);
    const int d = (int)(((uintptr_t)p / sizeof(GT)) & 3);
    u.decay = tab.decay[sg];
    u.g[0] = load4(p, first, end, d);
    u.g[1] = load4(p + 128, first, end, d);
    return true;
}

// ---- fp32 moments ---------------------------------------------------------------------

template <class GT, class Tab>
__global__ void __launch_bounds__(FC_ADAM_BLOCK)
    k_adamw(const __grid_constant__ Tab tab, const int64_t N, const AdamHyper h,
            const float *__restrict__ scale, float *__restrict__ w, void *__restrict__ low,
            const int ltype, float *__restrict__ m, float *__restrict__ v,
            int32_t *__restrict__ steps)
{
    __shared__ StepScalars sh;
    wait_for_prior_grid();
    allow_dependent_launch();
    const int lane = threadIdx.x & 31;
    const int64_t units = (N + FC_STATE_BLOCK - 1) / FC_STATE_BLOCK;
    const int64_t stride = (int64_t)gridDim.x * (FC_ADAM_BLOCK / 32);
    int64_t un = (int64_t)blockIdx.x * (FC_ADAM_BLOCK / 32) + (threadIdx.x >> 5);
    int sg = 0;
    UnitGrad<GT> u;
    float4 w4[2], m4[2], v4[2];
    bool whole = false;

    auto load = [&]() {
        const int64_t lo = un * FC_STATE_BLOCK;
        whole = load_unit_grad<GT>(tab, lo, N, lane, sg, u);
        if (!whole) return;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int64_t a = lo + 4 * lane + 128 * i;
            w4[i] = __ldcs(reinterpret_cast<const float4 *>(w + a));
            m4[i] = __ldcs(reinterpret_cast<const float4 *>(m + a));
            v4[i] = __ldcs(reinterpret_cast<const float4 *>(v + a));
        }
    };
    if (un < units) load();
    if (threadIdx.x == 0) {
        StepScalars t;
        load_scalars(t, h, scale, steps, 0);
        sh = t;
    }
    __syncthreads();
    const StepScalars sc = sh;
    if (sc.skip && !low) return;
    for (; un < units;) {
        const int64_t lo = un * FC_STATE_BLOCK;
        if (whole) {
            if (sc.skip) {
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    store_low4(low, ltype, lo + 4 * lane + 128 * i, &w4[i].x);
            } else {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float g[4];
                    unpack4(u.g[i], g);
                    adam1(g[0], u.decay, h, sc, m4[i].x, v4[i].x, w4[i].x);
                    adam1(g[1], u.decay, h, sc, m4[i].y, v4[i].y, w4[i].y);
                    adam1(g[2], u.decay, h, sc, m4[i].z, v4[i].z, w4[i].z);
                    adam1(g[3], u.decay, h, sc, m4[i].w, v4[i].w, w4[i].w);
                    const int64_t a = lo + 4 * lane + 128 * i;
                    __stcs(reinterpret_cast<float4 *>(w + a), w4[i]);
                    __stcs(reinterpret_cast<float4 *>(m + a), m4[i]);
                    __stcs(reinterpret_cast<float4 *>(v + a), v4[i]);
                    if (low) store_low4(low, ltype, a, &w4[i].x);
                }
            }
        } else {
            for (int e = 0; e < 8; ++e) {
                const int64_t a = lo + lane + 32 * e;
                if (a >= N) break;
                const int sa = find_segment(tab, a);
                float wi = w[a];
                if (!sc.skip) {
                    const float g = as_f32(static_cast<const GT *>(tab.ptr[sa])[a - tab.off[sa]]);
                    float mi = m[a], vi = v[a];
                    adam1(g, tab.decay[sa], h, sc, mi, vi, wi);
                    w[a] = wi;
                    m[a] = mi;
                    v[a] = vi;
                }
                if (low) store_low1(low, ltype, a, wi);
            }
        }
        un += stride;
        if (un < units) load();
    }
}

// ---- 8-bit moments --------------------------------------------------------------------

#define FC_E4M3_TOP 448.f

// The step with 8-bit moments runs in units of 2^-20: gradient, moments and
// eps are multiplied by 2^20 (exact, and folded into factors that are there
// anyway), so that g^2 stays a normal fp32 number down to |g| = 1e-24, well
// below the smallest moments that the blocks can hold relative to each other
// (fp32 moments end at |g| = 1e-19).
#define FC_ADAM8_UNIT 0x1p20f

// Factor onto the e4m3 range for a block whose largest value is `top` units,
// and the scale that undoes it; a block below 2^-110 (near where its scale
// would leave the normal numbers) holds zeros.  A NaN or an infinity in the
// block goes into the scale.
__device__ __forceinline__ void block_scale(float top, float &to, float &scale)
{
    const bool dead = top < 0x1p-110f * FC_ADAM8_UNIT;
    to = dead ? 0.f : __fdiv_rn(FC_E4M3_TOP, top);
    scale = dead ? 0.f : top * (1.f / FC_E4M3_TOP) * (1.f / FC_ADAM8_UNIT);
}

__device__ __forceinline__ void from_e4m3(uint32_t q, float scale, float *x)
{
    const __half2_raw a =
        __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(q & 0xffffu), __NV_E4M3);
    const __half2_raw b = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(q >> 16), __NV_E4M3);
    const float2 fa = __half22float2(__half2(a)), fb = __half22float2(__half2(b));
    x[0] = fa.x * scale;
    x[1] = fa.y * scale;
    x[2] = fb.x * scale;
    x[3] = fb.y * scale;
}

// Nearest e4m3, magnitudes above 448 (from the factor's rounding) to 448.
__device__ __forceinline__ uint32_t to_e4m3(float a, float b, float c, float d)
{
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
    return lo | hi << 16;
}

// The e4m3 value below or above y in [0, 448], by 16 random bits.  Normal
// e4m3 values differ from fp32 by 20 cut mantissa bits; below 2^-6 the
// spacing is 2^-9, which is what fp32 values in [2^-6, 2^-5) are cut to.
__device__ __forceinline__ float stochastic_e4m3(float y, unsigned bits16)
{
    y = fminf(y, FC_E4M3_TOP);
    const float base = y < 0x1p-6f ? 0x1p-6f : 0.f;
    const unsigned t = (__float_as_uint(y + base) + (bits16 * 16u + 8u)) & ~0xfffffu;
    const float q = fmaxf(__uint_as_float(t) - base, 0x1p-9f);
    return y > 0.f ? q : 0.f;
}

__device__ __forceinline__ unsigned pair_bits(unsigned key, int64_t i)
{
    const uint64_t p = (uint64_t)i >> 1;
    return mix32((unsigned)p + key + (unsigned)(p >> 32) * 0x9E3779B9u);
}

template <class GT, class Tab>
__global__ void __launch_bounds__(FC_ADAM_BLOCK)
    k_adamw8(const __grid_constant__ Tab tab, const int64_t N, const AdamHyper h,
             const float *__restrict__ scale, float *__restrict__ w, void *__restrict__ low,
             const int ltype, uint8_t *__restrict__ m8, float *__restrict__ m_scale,
             uint8_t *__restrict__ r8, float *__restrict__ r_scale,
             int32_t *__restrict__ steps, const uint64_t seed)
{
    // h.eps comes in units
    __shared__ StepScalars sh;
    wait_for_prior_grid();
    allow_dependent_launch();
    const int lane = threadIdx.x & 31;
    const int64_t units = (N + FC_STATE_BLOCK - 1) / FC_STATE_BLOCK;
    const int64_t stride = (int64_t)gridDim.x * (FC_ADAM_BLOCK / 32);
    int64_t un = (int64_t)blockIdx.x * (FC_ADAM_BLOCK / 32) + (threadIdx.x >> 5);
    int sg = 0;
    UnitGrad<GT> u;
    float4 w4[2];
    uint32_t mq[2], rq[2];
    float ms = 0.f, rs = 0.f;
    bool whole = false;

    auto load = [&]() {
        const int64_t lo = un * FC_STATE_BLOCK;
        whole = load_unit_grad<GT>(tab, lo, N, lane, sg, u);
        ms = __ldcs(m_scale + un) * FC_ADAM8_UNIT;
        rs = __ldcs(r_scale + un) * FC_ADAM8_UNIT;
        if (!whole) return;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int64_t a = lo + 4 * lane + 128 * i;
            w4[i] = __ldcs(reinterpret_cast<const float4 *>(w + a));
            mq[i] = __ldcs(reinterpret_cast<const unsigned *>(m8 + a));
            rq[i] = __ldcs(reinterpret_cast<const unsigned *>(r8 + a));
        }
    };
    if (un < units) load();
    if (threadIdx.x == 0) {
        StepScalars t;
        load_scalars(t, h, scale, steps, seed);
        t.s *= FC_ADAM8_UNIT;
        sh = t;
    }
    __syncthreads();
    const StepScalars sc = sh;
    if (sc.skip && !low) return;
    for (; un < units;) {
        const int64_t lo = un * FC_STATE_BLOCK;
        if (sc.skip) {
            for (int e = 0; e < 8; ++e) {
                const int64_t a = lo + lane + 32 * e;
                if (a < N) store_low1(low, ltype, a, w[a]);
            }
        } else {
            // element order of x[8]: of the lane's two groups where the unit
            // is whole, lo + lane + 32 e where it is not
            float mv[8], rv[8];
            unsigned mtop = 0u, rtop = 0u;
            if (whole) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int64_t a = lo + 4 * lane + 128 * i;
                    float g[4];
                    unpack4(u.g[i], g);
                    from_e4m3(mq[i], ms, mv + 4 * i);
                    from_e4m3(rq[i], rs, rv + 4 * i);
                    float *wp = &w4[i].x;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float v = rv[4 * i + e] * rv[4 * i + e];
                        rv[4 * i + e] = adam1(g[e], u.decay, h, sc, mv[4 * i + e], v, wp[e]);
                    }
                    __stcs(reinterpret_cast<float4 *>(w + a), w4[i]);
                    if (low) store_low4(low, ltype, a, wp);
                }
            } else {
                for (int e = 0; e < 8; ++e) {
                    const int64_t a = lo + lane + 32 * e;
                    mv[e] = rv[e] = 0.f;
                    if (a >= N) continue;
                    const int sa = find_segment(tab, a);
                    const float g = as_f32(static_cast<const GT *>(tab.ptr[sa])[a - tab.off[sa]]);
                    float wi = w[a];
                    const __half_raw hm = __nv_cvt_fp8_to_halfraw(m8[a], __NV_E4M3);
                    const __half_raw hr = __nv_cvt_fp8_to_halfraw(r8[a], __NV_E4M3);
                    mv[e] = __half2float(__half(hm)) * ms;
                    const float r = __half2float(__half(hr)) * rs;
                    float v = r * r;
                    rv[e] = adam1(g, tab.decay[sa], h, sc, mv[e], v, wi);
                    w[a] = wi;
                    if (low) store_low1(low, ltype, a, wi);
                }
            }
            // magnitudes compare as their bit patterns; a NaN is above all
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                mtop = max(mtop, __float_as_uint(mv[e]) & 0x7fffffffu);
                rtop = max(rtop, __float_as_uint(rv[e]) & 0x7fffffffu);
            }
            mtop = __reduce_max_sync(0xffffffffu, mtop);
            rtop = __reduce_max_sync(0xffffffffu, rtop);
            float mto, mnew, rto, rnew;
            block_scale(__uint_as_float(mtop), mto, mnew);
            block_scale(__uint_as_float(rtop), rto, rnew);
            if (lane == 0) {
                __stcs(m_scale + un, mnew);
                __stcs(r_scale + un, rnew);
            }
            if (whole) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int64_t a = lo + 4 * lane + 128 * i;
                    const float *x = mv + 4 * i;
                    __stcs(reinterpret_cast<unsigned *>(m8 + a),
                           to_e4m3(x[0] * mto, x[1] * mto, x[2] * mto, x[3] * mto));
                    const unsigned h0 = pair_bits(sc.key, a), h1 = pair_bits(sc.key, a + 2);
                    const float *y = rv + 4 * i;
                    __stcs(reinterpret_cast<unsigned *>(r8 + a),
                           to_e4m3(stochastic_e4m3(y[0] * rto, h0 & 0xffffu),
                                   stochastic_e4m3(y[1] * rto, h0 >> 16),
                                   stochastic_e4m3(y[2] * rto, h1 & 0xffffu),
                                   stochastic_e4m3(y[3] * rto, h1 >> 16)));
                }
            } else {
                for (int e = 0; e < 8; ++e) {
                    const int64_t a = lo + lane + 32 * e;
                    if (a >= N) continue;
                    m8[a] = (uint8_t)to_e4m3(mv[e] * mto, 0.f, 0.f, 0.f);
                    const unsigned hb = pair_bits(sc.key, a);
                    const float q = stochastic_e4m3(rv[e] * rto, a & 1 ? hb >> 16 : hb & 0xffffu);
                    r8[a] = (uint8_t)to_e4m3(q, 0.f, 0.f, 0.f);
                }
            }
        }
        un += stride;
        if (un < units) load();
    }
}

template <class F>
static int units_grid(F kernel, int64_t N)
{
    const int64_t per = FC_ADAM_BLOCK / 32;
    const int64_t ctas = ((N + FC_STATE_BLOCK - 1) / FC_STATE_BLOCK + per - 1) / per;
    int grid = grid_for((const void *)kernel, FC_ADAM_BLOCK, 0, ctas);
    if (ctas > grid) {  // as many rounds as needed, all of the same length
        const int64_t rounds = (ctas + grid - 1) / grid;
        grid = (int)((ctas + rounds - 1) / rounds);
    }
    return grid;
}

template <class GT, class Tab>
static cudaError_t launch_typed(const Tab &tab, int64_t N, const AdamHyper &h, const float *scale,
                                float *w, void *low, int ltype, float *m, float *v,
                                int32_t *steps, cudaStream_t s)
{
    return launch_after_prior(k_adamw<GT, Tab>, (unsigned)units_grid(k_adamw<GT, Tab>, N),
                              FC_ADAM_BLOCK, 0, s, tab, N, h, scale, w, low, ltype, m, v, steps);
}

template <class GT, class Tab>
static cudaError_t launch_typed8(const Tab &tab, int64_t N, const AdamHyper &h,
                                 const float *scale, float *w, void *low, int ltype, uint8_t *m8,
                                 float *m_scale, uint8_t *r8, float *r_scale, int32_t *steps,
                                 uint64_t seed, cudaStream_t s)
{
    AdamHyper units = h;
    units.eps *= FC_ADAM8_UNIT;
    return launch_after_prior(k_adamw8<GT, Tab>, (unsigned)units_grid(k_adamw8<GT, Tab>, N),
                              FC_ADAM_BLOCK, 0, s, tab, N, units, scale, w, low, ltype, m8, m_scale,
                              r8, r_scale, steps, seed);
}

template <class Tab>
cudaError_t launch_adamw(const Tab &tab, int gtype, int64_t N, const AdamHyper &h,
                         const float *scale, float *w, void *low, int ltype, float *m, float *v,
                         int32_t *steps, cudaStream_t s)
{
    if (gtype == FC_TYPE_F32)
        return launch_typed<float>(tab, N, h, scale, w, low, ltype, m, v, steps, s);
    if (gtype == FC_TYPE_F16)
        return launch_typed<__half>(tab, N, h, scale, w, low, ltype, m, v, steps, s);
    return launch_typed<__nv_bfloat16>(tab, N, h, scale, w, low, ltype, m, v, steps, s);
}

template <class Tab>
cudaError_t launch_adamw8(const Tab &tab, int gtype, int64_t N, const AdamHyper &h,
                          const float *scale, float *w, void *low, int ltype, uint8_t *m8,
                          float *m_scale, uint8_t *r8, float *r_scale, int32_t *steps,
                          uint64_t seed, cudaStream_t s)
{
    if (gtype == FC_TYPE_F32)
        return launch_typed8<float>(tab, N, h, scale, w, low, ltype, m8, m_scale, r8, r_scale,
                                    steps, seed, s);
    if (gtype == FC_TYPE_F16)
        return launch_typed8<__half>(tab, N, h, scale, w, low, ltype, m8, m_scale, r8, r_scale,
                                     steps, seed, s);
    return launch_typed8<__nv_bfloat16>(tab, N, h, scale, w, low, ltype, m8, m_scale, r8, r_scale,
                                        steps, seed, s);
}

#define FC_INST(Tab)                                                                            \
    template cudaError_t launch_adamw<Tab>(const Tab &, int, int64_t, const AdamHyper &,        \
                                           const float *, float *, void *, int, float *,       \
                                           float *, int32_t *, cudaStream_t);                   \
    template cudaError_t launch_adamw8<Tab>(const Tab &, int, int64_t, const AdamHyper &,       \
                                            const float *, float *, void *, int, uint8_t *,    \
                                            float *, uint8_t *, float *, int32_t *, uint64_t,  \
                                            cudaStream_t);
FC_INST(OptTableS)
FC_INST(OptTableL)

}  // namespace fc
