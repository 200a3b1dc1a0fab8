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
// wide loads for layers of any size.  A unit that holds a layer boundary
// reads its gradient element by element (at most two units a layer), and so
// does everything of the last unit where N is not a multiple of 256.
//
// Two kernels hold the same arithmetic: k_adamw_ring streams weights and
// moments through shared memory with bulk copies in both directions;
// k_adamw_direct loads and stores them from registers, which starts faster and
// serves what is resident at once.  Measured (ring): 278 us for 62.4M elements
// with fp32 moments, fp32 gradients and an fp16 copy (1.87 GB, 6.7 TB/s); 159
// us with 8-bit moments and fp16 gradients (1.0 GB, 6.3 TB/s); direct: 3.9 us
// for 133k elements.
#include <cuda_fp8.h>

#include <algorithm>
#include <atomic>

#include "fc_bulk.cuh"
#include "fc_opt.h"
#include "fc_pairs.cuh"

namespace fc {

#define FC_ADAM_BLOCK 256

// Consumer warps of the ring kernel (so units a tile) and its stages.  A tile
// of 19 units is copied in pieces of 19 KB; with 8 KB pieces the 62M-element
// step with fp32 moments took 320 us, with 16 KB 286, with 19 and 20 KB 278 and 280
// (fp32 gradients in 600 layers, 20M elements: 96 and 103 us: 20 warps and the copying
// one have 80 registers each, 19 have 96).  With 8-bit moments the update itself
// needs the warps: 23 of them have 80 registers, 24 to 27 have 72.  62M elements of
// fp16 / bf16 / fp32 159 / 159 / 176 us with 27 (23: 160 / 160 / 176, 24: 173 / 176 /
// 185); where gradients are shifted the selecting needs the registers, 7M elements in
// odd layers 24.1 / 24.2 / 29.6 with 23 (24: 28.4 / 28.4 / 29.7, 27: bf16 27.2).
#define FC_ADAM_CW32 19
#define FC_ADAM_S32 3
#define FC_ADAM_CW8 27
#define FC_ADAM_CW8_SHIFTED 23
#define FC_ADAM_S8 4

#define FC_ADAM_WAIT_NS 2000000000ull

struct AdamState {
    int64_t N;
    AdamHyper h;
    const float *scale;
    float *w;
    void *low;
    int ltype;
    float *m, *v;                // fp32 moments
    uint8_t *m8, *r8;            // 8-bit moments
    float *m_scale, *r_scale;
    int32_t *steps;
    uint64_t seed;
    uint64_t limit_ns;  // of a wait for a copy or for the consumers
    int64_t drop;       // tile that is not copied in (test hook), -1: none
};

struct StepScalars {
    float s;     // factor on the gradient (times 2^20 for 8-bit moments)
    float lrc;   // lr / c1
    float rc2;   // 1 / sqrt(c2)
    unsigned key;
    int skip;
};

// The step with 8-bit moments runs in units of 2^-20: gradient, moments and
// eps are multiplied by 2^20 (exact, and folded into factors that are there
// anyway), so that g^2 stays a normal fp32 number down to |g| = 1e-24, well
// below the smallest moments that the blocks can hold relative to each other
// (fp32 moments end at |g| = 1e-19).  A unit of 256 elements with a v that is then
// too large for fp32 (|g| from 1.8e13 on) is done again in units of 2^20.
#define FC_ADAM8_UNIT 0x1p20f
#define FC_ADAM8_LARGE 0x1p-20f

// 32-bit mixing by multiplications and xor-shifts (a bijection of 32 bits), with a
// pair of multipliers from Chris Wellons' published search for mixers of this form
// (2018), chosen for the low bias of each output bit.
__device__ __forceinline__ unsigned mix32(unsigned x)
{
    x ^= x >> 16;
    x *= 0x7feb352du;
    x ^= x >> 15;
    x *= 0x846ca68bu;
    x ^= x >> 16;
    return x;
}

// Called by one warp of each CTA; the caller's barrier shows `sh` to the rest.
template <int BITS>
__device__ __forceinline__ void load_scalars(StepScalars &sh, const AdamState &st)
{
    const int lane = threadIdx.x & 31;
    const float s = st.scale ? __ldcg(st.scale) : 1.f;
    const int32_t t = __ldcg(st.steps) + 1;
    // lane 0 forms c1, lane 1 c2
    const float c = -expm1f((float)t * (lane == 0 ? st.h.lnb1 : st.h.lnb2));
    if (lane == 0) {
        sh.lrc = __fdividef(st.h.lr, c);
        sh.s = BITS == 8 ? s * FC_ADAM8_UNIT : s;
        sh.skip = !isfinite(s);
        sh.key = mix32((unsigned)st.seed ^ mix32((unsigned)(st.seed >> 32) ^ mix32((unsigned)t)));
    } else if (lane == 1) {
        sh.rc2 = rsqrtf(c);
    }
}

// Each CTA arrives at steps[1] once it has read steps[0], and the last to
// arrive counts the step, so no CTA can read the new count.  The arrival is
// issued early and its answer only looked at when the CTA's work is done.
//
// Bit 31 of steps[1] says that a wait has run out, in this launch or an earlier one
// (FC_ADAM_LOST), and no such step is counted.  It may be set before the last CTA
// arrives, which sees it then, or later: then the step is counted, or will be,
// and whoever sets the bit takes the count back.  Additions on both sides, so
// their order does not matter, and nothing that is waited for.
#define FC_ADAM_LOST 0x80000000u

__device__ __forceinline__ unsigned arrive_step(int32_t *steps)
{
    unsigned old;
    asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;"
                 : "=r"(old)
                 : "l"(steps + 1)
                 : "memory");
    return old;
}

__device__ __forceinline__ void count_step(int32_t *steps, unsigned arrived)
{
    if ((arrived & ~FC_ADAM_LOST) == gridDim.x - 1) {
        if (!(arrived & FC_ADAM_LOST)) atomicAdd(steps, 1);
        atomicSub(reinterpret_cast<unsigned *>(steps) + 1, gridDim.x);
    }
}

// A wait has run out in a CTA that has arrived (skip: none does).
__device__ __forceinline__ void step_lost(int32_t *steps, int skip)
{
    const unsigned old = atomicOr(reinterpret_cast<unsigned *>(steps) + 1, FC_ADAM_LOST);
    const unsigned arrived = old & ~FC_ADAM_LOST;
    // all have arrived, or that is over
    if (!(old & FC_ADAM_LOST) && !skip && (arrived == gridDim.x || arrived == 0))
        atomicSub(steps, 1);
}

__device__ __forceinline__ float as_f32(float x) { return x; }
__device__ __forceinline__ float as_f32(__half x) { return __half2float(x); }
__device__ __forceinline__ float as_f32(__nv_bfloat16 x) { return __bfloat162float(x); }

// ---- gradients ------------------------------------------------------------------------

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

// The gradient of a unit that lies inside one segment.  SHIFTED: some segment
// is shifted against the fused index; then both groups around a lane's four
// elements are kept as they were loaded and selected when they are used, so
// that no load is waited for before its unit's turn.
template <class GT, bool SHIFTED>
struct UnitGrad {
    Raw4<GT> g[SHIFTED ? 4 : 2];
    float decay;
    int d;   // the segment's shift; -1: the unit is not whole
    int sg;  // segment of the unit's first element
    __device__ __forceinline__ void unpack(float *x) const
    {
        if constexpr (SHIFTED) {
            Raw4<GT> a = g[0], b = g[2];
            if (d) {
                a.q = select4(a.q, g[1].q, d);
                b.q = select4(b.q, g[3].q, d);
            }
            unpack4(a, x);
            unpack4(b, x + 4);
        } else {
            unpack4(g[0], x);
            unpack4(g[1], x + 4);
        }
    }
};

// Issues the gradient loads of the unit at `lo` if it is whole and lies inside
// one segment together with the aligned groups around it; `sg` is moved on to
// the unit's first segment.
template <class GT, bool SHIFTED, class Tab>
__device__ __forceinline__ void load_unit_grad(const Tab &tab, int64_t lo, int lane, int &sg,
                                               UnitGrad<GT, SHIFTED> &u)
{
    if (!(tab.off[sg] <= lo && lo < tab.off[sg + 1])) sg = find_segment(tab, lo);
    const int64_t at = lo - tab.off[sg], len = tab.off[sg + 1] - tab.off[sg];
    const GT *p = static_cast<const GT *>(tab.ptr[sg]) + at;
    const int d = SHIFTED ? (int)(((uintptr_t)p / sizeof(GT)) & 3) : 0;
    u.sg = sg;
    u.d = -1;
    if (at < d || at + FC_STATE_BLOCK + (d ? 4 - d : 0) > len) return;
    using Q = decltype(Raw4<GT>::q);
    const Q *q = reinterpret_cast<const Q *>(p - d) + lane;
    u.d = d;
    u.decay = tab.decay[sg];
    if constexpr (SHIFTED) {
        u.g[0].q = __ldg(q);
        u.g[2].q = __ldg(q + 32);
        if (d) {
            u.g[1].q = __ldg(q + 1);
            u.g[3].q = __ldg(q + 33);
        }
    } else {
        u.g[0].q = __ldcs(q);
        u.g[1].q = __ldcs(q + 32);
    }
}

// Gradient and decay of a lane's eight elements of any unit (0 past N), `sg`
// the segment of the unit's first element.  All eight loads are in flight
// before the first is used.
template <class GT, class Tab>
__device__ __forceinline__ void gather_unit(const Tab &tab, int64_t N, int64_t lo, int lane,
                                            int sg, float *g, float *d)
{
    GT x[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int64_t a = lo + 4 * lane + 128 * (j >> 2) + (j & 3);
        const int64_t f = a < N ? a : N - 1;
        while (tab.off[sg + 1] <= f) ++sg;
        x[j] = static_cast<const GT *>(tab.ptr[sg])[f - tab.off[sg]];
        d[j] = tab.decay[sg];
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int64_t a = lo + 4 * lane + 128 * (j >> 2) + (j & 3);
        g[j] = a < N ? as_f32(x[j]) : 0.f;
    }
}

// ---- arithmetic -----------------------------------------------------------------------

__device__ __forceinline__ float fast_sqrt(float x)
{
    float y;  // at most one unit in the last place off
    asm("sqrt.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// sqrt(x) for x = 0 or in [2^-126, 2^127]: the approximate reciprocal root, and
// one Newton step on the root's remainder, after which all but about one root
// in a million is the nearest fp32 number.
__device__ __forceinline__ F2 newton_sqrt2(F2 x)
{
    const float2 u = un2(x);
    float2 y;
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y.x) : "f"(fmaxf(u.x, 0x1p-126f)));
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y.y) : "f"(fmaxf(u.y, 0x1p-126f)));
    const F2 y2 = f2(y.x, y.y), s = mul2(x, y2), half = mul2(f2(-0.5f, -0.5f), y2);
    // s - (s^2 - x) y / 2
    return fma2(fma2(s, s, f2(-u.x, -u.y)), half, s);
}

// One element with fp32 moments.  The quotient is the fast division (2 units
// in the last place): it enters w scaled by lr, far below w's own rounding.
__device__ __forceinline__ void adam1(float graw, float decay, const AdamHyper &h,
                                      const StepScalars &sc, float &m, float &v, float &w)
{
    const float g = graw * sc.s;
    m = fmaf(h.b1, m, h.omb1 * g);
    v = fmaf(h.b2, v, h.omb2 * g * g);
    const float step = __fdividef(sc.lrc * m, fmaf(fast_sqrt(v), sc.rc2, h.eps));
    w = fmaf(-h.lrwd * decay, w, w) - step;
}

// a + b, one by one: the compiler joins a packed sum (one rounding) with a packed
// product before it.
__device__ __forceinline__ F2 add_once(F2 a, F2 b)
{
    const float2 x = un2(a), y = un2(b);
    return f2(__fadd_rn(x.x, y.x), __fadd_rn(x.y, y.y));
}

__device__ __forceinline__ float max3_nan(float a, float b, float c)
{
    float y;  // a NaN among the three is the result
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
    return y;
}

// x, or the limit with x's sign beyond it; an infinity and a NaN stay.
__device__ __forceinline__ float finite_at_most(float x, float limit)
{
    return fabsf(x) < INFINITY ? fminf(fmaxf(x, -limit), limit) : x;
}

// A lane's eight elements of a unit with 8-bit moments.  w: updated; mq, rq:
// e4m3 codes in and out; ms, rs: block scales in and out.  UNIFORM: d[0] is
// the decay of all eight.
//
// The moments are formed by the definition's operations one by one, each
// rounded once (no fused multiply-add), and the root and the blocks' factors
// to the nearest: a code is a step function of its value, so a last place
// would turn some code in a million into its neighbour, 6 % away, and the
// next step's block maximum with it.  The weights take the fast quotient.
//
// The unit is bound by the issue of its instructions where it is not by HBM, so
// two elements share one wherever they can (7M elements in odd layers 25.2 us
// so, one by one 26.2, with the loads as they then were).
//
// Rounding r by chance: y = r * 448 / top lies in [0, 448].  Scaled by 2^-120
// an e4m3 number is the top of an fp32 number's bits: e4m3's smallest normal
// 2^-6 falls on fp32's 2^-126, so that below it both formats are linear, and
// the code is the bits above bit 20 everywhere.  Adding 20 random bits (16
// drawn, centred) below the code and cutting rounds up with the probability
// of what is cut off.  A code of 0 for r > 0 becomes 1.
//
// False, for the whole warp: some v is not finite.  The codes and scales are then
// untouched and w is lost; marked_units does the step with LARGE.  That always
// succeeds, and a finite gradient beyond 2^83 (9.7e24) counts as 2^83 there, so that
// it leaves finite moments and weights; an infinity or a NaN goes through.
template <bool UNIFORM, bool LARGE = false>
__device__ __forceinline__ bool adam8_unit(const float *graw, const float *d, const AdamHyper &h,
                                           const StepScalars &sc, int64_t i0, float *w,
                                           uint32_t *mq, uint32_t *rq, float &ms, float &rs)
{
    F2 m[4], r[4];
    constexpr float UNIT = LARGE ? FC_ADAM8_LARGE : FC_ADAM8_UNIT;
    constexpr float FROM = LARGE ? FC_ADAM8_LARGE / FC_ADAM8_UNIT : 1.f;  // the caller's units
    const float ma = ms * UNIT, ra = rs * UNIT, s = sc.s * FROM;
    const float eps = LARGE ? fmaxf(h.eps * FROM, 0x1p-126f) : h.eps;
    const F2 ma2 = f2(ma, ma), ra2 = f2(ra, ra), s2 = f2(s, s);
    const F2 b12 = f2(h.b1, h.b1), b22 = f2(h.b2, h.b2);
    const F2 omb12 = f2(h.omb1, h.omb1), omb22 = f2(h.omb2, h.omb2);
    const F2 rc22 = f2(sc.rc2, sc.rc2), eps2 = f2(eps, eps), lrc2 = f2(-sc.lrc, -sc.lrc);
    const float wd0 = -h.lrwd * d[0];
    float mtop = 0.f, rtop = 0.f;
#pragma unroll
    for (int p = 0; p < 4; ++p) {
        const float2 cm = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(
            (__nv_fp8x2_storage_t)(mq[p >> 1] >> (16 * (p & 1))), __NV_E4M3)));
        const float2 cr = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(
            (__nv_fp8x2_storage_t)(rq[p >> 1] >> (16 * (p & 1))), __NV_E4M3)));
        F2 g = mul2(f2(graw[2 * p], graw[2 * p + 1]), s2);
        if constexpr (LARGE) {
            const float2 u = un2(g);
            g = f2(finite_at_most(u.x, 0x1p63f), finite_at_most(u.y, 0x1p63f));
        }
        const F2 r0 = mul2(f2(cr.x, cr.y), ra2);
        m[p] = add_once(mul2(mul2(f2(cm.x, cm.y), ma2), b12), mul2(g, omb12));
        const F2 v = add_once(mul2(mul2(r0, r0), b22), mul2(mul2(g, g), omb22));
        r[p] = newton_sqrt2(v);
        const float2 den = un2(fma2(r[p], rc22, eps2));
        const F2 rden = f2(rcp_ftz(den.x), rcp_ftz(den.y));
        const F2 w2 = f2(w[2 * p], w[2 * p + 1]);
        const F2 wd = UNIFORM ? f2(wd0, wd0) : f2(-h.lrwd * d[2 * p], -h.lrwd * d[2 * p + 1]);
        const float2 wn = un2(fma2(mul2(lrc2, m[p]), rden, fma2(wd, w2, w2)));
        w[2 * p] = wn.x;
        w[2 * p + 1] = wn.y;
        const float2 mu = un2(m[p]), ru = un2(r[p]);
        mtop = max3_nan(mtop, fabsf(mu.x), fabsf(mu.y));
        rtop = max3_nan(rtop, ru.x, ru.y);
    }
    // magnitudes compare as their bits; a NaN is above all numbers
    mtop = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(mtop)));
    rtop = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(rtop)));
    // the root of an infinite v is NaN
    if constexpr (!LARGE)
        if (!(rtop < INFINITY)) return false;
    // a block below 2^-110 holds zeros; a NaN or an infinity goes into the scale
    const bool mdead = mtop < 0x1p-110f * UNIT;
    const bool rdead = rtop < 0x1p-110f * UNIT;
    ms = mdead ? 0.f : mtop * (1.f / 448.f / UNIT);
    rs = rdead ? 0.f : rtop * (1.f / 448.f / UNIT);
    // even lanes divide for m, odd ones for r
    const float q448 = 448.f * __frcp_rn((threadIdx.x & 1) ? rtop : mtop);
    const float mto = mdead ? 0.f : __shfl_sync(0xffffffffu, q448, 0);
    const float rto = rdead ? 0.f : __shfl_sync(0xffffffffu, q448, 1);
    const F2 mto2 = f2(mto, mto), rto2 = f2(rto, rto);
    const float least = rdead ? 0.f : 0x1p-129f;  // e4m3's 2^-9
    const uint64_t pair = (uint64_t)i0 >> 1;
    const uint32_t x = (uint32_t)pair + sc.key + (uint32_t)(pair >> 32) * 0x9E3779B9u;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        mq[q] = (uint32_t)__nv_cvt_float2_to_fp8x2(un2(mul2(m[2 * q], mto2)), __NV_SATFINITE,
                                                   __NV_E4M3) |
                (uint32_t)__nv_cvt_float2_to_fp8x2(un2(mul2(m[2 * q + 1], mto2)), __NV_SATFINITE,
                                                   __NV_E4M3)
                    << 16;
        uint32_t u[4];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const uint32_t bits = mix32(x + 64 * q + e);
            // 24 bits: the 16 drawn, then 0x80
            const uint32_t lo = __byte_perm(bits, 0x80u, 0x5104);
            const uint32_t hi = __byte_perm(bits, 0x80u, 0x5324);
            const float2 ru = un2(r[2 * q + e]);
            const float2 y = un2(mul2(mul2(r[2 * q + e], rto2), f2(0x1p-120f, 0x1p-120f)));
            // r > 0 is at least 2^-63 here
            const float y0 = fmaxf(y.x, fminf(ru.x, least));
            const float y1 = fmaxf(y.y, fminf(ru.y, least));
            u[2 * e] = (__float_as_uint(y0) << 4) + lo;
            u[2 * e + 1] = (__float_as_uint(y1) << 4) + hi;
        }
        rq[q] = __byte_perm(__byte_perm(u[0], u[1], 0x0073), __byte_perm(u[2], u[3], 0x0073),
                            0x5410);
    }
    return true;
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

// ---- units from and to global memory ----------------------------------------------------

// Any unit in registers: weights, moments, gradient and decay of a lane's
// eight elements (0 past N).  Groups that lie inside one layer and inside the
// vector are read and written as vectors, the others element by element.
template <int BITS>
struct UnitRegs {
    float w[8], g[8], d[8];
    float m[BITS == 32 ? 8 : 1], v[BITS == 32 ? 8 : 1];
    uint32_t mq[2], rq[2];
    float ms, rs;
};

__device__ __forceinline__ void get4(float *to, const float *from, bool whole, int have)
{
    if (whole) {
        const float4 x = __ldcs(reinterpret_cast<const float4 *>(from));
        to[0] = x.x;
        to[1] = x.y;
        to[2] = x.z;
        to[3] = x.w;
    } else {
        to[0] = have > 0 ? from[0] : 0.f;
        to[1] = have > 1 ? from[1] : 0.f;
        to[2] = have > 2 ? from[2] : 0.f;
        to[3] = 0.f;
    }
}

__device__ __forceinline__ void put4(float *to, const float *from, bool whole, int have)
{
    if (whole) {
        __stcs(reinterpret_cast<float4 *>(to), make_float4(from[0], from[1], from[2], from[3]));
    } else {
        if (have > 0) to[0] = from[0];
        if (have > 1) to[1] = from[1];
        if (have > 2) to[2] = from[2];
    }
}

__device__ __forceinline__ uint32_t get4(const uint8_t *from, bool whole, int have)
{
    if (whole) return __ldcs(reinterpret_cast<const unsigned *>(from));
    uint32_t q = 0;
#pragma unroll
    for (int e = 0; e < 3; ++e)
        if (e < have) q |= (uint32_t)from[e] << (8 * e);
    return q;
}

__device__ __forceinline__ void put4(uint8_t *to, uint32_t q, bool whole, int have)
{
    if (whole) {
        __stcs(reinterpret_cast<unsigned *>(to), q);
        return;
    }
#pragma unroll
    for (int e = 0; e < 3; ++e)
        if (e < have) to[e] = (uint8_t)(q >> (8 * e));
}

template <class GT, int BITS, class Tab>
__device__ __forceinline__ void load_unit(const Tab &tab, const AdamState &st, int64_t un,
                                          int lane, UnitRegs<BITS> &u)
{
    const int64_t lo = un * FC_STATE_BLOCK;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int64_t a = lo + 4 * lane + 128 * i;
        const bool whole = a + 4 <= st.N;
        const int have = a < st.N ? (int)(st.N - a) : 0;  // only looked at if not whole
        get4(u.w + 4 * i, st.w + a, whole, have);
        if constexpr (BITS == 32) {
            get4(u.m + 4 * i, st.m + a, whole, have);
            get4(u.v + 4 * i, st.v + a, whole, have);
        } else {
            u.mq[i] = get4(st.m8 + a, whole, have);
            u.rq[i] = get4(st.r8 + a, whole, have);
        }
    }
    if constexpr (BITS == 8) {
        u.ms = __ldcs(st.m_scale + un);
        u.rs = __ldcs(st.r_scale + un);
    }
    int sg = find_segment(tab, lo);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int64_t a = lo + 4 * lane + 128 * i;
        float *const g = u.g + 4 * i, *const d = u.d + 4 * i;
        while (sg + 1 < tab.L && tab.off[sg + 1] <= a) ++sg;
        const int64_t off = tab.off[sg], oend = tab.off[sg + 1];
        const GT *first = static_cast<const GT *>(tab.ptr[sg]);
        d[0] = d[1] = d[2] = d[3] = tab.decay[sg];
        if (a + 4 <= oend) {
            const GT *p = first + (a - off);
            unpack4(load4(p, first, first + (oend - off), (int)(((uintptr_t)p / sizeof(GT)) & 3)),
                    g);
        } else {
            int se = sg;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                g[e] = 0.f;
                if (a + e < st.N) {
                    while (tab.off[se + 1] <= a + e) ++se;
                    g[e] = as_f32(static_cast<const GT *>(tab.ptr[se])[a + e - tab.off[se]]);
                    d[e] = tab.decay[se];
                }
            }
        }
    }
}

// What update_unit or marked_units has made of a unit; of a skipped one the
// low-precision copy alone.
template <int BITS>
__device__ __forceinline__ void store_unit(const AdamState &st, int skip, int64_t un, int lane,
                                           const UnitRegs<BITS> &u)
{
    const int64_t lo = un * FC_STATE_BLOCK;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int64_t a = lo + 4 * lane + 128 * i;
        const bool whole = a + 4 <= st.N;
        const int have = a < st.N ? (int)(st.N - a) : 0;
        if (!skip) {
            put4(st.w + a, u.w + 4 * i, whole, have);
            if constexpr (BITS == 32) {
                put4(st.m + a, u.m + 4 * i, whole, have);
                put4(st.v + a, u.v + 4 * i, whole, have);
            } else {
                put4(st.m8 + a, u.mq[i], whole, have);
                put4(st.r8 + a, u.rq[i], whole, have);
            }
        }
        if (st.low) {
            if (whole) {
                store_low4(st.low, st.ltype, a, u.w + 4 * i);
            } else {
#pragma unroll
                for (int e = 0; e < 3; ++e)
                    if (e < have) store_low1(st.low, st.ltype, a + e, u.w[4 * i + e]);
            }
        }
    }
    if constexpr (BITS == 8) {
        if (lane == 0 && !skip) {
            st.m_scale[un] = u.ms;
            st.r_scale[un] = u.rs;
        }
    }
}

// Leaves a unit whose v does not fit the usual units as it is and marks it by the
// sign of its r_scale.
__device__ __forceinline__ void mark_unit(const AdamState &st, int64_t un, int lane, float rs)
{
    if (lane == 0) st.r_scale[un] = __int_as_float(__float_as_int(rs) | 0x80000000);
}

// The marked ones of a warp's units, in global memory, once all else is done: CW
// units a tile, tile after tile of the CTA, and (the last CTA) those behind the last.
// `drained`: barrier of the copies out, which write what came in, or 0.  Out of
// line, called once and with little in its arguments: in the loops, or with their
// variables alive, it cost the usual path 2 to 40 % by the registers that it took.
template <class GT, class Tab>
__device__ __noinline__ void marked_units(const Tab *tab, const AdamState *st,
                                          const StepScalars *sc, int64_t tiles, int CW,
                                          uint32_t drained)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    __syncwarp();
    if (drained && !mbar_wait(drained, 0, st->limit_ns)) {
        if (lane == 0) step_lost(st->steps, 0);
        return;
    }
    int64_t t = blockIdx.x < tiles ? blockIdx.x : tiles;
    while (t <= tiles) {
        const int64_t un = t * CW + warp;
        const bool own = t < tiles || blockIdx.x == gridDim.x - 1;
        if (own && un * FC_STATE_BLOCK < st->N &&
            __float_as_int(__ldcg(st->r_scale + un)) < 0) {
            UnitRegs<8> u;
            load_unit<GT, 8>(*tab, *st, un, lane, u);
            adam8_unit<false, true>(u.g, u.d, st->h, *sc, un * FC_STATE_BLOCK + 4 * lane, u.w,
                                    u.mq, u.rq, u.ms, u.rs);
            store_unit<8>(*st, false, un, lane, u);
        }
        // behind the CTA's last tile comes what is left behind all of them
        t = t < tiles && t + gridDim.x > tiles ? tiles : t + gridDim.x;
    }
}

// False: the unit has been marked.
template <int BITS>
__device__ __forceinline__ bool update_unit(const AdamState &st, const StepScalars &sc, int64_t un,
                                            int lane, UnitRegs<BITS> &u)
{
    if (!sc.skip) {
        if constexpr (BITS == 32) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                adam1(u.g[j], u.d[j], st.h, sc, u.m[j], u.v[j], u.w[j]);
        } else if (!adam8_unit<false>(u.g, u.d, st.h, sc, un * FC_STATE_BLOCK + 4 * lane, u.w,
                                      u.mq, u.rq, u.ms, u.rs)) {
            mark_unit(st, un, lane, u.rs);
            return false;
        }
    }
    store_unit<BITS>(st, sc.skip, un, lane, u);
    return true;
}

// ---- direct kernel ----------------------------------------------------------------------

template <class GT, int BITS, class Tab>
__global__ void __launch_bounds__(FC_ADAM_BLOCK)
    k_adamw_direct(const __grid_constant__ Tab tab, const __grid_constant__ AdamState st)
{
    __shared__ StepScalars sh;
    wait_for_prior_grid();
    allow_dependent_launch();
    const int lane = threadIdx.x & 31;
    const int64_t units = (st.N + FC_STATE_BLOCK - 1) / FC_STATE_BLOCK;
    const int64_t stride = (int64_t)gridDim.x * (FC_ADAM_BLOCK / 32);
    int64_t un = (int64_t)blockIdx.x * (FC_ADAM_BLOCK / 32) + (threadIdx.x >> 5);
    UnitRegs<BITS> u;
    // the first unit's loads before the step's scalars are awaited
    if (un < units) load_unit<GT, BITS>(tab, st, un, lane, u);
    if (threadIdx.x < 32) load_scalars<BITS>(sh, st);
    __syncthreads();
    const StepScalars sc = sh;
    unsigned arrived = 0;
    if (threadIdx.x == 0 && !sc.skip) arrived = arrive_step(st.steps);
    bool done = true;
    while (un < units) {
        done &= update_unit<BITS>(st, sc, un, lane, u);
        un += stride;
        if (un < units) load_unit<GT, BITS>(tab, st, un, lane, u);
    }
    if (threadIdx.x == 0 && !sc.skip) count_step(st.steps, arrived);
    if constexpr (BITS == 8)
        if (!done)
            marked_units<GT>(&tab, &st, &sh, units / (FC_ADAM_BLOCK / 32), FC_ADAM_BLOCK / 32, 0);
}

// ---- ring kernel ------------------------------------------------------------------------
//
// One CTA per SM.  A tile is CW units; a stage holds a tile's weights and
// moments.  One thread copies tiles in (bulk copies counted on the stage's
// `full` barrier), CW warps update one unit each in place, and the same
// thread copies the stage out again once all have arrived at its `done`
// barrier; a stage is refilled when its copy out has read it.  That thread also
// counts the step: the warps have no registers to spare.  The gradient
// comes straight from its tensor (any alignment), one tile ahead in
// registers, and the low-precision copy goes out from registers.  A unit with
// 8-bit moments that does not fit the usual units is left as it is, its r_scale's
// sign marks it, and its warp does it from global memory at the end.

template <int BITS, int CW>
struct RingStage {
    static constexpr int T = CW * FC_STATE_BLOCK;
    static constexpr int WB = T * 4;
    static constexpr int AB = BITS == 32 ? T * 4 : T;
    static constexpr int BYTES = WB + 2 * AB;
};

template <class GT, int BITS, int CW, bool SHIFTED, class Tab>
__global__ void __launch_bounds__((CW + 1) * 32)
    k_adamw_ring(const __grid_constant__ Tab tab, const __grid_constant__ AdamState st,
                 const int64_t tiles, const int S)
{
    using St = RingStage<BITS, CW>;
    extern __shared__ __align__(128) unsigned char stages[];
    __shared__ uint64_t bars[2 * 32];  // full [S], done [S]
    __shared__ uint64_t drained;       // all copies out are done
    __shared__ int large[CW];          // whether a warp has marked units
    __shared__ StepScalars sh;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(smem_u32(&bars[s]), 1);
            mbar_init(smem_u32(&bars[S + s]), CW);
        }
        mbar_init(smem_u32(&drained), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (threadIdx.x < CW) large[threadIdx.x] = 0;
    __syncthreads();
    wait_for_prior_grid();
    allow_dependent_launch();
    const int64_t n = blockIdx.x < tiles ? (tiles - 1 - blockIdx.x) / gridDim.x + 1 : 0;

    if (warp == CW) {
        if (lane != 0) return;
        const char *const gw = reinterpret_cast<const char *>(st.w);
        const char *const ga = BITS == 32 ? reinterpret_cast<const char *>(st.m)
                                          : reinterpret_cast<const char *>(st.m8);
        const char *const gb = BITS == 32 ? reinterpret_cast<const char *>(st.v)
                                          : reinterpret_cast<const char *>(st.r8);
        auto fill = [&](int64_t it) {
            const int s = (int)(it % S);
            const int64_t t = blockIdx.x + it * gridDim.x;
            const uint32_t full = smem_u32(&bars[s]);
            const uint32_t to = smem_u32(stages) + (uint32_t)s * St::BYTES;
            if (t == st.drop) return;
            mbar_expect_tx(full, St::BYTES);
            bulk_g2s(to, gw + t * St::WB, St::WB, full);
            bulk_g2s(to + St::WB, ga + t * St::AB, St::AB, full);
            bulk_g2s(to + St::WB + St::AB, gb + t * St::AB, St::AB, full);
        };
        int64_t filled = 0;
        unsigned arrived = 0;
        int skip = 0;
        for (; filled < n && filled < S; ++filled) fill(filled);
        for (int64_t it = 0; it < n; ++it) {
            const int s = (int)(it % S);
            const bool done = mbar_wait(smem_u32(&bars[S + s]), (uint32_t)(it / S) & 1, st.limit_ns);
            if (it == 0) {
                // the consumers have read the step's scalars (long ago, if one of
                // them has given up)
                skip = *(volatile int *)&sh.skip;
                if (!skip) arrived = arrive_step(st.steps);
            }
            if (!done) {
                // not expected: no more copies out; those coming in must have
                // landed before the shared memory may go
                step_lost(st.steps, skip);
                for (int64_t j = it; j < filled; ++j)
                    mbar_wait(smem_u32(&bars[j % S]), (uint32_t)(j / S) & 1, st.limit_ns);
                break;
            }
            if (!skip) {
                const int64_t t = blockIdx.x + it * gridDim.x;
                const uint32_t from = smem_u32(stages) + (uint32_t)s * St::BYTES;
                bulk_s2g(const_cast<char *>(gw) + t * St::WB, from, St::WB);
                bulk_s2g(const_cast<char *>(ga) + t * St::AB, from + St::WB, St::AB);
                bulk_s2g(const_cast<char *>(gb) + t * St::AB, from + St::WB + St::AB, St::AB);
            }
            bulk_commit();
            // the stage before this one has been read by now, or nearly
            if (it >= 1 && filled < n) {
                bulk_wait_read<1>();
                fill(filled++);
            }
        }
        // while the last copies out are on their way
        if (!skip) count_step(st.steps, arrived);
        bulk_wait_all();
        mbar_arrive(smem_u32(&drained));
        return;
    }

    // the consumers
    int sg = 0;
    UnitGrad<GT, SHIFTED> next;
    float nms = 0.f, nrs = 0.f;
    auto unit = [&](int64_t it) { return (blockIdx.x + it * gridDim.x) * CW + warp; };
    auto load = [&](int64_t un) {
        load_unit_grad(tab, un * FC_STATE_BLOCK, lane, sg, next);
        if constexpr (BITS == 8) {
            nms = __ldcs(st.m_scale + un);
            nrs = __ldcs(st.r_scale + un);
        }
    };
    if (n > 0) load(unit(0));
    if (warp == 0) load_scalars<BITS>(sh, st);
    asm volatile("bar.sync 1, %0;" ::"n"(CW * 32) : "memory");
    const StepScalars sc = sh;
    int s = 0;
    uint32_t phase = 0;
    for (int64_t it = 0; it < n; ++it) {
        unsigned char *const stage = stages + (size_t)s * St::BYTES;
        // given up, it is missed at the stage's `done` barrier
        if (!mbar_wait(smem_u32(&bars[s]), phase, st.limit_ns)) return;
        const int64_t un = unit(it);
        const int64_t lo = un * FC_STATE_BLOCK;
        const UnitGrad<GT, SHIFTED> cur = next;
        float ms = nms, rs = nrs;
        if (it + 1 < n) load(unit(it + 1));
        const int at = warp * 64 + lane;  // in groups of 4 elements
        float4 *const sw = reinterpret_cast<float4 *>(stage) + at;
        float w[8];
        {
            const float4 a = sw[0], b = sw[32];
            w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
            w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
        }
        if (!sc.skip) {
            if constexpr (BITS == 32) {
                float4 *sm = reinterpret_cast<float4 *>(stage + St::WB) + at;
                float4 *sv = reinterpret_cast<float4 *>(stage + St::WB + St::AB) + at;
                float4 m4[2] = {sm[0], sm[32]}, v4[2] = {sv[0], sv[32]};
                float g[8], d[8];
                if (cur.d >= 0) {
                    cur.unpack(g);
#pragma unroll
                    for (int j = 0; j < 8; ++j) d[j] = cur.decay;
                } else {
                    gather_unit<GT>(tab, st.N, lo, lane, cur.sg, g, d);
                }
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    adam1(g[j], d[j], st.h, sc, (&m4[j >> 2].x)[j & 3], (&v4[j >> 2].x)[j & 3],
                          w[j]);
                sm[0] = m4[0];
                sm[32] = m4[1];
                sv[0] = v4[0];
                sv[32] = v4[1];
            } else {
                uint32_t *qm = reinterpret_cast<uint32_t *>(stage + St::WB) + at;
                uint32_t *qr =
                    reinterpret_cast<uint32_t *>(stage + St::WB + St::AB) + at;
                uint32_t mq[2] = {qm[0], qm[32]}, rq[2] = {qr[0], qr[32]};
                float g[8];
                bool fits;
                if (cur.d >= 0) {
                    cur.unpack(g);
                    fits = adam8_unit<true>(g, &cur.decay, st.h, sc, lo + 4 * lane, w, mq, rq, ms,
                                            rs);
                } else {
                    float d[8];
                    gather_unit<GT>(tab, st.N, lo, lane, cur.sg, g, d);
                    fits = adam8_unit<false>(g, d, st.h, sc, lo + 4 * lane, w, mq, rq, ms, rs);
                }
                if (!fits) {
                    // the stage goes out as it came; the mark is taken up at the end
                    mark_unit(st, un, lane, rs);
                    if (lane == 0) large[warp] = 1;
                    goto done;
                }
                qm[0] = mq[0];
                qm[32] = mq[1];
                qr[0] = rq[0];
                qr[32] = rq[1];
                if (lane == 0) {
                    __stcs(st.m_scale + un, ms);
                    __stcs(st.r_scale + un, rs);
                }
            }
            sw[0] = make_float4(w[0], w[1], w[2], w[3]);
            sw[32] = make_float4(w[4], w[5], w[6], w[7]);
        }
        if (st.low) {
            store_low4(st.low, st.ltype, lo + 4 * lane, w);
            store_low4(st.low, st.ltype, lo + 4 * lane + 128, w + 4);
        }
    done:
        fence_async_shared();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bars[S + s]));
        if (++s == S) {
            s = 0;
            phase ^= 1;
        }
    }
    // what is left behind the last whole tile, by the CTA with the fewest tiles
    if (blockIdx.x == gridDim.x - 1) {
        for (int64_t un = tiles * CW + warp; un * FC_STATE_BLOCK < st.N; un += CW) {
            UnitRegs<BITS> u;
            load_unit<GT, BITS>(tab, st, un, lane, u);
            if (!update_unit<BITS>(st, sc, un, lane, u) && lane == 0) large[warp] = 1;
        }
    }
    if constexpr (BITS == 8) {
        __syncwarp();
        if (large[warp]) marked_units<GT>(&tab, &st, &sh, tiles, CW, smem_u32(&drained));
    }
}

// ---- launches ---------------------------------------------------------------------------

// Passes the table by address: the launch copies it once into the launch's
// own parameters.
template <class Tab, class... Args>
static cudaError_t launch_table(const void *kernel, unsigned grid, unsigned block, size_t smem,
                                cudaStream_t s, const Tab &tab, const Args &...args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    void *p[] = {const_cast<Tab *>(&tab), const_cast<Args *>(&args)...};
    return cudaLaunchKernelExC(&cfg, kernel, p);
}

// Whether the gradient of some whole unit starts off a boundary of 4 elements.
template <class GT, class Tab>
static bool any_shifted(const Tab &tab)
{
    for (int l = 0; l < tab.L; ++l)
        if (tab.off[l + 1] - tab.off[l] >= FC_STATE_BLOCK &&
            (((uintptr_t)tab.ptr[l] / sizeof(GT) - (uintptr_t)tab.off[l]) & 3))
            return true;
    return false;
}

// Test hook (fc_test_adamw_loss): a tile that the next streamed launch does not copy
// in, and the limit of that launch's waits.
static std::atomic<int64_t> g_drop_tile{-1};
static std::atomic<uint64_t> g_drop_limit_ns{0};

template <class GT, int BITS, bool SHIFTED, class Tab>
static cudaError_t launch_ring(const Tab &tab, AdamState st, cudaStream_t s)
{
    constexpr int CW = BITS == 32 ? FC_ADAM_CW32 : SHIFTED ? FC_ADAM_CW8_SHIFTED : FC_ADAM_CW8;
    constexpr int S = BITS == 32 ? FC_ADAM_S32 : FC_ADAM_S8;
    static_assert(S >= 2 && S <= 32, "a stage is refilled while the next one is worked on");
    using St = RingStage<BITS, CW>;
    const size_t smem = (size_t)S * St::BYTES;
    const int64_t tiles = st.N / St::T;
    st.drop = g_drop_tile.exchange(-1);
    if (st.drop >= 0) {
        st.drop = std::min(st.drop, tiles - 1);
        st.limit_ns = g_drop_limit_ns.load();
    }
    const void *ring = (const void *)k_adamw_ring<GT, BITS, CW, SHIFTED, Tab>;
    cudaError_t e =
        cudaFuncSetAttribute(ring, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    const int grid = grid_for(ring, (CW + 1) * 32, smem, tiles);
    return launch_table(ring, (unsigned)grid, (CW + 1) * 32, smem, s, tab, st, tiles, S);
}

template <class GT, int BITS, class Tab>
static cudaError_t launch_typed(const Tab &tab, const AdamState &st, cudaStream_t s)
{
    const int64_t units = (st.N + FC_STATE_BLOCK - 1) / FC_STATE_BLOCK;
    const int64_t ctas = (units + FC_ADAM_BLOCK / 32 - 1) / (FC_ADAM_BLOCK / 32);
    const void *direct = (const void *)k_adamw_direct<GT, BITS, Tab>;
    const int resident = grid_for(direct, FC_ADAM_BLOCK, 0, INT64_MAX);
    // The direct kernel serves what its resident CTAs take in one round (0.93M
    // elements).  Measured, direct against ring: fp32 4.8 and 6.0 us at 0.8M
    // elements, 7.9 and 6.3 us at 1.1M; 8-bit 4.3 and 5.4 us, 7.0 and 6.5 us.
    if (ctas <= resident)
        return launch_table(direct, (unsigned)ctas, FC_ADAM_BLOCK, 0, s, tab, st);
    if (any_shifted<GT>(tab)) return launch_ring<GT, BITS, true>(tab, st, s);
    return launch_ring<GT, BITS, false>(tab, st, s);
}

template <int BITS, class Tab>
static cudaError_t launch_bits(const Tab &tab, int gtype, const AdamState &st, cudaStream_t s)
{
    if (gtype == FC_TYPE_F32) return launch_typed<float, BITS>(tab, st, s);
    if (gtype == FC_TYPE_F16) return launch_typed<__half, BITS>(tab, st, s);
    return launch_typed<__nv_bfloat16, BITS>(tab, st, s);
}

template <class Tab>
cudaError_t launch_adamw(const Tab &tab, int gtype, int64_t N, const AdamHyper &h,
                         const float *scale, float *w, void *low, int ltype, float *m, float *v,
                         int32_t *steps, cudaStream_t s)
{
    AdamState st = {};
    st.N = N;
    st.h = h;
    st.scale = scale;
    st.w = w;
    st.low = low;
    st.ltype = ltype;
    st.m = m;
    st.v = v;
    st.steps = steps;
    st.limit_ns = FC_ADAM_WAIT_NS;
    st.drop = -1;
    return launch_bits<32>(tab, gtype, st, s);
}

template <class Tab>
cudaError_t launch_adamw8(const Tab &tab, int gtype, int64_t N, const AdamHyper &h,
                          const float *scale, float *w, void *low, int ltype, uint8_t *m8,
                          float *m_scale, uint8_t *r8, float *r_scale, int32_t *steps,
                          uint64_t seed, cudaStream_t s)
{
    AdamState st = {};
    st.N = N;
    st.h = h;
    // a normal number: the quotient's reciprocal takes a subnormal one for zero, and
    // an element that never had a gradient would divide 0 by 0
    st.h.eps = std::max(h.eps * FC_ADAM8_UNIT, 0x1p-126f);
    st.scale = scale;
    st.w = w;
    st.low = low;
    st.ltype = ltype;
    st.m8 = m8;
    st.r8 = r8;
    st.m_scale = m_scale;
    st.r_scale = r_scale;
    st.steps = steps;
    st.seed = seed;
    st.limit_ns = FC_ADAM_WAIT_NS;
    st.drop = -1;
    return launch_bits<8>(tab, gtype, st, s);
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

extern "C" fc_status fc_test_adamw_loss(int64_t tile, uint64_t wait_limit_ns)
{
    if (tile >= 0 && (wait_limit_ns < 1000000ull || wait_limit_ns > 2000000000ull))
        return fc::set_error(FC_ERR_INVALID_ARG, "wait_limit_ns must be in [1 ms, 2 s]");
    fc::g_drop_limit_ns.store(wait_limit_ns);
    fc::g_drop_tile.store(tile < 0 ? -1 : tile);
    return FC_OK;
}
