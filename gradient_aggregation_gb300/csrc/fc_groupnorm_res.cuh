// Group norm with the maps held in shared memory between the statistics and the
// result: every element crosses HBM once each way.
//
// A cluster of K blocks holds a slab of whole groups of one sample, each block a
// part of the positions.  A thread copies its vectors into slots of its own
// (cp.async), so reading them back needs no barrier, and nothing of the wait for
// memory holds up another warp.  Sums go from the threads' registers to shared
// memory (one value for each group that a vector touches), from there by one warp a
// group to the block's sum, and from block to block through the cluster's shared
// memory.  A cluster goes from sample to sample; a slot whose result is on its way takes
// the next sample's vector, and several blocks to an SM keep loads, arithmetic and
// stores of different samples going side by side.
//
// 64 x 4096 x 512 bf16 with SiLU: 108 us forward (floor 79) and 212 backward (118); read two
// and three times over, without holding the maps, 245 and 380.  A copy through the same
// slots takes 97 us, so the forward pass is bound by how many bytes they keep in flight; the
// backward pass by its instructions, of which 10 warps an SM issue in 0.45 of the cycles.
#pragma once

#include "fc_groupnorm.cuh"

namespace fc {

struct GnPlan {
    int threads, K, logk;  // of a block; blocks of a cluster
    int sc, nslab;         // channels of a slab; slabs
    int cpg, gs, ns;       // channels of a group; groups of a slab; that a vector touches at most
    int V, R;              // vectors of a slab's row; rows that a block's threads hold at a time
    int divv, divn;        // t / V = t * divv >> 20 (t < 1024), and by a group's vectors
    int rows, iters;       // positions of a block; slots of a thread
    int per;               // clusters that share a slab's samples
    int part;              // bytes of the slots of one tensor
    float total;           // elements of a group
    size_t smem;
};

#define FC_GN_THREADS 512   // of a block at most
// of an SM that the registers leave room for: the backward pass holds three times the
// values a channel, and with 80 registers it spilled
#define FC_GN_RESIDENT 768
#define FC_GN_RESIDENT_BWD 512

// Where a thread of a resident kernel stands.
struct GnSpot {
    int rank, v, r;      // block of the cluster; vector and row of the thread
    int slab, gs;        // the block's slab, its groups (the last slab may have fewer)
    int g0, off;         // group of the vector's first channel, its place there
    int have, rows;      // the block's positions, the thread's
    int64_t row;         // the thread's first position
    int first;           // the cluster's first sample
    bool on;
};

template <int NE, bool ONE>
__device__ __forceinline__ GnSpot gn_spot(const GnPlan &p, const GnShape &n)
{
    GnSpot s;
    s.rank = (int)blockIdx.x & (p.K - 1);
    s.r = (int)threadIdx.x * p.divv >> 20;
    s.v = (int)threadIdx.x - s.r * p.V;
    const int cluster = (int)(blockIdx.x >> p.logk);
    s.first = cluster / p.nslab;
    s.slab = cluster - s.first * p.nslab;
    s.gs = min(p.gs, n.groups - s.slab * p.gs);
    s.on = s.r < p.R && s.v * NE < s.gs * p.cpg;
    if (ONE) {
        s.g0 = s.v * p.divn >> 20;
        s.off = 0;
    } else {
        s.g0 = s.v * NE / p.cpg;
        s.off = s.v * NE - s.g0 * p.cpg;
    }
    const int row0 = s.rank * p.rows;
    s.have = max(0, min(p.rows, (int)n.positions - row0));
    s.row = row0 + s.r;
    s.rows = s.on && s.r < s.have ? (s.have - s.r + p.R - 1) / p.R : 0;
    return s;
}

// Positions of block j of the cluster.
__device__ __forceinline__ float gn_rows(const GnPlan &p, const GnShape &n, int j)
{
    return (float)max(0, min(p.rows, (int)n.positions - j * p.rows));
}

// Copies AB bytes into a slot of the thread's own, where they are there once the copies
// have been waited for.
template <int AB>
__device__ __forceinline__ void gn_copy(char *to, const char *from)
{
    if constexpr (AB == 16)
        cp_async16((uint32_t)__cvta_generic_to_shared(to), from);
    else if constexpr (AB == 8)
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(
                         (uint32_t)__cvta_generic_to_shared(to)),
                     "l"(from)
                     : "memory");
    else if constexpr (AB == 4)
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(
                         (uint32_t)__cvta_generic_to_shared(to)),
                     "l"(from)
                     : "memory");
    else  // there on return: no asynchronous copy is as small
        *reinterpret_cast<unsigned short *>(to) = __ldcs(reinterpret_cast<const unsigned short *>(from));
}

// A thread's vectors of one tensor: the first of sample 0 and slab 0, and the bytes from
// one to the next.
struct GnWalk {
    char *p;
    int64_t step;
};

template <class T, int NE>
__device__ __forceinline__ GnWalk gn_walk(const GnImages &x, const GnSpot &s, const GnPlan &p)
{
    GnWalk w;
    w.p = (char *)x.p + (s.row * x.ld + s.v * NE) * (int)sizeof(T);
    w.step = p.R * x.ld * (int)sizeof(T);
    return w;
}

// The thread's first vector of a sample and slab.
template <class T>
__device__ __forceinline__ char *gn_at(const GnWalk &w, const GnImages &x, int n, int c0)
{
    return w.p + (n * x.ss + c0) * (int)sizeof(T);
}

// ---- values of a group among the threads --------------------------------------------------
//
// ONE: every vector lies in one group.  Otherwise a thread has a value for each group
// that its vector touches, value j of thread t at [j * threads + t].

// Calls f(index, elements, r) for each value that the threads have for group g, 32 lanes
// side by side.
template <int NE, bool ONE, class F>
__device__ __forceinline__ void gn_values(const GnPlan &p, int g, F f)
{
    const int lane = threadIdx.x & 31;
    int lo, nv, r, dr, j0 = 0;
    if (ONE) {
        nv = p.cpg / NE;
        lo = g * nv;
        r = lane * p.divn >> 20;
        dr = 32 * p.divn >> 20;
    } else {
        lo = g * p.cpg / NE;
        nv = ((g + 1) * p.cpg - 1) / NE - lo + 1;
        r = lane / nv;
        dr = 32 / nv;
        j0 = g - lo * NE / p.cpg;
    }
    int v = lane - r * nv;
    const int dv = 32 - dr * nv;
    while (r < p.R) {
        int at = r * p.V + lo + v, n = NE;
        if (!ONE) {
            if (v == 0) at += j0 * (int)blockDim.x;
            n = min((lo + v + 1) * NE, (g + 1) * p.cpg) - max((lo + v) * NE, g * p.cpg);
        }
        f(at, n, r);
        r += dr;
        v += dv;
        if (v >= nv) {
            v -= nv;
            ++r;
        }
    }
}

// Sum over the K lanes of a cluster's blocks.
__device__ __forceinline__ float gn_blocks_sum(float x, int K)
{
    for (int o = K >> 1; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

__device__ __forceinline__ void gn_block_or_cluster_sync(int K)
{
    if (K > 1)
        cluster_sync();
    else
        __syncthreads();
}

template <class T, int AB, int ACT, bool ONE>
__global__ void __launch_bounds__(FC_GN_RESIDENT)
    k_gn_fwd(const __grid_constant__ GnForward a, const __grid_constant__ GnPlan p)
{
    using V = Gv<T, AB>;
    using Raw = typename V::Raw;
    constexpr int NE = V::NE, NP = V::NP;
    extern __shared__ uint4 dyn[];
    const int T_ = (int)blockDim.x, hop = T_ * AB;
    char *const mine = reinterpret_cast<char *>(dyn) + (int)threadIdx.x * AB;
    float *const s_mean = reinterpret_cast<float *>(reinterpret_cast<char *>(dyn) + p.part);
    float *const s_sq = s_mean + p.ns * T_, *const g = s_sq + p.ns * T_;
    const GnSpot s = gn_spot<NE, ONE>(p, a.n);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = T_ >> 5;
    const int half = min((p.iters + 1) >> 1, s.rows);
    const GnWalk x = gn_walk<T, NE>(a.x, s, p), y = gn_walk<T, NE>(a.y, s, p);
    const int q0 = s.first, c0 = s.slab * p.sc;
    const int base = s.have / p.R, rest = s.have - base * p.R;  // threads r >= rest: base rows
    const float have = (float)s.rows, inv = s.rows > 0 ? 1.f / have : 0.f;
    const float block = s.have > 0 ? 1.f / (float)(s.have * p.cpg) : 0.f, all = 1.f / p.total;
    wait_for_prior_grid();
    allow_dependent_launch();
    auto copy = [&](int n, int first, int last) {
        const char *q = gn_at<T>(x, a.x, n, c0) + first * x.step;
        char *to = mine + first * hop;
#pragma unroll 4
        for (int k = first; k < last; ++k, to += hop, q += x.step) gn_copy<AB>(to, q);
        cp_async_commit();
    };
    copy(q0, 0, half);
    copy(q0, half, s.rows);
    F2 w[NP], b[NP];
    if (s.on) {
        gn_params<T, NE>(a.weight, a.ptype, c0 + s.v * NE, 1.f, w);
        gn_params<T, NE>(a.bias, a.ptype, c0 + s.v * NE, 0.f, b);
    }
    for (int n = q0;; n += p.per) {
        // per channel of the thread: a pivot, and the sums of x - p and (x - p)^2 (the
        // error is as many roundings as the thread has rows, even if p lies far from all
        // other values, as p itself adds as much to the sum)
        F2 neg[NP], sum[NP], sq[NP];
#pragma unroll
        for (int j = 0; j < NP; ++j) sum[j] = sq[j] = f2(0.f, 0.f);
        auto add = [&](int first, int last) {
            const char *from = mine + first * hop;
#pragma unroll 4
            for (int k = first; k < last; ++k, from += hop) {
                F2 f[NP];
                V::get(*reinterpret_cast<const Raw *>(from), f);
#pragma unroll
                for (int j = 0; j < NP; ++j) {
                    const F2 d = add2(f[j], neg[j]);
                    sum[j] = add2(sum[j], d);
                    sq[j] = fma2(d, d, sq[j]);
                }
            }
        };
        cp_async_wait<1>();
        V::get(*reinterpret_cast<const Raw *>(mine), neg);
#pragma unroll
        for (int j = 0; j < NP; ++j) neg[j] = neg2(neg[j]);
        add(0, half);
        cp_async_wait<0>();
        add(half, s.rows);
        // of each of the vector's pieces: the mean, and the squares about it
        if (s.rows > 0) {
#pragma unroll
            for (int j = 0; j < NP; ++j) {
                const F2 ms = mul2(sum[j], f2(inv, inv));
                sq[j] = fma2(neg2(ms), sum[j], sq[j]);
                sum[j] = add2(ms, neg2(neg[j]));
            }
        }
        if (s.on) {
            gn_pieces<NE, ONE>(s.off, p.cpg, [&](int j, int first, int last) {
                const float m = s.rows > 0
                                    ? gn_add<NE, ONE>(sum, first, last) / (float)(last - first) : 0.f;
                F2 q[NP];
#pragma unroll
                for (int k = 0; k < NP; ++k) {
                    const F2 d = add2(sum[k], f2(-m, -m));
                    q[k] = fma2(mul2(d, d), f2(have, have), sq[k]);
                }
                s_mean[j * T_ + threadIdx.x] = m;
                s_sq[j * T_ + threadIdx.x] = s.rows > 0 ? gn_add<NE, ONE>(q, first, last) : 0.f;
            });
        }
        __syncthreads();
        for (int k = warp; k < s.gs; k += warps) {
            float t = 0.f, q = 0.f;
            gn_values<NE, ONE>(p, k, [&](int at, int e, int r) {
                t = fmaf((float)((base + (r < rest)) * e), s_mean[at], t);
            });
            const float m = warp_sum_f32(t) * block;
            gn_values<NE, ONE>(p, k, [&](int at, int e, int r) {
                const float d = s_mean[at] - m, c = (float)((base + (r < rest)) * e);
                q += c > 0.f ? fmaf(c * d, d, s_sq[at]) : 0.f;
            });
            q = warp_sum_f32(q);
            if (lane == 0) {
                g[k] = m;
                g[p.gs + k] = q;
            }
        }
        gn_block_or_cluster_sync(p.K);
        // a lane for each block of the cluster
        for (int k = threadIdx.x; k < (((s.gs << p.logk) + 31) & ~31); k += T_) {
            const int at = min(k >> p.logk, s.gs - 1), j = k & (p.K - 1);
            float m, q;
            if (p.K > 1) {
                const float bm = ld_cluster_f32(g + at, j), bq = ld_cluster_f32(g + p.gs + at, j);
                const float e = gn_rows(p, a.n, j) * (float)p.cpg;
                m = gn_blocks_sum(e * bm, p.K) * all;
                const float d = bm - m;
                q = gn_blocks_sum(fmaf(e * d, d, bq), p.K);
            } else {
                m = g[at];
                q = g[p.gs + at];
            }
            if (j == 0 && k >> p.logk < s.gs) {
                const float r = 1.f / sqrtf(q * all + a.eps);
                g[2 * p.gs + at] = -m;
                g[3 * p.gs + at] = r;
                if (s.rank == 0 && a.mean) {
                    const int64_t to = (int64_t)n * a.n.groups + s.slab * p.gs + at;
                    a.mean[to] = m;
                    a.rstd[to] = r;
                }
            }
        }
        __syncthreads();
        if (p.K > 1) cluster_arrive_relaxed();  // the other blocks may change what was read here
        const bool more = n + p.per < a.n.samples;
        if (s.on) {
            GnOf<NE, ONE> m, r;
            m.load(s.g0, s.off, p.cpg, [&](int k) { return g[2 * p.gs + k]; });
            r.load(s.g0, s.off, p.cpg, [&](int k) { return g[3 * p.gs + k]; });
            F2 wk[NP];
#pragma unroll
            for (int j = 0; j < NP; ++j) wk[j] = mul2(r[j], w[j]);
            char *const to_y = gn_at<T>(y, a.y, n, c0);
            const char *const next = gn_at<T>(x, a.x, n + p.per, c0);
            // a slot that has been read takes the next sample's vector
            auto put = [&](int first, int last, auto ahead) {
                char *slot = mine + first * hop;
                char *to = to_y + first * y.step;
                const char *q = next + first * x.step;
#pragma unroll 4
                for (int k = first; k < last; ++k, slot += hop, to += y.step) {
                    F2 f[NP];
                    V::get(*reinterpret_cast<const Raw *>(slot), f);
#pragma unroll
                    for (int j = 0; j < NP; ++j) f[j] = fma2(add2(f[j], m[j]), wk[j], b[j]);
                    gn_act<ACT, NP>(f);
                    __stcs(reinterpret_cast<Raw *>(to), V::put(f));
                    if constexpr (decltype(ahead)::value) {
                        gn_copy<AB>(slot, q);
                        q += x.step;
                    }
                }
                if constexpr (decltype(ahead)::value) cp_async_commit();
            };
            if constexpr (AB == 2) {
                put(0, s.rows, Yes<false>());
                if (more) copy(n + p.per, 0, s.rows);
            } else if (more) {
                put(0, half, Yes<true>());
                put(half, s.rows, Yes<true>());
            } else {
                put(0, s.rows, Yes<false>());
            }
        }
        if (p.K > 1) cluster_wait();
        if (!more) break;
    }
}

// The channels' sums: over the block's rows of threads (in place of the maps' slots),
// over the cluster, into this cluster's set.
template <class T, int NE>
__device__ __forceinline__ void gn_leave_sums(const GnBackward &a, const GnPlan &p, const GnSpot &s,
                                              float *all, const F2 (&th)[(NE + 1) / 2],
                                              const F2 (&td)[(NE + 1) / 2])
{
    const int T_ = (int)blockDim.x, plane = p.R * p.sc;
    float *const some = all + 2 * plane;
    __syncthreads();
    if (s.on) {
#pragma unroll
        for (int e = 0; e < NE; ++e) {
            all[(int)threadIdx.x * NE + e] = gn_element<NE>(th, e);
            all[plane + (int)threadIdx.x * NE + e] = gn_element<NE>(td, e);
        }
    }
    __syncthreads();
    const int teams = max(1, min(p.R, T_ / (2 * p.sc)));
    for (int i = threadIdx.x; i < 2 * p.sc * teams; i += T_) {
        const int k = i / (2 * p.sc), j = i - k * 2 * p.sc;
        const float *q = all + (j >= p.sc ? plane + j - p.sc : j) + k * p.sc;
        float v = 0.f;
#pragma unroll 4
        for (int r = k; r < p.R; r += teams, q += teams * p.sc) v += *q;
        some[i] = v;
    }
    __syncthreads();
    float *const sums = all;
    for (int j = threadIdx.x; j < 2 * p.sc; j += T_) {
        float v = 0.f;
        for (int k = 0; k < teams; ++k) v += some[k * 2 * p.sc + j];
        sums[j] = v;
    }
    gn_block_or_cluster_sync(p.K);
    const int64_t padded = (a.n.channels + 7) & ~7;
    for (int j = s.rank * T_ + (int)threadIdx.x; j < 2 * p.sc; j += p.K * T_) {
        float v = 0.f;
        if (p.K > 1) {
#pragma unroll 4
            for (int k = 0; k < p.K; ++k) v += ld_cluster_f32(sums + j, k);
        } else {
            v = sums[j];
        }
        const int which = j >= p.sc, c = j - which * p.sc;
        if (c < s.gs * p.cpg)
            a.ws[(which * p.per + s.first) * padded + s.slab * p.sc + c] = v;
    }
    if (p.K > 1) cluster_sync();  // no block leaves while another reads its sums
}

template <class T, int AB, int ACT, bool ONE>
__global__ void __launch_bounds__(FC_GN_RESIDENT_BWD)
    k_gn_bwd(const __grid_constant__ GnBackward a, const __grid_constant__ GnPlan p)
{
    using V = Gv<T, AB>;
    using Raw = typename V::Raw;
    constexpr int NE = V::NE, NP = V::NP;
    extern __shared__ uint4 dyn[];
    const int T_ = (int)blockDim.x, hop = T_ * AB;
    char *const mine = reinterpret_cast<char *>(dyn) + (int)threadIdx.x * AB;
    float *const s_1 = reinterpret_cast<float *>(reinterpret_cast<char *>(dyn) + 2 * p.part);
    float *const s_2 = s_1 + p.ns * T_, *const g = s_2 + p.ns * T_;
    // the groups' mean and rstd, copied like the maps
    float *own = g + 4 * p.gs + (int)threadIdx.x, *ahead_own = own + 2 * p.ns * T_;
    const GnSpot s = gn_spot<NE, ONE>(p, a.n);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = T_ >> 5;
    const int half = min((p.iters + 1) >> 1, s.rows);
    const GnWalk x = gn_walk<T, NE>(a.x, s, p), dy = gn_walk<T, NE>(a.dy, s, p);
    const GnWalk dx = gn_walk<T, NE>(a.dx, s, p);
    const int q0 = s.first, c0 = s.slab * p.sc;
    const float inv = -1.f / p.total;
    wait_for_prior_grid();
    allow_dependent_launch();
    auto copy = [&](int n, int first, int last) {
        const char *q = gn_at<T>(x, a.x, n, c0) + first * x.step;
        const char *u = gn_at<T>(dy, a.dy, n, c0) + first * dy.step;
        char *to = mine + first * hop;
#pragma unroll 4
        for (int k = first; k < last; ++k, to += hop, q += x.step, u += dy.step) {
            gn_copy<AB>(to, q);
            gn_copy<AB>(to + p.part, u);
        }
        cp_async_commit();
    };
    auto copy_stats = [&](int n, float *to) {
        if (!s.on) return;
        const int64_t at = (int64_t)n * a.n.groups + s.slab * p.gs + s.g0;
        gn_pieces<NE, ONE>(s.off, p.cpg, [&](int j, int, int) {
            gn_copy<4>(reinterpret_cast<char *>(to + 2 * j * T_),
                       reinterpret_cast<const char *>(a.mean + at + j));
            gn_copy<4>(reinterpret_cast<char *>(to + (2 * j + 1) * T_),
                       reinterpret_cast<const char *>(a.rstd + at + j));
        });
    };
    copy_stats(q0, own);
    copy(q0, 0, half);
    copy(q0, half, s.rows);
    F2 th[NP], td[NP];  // over the samples, of dz h and of dz
    GnChannels<T, NE, ONE> ch;
#pragma unroll
    for (int j = 0; j < NP; ++j) th[j] = td[j] = f2(0.f, 0.f);
    if (s.on) gn_params<T, NE>(a.bias, a.ptype, c0 + s.v * NE, 0.f, ch.b);
    auto take = [&](const char *from, F2 (&d)[NP], F2 (&dz)[NP]) {
        F2 f[NP], e[NP];
        V::get(*reinterpret_cast<const Raw *>(from), f);
        V::get(*reinterpret_cast<const Raw *>(from + p.part), e);
        ch.template at<ACT>(f, e, d, dz, [&] {
            return GnSource{from, own, own + T_, 2 * T_, s.off, p.cpg, a.weight, a.bias, a.ptype,
                            c0 + s.v * NE};
        });
    };
    for (int n = q0;; n += p.per) {
        F2 w[NP];  // needed up to the groups' sums only: not worth registers beyond
        if (s.on) gn_params<T, NE>(a.weight, a.ptype, c0 + s.v * NE, 1.f, w);
        cp_async_wait<1>();  // of the sample's two groups the first: its statistics, half its rows
        if (s.on) {
            ch.mean.load(0, s.off, p.cpg, [&](int k) { return own[2 * k * T_]; });
            ch.rstd.load(0, s.off, p.cpg, [&](int k) { return own[(2 * k + 1) * T_]; });
            ch.scale(w);
        }
        F2 sh[NP], sd[NP];
#pragma unroll
        for (int j = 0; j < NP; ++j) sh[j] = sd[j] = f2(0.f, 0.f);
        auto add = [&](int first, int last) {
            const char *from = mine + first * hop;
#pragma unroll 2
            for (int k = first; k < last; ++k, from += hop) {
                F2 d[NP], dz[NP];
                take(from, d, dz);
#pragma unroll
                for (int j = 0; j < NP; ++j) {
                    sh[j] = fma2(dz[j], d[j], sh[j]);
                    sd[j] = add2(sd[j], dz[j]);
                }
            }
        };
        add(0, half);
        cp_async_wait<0>();
        add(half, s.rows);
        if (s.on) {
            F2 q1[NP], q2[NP];
#pragma unroll
            for (int j = 0; j < NP; ++j) {
                th[j] = fma2(sh[j], ch.rstd[j], th[j]);
                td[j] = add2(td[j], sd[j]);
                q1[j] = mul2(sd[j], w[j]);
                q2[j] = mul2(sh[j], ch.rw[j]);
            }
            gn_pieces<NE, ONE>(s.off, p.cpg, [&](int j, int first, int last) {
                s_1[j * T_ + threadIdx.x] = gn_add<NE, ONE>(q1, first, last);
                s_2[j * T_ + threadIdx.x] = gn_add<NE, ONE>(q2, first, last);
            });
        }
        __syncthreads();
        for (int k = warp; k < s.gs; k += warps) {
            float x1 = 0.f, x2 = 0.f;
            gn_values<NE, ONE>(p, k, [&](int at, int, int) {
                x1 += s_1[at];
                x2 += s_2[at];
            });
            x1 = warp_sum_f32(x1);
            x2 = warp_sum_f32(x2);
            if (lane == 0) {
                g[k] = x1;
                g[p.gs + k] = x2;
            }
        }
        gn_block_or_cluster_sync(p.K);
        // a lane for each block of the cluster
        for (int k = threadIdx.x; k < (((s.gs << p.logk) + 31) & ~31); k += T_) {
            const int at = min(k >> p.logk, s.gs - 1), j = k & (p.K - 1);
            float x1, x2;
            if (p.K > 1) {
                x1 = gn_blocks_sum(ld_cluster_f32(g + at, j), p.K);
                x2 = gn_blocks_sum(ld_cluster_f32(g + p.gs + at, j), p.K);
            } else {
                x1 = g[at];
                x2 = g[p.gs + at];
            }
            if (j == 0 && k >> p.logk < s.gs) {
                g[2 * p.gs + at] = x1 * inv;
                g[3 * p.gs + at] = x2 * inv;
            }
        }
        __syncthreads();
        if (p.K > 1) cluster_arrive_relaxed();  // the other blocks may change what was read here
        const bool more = n + p.per < a.n.samples;
        if (more) copy_stats(n + p.per, ahead_own);
        if (s.on) {
            GnSlope<NE, ONE> slope;
            slope.k1.load(s.g0, s.off, p.cpg, [&](int k) { return g[2 * p.gs + k]; });
            slope.k2.load(s.g0, s.off, p.cpg, [&](int k) { return g[3 * p.gs + k]; });
            slope.scale(ch.rstd);
            char *const to_dx = gn_at<T>(dx, a.dx, n, c0);
            const char *const next_x = gn_at<T>(x, a.x, n + p.per, c0);
            const char *const next_dy = gn_at<T>(dy, a.dy, n + p.per, c0);
            // a slot that has been read takes the next sample's vector
            auto put = [&](int first, int last, auto ahead) {
                char *slot = mine + first * hop;
                char *to = to_dx + first * dx.step;
                const char *q = next_x + first * x.step, *u = next_dy + first * dy.step;
#pragma unroll 2
                for (int k = first; k < last; ++k, slot += hop, to += dx.step) {
                    F2 d[NP], dz[NP];
                    take(slot, d, dz);
                    slope.dx(d, ch.rw, dz);
                    __stcs(reinterpret_cast<Raw *>(to), V::put(dz));
                    if constexpr (decltype(ahead)::value) {
                        gn_copy<AB>(slot, q);
                        gn_copy<AB>(slot + p.part, u);
                        q += x.step;
                        u += dy.step;
                    }
                }
                if constexpr (decltype(ahead)::value) cp_async_commit();
            };
            if constexpr (AB == 2) {
                put(0, s.rows, Yes<false>());
                if (more) {  // the statistics are in the first of two groups here too
                    copy(n + p.per, 0, half);
                    copy(n + p.per, half, s.rows);
                }
            } else if (more) {
                put(0, half, Yes<true>());
                put(half, s.rows, Yes<true>());
            } else {
                put(0, s.rows, Yes<false>());
            }
        }
        if (p.K > 1) cluster_wait();
        if (!more) break;
        float *const used = own;
        own = ahead_own;
        ahead_own = used;
    }
    if (a.dweight || a.dbias)
        gn_leave_sums<T, NE>(a, p, s, reinterpret_cast<float *>(dyn), th, td);
}

// ---- host ------------------------------------------------------------------------------------

#define FC_GN_SMEM (226 * 1024)  // a block's most; an SM has 1 KB a block more
#define FC_GN_SETS 1024          // most sets of channel sums

// How to hold the maps; false where a slab does not fit a cluster, or the device
// takes no cluster of the size.
bool gn_plan(const GnShape &n, int ab, int ne, int tensors, const void *kernel, GnPlan *out);

template <class Args>
cudaError_t gn_launch(void (*kernel)(Args, GnPlan), const Args &a, const GnPlan &p, cudaStream_t s)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(p.nslab * p.per * p.K));
    cfg.blockDim = dim3(p.threads);
    cfg.dynamicSmemBytes = p.smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)p.K;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.K > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, a, p);
}

}  // namespace fc
