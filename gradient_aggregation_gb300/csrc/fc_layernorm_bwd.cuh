// Layer norm, backward: the kernels, for one element type T.
//
//   h = (x - mean) * rstd;  q = dy * w
//   dx = rstd * (q - sum(q) / n - h * sum(q h) / n)
//   dweight = sum over rows of dy * h;  dbias = sum over rows of dy
//
// Bound by HBM: dy and x are read once and dx written once.  The two row sums
// cost one shuffle reduction and, where a row spans several warps, one
// exchange and one barrier.  A thread owns the same columns in every row, so
// the column sums stay in its registers until its block has no more rows; each
// block then leaves one set of sums, and a second kernel (for few narrow rows
// the same one, as a cluster) adds the sets in their order (no atomics: the same
// inputs give the same bits).
#pragma once

#include <algorithm>

#include "fc_cluster.cuh"
#include "fc_layernorm.cuh"
#include "fc_pairs.cuh"

namespace fc {

// Columns of one set of sums in the workspace.
__host__ __device__ __forceinline__ int64_t ln_padded(int64_t cols) { return (cols + 7) & ~(int64_t)7; }

cudaError_t ln_join(const LnBackward &a, int parts, cudaStream_t s);

__device__ __forceinline__ void store_sum(void *out, int gtype, int64_t c, float s)
{
    if (gtype == FC_TYPE_F32)
        static_cast<float *>(out)[c] = s;
    else if (gtype == FC_TYPE_F16)
        static_cast<__half *>(out)[c] = __float2half_rn(s);
    else
        static_cast<__nv_bfloat16 *>(out)[c] = __float2bfloat16_rn(s);
}

// Few narrow rows: the grid is one cluster, whose CTAs add the sets of column
// sums that they have just left in the workspace, a slice of the columns each.
// (Reading the sets from the other CTAs' shared memory instead took 0.4 to 0.7 us
// more for 256 to 1024 columns.)
#define FC_LN_CLUSTER 8

template <int BLOCK>
__device__ __forceinline__ void join_in_cluster(const LnBackward &a)
{
    cluster_sync();
    const int cols = (int)a.cols, parts = (int)gridDim.x;
    const int64_t padded = ln_padded(a.cols);
    for (int i = blockIdx.x * BLOCK + threadIdx.x; i < 2 * cols; i += parts * BLOCK) {
        const int which = i >= cols, c = which ? i - cols : i;
        void *const out = which ? a.dbias : a.dweight;
        if (!out) continue;
        const float *const p = a.partials + which * parts * padded + c;
        float v[FC_LN_CLUSTER], s = 0.f;
#pragma unroll
        for (int q = 0; q < FC_LN_CLUSTER; ++q) v[q] = q < parts ? __ldcg(p + q * padded) : 0.f;
#pragma unroll
        for (int q = 0; q < FC_LN_CLUSTER; ++q) s += v[q];
        store_sum(out, a.gtype, c, s);
    }
}

// Rows of at most 128 columns: TPR lanes of a warp hold a row, several rows a
// warp; the next row is loaded while one is worked on.
template <class T, int VEC, int K, int TPR, int BLOCK>
__global__ void __launch_bounds__(BLOCK)
    k_ln_bwd(const LnBackward a, const bool pvec, const bool joins)
{
    constexpr int G = BLOCK / TPR, W = TPR * K * VEC;
    __shared__ float sums[2][G][W];
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

    float pw[K][VEC], dw[K][VEC], db[K][VEC];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        if (t + k * TPR < nvec)
            load_params<T, VEC>(a.weight, a.ptype, pvec, (t + k * TPR) * VEC, 1.f, pw[k]);
#pragma unroll
        for (int e = 0; e < VEC; ++e) dw[k][e] = db[k][e] = 0.f;
    }

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
    for (int64_t it = 0; it < rounds; ++it, row += stride) {
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
                float fx[VEC], fy[VEC];
                vx[k].get(fx);
                vy[k].get(fy);
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const float h = (fx[e] - mean) * rstd;
                    const float q = fy[e] * pw[k][e];
                    s1 += q;
                    s2 = fmaf(q, h, s2);
                    dw[k][e] = fmaf(fy[e], h, dw[k][e]);
                    db[k][e] += fy[e];
                }
            }
        }
        s1 = lanes_sum<TPR>(s1) * inv_n;
        s2 = lanes_sum<TPR>(s2) * inv_n;
        if (row < a.rows) {
#pragma unroll
            for (int k = 0; k < K; ++k) {
                if (t + k * TPR < nvec) {
                    float fx[VEC], fy[VEC];
                    vx[k].get(fx);
                    vy[k].get(fy);
#pragma unroll
                    for (int e = 0; e < VEC; ++e) {
                        const float h = (fx[e] - mean) * rstd;
                        fx[e] = rstd * (fmaf(fy[e], pw[k][e], -s1) - h * s2);
                    }
                    Vec<T, VEC>::store(dx + row * a.lddx + (t + k * TPR) * VEC, fx);
                }
            }
        }
    }
    if (!a.partials) return;
    // the row groups of the block are added in their order
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            sums[0][g][(t + k * TPR) * VEC + e] = dw[k][e];
            sums[1][g][(t + k * TPR) * VEC + e] = db[k][e];
        }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * W; i += BLOCK) {
        const int which = i / W, c = i % W;
        float v = sums[which][0][c];
#pragma unroll
        for (int r = 1; r < G; ++r) v += sums[which][r][c];
        if (c < cols)
            a.partials[(which * (int64_t)gridDim.x + blockIdx.x) * ln_padded(cols) + c] = v;
    }
    if (joins) join_in_cluster<BLOCK>(a);
}

// ---- rows of more than 128 columns ----------------------------------------------------------
//
// A row is held by TPR threads, as pairs of fp32 that one instruction works on.
// The vectors of the next D - 1 rows are on their way into shared memory
// (cp.async, each warp into slots of its own, so no barrier of the block guards
// them) while a row is worked on: that keeps rows in flight without holding
// registers, which the column sums need.
//
// ANY = false: every row starts on a 16-byte boundary and is whole vectors; a
// lane holds K of them.  ANY = true: rows that start at any element and have any
// width; a warp copies the 32 K + 1 aligned granules around its columns and
// reads its pairs out of them word by word (see fc_pairs.cuh).
//
// h is (x - mean) * rstd, the difference first: a row far from zero has its mean's
// digits cancelled exactly there (as x * rstd - mean * rstd the rounding of the
// product, |mean| rstd 2^-24, is an error that the whole row's h has in common).
// dx is rstd ((q - s1) - (rstd s2) (x - mean)), with s1 and s2 the means of q and
// q h: no h, and rstd is never squared (it may be 1e19 where eps is 0).
//
// Measured at 134M elements of bf16 (805 MB), 768 / 1024 / 2048 / 4096 columns:
// 123 / 130 / 131 / 131 us, 0.9 of the copy rate; with the rows loaded one ahead
// into registers 197 / 161 / 178 / 200 us.
template <class T, int K, int TPR, int BLOCK, int D, bool ANY, int CL>
__global__ void __launch_bounds__(BLOCK, BLOCK == 512 ? 1 : K == 1 ? 4 : 2)
    k_ln_bwd_ring(const LnBackward a, const bool pvec, const bool joins)
{
    constexpr int VEC = 16 / (int)sizeof(T), NP = K * VEC / 2;
    constexpr int G = BLOCK / TPR, WARPS = TPR / 32, STEP = pair_step<T>();
    constexpr int SLOTS = warp_slots<K, ANY>();  // of one row of one matrix
    constexpr int ROW = BLOCK / 32 * 2 * SLOTS;
    // three vectors of a 16-bit type do not fit beside their sums: the row is read
    // from its slots again for dx (67M bf16 elements in rows of 1536 / 3000 / 6144 /
    // 12288 columns: 66 / 69 / 70 / 80 us; held in registers and spilled in part 83 /
    // 94 / 71 / 96), and where the block has one row it is read vector by vector
    // for the sums, too (12288 columns 75 us, but 3000 columns 71.5)
    constexpr bool AGAIN = !ANY && K == 3 && sizeof(T) == 2, BY_VECTOR = AGAIN && TPR == 512;
    extern __shared__ __align__(16) uint4 ring[];  // [D][warps][2][SLOTS]
    static_assert(CL == 1 || (G == 1 && CL * WARPS == 32), "a cluster's sums are one a lane");
    __shared__ float2 part[2][CL == 1 ? G : CL][WARPS];
    wait_for_prior_grid();
    allow_dependent_launch();
    const int t = threadIdx.x % TPR, g = threadIdx.x / TPR, lane = threadIdx.x & 31;
    const int cols = (int)a.cols;
    const uint32_t rank = CL == 1 ? 0 : cluster_rank();
    const int first = (int)rank * (TPR * K * VEC);  // the CTA's first column
    const int base = first + (t >> 5) * (64 * NP);  // the warp's
    const uint4 *const mine = ring + (threadIdx.x >> 5) * (2 * SLOTS);
    const uint32_t slot = (uint32_t)__cvta_generic_to_shared(mine + lane);
    const T *const x = static_cast<const T *>(a.x), *const dy = static_cast<const T *>(a.dy);
    T *const dx = static_cast<T *>(a.dx);
    const int64_t stride = (int64_t)gridDim.x / CL * G;

    // first column of pair p: vectors are contiguous, words interleaved
    auto column = [&](int p) {
        return ANY ? pair_column<T>(base, lane, p)
                   : base + VEC * (lane + 32 * (p / (VEC / 2))) + 2 * (p % (VEC / 2));
    };
    constexpr int SECOND = ANY ? STEP : 1;

    auto issue = [&](int64_t r, int d) {
        if (r < a.rows) {
            copy_row<T, K, ANY>(x, a.ldx, r, cols, base, slot + (uint32_t)(d * ROW) * 16);
            copy_row<T, K, ANY>(dy, a.lddy, r, cols, base, slot + (uint32_t)(d * ROW + SLOTS) * 16);
        }
        cp_async_commit();
    };

    int64_t row = (int64_t)blockIdx.x / CL * G + g;
    if constexpr (ANY) {
        for (int i = threadIdx.x; i < D * ROW; i += BLOCK) ring[i] = make_uint4(0, 0, 0, 0);
        __syncthreads();
    }
#pragma unroll
    for (int d = 0; d < D - 1; ++d) issue(row + d * stride, d);
    F2 pw[NP], dw[NP], db[NP];
#pragma unroll
    for (int p = 0; p < NP; ++p) pw[p] = dw[p] = db[p] = f2(0.f, 0.f);
    if constexpr (ANY) {
#pragma unroll
        for (int p = 0; p < NP; ++p) {
            float w0[1] = {0.f}, w1[1] = {0.f};
            const int c = column(p);
            if (c < cols) load_params<T, 1>(a.weight, a.ptype, false, c, 1.f, w0);
            if (c + SECOND < cols) load_params<T, 1>(a.weight, a.ptype, false, c + SECOND, 1.f, w1);
            pw[p] = f2(w0[0], w1[0]);
        }
    } else {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = base + VEC * (lane + 32 * k);
            if (c >= cols) continue;
            float w[VEC];
            load_params<T, VEC>(a.weight, a.ptype, pvec, c, 1.f, w);
#pragma unroll
            for (int p = 0; p < VEC / 2; ++p) pw[k * (VEC / 2) + p] = f2(w[2 * p], w[2 * p + 1]);
        }
    }
    const float inv_n = 1.f / (float)cols;
    if constexpr (CL > 1) cluster_sync();  // the other CTAs run before they are written to
    int buf = 0, d = 0;
    float nmean = 0.f, nrstd = 0.f;
    if (row < a.rows) {
        nmean = __ldg(a.mean + row);
        nrstd = __ldg(a.rstd + row);
    }
    for (; row < a.rows; row += stride) {
        issue(row + (D - 1) * stride, d == 0 ? D - 1 : d - 1);
        const float mean = nmean, rstd = nrstd;
        if (row + stride < a.rows) {
            nmean = __ldg(a.mean + row + stride);
            nrstd = __ldg(a.rstd + row + stride);
        }
        cp_async_wait<D - 1>();
        if constexpr (ANY) __syncwarp();
        uint32_t vx[4 * K], vy[4 * K];
        const uint4 *const held = mine + d * ROW;
        auto take = [&]() {
            take_row<T, K, ANY>(held, ANY ? past16(x + row * a.ldx) : 0, cols, base, vx);
            take_row<T, K, ANY>(held + SLOTS, ANY ? past16(dy + row * a.lddy) : 0, cols, base, vy);
        };
        if constexpr (!BY_VECTOR) take();
        if (++d == D) d = 0;
        const F2 rr = f2(rstd, rstd), mm = f2(-mean, -mean);
        auto centred = [&](int p) { return add2(pair_of<T>(vx, p), mm); };
        F2 a1 = f2(0.f, 0.f), a2 = f2(0.f, 0.f);
        // in blocks of a vector's pairs, each behind a branch of its own: without
        // it the compiler works on all of them at once and runs out of registers
#pragma unroll
        for (int k = 0; k < K; ++k) {
            if (column(k * (VEC / 2)) >= cols) continue;
            if constexpr (BY_VECTOR) {
                const uint4 qx = held[lane + 32 * k], qy = held[SLOTS + lane + 32 * k];
                vx[4 * k] = qx.x; vx[4 * k + 1] = qx.y; vx[4 * k + 2] = qx.z; vx[4 * k + 3] = qx.w;
                vy[4 * k] = qy.x; vy[4 * k + 1] = qy.y; vy[4 * k + 2] = qy.z; vy[4 * k + 3] = qy.w;
            }
#pragma unroll
            for (int p = k * (VEC / 2); p < (k + 1) * (VEC / 2); ++p) {
                const F2 fy = pair_of<T>(vy, p);
                const F2 h = mul2(centred(p), rr);
                const F2 q = mul2(fy, pw[p]);
                a1 = add2(a1, q);
                a2 = fma2(q, h, a2);
                dw[p] = fma2(fy, h, dw[p]);
                db[p] = add2(db[p], fy);
            }
        }
        const float2 u1 = un2(a1), u2 = un2(a2);
        float s1 = lanes_sum<32>(u1.x + u1.y);
        float s2 = lanes_sum<32>(u2.x + u2.y);
        if constexpr (CL > 1) {
            if (lane < CL) {
                const float2 *const to = &part[buf][rank][t >> 5];
                st_cluster_u32(&to->x, (uint32_t)lane, __float_as_uint(s1));
                st_cluster_u32(&to->y, (uint32_t)lane, __float_as_uint(s2));
            }
            cluster_sync();
            const float2 p = part[buf][lane / WARPS][lane % WARPS];
            s1 = lanes_sum<32>(p.x);
            s2 = lanes_sum<32>(p.y);
            buf ^= 1;
        } else if constexpr (WARPS > 1) {
            if (lane == 0) part[buf][g][t >> 5] = make_float2(s1, s2);
            group_sync<TPR, BLOCK>(g);
            const float2 p = part[buf][g][threadIdx.x & (WARPS - 1)];
            s1 = lanes_sum<WARPS>(p.x);
            s2 = lanes_sum<WARPS>(p.y);
            buf ^= 1;
        }
        if constexpr (AGAIN) {
            asm volatile("" ::: "memory");
            take();
        }
        s1 *= inv_n;
        s2 *= inv_n;
        const float c = -rstd * s2;
        const F2 c2 = f2(c, c), c1 = f2(-s1, -s1);
        T *const out = dx + row * a.lddx;
        auto grad = [&](int p) {
            return mul2(fma2(centred(p), c2, fma2(pair_of<T>(vy, p), pw[p], c1)), rr);
        };
        if constexpr (ANY) {
            F2 f[NP];
#pragma unroll
            for (int p = 0; p < NP; ++p) f[p] = grad(p);
            store_pairs<T, NP>(out, cols, base, f);
        } else {
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const int c = base + VEC * (lane + 32 * k);
                if (c >= cols) continue;
                F2 u[VEC / 2];
#pragma unroll
                for (int p = 0; p < VEC / 2; ++p) u[p] = grad(k * (VEC / 2) + p);
                __stcs(reinterpret_cast<uint4 *>(out + c), from_pairs<T>(u));
            }
        }
    }
    cp_async_wait<0>();
    if (!a.partials) return;
    // Every group leaves its sums in shared memory (no more than the ring
    // held), and the block adds them in the groups' order.
    const int padded = (int)ln_padded(cols);
    const int width = CL == 1 ? padded : min(padded - first, TPR * K * VEC);
    float *const sums = reinterpret_cast<float *>(ring);  // [2][G][width]
    __syncthreads();
#pragma unroll
    for (int p = 0; p < NP; ++p) {
        const int c = column(p);
        if (c >= cols) continue;
        float *const to = sums + g * width + (c - first);
        const float2 w = un2(dw[p]), b = un2(db[p]);
        if constexpr (SECOND == 1) {
            *reinterpret_cast<float2 *>(to) = w;
            *reinterpret_cast<float2 *>(to + G * width) = b;
        } else {
            to[0] = w.x;
            to[G * width] = b.x;
            if (c + SECOND < cols) {
                to[SECOND] = w.y;
                to[G * width + SECOND] = b.y;
            }
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * (width / 4); i += BLOCK) {
        const int which = i >= width / 4, q = which ? i - width / 4 : i;
        const float4 *from = reinterpret_cast<const float4 *>(sums + which * G * width) + q;
        float4 v = from[0];
#pragma unroll
        for (int r = 1; r < G; ++r) {
            const float4 u = from[r * (width / 4)];
            v = make_float4(v.x + u.x, v.y + u.y, v.z + u.z, v.w + u.w);
        }
        const int64_t set = which * (int64_t)gridDim.x / CL + blockIdx.x / CL;
        reinterpret_cast<float4 *>(a.partials + set * padded + first)[q] = v;
    }
    if constexpr (CL == 1) {
        if (joins) join_in_cluster<BLOCK>(a);
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
    a.partials[blockIdx.y * ln_padded(a.cols) + c] = dw;
    a.partials[(gridDim.y + blockIdx.y) * ln_padded(a.cols) + c] = db;
}

// ---- launches -------------------------------------------------------------------------------

// CTAs of the one cluster that serves the call, if a CTA takes `group` rows at
// a time, or 0 if the sums are joined by a launch of their own.  For rows of up
// to 32 vectors (64 where they are aligned).  One launch saves 1.6 us of host
// time a call (5.0 and 3.4 us); on the GPU, two launches and one, in us: 64
// columns, bf16 3.0 and 2.5 for 128 rows, 3.2 and 3.3 for 512; 256 columns,
// bf16 3.4 and 3.4 for 128 rows, 3.5 and 4.2 for 256, fp32 3.1 and 3.6 for 128
// rows, 3.2 and 4.2 for 256; 1024 fp32 columns 3.1 and 3.7 for 8 rows, 3.3 and
// 4.2 for 64.
#define FC_LN_ONE_ROWS 128

inline int joining_ctas(const LnBackward &a, int group)
{
    if (!a.partials || a.rows > FC_LN_ONE_ROWS) return 0;
    int ctas = 1;
    while (ctas < FC_LN_CLUSTER && ctas * group < a.rows && 2 * ctas <= a.rows) ctas *= 2;
    return ctas;
}

// A launch in clusters of `cluster` blocks.
template <class... KArgs, class... Args>
static cudaError_t launch_clusters(void (*kernel)(KArgs...), int grid, int cluster, unsigned block,
                                   size_t smem, cudaStream_t s, Args... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...);
}

template <class T, int VEC, int K, int TPR, int BLOCK>
static cudaError_t go(const LnBackward &a, bool pvec, cudaStream_t s)
{
    if (const int ctas = joining_ctas(a, BLOCK / TPR))
        return launch_clusters(k_ln_bwd<T, VEC, K, TPR, BLOCK>, ctas, ctas, BLOCK, 0, s, a, pvec,
                               true);
    const auto kernel = k_ln_bwd<T, VEC, K, TPR, BLOCK>;
    const int64_t ctas = (a.rows + BLOCK / TPR - 1) / (BLOCK / TPR);
    int grid = grid_for((const void *)kernel, BLOCK, 0, ctas);
    const int64_t most = ln_max_parts(a.rows, a.cols);
    if (grid > most) grid = (int)most;
    cudaError_t e = launch_after_prior(kernel, (unsigned)grid, BLOCK, 0, s, a, pvec, false);
    return e != cudaSuccess ? e : ln_join(a, grid, s);
}

template <class T, int K, int TPR, int BLOCK, bool ANY, int CL = 1>
struct RingLaunch {
    static constexpr int D = CL == 1 && K == 4 ? 2 : 3, G = BLOCK / TPR;
    static constexpr auto kernel = k_ln_bwd_ring<T, K, TPR, BLOCK, D, ANY, CL>;
    size_t smem;
    int64_t ctas;
    int resident;

    cudaError_t prepare(const LnBackward &a)
    {
        const void *k = (const void *)kernel;
        // the same for every width: the ring has room for the sums of the widest row
        smem = (size_t)D * (BLOCK / 32) * 2 * warp_slots<K, ANY>() * 16;
        static_assert((size_t)D * (BLOCK / 32) * 2 * 32 * K * 16 >=
                          2 * sizeof(float) * (size_t)G * TPR * K * (16 / sizeof(T)),
                      "the sums lie where the ring was");
        ctas = (a.rows + G - 1) / G;
        cudaError_t e =
            cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e == cudaSuccess)
            resident = grid_for(k, BLOCK, smem, INT64_MAX, cudaSharedmemCarveoutMaxShared);
        return e;
    }
    // in groups of CL blocks, each of which leaves one set of sums
    cudaError_t run(const LnBackward &a, bool pvec, cudaStream_t s) const
    {
        const int64_t most = std::min<int64_t>(resident / CL, ln_max_parts(a.rows, a.cols));
        const int grid = (int)std::min(ctas, most);
        cudaError_t e;
        if constexpr (CL == 1)
            e = launch_after_prior(kernel, (unsigned)grid, BLOCK, smem, s, a, pvec, false);
        else
            e = launch_clusters(kernel, grid * CL, CL, BLOCK, smem, s, a, pvec, false);
        return e != cudaSuccess ? e : ln_join(a, grid, s);
    }
    cudaError_t run_cluster(const LnBackward &a, bool pvec, int n, cudaStream_t s) const
    {
        return launch_clusters(kernel, n, n, BLOCK, smem, s, a, pvec, true);
    }
};

// Blocks of 512 threads leave half as many sets of sums as blocks of 256, which
// spread few rows over more SMs.  Measured with 256 and 512 threads: 128 rows of
// 256 fp32 columns 3.1 and 3.9 us, 512 rows of 1024 bf16 columns 5.2 and 5.7,
// 1024 rows 7.7 and 7.0, 2048 rows 9.3 and 8.0.
template <class T, int K, int TPR, bool ANY>
static cudaError_t go_ring(const LnBackward &a, bool pvec, cudaStream_t s)
{
    constexpr int SMALL = TPR == 512 ? 512 : 256, LARGE = K == 1 ? 256 : 512;
    if constexpr (K <= (ANY ? 1 : 2) && TPR == 32) {
        if (const int ctas = joining_ctas(a, LARGE / TPR)) {
            RingLaunch<T, K, TPR, LARGE, ANY> one;
            cudaError_t e = one.prepare(a);
            return e != cudaSuccess ? e : one.run_cluster(a, pvec, ctas, s);
        }
    }
    RingLaunch<T, K, TPR, SMALL, ANY> small;
    cudaError_t e = small.prepare(a);
    if (e != cudaSuccess) return e;
    // a block of the small kind on every SM at most
    constexpr int per_sm = SMALL == 512 ? 1 : K == 1 ? 4 : 2;
    if (SMALL == LARGE || small.ctas <= small.resident / per_sm) return small.run(a, pvec, s);
    RingLaunch<T, K, TPR, LARGE, ANY> large;
    e = large.prepare(a);
    return e != cudaSuccess ? e : large.run(a, pvec, s);
}

// Rows wider than one CTA's registers hold with their sums: half a row in each
// of two CTAs, which exchange the sums of their warps.  Measured at 805 MB: 16384
// bf16 columns 214 us (one CTA of four vectors a thread, which spills: 234), 12288
// and 16384 fp32 columns 170 and 151 us (two passes over the row: 360 and 387).  A
// quarter of a row in each of four CTAs, two to an SM: 311, 241 and 211 us.
template <class T, int K, bool ANY>
static cudaError_t go_halves(const LnBackward &a, bool pvec, cudaStream_t s)
{
    RingLaunch<T, K, 512, 512, ANY, 2> halves;
    const cudaError_t e = halves.prepare(a);
    return e != cudaSuccess ? e : halves.run(a, pvec, s);
}

// The smallest TPR * K that holds a row of n vectors.
template <class T, bool ANY>
static cudaError_t ring(const LnBackward &a, int64_t n, bool pvec, cudaStream_t s)
{
    if (n <= 32) return go_ring<T, 1, 32, ANY>(a, pvec, s);
    if (n <= 64) return go_ring<T, 2, 32, ANY>(a, pvec, s);
    if constexpr (!ANY) {  // 3 vectors' words and their masks would not fit the registers
        if (n <= 96) return go_ring<T, 3, 32, ANY>(a, pvec, s);
        if (n > 128 && n <= 192) return go_ring<T, 3, 64, ANY>(a, pvec, s);
        if (n > 256 && n <= 384) return go_ring<T, 3, 128, ANY>(a, pvec, s);
        if (n > 512 && n <= 768) return go_ring<T, 3, 256, ANY>(a, pvec, s);
        if (n > 1024 && n <= 1536) return go_ring<T, 3, 512, ANY>(a, pvec, s);
    }
    if (n <= 128) return go_ring<T, 2, 64, ANY>(a, pvec, s);
    if (n <= 256) return go_ring<T, 2, 128, ANY>(a, pvec, s);
    if (n <= 512) return go_ring<T, 2, 256, ANY>(a, pvec, s);
    if (n <= 1024) return go_ring<T, 2, 512, ANY>(a, pvec, s);
    if constexpr (sizeof(T) == 4) {
        if (n <= 2048) return go_ring<T, 4, 512, ANY>(a, pvec, s);
        if constexpr (!ANY)
            if (n <= 3072) return go_halves<T, 3, ANY>(a, pvec, s);
        return go_halves<T, 4, ANY>(a, pvec, s);
    } else {
        return go_halves<T, 2, ANY>(a, pvec, s);
    }
}

template <class T>
static cudaError_t wide_rows(const LnBackward &a, cudaStream_t s)
{
    const auto wide = k_ln_bwd_wide<T>;
    const int grid = grid_for((const void *)wide, FC_LN_WIDE_BLOCK, 0, a.rows);
    cudaError_t e = launch_after_prior(wide, (unsigned)grid, FC_LN_WIDE_BLOCK, 0, s, a);
    if (e != cudaSuccess || !a.partials) return e;
    const int64_t strips = (a.cols + 127) / 128;
    const int64_t parts = ln_max_parts(a.rows, a.cols);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)strips, (unsigned)parts);
    cfg.blockDim = dim3(128);
    cfg.stream = s;
    e = cudaLaunchKernelEx(&cfg, k_ln_colsum_wide<T>, a);
    return e != cudaSuccess ? e : ln_join(a, (int)parts, s);
}

template <class T>
cudaError_t ln_backward(const LnBackward &a, cudaStream_t s)
{
    constexpr int V = 16 / (int)sizeof(T);
    auto on16 = [](const void *p, int64_t ld) {
        return ((uintptr_t)p & 15) == 0 && (ld * (int64_t)sizeof(T)) % 16 == 0;
    };
    const bool pvec = ((uintptr_t)a.weight & 15) == 0;
    const int64_t c = a.cols, n = (c + V - 1) / V;
    const bool vectors = c % V == 0 && on16(a.x, a.ldx) && on16(a.dy, a.lddy) && on16(a.dx, a.lddx);
    // narrow rows: several to a warp, or one element a thread
    if (vectors && n <= 8) return go<T, V, 1, 8, 128>(a, pvec, s);
    if (vectors && n <= 16) return go<T, V, 1, 16, 128>(a, pvec, s);
    if (!vectors && c <= 32) return go<T, 1, 1, 32, 128>(a, pvec, s);
    if (!vectors && c <= 128) return go<T, 1, 4, 32, 128>(a, pvec, s);
    if (n > (sizeof(T) == 4 ? 4096 : 2048)) return wide_rows<T>(a, s);
    return vectors ? ring<T, false>(a, n, pvec, s) : ring<T, true>(a, n, pvec, s);
}

}  // namespace fc
