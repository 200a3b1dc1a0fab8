// Packed pairs of fp32 (one instruction for two elements), 16-byte vectors of
// the three element types as pairs, and rows that start anywhere.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "fc_common.cuh"

namespace fc {

struct F2 {
    unsigned long long v;
};

__device__ __forceinline__ F2 f2(float a, float b)
{
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
    return r;
}

__device__ __forceinline__ float2 un2(F2 a)
{
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a.v));
    return r;
}

__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c)
{
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}

__device__ __forceinline__ F2 mul2(F2 a, F2 b)
{
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}

__device__ __forceinline__ F2 add2(F2 a, F2 b)
{
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}

// A 16-byte vector of its pairs: 4 of a 16-bit type, 2 of fp32, each rounded once.
template <class T>
__device__ __forceinline__ uint4 from_pairs(const F2 (&f)[8 / sizeof(T)])
{
    uint32_t w[4];
    if constexpr (sizeof(T) == 4) {
        const float2 a = un2(f[0]), b = un2(f[1]);
        w[0] = __float_as_uint(a.x);
        w[1] = __float_as_uint(a.y);
        w[2] = __float_as_uint(b.x);
        w[3] = __float_as_uint(b.y);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 a = un2(f[i]);
            if constexpr (__is_same(T, __half)) {
                const __half2 h = __floats2half2_rn(a.x, a.y);
                w[i] = *reinterpret_cast<const uint32_t *>(&h);
            } else {
                const __nv_bfloat162 h = __floats2bfloat162_rn(a.x, a.y);
                w[i] = *reinterpret_cast<const uint32_t *>(&h);
            }
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// ---- rows that start at any element and have any width ---------------------------------------
//
// A warp holds NP pairs a lane of 64 NP columns that follow one another from
// column `base`: with 16-bit types pair p of lane l is columns base + 2 (l + 32 p)
// and the next, so that a pair is one 32-bit word; with fp32 it is columns
// base + l + 64 p and base + l + 64 p + 32.  Every access is then one word a
// lane, contiguous over the warp, and 16-bit rows that start at an odd element
// are put together from halves of two words.

// Elements of T by which p lies past a 16-byte boundary.
template <class T>
__device__ __forceinline__ int past16(const T *p)
{
    return (int)(((uintptr_t)p & 15) / sizeof(T));
}

template <class T>
__device__ __forceinline__ F2 pair_of_word(uint32_t w)
{
    if constexpr (__is_same(T, __half)) {
        const float2 v = __half22float2(*reinterpret_cast<const __half2 *>(&w));
        return f2(v.x, v.y);
    } else {
        return f2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    }
}

template <class T>
__device__ __forceinline__ uint32_t word_of_pair(F2 f)
{
    const float2 a = un2(f);
    if constexpr (__is_same(T, __half)) {
        const __half2 h = __floats2half2_rn(a.x, a.y);
        return *reinterpret_cast<const uint32_t *>(&h);
    } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a.x, a.y);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
}

// First column of pair p of lane l, and the distance to its second.
template <class T>
__device__ __forceinline__ int pair_column(int base, int lane, int p)
{
    return sizeof(T) == 2 ? base + 2 * (lane + 32 * p) : base + lane + 64 * p;
}

template <class T>
__host__ __device__ __forceinline__ constexpr int pair_step()
{
    return sizeof(T) == 2 ? 1 : 32;
}

// Writes a warp's pairs to columns of `row`.
template <class T, int NP>
__device__ __forceinline__ void store_pairs(T *row, int cols, int base, const F2 (&f)[NP])
{
    const int lane = threadIdx.x & 31;
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int p = 0; p < NP; ++p) {
            const int c = pair_column<T>(base, lane, p);
            const float2 v = un2(f[p]);
            if (c < cols) __stcs(row + c, v.x);
            if (c + 32 < cols) __stcs(row + c + 32, v.y);
        }
    } else {
        unsigned short *const h = reinterpret_cast<unsigned short *>(row) + base + 2 * lane;
        const int left = cols - base;  // of the row from the warp's first column on
        if (((uintptr_t)row & 2) == 0) {
#pragma unroll
            for (int b = 0; b < NP; b += 4) {
                if (left >= 64 * (b + 4)) {  // inside the row for every lane
#pragma unroll
                    for (int p = b; p < b + 4; ++p)
                        __stcs(reinterpret_cast<uint32_t *>(h + 64 * p), word_of_pair<T>(f[p]));
                } else {
#pragma unroll
                    for (int p = b; p < b + 4; ++p) {
                        const int n = left - 64 * p - 2 * lane;
                        const uint32_t w = word_of_pair<T>(f[p]);
                        if (n >= 2)
                            __stcs(reinterpret_cast<uint32_t *>(h + 64 * p), w);
                        else if (n == 1)
                            h[64 * p] = (unsigned short)w;
                    }
                }
            }
            return;
        }
        // memory's words hold the second of one pair and the first of the next
        uint32_t before = 0;
#pragma unroll
        for (int b = 0; b < NP; b += 4) {
            const bool inside = left > 64 * (b + 4);  // and a pair follows for every lane
            if (b > 0 && b + 4 < NP && inside) {
#pragma unroll
                for (int p = b; p < b + 4; ++p) {
                    const uint32_t w = word_of_pair<T>(f[p]);
                    const uint32_t r = __shfl_sync(0xffffffffu, w, (lane + 31) & 31);
                    __stcs(reinterpret_cast<uint32_t *>(h + 64 * p - 1),
                           __byte_perm(lane == 0 ? before : r, w, 0x5432));
                    before = r;
                }
                continue;
            }
#pragma unroll
            for (int p = b; p < b + 4; ++p) {
                const uint32_t w = word_of_pair<T>(f[p]);
                const uint32_t r = __shfl_sync(0xffffffffu, w, (lane + 31) & 31);
                const uint32_t joined = __byte_perm(lane == 0 ? before : r, w, 0x5432);
                before = r;
                const int n = left - 64 * p - 2 * lane;
                if (n >= 1) {
                    if (p == 0 && lane == 0)
                        h[0] = (unsigned short)w;
                    else
                        __stcs(reinterpret_cast<uint32_t *>(h + 64 * p - 1), joined);
                }
                if (n >= 2 && ((p == NP - 1 && lane == 31) || n == 2))
                    h[64 * p + 1] = (unsigned short)(w >> 16);
            }
        }
    }
}

__device__ __forceinline__ void cp_async16(uint32_t to, const void *from)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}

// The first `bytes` of 16, zeros behind them.
__device__ __forceinline__ void cp_async16(uint32_t to, const void *from, int bytes)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(bytes)
                 : "memory");
}

__device__ __forceinline__ void cp_async_commit()
{
    asm volatile("cp.async.commit_group;" ::: "memory");
}

// Until all but the latest KEEP groups of this thread have landed.
template <int KEEP>
__device__ __forceinline__ void cp_async_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(KEEP) : "memory");
}

// Shared-memory slots (16 bytes) that a warp needs for K vectors a lane of one row.
template <int K, bool ANY>
constexpr int warp_slots()
{
    return 32 * K + (ANY ? 1 : 0);
}

// Issues the copies of the granules around a warp's columns of row r of a
// matrix, into slots from `to` (this lane's first) on.  ANY: what lies past the
// row comes out as zeros, if the slots were zeros before their first row.
template <class T, int K, bool ANY>
__device__ __forceinline__ void copy_row(const T *m, int64_t ld, int64_t r, int cols, int base,
                                         uint32_t to)
{
    constexpr int VEC = 16 / (int)sizeof(T);
    const int lane = threadIdx.x & 31;
    const T *const row = m + r * ld;
    const int past = ANY ? past16(row) : 0;
#pragma unroll
    for (int k = 0; k < K + (ANY ? 1 : 0); ++k) {
        if (k == K && lane != 0) break;
        const int c = base + VEC * (lane + 32 * k) - past;  // may be before the row
        if (c >= cols + (ANY ? VEC : 0)) continue;
        if (!ANY) {
            cp_async16(to + 32 * k * 16, row + c);
        } else if (c >= 0 || r > 0) {
            // the granule behind the row's last is all zeros: another row, shifted
            // otherwise, may have ended in it
            const int n = min(VEC, max(cols - c, 0));
            cp_async16(to + 32 * k * 16, n ? row + c : row + c - VEC, n * (int)sizeof(T));
        } else {  // before the matrix itself: its first elements one by one
            uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
            for (int e = 0; e < VEC; ++e)
                if (c + e >= 0 && c + e < cols) {
                    if constexpr (sizeof(T) == 2)
                        w[e / 2] |= (uint32_t)reinterpret_cast<const unsigned short *>(row)[c + e]
                                    << (16 * (e & 1));
                    else
                        w[e] = reinterpret_cast<const uint32_t *>(row)[c + e];
                }
            asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(to + 32 * k * 16),
                         "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3])
                         : "memory");
        }
    }
}

// The lane's words out of the warp's slots p, where the warp's first column lies
// `past` elements in: its vectors, or (ANY) one word a pair, two of fp32.  What
// lies past the row is zero.
template <class T, int K, bool ANY>
__device__ __forceinline__ void take_row(const uint4 *p, int past, int cols, int base,
                                         uint32_t (&w)[4 * K])
{
    constexpr int VEC = 16 / (int)sizeof(T);
    const int lane = threadIdx.x & 31;
    if constexpr (!ANY) {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const uint4 q = base + VEC * (lane + 32 * k) < cols ? p[lane + 32 * k]
                                                                : make_uint4(0, 0, 0, 0);
            w[4 * k] = q.x;
            w[4 * k + 1] = q.y;
            w[4 * k + 2] = q.z;
            w[4 * k + 3] = q.w;
        }
    } else if constexpr (sizeof(T) == 4) {
        const uint32_t *const u = reinterpret_cast<const uint32_t *>(p) + past + lane;
#pragma unroll
        for (int i = 0; i < 4 * K; ++i) w[i] = u[32 * i];
    } else {
        const uint32_t *const u = reinterpret_cast<const uint32_t *>(p) + (past >> 1) + lane;
#pragma unroll
        for (int i = 0; i < 4 * K; ++i) w[i] = u[32 * i];
        if (past & 1) {
#pragma unroll
            for (int i = 0; i < 4 * K; ++i) w[i] = __byte_perm(w[i], u[32 * i + 1], 0x5432);
        }
    }
}

// Pair p of such words.
template <class T, int NW>
__device__ __forceinline__ F2 pair_of(const uint32_t (&w)[NW], int p)
{
    if constexpr (sizeof(T) == 4)
        return f2(__uint_as_float(w[2 * p]), __uint_as_float(w[2 * p + 1]));
    else
        return pair_of_word<T>(w[p]);
}

}  // namespace fc
