// Pieces that the layer norm kernels share.
//
// A row is held by TPR threads (8 to 1024), K vectors of VEC elements each:
// vector k of thread t covers columns (t + k*TPR)*VEC.., so a warp's access is
// contiguous.  VEC is 16 bytes' worth where every row starts on a 16-byte
// boundary and the width is whole vectors, else 1.  The row is read once and
// kept in registers in its own type; a block holds BLOCK / TPR rows.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fc.h"
#include "fc_internal.h"
#include "fc_layernorm.h"

namespace fc {

__device__ __forceinline__ float ln_f32(float x) { return x; }
__device__ __forceinline__ float ln_f32(__half x) { return __half2float(x); }
__device__ __forceinline__ float ln_f32(__nv_bfloat16 x) { return __bfloat162float(x); }

template <class T>
__device__ __forceinline__ T ln_round(float x);
template <>
__device__ __forceinline__ float ln_round<float>(float x) { return x; }
template <>
__device__ __forceinline__ __half ln_round<__half>(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ __nv_bfloat16 ln_round<__nv_bfloat16>(float x)
{
    return __float2bfloat16_rn(x);
}

// VEC elements as they lie in memory: 16 bytes, or one element.
template <class T, int VEC>
struct Vec {
    static_assert(VEC * sizeof(T) == 16, "a vector is 16 bytes or one element");
    uint4 q;
    __device__ __forceinline__ void load(const T *p)
    {
        q = __ldcs(reinterpret_cast<const uint4 *>(p));
    }
    __device__ __forceinline__ void clear() { q = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void get(float (&f)[VEC]) const
    {
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (VEC == 4) {
                f[i] = __uint_as_float(w[i]);
            } else if constexpr (sizeof(T) == 2) {
                float2 v;
                if constexpr (__is_same(T, __half)) {
                    v = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
                } else {
                    v.x = __uint_as_float(w[i] << 16);
                    v.y = __uint_as_float(w[i] & 0xffff0000u);
                }
                f[2 * i] = v.x;
                f[2 * i + 1] = v.y;
            }
        }
    }
    static __device__ __forceinline__ void store(T *p, const float (&f)[VEC])
    {
        uint4 o;
        uint32_t *w = &o.x;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (VEC == 4) {
                w[i] = __float_as_uint(f[i]);
            } else if constexpr (__is_same(T, __half)) {
                const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
                w[i] = *reinterpret_cast<const uint32_t *>(&h);
            } else if constexpr (sizeof(T) == 2) {
                const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
                w[i] = *reinterpret_cast<const uint32_t *>(&h);
            }
        }
        __stcs(reinterpret_cast<uint4 *>(p), o);
    }
};

template <class T>
struct Vec<T, 1> {
    T q;
    __device__ __forceinline__ void load(const T *p) { q = __ldcs(p); }
    __device__ __forceinline__ void clear() { q = ln_round<T>(0.f); }
    __device__ __forceinline__ void get(float (&f)[1]) const { f[0] = ln_f32(q); }
    static __device__ __forceinline__ void store(T *p, const float (&f)[1])
    {
        __stcs(p, ln_round<T>(f[0]));
    }
};

// VEC parameters of type fp32 or T from column c; pvec: the pointer is
// 16-byte aligned and VEC elements may be read as vectors.
template <class T, int VEC>
__device__ __forceinline__ void load_params(const void *p, int ptype, bool pvec, int64_t c,
                                            float none, float (&f)[VEC])
{
    if (!p) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) f[e] = none;
    } else if (sizeof(T) == 4 || ptype == FC_TYPE_F32) {
        const float *q = static_cast<const float *>(p) + c;
        if (VEC >= 4 && pvec) {
#pragma unroll
            for (int e = 0; e + 3 < VEC; e += 4) {
                const float4 v = __ldg(reinterpret_cast<const float4 *>(q + e));
                f[e] = v.x;
                f[e + 1] = v.y;
                f[e + 2] = v.z;
                f[e + 3] = v.w;
            }
        } else {
#pragma unroll
            for (int e = 0; e < VEC; ++e) f[e] = __ldg(q + e);
        }
    } else {
        const T *q = static_cast<const T *>(p) + c;
        if (VEC > 1 && pvec) {
            Vec<T, VEC> v;
            v.q = __ldg(reinterpret_cast<const decltype(v.q) *>(q));
            v.get(f);
        } else {
#pragma unroll
            for (int e = 0; e < VEC; ++e) f[e] = ln_f32(q[e]);
        }
    }
}

// Sum over the min(TPR, 32) lanes that hold a row's part of one warp.
template <int TPR>
__device__ __forceinline__ float lanes_sum(float x)
{
#pragma unroll
    for (int o = (TPR < 32 ? TPR : 32) / 2; o > 0; o >>= 1)
        x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// Barrier of the TPR threads of row group g (TPR > 32).
template <int TPR, int BLOCK>
__device__ __forceinline__ void group_sync(int g)
{
    if constexpr (TPR == BLOCK)
        __syncthreads();
    else
        asm volatile("bar.sync %0, %1;" ::"r"(g + 1), "n"(TPR) : "memory");
}

}  // namespace fc
