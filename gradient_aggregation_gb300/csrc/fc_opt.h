// What the gradient norm and the AdamW steps share: the layer table, the
// loads of one gradient from many tensors, and the launchers.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "fc.h"
#include "fc_internal.h"

namespace fc {

// Layers of the fused vector and where their gradients lie, passed by value
// as a __grid_constant__ kernel parameter.  Empty layers are dropped, and
// layers that lie back to back in memory (views of one fused gradient) with
// the same decay are one segment.  64 segments serve most models' small
// tables; 1536 is what fits the 32 KB of kernel parameters.
template <int MAXL>
struct OptTable {
    int32_t L;
    int64_t off[MAXL + 1];   // fused offsets, off[L] = N
    const void *ptr[MAXL];
    float decay[MAXL];
};
using OptTableS = OptTable<64>;
using OptTableL = OptTable<FC_MAX_OPT_LAYERS>;

// The norm needs no fused index: its tiles are cut from each segment's own
// addresses, so that every load is aligned whatever the layer sizes are.
template <int MAXL>
struct NormTable {
    int32_t L;
    int32_t tile0[MAXL + 1];  // first tile of each segment, tile0[L] = tiles
    const void *ptr[MAXL];
    int64_t n[MAXL];          // elements
};
using NormTableS = NormTable<64>;
using NormTableL = NormTable<FC_MAX_OPT_LAYERS>;

struct AdamHyper {
    float b1, omb1, b2, omb2;  // betas, and 1 - beta rounded once from binary64
    float lnb1, lnb2;          // ln(beta): 1 - beta^t = -expm1(t ln beta)
    float lr, eps, lrwd;       // lrwd = lr * weight_decay
};

// partials: FF [FC_NORM_MAX_GRID]; done: zero on entry and on exit.
#define FC_NORM_MAX_GRID 4096
#define FC_NORM_TILE 8192  // bytes of gradient a block takes at a time
template <class Tab>
cudaError_t launch_grad_norm(const Tab &tab, int gtype, float loss_scale, float max_norm,
                             FF *partials, unsigned *done, float *norm, float *scale,
                             cudaStream_t s);

template <class Tab>
cudaError_t launch_adamw(const Tab &tab, int gtype, int64_t N, const AdamHyper &h,
                         const float *scale, float *w, void *low, int ltype, float *m,
                         float *v, int32_t *steps, cudaStream_t s);

template <class Tab>
cudaError_t launch_adamw8(const Tab &tab, int gtype, int64_t N, const AdamHyper &h,
                          const float *scale, float *w, void *low, int ltype, uint8_t *m8,
                          float *m_scale, uint8_t *r8, float *r_scale, int32_t *steps,
                          uint64_t seed, cudaStream_t s);

}  // namespace fc
