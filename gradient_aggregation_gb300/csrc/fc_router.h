// Arguments of the router's launchers (checked by the C entry points).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "fc_router_cut.h"

namespace fc {

struct RouterForward {
    const void *logits;
    int64_t ld;
    RouterShape n;
    const int32_t *lengths;
    int32_t *chosen;
    float *weights, *lse;
    int32_t *counts, *routed;
    float *probs, *loss;
    void *ws;
};

struct RouterBackward {
    const void *logits;
    int64_t ld;
    RouterShape n;
    const int32_t *chosen;
    const float *weights, *lse;
    const int32_t *counts, *routed;
    const float *dweights, *dloss;
    void *dlogits;
    int64_t lddl;
};

// The workspace: what each block of the first kernel leaves, then the groups' shares
// of the losses, then a counter.
size_t router_workspace(int64_t sequences, int64_t tokens, int64_t experts, int64_t groups);

cudaError_t launch_router_forward(const RouterForward &a, int type, cudaStream_t s);
cudaError_t launch_router_backward(const RouterBackward &a, int type, cudaStream_t s);

}  // namespace fc
