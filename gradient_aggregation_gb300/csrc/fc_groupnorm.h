// Arguments of the group norm launchers (checked by the C entry points).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace fc {

// Images [samples, positions, channels]: channels next to one another, positions
// `ld` and samples `ss` elements apart.
struct GnImages {
    const void *p;
    int64_t ld, ss;
};

struct GnShape {
    int64_t samples, positions;
    int channels, groups;
};

struct GnForward {
    GnImages x;
    GnShape n;
    const void *weight, *bias;
    int ptype;  // type of weight and bias
    float eps;
    GnImages y;
    float *mean, *rstd;
    float *ws;
};

struct GnBackward {
    GnImages dy, x;
    GnShape n;
    const void *weight, *bias;
    int ptype;
    const float *mean, *rstd;
    GnImages dx;
    void *dweight, *dbias;
    int gtype;  // type of dweight and dbias
    float *ws;
};

// The workspace: sets of two values a channel (what blocks leave), then two values a
// group and sample.
int64_t gn_parts(const GnShape &n);  // parts of a sample's positions, streaming
int64_t gn_chunk(const GnShape &n);  // samples at a time, streaming
int64_t gn_held(const GnShape &n);   // most clusters that work on a slab's samples
int64_t gn_sets(const GnShape &n);
bool gn_may_stream(const GnShape &n);  // else the workspace has no room for it
inline int64_t gn_padded(int channels) { return ((int64_t)channels + 7) & ~(int64_t)7; }

cudaError_t launch_gn_forward(const GnForward &a, int type, int act, cudaStream_t s);
cudaError_t launch_gn_backward(const GnBackward &a, int type, int act, cudaStream_t s);

}  // namespace fc
