// Group norm, backward, for one element type T.
#pragma once

#include "fc_groupnorm_res.cuh"
#include "fc_layernorm_bwd.cuh"

namespace fc {

// dweight and dbias from `sets` sets of the channels' sums, as layer norm joins its own.
inline cudaError_t gn_join(const GnBackward &a, const float *in, int64_t sets, cudaStream_t s)
{
    if (!a.dweight && !a.dbias) return cudaSuccess;
    LnBackward l = {};
    l.cols = a.n.channels;
    l.dweight = a.dweight;
    l.dbias = a.dbias;
    l.gtype = a.gtype;
    l.partials = const_cast<float *>(in);
    return ln_join(l, (int)sets, s);
}

// Some of a call's samples, whose sums go to dweight and dbias; `stat` has room for two values
// a group of each.
template <class T, int AB, int ACT>
cudaError_t gn_backward_chunk(const GnBackward &a, const GnTile &t, float *stat, cudaStream_t s)
{
    const unsigned grid = gn_grid(a.n, t);
    float *part = a.ws;
    int64_t sets = a.n.samples * t.parts;
    int parts = t.parts;
    cudaError_t e = launch_after_prior(k_gn_sums<T, AB, ACT>, grid, FC_GN_BLOCK, 0, s, a, t, part,
                                       sets);
    if (e != cudaSuccess) return e;
    const int64_t groups = a.n.samples * a.n.groups;
    const int cpg = a.n.channels / a.n.groups;
    if ((int64_t)parts * cpg > FC_GN_ENTRIES && parts > 1) {
        float *const joined = part + 2 * sets * gn_padded(a.n.channels);
        e = gn_join_parts(false, a.n, t, part, sets, joined, s);
        if (e != cudaSuccess) return e;
        part = joined;
        sets = a.n.samples;
        parts = 1;
    }
    if ((int64_t)parts * cpg <= 1024)
        e = launch_after_prior(k_gn_finish_sums<T, 32>, (unsigned)((groups + 7) / 8), 256, 0, s, a,
                               parts, part, sets, stat);
    else
        e = launch_after_prior(k_gn_finish_sums<T, 1024>, (unsigned)groups, 1024, 0, s, a, parts,
                               part, sets, stat);
    if (e != cudaSuccess) return e;
    e = launch_after_prior(k_gn_apply_bwd<T, AB, ACT>, grid, FC_GN_BLOCK, 0, s, a, t, stat);
    if (e != cudaSuccess) return e;
    return gn_join(a, part, sets, s);
}

template <class T, int AB, int ACT>
cudaError_t gn_backward_streaming(const GnBackward &a, cudaStream_t s)
{
    const GnTile t = gn_tile(a.n, Gv<T, AB>::NE);
    const int64_t padded = gn_padded(a.n.channels);
    float *const stat = a.ws + 2 * gn_sets(a.n) * padded;
    const int64_t chunk = gn_chunk(a.n), chunks = (a.n.samples + chunk - 1) / chunk;
    if (chunks == 1) return gn_backward_chunk<T, AB, ACT>(a, t, stat, s);
    float *const sums = a.ws + 2 * chunk * padded;  // behind what a chunk leaves: a set for each
    for (int64_t k = 0; k < chunks; ++k) {
        const int64_t first = k * chunk;
        GnBackward c = a;
        c.n.samples = std::min(chunk, a.n.samples - first);
        c.dy = gn_from<T>(a.dy, first);
        c.x = gn_from<T>(a.x, first);
        c.dx = gn_from<T>(a.dx, first);
        c.mean += first * a.n.groups;
        c.rstd += first * a.n.groups;
        c.gtype = FC_TYPE_F32;
        if (a.dweight) c.dweight = sums + k * padded;
        if (a.dbias) c.dbias = sums + (chunks + k) * padded;
        const cudaError_t e = gn_backward_chunk<T, AB, ACT>(c, t, stat, s);
        if (e != cudaSuccess) return e;
    }
    return gn_join(a, sums, chunks, s);
}

template <class T, int AB, int ACT, bool ONE>
cudaError_t gn_backward_one(const GnBackward &a, cudaStream_t s)
{
    GnPlan p;
    if (!gn_plan(a.n, AB, Gv<T, AB>::NE, 2, (const void *)k_gn_bwd<T, AB, ACT, ONE>, &p)) {
        if (!gn_may_stream(a.n)) return cudaErrorInvalidConfiguration;
        return gn_backward_streaming<T, AB, ACT>(a, s);
    }
    const cudaError_t e = gn_launch(k_gn_bwd<T, AB, ACT, ONE>, a, p, s);
    return e == cudaSuccess ? gn_join(a, a.ws, p.per, s) : e;
}

// A thread holds five values a channel, and two or four more of each group that its
// vector touches: vectors that cross groups are halved.
template <class T, int AB, int ACT>
cudaError_t gn_backward_groups(const GnBackward &a, cudaStream_t s)
{
    constexpr int NE = Gv<T, AB>::NE;
    const int cpg = a.n.channels / a.n.groups;
    if (cpg % NE == 0) return gn_backward_one<T, AB, ACT, true>(a, s);
    if constexpr (AB == 16) {
        if (cpg % (NE / 2) == 0) return gn_backward_one<T, AB / 2, ACT, true>(a, s);
        return gn_backward_one<T, AB / 2, ACT, false>(a, s);
    } else {
        return gn_backward_one<T, AB, ACT, NE == 1>(a, s);  // a vector of one lies in one group
    }
}

template <class T, int AB>
cudaError_t gn_backward_act(const GnBackward &a, int act, cudaStream_t s)
{
    if (act == FC_ACT_RELU) return gn_backward_groups<T, AB, FC_ACT_RELU>(a, s);
    if (act == FC_ACT_SILU) return gn_backward_groups<T, AB, FC_ACT_SILU>(a, s);
    return gn_backward_groups<T, AB, FC_ACT_NONE>(a, s);
}

template <class T>
cudaError_t gn_backward(const GnBackward &a, int act, cudaStream_t s)
{
    const int ab = gn_access<T>(a.n, {&a.x, &a.dy, &a.dx});
    if (ab == 16) return gn_backward_act<T, 16>(a, act, s);
    if (sizeof(T) == 2 && ab == 2) return gn_backward_act<T, sizeof(T) == 2 ? 2 : 4>(a, act, s);
    return gn_backward_act<T, 4>(a, act, s);
}

}  // namespace fc
