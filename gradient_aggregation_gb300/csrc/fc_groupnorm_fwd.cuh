// Group norm, forward, for one element type T.
#pragma once

#include "fc_groupnorm_res.cuh"

namespace fc {

// Some of a call's samples; `stat` has room for two values a group of each.
template <class T, int AB, int ACT>
cudaError_t gn_forward_chunk(const GnForward &a, const GnTile &t, float *stat, cudaStream_t s)
{
    const unsigned grid = gn_grid(a.n, t);
    float *part = a.ws;
    int64_t sets = a.n.samples * t.parts, rows = t.rows;
    int parts = t.parts;
    cudaError_t e = launch_after_prior(k_gn_stats<T, AB>, grid, FC_GN_BLOCK, 0, s, a.x, a.n, t, part,
                                       sets);
    if (e != cudaSuccess) return e;
    const int64_t groups = a.n.samples * a.n.groups;
    const int cpg = a.n.channels / a.n.groups;
    if ((int64_t)parts * cpg > FC_GN_ENTRIES && parts > 1) {
        float *const joined = part + 2 * sets * gn_padded(a.n.channels);
        e = gn_join_parts(true, a.n, t, part, sets, joined, s);
        if (e != cudaSuccess) return e;
        part = joined;
        sets = a.n.samples;
        parts = 1;
        rows = a.n.positions;
    }
    if ((int64_t)parts * cpg <= 1024)
        e = launch_after_prior(k_gn_finish<32>, (unsigned)((groups + 7) / 8), 256, 0, s, a.n, parts,
                               rows, part, sets, a.eps, stat, a.mean, a.rstd);
    else
        e = launch_after_prior(k_gn_finish<1024>, (unsigned)groups, 1024, 0, s, a.n, parts, rows,
                               part, sets, a.eps, stat, a.mean, a.rstd);
    if (e != cudaSuccess) return e;
    return launch_after_prior(k_gn_apply<T, AB, ACT>, grid, FC_GN_BLOCK, 0, s, a, t, stat);
}

template <class T, int AB, int ACT>
cudaError_t gn_forward_streaming(const GnForward &a, cudaStream_t s)
{
    const GnTile t = gn_tile(a.n, Gv<T, AB>::NE);
    float *const stat = a.ws + 2 * gn_sets(a.n) * gn_padded(a.n.channels);
    const int64_t chunk = gn_chunk(a.n);
    for (int64_t first = 0; first < a.n.samples; first += chunk) {
        GnForward c = a;
        c.n.samples = std::min(chunk, a.n.samples - first);
        c.x = gn_from<T>(a.x, first);
        c.y = gn_from<T>(a.y, first);
        if (a.mean) {
            c.mean += first * a.n.groups;
            c.rstd += first * a.n.groups;
        }
        const cudaError_t e = gn_forward_chunk<T, AB, ACT>(c, t, stat, s);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

template <class T, int AB, int ACT, bool ONE>
cudaError_t gn_forward_one(const GnForward &a, cudaStream_t s)
{
    GnPlan p;
    if (gn_plan(a.n, AB, Gv<T, AB>::NE, 1, (const void *)k_gn_fwd<T, AB, ACT, ONE>, &p))
        return gn_launch(k_gn_fwd<T, AB, ACT, ONE>, a, p, s);
    if (!gn_may_stream(a.n)) return cudaErrorInvalidConfiguration;
    return gn_forward_streaming<T, AB, ACT>(a, s);
}

template <class T, int AB, int ACT>
cudaError_t gn_forward_groups(const GnForward &a, cudaStream_t s)
{
    constexpr int NE = Gv<T, AB>::NE;
    if (a.n.channels / a.n.groups % NE == 0) return gn_forward_one<T, AB, ACT, true>(a, s);
    return gn_forward_one<T, AB, ACT, NE == 1>(a, s);  // a vector of one lies in one group
}

template <class T, int AB>
cudaError_t gn_forward_act(const GnForward &a, int act, cudaStream_t s)
{
    if (act == FC_ACT_RELU) return gn_forward_groups<T, AB, FC_ACT_RELU>(a, s);
    if (act == FC_ACT_SILU) return gn_forward_groups<T, AB, FC_ACT_SILU>(a, s);
    return gn_forward_groups<T, AB, FC_ACT_NONE>(a, s);
}

template <class T>
cudaError_t gn_forward(const GnForward &a, int act, cudaStream_t s)
{
    const int ab = gn_access<T>(a.n, {&a.x, &a.y});
    if (ab == 16) return gn_forward_act<T, 16>(a, act, s);
    if (sizeof(T) == 2 && ab == 2) return gn_forward_act<T, sizeof(T) == 2 ? 2 : 4>(a, act, s);
    return gn_forward_act<T, 4>(a, act, s);
}

}  // namespace fc
