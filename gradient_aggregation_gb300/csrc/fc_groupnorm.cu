// Group norm: the workspace's layout and the choice of the element type.  The
// kernels are in fc_groupnorm.cuh; each element type and direction is compiled
// in a file of its own, so that they build side by side.
#include <algorithm>
#include <mutex>
#include <new>
#include <numeric>
#include <unordered_map>

#include "fc_groupnorm_bwd.cuh"
#include "fc_groupnorm_fwd.cuh"

namespace fc {

extern template cudaError_t gn_forward<float>(const GnForward &, int, cudaStream_t);
extern template cudaError_t gn_forward<__half>(const GnForward &, int, cudaStream_t);
extern template cudaError_t gn_forward<__nv_bfloat16>(const GnForward &, int, cudaStream_t);
extern template cudaError_t gn_backward<float>(const GnBackward &, int, cudaStream_t);
extern template cudaError_t gn_backward<__half>(const GnBackward &, int, cudaStream_t);
extern template cudaError_t gn_backward<__nv_bfloat16>(const GnBackward &, int, cudaStream_t);

// Whether a call may stream, whatever its type and alignment: not where the group of a
// sample fits a cluster of any kind (see find_plan) for two tensors of 4 bytes, unless the
// images are large enough for streaming to be the faster.
bool gn_may_stream(const GnShape &n)
{
    const int64_t cpg = n.channels / n.groups;
    return cpg > 256 || n.positions * cpg > 1 << 16 ||
           (n.positions >= 64 && n.samples * n.positions * n.channels >= 1 << 22);
}

// As many parts as make 1024 blocks over the samples, of 16 positions or more and of 4096
// elements or more (16 a thread); none is empty.
int64_t gn_parts(const GnShape &n)
{
    const int64_t most = std::max<int64_t>(1, 1024 / std::max<int64_t>(1, n.samples));
    const int64_t least = std::max<int64_t>(16, 4096 / n.channels);
    const int64_t want = std::min(most, (n.positions + least - 1) / least);
    const int64_t rows = (n.positions + want - 1) / want;
    return (n.positions + rows - 1) / rows;
}

// Many samples of few positions are streamed some at a time, so that what they leave is 64 MB
// at most (a set of two sums is up to 8 bytes for each element of them, which L2 holds so) and
// no thread adds up more than 256 sets.  All at once, 65536 x 1 x 4096 bf16 at an odd pitch
// left 2148 MB: 8.77 and 10.44 ms, in chunks 8.71 and 10.26; 9000 x 16 x 2000: 915 and 1356 us,
// in chunks 951 and 1388.
int64_t gn_chunk(const GnShape &n)
{
    if (gn_parts(n) > 1) return n.samples;  // 512 samples at most
    const int64_t most = std::min<int64_t>(8192, (1 << 23) / gn_padded(n.channels));
    return std::min<int64_t>(n.samples, std::max<int64_t>(1, most));
}

// The same limit for the sets of the resident kernels, above what the GPU holds: clusters run
// at a time, 2048 threads of an SM at most with 8 channels each.
int64_t gn_held(const GnShape &n)
{
    const int64_t most = std::min<int64_t>(FC_GN_SETS, (1 << 23) / gn_padded(n.channels));
    return std::min<int64_t>(n.samples, std::max<int64_t>(1, most));
}

// Streaming leaves one for each part, one for each sample that has several, and one for each
// chunk of samples where there are several; the resident kernels one for each cluster that
// works on a slab's samples.
int64_t gn_sets(const GnShape &n)
{
    if (n.samples == 0 || !gn_may_stream(n)) return gn_held(n);
    const int64_t parts = gn_parts(n), chunk = gn_chunk(n);
    const int64_t chunks = (n.samples + chunk - 1) / chunk;
    return std::max(gn_held(n), chunk * (parts + (parts > 1)) + (chunks > 1 ? chunks : 0));
}

namespace {

// What a kernel's launches ask the device, kept: each is looked up once.
struct Fact {
    const void *kernel;
    int dev, K, threads, smem;
    bool operator==(const Fact &o) const
    {
        return kernel == o.kernel && dev == o.dev && K == o.K && threads == o.threads &&
               smem == o.smem;
    }
};

struct FactHash {
    size_t operator()(const Fact &f) const
    {
        return ((size_t)f.kernel >> 4) * 31 + (size_t)(f.dev * 7 + f.K) * 1031 +
               (size_t)f.threads * 17 + (size_t)f.smem;
    }
};

template <class F>
int looked_up(const Fact &f, F find)
{
    static std::mutex mu;
    // never destroyed: calls may come from threads that outlive the statics
    static auto *const cache = new (std::nothrow) std::unordered_map<Fact, int, FactHash>;
    std::lock_guard<std::mutex> lock(mu);
    if (cache) {
        const auto it = cache->find(f);
        if (it != cache->end()) return it->second;
    }
    const int v = find();
    try {
        if (cache) cache->emplace(f, v);
    } catch (const std::bad_alloc &) {  // looked up again next time
    }
    return v;
}

// Clusters of K blocks that the device holds at a time (0: none).
int clusters_held(const void *kernel, int K, int threads, size_t smem)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(K);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = K;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int clusters = 0;
    if (cudaOccupancyMaxActiveClusters(&clusters, kernel, &cfg) != cudaSuccess) clusters = 0;
    cudaGetLastError();  // a refusal is an answer
    return clusters;
}

// Largest cluster of the kernel's largest blocks that the device takes (0: it takes no
// such block); raises the kernel's limits.
int cluster_limit(const void *kernel)
{
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, FC_GN_SMEM) !=
        cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
    const bool wide = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed,
                                           1) == cudaSuccess;
    cudaGetLastError();
    for (int k = wide ? 16 : 8; k > 1; k /= 2)
        if (clusters_held(kernel, k, FC_GN_THREADS, FC_GN_SMEM) > 0) return k;
    return 1;
}

bool find_plan(const GnShape &n, int ab, int ne, int tensors, const void *kernel, int dev,
               GnPlan *out)
{
    const int cpg = n.channels / n.groups;
    const int64_t unit = std::lcm((int64_t)cpg, (int64_t)ne);  // channels; divides all of them
    const int64_t uv = unit / ne;
    if (uv > FC_GN_THREADS || n.positions > (1 << 24)) return false;
    const int limit = looked_up({kernel, dev, 0, 0, 0}, [&] { return cluster_limit(kernel); });
    const int64_t units = n.channels / unit;
    const int ns = ne % cpg == 0 ? ne / cpg : cpg % ne == 0 ? 1 : (ne + cpg - 2) / cpg + 1;
    double best = 1e30;
    GnPlan p = {};
    p.cpg = cpg;
    p.ns = ns;
    p.total = (float)n.positions * (float)cpg;
    p.divn = cpg % ne == 0 ? (int)(((1 << 20) + cpg / ne - 1) / (cpg / ne)) : 0;
    // units of a slab; the last slab may have fewer
    const int64_t slabs[] = {1, 2, 3, 4, 6, 8, 12, 16, 24, 32, 48, 64, 96, 128, 192, 256, 384, 512, units};
    for (int T = 128; T <= FC_GN_THREADS; T *= 2) {
        for (const int64_t u : slabs) {
            if (u > units || u * uv > T) continue;
            const int V = (int)(u * uv), R = T / V, gs = (int)(u * unit / cpg);
            const int64_t nslab = (units + u - 1) / u, items = n.samples * nslab;
            for (int K = 1; K <= limit && (K == 1 || K <= n.positions); K *= 2) {
                const int64_t rows = (n.positions + K - 1) / K, iters = (rows + R - 1) / R;
                const int64_t part = (iters * T * ab + 15) / 16 * 16;
                int64_t smem = tensors * part + 2 * (int64_t)ns * T * 4 + 16 * gs;
                if (tensors == 2)
                    smem = std::max<int64_t>(smem + 4 * (int64_t)ns * T * 4,
                                             (2 * T * ne + std::max(T, 2 * V * ne)) * 4);
                smem = (smem + 4095) / 4096 * 4096;  // few sizes to look up
                if (smem > FC_GN_SMEM || items * K > INT32_MAX) continue;
                // what an SM and the GPU hold at a time
                const int64_t occ = std::min<int64_t>(
                    233472 / (smem + 1024), (tensors == 2 ? FC_GN_RESIDENT_BWD : FC_GN_RESIDENT) / T);
                const int64_t held = std::max<int64_t>(
                    1, (int64_t)(152 * occ * (K <= 2 ? 1. : K == 4 ? .96 : K == 8 ? .88 : .74) / K));
                const int64_t per = std::max<int64_t>(1, std::min(n.samples, held / nslab));
                const int64_t at_once = std::min(per * nslab, held);
                const int64_t rounds = (items + at_once - 1) / at_once;
                const int64_t an_sm = std::min(occ, (at_once * K + 151) / 152);
                // us of a round: HBM's, the instructions', and what neither hides
                const double wide = V * ab >= 128 ? 1 : V * ab >= 64 ? 1.03 : V * ab >= 32 ? 1.35
                                    : V * ab >= 16 ? 2 : V * ab >= 8 ? 3 : 24. / (V * ab);
                const double mem = (double)at_once * rows * K * V * ab * (tensors + 1) * wide / 6.6e6;
                const double inst = (tensors == 2 ? 22 : 11) * ne + 10;
                const double issue = an_sm * (T / 32) * (iters * inst + 600) / 7600.;
                const double lat = 1 + (K > 1 ? .4 : 0) + (K > 8 ? 1.5 : 0) +
                                   (an_sm == 1 && rounds > 1 ? 1.2 : 0) +
                                   iters * (tensors == 2 ? .06 : .03) + (V * ab < 32 ? .5 : 0);
                const double cost = 2 + .3 * T / 256 +
                                    rounds * (std::max(mem, issue) + .35 * std::min(mem, issue) + lat);
                if (cost < best) {
                    best = cost;
                    p.threads = T;
                    p.K = K;
                    p.sc = (int)(u * unit);
                    p.nslab = (int)nslab;
                    p.gs = gs;
                    p.V = V;
                    p.R = R;
                    p.rows = (int)rows;
                    p.iters = (int)iters;
                    p.part = (int)part;
                    p.smem = (size_t)smem;
                }
            }
        }
    }
    if (best == 1e30) return false;
    // Long maps at less than 16 bytes an access: a round of one block an SM takes 1.1 to 5
    // times as long as reckoned above, and streaming, which has no rounds, 2.5 to 5 times the
    // floor and 18 us at the least.  8 x 16427 x 384 bf16 at an odd pitch, backward: 640 us held
    // in shared memory, 233 streamed; 10 x 11404 x 480 in groups of 30: 314 and 137; the other
    // way round 40 x 1352 x 211 in 211 groups, forward: 27 and 32.
    const double bytes = (double)n.samples * n.positions * n.channels * (ab / ne) * (tensors + 1);
    const double floors = ab == 2 ? (tensors == 2 ? 4.5 : 4) : 3.1;
    if (ab < 16 && gn_may_stream(n) && 1.7 * best > 18 + floors * bytes / 6.8e6) return false;
    for (p.logk = 0; 1 << p.logk < p.K;) ++p.logk;
    p.divv = ((1 << 20) + p.V - 1) / p.V;
    const int held = looked_up({kernel, dev, p.K, p.threads, (int)p.smem}, [&] {
        return clusters_held(kernel, p.K, p.threads, p.smem);
    });
    if (held < 1) return false;
    // as many clusters as run at a time, each with as many samples as the others
    const int64_t most = std::max<int64_t>(1, std::min<int64_t>(held / p.nslab, gn_held(n)));
    const int64_t rounds = (n.samples + most - 1) / most;
    p.per = (int)((n.samples + rounds - 1) / rounds);
    *out = p;
    return true;
}

}  // namespace

// The search takes 3 us of host time: each thread keeps its latest plans.
bool gn_plan(const GnShape &n, int ab, int ne, int tensors, const void *kernel, GnPlan *out)
{
    struct Kept {
        GnShape n;
        const void *kernel;  // one for each type, access, direction, activation
        int dev;
        bool found, used;
        GnPlan plan;
    };
    constexpr int kKept = 64;
    static thread_local Kept kept[kKept];
    int dev = 0;
    cudaGetDevice(&dev);
    const uint64_t mixed = ((uint64_t)n.samples * 0x9E3779B97F4A7C15ull +
                            (uint64_t)n.positions * 0xC2B2AE3D27D4EB4Full +
                            (uint64_t)n.channels * 0x165667B19E3779F9ull + (uint64_t)n.groups +
                            ((uint64_t)(uintptr_t)kernel >> 4) * 0x27D4EB2F165667C5ull);
    Kept &k = kept[(mixed >> 32) % kKept];
    if (!k.used || k.kernel != kernel || k.dev != dev || k.n.samples != n.samples ||
        k.n.positions != n.positions || k.n.channels != n.channels || k.n.groups != n.groups) {
        k.used = false;
        k.found = find_plan(n, ab, ne, tensors, kernel, dev, &k.plan);
        k.n = n;
        k.kernel = kernel;
        k.dev = dev;
        k.used = true;
    }
    *out = k.plan;
    return k.found;
}

cudaError_t launch_gn_forward(const GnForward &a, int type, int act, cudaStream_t s)
{
    if (type == FC_TYPE_F32) return gn_forward<float>(a, act, s);
    if (type == FC_TYPE_F16) return gn_forward<__half>(a, act, s);
    return gn_forward<__nv_bfloat16>(a, act, s);
}

cudaError_t launch_gn_backward(const GnBackward &a, int type, int act, cudaStream_t s)
{
    if (a.n.samples == 0) return gn_join(a, a.ws, 0, s);
    if (type == FC_TYPE_F32) return gn_backward<float>(a, act, s);
    if (type == FC_TYPE_F16) return gn_backward<__half>(a, act, s);
    return gn_backward<__nv_bfloat16>(a, act, s);
}

}  // namespace fc
