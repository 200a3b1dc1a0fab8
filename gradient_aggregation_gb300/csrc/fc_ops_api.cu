// C entry points of the training-step operators: gradient norm, AdamW and
// layer norm.  Argument checks and launches; contracts in include/fc.h.
#include <math.h>
#include <stdarg.h>
#include <stdio.h>

#include <nvtx3/nvToolsExt.h>

#include "fc.h"
#include "fc_layernorm.h"
#include "fc_opt.h"

using namespace fc;

namespace {

struct TraceRange {
    explicit TraceRange(const char *name) { nvtxRangePushA(name); }
    ~TraceRange() { nvtxRangePop(); }
};

fc_status fail(fc_status st, const char *fmt, ...)
{
    char msg[384];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(msg, sizeof(msg), fmt, ap);
    va_end(ap);
    return set_error(st, msg);
}

fc_status ok() { return set_error(FC_OK, ""); }

fc_status launched(cudaError_t e, const char *what)
{
    if (e == cudaSuccess) return ok();
    return fail(FC_ERR_CUDA, "%s: %s (%s)", what, cudaGetErrorName(e), cudaGetErrorString(e));
}

#define TRY(x)                        \
    do {                              \
        fc_status _st = (x);          \
        if (_st != FC_OK) return _st; \
    } while (0)

int type_size(int32_t type) { return type == FC_TYPE_F32 ? 4 : 2; }

fc_status check_type(int32_t type, const char *name)
{
    if (type < FC_TYPE_F32 || type > FC_TYPE_BF16)
        return fail(FC_ERR_INVALID_ARG, "%s = %d is not an FC_TYPE_* value", name, type);
    return FC_OK;
}

fc_status check_ptr(const void *p, const char *name, uintptr_t align, bool may_be_null)
{
    if (!p) return may_be_null ? FC_OK : fail(FC_ERR_INVALID_ARG, "%s is NULL", name);
    if ((uintptr_t)p & (align - 1))
        return fail(FC_ERR_ALIGNMENT, "%s is not %d-byte aligned", name, (int)align);
    return FC_OK;
}

// Layers of a table call; the fused length goes to *N_out.
fc_status check_layers(const void *const *grads, int32_t grad_type, int32_t L,
                       const int64_t *sizes, int64_t *N_out)
{
    TRY(check_type(grad_type, "grad_type"));
    if (!grads) return fail(FC_ERR_INVALID_ARG, "grads is NULL");
    if (!sizes) return fail(FC_ERR_INVALID_ARG, "sizes is NULL");
    if (L < 1) return fail(FC_ERR_INVALID_ARG, "L = %d must be >= 1", L);
    if (L > FC_MAX_OPT_LAYERS)
        return fail(FC_ERR_LIMIT, "L = %d exceeds FC_MAX_OPT_LAYERS = %d", L, FC_MAX_OPT_LAYERS);
    const uintptr_t align = (uintptr_t)type_size(grad_type);
    int64_t N = 0;
    for (int32_t l = 0; l < L; ++l) {
        if (sizes[l] < 0)
            return fail(FC_ERR_INVALID_ARG, "sizes[%d] = %lld < 0", l, (long long)sizes[l]);
        if (sizes[l] == 0) continue;
        // the norm counts its tiles in 32 bits: 2^31 tiles of 8 KB
        if (sizes[l] > ((int64_t)1 << 41) || (N += sizes[l]) > ((int64_t)1 << 41))
            return fail(FC_ERR_INVALID_ARG, "sizes too large");
        if (!grads[l]) return fail(FC_ERR_INVALID_ARG, "grads[%d] is NULL", l);
        if ((uintptr_t)grads[l] & (align - 1))
            return fail(FC_ERR_ALIGNMENT, "grads[%d] is not aligned to its element", l);
    }
    if (N < 1) return fail(FC_ERR_INVALID_ARG, "the sizes sum to 0");
    *N_out = N;
    return FC_OK;
}

// Calls seg(first layer, elements) for every segment: layers that follow
// one another in memory with equal decay.
template <class F>
void for_segments(const void *const *grads, int es, int32_t L, const int64_t *sizes,
                  const float *decay, F seg)
{
    int first = -1;
    int64_t len = 0;
    for (int32_t l = 0; l < L; ++l) {
        if (sizes[l] == 0) continue;
        if (first >= 0 && (const char *)grads[first] + len * es == (const char *)grads[l] &&
            (!decay || decay[l] == decay[first])) {
            len += sizes[l];
            continue;
        }
        if (first >= 0) seg(first, len);
        first = l;
        len = sizes[l];
    }
    seg(first, len);
}

int count_segments(const void *const *grads, int es, int32_t L, const int64_t *sizes,
                   const float *decay)
{
    int n = 0;
    for_segments(grads, es, L, sizes, decay, [&](int, int64_t) { ++n; });
    return n;
}

template <class Tab>
void fill(Tab &t, const void *const *grads, int es, int32_t L, const int64_t *sizes,
          const float *decay)
{
    t.L = 0;
    int64_t acc = 0;
    for_segments(grads, es, L, sizes, decay, [&](int l, int64_t n) {
        t.off[t.L] = acc;
        t.ptr[t.L] = grads[l];
        t.decay[t.L] = decay ? decay[l] : 1.f;
        acc += n;
        ++t.L;
    });
    t.off[t.L] = acc;
}

template <class Tab>
void fill_norm(Tab &t, const void *const *grads, int es, int32_t L, const int64_t *sizes)
{
    t.L = 0;
    int64_t tiles = 0;
    for_segments(grads, es, L, sizes, nullptr, [&](int l, int64_t n) {
        t.tile0[t.L] = (int32_t)tiles;
        t.ptr[t.L] = grads[l];
        t.n[t.L] = n;
        const int64_t bytes = n * es + (int64_t)((uintptr_t)grads[l] & 15);
        tiles += (bytes + FC_NORM_TILE - 1) / FC_NORM_TILE;
        ++t.L;
    });
    t.tile0[t.L] = (int32_t)tiles;
}

constexpr size_t kNormCounter = 256;

struct AdamArgs {
    int64_t N;
    AdamHyper h;
};

fc_status check_adam(const void *const *grads, int32_t grad_type, int32_t L,
                     const int64_t *sizes, const float *decay, const float *grad_scale, double lr,
                     double beta1, double beta2, double eps, double weight_decay,
                     const float *weights, const void *weights_low, int32_t low_type,
                     const int32_t *steps, AdamArgs *out)
{
    TRY(check_layers(grads, grad_type, L, sizes, &out->N));
    for (int32_t l = 0; decay && l < L; ++l)
        if (!(decay[l] >= 0.f) || !isfinite(decay[l]))
            return fail(FC_ERR_INVALID_ARG, "decay[%d] must be finite and >= 0", l);
    TRY(check_ptr(grad_scale, "grad_scale", 4, true));
    if (!(lr >= 0) || !isfinite((float)lr))
        return fail(FC_ERR_INVALID_ARG, "lr must be finite and >= 0");
    if (!(weight_decay >= 0) || !isfinite((float)(lr * weight_decay)))
        return fail(FC_ERR_INVALID_ARG, "weight_decay must be finite and >= 0");
    if (!(beta1 >= 0 && beta1 < 1) || !(beta2 >= 0 && beta2 < 1))
        return fail(FC_ERR_INVALID_ARG, "beta1 and beta2 must be in [0, 1)");
    // betas that fp32 rounds to 1 would leave 1 - beta^t at zero
    if ((float)beta1 == 1.f || (float)beta2 == 1.f)
        return fail(FC_ERR_INVALID_ARG, "beta1 and beta2 must be below 1 in fp32");
    if (!((float)eps > 0.f) || !isfinite((float)eps))
        return fail(FC_ERR_INVALID_ARG, "eps must be finite and > 0 in fp32");
    TRY(check_ptr(weights, "weights", 16, false));
    TRY(check_ptr(weights_low, "weights_low", 16, true));
    if (weights_low && low_type != FC_TYPE_F16 && low_type != FC_TYPE_BF16)
        return fail(FC_ERR_INVALID_ARG, "low_type = %d must be FC_TYPE_F16 or FC_TYPE_BF16",
                    low_type);
    TRY(check_ptr(steps, "steps", 8, false));
    AdamHyper &h = out->h;
    h.b1 = (float)beta1;
    h.omb1 = (float)(1 - beta1);
    h.b2 = (float)beta2;
    h.omb2 = (float)(1 - beta2);
    h.lnb1 = (float)log(beta1);  // -inf for 0: 1 - beta^t is then 1
    h.lnb2 = (float)log(beta2);
    h.lr = (float)lr;
    h.eps = (float)eps;
    h.lrwd = (float)(lr * weight_decay);
    return FC_OK;
}

// Runs f with the smallest table that holds the layers.
template <class F>
cudaError_t with_table(const void *const *grads, int es, int32_t L, const int64_t *sizes,
                       const float *decay, F f)
{
    if (count_segments(grads, es, L, sizes, decay) <= 64) {
        OptTableS tab;
        fill(tab, grads, es, L, sizes, decay);
        return f(tab);
    }
    static thread_local OptTableL tab;
    fill(tab, grads, es, L, sizes, decay);
    return f(tab);
}

}  // namespace

extern "C" {

size_t fc_grad_norm_workspace_size(void)
{
    return kNormCounter + FC_NORM_MAX_GRID * sizeof(FF);
}

fc_status fc_grad_norm(const void *const *grads, int32_t grad_type, int32_t L,
                       const int64_t *sizes, float loss_scale, float max_norm, float *norm,
                       float *scale, void *workspace, size_t workspace_bytes, void *stream)
{
    TraceRange trace("fc_grad_norm");
    int64_t N = 0;
    TRY(check_layers(grads, grad_type, L, sizes, &N));
    if (!(loss_scale > 0.f) || !isfinite(loss_scale))
        return fail(FC_ERR_INVALID_ARG, "loss_scale must be finite and > 0");
    if (!(max_norm >= 0.f) || !isfinite(max_norm))
        return fail(FC_ERR_INVALID_ARG, "max_norm must be finite and >= 0");
    TRY(check_ptr(norm, "norm", 4, false));
    TRY(check_ptr(scale, "scale", 4, false));
    if (!workspace || workspace_bytes < fc_grad_norm_workspace_size())
        return fail(FC_ERR_WORKSPACE, "workspace of %zu bytes, %zu needed",
                    workspace ? workspace_bytes : (size_t)0, fc_grad_norm_workspace_size());
    TRY(check_ptr(workspace, "workspace", 256, false));
    DeviceScope scope;
    TRY(scope.bind(norm));
    unsigned *done = (unsigned *)workspace;
    FF *partials = (FF *)((char *)workspace + kNormCounter);
    const int es = type_size(grad_type);
    if (count_segments(grads, es, L, sizes, nullptr) <= 64) {
        NormTableS tab;
        fill_norm(tab, grads, es, L, sizes);
        return launched(launch_grad_norm(tab, grad_type, loss_scale, max_norm, partials, done,
                                         norm, scale, (cudaStream_t)stream),
                        "grad_norm launch");
    }
    static thread_local NormTableL tab;
    fill_norm(tab, grads, es, L, sizes);
    return launched(launch_grad_norm(tab, grad_type, loss_scale, max_norm, partials, done, norm,
                                     scale, (cudaStream_t)stream),
                    "grad_norm launch");
}

fc_status fc_adamw_step(const void *const *grads, int32_t grad_type, int32_t L,
                        const int64_t *sizes, const float *decay, const float *grad_scale,
                        double lr, double beta1, double beta2, double eps, double weight_decay,
                        float *weights, void *weights_low, int32_t low_type, float *exp_avg,
                        float *exp_avg_sq, int32_t *steps, void *stream)
{
    TraceRange trace("fc_adamw_step");
    AdamArgs a;
    TRY(check_adam(grads, grad_type, L, sizes, decay, grad_scale, lr, beta1, beta2, eps,
                   weight_decay, weights, weights_low, low_type, steps, &a));
    TRY(check_ptr(exp_avg, "exp_avg", 16, false));
    TRY(check_ptr(exp_avg_sq, "exp_avg_sq", 16, false));
    DeviceScope scope;
    TRY(scope.bind(weights));
    return launched(with_table(grads, type_size(grad_type), L, sizes, decay,
                               [&](const auto &tab) {
                                   return launch_adamw(tab, grad_type, a.N, a.h, grad_scale,
                                                       weights, weights_low, low_type, exp_avg,
                                                       exp_avg_sq, steps, (cudaStream_t)stream);
                               }),
                    "adamw launch");
}

fc_status fc_adamw8_step(const void *const *grads, int32_t grad_type, int32_t L,
                         const int64_t *sizes, const float *decay, const float *grad_scale,
                         double lr, double beta1, double beta2, double eps, double weight_decay,
                         float *weights, void *weights_low, int32_t low_type, void *exp_avg_q,
                         float *exp_avg_scale, void *exp_rms_q, float *exp_rms_scale,
                         int32_t *steps, uint64_t seed, void *stream)
{
    TraceRange trace("fc_adamw8_step");
    AdamArgs a;
    TRY(check_adam(grads, grad_type, L, sizes, decay, grad_scale, lr, beta1, beta2, eps,
                   weight_decay, weights, weights_low, low_type, steps, &a));
    TRY(check_ptr(exp_avg_q, "exp_avg_q", 16, false));
    TRY(check_ptr(exp_avg_scale, "exp_avg_scale", 4, false));
    TRY(check_ptr(exp_rms_q, "exp_rms_q", 16, false));
    TRY(check_ptr(exp_rms_scale, "exp_rms_scale", 4, false));
    DeviceScope scope;
    TRY(scope.bind(weights));
    return launched(with_table(grads, type_size(grad_type), L, sizes, decay,
                               [&](const auto &tab) {
                                   return launch_adamw8(tab, grad_type, a.N, a.h, grad_scale,
                                                        weights, weights_low, low_type,
                                                        (uint8_t *)exp_avg_q, exp_avg_scale,
                                                        (uint8_t *)exp_rms_q, exp_rms_scale,
                                                        steps, seed, (cudaStream_t)stream);
                               }),
                    "adamw8 launch");
}

static fc_status check_matrix(const void *p, const char *name, int32_t type, int64_t rows,
                              int64_t cols, int64_t ld)
{
    if (rows > 0) TRY(check_ptr(p, name, (uintptr_t)type_size(type), false));
    if (ld < cols)
        return fail(FC_ERR_INVALID_ARG, "the rows of %s are %lld elements apart, less than cols = %lld",
                    name, (long long)ld, (long long)cols);
    // element offsets stay inside 64 bits
    if (ld > ((int64_t)1 << 40) || (rows > 0 && ld > ((int64_t)1 << 60) / rows))
        return fail(FC_ERR_INVALID_ARG, "%s is too large", name);
    return FC_OK;
}

static fc_status check_layernorm(int32_t type, int32_t param_type, int64_t rows, int64_t cols)
{
    TRY(check_type(type, "type"));
    if (param_type != FC_TYPE_F32 && param_type != type)
        return fail(FC_ERR_INVALID_ARG, "param_type = %d must be FC_TYPE_F32 or the type of x",
                    param_type);
    if (rows < 0) return fail(FC_ERR_INVALID_ARG, "rows = %lld must be >= 0", (long long)rows);
    if (cols < 1 || cols > ((int64_t)1 << 31))
        return fail(FC_ERR_INVALID_ARG, "cols = %lld out of [1, 2^31]", (long long)cols);
    return FC_OK;
}

fc_status fc_layernorm_forward(const void *x, int64_t rows, int64_t cols, int64_t ldx,
                               int32_t type, const void *weight, const void *bias,
                               int32_t param_type, float eps, void *y, int64_t ldy, float *mean,
                               float *rstd, void *stream)
{
    TraceRange trace("fc_layernorm_forward");
    TRY(check_layernorm(type, param_type, rows, cols));
    TRY(check_matrix(x, "x", type, rows, cols, ldx));
    TRY(check_matrix(y, "y", type, rows, cols, ldy));
    TRY(check_ptr(weight, "weight", (uintptr_t)type_size(param_type), true));
    TRY(check_ptr(bias, "bias", (uintptr_t)type_size(param_type), true));
    if (!(eps >= 0.f) || !isfinite(eps))
        return fail(FC_ERR_INVALID_ARG, "eps must be finite and >= 0");
    if (!mean != !rstd)
        return fail(FC_ERR_INVALID_ARG, "mean and rstd must both be given or both be NULL");
    TRY(check_ptr(mean, "mean", 4, true));
    TRY(check_ptr(rstd, "rstd", 4, true));
    if (rows == 0) return ok();
    DeviceScope scope;
    TRY(scope.bind(y));
    const LnForward a = {x, rows, cols, ldx, weight, bias, param_type, eps, y, ldy, mean, rstd};
    return launched(launch_ln_forward(a, type, (cudaStream_t)stream), "layernorm launch");
}

size_t fc_layernorm_backward_workspace_size(int64_t rows, int64_t cols)
{
    if (rows < 0 || cols < 1 || cols > ((int64_t)1 << 31)) return 0;
    const int64_t parts = ln_max_parts(rows, cols) < 1 ? 1 : ln_max_parts(rows, cols);
    // sets of column sums, rows of whole 32-byte groups
    return (size_t)parts * (size_t)((cols + 7) / 8 * 8) * 2 * sizeof(float);
}

fc_status fc_layernorm_backward(const void *dy, int64_t lddy, const void *x, int64_t ldx,
                                int32_t type, const void *weight, int32_t param_type,
                                const float *mean, const float *rstd, int64_t rows, int64_t cols,
                                void *dx, int64_t lddx, void *dweight, void *dbias,
                                int32_t grad_type, void *workspace, size_t workspace_bytes,
                                void *stream)
{
    TraceRange trace("fc_layernorm_backward");
    TRY(check_layernorm(type, param_type, rows, cols));
    TRY(check_type(grad_type, "grad_type"));
    TRY(check_matrix(dy, "dy", type, rows, cols, lddy));
    TRY(check_matrix(x, "x", type, rows, cols, ldx));
    TRY(check_matrix(dx, "dx", type, rows, cols, lddx));
    TRY(check_ptr(weight, "weight", (uintptr_t)type_size(param_type), true));
    TRY(check_ptr(mean, "mean", 4, rows == 0));
    TRY(check_ptr(rstd, "rstd", 4, rows == 0));
    TRY(check_ptr(dweight, "dweight", (uintptr_t)type_size(grad_type), true));
    TRY(check_ptr(dbias, "dbias", (uintptr_t)type_size(grad_type), true));
    const bool sums = dweight || dbias;
    if (sums) {
        const size_t need = fc_layernorm_backward_workspace_size(rows, cols);
        if (!workspace || workspace_bytes < need)
            return fail(FC_ERR_WORKSPACE, "workspace of %zu bytes, %zu needed",
                        workspace ? workspace_bytes : (size_t)0, need);
        TRY(check_ptr(workspace, "workspace", 256, false));
    }
    if (rows == 0 && !sums) return ok();
    DeviceScope scope;
    TRY(scope.bind(rows ? dx : dweight ? dweight : dbias));
    const LnBackward a = {dy,   lddy, x,       ldx,   weight,    param_type, mean, rstd, rows, cols,
                          dx,   lddx, dweight, dbias, grad_type, sums ? (float *)workspace : nullptr};
    return launched(launch_ln_backward(a, type, (cudaStream_t)stream), "layernorm launch");
}

}  // extern "C"
