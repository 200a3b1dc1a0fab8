"""Plain 64-bit forms of the training-step operators (torch float64 on whatever
device the inputs are on), and the error bounds their tests use.

U is the relative error of one fp32 rounding.  The bounds follow the number of
roundings in the definitions that include/fc.h gives, with room for the order of
a sum: they were fixed before the first run.
"""

import math

import torch

U = 2.0 ** -24
HALF_ULP = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINIEST = {torch.float32: 2.0 ** -149, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}
BLOCK = 256


def rounded(bound, value, dtype):
    """A bound on an fp32 result, and the rounding of that result to dtype."""
    return bound + HALF_ULP[dtype] * (value.abs() + bound) + TINIEST[dtype]


def grad_norm(grads, loss_scale, max_norm):
    ss = sum(float((g.double() ** 2).sum()) for g in grads)
    norm = math.sqrt(ss) / loss_scale if math.isfinite(ss) else ss
    if not math.isfinite(norm):
        return norm, math.nan
    f = min(1.0, max_norm / norm) if max_norm > 0 and norm > 0 else 1.0
    return norm, f / loss_scale


def adamw(w, m, v, g, decay, t, lr, b1, b2, eps, wd):
    """(w, m, v) after step t, and bounds on the errors of fp32 arithmetic."""
    w, m, v, g, decay = (x.double() for x in (w, m, v, g, decay))
    size = b1 * m.abs() + (1 - b1) * g.abs()
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g * g
    den = torch.sqrt(v) / math.sqrt(1 - b2 ** t) + eps
    to = lr / (1 - b1 ** t)
    step = to * m / den
    new = w - lr * wd * decay * w - step
    # m: roundings of s*g, 1-b1, their product, b1 and the sum; v twice g's.
    # The quotient adds c1, c2 (4 roundings each, halved by the root for c2),
    # the root (2), the division (2) and the products (3).
    em = 6 * U * size
    ev = 8 * U * v + 2.0 ** -148
    ew = 3 * U * w.abs() + to * em / den + 20 * U * step.abs()
    return (new, m, v), (ew, em, ev)


def mix32(x):
    x = x & 0xFFFFFFFF
    x = ((x ^ (x >> 16)) * 0x7FEB352D) & 0xFFFFFFFF
    x = ((x ^ (x >> 15)) * 0x846CA68B) & 0xFFFFFFFF
    return x ^ (x >> 16)


def random16(seed, t, i):
    """The 16 random bits of element i (an int64 tensor) at step t."""
    key = mix32((seed & 0xFFFFFFFF) ^ mix32((seed >> 32) ^ mix32(t)))
    p = i >> 1
    h = mix32((p & 0xFFFFFFFF) + key + (p >> 32) * 0x9E3779B9)
    return torch.where(i % 2 == 0, h & 0xFFFF, h >> 16)


def e4m3_quantum(y):
    """Distance of neighbouring e4m3 values at y >= 0 (float64)."""
    _, e = torch.frexp(y)
    # 2^(e - 4) by its bits: a power taken on the GPU may be a rounding off
    return ((torch.clamp(e - 4, min=-9).long() + 1023) << 52).view(torch.float64)


def block_top(x):
    pad = -x.numel() % BLOCK
    x = torch.cat((x.abs(), torch.zeros(pad, dtype=x.dtype, device=x.device)))
    return x.view(-1, BLOCK).amax(1)


def spread(per_block, n):
    return torch.repeat_interleave(per_block, BLOCK)[:n]


def layernorm(x, weight, bias, eps):
    """(y, mean, rstd) and bounds for fp32 arithmetic before y is rounded."""
    x = x.double()
    n = x.shape[1]
    mean = x.mean(1, keepdim=True)
    c = x - mean
    rstd = 1 / torch.sqrt((c * c).mean(1, keepdim=True) + eps)
    w = torch.ones(n, dtype=torch.float64, device=x.device) if weight is None else weight.double()
    b = torch.zeros(n, dtype=torch.float64, device=x.device) if bias is None else bias.double()
    h = c * rstd
    y = h * w + b
    # a sum of at most 2^14 terms, 32 of them in a row and the rest in a tree
    emean = 40 * U * x.abs().mean(1, keepdim=True)
    erstd = rstd * (50 * U + 0.5 * (rstd * emean) ** 2)
    eh = rstd * (emean + U * (x.abs() + mean.abs())) + h.abs() * (erstd / rstd + 3 * U)
    return (y, mean[:, 0], rstd[:, 0]), (eh * w.abs() + 2 * U * (y.abs() + b.abs()),
                                         emean[:, 0], erstd[:, 0])


def layernorm_backward(dy, x, weight, mean, rstd, run=64):
    """(dx, dweight, dbias) and bounds; `run`: rows that one thread adds in a row."""
    dy, x = dy.double(), x.double()
    mean, rstd = mean.double()[:, None], rstd.double()[:, None]
    n = x.shape[1]
    w = torch.ones(n, dtype=torch.float64, device=x.device) if weight is None else weight.double()
    h = (x - mean) * rstd
    q = dy * w
    s1, s2 = q.mean(1, keepdim=True), (q * h).mean(1, keepdim=True)
    dx = rstd * (q - s1 - h * s2)
    eh = 3 * U * (x.abs() + mean.abs()) * rstd
    e1 = 45 * U * q.abs().mean(1, keepdim=True)
    e2 = 45 * U * (q * h).abs().mean(1, keepdim=True) + (q.abs() * eh).mean(1, keepdim=True)
    edx = rstd * (3 * U * (q.abs() + s1.abs() + (h * s2).abs()) + e1 + h.abs() * e2
                  + eh * s2.abs()) + 2 * U * dx.abs()
    add = (run + 24) * U
    edw = add * (dy * h).abs().sum(0) + (dy.abs() * eh).sum(0)
    return (dx, (dy * h).sum(0), dy.sum(0)), (edx, edw, add * dy.abs().sum(0))


def assert_within(name, got, want, bound):
    got, want, bound = got.double(), want.double(), bound.double()
    over = (got - want).abs() - bound
    bad = ~(over <= 0)
    assert not bool(bad.any()), "%s: %d of %d outside, worst at %d: got %r, want %r within %r" % (
        name, int(bad.sum()), got.numel(), int(torch.where(bad, over, -1.0).argmax()),
        float(got.flatten()[torch.where(bad, over, -1.0).argmax()]),
        float(want.flatten()[torch.where(bad, over, -1.0).argmax()]),
        float(bound.flatten()[torch.where(bad, over, -1.0).argmax()]))
