"""Plain 64-bit forms of group norm and the router (torch float64 on whatever device
the inputs are on), and the error bounds their tests use.

U is the relative error of one fp32 rounding.  RUN is more than the longest chain of
additions behind any sum of the kernels (a thread's own run, the threads of a block,
the blocks): a sum of n terms is off by at most RUN * U of the sum of their sizes.
The bounds were fixed before the first run.
"""

import torch

from tests.ops_ref import U

RUN = 500


def _spread(t, channels):
    """[N, G] -> [N, 1, C]"""
    return t.repeat_interleave(channels // t.shape[1], 1)[:, None, :]


def _by_group(t, groups):
    """Mean over positions and a group's channels: [N, S, C] -> [N, G]"""
    n, s, c = t.shape
    return t.view(n, s, groups, c // groups).mean((1, 3))


def act(z, kind):
    if kind == 1:
        return torch.relu(z)
    return z * torch.sigmoid(z) if kind == 2 else z


def dact(z, kind):
    if kind == 1:
        return (z > 0).double()
    if kind == 2:
        s = torch.sigmoid(z)
        return s + z * s * torch.sigmoid(-z)
    return torch.ones_like(z)


def _params(c, weight, bias, dev):
    w = torch.ones(c, dtype=torch.float64, device=dev) if weight is None else weight.double()
    b = torch.zeros(c, dtype=torch.float64, device=dev) if bias is None else bias.double()
    return w, b


def groupnorm(x, groups, weight, bias, eps, kind):
    """(y, mean, rstd) and bounds for fp32 arithmetic before y is rounded."""
    x = x.double().contiguous()
    c = x.shape[2]
    w, b = _params(c, weight, bias, x.device)
    mean = _by_group(x, groups)
    d = x - _spread(mean, c)
    var = _by_group(d * d, groups)
    rstd = 1 / torch.sqrt(var + eps)
    h = d * _spread(rstd, c)
    z = h * w + b
    y = act(z, kind)
    emean = RUN * U * _by_group(x.abs(), groups)
    # squares: three roundings and the chain; a thread's pivot costs as much again
    evar = 2 * RUN * U * var + emean ** 2
    erstd = rstd * (0.5 * evar / (var + eps) + 4 * U)
    eh = (_spread(rstd * emean, c) + U * (x.abs() + _spread(mean.abs(), c)) * _spread(rstd, c)
          + h.abs() * (_spread(erstd / rstd, c) + 3 * U))
    ez = eh * w.abs() + 3 * U * (z.abs() + b.abs())
    # the exponential's argument is off by half a unit of its size; |silu'| < 1.1
    ey = ez if kind != 2 else 1.1 * ez + y.abs() * (10 + 3 * z.abs()) * U + 2.0 ** -120
    return (y, mean, rstd), (ey, emean + U * mean.abs(), erstd)


def groupnorm_backward(dy, x, groups, weight, bias, kind, mean, rstd):
    """(dx, dweight, dbias) and bounds."""
    dy, x = dy.double().contiguous(), x.double().contiguous()
    c = x.shape[2]
    w, b = _params(c, weight, bias, x.device)
    m, r = _spread(mean.double(), c), _spread(rstd.double(), c)
    h = (x - m) * r
    z = h * w + b
    dz = dy * dact(z, kind)
    q = dz * w
    s1, s2 = _spread(_by_group(q, groups), c), _spread(_by_group(q * h, groups), c)
    dx = r * (q - s1 - h * s2)
    eh = 3 * U * (x.abs() + m.abs()) * r
    edz = torch.zeros_like(dz)
    if kind == 2:  # |silu''| <= 1/2; the sigmoid's own roundings
        ez = eh * w.abs() + 3 * U * (z.abs() + b.abs())
        edz = dy.abs() * (0.5 * ez + (12 + 6 * z.abs()) * U)
    e1 = _spread(_by_group(RUN * U * q.abs() + edz * w.abs(), groups), c)
    e2 = _spread(_by_group(RUN * U * (q * h).abs() + edz * (w * h).abs() + q.abs() * eh, groups), c)
    edx = r * (4 * U * (q.abs() + s1.abs() + (h * s2).abs()) + edz * w.abs() + e1 + h.abs() * e2
               + eh * s2.abs()) + 3 * U * dx.abs()
    edw = (RUN * U * (dz * h).abs() + edz * h.abs() + dz.abs() * eh).sum((0, 1))
    edb = (RUN * U * dz.abs() + edz).sum((0, 1))
    return (dx, (dz * h).sum((0, 1)), dz.sum((0, 1))), (edx, edw, edb)


def router(logits, sequences, lengths, k, normalise, per_sequence):
    """The eight outputs by name, and bounds of the computed ones."""
    x = logits.double()
    rows, e = x.shape
    dev = x.device
    at = torch.arange(rows, device=dev)
    live = (x != -torch.inf).any(1)
    if lengths is not None:
        tokens = rows // sequences
        live &= at % tokens < lengths.long()[at // tokens]
    groups = sequences if per_sequence else 1
    group = at // max(1, rows // max(1, groups))
    lse = torch.where(live, torch.logsumexp(x, 1), -torch.inf)
    top = x.amax(1, keepdim=True)
    # not from lse: among the largest numbers its last bits are more than a logarithm
    p = torch.where(live[:, None], torch.softmax(x, 1), 0.0)
    # by value from the largest, equal ones by place
    order = torch.sort(x, dim=1, descending=True, stable=True)[1][:, :k]
    taken = live[:, None] & (x.gather(1, order) > -torch.inf)
    chosen = torch.where(taken, order, -1).int()
    weights = torch.where(taken, p.gather(1, order), 0.0)
    total = weights.sum(1, keepdim=True)
    if normalise:
        weights = torch.where(total > 0, weights / total, 0.0)
    counts = torch.bincount((group[:, None] * e + order)[taken], minlength=groups * e)
    counts = counts.view(groups, e)
    routed = torch.bincount(group[live], minlength=groups)
    n = routed.clamp(min=1).double()
    probs = torch.zeros(groups, e, dtype=torch.float64, device=dev).index_add_(0, group, p)
    probs = probs / n[:, None]
    square = torch.zeros(groups, dtype=torch.float64, device=dev)
    square.index_add_(0, group, torch.where(live, lse, 0.0) ** 2)
    loss = torch.stack((((counts * probs).sum(1) * e / (k * n)).sum(),
                        (square / n).sum())) / max(1, groups)
    out = {"chosen": chosen, "weights": weights, "lse": lse, "counts": counts.int(),
           "routed": routed.int(), "probs": probs, "loss": loss}
    # an exponential: 2 roundings of its own, one of its argument's size; a row's sum: E / 32
    # in a row, a tree of 5
    far = (x - top).abs()
    far = torch.where(far < 110, far, 0.0)  # what lies further is 0 in fp32
    term = (far + e / 32 + 20) * U
    eall = torch.where(live, term.amax(1), 0.0)
    low = 2.0 ** -126
    bound = {"weights": 2 * weights * eall[:, None] + low,
             "lse": torch.where(live, eall + 3 * U * lse.abs(), 0.0),
             "probs": probs * (2 * (eall.max() if rows else 0) + RUN * U) + low,
             "loss": loss * (3 * (eall.max() if rows else 0) + 2 * RUN * U) + 2.0 ** -100}
    return out, bound


def router_backward(logits, sequences, k, normalise, per_sequence, chosen, weights, lse, counts,
                    routed, dweights, dloss):
    """dlogits and its bound."""
    x = logits.double()
    rows, e = x.shape
    groups = sequences if per_sequence else 1
    group = torch.arange(rows, device=x.device) // max(1, rows // max(1, groups))
    lse = lse.double()
    live = lse > -torch.inf
    lse = torch.where(live, lse, 0.0)
    p = torch.where(live[:, None], torch.softmax(x, 1), 0.0)
    n = routed.clamp(min=1).double()
    d0, d1 = (0.0, 0.0) if dloss is None else (float(dloss[0]), float(dloss[1]))
    c = (d0 * counts.double() * e / (k * n * n * groups)[:, None])[group]
    z = (2 * d1 * lse / (groups * n[group]))[:, None]
    taken = chosen >= 0
    at = chosen.clamp(min=0).long()
    w = weights.double()
    dw = torch.zeros_like(w) if dweights is None else torch.where(taken, dweights.double(), 0.0)
    inner = (w * dw).sum(1, keepdim=True)
    mean = (p * c).sum(1, keepdim=True)
    if normalise:
        v = torch.zeros_like(p).scatter_add_(1, at, torch.where(taken, w * (dw - inner), 0.0))
        factor = c.abs() + (p * c.abs()).sum(1, keepdim=True) + z.abs()
        sizev = w * (dw.abs() + (w * dw).abs().sum(1, keepdim=True))
    else:
        v = torch.zeros_like(p).scatter_add_(1, at, w * dw) - p * inner
        factor = (c.abs() + (p * c.abs()).sum(1, keepdim=True) + z.abs()
                  + (w * dw).abs().sum(1, keepdim=True))
        sizev = w * dw.abs()
    out = p * (c - mean + z) + v
    far = torch.where(live[:, None], (x - lse[:, None]).abs(), 0.0)
    far = torch.where(far < 110, far, 0.0)
    add = (e / 32 + 30 + far.amax(1, keepdim=True) + 2 * lse.abs()[:, None]) * U
    # a probability below 2^-126 is taken as 0: what it would have been multiplied by, times
    # that (and a product below 2^-126 may itself be 0)
    bound = (add * (p * factor + torch.zeros_like(p).scatter_add_(1, at, sizev * taken))
             + 2.0 ** -126 * (1 + factor))
    return torch.where(live[:, None], out, 0.0), torch.where(live[:, None], bound, 0.0)
