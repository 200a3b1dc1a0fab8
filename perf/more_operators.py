"""What is measured of the operators that a worker's model has beside its products:
group norm with an activation over channels-last images, both passes, and the
router of a mixture of experts with its balance loss and per-expert counts,
both passes.

`own` false: the plain form, elementary torch operations in fp32, rounded once
at the end.  `own` true: the calls of gradient_aggregation_gb300.fc.
"""

import math
import random

import torch

own = False

GN_EPS = 1e-5
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}
MOST = 1 << 27  # elements of the largest case


def listed():
    return [
        # one small feature map while a single image is answered: latency
        {"name": "gn_fwd_one_image_bf16", "op": "gn_fwd", "samples": 1, "positions": 64,
         "channels": 256, "groups": 32, "pad": 0, "type": "bf16", "param": "bf16",
         "affine": True, "act": "silu"},
        # 55 x 55 maps of 96 channels (the AlexNet-shaped workload's first layer), 3 to a group
        {"name": "gn_fwd_odd_f16", "op": "gn_fwd", "samples": 128, "positions": 3025,
         "channels": 96, "groups": 32, "pad": 0, "type": "f16", "param": "f32",
         "affine": True, "act": "relu"},
        # a training batch of 64 x 64 maps
        {"name": "gn_fwd_large_bf16", "op": "gn_fwd", "samples": 64, "positions": 4096,
         "channels": 512, "groups": 32, "pad": 0, "type": "bf16", "param": "f32",
         "affine": True, "act": "silu"},
        # 7 x 7 maps of 1024 channels in fp32: latency
        {"name": "gn_bwd_small_f32", "op": "gn_bwd", "samples": 4, "positions": 49,
         "channels": 1024, "groups": 32, "pad": 0, "type": "f32", "param": "f32",
         "affine": True, "act": "none", "grad": "f32"},
        # 13 x 13 maps of 384 channels (the AlexNet-shaped workload's third layer), parameter
        # gradients in the engine's fp16
        {"name": "gn_bwd_mid_f16", "op": "gn_bwd", "samples": 64, "positions": 169,
         "channels": 384, "groups": 32, "pad": 0, "type": "f16", "param": "f16",
         "affine": True, "act": "relu", "grad": "f16"},
        # a training batch of 64 x 64 maps
        {"name": "gn_bwd_large_bf16", "op": "gn_bwd", "samples": 64, "positions": 4096,
         "channels": 512, "groups": 32, "pad": 0, "type": "bf16", "param": "f32",
         "affine": True, "act": "silu", "grad": "f32"},
        # a handful of tokens and experts: latency
        {"name": "router_fwd_small_f32", "op": "router_fwd", "sequences": 1, "tokens": 64,
         "experts": 8, "k": 2, "pad": 0, "type": "f32", "normalise": True,
         "per_sequence": False, "length_seed": -1, "masked": False},
        # a padded batch of sequences, each balanced by itself, an odd number of experts
        {"name": "router_fwd_padded_f32", "op": "router_fwd", "sequences": 16, "tokens": 2048,
         "experts": 60, "k": 4, "pad": 0, "type": "f32", "normalise": False,
         "per_sequence": True, "length_seed": 3, "masked": False},
        # a training batch's tokens over many experts
        {"name": "router_fwd_large_bf16", "op": "router_fwd", "sequences": 32, "tokens": 4096,
         "experts": 256, "k": 8, "pad": 0, "type": "bf16", "normalise": True,
         "per_sequence": False, "length_seed": -1, "masked": False},
        # a handful of tokens and experts: latency
        {"name": "router_bwd_small_f32", "op": "router_bwd", "sequences": 1, "tokens": 64,
         "experts": 8, "k": 2, "pad": 0, "type": "f32", "normalise": True,
         "per_sequence": False, "length_seed": -1, "masked": False},
        # a padded batch of sequences, each balanced by itself, an odd number of experts
        {"name": "router_bwd_padded_f32", "op": "router_bwd", "sequences": 16, "tokens": 2048,
         "experts": 60, "k": 4, "pad": 0, "type": "f32", "normalise": False,
         "per_sequence": True, "length_seed": 3, "masked": False},
        # a training batch's tokens over many experts
        {"name": "router_bwd_large_bf16", "op": "router_bwd", "sequences": 32, "tokens": 4096,
         "experts": 256, "k": 8, "pad": 0, "type": "bf16", "normalise": True,
         "per_sequence": False, "length_seed": -1, "masked": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("gn_fwd", "gn_bwd", "router_fwd", "router_bwd"))
    case = {"op": op, "pad": rng.choice((0, 0, 0, 8, 24, 5)),
            "type": rng.choice(("bf16", "bf16", "f16", "f32"))}
    if op in ("gn_fwd", "gn_bwd"):
        channels = _log(rng, 8, 2048)
        if rng.random() < 0.7:
            channels = max(16, channels // 16 * 16)
        positions = _log(rng, 1, 65536)
        if positions * channels > 1 << 26:
            positions = (1 << 26) // channels
        samples = _log(rng, 1, max(1, min(512, (MOST >> 1) // (positions * channels))))
        # at least 16 elements to a group
        fits = [g for g in (1, 2, 4, 8, 16, 32, 64, channels)
                if channels % g == 0 and channels // g * positions >= 16]
        if not fits:
            positions, fits = positions + 15, [1]
        case |= {"samples": samples, "positions": positions, "channels": channels,
                 "groups": rng.choice(fits[-4:]), "affine": rng.random() < 0.85,
                 "param": rng.choice(("f32", case["type"])),
                 "act": rng.choice(("silu", "silu", "relu", "none"))}
        if op == "gn_bwd":
            case["grad"] = rng.choice(("f32", case["type"]))
        return case
    experts = _log(rng, 2, 512)
    if rng.random() < 0.6:
        experts = max(2, experts // 8 * 8)
    sequences = _log(rng, 1, 64)
    tokens = _log(rng, 1, min(131072 // sequences, (1 << 25) // (experts * sequences)))
    return case | {
        "sequences": sequences, "tokens": tokens, "experts": experts,
        "k": min(experts, rng.choice((1, 2, 2, 4, 6, 8, 8))), "normalise": rng.random() < 0.5,
        "per_sequence": rng.random() < 0.4,
        "length_seed": rng.choice((-1, -1, rng.randrange(1 << 30))),
        "masked": rng.random() < 0.15}


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


# ---- group norm's inputs ------------------------------------------------------------

def _prepare_groupnorm(case, seed):
    gen, dtype = _generator(seed), DTYPES[case["type"]]
    n, s, c, pad = case["samples"], case["positions"], case["channels"], case["pad"]
    groups = case["groups"]

    def images(scale):
        # drawn in the output's own type: nothing is as large as an fp32 copy
        m = torch.randn(n, s, c + pad, generator=gen, device="cuda", dtype=dtype)
        return m.mul_(scale)[:, :, :c]

    def empty():
        return torch.empty(n, s, c + pad, device="cuda", dtype=dtype)[:, :, :c]

    x = images(1.5)
    # each channel has a mean of its own
    x.add_(torch.randn(c, generator=gen, device="cuda").to(dtype))
    state = {"case": case, "x": x, "weight": None, "bias": None}
    if case["affine"]:
        param = DTYPES[case["param"]]
        state["weight"] = (1 + 0.1 * torch.randn(c, generator=gen, device="cuda")).to(param)
        state["bias"] = (0.1 * torch.randn(c, generator=gen, device="cuda")).to(param)
    if own:
        from gradient_aggregation_gb300 import fc
        state["workspace"] = torch.empty(fc.fc_groupnorm_workspace_size(n, s, c, groups),
                                         dtype=torch.uint8, device="cuda")
    if case["op"] == "gn_fwd":
        return state | {"y": empty(), "mean": torch.empty(n, groups, device="cuda"),
                        "rstd": torch.empty(n, groups, device="cuda")}
    state["dy"] = images(0.5)
    mean, rstd = [], []
    for i in range(n):  # one by one: no fp32 copy of the whole
        g = x[i].float().view(s, groups, c // groups)
        m = g.mean((0, 2), keepdim=True)
        mean.append(m.view(-1))
        rstd.append(torch.rsqrt((g - m).square().mean((0, 2)) + GN_EPS))
    state["mean"], state["rstd"] = torch.stack(mean), torch.stack(rstd)
    state["dx"], state["dweight"], state["dbias"] = empty(), None, None
    if case["affine"]:
        state["dweight"] = torch.empty(c, device="cuda", dtype=DTYPES[case["grad"]])
        state["dbias"] = torch.empty(c, device="cuda", dtype=DTYPES[case["grad"]])
    return state


# ---- the router's inputs --------------------------------------------------------------

def _lengths(case):
    """Tokens of each sequence: all, or for a padded batch anything from none to all."""
    count, most = case["sequences"], case["tokens"]
    if case["length_seed"] < 0:
        return [most] * count
    rng = random.Random(case["length_seed"])
    return [0 if rng.random() < 0.05 else rng.randint(1, most) for _ in range(count)]


def _prepare_router(case, seed):
    gen, dtype = _generator(seed), DTYPES[case["type"]]
    rows, e, k, pad = case["sequences"] * case["tokens"], case["experts"], case["k"], case["pad"]
    logits = torch.randn(rows, e + pad, generator=gen, device="cuda", dtype=dtype)[:, :e]
    # some experts are liked better than others
    logits.add_((0.7 * torch.randn(e, generator=gen, device="cuda")).to(dtype))
    if case["masked"]:
        # every token may go to the experts of about half of the places only
        shut = torch.rand(rows, e, generator=gen, device="cuda") < 0.5
        logits.masked_fill_(shut, -math.inf)
    padded = case["length_seed"] >= 0
    state = {"case": case, "logits": logits, "lengths": None}
    if padded:
        state["lengths"] = torch.tensor(_lengths(case), dtype=torch.int32, device="cuda")
    groups = case["sequences"] if case["per_sequence"] else 1
    if case["op"] == "router_fwd":
        new = dict(device="cuda", dtype=torch.float32)
        state |= {"experts": torch.empty(rows, k, dtype=torch.int32, device="cuda"),
                  "weights": torch.empty(rows, k, **new), "lse": torch.empty(rows, **new),
                  "counts": torch.empty(groups, e, dtype=torch.int32, device="cuda"),
                  "routed": torch.empty(groups, dtype=torch.int32, device="cuda"),
                  "probs": torch.empty(groups, e, **new), "loss": torch.empty(2, **new)}
        if own:
            from gradient_aggregation_gb300 import fc
            size = fc.fc_router_workspace_size(case["sequences"], case["tokens"], e,
                                               case["per_sequence"])
            state["workspace"] = torch.empty(size, dtype=torch.uint8, device="cuda")
        return state
    # what the forward pass left
    state |= {q: v for q, v in _router_fwd_plain(state).items() if q not in ("probs", "loss")}
    state["dweights"] = torch.randn(rows, k, generator=gen, device="cuda") * (1.0 / rows)
    state["dloss"] = torch.tensor([0.01, 0.001], device="cuda")
    state["dlogits"] = torch.empty(rows, e + pad, device="cuda", dtype=dtype)[:, :e]
    if dtype == torch.float16:  # the gradients of a scaled loss
        state["dweights"] *= 1024.0
        state["dloss"] *= 1024.0
    return state


def prepare(case, seed):
    if case["op"] in ("gn_fwd", "gn_bwd"):
        return _prepare_groupnorm(case, seed)
    return _prepare_router(case, seed)


# ---- the plain forms --------------------------------------------------------------------

def _gn_fwd_plain(s):
    case = s["case"]
    n, p, c, groups = case["samples"], case["positions"], case["channels"], case["groups"]
    x = s["x"].float().reshape(n, p, groups, c // groups)
    mean = x.mean((1, 3), keepdim=True)
    d = x - mean
    rstd = torch.rsqrt((d * d).mean((1, 3), keepdim=True) + GN_EPS)
    z = (d * rstd).view(n, p, c)
    if s["weight"] is not None:
        z = z * s["weight"].float() + s["bias"].float()
    if case["act"] == "relu":
        z = z.clamp(min=0)
    elif case["act"] == "silu":
        z = z / (1 + torch.exp(-z))
    return {"y": z.to(s["x"].dtype), "mean": mean.view(n, groups), "rstd": rstd.view(n, groups)}


def _gn_bwd_plain(s):
    case = s["case"]
    n, p, c, groups = case["samples"], case["positions"], case["channels"], case["groups"]
    mean, rstd = s["mean"].view(n, 1, groups, 1), s["rstd"].view(n, 1, groups, 1)
    h = ((s["x"].float().reshape(n, p, groups, c // groups) - mean) * rstd).view(n, p, c)
    dz = s["dy"].float()
    if case["act"] == "relu":
        # in 64 bits: which side of 0 a value lies on
        z = (s["x"].double().reshape(n, p, groups, c // groups) - mean) * rstd.double()
        z = z.view(n, p, c)
        if s["weight"] is not None:
            z = z * s["weight"].double() + s["bias"].double()
        dz = dz * (z > 0)
    elif case["act"] == "silu":
        z = h if s["weight"] is None else h * s["weight"].float() + s["bias"].float()
        sig = 1 / (1 + torch.exp(-z))
        dz = dz * (sig * (1 + z * (1 - sig)))
    out = {}
    g = dz
    if s["weight"] is not None:
        out["dweight"] = (dz * h).sum((0, 1)).to(s["dweight"].dtype)
        out["dbias"] = dz.sum((0, 1)).to(s["dbias"].dtype)
        g = dz * s["weight"].float()
    g, h = g.view(n, p, groups, c // groups), h.view(n, p, groups, c // groups)
    dx = rstd * (g - g.mean((1, 3), keepdim=True) - h * (g * h).mean((1, 3), keepdim=True))
    return out | {"dx": dx.view(n, p, c).to(s["x"].dtype)}


def _live(s):
    """Which tokens are routed: those inside their sequence, with an expert open to them."""
    case, x = s["case"], s["logits"]
    live = x.amax(1) > -math.inf
    if s["lengths"] is not None:
        at = torch.arange(case["tokens"], device="cuda")
        live = live & (at < s["lengths"][:, None]).view(-1)
    return live


def _router_fwd_plain(s):
    case = s["case"]
    e, k = case["experts"], case["k"]
    groups = case["sequences"] if case["per_sequence"] else 1
    live = _live(s)
    x = torch.where(live[:, None], s["logits"].float(), 0.0)
    top = x.amax(1, keepdim=True)
    p = torch.exp(x - top)
    total = p.sum(1, keepdim=True)
    p = p / total * live[:, None]
    lse = torch.where(live, (top + torch.log(total)).view(-1), -math.inf)
    # the largest first, equal ones by their place
    order = torch.sort(x, dim=1, descending=True, stable=True)[1][:, :k]
    open_ = (torch.gather(x, 1, order) > -math.inf) & live[:, None]
    weights = torch.gather(p, 1, order) * open_
    if case["normalise"]:
        weights = weights / torch.where(live, weights.sum(1), 1.0)[:, None]
    experts = torch.where(open_, order, -1).int()
    # per group: tokens, tokens of each expert, mean probability of each expert
    routed = live.view(groups, -1).sum(1)
    slot = torch.arange(groups, device="cuda").repeat_interleave(live.numel() // groups)
    slot = torch.where(open_, slot[:, None] * e + order, groups * e)
    counts = torch.zeros(groups * e + 1, dtype=torch.int64, device="cuda")
    counts = counts.index_add(0, slot.view(-1), torch.ones_like(slot.view(-1)))
    counts = counts[:-1].view(groups, e)
    each = routed.clamp(min=1)[:, None].float()
    probs = p.view(groups, -1, e).sum(1) / each
    share = counts.float() * (e / k) / each
    square = torch.where(live, lse, 0.0).square().view(groups, -1).sum(1, keepdim=True) / each
    loss = torch.stack(((share * probs).sum(), square.sum())) / groups
    return {"experts": experts, "weights": weights, "lse": lse, "counts": counts.int(),
            "routed": routed.int(), "probs": probs, "loss": loss}


def _router_bwd_plain(s):
    case = s["case"]
    e, k = case["experts"], case["k"]
    groups = case["sequences"] if case["per_sequence"] else 1
    live = (s["lse"] > -math.inf)[:, None]
    lse = torch.where(live, s["lse"][:, None], 0.0)
    p = torch.where(live, torch.exp(s["logits"].float() - lse), 0.0)
    rows = p.shape[0]
    each = s["routed"].clamp(min=1)[:, None].float()
    # what the balance loss asks of every probability of a group
    ask = s["dloss"][0] * (e / k) * s["counts"].float() / (each * each * groups)
    ask = ask.repeat_interleave(rows // groups, 0)
    per_token = (1 / (each * groups)).repeat_interleave(rows // groups, 0)
    z_part = 2 * s["dloss"][1] * lse * per_token
    chosen = s["experts"] >= 0
    at = s["experts"].clamp(min=0).long()
    w, dw = s["weights"], torch.where(chosen, s["dweights"], 0.0)
    inner = (w * dw).sum(1, keepdim=True)
    if case["normalise"]:
        d = p * (ask - (p * ask).sum(1, keepdim=True) + z_part)
        d = d.scatter_add(1, at, w * torch.where(chosen, dw - inner, 0.0))
    else:
        d = p * (ask - (p * ask).sum(1, keepdim=True) + z_part - inner)
        d = d.scatter_add(1, at, w * dw)
    return {"dlogits": d.to(s["logits"].dtype)}


PLAIN = {"gn_fwd": _gn_fwd_plain, "gn_bwd": _gn_bwd_plain, "router_fwd": _router_fwd_plain,
         "router_bwd": _router_bwd_plain}


# ---- the framework's calls ------------------------------------------------------------------

def _run_own(s):
    from gradient_aggregation_gb300 import fc
    case = s["case"]
    op = case["op"]
    if op == "gn_fwd":
        act = {"none": fc.FC_ACT_NONE, "relu": fc.FC_ACT_RELU, "silu": fc.FC_ACT_SILU}[case["act"]]
        fc.fc_groupnorm_forward(s["x"], case["groups"], s["weight"], s["bias"], GN_EPS, act,
                                s["y"], s["mean"], s["rstd"], s["workspace"])
        return {"y": s["y"], "mean": s["mean"], "rstd": s["rstd"]}
    if op == "gn_bwd":
        act = {"none": fc.FC_ACT_NONE, "relu": fc.FC_ACT_RELU, "silu": fc.FC_ACT_SILU}[case["act"]]
        fc.fc_groupnorm_backward(s["dy"], s["x"], case["groups"], s["weight"], s["bias"], act,
                                 s["mean"], s["rstd"], s["dx"], s["dweight"], s["dbias"],
                                 s["workspace"])
        if s["dweight"] is None:
            return {"dx": s["dx"]}
        return {"dx": s["dx"], "dweight": s["dweight"], "dbias": s["dbias"]}
    if op == "router_fwd":
        fc.fc_router_forward(s["logits"], case["sequences"], s["lengths"], case["normalise"],
                             case["per_sequence"], s["experts"], s["weights"], s["lse"],
                             s["counts"], s["routed"], s["probs"], s["loss"], s["workspace"])
        return {q: s[q] for q in ("experts", "weights", "lse", "counts", "routed", "probs",
                                  "loss")}
    fc.fc_router_backward(s["logits"], case["sequences"], case["normalise"],
                          case["per_sequence"], s["experts"], s["weights"], s["lse"], s["counts"],
                          s["routed"], s["dweights"], s["dloss"], s["dlogits"])
    return {"dlogits": s["dlogits"]}


def run(state):
    return _run_own(state) if own else PLAIN[state["case"]["op"]](state)


# ---- the work that no path can do without -----------------------------------------------------

def work(case):
    op, b = case["op"], BYTES[case["type"]]
    if op in ("gn_fwd", "gn_bwd"):
        size = case["samples"] * case["positions"] * case["channels"]
        stats = 8 * case["samples"] * case["groups"]
        param = BYTES[case["param"]] if case["affine"] else 0
        if op == "gn_fwd":
            return {"bytes": 2 * b * size + 2 * param * case["channels"] + stats,
                    "flops": 10 * size}
        grad = BYTES[case["grad"]] if case["affine"] else 0
        return {"bytes": 3 * b * size + 2 * (param + grad) * case["channels"] + stats,
                "flops": 20 * size}
    rows, e, k = case["sequences"] * case["tokens"], case["experts"], case["k"]
    live = sum(_lengths(case))
    groups = case["sequences"] if case["per_sequence"] else 1
    if op == "router_fwd":
        return {"bytes": b * live * e + 8 * rows * k + 4 * rows + 8 * groups * e + 4 * groups + 8,
                "flops": (8 + k) * live * e}
    taken = (8 if case["normalise"] else 12) + (4 if case["normalise"] else 0)
    return {"bytes": b * (live + rows) * e + taken * live * k + 4 * rows + 4 * groups * (e + 1) + 8,
            "flops": 8 * live * e}


# ---- the definitions in 64 bits -----------------------------------------------------------------

def _exact_groupnorm(case, seed):
    s = _prepare_groupnorm(case, seed)
    n, p, c, groups = case["samples"], case["positions"], case["channels"], case["groups"]
    w = b = None
    if s["weight"] is not None:
        w, b = s["weight"].double(), s["bias"].double()
    keep = {"y": [], "mean": [], "rstd": [], "dx": []}
    dweight = dbias = 0.0
    for i in range(n):  # one image after another
        x = s["x"][i].double().reshape(p, groups, c // groups).transpose(0, 1).reshape(groups, -1)
        if case["op"] == "gn_fwd":
            var, mean = torch.var_mean(x, dim=1, correction=0)
            rstd = 1 / torch.sqrt(var + GN_EPS)
            keep["mean"].append(mean)
            keep["rstd"].append(rstd)
        else:
            mean, rstd = s["mean"][i].double(), s["rstd"][i].double()
        h = (x - mean[:, None]) * rstd[:, None]
        h = h.view(groups, p, c // groups).transpose(0, 1).reshape(p, c)
        z = h if w is None else h * w + b
        if case["op"] == "gn_fwd":
            y = {"none": lambda t: t, "relu": torch.relu,
                 "silu": lambda t: t * torch.sigmoid(t)}[case["act"]](z)
            keep["y"].append(y)
            continue
        d = s["dy"][i].double()
        if case["act"] == "relu":
            d = torch.where(z > 0, d, 0.0)
        elif case["act"] == "silu":
            q = torch.sigmoid(z)
            d = d * (q + z * q * torch.sigmoid(-z))
        dweight, dbias = dweight + (d * h).sum(0), dbias + d.sum(0)
        if w is not None:
            d = d * w
        per = p * (c // groups)
        one = d.sum(0).view(groups, -1).sum(1) / per
        two = (d * h).sum(0).view(groups, -1).sum(1) / per
        spread = lambda t: t.repeat_interleave(c // groups)  # noqa: E731
        keep["dx"].append(spread(rstd) * (d - spread(one) - h * spread(two)))
    if case["op"] == "gn_fwd":
        return {q: torch.stack(keep[q]) for q in ("y", "mean", "rstd")}
    out = {"dx": torch.stack(keep["dx"])}
    return out if w is None else out | {"dweight": dweight, "dbias": dbias}


def _exact_router(case, seed):
    s = _prepare_router(case, seed)
    e, k, tokens = case["experts"], case["k"], case["tokens"]
    groups = case["sequences"] if case["per_sequence"] else 1
    x = s["logits"].double()
    rows = x.shape[0]
    where = torch.arange(rows, device=x.device)
    group_of = where // (rows // groups)
    if case["op"] == "router_fwd":
        live = torch.isfinite(x).any(1)
        if s["lengths"] is not None:
            live &= where % tokens < s["lengths"].long()[where // tokens]
        lse = torch.where(live, torch.logsumexp(x, 1), -math.inf)
        p = torch.where(live[:, None], torch.softmax(x, 1), 0.0)
        left, experts = x.clone(), []
        for _ in range(k):
            top = left.amax(1, keepdim=True)
            places = torch.where(left == top, torch.arange(e, device=x.device), e)
            first = places.amin(1)
            taken = live & (top.view(-1) > -math.inf)
            experts.append(torch.where(taken, first, -1))
            left.scatter_(1, first[:, None], -math.inf)
        experts = torch.stack(experts, 1)
        chosen = experts >= 0
        weights = torch.where(chosen, p.gather(1, experts.clamp(min=0)), 0.0)
        if case["normalise"]:
            norm = weights.sum(1, keepdim=True)
            weights = torch.where(norm > 0, weights / torch.where(norm > 0, norm, 1.0), 0.0)
        flat = (group_of[:, None] * e + experts)[chosen]
        counts = torch.bincount(flat, minlength=groups * e).view(groups, e)
        routed = torch.bincount(group_of[live], minlength=groups)
        probs = torch.zeros(groups, e, dtype=torch.float64, device=x.device)
        probs.index_add_(0, group_of, p)
        z = torch.zeros(groups, dtype=torch.float64, device=x.device)
        z.index_add_(0, group_of, torch.where(live, lse, 0.0) ** 2)
        n = routed.clamp(min=1).double()
        probs = probs / n[:, None]
        balance = (probs * counts.double() * e).sum(1) / (k * n)
        loss = torch.stack((balance.mean(), (z / n).mean()))
        return {"experts": experts.int(), "weights": weights, "lse": lse, "counts": counts.int(),
                "routed": routed.int(), "probs": probs, "loss": loss}
    lse = s["lse"].double()
    live = lse > -math.inf
    p = torch.where(live[:, None], torch.exp(x - torch.where(live, lse, 0.0)[:, None]), 0.0)
    n = s["routed"].clamp(min=1).double()
    want = s["counts"].double() / (k * n)[:, None] * e  # the shares f
    # the derivative by each probability, then through the softmax
    dp = float(s["dloss"][0]) / groups * (want / n[:, None])[group_of]
    chosen = s["experts"] >= 0
    at = s["experts"].clamp(min=0).long()
    dw = torch.where(chosen, s["dweights"].double(), 0.0)
    w = s["weights"].double()
    out = p * (float(s["dloss"][1]) * 2 / groups * torch.where(live, lse, 0.0) / n[group_of])[:, None]
    if case["normalise"]:
        # a softmax over the chosen ones alone
        out.scatter_add_(1, at, torch.where(chosen, w * (dw - (w * dw).sum(1, keepdim=True)), 0.0))
    else:
        dp = dp.scatter_add(1, at, dw)
    out += p * (dp - (p * dp).sum(1, keepdim=True))
    return {"dlogits": out}


def exact(case, seed):
    if case["op"] in ("gn_fwd", "gn_bwd"):
        return _exact_groupnorm(case, seed)
    return _exact_router(case, seed)
