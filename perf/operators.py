"""What is measured of the training-step operators beside the aggregation:
layer norm's two passes, the global gradient norm, and the AdamW step with
its states in 32 or in 8 bits.

`own` false: the plain form, elementary torch operations in fp32, rounded once
at the end.  `own` true: the calls of gradient_aggregation_gb300.fc.  The
optimiser's tensors live in the fused layout of the engine: L layers one
after another, without padding, in one vector of N elements; the gradients
are the L separate tensors that a backward pass leaves.
"""

import math
import random

import torch

own = False

BLOCK = 256         # elements that share one scale of an 8-bit state
TOP = 448.0         # largest e4m3 value
TINY = 2.0 ** -110  # a block whose largest moment is below this holds zeros
LR, WD, EPS, B1, B2 = 1e-4, 0.01, 1e-8, 0.9, 0.999
LN_EPS = 1e-5
STEPS_DONE = 100

# Layer sizes of the repository's Tiny and AlexNet-shaped workloads.
TINY_SIZES = "1728,131072,256"
ALEXNET_SIZES = ("34848,96,614400,256,884736,384,1327104,384,884736,256,"
                 "37748736,4096,16777216,4096,4096000,1000")

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}


def listed():
    return [
        # the gradient of a small model, as its backward pass leaves it
        {"name": "norm_tiny_f16", "op": "norm", "sizes": TINY_SIZES, "grad": "f16", "shift": 0,
         "loss_scale": 1024.0, "clip": 1.0, "overflow": False},
        # 16 large and small layers of the reduced fp32 gradient
        {"name": "norm_alexnet_f32", "op": "norm", "sizes": ALEXNET_SIZES, "grad": "f32",
         "shift": 0, "loss_scale": 1.0, "clip": 1.0, "overflow": False},
        # a small model's update: latency
        {"name": "adamw_tiny_f16", "op": "adamw", "sizes": TINY_SIZES, "grad": "f16", "shift": 0,
         "low": "f16", "overflow": False},
        # the AlexNet-shaped update from the reduced fp32 gradient
        {"name": "adamw_alexnet_f32", "op": "adamw", "sizes": ALEXNET_SIZES, "grad": "f32",
         "shift": 0, "low": "f16", "overflow": False},
        # 57 layers of odd sizes (the GoogLeNet-shaped workload's count and sum)
        {"name": "adamw8_odd_layers_bf16", "op": "adamw8", "layers": 57, "total": 6998552,
         "size_seed": 2, "grad": "bf16", "shift": 0, "low": "bf16", "overflow": False},
        # the AlexNet-shaped update with 8-bit states from fp16 gradients
        {"name": "adamw8_alexnet_f16", "op": "adamw8", "sizes": ALEXNET_SIZES, "grad": "f16",
         "shift": 0, "low": "f16", "overflow": False},
        # one token while a model answers: latency
        {"name": "ln_fwd_one_row_bf16", "op": "ln_fwd", "rows": 1, "cols": 4096, "pad": 0,
         "type": "bf16", "param": "bf16", "affine": True},
        # a width that is not a multiple of anything
        {"name": "ln_fwd_odd_f16", "op": "ln_fwd", "rows": 20000, "cols": 1001, "pad": 0,
         "type": "f16", "param": "f32", "affine": True},
        # a training batch of long sequences
        {"name": "ln_fwd_large_bf16", "op": "ln_fwd", "rows": 32768, "cols": 4096, "pad": 0,
         "type": "bf16", "param": "f32", "affine": True},
        # a short batch in fp32: latency
        {"name": "ln_bwd_small_f32", "op": "ln_bwd", "rows": 128, "cols": 256, "pad": 0,
         "type": "f32", "param": "f32", "affine": True, "grad": "f32"},
        # an ordinary batch, parameter gradients in the engine's fp16
        {"name": "ln_bwd_mid_f16", "op": "ln_bwd", "rows": 8192, "cols": 1024, "pad": 0,
         "type": "f16", "param": "f16", "affine": True, "grad": "f16"},
        # a training batch of long sequences
        {"name": "ln_bwd_large_bf16", "op": "ln_bwd", "rows": 32768, "cols": 4096, "pad": 0,
         "type": "bf16", "param": "f32", "affine": True, "grad": "f32"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("norm", "adamw", "adamw8", "ln_fwd", "ln_bwd"))
    if op in ("norm", "adamw", "adamw8"):
        total = _log(rng, 1000, 60_000_000)
        case = {"op": op, "layers": min(total // 4, _log(rng, 1, 600)), "total": total,
                "size_seed": rng.randrange(1 << 30), "grad": rng.choice(("f32", "f16", "bf16")),
                "shift": rng.choice((0, 0, 0, rng.randrange(1, 8))),
                "overflow": rng.random() < 0.08}
        if op == "norm":
            case |= {"loss_scale": rng.choice((1.0, 128.0, 1024.0)),
                     "clip": rng.choice((0.0, 0.5, 1.0, 1e6))}
        else:
            case |= {"low": rng.choice(("none", "f16", "bf16"))}
        return case
    cols = _log(rng, 32, 16384)
    if rng.random() < 0.6:
        cols = max(32, cols // 64 * 64)
    rows = _log(rng, 1, min(65536, (1 << 27) // cols))
    case = {"op": op, "rows": rows, "cols": cols, "pad": rng.choice((0, 0, 0, 8, 24, 5)),
            "type": rng.choice(("bf16", "bf16", "f16", "f32")), "affine": rng.random() < 0.85}
    if case["pad"] and rows * (cols + 24) > 1 << 27:
        case["pad"] = 0
    case["param"] = rng.choice(("f32", case["type"]))
    if op == "ln_bwd":
        case["grad"] = rng.choice(("f32", case["type"]))
    return case


def _sizes(case):
    if "sizes" in case:
        return [int(t) for t in case["sizes"].split(",")]
    rng = random.Random(case["size_seed"])
    layers, total = case["layers"], case["total"]
    raw = [math.exp(rng.uniform(0.0, math.log(10000.0))) for _ in range(layers)]
    f = total / sum(raw)
    sizes = [max(1, int(r * f)) for r in raw]
    big = sizes.index(max(sizes))
    sizes[big] += total - sum(sizes)
    return sizes


def _blocks(n):
    return -(-n // BLOCK)


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _layers(flat, sizes, shift):
    """The layers' own tensors: each starts `shift` elements past a 128-byte boundary."""
    at, views = 0, []
    for n in sizes:
        views.append(flat[at + shift: at + shift + n])
        at += -(-(n + shift) // 64) * 64
    return views


def _prepare_optimiser(case, seed):
    sizes = _sizes(case)
    n, gen = sum(sizes), _generator(seed)
    dtype = DTYPES[case["grad"]]
    loss_scale = case.get("loss_scale", 512.0 if case["grad"] == "f16" else 1.0)
    room = sum(-(-(k + case["shift"]) // 64) * 64 for k in sizes)
    flat = torch.randn(room, generator=gen, device="cuda")
    flat = flat.mul_(1e-3 * loss_scale).to(dtype)
    grads = _layers(flat, sizes, case["shift"])
    if case["op"] == "norm":
        if case["overflow"]:
            grads[len(grads) // 2][0] = math.inf
        s = {"case": case, "grads": grads, "norm": torch.zeros(1, device="cuda"),
             "scale": torch.zeros(1, device="cuda")}
        if own:
            from gradient_aggregation_gb300 import fc
            s["table"] = fc.LayerGrads(grads)
            s["workspace"] = torch.zeros(fc.fc_grad_norm_workspace_size(), dtype=torch.uint8,
                                         device="cuda")
        return s
    # small layers (biases, norm weights) are not decayed
    decay = [1.0 if k > 4096 else 0.0 for k in sizes]
    s = {"case": case, "grads": grads, "n": n, "seed": int(seed) * 2654435761 % (1 << 63),
         "decay": torch.repeat_interleave(torch.tensor(decay, device="cuda"),
                                          torch.tensor(sizes, device="cuda")),
         "weights": torch.randn(n, generator=gen, device="cuda") * 0.05,
         "low": None if case["low"] == "none" else torch.empty(n, dtype=DTYPES[case["low"]], device="cuda"),
         "grad_scale": torch.tensor([math.nan if case["overflow"] else 0.7 / loss_scale], device="cuda"),
         "steps": torch.tensor([STEPS_DONE, 0], dtype=torch.int32, device="cuda")}
    if own:
        from gradient_aggregation_gb300 import fc
        s["table"] = fc.LayerGrads(grads, decay)
    padded = _blocks(n) * BLOCK if case["op"] == "adamw8" else n
    m = torch.randn(padded, generator=gen, device="cuda") * 3e-4
    v = (torch.rand(padded, generator=gen, device="cuda") + 0.1) * 1e-6
    m[n:] = 0
    v[n:] = 0
    if case["op"] == "adamw":
        return s | {"m": m, "v": v}
    s["m8"], s["m_scale"] = _to_8_bits(m)
    s["r8"], s["r_scale"] = _to_8_bits(v.sqrt())
    return s


def _to_8_bits(x):
    x = x.view(-1, BLOCK)
    top = x.abs().amax(1)
    inv = torch.where(top >= TINY, TOP / top, 0.0)
    q = (x * inv[:, None]).clamp_(-TOP, TOP).to(torch.float8_e4m3fn)
    return q.view(-1), torch.where(top >= TINY, top * (1 / TOP), 0.0)


def _prepare_layernorm(case, seed):
    gen, dtype = _generator(seed), DTYPES[case["type"]]
    rows, cols, pad = case["rows"], case["cols"], case["pad"]

    def matrix(scale, shift):
        # drawn in the output's own type: nothing is as large as an fp32 copy
        m = torch.randn(rows, cols + pad, generator=gen, device="cuda", dtype=dtype)
        return m.mul_(scale).add_(shift)[:, :cols]

    def empty():
        return torch.empty(rows, cols + pad, device="cuda", dtype=dtype)[:, :cols]

    s = {"case": case, "x": matrix(1.5, 0.25), "weight": None, "bias": None}
    if case["affine"]:
        param = DTYPES[case["param"]]
        s["weight"] = (1 + 0.1 * torch.randn(cols, generator=gen, device="cuda")).to(param)
        s["bias"] = (0.1 * torch.randn(cols, generator=gen, device="cuda")).to(param)
    if case["op"] == "ln_fwd":
        return s | {"y": empty(), "mean": torch.empty(rows, device="cuda"),
                    "rstd": torch.empty(rows, device="cuda")}
    s["dy"] = matrix(0.5, 0.0)
    x = s["x"]
    s["mean"] = x.mean(1, dtype=torch.float32)
    s["rstd"] = torch.empty(rows, device="cuda")
    for a in range(0, rows, 4096):  # in pieces: no fp32 copy of the whole
        c = x[a:a + 4096].float() - s["mean"][a:a + 4096, None]
        s["rstd"][a:a + 4096] = torch.rsqrt(c.square_().mean(1) + LN_EPS)
    s["dx"] = empty()
    if case["affine"]:
        s["dweight"] = torch.empty(cols, device="cuda", dtype=DTYPES[case["grad"]])
        s["dbias"] = torch.empty(cols, device="cuda", dtype=DTYPES[case["grad"]])
    else:
        s["dweight"] = s["dbias"] = None
    if own:
        from gradient_aggregation_gb300 import fc
        s["workspace"] = torch.empty(fc.fc_layernorm_backward_workspace_size(rows, cols),
                                     dtype=torch.uint8, device="cuda")
    return s


def prepare(case, seed):
    if case["op"] in ("norm", "adamw", "adamw8"):
        return _prepare_optimiser(case, seed)
    return _prepare_layernorm(case, seed)


# ---- the plain forms ----------------------------------------------------------

def _flat(grads, more=0):
    parts = [g.reshape(-1) for g in grads]
    if more:
        parts.append(torch.zeros(more, dtype=parts[0].dtype, device="cuda"))
    return torch.cat(parts).float()


def _norm_plain(s):
    case = s["case"]
    norm = _flat(s["grads"]).square().sum(dtype=torch.float32).sqrt() / case["loss_scale"]
    clip = torch.clamp(case["clip"] / norm, max=1.0) if case["clip"] > 0 else torch.ones_like(norm)
    scale = torch.where(torch.isfinite(norm), clip / case["loss_scale"], math.nan)
    return {"norm": norm.reshape(1), "scale": scale.reshape(1)}


def _moments_plain(s, g, m, v):
    """The new moments and weights, before any step is skipped."""
    t = (s["steps"][0] + 1).float()
    c1, c2 = -torch.expm1(t * math.log(B1)), -torch.expm1(t * math.log(B2))
    m = m * B1 + g * (1 - B1)
    v = v * B2 + g * g * (1 - B2)
    n = s["n"]
    root = v.sqrt()
    w = s["weights"] * (1 - LR * WD * s["decay"])
    w = w - (LR / c1) * m[:n] / (root[:n] / c2.sqrt() + EPS)
    return m, v, root, w


def _finish_plain(s, applied, w):
    s["weights"] = torch.where(applied, w, s["weights"])
    s["steps"] = s["steps"] + torch.stack((applied[0], torch.zeros_like(applied[0])))
    out = {"weights": s["weights"], "steps": s["steps"]}
    if s["low"] is not None:
        out["low"] = s["weights"].to(s["low"].dtype)
    return out


def _adamw_plain(s):
    applied = torch.isfinite(s["grad_scale"])
    g = _flat(s["grads"]) * s["grad_scale"]
    m, v, _, w = _moments_plain(s, g, s["m"], s["v"])
    s["m"], s["v"] = torch.where(applied, m, s["m"]), torch.where(applied, v, s["v"])
    return _finish_plain(s, applied, w) | {"m": s["m"], "v": s["v"]}


def _mix(x):
    """A mixing of 32 bits held in int64: multiply and xor-shift, twice."""
    x = x & 0xFFFFFFFF
    x = ((x ^ (x >> 16)) * 0x7FEB352D) & 0xFFFFFFFF
    x = ((x ^ (x >> 15)) * 0x846CA68B) & 0xFFFFFFFF
    return x ^ (x >> 16)


def _stochastic_e4m3(y, seed, t):
    """e4m3 of values in [0, 448], rounded up with the probability of what is cut off; a
    value above 0 never becomes 0."""
    key = _mix((seed & 0xFFFFFFFF) ^ _mix((seed >> 32) ^ _mix(t.long())))
    pair = torch.arange(y.numel() // 2, device="cuda")
    h = _mix((pair & 0xFFFFFFFF) + key + (pair >> 32) * 0x9E3779B9)
    bits = torch.stack((h & 0xFFFF, h >> 16), 1).view(-1) * 16 + 8
    base = torch.where(y < 2.0 ** -6, 2.0 ** -6, 0.0)
    cut = ((y + base).view(torch.int32) + bits.int()) & ~0xFFFFF
    q = cut.view(torch.float32) - base
    return torch.where(y > 0, q.clamp(min=2.0 ** -9), 0.0).to(torch.float8_e4m3fn)


def _adamw8_plain(s):
    applied = torch.isfinite(s["grad_scale"])
    m8, r8, n = s["m8"], s["r8"], s["n"]
    g = _flat(s["grads"], m8.numel() - n) * s["grad_scale"]
    m = (m8.float().view(-1, BLOCK) * s["m_scale"][:, None]).view(-1)
    r = (r8.float().view(-1, BLOCK) * s["r_scale"][:, None]).view(-1)
    m, _, root, w = _moments_plain(s, g, m, r * r)
    new_m8, m_scale = _to_8_bits(m)
    root = root.view(-1, BLOCK)
    top = root.amax(1)
    inv = torch.where(top >= TINY, TOP / top, 0.0)
    y = (root * inv[:, None]).clamp_(max=TOP).view(-1)
    new_r8 = _stochastic_e4m3(y, s["seed"], s["steps"][0] + 1)
    r_scale = torch.where(top >= TINY, top * (1 / TOP), 0.0)

    def keep(new, old):
        return torch.where(applied, new.view(torch.uint8), old.view(torch.uint8)).view(new.dtype)

    s["m8"], s["r8"] = keep(new_m8, m8), keep(new_r8, r8)
    s["m_scale"] = torch.where(applied, m_scale, s["m_scale"])
    s["r_scale"] = torch.where(applied, r_scale, s["r_scale"])
    return _finish_plain(s, applied, w) | {"m8": s["m8"][:n], "r8": s["r8"][:n],
                                           "m_scale": s["m_scale"], "r_scale": s["r_scale"]}


def _ln_fwd_plain(s):
    x = s["x"].float()
    mean = x.mean(1, keepdim=True)
    c = x - mean
    rstd = torch.rsqrt((c * c).mean(1, keepdim=True) + LN_EPS)
    y = c * rstd
    if s["weight"] is not None:
        y = y * s["weight"].float() + s["bias"].float()
    return {"y": y.to(s["x"].dtype), "mean": mean.view(-1), "rstd": rstd.view(-1)}


def _ln_bwd_plain(s):
    dy, rstd = s["dy"].float(), s["rstd"][:, None]
    h = (s["x"].float() - s["mean"][:, None]) * rstd
    out = {}
    g = dy
    if s["weight"] is not None:
        g = dy * s["weight"].float()
        out["dweight"] = (dy * h).sum(0).to(s["dweight"].dtype)
        out["dbias"] = dy.sum(0).to(s["dbias"].dtype)
    dx = (g - g.mean(1, keepdim=True) - h * (g * h).mean(1, keepdim=True)) * rstd
    return out | {"dx": dx.to(s["x"].dtype)}


PLAIN = {"norm": _norm_plain, "adamw": _adamw_plain, "adamw8": _adamw8_plain,
         "ln_fwd": _ln_fwd_plain, "ln_bwd": _ln_bwd_plain}


# ---- the framework's calls --------------------------------------------------------

def _run_own(s):
    from gradient_aggregation_gb300 import fc
    case = s["case"]
    op = case["op"]
    if op == "norm":
        fc.fc_grad_norm(s["table"], case["loss_scale"], case["clip"], s["norm"], s["scale"],
                        s["workspace"])
        return {"norm": s["norm"], "scale": s["scale"]}
    if op == "adamw":
        fc.fc_adamw_step(s["table"], s["grad_scale"], LR, B1, B2, EPS, WD, s["weights"], s["low"],
                         s["m"], s["v"], s["steps"])
        out = {"weights": s["weights"], "steps": s["steps"], "m": s["m"], "v": s["v"]}
        return out if s["low"] is None else out | {"low": s["low"]}
    if op == "adamw8":
        n = s["n"]
        fc.fc_adamw8_step(s["table"], s["grad_scale"], LR, B1, B2, EPS, WD, s["weights"], s["low"],
                          s["m8"], s["m_scale"], s["r8"], s["r_scale"], s["steps"], s["seed"])
        out = {"weights": s["weights"], "steps": s["steps"], "m8": s["m8"][:n], "r8": s["r8"][:n],
               "m_scale": s["m_scale"], "r_scale": s["r_scale"]}
        return out if s["low"] is None else out | {"low": s["low"]}
    if op == "ln_fwd":
        fc.fc_layernorm_forward(s["x"], s["weight"], s["bias"], LN_EPS, s["y"], s["mean"],
                                s["rstd"])
        return {"y": s["y"], "mean": s["mean"], "rstd": s["rstd"]}
    fc.fc_layernorm_backward(s["dy"], s["x"], s["weight"], s["mean"], s["rstd"], s["dx"],
                             s["dweight"], s["dbias"], s["workspace"])
    if s["dweight"] is None:
        return {"dx": s["dx"]}
    return {"dx": s["dx"], "dweight": s["dweight"], "dbias": s["dbias"]}


def run(state):
    return _run_own(state) if own else PLAIN[state["case"]["op"]](state)


# ---- the work that no path can do without ------------------------------------------

def work(case):
    op = case["op"]
    if op in ("norm", "adamw", "adamw8"):
        n = sum(_sizes(case))
        g = BYTES[case["grad"]] * n
        if op == "norm":
            return {"bytes": g + 8, "flops": 2 * n}
        low = 0 if case["low"] == "none" else 2 * n
        if op == "adamw":
            return {"bytes": g + 24 * n + low, "flops": 16 * n}
        return {"bytes": g + 12 * n + low + 16 * _blocks(n), "flops": 24 * n}
    size = case["rows"] * case["cols"]
    b = BYTES[case["type"]]
    param = BYTES[case["param"]] if case["affine"] else 0
    if op == "ln_fwd":
        return {"bytes": 2 * b * size + 2 * param * case["cols"] + 8 * case["rows"],
                "flops": 8 * size}
    grad = BYTES[case["grad"]] if case["affine"] else 0
    return {"bytes": 3 * b * size + (param + 2 * grad) * case["cols"] + 8 * case["rows"],
            "flops": 14 * size}


# ---- the definitions in 64 bits -----------------------------------------------------

def _round_e4m3(x):
    """Nearest e4m3 value of a float64 in [-448, 448], ties to even, in float64."""
    _, e = torch.frexp(x)
    quantum = torch.ldexp(torch.ones_like(x), torch.clamp(e - 4, min=-9))
    return torch.round(x / quantum) * quantum


def _chance_e4m3(y, chance):
    """e4m3 value next below y >= 0 or the one above it, as `chance` in (0, 1) says."""
    _, e = torch.frexp(y)
    quantum = torch.ldexp(torch.ones_like(y), torch.clamp(e - 4, min=-9))
    q = torch.floor(y / quantum + chance) * quantum
    return torch.where(y > 0, torch.clamp(q, min=2.0 ** -9), 0.0)


def _exact_optimiser(case, seed):
    s = _prepare_optimiser(case, seed)
    n = sum(_sizes(case))
    g = torch.cat([t.double() for t in s["grads"]])
    if case["op"] == "norm":
        norm = float(torch.sqrt(torch.sum(g * g))) / case["loss_scale"]
        scale = 1 / case["loss_scale"]
        if not math.isfinite(norm):
            scale = math.nan
        elif case["clip"] > 0 and norm > case["clip"]:
            scale = scale * case["clip"] / norm
        as_one = lambda x: torch.tensor([x], dtype=torch.float64)  # noqa: E731
        return {"norm": as_one(norm), "scale": as_one(scale)}
    k = float(s["grad_scale"])
    skipped = not math.isfinite(k)
    t = STEPS_DONE + 1
    if case["op"] == "adamw":
        m0, v0 = s["m"].double(), s["v"].double()
    else:
        spread = lambda q, f: q.double() * torch.repeat_interleave(f.double(), BLOCK)  # noqa: E731
        m0 = spread(s["m8"], s["m_scale"])[:n]
        v0 = spread(s["r8"], s["r_scale"])[:n] ** 2
    g = g * (0.0 if skipped else k)
    m = B1 * m0 + (1 - B1) * g
    v = B2 * v0 + (1 - B2) * g * g
    w0 = s["weights"].double()
    step = (m / (1 - B1 ** t)) / (torch.sqrt(v / (1 - B2 ** t)) + EPS)
    w = w0 - LR * WD * s["decay"].double() * w0 - LR * step
    out = {"weights": w0 if skipped else w, "steps": None}
    if s["low"] is not None:
        out["low"] = out["weights"]
    if case["op"] == "adamw":
        return out | {"m": m0 if skipped else m, "v": v0 if skipped else v}
    if skipped:
        return out | {"m8": s["m8"][:n].double(), "r8": s["r8"][:n].double(),
                      "m_scale": s["m_scale"].double(), "r_scale": s["r_scale"].double()}

    def blocks(x):
        x = torch.cat((x, torch.zeros(_blocks(n) * BLOCK - n, dtype=x.dtype, device=x.device)))
        x = x.view(-1, BLOCK)
        top = x.abs().amax(1, keepdim=True)
        live = top >= TINY
        y = torch.where(live, x / torch.where(live, top, 1.0) * TOP, 0.0)
        return y.reshape(-1), torch.where(live, top / TOP, 0.0).view(-1)

    ym, m_scale = blocks(m)
    yr, r_scale = blocks(torch.sqrt(v))

    def mix(x):
        x = x & 0xFFFFFFFF
        x = ((x ^ (x >> 16)) * 0x7FEB352D) & 0xFFFFFFFF
        x = ((x ^ (x >> 15)) * 0x846CA68B) & 0xFFFFFFFF
        return x ^ (x >> 16)

    at = torch.arange(yr.numel(), device="cuda") // 2
    key = mix((s["seed"] & 0xFFFFFFFF) ^ mix((s["seed"] >> 32) ^ mix(t)))
    h = mix((at & 0xFFFFFFFF) + key + (at >> 32) * 0x9E3779B9)
    h = torch.where(torch.arange(yr.numel(), device="cuda") % 2 == 0, h & 0xFFFF, h >> 16)
    chance = (h.double() + 0.5) / 65536
    return out | {"m8": _round_e4m3(ym)[:n], "m_scale": m_scale,
                  "r8": _chance_e4m3(yr, chance)[:n], "r_scale": r_scale}


def _exact_layernorm(case, seed):
    s = _prepare_layernorm(case, seed)
    x = s["x"].double()
    w = None if s["weight"] is None else s["weight"].double()
    if case["op"] == "ln_fwd":
        var, mean = torch.var_mean(x, dim=1, correction=0)
        rstd = 1 / torch.sqrt(var + LN_EPS)
        y = (x - mean[:, None]) * rstd[:, None]
        if w is not None:
            y = y * w + s["bias"].double()
        return {"y": y, "mean": mean, "rstd": rstd}
    rstd = s["rstd"].double()[:, None]
    h = (x - s["mean"].double()[:, None]) * rstd
    dy = s["dy"].double()
    g = dy if w is None else dy * w
    cols = case["cols"]
    dx = rstd * (g - (g.sum(1, keepdim=True) + h * (g * h).sum(1, keepdim=True)) / cols)
    if w is None:
        return {"dx": dx}
    return {"dx": dx, "dweight": (dy * h).sum(0), "dbias": dy.sum(0)}


def exact(case, seed):
    if case["op"] in ("norm", "adamw", "adamw8"):
        return _exact_optimiser(case, seed)
    return _exact_layernorm(case, seed)
